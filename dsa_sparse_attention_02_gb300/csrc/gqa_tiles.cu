// Grouped-query attention over the paged 8-bit cache for many query rows per key head:
// prompts (the definition is at dsa_gqa_attend in include/dsa.h).
//
// 256 query rows (tokens x heads of a key head, in two tiles of 128) against a key head's
// blocks on tcgen05: for each block of 64 keys S = Q K^T (128 x 64 x D) and O += P V
// (128 x D x 64) per tile, f16 operands with fp32 sums. The tensor cores bound it: 4 * 64 *
// 256 * D operations per block, at D = 128 about 1,000 clocks of an SM.
//
//   * tensor memory holds, per tile, two S of 64 columns (P, packed f16, takes the place of
//     the S it comes from) and O (D columns): with two tiles of D = 128 all 512. So the next
//     block's scores are computed while this one's softmax runs, and the softmax of a tile
//     never waits for its own products. P is the A operand from tensor memory; Q is read from
//     shared memory. (With Q in tensor memory and one S per tile the MMAs read half as much
//     shared memory, but each block went through softmax, product and scores one after the
//     other: 1,950 clocks a block.)
//   * four warps convert the codes of each block to f16 (exact) once for all 256 rows, into
//     a ring of 128-byte-swizzled stages: K row by row (K-major), V row by row as well (read
//     MN-major). Their loads run one block ahead in registers.
//     At D = 128 column d of a row goes to atom (d/8) % 2, 16-byte chunk d/16: the eight lanes
//     that load a row's 128 bytes of codes then store to eight different bank groups. Q is
//     laid out the same way, and the outputs' columns come out of O in that order.
//   * eight warps do the softmax, one thread per row: while tile 0's four work, the tensor
//     cores do tile 1's products, and the other way round. The block's value scale is part
//     of the exponent, as in gqa_attend.cu; the reference maximum M moves only when a score
//     passes it by more than 2^4, and only then O is rescaled. P at M is 2^11, so that f16 holds
//     it up to 2^4 above, and keeps 2^-11 of every weight down to 2^-25 of the largest one, 2^-36 of
//     the largest below that.
//   * one thread per tile issues its MMAs (each costs the issuer some 40 clocks: with one thread
//     for both tiles the tensor cores waited for it).
// Items (request, key head, 256 rows) have as many units as blocks their last token sees;
// all units are laid end to end and cut into equal runs, one per SM, so that the causal
// triangle and ragged requests leave no SM idle; cut items are merged afterwards.
//
// 2048 tokens over 16384, 64 query heads over 8 of 128 (1.03 TFLOP): 804 us, 1.28 PFLOP/s, the
// tensor pipe 70% busy. A block takes some 1,800 clocks, where products and shared-memory reads
// alone would take 1,280: the rest is the softmax between a tile's scores and its products. (A
// reference that moves at 2^8 would take 788 us and keep 4 bits less of the range, one that moves
// at 2^2 826 and 2 more; weights of at most 2^8 as they were took 782.)
//
// A block that some rows see only in part has the keys past each row's position at weight
// 0, and values that no row sees zeroed. An e4m3 NaN value in such a block is taken out and
// its position noted per column: a row whose position has reached it gets NaN there.
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kConvWarp0 = 8, kConvWarps = 4;   // warps 0-3 and 4-7: the softmax of tile 0 and 1
constexpr int kMmaWarp = 12;                    // and 13: the products of tile 0 and 1
constexpr int kThreads = 14 * 32;
constexpr int kStages = 4;
constexpr int kDeep = 3;                    // units between a prefetch and the loads
constexpr int kNanSlots = 16;               // segments whose NaN notes are alive: converters run at most kStages units ahead
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTileCols = 256, kSCols = 64, kOCol = 128;   // of a tile: S / P at 0 and 64
constexpr float kRescale = 4.f;             // log2 of what a weight may pass the reference by,
constexpr float kLift = 11.f, kDown = 1.f / 2048.f;   // of the weight at the reference, and what takes that back

template <int D>
struct TileShape {
  static constexpr int kAtom = kPage * 128;              // 64 rows x 64 f16
  static constexpr int kOperand = kPage * D * 2;         // K or V of a block
  static constexpr int kQAtom = 128 * 128;               // 128 rows x 64 f16
  static constexpr int kQTile = D / 64 * kQAtom;
  static constexpr size_t kSmem = 2 * kQTile + (size_t)kStages * 2 * kOperand + 1024;
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
// Pairs of fp32 operations (one instruction for two lanes' worth of the same thread).
__device__ __forceinline__ void fma2(float& a, float& b, float m, float c) {   // a = a * m + c, b = b * m + c
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(m), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {   // a += c, b += d
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

// Requests as the items see them.
struct Prompt {
  int q0, n, start;      // first token, tokens, position of the first (may be negative)
  int tiles;
  bool bad, none;        // none: nothing visible (inconsistent geometry)
};
__device__ __forceinline__ Prompt prompt_of(const GqaAttendArgs& A, int b) {
  Prompt r;
  const int c0 = __ldg(A.g.cu_q + b), c1 = __ldg(A.g.cu_q + b + 1);
  const int len = __ldg(A.g.seq_lens + b);
  r.bad = c0 < 0 || c1 < c0 || c1 > A.g.T || len > A.g.max_seq_len;
  r.q0 = min(max(c0, 0), A.g.T);
  r.n = max(min(c1, A.g.T) - r.q0, 0);
  r.none = r.bad || len <= 0;
  r.start = len - r.n;
  r.tiles = (int)(((int64_t)r.n * A.G + kGqaTileRows - 1) / kGqaTileRows);
  return r;
}
// Blocks that the last token of tile i sees (at least one unit: empty rows are written too).
__device__ __forceinline__ int tile_units(const GqaAttendArgs& A, const Prompt& r, int i) {
  if (r.none) return 1;
  const int last = (int)min((int64_t)r.n - 1, ((int64_t)i * kGqaTileRows + kGqaTileRows - 1) / A.G);
  return max(r.start + last, 0) / kPage + 1;
}
__device__ __forceinline__ int64_t head_units(const GqaAttendArgs& A, const Prompt& r) {
  int64_t s = 0;
  for (int i = 0; i < r.tiles; ++i) s += tile_units(A, r, i);
  return s;
}

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads, 1) gqa_tiles_kernel(const GqaAttendArgs A, const GqaParts parts, const int deep) {
  using S = TileShape<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_empty[kStages];
  __shared__ uint64_t s_sfull[2][2], s_pfull[2][2], s_odone[2][2],   // [tile][unit % 2]
       s_qfull[2], s_drain[2];
  __shared__ Unit s_unit[kStages];
  __shared__ int s_nan[I8 ? 1 : kNanSlots][D];
  __shared__ int64_t s_begin, s_end, s_base, s_total;
  __shared__ int s_req, s_grid, s_abort;
  __shared__ uint32_t s_tmem;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* q_smem = smem + (size_t)kStages * 2 * S::kOperand;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  if (tid == 32 * kMmaWarp) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s_full[i]), kConvWarps);
      mbar_init(smem_u32(&s_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(smem_u32(&s_sfull[i][k]), 1);
        mbar_init(smem_u32(&s_pfull[i][k]), 4);
        mbar_init(smem_u32(&s_odone[i][k]), 1);
      }
      mbar_init(smem_u32(&s_qfull[i]), 4);
      mbar_init(smem_u32(&s_drain[i]), 1);
    }
    s_abort = 0;
    fence_mbar_init();
    parts.cuts[blockIdx.x].follow = 0;
  }
  if (!I8)
    for (int i = tid; i < kNanSlots * D; i += kThreads) (&s_nan[0][0])[i] = INT32_MAX;
  // The run [s_begin, s_end) of all units, the request it starts in and where that begins.
  if (warp == 0) {
    int64_t total = 0;
    for (int b0 = 0; b0 < A.g.B; b0 += 32) {
      if (b0 + lane < A.g.B) {
        const Prompt r = prompt_of(A, b0 + lane);
        total += A.c.Hkv * head_units(A, r);
        if (r.bad && blockIdx.x == 0) record_error(A.err, kDevBadIndex);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int grid = (int)min((int64_t)gridDim.x, total);
    int64_t begin = 0, end = 0, base = 0;
    int req = 0;
    if ((int)blockIdx.x < grid) {
      begin = split_begin(blockIdx.x, total, grid);
      end = split_begin(blockIdx.x + 1, total, grid);
      for (int b0 = 0; b0 < A.g.B; b0 += 32) {
        const int64_t w = b0 + lane < A.g.B ? A.c.Hkv * head_units(A, prompt_of(A, b0 + lane)) : 0;
        int64_t upto = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const unsigned m = __ballot_sync(0xffffffffu, base + upto > begin);
        if (m) {
          const int l = __ffs(m) - 1;
          req = b0 + l;
          base += __shfl_sync(0xffffffffu, upto - w, l);
          break;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (lane == 0) {
      s_begin = begin, s_end = end, s_base = base, s_total = total;
      s_req = req, s_grid = grid;
    }
  }
  __syncthreads();
  const int64_t begin = s_begin, end = s_end;
  if (begin >= end) return;                       // (the whole block)
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort = &s_abort;
  const int count = (int)(end - begin);           // at most total / grid + 1

  if (warp >= kConvWarp0 && warp < kConvWarp0 + kConvWarps) {
    // ------------------------------------------------------------ conversion
    const int ct = tid - 32 * kConvWarp0;
    const bool writer = warp == kConvWarp0;
    const int64_t total = s_total;
    const int grid = s_grid;
    // the cursor: request, key head, tile, block of the next batch's first unit
    int b = s_req, h = 0, tile_i = 0, c = 0;
    Prompt r = prompt_of(A, b);
    {
      const int64_t per = head_units(A, r);
      int64_t o = begin - s_base;
      h = (int)(o / per);
      o -= h * per;
      while (o >= tile_units(A, r, tile_i)) o -= tile_units(A, r, tile_i++);
      c = (int)o;
    }
    // up to 32 units at a time, one per lane
    Unit x{};
    int page_tile = 0, cnt = 0, at = 0, seen = 0, whole_all = 0;
    auto batch = [&](int64_t u) {
      cnt = (int)min((int64_t)32, end - u);
      int bb = b, hh = h, ti = tile_i, cc = c;
      Prompt rr = r;
      int units = tile_units(A, rr, ti);
      for (int step = lane; step > 0 && lane < cnt;) {          // forward by `lane` units
        const int left = units - cc;
        if (step < left) {
          cc += step;
          break;
        }
        step -= left;
        cc = 0;
        if (++ti == rr.tiles) {
          ti = 0;
          if (++hh == A.c.Hkv) {
            hh = 0;
            do rr = prompt_of(A, ++bb);
            while (rr.tiles == 0 && bb + 1 < A.g.B);
          }
        }
        units = tile_units(A, rr, ti);
      }
      __syncwarp();
      if (lane < cnt) {
        const int64_t me = u + lane, ib = me - cc, ie = ib + units;
        x.q0 = rr.q0, x.n = rr.n, x.h = hh, x.c = cc;
        x.row0 = ti * kGqaTileRows;
        x.rel = rr.start - cc * kPage;
        const int lo = x.row0 / A.G, hi = min(rr.n - 1, (x.row0 + kGqaTileRows - 1) / A.G);
        int page = -1;
        if (!rr.none && x.rel + hi >= 0) {
          page = gqa_page(A.g, bb, cc);
          if (page < 0 && writer) record_error(A.err, kDevBadIndex);
        }
        x.kf = 0.f, x.lv = 0.f, x.ivs = 1.f;
        page_tile = 0;
        if (page >= 0) {
          page_tile = page * A.c.Hkv + hh;
          const float vs = __ldg(A.c.v_scale + page_tile);
          x.kf = __ldg(A.c.k_scale + page_tile) * A.scale_log2;
          x.lv = log2f(vs);
          x.ivs = 1.f / vs;
        }
        seen = page >= 0 ? min(x.rel + hi, kPage - 1) : -1;
        whole_all = page >= 0 && x.rel + lo >= kPage - 1;
        const bool first = me == ib || me == begin, last = me + 1 == ie || me + 1 == end;
        x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (page >= 0 ? 0 : kVoid);
        const bool cut = ib < begin || ie > end;
        x.slot = !cut ? -1 : 2 * (int)blockIdx.x + (max(ib, begin) == begin ? 0 : 1);
        if (writer && last && cut && ib >= begin) {
          Cut k{};
          k.follow = (int)split_owner(ie - 1, total, grid) - (int)blockIdx.x;
          k.slot = x.slot;
          k.q0 = x.q0, k.n = x.n, k.row0 = x.row0, k.h = x.h;
          parts.cuts[blockIdx.x] = k;
        }
      }
      // the cursor behind the batch: its last lane's unit, one further
      const int l = cnt - 1;
      b = __shfl_sync(0xffffffffu, bb, l), h = __shfl_sync(0xffffffffu, hh, l);
      tile_i = __shfl_sync(0xffffffffu, ti, l), c = __shfl_sync(0xffffffffu, cc, l) + 1;
      r = prompt_of(A, b);
      if (u + cnt < end && c == tile_units(A, r, tile_i)) {
        c = 0;
        if (++tile_i == r.tiles) {
          tile_i = 0;
          if (++h == A.c.Hkv) {
            h = 0;
            do r = prompt_of(A, ++b);
            while (r.tiles == 0 && b + 1 < A.g.B);
          }
        }
      }
      at = 0;
    };
    // a thread's share of a tensor's codes: kLoads pieces of 16, piece i in row prow + kStep * i
    constexpr int kLoads = D / 32, kLanes = D / 16, kStep = 32 * kConvWarps / kLanes;
    const int prow = ct / kLanes, pch = ct % kLanes;
    uint4 kr[kLoads], vr[kLoads];
    auto fetch = [&](const uint8_t* base, int t, uint4 (&dst)[kLoads]) {
      const uint4* src = reinterpret_cast<const uint4*>(base + (int64_t)t * (kPage * D)) + ct;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) dst[i] = __ldg(src + i * 32 * kConvWarps);
    };
    auto put = [&](uint8_t* dst, int i, const uint4& v) {
      const int row = prow + kStep * i;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) codes_f16<I8>(w[k], f[2 * k], f[2 * k + 1]);
      uint8_t* line = dst + row * 128;
      uint8_t* lo = D == 128 ? line + ((pch ^ (row & 7)) << 4) : line + (((2 * pch) ^ (row & 7)) << 4);
      uint8_t* hi = D == 128 ? lo + S::kAtom : line + (((2 * pch + 1) ^ (row & 7)) << 4);
      *reinterpret_cast<uint4*>(lo) = make_uint4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<uint4*>(hi) = make_uint4(f[4], f[5], f[6], f[7]);
    };
    // A unit of the batch towards L2, a line a thread, `deep` units before its loads: one unit on
    // the way an SM does not fill HBM's latency.
    auto prefetch = [&](int k) {
      if (deep == 0 || k >= cnt) return;
      const int t = __shfl_sync(0xffffffffu, page_tile, k);
      constexpr int kLines = kPage * D / 128;
      if (ct < 2 * kLines) prefetch_l2((ct < kLines ? A.c.k : A.c.v) + (int64_t)t * (kPage * D) + (ct & (kLines - 1)) * 128);
    };
    batch(begin);
    for (int k = 1; k < deep; ++k) prefetch(k);
    int t_next = __shfl_sync(0xffffffffu, page_tile, 0);
    fetch(A.c.k, t_next, kr);
    fetch(A.c.v, t_next, vr);
    int seg = -1;
    for (int n = 0; n < count; ++n) {
      const int stage = n % kStages;
      if (!warp_wait(&s_empty[stage], ((n / kStages) & 1) ^ 1, abort, A.err)) break;
      if (writer && lane == at) s_unit[stage] = x;
      const int flags = __shfl_sync(0xffffffffu, x.flags, at), my_seen = __shfl_sync(0xffffffffu, seen, at);
      const int my_whole = __shfl_sync(0xffffffffu, whole_all, at), my_c = __shfl_sync(0xffffffffu, x.c, at);
      if (flags & kFirst) {
        ++seg;
        // notes of the segment eight ahead: its slot's last user ended more than kStages units ago
        if (!I8 && ct < D) s_nan[(seg + kNanSlots / 2) % kNanSlots][ct] = INT32_MAX;
      }
      uint8_t* kd = smem + (size_t)stage * 2 * S::kOperand;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) put(kd, i, kr[i]);
      if (n + 1 < count) {
        if (++at == cnt) {
          batch(begin + n + 1);
          for (int k = 1; k < deep; ++k) prefetch(k);
        }
        prefetch(at + deep);
        t_next = __shfl_sync(0xffffffffu, page_tile, at);
        fetch(A.c.k, t_next, kr);
      }
      if (!my_whole) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int row = prow + kStep * i;
          if (row > my_seen) vr[i] = make_uint4(0, 0, 0, 0);
          if (!I8) {
            uint32_t* w = &vr[i].x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t bad = __vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              if (bad) {
                w[k] &= ~bad;
                for (int e = 0; e < 4; ++e)
                  if ((bad >> (8 * e)) & 1u) atomicMin(&s_nan[seg % kNanSlots][16 * pch + 4 * k + e], my_c * kPage + row);
              }
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) put(kd + S::kOperand, i, vr[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_full[stage]));
      if (n + 1 < count) fetch(A.c.v, t_next, vr);
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp runs the loop, so that descriptors and addresses are uniform values (an
    // MMA takes them from uniform registers); one lane issues. All 512 columns are this
    // block's: tensor memory starts at column 0.
    constexpr uint32_t idesc_s = make_idesc(128, kPage, kFmtF16, kFmtF16, 0, 0);
    constexpr uint32_t idesc_o = make_idesc(128, D, kFmtF16, kFmtF16, 0, 1);
    const int i = warp - kMmaWarp;                // tile
    const uint32_t tcol = i * kTileCols;
    const uint64_t dk = smem_desc(smem_u32(smem), 0, 1024, kSwizzle128B);
    const uint64_t dv = smem_desc(smem_u32(smem) + S::kOperand, S::kAtom, 1024, kSwizzle128B);
    const bool issuer = elect_one();
    uint32_t qphase = 0, fresh = 0;               // fresh: unit n begins a segment
    int stage = 0, before = 0;                    // of units n + 1 and n
    uint32_t phase = 0;
    bool ok = tmem == 0;
    if (!ok) {
      *abort = 1;
      record_error(A.err, kDevTimeout);
    }
    const uint64_t dq = smem_desc(smem_u32(q_smem) + i * S::kQTile, 0, 1024, kSwizzle128B);
    auto scores = [&](int n) {                    // of unit n, in `stage`
      tc_fence_after();
      if (issuer) {
        const uint64_t kd = desc_add(dk, stage * 2 * S::kOperand);
        const uint32_t d = tcol + (n & 1) * kSCols;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ss(d, desc_add(dq, (k >> 2) * S::kQAtom + (k & 3) * 32), desc_add(kd, (k >> 2) * S::kAtom + (k & 3) * 32),
                     idesc_s, k != 0);
        mma_commit(smem_u32(&s_sfull[i][n & 1]));
      }
    };
    for (int n = -1; n < count; ++n) {
      // unit n + 1's scores, then unit n's values; where n + 1 begins a segment, its queries
      // come after unit n's outputs, so the other way round
      uint32_t next = 0;
      if (n + 1 < count) {
        ok = ok && warp_wait(&s_full[stage], phase, abort, A.err);
        if (!ok) break;
        next = s_unit[stage].flags & kFirst;
        static_assert(kFirst == 1, "next is a flag and an operand");
        next = __any_sync(0xffffffffu, next) ? 1u : 0u;
        if (!next) scores(n + 1);
      }
      if (n >= 0) {
        ok = warp_wait(&s_pfull[i][n & 1], (n >> 1) & 1, abort, A.err);
        if (!ok) break;
        tc_fence_after();
        if (issuer) {
          const uint64_t vd = desc_add(dv, before * 2 * S::kOperand);
          const uint32_t p = tcol + (n & 1) * kSCols;
#pragma unroll
          for (int k = 0; k < kPage / 16; ++k)
            mma_f16_ts(tcol + kOCol, p + 8 * k, desc_add(vd, k * 2048), idesc_o, k != 0 ? 1u : fresh ^ 1u);
          mma_commit(smem_u32(&s_odone[i][n & 1]));
          mma_commit(smem_u32(&s_empty[before]));
        }
      }
      if (next) {
        ok = warp_wait(&s_qfull[i], qphase, abort, A.err);
        qphase ^= 1u;
        if (!ok) break;
        scores(n + 1);
      }
      fresh = next;
      before = stage;
      if (++stage == kStages) stage = 0, phase ^= 1u;
    }
    // Everything issued has finished before tensor and shared memory are given back.
    __syncwarp();
    if (issuer) {
      mma_commit(smem_u32(&s_drain[i]));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&s_drain[i]), 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort = 1;
          record_error(A.err, kDevTimeout);
          break;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax: a thread per row
    const int i = warp >> 2;                       // tile
    const uint32_t tile = tmem + i * kTileCols + ((uint32_t)(32 * (warp & 3)) << 16);
    const int G = A.G, H = A.G * A.c.Hkv;
    const int r_in = 128 * i + 32 * (warp & 3) + lane;
    float M = kNone, l = 0.f, rowf = 1.f;
    int tok = 0, tok_lo = 0, seg = -1;
    bool valid = false;
    // Of the next unit what every row needs (the rest is read where a segment begins or
    // ends): fetched while this one's exponentials run.
    struct Short { float kf, lv, ivs; int flags, rel; } x, x_next;
    int stage = 0;
    uint32_t phase = 0;
    auto peek = [&](Short& s) {
      if (!warp_wait(&s_full[stage], phase, abort, A.err)) return false;
      const Unit* u = &s_unit[stage];
      s = Short{u->kf, u->lv, u->ivs, u->flags, u->rel};
      return true;
    };
    bool ok = peek(x_next);
    for (int n = 0; n < count && ok; ++n) {
      x = x_next;
      const Unit& unit = s_unit[stage];
      if (x.flags & kFirst) {
        ++seg;
        const struct { int q0, n, row0, h; } u = {unit.q0, unit.n, unit.row0, unit.h};
        const int row = u.row0 + r_in;
        valid = row < u.n * G;
        tok = valid ? row / G : -(1 << 30);
        tok_lo = (u.row0 + 128 * i + 32 * (warp & 3)) / G;        // of the warp's rows
        M = kNone, l = 0.f;
        const uint4* src = reinterpret_cast<const uint4*>(
            A.q + (int64_t)(u.q0 + (valid ? tok : 0)) * A.q_stride + (int64_t)(u.h * G + (valid ? row - tok * G : 0)) * D);
        float big = 0.f;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 v = valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          big = fmaxf(big, fmaxf(fmaxf(fabsf(bf16_lo(v.x)), fabsf(bf16_hi(v.x))), fmaxf(fabsf(bf16_lo(v.y)), fabsf(bf16_hi(v.y)))));
          big = fmaxf(big, fmaxf(fmaxf(fabsf(bf16_lo(v.z)), fabsf(bf16_hi(v.z))), fmaxf(fabsf(bf16_lo(v.w)), fabsf(bf16_hi(v.w)))));
        }
        const int e = min(max((int)(__float_as_uint(big) >> 23), 15), 254);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        rowf = __uint_as_float((uint32_t)(e - 14) << 23);
        uint8_t* mine = q_smem + i * S::kQTile + (r_in & 127) * 128;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 v = valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          const int atom = D == 128 ? k & 1 : 0, chunk = D == 128 ? k >> 1 : k;
          *reinterpret_cast<uint4*>(mine + atom * S::kQAtom + ((chunk ^ (r_in & 7)) << 4)) =
              make_uint4(pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up), pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                         pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up), pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_qfull[i]));
      }
      if (!warp_wait(&s_sfull[i][n & 1], (n >> 1) & 1, abort, A.err)) break;
      tc_fence_after();
      float s[64];
      const uint32_t sp = tile + (n & 1) * kSCols;
      tmem_ld64(sp, s);
      tmem_ld_wait();
      if (x.rel + tok_lo < kPage - 1 || (x.flags & kVoid)) {   // some row of the warp does not see every key
        const int lim = (x.flags & kVoid) ? -1 : x.rel + tok;
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (k > lim) s[k] = -INFINITY;
      }
      float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int k = 4; k < 60; k += 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) m4[j] = max3(m4[j], s[k + 2 * j], s[k + 2 * j + 1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], s[60 + j]);
      // (a scale of 0 would make masked scores NaN)
      const float f = fmaxf(x.kf * rowf, 1.17549435e-38f);
      const float mf = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f;
      const float top = mf + x.lv;
      bool rose = false;
      if (__any_sync(0xffffffffu, top > M + kRescale)) {
        const float Mn = fmaxf(M, top), keep = ex2(M - Mn);
        rose = top >= M;
        M = Mn;
        l *= keep;
        if (!(x.flags & kFirst)) {                 // O so far, once its last product is done
          if (!warp_wait(&s_odone[i][(n - 1) & 1], ((n - 1) >> 1) & 1, abort, A.err)) break;
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            float v[16];
            tmem_ld16(tile + kOCol + k, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= keep;
            tmem_st16(tile + kOCol + k, v);
          }
          tmem_st_wait();
        }
      }
      // (where scores are so large that M and lv do not add exactly, this block's largest weight is
      // still 2^11 if M is its own, and not above 2^15 if not)
      const float ref = rose ? kLift - mf : fminf(x.lv - M + kLift, kLift + kRescale - mf);
      struct { int q0, row0, h, slot, c; } end{};   // (read before the stage may be given back)
      if (x.flags & kLast) end = {unit.q0, unit.row0, unit.h, unit.slot, unit.c};
      if (n + 1 < count) {
        if (++stage == kStages) stage = 0, phase ^= 1u;
        ok = peek(x_next);
        if (!ok) break;
      }
      float a[4] = {};
      uint32_t p[32];
#pragma unroll
      for (int k = 0; k < 64; k += 4) {
        fma2(s[k], s[k + 1], f, ref);
        fma2(s[k + 2], s[k + 3], f, ref);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[k + j] = ex2(s[k + j]);
        add2(a[0], a[1], s[k], s[k + 1]);
        add2(a[2], a[3], s[k + 2], s[k + 3]);
        p[k / 2] = pack_weights(s[k], s[k + 1]);
        p[k / 2 + 1] = pack_weights(s[k + 2], s[k + 3]);
      }
      tmem_st32(sp, p);
      l += ((a[0] + a[1]) + (a[2] + a[3])) * kDown * x.ivs;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_pfull[i][n & 1]));
      if (!(x.flags & kLast)) continue;

      // ---- the segment's outputs, or its part
      // (one barrier for every second unit: the warps of a tile run up to a unit apart, so the
      // products of unit n - 1 may still be to come, and a single barrier's parity would let n pass)
      if (!warp_wait(&s_odone[i][n & 1], (n >> 1) & 1, abort, A.err)) break;
      tc_fence_after();
      const int pos = x.rel + tok + end.c * kPage;
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const int64_t at = valid ? (int64_t)(end.q0 + tok) * H + end.h * G + (end.row0 + r_in - tok * G) : 0;
      const int64_t part = (int64_t)end.slot * kGqaTileRows + r_in;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {            // columns k .. k + 31
        float v[32];
        {
          float a[16], b[16];
          tmem_ld16(tile + kOCol + (D == 128 ? k / 2 : k), a);
          tmem_ld16(tile + kOCol + (D == 128 ? 64 + k / 2 : k + 16), b);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = kDown * (D == 128 ? ((j >> 3) & 1 ? b[(j & 7) + 8 * (j >> 4)] : a[(j & 7) + 8 * (j >> 4)]) : (j < 16 ? a[j] : b[j - 16]));
        }
        if (!I8) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!none && pos >= s_nan[seg % kNanSlots][k + j]) v[j] = NAN;
        }
        if (!valid) {
        } else if (end.slot < 0) {
          uint4* dst = reinterpret_cast<uint4*>(A.out + at * D + k);
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 o =
                  __floats2bfloat162_rn(none ? 0.f : v[j + 2 * e] * inv, none ? 0.f : v[j + 2 * e + 1] * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&o);
            }
            dst[j / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(parts.o + part * D + k);
#pragma unroll
          for (int j = 0; j < 32; j += 4) dst[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      if (valid) {
        if (end.slot >= 0) *reinterpret_cast<float2*>(parts.ml + part * 2) = make_float2(M, l);
        else if (A.lse) A.lse[at] = none ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool I8>
cudaError_t launch(const GqaAttendArgs& A, int num_sms, cudaStream_t st) {
  const GqaParts s = gqa_parts(A.scratch, num_sms, kGqaTileRows);
  auto kern = gqa_tiles_kernel<D, I8>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, TileShape<D>::kSmem, allowed);
  if (e != cudaSuccess) return e;
  // Requests of few items read their keys from HBM, where the prefetch helps (32 requests of 4096
  // to 16384 tokens: 256 rows 389 -> 349 us; 8 of them, 1024 rows: 370 -> 336). A long prompt finds
  // them in L2 after its first items, and the prefetch only costs issue (16384 rows: 783 -> 788).
  const int deep = ((int64_t)A.g.T + A.g.B - 1) / A.g.B * A.G <= 16 * kGqaTileRows ? kDeep : 0;
  kern<<<num_sms, kThreads, TileShape<D>::kSmem, st>>>(A, s, deep);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : gqa_merge_launch(A, s, num_sms, st);
}

}  // namespace

cudaError_t gqa_tiles_launch(const GqaAttendArgs& A, int num_sms, cudaStream_t st) {
  if (A.c.D == 128) return A.c.i8 ? launch<128, true>(A, num_sms, st) : launch<128, false>(A, num_sms, st);
  return A.c.i8 ? launch<64, true>(A, num_sms, st) : launch<64, false>(A, num_sms, st);
}

}  // namespace dsa
