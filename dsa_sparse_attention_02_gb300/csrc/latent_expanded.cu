// Causal attention over keys and values expanded by head, the rotated part of the key shared by
// all heads (the definition is at dsa_latent_attend_expanded in include/dsa.h).
//
// An item is (request, head, 256 query tokens in two tiles of 128; or 128 in one, where the mean
// request has no more), a unit 128 of its keys. For each unit and tile, on tcgen05 with bf16
// operands and fp32 sums:
//   S = Q K^T  128 x 128 x 192,  O += P V  128 x 128 x 128
// 2,560 clocks of an SM's tensor cores for two tiles. A unit of a long prompt takes 3,980: the tensor
// cores wait for the softmax between scores and values (2048 tokens over 16384, 32 heads: 470 to 520 us by card
// and clock, 1.24 to 1.37 PFLOP/s); both products read as many operand bytes from
// shared memory as 128 bytes a clock allow in 2,560. Few rows over many keys are bound by HBM
// (16 requests of 100 rows over 1500 keys in the mean, 16 heads: 51 us, 4.4 TB/s).
//
//   * tensor memory holds S (128 columns; P, packed bf16, takes its place) and O (128) in each of
//     two places: all 512. A tile goes through scores, softmax and values one after the other;
//     the tensor cores do one place's products while the other's softmax runs. Two tiles have a
//     place each; one tile's units take them in turn (see ExpShape).
//   * shared memory holds the queries (48 KB a tile), two units of keys (the rotated 64 columns
//     as a third atom beside the head's own 128) and one or two of values in two halves (keys 64 to
//     127 first), each loaded by TMA when its last reader has finished.
//   * eight warps do the softmax, one thread per row. P is handed over in two halves, so that
//     the values' product begins while the second half's exponentials run. The reference
//     maximum moves only when a score passes it by more than 2^8; only then O is rescaled
//     (a unit's scores are behind the unit before it in the tensor cores' order, so O is at rest).
//     Weights meet the values in bf16, as both operands of a product are of one type; their sum is of the
//     fp32 weights. (Against 64 bits outputs are off by 0.0020 to 0.0024 of their norm, with fp32 weights 0.0017.)
//   * one thread per place issues its products.
//   * four warps look through the values of units that some row does not see whole: keys
//     that no row sees are zeroed, and NaN and infinities taken out and noted per column, for
//     rows that reach them (a weight of zero would not keep them out of the sum).
// All units are laid end to end and cut into runs of equal cost, one per SM; cut items are merged.
#include "latent_common.cuh"

namespace dsa {

namespace {

constexpr int kKeys = 128, kTile = 128, kV = 128;
constexpr int kAtom = 128 * 128;               // 128 rows x 64 bf16
constexpr int kKBytes = 3 * kAtom, kVHalf = 2 * 64 * 128, kQTile = 3 * kAtom;
constexpr int kKStages = 2;
// Tiles of an item, and stages of values beside them. With one tile its units go alternately through
// the two places in tensor memory, each with the softmax warps, issuer, maximum, sum and O of
// its own (joined at the item's end): the products of one unit again run during the other's
// softmax, and a second stage of values has the second tile's place in shared memory.
template <int TILES>
struct ExpShape {
  static constexpr int kRows = TILES * kTile, kVStages = TILES == 1 ? 2 : 1;
  // An item's cost beside its units'. (Ragged prompts of 100 rows in the mean over 1500 keys: 82 us
  // with 0, 57 with 1, 54 with 2, 52 with 3 and with 4; a chunk of 2048 tokens: 476, 478 and 484 with 1, 2 and 3.)
  static constexpr int kItemCost = TILES == 1 ? 3 : 2;
  static constexpr int kSmem = 1024 + TILES * kQTile + kKStages * kKBytes + kVStages * 2 * kVHalf;
};
constexpr int kUnits = 4;                      // units described ahead
constexpr int kMmaWarp = 8, kLoadWarp = 10, kValueWarp = 11, kFixWarp0 = 12;   // 0-3, 4-7: softmax of tile 0, 1
constexpr int kFixWarps = 4;
constexpr int kThreads = 16 * 32;
constexpr uint32_t kTmem = 512, kTileCols = 256, kOCol = 128;
constexpr float kMove = 8.f;                   // log2 of what a weight may pass the reference by
enum : int { kEdge = 8 };                      // some row of the item does not see the whole unit

struct __align__(16) ExpUnit {
  int flags, rel;        // position of the item's first row less the unit's first position
  int q0, rows;          // the item's first token, its rows in use
  int h, key0;           // head; row of k, v of the unit's first key
  int slot, last;        // partial slot or -1; last key of the unit that some row sees, or -1
};

struct ExpReq {
  int q0, n, k0, start;  // first token, tokens, first key row, position of the first token (may be negative)
  int tiles;
  bool bad, none;
};
template <int kRows>
__device__ __forceinline__ ExpReq exp_req(const LatentExpandedArgs& A, int b) {
  ExpReq r;
  const int c0 = __ldg(A.cu_q + b), c1 = __ldg(A.cu_q + b + 1), k0 = __ldg(A.cu_k + b), k1 = __ldg(A.cu_k + b + 1);
  r.bad = c0 < 0 || c1 < c0 || c1 > A.T || k0 < 0 || k1 < k0 || k1 > A.S;
  r.q0 = min(max(c0, 0), A.T);
  r.n = max(min(c1, A.T) - r.q0, 0);
  r.none = r.bad || k1 == k0;
  r.k0 = k0;
  r.start = r.bad ? 0 : (k1 - k0) - r.n;
  r.tiles = (r.n + kRows - 1) / kRows;
  return r;
}
struct ExpStart { ExpReq r; int b, h, ti, c; int64_t item; };   // unit c of tile ti of head h of request b, the item's number
// Units that tile i's last token sees (at least one: empty rows are written too).
template <int kRows>
__device__ __forceinline__ int exp_units(const ExpReq& r, int i) {
  if (r.none) return 1;
  return max(r.start + min(r.n - 1, i * kRows + kRows - 1), 0) / kKeys + 1;
}
template <int kRows>
__device__ __forceinline__ int64_t exp_head(const ExpReq& r) {
  int64_t s = 0;
  for (int i = 0; i < r.tiles; ++i) s += exp_units<kRows>(r, i);
  return s;
}

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
// Pairs of fp32 operations (one instruction for both).
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

// Notes: the least relative key with a value that is not finite, 16 bits a column.
constexpr int kNoNote = 0x7FFF;
__device__ __forceinline__ void note_min(uint32_t* notes, int col, int key) {
  uint32_t* w = notes + (col >> 1);
  const int sh = 16 * (col & 1);
  uint32_t old = *w;
  while ((int)(int16_t)(old >> sh) > key) {
    const uint32_t want = (old & ~(0xFFFFu << sh)) | ((uint32_t)(uint16_t)(int16_t)key << sh);
    const uint32_t got = atomicCAS(w, old, want);
    if (got == old) break;
    old = got;
  }
}

template <int TILES>
__global__ void __launch_bounds__(kThreads, 1)
    latent_expanded_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_rope, const __grid_constant__ CUtensorMap map_v,
                           const LatentExpandedArgs A, const LatentParts parts) {
  constexpr int kRows = ExpShape<TILES>::kRows, kVStages = ExpShape<TILES>::kVStages;
  constexpr int kItemCost = ExpShape<TILES>::kItemCost;
  constexpr bool kSplit = TILES == 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_buf = smem;
  uint8_t* k_buf = q_buf + TILES * kQTile;
  uint8_t* v_buf = k_buf + kKStages * kKBytes;
  __shared__ uint64_t u_full[kUnits], u_loaded[kUnits], u_empty[kUnits], e_full[kUnits];
  __shared__ uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages][2], v_empty[kVStages][2];
  __shared__ uint64_t q_full[2], q_free[2], s_full[2], p_full[2][2], o_done[2], drain[2];
  __shared__ uint64_t x_full, x_done;            // one tile: both places' results of an item are there, have been read
  __shared__ ExpUnit s_unit[kUnits];
  __shared__ uint32_t s_note[kUnits][kV / 2];
  __shared__ float2 s_ml[kSplit ? 2 : 1][kSplit ? kTile : 1];
  __shared__ int s_count, s_abort;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&u_full[i]), 1);
      mbar_init(smem_u32(&u_loaded[i]), 1);
      mbar_init(smem_u32(&u_empty[i]), 8 + kFixWarps + 1);
      mbar_init(smem_u32(&e_full[i]), kFixWarps);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), TILES);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < kVStages; ++j) {
        mbar_init(smem_u32(&v_full[j][i]), 1);
        mbar_init(smem_u32(&v_empty[j][i]), TILES);
      }
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_free[i]), kSplit ? 2 : 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i][0]), 4);
      mbar_init(smem_u32(&p_full[i][1]), 4);
      mbar_init(smem_u32(&o_done[i]), 1);
      mbar_init(smem_u32(&drain[i]), 1);
    }
    mbar_init(smem_u32(&x_full), 8);
    mbar_init(smem_u32(&x_done), 8);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem), kTmem);
    tmem_relinquish();
  }
  // Runs are equal in cost: an item's units, and kItemCost for it (its queries, and its outputs, which
  // no product hides). This block's run is the units [begin, end); it starts at `first`.
  int64_t begin = 0, end = 0, total = 0;
  int runs = 1;
  ExpStart first{};
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_rope);
      tma_prefetch_desc(&map_v);
      parts.cuts[blockIdx.x].follow = 0;
    }
    // (32 requests at most are read once: each look takes half a microsecond)
    ExpReq front{};
    int64_t front_head = 0;
    auto look = [&](int b0) {
      front = ExpReq{};
      front_head = 0;
      if (b0 + lane < A.B) {
        front = exp_req<kRows>(A, b0 + lane);
        front_head = exp_head<kRows>(front);
      }
    };
    auto weight = [&]() { return A.H * (front_head + (int64_t)kItemCost * front.tiles); };
    for (int b0 = (A.B - 1) / 32 * 32; b0 >= 0; b0 -= 32) {      // (the first ones stay)
      look(b0);
      total += weight();
      if (front.bad && blockIdx.x == 0) record_error(A.err, kDevBadIndex);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    runs = (int)min((int64_t)gridDim.x, max(total, (int64_t)1));
    if ((int)blockIdx.x < runs && total > 0) {
      const int64_t lo = run_begin(blockIdx.x, total, runs), hi = run_begin(blockIdx.x + 1, total, runs);
      int64_t cost = 0, units = 0, items = 0;                    // of the requests before b0
      bool found = false;
      end = -1;
      for (int b0 = 0; b0 < A.B && end < 0; b0 += 32) {
        if (b0 > 0) look(b0);
        int64_t up[3] = {weight(), A.H * front_head, (int64_t)A.H * front.tiles};
        const int64_t own[3] = {up[0], up[1], up[2]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int64_t v = __shfl_up_sync(0xffffffffu, up[i], o);
            if (lane >= o) up[i] += v;
          }
        }
        // the unit at cost `at`, or the first behind it
        auto locate = [&](int64_t at, int l, ExpStart& k) {
          ExpReq& r = k.r;
          r.q0 = __shfl_sync(0xffffffffu, front.q0, l), r.n = __shfl_sync(0xffffffffu, front.n, l);
          r.k0 = __shfl_sync(0xffffffffu, front.k0, l), r.start = __shfl_sync(0xffffffffu, front.start, l);
          r.tiles = __shfl_sync(0xffffffffu, front.tiles, l);
          r.bad = __shfl_sync(0xffffffffu, front.bad, l), r.none = __shfl_sync(0xffffffffu, front.none, l);
          const int64_t head = __shfl_sync(0xffffffffu, front_head, l), whole = head + (int64_t)kItemCost * r.tiles;
          int64_t o = at - cost - __shfl_sync(0xffffffffu, up[0] - own[0], l), before = 0;
          k.b = b0 + l;
          k.h = (int)quotient(o, whole);
          o -= k.h * whole;
          k.ti = 0;
          for (int n = exp_units<kRows>(r, 0); o >= n + kItemCost; n = exp_units<kRows>(r, ++k.ti)) o -= n + kItemCost, before += n;
          k.c = max((int)o - kItemCost, 0);
          k.item = items + __shfl_sync(0xffffffffu, up[2] - own[2], l) + (int64_t)k.h * r.tiles + k.ti;
          return units + __shfl_sync(0xffffffffu, up[1] - own[1], l) + k.h * head + before + k.c;
        };
        const unsigned m_lo = __ballot_sync(0xffffffffu, cost + up[0] > lo), m_hi = __ballot_sync(0xffffffffu, cost + up[0] > hi);
        if (!found && m_lo) begin = locate(lo, __ffs(m_lo) - 1, first), found = true;
        ExpStart behind;
        if (m_hi) end = locate(hi, __ffs(m_hi) - 1, behind);
        cost += __shfl_sync(0xffffffffu, up[0], 31), units += __shfl_sync(0xffffffffu, up[1], 31);
        items += __shfl_sync(0xffffffffu, up[2], 31);
      }
      if (end < 0) end = units;                                  // (the last run)
    }
    if (lane == 0) s_count = (int)(end - begin);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int count = s_count;
  const uint32_t tmem = s_tmem;
  volatile int* abort = &s_abort;

  if (warp >= kMmaWarp) {
    if (count == 0) {
      // nothing of this batch for this block
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- units, keys and queries
      int b = first.b, h = first.h, ti = first.ti, c = first.c;
      int64_t item = first.item;                  // the item's number among all
      ExpReq r = first.r;
      ExpUnit x{};
      int cnt = 0, at = 0;
      // up to 32 units at a time, one per lane
      auto batch = [&](int64_t u) {
        cnt = (int)min((int64_t)32, end - u);
        int bb = b, hh = h, tt = ti, cc = c;
        int64_t it = item;
        ExpReq rr = r;
        int units = exp_units<kRows>(rr, tt);
        auto turn = [&](int& b_, int& h_, int& t_, int64_t& i_, ExpReq& r_) {   // the item behind this one
          ++i_;
          if (++t_ < r_.tiles) return;
          t_ = 0;
          if (++h_ < A.H) return;
          h_ = 0;
          do r_ = exp_req<kRows>(A, ++b_);
          while (r_.tiles == 0 && b_ + 1 < A.B);
        };
        for (int step = lane; step > 0 && lane < cnt;) {              // forward by `lane` units
          const int left = units - cc;
          if (step < left) {
            cc += step;
            break;
          }
          step -= left;
          cc = 0;
          turn(bb, hh, tt, it, rr);
          units = exp_units<kRows>(rr, tt);
        }
        __syncwarp();
        if (lane < cnt) {
          const int64_t me = u + lane, ib = me - cc, ie = ib + units;
          const int row0 = tt * kRows;
          x.q0 = rr.q0 + row0, x.h = hh;
          x.rows = min(kRows, rr.n - row0);
          x.rel = rr.start + row0 - cc * kKeys;
          x.key0 = rr.k0 + cc * kKeys;
          const bool seen = !rr.none && x.rel + x.rows - 1 >= 0;
          x.last = seen ? min(x.rel + x.rows - 1, kKeys - 1) : -1;
          const bool first = me == ib || me == begin, last = me + 1 == ie || me + 1 == end;
          x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (seen ? 0 : kVoid) | (!seen || x.rel < kKeys - 1 ? kEdge : 0);
          const bool cut = ib < begin || ie > end;
          x.slot = !cut ? -1 : 2 * (int)blockIdx.x + (max(ib, begin) == begin ? 0 : 1);
          if (last && cut && ib >= begin) {
            LatentCut k{};
            // (the last unit's cost: the units before it, and its item and those before)
            k.follow = (int)run_owner(ie - 1 + kItemCost * (it + 1), total, runs) - (int)blockIdx.x;
            k.slot = x.slot, k.rows = x.rows, k.step = A.H, k.out = (int64_t)x.q0 * A.H + hh;
            parts.cuts[blockIdx.x] = k;
          }
        }
        // the cursor behind the batch: its last lane's unit, one further
        const int l = cnt - 1;
        b = __shfl_sync(0xffffffffu, bb, l), h = __shfl_sync(0xffffffffu, hh, l);
        ti = __shfl_sync(0xffffffffu, tt, l), c = __shfl_sync(0xffffffffu, cc, l) + 1, item = __shfl_sync(0xffffffffu, it, l);
        r = exp_req<kRows>(A, b);
        if (u + cnt < end && c == exp_units<kRows>(r, ti)) {
          c = 0;
          turn(b, h, ti, item, r);
        }
        at = 0;
      };
      int seg = 0;
      bool ok = true;
      for (int n = 0; n < count && ok; ++n) {
        if (at == cnt) batch(begin + n);
        const int us = n % kUnits, ks = n % kKStages;
        ok = warp_wait(&u_empty[us], ((n / kUnits) & 1) ^ 1, abort, A.err);
        if (!ok) break;
        if (lane == at) s_unit[us] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&u_full[us]));
        const int flags = __shfl_sync(0xffffffffu, x.flags, at), head = __shfl_sync(0xffffffffu, x.h, at);
        const int key0 = __shfl_sync(0xffffffffu, x.key0, at), q0 = __shfl_sync(0xffffffffu, x.q0, at);
        ++at;
        ok = warp_wait(&k_empty[ks], ((n / kKStages) & 1) ^ 1, abort, A.err);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&k_full[ks]);
          if (!(flags & kVoid)) {
            const uint32_t dst = smem_u32(k_buf + ks * kKBytes);
            mbar_arrive_expect_tx(bar, kKBytes);
            tma_load_3d(dst, &map_k, bar, 0, head, key0);
            tma_load_3d(dst + kAtom, &map_k, bar, 64, head, key0);
            tma_load_2d(dst + 2 * kAtom, &map_rope, bar, 0, key0);
          } else {
            mbar_arrive(bar);
          }
        }
        __syncwarp();
        if (flags & kFirst) {                     // the last segment's scores have left the queries' place
          for (int i = 0; i < TILES && ok; ++i) {
            ok = seg == 0 || warp_wait(&q_free[i], (seg - 1) & 1, abort, A.err);
            if (ok && lane == 0) {
              const uint32_t bar = smem_u32(&q_full[i]), dst = smem_u32(q_buf + i * kQTile);
              mbar_arrive_expect_tx(bar, kQTile);
#pragma unroll
              for (int a = 0; a < 3; ++a) tma_load_3d(dst + a * kAtom, &map_q, bar, 64 * a, head, q0 + i * kTile);
            }
            __syncwarp();
          }
          ++seg;
        }
      }
      // Copies in flight land before shared memory is given back: each is waited for by its
      // reader, or, when the run was given up, here.
      if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {}
      }
    } else if (warp == kValueWarp) {
      // ---------------------------------------------------------- values
      bool ok = true;
      for (int n = 0; n < count && ok; ++n) {
        const int us = n % kUnits;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        const int flags = s_unit[us].flags, head = s_unit[us].h, key0 = s_unit[us].key0;
        for (int i = 0; i < 2 && ok; ++i) {
          ok = warp_wait(&v_empty[n % kVStages][i], ((n / kVStages) & 1) ^ 1, abort, A.err);
          if (ok && lane == 0) {
            const uint32_t bar = smem_u32(&v_full[n % kVStages][i]), dst = smem_u32(v_buf + (n % kVStages * 2 + i) * kVHalf);
            if (!(flags & kVoid)) {
              mbar_arrive_expect_tx(bar, kVHalf);
              tma_load_3d(dst, &map_v, bar, 0, head, key0 + 64 * (1 - i));
              tma_load_3d(dst + kVHalf / 2, &map_v, bar, 64, head, key0 + 64 * (1 - i));
            } else {
              mbar_arrive(bar);
            }
          }
          __syncwarp();
        }
        if (ok && lane == 0) {
          mbar_arrive(smem_u32(&u_loaded[us]));
          mbar_arrive(smem_u32(&u_empty[us]));
        }
      }
      if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {}
      }
    } else if (warp < kLoadWarp) {
      // ---------------------------------------------------------- MMA issue, a warp per tile (or place)
      constexpr uint32_t idesc_s = make_idesc(kTile, kKeys, kFmtBF16, kFmtBF16, 0, 0);
      constexpr uint32_t idesc_o = make_idesc(kTile, kV, kFmtBF16, kFmtBF16, 0, 1);
      const int i = warp - kMmaWarp;
      const uint32_t col = i * kTileCols;         // all 512 columns are this block's: they start at 0
      const uint64_t dq = smem_desc(smem_u32(q_buf) + (kSplit ? 0 : i * kQTile), 0, 1024, kSwizzle128B);
      const uint64_t dk = smem_desc(smem_u32(k_buf), 0, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(smem_u32(v_buf), kVHalf / 2, 1024, kSwizzle128B);
      const bool issuer = elect_one();
      bool ok = tmem == 0;
      if (!ok) {
        *abort = 1;
        record_error(A.err, kDevTimeout);
      }
      uint32_t seg = 0, kept = 0;                 // kept: O holds something of this item
      int edges = 0;
      for (int n = 0; n < count && ok; ++n) {
        const int us = n % kUnits, ks = n % kKStages;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        const int flags = s_unit[us].flags;
        const uint32_t par = (kSplit ? n >> 1 : n) & 1;
        if (flags & kFirst) {
          ok = warp_wait(&q_full[kSplit ? 0 : i], seg++ & 1, abort, A.err);
          kept = 0;
        }
        if (kSplit && (n & 1) != i) {             // the other's unit
          if (flags & kEdge) ++edges;
          if ((flags & kLast) && issuer) mma_commit(smem_u32(&q_free[0]));
          __syncwarp();
          continue;
        }
        ok = ok && warp_wait(&k_full[ks], (n / kKStages) & 1, abort, A.err);
        if (!ok) break;
        tc_fence_after();
        if (issuer) {
          const uint64_t kd = desc_add(dk, ks * kKBytes);
#pragma unroll
          for (int k = 0; k < 12; ++k)
            mma_f16_ss(col, desc_add(dq, (k >> 2) * kAtom + (k & 3) * 32), desc_add(kd, (k >> 2) * kAtom + (k & 3) * 32), idesc_s,
                       k != 0);
          mma_commit(smem_u32(&s_full[i]));
          mma_commit(smem_u32(&k_empty[ks]));
          if (flags & kLast) mma_commit(smem_u32(&q_free[kSplit ? 0 : i]));
        }
        __syncwarp();
        if (flags & kEdge) {
          ok = warp_wait(&e_full[edges % kUnits], (edges / kUnits) & 1, abort, A.err);
          ++edges;
        }
#pragma unroll 1
        for (int half = 0; half < 2 && ok; ++half) {
          ok = warp_wait(&v_full[n % kVStages][half], (n / kVStages) & 1, abort, A.err) &&
               warp_wait(&p_full[i][half], par, abort, A.err);
          if (!ok) break;
          tc_fence_after();
          if (issuer) {
            const uint64_t vd = desc_add(dv, (n % kVStages * 2 + half) * kVHalf);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_ts(col + kOCol, col + 64 * (1 - half) + 8 * k, desc_add(vd, k * 2048), idesc_o,
                         (half | k) != 0 ? 1u : kept);
            mma_commit(smem_u32(&v_empty[n % kVStages][half]));
            if (half == 1) mma_commit(smem_u32(&o_done[i]));
          }
          __syncwarp();
        }
        kept = 1;
      }
      // Everything issued has finished before tensor and shared memory are given back.
      __syncwarp();
      if (issuer) {
        mma_commit(smem_u32(&drain[i]));
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&drain[i]), 0)) {
          if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_error(A.err, kDevTimeout);
            break;
          }
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- values of units not seen whole
      // (each warp has 32 columns, and so their notes, to itself)
      const int fw = warp - kFixWarp0;
      int seg = -1, edges = 0;
      bool ok = true;
      for (int n = 0; n < count && ok; ++n) {
        const int us = n % kUnits;
        // (its loads have been issued, so the values' barriers are in this unit's phase)
        ok = warp_wait(&u_loaded[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        const ExpUnit x = s_unit[us];
        if (x.flags & kFirst) {
          // (the slot's last segment ended four units ago at least, and u_empty has told so)
          ++seg;
          if (lane < 16) s_note[seg % kUnits][16 * fw + lane] = (uint32_t)kNoNote << 16 | kNoNote;
          __syncwarp();
        }
        if (x.flags & kEdge) {
          for (int i = 0; i < 2 && ok; ++i) {
            ok = warp_wait(&v_full[n % kVStages][i], (n / kVStages) & 1, abort, A.err);
            if (!ok) break;
            uint4* atom = reinterpret_cast<uint4*>(v_buf + (n % kVStages * 2 + i) * kVHalf + (fw >> 1) * (kVHalf / 2));
            const int ch = 4 * (fw & 1) + (lane & 3), key0 = 64 * (1 - i) + (lane >> 2);   // keys key0 + 8 k
            auto chunk = [&](int k) { return atom + (8 * k + (lane >> 2)) * 8 + (ch ^ (lane >> 2)); };
            // zero times a value is NaN exactly where the value is not finite
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = key0 + 8 * k <= x.last ? *chunk(k) : make_uint4(0, 0, 0, 0);
            __nv_bfloat162 sum = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t o[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&o[e]), __float2bfloat162_rn(0.f), sum);
              if (key0 + 8 * k > x.last) *chunk(k) = v[k];
            }
            if (__low2float(sum) != 0.f || __high2float(sum) != 0.f) {
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                if (key0 + 8 * k > x.last) break;
                const uint4 u = *chunk(k);
                const uint32_t o[4] = {u.x, u.y, u.z, u.w};
                uint32_t keep[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  keep[e] = o[e];
                  if ((o[e] & 0x7F80u) == 0x7F80u) keep[e] &= 0xFFFF0000u;
                  if ((o[e] & 0x7F800000u) == 0x7F800000u) keep[e] &= 0xFFFFu;
                }
                *chunk(k) = make_uint4(keep[0], keep[1], keep[2], keep[3]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if ((o[e >> 1] ^ keep[e >> 1]) >> (16 * (e & 1)) & 0xFFFFu)
                    note_min(s_note[seg % kUnits], 32 * fw + 8 * (lane & 3) + e, key0 + 8 * k - x.rel);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(smem_u32(&e_full[edges % kUnits]));
          ++edges;
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&u_empty[us]));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax: a thread per row
    const int i = warp >> 2;                       // tile
    const uint32_t tile = tmem + i * kTileCols + ((uint32_t)(32 * (warp & 3)) << 16);
    const int row = (kSplit ? 0 : kTile * i) + 32 * (warp & 3) + lane;
    const float f = fmaxf(A.scale_log2, 1.17549435e-38f);   // (a scale of 0 would make masked scores NaN)
    float M = kNone, l = 0.f;
    int seg = -1;
    bool notes = false, have = false;              // the segment had a unit with notes, one of this tile's
    for (int n = 0; n < count; ++n) {
      const int us = n % kUnits;
      if (!warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err)) break;
      const int flags = s_unit[us].flags;
      if (flags & kFirst) {
        ++seg;
        M = kNone, l = 0.f, notes = have = false;
      }
      const bool edge = (flags & kEdge) != 0;
      notes |= edge;
      const uint32_t par = (kSplit ? n >> 1 : n) & 1;
      if (!kSplit || (n & 1) == i) {
        if (!warp_wait(&s_full[i], par, abort, A.err)) break;
        tc_fence_after();
        // Keys 0 .. 63 are read for the maximum, then 64 .. 127, whose weights are formed first; then
        // the others again (all 128 at once would not fit beside the rest in 128 registers).
        const int lim = !edge ? kKeys : (flags & kVoid) || row >= s_unit[us].rows ? -1 : s_unit[us].rel + row;
        float s[64];
        auto read = [&](int key) {
          tmem_ld64(tile + key, s);
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (key + k > lim) s[k] = -INFINITY;
          }
        };
        auto most = [&]() {
          float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < 60; k += 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m4[j] = max3(m4[j], s[k + 2 * j], s[k + 2 * j + 1]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], s[60 + j]);
          return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        };
        read(0);
        float top = most();
        read(64);
        top = fmaxf(top, most()) * f;
        if (!have) {
          M = fmaxf(top, kNone);
        } else if (__any_sync(0xffffffffu, top > M + kMove)) {
          float keep = 1.f;
          if (top > M + kMove) keep = ex2(M - top), M = top;
          l *= keep;
#pragma unroll 1
          for (int k = 0; k < kV; k += 16) {
            float v[16];
            tmem_ld16(tile + kOCol + k, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= keep;
            tmem_st16(tile + kOCol + k, v);
          }
          tmem_st_wait();
        }
        float a[4] = {};
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (half) read(0);
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            fma2(s[k], s[k + 1], f, -M);
            fma2(s[k + 2], s[k + 3], f, -M);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[k + j] = ex2(s[k + j]);
            add2(a[0], a[1], s[k], s[k + 1]);
            add2(a[2], a[3], s[k + 2], s[k + 3]);
            p[k / 2] = pack_bf16(s[k], s[k + 1]);
            p[k / 2 + 1] = pack_bf16(s[k + 2], s[k + 3]);
          }
          tmem_st32(tile + 64 * (1 - half), p);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&p_full[i][half]));
        }
        l += (a[0] + a[1]) + (a[2] + a[3]);
        have = true;
      }
      if (kSplit && (flags & kLast)) {
        // ---- both places' maxima, sums and O are one; a place's warps take 64 of the columns
        const bool mine = (n & 1) == i;
        s_ml[kSplit ? i : 0][kSplit ? row : 0] = make_float2(M, have ? l : -1.f);
        if (have && !warp_wait(&o_done[i], mine ? par : (n - 1) >> 1 & 1, abort, A.err)) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&x_full));
        if (!warp_wait(&x_full, seg & 1, abort, A.err)) break;
        tc_fence_after();
        const ExpUnit x = s_unit[us];
        const float2 other = s_ml[kSplit ? 1 - i : 0][kSplit ? row : 0];
        const bool there = other.y != -1.f;       // (the same for all rows)
        const float Mx = !there ? M : have ? fmaxf(M, other.x) : other.x;
        const float fa = have ? ex2(M - Mx) : 0.f, fb = there ? ex2(other.x - Mx) : 0.f;
        const float sum = (have ? l * fa : 0.f) + (there ? other.y * fb : 0.f);
        const bool valid = row < x.rows, none = sum == 0.f;
        const float inv = none ? 0.f : x.slot < 0 ? 1.f / sum : 1.f;
        const int64_t at = (int64_t)(x.q0 + (valid ? row : 0)) * A.H + x.h;
        const int64_t part = (int64_t)x.slot * kRows + row;
        const uint32_t far = tmem + (1 - i) * kTileCols + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
        for (int k = 64 * i; k < 64 * i + 64; k += 16) {
          float v[16], u[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = u[j] = 0.f;
          if (have) tmem_ld16(tile + kOCol + k, v);
          if (__any_sync(0xffffffffu, there)) tmem_ld16(far + kOCol + k, u);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = (v[j] * fa + u[j] * fb) * inv;
            if (notes && !none && row >= (int)(int16_t)(s_note[seg % kUnits][(k + j) >> 1] >> (16 * (j & 1)))) v[j] = NAN;
          }
          if (!valid) {
          } else if (x.slot < 0) {
            uint4* dst = reinterpret_cast<uint4*>(A.out + at * kV + k);
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              dst[j / 8] = none ? make_uint4(0, 0, 0, 0)
                                : make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]), pack_bf16(v[j + 4], v[j + 5]),
                                             pack_bf16(v[j + 6], v[j + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(parts.o + part * kV + k);
#pragma unroll
            for (int j = 0; j < 16; j += 4) dst[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
          __syncwarp();
        }
        if (valid && i == 0) {
          if (x.slot >= 0) *reinterpret_cast<float2*>(parts.ml + part * 2) = make_float2(Mx, sum);
          else if (A.lse) A.lse[at] = none ? -INFINITY : (Mx + log2f(sum)) * 0.6931471805599453f;
        }
        // (the next item's products overwrite both)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&x_done));
        if (!warp_wait(&x_done, seg & 1, abort, A.err)) break;
      } else if (flags & kLast) {
        // ---- the segment's outputs, or its part
        if (!warp_wait(&o_done[i], par, abort, A.err)) break;
        tc_fence_after();
        const ExpUnit x = s_unit[us];
        const bool valid = row < x.rows, none = l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        const int64_t at = (int64_t)(x.q0 + (valid ? row : 0)) * A.H + x.h;
        const int64_t part = (int64_t)x.slot * kRows + row;
#pragma unroll 1
        for (int k = 0; k < kV; k += 16) {
          float v[16];
          tmem_ld16(tile + kOCol + k, v);
          tmem_ld_wait();
          if (notes && !none) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (row >= (int)(int16_t)(s_note[seg % kUnits][(k + j) >> 1] >> (16 * (j & 1)))) v[j] = NAN;
          }
          if (!valid) {
          } else if (x.slot < 0) {
            uint4* dst = reinterpret_cast<uint4*>(A.out + at * kV + k);
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              dst[j / 8] = none ? make_uint4(0, 0, 0, 0)
                                : make_uint4(pack_bf16(v[j] * inv, v[j + 1] * inv), pack_bf16(v[j + 2] * inv, v[j + 3] * inv),
                                             pack_bf16(v[j + 4] * inv, v[j + 5] * inv), pack_bf16(v[j + 6] * inv, v[j + 7] * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(parts.o + part * kV + k);
#pragma unroll
            for (int j = 0; j < 16; j += 4) dst[j / 4] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
        if (valid) {
          if (x.slot >= 0) *reinterpret_cast<float2*>(parts.ml + part * 2) = make_float2(M, l);
          else if (A.lse) A.lse[at] = none ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&u_empty[us]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

}  // namespace

// Tiles of an item: two (products of one while the other's softmax runs), but one where the mean
// request has no more rows than that. (16 requests of 100 rows in the mean over 1500 keys, 16 heads:
// 52 us with one tile, 79 with two.)
static int exp_tiles(int B, int T) { return T <= (int64_t)B * kTile ? 1 : 2; }

template <int TILES>
static cudaError_t exp_launch(const LatentExpandedArgs& A, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& rope,
                              const CUtensorMap& v, int num_sms, cudaStream_t st) {
  using S = ExpShape<TILES>;
  const LatentParts parts = latent_parts(A.scratch, num_sms, S::kRows, kV);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(latent_expanded_kernel<TILES>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  latent_expanded_kernel<TILES><<<num_sms, kThreads, S::kSmem, st>>>(q, k, rope, v, A, parts);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : latent_merge_launch<kV>(parts, num_sms, A.out, A.lse, st);
}

// (of two tiles, which serve any batch)
size_t latent_expanded_scratch_bytes(int num_sms) { return latent_parts_bytes(num_sms, ExpShape<2>::kRows, kV); }

cudaError_t latent_expanded_launch(const LatentExpandedArgs& A, const CUtensorMap& q, const CUtensorMap& k,
                                   const CUtensorMap& rope, const CUtensorMap& v, int num_sms, cudaStream_t st) {
  return exp_tiles(A.B, A.T) == 1 ? exp_launch<1>(A, q, k, rope, v, num_sms, st) : exp_launch<2>(A, q, k, rope, v, num_sms, st);
}

}  // namespace dsa
