// Grouped-query attention over the paged 8-bit cache for few query rows per key head:
// decode and verification over whole contexts, and listed blocks (the definitions are at
// dsa_gqa_attend and dsa_gqa_attend_blocks in include/dsa.h).
//
// A block (64 keys and values of one head, 2 * 64 * D bytes) is the unit of work; the time
// goes into bringing units from HBM (D = 128: 16 KB, which an SM's share of the bandwidth
// takes about 700 clocks to load). So the units of all (request, key head, row tile) items
// are laid end to end and cut into equal runs, and every run belongs to one warp, or a team
// of two or four warps where an item has more than 16 query rows. The warps of an SM work
// without meeting: each team brings its units' keys and values through a ring of its own by
// TMA and keeps its rows' sums in registers. An item that crosses a cut leaves partial results
// that a second kernel merges.
//
//   * 16 keys x 8 query rows per step on mma.sync m16n8k16 (f16, fp32 sums), the keys (and
//     the values' columns) as the 16 rows of A, so that a group of up to 8 heads wastes
//     nothing. tcgen05 would take its operands from shared memory or TMEM, i.e. a write and
//     a second read of every key and value converted to 16 bits; here the codes go from
//     shared memory to registers once, are converted there, and are fragments already. The
//     order of the summation index is free, so a lane's fragments are D/4 consecutive bytes
//     of a key, and a value pair's halves are put side by side by one byte permute.
//   * both 8-bit types are exact in f16. Queries are scaled by a power of two per row (so
//     that bf16's range fits f16) and are exact to 2^-38 of the row's largest value. (The e4m3
//     form of mma.sync, with the query as two e4m3 parts and the keys' codes as they are, was
//     slower: 1,184 us instead of 837 for the blocks of 2048 tokens.)
//   * the block's key scale multiplies the scores. Its value scale enters the exponent: with
//     M the running maximum of z + log2(v_scale), the weights p = 2^(z - M + log2(v_scale) + 15)
//     multiply the codes directly, and the softmax's sum is of p / v_scale / 2^15. p is rounded
//     to f16 for the product, the sum and all else is fp32. The largest p of a run's part is
//     2^15, so that all of f16's range lies below it: a p is off by 2^-11 of itself down to
//     2^-29 of the largest one, and by 2^-40 of the largest below that. (Behind a sink key
//     whose value is 0, or a block whose value scale dwarfs the others', the small weights are
//     what the output is made of; with p up to 1 they were lost from 2^-25 on.)
//
// 64 requests of 2048 to 8192 tokens with 64 query heads over 8 of 128 (671 MB) take 122 us in a
// graph, 8 of 131072 (2.15 GB) 340, 6.3 TB/s: HBM. 32 requests of 4096 to 16384 with 20 rows
// (685 MB) take 149: a unit takes a warp some 4,100 clocks, and rows 17 to 20 read the keys again.
//
// A lane whose row does not see a key sets p = 0; values that no row of the tile sees are
// zeroed, and where some rows see an e4m3 NaN value that others do not, the product is made
// token by token (0 * NaN would reach the others).
#include <algorithm>
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr float kLift = 15.f, kDown = 1.f / 32768.f;   // log2 of the largest weight, and what takes it back

// An 8x8 matrix of 16-bit values, a row per four lanes and two values per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The A fragments of a slice's values, 16 columns at a time: take(tile, a0, a1, a2, a3).
template <int D, bool I8, typename F>
__device__ __forceinline__ void value_tiles(const uint32_t (&v)[4][D / 32], F take) {
  uint32_t f[2][4];
  auto convert = [&](int j, uint32_t (&to)[4]) {
    const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
    codes_f16<I8>(__byte_perm(v[0][j >> 1], v[1][j >> 1], sel), to[0], to[1]);
    codes_f16<I8>(__byte_perm(v[2][j >> 1], v[3][j >> 1], sel), to[2], to[3]);
  };
  convert(0, f[0]);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {               // (the next tile is converted while this one is multiplied)
    if (j + 1 < D / 16) convert(j + 1, f[(j + 1) & 1]);
    take(j, f[j & 1][0], f[j & 1][1], f[j & 1][2], f[j & 1][3]);
  }
}

// Requests as the items see them: tokens [q0, q0 + n), items of `units` units each.
struct Request {
  int q0, n, len;
  int tiles, units;
  bool bad;
};
__device__ __forceinline__ Request request_of(const GqaAttendArgs& A, int b, int tile_rows) {
  Request r;
  const int c0 = __ldg(A.g.cu_q + b), c1 = __ldg(A.g.cu_q + b + 1);
  r.len = __ldg(A.g.seq_lens + b);
  r.bad = c0 < 0 || c1 < c0 || c1 > A.g.T || r.len > A.g.max_seq_len;
  r.q0 = min(max(c0, 0), A.g.T);
  r.n = max(min(c1, A.g.T) - r.q0, 0);
  if (r.bad || r.len < 0) r.len = 0;
  r.tiles = (r.n * A.G + tile_rows - 1) / tile_rows;
  r.units = max((r.len + kPage - 1) / kPage, 1);
  return r;
}

// A warp has NT tiles of 8 query rows; a team of MT warps shares its units, each with rows of
// its own. The team's ring holds halves (a unit's keys, or its values) in turn. kWarps: a block
// of threads per SM.
template <int D, int NT, int MT, int kWarps = 8>
struct Shape {
  static constexpr int kRows = 8 * NT * MT;
  static constexpr int kTeams = kWarps / MT;
  static constexpr int kHalf = kPage * D;                        // bytes
  static constexpr int kRing = (kWarps == 12 ? 2 : 3 * MT) * (128 / D);   // halves
  // Halves that a lead warp stays behind with new loads, so that it does not wait for the
  // others to have read the slot.
  static constexpr int kLag = MT == 1 ? 0 : 2;
  static constexpr size_t kSmem = (size_t)kTeams * kRing * kHalf + 1024;
};

template <int D, bool I8, int NT, int MT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 1)
    gqa_rows_kernel(const GqaAttendArgs A, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const GqaParts parts) {
  using S = Shape<D, NT, MT, kWarps>;
  constexpr int kRows = S::kRows, kRing = S::kRing, kAhead = S::kRing - S::kLag;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[S::kTeams][kRing], s_empty[S::kTeams][kRing];
  __shared__ int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int team = warp / MT, m = warp % MT;
  const int run = team * gridDim.x + blockIdx.x, runs = S::kTeams * gridDim.x;   // teams of an SM far apart
  const bool listed = A.blocks != nullptr;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < S::kTeams * kRing; ++i) {
      mbar_init(smem_u32(&s_full[0][0] + i), 1);
      mbar_init(smem_u32(&s_empty[0][0] + i), MT);
    }
    s_abort = 0;
    fence_mbar_init();
  }
  if (m == 0 && lane == 0) parts.cuts[run].follow = 0;
  __syncthreads();

  // ---- the run [begin, end) of all units; whole contexts: the request it starts in and where
  // that request's units begin. A.whole: runs are cut between items (few units each), and
  // nothing has to be merged.
  int64_t total = 0, begin, end, base = 0;
  int req = 0;
  if (listed) {
    total = (int64_t)A.g.T * A.c.Hkv * (A.whole ? 1 : A.n_sel);
    // (the last runs first: they have no work in small batches)
    const int64_t at = ((int64_t)(kWarps - 1 - warp) * gridDim.x + (gridDim.x - 1 - blockIdx.x)) * 32 + lane;
    RequestCheck(A.g, at).report(A.g, at, (int64_t)gridDim.x * (32 * kWarps), A.err);
  } else {
    for (int b0 = 0; b0 < A.g.B; b0 += 32) {
      if (b0 + lane < A.g.B) {
        const Request r = request_of(A, b0 + lane, kRows);
        total += (int64_t)A.c.Hkv * r.tiles * (A.whole ? 1 : r.units);
        if (r.bad && run == 0 && m == 0) record_error(A.err, kDevBadIndex);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const int used = (int)min((int64_t)runs, (total + A.min_run - 1) / A.min_run);
  if (run >= used) return;
  begin = split_begin(run, total, used);
  end = split_begin(run + 1, total, used);
  if (listed) {
    if (A.whole) begin *= A.n_sel, end *= A.n_sel;
  } else {
    // the request that item or unit `at` lies in, and the unit that it is or begins with
    auto locate = [&](int64_t at, int& in, int64_t& in_base) {
      int64_t before = 0, unit = 0;                // items or units, and units, of the requests before
      for (int b0 = 0; b0 < A.g.B; b0 += 32) {
        int64_t w = 0, u = 0;
        int each = 1;
        if (b0 + lane < A.g.B) {
          const Request r = request_of(A, b0 + lane, kRows);
          u = (int64_t)A.c.Hkv * r.tiles * r.units;
          w = A.whole ? (int64_t)A.c.Hkv * r.tiles : u;
          each = A.whole ? r.units : 1;
        }
        int64_t wsum = w, usum = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, wsum, o), z = __shfl_up_sync(0xffffffffu, usum, o);
          if (lane >= o) wsum += v, usum += z;
        }
        const unsigned mask = __ballot_sync(0xffffffffu, before + wsum > at);
        if (mask) {
          const int l = __ffs(mask) - 1;
          in = b0 + l;
          in_base = unit + __shfl_sync(0xffffffffu, usum - u, l);
          return in_base + (at - before - __shfl_sync(0xffffffffu, wsum - w, l)) * __shfl_sync(0xffffffffu, each, l);
        }
        before += __shfl_sync(0xffffffffu, wsum, 31);
        unit += __shfl_sync(0xffffffffu, usum, 31);
      }
      return unit;                                 // (at == total)
    };
    if (A.whole) {
      int64_t b2 = 0;
      int r2 = 0;
      end = locate(end, r2, b2);
    }
    begin = locate(begin, req, base);
  }
  volatile int* abort = &s_abort;

  // ---- units, up to 32 at a time, one per lane; a batch stays within a request
  struct Lane {
    float ks, vs;               // the block's scales
    int flags, rel;             // position of token 0, less the block's first position
    int q0, n, row0, h, slot;
    int tile;                   // page * Hkv + h, or -1: nothing to see
  };
  int64_t bu = begin;           // the next batch's first unit
  Request r{};
  if (!listed) r = request_of(A, req, kRows);
  auto batch = [&](Lane& x) {
    x = Lane{};
    x.tile = -1;
    int64_t item_begin = 0, item_end = 0;
    int c = 0, bb = req, cnt;
    bool sees = false;
    if (!listed) {
      int64_t mine = (int64_t)A.c.Hkv * r.tiles * r.units;
      while (bu >= base + mine) {                // the next request with tokens
        base += mine;
        r = request_of(A, ++req, kRows);
        mine = (int64_t)A.c.Hkv * r.tiles * r.units;
      }
      bb = req;
      cnt = (int)min((int64_t)32, min(end, base + mine) - bu);
      if (lane < cnt) {
        const int64_t o = bu + lane - base, item = o / r.units;
        c = (int)(o - item * r.units);
        item_begin = base + item * r.units;
        item_end = item_begin + r.units;
        x.h = (int)(item / r.tiles);
        x.row0 = (int)(item % r.tiles) * kRows;
        x.q0 = r.q0;
        x.n = r.n;
        x.rel = r.len - r.n - c * kPage;
        const int last = min(r.n - 1, (x.row0 + kRows - 1) / A.G);    // the tile's last token
        sees = c * kPage < r.len && x.rel + last >= 0;
      }
    } else {
      cnt = (int)min((int64_t)32, end - bu);
      if (lane < cnt) {
        const int64_t item = (bu + lane) / A.n_sel;
        const int i = (int)(bu + lane - item * A.n_sel);
        item_begin = item * A.n_sel;
        item_end = item_begin + A.n_sel;
        const int t = (int)(item / A.c.Hkv);
        x.h = (int)(item % A.c.Hkv);
        x.q0 = t;
        const bool real = t < __ldg(A.g.cu_q + A.g.B);
        x.n = real ? 1 : 0;                      // no rows: a padding token's outputs stay
        const QueryInfo qi = query_info(A.g, t);
        bb = qi.b;
        const bool bad = real && (t < __ldg(A.g.cu_q + bb) || t >= __ldg(A.g.cu_q + bb + 1) ||
                                  __ldg(A.g.cu_q + bb + 1) > A.g.T || qi.len > A.g.max_seq_len);
        if (bad) record_error(A.err, kDevBadIndex);
        if (real && !bad && qi.pos >= 0 && qi.pos < qi.len) {
          const int* list = A.blocks + item * A.n_sel;
          c = __ldg(list + i);
          sees = c >= 0 && c <= (qi.pos >> 6);
          if (sees && i > 0) {
            const int before = __ldg(list + i - 1);
            if (before < 0 || before >= c) {
              record_error(A.err, kDevBadIndex);
              sees = false;
            }
          }
          x.rel = qi.pos - c * kPage;
        }
      }
    }
    if (lane < cnt) {
      if (sees) {
        const int page = gqa_page(A.g, bb, c);
        if (page < 0) {
          record_error(A.err, kDevBadIndex);
          sees = false;
        } else {
          x.tile = page * A.c.Hkv + x.h;
          x.vs = __ldg(A.c.v_scale + x.tile);
          x.ks = __ldg(A.c.k_scale + x.tile);
        }
      }
      const int64_t at = bu + lane;
      const bool first = at == item_begin || at == begin, last = at + 1 == item_end || at + 1 == end;
      x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (sees ? 0 : kVoid);
      const bool cut = item_begin < begin || item_end > end;
      x.slot = !cut ? -1 : 2 * run + (max(item_begin, begin) == begin ? 0 : 1);
      if (!A.whole && m == 0 && last && cut && item_begin >= begin) {   // the item's merge goes by this run's index
        Cut k{};
        k.follow = (int)split_owner(item_end - 1, total, used) - run;
        k.slot = x.slot;
        k.q0 = x.q0, k.n = x.n, k.row0 = x.row0, k.h = x.h;
        parts.cuts[run] = k;
      }
    }
    __syncwarp();
    bu += cnt;
    return cnt;
  };

  // ---- loads: half j (unit j / 2's keys or values) goes to ring slot j % kRing
  uint8_t* ring = smem + (size_t)team * kRing * S::kHalf;
  uint64_t* full = s_full[team];
  uint64_t* empty = s_empty[team];
  Lane x, y;                                     // the batch of the unit at work, and the next one
  int cnt = batch(x), at = 0;                    // lane of the unit at work
  int ycnt = 0, lat = 0;                         // lane of the next load, in x, or in y if ycnt
  int lslot = 0;
  uint32_t lphase = 1;
  int left = 2 * (int)(end - begin);             // halves to load
  int ahead = 0;                                 // halves loaded and not yet read
  const bool issuer = elect_one();
  bool lvalues = false;
  int ltile = -1;
  const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full);

  // ---- computing
  constexpr int kSteps = D / 16;                 // k16 steps of a score = words of a lane's D/4 key bytes
  constexpr int kTiles = D / 16;                 // 16-column tiles of the output
  constexpr int kVw = D / 32;                    // words of a lane's D/8 bytes of a value
  constexpr int kSlices = kPage / 16, kPair = 2;
  const int q = lane & 3, lrow = lane >> 2;
  const int G = A.G, H = A.G * A.c.Hkv;
  uint32_t qf[NT][kSteps][2];
  float o[NT][kTiles][4];                        // [.][j]: columns lrow*D/8 + 2j (0, 1) and + 1 (2, 3) of rows 2q, 2q+1
  float M[NT][2], l[NT][2], rowf[NT][2];         // of rows 8i + 2q and + 1
  int tok[NT][2];                                // their tokens, or far below any limit
  int tok_lo = 0, tok_hi = 0;                    // of the warp's rows (tok_hi < 0: none)
  uint32_t pb[kSlices][NT][2];                   // weights, f16: rows by lane group, keys 2q, 2q+1 (0) and + 8 (1)
  int flags = 0, rel = 0, seen = 0;
  bool some = false, whole = false, values = false, ok = true;
  int slot = 0;
  uint32_t phase = 0;

  // Each turn loads ahead, then works on one half.
#pragma unroll 1
  for (int todo = left; todo > 0; --todo) {
    // up to kAhead halves ahead, but not past the batch after the one at work
    while (left > 0 && ahead < kAhead) {
      if (!lvalues && lat == (ycnt ? ycnt : cnt)) {
        if (ycnt) break;
        ycnt = batch(y);
        lat = 0;
      }
      if (!lvalues) ltile = __shfl_sync(0xffffffffu, ycnt ? y.tile : x.tile, lat);
      if (m == 0) {
        if (MT > 1) {
          ok = warp_wait(&empty[lslot], lphase, abort, A.err);
          if (!ok) break;
        }
        if (issuer) {
          const uint32_t bar = full0 + 8 * lslot, dst = ring0 + lslot * S::kHalf;
          if (ltile < 0) {
            mbar_arrive(bar);
          } else {
            mbar_arrive_expect_tx(bar, S::kHalf);
            if (lvalues) tma_load_3d(dst, &map_v, bar, 0, 0, ltile);
            else tma_load_3d(dst, &map_k, bar, 0, 0, ltile);
          }
        }
        __syncwarp();
      }
      --left, ++ahead;
      if (lvalues) ++lat;
      lvalues = !lvalues;
      if (++lslot == kRing) lslot = 0, lphase ^= 1u;
    }
    ok = ok && warp_wait(&full[slot], phase, abort, A.err);
    if (!ok) {
      if (m == 0 && lane == 0) {
        // Gave up: copies still in flight must land before the shared memory is given back (each
        // slot's last phase; one that was never filled counts as complete).
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < kRing; ++i) {
          const uint32_t par = i < lslot ? lphase ^ 1u : lphase;
          while (!mbar_test_wait(smem_u32(&full[i]), par) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
      return;
    }
    if (!values) {
      // ============================================================ keys
      flags = __shfl_sync(0xffffffffu, x.flags, at), rel = __shfl_sync(0xffffffffu, x.rel, at);
      const float kf = __shfl_sync(0xffffffffu, x.ks, at) * A.scale_log2, vs = __shfl_sync(0xffffffffu, x.vs, at);
      const float lv = __log2f(vs), ivs = __frcp_rn(vs);
      if (flags & kFirst) {
        const int q0 = __shfl_sync(0xffffffffu, x.q0, at), n = __shfl_sync(0xffffffffu, x.n, at);
        const int h = __shfl_sync(0xffffffffu, x.h, at), r0 = __shfl_sync(0xffffffffu, x.row0, at) + m * 8 * NT;
        const int rows = n * G;
        tok_lo = r0 / G;
        tok_hi = r0 < rows ? min(n - 1, (r0 + 8 * NT - 1) / G) : -1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int row = r0 + 8 * i + lrow;
          const bool valid = row < rows;
          const int t = valid ? row / G : 0;
          const uint4* src = reinterpret_cast<const uint4*>(
              A.q + (int64_t)(q0 + t) * A.q_stride + (int64_t)(h * G + (valid ? row - t * G : 0)) * D + q * (D / 4));
          uint32_t w[D / 8];
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint4 v = valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
            w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
          }
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) big = max3(big, fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k])));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // the row times 2^(14 - e), e the exponent of its largest value (none for infinities)
          const int e = min(max((int)(__float_as_uint(big) >> 23), 15), 254);
          const float up = __uint_as_float((uint32_t)(268 - e) << 23);
          const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
          for (int k = 0; k < D / 8; ++k) qf[i][k >> 1][k & 1] = pack_f16(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int mine = r0 + 8 * i + 2 * q + hh;
            rowf[i][hh] = __shfl_sync(0xffffffffu, down, 4 * (2 * q + hh));
            tok[i][hh] = mine < rows ? mine / G : -(1 << 30);
            M[i][hh] = kNone;
            l[i][hh] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kTiles; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
        }
      }
      seen = (flags & kVoid) ? -1 : min(rel + tok_hi, kPage - 1);   // last key any row of the warp sees
      some = tok_hi >= 0 && seen >= 0;
      whole = rel + tok_lo >= kPage - 1;                            // every row sees every key
      if (some) {
        // ---- scores: s[sl][i][0..3] are keys lrow (0, 1) and lrow + 8 (2, 3) of slice sl with rows 2q,
        // 2q+1 (the steps of kPair slices in turn: each waits for its own previous one only)
        float s[kSlices][NT][4];
        const uint32_t kt = ring0 + slot * S::kHalf;
#pragma unroll
        for (int s0 = 0; s0 < kSlices; s0 += kPair) {
#pragma unroll
          for (int sl = s0; sl < s0 + kPair; ++sl)
#pragma unroll
            for (int i = 0; i < NT; ++i) s[sl][i][0] = s[sl][i][1] = s[sl][i][2] = s[sl][i][3] = 0.f;
#pragma unroll
          for (int part = 0; part < D / 64; ++part) {
            uint4 kw[kPair][2];
#pragma unroll
            for (int sl = 0; sl < kPair; ++sl)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t row = kt + (16 * (s0 + sl) + 8 * j + lrow) * D;
                kw[sl][j] = lds128(row + ((D == 128 ? (2 * q + part) ^ lrow : q ^ ((lrow >> 1) & 3)) << 4));
              }
            // (a step's fragments are converted while the step before is multiplied)
            uint32_t f[2][kPair][4];
            auto convert = [&](int k, uint32_t (&to)[kPair][4]) {
#pragma unroll
              for (int sl = 0; sl < kPair; ++sl) {
                codes_f16<I8>(word(kw[sl][0], k), to[sl][0], to[sl][2]);
                codes_f16<I8>(word(kw[sl][1], k), to[sl][1], to[sl][3]);
              }
            };
            convert(0, f[0]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k < 3) convert(k + 1, f[(k + 1) & 1]);
#pragma unroll
              for (int sl = 0; sl < kPair; ++sl)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                  mma16816(s[s0 + sl][i], f[k & 1][sl][0], f[k & 1][sl][1], f[k & 1][sl][2], f[k & 1][sl][3],
                           qf[i][4 * part + k][0], qf[i][4 * part + k][1]);
            }
          }
        }
        // ---- softmax
        bool grew = false;
        float keep[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = kf * rowf[i][h];
            float mx = -INFINITY;
#pragma unroll
            for (int sl = 0; sl < kSlices; ++sl) {
              s[sl][i][h] *= f, s[sl][i][2 + h] *= f;
              if (!whole) {
                const int lim = rel + tok[i][h] - 16 * sl;
                if (lrow > lim) s[sl][i][h] = -INFINITY;
                if (lrow + 8 > lim) s[sl][i][2 + h] = -INFINITY;
              }
              mx = max3(mx, s[sl][i][h], s[sl][i][2 + h]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float Mo = M[i][h], Mn = fmaxf(Mo, mx + lv);
            grew |= Mn > Mo;
            keep[i][h] = ex2(Mo - Mn);
            M[i][h] = Mn;
            // (where scores are so large that M and lv do not add exactly, this block's largest
            // weight is still 2^15 if M is its own, and not above it if not)
            const float ref = (mx + lv >= Mo ? mx : fmaxf(Mn - lv, mx)) - kLift;
            float sum = 0.f;
#pragma unroll
            for (int sl = 0; sl < kSlices; ++sl) {
              s[sl][i][h] = ex2(s[sl][i][h] - ref);
              s[sl][i][2 + h] = ex2(s[sl][i][2 + h] - ref);
              sum += s[sl][i][h] + s[sl][i][2 + h];
            }
            l[i][h] = l[i][h] * keep[i][h] + sum * kDown * ivs;
          }
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl) {
            pb[sl][i][0] = transpose8(pack_weights(s[sl][i][0], s[sl][i][1]));
            pb[sl][i][1] = transpose8(pack_weights(s[sl][i][2], s[sl][i][3]));
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
              o[i][j][0] *= keep[i][0], o[i][j][1] *= keep[i][1], o[i][j][2] *= keep[i][0], o[i][j][3] *= keep[i][1];
        }
      }
    } else {
      // ============================================================ values times weights
      if (some) {
        const uint32_t vt = ring0 + slot * S::kHalf;
#pragma unroll
        for (int sl = 0; sl < kSlices; ++sl) {
          // vw[k]: token 2q + (k & 1) + 8 * (k >> 1) of the slice, D/8 bytes from column (D/8) * lrow
          uint32_t vw[4][kVw];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tk = 16 * sl + 2 * q + (k & 1) + 8 * (k >> 1);
            if constexpr (D == 128) {
              const uint4 a = lds128(vt + tk * D + ((lrow ^ (tk & 7)) << 4));
              vw[k][0] = a.x, vw[k][1] = a.y, vw[k][2] = a.z, vw[k][3] = a.w;
            } else {
              const uint2 a = lds64(vt + tk * D + (((lrow >> 1) ^ ((tk >> 1) & 3)) << 4) + (lrow & 1) * 8);
              vw[k][0] = a.x, vw[k][1] = a.y;
            }
          }
          bool apart = false;                     // a NaN value that only some rows may meet
          if (!whole) {
            bool nan = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool out = 16 * sl + 2 * q + (k & 1) + 8 * (k >> 1) > seen;
#pragma unroll
              for (int w = 0; w < kVw; ++w) {
                if (out) vw[k][w] = 0u;
                if (!I8) nan |= __vcmpeq4(vw[k][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
              }
            }
            apart = !I8 && __any_sync(0xffffffffu, nan);
          }
          if (!apart) {
            value_tiles<D, I8>(vw, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
              for (int i = 0; i < NT; ++i) mma16816(o[i][j], a0, a1, a2, a3, pb[sl][i][0], pb[sl][i][1]);
            });
          } else {
#pragma unroll 1
            for (int t = tok_lo; t <= tok_hi; ++t) {
              uint32_t v[4][kVw];
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int w = 0; w < kVw; ++w)
                  v[k][w] = 16 * sl + 2 * q + (k & 1) + 8 * (k >> 1) > rel + t ? 0u : vw[k][w];
              value_tiles<D, I8>(v, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                  float c[4] = {o[i][j][0], o[i][j][1], o[i][j][2], o[i][j][3]};
                  mma16816(c, a0, a1, a2, a3, pb[sl][i][0], pb[sl][i][1]);
                  if (tok[i][0] == t) o[i][j][0] = c[0], o[i][j][2] = c[2];
                  if (tok[i][1] == t) o[i][j][1] = c[1], o[i][j][3] = c[3];
                }
              });
            }
          }
        }
      }
      if (flags & kLast) {
        // ---- the item's outputs, or the run's part of it; a lane holds columns lrow*D/8 .. of its rows
        const int q0 = __shfl_sync(0xffffffffu, x.q0, at), h0 = __shfl_sync(0xffffffffu, x.h, at);
        const int row0 = __shfl_sync(0xffffffffu, x.row0, at), pslot = __shfl_sync(0xffffffffu, x.slot, at);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float sum = l[i][h];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            if (tok[i][h] >= 0) {
              const int rr = m * 8 * NT + 8 * i + 2 * q + h;             // row of the item's tile
              auto col = [&](int d) { return o[i][d >> 1][2 * (d & 1) + h] * kDown; };
              if (pslot < 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t to = (int64_t)(q0 + tok[i][h]) * H + h0 * G + (row0 + rr - tok[i][h] * G);
                uint4* dst = reinterpret_cast<uint4*>(A.out + to * D + lrow * (D / 8));
#pragma unroll
                for (int d = 0; d < D / 8; d += 8) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(col(d + 2 * k) * inv, col(d + 2 * k + 1) * inv);
                    w[k] = *reinterpret_cast<const uint32_t*>(&v);
                  }
                  dst[d / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (A.lse && lrow == 0) A.lse[to] = sum == 0.f ? -INFINITY : (M[i][h] + log2f(sum)) * 0.6931471805599453f;
              } else {
                const int64_t to = (int64_t)pslot * kRows + rr;
                float4* dst = reinterpret_cast<float4*>(parts.o + to * D + lrow * (D / 8));
#pragma unroll
                for (int d = 0; d < D / 8; d += 4) dst[d / 4] = make_float4(col(d), col(d + 1), col(d + 2), col(d + 3));
                if (lrow == 0) *reinterpret_cast<float2*>(parts.ml + to * 2) = make_float2(M[i][h], sum);
              }
            }
            __syncwarp();
          }
      }
      if (++at == cnt) {                           // on to the next batch (which the loads have reached)
        x = y;
        cnt = ycnt, at = 0, ycnt = 0;
      }
    }
    // the half has been read: by the whole warp, then by the team
    values = !values;
    __syncwarp();
    if (MT > 1 && lane == 0) mbar_arrive(smem_u32(&empty[slot]));
    if (++slot == kRing) slot = 0, phase ^= 1u;
    --ahead;
  }
}

// Merges the parts of items that were cut, in the order of the runs: block c (x) looks whether
// run c holds an item's first part, and if so merges eight of its rows (y). The warps share the
// parts, each adding its own for all eight rows (so that eight rows' loads are in flight), then
// each finishes one row.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) gqa_merge_kernel(const GqaAttendArgs A, const GqaParts s) {
  constexpr int V = D / 32, kRows = 8;
  __shared__ float s_o[kMergeWarps][kRows][D];
  __shared__ float2 s_ml[kMergeWarps][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const Cut k = s.cuts[blockIdx.x];
  if (k.follow <= 0) return;
  const int parts = k.follow + 1, r0 = blockIdx.y * kRows;
  if (k.row0 + r0 >= k.n * A.G) return;
  float M[kRows], l[kRows], o[kRows][V];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    M[r] = kNone, l[r] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) o[r][j] = 0.f;
  }
  const unsigned rows = __ballot_sync(0xffffffffu, k.row0 + r0 + (lane & 7) < k.n * A.G) & 0xFFu;   // (others were not written)
  for (int p = warp; p < parts; p += kMergeWarps) {
    const int64_t slot = p == 0 ? k.slot : 2 * (int64_t)(blockIdx.x + p);
    const int64_t at = slot * s.rows + r0;
    float2 ml[kRows];
    float v[kRows][V];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!((rows >> r) & 1u)) continue;
      ml[r] = __ldcg(reinterpret_cast<const float2*>(s.ml + (at + r) * 2));
      if constexpr (V == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(s.o + (at + r) * D) + lane);
        v[r][0] = f.x, v[r][1] = f.y, v[r][2] = f.z, v[r][3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(s.o + (at + r) * D) + lane);
        v[r][0] = f.x, v[r][1] = f.y;
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!((rows >> r) & 1u)) continue;
      const float Mn = fmaxf(M[r], ml[r].x), a = ex2(M[r] - Mn), b = ex2(ml[r].x - Mn);
      M[r] = Mn;
      l[r] = l[r] * a + ml[r].y * b;
#pragma unroll
      for (int j = 0; j < V; ++j) o[r][j] = o[r][j] * a + v[r][j] * b;
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int j = 0; j < V; ++j) s_o[warp][r][lane * V + j] = o[r][j];
    if (lane == 0) s_ml[warp][r] = make_float2(M[r], l[r]);
  }
  __syncthreads();
  const int row = k.row0 + r0 + warp;
  if (row >= k.n * A.G) return;
  float Mt = kNone, lt = 0.f, ot[V] = {};
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) Mt = fmaxf(Mt, s_ml[w][warp].x);
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float2 ml = s_ml[w][warp];
    const float b = ex2(ml.x - Mt);
    lt += ml.y * b;
#pragma unroll
    for (int j = 0; j < V; ++j) ot[j] += s_o[w][warp][lane * V + j] * b;
  }
  const int t = row / A.G;
  const int64_t at = (int64_t)(k.q0 + t) * (A.G * A.c.Hkv) + k.h * A.G + (row - t * A.G);
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  __nv_bfloat162 w[V / 2];
#pragma unroll
  for (int j = 0; j < V / 2; ++j) w[j] = __floats2bfloat162_rn(ot[2 * j] * inv, ot[2 * j + 1] * inv);
  if constexpr (V == 4) *(reinterpret_cast<uint2*>(A.out + at * D) + lane) = *reinterpret_cast<uint2*>(w);
  else *(reinterpret_cast<uint32_t*>(A.out + at * D) + lane) = *reinterpret_cast<uint32_t*>(w);
  if (A.lse && lane == 0) A.lse[at] = lt == 0.f ? -INFINITY : (Mt + log2f(lt)) * 0.6931471805599453f;
}

// Items of at most this many units are not cut: a warp takes them about as long as the launch
// of the merge.
constexpr int kWhole = 2;

// Query rows (tokens x heads of a key head) that meet a unit together. Up to 16 rows: a warp
// has them all. More: a unit's codes are converted by two or four warps, each for 16 of the
// rows. Above 64: gqa_tiles.cu; above 32 as well if the contexts may have 64 units an SM and
// more, for it is quicker by unit but slower to start (48 rows, 32 requests of 4096 to 16384
// tokens: 302 instead of 412 us, one request of 100000: 97 instead of 137; 96 requests of 100
// to 400 tokens, 35 units an SM: 85 instead of 73, one request of 2000: 20 instead of 17).
int rows_per_item(const GeomDev& g, int Hkv, int G, bool listed, int num_sms) {
  const int64_t rows = listed ? G : ((int64_t)g.T + g.B - 1) / g.B * G;
  const int64_t units = (int64_t)g.B * Hkv * ((g.max_seq_len + kPage - 1) / kPage);
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 && units < (int64_t)64 * num_sms ? 64 : kGqaTileRows;
}

// Warps per SM. Lists that give twelve warps 32 units each take twelve: the codes' conversion
// bounds them (their blocks come from L2), and three warps a sub-partition hide more of its
// latency than two (2048 tokens, 32 of 256 blocks each: 837 us instead of 954). Otherwise eight,
// with deeper rings and fewer parts to merge (decode 121 instead of 124 us, 32 blocks of 131072
// tokens for 8 requests 19 instead of 25).
int rows_warps(int64_t T, int Hkv, int rows, int n_sel, int num_sms) {
  return rows == 8 && T * Hkv * n_sel >= (int64_t)32 * 12 * num_sms ? 12 : 8;
}

int rows_runs(int rows, int warps, int num_sms) { return warps / (rows <= 16 ? 1 : rows / 16) * num_sms; }

template <int D, bool I8, int NT, int MT, int kWarps>
cudaError_t launch(GqaAttendArgs A, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms, cudaStream_t st) {
  using S = Shape<D, NT, MT, kWarps>;
  constexpr int rows = S::kRows;
  const int runs = rows_runs(rows, kWarps, num_sms);
  const GqaParts s = gqa_parts(A.scratch, runs, rows);
  // The shortest run: with few items of many units, shorter runs save a warp time that merging
  // their parts costs again (a unit takes a lone warp about as long as the merge takes for 16 parts).
  const int most = A.blocks ? A.n_sel : (A.g.max_seq_len + kPage - 1) / kPage;
  A.min_run = 1;
  A.whole = most <= kWhole;
  while (!A.whole && (A.min_run + 1) * (A.min_run + 1) * 16 <= most) ++A.min_run;
  auto kern = gqa_rows_kernel<D, I8, NT, MT, kWarps>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kern<<<num_sms, 32 * kWarps, S::kSmem, st>>>(A, mk, mv, s);
  e = cudaGetLastError();
  return e != cudaSuccess || A.whole ? e : gqa_merge_launch(A, s, runs, st);
}

template <int D, bool I8>
cudaError_t launch_rows(const GqaAttendArgs& A, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms, cudaStream_t st) {
  switch (rows_per_item(A.g, A.c.Hkv, A.G, A.blocks != nullptr, num_sms)) {
    case 8:
      if (rows_warps(A.g.T, A.c.Hkv, 8, A.blocks ? A.n_sel : 0, num_sms) == 12)
        return launch<D, I8, 1, 1, 12>(A, mk, mv, num_sms, st);
      return launch<D, I8, 1, 1, 8>(A, mk, mv, num_sms, st);
    case 16: return launch<D, I8, 2, 1, 8>(A, mk, mv, num_sms, st);
    case 32: return launch<D, I8, 2, 2, 8>(A, mk, mv, num_sms, st);
    default: return launch<D, I8, 2, 4, 8>(A, mk, mv, num_sms, st);
  }
}

}  // namespace

cudaError_t gqa_merge_launch(const GqaAttendArgs& A, const GqaParts& s, int grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, s.rows / kMergeWarps);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return A.c.D == 128 ? cudaLaunchKernelEx(&cfg, gqa_merge_kernel<128>, A, s) : cudaLaunchKernelEx(&cfg, gqa_merge_kernel<64>, A, s);
}

// Enough for any smaller T as well: a buffer sized for a batch's largest step serves its others.
size_t gqa_attend_scratch_bytes(const dsa_geom_t* g, int Hkv, int D, int G, int n_sel, int num_sms) {
  GeomDev gd{};
  gd.B = g->B, gd.T = g->T, gd.max_seq_len = g->max_seq_len;
  const int most = rows_per_item(gd, Hkv, G, n_sel > 0, num_sms);
  size_t need = 0;
  for (int rows : {8, 16, 32, 64, kGqaTileRows}) {
    if (rows > most) break;
    const int runs = rows > 64 ? num_sms : rows_runs(rows, rows_warps(g->T, Hkv, rows, n_sel, num_sms), num_sms);
    need = std::max(need, gqa_parts_bytes(runs, rows, D));
  }
  return need;
}

cudaError_t gqa_attend_launch(const GqaAttendArgs& A, int num_sms, cudaStream_t st) {
  if (rows_per_item(A.g, A.c.Hkv, A.G, A.blocks != nullptr, num_sms) > 64) return gqa_tiles_launch(A, num_sms, st);
  CUtensorMap mk, mv;
  const uint64_t tiles = (uint64_t)A.g.num_pages * A.c.Hkv;
  if (!encode_code_tiles(&mk, A.c.k, A.c.D, tiles) || !encode_code_tiles(&mv, A.c.v, A.c.D, tiles))
    return cudaErrorInvalidValue;
  if (A.c.D == 128) return A.c.i8 ? launch_rows<128, true>(A, mk, mv, num_sms, st) : launch_rows<128, false>(A, mk, mv, num_sms, st);
  return A.c.i8 ? launch_rows<64, true>(A, mk, mv, num_sms, st) : launch_rows<64, false>(A, mk, mv, num_sms, st);
}

}  // namespace dsa
