// Grouped-query attention over the paged 8-bit cache for few query rows per key head:
// decode and verification over whole contexts, and listed blocks (the definitions are at
// dsa_gqa_attend and dsa_gqa_attend_blocks in include/dsa.h).
//
// A block (64 keys and values of one head, 2 * 64 * D bytes) is the unit of work; the time
// goes into bringing units from HBM (D = 128: 16 KB, which the tensor cores multiply with
// up to 64 query rows in less time than the SM's share of the bandwidth needs to load it).
// So the units of all (request, key head, row tile) items are laid end to end and cut into
// equal runs, one per block of threads (two of those per SM); an item that crosses a cut
// leaves partial results that a second kernel merges. A producer warp brings units through
// a ring of TMA stages; four warps compute straight from the codes:
//
//   * 16 keys x 8 query rows per step on mma.sync m16n8k16 (f16, fp32 sums), the keys (and
//     the values' columns) as the 16 rows of A, so that a group of up to 8 heads wastes
//     nothing. tcgen05 would take its operands from shared memory or TMEM, i.e. a write and
//     a second read of every key and value converted to 16 bits; here the codes go from
//     shared memory to registers once, are converted there, and are fragments already. The
//     order of the summation index is free, so a lane's fragments are D/4 consecutive bytes
//     of a key, and a value pair's halves are put side by side by one byte permute.
//   * both 8-bit types are exact in f16. Queries are scaled by a power of two per row (so
//     that bf16's range fits f16) and are exact to 2^-38 of the row's largest value.
//   * the block's key scale multiplies the scores. Its value scale enters the exponent: with
//     M the running maximum of z + log2(v_scale), the weights p = 2^(z - M + log2(v_scale))
//     are at most 1, multiply the codes directly, and the softmax's sum is of p / v_scale.
//     p is rounded to f16 for the product (2^-11 of it), the sum and all else is fp32.
//
// A lane whose row does not see a key sets p = 0; values that no row of the tile sees are
// zeroed, and where some rows see an e4m3 NaN value that others do not, the product is made
// token by token (0 * NaN would reach the others).
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kConsumers = 4;               // computing warps; one more brings the units
constexpr int kThreads = 32 * (kConsumers + 1);


__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The A fragments of a slice's values, 16 columns at a time: take(tile, a0, a1, a2, a3).
template <int D, bool I8, typename F>
__device__ __forceinline__ void value_tiles(const uint32_t (&v)[4][D / 32], F take) {
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t sel = e ? 0x7362u : 0x5140u;
      uint32_t a0, a1, a2, a3;
      codes_f16<I8>(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
      codes_f16<I8>(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
      take(2 * w + e, a0, a1, a2, a3);
    }
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

// A warp has NT tiles of 8 query rows; MT warps share a unit's keys, each with rows of its own.
template <int D, int NT, int MT>
struct Shape {
  static constexpr int kRows = 8 * NT * MT;
  static constexpr int kTile = kPage * D;                        // bytes of a unit's keys (and of its values)
  static constexpr int kAcc = NT * D / 4;                        // fp32 sums per lane
  static constexpr int kGroups = kConsumers / MT;                // warps that share a row tile, each with its keys
  static constexpr int kMergeBufs = (kGroups - 1) * MT;
  static constexpr int kMergeFloats = (kAcc + 4 * NT) * 32;
  static constexpr int kCtas = NT == 1 ? 3 : 2;                  // per SM
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr size_t kSmem = (size_t)kStages * 2 * kTile + (size_t)kMergeBufs * kMergeFloats * 4 + 1024;
};

template <int D, bool I8, int NT, int MT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT, MT>::kCtas)
    gqa_rows_kernel(const GqaAttendArgs A, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const GqaParts parts) {
  using S = Shape<D, NT, MT>;
  constexpr int kRows = S::kRows, kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[kStages], s_empty[kStages], s_meet;
  __shared__ Unit s_unit[kStages];
  __shared__ int64_t s_begin, s_end, s_base, s_total;
  __shared__ int s_req, s_grid, s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* merge = reinterpret_cast<float*>(smem + kStages * 2 * S::kTile);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool listed = A.blocks != nullptr;
  griddep_launch_dependents();

  if (tid == 32) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), kConsumers);
    }
    s_abort = 0;
    mbar_init(smem_u32(&s_meet), kConsumers);
    fence_mbar_init();
    parts.cuts[blockIdx.x].follow = 0;
  }
  // This block's run [s_begin, s_end) of all units. Whole contexts: the request it starts in
  // and where that request's units begin.
  if (warp == 0) {
    int64_t total = 0;
    if (listed) {
      total = (int64_t)A.g.T * A.c.Hkv * A.n_sel;
    } else {
      for (int b0 = 0; b0 < A.g.B; b0 += 32) {
        int64_t w = 0;
        if (b0 + lane < A.g.B) {
          const Request r = request_of(A, b0 + lane, kRows);
          w = (int64_t)A.c.Hkv * r.tiles * r.units;
          if (r.bad && blockIdx.x == 0) record_error(A.err, kDevBadIndex);
        }
        total += w;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    const int grid = (int)min((int64_t)gridDim.x, total);
    int64_t begin = 0, end = 0;
    if ((int)blockIdx.x < grid) {
      begin = split_begin(blockIdx.x, total, grid);
      end = split_begin(blockIdx.x + 1, total, grid);
    }
    int req = 0;
    int64_t base = 0;
    if (!listed && begin < end) {
      for (int b0 = 0; b0 < A.g.B; b0 += 32) {
        int64_t w = 0;
        if (b0 + lane < A.g.B) {
          const Request r = request_of(A, b0 + lane, kRows);
          w = (int64_t)A.c.Hkv * r.tiles * r.units;
        }
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
  if (begin >= end) return;
  volatile int* abort = &s_abort;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0;
    int64_t u = begin, base = s_base;
    int b = s_req;
    Request r{};
    if (!listed) r = request_of(A, b, kRows);
    const int grid = s_grid;
    const int64_t total = s_total;
    bool ok = true;
    while (u < end && ok) {
      // up to 32 units at a time, one per lane
      int cnt;
      int64_t item_begin = 0, item_end = 0;      // of the lane's unit
      int c = 0, bb = b;
      bool sees = false;
      Unit x{};
      if (!listed) {
        const int64_t mine = (int64_t)A.c.Hkv * r.tiles * r.units;
        if (u >= base + mine) {                  // next request with tokens
          base += mine;
          r = request_of(A, ++b, kRows);
          continue;
        }
        cnt = (int)min((int64_t)32, min(end, base + mine) - u);
        if (lane < cnt) {
          const int64_t o = u + lane - base;
          const int64_t item = o / r.units;
          c = (int)(o - item * r.units);
          item_begin = base + item * r.units;
          item_end = item_begin + r.units;
          x.h = (int)(item / r.tiles);
          x.row0 = (int)(item % r.tiles) * kRows;
          x.q0 = r.q0;
          x.n = r.n;
          x.rel = r.len - r.n - c * kPage;
          // the tile's last token
          const int last = min(r.n - 1, (x.row0 + kRows - 1) / A.G);
          sees = c * kPage < r.len && x.rel + last >= 0;
        }
      } else {
        cnt = (int)min((int64_t)32, end - u);
        if (lane < cnt) {
          const int64_t item = (u + lane) / A.n_sel;
          const int i = (int)(u + lane - item * A.n_sel);
          item_begin = item * A.n_sel;
          item_end = item_begin + A.n_sel;
          const int t = (int)(item / A.c.Hkv);
          x.h = (int)(item % A.c.Hkv);
          x.q0 = t;
          const bool real = t < __ldg(A.g.cu_q + A.g.B);
          x.n = real ? 1 : 0;                    // no rows: a padding token's outputs stay
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
      int tile = 0;
      if (lane < cnt) {
        if (sees) {
          const int page = gqa_page(A.g, bb, c);
          if (page < 0) {
            record_error(A.err, kDevBadIndex);
            sees = false;
          } else {
            tile = page * A.c.Hkv + x.h;
            const float vs = __ldg(A.c.v_scale + tile);
            x.kf = __ldg(A.c.k_scale + tile) * A.scale_log2;
            x.lv = log2f(vs);
            x.ivs = 1.f / vs;
          }
        }
        const int64_t at = u + lane;
        const bool first = at == item_begin || at == begin, last = at + 1 == item_end || at + 1 == end;
        x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (sees ? 0 : kVoid);
        const bool cut = item_begin < begin || item_end > end;
        x.slot = !cut ? -1 : 2 * (int)blockIdx.x + (max(item_begin, begin) == begin ? 0 : 1);
        if (last && cut && item_begin >= begin) {   // this block merges the item
          Cut k{};
          k.follow = (int)split_owner(item_end - 1, total, grid) - (int)blockIdx.x;
          k.slot = x.slot;
          k.q0 = x.q0, k.n = x.n, k.row0 = x.row0, k.h = x.h;
          parts.cuts[blockIdx.x] = k;
        }
      }
      for (int i = 0; i < cnt; ++i) {
        ok = warp_wait(&s_empty[stage], phase ^ 1u, abort, A.err);
        if (!ok) break;
        if (lane == i) {
          s_unit[stage] = x;
          const uint32_t bar = smem_u32(&s_full[stage]);
          if (sees) {
            const uint32_t dst = smem_u32(smem + stage * 2 * S::kTile);
            mbar_arrive_expect_tx(bar, 2 * S::kTile);
            tma_load_3d(dst, &map_k, bar, 0, 0, tile);
            tma_load_3d(dst + S::kTile, &map_v, bar, 0, 0, tile);
          } else {
            mbar_arrive(bar);
          }
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
      u += cnt;
    }
    if (!ok) {
      // Gave up: copies still in flight must land before the shared memory is given back
      // (each stage's last phase; one that was never filled counts as complete).
      if (lane == 0) {
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < kStages; ++i) {
          const uint32_t par = i < stage ? phase : phase ^ 1u;
          while (!mbar_test_wait(smem_u32(&s_full[i]), par) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- computing warps
  constexpr int kSteps = D / 16;                 // k16 steps of a score = words of a lane's D/4 key bytes
  constexpr int kTiles = D / 16;                 // 16-column tiles of the output
  constexpr int kVw = D / 32;                    // words of a lane's D/8 bytes of a value
  const int m = warp % MT, group = warp / MT;
  const int q = lane & 3, lrow = lane >> 2;
  const int G = A.G, H = A.G * A.c.Hkv;
  uint32_t qf[NT][kSteps][2];
  float o[NT][kTiles][4];                        // [.][j]: columns lrow*D/8 + 2j (0, 1) and + 1 (2, 3) of rows 2q, 2q+1
  float M[NT][2], l[NT][2], rowf[NT][2];         // of rows 8i + 2q and + 1
  int tok[NT][2];                                // their tokens, or far below any limit
  int tok_lo = 0, tok_hi = 0;                    // of the warp's rows (tok_hi < 0: none)
  int stage = 0;
  uint32_t phase = 0, met = 0;
  // All computing warps meet here (a bounded wait: a warp that gave up does not come).
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s_meet));
    const bool all = warp_wait(&s_meet, met, abort, A.err);
    met ^= 1u;
    return all;
  };

  for (int64_t u = begin; u < end; ++u) {
    if (!warp_wait(&s_full[stage], phase, abort, A.err)) break;
    const Unit x = s_unit[stage];
    if (x.flags & kFirst) {
      const int r0 = x.row0 + m * 8 * NT, rows = x.n * G;
      tok_lo = r0 / G;
      tok_hi = r0 < rows ? min(x.n - 1, (r0 + 8 * NT - 1) / G) : -1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = r0 + 8 * i + lrow;
        const bool valid = row < rows;
        const int t = valid ? row / G : 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            A.q + (int64_t)(x.q0 + t) * A.q_stride + (int64_t)(x.h * G + (valid ? row - t * G : 0)) * D + q * (D / 4));
        uint32_t w[D / 8];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint4 v = valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
        }
        float big = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) big = fmaxf(big, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // the row times 2^(14 - e), e the exponent of its largest value (none for infinities)
        const int e = min(max((int)(__float_as_uint(big) >> 23), 15), 254);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) qf[i][k >> 1][k & 1] = pack_f16(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int mine = r0 + 8 * i + 2 * q + h;
          rowf[i][h] = __shfl_sync(0xffffffffu, down, 4 * (2 * q + h));
          tok[i][h] = mine < rows ? mine / G : -(1 << 30);
          M[i][h] = kNone;
          l[i][h] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
      }
    }
    const uint32_t kt = smem_u32(smem + stage * 2 * S::kTile), vt = kt + S::kTile;
    const int seen = (x.flags & kVoid) ? -1 : min(x.rel + tok_hi, kPage - 1);   // last key any row of the warp sees
    const bool whole = x.rel + tok_lo >= kPage - 1;                             // every row sees every key
#pragma unroll 1
    for (int sub = 0; sub < MT; ++sub) {
      const int ts = (group * MT + sub) * 16;
      if (tok_hi < 0 || ts > seen) break;
      // ---- scores: s[i][0..3] are key lrow (0, 1) and lrow + 8 (2, 3) with rows 2q, 2q+1
      float s[NT][4] = {};
      {
        uint32_t kw[2][kSteps];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t row = kt + (ts + 8 * j + lrow) * D;
          if constexpr (D == 128) {
            const uint4 a = lds128(row + (((2 * q) ^ lrow) << 4)), b = lds128(row + (((2 * q + 1) ^ lrow) << 4));
            kw[j][0] = a.x, kw[j][1] = a.y, kw[j][2] = a.z, kw[j][3] = a.w;
            kw[j][4] = b.x, kw[j][5] = b.y, kw[j][6] = b.z, kw[j][7] = b.w;
          } else {
            const uint4 a = lds128(row + ((q ^ ((lrow >> 1) & 3)) << 4));
            kw[j][0] = a.x, kw[j][1] = a.y, kw[j][2] = a.z, kw[j][3] = a.w;
          }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a0, a1, a2, a3;
          codes_f16<I8>(kw[0][k], a0, a2);
          codes_f16<I8>(kw[1][k], a1, a3);
#pragma unroll
          for (int i = 0; i < NT; ++i) mma16816(s[i], a0, a1, a2, a3, qf[i][k][0], qf[i][k][1]);
        }
      }
      // ---- values (read early: their latency passes under the softmax). vw[k]: token
      // 2q + (k & 1) + 8 * (k >> 1) of the slice, D/8 bytes from column (D/8) * lrow
      uint32_t vw[4][kVw];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tk = ts + 2 * q + (k & 1) + 8 * (k >> 1);
        if constexpr (D == 128) {
          const uint4 a = lds128(vt + tk * D + ((lrow ^ (tk & 7)) << 4));
          vw[k][0] = a.x, vw[k][1] = a.y, vw[k][2] = a.z, vw[k][3] = a.w;
        } else {
          const uint2 a = lds64(vt + tk * D + (((lrow >> 1) ^ ((tk >> 1) & 3)) << 4) + (lrow & 1) * 8);
          vw[k][0] = a.x, vw[k][1] = a.y;
        }
      }
      // ---- softmax
      bool grew = false;
      float keep[NT][2];
      uint32_t pb[NT][2];                         // weights, f16: rows by lane group, keys 2q, 2q+1 (0) and + 8 (1)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = x.kf * rowf[i][h];
          float z0 = s[i][h] * f, z1 = s[i][2 + h] * f;
          if (!whole) {
            const int lim = x.rel + tok[i][h] - ts;
            if (lrow > lim) z0 = -INFINITY;
            if (lrow + 8 > lim) z1 = -INFINITY;
          }
          float mx = fmaxf(z0, z1);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float Mn = fmaxf(M[i][h], mx + x.lv);
          grew |= Mn > M[i][h];
          keep[i][h] = ex2(M[i][h] - Mn);
          M[i][h] = Mn;
          const float ref = Mn - x.lv;
          z0 = ex2(z0 - ref);
          z1 = ex2(z1 - ref);
          l[i][h] = l[i][h] * keep[i][h] + (z0 + z1) * x.ivs;
          s[i][h] = z0, s[i][2 + h] = z1;
        }
        pb[i][0] = transpose8(pack_f16(s[i][0], s[i][1]));
        pb[i][1] = transpose8(pack_f16(s[i][2], s[i][3]));
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
            o[i][j][0] *= keep[i][0], o[i][j][1] *= keep[i][1], o[i][j][2] *= keep[i][0], o[i][j][3] *= keep[i][1];
      }
      // ---- values times weights
      bool apart = false;                         // a NaN value that only some rows may meet
      if (!whole) {
        bool nan = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool out = ts + 2 * q + (k & 1) + 8 * (k >> 1) > seen;
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
          for (int i = 0; i < NT; ++i) mma16816(o[i][j], a0, a1, a2, a3, pb[i][0], pb[i][1]);
        });
      } else {
        for (int t = tok_lo; t <= tok_hi; ++t) {
          uint32_t v[4][kVw];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < kVw; ++w)
              v[k][w] = ts + 2 * q + (k & 1) + 8 * (k >> 1) > x.rel + t ? 0u : vw[k][w];
          value_tiles<D, I8>(v, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float c[4] = {o[i][j][0], o[i][j][1], o[i][j][2], o[i][j][3]};
              mma16816(c, a0, a1, a2, a3, pb[i][0], pb[i][1]);
              if (tok[i][0] == t) o[i][j][0] = c[0], o[i][j][2] = c[2];
              if (tok[i][1] == t) o[i][j][1] = c[1], o[i][j][3] = c[3];
            }
          });
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s_empty[stage]));
    if (++stage == kStages) stage = 0, phase ^= 1u;
    if (!(x.flags & kLast)) continue;

    // ---- end of the run's part of the item: the sums of the warps that shared its rows
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 4);
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 8);
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 16);
      }
    if (S::kGroups > 1) {
      if (!meet()) break;                         // the last merge has been read
      if (group > 0) {
        float* buf = merge + ((group - 1) * MT + m) * S::kMergeFloats + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int j = 0; j < 4 * kTiles; ++j) buf[(i * 4 * kTiles + j) * 32] = o[i][j >> 2][j & 3];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            buf[(S::kAcc + 4 * i + h) * 32] = M[i][h];
            buf[(S::kAcc + 4 * i + 2 + h) * 32] = l[i][h];
          }
        }
      }
      if (!meet()) break;
      if (group > 0) continue;
#pragma unroll 1
      for (int gr = 1; gr < S::kGroups; ++gr) {
        const float* buf = merge + ((gr - 1) * MT + m) * S::kMergeFloats + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float mine[2], other[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float Mo = buf[(S::kAcc + 4 * i + h) * 32], Mn = fmaxf(M[i][h], Mo);
            mine[h] = ex2(M[i][h] - Mn);
            other[h] = ex2(Mo - Mn);
            l[i][h] = l[i][h] * mine[h] + buf[(S::kAcc + 4 * i + 2 + h) * 32] * other[h];
            M[i][h] = Mn;
          }
#pragma unroll
          for (int j = 0; j < 4 * kTiles; ++j)
            o[i][j >> 2][j & 3] = o[i][j >> 2][j & 3] * mine[j & 1] + buf[(i * 4 * kTiles + j) * 32] * other[j & 1];
        }
      }
    }
    // a lane holds columns lrow*D/8 .. of its rows
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tok[i][h] < 0) continue;
        const int r = m * 8 * NT + 8 * i + 2 * q + h;                 // row of the item's tile
        auto col = [&](int d) { return o[i][d >> 1][2 * (d & 1) + h]; };
        if (x.slot < 0) {
          const float inv = l[i][h] == 0.f ? 0.f : 1.f / l[i][h];
          const int64_t at = (int64_t)(x.q0 + tok[i][h]) * H + x.h * G + (x.row0 + r - tok[i][h] * G);
          uint4* dst = reinterpret_cast<uint4*>(A.out + at * D + lrow * (D / 8));
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
          if (A.lse && lrow == 0) A.lse[at] = l[i][h] == 0.f ? -INFINITY : (M[i][h] + log2f(l[i][h])) * 0.6931471805599453f;
        } else {
          const int64_t at = (int64_t)x.slot * kRows + r;
          float4* dst = reinterpret_cast<float4*>(parts.o + at * D + lrow * (D / 8));
#pragma unroll
          for (int d = 0; d < D / 8; d += 4) dst[d / 4] = make_float4(col(d), col(d + 1), col(d + 2), col(d + 3));
          if (lrow == 0) *reinterpret_cast<float2*>(parts.ml + at * 2) = make_float2(M[i][h], l[i][h]);
        }
      }
  }
}

// Merges the parts of items that were cut, in the order of the blocks of threads: block c
// (x) looks whether it holds an item's first part; eight rows per block (y), a warp each,
// or all warps on one row after another where an item has many parts.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    gqa_merge_kernel(const GqaAttendArgs A, const GqaParts s) {
  constexpr int V = D / 32;
  __shared__ float s_o[kMergeWarps][D];
  __shared__ float s_ml[kMergeWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const Cut k = s.cuts[blockIdx.x];
  if (k.follow <= 0) return;
  const int rows = s.rows, parts = k.follow + 1, H = A.G * A.c.Hkv;
  const bool many = parts > 2 * kMergeWarps;
  const int first = many ? warp : 0, step = many ? kMergeWarps : 1;
  for (int i = many ? 0 : warp; i < kMergeWarps; i += many ? 1 : kMergeWarps) {
    const int r = blockIdx.y * kMergeWarps + i, row = k.row0 + r;
    if (row >= k.n * A.G) break;
    float M = kNone, l = 0.f, o[V] = {};
    for (int p = first; p < parts; p += step) {
      const int64_t slot = p == 0 ? k.slot : 2 * (int64_t)(blockIdx.x + p);
      const int64_t at = slot * rows + r;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(s.ml + at * 2));
      float v[V];
      if constexpr (V == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(s.o + at * D) + lane);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(s.o + at * D) + lane);
        v[0] = f.x, v[1] = f.y;
      }
      const float Mn = fmaxf(M, ml.x), a = ex2(M - Mn), b = ex2(ml.x - Mn);
      M = Mn;
      l = l * a + ml.y * b;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = o[j] * a + v[j] * b;
    }
    if (many) {
#pragma unroll
      for (int j = 0; j < V; ++j) s_o[warp][lane * V + j] = o[j];
      if (lane == 0) s_ml[warp][0] = M, s_ml[warp][1] = l;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < kMergeWarps; ++w) {
          const float Mn = fmaxf(M, s_ml[w][0]), a = ex2(M - Mn), b = ex2(s_ml[w][0] - Mn);
          M = Mn;
          l = l * a + s_ml[w][1] * b;
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = o[j] * a + s_o[w][lane * V + j] * b;
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int t = row / A.G;
    const int64_t at = (int64_t)(k.q0 + t) * H + k.h * A.G + (row - t * A.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat162 w[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) w[j] = __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
    if constexpr (V == 4) *(reinterpret_cast<uint2*>(A.out + at * D) + lane) = *reinterpret_cast<uint2*>(w);
    else *(reinterpret_cast<uint32_t*>(A.out + at * D) + lane) = *reinterpret_cast<uint32_t*>(w);
    if (A.lse && lane == 0) A.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
  }
}

// Query rows (tokens x heads of a key head) that meet a unit together. Up to 16 rows: every
// warp has them all and a quarter of the keys. More: a unit's codes are converted by two or
// four warps, each for 16 of the rows. Above 64: gqa_tiles.cu.
int rows_per_item(int T, int B, int G, bool listed) {
  const int64_t rows = listed ? G : ((int64_t)T + B - 1) / B * G;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : kGqaTileRows;
}

int rows_grid(int rows, int num_sms) { return (rows == 8 ? Shape<128, 1, 1>::kCtas : Shape<128, 2, 1>::kCtas) * num_sms; }

template <int D, bool I8, int NT, int MT>
cudaError_t launch(const GqaAttendArgs& A, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms, cudaStream_t st) {
  using S = Shape<D, NT, MT>;
  constexpr int rows = S::kRows;
  const int grid = rows_grid(rows, num_sms);
  const GqaParts s = gqa_parts(A.scratch, grid, rows);
  auto kern = gqa_rows_kernel<D, I8, NT, MT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, S::kSmem, st>>>(A, mk, mv, s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return gqa_merge_launch(A, s, grid, st);
}

template <int D, bool I8>
cudaError_t launch_rows(const GqaAttendArgs& A, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms, cudaStream_t st) {
  switch (rows_per_item(A.g.T, A.g.B, A.G, A.blocks != nullptr)) {
    case 8: return launch<D, I8, 1, 1>(A, mk, mv, num_sms, st);
    case 16: return launch<D, I8, 2, 1>(A, mk, mv, num_sms, st);
    case 32: return launch<D, I8, 2, 2>(A, mk, mv, num_sms, st);
    default: return launch<D, I8, 2, 4>(A, mk, mv, num_sms, st);
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

size_t gqa_attend_scratch_bytes(const dsa_geom_t* g, int, int D, int G, int n_sel, int num_sms) {
  const int rows = rows_per_item(g->T, g->B, G, n_sel > 0);
  return rows > 64 ? gqa_parts_bytes(num_sms, kGqaTileRows, D) : gqa_parts_bytes(rows_grid(rows, num_sms), rows, D);
}

cudaError_t gqa_attend_launch(const GqaAttendArgs& A, int num_sms, cudaStream_t st) {
  if (rows_per_item(A.g.T, A.g.B, A.G, A.blocks != nullptr) > 64) return gqa_tiles_launch(A, num_sms, st);
  CUtensorMap mk, mv;
  const uint64_t tiles = (uint64_t)A.g.num_pages * A.c.Hkv;
  if (!encode_code_tiles(&mk, A.c.k, A.c.D, tiles) || !encode_code_tiles(&mv, A.c.v, A.c.D, tiles))
    return cudaErrorInvalidValue;
  if (A.c.D == 128) return A.c.i8 ? launch_rows<128, true>(A, mk, mv, num_sms, st) : launch_rows<128, false>(A, mk, mv, num_sms, st);
  return A.c.i8 ? launch_rows<64, true>(A, mk, mv, num_sms, st) : launch_rows<64, false>(A, mk, mv, num_sms, st);
}

}  // namespace dsa
