// Block selection: scores of the blocks' int8 key means against the pooled, int8-coded
// query of each (token, key head), and the n_sel best blocks (the definition is at
// dsa_block_select in include/dsa.h).
//
// The dot products are whole numbers below 2^21 (dp4a), so a score is one fp32 product of
// exact factors and the selection is the same for every split of the work. A block of
// threads keeps the scores' order-preserving keys of its tokens in shared memory and
// selects there by radix (8 bits a pass), then lists the taken blocks in ascending order
// with ballots; nothing but the lists goes back to memory.
//
// Two shapes. One token per block of threads (decode): every warp scores on dp4a, all of them
// select by radix. Tiles of 16 or 8 consecutive tokens (prompts): a block's mean, converted to
// f16 once, meets the tile's tokens of the same request on the tensor cores (the codes' products
// and sums are whole numbers that f16 operands and fp32 sums hold exactly), and each warp selects
// for one or two tokens, by bisection between its largest and smallest score where a lane can
// hold its share of the scores in registers.
//
// 8 tokens over 131072 each (17 MB of means) take 10.2 us in a graph: a chain of lookups, four
// radix passes and their barriers. 2048 tokens over 16384 (36 MB, nearly all of it the queries)
// take 39: issue, 17 for lookups and pooled queries, 4 for scores, 4 for keys, 13 for choosing.
// One token per block of threads took 55 there. (32 tokens a tile spill registers: 42.)
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kTileWarps = 16;   // warps in the tile shape
constexpr int kOneWarps = 32;    // warps in the one-token shape
constexpr int kHeld = 16;        // scores that a lane can hold in registers: rows of up to 512 blocks

// The n_sel largest of nv keys (n_sel < nv), ties to the lower index, ascending into out.
// NW warps take part; scr: 256 + 2 * NW + 4 ints.
template <int NW>
__device__ __forceinline__ void choose(const uint32_t* keys, int nv, int n_sel, int* out, int* scr, int warp, int lane) {
  auto sync = [] {
    if (NW == 1) __syncwarp();
    else __syncthreads();
  };
  int* hist = scr;
  int* found = scr + 256;
  int* counts = found + 4;
  uint32_t prefix = 0, mask = 0;
  int need = n_sel;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = warp * 32 + lane; i < 256; i += NW * 32) hist[i] = 0;
    sync();
    for (int i = warp * 32 + lane; i < nv; i += NW * 32) {
      const uint32_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(hist + ((k >> shift) & 255u), 1);
    }
    sync();
    if (warp == 0) {   // bins from the top, eight a lane
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - 8 * lane - i];
        sum += c[i];
      }
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      int before = upto - sum;
      if (before < need && upto >= need) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + c[i] >= need) {
            found[0] = 255 - 8 * lane - i;
            found[1] = need - before;
            found[2] = c[i];
          }
          before += c[i];
        }
      }
    }
    sync();
    prefix |= (uint32_t)found[0] << shift;
    mask |= 255u << shift;
    need = found[1];
    if (found[2] == need) break;   // the whole bin is taken
  }
  // the warp's run of blocks: those above the bin, and the bin's first `need`
  const int per = (nv + 32 * NW - 1) / (32 * NW) * 32;
  const int s0 = min(nv, warp * per), s1 = min(nv, s0 + per);
  int above = 0, equal = 0;
  if (NW > 1) {
    for (int i = s0 + lane; i < s1; i += 32) {
      const uint32_t k = keys[i] & mask;
      above += k > prefix;
      equal += k == prefix;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) counts[2 * warp] = above, counts[2 * warp + 1] = equal;
    sync();
    above = equal = 0;
    for (int w = 0; w < warp; ++w) above += counts[2 * w], equal += counts[2 * w + 1];
  }
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < s1 ? keys[i] & mask : 0u;
    const bool a = i < s1 && k > prefix, e = i < s1 && k == prefix;
    const unsigned ma = __ballot_sync(0xffffffffu, a), me = __ballot_sync(0xffffffffu, e);
    const unsigned below = (1u << lane) - 1u;
    const int eq = equal + __popc(me & below);
    if (a || (e && eq < need)) out[above + __popc(ma & below) + min(eq, need)] = i;
    above += __popc(ma);
    equal += __popc(me);
  }
}

// The query token's pooled int8 code of key head kvh (D bytes at dst), by one warp; the first
// eight heads' loads are issued at construction, to pass under other lookups.
template <int D>
struct PooledQuery {
  static constexpr int V = D / 32;
  const __nv_bfloat16* row;
  uint32_t w[8][V / 2];
  __device__ __forceinline__ void load(int G, int h0) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      if (h0 + h >= G) continue;
      if constexpr (V == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + (h0 + h) * D));
        w[h][0] = v.x, w[h][1] = v.y;
      } else {
        w[h][0] = __ldg(reinterpret_cast<const uint32_t*>(row + (h0 + h) * D));
      }
    }
  }
  __device__ __forceinline__ PooledQuery(const GqaSelectArgs& A, int t, int kvh, int lane)
      : row(A.q + (int64_t)t * A.q_stride + (int64_t)kvh * A.G * D + lane * V) {
    load(A.G, 0);
  }
  __device__ __forceinline__ void finish(int G, uint8_t* dst, int lane) {
    float x[V] = {};
    for (int h0 = 0; h0 < G; h0 += 8) {
      if (h0) load(G, h0);
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        if (h0 + h >= G) continue;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          x[2 * j] = h0 + h ? __fadd_rn(x[2 * j], bf16_lo(w[h][j])) : bf16_lo(w[h][j]);
          x[2 * j + 1] = h0 + h ? __fadd_rn(x[2 * j + 1], bf16_hi(w[h][j])) : bf16_hi(w[h][j]);
        }
      }
    }
    float u = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) u = fmaxf(u, fabsf(x[j]));
    u = __fdiv_rn(warp_max(u), 127.f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = u > 0.f ? max(-127, min(127, __float2int_rn(__fdiv_rn(x[j], u)))) : 0;
      dst[lane * V + j] = (uint8_t)(c & 0xFF);
    }
  }
};

// The key that block c of nv is ranked by.
__device__ __forceinline__ uint32_t score_key(const GqaSelectArgs& A, float s, int c, int nv, int page) {
  if (c < A.n_first || c >= nv - A.n_last) return 0xFFFFFFFFu;
  return page < 0 ? 0u : s == s ? max(orderable_key(s), 2u) : 1u;
}

// Keys of 32 blocks c0..c0+31, by the whole warp; page: the lane's block's, or -1.
template <int D>
__device__ __forceinline__ void score_blocks(const GqaSelectArgs& A, int kvh, int c0, int nv, int page,
                                             const uint8_t* codes, uint32_t* keys, int lane) {
  constexpr int kLpb = D / 16;                   // lanes to a block's mean, 16 bytes each
  const int sub = lane % kLpb, grp = lane / kLpb;
  const int c = c0 + lane;
  if (c < nv && page < 0) record_error(A.err, kDevBadIndex);
  const float scale = page >= 0 ? __ldg(A.c.k_mean_scale + (int64_t)page * A.c.Hkv + kvh) : 0.f;
  int v[kLpb];
  const uint4 q = *reinterpret_cast<const uint4*>(codes + sub * 16);
  uint4 mean[kLpb];
#pragma unroll
  for (int j = 0; j < kLpb; ++j) {
    const int p = __shfl_sync(0xffffffffu, page, grp * kLpb + j);
    mean[j] = p >= 0 ? __ldg(reinterpret_cast<const uint4*>(A.c.k_mean + ((int64_t)p * A.c.Hkv + kvh) * D) + sub)
                     : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < kLpb; ++j) {
    v[j] = __dp4a((int)mean[j].x, (int)q.x, 0);
    v[j] = __dp4a((int)mean[j].y, (int)q.y, v[j]);
    v[j] = __dp4a((int)mean[j].z, (int)q.z, v[j]);
    v[j] = __dp4a((int)mean[j].w, (int)q.w, v[j]);
  }
  // sums over the lanes of a block, lane `sub` keeping the group's block `sub`
#pragma unroll
  for (int o = kLpb / 2; o > 0; o >>= 1) {
    const bool up = (sub & o) != 0;
#pragma unroll
    for (int j = 0; j < kLpb / 2; ++j) {
      if (j < o) {
        const int keep = up ? v[j + o] : v[j], send = up ? v[j] : v[j + o];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
  }
  if (c < nv) keys[c] = score_key(A, __fmul_rn((float)v[0], scale), c, nv, page);
}

// The same choice by one warp, for nv <= 32 * kHeld: the keys of the lane's blocks lane, lane +
// 32, ... in registers, the smallest key taken found by bisection. kForced keys are all taken.
constexpr uint32_t kForced = 0xFFFFFFFFu;

__device__ __forceinline__ float key_value(uint32_t k) {   // inverse of orderable_key
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
template <int kHeld>
__device__ __forceinline__ void choose_held(const uint32_t* keys, int nv, int n_sel, int* out, int lane) {
  uint32_t k[kHeld];
  uint32_t top = 0, low = kForced;
  int forced = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = lane + 32 * i;
    k[i] = c < nv ? keys[c] : 0u;                 // (a key of 0, a bad page's, ranks with what is not there: see below)
    if (k[i] == kForced) ++forced;
    else if (c < nv) top = max(top, k[i]), low = min(low, k[i]);
  }
  forced = __reduce_add_sync(0xffffffffu, forced);
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  // at least n_sel keys are >= lo, fewer than n_sel are >= hi; more: those >= hi
  uint32_t lo = low, hi = top + 1u;
  int more = forced;
  bool exact = more == n_sel;
  if (exact) lo = hi;
  float flo = key_value(lo), fhi = key_value(top);
  bool by_value = true;                           // halve the scores' range, later the keys'
  while (!exact && hi - lo > 1u) {
    uint32_t mid = lo + (hi - lo) / 2u;
    if (by_value) {
      const float fm = 0.5f * flo + 0.5f * fhi;
      const uint32_t m = orderable_key(fm);
      by_value = m > lo && m < hi;                // (also false for what is no number)
      if (by_value) mid = m;
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) n += k[i] >= mid;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= n_sel) {
      lo = mid, flo = key_value(mid);
      exact = n == n_sel;
    } else {
      hi = mid, fhi = key_value(mid);
      more = n;
    }
  }
  const unsigned below = (1u << lane) - 1u;
  if (exact) {                                    // the keys from lo on (the usual end)
    int n = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (32 * i >= nv) break;
      const bool in = lane + 32 * i < nv && k[i] >= lo;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (in) out[n + __popc(m & below)] = lane + 32 * i;
      n += __popc(m);
    }
    return;
  }
  // keys above lo, and the first of those equal to it
  const int need = n_sel - more;
  int above = 0, equal = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (32 * i >= nv) break;
    const bool there = lane + 32 * i < nv;
    const bool a = there && k[i] > lo, e = there && k[i] == lo;
    const unsigned ma = __ballot_sync(0xffffffffu, a), me = __ballot_sync(0xffffffffu, e);
    const int eq = equal + __popc(me & below);
    if (a || (e && eq < need)) out[above + __popc(ma & below) + min(eq, need)] = lane + 32 * i;
    above += __popc(ma);
    equal += __popc(me);
  }
}

// A token's list where nothing has to be chosen: all of its nv <= n_sel blocks. (Their pages are
// looked up only to report bad ones, as where blocks are scored.)
__device__ __forceinline__ void list_all(const GqaSelectArgs& A, int* out, int b, int nv, int at, int step) {
  for (int i = at; i < A.n_sel; i += step) out[i] = i < nv ? i : -1;
  for (int i = at; i < nv; i += step)
    if (gqa_page(A.g, b, i) < 0) record_error(A.err, kDevBadIndex);
}

// One token.
template <int D>
__global__ void __launch_bounds__(32 * kOneWarps) gqa_select_one_kernel(const GqaSelectArgs A) {
  extern __shared__ __align__(16) uint8_t select_smem[];
  __shared__ __align__(16) uint8_t s_codes[D];
  __shared__ int s_scr[256 + 4 + 2 * kOneWarps];
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, kvh = blockIdx.y;
  const int64_t at = ((int64_t)kvh * gridDim.x + t) * (32 * kOneWarps) + threadIdx.x;
  RequestCheck check(A.g, at);
  if (warp == kOneWarps - 1) {                    // (meanwhile the others look the token up)
    PooledQuery<D> pooled(A, t, kvh, lane);
    pooled.finish(A.G, s_codes, lane);
  }
  bool bad;
  const GqaToken k = gqa_token_warp(A.g, t, &bad);
  if (bad && threadIdx.x == 0) record_error(A.err, kDevBadIndex);
  check.report(A.g, at, (int64_t)gridDim.x * gridDim.y * (32 * kOneWarps), A.err);
  if (k.row == kRowPadding) return;
  int* out = A.blocks + ((int64_t)t * A.c.Hkv + kvh) * A.n_sel;
  const int nv = k.row == kRowSees ? (k.pos >> 6) + 1 : 0;
  if (nv <= A.n_sel) {
    list_all(A, out, k.b, nv, threadIdx.x, 32 * kOneWarps);
    return;
  }
  int c0 = warp * 32, page = c0 + lane < nv ? gqa_page(A.g, k.b, c0 + lane) : -1;
  __syncthreads();
  for (; c0 < nv; c0 += kOneWarps * 32) {
    const int next = c0 + kOneWarps * 32 + lane;
    const int after = next < nv ? gqa_page(A.g, k.b, next) : -1;
    score_blocks<D>(A, kvh, c0, nv, page, s_codes, keys, lane);
    page = after;
  }
  __syncthreads();
  choose<kOneWarps>(keys, nv, A.n_sel, out, s_scr, warp, lane);
}

// TQ consecutive tokens (a multiple of 8); stride: words between tokens' keys.
template <int D, int TQ>
__global__ void __launch_bounds__(32 * kTileWarps, 2) gqa_select_tile_kernel(const GqaSelectArgs A, int stride) {
  constexpr int kSteps = D / 16, kNT = TQ / 8;
  extern __shared__ __align__(16) uint8_t select_smem[];
  __shared__ __align__(16) uint8_t s_codes[TQ][D];
  __shared__ uint2 s_qf[kNT][kSteps][32];
  __shared__ int s_nv[TQ], s_b[TQ], s_row[TQ];
  __shared__ int s_scr[TQ][256 + 4 + 2];
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, lrow = lane >> 2;
  const int t0 = blockIdx.x * TQ, kvh = blockIdx.y;
  static_assert(TQ <= kTileWarps, "a warp per token");
  const int64_t at = ((int64_t)kvh * gridDim.x + blockIdx.x) * (32 * kTileWarps) + threadIdx.x;
  RequestCheck check(A.g, at);
  if (warp < TQ) {
    const int t = t0 + warp;
    PooledQuery<D> pooled(A, min(t, A.g.T - 1), kvh, lane);
    GqaToken k{0, -1, kRowPadding};
    bool bad = false;
    if (t < A.g.T) k = gqa_token_warp(A.g, t, &bad);
    if (lane == 0) {
      if (bad) record_error(A.err, kDevBadIndex);
      s_row[warp] = k.row;
      s_b[warp] = k.b;
      s_nv[warp] = k.row == kRowSees ? (k.pos >> 6) + 1 : 0;
    }
    pooled.finish(A.G, s_codes[warp], lane);
  }
  check.report(A.g, at, (int64_t)gridDim.x * gridDim.y * (32 * kTileWarps), A.err);
  __syncthreads();
  // 16 blocks' means and scales of a request, as they are
  struct Means {
    uint4 v[2][D / 64];
    float scale[2];
    int page[2];
  };
  auto means = [&](Means& m, int b, int c0, int most) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + lrow + 8 * h;
      m.page[h] = c < most ? gqa_page(A.g, b, c) : -1;
      if (c < most && m.page[h] < 0) record_error(A.err, kDevBadIndex);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t tile = (int64_t)max(m.page[h], 0) * A.c.Hkv + kvh;
      m.scale[h] = __ldg(A.c.k_mean_scale + tile);
      const uint4* src = reinterpret_cast<const uint4*>(A.c.k_mean + tile * D + q * (D / 4));
#pragma unroll
      for (int k = 0; k < D / 64; ++k) m.v[h][k] = __ldg(src + k);
    }
  };
  // the first run of tokens of one request: its first slice is loaded under what follows
  int w0 = 0, w1, most;
  auto run = [&]() {
    w1 = w0 + 1, most = s_nv[w0];
    while (w1 < TQ && s_b[w1] == s_b[w0]) {
      most = max(most, s_nv[w1]);
      ++w1;
    }
  };
  run();
  Means m;
  if (most > A.n_sel && 16 * warp < most) means(m, s_b[0], 16 * warp, most);
  // the tokens' codes as B fragments: token lrow of each eight, columns q*D/4 ..
  for (int i = warp; i < kNT * kSteps; i += kTileWarps) {
    const int n = i / kSteps, k = i % kSteps;
    uint2 f;
    codes_f16<true>(*reinterpret_cast<const uint32_t*>(&s_codes[8 * n + lrow][q * (D / 4) + 4 * k]), f.x, f.y);
    s_qf[n][k][lane] = f;
  }
  __syncthreads();
  // scores, 16 blocks a warp and step
  for (;;) {
    if (most > A.n_sel) {
      for (int c0 = 16 * warp; c0 < most; c0 += 16 * kTileWarps) {
        if (w0 > 0 || c0 > 16 * warp) means(m, s_b[w0], c0, most);
        uint32_t a[kSteps][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < kSteps; k += 4) {
            const uint4 v = m.v[h][k / 4];
            codes_f16<true>(v.x, a[k][h], a[k][2 + h]);
            codes_f16<true>(v.y, a[k + 1][h], a[k + 1][2 + h]);
            codes_f16<true>(v.z, a[k + 2][h], a[k + 2][2 + h]);
            codes_f16<true>(v.w, a[k + 3][h], a[k + 3][2 + h]);
          }
#pragma unroll
        for (int i = 0; i < kNT; ++i) {
          float s[4] = {};
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const uint2 f = s_qf[i][k][lane];
            mma16816(s, a[k][0], a[k][1], a[k][2], a[k][3], f.x, f.y);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int w = 8 * i + 2 * q + (j & 1), c = c0 + lrow + 8 * (j >> 1);
            if (w < w0 || w >= w1 || c >= s_nv[w]) continue;
            keys[w * stride + c] = score_key(A, __fmul_rn(s[j], m.scale[j >> 1]), c, s_nv[w], m.page[j >> 1]);
          }
        }
      }
    }
    w0 = w1;
    if (w0 >= TQ) break;
    run();
  }
  __syncthreads();
  for (int w = warp; w < TQ; w += kTileWarps) {
    if (s_row[w] == kRowPadding) continue;
    int* out = A.blocks + ((int64_t)(t0 + w) * A.c.Hkv + kvh) * A.n_sel;
    if (s_nv[w] <= A.n_sel) list_all(A, out, s_b[w], s_nv[w], lane, 32);
    else if (s_nv[w] <= 32 * kHeld / 2) choose_held<kHeld / 2>(keys + w * stride, s_nv[w], A.n_sel, out, lane);
    else if (s_nv[w] <= 32 * kHeld) choose_held<kHeld>(keys + w * stride, s_nv[w], A.n_sel, out, lane);
    else choose<1>(keys + w * stride, s_nv[w], A.n_sel, out, s_scr[w], 0, lane);
    __syncwarp();
  }
}

template <int D, int TQ>
cudaError_t launch_tile(const GqaSelectArgs& A, int stride, cudaStream_t st) {
  const size_t bytes = (size_t)stride * 4 * TQ;
  auto kern = gqa_select_tile_kernel<D, TQ>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, 98304, allowed);
  if (e != cudaSuccess) return e;
  kern<<<dim3((A.g.T + TQ - 1) / TQ, A.c.Hkv), 32 * kTileWarps, bytes, st>>>(A, stride);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const GqaSelectArgs& A, int num_sms, cudaStream_t st) {
  const int nb = (A.g.max_seq_len + kPage - 1) / kPage;
  const int stride = (nb + 15) / 16 * 16 + 4;     // (a warp's 8 x 8 keys then fall into 32 banks)
  // Tiles of tokens pay once they alone fill the SMs and their scores fit beside others'.
  const int64_t rows = (int64_t)A.g.T * A.c.Hkv;
  const bool runs = A.g.T / A.g.B >= 8;
  if (runs && rows >= (int64_t)16 * num_sms && (size_t)stride * 4 * 16 <= 98304) return launch_tile<D, 16>(A, stride, st);
  if (runs && rows >= (int64_t)16 * num_sms && (size_t)stride * 4 * 8 <= 98304) return launch_tile<D, 8>(A, stride, st);
  auto kern = gqa_select_one_kernel<D>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, 131072, allowed);
  if (e != cudaSuccess) return e;
  kern<<<dim3(A.g.T, A.c.Hkv), 32 * kOneWarps, (size_t)nb * 4, st>>>(A);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gqa_select_launch(const GqaSelectArgs& A, int num_sms, cudaStream_t st) {
  return A.c.D == 128 ? launch<128>(A, num_sms, st) : launch<64>(A, num_sms, st);
}

}  // namespace dsa
