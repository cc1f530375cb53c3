// Append to the grouped-query cache: rotation of the new tokens' keys and queries,
// quantisation of keys and values into their blocks, and the blocks' key means, in one
// launch (the definition is at dsa_gqa_append in include/dsa.h).
//
// Two kinds of blocks of threads. Queries: a thread owns W rotated pairs of a token (W 8 where
// the halves allow 16-byte accesses, else 4) and takes its head group's rows with the cosines
// and sines in registers. Keys and values:
//
// A block's scale is a maximum over its tokens, so one block of threads owns the new
// tokens of one (page, key head): it holds their values in registers, reduces the two
// magnitudes, and only then encodes. A scale that grows moves the older codes of the
// block; that, and the mean, are the only reads of the cache. Sums of at most 64 codes
// are exact in fp32 (e4m3 codes are multiples of 2^-9 below 2^9), so the mean does not
// depend on the order in which the shared-memory atomics add them.
//
// Which tokens a block of threads owns follows from its slot: request b's touched pages
// take slots cu_q[b]/64 + 2b onward (n new tokens touch at most n/64 + 2 pages), so the
// host needs only T and B. (Where offsets decrease the search may miss slots of good requests
// too: their tokens are not stored, and the error is set.) Rotation, scale, quotient and code
// are single IEEE operations in a fixed order: the stored state does not depend on the launch.
//
// A chunk of 2048 tokens with 64 + 8 + 8 heads of 128 (81 MB) takes 19.8 us in a graph, 4.1 TB/s:
// every block of threads loads, waits for its maximum and encodes, and two of them an SM
// overlap (one: 27). One to four tokens take 6.9 to 7.9: a chain of loads behind the launch.
#include <type_traits>
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kQHeads = 4;                    // query heads per thread
constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100
constexpr float kFltMax = 3.4028234663852886e38f;

template <int V>
struct Raw { uint32_t w[V / 2]; };

template <int V>
__device__ __forceinline__ Raw<V> load_row(const __nv_bfloat16* row, int lane) {
  Raw<V> r;
  if constexpr (V == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row) + lane);
  }
  return r;
}
template <int V>
__device__ __forceinline__ void unpack(const Raw<V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x[2 * i] = bf16_lo(r.w[i]);
    x[2 * i + 1] = bf16_hi(r.w[i]);
  }
}

// The lane's cos and sin at position pos: lanes below r/V hold first halves of the
// rotated pairs, the next r/V lanes their partners.
template <int V>
__device__ __forceinline__ void load_turn(const GqaAppendArgs& A, int pos, int lane, float (&c)[V], float (&s)[V]) {
  const int r = A.rope_dim >> 1, hl = r / V;
  if (lane < 2 * hl) {
    const int64_t at = (int64_t)pos * r + (lane < hl ? lane : lane - hl) * V;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 cc = __ldg(reinterpret_cast<const float2*>(A.rope_cos + at + j));
      const float2 ss = __ldg(reinterpret_cast<const float2*>(A.rope_sin + at + j));
      c[j] = cc.x, c[j + 1] = cc.y, s[j] = ss.x, s[j + 1] = ss.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void turn(const GqaAppendArgs& A, int lane, float (&x)[V], const float (&c)[V], const float (&s)[V]) {
  const int hl = (A.rope_dim >> 1) / V;
  const bool first = lane < hl, second = lane >= hl && lane < 2 * hl;
  const int src = first ? lane + hl : second ? lane - hl : lane;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float o = __shfl_sync(0xffffffffu, x[j], src);
    if (first) x[j] = __fsub_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o, s[j]));
    if (second) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o, s[j]));
  }
}

// Code of one value (already divided by its scale).
template <bool I8>
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  if constexpr (I8) {
    const int x = max(-127, min(127, __float2int_rn(a))), y = max(-127, min(127, __float2int_rn(b)));
    return (uint32_t)(x & 0xFF) | ((uint32_t)(y & 0xFF) << 8);
  } else {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  }
}
template <bool I8>
__device__ __forceinline__ float2 decode2(uint32_t v) {
  if constexpr (I8) return make_float2((float)(int8_t)(v & 0xFF), (float)(int8_t)((v >> 8) & 0xFF));
  else return e4m3x2_f32(v);
}
__device__ __forceinline__ float or_zero(float x) { return x == x ? x : 0.f; }
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= kFltMax ? a : 0.f;
}

// Older codes of one tensor's block: rows [0, rows) of the block, multiplied by ratio if
// grown; their sums per column into sum (shared) if kSum.
template <int D, bool I8, bool kSum, int kWarps>
__device__ __forceinline__ void older_codes(uint8_t* block, int rows, bool grown, float ratio, float* sum) {
  constexpr int kCh = D / 16;
  const int tid = threadIdx.x, ch = tid % kCh;
  float acc[16] = {};
  for (int p = tid; p < rows * kCh; p += 32 * kWarps) {
    uint4* at = reinterpret_cast<uint4*>(block) + p;
    uint4 v = *at;
    uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t c = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      if (grown) {
        const float2 f = decode2<I8>(c);
        c = encode2<I8>(__fmul_rn(f.x, ratio), __fmul_rn(f.y, ratio));
        w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xFFFFu) | (c << 16) : (w[i >> 1] & 0xFFFF0000u) | c;
      }
      if (kSum) {
        const float2 f = decode2<I8>(c);
        acc[2 * i] += or_zero(f.x);
        acc[2 * i + 1] += or_zero(f.y);
      }
    }
    if (grown) *at = v;
  }
  if (kSum && rows > 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int o = kCh; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    if ((tid & 31) < kCh) {
#pragma unroll
      for (int i = 0; i < 16; ++i) atomicAdd(sum + ch * 16 + i, acc[i]);
    }
  }
}

// Query rows: blocks of threads cover 32 * kWarps / (D / 2W) tokens and kQHeads heads.
template <int D, int W, int kWarps>
__device__ __forceinline__ void rotate_queries(const GqaAppendArgs& A, int index) {
  constexpr int kPer = D / (2 * W);              // threads per row
  constexpr int kTokens = 32 * kWarps / kPer;
  const int H = A.G * A.c.Hkv, groups = (H + kQHeads - 1) / kQHeads;
  const int t = (index / groups) * kTokens + threadIdx.x / kPer, h0 = (index % groups) * kQHeads, ch = threadIdx.x % kPer;
  const int r = A.rope_dim >> 1;
  const bool turned = ch < r / W;
  // the thread's values: W at first, W at second
  const int first = turned ? ch * W : 2 * r + (ch - r / W) * 2 * W, second = turned ? first + r : first + W;
  const __nv_bfloat16* src = A.q_in + (int64_t)t * A.q_stride + (int64_t)h0 * D;
  __nv_bfloat16* dst = A.q_out + ((int64_t)t * H + h0) * D;
  using Vec = typename std::conditional<W == 8, uint4, uint2>::type;
  Vec lo[kQHeads], hi[kQHeads];
#pragma unroll
  for (int i = 0; i < kQHeads; ++i)
    if (t < A.g.T && h0 + i < H) {
      lo[i] = __ldg(reinterpret_cast<const Vec*>(src + i * D + first));
      hi[i] = __ldg(reinterpret_cast<const Vec*>(src + i * D + second));
    }
  // position of each of the warp's tokens, or -1: left as it is
  int pos = -1;
#pragma unroll
  for (int k = 0; k < 32 / kPer; ++k) {
    const int tk = __shfl_sync(0xffffffffu, t, k * kPer);
    if (tk >= A.g.T || tk >= __ldg(A.g.cu_q + A.g.B)) continue;
    const QueryInfo qi = query_info_warp(A.g, tk);
    const int q0 = __ldg(A.g.cu_q + qi.b), q1 = __ldg(A.g.cu_q + qi.b + 1);
    const bool ok = tk >= q0 && tk < q1 && q0 >= 0 && q1 <= A.g.T && qi.len <= A.g.max_seq_len && qi.pos < qi.len;
    if (ok && tk == t) pos = qi.pos;
  }
  if (pos < 0) return;
  float c[W], s[W];
  if (turned) {
#pragma unroll
    for (int j = 0; j < W; j += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(A.rope_cos + (int64_t)pos * r + first + j));
      const float4 b = __ldg(reinterpret_cast<const float4*>(A.rope_sin + (int64_t)pos * r + first + j));
      c[j] = a.x, c[j + 1] = a.y, c[j + 2] = a.z, c[j + 3] = a.w;
      s[j] = b.x, s[j + 1] = b.y, s[j + 2] = b.z, s[j + 3] = b.w;
    }
  }
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    if (h0 + i >= H) break;
    if (turned) {
      uint32_t* a = reinterpret_cast<uint32_t*>(&lo[i]);
      uint32_t* b = reinterpret_cast<uint32_t*>(&hi[i]);
#pragma unroll
      for (int j = 0; j < W; j += 2) {
        const float x0 = bf16_lo(a[j / 2]), x1 = bf16_hi(a[j / 2]), y0 = bf16_lo(b[j / 2]), y1 = bf16_hi(b[j / 2]);
        const __nv_bfloat162 u = __floats2bfloat162_rn(__fsub_rn(__fmul_rn(x0, c[j]), __fmul_rn(y0, s[j])),
                                                       __fsub_rn(__fmul_rn(x1, c[j + 1]), __fmul_rn(y1, s[j + 1])));
        const __nv_bfloat162 v = __floats2bfloat162_rn(__fadd_rn(__fmul_rn(y0, c[j]), __fmul_rn(x0, s[j])),
                                                       __fadd_rn(__fmul_rn(y1, c[j + 1]), __fmul_rn(x1, s[j + 1])));
        a[j / 2] = *reinterpret_cast<const uint32_t*>(&u);
        b[j / 2] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *reinterpret_cast<Vec*>(dst + i * D + first) = lo[i];
    *reinterpret_cast<Vec*>(dst + i * D + second) = hi[i];
  }
}

// Blocks of threads below kv_blocks own (slot, key head)s, the others query rows; the last one
// looks the requests over. (In the blocks that store, that took 0.25 us more of one or two tokens.)
template <int D, bool I8, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 16 ? 2 : 4) gqa_append_kernel(const GqaAppendArgs A, int slots, int kv_blocks) {
  constexpr int V = D / 32, kTok = kPage / kWarps;   // kTok: new tokens of a block per warp
  __shared__ float s_amax[2][kWarps];
  __shared__ float s_sum[D];
  if ((int)blockIdx.x >= kv_blocks) {
    if (blockIdx.x == gridDim.x - 1) {
      RequestCheck(A.g, threadIdx.x).report(A.g, threadIdx.x, 32 * kWarps, A.err);
      return;
    }
    if ((A.rope_dim & 15) == 0) rotate_queries<D, 8, kWarps>(A, blockIdx.x - kv_blocks);
    else rotate_queries<D, 4, kWarps>(A, blockIdx.x - kv_blocks);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const GeomDev& g = A.g;
  const int slot = blockIdx.x % slots, kvh = blockIdx.x / slots;

  // request of this slot: the last b with cu_q[b]/64 + 2b <= slot (32 probes a round)
  int lo = 0, n = g.B;
  while (n > 32) {
    const int step = (n + 31) / 32, idx = lo + lane * step;
    const bool le = idx < lo + n && (__ldg(g.cu_q + idx) >> 6) + 2 * idx <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const bool le = lane < n && (__ldg(g.cu_q + lo + lane) >> 6) + 2 * (lo + lane) <= slot;
  const unsigned m = __ballot_sync(0xffffffffu, le);
  const int b = lo + (m ? 31 - __clz(m) : 0);
  const int q0 = __ldg(g.cu_q + b), q1 = __ldg(g.cu_q + b + 1), len = __ldg(g.seq_lens + b);
  const int nth = slot - ((q0 >> 6) + 2 * b);
  if (q0 < 0 || q1 < q0 || q1 > g.T || len > g.max_seq_len) return;
  const int start = max(0, len - (q1 - q0));           // first new position that exists
  if (nth < 0 || start >= len) return;
  const int blk = (start >> 6) + nth;
  const int p0 = max(start, blk << 6), p1 = min(len, (blk + 1) << 6);   // new positions of this block
  if (p0 >= p1) return;
  const int cnt = p1 - p0, t0 = q1 - len + p0;         // token of position p0

  // ---- keys and values
  const int page = gqa_page(g, b, blk);
  const int off = p0 - (blk << 6);                     // older tokens of the block
  Raw<V> rk[kTok], rv[kTok];                           // (before the page is known)
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const int tt = warp + i * kWarps;
    if (tt < cnt) {
      rk[i] = load_row<V>(A.k_new + (int64_t)(t0 + tt) * A.k_stride + kvh * D, lane);
      rv[i] = load_row<V>(A.v_new + (int64_t)(t0 + tt) * A.v_stride + kvh * D, lane);
    }
  }
  if (page < 0) {
    if (tid == 0) record_error(A.err, kDevBadIndex);
    return;
  }
  const int64_t tile = (int64_t)page * A.c.Hkv + kvh;
  const float ks_old = off > 0 ? A.c.k_scale[tile] : 0.f, vs_old = off > 0 ? A.c.v_scale[tile] : 0.f;
  for (int d = tid; d < D; d += 32 * kWarps) s_sum[d] = 0.f;
  float xk[kTok][V], mk = 0.f, mv = 0.f;
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const int tt = warp + i * kWarps;
    if (tt >= cnt) break;
    float c[V], s[V], xv[V];
    unpack<V>(rk[i], xk[i]);
    load_turn<V>(A, p0 + tt, lane, c, s);
    turn<V>(A, lane, xk[i], c, s);
    unpack<V>(rv[i], xv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mk = fmaxf(mk, finite_abs(xk[i][j]));
      mv = fmaxf(mv, finite_abs(xv[j]));
    }
  }
  mk = warp_max(mk);
  mv = warp_max(mv);
  if (lane == 0) s_amax[0][warp] = mk, s_amax[1][warp] = mv;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mk = fmaxf(mk, s_amax[0][w]), mv = fmaxf(mv, s_amax[1][w]);
  constexpr float kQmax = I8 ? 127.f : 448.f;
  const float ks = fmaxf(ks_old, fmaxf(__fdiv_rn(mk, kQmax), kScaleFloor));
  const float vs = fmaxf(vs_old, fmaxf(__fdiv_rn(mv, kQmax), kScaleFloor));
  uint8_t* kb = A.c.k + tile * (kPage * D);
  uint8_t* vb = A.c.v + tile * (kPage * D);
  if (tid == 0) A.c.k_scale[tile] = ks, A.c.v_scale[tile] = vs;
  const bool mean = A.c.k_mean != nullptr;
  const bool kgrown = off > 0 && ks > ks_old, vgrown = off > 0 && vs > vs_old;
  if (mean) older_codes<D, I8, true, kWarps>(kb, off, kgrown, __fdiv_rn(ks_old, ks), s_sum);
  else if (kgrown) older_codes<D, I8, false, kWarps>(kb, off, true, __fdiv_rn(ks_old, ks), nullptr);
  if (vgrown) older_codes<D, I8, false, kWarps>(vb, off, true, __fdiv_rn(vs_old, vs), nullptr);

  float sum[V] = {};
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    const int tt = warp + i * kWarps;
    if (tt >= cnt) break;
    float xv[V];
    unpack<V>(rv[i], xv);
    uint32_t ck[V / 2], cv[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      ck[j] = encode2<I8>(__fdiv_rn(xk[i][2 * j], ks), __fdiv_rn(xk[i][2 * j + 1], ks));
      cv[j] = encode2<I8>(__fdiv_rn(xv[2 * j], vs), __fdiv_rn(xv[2 * j + 1], vs));
      const float2 f = decode2<I8>(ck[j]);
      sum[2 * j] += or_zero(f.x);
      sum[2 * j + 1] += or_zero(f.y);
    }
    const int at = (off + tt) * D + lane * V;
    if constexpr (V == 4) {
      *reinterpret_cast<uint32_t*>(kb + at) = ck[0] | (ck[1] << 16);
      *reinterpret_cast<uint32_t*>(vb + at) = cv[0] | (cv[1] << 16);
    } else {
      *reinterpret_cast<uint16_t*>(kb + at) = (uint16_t)ck[0];
      *reinterpret_cast<uint16_t*>(vb + at) = (uint16_t)cv[0];
    }
  }
  if (!mean) return;
  if (warp < cnt) {
#pragma unroll
    for (int j = 0; j < V; ++j) atomicAdd(s_sum + lane * V + j, sum[j]);
  }
  __syncthreads();
  if (warp == 0) {
    float x[V], u = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = s_sum[lane * V + j];
      u = fmaxf(u, fabsf(x[j]));
    }
    u = __fdiv_rn(warp_max(u), 127.f);
    uint32_t code[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      code[j] = u > 0.f ? encode2<true>(__fdiv_rn(x[2 * j], u), __fdiv_rn(x[2 * j + 1], u)) : 0u;
    int8_t* dst = A.c.k_mean + tile * D + lane * V;
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(dst) = code[0] | (code[1] << 16);
    else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code[0];
    if (lane == 0) A.c.k_mean_scale[tile] = __fdiv_rn(__fmul_rn(u, ks), (float)(off + cnt));
  }
}

template <int D, bool I8, int kWarps>
cudaError_t launch(const GqaAppendArgs& A, cudaStream_t st) {
  const int slots = A.g.T / kPage + 2 * A.g.B, kv = slots * A.c.Hkv;
  const int W = (A.rope_dim & 15) == 0 ? 8 : 4, tokens = 32 * kWarps * 2 * W / D, H = A.G * A.c.Hkv;
  const int64_t blocks = kv + (A.q_in ? (int64_t)((A.g.T + tokens - 1) / tokens) * ((H + kQHeads - 1) / kQHeads) : 0);
  if (blocks >= INT32_MAX) return cudaErrorInvalidValue;
  gqa_append_kernel<D, I8, kWarps><<<(unsigned)blocks + 1, 32 * kWarps, 0, st>>>(A, slots, kv);
  return cudaGetLastError();
}

// Warps of a block: full blocks of new tokens keep sixteen busy, a few tokens not even four.
template <int D>
cudaError_t launch_warps(const GqaAppendArgs& A, cudaStream_t st) {
  if (A.g.T / A.g.B >= 16) return A.c.i8 ? launch<D, true, 16>(A, st) : launch<D, false, 16>(A, st);
  return A.c.i8 ? launch<D, true, 4>(A, st) : launch<D, false, 4>(A, st);
}

}  // namespace

cudaError_t gqa_append_launch(const GqaAppendArgs& A, cudaStream_t st) {
  return A.c.D == 128 ? launch_warps<128>(A, st) : launch_warps<64>(A, st);
}

}  // namespace dsa
