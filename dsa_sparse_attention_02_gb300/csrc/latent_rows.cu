// Rows of the paged latent cache, in and out (the definitions are at dsa_latent_append and
// dsa_latent_gather in include/dsa.h).
//
// Append: HBM bounds it where a chunk's queries are many, lookups and launch where they are few (2048
// tokens, 64 heads, e4m3 records and bf16 rows: 40 MB in 10.2 us, 3.9 TB/s; a token of two requests 2.9).
// A token's work is cut into warps: one norms, rotates and stores the row, the others rotate
// kWarpHeads query heads each (two rounds of eight heads by four threads, whose loads are all
// issued before the lookups that give the position). Angles are counted in turns, as fractions
// of 2^64: position times frequency is one 64-bit product whose overflow drops whole turns, so
// far positions lose nothing, and no table is read. Each lane of a warp takes one
// frequency's sine and cosine; shuffles hand them out.
// The sum of squares is held as a pair of fp32 (the squares of bf16 are exact in one) and the
// reciprocal root is corrected from that pair, so that stored codes do not depend on the
// order of the sum: it is the exact sum's but where that lies at a rounding's border.
//
// Gather: HBM bounds it (143 MB of e4m3 records and rows in 24.7 us, 5.8 TB/s). A warp takes kGatherRows rows, lane i the lookups of row i, with all
// rows' loads in flight together.
#include "latent_common.cuh"

namespace dsa {

namespace {

constexpr int kRowsWarps = 4;
constexpr int kWarpHeads = 16;
constexpr int kGatherRows = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// (h, l) += x, and the sum of two pairs, each keeping the roundings' errors.
__device__ __forceinline__ void pair_add(float& h, float& l, float x) {
  const float s = __fadd_rn(h, x), b = __fsub_rn(s, h);
  l = __fadd_rn(l, __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(x, b)));
  h = s;
}

// Four values' codes (e4m3 or int8), byte i from value i, as dsa_cache_append stores them.
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (I8) {
    const float f[4] = {a, b, c, d};
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (uint32_t)(max(-127, min(127, __float2int_rn(f[i]))) & 0xFF) << (8 * i);
    return r;
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xFFFFu) | (hi << 16);
  }
}

// Sines and cosines of a token's position: lane i has frequency i's.
struct Turn {
  float c, s;
  __device__ __forceinline__ Turn(const dsa_rope_t& r, int pos) {
    const int i = threadIdx.x & 31;
    const uint64_t at = i < r.dim / 2 ? r.turns[i] * (uint64_t)max(pos, 0) : 0;
    // the nearest fraction of half a turn in [-1, 1)
    const float half = (float)(int32_t)((at + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
    sincospif(half, &s, &c);
    c *= r.scale, s *= r.scale;
  }
};

// Rotates chunk a (values 8 g ..) and chunk b (8 g + dim / 2 ..) of a head's dim rotated values;
// whole warp, g = this thread's chunk.
__device__ __forceinline__ void rotate(const Turn& t, bool interleaved, int dim, int g, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // half: pair 8 g + i is (a[i], b[i]); interleaved: a holds pairs 4 g .., b pairs 4 g + dim / 4 ..
    const int f = interleaved ? 4 * g + (i >> 1) + (i & 1) * (dim / 4) : 8 * g + i;
    const float c = __shfl_sync(0xffffffffu, t.c, f & 31), s = __shfl_sync(0xffffffffu, t.s, f & 31);
    float& x = interleaved ? ((i & 1) ? b[i & 6] : a[i & 6]) : a[i];
    float& y = interleaved ? ((i & 1) ? b[i | 1] : a[i | 1]) : b[i];
    const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)), v = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = u, y = v;
  }
}

// The token's place: position (0 where it has none) and its row in the cache, or -1.
struct Place { int pos; int64_t row; bool padding; };
__device__ __forceinline__ Place place_of(const LatentAppendArgs& A, int t, bool want_row) {
  bool bad;
  const GqaToken k = gqa_token_warp(A.g, t, &bad);
  Place p{max(k.pos, 0), -1, k.row == kRowPadding};
  if (k.row == kRowEmpty) p.pos = 0;
  if (want_row && k.row == kRowSees) {
    p.row = physical_row(A.g, k.b, k.pos);
    if (p.row < 0) record_error(A.err, kDevBadIndex);
  }
  return p;
}

template <int KV>
__global__ void __launch_bounds__(32 * kRowsWarps) latent_append_kernel(const LatentAppendArgs A) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRowsWarps + (threadIdx.x >> 5);
  const int per = (A.kv_in ? 1 : 0) + (A.q_in ? (A.H + kWarpHeads - 1) / kWarpHeads : 0);
  if (blockIdx.x == 0 && threadIdx.x < 32) RequestCheck(A.g, lane).report(A.g, lane, 32, A.err);
  const int64_t t64 = w / per;
  if (t64 >= A.g.T) return;
  const int t = (int)t64, part = (int)(w - t64 * per);
  const int dim = A.rope.dim, half = dim / 16;      // chunks of 8 values: rotated ones of each half
  const bool inter = A.rope.interleaved != 0;
  if (A.kv_in && part == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(A.kv_in + (int64_t)t * A.kv_stride);
    const uint4 d0 = __ldg(src + 2 * lane), d1 = __ldg(src + 2 * lane + 1);
    // rotated part: thread g < half has chunks g and g + half, then the rest pass through
    const int rest = dim / 8 + (lane - half);       // chunk that lane >= half passes on, if below 8
    uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
    if (lane < half) ra = __ldg(src + 64 + lane), rb = __ldg(src + 64 + lane + half);
    else if (rest < 8) ra = __ldg(src + 64 + rest);
    float4 gm[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      gm[i] = A.gamma ? __ldg(reinterpret_cast<const float4*>(A.gamma) + 4 * lane + i) : make_float4(1.f, 1.f, 1.f, 1.f);
    const Place p = place_of(A, t, true);
    if (p.padding) return;
    const Turn turn(A.rope, p.pos);

    float v[16];
    {
      float a[8], b[8];
      unpack8(d0, a);
      unpack8(d1, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[i], v[8 + i] = b[i];
    }
    float h = 0.f, l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) pair_add(h, l, __fmul_rn(v[i], v[i]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, h, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      // (each lane of a pair must come to the same sum: the larger first)
      float a = fmaxf(h, h2), b = fminf(h, h2);
      if (h != h || h2 != h2) a = b = NAN;
      l = __fadd_rn(l, l2);
      pair_add(a, l, b);
      h = a;
    }
    // m = sum / 512 + eps as a pair, r = m^-1/2 with one correction from its residue
    h *= 1.f / kDimLatent, l *= 1.f / kDimLatent;
    pair_add(h, l, A.eps);
    const float r0 = rsqrtf(h), sq = __fmul_rn(r0, r0), sl = __fmaf_rn(r0, r0, -sq);
    const float res = __fmaf_rn(-l, sq, __fmaf_rn(-h, sl, __fmaf_rn(-h, sq, 1.f)));
    const float r = h > 0.f && r0 < INFINITY ? __fmaf_rn(__fmul_rn(0.5f, r0), res, r0) : r0;
    const float* g = reinterpret_cast<const float*>(gm);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], r), g[i]);

    float a[8], b[8];
    unpack8(ra, a);
    unpack8(rb, b);
    rotate(turn, inter, dim, min(lane, half - 1), a, b);
    const uint4 ka = lane < half ? pack8(a) : ra, kb = pack8(b);
    // the rotated part's chunk `lane` of the row, from whoever has it
    auto store_rope = [&](uint4* dst) {
      if (lane < half) dst[lane] = ka, dst[lane + half] = kb;
      else if (rest < 8) dst[rest] = ka;
    };
    uint4 o0, o1;
    {
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[i], y[i] = v[8 + i];
      o0 = pack8(x), o1 = pack8(y);
    }
    if (A.kv_out) {
      uint4* dst = reinterpret_cast<uint4*>(A.kv_out + (int64_t)t * kDimQK);
      dst[2 * lane] = o0, dst[2 * lane + 1] = o1;
      store_rope(dst + 64);
    }
    if (p.row < 0) return;
    if constexpr (KV == kKvBf16) {
      uint4* dst = reinterpret_cast<uint4*>(A.kv_cache + p.row * (kDimQK * 2));
      dst[2 * lane] = o0, dst[2 * lane + 1] = o1;
      store_rope(dst + 64);
    } else {
      constexpr bool kI8 = KV == kKvInt8;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));   // the lane's 128 values
      const float scale = m > 0.f ? __fdiv_rn(m, kI8 ? 127.f : 448.f) : 1.f;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = codes4<kI8>(__fdiv_rn(v[4 * i], scale), __fdiv_rn(v[4 * i + 1], scale), __fdiv_rn(v[4 * i + 2], scale),
                           __fdiv_rn(v[4 * i + 3], scale));
      *reinterpret_cast<uint4*>(A.kv_cache + rec_codes_at(p.row) + 16 * lane) = make_uint4(c[0], c[1], c[2], c[3]);
      if ((lane & 7) == 0) *reinterpret_cast<float*>(A.kv_cache + rec_scales_at(p.row) + 4 * (lane >> 3)) = scale;
      store_rope(reinterpret_cast<uint4*>(A.kv_cache + rec_rope_at(p.row)));
    }
    return;
  }
  // ---- query heads: four threads a head (chunks g and g + 4, or what of them is rotated)
  const int h0 = (part - (A.kv_in ? 1 : 0)) * kWarpHeads, g = lane & 3;
  const int ca = g < half ? g : dim / 8 + 2 * (g - half), cb = g < half ? g + half : ca + 1;   // this thread's two chunks
  constexpr int kRounds = kWarpHeads / 8;
  uint4 xa[kRounds], xb[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int h = h0 + 8 * i + (lane >> 2);
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (h < A.H) {
      const uint4* src = reinterpret_cast<const uint4*>(A.q_in + (int64_t)t * A.qi_token + (int64_t)h * A.qi_head);
      xa[i] = src[ca], xb[i] = src[cb];
    }
  }
  const Place p = place_of(A, t, false);
  if (p.padding) return;
  const Turn turn(A.rope, p.pos);
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    float a[8], b[8];
    unpack8(xa[i], a);
    unpack8(xb[i], b);
    rotate(turn, inter, dim, min(g, half - 1), a, b);
    const int h = h0 + 8 * i + (lane >> 2);
    if (h < A.H) {
      uint4* dst = reinterpret_cast<uint4*>(A.q_out + (int64_t)t * A.qo_token + (int64_t)h * A.qo_head);
      dst[ca] = g < half ? pack8(a) : xa[i];
      dst[cb] = g < half ? pack8(b) : xb[i];
    }
  }
}

template <int KV>
__global__ void __launch_bounds__(32 * kRowsWarps) latent_gather_kernel(const LatentGatherArgs A) {
  const int lane = threadIdx.x & 31;
  const int64_t s0 = ((int64_t)blockIdx.x * kRowsWarps + (threadIdx.x >> 5)) * kGatherRows;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < A.g.B; b += 32 * kRowsWarps) {
      const int c0 = __ldg(A.cu_k + b), c1 = __ldg(A.cu_k + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > A.S || __ldg(A.g.seq_lens + b) > A.g.max_seq_len) record_error(A.err, kDevBadIndex);
    }
  }
  // lane i: output row s0 + i; -2 where it is none of a request's, -1 where it has no row in the cache
  int64_t mine = -2;
  const int64_t s = s0 + lane;
  if (lane < kGatherRows && s < A.S && s >= __ldg(A.cu_k) && s < __ldg(A.cu_k + A.g.B)) {
    int lo = 0, hi = A.g.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(A.cu_k + mid) <= s) lo = mid; else hi = mid - 1;
    }
    const int64_t pos = (A.first ? (int64_t)__ldg(A.first + lo) : 0) + (s - __ldg(A.cu_k + lo));
    const int len = __ldg(A.g.seq_lens + lo);
    mine = -1;
    if (s >= __ldg(A.cu_k + lo) && s < __ldg(A.cu_k + lo + 1) && pos >= 0 && pos < len && len <= A.g.max_seq_len)
      mine = physical_row(A.g, lo, (int)pos);
    if (mine < 0) record_error(A.err, kDevBadIndex);
  }
  int64_t row[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) row[i] = __shfl_sync(0xffffffffu, mine, i);
  if constexpr (KV == kKvBf16) {
    uint4 v[kGatherRows][3];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        v[i][k] = make_uint4(0, 0, 0, 0);
        if (row[i] >= 0 && (k < 2 || lane < 8))
          v[i][k] = __ldg(reinterpret_cast<const uint4*>(A.kv + row[i] * (kDimQK * 2)) + 32 * k + lane);
      }
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      if (row[i] < -1) continue;
      uint4* dst = reinterpret_cast<uint4*>(A.out + (s0 + i) * A.out_stride);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < 2 || lane < 8) dst[32 * k + lane] = v[i][k];
    }
  } else {
    uint2 c[kGatherRows][2];
    uint4 r[kGatherRows];
    float sc[kGatherRows][2];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      r[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c[i][k] = make_uint2(0, 0), sc[i][k] = 0.f;
        if (row[i] >= 0) {
          c[i][k] = __ldg(reinterpret_cast<const uint2*>(A.kv + rec_codes_at(row[i])) + 32 * k + lane);
          sc[i][k] = __ldg(reinterpret_cast<const float*>(A.kv + rec_scales_at(row[i])) + 2 * k + (lane >> 4));
        }
      }
      if (row[i] >= 0 && lane < 8) r[i] = __ldg(reinterpret_cast<const uint4*>(A.kv + rec_rope_at(row[i])) + lane);
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      if (row[i] < -1) continue;
      uint4* dst = reinterpret_cast<uint4*>(A.out + (s0 + i) * A.out_stride);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a, b;
          codes_f16<KV == kKvInt8>(h ? c[i][k].y : c[i][k].x, a, b);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&b));
          o[2 * h] = pack_bf16(f.x * sc[i][k], f.y * sc[i][k]);
          o[2 * h + 1] = pack_bf16(g.x * sc[i][k], g.y * sc[i][k]);
        }
        dst[32 * k + lane] = row[i] >= 0 ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0, 0, 0, 0);
      }
      if (lane < 8) dst[64 + lane] = r[i];
    }
  }
}

}  // namespace

int64_t latent_append_blocks(int T, int H, bool rows, bool queries) {
  const int64_t per = (rows ? 1 : 0) + (queries ? (H + kWarpHeads - 1) / kWarpHeads : 0);
  return (T * per + kRowsWarps - 1) / kRowsWarps;
}

cudaError_t latent_append_launch(const LatentAppendArgs& A, cudaStream_t st) {
  const int grid = (int)latent_append_blocks(A.g.T, A.H, A.kv_in != nullptr, A.q_in != nullptr);
  switch (A.kv_format) {
    case kKvBf16: latent_append_kernel<kKvBf16><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
    case kKvE4m3: latent_append_kernel<kKvE4m3><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
    default: latent_append_kernel<kKvInt8><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
  }
  return cudaGetLastError();
}

cudaError_t latent_gather_launch(const LatentGatherArgs& A, cudaStream_t st) {
  const int grid = (int)(((int64_t)A.S + kGatherRows * kRowsWarps - 1) / (kGatherRows * kRowsWarps));
  switch (A.kv_format) {
    case kKvBf16: latent_gather_kernel<kKvBf16><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
    case kKvE4m3: latent_gather_kernel<kKvE4m3><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
    default: latent_gather_kernel<kKvInt8><<<grid, 32 * kRowsWarps, 0, st>>>(A); break;
  }
  return cudaGetLastError();
}

}  // namespace dsa
