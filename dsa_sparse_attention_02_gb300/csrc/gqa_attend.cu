// Grouped-query attention over the paged 8-bit cache, whole contexts or listed blocks
// (the definitions are at dsa_gqa_attend and dsa_gqa_attend_blocks in include/dsa.h).
//
// One warp per (token, head): a lane scores one key at a time, the warp keeps the running
// maximum and sum, and all lanes add the 32 values in turn.
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;

template <bool I8>
__device__ __forceinline__ float2 code2(uint32_t v) {
  if constexpr (I8) return make_float2((float)(int8_t)(v & 0xFF), (float)(int8_t)((v >> 8) & 0xFF));
  else return e4m3x2_f32(v);
}

template <int D, bool I8>
__global__ void __launch_bounds__(32 * kWarps) gqa_attend_kernel(const GqaAttendArgs A) {
  constexpr int V = D / 32;
  __shared__ float s_q[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = A.G * A.c.Hkv;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= (int64_t)A.g.T * H) return;
  const int t = (int)(row / H), h = (int)(row % H), kvh = h / A.G;
  bool bad;
  const GqaToken k = gqa_token_warp(A.g, t, &bad);
  if (bad && lane == 0) record_error(A.err, kDevBadIndex);
  if (k.row == kRowPadding) return;
  for (int d = lane; d < D; d += 32) s_q[warp][d] = __bfloat162float(A.q[(int64_t)t * A.q_stride + h * D + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[V] = {};
  const int n = k.row != kRowSees ? 0 : A.blocks ? A.n_sel : (k.pos >> 6) + 1;
  const int* list = A.blocks ? A.blocks + ((int64_t)t * A.c.Hkv + kvh) * A.n_sel : nullptr;
  for (int i = 0; i < n; ++i) {
    int c = i;
    if (list) {
      c = __ldg(list + i);
      if (c < 0 || c > (k.pos >> 6)) continue;
      if (i > 0) {
        const int p = __ldg(list + i - 1);
        if (p < 0 || p >= c) {
          if (lane == 0) record_error(A.err, kDevBadIndex);
          continue;
        }
      }
    }
    const int page = gqa_page(A.g, k.b, c);
    if (page < 0) {
      if (lane == 0) record_error(A.err, kDevBadIndex);
      continue;
    }
    const int64_t tile = (int64_t)page * A.c.Hkv + kvh;
    const float ks = A.c.k_scale[tile] * A.scale_log2, vs = A.c.v_scale[tile];
    const uint8_t* kb = A.c.k + tile * (kPage * D);
    const uint8_t* vb = A.c.v + tile * (kPage * D);
    for (int s0 = 0; s0 < kPage; s0 += 32) {
      const int seen = min(32, k.pos + 1 - c * kPage - s0);
      if (seen <= 0) break;
      float z = -INFINITY;
      if (lane < seen) {
        float dot = 0.f;
        for (int d = 0; d < D; d += 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(kb + (s0 + lane) * D + d);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = code2<I8>(u[j >> 1] >> (16 * (j & 1)));
            dot += f.x * s_q[warp][d + 2 * j] + f.y * s_q[warp][d + 2 * j + 1];
          }
        }
        z = dot * ks;
      }
      const float mn = fmaxf(m, warp_max(z));
      const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float p = lane < seen ? exp2f(z - mn) : 0.f;
      l = l * keep + warp_sum(p);
      m = mn;
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] *= keep;
      for (int s = 0; s < seen; ++s) {
        const float w = __shfl_sync(0xffffffffu, p, s) * vs;
        const uint8_t* v = vb + (s0 + s) * D + lane * V;
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float2 f = code2<I8>(*reinterpret_cast<const uint16_t*>(v + j));
          o[j] += w * f.x;
          o[j + 1] += w * f.y;
        }
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* out = A.out + row * D + lane * V;
#pragma unroll
  for (int j = 0; j < V; ++j) out[j] = __float2bfloat16(o[j] * inv);
  if (A.lse && lane == 0) A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t gqa_attend_scratch_bytes(const dsa_geom_t*, int, int, int, int, int) { return 0; }

cudaError_t gqa_attend_launch(const GqaAttendArgs& A, int, cudaStream_t st) {
  const int64_t rows = (int64_t)A.g.T * A.G * A.c.Hkv;
  const unsigned grid = (unsigned)((rows + kWarps - 1) / kWarps);
  if (A.c.D == 128) {
    if (A.c.i8) gqa_attend_kernel<128, true><<<grid, 32 * kWarps, 0, st>>>(A);
    else gqa_attend_kernel<128, false><<<grid, 32 * kWarps, 0, st>>>(A);
  } else {
    if (A.c.i8) gqa_attend_kernel<64, true><<<grid, 32 * kWarps, 0, st>>>(A);
    else gqa_attend_kernel<64, false><<<grid, 32 * kWarps, 0, st>>>(A);
  }
  return cudaGetLastError();
}

}  // namespace dsa
