// What the dense latent-attention kernels share (latent_*.cu; entry points in latent_api.cu).
#pragma once
#include <cstdint>
#include "gqa_common.cuh"

namespace dsa {

// Partial results of cut items, in the workspace: two slots a run, `rows` rows of `width` each.
// Item i's first part lies in run c's slot `slot`, the next `follow` runs each hold one in slot 0.
struct __align__(16) LatentCut { int follow, slot, rows, step; int64_t out, pad; };   // output rows out, out + step, ...
struct LatentParts {
  int rows, width;
  LatentCut* cuts;   // one per run
  float* ml;         // [2 * runs, rows, 2] running maximum (log2 units) and sum
  float* o;          // [2 * runs, rows, width]
};
inline size_t latent_parts_bytes(int runs, int rows, int width) {
  return align_up(sizeof(LatentCut) * runs, 256) + align_up((size_t)2 * runs * rows * 2 * sizeof(float), 256) +
         (size_t)2 * runs * rows * width * sizeof(float);
}
inline LatentParts latent_parts(void* scratch, int runs, int rows, int width) {
  uint8_t* p = reinterpret_cast<uint8_t*>(scratch);
  LatentParts s;
  s.rows = rows, s.width = width;
  s.cuts = reinterpret_cast<LatentCut*>(p);
  p += align_up(sizeof(LatentCut) * runs, 256);
  s.ml = reinterpret_cast<float*>(p);
  s.o = reinterpret_cast<float*>(p + align_up((size_t)2 * runs * rows * 2 * sizeof(float), 256));
  return s;
}

// Run c of g starts at unit run_begin of n; unit x lies in run run_owner. (As split_begin and
// split_owner, but 64-bit divisions, some 200 clocks each, only where the numbers need them.)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {   // of numbers >= 0
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t run_begin(int64_t c, int64_t n, int64_t g) { return quotient(c * n, g); }
__device__ __forceinline__ int64_t run_owner(int64_t x, int64_t n, int64_t g) { return quotient((x + 1) * g - 1, n); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Barrier `id` among `count` threads that also tells whether any / all of them say so.
__device__ __forceinline__ bool bar_any(int id, int count, bool p) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)p), "r"(id), "r"(count)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ bool bar_all(int id, int count, bool p) { return !bar_any(id, count, !p); }

// 16 lanes x 32 columns, spread over the warp: thread i gets rows i / 4 (v[4j], v[4j+1]) and
// i / 4 + 8 (v[4j+2], v[4j+3]), columns 8j + 2 (i % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 matrices of 16-bit values to shared memory: lane i gives the address of matrix i / 8's row i % 8, and holds
// of each matrix row i / 4, columns 2 (i % 4) and the next.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Merges the parts of cut items in the order of the runs: block (c, y) looks whether run c holds
// an item's first part, and if so merges eight of its rows, one a warp.
constexpr int kLatentMergeWarps = 8;

template <int WIDTH>
__global__ void __launch_bounds__(32 * kLatentMergeWarps) latent_merge_kernel(const LatentParts s, __nv_bfloat16* out,
                                                                              float* lse) {
  constexpr int V = WIDTH / 128;                   // float4 pieces a lane has, 128 values apart
  constexpr int kBatch = V == 1 ? 8 : 4;           // parts whose loads are in flight together
  griddep_wait();
  const LatentCut k = s.cuts[blockIdx.x];
  const int row = blockIdx.y * kLatentMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (k.follow <= 0 || row >= k.rows) return;
  float M = kNone, l = 0.f, o[4 * V] = {};
  for (int p0 = 0; p0 <= k.follow; p0 += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch][V];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 + i;
      if (p > k.follow) break;
      const int64_t at = (p == 0 ? (int64_t)k.slot : 2 * (int64_t)(blockIdx.x + p)) * s.rows + row;
      ml[i] = __ldcg(reinterpret_cast<const float2*>(s.ml + at * 2));
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = __ldcg(reinterpret_cast<const float4*>(s.o + at * WIDTH) + 32 * j + lane);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (p0 + i > k.follow) break;
      const float Mn = fmaxf(M, ml[i].x), a = ex2(M - Mn), b = ex2(ml[i].x - Mn);
      M = Mn;
      l = l * a + ml[i].y * b;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[4 * j] = o[4 * j] * a + v[i][j].x * b, o[4 * j + 1] = o[4 * j + 1] * a + v[i][j].y * b;
        o[4 * j + 2] = o[4 * j + 2] * a + v[i][j].z * b, o[4 * j + 3] = o[4 * j + 3] * a + v[i][j].w * b;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = k.out + (int64_t)row * k.step;
  uint2* dst = reinterpret_cast<uint2*>(out + at * WIDTH) + lane;
#pragma unroll
  for (int j = 0; j < V; ++j)
    dst[32 * j] = make_uint2(pack_bf16(o[4 * j] * inv, o[4 * j + 1] * inv), pack_bf16(o[4 * j + 2] * inv, o[4 * j + 3] * inv));
  if (lse && lane == 0) lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <int WIDTH>
inline cudaError_t latent_merge_launch(const LatentParts& s, int runs, __nv_bfloat16* out, float* lse, cudaStream_t st) {
  // As much shared memory as the attention kernels ask for: between two kernels that want different
  // shares of it, an SM has to run empty and set its memory up anew.
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(latent_merge_kernel<WIDTH>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(runs, s.rows / kLatentMergeWarps);
  cfg.blockDim = dim3(32 * kLatentMergeWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<WIDTH>, s, out, lse);
}

}  // namespace dsa
