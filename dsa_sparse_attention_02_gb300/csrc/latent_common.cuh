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
// 32 lanes x 32 columns: thread i gets lane i.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 matrices of 16-bit values to shared memory: lane i gives the address of matrix i / 8's row i % 8, and holds
// of each matrix row i / 4, columns 2 (i % 4) and the next.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Merges the parts of cut items in the order of the runs: blocks (c, y) look whether run c holds an
// item's first part, and if so merge rows of it, a warp one of 512 columns or four of 128 at a time.
// (128 columns: with one row a warp two short prompts took 11.6 us instead of 10.4. 512: with one, two or four
// rows of 128 columns a warp long contexts took 286 to 299 us instead of 280, two short requests 10.8 to 11.1 instead of 10.4.)
constexpr int kLatentMergeWarps = 8, kLatentMergeBlocks = 8;   // blocks of a run at most
template <int WIDTH>
constexpr int kLatentMergeRows = WIDTH == 128 ? 4 : 1;

template <int WIDTH>
__global__ void __launch_bounds__(32 * kLatentMergeWarps) latent_merge_kernel(const LatentParts s, __nv_bfloat16* out,
                                                                              float* lse) {
  constexpr int V = WIDTH / 128;                   // float4 pieces a lane has, 128 values apart
  constexpr int kRows = kLatentMergeRows<WIDTH>;
  constexpr int kBatch = V == 1 ? 2 : 4;           // parts whose loads are in flight together
  griddep_wait();
  const LatentCut k = s.cuts[blockIdx.x];
  if (k.follow <= 0) return;
  const int lane = threadIdx.x & 31;
  for (int row0 = (blockIdx.y * kLatentMergeWarps + (threadIdx.x >> 5)) * kRows; row0 < k.rows;
       row0 += gridDim.y * kLatentMergeWarps * kRows) {
    float M[kRows], l[kRows] = {};
    float4 o[kRows][V] = {};
#pragma unroll
    for (int r = 0; r < kRows; ++r) M[r] = kNone;
    for (int p0 = 0; p0 <= k.follow; p0 += kBatch) {
      float2 ml[kBatch][kRows];
      float4 v[kBatch][kRows][V];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = p0 + i;
        if (p > k.follow) break;
        const int64_t part = (p == 0 ? (int64_t)k.slot : 2 * (int64_t)(blockIdx.x + p)) * s.rows;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int64_t at = part + min(row0 + r, k.rows - 1);
          ml[i][r] = __ldcg(reinterpret_cast<const float2*>(s.ml + at * 2));
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][r][j] = __ldcg(reinterpret_cast<const float4*>(s.o + at * WIDTH) + 32 * j + lane);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (p0 + i > k.follow) break;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float Mn = fmaxf(M[r], ml[i][r].x), a = ex2(M[r] - Mn), b = ex2(ml[i][r].x - Mn);
          M[r] = Mn;
          l[r] = l[r] * a + ml[i][r].y * b;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o[r][j].x = o[r][j].x * a + v[i][r][j].x * b, o[r][j].y = o[r][j].y * a + v[i][r][j].y * b;
            o[r][j].z = o[r][j].z * a + v[i][r][j].z * b, o[r][j].w = o[r][j].w * a + v[i][r][j].w * b;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row0 + r >= k.rows) break;
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
      const int64_t at = k.out + (int64_t)(row0 + r) * k.step;
      uint2* dst = reinterpret_cast<uint2*>(out + at * WIDTH) + lane;
#pragma unroll
      for (int j = 0; j < V; ++j)
        dst[32 * j] = make_uint2(pack_bf16(o[r][j].x * inv, o[r][j].y * inv), pack_bf16(o[r][j].z * inv, o[r][j].w * inv));
      if (lse && lane == 0) lse[at] = l[r] == 0.f ? -INFINITY : (M[r] + log2f(l[r])) * 0.6931471805599453f;
    }
  }
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
  cfg.gridDim = dim3(runs, min(s.rows / (kLatentMergeWarps * kLatentMergeRows<WIDTH>), kLatentMergeBlocks));
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
