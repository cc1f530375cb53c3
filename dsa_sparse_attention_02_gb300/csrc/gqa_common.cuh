// What the grouped-query kernels share: tokens of a padded flattened batch, and codes.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "kernels.cuh"

namespace dsa {

// Request search as in query_info_warp, for batches whose last rows may be padding.
enum GqaRow : int { kRowSees = 0, kRowEmpty = 1, kRowPadding = 2 };
struct GqaToken {
  int b, pos;
  int row;      // kRowSees: keys 0..pos; kRowEmpty: sees no key; kRowPadding: outputs stay as they are
};

// Whole warp, every lane the same result. bad: the request's geometry is inconsistent.
__device__ __forceinline__ GqaToken gqa_token_warp(const GeomDev& g, int t, bool* bad) {
  *bad = false;
  GqaToken k{0, -1, kRowPadding};
  if (t >= __ldg(g.cu_q + g.B)) return k;
  const QueryInfo qi = query_info_warp(g, t);
  const int q0 = __ldg(g.cu_q + qi.b), q1 = __ldg(g.cu_q + qi.b + 1);
  *bad = t < q0 || t >= q1 || q1 > g.T || qi.len > g.max_seq_len;
  k.b = qi.b;
  k.pos = qi.pos;
  k.row = *bad || qi.pos < 0 || qi.pos >= qi.len ? kRowEmpty : kRowSees;
  return k;
}

// Reports inconsistent requests: thread `at` of `step` looks at every step-th one. (A search by
// token or slot can pass such a request over: none of its tokens has to exist.) The first one's
// loads are issued at construction, to pass under other lookups.
struct RequestCheck {
  int c0 = 0, c1 = 0, len = 0;
  __device__ __forceinline__ void load(const GeomDev& g, int64_t b) {
    c0 = __ldg(g.cu_q + b), c1 = __ldg(g.cu_q + b + 1), len = __ldg(g.seq_lens + b);
  }
  __device__ __forceinline__ RequestCheck(const GeomDev& g, int64_t at) {
    if (at < g.B) load(g, at);
  }
  __device__ __forceinline__ void report(const GeomDev& g, int64_t at, int64_t step, int* err) {
    for (int64_t b = at; b < g.B; b += step) {
      if (b != at) load(g, b);
      if (c0 < 0 || c1 < c0 || c1 > g.T || len > g.max_seq_len) record_error(err, kDevBadIndex);
    }
  }
};

// Page of request b's block c, or -1.
__device__ __forceinline__ int gqa_page(const GeomDev& g, int b, int c) {
  const int page = __ldg(g.block_table + (int64_t)b * g.bt_stride + c);
  return page >= 0 && page < g.num_pages ? page : -1;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Values of the two e4m3 codes in the low 16 bits.
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Lets a kernel use `bytes` of dynamic shared memory; the driver is asked once per device.
template <typename K>
inline cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---- attention: runs of units (gqa_attend.cu, gqa_tiles.cu)
constexpr float kNone = -3.0e38f;           // running maximum before the first key

// What a unit's stage says to the computing warps.
struct __align__(16) Unit {
  float kf;       // k_scale * sm_scale * log2(e)
  float lv, ivs;  // log2(v_scale), 1 / v_scale
  int flags;
  int rel;        // position of token 0, less the block's first position
  int q0, n;      // the request's first token and its number of tokens (listed blocks: the token, 1)
  int row0;       // first row of the tile (row r: token r / G, head r % G of key head h)
  int h;
  int slot;       // partial slot, or -1: the item ends in its outputs
  int c;          // the block's number in the request
  int pad;
};
enum : int { kFirst = 1, kLast = 2, kVoid = 4 };   // first / last unit of the run's part of an item; nothing to see

// Merge order of an item that was cut: run c holds its first part in `slot`, the next `follow`
// runs each a part in their slot 0. (A run belongs to a warp or a team of warps in gqa_attend.cu,
// to a block of threads in gqa_tiles.cu.)
struct __align__(16) Cut { int follow, slot, q0, n, row0, h, pad[2]; };

// A bounded wait by a whole warp: all lanes go on, or all give up. The waiting loop stays
// out of line: the roles of a block together outgrow the instruction caches, and a phase
// that is already complete should cost a few instructions.
static __device__ __noinline__ bool warp_wait_loop(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  const uint32_t a = smem_u32(bar);
  return __all_sync(0xffffffffu, mbar_try_wait(a, parity)) || warp_wait_loop(a, parity, abort, err);
}

// Partial results of cut items, in the workspace: two slots a run, `rows` rows each.
struct GqaParts {
  int rows;
  Cut* cuts;      // one per run
  float* ml;      // [2 * runs, rows, 2] running maximum (log2 units) and sum
  float* o;       // [2 * runs, rows, D]
};
inline size_t gqa_parts_bytes(int runs, int rows, int D) {
  return align_up(sizeof(Cut) * runs, 256) + align_up((size_t)2 * runs * rows * 2 * sizeof(float), 256) +
         (size_t)2 * runs * rows * D * sizeof(float);
}
inline GqaParts gqa_parts(void* scratch, int runs, int rows) {
  uint8_t* p = reinterpret_cast<uint8_t*>(scratch);
  GqaParts s;
  s.rows = rows;
  s.cuts = reinterpret_cast<Cut*>(p);
  p += align_up(sizeof(Cut) * runs, 256);
  s.ml = reinterpret_cast<float*>(p);
  s.o = reinterpret_cast<float*>(p + align_up((size_t)2 * runs * rows * 2 * sizeof(float), 256));
  return s;
}
cudaError_t gqa_merge_launch(const GqaAttendArgs& A, const GqaParts& s, int runs, cudaStream_t st);

// Rows of an item in the kernel for many query rows (gqa_tiles.cu).
constexpr int kGqaTileRows = 256;
cudaError_t gqa_tiles_launch(const GqaAttendArgs& A, int num_sms, cudaStream_t st);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The same of weights (cut at f16's largest value; a NaN stays one).
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// c += A B, m16n8k16, f16 with fp32 sums, in fragments.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// f16 pairs of a word's four codes: (byte 0, byte 1) and (byte 2, byte 3).
template <bool I8>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (I8) {
    // 0x64xx is 1024 + xx in f16; with the sign bit flipped xx is code + 128
    const uint32_t u = w ^ 0x80808080u, bias = 0x64806480u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

}  // namespace dsa
