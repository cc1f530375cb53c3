// What the grouped-query kernels share: tokens of a padded flattened batch, and codes.
#pragma once
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

}  // namespace dsa
