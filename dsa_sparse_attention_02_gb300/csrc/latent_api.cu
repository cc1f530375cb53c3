// Host side of the dense latent-attention operators (include/dsa.h): argument checks and launches.
#include <cmath>
#include <cstdint>
#include "dsa.h"
#include "kernels.cuh"

using namespace dsa;

namespace {

constexpr int kMaxHeads = 128;
constexpr int kRope = 64;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}
bool format_of(dsa_dtype_t dt, int* f) {
  *f = dt == DSA_E4M3 ? kKvE4m3 : dt == DSA_I8 ? kKvInt8 : kKvBf16;
  return dt == DSA_BF16 || dt == DSA_E4M3 || dt == DSA_I8;
}
bool stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0; }

bool rope_ok(const dsa_rope_t* r) {
  return r && r->dim >= 16 && r->dim <= kRope && r->dim % 16 == 0 && std::isfinite(r->scale);
}

size_t attend_ws(const dsa_geom_t* g, int H) {
  if (check_geom(g) != DSA_OK || H < 1 || H > kMaxHeads || g->T == 0) return kHeaderBytes;
  return kHeaderBytes + align_up(latent_attend_scratch_bytes(g, H, num_sms()), 256);
}

}  // namespace

extern "C" {

dsa_status_t dsa_rope_init(dsa_rope_t* rope, int32_t dim, int32_t interleaved, float base, float factor,
                           int64_t original_len, float beta_fast, float beta_slow, float scale) {
  if (!rope || dim < 16 || dim > kRope || dim % 16 != 0) return DSA_ERR_INVALID_ARG;
  if (!(base > 1.f) || !std::isfinite(base) || !(factor >= 1.f) || !std::isfinite(factor) || !std::isfinite(scale))
    return DSA_ERR_INVALID_ARG;
  if (original_len < 0) return DSA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  double lo = 0.0, hi = 0.0;
  if (original_len > 0) {
    if (!(beta_slow > 0.f) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)) return DSA_ERR_INVALID_ARG;
    auto at = [&](double turns) { return dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log((double)base)); };
    lo = std::fmax(std::floor(at(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(at(beta_slow)), (double)dim - 1);
  }
  dsa_rope_t r{};
  r.dim = dim;
  r.interleaved = interleaved != 0;
  r.scale = scale;
  for (int i = 0; i < dim / 2; ++i) {
    double ramp = 1.0;                      // the share of the scaled frequency
    if (original_len > 0) ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
    const double f = std::pow((double)base, -2.0 * i / dim);
    const double turns = (f / factor * ramp + f * (1.0 - ramp)) / two_pi;
    r.turns[i] = (uint64_t)(turns * 18446744073709551616.0);   // below a sixth of 2^64
  }
  *rope = r;
  return DSA_OK;
}

size_t dsa_latent_append_workspace_size(const dsa_geom_t*) { return kHeaderBytes; }

dsa_status_t dsa_latent_append(const dsa_geom_t* geom, dsa_dtype_t kv_dtype, const void* kv_in, int64_t kv_stride,
                               const float* gamma, float eps, const dsa_rope_t* rope, void* kv_cache, void* kv_out,
                               int32_t H, const void* q_in, int64_t q_in_token, int64_t q_in_head, void* q_out,
                               int64_t q_out_token, int64_t q_out_head, void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t s = check_geom(geom);
  if (s != DSA_OK) return s;
  LatentAppendArgs A{};
  if (!format_of(kv_dtype, &A.kv_format) || !rope_ok(rope)) return DSA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DSA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, kHeaderBytes)) return DSA_ERR_WORKSPACE;
  if (geom->T == 0) return DSA_OK;                 // (tensors without elements have no address)
  if ((q_in == nullptr) != (q_out == nullptr)) return DSA_ERR_INVALID_ARG;
  if (q_in && (H < 1 || H > kMaxHeads)) return DSA_ERR_INVALID_ARG;
  if (!kv_in && (kv_cache || kv_out)) return DSA_ERR_INVALID_ARG;
  if (!kv_in && !q_in) return DSA_ERR_INVALID_ARG;
  if (kv_in && (!kv_cache || !aligned16(kv_in) || !aligned16(kv_cache) || !stride_ok(kv_stride, 576) ||
                (gamma && !aligned16(gamma)) || (kv_out && !aligned16(kv_out))))
    return DSA_ERR_INVALID_ARG;
  if (q_in && (!aligned16(q_in) || !aligned16(q_out) || !stride_ok(q_in_head, kRope) || !stride_ok(q_out_head, kRope) ||
               !stride_ok(q_in_token, kRope) || !stride_ok(q_out_token, kRope)))
    return DSA_ERR_INVALID_ARG;
  if (latent_append_blocks(geom->T, H, kv_in != nullptr, q_in != nullptr) > INT32_MAX) {
    set_last_error("dsa_latent_append", "T * H too large for a launch");
    return DSA_ERR_UNSUPPORTED;
  }
  A.g = to_dev(geom);
  A.kv_in = reinterpret_cast<const __nv_bfloat16*>(kv_in);
  A.kv_stride = kv_stride;
  A.gamma = gamma;
  A.eps = eps;
  A.rope = *rope;
  A.kv_cache = reinterpret_cast<uint8_t*>(kv_cache);
  A.kv_out = reinterpret_cast<__nv_bfloat16*>(kv_out);
  A.H = H;
  A.q_in = reinterpret_cast<const __nv_bfloat16*>(q_in);
  A.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  A.qi_token = q_in_token, A.qi_head = q_in_head, A.qo_token = q_out_token, A.qo_head = q_out_head;
  A.err = reinterpret_cast<int*>(ws);
  return from_cuda(latent_append_launch(A, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsa_latent_gather_workspace_size(const dsa_geom_t*) { return kHeaderBytes; }

dsa_status_t dsa_latent_gather(const dsa_geom_t* geom, dsa_dtype_t kv_dtype, const void* kv_cache, const int32_t* first,
                               const int32_t* cu_k, int32_t S, void* out, int64_t out_stride, void* ws, size_t ws_bytes,
                               void* stream) {
  dsa_status_t s = check_geom(geom);
  if (s != DSA_OK) return s;
  LatentGatherArgs A{};
  if (!format_of(kv_dtype, &A.kv_format) || S < 0) return DSA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, kHeaderBytes)) return DSA_ERR_WORKSPACE;
  if (S == 0) return DSA_OK;
  if (geom->B < 1 || !kv_cache || !cu_k || !out || !aligned16(kv_cache) || !aligned16(out) || !aligned4(cu_k) ||
      (first && !aligned4(first)) || !stride_ok(out_stride, 576))
    return DSA_ERR_INVALID_ARG;
  A.g = to_dev(geom);
  A.kv = reinterpret_cast<const uint8_t*>(kv_cache);
  A.first = first;
  A.cu_k = cu_k;
  A.S = S;
  A.out = reinterpret_cast<__nv_bfloat16*>(out);
  A.out_stride = out_stride;
  A.err = reinterpret_cast<int*>(ws);
  return from_cuda(latent_gather_launch(A, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsa_latent_attend_workspace_size(const dsa_geom_t* geom, int32_t H) { return attend_ws(geom, H); }

dsa_status_t dsa_latent_attend(const dsa_geom_t* geom, dsa_dtype_t kv_dtype, int32_t H, const void* q,
                               const void* kv_cache, float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
  dsa_status_t s = check_geom(geom);
  if (s != DSA_OK) return s;
  LatentAttendArgs A{};
  if (!format_of(kv_dtype, &A.kv_format) || H < 1 || H > kMaxHeads) return DSA_ERR_INVALID_ARG;
  const float scale_log2 = sm_scale * 1.4426950408889634f;   // scores in powers of two
  if (!std::isfinite(scale_log2) || sm_scale < 0.f) return DSA_ERR_INVALID_ARG;
  if ((int64_t)geom->T * H > INT32_MAX - 127) {        // (rounded up to items, of 128 rows at most, in 32 bits)
    set_last_error("dsa_latent_attend", "T * H above 2^31 - 128");
    return DSA_ERR_UNSUPPORTED;
  }
  if (!ws_ok(ws, ws_bytes, attend_ws(geom, H))) return DSA_ERR_WORKSPACE;
  if (geom->T == 0) return DSA_OK;
  if (!q || !kv_cache || !out || !aligned16(q) || !aligned16(kv_cache) || !aligned16(out) || (lse && !aligned4(lse)))
    return DSA_ERR_INVALID_ARG;
  A.g = to_dev(geom);
  A.H = H;
  A.kv = reinterpret_cast<const uint8_t*>(kv_cache);
  A.scale_log2 = scale_log2;
  A.out = reinterpret_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.scratch = reinterpret_cast<uint8_t*>(ws) + kHeaderBytes;
  A.err = reinterpret_cast<int*>(ws);
  LatentMaps m;
  const uint64_t rows = (uint64_t)geom->T * H, pages = (uint64_t)geom->num_pages;
  const uint32_t n = (uint32_t)latent_attend_rows(A.g, H);
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  bool ok = encode_tensor_map_3d(&m.q, bf16, q, {64, rows, 9}, {1152, 128}, {64, n, 9}, true);
  if (kv_dtype == DSA_BF16) {
    ok = ok && encode_tensor_map_3d(&m.pair, bf16, kv_cache, {64, pages * 64, 9}, {1152, 128}, {64, 64, 2}, true) &&
         encode_tensor_map_3d(&m.rope, bf16, kv_cache, {64, pages * 64, 9}, {1152, 128}, {64, 64, 1}, true);
  } else {
    ok = ok && encode_tensor_map_3d(&m.pair, CU_TENSOR_MAP_DATA_TYPE_UINT8, kv_cache, {512, 64, pages},
                                    {512, kRecPageBytes}, {128, 64, 1}, false) &&
         encode_tensor_map_3d(&m.rope, bf16, A.kv + kRecRopeAt, {64, 64, pages}, {128, kRecPageBytes}, {64, 64, 1}, true);
  }
  if (!ok) return DSA_ERR_CUDA;
  return from_cuda(latent_attend_launch(A, m, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsa_latent_attend_expanded_workspace_size(int32_t B, int32_t T, int32_t S, int32_t H) {
  if (B < 1 || T < 1 || S < 0 || H < 1 || H > kMaxHeads) return kHeaderBytes;
  return kHeaderBytes + align_up(latent_expanded_scratch_bytes(num_sms()), 256);
}

dsa_status_t dsa_latent_attend_expanded(int32_t B, int32_t T, int32_t S, const int32_t* cu_q, const int32_t* cu_k, int32_t H,
                                        const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                                        int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                        const void* k_rope, int64_t rope_token, float sm_scale, void* out, float* lse,
                                        void* ws, size_t ws_bytes, void* stream) {
  if (B < 0 || T < 0 || S < 0 || (T > 0 && B < 1) || H < 1 || H > kMaxHeads) return DSA_ERR_INVALID_ARG;
  LatentExpandedArgs A{};
  const float scale_log2 = sm_scale * 1.4426950408889634f;   // scores in powers of two
  if (!std::isfinite(scale_log2) || sm_scale < 0.f) return DSA_ERR_INVALID_ARG;
  if (T > INT32_MAX - 65536 || S > INT32_MAX - 65536) return DSA_ERR_UNSUPPORTED;   // (rounded up to tiles in 32 bits)
  if (!ws_ok(ws, ws_bytes, dsa_latent_attend_expanded_workspace_size(B, T, S, H))) return DSA_ERR_WORKSPACE;
  if (T == 0) return DSA_OK;
  if (!cu_q || !cu_k || !aligned4(cu_q) || !aligned4(cu_k) || !q || !out || !aligned16(q) || !aligned16(out) ||
      (lse && !aligned4(lse)) || !stride_ok(q_token, 192) || !stride_ok(q_head, 192))
    return DSA_ERR_INVALID_ARG;
  if (S > 0 && (!k || !v || !k_rope || !aligned16(k) || !aligned16(v) || !aligned16(k_rope) || !stride_ok(k_token, 128) ||
                !stride_ok(k_head, 128) || !stride_ok(v_token, 128) || !stride_ok(v_head, 128) || !stride_ok(rope_token, 64)))
    return DSA_ERR_INVALID_ARG;
  A.B = B, A.T = T, A.S = S, A.H = H;
  A.cu_q = cu_q;
  A.cu_k = cu_k;
  A.scale_log2 = scale_log2;
  A.out = reinterpret_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.scratch = reinterpret_cast<uint8_t*>(ws) + kHeaderBytes;
  A.err = reinterpret_cast<int*>(ws);
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t h = (uint64_t)H, t = (uint64_t)T, n = (uint64_t)S;
  CUtensorMap mq, mk, mr, mv;
  if (!encode_tensor_map_3d(&mq, bf16, q, {192, h, t}, {(uint64_t)q_head * 2, (uint64_t)q_token * 2}, {64, 1, 128}, true))
    return DSA_ERR_CUDA;
  if (S > 0) {
    if (!encode_tensor_map_3d(&mk, bf16, k, {128, h, n}, {(uint64_t)k_head * 2, (uint64_t)k_token * 2}, {64, 1, 128}, true) ||
        !encode_tensor_map_3d(&mv, bf16, v, {128, h, n}, {(uint64_t)v_head * 2, (uint64_t)v_token * 2}, {64, 1, 64}, true) ||
        !encode_tensor_map_2d(&mr, bf16, k_rope, 64, n, (uint64_t)rope_token * 2, 64, 128))
      return DSA_ERR_CUDA;
  } else {
    mk = mv = mr = mq;               // (no unit loads through them)
  }
  return from_cuda(latent_expanded_launch(A, mq, mk, mr, mv, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
