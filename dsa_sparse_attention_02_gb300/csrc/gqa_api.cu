// Host side of the grouped-query operators (include/dsa.h): argument checks and launches.
#include <cmath>
#include <cstdint>
#include "dsa.h"
#include "kernels.cuh"

using namespace dsa;

namespace {

constexpr int kMaxSelect = 1024;
constexpr int kMaxListed = 32768;
constexpr int kMaxGroup = 16;
constexpr int kMaxSelectLen = 1 << 21;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dsa_status_t check_cache(const dsa_gqa_cache_t* c) {
  if (!c) return DSA_ERR_INVALID_ARG;
  if (c->dtype != DSA_E4M3 && c->dtype != DSA_I8) return DSA_ERR_INVALID_ARG;
  if (c->Hkv < 1 || c->Hkv > 128) return DSA_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// Codes and scales there and aligned (not asked of calls without work).
bool has_codes(const dsa_gqa_cache_t* c) {
  return c->k && c->v && c->k_scale && c->v_scale && aligned16(c->k) && aligned16(c->v) && aligned4(c->k_scale) &&
         aligned4(c->v_scale);
}
bool has_mean(const dsa_gqa_cache_t* c) {
  return c->k_mean && c->k_mean_scale && aligned16(c->k_mean) && aligned4(c->k_mean_scale);
}

bool heads_ok(const dsa_gqa_cache_t* c, int H) { return H >= 1 && H % c->Hkv == 0 && H / c->Hkv <= kMaxGroup; }

bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && aligned16(p) && stride >= width && stride % 8 == 0;
}

bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

GqaCacheDev cache_dev(const dsa_gqa_cache_t* c) {
  GqaCacheDev d;
  d.i8 = c->dtype == DSA_I8;
  d.Hkv = c->Hkv;
  d.D = c->D;
  d.k = reinterpret_cast<uint8_t*>(c->k);
  d.v = reinterpret_cast<uint8_t*>(c->v);
  d.k_scale = c->k_scale;
  d.v_scale = c->v_scale;
  d.k_mean = c->k_mean;
  d.k_mean_scale = c->k_mean_scale;
  return d;
}

size_t attend_ws(const dsa_geom_t* g, const dsa_gqa_cache_t* c, int H, int n_sel) {
  if (check_geom(g) != DSA_OK || check_cache(c) != DSA_OK || !heads_ok(c, H) || g->T == 0) return kHeaderBytes;
  return kHeaderBytes + align_up(gqa_attend_scratch_bytes(g, c->Hkv, c->D, H / c->Hkv, n_sel, num_sms()), 256);
}

dsa_status_t attend(const dsa_geom_t* g, const dsa_gqa_cache_t* c, int H, const void* q, int64_t q_stride,
                    const int32_t* blocks, int n_sel, float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                    void* stream) {
  dsa_status_t s = check_geom(g);
  if (s == DSA_OK) s = check_cache(c);
  if (s != DSA_OK) return s;
  const float scale_log2 = sm_scale * 1.4426950408889634f;   // scores in powers of two
  if (!heads_ok(c, H) || !std::isfinite(scale_log2) || sm_scale < 0.f) return DSA_ERR_INVALID_ARG;
  if ((int64_t)g->num_pages * c->Hkv > INT32_MAX) {
    set_last_error("grouped-query attention", "num_pages * Hkv above 2^31 - 1");
    return DSA_ERR_UNSUPPORTED;
  }
  if (!ws_ok(ws, ws_bytes, attend_ws(g, c, H, n_sel))) return DSA_ERR_WORKSPACE;
  if (g->T == 0) return DSA_OK;
  if (!has_codes(c) || !rows_ok(q, q_stride, (int64_t)H * c->D) || !out || !aligned16(out) || (lse && !aligned4(lse)))
    return DSA_ERR_INVALID_ARG;
  GqaAttendArgs A;
  A.g = to_dev(g);
  A.c = cache_dev(c);
  A.q = reinterpret_cast<const __nv_bfloat16*>(q);
  A.q_stride = q_stride;
  A.G = H / c->Hkv;
  A.scale_log2 = scale_log2;
  A.blocks = blocks;
  A.n_sel = n_sel;
  A.out = reinterpret_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  A.scratch = reinterpret_cast<uint8_t*>(ws) + kHeaderBytes;
  A.err = reinterpret_cast<int*>(ws);
  return from_cuda(gqa_attend_launch(A, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t dsa_gqa_append_workspace_size(const dsa_geom_t*, const dsa_gqa_cache_t*) { return kHeaderBytes; }

dsa_status_t dsa_gqa_append(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, const void* k_new, int64_t k_stride,
                            const void* v_new, int64_t v_stride, int32_t H, const void* q_in, int64_t q_stride,
                            void* q_out, int32_t rope_dim, const float* rope_cos, const float* rope_sin, void* ws,
                            size_t ws_bytes, void* stream) {
  dsa_status_t s = check_geom(geom);
  if (s == DSA_OK) s = check_cache(cache);
  if (s != DSA_OK) return s;
  if (rope_dim < 0 || rope_dim > cache->D || rope_dim % 8 != 0) return DSA_ERR_INVALID_ARG;
  if ((q_in == nullptr) != (q_out == nullptr)) return DSA_ERR_INVALID_ARG;
  if ((cache->k_mean == nullptr) != (cache->k_mean_scale == nullptr)) return DSA_ERR_INVALID_ARG;
  if (q_in && !heads_ok(cache, H)) return DSA_ERR_INVALID_ARG;
  // (blocks of threads of the launch: one for each page that may receive tokens and key head)
  if (((int64_t)geom->T / 64 + 2 * (int64_t)geom->B) * cache->Hkv > INT32_MAX) {
    set_last_error("dsa_gqa_append", "(T / 64 + 2 * B) * Hkv above 2^31 - 1");
    return DSA_ERR_UNSUPPORTED;
  }
  if (!ws_ok(ws, ws_bytes, kHeaderBytes)) return DSA_ERR_WORKSPACE;
  if (geom->T == 0) return DSA_OK;
  const int64_t width = (int64_t)cache->Hkv * cache->D;
  if (!has_codes(cache) || !rows_ok(k_new, k_stride, width) || !rows_ok(v_new, v_stride, width)) return DSA_ERR_INVALID_ARG;
  if (cache->k_mean && !has_mean(cache)) return DSA_ERR_INVALID_ARG;
  if (q_in && (!rows_ok(q_in, q_stride, (int64_t)H * cache->D) || !aligned16(q_out))) return DSA_ERR_INVALID_ARG;
  if (rope_dim > 0 && (!rope_cos || !rope_sin || !aligned16(rope_cos) || !aligned16(rope_sin))) return DSA_ERR_INVALID_ARG;
  GqaAppendArgs A;
  A.g = to_dev(geom);
  A.c = cache_dev(cache);
  A.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  A.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  A.q_in = reinterpret_cast<const __nv_bfloat16*>(q_in);
  A.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  A.q_stride = q_stride;
  A.G = q_in ? H / cache->Hkv : 0;
  A.rope_dim = rope_dim;
  A.rope_cos = rope_cos;
  A.rope_sin = rope_sin;
  A.err = reinterpret_cast<int*>(ws);
  return from_cuda(gqa_append_launch(A, reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsa_block_select_workspace_size(const dsa_geom_t*, const dsa_gqa_cache_t*, int32_t) { return kHeaderBytes; }

dsa_status_t dsa_block_select(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, int32_t H, const void* q,
                              int64_t q_stride, int32_t n_sel, int32_t n_first, int32_t n_last, int32_t* blocks,
                              void* ws, size_t ws_bytes, void* stream) {
  dsa_status_t s = check_geom(geom);
  if (s == DSA_OK) s = check_cache(cache);
  if (s != DSA_OK) return s;
  if (!heads_ok(cache, H)) return DSA_ERR_INVALID_ARG;
  if (n_sel < 1 || n_sel > kMaxSelect || n_first < 0 || n_last < 1 || n_first > n_sel || n_last > n_sel - n_first)
    return DSA_ERR_INVALID_ARG;
  if (geom->max_seq_len > kMaxSelectLen) {
    set_last_error("dsa_block_select", "max_seq_len above 2097152");
    return DSA_ERR_UNSUPPORTED;
  }
  if (!ws_ok(ws, ws_bytes, kHeaderBytes)) return DSA_ERR_WORKSPACE;
  if (geom->T == 0) return DSA_OK;
  if (!has_mean(cache) || !rows_ok(q, q_stride, (int64_t)H * cache->D) || !blocks || !aligned4(blocks))
    return DSA_ERR_INVALID_ARG;
  GqaSelectArgs A;
  A.g = to_dev(geom);
  A.c = cache_dev(cache);
  A.q = reinterpret_cast<const __nv_bfloat16*>(q);
  A.q_stride = q_stride;
  A.G = H / cache->Hkv;
  A.n_sel = n_sel;
  A.n_first = n_first;
  A.n_last = n_last;
  A.blocks = blocks;
  A.err = reinterpret_cast<int*>(ws);
  return from_cuda(gqa_select_launch(A, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t dsa_gqa_attend_workspace_size(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, int32_t H) {
  return attend_ws(geom, cache, H, 0);
}

dsa_status_t dsa_gqa_attend(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, int32_t H, const void* q,
                            int64_t q_stride, float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                            void* stream) {
  return attend(geom, cache, H, q, q_stride, nullptr, 0, sm_scale, out, lse, ws, ws_bytes, stream);
}

size_t dsa_gqa_attend_blocks_workspace_size(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, int32_t H,
                                            int32_t n_sel) {
  if (n_sel < 1 || n_sel > kMaxListed) return kHeaderBytes;
  return attend_ws(geom, cache, H, n_sel);
}

dsa_status_t dsa_gqa_attend_blocks(const dsa_geom_t* geom, const dsa_gqa_cache_t* cache, int32_t H, const void* q,
                                   int64_t q_stride, const int32_t* blocks, int32_t n_sel, float sm_scale, void* out,
                                   float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (n_sel < 1 || n_sel > kMaxListed) return DSA_ERR_INVALID_ARG;
  if (geom && geom->T > 0 && (!blocks || !aligned4(blocks))) return DSA_ERR_INVALID_ARG;
  return attend(geom, cache, H, q, q_stride, blocks, n_sel, sm_scale, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
