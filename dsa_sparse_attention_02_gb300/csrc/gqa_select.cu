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
// Two shapes: one token per block of threads (decode: every warp scores, all of them
// select), or eight consecutive tokens (prompts: the mean of a block, read once, meets all
// tokens of the same request, and each warp selects for one token).
#include "gqa_common.cuh"

namespace dsa {

namespace {

constexpr int kTokTile = 8;      // tokens per block of threads in the prompt shape
constexpr int kOneWarps = 16;    // warps in the one-token shape

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

// The query token's pooled int8 code of key head kvh (D bytes at dst), by one warp.
template <int D>
__device__ __forceinline__ void pool_query(const GqaSelectArgs& A, int t, int kvh, uint8_t* dst, int lane) {
  constexpr int V = D / 32;
  const __nv_bfloat16* row = A.q + (int64_t)t * A.q_stride + (int64_t)kvh * A.G * D + lane * V;
  float x[V] = {};
  for (int h = 0; h < A.G; ++h) {
    uint32_t w[V / 2];
    if constexpr (V == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + h * D));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + h * D));
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      x[2 * j] = h ? __fadd_rn(x[2 * j], bf16_lo(w[j])) : bf16_lo(w[j]);
      x[2 * j + 1] = h ? __fadd_rn(x[2 * j + 1], bf16_hi(w[j])) : bf16_hi(w[j]);
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

// Keys of 32 blocks c0..c0+31 of request b for the tokens [w0, w1) of the tile; the whole
// warp. keys + w * stride receives token w's.
template <int D>
__device__ __forceinline__ void score_blocks(const GqaSelectArgs& A, int b, int kvh, int c0, int nv_max, int w0, int w1,
                                             const uint8_t* codes, const int* nv, uint32_t* keys, int stride, int lane) {
  constexpr int kLpb = D / 16;                   // lanes to a block's mean, 16 bytes each
  const int sub = lane % kLpb, grp = lane / kLpb;
  const int c = c0 + lane;
  const int page = c < nv_max ? gqa_page(A.g, b, c) : -1;
  if (c < nv_max && page < 0) record_error(A.err, kDevBadIndex);
  const float scale = page >= 0 ? __ldg(A.c.k_mean_scale + (int64_t)page * A.c.Hkv + kvh) : 0.f;
  uint4 mean[kLpb];
#pragma unroll
  for (int j = 0; j < kLpb; ++j) {
    const int p = __shfl_sync(0xffffffffu, page, grp * kLpb + j);
    mean[j] = p >= 0 ? __ldg(reinterpret_cast<const uint4*>(A.c.k_mean + ((int64_t)p * A.c.Hkv + kvh) * D) + sub)
                     : make_uint4(0, 0, 0, 0);
  }
  for (int w = w0; w < w1; ++w) {
    if (c0 >= nv[w]) continue;                   // (uniform)
    const uint4 q = *reinterpret_cast<const uint4*>(codes + w * D + sub * 16);
    int v[kLpb];
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
    if (c < nv[w]) {
      const float s = __fmul_rn((float)v[0], scale);
      uint32_t key = s == s ? max(orderable_key(s), 2u) : 1u;
      if (page < 0) key = 0u;
      if (c < A.n_first || c >= nv[w] - A.n_last) key = 0xFFFFFFFFu;
      keys[w * stride + c] = key;
    }
  }
}

// A token's list where nothing has to be chosen: all of its nv <= n_sel blocks.
__device__ __forceinline__ void list_all(int* out, int nv, int n_sel, int at, int step) {
  for (int i = at; i < n_sel; i += step) out[i] = i < nv ? i : -1;
}

template <int D, int TQ, int NW>
__global__ void __launch_bounds__(32 * NW) gqa_select_kernel(const GqaSelectArgs A, int stride) {
  extern __shared__ __align__(16) uint8_t select_smem[];
  __shared__ __align__(16) uint8_t s_codes[TQ][D];
  __shared__ int s_nv[TQ], s_b[TQ], s_row[TQ];
  constexpr int kSelWarps = TQ == 1 ? NW : 1;               // warps that select for one token
  __shared__ int s_scr[TQ][256 + 4 + 2 * kSelWarps];
  uint32_t* keys = reinterpret_cast<uint32_t*>(select_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * TQ, kvh = blockIdx.y;

  if (warp < TQ) {
    const int t = t0 + warp;
    GqaToken k{0, -1, kRowPadding};
    bool bad = false;
    if (t < A.g.T) k = gqa_token_warp(A.g, t, &bad);
    if (lane == 0) {
      if (bad) record_error(A.err, kDevBadIndex);
      s_row[warp] = k.row;
      s_b[warp] = k.b;
      s_nv[warp] = k.row == kRowSees ? (k.pos >> 6) + 1 : 0;
    }
    if (k.row == kRowSees && (k.pos >> 6) + 1 > A.n_sel) pool_query<D>(A, t, kvh, s_codes[warp], lane);
  }
  __syncthreads();
  // scores: runs of tokens of one request
  for (int w0 = 0; w0 < TQ;) {
    int w1 = w0 + 1, most = s_nv[w0];
    while (w1 < TQ && s_b[w1] == s_b[w0]) {
      most = max(most, s_nv[w1]);
      ++w1;
    }
    if (most > A.n_sel)
      for (int c0 = warp * 32; c0 < most; c0 += NW * 32)
        score_blocks<D>(A, s_b[w0], kvh, c0, most, w0, w1, &s_codes[0][0], s_nv, keys, stride, lane);
    w0 = w1;
  }
  __syncthreads();
  if (TQ == 1) {
    if (s_row[0] == kRowPadding) return;
    int* out = A.blocks + ((int64_t)t0 * A.c.Hkv + kvh) * A.n_sel;
    if (s_nv[0] <= A.n_sel) list_all(out, s_nv[0], A.n_sel, threadIdx.x, 32 * NW);
    else choose<kSelWarps>(keys, s_nv[0], A.n_sel, out, s_scr[0], warp, lane);
  } else if (warp < TQ && s_row[warp] != kRowPadding) {
    int* out = A.blocks + ((int64_t)(t0 + warp) * A.c.Hkv + kvh) * A.n_sel;
    if (s_nv[warp] <= A.n_sel) list_all(out, s_nv[warp], A.n_sel, lane, 32);
    else choose<kSelWarps>(keys + warp * stride, s_nv[warp], A.n_sel, out, s_scr[warp], warp % kSelWarps, lane);
  }
}

template <int D>
cudaError_t launch(const GqaSelectArgs& A, int num_sms, cudaStream_t st) {
  const int nb = (A.g.max_seq_len + kPage - 1) / kPage, stride = (nb + 3) / 4 * 4;
  const size_t tile = (size_t)stride * 4 * kTokTile;
  // Tiles of tokens pay once they alone fill the SMs and their scores fit beside others'.
  const bool tiles = (int64_t)A.g.T * A.c.Hkv >= (int64_t)2 * kTokTile * num_sms && A.g.T / A.g.B >= kTokTile && tile <= 98304;
  if (tiles) {
    auto kern = gqa_select_kernel<D, kTokTile, kTokTile>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tile);
    if (e != cudaSuccess) return e;
    kern<<<dim3((A.g.T + kTokTile - 1) / kTokTile, A.c.Hkv), 32 * kTokTile, tile, st>>>(A, stride);
  } else {
    auto kern = gqa_select_kernel<D, 1, kOneWarps>;
    const size_t bytes = (size_t)stride * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kern<<<dim3(A.g.T, A.c.Hkv), 32 * kOneWarps, bytes, st>>>(A, stride);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t gqa_select_launch(const GqaSelectArgs& A, int num_sms, cudaStream_t st) {
  return A.c.D == 128 ? launch<128>(A, num_sms, st) : launch<64>(A, num_sms, st);
}

}  // namespace dsa
