// Dense causal attention in the absorbed form over the paged latent cache (the definition is
// at dsa_latent_attend in include/dsa.h).
//
// All heads of a token share one row per key, so a request's tokens x heads are query rows
// against the same pages. An item is (request, N of those rows); a unit is a page of 64 keys of
// an item. For each unit, on tcgen05 with bf16 operands and fp32 sums:
//   S = Q K^T      64 x 64 x 576 (Q rows past N are whatever lies behind: their lanes are not read)
//   O^T += C^T P^T 4 x (128 x N x 64), C the page's 512 latent columns, read MN-major from the
//                  same shared memory that S reads K-major
// so that O takes 4 N columns of tensor memory (with O by rows, its 512 columns would fill it),
// a page is read once for both products, and one 64-key page is what has to be whole: the rows
// of N = 64 queries alone take 74 KB, and 128 keys would leave no room for the next ones.
//
//   warps 0-7   softmax: S has 16 rows in each lane quarter; a 16 x 256-bit load spreads them
//               over all lanes, warp w has rows 16 (w % 4) on (those below N) and the keys of half
//               w / 4, a thread two rows with 8 keys each. P^T goes to shared memory by matrix
//               stores. The reference maximum moves only when a score passes it by more than 2^8;
//               then, and at an item's end, all eight read O^T (a quarter's lanes, half the columns).
//   then two issue scores and two (records: one) values: an MMA costs its issuer some 50 clocks,
//               more than it costs the tensor cores at these shapes (32 and 40 to 48)
//   one         finds the units of this block's run, loads pages by TMA in pairs of 64-column atoms
//   the rest    bf16: in a page that some row of the item does not see whole, zero the keys that no
//               row sees, and where rows see different keys those with a NaN or infinity, which rows
//               that do see them get as a NaN score (a weight of zero would not keep them out of
//               the sum). The scores do not wait for that.
//               records: convert codes to f16, exact; scales are applied in fp32 to each scale's
//               scores, and to the weights: P^T of each scale's 128 columns is its own. (With code *
//               scale rounded to bf16 instead, log-sum-exps were off by 0.3%.) The queries' latent part
//               is brought to f16 by an exact power of two a row.
//
// Weights meet bf16 rows in bf16, as both operands of a product are of one type; their sum is of the fp32
// weights. (Against 64 bits outputs are off by 0.0019 to 0.0021 of their norm, with fp32 weights 0.0017, which is the
// output's own rounding.) Weights times scales meet records in f16, where that is not to be seen.
//
// What bounds it. bf16 rows, 16 heads: HBM (376 MB in 71 us, of which 57 at 6.6 TB/s). 64 rows an item:
// the chain of a page, as two pages are all that fits beside the queries: loads (1900 clocks) ->
// scores (2000) -> softmax (1200) -> values (1500), 3,030 clocks a page (128 heads: 129.5 us, pages read
// from HBM once for two items in neighbouring blocks, 3.0 TB/s). Records, 64 rows: values -> conversion of the next page's last two pairs ->
// their scores -> softmax -> weights, and the softmax warps' own steps (each wait 200 clocks), which
// are as long: 4,500 to 4,700 clocks a page, with fewer rows too (8 contexts of 131072 in e4m3, 64 rows: 269 us,
// 2.6 TB/s; issue slots 51%, tensor pipe 35% busy).
// All units are laid end to end and cut into runs of equal cost, one per SM; cut items are merged.
#include "latent_units.cuh"

namespace dsa {

namespace {

constexpr int kSoftWarps = 8, kScoreWarp0 = 8, kValueWarp0 = 10;
constexpr uint32_t kSCol = 256;              // scores' first column in tensor memory
constexpr int kAhead = 1;                    // pages
constexpr float kMove = 8.f;                 // log2 of what a weight may pass the reference by

template <int N, int KV>
struct LatentShape {
  static constexpr bool kRecord = KV != kKvBf16;
  // Rings as deep as shared memory allows.
  static constexpr int kPairs = !kRecord ? (N == 16 ? 11 : N == 32 ? 10 : 8) : (N == 16 ? 8 : 6);
  static constexpr int kRopes = !kRecord && N == 16 ? 3 : kRecord && N == 64 ? 1 : 2;
  static constexpr int kCodes = !kRecord ? 0 : N == 64 ? 2 : 6;
  // (Records: the two groups of converting warps, and the two that issue scores, take every other place. In
  // an odd ring one would come to a place that the other's load has not reached yet, and take the phase
  // before that for the one it waits for.)
  static_assert(!kRecord || (kPairs % 2 == 0 && kCodes % 2 == 0), "a place has one user");
  // (bf16 rows: the ring may be odd. An issuer of scores comes to pair 4 n + j only when those of page n - 2 have been
  // read, for which all its pairs, up to 4 n - 5, had arrived: the load before in that place, 4 n + j - kPairs, as well.)
  static_assert(kRecord || kPairs >= 8, "the place's last load is behind the issuer");
  // Scores, from column 256 on. bf16 rows: a page's in one place (two, one of each issuer), two pages at a
  // time. Records: the rotated part's and three of the scales' in a place each, the last scale's in the
  // rotated part's. P: one of a page, or three, the last scale's in the first's place.
  static constexpr int kPs = kRecord ? 3 : 1;
  // (20 and 16 warps: a whole number for each quarter of the SM, whose registers they share)
  static constexpr int kValueWarps = kRecord ? 1 : 2, kFixWarps = kRecord ? 8 : 3;
  static constexpr int kLoadWarp = kValueWarp0 + kValueWarps, kFixWarp0 = kLoadWarp + 1;
  static constexpr int kThreads = 32 * (kFixWarp0 + kFixWarps);
  // An item's cost beside its units'. (0, 1, 2, 3, 4, 6: decode of 16 heads 71.1, 70.3, 70.6, 70.9, 71.4, 72.6 us; of
  // 128 heads 149, 149, 147, 147, 145, 143; verification int8, 64 rows, 107, 106, 103, 103, 103, 105)
  static constexpr int kItemCost = N == 64 ? 4 : N == 32 ? 2 : 1;
  static constexpr int kQBytes = 9 * N * 128, kPBytes = N * 128;   // of one P
  static constexpr int kSmem = 1024 + kQBytes + kPs * kPBytes + kRopes * kRopeBytes + kPairs * kPairBytes + kCodes * kCodeStage +
                               (kRecord ? kScaleSlots * 1024 : 0);
  static_assert(kSmem <= 227 * 1024 - (kRecord ? 3328 : 2048), "and barriers, units and row statistics beside it");
};

// Queries of records: the latent part of N rows in shared memory, bf16 to f16, each row by a power of
// two that brings its largest magnitude into [2^13, 2^14) (what lies 2^31 below that may round; the
// rest is exact). factor[row] undoes it. For 256 threads.
// (Eight lanes have a row's 128 bytes of an atom, so that no two meet in a bank; each value is read once.)
template <int N>
__device__ __forceinline__ void queries_f16(uint8_t* q_buf, int tid, float* factor) {
  constexpr int kWarpRows = N / kSoftWarps;                      // 8, 4 or 2
  constexpr int kLanes = kWarpRows == 2 ? 16 : 8, kAtoms = 64 / kLanes, kAtomStep = kLanes / 8;
  const int lane = tid & 31;
#pragma unroll 1
  for (int r = 0; r < kWarpRows; r += 32 / kLanes) {
    const int row = (tid >> 5) * kWarpRows + r + lane / kLanes;
    uint8_t* at = q_buf + (lane >> 3) % kAtomStep * (N * 128) + row * 128 + (((lane ^ row) & 7) << 4);
    uint4 v[kAtoms];
    uint32_t top = 0;                            // largest magnitude, as bf16 bits
#pragma unroll
    for (int i = 0; i < kAtoms; ++i) {
      v[i] = *reinterpret_cast<const uint4*>(at + i * kAtomStep * (N * 128));
      const uint32_t o[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(o[e] & 0x7FFFu, o[e] >> 16 & 0x7FFFu));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = min(max((int)(top >> 7) - 127, -60), 127);
    const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
    if (lane % kLanes == 0) factor[row] = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
    for (int i = 0; i < kAtoms; ++i)
      *reinterpret_cast<uint4*>(at + i * kAtomStep * (N * 128)) =
          make_uint4(pack_f16(bf16_lo(v[i].x) * up, bf16_hi(v[i].x) * up), pack_f16(bf16_lo(v[i].y) * up, bf16_hi(v[i].y) * up),
                     pack_f16(bf16_lo(v[i].z) * up, bf16_hi(v[i].z) * up), pack_f16(bf16_lo(v[i].w) * up, bf16_hi(v[i].w) * up));
  }
}

// Place and phase of a ring's user that takes more than one step at a time.
template <int K>
struct Ring {
  int at;
  uint32_t ph = 0;
  __device__ __forceinline__ explicit Ring(int first) : at(0) { step(first); }
  __device__ __forceinline__ void step(int k) {
    at += k;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at >= K) at -= K, ph ^= 1u;
  }
};

// BL: blocks of a run, which have neighbouring items of N rows each over the same pages at about the same
// time, so that a page is read from HBM by the first and found in L2 by the other.
template <int N, int KV, int BL>
__global__ void __launch_bounds__(LatentShape<N, KV>::kThreads, 1)
    latent_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_pair,
                         const __grid_constant__ CUtensorMap map_rope, const LatentAttendArgs A, const LatentParts parts) {
  using S = LatentShape<N, KV>;
  constexpr bool kRecord = S::kRecord;
  constexpr int kLoadWarp = S::kLoadWarp, kFixWarp0 = S::kFixWarp0;
  constexpr uint32_t kFmt = kRecord ? kFmtF16 : kFmtBF16;   // of latents, and of weights
  static_assert(BL == 1 || !kRecord, "records have no form of two blocks");
  constexpr int R = BL * N;                     // rows of an item as the units and the parts see it
  const int rank = BL == 1 ? 0 : (int)blockIdx.x % BL;
  // Weights in f16 use its range upwards as well: 2^7 at the reference, and so below 2^16.
  constexpr float kLift = kRecord ? 7.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_buf = smem;                                  // (S reads 64 rows of each atom: up to 6 KB past the last)
  uint8_t* p_buf = q_buf + S::kQBytes;
  uint8_t* rope_buf = p_buf + S::kPs * S::kPBytes;
  uint8_t* pair_buf = rope_buf + S::kRopes * kRopeBytes;
  uint8_t* code_buf = pair_buf + S::kPairs * kPairBytes;
  float* scale_buf = reinterpret_cast<float*>(code_buf + S::kCodes * kCodeStage);
  __shared__ uint64_t u_full[kUnits], u_loaded[kUnits], u_empty[kUnits], e_full[kUnits];
  __shared__ uint64_t pair_full[S::kPairs], pair_empty[S::kPairs], rope_full[S::kRopes], rope_empty[S::kRopes];
  __shared__ uint64_t code_full[kRecord ? S::kCodes : 1], code_empty[kRecord ? S::kCodes : 1];
  __shared__ uint64_t scale_full[kRecord ? kScaleSlots : 1];
  __shared__ uint64_t q_full, q_free, s_full[2], s_empty[2], p_full;   // (bf16 rows)
  // records, each once a page: the rotated part's and the first scale's scores are there (and the last
  // page's first weights used), the next two's, the last's (and the last page's last weights used); the
  // first two have been read, the others; the first scale's weights are there, the next two's, the
  // last's; the first's have been used
  __shared__ uint64_t f_front, f_mid, f_last, e_front, e_rest, p_front, p_mid, p_last, p_used;
  __shared__ uint64_t q_ready;                            // records: the queries are in f16
  __shared__ uint64_t o_done[2], drain[4];                // o_done: of even and odd units
  __shared__ LatentUnit s_unit[kUnits];
  __shared__ uint32_t s_bad[kUnits][2];                   // keys with a value that is not finite
  __shared__ __align__(16) float s_keep[N], s_top[2][N], s_sum[2][N], s_qf[kRecord ? N : 1], s_lg[kRecord ? kUnits : 1][kPage];
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&u_full[i]), 1);
      mbar_init(smem_u32(&u_loaded[i]), 1);
      mbar_init(smem_u32(&u_empty[i]), kSoftWarps + S::kFixWarps);
      mbar_init(smem_u32(&e_full[i]), S::kFixWarps);
    }
    for (int i = 0; i < S::kPairs; ++i) {
      mbar_init(smem_u32(&pair_full[i]), kRecord ? S::kFixWarps / 2 : 1);
      mbar_init(smem_u32(&pair_empty[i]), 1);
    }
    for (int i = 0; i < S::kRopes; ++i) {
      mbar_init(smem_u32(&rope_full[i]), 1);
      mbar_init(smem_u32(&rope_empty[i]), 1);
    }
    if (kRecord) {
      for (int i = 0; i < kScaleSlots; ++i) mbar_init(smem_u32(&scale_full[i]), 1);
      for (int i = 0; i < S::kCodes; ++i) {
        mbar_init(smem_u32(&code_full[i]), 1);
        mbar_init(smem_u32(&code_empty[i]), S::kFixWarps / 2);
      }
    }
    mbar_init(smem_u32(&q_full), 1);
    mbar_init(smem_u32(&q_free), 2);
    mbar_init(smem_u32(&q_ready), kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 2);
      mbar_init(smem_u32(&s_empty[i]), N / 8);
    }
    mbar_init(smem_u32(&p_full), kSoftWarps);
    mbar_init(smem_u32(&f_front), 2);
    mbar_init(smem_u32(&f_mid), 2);
    mbar_init(smem_u32(&f_last), 2);
    mbar_init(smem_u32(&e_front), N / 8);
    mbar_init(smem_u32(&e_rest), N / 8);
    mbar_init(smem_u32(&p_front), N / 8);
    mbar_init(smem_u32(&p_mid), N / 8);
    mbar_init(smem_u32(&p_last), N / 8);
    mbar_init(smem_u32(&p_used), 1);
    mbar_init(smem_u32(&o_done[0]), S::kValueWarps);
    mbar_init(smem_u32(&o_done[1]), S::kValueWarps);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&drain[i]), 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kScoreWarp0) {
    tmem_alloc(smem_u32(&s_tmem), kTmem);
    tmem_relinquish();
  }
  LatentCursor<R, S::kItemCost> at(A, parts, blockIdx.x / BL, gridDim.x / BL, rank == 0);
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_pair);
      tma_prefetch_desc(&map_rope);
    }
    at.find();
    if (at.begin < at.end) at.batch(at.begin);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort = &s_abort;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ units and loads
    const int count = (int)(at.end - at.begin);
    if (count == 0 && lane == 0) {
      s_unit[0].flags = kStop;
      mbar_arrive(smem_u32(&u_full[0]));
    }
    int pair = 0, rope = 0, code = 0;
    uint32_t pair_ph = 0, rope_ph = 0, code_ph = 0;
    bool ok = true;
    for (int n = 0; n < count && ok; ++n) {
      if (at.at == at.cnt) at.batch(at.begin + n);
      {
        // The page kAhead units on into L2, ahead of its loads: too few of those are under way for HBM's latency
        // (records: 304 us without, 284, 286, 288 and 305 with 1, 2, 3 and 6; bf16 rows gain 1%)
        constexpr uint32_t kPageBytes = kRecord ? kRecPageBytes : kPage * kDimQK * 2;
        const bool mine = at.at == 0 ? lane <= kAhead : lane == at.at + kAhead;
        if (mine && lane < at.cnt && at.page >= 0 && rank == 0) bulk_prefetch_l2(A.kv + (int64_t)at.page * kPageBytes, kPageBytes);
      }
      const int us = n % kUnits;
      ok = warp_wait(&u_empty[us], ((n / kUnits) & 1) ^ 1, abort, A.err);
      if (!ok) break;
      if (lane == at.at) {
        LatentUnit x = at.x;
        if (BL > 1) x.row0 += N * rank, x.out += N * rank, x.rows = min(max(x.rows - N * rank, 0), N);
        s_unit[us] = x;
        s_bad[us][0] = s_bad[us][1] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&u_full[us]));
      const int pg = __shfl_sync(0xffffffffu, at.page, at.at++);
      auto load_rope = [&]() {
        ok = warp_wait(&rope_empty[rope], rope_ph ^ 1, abort, A.err);
        if (!ok) return;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&rope_full[rope]);
          if (pg >= 0) {
            mbar_arrive_expect_tx(bar, kRopeBytes);
            if (kRecord) tma_load_3d(smem_u32(rope_buf + rope * kRopeBytes), &map_rope, bar, 0, 0, pg);
            else tma_load_3d(smem_u32(rope_buf + rope * kRopeBytes), &map_rope, bar, 0, pg * kPage, 8);
          } else {
            mbar_arrive(bar);
          }
        }
        if (++rope == S::kRopes) rope = 0, rope_ph ^= 1u;
      };
      if (!kRecord) load_rope();
      if (!ok) break;
      if (kRecord && lane == 0) {                 // (the slot's last reader has given back its unit)
        const uint32_t bar = smem_u32(&scale_full[n % kScaleSlots]);
        if (pg >= 0) {
          mbar_arrive_expect_tx(bar, 1024);
          bulk_load(smem_u32(scale_buf + (n % kScaleSlots) * 256), A.kv + (int64_t)pg * kRecPageBytes + kRecScalesAt, 1024, bar);
        } else {
          mbar_arrive(bar);
        }
      }
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        if (kRecord) {
          // (the rotated part's one place is free later than the first codes')
          if (j == 2) load_rope();
          ok = ok && warp_wait(&code_empty[code], code_ph ^ 1, abort, A.err);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&code_full[code]);
            if (pg >= 0) {
              mbar_arrive_expect_tx(bar, kCodeStage);
              tma_load_3d(smem_u32(code_buf + code * kCodeStage), &map_pair, bar, 128 * j, 0, pg);
            } else {
              mbar_arrive(bar);
            }
          }
          if (++code == S::kCodes) code = 0, code_ph ^= 1u;
        } else {
          ok = warp_wait(&pair_empty[pair], pair_ph ^ 1, abort, A.err);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&pair_full[pair]);
            if (pg >= 0) {
              mbar_arrive_expect_tx(bar, kPairBytes);
              tma_load_3d(smem_u32(pair_buf + pair * kPairBytes), &map_pair, bar, 0, pg * kPage, 2 * j);
            } else {
              mbar_arrive(bar);
            }
          }
          if (++pair == S::kPairs) pair = 0, pair_ph ^= 1u;
        }
      }
      if (ok && lane == 0) mbar_arrive(smem_u32(&u_loaded[us]));
    }
    // Copies in flight land before shared memory is given back: every slot's last copy is waited
    // for by its reader, or, when the run was given up, here.
    if (!ok) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {}
    }
  } else if (warp >= kScoreWarp0 && warp < kLoadWarp) {
    // ------------------------------------------------------------ MMA issue: scores, values
    const bool issuer = elect_one();
    const int half = (warp - kScoreWarp0) & 1;    // pairs half and half + 2 of a page; the first has the rotated part
    bool ok = tmem == 0;                          // all 512 columns are this block's
    if (!ok) {
      *abort = 1;
      record_error(A.err, kDevTimeout);
    }
    if (warp < kValueWarp0) {
      Ring<S::kPairs> pair(half);
      constexpr uint32_t idesc_rope = make_idesc(64, kPage, kFmtBF16, kFmtBF16, 0, 0);
      constexpr uint32_t idesc = make_idesc(64, kPage, kFmt, kFmt, 0, 0);
      const uint64_t dq = smem_desc(smem_u32(q_buf), 0, 1024, kSwizzle128B);
      const uint64_t dk = smem_desc(smem_u32(pair_buf), 0, 1024, kSwizzle128B);
      const uint64_t dr = smem_desc(smem_u32(rope_buf), 0, 1024, kSwizzle128B);
      Ring<S::kRopes> rope(0);
      uint32_t seg = 0;
      for (int n = 0, flags = 0; ok && !(flags & kEnd); ++n) {
        const int us = n % kUnits;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        flags = s_unit[us].flags;
        if (flags & kStop) break;
        if (flags & kFirst) {
          if (half == 0) {
            // the last segment's scores have left the queries' place
            if (seg > 0) ok = warp_wait(&q_free, (seg - 1) & 1, abort, A.err);
            if (ok && issuer) {
              const uint32_t bar = smem_u32(&q_full);
              mbar_arrive_expect_tx(bar, S::kQBytes);
              tma_load_3d(smem_u32(q_buf), &map_q, bar, 0, (int)s_unit[us].out, 0);
            }
            __syncwarp();
          }
          ok = ok && warp_wait(kRecord ? &q_ready : &q_full, seg & 1, abort, A.err);
          ++seg;
        }
        // the place (records: all but the first scale's, and that too) has been read
        ok = ok && (kRecord ? warp_wait(&e_rest, (n & 1) ^ 1, abort, A.err) : warp_wait(&s_empty[n & 1], ((n >> 1) & 1) ^ 1, abort, A.err));
        uint32_t d = kRecord ? kSCol : kSCol + (n & 1) * 2 * kPage + half * kPage;
        if (half == 0) {
          ok = ok && warp_wait(&rope_full[rope.at], rope.ph, abort, A.err);
          if (!ok) break;
          tc_fence_after();
          if (issuer) {
            const uint64_t kd = desc_add(dr, rope.at * kRopeBytes), qd = desc_add(dq, 8 * N * 128);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ss(d, desc_add(qd, k * 32), desc_add(kd, k * 32), idesc_rope, k != 0);
            mma_commit(smem_u32(&rope_empty[rope.at]));
          }
          __syncwarp();
          rope.step(1);
        }
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
          const int j = half + 2 * i;
          if (kRecord) {                          // each scale's scores go to a place of their own
            d = kSCol + ((j + 1) & 3) * kPage;
            if (j == 3) ok = warp_wait(&e_front, n & 1, abort, A.err);
          }
          ok = ok && warp_wait(&pair_full[pair.at], pair.ph, abort, A.err);
          if (!ok) break;
          tc_fence_after();
          if (issuer) {
            const uint64_t kd = desc_add(dk, pair.at * kPairBytes), qd = desc_add(dq, 2 * j * N * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16_ss(d, desc_add(qd, (k >> 2) * N * 128 + (k & 3) * 32),
                         desc_add(kd, (k >> 2) * (kPage * 128) + (k & 3) * 32), idesc, kRecord || (half && i == 0) ? k != 0 : 1);
            if (kRecord) mma_commit(smem_u32(j == 0 ? &f_front : j == 3 ? &f_last : &f_mid));
            else if (i == 1) mma_commit(smem_u32(&s_full[n & 1]));
            if (i == 1 && (flags & kLast)) mma_commit(smem_u32(&q_free));
          }
          __syncwarp();
          pair.step(2);
        }
      }
    } else {
      constexpr uint32_t idesc = make_idesc(128, N, kFmt, kFmt, 1, 0);
      const uint64_t dv = smem_desc(smem_u32(pair_buf), kPage * 128, 1024, kSwizzle128B);
      const uint64_t dp = smem_desc(smem_u32(p_buf), 0, 1024, kSwizzle128B);
      constexpr int kStep = S::kValueWarps;       // a warp's pairs: half and every kStep-th from there
      Ring<S::kPairs> pair(half);
      for (int n = 0, flags = 0; ok && !(flags & kEnd); ++n) {
        const int us = n % kUnits;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        flags = s_unit[us].flags;
        if (flags & kStop) break;
        const uint32_t kept = flags & kFirst ? 0u : 1u;
        // pairs j, j + kStep, .. below `to` (P is behind the scores, and so behind the pairs' arrival)
        auto values = [&](int j, int to, uint64_t* bar) {
          ok = ok && warp_wait(bar, n & 1, abort, A.err);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j + i * kStep >= to) break;
            if (issuer) {
              const int jj = j + i * kStep;
              const uint64_t vd = desc_add(dv, pair.at * kPairBytes), pd = desc_add(dp, kRecord ? jj % 3 * S::kPBytes : 0);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_ss(jj * N, desc_add(vd, k * 2048), desc_add(pd, k * 32), idesc, k != 0 ? 1u : kept);
              mma_commit(smem_u32(&pair_empty[pair.at]));
              if (kRecord && jj == 0) mma_commit(smem_u32(&p_used)), mma_commit(smem_u32(&f_front));
              if (jj + kStep >= 4) mma_commit(smem_u32(&o_done[n & 1]));
              if (kRecord && jj == 3) mma_commit(smem_u32(&f_last));
            }
            pair.step(kStep);
          }
          __syncwarp();
        };
        if constexpr (kRecord) {
          if (n == 0 && lane == 0) {              // (no page before it)
            mbar_arrive(smem_u32(&f_front));
            mbar_arrive(smem_u32(&f_last));
          }
          values(0, 1, &p_front);
          values(1, 3, &p_mid);
          values(3, 4, &p_last);
        } else {
          values(half, 4, &p_full);
        }
      }
    }
    // Everything issued has finished before tensor and shared memory are given back.
    __syncwarp();
    if (issuer) {
      const uint32_t bar = smem_u32(&drain[warp - kScoreWarp0]);
      mma_commit(bar);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar, 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort = 1;
          record_error(A.err, kDevTimeout);
          break;
        }
      }
    }
    __syncwarp();
  } else if (warp >= kFixWarp0) {
    const int ct = tid - 32 * kFixWarp0;
    if constexpr (kRecord) {
      // ---------------------------------------------------------- conversion
      // (half of the warps take every other pair: what a pair waits for is not what the next does)
      const int group = ct / (16 * S::kFixWarps), gt = ct % (16 * S::kFixWarps);
      Ring<S::kPairs> pair(group);
      Ring<S::kCodes> code(group);
      bool ok = true;
      for (int n = 0, flags = 0; ok && !(flags & kEnd); ++n) {
        const int us = n % kUnits;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        flags = s_unit[us].flags;
        if (flags & kStop) break;
        const bool edge = (flags & kEdge) != 0;
        const int last = s_unit[us].last;
        // Each key's largest scale, for the weights' reference. In a page not seen whole: scales of keys that no
        // row sees become 0, and so do those of a key with a NaN or infinity, which is noted.
        ok = warp_wait(&scale_full[n % kScaleSlots], (n / kScaleSlots) & 1, abort, A.err);
        if (!ok) break;
        if (ct < kPage) {                         // (of the first group, before its first pair is there)
          float4* at = reinterpret_cast<float4*>(scale_buf) + (n % kScaleSlots) * kPage + ct;
          const float4 c = *at;
          const float top = fmaxf(max3(fabsf(c.x), fabsf(c.y), fabsf(c.z)), fabsf(c.w));
          if (edge) {
            const bool bad = !(fabsf(c.x) + fabsf(c.y) + fabsf(c.z) + fabsf(c.w) < INFINITY);
            if (bad && ct <= last) atomicOr(&s_bad[us][ct >> 5], 1u << (ct & 31));
            if (bad || ct > last) *at = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          // (2^-88 at least: all four may be 0. A weight is then below 2^(88 + kLift + kMove) = 2^103, and
          // 2^25 of them in a run's sum below 2^128.)
          s_lg[us][ct] = lg2(fmaxf(top, 3.2311743e-27f));
        }
        // eight codes a thread and round: half a warp reads a row's 128, and eight threads write a row of an atom
        constexpr int kRounds = kPage * 16 / (16 * S::kFixWarps), kRows = S::kFixWarps;
        const int row = gt >> 4, ch = gt & 15;
        const int from = row * 128 + ch * 8, to = (ch >> 3) * (kPage * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        static_assert(kRows % 8 == 0, "rows of a round have the swizzle of the first");
#pragma unroll 1
        for (int j = group; j < 4; j += 2) {
          ok = warp_wait(&code_full[code.at], code.ph, abort, A.err) && warp_wait(&pair_empty[pair.at], pair.ph ^ 1, abort, A.err);
          if (!ok) break;
          const uint8_t* src = code_buf + code.at * kCodeStage + from;
          uint8_t* dst = pair_buf + pair.at * kPairBytes + to;
          uint2 w[kRounds];
#pragma unroll
          for (int i = 0; i < kRounds; ++i) w[i] = *reinterpret_cast<const uint2*>(src + i * kRows * 128);
          if (KV == kKvE4m3 && edge) {
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
              const uint32_t b0 = __vcmpeq4(w[i].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), b1 = __vcmpeq4(w[i].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              const int key = row + i * kRows;
              if ((b0 | b1) && key <= last) atomicOr(&s_bad[us][key >> 5], 1u << (key & 31));
              w[i].x &= ~b0, w[i].y &= ~b1;
            }
          }
#pragma unroll
          for (int i = 0; i < kRounds; ++i) {
            uint4 o;
            codes_f16<KV == kKvInt8>(w[i].x, o.x, o.y);
            codes_f16<KV == kKvInt8>(w[i].y, o.z, o.w);
            *reinterpret_cast<uint4*>(dst + i * kRows * 128) = o;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&pair_full[pair.at]));
            mbar_arrive(smem_u32(&code_empty[code.at]));
            if (j >= 2) mbar_arrive(smem_u32(&u_empty[us]));
          }
          pair.step(2);
          code.step(2);
        }
      }
    } else {
      // ---------------------------------------------------------- pages not seen whole
      int pair = 0, edges = 0;
      uint32_t pair_ph = 0;
      bool ok = true;
      for (int n = 0, flags = 0; ok && !(flags & kEnd); ++n) {
        const int us = n % kUnits;
        ok = warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        flags = s_unit[us].flags;
        if (flags & kStop) break;
        const bool edge = (flags & kEdge) != 0;
        // (once the unit's loads have been issued, its slots' barriers are in its phase)
        ok = warp_wait(&u_loaded[us], (n / kUnits) & 1, abort, A.err);
        if (!ok) break;
        const int last = s_unit[us].last;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          if (edge) {
            ok = ok && warp_wait(&pair_full[pair], pair_ph, abort, A.err);
            if (!ok) break;
            uint4* at = reinterpret_cast<uint4*>(pair_buf + pair * kPairBytes);
            // (a row's eight chunks of an atom by eight threads: the swizzle permutes within the row)
            constexpr int kChunks = kPage * 8, kStep = 32 * S::kFixWarps;
            for (int i = 8 * (last + 1) + ct; i < kChunks; i += kStep) at[i] = at[kChunks + i] = make_uint4(0, 0, 0, 0);
            // where all rows see the same keys, the others may do as they like
            if (flags & kMixed) {
              for (int i = ct; i < 8 * (last + 1); i += kStep) {
                const uint4 v[2] = {at[i], at[kChunks + i]};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t o[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
                  bool bad = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) bad |= (o[e] & 0x7F80u) == 0x7F80u || (o[e] & 0x7F800000u) == 0x7F800000u;
                  if (bad) {
                    atomicOr(&s_bad[us][i >> 8], 1u << (i >> 3 & 31));
                    at[h * kChunks + i] = make_uint4(0, 0, 0, 0);
                  }
                }
              }
            }
          }
          if (++pair == S::kPairs) pair = 0, pair_ph ^= 1u;
        }
        if (!ok) break;
        if (edge) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (edge) mbar_arrive(smem_u32(&e_full[edges % kUnits]));
          mbar_arrive(smem_u32(&u_empty[us]));
        }
        if (edge) ++edges;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int w4 = warp & 3, half = warp >> 2;    // lane quarter; keys 32 * half and on
    const bool active = 16 * w4 < N;
    const uint32_t quarter = tmem + ((uint32_t)(32 * w4) << 16);
    const int r0 = 16 * w4 + (lane >> 2);         // this thread's rows: r0 and r0 + 8
    const int key0 = 32 * half + 2 * (lane & 3);  // and keys: key0 + 8 j and the next, j < 4
    const float f = fmaxf(A.scale_log2, 1.17549435e-38f);   // (a scale of 0 would make masked scores NaN)
    float M[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
    float qf[2], up[2];                           // records: factors of the rows' scores, and of the rotated part's to theirs
    uint32_t seg = 0;
    int edges = 0;
    bool ok = true;
    // Records: the rotated part's scores and the first scale's, of page n (both by the first issuer, so
    // the second are behind the first; the scales are there, and as the conversion leaves them).
    float early[kRecord ? 16 : 1];
    bool ahead = false;                           // they have been read
    auto front = [&](int n) {
      if constexpr (kRecord) {
        ok = ok && warp_wait(&f_front, n & 1, abort, A.err);
        if (!ok) return;
        float t[2][16], c[8];
        tc_fence_after();
        tmem_ld_16x32(quarter + kSCol + 32 * half, t[0]);
        tmem_ld_16x32(quarter + kSCol + kPage + 32 * half, t[1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = scale_buf[((n % kScaleSlots) * kPage + key0 + 8 * (j >> 1) + (j & 1)) * 4];
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&e_front));
#pragma unroll
        for (int j = 0; j < 16; ++j) early[j] = fmaf(t[1][j], c[2 * (j >> 2) + (j & 1)], t[0][j] * up[j >> 1 & 1]);
      }
    };
    for (int n = 0;; ++n) {
      const int us = n % kUnits;
      ok = ok && (ahead || warp_wait(&u_full[us], (n / kUnits) & 1, abort, A.err));
      LatentUnit x{};
      if (ok) x = s_unit[us];
      if (x.flags & kFirst) {
        M[0] = M[1] = kNone, l[0] = l[1] = 0.f;
        if constexpr (kRecord) {
          ok = ok && warp_wait(&q_full, seg & 1, abort, A.err);
          if (ok) queries_f16<N>(q_buf, tid, s_qf);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(smem_u32(&q_ready));
          ok = ok && warp_wait(&q_ready, seg++ & 1, abort, A.err);
          if (active) {
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[i] = s_qf[r0 + 8 * i], up[i] = __frcp_rn(qf[i]), qf[i] *= f;
          }
        }
      }
      float s[16], lg[8] = {};                    // lg: records, logarithms of the keys' largest scales
      const float* scales = scale_buf + ((n % kScaleSlots) * kPage + key0) * 4;   // of this thread's keys
      // (warps without rows do not look at the scores' barriers, which may be two pages ahead of them)
      if (!active || (x.flags & kStop)) {
      } else if constexpr (!kRecord) {
        ok = ok && warp_wait(&s_full[n & 1], (n >> 1) & 1, abort, A.err);
        if (ok) {
          float t[16];
          tc_fence_after();
          tmem_ld_16x32(quarter + kSCol + (n & 1) * 2 * kPage + 32 * half, s);
          tmem_ld_16x32(quarter + kSCol + (n & 1) * 2 * kPage + kPage + 32 * half, t);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_empty[n & 1]));
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] += t[j];
        }
      } else {
        if (!ahead) front(n);
        // the next two scales', then the last one's, before whose arrival the rest is at hand: the chain of
        // a page is values -> conversion of its last pairs -> their scores -> from here to the weights
        auto more = [&](int g, const float (&t)[16], const float (&c)[8]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = fmaf(t[j], c[2 * (j >> 2) + (j & 1)], g == 1 ? early[j] : s[j]);
        };
        auto scale = [&](int g, float (&c)[8]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) c[j] = scales[4 * (8 * (j >> 1) + (j & 1)) + g];
        };
        float t[16], c[8];
        ok = ok && warp_wait(&f_mid, n & 1, abort, A.err);
        if (ok) {
          float u[16], d[8];
          tc_fence_after();
          tmem_ld_16x32(quarter + kSCol + 2 * kPage + 32 * half, t);
          tmem_ld_16x32(quarter + kSCol + 3 * kPage + 32 * half, u);
          scale(1, c);
          scale(2, d);
          tmem_ld_wait();
          more(1, t, c);
          more(2, u, d);
          scale(3, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = *reinterpret_cast<const float2*>(&s_lg[us][key0 + 8 * j]);
            lg[2 * j] = v.x, lg[2 * j + 1] = v.y;
          }
        }
        ok = ok && warp_wait(&f_last, n & 1, abort, A.err);
        if (ok) {
          tc_fence_after();
          tmem_ld_16x32(quarter + kSCol + 32 * half, t);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&e_rest));
          more(3, t, c);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] *= qf[j >> 1 & 1];    // in powers of two
        }
      }
      bool need = false;
      if (active && ok && !(x.flags & kStop)) {
        if (x.flags & kEdge) {
          // bf16: what rows that do not see them must not meet has left the values (the scores need no
          // waiting: those of such keys are replaced here). Records: the conversion has done it.
          if (!kRecord) ok = warp_wait(&e_full[edges % kUnits], (edges / kUnits) & 1, abort, A.err);
          const uint64_t bad = (uint64_t)s_bad[us][0] | (uint64_t)s_bad[us][1] << 32;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = r0 + 8 * i;
            const int lim = row < x.rows && !(x.flags & kVoid) ? x.rel + (x.row0 + row) / A.H : -1;   // last key that it sees
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + 8 * j + e;
                float& v = s[4 * j + 2 * i + e];
                if (key > lim) v = -INFINITY;
                else if (bad >> key & 1) v = NAN;
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (kRecord) m = max3(m, s[4 * j + 2 * i] + lg[2 * j], s[4 * j + 2 * i + 1] + lg[2 * j + 1]);
            else m = max3(m, s[4 * j + 2 * i], s[4 * j + 2 * i + 1]);
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (!kRecord) m *= f;
          if ((lane & 3) == 0) s_top[half][r0 + 8 * i] = m;
          need |= r0 + 8 * i < x.rows && m - kLift > M[i] + kMove;
        }
      }
      if (x.flags & kEdge) ++edges;
      // The reference moves. (All eight warps come here in every round, those that gave up too;
      // an item's first unit comes here whether or not a row sees a key of it.)
      if (bar_any(1, 32 * kSoftWarps, need || !ok || (x.flags & kFirst))) {
        if (active && ok && !(x.flags & kStop)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m = fmaxf(s_top[0][r0 + 8 * i], s_top[1][r0 + 8 * i]) - kLift;
            float keep = 1.f;
            if (x.flags & kFirst) M[i] = fmaxf(m, kNone);
            else if (m > M[i] + kMove) keep = ex2(M[i] - m), M[i] = m, l[i] *= keep;
            if (half == 0 && (lane & 3) == 0) s_keep[r0 + 8 * i] = keep;
          }
        }
        if (!bar_all(1, 32 * kSoftWarps, ok)) break;
        if (!(x.flags & (kFirst | kStop))) {      // O so far, once its last product is done
          ok = warp_wait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort, A.err);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 2 * N * half; k < 2 * N * (half + 1); k += 16) {
              float v[16];
              tmem_ld16(quarter + k, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] *= s_keep[(k + j) % N];
              tmem_st16(quarter + k, v);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          // (records: warps without rows hand over no weights, so the others wait for theirs)
          if (kRecord && N < 64 && !bar_all(1, 32 * kSoftWarps, ok)) break;
        }
      }
      if (x.flags & kStop) break;
      if (active && ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a = 0.f, b = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float &u = s[4 * j + 2 * i], &w = s[4 * j + 2 * i + 1];
            u = ex2(kRecord ? u - M[i] : fmaf(u, f, -M[i])), w = ex2(kRecord ? w - M[i] : fmaf(w, f, -M[i]));
            a += u, b += w;
          }
          l[i] += a + b;
        }
      }
      // this lane's row of a 16 x 32 piece's four 8 x 8 matrices (stored with rows r0 of all, then r0 + 8)
      const uint32_t p_row = smem_u32(p_buf) + (16 * w4 + (lane & 7)) * 128 + (((4 * half + (lane >> 3)) ^ (lane & 7)) << 4);
      if constexpr (!kRecord) {
        // the last page's values have left P's place
        if (n > 0) ok = ok && warp_wait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort, A.err);
        if (active && ok) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            store_matrices(p_row + i * 1024, pack_bf16(s[2 * i], s[2 * i + 1]), pack_bf16(s[4 + 2 * i], s[5 + 2 * i]),
                           pack_bf16(s[8 + 2 * i], s[9 + 2 * i]), pack_bf16(s[12 + 2 * i], s[13 + 2 * i]));
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&p_full));
      } else if (active) {
        // each scale's codes get its weights
        auto weights = [&](int g) {
          float v[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float c = scales[4 * (8 * (k >> 1) + (k & 1)) + g];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int j = 4 * (k >> 1) + 2 * i + (k & 1);
              v[j] = s[j] * c;
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            store_matrices(p_row + g % 3 * S::kPBytes + i * 1024, pack_weights(v[2 * i], v[2 * i + 1]),
                           pack_weights(v[4 + 2 * i], v[5 + 2 * i]), pack_weights(v[8 + 2 * i], v[9 + 2 * i]),
                           pack_weights(v[12 + 2 * i], v[13 + 2 * i]));
        };
        auto hand_over = [&](uint64_t* bar) {
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(bar));
        };
        if (ok) {
          weights(0);
          hand_over(&p_front);
          weights(1);
          weights(2);
          hand_over(&p_mid);
        }
        // While their values are on the way: the next page's first scores, whose place its last ones
        // need. (Not of another item, whose queries these warps have yet to convert.)
        ahead = ok && !(x.flags & kLast);
        if (ahead) front(n + 1);                  // (which waits for the first weights' use as well)
        else ok = ok && warp_wait(&p_used, n & 1, abort, A.err);
        if (ok) {
          weights(3);
          hand_over(&p_last);
        }
      }
      if (x.flags & kLast) {
        // ---- the segment's outputs, or its part
        if (active && ok) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if ((lane & 3) == 0) s_sum[half][r0 + 8 * i] = l[i];
          }
        }
        if (!bar_all(1, 32 * kSoftWarps, ok)) break;
        if (tid < N) {                            // (keep is for the next rescaling: now the sums' reciprocals)
          const float sum = s_sum[0][tid] + s_sum[1][tid];
          s_keep[tid] = sum == 0.f ? 0.f : 1.f / sum;
        }
        if (!bar_all(1, 32 * kSoftWarps, ok)) break;
        // (two barriers, for a warp may come here before unit n - 1's values are done or after unit n's)
        ok = warp_wait(&o_done[n & 1], (n >> 1) & 1, abort, A.err);
        if (ok) {
          tc_fence_after();
          const int t = w4 * 32 + lane;
          if (half == 0 && active && (lane & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = r0 + 8 * i;
              const float sum = s_sum[0][row] + s_sum[1][row];
              if (row >= x.rows) continue;
              if (x.slot >= 0) *reinterpret_cast<float2*>(parts.ml + ((int64_t)x.slot * R + N * rank + row) * 2) = make_float2(M[i], sum);
              else if (A.lse) A.lse[x.out + row] = sum == 0.f ? -INFINITY : (M[i] + log2f(sum)) * 0.6931471805599453f;
            }
          }
          constexpr int kCols = N == 16 ? 16 : 32;  // at a time: each look at tensor memory is waited for
#pragma unroll 1
          for (int k = 2 * N * half; k < 2 * N * (half + 1); k += kCols) {
            float v[kCols];
            if constexpr (kCols == 16) tmem_ld16(quarter + k, v);
            else tmem_ld32(quarter + k, v);
            tmem_ld_wait();
            const int dim = k / N * 128 + t, row = k % N;
            // (rows all in use as a case of its own: 16 branches a look at tensor memory otherwise)
            auto part = [&](auto used) {
              float* dst = parts.o + ((int64_t)x.slot * R + N * rank + row) * kDimLatent + dim;
#pragma unroll
              for (int j = 0; j < kCols; ++j)
                if (used(j)) dst[(int64_t)j * kDimLatent] = v[j];
            };
            auto output = [&](auto used) {
              // neighbouring lanes share two rows: the even one writes both columns of the first
              __nv_bfloat16* dst = A.out + (x.out + row + (lane & 1)) * kDimLatent + (dim & ~1);
#pragma unroll
              for (int j = 0; j < kCols; j += 4) {
                // (a row that saw nothing has zeros in O as well: all its weights were 0)
                const float4 inv = *reinterpret_cast<const float4*>(&s_keep[row + j]);
                const float w[4] = {v[j] * inv.x, v[j + 1] * inv.y, v[j + 2] * inv.z, v[j + 3] * inv.w};
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                  const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? w[i] : w[i + 1], 1);
                  const uint32_t two = lane & 1 ? pack_bf16(other, w[i + 1]) : pack_bf16(w[i], other);
                  if (used(j + i + (lane & 1))) *reinterpret_cast<uint32_t*>(dst + (int64_t)(j + i) * kDimLatent) = two;
                }
              }
            };
            auto some = [&](int j) { return row + j < x.rows; };
            auto all = [](int) { return true; };
            const bool whole = row + kCols <= x.rows;
            if (x.slot >= 0) whole ? part(all) : part(some);
            else whole ? output(all) : output(some);
          }
          tc_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&u_empty[us]));
      // (past the round's vote all eight warps know the unit, and so leave together)
      if (x.flags & kEnd) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// Query rows of an item: as many as a request has in the mean, up to 64 (more rows a page read).
int latent_rows(const GeomDev& g, int H) {
  const int64_t rows = ((int64_t)g.T + g.B - 1) / g.B * H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Whether two items of a request go to two neighbouring blocks: where it has just two in the mean. (64 requests
// of 128 rows over 5000 keys 129.5 us, without 143; 40 of 80 rows over 6750 108 and 118; 32 of 128 over 2250 43 and
// 44; 8 over 3000 28 and 27; a single one over 30000 50 and 39.5, for its parts are merged by fewer blocks. With more
// rows the other items are mostly found in L2, and an odd one leaves half of a run idle: 40 of 192 rows over 6750 200
// and 167.5; 16 of 192 over 3000 51 and 44.5; 8 of 256 over 3000 35 and 34; but 64 of 256 over 6100 279 and 302.)
bool latent_pairs(const GeomDev& g, int H) {
  const int64_t rows = ((int64_t)g.T + g.B - 1) / g.B * H;
  return rows > 64 && rows <= 128;
}

template <int N, int KV, int BL>
cudaError_t launch(const LatentAttendArgs& A, const LatentMaps& m, int num_sms, cudaStream_t st) {
  using S = LatentShape<N, KV>;
  const int runs = num_sms / BL;
  const LatentParts parts = latent_parts(A.scratch, runs, BL * N, kDimLatent);
  auto kern = latent_attend_kernel<N, KV, BL>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  kern<<<runs * BL, S::kThreads, S::kSmem, st>>>(m.q, m.pair, m.rope, A, parts);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : latent_merge_launch<kDimLatent>(parts, runs, A.out, A.lse, st);
}
template <int KV>
cudaError_t launch_rows(const LatentAttendArgs& A, const LatentMaps& m, int num_sms, cudaStream_t st) {
  switch (latent_rows(A.g, A.H)) {
    case 16: return launch<16, KV, 1>(A, m, num_sms, st);
    case 32: return launch<32, KV, 1>(A, m, num_sms, st);
    default:
      if constexpr (KV == kKvBf16) {
        if (latent_pairs(A.g, A.H) && num_sms > 1) return launch<64, KV, 2>(A, m, num_sms, st);
      }
      return launch<64, KV, 1>(A, m, num_sms, st);
  }
}

}  // namespace

int latent_attend_rows(const GeomDev& g, int H) { return latent_rows(g, H); }

// Enough for any smaller T as well: a buffer sized for a batch's largest step serves its others.
size_t latent_attend_scratch_bytes(const dsa_geom_t* g, int H, int num_sms) {
  GeomDev gd{};
  gd.B = g->B, gd.T = g->T;
  return latent_parts_bytes(num_sms, latent_rows(gd, H), kDimLatent);
}

cudaError_t latent_attend_launch(const LatentAttendArgs& A, const LatentMaps& m, int num_sms, cudaStream_t st) {
  switch (A.kv_format) {
    case kKvBf16: return launch_rows<kKvBf16>(A, m, num_sms, st);
    case kKvE4m3: return launch_rows<kKvE4m3>(A, m, num_sms, st);
    default: return launch_rows<kKvInt8>(A, m, num_sms, st);
  }
}

}  // namespace dsa
