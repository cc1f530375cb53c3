// Units of the dense absorbed attention (latent_attend.cu, latent_cluster.cu): an item is (request,
// N of its tokens x heads), a unit a page of 64 keys that some row of the item sees. All units are
// laid end to end and cut into equal runs.
#pragma once
#include "latent_common.cuh"

namespace dsa {

constexpr int kUnits = 4;                    // units described ahead
constexpr int kPairBytes = 2 * kPage * 128;  // two atoms of 64 rows x 64 bf16: 128 latent columns of a page
constexpr int kRopeBytes = kPage * 128;
constexpr int kCodeStage = kPage * 128;      // a pair's codes
constexpr int kScaleSlots = 4;
constexpr uint32_t kTmem = 512;
// Beside first, last and void: some row of the item does not see the whole page; the run's last
// unit; a run without units (nothing in it to do); a key that some rows see and others do not.
enum : int { kEdge = 8, kEnd = 16, kStop = 32, kMixed = 64 };

struct __align__(16) LatentUnit {
  int flags, rel;       // position of token 0 less the page's first position
  int row0, rows;       // first row of the item in its request (token row / H, head row % H); rows in use
  int slot, last;       // partial slot or -1; last key of the page that some row sees, or -1
  int64_t out;          // global number of the item's first row
};

// Requests as the items see them.
struct LatentReq {
  int q0, n, start;      // first token, tokens, position of the first (may be negative)
  int tiles;
  bool bad, none;        // none: nothing visible (inconsistent geometry)
};
template <int N>
__device__ __forceinline__ LatentReq latent_req(const LatentAttendArgs& A, int b) {
  LatentReq r;
  const int c0 = __ldg(A.g.cu_q + b), c1 = __ldg(A.g.cu_q + b + 1), len = __ldg(A.g.seq_lens + b);
  r.bad = c0 < 0 || c1 < c0 || c1 > A.g.T || len > A.g.max_seq_len;
  r.q0 = min(max(c0, 0), A.g.T);
  r.n = max(min(c1, A.g.T) - r.q0, 0);
  r.none = r.bad || len <= 0;
  r.start = len - r.n;
  r.tiles = (r.n * A.H + N - 1) / N;      // (T * H stays below 2^31)
  return r;
}
// Pages that tile i's last token sees; at least one unit, so that empty rows are written too.
template <int N>
__device__ __forceinline__ int latent_units(const LatentAttendArgs& A, const LatentReq& r, int i) {
  if (r.none) return 1;
  const int last = min((uint32_t)(r.n - 1), ((uint32_t)i * N + N - 1) / (uint32_t)A.H);
  return max(r.start + last, 0) / kPage + 1;
}
// Units of tiles 0 .. i - 1: tile j sees page k if its last token reaches position 64 k, which
// tiles from (64 k - start) H / N on do.
template <int N>
__device__ __forceinline__ int64_t latent_before(const LatentAttendArgs& A, const LatentReq& r, int i) {
  if (r.none || i <= 0) return i;
  const int k0 = max(r.start, 0) / kPage, k1 = max(r.start + r.n - 1, 0) / kPage;
  int64_t s = (int64_t)i * (k0 + 1);
  for (int k = k0 + 1; k <= k1; ++k) s += max((int64_t)i - (int64_t)(k * kPage - r.start) * A.H / N, (int64_t)0);
  return s;
}

// Finds the units of run `id` of `grid`; whole warp, which keeps up to 32 units at a time, one a lane.
template <int N>
struct LatentCursor {
  const LatentAttendArgs& A;
  const LatentParts& parts;
  const int id;
  const bool writer;                         // notes the run's cut item
  int64_t begin = 0, end = 0, base = 0, total = 0;
  int runs = 1;
  int b = 0, ti = 0, c = 0;                  // request, tile and page of the next batch's first unit
  LatentReq r{};
  LatentUnit x{};                            // the batch: this lane's unit and its page
  int page = -1, cnt = 0, at = 0;

  __device__ __forceinline__ LatentCursor(const LatentAttendArgs& args, const LatentParts& p, int id_, bool writer_)
      : A(args), parts(p), id(id_), writer(writer_) {}

  // Finds the run. (What the requests say is read once where there are 32 at most: each look takes
  // half a microsecond, before which no load of a page can begin.)
  __device__ __forceinline__ void find(int grid) {
    const int lane = threadIdx.x & 31;
    LatentReq front{};                       // of request `lane`
    int64_t w_front = 0;
    for (int b0 = 0; b0 < A.g.B; b0 += 32) {
      if (b0 + lane < A.g.B) {
        const LatentReq q = latent_req<N>(A, b0 + lane);
        const int64_t w = latent_before<N>(A, q, q.tiles);
        if (b0 == 0) front = q, w_front = w;
        total += w;
        if (q.bad && id == 0 && writer) record_error(A.err, kDevBadIndex);
      }
    }
    if (lane == 0 && writer) parts.cuts[id].follow = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    runs = (int)min((int64_t)grid, max(total, (int64_t)1));
    if (id >= runs || total == 0) return;
    begin = run_begin(id, total, runs);
    end = run_begin(id + 1, total, runs);
    for (int b0 = 0; b0 < A.g.B; b0 += 32) {
      int64_t w = w_front;
      if (b0 > 0) {
        w = 0;
        if (b0 + lane < A.g.B) {
          front = latent_req<N>(A, b0 + lane);
          w = latent_before<N>(A, front, front.tiles);
        }
      }
      int64_t upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, base + upto > begin);
      if (m) {
        const int l = __ffs(m) - 1;
        b = b0 + l;
        base += __shfl_sync(0xffffffffu, upto - w, l);
        r.q0 = __shfl_sync(0xffffffffu, front.q0, l), r.n = __shfl_sync(0xffffffffu, front.n, l);
        r.start = __shfl_sync(0xffffffffu, front.start, l), r.tiles = __shfl_sync(0xffffffffu, front.tiles, l);
        r.bad = __shfl_sync(0xffffffffu, front.bad, l), r.none = __shfl_sync(0xffffffffu, front.none, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    // the last tile that begins at or before unit `begin`
    const int64_t o = begin - base;
    int lo = 0, hi = r.tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (latent_before<N>(A, r, mid) <= o) lo = mid; else hi = mid - 1;
    }
    ti = lo;
    c = (int)(o - latent_before<N>(A, r, lo));
  }

  __device__ __forceinline__ void turn(int& b_, int& t_, LatentReq& r_) const {   // the item behind this one
    if (++t_ < r_.tiles) return;
    t_ = 0;
    do r_ = latent_req<N>(A, ++b_);
    while (r_.tiles == 0 && b_ + 1 < A.g.B);
  }

  __device__ __forceinline__ void batch(int64_t u) {
    const int lane = threadIdx.x & 31;
    cnt = (int)min((int64_t)32, end - u);
    int bb = b, tt = ti, cc = c;
    LatentReq rr = r;
    int units = latent_units<N>(A, rr, tt);
    for (int step = lane; step > 0 && lane < cnt;) {            // forward by `lane` units
      const int left = units - cc;
      if (step < left) {
        cc += step;
        break;
      }
      step -= left;
      cc = 0;
      turn(bb, tt, rr);
      units = latent_units<N>(A, rr, tt);
    }
    __syncwarp();
    if (lane < cnt) {
      const int64_t me = u + lane, ib = me - cc, ie = ib + units;
      x.row0 = tt * N;
      x.rows = min(N, rr.n * A.H - x.row0);
      x.out = (int64_t)rr.q0 * A.H + x.row0;
      x.rel = rr.start - cc * kPage;
      const int lo = (uint32_t)x.row0 / (uint32_t)A.H, hi = (uint32_t)(x.row0 + x.rows - 1) / (uint32_t)A.H;
      page = -1;
      if (!rr.none && x.rel + hi >= 0) {
        page = gqa_page(A.g, bb, cc);
        if (page < 0) record_error(A.err, kDevBadIndex);
      }
      x.last = page >= 0 ? min(x.rel + hi, kPage - 1) : -1;
      const bool first = me == ib || me == begin, last = me + 1 == ie || me + 1 == end;
      x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (page >= 0 ? 0 : kVoid) |
                (page < 0 || x.rel + lo < kPage - 1 ? kEdge : 0) | (page >= 0 && max(x.rel + lo, -1) < x.last ? kMixed : 0) |
                (me + 1 == end ? kEnd : 0);
      const bool cut = ib < begin || ie > end;
      x.slot = !cut ? -1 : 2 * id + (max(ib, begin) == begin ? 0 : 1);
      if (last && cut && ib >= begin && writer) {
        LatentCut k{};
        k.follow = (int)run_owner(ie - 1, total, runs) - id;
        k.slot = x.slot, k.rows = x.rows, k.step = 1, k.out = x.out;
        parts.cuts[id] = k;
      }
    }
    at = 0;
    if (u + cnt == end) return;
    // the cursor behind the batch: its last lane's unit, one further
    const int l = cnt - 1;
    b = __shfl_sync(0xffffffffu, bb, l), ti = __shfl_sync(0xffffffffu, tt, l), c = __shfl_sync(0xffffffffu, cc, l) + 1;
    r = latent_req<N>(A, b);
    if (c == latent_units<N>(A, r, ti)) {
      c = 0;
      turn(b, ti, r);
    }
  }
};

}  // namespace dsa
