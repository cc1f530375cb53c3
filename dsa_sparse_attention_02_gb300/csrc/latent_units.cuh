// Units of the dense absorbed attention (latent_attend.cu): an item is (request, N of its tokens x
// heads), a unit a page of 64 keys that some row of the item sees. All units are laid end to end
// and cut into runs of equal cost.
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
  r.tiles = (r.n * A.H + N - 1) / N;      // (T * H <= 2^31 - 128)
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

// Finds the units of run `id` of `grid` (a block's, or that of two neighbours); whole warp, which keeps up to 32 units at a time, one a lane.
// Runs are equal in cost: an item's units, and COST for it (its queries, and its outputs, which no
// product hides).
template <int N, int COST>
struct LatentCursor {
  const LatentAttendArgs& A;
  const LatentParts& parts;
  const int id, grid;
  const bool writer;                         // reports, and notes the run's cut item
  int64_t begin = 0, end = 0, total = 0;     // the run's units; the cost of all
  int runs = 1;
  // Of the next batch's first unit: request, tile and page, and the item's number among all.
  struct Place {
    LatentReq r;
    int b, ti, c;
    int64_t item;
  } p{};
  LatentUnit x{};                            // the batch: this lane's unit and its page
  int page = -1, cnt = 0, at = 0;

  __device__ __forceinline__ LatentCursor(const LatentAttendArgs& args, const LatentParts& parts_, int id_, int grid_, bool writer_)
      : A(args), parts(parts_), id(id_), grid(grid_), writer(writer_) {}

  // Finds the run. (What the requests say is read once where there are 32 at most: each look takes
  // half a microsecond, before which no load of a page can begin.)
  __device__ __forceinline__ void find() {
    const int lane = threadIdx.x & 31;
    LatentReq front{};                       // of request b0 + lane
    int64_t units_of = 0;
    auto look = [&](int b0) {
      front = LatentReq{};
      units_of = 0;
      if (b0 + lane < A.g.B) {
        front = latent_req<N>(A, b0 + lane);
        units_of = latent_before<N>(A, front, front.tiles);
      }
    };
    for (int b0 = (A.g.B - 1) / 32 * 32; b0 >= 0; b0 -= 32) {      // (the first ones stay)
      look(b0);
      total += units_of + (int64_t)COST * front.tiles;
      if (front.bad && id == 0 && writer) record_error(A.err, kDevBadIndex);
    }
    if (lane == 0 && writer) parts.cuts[id].follow = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    runs = (int)min((int64_t)grid, max(total, (int64_t)1));
    if (id >= runs || total == 0) return;
    const int64_t lo = run_begin(id, total, runs), hi = run_begin(id + 1, total, runs);
    int64_t units = 0, items = 0;                                  // of the requests before b0
    bool found = false;
    end = -1;
    for (int b0 = 0; b0 < A.g.B && end < 0; b0 += 32) {
      if (b0 > 0) look(b0);
      int64_t up = units_of;
      int it = front.tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
        const int i = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) up += v, it += i;
      }
      const int64_t cost = units + up + COST * (items + it);       // up to this lane's request, with it
      // the unit at cost `to`, or the first behind it: its number, and where it is
      auto locate = [&](int64_t to, int l, Place& k) {
        LatentReq& r = k.r;
        r.q0 = __shfl_sync(0xffffffffu, front.q0, l), r.n = __shfl_sync(0xffffffffu, front.n, l);
        r.start = __shfl_sync(0xffffffffu, front.start, l), r.tiles = __shfl_sync(0xffffffffu, front.tiles, l);
        r.bad = __shfl_sync(0xffffffffu, front.bad, l), r.none = __shfl_sync(0xffffffffu, front.none, l);
        const int64_t u0 = units + __shfl_sync(0xffffffffu, up - units_of, l);
        const int64_t i0 = items + __shfl_sync(0xffffffffu, it - front.tiles, l);
        const int64_t o = to - u0 - COST * i0;
        int lo = 0, hi = r.tiles - 1;                              // the last tile that begins at `to` or before it
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (latent_before<N>(A, r, mid) + (int64_t)COST * mid <= o) lo = mid; else hi = mid - 1;
        }
        const int64_t before = latent_before<N>(A, r, lo);
        k.b = b0 + l;
        k.ti = lo;
        k.c = (int)max(o - before - (int64_t)COST * (lo + 1), (int64_t)0);
        k.item = i0 + lo;
        return u0 + before + k.c;
      };
      const unsigned m_lo = __ballot_sync(0xffffffffu, cost > lo), m_hi = __ballot_sync(0xffffffffu, cost > hi);
      if (!found && m_lo) begin = locate(lo, __ffs(m_lo) - 1, p), found = true;
      Place behind;
      if (m_hi) end = locate(hi, __ffs(m_hi) - 1, behind);
      units += __shfl_sync(0xffffffffu, up, 31), items += __shfl_sync(0xffffffffu, it, 31);
    }
    if (end < 0) end = units;                                      // (the last run)
  }

  __device__ __forceinline__ void turn(Place& k) const {   // to the item behind this one
    ++k.item;
    if (++k.ti < k.r.tiles) return;
    k.ti = 0;
    do k.r = latent_req<N>(A, ++k.b);
    while (k.r.tiles == 0 && k.b + 1 < A.g.B);
  }

  __device__ __forceinline__ void batch(int64_t u) {
    const int lane = threadIdx.x & 31;
    cnt = (int)min((int64_t)32, end - u);
    Place k = p;
    int units = latent_units<N>(A, k.r, k.ti);
    for (int step = lane; step > 0 && lane < cnt;) {            // forward by `lane` units
      const int left = units - k.c;
      if (step < left) {
        k.c += step;
        break;
      }
      step -= left;
      k.c = 0;
      turn(k);
      units = latent_units<N>(A, k.r, k.ti);
    }
    __syncwarp();
    if (lane < cnt) {
      const int64_t me = u + lane, ib = me - k.c, ie = ib + units;
      x.row0 = k.ti * N;
      x.rows = min(N, k.r.n * A.H - x.row0);
      x.out = (int64_t)k.r.q0 * A.H + x.row0;
      x.rel = k.r.start - k.c * kPage;
      const int lo = (uint32_t)x.row0 / (uint32_t)A.H, hi = (uint32_t)(x.row0 + x.rows - 1) / (uint32_t)A.H;
      page = -1;
      if (!k.r.none && x.rel + hi >= 0) {
        page = gqa_page(A.g, k.b, k.c);
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
        LatentCut w{};
        // (the last unit's cost: the units before it, and its item and those before)
        w.follow = (int)run_owner(ie - 1 + COST * (k.item + 1), total, runs) - id;
        w.slot = x.slot, w.rows = x.rows, w.step = 1, w.out = x.out;
        parts.cuts[id] = w;
      }
    }
    at = 0;
    if (u + cnt == end) return;
    // the cursor behind the batch: its last lane's unit, one further
    const int l = cnt - 1;
    p.b = __shfl_sync(0xffffffffu, k.b, l), p.ti = __shfl_sync(0xffffffffu, k.ti, l);
    p.c = __shfl_sync(0xffffffffu, k.c, l) + 1, p.item = __shfl_sync(0xffffffffu, k.item, l);
    p.r = latent_req<N>(A, p.b);
    if (p.c == latent_units<N>(A, p.r, p.ti)) {
      p.c = 0;
      turn(p);
    }
  }
};

}  // namespace dsa
