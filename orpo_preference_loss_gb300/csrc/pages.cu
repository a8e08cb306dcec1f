// pages.cu — beam states in shared pages (orpo_pages.h): page tables follow the beams' parents, pages are taken, copied on
// write, released and compacted.
//
// A page is free when its count of holders is 0, and free pages are always taken lowest first, so there is no list of free
// pages to keep and no order for atomics to change: counts are integers, and every choice follows the order of rows,
// columns and page numbers.
//
// The plans (which page goes where) touch a few kilobytes: they are bound by the way to memory and back, which each step of
// "length, parent, table entry, count of holders, free page" takes once, and by barriers.  So a decode step's plan is one CTA that
// takes those ways twice (captured in a graph: 4 beams, 100 pages 3.8 us; 16 x 8 beams, 3000 pages about 8), larger ones a cluster of 8
// CTAs that tell each other sums through shared memory (64 prompts of up to 512 pages into 164k pages: 16).  The copies are
// bound by the bytes moved: 1.06 GB in 161 us, 97% of the rate of a plain copy.
#include <algorithm>

#include "../../include/orpo_pages.h"
#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

struct TableArgs {
  int32_t* table;
  int64_t ld, columns;
  int32_t* refs;
  int32_t pages, page;
  const int32_t* parent;
  int64_t ld_parent;
  const int32_t* length;
  const int32_t* more;
  int32_t most;
  int64_t batch;
  int beams;
  int32_t* status;
};

__device__ __forceinline__ bool is_page(const TableArgs& a, int32_t e) { return e >= 0 && e < a.pages; }

// Positions [begin, end) that entry b asks for; false where they are out of range.
__device__ __forceinline__ bool wanted(const TableArgs& a, int64_t b, int64_t& begin, int64_t& end) {
  begin = a.length[b];
  const int64_t more = a.more ? (int64_t)a.more[b] : a.most;
  end = begin + more;
  return begin >= 0 && more >= 0 && more <= a.most && end <= a.columns * a.page;
}

// ------------------------------------------------------------------ fork
// One thread owns a column of all rows of an entry and reads it whole before it writes.  A row that keeps its page number
// (the shared past) costs no atomics.

// Column c of entry b, whose parents are par.
template <int KB, class Parents>
__device__ __forceinline__ void fork_column(const TableArgs& a, int64_t b, int64_t c, const Parents& par) {
  const int64_t b0 = b * a.beams * a.ld, all = a.batch * a.beams * a.ld;
  int32_t* const column = a.table + b0 + c;
  constexpr bool kHold = KB <= 16;  // above, a row's own page is read when it is written: both sets spill
  int32_t was[KB], now[KB];
#pragma unroll
  for (int k = 0; k < KB; ++k)
    if (par[k] != k && in_bounds(a.status, b0 + c + k * a.ld, all)) {
      if (kHold) was[k] = column[k * a.ld];
      now[k] = column[par[k] * a.ld];
    }
#pragma unroll
  for (int k = 0; k < KB; ++k)
    if (par[k] != k && in_bounds(a.status, b0 + c + k * a.ld, all)) {
      if (!kHold) was[k] = column[k * a.ld];
      if (was[k] == now[k]) continue;
      column[k * a.ld] = now[k];
      if (is_page(a, now[k])) atomicAdd(a.refs + now[k], 1);
      if (is_page(a, was[k])) atomicSub(a.refs + was[k], 1);
      if (now[k] < -1 || now[k] >= a.pages || was[k] < -1 || was[k] >= a.pages) atomicOr(a.status, ORPO_STATUS_PAGE);
    }
}

constexpr int kForkThreads = 128;

template <int KB>
__global__ void __launch_bounds__(kForkThreads) fork_kernel(TableArgs a, int32_t* left_alone) {
  __shared__ int par[KB];
  grid_trigger();
  grid_wait();
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  int64_t begin, end;
  bool bad = !wanted(a, b, begin, end);
  if (tid < KB) {
    const int p = tid < a.beams ? a.parent[b * a.ld_parent + tid] : tid;
    bad |= tid < a.beams && (p < 0 || p >= a.beams);
    par[tid] = p;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && blockIdx.y == 0) {
    if (in_bounds(a.status, b, a.batch)) left_alone[b] = bad;
    if (bad) atomicOr(a.status, ORPO_STATUS_PARENT);
  }
  if (bad) return;
  const int64_t used = (begin + a.page - 1) / a.page;
  for (int64_t c = (int64_t)blockIdx.y * kForkThreads + tid; c < used; c += (int64_t)gridDim.y * kForkThreads) fork_column<KB>(a, b, c, par);
}

// ------------------------------------------------------------------ one CTA, or a cluster of them
constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;
constexpr int kMaxCtas = 8;

// Exclusive sum of x over the threads of a CTA of kW warps, and the total.  `part` is kW words of shared memory, free again after
// the call.
template <int kW = kWarps>
__device__ __forceinline__ uint32_t scan(uint32_t x, uint32_t* part, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t sum = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t y = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == 31) part[warp] = sum;
  __syncthreads();
  const uint32_t w = lane < kW ? part[lane] : 0;
  uint32_t before = w;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t y = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += y;
  }
  total = __shfl_sync(~0u, before, 31);
  before = __shfl_sync(~0u, before - w, warp);
  __syncthreads();
  return before + sum - x;
}

__device__ __forceinline__ void plan_sync(int ctas) {
  if (ctas > 1) cluster_sync(); else __syncthreads();
}

// What each CTA of the cluster tells the others; read between two plan_syncs.
struct Totals {
  uint32_t v[4];
};
// Sum over the CTAs before this one, and over all.  A lane asks a CTA; whole warps.
__device__ __forceinline__ uint32_t told_before(const Totals* mine, int what, int cta, int ctas, uint32_t& all) {
  if (ctas == 1) {
    all = mine->v[what];
    return 0;
  }
  const int lane = threadIdx.x & 31;
  uint32_t at, x = 0;
  if (lane < ctas) {
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&mine->v[what])), "r"(lane));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  }
  all = __reduce_add_sync(~0u, x);
  return __reduce_add_sync(~0u, lane < cta ? x : 0);
}

// A CTA's stretch of pages, a run of 32-page words per warp: who is in use, as ballots.  A lane keeps the word of its own
// number; runs of more than 32 words are looked up again.
template <int kW = kWarps>
struct PageRun {
  int32_t begin, words;
  uint32_t kept;
  __device__ __forceinline__ PageRun(int32_t p_begin, int32_t p_end) : kept(0) {
    words = (p_end - p_begin + 32 * kW - 1) / (32 * kW);
    begin = p_begin + (int32_t)(threadIdx.x >> 5) * words * 32;
  }
  // How many pages of the run, of those below p_end, are in use.
  __device__ __forceinline__ uint32_t count(const int32_t* refs, int32_t p_end) {
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    constexpr int kAhead = 8;
    for (int i = 0; i < words; i += kAhead) {
      int32_t v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int32_t p = begin + (i + k) * 32 + lane;
        v[k] = i + k < words && p < p_end ? __ldcg(refs + p) : 0;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= words) break;
        const uint32_t bits = __ballot_sync(~0u, v[k] > 0);
        if (lane == i + k) kept = bits;
        n += __popc(bits);
      }
    }
    return n;
  }
  __device__ __forceinline__ uint32_t word(const int32_t* refs, int32_t p_end, int i) const {
    if (words <= 32) return __shfl_sync(~0u, kept, i);
    const int32_t p = begin + i * 32 + (int32_t)(threadIdx.x & 31);
    return __ballot_sync(~0u, p < p_end && __ldcg(refs + p) > 0);
  }
};

// ------------------------------------------------------------------ reserve
// Items are (row, column) pairs of the positions asked for, in order; a row has `width` of them, of which those from the
// end of its positions on ask for nothing.
struct ReserveArgs {
  TableArgs t;
  int32_t* left_alone;  // [batch] entries that the fork found wrong; nullptr: there was no fork
  int32_t* moves;
  int32_t* n_moves;
  int32_t width;     // items per row, with padding: see padded_width
  int32_t items;     // so many in all
  int32_t units_per; // CTA
  int32_t* count;    // [pages] how many items hold a page that others hold too,
  int32_t* last;     // [pages] and the last of them
  uint32_t* needs;   // [units][kUnit / 32] items that need a page, as bits
  uint32_t* copies;  // [units] moves of a unit
  uint32_t* before;  // [units][2] pages needed and moves of the CTA's units before
  uint32_t* free;    // [pages / kTile] free pages
  int32_t* fresh;    // [items] the new pages, in order
};

enum { kNone = 0, kNeed = 1, kShared = 2 };

// What row asks for: columns first .. first + n - 1, of which the first holds `fill` positions in use.
struct Wanted {
  uint32_t first, n, fill;
};
__device__ __forceinline__ Wanted wanted_columns(const TableArgs& a, uint32_t b) {
  int64_t begin, end;
  if (!wanted(a, b, begin, end) || begin == end) return {0, 0, 0};
  const uint32_t page = (uint32_t)a.page, first = (uint32_t)begin / page, last = ((uint32_t)end - 1) / page;
  return {first, last - first + 1, (uint32_t)begin - first * page};
}

// ---- a decode step's worth: up to kSmallItems items, in one CTA.
// KB: a fork of up to KB beams is done here too, for (entry, column) pairs of at most one per thread; the counts of holders are
// then in shared memory, where what the fork changes can be looked up at once.  0: no fork here, and the counts stay
// where they are.  kQ: items per thread, one after the other.  kT: threads.
constexpr int kSmallThreads = 1024;
constexpr int kSmallMost = 4;               // items per thread at most
constexpr int kSmallItems = kSmallMost * kSmallThreads;
// Where items, pairs and pages are few, so are the threads: the barriers are then shorter (a step of 4 beams in 27 pages with its
// copy 6.3 us captured, with 1024 threads 6.9; the plan alone, fork included, in 27 pages 4.1 and 4.5, in 4000 4.5 and
// 5.3), but each looks through more pages (in 8192 5.2 and 4.9).
constexpr int kFewThreads = 256;
constexpr int kFewPages = 8192;
// In turns, 128 x 256 pairs took 14.5 us here, by a kernel of their own and a plan without a fork 8.3; two to some thirty turns were
// not measured.  Up to one turn it is a launch less: with the copy 5.1 us to enqueue, else 6.4.
constexpr int kForkHere = kSmallThreads;    // pairs
constexpr int kForkPages = 32768;           // 128 KB of counts
inline int32_t padded_pages(int64_t pages, int threads) { return (int32_t)(cdiv(pages, threads) * threads); }

// Pages that several items hold, in shared memory: twice as many slots as items.
template <int kItems>
struct SmallTables {
  int32_t keys[2 * kItems], count[2 * kItems], last[2 * kItems];  // page, how many items, and the last of them
  int32_t fresh[kItems];                                           // the new pages
  uint8_t bad[kItems];                                             // entries
};

template <int KB, int kQ, int kT>
__global__ void __launch_bounds__(kT) small_reserve_kernel(ReserveArgs a, int32_t padded) {
  constexpr int kItems = kQ * kT, kW = kT / 32;
  constexpr uint32_t kSlots = 2 * kItems;
  extern __shared__ __align__(16) uint8_t small_raw[];
  SmallTables<kItems>& s = *reinterpret_cast<SmallTables<kItems>*>(small_raw);
  int32_t* const refs = reinterpret_cast<int32_t*>(small_raw + sizeof(SmallTables<kItems>));  // KB > 0: [padded] counts of holders
  __shared__ uint32_t part[kW];
  const TableArgs& t = a.t;
  const int tid = threadIdx.x, lane = tid & 31;
  grid_trigger();
  for (int i = tid; i < kItems; i += kT) s.bad[i] = 0;
  for (int i = tid; i < (int)kSlots; i += kT) s.keys[i] = -1, s.count[i] = 0, s.last[i] = -1;
  __syncthreads();
  grid_wait();
  const int rows = (int)t.batch * t.beams;
  // ---- counts, lengths, parents
  PageRun<kW> run(0, KB > 0 ? padded : t.pages);
  uint32_t used = 0;
  if constexpr (KB > 0) {
#pragma unroll 8
    for (int p = tid; p < padded; p += kT) refs[p] = p < t.pages ? t.refs[p] : 1;
  } else {
    used = run.count(t.refs, t.pages);
  }
  for (int r = tid; r < rows; r += kT) {
    const int e = r / t.beams;
    int64_t begin, end;
    bool wrong = !wanted(t, e, begin, end);
    if constexpr (KB > 0) {
      const int p = t.parent[e * t.ld_parent + r - e * t.beams];
      wrong |= p < 0 || p >= t.beams;
    } else if (a.left_alone) {
      wrong |= a.left_alone[e] != 0;
    }
    if (wrong) {
      if (in_bounds(t.status, e, kItems)) s.bad[e] = 1;
      atomicOr(t.status, ORPO_STATUS_PARENT);
    }
  }
  Wanted w[kQ];
  uint32_t row[kQ], j[kQ];
  int32_t from[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const uint32_t i = (uint32_t)tid * kQ + q;
    row[q] = i / (uint32_t)a.width;
    j[q] = i - row[q] * (uint32_t)a.width;
    w[q] = i < (uint32_t)a.items ? wanted_columns(t, row[q] / (uint32_t)t.beams) : Wanted{0, 0, 0};
    from[q] = (int32_t)row[q];
    if constexpr (KB > 0) {
      const uint32_t b = row[q] / (uint32_t)t.beams;
      if (w[q].fill > 0 && j[q] == 0) from[q] = (int32_t)(b * t.beams) + t.parent[b * t.ld_parent + row[q] - b * t.beams];
    }
  }
  __syncthreads();
  // ---- the table: each item's page after the fork, and the columns to fork
  int32_t old[kQ];
  bool asks[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    asks[q] = j[q] < w[q].n && !s.bad[row[q] / (uint32_t)t.beams];
    old[q] = -1;
    if (asks[q] && in_bounds(t.status, from[q], rows) && in_bounds(t.status, w[q].first + j[q], t.columns))
      old[q] = t.table[from[q] * t.ld + w[q].first + j[q]];
  }
  if constexpr (KB > 0) {
    const uint32_t columns = (uint32_t)t.columns, e = columns > 0 ? (uint32_t)tid / columns : 0, c = (uint32_t)tid - e * columns;
    const bool on = e < (uint32_t)t.batch && columns > 0 && !s.bad[e] && (int64_t)c * t.page < t.length[e];
    const int64_t b0 = (int64_t)e * t.beams * t.ld, all = t.batch * t.beams * t.ld;
    int32_t* const column = t.table + b0 + c;
    int par[KB];
    int32_t was[KB], now[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      par[k] = on && k < t.beams ? t.parent[e * t.ld_parent + k] : k;
      if (par[k] != k && in_bounds(t.status, b0 + c + k * t.ld, all)) {
        was[k] = column[k * t.ld];
        now[k] = column[par[k] * t.ld];
      }
    }
    __syncthreads();  // all that the fork overwrites is read
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k && was[k] != now[k] && in_bounds(t.status, b0 + c + k * t.ld, all)) {
        column[k * t.ld] = now[k];
        if (is_page(t, now[k])) atomicAdd(t.refs + now[k], 1), atomicAdd(refs + now[k], 1);
        if (is_page(t, was[k])) atomicSub(t.refs + was[k], 1), atomicSub(refs + was[k], 1);
        if (now[k] < -1 || now[k] >= t.pages || was[k] < -1 || was[k] >= t.pages) atomicOr(t.status, ORPO_STATUS_PAGE);
      }
    __syncthreads();
  }
  // ---- what the items ask for; of the items that hold a page together the last keeps it, where nothing else holds it
  int what[kQ];
  int32_t held[kQ];
  bool shared = false;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const bool is = asks[q] && is_page(t, old[q]);
    if (asks[q] && (old[q] < -1 || old[q] >= t.pages)) atomicOr(t.status, ORPO_STATUS_PAGE);
    held[q] = is ? (KB > 0 ? refs[old[q]] : __ldcg(t.refs + old[q])) : 0;
    what[q] = asks[q] && old[q] == -1 ? kNeed : held[q] > 1 ? kShared : kNone;
    shared |= what[q] == kShared;
  }
  if (__syncthreads_or(shared)) {
    uint32_t slot[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (what[q] != kShared) continue;
      slot[q] = (uint32_t)old[q] * 2654435769u / (0xffffffffu / kSlots + 1u);
      for (;;) {  // an empty slot is always met
        const int32_t key = atomicCAS(s.keys + slot[q], -1, old[q]);
        if (key == -1 || key == old[q]) break;
        slot[q] = (slot[q] + 1) % kSlots;
      }
      atomicAdd(s.count + slot[q], 1);
      atomicMax(s.last + slot[q], tid * kQ + q);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (what[q] == kShared && s.count[slot[q]] == held[q] && s.last[slot[q]] == tid * kQ + q) what[q] = kNone;
  }
  uint32_t mine = 0, total;
#pragma unroll
  for (int q = 0; q < kQ; ++q) mine += (uint32_t)(what[q] != kNone) | (uint32_t)(what[q] == kShared && j[q] == 0 && w[q].fill > 0) << 16;
  const uint32_t before = scan<kW>(mine, part, total), needed = total & 0xffff;
  // ---- free pages, lowest first
  if constexpr (KB > 0)
    for (int i = 0; i < run.words; ++i) used += __popc(__ballot_sync(~0u, refs[run.begin + i * 32 + lane] > 0));
  const int run_pages = min(max((KB > 0 ? padded : t.pages) - run.begin, 0), run.words * 32);
  uint32_t found;
  uint32_t rank = scan<kW>(lane == 0 ? (uint32_t)run_pages - used : 0, part, found);
  rank = __shfl_sync(~0u, rank, 0);
  if (found < needed) {
    if (tid == 0) {
      atomicOr(t.status, ORPO_STATUS_FULL);
      *a.n_moves = 0;
    }
    return;
  }
  for (int i = 0; i < run.words && rank < needed; ++i) {
    const int32_t p = run.begin + i * 32 + lane;
    const uint32_t taken = KB > 0 ? __ballot_sync(~0u, refs[p] > 0) : run.word(t.refs, t.pages, i);
    const uint32_t bits = __ballot_sync(~0u, !(taken >> lane & 1u) && p < t.pages), to = rank + __popc(bits & ((1u << lane) - 1u));
    if (bits >> lane & 1u && to < needed && in_bounds(t.status, to, kItems)) s.fresh[to] = p;
    rank += __popc(bits);
  }
  __syncthreads();
  if (tid == 0) *a.n_moves = (int32_t)(total >> 16);
  uint32_t at = before & 0xffff, m = before >> 16;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (what[q] == kNone) continue;
    const int32_t p = s.fresh[at++];
    t.table[row[q] * t.ld + w[q].first + j[q]] = p;
    t.refs[p] = 1;
    if (what[q] != kShared) continue;
    atomicSub(t.refs + old[q], 1);
    if (j[q] != 0 || w[q].fill == 0 || !in_bounds(t.status, m, rows)) continue;
    a.moves[3 * m] = old[q];
    a.moves[3 * m + 1] = p;
    a.moves[3 * m++ + 2] = (int32_t)w[q].fill;
  }
}

// ---- any number of items and pages, on a cluster of CTAs.  A warp takes a unit of kUnit items, a row's or several rows', at
// a time, and a tile of kTile pages.  Each CTA has a stretch of units, and every ctas-th tile, so that the lowest free pages, which
// are the ones that are taken, are everybody's; the CTAs tell each other how many pages their units need and how many of each
// tile's are free, and then every item's new page is known.
constexpr int kTile = 1024;
constexpr int kUnit = 128;
constexpr int kPer = kUnit / 32;  // items of a lane

struct Items {
  int32_t row[kPer], old[kPer];
  Wanted w[kPer];
  uint32_t j[kPer];
  bool asks[kPer];
};

// The units of a warp, one after the other: next() gives their items and the pages that those have.  What the rows of up to
// 32 units ask for is looked up at once, a unit per lane, where every unit is of one row.
struct Units {
  const ReserveArgs& a;
  int32_t unit, end;
  int32_t row;  // of this lane's unit
  uint32_t j;
  Wanted w;
  int at = 32;
  __device__ Units(const ReserveArgs& args, int32_t begin, int32_t end_)
      : a(args), unit(begin + (int32_t)(threadIdx.x >> 5) - kWarps), end(end_), row(0), j(0), w{0, 0, 0} {}

  __device__ __forceinline__ Wanted of_row(uint32_t r) const {
    const uint32_t b = r / (uint32_t)a.t.beams;
    return (int64_t)r < a.t.batch * a.t.beams && !(a.left_alone && a.left_alone[b]) ? wanted_columns(a.t, b) : Wanted{0, 0, 0};
  }
  // false: there is no other unit.  any: whether the unit's items ask for anything; else `it` is not filled.
  __device__ __forceinline__ bool next(Items& it, bool& any) {
    unit += kWarps;
    if (unit >= end) return false;
    const int lane = threadIdx.x & 31;
    if (a.width % kUnit == 0) {
      if (at == 32) {
        const int64_t mine = (int64_t)unit + lane * kWarps;
        const uint32_t i = mine < end ? (uint32_t)mine * kUnit : 0;
        row = (int32_t)(i / (uint32_t)a.width);
        j = i - (uint32_t)row * (uint32_t)a.width;
        w = mine < end ? of_row((uint32_t)row) : Wanted{0, 0, 0};
        at = 0;
      }
      const int32_t r = __shfl_sync(~0u, row, at);
      const uint32_t j0 = __shfl_sync(~0u, j, at);
      const Wanted x{__shfl_sync(~0u, w.first, at), __shfl_sync(~0u, w.n, at), __shfl_sync(~0u, w.fill, at)};
      ++at;
      any = j0 < x.n;
      if (!any) return true;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        it.row[u] = r;
        it.j[u] = j0 + u * 32 + lane;
        it.w[u] = x;
        it.asks[u] = it.j[u] < x.n;
      }
    } else {
      any = true;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const uint32_t i = (uint32_t)unit * kUnit + u * 32 + lane, r = i / (uint32_t)a.width;
        it.row[u] = (int32_t)r;
        it.j[u] = i - r * (uint32_t)a.width;
        it.w[u] = of_row(r);
        it.asks[u] = it.j[u] < it.w[u].n;
      }
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t c = (int64_t)it.w[u].first + it.j[u];
      it.old[u] = it.asks[u] && in_bounds(a.t.status, c, a.t.columns) ? __ldcg(a.t.table + it.row[u] * a.t.ld + c) : -1;
    }
    return true;
  }
};

// A tile's free pages: a lane has the word of its own number.
__device__ __forceinline__ uint32_t free_word(const int32_t* refs, int32_t tile, int32_t pages) {
  const int lane = threadIdx.x & 31;
  uint32_t kept = 0;
#pragma unroll 1
  for (int i = 0; i < 32; i += 8) {
    int32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int32_t p = tile * kTile + (i + k) * 32 + lane;
      v[k] = p < pages ? __ldcg(refs + p) : 1;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t bits = __ballot_sync(~0u, v[k] <= 0);
      if (lane == i + k) kept = bits;
    }
  }
  return kept;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(ReserveArgs a) {
  __shared__ uint32_t part[kWarps];
  __shared__ Totals totals;
  const TableArgs& t = a.t;
  grid_trigger();
  grid_wait();
  const int tid = threadIdx.x, lane = tid & 31, ctas = gridDim.x, cta = blockIdx.x;
  if (!a.left_alone)
    for (int64_t b = (int64_t)cta * kPlanThreads + tid; b < t.batch; b += (int64_t)ctas * kPlanThreads) {
      int64_t begin, end;
      if (!wanted(t, b, begin, end)) atomicOr(t.status, ORPO_STATUS_PARENT);
    }
  if (a.items == 0) {  // a fork alone
    if (tid == 0 && cta == 0) *a.n_moves = 0;
    return;
  }
  const int32_t units = (int32_t)(((int64_t)a.items + kUnit - 1) / kUnit);
  const int32_t u_begin = (int32_t)min((int64_t)cta * a.units_per, (int64_t)units), u_end = (int32_t)min((int64_t)u_begin + a.units_per, (int64_t)units);
  const int32_t tiles = (t.pages + kTile - 1) / kTile, first_tile = (tid >> 5) * ctas + cta, tile_step = kWarps * ctas;
  Items it;
  bool asked;

  // ---- how many pages of each tile are free
  uint32_t first_word = 0;  // of the warp's first tile
  for (int32_t tile = first_tile; tile < tiles; tile += tile_step) {
    const uint32_t word = free_word(t.refs, tile, t.pages), n = __reduce_add_sync(~0u, (uint32_t)__popc(word));
    if (tile == first_tile) first_word = word;
    if (lane == 0) a.free[tile] = n;
  }
  // ---- what each item asks for.  Pages that others hold too are counted below
  int shared = 0;
  for (Units list(a, u_begin, u_end); list.next(it, asked);) {
    const int32_t unit = list.unit;
    uint32_t need = 0;
    if (asked) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const bool wrong = it.old[u] < -1 || it.old[u] >= t.pages;
        if (wrong) atomicOr(t.status, ORPO_STATUS_PAGE);
        if (it.old[u] >= 0 && !wrong && __ldcg(t.refs + it.old[u]) > 1) a.count[it.old[u]] = 0, a.last[it.old[u]] = -1, shared = 1;
        const uint32_t bits = __ballot_sync(~0u, it.asks[u] && it.old[u] == -1);
        if (lane == u) need = bits;
      }
    }
    if (lane < kPer && in_bounds(t.status, unit, units)) a.needs[unit * kPer + lane] = need;
    if (lane == kPer && in_bounds(t.status, unit, units)) a.copies[unit] = 0;
  }
  shared = __syncthreads_or(shared);
  // ---- sums over the CTA's units, told to the others
  const auto sum_up = [&] {
    uint32_t needed = 0, moved = 0;
    for (int32_t u0 = u_begin; u0 < u_end; u0 += kPlanThreads) {
      const int32_t unit = u0 + tid;
      const bool mine = unit < u_end && in_bounds(t.status, unit, units);
      uint32_t need = 0, all_need, all_moves;
#pragma unroll
      for (int u = 0; u < kPer; ++u) need += mine ? __popc(a.needs[unit * kPer + u]) : 0;
      const uint32_t at_need = scan(need, part, all_need), at_move = scan(mine ? a.copies[unit] : 0, part, all_moves);
      if (mine) a.before[2 * unit] = needed + at_need, a.before[2 * unit + 1] = moved + at_move;
      needed += all_need;
      moved += all_moves;
    }
    if (tid == 0) totals.v[1] = needed, totals.v[2] = moved;
  };
  sum_up();
  if (tid == 0) totals.v[0] = shared;
  plan_sync(ctas);
  uint32_t any;
  told_before(&totals, 0, cta, ctas, any);
  // ---- of the items that hold a page together the last keeps it, where nothing else holds it
  if (any) {
    if (shared)
      for (Units list(a, u_begin, u_end); list.next(it, asked);) {
        if (!asked) continue;
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (it.old[u] >= 0 && it.old[u] < t.pages && __ldcg(t.refs + it.old[u]) > 1) {
            atomicAdd(a.count + it.old[u], 1);
            atomicMax(a.last + it.old[u], list.unit * kUnit + u * 32 + lane);
          }
      }
    plan_sync(ctas);
    if (shared)
      for (Units list(a, u_begin, u_end); list.next(it, asked);) {
        if (!asked) continue;
        const int32_t unit = list.unit;
        uint32_t moves = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          bool copies = false;
          if (it.old[u] >= 0 && it.old[u] < t.pages) {
            const int32_t held = __ldcg(t.refs + it.old[u]);
            copies = held > 1 && !(__ldcg(a.count + it.old[u]) == held && __ldcg(a.last + it.old[u]) == unit * kUnit + u * 32 + lane);
          }
          const uint32_t bits = __ballot_sync(~0u, copies || (it.asks[u] && it.old[u] == -1));
          moves += __popc(__ballot_sync(~0u, copies && it.j[u] == 0 && it.w[u].fill > 0));
          if (lane == 0 && in_bounds(t.status, unit, units)) a.needs[unit * kPer + u] = bits;
        }
        if (lane == 0 && in_bounds(t.status, unit, units)) a.copies[unit] = moves;
      }
    __syncthreads();
    sum_up();
    plan_sync(ctas);
  }
  uint32_t all_needed, all_moved;
  const uint32_t at_item = told_before(&totals, 1, cta, ctas, all_needed);
  const uint32_t at_move = told_before(&totals, 2, cta, ctas, all_moved);
  // ---- the new pages, lowest first.  rank: free pages before the tile; then all of them
  uint32_t rank = 0;
  int32_t seen = 0;  // tiles counted in rank
  const auto count_to = [&](int32_t tile) {
    uint32_t mine = 0;
    for (int32_t i = seen + lane; i < tile; i += 32) mine += __ldcg(a.free + i);
    rank += __reduce_add_sync(~0u, mine);
    seen = tile;
  };
  for (int32_t tile = first_tile; tile < tiles; tile += tile_step) {
    count_to(tile);
    if (rank >= all_needed) break;
    const uint32_t word = tile == first_tile ? first_word : free_word(t.refs, tile, t.pages);
    uint32_t start = __popc(word);  // free pages of the tile before the lane's word
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(~0u, start, d);
      if (lane >= d) start += y;
    }
    start -= __popc(word);
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
      const uint32_t bits = __shfl_sync(~0u, word, i), at = rank + __shfl_sync(~0u, start, i) + __popc(bits & ((1u << lane) - 1u));
      if (bits >> lane & 1u && at < all_needed && in_bounds(t.status, at, a.items)) a.fresh[at] = tile * kTile + i * 32 + lane;
    }
  }
  if (rank < all_needed) count_to(tiles);
  const bool full = rank < all_needed;  // the same for everybody: all tiles are counted, or enough of them
  if (tid == 0 && cta == 0) {
    *a.n_moves = full ? 0 : (int32_t)all_moved;
    if (full) atomicOr(t.status, ORPO_STATUS_FULL);
  }
  plan_sync(ctas);  // the last look at another CTA's totals is behind
  if (full) return;
  for (Units list(a, u_begin, u_end); list.next(it, asked);) {
    if (!asked) continue;
    const int32_t unit = list.unit;
    uint32_t bits[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) bits[u] = a.needs[unit * kPer + u];
    uint32_t at = at_item + a.before[2 * unit], to = at_move + a.before[2 * unit + 1];
    int32_t page[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const uint32_t mine = at + __popc(bits[u] & ((1u << lane) - 1u));
      page[u] = bits[u] >> lane & 1u && in_bounds(t.status, mine, a.items) ? __ldcg(a.fresh + mine) : -1;
      at += __popc(bits[u]);
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const bool move = page[u] >= 0 && it.old[u] >= 0 && it.j[u] == 0 && it.w[u].fill > 0;
      const uint32_t moves = __ballot_sync(~0u, move), m = to + __popc(moves & ((1u << lane) - 1u));
      to += __popc(moves);
      if (page[u] < 0) continue;
      t.table[it.row[u] * t.ld + it.w[u].first + it.j[u]] = page[u];
      t.refs[page[u]] = 1;
      if (it.old[u] >= 0) atomicSub(t.refs + it.old[u], 1);
      if (move && in_bounds(t.status, m, t.batch * t.beams)) {
        a.moves[3 * m] = it.old[u];
        a.moves[3 * m + 1] = page[u];
        a.moves[3 * m + 2] = (int32_t)it.w[u].fill;
      }
    }
  }
}

// ------------------------------------------------------------------ copy
struct CopyArgs {
  uint8_t* pool;
  int64_t outer, rows, page_bytes;  // page_bytes: of one (slab, page)
  int32_t pages, page, unit;
  const int32_t* moves;
  int32_t max_moves;
  const int32_t* n_moves;
  int32_t* status;
  int64_t stretches;  // of one (slab, page), at most
  int64_t stretch;    // pieces of one, a multiple of 32
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;  // pieces of a lane in flight

// A warp takes a stretch of at most kCopyUnroll * 32 pieces of one (move, slab): of the page's bytes there, all rows one after
// the other, those whose positions move.
template <class Piece>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  constexpr int kSize = (int)sizeof(Piece);
  grid_trigger();
  grid_wait();
  const int32_t n = *a.n_moves;
  const int64_t warp = ((int64_t)blockIdx.x * kCopyThreads + threadIdx.x) / 32, warps = (int64_t)gridDim.x * kCopyThreads / 32;
  const int lane = threadIdx.x & 31;
  if (n < 0 || n > a.max_moves) {
    if (warp == 0 && lane == 0) atomicOr(a.status, ORPO_STATUS_PAGE);
    return;
  }
  const uint32_t row_pieces = (uint32_t)((int64_t)a.page * a.unit / kSize);
  const int64_t pieces = a.rows * row_pieces, per_move = a.outer * a.stretches, all = a.outer * a.pages * a.page_bytes;
  for (int64_t w = warp; w < n * per_move; w += warps) {
    const int64_t m = w / per_move, left = w - m * per_move, o = left / a.stretches, s = left - o * a.stretches;
    const int32_t from = a.moves[3 * m], to = a.moves[3 * m + 1], positions = a.moves[3 * m + 2];
    if (from < 0 || from >= a.pages || to < 0 || to >= a.pages || from == to || positions < 0 || positions > a.page) {
      if (left == 0 && lane == 0) atomicOr(a.status, ORPO_STATUS_PAGE);
      continue;
    }
    const int64_t first = s * a.stretch, begin = first + lane, end = min(pieces, first + a.stretch);
    uint32_t moves = 0, cut = 0;  // which of the lane's pieces move, and which in part
    const uint32_t bytes = (uint32_t)positions * (uint32_t)a.unit;  // of a row
    if (positions == a.page) {
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u) moves |= (uint32_t)(begin + u * 32 < end) << u;
    } else {
      const uint32_t in_row = (uint32_t)(first - first / row_pieces * row_pieces) + lane;  // counted from the row that `first` is in
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u) {
        uint32_t i = in_row + u * 32;
        if (row_pieces >= kCopyUnroll * 32) i -= i >= row_pieces ? row_pieces : 0;  // at most one row on
        else i %= row_pieces;
        const int64_t byte = (int64_t)i * kSize;
        const bool mine = begin + u * 32 < end && byte < bytes, part = byte + kSize > bytes;
        moves |= (uint32_t)(mine && !part) << u;
        cut |= (uint32_t)(mine && part) << u;
      }
    }
    const int64_t src_at = (o * a.pages + from) * a.page_bytes + begin * kSize, dst_at = (o * a.pages + to) * a.page_bytes + begin * kSize;
    const Piece* const src = reinterpret_cast<const Piece*>(a.pool + src_at);
    Piece* const dst = reinterpret_cast<Piece*>(a.pool + dst_at);
    Piece v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (moves >> u & 1u && in_bounds(a.status, src_at + (u * 32 + 1) * kSize - 1, all)) v[u] = src[u * 32];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (moves >> u & 1u && in_bounds(a.status, dst_at + (u * 32 + 1) * kSize - 1, all)) dst[u * 32] = v[u];
    for (; cut != 0; cut &= cut - 1) {  // positions that end inside a piece
      const int u = __ffs(cut) - 1;
      for (uint32_t i = 0; i < bytes % kSize; ++i)
        if (in_bounds(a.status, src_at + u * 32 * kSize + i, all) && in_bounds(a.status, dst_at + u * 32 * kSize + i, all))
          a.pool[dst_at + u * 32 * kSize + i] = a.pool[src_at + u * 32 * kSize + i];
    }
  }
}

// ------------------------------------------------------------------ release
constexpr int kReleaseThreads = 256;

__global__ void __launch_bounds__(kReleaseThreads) release_kernel(TableArgs a, const uint8_t* ended) {
  grid_trigger();
  grid_wait();
  const int64_t row = blockIdx.x;
  if (ended && !ended[row / a.beams]) return;
  int wrong = 0;
  for (int64_t c = (int64_t)blockIdx.y * kReleaseThreads + threadIdx.x; c < a.columns; c += (int64_t)gridDim.y * kReleaseThreads) {
    if (!in_bounds(a.status, row * a.ld + c, a.batch * a.beams * a.ld)) continue;
    int32_t* const at = a.table + row * a.ld + c;
    const int32_t e = *at;
    if (e == -1) continue;
    *at = -1;
    if (!is_page(a, e)) {
      wrong = 1;
    } else if (atomicSub(a.refs + e, 1) <= 0) {
      atomicAdd(a.refs + e, 1);
      wrong = 1;
    }
  }
  if (wrong) atomicOr(a.status, ORPO_STATUS_PAGE);
}

// ------------------------------------------------------------------ compact
// With u(p) pages in use below page p and n in use in all: a free page p < n is hole number p - u(p), a used page p >= n
// is mover number u(p) - u(n).  So one count of the pages in use, told between the CTAs, gives every number.
struct CompactArgs {
  const int32_t* table;
  int64_t ld, columns, rows;
  const int32_t* refs;
  int32_t pages, page;
  int32_t* new_table;
  int64_t ld_new;
  int32_t* new_refs;
  int32_t* live;
  int32_t* moves;
  int32_t* n_moves;
  int32_t pages_per;  // CTA, a multiple of 32 * kWarps
  int32_t* holes;   // [pages / 2] free pages below n, by number
  int32_t* movers;  // [pages] used pages at or above n, by the pages in use below them
  int32_t* below;   // [pages] the pages in use below, or -1 for a free page
  int32_t* status;
};

// Entries i, i + step, ... of the table.  first: u(n)
__device__ __forceinline__ void remap(const CompactArgs& a, int32_t live, int32_t first, int64_t i, int64_t step) {
  int wrong = 0;
  for (const int64_t n = a.rows * a.columns; i < n; i += step) {
    const uint32_t row = (uint32_t)i / (uint32_t)a.columns, c = (uint32_t)i - row * (uint32_t)a.columns;
    if (!in_bounds(a.status, row * a.ld + c, a.rows * a.ld) || !in_bounds(a.status, row * a.ld_new + c, a.rows * a.ld_new)) continue;
    int32_t e = a.table[row * a.ld + c];
    if (e < -1 || e >= a.pages) {
      wrong = 1;
    } else if (e >= 0) {
      const int32_t u = a.below[e];  // by now the counts of the holes may be those of the pages that move there
      if (u < 0) wrong = 1;
      else if (e >= live && in_bounds(a.status, u - first, a.pages / 2)) e = a.holes[u - first];
    }
    a.new_table[row * a.ld_new + c] = e;
  }
  if (wrong) atomicOr(a.status, ORPO_STATUS_PAGE);
}

// here: 0: the table is done by another kernel; 1: here; 2: here, with the lists in shared memory
__global__ void __launch_bounds__(kPlanThreads) compact_kernel(CompactArgs a, int here) {
  extern __shared__ __align__(16) int32_t own[];
  if (here == 2) {  // one CTA: its arrays fit shared memory
    a.below = own;
    a.movers = own + a.pages;
    a.holes = own + 2 * a.pages;
  }
  __shared__ uint32_t part[kWarps];
  __shared__ Totals totals;
  grid_trigger();
  grid_wait();
  const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x;
  const int32_t p_begin = (int32_t)min((int64_t)cta * a.pages_per, (int64_t)a.pages), p_end = (int32_t)min((int64_t)p_begin + a.pages_per, (int64_t)a.pages);
  const int lane = tid & 31;
  PageRun<> run(p_begin, p_end);
  const uint32_t run_used = run.count(a.refs, p_end);
  uint32_t used;
  const uint32_t run_before = scan(lane == 0 ? run_used : 0, part, used);
  if (tid == 0) totals.v[0] = used, totals.v[1] = 0;
  plan_sync(ctas);
  uint32_t n;
  uint32_t before = told_before(&totals, 0, cta, ctas, n) + __shfl_sync(~0u, run_before, 0);
  const int32_t live = (int32_t)n;
  for (int i = 0; i < run.words; ++i) {  // whole warps: the lanes past p_end take part in the ballots
    const uint32_t bits = run.word(a.refs, p_end, i);
    const int32_t p = run.begin + i * 32 + lane;
    const uint32_t u = before + __popc(bits & ((1u << lane) - 1u));  // pages in use below p
    const bool in_use = bits >> lane & 1u;
    before += __popc(bits);
    if (p >= p_end) continue;
    if (p == live) totals.v[1] = u + 1;  // u(n), told with 0 for "not mine"
    a.below[p] = in_use ? (int32_t)u : -1;
    if (p < live) {
      if (!in_use && in_bounds(a.status, p - (int32_t)u, a.pages / 2)) a.holes[p - (int32_t)u] = p;
      if (in_use && a.new_refs != a.refs) a.new_refs[p] = __ldcg(a.refs + p);
    } else {
      if (in_use && in_bounds(a.status, u, a.pages)) a.movers[u] = p;
      if (a.new_refs != a.refs) a.new_refs[p] = 0;
    }
  }
  plan_sync(ctas);
  uint32_t first;
  told_before(&totals, 1, cta, ctas, first);
  first = first ? first - 1 : n;  // every page is in use
  for (int32_t i = cta * kPlanThreads + tid; i < live - (int32_t)first; i += ctas * kPlanThreads) {
    if (!in_bounds(a.status, i, a.pages / 2)) continue;
    const int32_t from = a.movers[first + i], to = a.holes[i];
    a.moves[3 * i] = from;
    a.moves[3 * i + 1] = to;
    a.moves[3 * i + 2] = a.page;
    a.new_refs[to] = __ldcg(a.refs + from);
    if (a.new_refs == a.refs) a.new_refs[from] = 0;
  }
  if (tid == 0 && cta == 0) {
    *a.n_moves = live - (int32_t)first;
    *a.live = live;
  }
  if (here) remap(a, live, (int32_t)first, (int64_t)cta * kPlanThreads + tid, (int64_t)ctas * kPlanThreads);
  if (ctas > 1) cluster_sync();  // the totals may still be read
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads) remap_kernel(CompactArgs a) {
  grid_trigger();
  grid_wait();
  const int32_t live = *a.live;
  remap(a, live, live - *a.n_moves, (int64_t)blockIdx.x * kRemapThreads + threadIdx.x, (int64_t)gridDim.x * kRemapThreads);
}

// ------------------------------------------------------------------ host
constexpr int64_t kMaxPages = 1ll << 24, kMaxPage = 1ll << 16, kMaxInt = (1ll << 31) - 1, kMaxItems = 1ll << 30;

bool table_ok(int64_t table_rows, int64_t ld, int64_t columns, int64_t pages, int64_t page) {
  return table_rows >= 0 && table_rows <= (1ll << 20) && columns >= 0 && columns <= kMaxInt && ld >= columns && pages >= 1 &&
         pages <= kMaxPages && page >= 1 && page <= kMaxPage && columns * page <= kMaxInt && table_rows * columns <= kMaxInt;
}

int64_t width_of(int64_t most, int64_t page) { return most > 0 ? cdiv(most - 1, page) + 1 : 0; }

size_t align16(size_t n) { return (n + 15) / 16 * 16; }
// Items per row, rounded up to a power of two up to 32 or a multiple of kUnit, so that a warp's unit of items starts on a row.
int64_t rounded_width(int64_t width) {
  if (width > 32) return cdiv(width, kUnit) * kUnit;
  int64_t w = 1;
  while (w < width) w *= 2;
  return w;
}
// The same where that stays within kMaxItems; else no padding, and units hold the ends of rows.
int64_t padded_width(int64_t rows, int64_t width) {
  const int64_t w = rounded_width(width);
  return rows * w <= kMaxItems ? w : width;
}
// Never less for more rows or a larger width, so a workspace for the largest call serves all of them.
size_t reserve_bytes(int64_t batch, int64_t pages, int64_t rows, int64_t width) {
  const int64_t units = cdiv(std::min(rows * rounded_width(width), kMaxItems), kUnit);
  return align16(batch * 4) + 2 * align16(pages * 4) + align16(units * kPer * 4) + align16(units * 4) + align16(units * 8) +
         align16(cdiv(pages, kTile) * 4) + align16(std::min(pages, rows * width) * 4);
}
size_t compact_bytes(int64_t pages) { return align16(pages / 2 * 4) + 2 * align16(pages * 4); }

// CTAs of a plan over so many units and pages, and a CTA's share of n in whole tiles.
// Compaction of 4096 pages takes 5.5 us in one CTA, of 16384 13.8 in one and 6.7 in eight.
constexpr int64_t kOneCta = 4096;  // pages
int plan_ctas(int64_t units, int64_t pages) { return units <= kWarps && pages <= kOneCta ? 1 : kMaxCtas; }
int32_t share(int64_t n, int ctas, int tile) { return (int32_t)(cdiv(cdiv(n, ctas), tile) * tile); }
// Table entries per CTA up to which the compaction's own CTAs rewrite the table.  At 65536 entries that takes 15.4 to 16.1 us in 70000
// pages and 10 in 9000, by a kernel of their own 12.3 and 8, but that one is 1.4 us more to enqueue; at 33024 7.8 here.
constexpr int64_t kRemapHere = 8192;
// Pages whose counts one CTA looks through for a decode step: 512 rows in 16385 pages take 7 us in one CTA and 15 on a cluster, in
// 100000 13 and 17; one CTA takes 0.08 us per 1000 pages more, the cluster 0.01.  (Items: 1025 take 12 us in one CTA and 27 on a
// cluster, 4096 19 and 27.)
constexpr int64_t kSmallPages = 131072;

template <int KB, int kQ, int kT>
cudaError_t launch_small(const ReserveArgs& a, cudaStream_t st) {
  static std::atomic<int> done[64];
  constexpr int kTables = (int)sizeof(SmallTables<kQ * kT>), kMost = kTables + (KB > 0 ? kForkPages * 4 : 0);
  static_assert(kTables % 16 == 0 && kMost <= 227 << 10, "a CTA's shared memory");
  const cudaError_t e = opt_in_smem(small_reserve_kernel<KB, kQ, kT>, kMost, done);
  if (e != cudaSuccess) return e;
  const int32_t padded = KB > 0 ? padded_pages(a.t.pages, kT) : 0;
  return launch_dependent(small_reserve_kernel<KB, kQ, kT>, dim3(1), kT, (size_t)kTables + (size_t)padded * 4, st, a, padded);
}
template <int KB>
cudaError_t launch_small(const ReserveArgs& a, bool few, cudaStream_t st) {
  return few ? launch_small<KB, 1, kFewThreads>(a, st) : launch_small<KB, 1, kSmallThreads>(a, st);
}

bool misaligned(std::initializer_list<const void*> p) {
  uintptr_t at = 0;
  for (const void* x : p) at |= reinterpret_cast<uintptr_t>(x);
  return at & 3;
}

template <class Piece>
cudaError_t launch_copy(CopyArgs a, int sms, cudaStream_t st) {
  const int64_t pieces = cdiv(a.page_bytes, (int64_t)sizeof(Piece));
  a.stretches = cdiv(pieces, kCopyUnroll * 32);
  a.stretch = cdiv(cdiv(pieces, a.stretches), 32) * 32;
  const int64_t warps = (int64_t)a.max_moves * a.outer * a.stretches;  // at most
  const int grid = (int)std::min<int64_t>((int64_t)sms * 8, cdiv(warps, kCopyThreads / 32));
  prof_begin(K_PAGECOPY, st);
  const cudaError_t e = launch_dependent(copy_kernel<Piece>, grid, kCopyThreads, 0, st, a);
  prof_end(K_PAGECOPY, st);
  return e;
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" {

size_t orpo_pages_workspace_bytes(int64_t table_rows, int64_t pages, int64_t page, int64_t most) {
  if (!table_ok(table_rows, 0, 0, pages, page) || most < 0 || most > kMaxInt) return 0;
  const int64_t width = width_of(most, page);
  if (table_rows * width > kMaxItems) return 0;
  return std::max(std::max(reserve_bytes(table_rows, pages, table_rows, width), compact_bytes(pages)), (size_t)16);
}

int orpo_pages_advance(int32_t* table, int64_t ld_table, int64_t columns, int32_t* refs, int64_t pages, int64_t page,
                       const int32_t* parent, int64_t ld_parent, const int32_t* length, const int32_t* more, int64_t most,
                       int64_t batch, int beams, int32_t* moves, int64_t max_moves, int32_t* n_moves, void* workspace,
                       size_t ws_bytes, int32_t* status, void* stream) {
  if (batch < 0 || batch > (1ll << 20) || beams < 1 || beams > ORPO_MAX_BEAMS ||
      !table_ok(batch * beams, ld_table, columns, pages, page) || most < 0 || most > kMaxInt || (parent && ld_parent < beams) ||
      max_moves < batch * beams)
    return ORPO_ERR_SHAPE;
  const int64_t rows = batch * beams, width = width_of(most, page);
  if (rows * width > kMaxItems) return ORPO_ERR_SHAPE;
  if (!n_moves || !status || (batch > 0 && ((columns > 0 && !table) || !refs || !length || !moves || !workspace))) return ORPO_ERR_NULL;
  if (misaligned({table, refs, parent, length, more, moves, n_moves, status}) || !aligned16(workspace)) return ORPO_ERR_ALIGN;
  if (ws_bytes < (batch > 0 ? reserve_bytes(batch, pages, rows, width) : 0)) return ORPO_ERR_WORKSPACE;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const TableArgs t{table, ld_table, columns, refs, (int32_t)pages, (int32_t)page, parent, ld_parent, length, more, (int32_t)most,
                    batch, beams, status};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool fork = parent && batch > 0;
  ReserveArgs a{};
  a.t = t;
  a.moves = moves;
  a.n_moves = n_moves;
  cudaError_t e = cudaSuccess;
  prof_begin(K_PAGES, st);
  const bool small = rows * width > 0 && rows * width <= kSmallItems && pages <= kSmallPages;
  const bool fork_there = fork && small && beams <= 8 && rows * width <= kSmallThreads && batch * columns <= kForkHere && pages <= kForkPages;
  if (fork && !fork_there) {
    a.left_alone = reinterpret_cast<int32_t*>(ws);
    const dim3 grid((unsigned)batch, (unsigned)std::max<int64_t>(1, std::min<int64_t>(65535, cdiv(columns, kForkThreads))));
    e = beams <= 4    ? launch_dependent(fork_kernel<4>, grid, kForkThreads, 0, st, t, a.left_alone)
        : beams <= 8  ? launch_dependent(fork_kernel<8>, grid, kForkThreads, 0, st, t, a.left_alone)
        : beams <= 16 ? launch_dependent(fork_kernel<16>, grid, kForkThreads, 0, st, t, a.left_alone)
        : beams <= 32 ? launch_dependent(fork_kernel<32>, grid, kForkThreads, 0, st, t, a.left_alone)
                      : launch_dependent(fork_kernel<64>, grid, kForkThreads, 0, st, t, a.left_alone);
  }
  if (e == cudaSuccess && small) {
    a.width = (int32_t)width;
    a.items = (int32_t)(rows * width);
    const bool few = a.items <= kFewThreads && pages <= kFewPages && (!fork_there || batch * columns <= kFewThreads);
    e = a.items > kSmallThreads ? launch_small<0, kSmallMost, kSmallThreads>(a, st)
        : !fork_there           ? launch_small<0>(a, few, st)
        : beams <= 4            ? launch_small<4>(a, few, st)
                                : launch_small<8>(a, few, st);
  } else if (e == cudaSuccess) {
    a.width = (int32_t)padded_width(rows, width);
    a.items = width > 0 ? (int32_t)(rows * a.width) : 0;
    const int64_t units = cdiv(a.items, kUnit);
    const int ctas = a.items > 0 ? plan_ctas(units, pages) : 1;
    a.units_per = share(units, ctas, 1);
    a.count = reinterpret_cast<int32_t*>(ws += align16(batch * 4));
    a.last = reinterpret_cast<int32_t*>(ws += align16(pages * 4));
    a.needs = reinterpret_cast<uint32_t*>(ws += align16(pages * 4));
    a.copies = reinterpret_cast<uint32_t*>(ws += align16(units * kPer * 4));
    a.before = reinterpret_cast<uint32_t*>(ws += align16(units * 4));
    a.free = reinterpret_cast<uint32_t*>(ws += align16(units * 8));
    a.fresh = reinterpret_cast<int32_t*>(ws += align16(cdiv(pages, kTile) * 4));
    e = launch_cluster_dependent(reserve_kernel, ctas, kPlanThreads, 0, st, a);
  }
  prof_end(K_PAGES, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}

int orpo_pages_copy(void* pool, int64_t outer, int64_t pages, int64_t rows, int64_t page, int64_t unit_bytes,
                    const int32_t* moves, int64_t max_moves, const int32_t* n_moves, int32_t* status, void* stream) {
  if (outer < 0 || pages < 1 || pages > kMaxPages || rows < 0 || page < 1 || page > kMaxPage || unit_bytes < 0 || max_moves < 0 ||
      max_moves > kMaxInt || (unit_bytes > 0 && page > kMaxInt / unit_bytes))
    return ORPO_ERR_SHAPE;
  if (outer == 0 || rows == 0 || unit_bytes == 0 || max_moves == 0) return ORPO_OK;
  const int64_t run = page * unit_bytes, most = 1ll << 62;
  if (rows >= most / run || outer >= most / (rows * run) || pages >= most / (outer * rows * run)) return ORPO_ERR_SHAPE;
  if (outer * rows >= most / max_moves / cdiv(run, 128)) return ORPO_ERR_SHAPE;
  if (!pool || !moves || !n_moves || !status) return ORPO_ERR_NULL;
  if (misaligned({moves, n_moves, status})) return ORPO_ERR_ALIGN;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  const CopyArgs a{static_cast<uint8_t*>(pool), outer, rows, rows * run, (int32_t)pages, (int32_t)page, (int32_t)unit_bytes, moves,
                   (int32_t)max_moves, n_moves, status, 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t at = (uint64_t)reinterpret_cast<uintptr_t>(pool) | (uint64_t)run;
  const cudaError_t e = at % 16 == 0  ? launch_copy<uint4>(a, sms, st)
                        : at % 8 == 0 ? launch_copy<uint2>(a, sms, st)
                        : at % 4 == 0 ? launch_copy<uint32_t>(a, sms, st)
                                      : launch_copy<uint8_t>(a, sms, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}

int orpo_pages_release(int32_t* table, int64_t ld_table, int64_t columns, int32_t* refs, int64_t pages, const uint8_t* ended,
                       int64_t batch, int beams, int32_t* status, void* stream) {
  if (batch < 0 || batch > (1ll << 20) || beams < 1 || beams > ORPO_MAX_BEAMS || !table_ok(batch * beams, ld_table, columns, pages, 1))
    return ORPO_ERR_SHAPE;
  if (batch == 0 || columns == 0) return ORPO_OK;
  if (!table || !refs || !status) return ORPO_ERR_NULL;
  if (misaligned({table, refs, status})) return ORPO_ERR_ALIGN;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  const TableArgs t{table, ld_table, columns, refs, (int32_t)pages, 1, nullptr, 0, nullptr, nullptr, 0, batch, beams, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(batch * beams), (unsigned)std::min<int64_t>(65535, cdiv(columns, kReleaseThreads)));
  prof_begin(K_PAGES, st);
  const cudaError_t e = launch_dependent(release_kernel, grid, kReleaseThreads, 0, st, t, ended);
  prof_end(K_PAGES, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}

int orpo_pages_compact(const int32_t* table, int64_t ld_table, int64_t columns, int64_t table_rows, const int32_t* refs,
                       int64_t pages, int64_t page, int32_t* new_table, int64_t ld_new, int32_t* new_refs, int32_t* live,
                       int32_t* moves, int64_t max_moves, int32_t* n_moves, void* workspace, size_t ws_bytes, int32_t* status,
                       void* stream) {
  if (!table_ok(table_rows, ld_table, columns, pages, page) || ld_new < columns || max_moves < pages / 2 ||
      (new_table == table && ld_new != ld_table))
    return ORPO_ERR_SHAPE;
  const bool entries = table_rows > 0 && columns > 0;
  if ((entries && (!table || !new_table)) || !refs || !new_refs || !live || (max_moves > 0 && !moves) || !n_moves || !workspace ||
      !status)
    return ORPO_ERR_NULL;
  if (misaligned({table, refs, new_table, new_refs, live, moves, n_moves, status}) || !aligned16(workspace)) return ORPO_ERR_ALIGN;
  if (ws_bytes < compact_bytes(pages)) return ORPO_ERR_WORKSPACE;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int ctas = plan_ctas(0, pages);
  CompactArgs a{table, ld_table, columns, table_rows, refs, (int32_t)pages, (int32_t)page, new_table, ld_new, new_refs, live, moves,
                n_moves, share(pages, ctas, 32 * kWarps), nullptr, nullptr, nullptr, status};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.holes = reinterpret_cast<int32_t*>(ws);
  a.movers = reinterpret_cast<int32_t*>(ws += align16(pages / 2 * 4));
  a.below = reinterpret_cast<int32_t*>(ws += align16(pages * 4));
  const int here = table_rows * columns > (int64_t)ctas * kRemapHere ? 0 : ctas > 1 ? 1 : 2;
  static std::atomic<int> done[64];
  const size_t smem = here == 2 ? (size_t)(2 * pages + pages / 2) * 4 : 0;
  cudaError_t e = opt_in_smem(compact_kernel, (int)kOneCta * 10, done);
  prof_begin(K_PAGES, st);
  if (e == cudaSuccess) e = launch_cluster_dependent(compact_kernel, ctas, kPlanThreads, smem, st, a, here);
  if (e == cudaSuccess && !here) {
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)sms * 8, cdiv(table_rows * columns, kRemapThreads));
    e = launch_dependent(remap_kernel, grid, kRemapThreads, 0, st, a);
  }
  prof_end(K_PAGES, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}

}  // extern "C"
