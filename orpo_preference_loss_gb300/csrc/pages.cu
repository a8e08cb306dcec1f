// pages.cu — beam states in shared pages (orpo_pages.h): page tables follow the beams' parents, pages are taken, copied on
// write, released and compacted.
//
// A page is free when its count of holders is 0, and free pages are always taken lowest first, so there is no list of free
// pages to keep and no order for atomics to change: counts are integers, and every choice follows the order of rows,
// columns and page numbers.
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
  const int64_t used = (begin + a.page - 1) / a.page, b0 = b * a.beams * a.ld, all = a.batch * a.beams * a.ld;
  for (int64_t c = (int64_t)blockIdx.y * kForkThreads + tid; c < used; c += (int64_t)gridDim.y * kForkThreads) {
    int32_t* const column = a.table + b0 + c;
    int32_t was[KB], now[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k && in_bounds(a.status, b0 + c + k * a.ld, all)) {
        was[k] = column[k * a.ld];
        now[k] = column[par[k] * a.ld];
      }
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k && was[k] != now[k] && in_bounds(a.status, b0 + c + k * a.ld, all)) {
        column[k * a.ld] = now[k];
        if (is_page(a, now[k])) atomicAdd(a.refs + now[k], 1);
        if (is_page(a, was[k])) atomicSub(a.refs + was[k], 1);
        if (now[k] < -1 || now[k] >= a.pages || was[k] < -1 || was[k] >= a.pages) atomicOr(a.status, ORPO_STATUS_PAGE);
      }
  }
}

// ------------------------------------------------------------------ scans over one CTA
constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;

// Exclusive sum of x over the CTA's threads, and the total.  `part` is kWarps words of shared memory, free again at the
// next barrier.
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
  const uint32_t w = part[lane];
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

// ------------------------------------------------------------------ reserve
// Items are (row, column) pairs of the positions asked for, in order: `width` columns per row, of which those from the
// end of the row's positions on ask for nothing.
struct ReserveArgs {
  TableArgs t;
  const int32_t* left_alone;  // entries that the fork found wrong; nullptr without a fork
  int32_t* moves;
  int32_t* n_moves;
  int32_t width;
  int32_t items;
  int32_t* count;  // [pages] how many items hold a page that others hold too,
  int32_t* last;   // [pages] and the last of them
  int32_t* rank;   // [items] number of the item's new page among the new ones, or -1
  int32_t* fresh;  // [items] the new pages
};

struct Item {
  bool inside;
  int32_t old, fill;
  int32_t* entry;
};

__device__ __forceinline__ Item item_at(const ReserveArgs& a, int32_t i) {
  Item it{false, -1, 0, nullptr};
  if (i >= a.items) return it;
  const int32_t row = i / a.width, j = i - row * a.width, b = row / a.t.beams;
  int64_t begin, end;
  if ((a.left_alone && a.left_alone[b]) || !wanted(a.t, b, begin, end) || begin == end) return it;
  const int64_t c = begin / a.t.page + j;
  if (c * a.t.page >= end || !in_bounds(a.t.status, c, a.t.columns)) return it;
  it.entry = a.t.table + row * a.t.ld + c;
  it.old = *it.entry;
  it.inside = it.old >= -1 && it.old < a.t.pages;
  it.fill = j == 0 ? (int32_t)(begin % a.t.page) : 0;
  return it;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(ReserveArgs a) {
  __shared__ uint32_t part[kWarps];
  grid_trigger();
  grid_wait();
  const int tid = threadIdx.x;
  const int32_t pages = a.t.pages;
  if (!a.left_alone)
    for (int64_t b = tid; b < a.t.batch; b += kPlanThreads) {
      int64_t begin, end;
      if (!wanted(a.t, b, begin, end)) atomicOr(a.t.status, ORPO_STATUS_PARENT);
    }
  // which of the items that hold a page together is the last: it keeps the page where nothing else holds it
  for (int32_t i = tid; i < a.items; i += kPlanThreads) {
    const Item it = item_at(a, i);
    if (it.inside && it.old >= 0 && a.t.refs[it.old] > 1) a.count[it.old] = 0, a.last[it.old] = -1;
    if (it.entry && !it.inside) atomicOr(a.t.status, ORPO_STATUS_PAGE);
  }
  __syncthreads();
  for (int32_t i = tid; i < a.items; i += kPlanThreads) {
    const Item it = item_at(a, i);
    if (it.inside && it.old >= 0 && a.t.refs[it.old] > 1) atomicAdd(a.count + it.old, 1), atomicMax(a.last + it.old, i);
  }
  __syncthreads();
  uint32_t needed = 0, moved = 0;
  for (int32_t i0 = 0; i0 < a.items; i0 += kPlanThreads) {
    const int32_t i = i0 + tid;
    const Item it = item_at(a, i);
    bool need = it.inside;
    if (need && it.old >= 0) {
      const int32_t held = a.t.refs[it.old];
      need = held > 1 && !(__ldcg(a.count + it.old) == held && __ldcg(a.last + it.old) == i);
    }
    uint32_t total;
    const uint32_t at = scan(need, part, total);
    if (i < a.items && in_bounds(a.t.status, i, a.items)) a.rank[i] = need ? (int32_t)(needed + at) : -1;
    needed += total;
  }
  uint32_t found = 0;
  for (int32_t p0 = 0; p0 < pages && found < needed; p0 += kPlanThreads) {
    const int32_t p = p0 + tid;
    const bool free = p < pages && a.t.refs[p] <= 0;
    uint32_t total;
    const uint32_t at = found + scan(free, part, total);
    if (free && at < needed && in_bounds(a.t.status, at, a.items)) a.fresh[at] = p;
    found += total;
  }
  if (found < needed) {
    if (tid == 0) {
      atomicOr(a.t.status, ORPO_STATUS_FULL);
      *a.n_moves = 0;
    }
    return;
  }
  __syncthreads();
  for (int32_t i0 = 0; i0 < a.items; i0 += kPlanThreads) {
    const int32_t i = i0 + tid;
    const Item it = item_at(a, i);
    const int32_t rank = i < a.items ? a.rank[i] : -1;
    const bool move = rank >= 0 && it.old >= 0 && it.fill > 0;
    uint32_t total;
    const uint32_t at = moved + scan(move, part, total);
    if (rank >= 0 && in_bounds(a.t.status, rank, a.items)) {
      const int32_t p = a.fresh[rank];
      *it.entry = p;
      a.t.refs[p] = 1;
      if (it.old >= 0) atomicSub(a.t.refs + it.old, 1);
      if (move && in_bounds(a.t.status, at, a.t.batch * a.t.beams)) {
        a.moves[3 * at] = it.old;
        a.moves[3 * at + 1] = p;
        a.moves[3 * at + 2] = it.fill;
      }
    }
    moved += total;
  }
  if (tid == 0) *a.n_moves = (int32_t)moved;
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
  int64_t stretches;  // of one (slab, page, row)
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;  // pieces of a lane in flight

// A warp takes a stretch of kCopyUnroll * 32 pieces of one (move, slab, row).
template <class Piece>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  constexpr int kStretch = kCopyUnroll * 32;
  grid_trigger();
  grid_wait();
  const int32_t n = *a.n_moves;
  const int64_t warp = ((int64_t)blockIdx.x * kCopyThreads + threadIdx.x) / 32, warps = (int64_t)gridDim.x * kCopyThreads / 32;
  const int lane = threadIdx.x & 31;
  if (n < 0 || n > a.max_moves) {
    if (warp == 0 && lane == 0) atomicOr(a.status, ORPO_STATUS_PAGE);
    return;
  }
  const int64_t run = (int64_t)a.page * a.unit, stretches = a.stretches, per_move = a.outer * a.rows * stretches;
  const int64_t all = a.outer * a.pages * a.page_bytes;
  for (int64_t w = warp; w < n * per_move; w += warps) {
    const int64_t m = w / per_move, left = w - m * per_move, run_at = left / stretches, s = left - run_at * stretches;
    const int64_t o = run_at / a.rows, r = run_at - o * a.rows;
    const int32_t from = a.moves[3 * m], to = a.moves[3 * m + 1], positions = a.moves[3 * m + 2];
    if (from < 0 || from >= a.pages || to < 0 || to >= a.pages || from == to || positions < 0 || positions > a.page) {
      if (left == 0 && lane == 0) atomicOr(a.status, ORPO_STATUS_PAGE);
      continue;
    }
    const int64_t bytes = (int64_t)positions * a.unit, pieces = bytes / (int64_t)sizeof(Piece);
    const int64_t src = (o * a.pages + from) * a.page_bytes + r * run, dst = (o * a.pages + to) * a.page_bytes + r * run;
    Piece v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int64_t i = s * kStretch + u * 32 + lane;
      if (i < pieces && in_bounds(a.status, src + (i + 1) * (int64_t)sizeof(Piece) - 1, all))
        v[u] = reinterpret_cast<const Piece*>(a.pool + src)[i];
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int64_t i = s * kStretch + u * 32 + lane;
      if (i < pieces && in_bounds(a.status, dst + (i + 1) * (int64_t)sizeof(Piece) - 1, all))
        reinterpret_cast<Piece*>(a.pool + dst)[i] = v[u];
    }
    // what is left of a run whose positions do not fill whole pieces
    const int64_t i = pieces * (int64_t)sizeof(Piece) + lane;
    if (s == 0 && i < bytes && in_bounds(a.status, dst + i, all) && in_bounds(a.status, src + i, all)) a.pool[dst + i] = a.pool[src + i];
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
  int32_t* holes;   // [pages / 2]
  int32_t* movers;  // [pages / 2]
  int32_t* to;      // [pages] where a page at or above `live` goes; -1: nowhere
  int32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) compact_kernel(CompactArgs a) {
  __shared__ uint32_t part[kWarps];
  grid_trigger();
  grid_wait();
  const int tid = threadIdx.x;
  uint32_t mine = 0, n;
  for (int32_t p = tid; p < a.pages; p += kPlanThreads) mine += a.refs[p] > 0;
  scan(mine, part, n);
  const int32_t live = (int32_t)n;
  uint32_t holes = 0, movers = 0;
  for (int32_t p0 = 0; p0 < a.pages; p0 += kPlanThreads) {
    const int32_t p = p0 + tid;
    const bool used = p < a.pages && a.refs[p] > 0;
    const bool hole = p < live && !used, mover = p >= live && used;
    uint32_t total;
    const uint32_t at = scan((uint32_t)hole | (uint32_t)mover << 16, part, total);
    if (hole && in_bounds(a.status, holes + (at & 0xffff), a.pages / 2)) a.holes[holes + (at & 0xffff)] = p;
    if (mover && in_bounds(a.status, movers + (at >> 16), a.pages / 2)) a.movers[movers + (at >> 16)] = p;
    if (p < a.pages && p >= live && !used) a.to[p] = -1;
    holes += total & 0xffff;
    movers += total >> 16;
  }
  __syncthreads();
  if (a.new_refs != a.refs)
    for (int32_t p = tid; p < a.pages; p += kPlanThreads)
      if (p >= live || a.refs[p] > 0) a.new_refs[p] = p < live ? a.refs[p] : 0;
  for (int32_t i = tid; i < (int32_t)movers; i += kPlanThreads) {
    if (!in_bounds(a.status, i, a.pages / 2)) continue;
    const int32_t from = a.movers[i], to = a.holes[i];
    a.moves[3 * i] = from;
    a.moves[3 * i + 1] = to;
    a.moves[3 * i + 2] = a.page;
    a.to[from] = to;
    a.new_refs[to] = a.refs[from];
    if (a.new_refs == a.refs) a.new_refs[from] = 0;
  }
  if (tid == 0) {
    *a.n_moves = (int32_t)movers;
    *a.live = live;
  }
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads) remap_kernel(CompactArgs a) {
  grid_trigger();
  grid_wait();
  const int32_t live = *a.live;
  const int64_t row = blockIdx.x;
  int wrong = 0;
  for (int64_t c = (int64_t)blockIdx.y * kRemapThreads + threadIdx.x; c < a.columns; c += (int64_t)gridDim.y * kRemapThreads) {
    if (!in_bounds(a.status, row * a.ld + c, a.rows * a.ld) || !in_bounds(a.status, row * a.ld_new + c, a.rows * a.ld_new)) continue;
    int32_t e = a.table[row * a.ld + c];
    if (e < -1 || e >= a.pages) {
      wrong = 1;
    } else if (e >= live) {
      const int32_t to = a.to[e];
      if (to >= 0) e = to; else wrong = 1;
    }
    a.new_table[row * a.ld_new + c] = e;
  }
  if (wrong) atomicOr(a.status, ORPO_STATUS_PAGE);
}

// ------------------------------------------------------------------ host
constexpr int64_t kMaxPages = 1ll << 24, kMaxPage = 1ll << 16, kMaxInt = (1ll << 31) - 1;

bool table_ok(int64_t table_rows, int64_t ld, int64_t columns, int64_t pages, int64_t page) {
  return table_rows >= 0 && table_rows <= (1ll << 20) && columns >= 0 && columns <= kMaxInt && ld >= columns && pages >= 1 &&
         pages <= kMaxPages && page >= 1 && page <= kMaxPage && columns * page <= kMaxInt && table_rows * columns <= kMaxInt;
}

int64_t width_of(int64_t most, int64_t page) { return most > 0 ? cdiv(most - 1, page) + 1 : 0; }

size_t align16(size_t n) { return (n + 15) / 16 * 16; }
size_t reserve_bytes(int64_t batch, int64_t pages, int64_t items) {
  return align16(batch * 4) + 2 * align16(pages * 4) + 2 * align16(items * 4);
}
size_t compact_bytes(int64_t pages) { return 2 * align16(pages / 2 * 4) + align16(pages * 4); }

bool misaligned(std::initializer_list<const void*> p) {
  uintptr_t at = 0;
  for (const void* x : p) at |= reinterpret_cast<uintptr_t>(x);
  return at & 3;
}

template <class Piece>
cudaError_t launch_copy(CopyArgs a, int sms, cudaStream_t st) {
  a.stretches = cdiv((int64_t)a.page * a.unit, (int64_t)sizeof(Piece) * kCopyUnroll * 32);
  const int64_t warps = (int64_t)a.max_moves * a.outer * a.rows * a.stretches;  // at most
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
  const int64_t items = table_rows * width_of(most, page);
  if (items > kMaxInt) return 0;
  return std::max(std::max(reserve_bytes(table_rows, pages, items), compact_bytes(pages)), (size_t)16);
}

int orpo_pages_advance(int32_t* table, int64_t ld_table, int64_t columns, int32_t* refs, int64_t pages, int64_t page,
                       const int32_t* parent, int64_t ld_parent, const int32_t* length, const int32_t* more, int64_t most,
                       int64_t batch, int beams, int32_t* moves, int64_t max_moves, int32_t* n_moves, void* workspace,
                       size_t ws_bytes, int32_t* status, void* stream) {
  if (batch < 0 || batch > (1ll << 20) || beams < 1 || beams > ORPO_MAX_BEAMS ||
      !table_ok(batch * beams, ld_table, columns, pages, page) || most < 0 || most > kMaxInt || (parent && ld_parent < beams) ||
      max_moves < batch * beams)
    return ORPO_ERR_SHAPE;
  const int64_t width = width_of(most, page), items = batch * beams * width;
  if (items > kMaxInt) return ORPO_ERR_SHAPE;
  if (!n_moves || !status || (batch > 0 && ((columns > 0 && !table) || !refs || !length || !moves || !workspace))) return ORPO_ERR_NULL;
  if (misaligned({table, refs, parent, length, more, moves, n_moves, status}) || !aligned16(workspace)) return ORPO_ERR_ALIGN;
  if (ws_bytes < (batch > 0 ? reserve_bytes(batch, pages, items) : 0)) return ORPO_ERR_WORKSPACE;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const TableArgs t{table, ld_table, columns, refs, (int32_t)pages, (int32_t)page, parent, ld_parent, length, more, (int32_t)most,
                    batch, beams, status};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ReserveArgs a{t, nullptr, moves, n_moves, (int32_t)std::max<int64_t>(width, 1), (int32_t)items, nullptr, nullptr, nullptr, nullptr};
  int32_t* const left_alone = reinterpret_cast<int32_t*>(ws);
  a.count = reinterpret_cast<int32_t*>(ws += align16(batch * 4));
  a.last = reinterpret_cast<int32_t*>(ws += align16(pages * 4));
  a.rank = reinterpret_cast<int32_t*>(ws += align16(pages * 4));
  a.fresh = reinterpret_cast<int32_t*>(ws += align16(items * 4));
  cudaError_t e = cudaSuccess;
  prof_begin(K_PAGES, st);
  if (parent && batch > 0) {
    a.left_alone = left_alone;
    const dim3 grid((unsigned)batch, (unsigned)std::max<int64_t>(1, std::min<int64_t>(65535, cdiv(columns, kForkThreads))));
    e = beams <= 4    ? launch_dependent(fork_kernel<4>, grid, kForkThreads, 0, st, t, left_alone)
        : beams <= 8  ? launch_dependent(fork_kernel<8>, grid, kForkThreads, 0, st, t, left_alone)
        : beams <= 16 ? launch_dependent(fork_kernel<16>, grid, kForkThreads, 0, st, t, left_alone)
                      : launch_dependent(fork_kernel<64>, grid, kForkThreads, 0, st, t, left_alone);
  }
  if (e == cudaSuccess) e = launch_dependent(reserve_kernel, dim3(1), kPlanThreads, 0, st, a);
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
                   (int32_t)max_moves, n_moves, status, 0};
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
  CompactArgs a{table, ld_table, columns, table_rows, refs, (int32_t)pages, (int32_t)page, new_table, ld_new, new_refs, live, moves,
                n_moves, nullptr, nullptr, nullptr, status};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.holes = reinterpret_cast<int32_t*>(ws);
  a.movers = reinterpret_cast<int32_t*>(ws += align16(pages / 2 * 4));
  a.to = reinterpret_cast<int32_t*>(ws += align16(pages / 2 * 4));
  prof_begin(K_PAGES, st);
  cudaError_t e = launch_dependent(compact_kernel, dim3(1), kPlanThreads, 0, st, a);
  if (e == cudaSuccess && entries) {
    const dim3 grid((unsigned)table_rows, (unsigned)std::min<int64_t>(65535, cdiv(columns, kRemapThreads)));
    e = launch_dependent(remap_kernel, grid, kRemapThreads, 0, st, a);
  }
  prof_end(K_PAGES, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}

}  // extern "C"
