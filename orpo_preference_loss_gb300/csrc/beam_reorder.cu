// beam_reorder.cu — per-beam states follow their parents, in place (orpo_beam_reorder).
//
//   state[o, b, k, r, t, :] <- state[o, b, parent[b, k], r, t, :]   for t < length[b]
//
// Units that start on 4, 8 or 16 bytes, in pieces of as many: one thread owns the same piece of a (slab, entry, row)
// in all beams of the entry: it reads every moved beam's source before it writes any, and no other thread touches
// those, so the parents may form any map (cycles, many children) without a second buffer.  A source that several
// beams take is asked for several times by one thread, of which L1 makes one.  Above 8 beams a thread's sources
// would leave too few threads their registers: there a CTA takes kTile pieces of all moved beams through shared memory
// (9 beams, 114 MB: 28 us; with 16 sources in registers 35).
// Units of any other size: beams start at any byte.  A CTA takes a window of a (slab, entry, row) through shared
// memory; each source lies there as far from a 16-byte boundary as in memory, and what goes out is put together for
// the destination's own boundaries by funnel shifts, so that all but the ends moves 16 bytes at a time (bf16 heads of
// 33, 6 beams, 254 MB: 72 us; in pieces of 2 bytes 91.  Heads of 36 in pieces of 8 bytes: 64, and by bytes 78).
// Bound by the bytes moved, so each CTA stays with one (slab, entry, row) for up to kMaxPer pieces, with 16
// loads of a thread in flight, and reads the parents once: one piece per thread and CTA cost a
// quarter of the rate.  Measured: 524 MB (16 slabs, 8 x 4 beams, 3 moved, heads of 128 bf16) 81 us, 6.5 TB/s or 96% of
// the rate of a plain copy.
#include <algorithm>

#include "../../include/orpo_decode.h"
#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

struct ReorderArgs {
  uint8_t* state;
  const int32_t* parent;
  int64_t ld_parent;
  const int32_t* length;
  int64_t outer, batch, rows, capacity, unit;
  int beams;
  int32_t* status;
  int64_t per;  // 16-byte pieces (other units: bytes) per CTA
};

constexpr int kThreads = 256;

// Whether `n` bytes from `p` on are this launch's (bounds-checked build).
__device__ __forceinline__ bool in_state(const ReorderArgs& a, const void* p, int n) {
  const int64_t at = static_cast<const uint8_t*>(p) - a.state, size = a.outer * a.batch * a.beams * a.rows * a.capacity * a.unit;
  return in_bounds(a.status, at, size) && in_bounds(a.status, at + n - 1, size);
}

// A CTA's (slab, entry, row), of at most 2^30.
struct Run {
  uint32_t o, b, row;
  __device__ __forceinline__ explicit Run(const ReorderArgs& a) {
    const uint32_t ob = blockIdx.x / (uint32_t)a.rows;
    row = blockIdx.x - ob * (uint32_t)a.rows;
    o = ob / (uint32_t)a.batch;
    b = ob - o * (uint32_t)a.batch;
  }
};

template <class T, int KB>
__global__ void __launch_bounds__(kThreads) reorder_kernel(ReorderArgs a) {
  constexpr int kUnroll = 16 / KB;  // pieces of a thread in flight per beam
  grid_trigger();
  grid_wait();
  const Run run(a);
  const int64_t row = run.row, b = run.b, o = run.o;
  __shared__ int par[KB];
  const int64_t len = a.length ? (int64_t)a.length[b] : a.capacity;
  const int64_t used = len * a.unit / (int64_t)sizeof(T);
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(begin + a.per, used);
  bool bad = len < 0 || len > a.capacity;
  if (threadIdx.x < KB) {
    const int k = threadIdx.x;
    const int p = k < a.beams && in_bounds(a.status, b, a.batch) ? a.parent[b * a.ld_parent + k] : k;
    bad |= k < a.beams && (p < 0 || p >= a.beams);
    par[k] = p;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(a.status, ORPO_STATUS_PARENT);
    return;
  }
  const int64_t beam_units = a.rows * a.capacity * a.unit / (int64_t)sizeof(T);
  T* base = reinterpret_cast<T*>(a.state) + (o * a.batch + b) * a.beams * beam_units +
            row * (a.capacity * a.unit / (int64_t)sizeof(T));
  for (int64_t i = begin + threadIdx.x; i < end; i += kThreads * kUnroll) {
    T v[kUnroll][KB];
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k) {
        const T* src = base + par[k] * beam_units + i;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if ((u == 0 || i + u * kThreads < end) && in_state(a, src + u * kThreads, sizeof(T))) v[u][k] = src[u * kThreads];
      }
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k) {
        T* dst = base + k * beam_units + i;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if ((u == 0 || i + u * kThreads < end) && in_state(a, dst + u * kThreads, sizeof(T))) dst[u * kThreads] = v[u][k];
      }
  }
}

// Any number of beams: kTile units of every moved beam's source into shared memory, then out.
constexpr int kTile = 128;

// The moved beams of an entry, in any order; false (for the whole CTA) on a bad parent or length.
struct Moves {
  int from[ORPO_MAX_BEAMS], to[ORPO_MAX_BEAMS], n;
};
__device__ __forceinline__ bool find_moves(const ReorderArgs& a, int64_t b, int64_t len, Moves& m) {
  bool bad = len < 0 || len > a.capacity;
  if (threadIdx.x == 0) m.n = 0;
  __syncthreads();
  if (threadIdx.x < a.beams) {
    const int k = threadIdx.x, p = in_bounds(a.status, b, a.batch) ? a.parent[b * a.ld_parent + k] : k;
    bad |= p < 0 || p >= a.beams;
    if (p != k) {
      const int j = atomicAdd(&m.n, 1);
      if (in_bounds(a.status, j, ORPO_MAX_BEAMS)) m.from[j] = p, m.to[j] = k;
    }
  }
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0) atomicOr(a.status, ORPO_STATUS_PARENT);
  return false;
}

template <class T>
__global__ void __launch_bounds__(kThreads) reorder_tile_kernel(ReorderArgs a) {
  extern __shared__ __align__(16) uint8_t tile_raw[];
  T* const tile = reinterpret_cast<T*>(tile_raw);  // [moved][kTile]
  grid_trigger();
  grid_wait();
  __shared__ Moves moves;
  const Run run(a);
  const int64_t row = run.row, b = run.b, o = run.o;
  const int64_t len = a.length ? (int64_t)a.length[b] : a.capacity;
  const int64_t used = len * a.unit / (int64_t)sizeof(T);
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(begin + a.per, used);
  if (!find_moves(a, b, len, moves)) return;
  const int64_t beam_units = a.rows * a.capacity * a.unit / (int64_t)sizeof(T);
  T* base = reinterpret_cast<T*>(a.state) + (o * a.batch + b) * a.beams * beam_units +
            row * (a.capacity * a.unit / (int64_t)sizeof(T));
  const int n = moves.n * kTile, slots = a.beams * kTile;
  for (int64_t i = begin; i < end; i += kTile) {
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const T* const src = base + moves.from[j / kTile] * beam_units + i + j % kTile;
      if (i + j % kTile < end && in_bounds(a.status, j, slots) && in_state(a, src, sizeof(T))) tile[j] = *src;
    }
    __syncthreads();  // every beam's units are read
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += kThreads) {
      T* const dst = base + moves.to[j / kTile] * beam_units + i + j % kTile;
      if (i + j % kTile < end && in_bounds(a.status, j, slots) && in_state(a, dst, sizeof(T))) *dst = tile[j];
    }
    __syncthreads();
  }
}

// Units of any size.  Windows of `window` bytes (a multiple of 16) of every moved beam.
__global__ void __launch_bounds__(kThreads) reorder_bytes_kernel(ReorderArgs a, int window) {
  extern __shared__ __align__(16) uint8_t tile_raw[];  // [moved][window + 32]: bytes from the boundary before the source on
  grid_trigger();
  grid_wait();
  __shared__ Moves moves;
  const Run run(a);
  const int64_t len = a.length ? (int64_t)a.length[run.b] : a.capacity;
  const int64_t used = len * a.unit;
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(begin + a.per, used);
  if (!find_moves(a, run.b, len, moves)) return;
  const int64_t run_bytes = a.capacity * a.unit, beam_bytes = a.rows * run_bytes;
  uint8_t* const base = a.state + ((int64_t)run.o * a.batch + run.b) * a.beams * beam_bytes + run.row * run_bytes;
  const uint32_t chunks = (uint32_t)window / 16, n = moves.n * chunks, ends = moves.n * 32;
  const int pitch = window + 32, tile_size = a.beams * pitch;
  for (int64_t w0 = begin; w0 < end; w0 += window) {
    const int size = (int)min((int64_t)window, end - w0);
    // of the bytes [p, p + size): those before the first boundary, and whole 16-byte chunks
    auto head_of = [&](const uint8_t* p) { return min(size, (int)(-reinterpret_cast<uintptr_t>(p) & 15u)); };
    // byte e (0..31) of a beam's ends: its place in the window, or -1
    auto end_byte = [&](int head, int e) {
      const int tail = head + (size - head) / 16 * 16 + e - 16;
      return e < 16 ? (e < head ? e : -1) : tail < size ? tail : -1;
    };
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t j = i / chunks, c = i - j * chunks;
      const uint8_t* const src = base + moves.from[j] * beam_bytes + w0;
      const int at = head_of(src) + (int)c * 16;
      const int to = (int)(j * pitch + (reinterpret_cast<uintptr_t>(src) & 15u)) + at;
      if (at + 16 <= size && in_bounds(a.status, to + 15, tile_size) && in_state(a, src + at, 16))
        *reinterpret_cast<uint4*>(tile_raw + to) = *reinterpret_cast<const uint4*>(src + at);
    }
    for (uint32_t i = threadIdx.x; i < ends; i += kThreads) {
      const uint32_t j = i / 32;
      const uint8_t* const src = base + moves.from[j] * beam_bytes + w0;
      const int at = end_byte(head_of(src), (int)(i & 31u));
      const int to = (int)(j * pitch + (reinterpret_cast<uintptr_t>(src) & 15u)) + at;
      if (at >= 0 && in_bounds(a.status, to, tile_size) && in_state(a, src + at, 1)) tile_raw[to] = src[at];
    }
    __syncthreads();  // every beam's window is read
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t j = i / chunks, c = i - j * chunks;
      const uint8_t* const src = base + moves.from[j] * beam_bytes + w0;
      uint8_t* const dst = base + moves.to[j] * beam_bytes + w0;
      const int at = head_of(dst) + (int)c * 16;
      if (at + 16 <= size) {
        const uint32_t off = j * pitch + (uint32_t)(reinterpret_cast<uintptr_t>(src) & 15u) + at, shift = (off & 3u) * 8;
        const uint32_t* const w = reinterpret_cast<const uint32_t*>(tile_raw) + off / 4;  // 5 words: inside the slot's slack
        if (!in_bounds(a.status, off / 4 * 4 + 19, tile_size) || !in_state(a, dst + at, 16)) continue;
        uint32_t x[5];
#pragma unroll
        for (int e = 0; e < 5; ++e) x[e] = w[e];
        *reinterpret_cast<uint4*>(dst + at) = make_uint4(__funnelshift_r(x[0], x[1], shift), __funnelshift_r(x[1], x[2], shift),
                                                         __funnelshift_r(x[2], x[3], shift), __funnelshift_r(x[3], x[4], shift));
      }
    }
    for (uint32_t i = threadIdx.x; i < ends; i += kThreads) {
      const uint32_t j = i / 32;
      const uint8_t* const src = base + moves.from[j] * beam_bytes + w0;
      uint8_t* const dst = base + moves.to[j] * beam_bytes + w0;
      const int at = end_byte(head_of(dst), (int)(i & 31u));
      const int from = (int)(j * pitch + (reinterpret_cast<uintptr_t>(src) & 15u)) + at;
      if (at >= 0 && in_bounds(a.status, from, tile_size) && in_state(a, dst + at, 1)) dst[at] = tile_raw[from];
    }
    __syncthreads();
  }
}

constexpr int64_t kMaxPer = 8192;  // pieces per CTA at most
constexpr int64_t kMinPer = 512;   // and at least, where a run has as many
constexpr int kBytesSmem = 36 << 10;

// Piece: uint4, uint2, uint32_t, or uint8_t for the kernel of any units (in 16-byte chunks)
template <class Piece>
cudaError_t launch(const ReorderArgs& a, int sms, cudaStream_t st) {
  constexpr bool kBytes = sizeof(Piece) == 1;
  constexpr int64_t kPiece = kBytes ? 16 : sizeof(Piece);
  // slabs in launches of at most 2^30 runs
  const int64_t runs = a.batch * a.rows;
  const int64_t slabs = std::max<int64_t>(1, (1ll << 30) / runs);
  const int64_t slab_bytes = a.batch * a.beams * a.rows * a.capacity * a.unit;
  const int64_t pieces = cdiv(a.capacity * a.unit, kPiece);
  const int window = std::min(4096, kBytesSmem / a.beams / 16 * 16 - 32);  // at least 544
  for (int64_t o = 0; o < a.outer; o += slabs) {
    ReorderArgs c = a;
    c.state = a.state + o * slab_bytes;
    c.outer = std::min(slabs, a.outer - o);
    // about sixteen CTAs per SM, but at most 65535 per run
    const int64_t want = cdiv(pieces * c.outer * runs, (int64_t)sms * 16);
    const int64_t per = std::max(std::min(kMaxPer, std::max(kMinPer, want)), cdiv(pieces, 65535));
    const int64_t step = kBytes ? window / 16 : kThreads;
    c.per = cdiv(per, step) * step;
    const dim3 grid((unsigned)(c.outer * runs), (unsigned)cdiv(pieces, c.per));
    prof_begin(K_REORDER, st);
    cudaError_t e;
    if constexpr (kBytes) {
      c.per *= 16;
      e = launch_dependent(reorder_bytes_kernel, grid, kThreads, (size_t)a.beams * (window + 32), st, c, window);
    } else if (a.beams <= 4) {
      e = launch_dependent(reorder_kernel<Piece, 4>, grid, kThreads, 0, st, c);
    } else if (a.beams <= 8) {
      e = launch_dependent(reorder_kernel<Piece, 8>, grid, kThreads, 0, st, c);
    } else {
      static std::atomic<int> done[64];
      e = opt_in_smem(reorder_tile_kernel<Piece>, ORPO_MAX_BEAMS * kTile * (int)sizeof(Piece), done);
      if (e == cudaSuccess) e = launch_dependent(reorder_tile_kernel<Piece>, grid, kThreads, a.beams * kTile * sizeof(Piece), st, c);
    }
    prof_end(K_REORDER, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// product of non-negative sizes, or -1 when it reaches 2^62
int64_t product(std::initializer_list<int64_t> f) {
  int64_t p = 1;
  for (int64_t x : f) {
    if (x == 0) return 0;
  }
  for (int64_t x : f) {
    if (p > ((1ll << 62) - 1) / x) return -1;
    p *= x;
  }
  return p;
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" int orpo_beam_reorder(void* state, const int32_t* parent, int64_t ld_parent, const int32_t* length,
                                 int64_t outer, int64_t batch, int beams, int64_t rows, int64_t capacity,
                                 int64_t unit_bytes, int32_t* status, void* stream) {
  if (outer < 0 || batch < 0 || beams < 1 || beams > ORPO_MAX_BEAMS || rows < 0 || capacity < 0 || unit_bytes < 0 ||
      ld_parent < beams)
    return ORPO_ERR_SHAPE;
  const int64_t bytes = product({outer, batch, (int64_t)beams, rows, capacity, unit_bytes});
  if (bytes < 0) return ORPO_ERR_SHAPE;
  if (bytes == 0) return ORPO_OK;
  if (batch * rows > (1ll << 30)) return ORPO_ERR_SHAPE;
  if (!state || !parent || !status) return ORPO_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(parent) | reinterpret_cast<uintptr_t>(length)) & 3) return ORPO_ERR_ALIGN;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  const ReorderArgs a{static_cast<uint8_t*>(state), parent, ld_parent, length, outer, batch, rows, capacity,
                      unit_bytes, beams, status, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t al = (uint64_t)reinterpret_cast<uintptr_t>(state) | (uint64_t)unit_bytes;
  const cudaError_t e = al % 16 == 0  ? launch<uint4>(a, sms, st)
                        : al % 8 == 0 ? launch<uint2>(a, sms, st)
                        : al % 4 == 0 ? launch<uint32_t>(a, sms, st)
                                      : launch<uint8_t>(a, sms, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
