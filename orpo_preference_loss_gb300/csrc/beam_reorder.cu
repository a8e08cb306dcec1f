// beam_reorder.cu — per-beam states follow their parents, in place (orpo_beam_reorder).
//
//   state[o, b, k, r, t, :] <- state[o, b, parent[b, k], r, t, :]   for t < length[b]
//
// One thread owns the same unit of a (slab, entry, row) in all beams of the entry: it reads every
// moved beam's source before it writes any, and no other thread touches that unit, so the parents
// may form any map (cycles, many children) without a second buffer.  A unit that several beams take is
// asked for several times by one thread, of which L1 makes one.  The unit is the widest of 16, 8, 4,
// 2 or 1 bytes that the address and the two byte strides allow.  Above 16 beams a thread's units would not
// fit its registers: there a CTA takes kTile units of all moved beams through shared memory.
// Bound by the bytes moved, so each CTA stays with one (slab, entry, row) for up to kMaxPer units, with 16
// loads of a thread in flight, and reads the parents once: one unit per thread and CTA cost a
// quarter of the rate.
#include <algorithm>

#include "../../include/orpo_decode.h"
#include "internal.h"

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
  int64_t per;  // units per CTA
};

constexpr int kThreads = 256;

template <class T, int KB>
__global__ void __launch_bounds__(kThreads) reorder_kernel(ReorderArgs a) {
  constexpr int kUnroll = KB <= 8 ? 16 / KB : 1;  // units of a thread in flight per beam
  const int64_t run = blockIdx.x;                 // (slab, entry, row)
  const int64_t row = run % a.rows, ob = run / a.rows, b = ob % a.batch, o = ob / a.batch;
  __shared__ int par[KB];
  const int64_t len = a.length ? (int64_t)a.length[b] : a.capacity;
  const int64_t used = len * a.unit / (int64_t)sizeof(T);
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(begin + a.per, used);
  bool bad = len < 0 || len > a.capacity;
  if (threadIdx.x < KB) {
    const int k = threadIdx.x, p = k < a.beams ? a.parent[b * a.ld_parent + k] : k;
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
          if (u == 0 || i + u * kThreads < end) v[u][k] = src[u * kThreads];
      }
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k) {
        T* dst = base + k * beam_units + i;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u == 0 || i + u * kThreads < end) dst[u * kThreads] = v[u][k];
      }
  }
}

// Any number of beams: kTile units of every moved beam's source into shared memory, then out.
constexpr int kTile = 128;

template <class T>
__global__ void __launch_bounds__(kThreads) reorder_tile_kernel(ReorderArgs a) {
  extern __shared__ __align__(16) uint8_t tile_raw[];
  T* const tile = reinterpret_cast<T*>(tile_raw);  // [moved][kTile]
  const int64_t run = blockIdx.x;
  const int64_t row = run % a.rows, ob = run / a.rows, b = ob % a.batch, o = ob / a.batch;
  __shared__ int from[ORPO_MAX_BEAMS], to[ORPO_MAX_BEAMS], moved;
  const int64_t len = a.length ? (int64_t)a.length[b] : a.capacity;
  const int64_t used = len * a.unit / (int64_t)sizeof(T);
  const int64_t begin = (int64_t)blockIdx.y * a.per, end = min(begin + a.per, used);
  bool bad = len < 0 || len > a.capacity;
  if (threadIdx.x == 0) moved = 0;
  __syncthreads();
  if (threadIdx.x < a.beams) {
    const int k = threadIdx.x, p = a.parent[b * a.ld_parent + k];
    bad |= p < 0 || p >= a.beams;
    if (p != k) {
      const int j = atomicAdd(&moved, 1);  // their order does not matter
      from[j] = p, to[j] = k;
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(a.status, ORPO_STATUS_PARENT);
    return;
  }
  const int64_t beam_units = a.rows * a.capacity * a.unit / (int64_t)sizeof(T);
  T* base = reinterpret_cast<T*>(a.state) + (o * a.batch + b) * a.beams * beam_units +
            row * (a.capacity * a.unit / (int64_t)sizeof(T));
  const int n = moved * kTile;
  for (int64_t i = begin; i < end; i += kTile) {
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += kThreads)
      if (i + j % kTile < end) tile[j] = base[from[j / kTile] * beam_units + i + j % kTile];
    __syncthreads();  // every beam's units are read
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += kThreads)
      if (i + j % kTile < end) base[to[j / kTile] * beam_units + i + j % kTile] = tile[j];
    __syncthreads();
  }
}

constexpr int64_t kMaxPer = 8192;  // units per CTA at most
constexpr int64_t kMinPer = 512;   // and at least, where a run has as many

template <class T, int KB>  // KB = 0: any number of beams
cudaError_t launch_kb(const ReorderArgs& a, int sms, cudaStream_t st) {
  // slabs in launches of at most 2^30 runs
  const int64_t runs = a.batch * a.rows;
  const int64_t slabs = std::max<int64_t>(1, (1ll << 30) / runs);
  const int64_t slab_bytes = a.batch * a.beams * a.rows * a.capacity * a.unit;
  const int64_t units = a.capacity * a.unit / (int64_t)sizeof(T);
  for (int64_t o = 0; o < a.outer; o += slabs) {
    ReorderArgs c = a;
    c.state = a.state + o * slab_bytes;
    c.outer = std::min(slabs, a.outer - o);
    // about sixteen CTAs per SM, but at most 65535 per run
    const int64_t want = cdiv(units * c.outer * runs, (int64_t)sms * 16);
    const int64_t per = std::max(std::min(kMaxPer, std::max(kMinPer, want)), cdiv(units, 65535));
    c.per = cdiv(per, kThreads) * kThreads;
    const dim3 grid((unsigned)(c.outer * runs), (unsigned)cdiv(units, c.per));
    prof_begin(K_REORDER, st);
    if constexpr (KB != 0) {
      reorder_kernel<T, KB><<<grid, kThreads, 0, st>>>(c);
    } else {
      static std::atomic<int> done[64];
      if (cudaError_t e = opt_in_smem(reorder_tile_kernel<T>, ORPO_MAX_BEAMS * kTile * (int)sizeof(T), done)) return e;
      reorder_tile_kernel<T><<<grid, kThreads, a.beams * kTile * sizeof(T), st>>>(c);
    }
    prof_end(K_REORDER, st);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  return cudaSuccess;
}

template <class T>
cudaError_t launch(const ReorderArgs& a, int sms, cudaStream_t st) {
  if (a.beams <= 4) return launch_kb<T, 4>(a, sms, st);
  if (a.beams <= 8) return launch_kb<T, 8>(a, sms, st);
  if (a.beams <= 16) return launch_kb<T, 16>(a, sms, st);
  return launch_kb<T, 0>(a, sms, st);
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
                        : al % 2 == 0 ? launch<uint16_t>(a, sms, st)
                                      : launch<uint8_t>(a, sms, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
