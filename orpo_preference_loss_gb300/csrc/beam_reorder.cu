// beam_reorder.cu — per-beam states follow their parents, in place (orpo_beam_reorder).
//
//   state[o, b, k, r, t, :] <- state[o, b, parent[b, k], r, t, :]   for t < length[b]
//
// One thread owns the same unit of a (slab, entry, row) in all beams of the entry: it reads every
// moved beam's source before it writes any, and no other thread touches that unit, so the parents
// may form any map (cycles, many children) without a second buffer.  The unit is the widest of 16,
// 8, 4, 2 or 1 bytes that the address and the two byte strides allow.  Bound by the bytes moved.
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
};

template <class T>
__global__ void __launch_bounds__(256) reorder_kernel(ReorderArgs a) {
  const int64_t run = blockIdx.x;  // (slab, entry, row)
  const int64_t row = run % a.rows, ob = run / a.rows, b = ob % a.batch, o = ob / a.batch;
  __shared__ int par[ORPO_MAX_BEAMS];
  const int64_t len = a.length ? (int64_t)a.length[b] : a.capacity;
  bool bad = len < 0 || len > a.capacity;
  for (int k = 0; k < a.beams; ++k) {
    const int p = a.parent[b * a.ld_parent + k];
    bad |= p < 0 || p >= a.beams;
    if (threadIdx.x == 0) par[k] = p;
  }
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.status, ORPO_STATUS_PARENT);
    return;
  }
  __syncthreads();
  const int64_t beam_units = a.rows * a.capacity * a.unit / (int64_t)sizeof(T);
  T* base = reinterpret_cast<T*>(a.state) + (o * a.batch + b) * a.beams * beam_units +
            row * (a.capacity * a.unit / (int64_t)sizeof(T));
  const int64_t used = len * a.unit / (int64_t)sizeof(T);
  for (int64_t i = blockIdx.y * 256ll + threadIdx.x; i < used; i += gridDim.y * 256ll) {
    T v[ORPO_MAX_BEAMS];
    for (int k = 0; k < a.beams; ++k)
      if (par[k] != k) v[k] = base[par[k] * beam_units + i];
    for (int k = 0; k < a.beams; ++k)
      if (par[k] != k) base[k * beam_units + i] = v[k];
  }
}

template <class T>
cudaError_t launch(const ReorderArgs& a, cudaStream_t st) {
  // slabs in launches of at most 2^30 runs
  const int64_t per = a.batch * a.rows;
  const int64_t slabs = std::max<int64_t>(1, (1ll << 30) / per);
  const int64_t slab_bytes = a.batch * a.beams * a.rows * a.capacity * a.unit;
  const int64_t units = a.capacity * a.unit / (int64_t)sizeof(T);
  for (int64_t o = 0; o < a.outer; o += slabs) {
    ReorderArgs c = a;
    c.state = a.state + o * slab_bytes;
    c.outer = std::min(slabs, a.outer - o);
    const dim3 grid((unsigned)(c.outer * per), (unsigned)std::min<int64_t>(cdiv(units, 256), 64));
    prof_begin(K_REORDER, st);
    reorder_kernel<T><<<grid, 256, 0, st>>>(c);
    prof_end(K_REORDER, st);
    if (cudaError_t e = cudaGetLastError()) return e;
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
                      unit_bytes, beams, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t al = (uint64_t)reinterpret_cast<uintptr_t>(state) | (uint64_t)unit_bytes;
  const cudaError_t e = al % 16 == 0  ? launch<uint4>(a, st)
                        : al % 8 == 0 ? launch<uint2>(a, st)
                        : al % 4 == 0 ? launch<uint32_t>(a, st)
                        : al % 2 == 0 ? launch<uint16_t>(a, st)
                                      : launch<uint8_t>(a, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
