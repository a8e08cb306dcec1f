// beam_history.cu — the beams' token histories follow their parents and get the new tokens (orpo_beam_history).
//
//   history[b, k, t] <- history[b, parent[b, k], t] for t < length[b];  history[b, k, length[b]] <- token[b, k]
//
// One thread owns the same piece of all beams of an entry: it reads every moved beam's source before it writes any, and
// no other thread touches those.  Pieces are 16 bytes for up to 8 beams (their sources are 32 registers), 4 above.  Bound by
// the launch and two ways to memory: 4 beams of 100 tokens 1.5 us captured in a graph, 32 x 8 of 8191 (9.5 MB) 3.3, 28 x 9 of
// them 5.4, 16 x 16 4.4, 4 x 64 5.9.
#include <algorithm>

#include "../../include/orpo_decode.h"
#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

struct HistoryArgs {
  int32_t* history;
  int64_t ld;
  int capacity;
  const int32_t* parent;
  int64_t ld_parent;
  const int32_t* token;
  int64_t ld_token;
  const int32_t* length;
  int64_t batch;
  int beams;
  int32_t* status;
};

constexpr int kThreads = 128;

// Piece: int4 or int.  KB: beams at most.
template <class Piece, int KB>
__global__ void __launch_bounds__(kThreads) history_kernel(HistoryArgs a) {
  constexpr int kInts = (int)sizeof(Piece) / 4;
  __shared__ int par[KB];
  grid_trigger();
  grid_wait();
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, len = a.length[b];
  bool bad = len < 0 || len >= a.capacity;
  if (tid < KB) {
    const int p = tid < a.beams ? a.parent[b * a.ld_parent + tid] : tid;
    bad |= tid < a.beams && (p < 0 || p >= a.beams);
    par[tid] = p;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.y == 0) atomicOr(a.status, ORPO_STATUS_PARENT);
    return;
  }
  int32_t* const base = a.history + b * a.beams * a.ld;
  const int64_t used = a.batch * a.beams * a.ld, b0 = b * a.beams * a.ld;
  auto move = [&](auto piece, int64_t t) {
    using P = decltype(piece);
    constexpr int n = (int)sizeof(P) / 4;
    P v[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k && in_bounds(a.status, b0 + par[k] * a.ld + t + n - 1, used))
        v[k] = *reinterpret_cast<const P*>(base + par[k] * a.ld + t);
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (par[k] != k && in_bounds(a.status, b0 + k * a.ld + t + n - 1, used)) *reinterpret_cast<P*>(base + k * a.ld + t) = v[k];
  };
  const int whole = len / kInts;
  for (int64_t i = (int64_t)blockIdx.y * kThreads + tid; i < whole; i += (int64_t)gridDim.y * kThreads) move(Piece(), i * kInts);
  if (blockIdx.y == 0) {
    if (kInts > 1 && tid < len - whole * kInts) move(int(), whole * kInts + tid);
    if (tid < a.beams && in_bounds(a.status, b0 + tid * a.ld + len, used)) base[tid * a.ld + len] = a.token[b * a.ld_token + tid];
  }
}

template <class Piece, int KB>
cudaError_t launch(const HistoryArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.batch, (unsigned)std::min<int64_t>(65535, cdiv(a.capacity, kThreads * ((int)sizeof(Piece) / 4))));
  prof_begin(K_HISTORY, st);
  const cudaError_t e = launch_dependent(history_kernel<Piece, KB>, grid, kThreads, 0, st, a);
  prof_end(K_HISTORY, st);
  return e;
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" int orpo_beam_history(int32_t* history, int64_t ld_history, int64_t capacity, const int32_t* parent, int64_t ld_parent,
                                 const int32_t* token, int64_t ld_token, const int32_t* length, int64_t batch, int beams,
                                 int32_t* status, void* stream) {
  if (batch < 0 || batch > (1ll << 20) || beams < 1 || beams > ORPO_MAX_BEAMS || batch * beams > (1ll << 20) || capacity < 1 ||
      capacity >= (1ll << 28) || ld_history < capacity || ld_parent < beams || ld_token < beams)
    return ORPO_ERR_SHAPE;
  if (batch == 0) return ORPO_OK;
  if (!history || !parent || !token || !length || !status) return ORPO_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(history) | reinterpret_cast<uintptr_t>(parent) | reinterpret_cast<uintptr_t>(token) |
       reinterpret_cast<uintptr_t>(length) | reinterpret_cast<uintptr_t>(status)) & 3)
    return ORPO_ERR_ALIGN;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  const HistoryArgs a{history, ld_history, (int)capacity, parent, ld_parent, token, ld_token, length, batch, beams, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = reinterpret_cast<uintptr_t>(history) % 16 == 0 && ld_history % 4 == 0;
  const cudaError_t e = beams <= 4    ? (wide ? launch<int4, 4>(a, st) : launch<int, 4>(a, st))
                        : beams <= 8  ? (wide ? launch<int4, 8>(a, st) : launch<int, 8>(a, st))
                        : beams <= 16 ? launch<int, 16>(a, st)
                        : beams <= 32 ? launch<int, 32>(a, st)
                                      : launch<int, 64>(a, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
