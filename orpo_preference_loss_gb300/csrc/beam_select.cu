// beam_select.cu — the n best continuations over beams x vocabulary (orpo_beam_select).
//
//   lse_r = log sum_v exp x_rv,  value(k, v) = score_k + (x_kv - lse_k)
//
// Within a beam the value grows with the logit, so a beam's proposals are its n largest logits and
// the softmax statistics are needed only for those.  Order inside a beam is a 64-bit key (the
// logit's bits mapped to an order-preserving integer, then the complement of the token), which is
// total, so ties and scheduling cannot change the result.
//
// Row kernel: one CTA per live beam finds the row's max and sum of exp and its n largest keys, by n
// rounds of "largest key below the last one".  Merge kernel: one warp per batch entry merges the
// beams' sorted proposals by value.
#include <math.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;

// order-preserving map of a non-NaN float to uint32 (-inf is the least value any float maps to)
__device__ __forceinline__ uint32_t ord_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ord_to_float(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int v) {
  return ((uint64_t)ord_of(x) << 32) | (uint32_t)~(uint32_t)v;
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* row, int v) {
  if constexpr (kBf16)
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(row) + v) << 16);
  else
    return __ldg(static_cast<const float*>(row) + v);
}

struct SelectArgs {
  const void* logits;
  int64_t ld;
  const float* score;
  const uint8_t* finished;
  int eos, beams, V, n;
  float* out_score;
  int32_t* out_parent;
  int32_t* out_token;
  uint8_t* out_finished;
  uint64_t* keys;  // [rows, n]
  float* lse;      // [rows]
  int32_t* status;
};

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t t = __shfl_xor_sync(0xffffffffu, k, o);
    k = t > k ? t : k;
  }
  return k;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) select_rows_kernel(SelectArgs a) {
  const int64_t r = blockIdx.x;
  if (a.finished != nullptr && a.finished[r]) return;
  const void* row = static_cast<const uint8_t*>(a.logits) + r * a.ld * (kBf16 ? 2 : 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ float sm[kThreads / 32], ss[kThreads / 32];
  __shared__ uint64_t sk[kThreads / 32];
  float m = -INFINITY, s = 0.f;
  bool bad = false;
  for (int v = tid; v < a.V; v += kThreads) {
    const float x = load_logit<kBf16>(row, v);
    if (x != x || x == INFINITY) bad = true;
    if (x != x || x == -INFINITY) continue;
    if (x > m) {
      s = s * ex2_approx((m - x) * kLog2e) + 1.f;
      m = x;
    } else {
      s += x == m ? 1.f : ex2_approx((x - m) * kLog2e);
    }
  }
  if (bad) atomicOr(a.status, ORPO_STATUS_NONFINITE);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float mm = fmaxf(m, m2);
    s = mm == -INFINITY ? 0.f : s * (m == mm ? 1.f : ex2_approx((m - mm) * kLog2e)) +
                                    s2 * (m2 == mm ? 1.f : ex2_approx((m2 - mm) * kLog2e));
    m = mm;
  }
  if (lane == 0) sm[warp] = m, ss[warp] = s;
  __syncthreads();
  if (tid == 0) {
    float mm = -INFINITY, t = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < kThreads / 32; ++w)
      if (sm[w] > -INFINITY) t += ss[w] * (sm[w] == mm ? 1.f : ex2_approx((sm[w] - mm) * kLog2e));
    a.lse[r] = mm == -INFINITY || mm == INFINITY ? mm : mm + logf(t);
  }
  uint64_t last = ~0ull;
  for (int i = 0; i < a.n; ++i) {
    uint64_t best = 0;
    for (int v = tid; v < a.V; v += kThreads) {
      float x = load_logit<kBf16>(row, v);
      if (x != x) x = -INFINITY;
      const uint64_t k = key_of(x, v);
      if (k < last && k > best) best = k;
    }
    best = warp_max(best);
    __syncthreads();
    if (lane == 0) sk[warp] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) best = sk[w] > best ? sk[w] : best;
    if (tid == 0) a.keys[r * a.n + i] = best;
    last = best;
  }
}

__global__ void __launch_bounds__(32) select_merge_kernel(SelectArgs a) {
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x;
  __shared__ float value[ORPO_MAX_BEAMS][ORPO_MAX_SELECT];
  __shared__ int token[ORPO_MAX_BEAMS][ORPO_MAX_SELECT];
  __shared__ uint8_t over[ORPO_MAX_BEAMS];
  for (int i = lane; i < a.beams * a.n; i += 32) {
    const int k = i / a.n, j = i - k * a.n;
    const int64_t r = b * a.beams + k;
    const float s = a.score[r];
    float x = -INFINITY;
    int t = a.eos;
    if (s != s) atomicOr(a.status, ORPO_STATUS_NONFINITE);
    if (a.finished != nullptr && a.finished[r]) {
      if (j == 0) x = s, over[k] = 1;
    } else {
      if (j == 0) over[k] = 0;
      const uint64_t key = a.keys[r * a.n + j];
      const float l = ord_to_float((uint32_t)(key >> 32)), lse = a.lse[r];
      t = (int)~(uint32_t)key;
      if (l > -INFINITY && fabsf(lse) < INFINITY) x = s + (l - lse);
    }
    value[k][j] = x == x ? x : -INFINITY;
    token[k][j] = t;
  }
  __syncwarp();
  int head0 = 0, head1 = 0;  // next proposal of beams lane and lane + 32
  for (int i = 0; i < a.n; ++i) {
    // (value, then the lower beam) as one key; 0 for an exhausted beam
    uint64_t k0 = 0, k1 = 0;
    if (lane < a.beams && head0 < a.n) k0 = key_of(value[lane][head0], lane);
    if (lane + 32 < a.beams && head1 < a.n) k1 = key_of(value[lane + 32][head1], lane + 32);
    const uint64_t best = warp_max(k0 > k1 ? k0 : k1);
    const int k = (int)~(uint32_t)best;
    const int h = __shfl_sync(0xffffffffu, k < 32 ? head0 : head1, k & 31);
    if (lane == 0) {
      const int64_t at = b * a.n + i;
      a.out_score[at] = value[k][h];
      a.out_parent[at] = k;
      a.out_token[at] = token[k][h];
      if (a.out_finished) a.out_finished[at] = over[k] || token[k][h] == a.eos;
    }
    if (k == lane) ++head0;
    if (k == lane + 32) ++head1;
  }
}

bool select_sizes_ok(int64_t batch, int beams, int64_t V, int n) {
  return batch >= 0 && beams >= 1 && beams <= ORPO_MAX_BEAMS && V >= 1 && V <= kMaxRows && n >= 1 &&
         n <= ORPO_MAX_SELECT && n <= V && batch <= (1 << 20) && batch * beams <= (1 << 20);
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" size_t orpo_beam_select_workspace_bytes(int64_t batch, int beams, int64_t V, int n) {
  if (!select_sizes_ok(batch, beams, V, n)) return 0;
  return (size_t)(batch * beams) * ((size_t)n * 8 + 8) + 16;
}

extern "C" int orpo_beam_select(const void* logits, int64_t ld_logits, int logits_bf16, const float* score,
                                const uint8_t* finished, int32_t eos, int64_t batch, int beams, int64_t V, int n,
                                float* out_score, int32_t* out_parent, int32_t* out_token, uint8_t* out_finished,
                                void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  if (!select_sizes_ok(batch, beams, V, n)) return ORPO_ERR_SHAPE;
  if (batch == 0) return ORPO_OK;
  if (ld_logits < V || ld_logits > (1ll << 40)) return ORPO_ERR_SHAPE;
  if (!logits || !score || !out_score || !out_parent || !out_token || !workspace || !status) return ORPO_ERR_NULL;
  if (eos < -1 || eos >= V || (finished && eos < 0)) return ORPO_ERR_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(score) | reinterpret_cast<uintptr_t>(out_score) |
                          reinterpret_cast<uintptr_t>(out_parent) | reinterpret_cast<uintptr_t>(out_token);
  if (!aligned16(workspace) || (words & 3) || (reinterpret_cast<uintptr_t>(logits) & (logits_bf16 ? 1 : 3)))
    return ORPO_ERR_ALIGN;
  if (ws_bytes < orpo_beam_select_workspace_bytes(batch, beams, V, n)) return ORPO_ERR_WORKSPACE;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = batch * beams;
  SelectArgs a{logits, ld_logits, score, finished, eos, beams, (int)V, n, out_score, out_parent, out_token,
               out_finished, static_cast<uint64_t*>(workspace), nullptr, status};
  a.lse = reinterpret_cast<float*>(a.keys + rows * n);
  prof_begin(K_BEAM, st);
  if (logits_bf16)
    select_rows_kernel<true><<<(unsigned)rows, kThreads, 0, st>>>(a);
  else
    select_rows_kernel<false><<<(unsigned)rows, kThreads, 0, st>>>(a);
  prof_end(K_BEAM, st);
  if (cudaGetLastError() != cudaSuccess) return ORPO_ERR_CUDA;
  prof_begin(K_BEAM, st);
  select_merge_kernel<<<(unsigned)batch, 32, 0, st>>>(a);
  prof_end(K_BEAM, st);
  return cudaGetLastError() == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
