// logits_adjust.cu — penalties for repeated tokens, biases and grammar masks on logits, in place (orpo_logits_adjust).
//
//   x' = x > 0 ? x / repetition : x * repetition          where the row's history holds the token
//   x' - (presence + frequency n)                         where its generated part holds it n > 0 times
//   + the token's biases;  -inf where a mask or an n-gram bans it
//
// Only the logits that one of these concerns are read or written, so the work is the history's length and the masked
// logits, not the vocabulary.  A CTA owns one row's logits of a range of `chunk` tokens.  It counts the history's tokens
// that fall into its range in a table in shared memory, one word per token, so there is nothing to hash or to overflow
// and the counts are exact; the first to meet a token lists it.  Then the masked logits are overwritten
// 16 bytes at a time, and each listed token's logit is read, adjusted and written by one thread.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "../../include/orpo_decode.h"
#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

struct AdjustArgs {
  void* logits;
  int64_t ld;
  int64_t rows, V;
  int beams;
  const int32_t* history;
  int64_t ld_history;
  int capacity;
  const int32_t* length;
  const int32_t* prompt;
  float repetition, presence, frequency;
  int ngram;
  const int32_t* bias_token;
  const float* bias_value;
  int64_t ld_bias;
  int n_bias;
  const uint32_t* masks;
  int64_t ld_masks, n_masks;
  const int32_t* mask_row;
  int32_t* status;
  int chunk;       // tokens per CTA, a multiple of 32
  int list_cap;    // listed tokens at most
};

constexpr int kThreads = 256;
// A token's word in the table: how often the generated part holds it, and
constexpr uint32_t kCount = (1u << 28) - 1;
constexpr uint32_t kBan = 1u << 28;     // it would end an n-gram for the second time
constexpr uint32_t kPrompt = 1u << 29;  // the prompt holds it
constexpr uint32_t kBias = 1u << 30;    // the bias list holds it: the list's thread handles it

template <class T>
struct Logit;
template <>
struct Logit<float> {
  static __device__ float load(const float* p) { return *p; }
  static __device__ float make(float x) { return x; }
  static constexpr uint32_t kNinf = 0xff800000u;  // of a 32-bit word
};
template <>
struct Logit<uint16_t> {
  static __device__ float load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  static __device__ uint16_t make(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }  // the one rounding
  static constexpr uint32_t kNinf = 0xff80ff80u;
};

__host__ __device__ inline int table_bytes(int chunk) { return chunk * 4; }
__host__ __device__ inline int words_bytes(int chunk) { return (chunk / 32 + 4) * 4; }  // a word of ones before, up to three behind

template <class T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int32_t tail[ORPO_MAX_NGRAM];
  __shared__ int listed, twice;
  const bool counts = a.history != nullptr || a.n_bias > 0;
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem);
  uint32_t* const table = reinterpret_cast<uint32_t*>(smem + words_bytes(a.chunk));
  uint16_t* const list = reinterpret_cast<uint16_t*>(smem + words_bytes(a.chunk) + table_bytes(a.chunk));
  const int tid = threadIdx.x;
  grid_trigger();
  const int64_t r = blockIdx.x, v0 = (int64_t)blockIdx.y * a.chunk;
  const int size = (int)min((int64_t)a.chunk, a.V - v0);
  if (counts)
    for (int i = tid; i < a.chunk / 4; i += kThreads)
      if (in_bounds(a.status, i, a.chunk / 4)) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) listed = 0, twice = 0;
  grid_wait();

  const int64_t b = r / a.beams;
  const int len = a.history ? a.length[b] : 0;
  const int mask = a.masks ? a.mask_row[r] : -1;
  const int wrong = (len < 0 || len > a.capacity ? ORPO_STATUS_PARENT : 0) |
                    (mask < -1 || (a.masks && mask >= a.n_masks) ? ORPO_STATUS_MASK : 0);
  if (wrong) {
    if (tid == 0 && blockIdx.y == 0) atomicOr(a.status, wrong);
    return;
  }
  const int n_words = (size + 31) / 32;
  for (int i = tid; i < a.chunk / 32 + 4; i += kThreads) {
    uint32_t w = ~0u;
    if (mask >= 0 && i >= 1 && i <= n_words) {
      w = a.masks[mask * a.ld_masks + v0 / 32 + i - 1];
      if (i == n_words && size % 32) w |= ~0u << (size % 32);
    }
    words[i] = w;
  }
  const int32_t* const h = a.history + r * a.ld_history;
  const int n_tail = a.ngram > 0 && len >= a.ngram ? a.ngram - 1 : -1;  // -1: no n-gram to look for
  bool bad_tail = false;
  if (tid < n_tail) {
    const int t = h[len - n_tail + tid];
    tail[tid] = t;
    bad_tail = t < 0 || t >= a.V;
  }
  const bool bans = !__syncthreads_or(bad_tail) && n_tail >= 0;
  const int prompt = a.prompt && a.history ? a.prompt[b] : 0;

  // ---- count
  auto add = [&](int t, int32_t token) {
    const uint32_t at = (uint32_t)(token - (int32_t)v0);
    if (token < 0 || at >= (uint32_t)size || !in_bounds(a.status, at, a.chunk)) return;
    const uint32_t old = t >= prompt ? atomicAdd(&table[at], 1u) : atomicOr(&table[at], kPrompt);
    if (old == 0) {
      const int j = atomicAdd(&listed, 1);
      if (in_bounds(a.status, j, a.list_cap)) list[j] = (uint16_t)at;
    }
    if (bans && t >= n_tail) {
      bool same = true;
      for (int i = 1; i <= n_tail && same; ++i) same = h[t - i] == tail[n_tail - i];
      if (same) atomicOr(&table[at], kBan);
    }
  };
  constexpr int kUnroll = 8;
  int t = tid;
  for (; t + (kUnroll - 1) * kThreads < len; t += kUnroll * kThreads) {
    int32_t v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = h[t + u * kThreads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add(t + u * kThreads, v[u]);
  }
  for (; t < len; t += kThreads) add(t, h[t]);
  const int32_t* const bias_token = a.bias_token + b * a.ld_bias;
  const float* const bias_value = a.bias_value + b * a.ld_bias;
  for (int j = tid; j < a.n_bias; j += kThreads) {
    const int32_t token = bias_token[j];
    const uint32_t at = (uint32_t)(token - (int32_t)v0);
    if (token < 0 || at >= (uint32_t)size || !in_bounds(a.status, at, a.chunk)) continue;
    if (atomicOr(&table[at], kBias) & kBias) twice = 1;
  }
  __syncthreads();

  // ---- adjust: one thread per token; masked tokens are left to the masks
  T* const x = static_cast<T*>(a.logits) + r * a.ld + v0;
  const bool penalties = a.repetition != 1.f || a.presence != 0.f || a.frequency != 0.f;
  auto adjust = [&](uint32_t at, uint32_t w, float bias) {
    if (!(words[1 + at / 32] >> (at % 32) & 1u)) return;
    if (!in_bounds(a.status, r * a.ld + v0 + at, a.rows * a.ld)) return;
    if (w & kBan) {
      x[at] = Logit<T>::make(-INFINITY);
      return;
    }
    float y = Logit<T>::load(x + at);
    if (w & (kCount | kPrompt)) y = y > 0.f ? y / a.repetition : y * a.repetition;
    if (w & kCount) y -= fmaf(a.frequency, (float)(w & kCount), a.presence);
    x[at] = Logit<T>::make(y + bias);
  };
  for (int j = tid; j < a.n_bias; j += kThreads) {
    const int32_t token = bias_token[j];
    const uint32_t at = (uint32_t)(token - (int32_t)v0);
    if (token < 0 || at >= (uint32_t)size || !in_bounds(a.status, at, a.chunk)) continue;
    float sum = bias_value[j];
    if (twice) {  // the first of a token's entries adds them all up, in order
      bool first = true;
      for (int i = 0; i < j && first; ++i) first = bias_token[i] != token;
      if (!first) continue;
      for (int i = j + 1; i < a.n_bias; ++i)
        if (bias_token[i] == token) sum += bias_value[i];
    }
    adjust(at, table[at], sum);
  }
  if (penalties || bans)
    for (int j = tid; j < listed; j += kThreads) {
      const uint32_t at = list[j], w = table[at];
      if (w & kBias || (!penalties && !(w & kBan))) continue;
      adjust(at, w, 0.f);
    }

  // ---- masks: pieces of 16 bytes from the boundary before the range on
  if (mask < 0) return;
  constexpr int E = 16 / (int)sizeof(T);
  const int before = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  for (int p = tid; p * E < size + before; p += kThreads) {
    const int at = p * E - before;  // first token of the piece
    const uint32_t bit = (uint32_t)(at + 32);
    const uint32_t ok = __funnelshift_r(words[bit / 32], words[bit / 32 + 1], bit % 32) & ((1u << E) - 1);
    if (ok == (1u << E) - 1) continue;
    if (ok == 0) {
      if (in_bounds(a.status, r * a.ld + v0 + at, a.rows * a.ld) && in_bounds(a.status, r * a.ld + v0 + at + E - 1, a.rows * a.ld))
        *reinterpret_cast<uint4*>(x + at) = make_uint4(Logit<T>::kNinf, Logit<T>::kNinf, Logit<T>::kNinf, Logit<T>::kNinf);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (!(ok >> i & 1u) && in_bounds(a.status, r * a.ld + v0 + at + i, a.rows * a.ld)) x[at + i] = Logit<T>::make(-INFINITY);
    }
  }
}

constexpr int kMaxChunk = 32768;  // list entries are 16 bits, and the table has to fit beside it

template <class T>
cudaError_t launch(AdjustArgs a, cudaStream_t st) {
  a.chunk = a.V > (int64_t)65535 * 8192 ? kMaxChunk : 8192;
  a.chunk = (int)std::min<int64_t>(a.chunk, cdiv(a.V, 128) * 128);
  const bool counts = a.history != nullptr || a.n_bias > 0;
  a.list_cap = (int)std::min<int64_t>(a.chunk, a.history ? a.capacity : 0);
  const int smem = words_bytes(a.chunk) + (counts ? table_bytes(a.chunk) + cdiv(a.list_cap * 2, 16) * 16 : 0);
  static std::atomic<int> done[64];
  constexpr int kMost = kMaxChunk * 6 + kMaxChunk / 8 + 16;
  static_assert(kMost <= 227 << 10, "a CTA's shared memory");
  cudaError_t e = opt_in_smem(adjust_kernel<T>, kMost, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.rows, (unsigned)cdiv(a.V, a.chunk));
  prof_begin(K_ADJUST, st);
  e = launch_dependent(adjust_kernel<T>, grid, kThreads, (size_t)smem, st, a);
  prof_end(K_ADJUST, st);
  return e;
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" int orpo_logits_adjust(void* logits, int64_t ld_logits, int logits_bf16, int64_t batch, int beams, int64_t V,
                                  const int32_t* history, int64_t ld_history, int64_t capacity, const int32_t* length,
                                  const int32_t* prompt, float repetition, float presence, float frequency, int no_repeat,
                                  const int32_t* bias_token, const float* bias_value, int64_t ld_bias, int64_t n_bias,
                                  const uint32_t* masks, int64_t ld_masks, int64_t n_masks, const int32_t* mask_row,
                                  int32_t* status, void* stream) {
  if (batch < 0 || batch > (1ll << 20) || beams < 1 || beams > (1 << 20) || batch * beams > (1ll << 20) || V < 1 ||
      V > kMaxRows || ld_logits < V || capacity < 0 || capacity >= (1ll << 28) || n_bias < 0 || n_bias > ORPO_MAX_BIAS)
    return ORPO_ERR_SHAPE;
  if (!std::isfinite(repetition) || repetition <= 0.f || !std::isfinite(presence) || !std::isfinite(frequency) ||
      no_repeat < 0 || no_repeat > ORPO_MAX_NGRAM)
    return ORPO_ERR_ARG;
  const bool reads = repetition != 1.f || presence != 0.f || frequency != 0.f || no_repeat > 0;
  if (reads && history && ld_history < capacity) return ORPO_ERR_SHAPE;
  if (n_bias > 0 && ld_bias != 0 && ld_bias < n_bias) return ORPO_ERR_SHAPE;
  if (masks && (n_masks < 1 || n_masks >= (1ll << 31) || ld_masks < cdiv(V, 32))) return ORPO_ERR_SHAPE;
  if (batch == 0) return ORPO_OK;
  if (!logits || !status || (reads && (!history || !length)) || (n_bias > 0 && (!bias_token || !bias_value)) ||
      (masks == nullptr) != (mask_row == nullptr))
    return ORPO_ERR_NULL;
  uintptr_t at = reinterpret_cast<uintptr_t>(status) | reinterpret_cast<uintptr_t>(masks) | reinterpret_cast<uintptr_t>(mask_row);
  if (reads) at |= reinterpret_cast<uintptr_t>(history) | reinterpret_cast<uintptr_t>(length) | reinterpret_cast<uintptr_t>(prompt);
  if (n_bias > 0) at |= reinterpret_cast<uintptr_t>(bias_token) | reinterpret_cast<uintptr_t>(bias_value);
  if ((at & 3) || (reinterpret_cast<uintptr_t>(logits) & (logits_bf16 ? 1 : 3))) return ORPO_ERR_ALIGN;
  if (!reads && n_bias == 0 && !masks) return ORPO_OK;
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  const AdjustArgs a{logits, ld_logits, batch * beams, V, beams, reads ? history : nullptr, ld_history, (int)capacity,
                     length, prompt, repetition, presence, frequency, no_repeat, bias_token, bias_value, ld_bias, (int)n_bias,
                     masks, ld_masks, n_masks, mask_row, status, 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_bf16 ? launch<uint16_t>(a, st) : launch<float>(a, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
