// logits_adjust.cu — penalties for repeated tokens, biases and grammar masks on logits, in place (orpo_logits_adjust).
//
//   x' = x > 0 ? x / repetition : x * repetition          where the row's history holds the token
//   x' - (presence + frequency n)                         where its generated part holds it n > 0 times
//   + the token's biases;  -inf where a mask or an n-gram bans it
//
// Only the logits that one of these concerns are read or written, so the work is the history's length and the masked
// logits, not the vocabulary.  Two kinds of CTAs share a launch; they never write the same logit, but for the -inf of a token that
// a mask and an n-gram both ban, so they need no order:
//   history CTAs   adjust the tokens that the history and the bias list hold, unless a mask bans them.
//     By bits: without a frequency penalty it is enough to know which tokens there are: one CTA per row, with a bit per token
//     of the vocabulary in shared memory, where masked tokens are set from the start.  Who sets a token's bit adjusts its
//     logit at once; the generated part is taken before the prompt, so that the first to come knows the penalty.
//     By counters: a CTA per range of the vocabulary, with a counter per token, which no history can overflow; each CTA reads
//     the whole history.
//     Neither has anything to probe or to sort, and integer atomics give the same whatever their order.  (With a hash table of
//     a row's tokens 16 rows of 262144 took 15.9 us; with counters 6.2: probes follow one another.)
//   mask CTAs      overwrite the masked logits of a range, 16 bytes per lane where 512 bytes in a row are all masked, else a
//                  lane per token: nothing is read but the mask.
// Bound, for few rows, by three ways to memory (length, tokens, logits) and the launch: 4 rows of 4096 2.9 us captured in a
// graph, 16 rows of 262144 with everything on 6.2.  For many rows (32 x 8 of 128256 bf16, histories of 4096, a grammar's masks:
// 20.4 us; the masks alone 11.4, the history alone 16.2) the logits' lookups are the largest known part: 32 different sectors a
// warp, read and written, for two rows on the busiest SM 2 x 3600 x 2 requests, about 7.6 us at one per clock.  With a frequency penalty
// every CTA of a row reads its whole history: 30.7 us, 22.6 without masks, 34 there with 32-bit counters.
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
  int parts;       // history CTAs per row
  int list_cap;    // listed tokens per range at most
  int list_words;  // 32-bit words of that list
  int bit_words;   // of a map of the vocabulary
  int sets;        // of words per mask CTA
  int clear;       // 16-byte pieces of shared memory to clear
};

constexpr int kThreads = 512;
// What is known of a token: how often the generated part holds it, and flags
constexpr uint32_t kCount = (1u << 28) - 1;
constexpr uint32_t kPrompt = 1u << 28;  // the prompt holds it
constexpr uint32_t kBan = 1u << 29;     // it would end an n-gram for the second time
constexpr uint32_t kBias = 1u << 30;    // the bias list holds it: the list's thread adjusts it
// as 16 bits, for histories of up to kFew tokens
constexpr int kFew = (1 << 13) - 1;
constexpr uint32_t kFewPrompt = 1u << 13, kFewBan = 1u << 14, kFewBias = 1u << 15;

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

// ------------------------------------------------------------------ the history's tokens
constexpr int kUnroll = 6;  // tokens of a thread in flight; with 4 and three CTAs per SM the wide case takes 25 us instead of 21, with 8 as many

// A thread's first kUnroll tokens of history positions [begin, end) (-1: none), asked for before they are needed.
struct First {
  int begin = -1;
  int32_t v[kUnroll];
  __device__ __forceinline__ void load(const int32_t* h, int from, int end) {
    begin = from;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = from + u * kThreads + (int)threadIdx.x;
      v[u] = t < end ? h[t] : -1;
    }
  }
};

// Calls each(t, token) with kUnroll tokens of history positions t[0], ... in [begin, end) (token -1: none), whole warps at
// a time.
template <class Each>
__device__ __forceinline__ void each_tokens(const int32_t* h, int begin, int end, const First& first, Each each) {
  const int lane = threadIdx.x & 31;
  for (int t0 = begin + (int)threadIdx.x - lane; t0 < end; t0 += kUnroll * kThreads) {
    int t[kUnroll];
    int32_t v[kUnroll];
    const bool ready = begin == first.begin && t0 < begin + kThreads;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      t[u] = t0 + u * kThreads + lane;
      v[u] = ready ? first.v[u] : t[u] < end ? h[t[u]] : -1;
    }
    each(t, v);
  }
}

// Whether the tokens before position t are the tail's; all lanes of a warp together, whose v are neighbours.
__device__ __forceinline__ bool ends_again(const int32_t* h, int t, int32_t v, int len, const int32_t* tail, int n_tail) {
  if (n_tail <= 0) return n_tail == 0 && t < len;
  int32_t before = __shfl_up_sync(~0u, v, 1);
  if (t < n_tail || t >= len) return false;
  if ((threadIdx.x & 31) == 0) before = h[t - 1];
  bool same = before == tail[n_tail - 1];
  for (int i = 2; i <= n_tail && same; ++i) same = h[t - i] == tail[n_tail - i];
  return same;
}

template <class T>
struct Row {
  T* x;                   // the row's logits
  const uint32_t* words;  // its mask, or nullptr
  int64_t at, all;        // where it starts, and all logits (bounds-checked build)
};

// N tokens (-1: none) that no mask bans, with what is known of them and their bias, all their logits on the way at once.
template <class T, int N>
__device__ __forceinline__ void adjust(const AdjustArgs& a, const Row<T>& row, const int32_t (&token)[N], const uint32_t (&w)[N],
                                       float bias) {
  float y[N];
  bool on[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    on[i] = token[i] >= 0 && in_bounds(a.status, row.at + token[i], row.all);
    y[i] = on[i] ? Logit<T>::load(row.x + token[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!on[i]) continue;
    if (w[i] & (kCount | kPrompt)) y[i] = y[i] > 0.f ? y[i] / a.repetition : y[i] * a.repetition;
    if (w[i] & kCount) y[i] -= fmaf(a.frequency, (float)(w[i] & kCount), a.presence);
    y[i] = w[i] & kBan ? -INFINITY : y[i] + bias;
    row.x[token[i]] = Logit<T>::make(y[i]);
  }
}

// The bias list's tokens in [v0, v0 + size): the first of a token's entries adds them all up, in order.  Where any token comes
// twice every entry searches the list: 4 rows of 128256 with 4096 entries take 6.7 us, with one of them repeated 790.
template <class T, class Known>
__device__ __forceinline__ void adjust_biased(const AdjustArgs& a, const Row<T>& row, const int32_t* token, const float* value, bool twice,
                                              int64_t v0, int size, Known known) {
  for (int j = kThreads - 1 - (int)threadIdx.x; j < a.n_bias; j += kThreads) {  // from the last thread on: the first have the history's
    const int32_t v = token[j];
    if (v < 0 || (uint32_t)(v - (int32_t)v0) >= (uint32_t)size) continue;
    if (row.words && !(row.words[v >> 5] >> (v & 31) & 1u)) continue;  // left to the masks
    float sum = value[j];
    if (twice) {
      bool first = true;
      for (int i = 0; i < j && first; ++i) first = token[i] != v;
      if (!first) continue;
      for (int i = j + 1; i < a.n_bias; ++i)
        if (token[i] == v) sum += value[i];
    }
    const int32_t tokens[1] = {v};
    const uint32_t w[1] = {known(v)};
    adjust<T, 1>(a, row, tokens, w, sum);
  }
}

// ------------------------------------------------------------------ masks
constexpr int kSetTokens = kThreads * 32;  // a word per thread
constexpr int kMaskSets = 2;               // of those per CTA, or one where so many CTAs are resident at once

template <class T>
__device__ __forceinline__ void mask_range(const AdjustArgs& a, const Row<T>& row, int64_t v0, int sets) {
  constexpr int kGroup = 512 / (32 * (int)sizeof(T));  // words whose logits are 512 bytes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n_words = (a.V + 31) / 32;
  const bool aligned = (reinterpret_cast<uintptr_t>(row.x) & 15u) == 0;
  uint32_t word[kMaskSets];
  int64_t first[kMaskSets];
#pragma unroll
  for (int s = 0; s < kMaskSets; ++s) {
    first[s] = v0 / 32 + (s * (kThreads / 32) + warp) * 32;
    const int64_t i = first[s] + lane;
    word[s] = s < sets && i < n_words ? row.words[i] : ~0u;
    if (i == n_words - 1 && a.V % 32) word[s] |= ~0u << (a.V % 32);
  }
#pragma unroll
  for (int s = 0; s < kMaskSets; ++s) {
    const uint32_t none = __ballot_sync(~0u, word[s] == 0), all = __ballot_sync(~0u, word[s] == ~0u);
    if (all == ~0u) continue;
    for (int g = 0; g < 32; g += kGroup) {
      constexpr uint32_t kOnes = (1u << kGroup) - 1u;
      if ((all >> g & kOnes) == kOnes) continue;
      T* const x = row.x + (first[s] + g) * 32;
      if (aligned && (none >> g & kOnes) == kOnes) {
        if (in_bounds(a.status, row.at + (first[s] + g + kGroup) * 32 - 1, row.all))
          reinterpret_cast<uint4*>(x)[lane] = make_uint4(Logit<T>::kNinf, Logit<T>::kNinf, Logit<T>::kNinf, Logit<T>::kNinf);
        continue;
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const uint32_t w = __shfl_sync(~0u, word[s], g + i);
        if (!(w & 1u << lane) && in_bounds(a.status, row.at + (first[s] + g + i) * 32 + lane, row.all)) x[i * 32 + lane] = Logit<T>::make(-INFINITY);
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
// How history CTAs know the tokens: bits, or 16- or 32-bit counters of a range.
enum { kBits = 0, kCount16 = 1, kCount32 = 2 };
constexpr int kTableBytes = 64 << 10;
__host__ __device__ constexpr int range_of(int form) { return kTableBytes / (form == kCount16 ? 2 : 4); }
constexpr int kMostBits = 200 << 10;  // bytes of all bitmaps

// One bit per token of the vocabulary, `stride` words a map: met; banned (n-grams); of the bias list; met in the generated part
// (kept for the bias list).
struct Bits {
  uint32_t *met, *ban, *bias, *gen;
  __device__ static bool get(const uint32_t* map, int32_t v) { return map[v >> 5] >> (v & 31) & 1u; }
  __device__ static bool set(uint32_t* map, int32_t v) {  // whether it was set before
    const uint32_t bit = 1u << (v & 31);
    return (atomicOr(map + (v >> 5), bit) & bit) != 0;
  }
};

template <class T>
__device__ __forceinline__ void by_bits(const AdjustArgs& a, const Row<T>& row, uint32_t* smem, const First& first, const int32_t* h, int len, int prompt,
                                        const int32_t* tail, int n_tail, const int32_t* bias_token, const float* bias_value, int* twice,
                                        bool penalties) {
  const int stride = a.bit_words;
  const bool biased = a.n_bias > 0;
  const Bits bits{smem, smem + stride, smem + (a.ngram > 0 ? 2 : 1) * stride, smem + (a.ngram > 0 ? 3 : 2) * stride};
  const int32_t V = (int32_t)a.V;
  for (int j = kThreads - 1 - (int)threadIdx.x; j < a.n_bias; j += kThreads) {  // from the last thread on: the first have the history's
    const int32_t v = bias_token[j];
    if (v >= 0 && v < V && Bits::set(bits.bias, v)) *twice = 1;
  }
  if (n_tail >= 0)
    each_tokens(h, 0, len, first, [&](const int (&t)[kUnroll], const int32_t (&v)[kUnroll]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (ends_again(h, t[u], v[u], len, tail, n_tail) && v[u] >= 0 && v[u] < V && !Bits::set(bits.ban, v[u]) &&
            in_bounds(a.status, row.at + v[u], row.all))
          row.x[v[u]] = Logit<T>::make(-INFINITY);  // as a mask would
    });
  if (penalties) {
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {  // what was generated, then the prompt
      if (part == 1 && prompt == 0) break;
      if (part == 1 || biased || n_tail >= 0) __syncthreads();
      each_tokens(h, part == 0 ? prompt : 0, part == 0 ? len : prompt, part == 0 ? first : First(), [&](const int (&)[kUnroll], const int32_t (&v)[kUnroll]) {
        int32_t token[kUnroll];
        uint32_t w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          w[u] = part == 0 ? 1u : kPrompt;
          token[u] = v[u] >= 0 && v[u] < V && !Bits::set(bits.met, v[u]) ? v[u] : -1;
          if (token[u] >= 0 && n_tail >= 0 && Bits::get(bits.ban, token[u])) token[u] = -1;
          if (token[u] >= 0 && biased && Bits::get(bits.bias, token[u])) {
            if (part == 0) Bits::set(bits.gen, token[u]);
            token[u] = -1;
          }
        }
        adjust<T, kUnroll>(a, row, token, w, 0.f);
      });
    }
  }
  if (!biased) return;
  __syncthreads();
  adjust_biased<T>(a, row, bias_token, bias_value, *twice, 0, V, [&](int32_t v) {
    return (penalties && Bits::get(bits.gen, v) ? 1u : 0u) | (penalties && Bits::get(bits.met, v) ? kPrompt : 0u) |
           (n_tail >= 0 && Bits::get(bits.ban, v) ? kBan : 0u);
  });
}

// The counters of a range.
template <int kForm>
struct Counters {
  uint32_t* table;
  // Adds one to, or sets flags of, the token at `at`; what was known before, in the form's own bits.
  __device__ uint32_t add(uint32_t at) const {
    if (kForm == kCount32) return atomicAdd(table + at, 1u);
    return atomicAdd(table + at / 2, 1u << (at & 1u) * 16) >> (at & 1u) * 16 & 0xffffu;
  }
  __device__ uint32_t flag(uint32_t at, uint32_t flag32, uint32_t flag16) const {
    if (kForm == kCount32) return atomicOr(table + at, flag32);
    return atomicOr(table + at / 2, flag16 << (at & 1u) * 16) >> (at & 1u) * 16 & 0xffffu;
  }
  __device__ uint32_t known(uint32_t at) const {
    if (kForm == kCount32) return table[at];
    const uint32_t w = table[at / 2] >> (at & 1u) * 16 & 0xffffu;
    return (w & (uint32_t)kFew) | (w & kFewPrompt ? kPrompt : 0u) | (w & kFewBan ? kBan : 0u) | (w & kFewBias ? kBias : 0u);
  }
};

template <class T, int kForm>
__device__ __forceinline__ void by_counts(const AdjustArgs& a, const Row<T>& row, uint32_t* smem, const First& first, int64_t v0, const int32_t* h, int len,
                                          int prompt, const int32_t* tail, int n_tail, const int32_t* bias_token, const float* bias_value,
                                          int* listed, int* twice, bool penalties) {
  constexpr int kRange = range_of(kForm);
  const Counters<kForm> counters{smem};
  uint16_t* const list = reinterpret_cast<uint16_t*>(smem + kTableBytes / 4);  // tokens met, each once
  const uint32_t size = (uint32_t)min((int64_t)kRange, a.V - v0);
  const uint32_t* const allowed = smem + kTableBytes / 4 + a.list_words;  // the mask's part
  each_tokens(h, 0, len, first, [&](const int (&t)[kUnroll], const int32_t (&v)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool banned = ends_again(h, t[u], v[u], len, tail, n_tail);
      const uint32_t at = (uint32_t)(v[u] - (int32_t)v0);
      if (v[u] < 0 || at >= size || !(penalties || banned) || !in_bounds(a.status, at, kRange)) continue;
      if (row.words && !(allowed[at / 32] >> (at % 32) & 1u)) continue;  // left to the masks
      const uint32_t old = t[u] >= prompt ? counters.add(at) : counters.flag(at, kPrompt, kFewPrompt);
      if (old == 0) {
        const int j = atomicAdd(listed, 1);
        if (in_bounds(a.status, j, a.list_cap)) list[j] = (uint16_t)at;
      }
      if (banned) counters.flag(at, kBan, kFewBan);
    }
  });
  for (int j = kThreads - 1 - (int)threadIdx.x; j < a.n_bias; j += kThreads) {  // from the last thread on: the first have the history's
    const int32_t v = bias_token[j];
    const uint32_t at = (uint32_t)(v - (int32_t)v0);
    if (v < 0 || at >= size || !in_bounds(a.status, at, kRange)) continue;
    if (counters.flag(at, kBias, kFewBias) & (kForm == kCount32 ? kBias : kFewBias)) *twice = 1;
  }
  __syncthreads();
  adjust_biased<T>(a, row, bias_token, bias_value, *twice, v0, (int)size, [&](int32_t v) { return counters.known(v - (int32_t)v0); });
  const int n = *listed;
  for (int j0 = threadIdx.x; j0 < n; j0 += kUnroll * kThreads) {
    int32_t token[kUnroll];
    uint32_t w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * kThreads, at = j < n ? list[j] : -1;
      w[u] = at >= 0 ? counters.known(at) : 0;
      token[u] = at >= 0 && !(w[u] & kBias) ? (int32_t)v0 + at : -1;
    }
    adjust<T, kUnroll>(a, row, token, w, 0.f);
  }
}

template <class T, int kForm>
__global__ void __launch_bounds__(kThreads, 2) adjust_kernel(AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int32_t tail[ORPO_MAX_NGRAM];
  __shared__ int listed, twice;
  const int tid = threadIdx.x;
  grid_trigger();
  const uint32_t part = blockIdx.x / (uint32_t)a.rows;  // history CTAs, which take longer, come first
  const int64_t r = blockIdx.x - part * (uint32_t)a.rows;
  const bool history = part < (uint32_t)a.parts;
  if (history)
    for (int i = tid; i < a.clear; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) listed = 0, twice = 0;
  __syncthreads();
  grid_wait();

  const int64_t b = (uint32_t)r / (uint32_t)a.beams;
  const int len = a.history ? a.length[b] : 0;
  const int mask = a.masks ? a.mask_row[r] : -1;
  const int prompt = a.prompt && a.history ? a.prompt[b] : 0;
  const int wrong = (len < 0 || len > a.capacity ? ORPO_STATUS_PARENT : 0) |
                    (mask < -1 || (a.masks && mask >= a.n_masks) ? ORPO_STATUS_MASK : 0);
  if (wrong) {
    if (tid == 0 && part == 0) atomicOr(a.status, wrong);
    return;
  }
  const Row<T> row{static_cast<T*>(a.logits) + r * a.ld, mask >= 0 ? a.masks + mask * a.ld_masks : nullptr, r * a.ld, a.rows * a.ld};
  if (!history) {
    if (mask >= 0) mask_range(a, row, (int64_t)(part - a.parts) * a.sets * kSetTokens, a.sets);
    return;
  }
  const int32_t* const h = a.history + r * a.ld_history;
  const int32_t* const bias_token = a.bias_token + b * a.ld_bias;
  const float* const bias_value = a.bias_value + b * a.ld_bias;
  // the n-gram to look for: the last n - 1 tokens, if all of them are tokens
  int n_tail = a.ngram > 0 && len >= a.ngram ? a.ngram - 1 : -1;
  bool bad_tail = false;
  if (tid < n_tail) {
    const int t = h[len - n_tail + tid];
    tail[tid] = t;
    bad_tail = t < 0 || t >= a.V;
  }
  // its mask: for bits, masked tokens count as met from the start, so that nobody adjusts them
  if (row.words) {
    constexpr int kRange = kForm == kBits ? 0 : range_of(kForm);
    const int64_t w0 = kForm == kBits ? 0 : (int64_t)part * (kRange / 32), words = (a.V + 31) / 32;
    uint32_t* const to = kForm == kBits ? smem : smem + kTableBytes / 4 + a.list_words;
    const int n = (int)(kForm == kBits ? words : min(words - w0, (int64_t)kRange / 32));
    for (int i = tid; i < n; i += kThreads) to[i] = kForm == kBits ? ~row.words[i] : row.words[w0 + i];
  }
  // the tokens that are looked at first: for bits the generated part's, where it has a penalty of its own
  const int generated = kForm == kBits && a.presence != 0.f ? min(max(prompt, 0), len) : 0;
  First first;
  first.load(h, n_tail >= 0 ? 0 : generated, len);
  if (__syncthreads_or(bad_tail)) n_tail = -1;
  const bool penalties = a.repetition != 1.f || a.presence != 0.f || a.frequency != 0.f;
  if constexpr (kForm == kBits)
    by_bits<T>(a, row, smem, first, h, len, generated, tail, n_tail, bias_token, bias_value, &twice, penalties);
  else
    by_counts<T, kForm>(a, row, smem, first, (int64_t)part * range_of(kForm), h, len, prompt, tail, n_tail, bias_token, bias_value, &listed, &twice,
                        penalties);
}

template <class T, int kForm>
cudaError_t launch_form(const AdjustArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  static std::atomic<int> done[64];
  cudaError_t e = opt_in_smem(adjust_kernel<T, kForm>, kForm == kBits ? kMostBits : kTableBytes + range_of(kForm) * 2 + range_of(kForm) / 8, done);
  if (e != cudaSuccess) return e;
  prof_begin(K_ADJUST, st);
  e = launch_dependent(adjust_kernel<T, kForm>, grid, kThreads, smem, st, a);
  prof_end(K_ADJUST, st);
  return e;
}

template <class T>
cudaError_t launch(AdjustArgs a, int sms, cudaStream_t st) {
  const bool history = a.history != nullptr || a.n_bias > 0;
  a.bit_words = (int)(cdiv(a.V, 128) * 4);
  const int64_t bits = (int64_t)a.bit_words * 4 * (1 + (a.ngram > 0) + 2 * (a.n_bias > 0));
  // Bits take one CTA per row, counters several, which is better while all of them are resident at once: 35 rows of 50257
  // 5.0 us by counters and 7.2 by bits, 16 of 262144 6.1 and 7.9, but 256 of 128256 31.0 and 20.5.  16-bit counters have twice
  // the range of 32-bit ones, so half the CTAs read the history: with 32 bits the three take 4.5, 7.0 and 44.0 us.
  const int counted = a.capacity <= kFew ? kCount16 : kCount32;
  const bool spread = a.rows * cdiv(a.V, range_of(counted)) <= (int64_t)sms * 2;
  const int form = a.frequency == 0.f && bits <= kMostBits && !spread ? kBits : counted;
  a.parts = !history ? 0 : form == kBits ? 1 : (int)cdiv(a.V, range_of(form));
  a.list_cap = std::min(range_of(form), a.history ? a.capacity : 0);
  a.list_words = (int)cdiv(a.list_cap, 8) * 4;
  const int64_t smem = !history ? 0 : form == kBits ? bits : kTableBytes + a.list_words * 4 + (a.masks ? range_of(form) / 8 : 0);
  a.clear = (int)((form == kBits ? bits : kTableBytes) / 16);
  a.sets = a.rows * cdiv(a.V, kSetTokens) <= (int64_t)sms * 2 ? 1 : kMaskSets;
  const dim3 grid((unsigned)(a.rows * (a.parts + (a.masks ? cdiv(a.V, a.sets * kSetTokens) : 0))));
  return form == kBits      ? launch_form<T, kBits>(a, grid, (size_t)smem, st)
         : form == kCount16 ? launch_form<T, kCount16>(a, grid, (size_t)smem, st)
                            : launch_form<T, kCount32>(a, grid, (size_t)smem, st);
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
      V > kMaxRows || batch * beams * V >= (1ll << 44) || ld_logits < V || capacity < 0 || capacity >= (1ll << 28) || n_bias < 0 || n_bias > ORPO_MAX_BIAS)
    return ORPO_ERR_SHAPE;
  if (!std::isfinite(repetition) || repetition <= 0.f || !std::isfinite(presence) || !std::isfinite(frequency) ||
      no_repeat < 0 || no_repeat > ORPO_MAX_NGRAM)
    return ORPO_ERR_ARG;
  const bool reads = capacity > 0 && (repetition != 1.f || presence != 0.f || frequency != 0.f || no_repeat > 0);
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
                     masks, ld_masks, n_masks, mask_row, status, 0, 0, 0, 0, 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_bf16 ? launch<uint16_t>(a, sms, st) : launch<float>(a, sms, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
