// beam_select.cu — the n best continuations over beams x vocabulary (orpo_beam_select).
//
//   lse_r = log sum_v exp x_rv,  value(k, v) = score_k + (x_kv - lse_k)
//
// lse is kept as the row's maximum m and log s, s = sum exp(x - m), and the value is score + ((x - m) - log s): rounded to one
// number, lse would lose half a unit in the last place of m (5e-4 at 1e4, all of log s at a mask's -1e9).
// Within a beam the value grows with the logit, so a beam's proposals are its n largest logits and
// the softmax statistics are needed only for those.  Order inside a beam is a 64-bit key (the
// logit's bits mapped to an order-preserving integer, then the complement of the token), which is
// total, so ties and scheduling cannot change the result.
//
// Row kernel: a CTA reads a part of one beam's row once, 8192 fp32 or 16384 bf16 logits at a time in
// registers (32 words per thread, all loads in flight together), and leaves the part's max, sum of exp
// and n largest keys.  A logit costs 12 to 15 instructions in all, of which about five are its own (bf16: unpack, half a
// packed max, and multiply-add, ex2 and add of the sum, two at a time); no unit is near its limit.
// The n largest come without sorting: the r-th largest of a warp's 32 lane maxima, r = ceil(n / warps),
// has r elements of that warp at or above it, so the least of these over the warps has n of the CTA;
// what reaches it (20 to 140 elements for n = 1 to 64 of well-mixed logits) goes to shared memory, and each
// finds its rank by counting.  Where more than kCap reach it (long runs of equal or sorted logits, masks of a finite value
// with fewer than n live tokens), the exact n-th largest is found by bisection on the key, which costs 5 to 25 times
// as much (32 x 8 rows of 128256 bf16, n 16: 370 to 720 us).
// Merge kernel: one CTA per entry merges the parts' sorted lists of every beam, then the beams' sorted proposals.  Up
// to 8 lists are merged neighbours by neighbours, more by taking the largest of their heads n times, a warp per beam:
// its warp-wide maxima share one slow unit, which costs 49 clocks a beam and key.  (15 x 14 rows of 12692, n = 28: 13.7 us
// by neighbours, 21.9 by heads; 4 x 4 rows of 262144, n = 8, 32 parts: 12.2 and 10.4.)
// Measured: 32 x 8 rows of 128256 bf16 (65.7 MB), n = 16: 28 us, 2.3 TB/s, of which the row kernel 23: a CTA's chunk
// takes 11 to 12 thousand clocks, 3 to 5 of them waiting for its loads and the rest a chain of short steps (threshold,
// sum, candidates, ranks) between six barriers, with 59% of issue slots used; without the sum it took 1.4 us less.
// 4 x 4 rows of 262144 fp32, n = 8: 10.4 us, 9.6 out of a graph.
#include <math.h>
#include <stddef.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kWords = 32;                      // 32-bit words of logits per thread and chunk
constexpr int chunk_of(bool bf16) { return kThreads * kWords * (bf16 ? 2 : 1); }
constexpr int kCap = 256;                       // candidates of a chunk, one per thread
constexpr int kMaxParts = 64;                   // parts of a row: two lists per lane of the merging warp
constexpr int kMergeThreads = 512;
constexpr int kFewParts = 8;                    // parts of a row that are merged by neighbours; more: by their heads
constexpr int kMergeSmem = 160 << 10;
constexpr uint32_t kNinf = 0x007FFFFFu;         // ord_of(-inf); 0 stands for no element

// packed maximum, which passes over NaN
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// order-preserving map of a non-NaN float to uint32 (-inf is the least value any float maps to)
__device__ __forceinline__ uint32_t ord_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ord_to_float(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
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
  uint64_t* keys;  // [rows, parts, n], descending; 0: none
  float2* stats;   // [rows, parts] max, sum of exp(x - max)
  int parts, chunks;  // parts of a row, chunks of a row (the last may be short, or empty)
  int group, area;    // merge: beams whose lists are merged at a time, keys of an area of them
  int64_t lists;      // lists of n keys that `keys` holds, and statistics
  int32_t* status;
};

constexpr int kVecCap = 256;  // vectors with a candidate
constexpr int kKeys = kCap + ORPO_MAX_SELECT;  // a chunk's candidates and the best of the chunks before

struct RowShared {
  alignas(16) uint32_t words[kWords][kThreads];  // the chunk, in the rare paths; else the vectors with a candidate
  uint64_t cand[kKeys];
  uint64_t best[ORPO_MAX_SELECT];
  uint32_t part[kWarps];
  float sum[kWarps];
  uint32_t thr[kWarps];
  int vecs, count, total;
};
static_assert(alignof(RowShared) >= alignof(uint4) && offsetof(RowShared, words) % alignof(uint4) == 0,
              "candidates' vectors are stored as uint4");

// Sum over the CTA of v; every thread gets it.
__device__ __forceinline__ int cta_sum(RowShared& sh, int v) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (threadIdx.x == 0) sh.total = 0;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) atomicAdd(&sh.total, v);
  __syncthreads();
  return sh.total;
}

// (a.x * b + c.x, a.y * b + c.y) and the like, two fp32 operations an instruction
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return ((uint64_t)__float_as_uint(y) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

// a thread's logits of a chunk, as loaded: word w of fp32, or words of two bf16
template <bool kBf16>
struct Elems {
  static constexpr int kVec = kBf16 ? 8 : 4;             // logits per 16-byte load
  static constexpr int kSize = kBf16 ? 2 : 4;
  static constexpr int kN = kWords * (kBf16 ? 2 : 1);    // logits
  static constexpr uint32_t kNone = kBf16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  uint32_t w[kWords];
  __device__ __forceinline__ void put(RowShared& sh) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) sh.words[i][threadIdx.x] = w[i];
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kBf16)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

__device__ __forceinline__ bool bf16_is_bad(uint32_t bits) {  // NaN or +inf
  return (bits & 0x7fffu) > 0x7f80u || bits == 0x7f80u;
}

// Rare paths, on the chunk in shared memory (words[i][thread]); NaN counts as -inf.
template <bool kBf16>
struct Chunk {
  const RowShared& sh;
  int first, last;  // logit of this thread's element 0; the chunk's end
  __device__ __forceinline__ int token_of(int i) const {
    return first + i / Elems<kBf16>::kVec * (kThreads * Elems<kBf16>::kVec) + i % Elems<kBf16>::kVec;
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = sh.words[kBf16 ? i / 2 : i][threadIdx.x];
    const float f = __uint_as_float(!kBf16 ? w : i & 1 ? w & 0xffff0000u : w << 16);
    return f == f ? f : -INFINITY;
  }
  template <class F>
  __device__ __forceinline__ int count(F f) const {
    int k = 0;
#pragma unroll 4
    for (int i = 0; i < Elems<kBf16>::kN; ++i) k += f(i) ? 1 : 0;
    return k;
  }
};

__device__ __forceinline__ uint64_t key_of(float x, int token) {
  return ((uint64_t)ord_of(x) << 32) | (uint32_t)~(uint32_t)token;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(SelectArgs a) {
  using E = Elems<kBf16>;
  constexpr int kVec = E::kVec, kSize = E::kSize, kN = E::kN, kLen = chunk_of(kBf16);
  grid_trigger();  // the merge kernel may be set up meanwhile
  grid_wait();
  const int64_t r = blockIdx.y;
  if (a.finished != nullptr && a.finished[r]) return;
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + r * a.ld * kSize;
  // the row's 16-byte grid starts `off` logits before it: element e of the grid is logit e - off
  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / kSize);
  const int64_t grid_len = (int64_t)a.V + off;
  const int c0 = (int)((uint32_t)a.chunks * blockIdx.x / (uint32_t)a.parts);
  const int c1 = (int)((uint32_t)a.chunks * (blockIdx.x + 1) / (uint32_t)a.parts);
  float run_m = -INFINITY, run_s = 0.f;
  int have = 0;  // keys in sh.best
  for (int c = c0; c < c1; ++c) {
    const int64_t e0 = min((int64_t)c * kLen, grid_len), e1 = min(e0 + kLen, grid_len);
    const int first = (int)(e0 - off) + tid * kVec;  // logit of this thread's element 0
    auto token_of = [&](int i) { return first + i / kVec * (kThreads * kVec) + i % kVec; };
    // ---- load; -inf where there is no logit
    E x;
    const int last = (int)(e1 - off);  // logits of the chunk end here (at most V)
    if (e0 >= off && e1 - e0 == kLen) {  // a whole chunk
      const uint4* src = reinterpret_cast<const uint4*>(row + (e0 - off) * kSize) + tid;
#pragma unroll
      for (int i = 0; i < kN / kVec; ++i) {
        if (!in_bounds(a.status, token_of(i * kVec), a.V - kVec + 1)) continue;
        const uint4 y = __ldg(src + i * kThreads);
        x.w[i * 4] = y.x, x.w[i * 4 + 1] = y.y, x.w[i * 4 + 2] = y.z, x.w[i * 4 + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN / kVec; ++i) {
        const int v = token_of(i * kVec);
        uint32_t* w = x.w + i * 4;
        if (v >= 0 && v <= last - kVec && in_bounds(a.status, v, a.V - kVec + 1)) {
          const uint4 y = __ldg(reinterpret_cast<const uint4*>(row + (int64_t)v * kSize));
          w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = E::kNone;
            if constexpr (kBf16) {
              const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + v + 2 * j;
              if (v + 2 * j >= 0 && v + 2 * j < last && in_bounds(a.status, v + 2 * j, a.V))
                w[j] = (w[j] & 0xffff0000u) | __ldg(p);
              if (v + 2 * j + 1 >= 0 && v + 2 * j + 1 < last && in_bounds(a.status, v + 2 * j + 1, a.V))
                w[j] = (w[j] & 0xffffu) | ((uint32_t)__ldg(p + 1) << 16);
            } else if (v + j >= 0 && v + j < last && in_bounds(a.status, v + j, a.V)) {
              w[j] = __ldg(reinterpret_cast<const uint32_t*>(row) + v + j);
            }
          }
        }
      }
    }
    // ---- maxima (which pass over NaN) of each vector and of the thread
    float vmax[kN / kVec], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN / kVec; ++i) {
      const uint32_t* w = x.w + i * 4;
      if constexpr (kBf16) {
        const uint32_t m2 = bf16x2_max(bf16x2_max(w[0], w[1]), bf16x2_max(w[2], w[3]));
        vmax[i] = fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
      } else {
        vmax[i] = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])), fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
      }
      top = fmaxf(top, vmax[i]);
    }
    // ---- CTA maximum; threshold
    // Warps all of whose lanes hold an element (the grid is dealt out 32 lanes x kVec at a time): one with a few would
    // bring the threshold down to its own few.
    const int active = max(1, min(kWarps, (int)(e1 - e0) / (32 * kVec)));
    const int need = active == kWarps ? (a.n + kWarps - 1) / kWarps : (a.n + active - 1) / active;
    uint32_t rest = ord_of(top), rth = 0, wmax = 0;
    for (int i = 0; i < min(need, 32); ++i) {
      rth = __reduce_max_sync(0xffffffffu, rest);
      if (i == 0) wmax = rth;
      const uint32_t who = __ballot_sync(0xffffffffu, rest == rth);
      if (lane == __ffs((int)who) - 1) rest = 0;
    }
    if (need > 32) rth = 0;  // more than a warp's lanes: no threshold
    __syncthreads();         // the previous chunk's readers of sh are done
    if (lane == 0) {
      sh.part[warp] = wmax;
      sh.thr[warp] = warp < active ? rth : 0xffffffffu;
    }
    if (tid == 0) sh.count = sh.vecs = 0;
    __syncthreads();
    uint32_t cmax = 0, thr = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cmax = max(cmax, sh.part[w]), thr = min(thr, sh.thr[w]);
    if (have == a.n) thr = max(thr, (uint32_t)(sh.best[a.n - 1] >> 32));  // the n-th best of the chunks before
    const float m = ord_to_float(cmax);
    // ---- sum of exp(x - m): 2^(x L - c) with c = m L rounded, which is put right after the sum.  Below 2^24 c is off by
    // half at most; far above, a term may overflow or vanish before it is put right.
    float s = 0.f;
    const float c2 = m * kLog2e;
    if (fabsf(c2) < 0x1p24f) {
      uint64_t s2 = 0;
      const uint64_t l2 = pack2(kLog2e, kLog2e), mc2 = pack2(-c2, -c2);
#pragma unroll
      for (int i = 0; i < kN; i += 2) {
        const uint64_t y = fma2(pack2(x.at(i), x.at(i + 1)), l2, mc2);
        s2 = add2(s2, pack2(ex2_approx(lo2(y)), ex2_approx(hi2(y))));
      }
      s = (lo2(s2) + hi2(s2)) * ex2_approx(-fmaf(m, kLog2e, -c2));
    } else if (m > -INFINITY && m < INFINITY) {  // a mask's value, most likely
      s = NAN;                                   // the slow sum below
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    // ---- NaN or +inf among the warp's logits (a NaN reaches every sum but that of a row without a maximum)
    if (s != s || !(m < INFINITY && m > -INFINITY)) {
      x.put(sh);
      const Chunk<kBf16> ch{sh, first, last};
      bool bad = false;
      s = 0.f;
#pragma unroll 2
      for (int i = 0; i < kWords; ++i) {
        const uint32_t w = sh.words[i][tid];
        bad |= kBf16 ? bf16_is_bad(w & 0xffffu) || bf16_is_bad(w >> 16) : !(__uint_as_float(w) < INFINITY);
      }
      if (m > -INFINITY && m < INFINITY) {
#pragma unroll 2
        for (int i = 0; i < kN; ++i) s += ex2_approx((ch.at(i) - m) * kLog2e);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (bad) atomicOr(a.status, ORPO_STATUS_NONFINITE);
    }
    if (lane == 0) sh.sum[warp] = s;
    // ---- candidates: what reaches the threshold; of masked logits only what is needed, below
    const float live = thr > kNinf ? ord_to_float(thr) : -3.402823466e38f;
    // first the vectors that hold one (most words of a warp's 32 x kVec have none), then their elements
    __syncthreads();  // rare path: its readers of sh.words are done
#pragma unroll
    for (int i = 0; i < kN / kVec; ++i)
      if (vmax[i] >= live) {
        const int at = atomicAdd(&sh.vecs, 1);
        if (at < kVecCap && in_bounds(a.status, at * 8 + 7, kWords * kThreads)) {
          uint32_t* v = &sh.words[0][0] + at * 8;
          v[0] = token_of(i * kVec);
          *reinterpret_cast<uint4*>(v + 4) = make_uint4(x.w[i * 4], x.w[i * 4 + 1], x.w[i * 4 + 2], x.w[i * 4 + 3]);
        }
      }
    __syncthreads();
    const int vecs = sh.vecs;
    if (vecs <= kVecCap) {
      for (int i = tid; i < vecs * kVec; i += kThreads) {
        const uint32_t* v = &sh.words[0][0] + i / kVec * 8;
        const int j = i % kVec;
        const uint32_t w = v[4 + (kBf16 ? j / 2 : j)];
        const float f = __uint_as_float(!kBf16 ? w : j & 1 ? w & 0xffff0000u : w << 16);
        if (f >= live) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kCap && in_bounds(a.status, at, kKeys)) sh.cand[at] = key_of(f, (int)v[0] + j);
        }
      }
    }
    __syncthreads();
    int count = vecs <= kVecCap ? sh.count : kCap + 1;
    __syncthreads();
    if (count > kCap) {
      // ---- exact: the largest t that n logits reach, by bisection, if that many reach `live` at all
      x.put(sh);
      const Chunk<kBf16> ch{sh, first, last};
      uint32_t lo = ord_of(live), hi = cmax;
      const int all = cta_sum(sh, ch.count([&](int i) { return ord_of(ch.at(i)) >= lo; }));
      const int want = min(a.n, all);
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (cta_sum(sh, ch.count([&](int i) { return ord_of(ch.at(i)) >= mid; })) >= want)
          lo = mid;
        else
          hi = mid - 1;
      }
      // of those equal to t the lowest tokens, so many as are missing: the least bound that they lie below
      const int equal = want - cta_sum(sh, ch.count([&](int i) { return ord_of(ch.at(i)) > lo; }));
      int b0 = (int)(e0 - off), b1 = last;
      while (b0 < b1) {
        const int mid = b0 + (b1 - b0) / 2;
        if (cta_sum(sh, ch.count([&](int i) { return ord_of(ch.at(i)) == lo && ch.token_of(i) < mid; })) >= equal)
          b1 = mid;
        else
          b0 = mid + 1;
      }
      if (tid == 0) sh.count = 0;
      __syncthreads();
#pragma unroll 2
      for (int i = 0; i < kN; ++i) {
        const float f = ch.at(i);
        const uint32_t o = ord_of(f);
        if (o > lo || (o == lo && ch.token_of(i) < b0)) {
          const int at = atomicAdd(&sh.count, 1);
          if (in_bounds(a.status, at, kKeys)) sh.cand[at] = key_of(f, ch.token_of(i));
        }
      }
      __syncthreads();
      count = sh.count;
      __syncthreads();
    }
    if (count < a.n && have < a.n) {
      // ---- too few live logits: masked ones by lowest token, all among the first n + count of the chunk
      x.put(sh);
      const Chunk<kBf16> ch{sh, first, last};
      const int from = max((int)(e0 - off), 0), bound = min(last, from + a.n + count);
#pragma unroll 2
      for (int i = 0; i < kN; ++i) {
        const int v = ch.token_of(i);
        if (v >= from && v < bound && ch.at(i) == -INFINITY) {
          const int at = atomicAdd(&sh.count, 1);
          if (in_bounds(a.status, at, kKeys)) sh.cand[at] = key_of(-INFINITY, v);
        }
      }
      __syncthreads();
      count = sh.count;
    }
    // ---- with the best so far: rank by counting (keys are distinct)
    if (tid < have && in_bounds(a.status, count + tid, kKeys)) sh.cand[count + tid] = sh.best[tid];
    __syncthreads();
    count += have;
    for (int i = tid; i < count && in_bounds(a.status, count - 1, kKeys); i += kThreads) {
      const uint64_t key = sh.cand[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < count; ++j) rank += sh.cand[j] > key;
      if (rank < a.n && in_bounds(a.status, rank, ORPO_MAX_SELECT)) sh.best[rank] = key;
    }
    have = min(count, a.n);
    // ---- running statistics (every thread keeps them)
    float cs = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cs += sh.sum[w];
    if (m == INFINITY || run_m == INFINITY) {
      run_m = INFINITY;
    } else if (m > -INFINITY) {
      const float mm = fmaxf(run_m, m);
      run_s = (run_m > -INFINITY ? run_s * ex2_approx((run_m - mm) * kLog2e) : 0.f) + cs * ex2_approx((m - mm) * kLog2e);
      run_m = mm;
    }
  }
  __syncthreads();
  const int64_t list = r * a.parts + blockIdx.x;
  if (!in_bounds(a.status, list, a.lists)) return;
  for (int i = tid; i < a.n; i += kThreads) a.keys[list * a.n + i] = i < have ? sh.best[i] : 0;
  if (tid == 0) a.stats[list] = make_float2(run_m, run_s);
}

// The n largest of each group's lists of n keys (descending, distinct but for the 0 of no key): neighbours are merged,
// a key's rank being its place in its own list plus the number of the other's that are greater (binary search), until
// one list is left.  Lists in `from`, in turns to `to`; returns where they end.  (Four at a time, three searches side
// by side, took 1 to 2 us longer.)  `size`: keys that both hold at least.
__device__ __forceinline__ uint64_t* merge_lists(uint64_t* from, uint64_t* to, int groups, int lists, int n, int size, int32_t* status) {
  while (lists > 1) {
    const int half = (lists + 1) / 2, total = groups * lists * n;
    for (int t = threadIdx.x; t < total && in_bounds(status, total - 1, size); t += blockDim.x) {
      const int list = t / n, j = t - list * n, g = list / lists, l = list - g * lists;
      const uint64_t key = from[t];
      int rank = j;
      if ((l ^ 1) < lists) {
        const uint64_t* const other = from + (g * lists + (l ^ 1)) * n;
        int lo = 0, hi = n - j;  // further ones do not matter
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (in_bounds(status, (g * lists + (l ^ 1)) * n + mid, total) && other[mid] > key)
            lo = mid + 1;
          else
            hi = mid;
        }
        rank += lo;
      }
      if (rank < n && in_bounds(status, (g * half + l / 2) * n + rank, size)) to[(g * half + l / 2) * n + rank] = key;
    }
    __syncthreads();
    uint64_t* const swap = from;
    from = to, to = swap, lists = half;
  }
  return from;
}

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// The same for up to kMaxParts lists by a warp per group: n times the largest of the lists' heads, of which a lane holds
// those of lists lane and lane + 32.
__device__ __forceinline__ void merge_heads(const uint64_t* from, uint64_t* to, int groups, int lists, int n, int size, int32_t* status) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x / 32; g < groups; g += blockDim.x / 32) {
    if (!in_bounds(status, (g + 1) * lists * n - 1, size) || !in_bounds(status, lists - 1, kMaxParts)) break;
    const uint64_t* const mine = from + g * lists * n;
    int h0 = 0, h1 = 0;
    uint64_t k0 = lane < lists ? mine[lane * n] : 0, k1 = lane + 32 < lists ? mine[(lane + 32) * n] : 0;
    for (int i = 0; i < n; ++i) {
      const uint64_t best = warp_max(k0 > k1 ? k0 : k1);
      if (lane == 0) to[g * n + i] = best;
      if (best == k0 && k0 != 0) k0 = ++h0 < n ? mine[lane * n + h0] : 0;
      if (best == k1 && k1 != 0) k1 = ++h1 < n ? mine[(lane + 32) * n + h1] : 0;
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kMergeThreads) select_merge_kernel(SelectArgs a) {
  extern __shared__ uint64_t lists[];  // two areas of `area` keys; then tokens [beams, n]
  grid_trigger();
  grid_wait();  // the row kernel's lists are there
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, n = a.n;
  __shared__ uint8_t over[ORPO_MAX_BEAMS];
  __shared__ float beam_score[ORPO_MAX_BEAMS], beam_max[ORPO_MAX_BEAMS], beam_log[ORPO_MAX_BEAMS];
  uint64_t* const area0 = lists;
  uint64_t* const area1 = lists + a.area;
  uint64_t* const best = area1 + a.area;  // [beams, n]: value, then beam and place
  int* const token = reinterpret_cast<int*>(best + a.beams * n);
  // log-sum-exp of every beam, as maximum and log of the sum: a warp takes its parts' statistics, at most two per lane
  for (int k = warp; k < a.beams; k += warps) {
    const int64_t r = b * a.beams + k;
    if (!in_bounds(a.status, (r + 1) * a.parts - 1, a.lists) || !in_bounds(a.status, k, ORPO_MAX_BEAMS)) break;
    const bool ended = a.finished != nullptr && a.finished[r];
    const float score = a.score[r];
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 s0 = !ended && lane < a.parts ? a.stats[r * a.parts + lane] : none;
    const float2 s1 = !ended && lane + 32 < a.parts ? a.stats[r * a.parts + lane + 32] : none;
    float m = fmaxf(s0.x, s1.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float log_s = 0.f;
    if (fabsf(m) < INFINITY) {
      float s = (s0.x > -INFINITY ? s0.y * ex2_approx((s0.x - m) * kLog2e) : 0.f) +
                (s1.x > -INFINITY ? s1.y * ex2_approx((s1.x - m) * kLog2e) : 0.f);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      log_s = logf(s);
    }
    if (lane == 0) {
      if (score != score) atomicOr(a.status, ORPO_STATUS_NONFINITE);
      over[k] = ended, beam_score[k] = score, beam_max[k] = m, beam_log[k] = log_s;
    }
  }
  __syncthreads();
  // every beam's n largest keys, as many beams at a time as their parts' lists fit, and their values
  for (int k0 = 0; k0 < a.beams; k0 += a.group) {
    const int group = min(a.group, a.beams - k0), per_beam = a.parts * n;
    const uint64_t* const src = a.keys + (b * a.beams + k0) * per_beam;
#pragma unroll 4
    for (int t = tid; t < group * per_beam; t += blockDim.x)
      if (in_bounds(a.status, t, a.area) && in_bounds(a.status, (b * a.beams + k0) * per_beam + t, a.lists * n))
        area0[t] = over[k0 + t / per_beam] ? 0 : src[t];
    __syncthreads();
    const uint64_t* top = area1;
    if (a.parts <= kFewParts)
      top = merge_lists(area0, area1, group, a.parts, n, a.area, a.status);
    else
      merge_heads(area0, area1, group, a.parts, n, a.area, a.status);
    for (int t = tid; t < group * n; t += blockDim.x) {
      const int k = k0 + t / n, j = t % n;
      if (!in_bounds(a.status, k, a.beams)) break;
      const float score = beam_score[k], m = beam_max[k];
      float y = -INFINITY;
      if (over[k]) {
        if (j == 0) y = score;
      } else {
        const float x = ord_to_float((uint32_t)(top[t] >> 32));
        if (x > -INFINITY && fabsf(m) < INFINITY) y = score + ((x - m) - beam_log[k]);
      }
      if (y != y) y = -INFINITY;
      const int at = k * n + j;
      token[at] = over[k] ? a.eos : (int)~(uint32_t)top[t];
      best[at] = key_of(y, at);  // of equal values the lower beam first, and within a beam its own order
    }
    __syncthreads();
  }
  const uint64_t* const top = a.beams > 1 ? merge_lists(best, area0, 1, a.beams, n, a.beams * n, a.status) : best;
  for (int i = tid; i < n; i += blockDim.x) {
    const uint64_t key = top[i];
    const int from = (int)~(uint32_t)key, k = from / n;
    if (!in_bounds(a.status, from, a.beams * n)) continue;
    const int64_t at = b * n + i;
    a.out_score[at] = ord_to_float((uint32_t)(key >> 32));
    a.out_parent[at] = k;
    a.out_token[at] = token[from];
    if (a.out_finished) a.out_finished[at] = over[k] || token[from] == a.eos;
  }
}

// Chunks of a row, and the parts (CTAs) they are dealt to.
struct RowPlan {
  int chunks, parts;
};
RowPlan row_plan(int64_t V, bool bf16, bool aligned) {
  RowPlan p;
  const int64_t grid = V + (aligned ? 0 : 7);  // up to 7 elements of a row's grid lie before it
  p.chunks = (int)cdiv(grid, chunk_of(bf16));
  p.parts = std::min(p.chunks, kMaxParts);
  return p;
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
  return (size_t)(batch * beams) * row_plan(V, false, false).parts * ((size_t)n * 8 + 8) + 16;
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
  const int size = logits_bf16 ? 2 : 4;
  const RowPlan plan = row_plan(V, logits_bf16 != 0, aligned16(logits) && (ld_logits * size) % 16 == 0);
  SelectArgs a{logits, ld_logits, score, finished, eos, beams, (int)V, n, out_score, out_parent, out_token,
               out_finished, static_cast<uint64_t*>(workspace), nullptr, plan.parts, plan.chunks, 0, 0, rows * plan.parts, status};
  a.stats = reinterpret_cast<float2*>(a.keys + rows * plan.parts * n);
  // rows in launches of at most 65535
  prof_begin(K_BEAM, st);
  cudaError_t e = cudaSuccess;
  for (int64_t r = 0; r < rows && e == cudaSuccess; r += 65535) {
    SelectArgs c = a;
    c.logits = static_cast<const uint8_t*>(logits) + r * ld_logits * size;
    if (finished) c.finished = finished + r;
    c.keys = a.keys + r * plan.parts * n;
    c.stats = a.stats + r * plan.parts;
    c.lists = a.lists - r * plan.parts;
    const dim3 grid((unsigned)plan.parts, (unsigned)std::min<int64_t>(65535, rows - r));
    e = logits_bf16 ? launch_dependent(select_rows_kernel<true>, grid, kThreads, 0, st, c)
                    : launch_dependent(select_rows_kernel<false>, grid, kThreads, 0, st, c);
  }
  prof_end(K_BEAM, st);
  if (e != cudaSuccess) return ORPO_ERR_CUDA;
  // as many beams' lists at a time as fit shared memory twice, beside every beam's n best and their tokens
  const int per_beam = plan.parts * n, bests = beams * n;
  a.group = std::min(beams, (int)((kMergeSmem - bests * 12) / (per_beam * 16)));  // at least 1: 16 * 4096 bytes of 112 KiB
  a.area = std::max(a.group * per_beam, bests);  // the beams' own lists are merged there too
  const size_t smem = (size_t)a.area * 16 + (size_t)bests * 12;
  static std::atomic<int> done[64];
  if (opt_in_smem(select_merge_kernel, kMergeSmem, done) != cudaSuccess) return ORPO_ERR_CUDA;
  prof_begin(K_BEAM, st);
  // it may be set up while the row kernel runs
  const int threads = std::min(kMergeThreads, std::max(128, (int)cdiv(a.group * per_beam, 32) * 32));
  e = launch_dependent(select_merge_kernel, dim3((unsigned)batch), threads, smem, st, a);
  prof_end(K_BEAM, st);
  return e == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
