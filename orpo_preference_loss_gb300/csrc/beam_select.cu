// beam_select.cu — the n best continuations over beams x vocabulary (orpo_beam_select).
//
//   lse_r = log sum_v exp x_rv,  value(k, v) = score_k + (x_kv - lse_k)
//
// Within a beam the value grows with the logit, so a beam's proposals are its n largest logits and
// the softmax statistics are needed only for those.  Order inside a beam is a 64-bit key (the
// logit's bits mapped to an order-preserving integer, then the complement of the token), which is
// total, so ties and scheduling cannot change the result.
//
// Row kernel: a CTA reads a part of one beam's row once, 8192 logits at a time in registers (32 per
// thread, all loads in flight together), and leaves the part's max, sum of exp and n largest keys.
// The n largest come without sorting: the r-th largest of a warp's 32 lane maxima, r = ceil(n / warps),
// has r elements of that warp at or above it, so the least of these over the warps has n of the CTA;
// what reaches it (20 to 140 elements for n = 1 to 64 of well-mixed logits) goes to shared memory, and each
// finds its rank by counting.  Where more than kCap reach it (long runs of equal or sorted logits), the exact
// n-th largest is found by bisection on the key.
// Merge kernel: one CTA per entry; a warp per beam merges its parts' sorted lists and statistics, then
// the beams' sorted proposals are ranked by value.
// Bound by reading the logits (largev, 32 x 8 rows, bf16: 65.7 MB).
#include <math.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kElems = 32;                      // logits per thread and chunk
constexpr int kChunk = kThreads * kElems;       // 8192
constexpr int kCap = 256;                       // candidates of a chunk, one per thread
constexpr int kMaxParts = 64;                   // parts of a row: two lists per lane of the merging warp
constexpr int kMergeThreads = 512;
constexpr int kMergeSmem = 160 << 10;
constexpr uint32_t kNinf = 0x007FFFFFu;         // ord_of(-inf); 0 stands for no element

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
  int parts, chunks;  // parts of a row, chunks of a row
  int list_warps;     // merge: warps that merge beams
  int32_t* status;
};

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

struct RowShared {
  uint64_t cand[kCap + ORPO_MAX_SELECT];
  uint64_t best[ORPO_MAX_SELECT];
  uint32_t part[kWarps];
  float sum[kWarps];
  uint32_t thr[kWarps];
  int count, total;
};

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

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(SelectArgs a) {
  constexpr int kVec = kBf16 ? 8 : 4;        // logits per 16-byte load
  constexpr int kSize = kBf16 ? 2 : 4;
  const int64_t r = blockIdx.y;
  if (a.finished != nullptr && a.finished[r]) return;
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + r * a.ld * kSize;
  // the row's 16-byte grid starts `off` logits before it: element e of the grid is logit e - off
  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / kSize);
  const int64_t grid_len = (int64_t)a.V + off;
  const int c0 = (int)((int64_t)a.chunks * blockIdx.x / a.parts), c1 = (int)((int64_t)a.chunks * (blockIdx.x + 1) / a.parts);
  // chunks of equal length, a multiple of 256 grid elements (the last may be short, or empty)
  const int64_t len = (grid_len + (int64_t)a.chunks * 256 - 1) / ((int64_t)a.chunks * 256) * 256;
  float run_m = -INFINITY, run_s = 0.f;
  int have = 0;  // keys in sh.best
  for (int c = c0; c < c1; ++c) {
    const int64_t e0 = c * len, e1 = min(e0 + len, grid_len);
    // ---- load: ord_of of each logit, 0 where there is none
    uint32_t o[kElems];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kElems / kVec; ++i) {
      const int64_t e = e0 + ((int64_t)i * kThreads + tid) * kVec, v = e - off;
      uint32_t w[kVec];  // fp32 bits
      if (e < e1 && v >= 0 && v + kVec <= a.V) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + v * kSize));
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < kVec; ++j) w[j] = kBf16 ? (j & 1 ? y[j / 2] & 0xffff0000u : y[j / 2] << 16) : y[j];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float f = __uint_as_float(w[j]);
          bad |= !(f < INFINITY);
          o[i * kVec + j] = f == f ? ord_of(f) : kNinf;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          o[i * kVec + j] = 0;
          if (e < e1 && v + j >= 0 && v + j < a.V) {
            float f;
            if constexpr (kBf16)
              f = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row) + v + j) << 16);
            else
              f = __ldg(reinterpret_cast<const float*>(row) + v + j);
            bad |= !(f < INFINITY);
            o[i * kVec + j] = f == f ? ord_of(f) : kNinf;
          }
        }
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, ORPO_STATUS_NONFINITE);
    // logit of element i of this thread
    auto token_of = [&](int i) { return (int)(e0 + ((int64_t)(i / kVec) * kThreads + tid) * kVec + i % kVec - off); };
    // ---- max; threshold
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kElems; ++i) top = max(top, o[i]);
    // warps that hold an element: the grid is dealt out 32 lanes x kVec at a time
    const int active = (int)max((int64_t)1, min((int64_t)kWarps, (e1 - e0 + 32 * kVec - 1) / (32 * kVec)));
    const int need = (a.n + active - 1) / active;
    uint32_t rest = top, rth = 0, wmax = 0;
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
    if (tid == 0) sh.count = 0;
    __syncthreads();
    uint32_t cmax = 0, thr = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cmax = max(cmax, sh.part[w]), thr = min(thr, sh.thr[w]);
    if (have == a.n) thr = max(thr, (uint32_t)(sh.best[a.n - 1] >> 32));  // the n-th best of the chunks before
    // ---- sum of exp(x - max)
    const float m = cmax > kNinf ? ord_to_float(cmax) : -INFINITY;
    float s = 0.f;
    if (m > -INFINITY && m < INFINITY) {
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (o[i] > kNinf) s += ex2_approx((ord_to_float(o[i]) - m) * kLog2e);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) sh.sum[warp] = s;
    // ---- candidates: what reaches the threshold; of masked logits only what is needed, below
    const uint32_t live = max(thr, kNinf + 1);
#pragma unroll
    for (int i = 0; i < kElems; ++i)
      if (o[i] >= live) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kCap) sh.cand[at] = ((uint64_t)o[i] << 32) | (uint32_t)~(uint32_t)token_of(i);
      }
    __syncthreads();
    int count = sh.count;
    __syncthreads();
    if (count > kCap) {
      // ---- exact: the largest t that n elements reach (at least kCap > n do reach `live`)
      uint32_t lo = live, hi = cmax;
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        int k = 0;
#pragma unroll
        for (int i = 0; i < kElems; ++i) k += o[i] >= mid;
        if (cta_sum(sh, k) >= a.n)
          lo = mid;
        else
          hi = mid - 1;
      }
      int k = 0;
#pragma unroll
      for (int i = 0; i < kElems; ++i) k += o[i] > lo;
      const int equal = a.n - cta_sum(sh, k);  // so many of those equal to t, the lowest tokens
      int64_t b0 = e0 - off, b1 = e1 - off;    // the least bound that so many lie below
      while (b0 < b1) {
        const int64_t mid = b0 + (b1 - b0) / 2;
        k = 0;
#pragma unroll
        for (int i = 0; i < kElems; ++i) k += o[i] == lo && token_of(i) < mid;
        if (cta_sum(sh, k) >= equal)
          b1 = mid;
        else
          b0 = mid + 1;
      }
      if (tid == 0) sh.count = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (o[i] > lo || (o[i] == lo && token_of(i) < b0))
          sh.cand[atomicAdd(&sh.count, 1)] = ((uint64_t)o[i] << 32) | (uint32_t)~(uint32_t)token_of(i);
      __syncthreads();
      count = sh.count;
    } else if (count < a.n && have < a.n) {
      // ---- too few live logits: masked ones by lowest token, all among the first n + count of the chunk
      const int64_t bound = max(e0 - off, (int64_t)0) + a.n + count;
#pragma unroll
      for (int i = 0; i < kElems; ++i)
        if (o[i] == kNinf && token_of(i) < bound)
          sh.cand[atomicAdd(&sh.count, 1)] = ((uint64_t)o[i] << 32) | (uint32_t)~(uint32_t)token_of(i);
      __syncthreads();
      count = sh.count;
    }
    // ---- with the best so far: rank by counting (keys are distinct)
    if (tid < have) sh.cand[count + tid] = sh.best[tid];
    __syncthreads();
    count += have;
    for (int i = tid; i < count; i += kThreads) {
      const uint64_t key = sh.cand[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < count; ++j) rank += sh.cand[j] > key;
      if (rank < a.n) sh.best[rank] = key;
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
  for (int i = tid; i < a.n; i += kThreads) a.keys[list * a.n + i] = i < have ? sh.best[i] : 0;
  if (tid == 0) a.stats[list] = make_float2(run_m, run_s);
}

__global__ void __launch_bounds__(kMergeThreads) select_merge_kernel(SelectArgs a) {
  extern __shared__ uint64_t lists[];  // one per warp: the keys of its beam's parts; then values and tokens
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ uint8_t over[ORPO_MAX_BEAMS];
  float* const value = reinterpret_cast<float*>(lists + (size_t)a.list_warps * a.parts * a.n);  // [beams, n]
  int* const token = reinterpret_cast<int*>(value + a.beams * a.n);
  for (int k = warp; warp < a.list_warps && k < a.beams; k += a.list_warps) {
    const int64_t r = b * a.beams + k;
    const float score = a.score[r];
    const bool ended = a.finished != nullptr && a.finished[r];
    if (score != score && lane == 0) atomicOr(a.status, ORPO_STATUS_NONFINITE);
    if (lane == 0) over[k] = ended;
    if (ended) {
      for (int i = lane; i < a.n; i += 32) {
        value[k * a.n + i] = i == 0 && score == score ? score : -INFINITY;
        token[k * a.n + i] = a.eos;
      }
      continue;
    }
    uint64_t* const mine = lists + (size_t)warp * a.parts * a.n;
    const uint64_t* src = a.keys + r * a.parts * a.n;
    for (int i = lane; i < a.parts * a.n; i += 32) mine[i] = src[i];
    // log-sum-exp of the parts, at most two per lane
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 s0 = lane < a.parts ? a.stats[r * a.parts + lane] : none;
    const float2 s1 = lane + 32 < a.parts ? a.stats[r * a.parts + lane + 32] : none;
    float m = fmaxf(s0.x, s1.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float lse = m;
    if (fabsf(m) < INFINITY) {
      float s = (s0.x > -INFINITY ? s0.y * ex2_approx((s0.x - m) * kLog2e) : 0.f) +
                (s1.x > -INFINITY ? s1.y * ex2_approx((s1.x - m) * kLog2e) : 0.f);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      lse = m + logf(s);
    }
    __syncwarp();
    // the n largest of the sorted lists: each lane holds the heads of lists lane and lane + 32
    int h0 = 0, h1 = 0;
    uint64_t k0 = lane < a.parts ? mine[lane * a.n] : 0, k1 = lane + 32 < a.parts ? mine[(lane + 32) * a.n] : 0;
    for (int i = 0; i < a.n; ++i) {
      const uint64_t best = warp_max(k0 > k1 ? k0 : k1);
      if (lane == 0) {
        const float x = ord_to_float((uint32_t)(best >> 32));
        float y = -INFINITY;
        if (x > -INFINITY && fabsf(lse) < INFINITY) y = score + (x - lse);
        value[k * a.n + i] = y == y ? y : -INFINITY;
        token[k * a.n + i] = (int)~(uint32_t)best;
      }
      if (best == k0) k0 = ++h0 < a.n ? mine[lane * a.n + h0] : 0;
      if (best == k1) k1 = ++h1 < a.n ? mine[(lane + 32) * a.n + h1] : 0;
    }
  }
  __syncthreads();
  // Each beam's proposals are in order, so a proposal's rank is its place in its own beam plus, for every
  // other beam, the number of that beam's proposals that come before it (a binary search).
  for (int i = threadIdx.x; i < a.beams * a.n; i += blockDim.x) {
    const int k = i / a.n, j = i - k * a.n;
    const float v = value[i];
    int rank = j;
    for (int q = 0; q < a.beams && rank < a.n; ++q) {
      if (q == k) continue;
      // of beam q those with a greater value, or an equal one if q < k
      int lo = 0, hi = a.n;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        const float w = value[q * a.n + mid];
        if (q < k ? w >= v : w > v)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank < a.n) {
      const int64_t at = b * a.n + rank;
      a.out_score[at] = v;
      a.out_parent[at] = k;
      a.out_token[at] = token[i];
      if (a.out_finished) a.out_finished[at] = over[k] || token[i] == a.eos;
    }
  }
}

// Chunks of a row, and the parts (CTAs) they are dealt to.
struct RowPlan {
  int chunks, parts;
};
RowPlan row_plan(int64_t V, bool aligned) {
  RowPlan p;
  p.chunks = (int)cdiv(V + (aligned ? 0 : 7), kChunk);  // up to 7 elements of a row's grid lie before it
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
  return (size_t)(batch * beams) * row_plan(V, false).parts * ((size_t)n * 8 + 8) + 16;
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
  const RowPlan plan = row_plan(V, aligned16(logits) && (ld_logits * size) % 16 == 0);
  SelectArgs a{logits, ld_logits, score, finished, eos, beams, (int)V, n, out_score, out_parent, out_token,
               out_finished, static_cast<uint64_t*>(workspace), nullptr, plan.parts, plan.chunks, 0, status};
  a.stats = reinterpret_cast<float2*>(a.keys + rows * plan.parts * n);
  // rows in launches of at most 65535
  prof_begin(K_BEAM, st);
  for (int64_t r = 0; r < rows; r += 65535) {
    SelectArgs c = a;
    c.logits = static_cast<const uint8_t*>(logits) + r * ld_logits * size;
    if (finished) c.finished = finished + r;
    c.keys = a.keys + r * plan.parts * n;
    c.stats = a.stats + r * plan.parts;
    const dim3 grid((unsigned)plan.parts, (unsigned)std::min<int64_t>(65535, rows - r));
    if (logits_bf16)
      select_rows_kernel<true><<<grid, kThreads, 0, st>>>(c);
    else
      select_rows_kernel<false><<<grid, kThreads, 0, st>>>(c);
  }
  prof_end(K_BEAM, st);
  if (cudaGetLastError() != cudaSuccess) return ORPO_ERR_CUDA;
  // a warp per beam, as many as their lists fit shared memory (one list: at most 32 KiB)
  const size_t out_bytes = (size_t)beams * n * 8, list_bytes = (size_t)plan.parts * n * 8;
  const int warps = (int)std::min<size_t>({(size_t)kMergeThreads / 32, (size_t)beams, (kMergeSmem - out_bytes) / list_bytes});
  const size_t smem = warps * list_bytes + out_bytes;
  a.list_warps = warps;
  static std::atomic<int> done[64];
  if (opt_in_smem(select_merge_kernel, kMergeSmem, done) != cudaSuccess) return ORPO_ERR_CUDA;
  prof_begin(K_BEAM, st);
  select_merge_kernel<<<(unsigned)batch, std::max(warps, 4) * 32, smem, st>>>(a);
  prof_end(K_BEAM, st);
  return cudaGetLastError() == cudaSuccess ? ORPO_OK : ORPO_ERR_CUDA;
}
