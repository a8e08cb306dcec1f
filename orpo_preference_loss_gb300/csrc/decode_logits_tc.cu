// decode_logits_tc.cu — logits of up to 64 rows of h per pass over the quantised head, on tcgen05.
//
//   D[v, m] = sum_k W[v, k] h[m, k],  W[v, k] = bf16(scale q + bias)
//
// A CTA takes tiles of 128 vocabulary rows.  The weights are the A operand (128 rows of the tile, in
// tensor memory) and h the B operand (N = 16, 32 or 64 columns, in shared memory), so the tensor core
// does as little more than the 2 M V d useful flop as its least N allows, and the dequantised weights
// never cross shared memory (at 40 weights a clock per SM, writing them there and reading them back
// would take 160 B/clk of its 128).  What a call costs beside reading the weights once is turning q
// into bf16: 9 instructions per 8 weights where the scales allow it (dequant4_scaled), 15 where not.
//
// Roles (warps):
//   0       TMA of q: segments (128 bytes of each of the tile's rows: 256 columns, 8-bit 128; one swizzled
//           16 KiB box) into a ring
//   1       MMA issue
//   2       streamed h (below)
//   4..7    scales and biases, 32 rows each: (scale, bias) words beside the segment of q in the ring; scales
//           multiplied by 2^133 where those of 32 rows are all small enough, which a flag of the stage says
//   8..     sums and output of the accumulators, a thread per vocabulary row and up to 32 columns
//   then    dequantisation: three groups of 4 warps in turns, a thread per vocabulary row of a segment
//
// Why turns and whole segments: a warp's fixed costs per segment (waits that find nothing to wait for take 90
// clocks each, first loads 150, releases) are hidden only by warps that are at another point of their segment.
// Four groups with a quarter of every segment each went in step and took 91 us where turns took 79 (one row,
// d 2560, V 262144), and with the plain form of the dequantisation in a loop apart 70.  Tensor memory holds A of three
// segments (8-bit: six) beside two sets of accumulators.
//
// Measured: one row, d 2560, V 262144, groups of 64, fp32 logits: 65 to 66 us, 5.8 TB/s or 86% of the rate of a plain copy;
// steady state 855 clocks a segment, where that rate would allow 790.  64 rows, d 4096, V 128256: 73 to 77 us, 4.2 TB/s
// and 900 TFLOP/s; without the products 63.  Calls with little work per SM (8 rows, 8 bits, d 2048, V 32000: 17 us for
// 74 MB) spend 4 us until the first product: memory answers the first requests of all SMs at once.
//
// Order of k: 4-bit dequantisation yields the pairs (0,4), (1,5), (2,6), (3,7) of 8 consecutive weights
// (8-bit: (0,2), (1,3) of 4), which go to tensor memory as they are; h gets the same order, 16 bytes at a
// time.  Rows of h that fit beside the weights (16 of d up to 3328, 64 of 768) are loaded and put in that order by
// each CTA, once.  More are streamed: a small kernel first writes h in that order, and as
// shared memory holds it, to the workspace, and each CTA fetches every segment with one plain bulk copy for each
// of its tiles.  At 64 rows that is twice the weights' bytes from L2, which keeps up: pairs of CTAs
// that shared each segment took no less.
// Accuracy: the tensor core truncates as it accumulates (measured: 1e-9 of the result per product, one
// sign), so an accumulator spans 512 columns and those sums are added in registers, rounding.
#include <math.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "decode_logits.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr int kTileRows = 128;
constexpr int kBoxBytes = kTileRows * 128;            // a TMA box: 128 bytes of every row, up to 16 KiB
constexpr int kUnitK = 128;                           // columns per unit of h
constexpr int kAccK = 512;                            // columns per accumulator
constexpr int seg_k(int bits) { return 1024 / bits; } // columns per segment: a box of q
constexpr int scale_bytes(int bits) { return seg_k(bits) / 32 * kTileRows * 4; }  // (scale, bias) words of a segment, at most one per 32 columns
constexpr int kMaxStages = 9;
constexpr int kMaxH = 8;  // streamed h: segments in the ring
constexpr int kGroups = 3;                            // dequantising groups
constexpr int kTmemA = 128, kTmemACols = 384;         // A in tensor memory, beside two sets of accumulators
constexpr int a_slots(int bits) { return kTmemACols / (seg_k(bits) / 2); }
constexpr int kMaxASlots = a_slots(8);
constexpr int kHWarp = 2, kScaleWarp = 4, kSumWarp = 8;
constexpr uint64_t kLimitNs = 4000000000ull;          // far above any legitimate wait
constexpr int kSmemLimit = 232448 - 1024;             // less the slack that aligns the base

struct TcCtl {
  uint64_t w_full[kMaxStages], w_empty[kMaxStages];
  uint64_t a_full[kMaxASlots], a_empty[kMaxASlots];
  uint64_t d_full[2], d_empty[2];          // [set]
  uint64_t h_full[kMaxH], h_empty[kMaxH];  // streamed h
  uint64_t h_ready;                        // resident h is there
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  uint8_t plain[kMaxStages][4];  // per stage a byte for each 32 rows: 1 if their scales are as they are, not times 2^133
};
constexpr int kCtlBytes = 1024;
static_assert(sizeof(TcCtl) <= kCtlBytes, "control block");

struct TcArgs {
  LogitsArgs a;
  int tiles, segs;        // tiles, segments per row
  int rows;               // vocabulary rows per tile, at most 128
  int units;              // 128-column units per row: segs * units per segment
  int ngroups;            // groups per row
  int seg_words, shift;   // scale words per segment: one per 2^shift times 32 columns
  uint32_t gmul;          // group of word j of a row: j if 0, else umulhi(j, gmul)
  int stages;             // weight ring
  int hslots;             // streamed h: segments in the ring
  const uint8_t* image;   // streamed h: [m tiles][units] units as shared memory holds them
  int64_t image_bytes;
  int word_groups;        // a scale word is a group (and its index that of the group)
  int wide_scales;        // and a segment's scales and biases are one aligned word of up to 16 bytes each
  int prefetch_scales;    // they start on 16 bytes
};

// One wait of up to kPollNs in the barrier unit: the polls of eight waiting warps at the default
// interval took as many issue slots as the dequantisation.
constexpr uint32_t kPollNs = 20000;
__device__ __forceinline__ bool poll_bar(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kPollNs)
      : "memory");
  return ok != 0;
}

// Bounded wait: false on a timeout (reported) or when another role gave up.
__device__ __forceinline__ bool wait_bar(TcCtl* ctl, uint64_t* bar, uint32_t parity, int32_t* status) {
  if (__builtin_expect(poll_bar(bar, parity), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!poll_bar(bar, parity)) {
    if (ctl->abort_flag) return false;
    if (globaltimer_ns() - t0 > kLimitNs) {
      atomicOr(status, ORPO_STATUS_TIMEOUT);
      ctl->abort_flag = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool wait_warp(TcCtl* ctl, uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, wait_bar(ctl, bar, parity, status));
}

__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 200000000ull) return;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 in, fp32 accumulate
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

// `bytes` (a multiple of 16) of global memory to shared memory, counted on the barrier
__device__ __forceinline__ void bulk_load(const void* src, uint32_t bytes, void* dst, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

#define ORPO_IN16(r, o)                                                                                              \
  "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7]), \
      "r"(r[o + 8]), "r"(r[o + 9]), "r"(r[o + 10]), "r"(r[o + 11]), "r"(r[o + 12]), "r"(r[o + 13]), "r"(r[o + 14]),  \
      "r"(r[o + 15])

// 32 columns of this thread's lane (warp's quadrant)
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      ORPO_IN16(r, 0), ORPO_IN16(r, 16)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}
// Bring `bytes` (a multiple of 16) from a 16-byte aligned address to L2.
__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// 8 values of h in the order of the dequantised weights' pairs
template <int kBits>
__device__ __forceinline__ uint4 reorder_pairs(const uint4& x) {
  if constexpr (kBits == 4)
    return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                      __byte_perm(x.y, x.w, 0x7632));
  else
    return make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x5410),
                      __byte_perm(x.z, x.w, 0x7632));
}

// f(0..3, word) over a vector's words
template <class F>
__device__ __forceinline__ void unpack(const uint4& v, F f) {
  f(0, v.x), f(1, v.y), f(2, v.z), f(3, v.w);
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t group_of(const TcArgs& p, uint32_t word) {
  return p.gmul ? __umulhi(word, p.gmul) : word;
}

// W values from any address: the aligned 8-byte words (W = 2: 4-byte ones) that hold them, and, once they are there, the
// values put together.  Reads less than a word before and past them.
template <int W>
struct Shifted {
  static constexpr int kWord = W > 2 ? 8 : 4, n = W * 2 / kWord, kWords = (n + 1) * kWord / 4;
  // whether what load(base + at) reads lies among `size` values from `base` on
  static __device__ __forceinline__ bool inside(const uint16_t* base, int64_t at, int64_t size, int32_t* status) {
    const int s = (int)(reinterpret_cast<uintptr_t>(base + at) & (kWord - 1)) / 2;
    return in_bounds(status, at - s, size) && in_bounds(status, at - s + (s != 0 ? n + 1 : n) * (kWord / 2) - 1, size);
  }
  static __device__ __forceinline__ void load(const uint16_t* p, uint32_t (&w)[kWords]) {
    const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(p) & (kWord - 1);
    const uint8_t* const q = reinterpret_cast<const uint8_t*>(p) - s;
#pragma unroll
    for (int i = 0; i <= n; ++i) {
      if constexpr (kWord == 8) {
        uint2 v = make_uint2(0u, 0u);
        if (i < n || s != 0) v = __ldg(reinterpret_cast<const uint2*>(q) + i);
        w[2 * i] = v.x, w[2 * i + 1] = v.y;
      } else {
        w[i] = i < n || s != 0 ? __ldg(reinterpret_cast<const uint32_t*>(q) + i) : 0u;
      }
    }
  }
  static __device__ __forceinline__ void take(const uint32_t (&w)[kWords], uint32_t s, uint32_t (&out)[W / 2]) {
    uint32_t t[W / 2 + 1];
#pragma unroll
    for (int i = 0; i <= W / 2; ++i) t[i] = kWord == 8 && (s & 4) ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) out[i] = __funnelshift_r(t[i], t[i + 1], (s & 2) * 8);
  }
};

// The rows' scales and biases of a tile, contiguous, to L2, by the two threads with lane 0 and 1.
__device__ __forceinline__ void prefetch_scales(const TcArgs& p, int64_t tile, int lane) {
  const LogitsArgs& a = p.a;
  const uint32_t bytes = (uint32_t)(p.rows * 2) * p.ngroups;  // a multiple of 16: p.rows is one of 8
  if (p.prefetch_scales && (lane == 0 || lane == 1) && (tile + 1) * p.rows <= a.V &&
      in_bounds(a.status, tile * bytes + bytes - 1, (int64_t)a.V * p.ngroups * 2))
    l2_prefetch(reinterpret_cast<const uint8_t*>(lane == 0 ? a.scales : a.biases) + tile * bytes, bytes);
}

// One of the four warps that bring scales and biases beside the segments of q: rows row0 + lane of the tile.
template <int kSegK>
struct ScaleRole {
  const TcArgs& p;
  TcCtl* ctl;
  uint32_t sring;
  int my_tiles, row0, lane;

  // W: words per segment, a group each, or 0: any number, groups repeated; kWide: loaded as one vector, else from any
  // address (24 rows, d 3232, V 96333, 101 groups a row: 56 us; element by element 69)
  template <int W, bool kWide>
  __device__ __forceinline__ void run() const {
    constexpr bool kShift = W > 1 && !kWide;
    constexpr int kWords = W ? W : kSegK / 32, kPairs = (kWords + 1) / 2, kRaw = kShift ? Shifted<W < 2 ? 2 : W>::kWords : kPairs;
    const LogitsArgs& a = p.a;
    struct Set {
      uint32_t sc[kRaw], bi[kRaw];  // the groups of the segment, in pairs, or what holds them
      uint32_t shift;               // kShift: bytes that they start after their word
    };
    // the next fetch: its segment, its tile's row that is mine, and where the row's scales and biases are
    int seg = 0;
    int64_t row = (int64_t)blockIdx.x * p.rows + row0 + lane, ahead = (int64_t)blockIdx.x + gridDim.x;
    const uint16_t *s, *b;
    // Scales are fetched two segments ahead, which covers the way from L2 and not from memory.  (Four ahead spilled.)
    auto enter_tile = [&]() {
      s = a.scales + row * p.ngroups;
      b = a.biases + row * p.ngroups;
      if (row0 == 0) prefetch_scales(p, ahead, lane);
      ahead += gridDim.x;
    };
    auto fetch = [&](Set& x) {
#pragma unroll
      for (int i = 0; i < kRaw; ++i) x.sc[i] = x.bi[i] = 0;
      x.shift = 0;
      const int g0 = W ? seg * W : (int)group_of(p, (uint32_t)(seg * p.seg_words));
      const uint16_t *sr = s + g0, *br = b + g0;
      const int64_t at = row * p.ngroups + g0, size = (int64_t)a.V * p.ngroups;
      if (row < a.V && in_bounds(a.status, at, size)) {
        if constexpr (kShift) {
          // (the row's first group + g0 + W, and the slack of a shifted load, stay inside the arrays)
          if (p.prefetch_scales && at + W + 4 <= size && Shifted<W>::inside(a.scales, at, size, a.status) &&
              Shifted<W>::inside(a.biases, at, size, a.status)) {
            x.shift = (uint32_t)reinterpret_cast<uintptr_t>(sr) & (Shifted<W>::kWord - 1);  // both arrays start on 16 bytes
            Shifted<W>::load(sr, x.sc);
            Shifted<W>::load(br, x.bi);
          } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (g0 + i < p.ngroups && in_bounds(a.status, at + i, size)) {
                x.sc[i / 2] |= (uint32_t)__ldg(sr + i) << (16 * (i & 1));
                x.bi[i / 2] |= (uint32_t)__ldg(br + i) << (16 * (i & 1));
              }
          }
        } else if (W && !in_bounds(a.status, at + W - 1, size)) {
        } else if constexpr (W == 8) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(sr)), v = __ldg(reinterpret_cast<const uint4*>(br));
          x.sc[0] = u.x, x.sc[1] = u.y, x.sc[2] = u.z, x.sc[3] = u.w;
          x.bi[0] = v.x, x.bi[1] = v.y, x.bi[2] = v.z, x.bi[3] = v.w;
        } else if constexpr (W == 4) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(sr)), v = __ldg(reinterpret_cast<const uint2*>(br));
          x.sc[0] = u.x, x.sc[1] = u.y, x.bi[0] = v.x, x.bi[1] = v.y;
        } else if constexpr (W == 2) {
          x.sc[0] = __ldg(reinterpret_cast<const uint32_t*>(sr)), x.bi[0] = __ldg(reinterpret_cast<const uint32_t*>(br));
        } else if constexpr (W == 1) {
          x.sc[0] = __ldg(sr), x.bi[0] = __ldg(br);
        } else {
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int gi = (int)group_of(p, (uint32_t)(seg * p.seg_words + i)) - g0;
            if (i < p.seg_words && g0 + gi < p.ngroups && in_bounds(a.status, at + gi, size)) {
              x.sc[i / 2] |= (uint32_t)__ldg(sr + gi) << (16 * (i & 1));
              x.bi[i / 2] |= (uint32_t)__ldg(br + gi) << (16 * (i & 1));
            }
          }
        }
      }
      if (++seg == p.segs) {
        seg = 0, row += (int64_t)gridDim.x * p.rows;
        enter_tile();
      }
    };
    uint32_t stage = 0, ph = 0;
    int at = 0;  // the segment to put
    auto put = [&](const Set& x) {
      if (!wait_warp(ctl, &ctl->w_empty[stage], ph ^ 1u, a.status)) return false;
      const uint32_t out = sring + stage * scale_bytes(1024 / kSegK) + (row0 + lane) * 4;
      if (!in_bounds(a.status, stage, p.stages) || !in_bounds(a.status, p.seg_words - 1, kSegK / 32)) return false;
      uint32_t sc[kPairs], bi[kPairs];
      if constexpr (kShift) {
        Shifted<W>::take(x.sc, x.shift, sc);
        Shifted<W>::take(x.bi, x.shift, bi);
        if (++at == p.segs) {
          const int own = p.ngroups - (p.segs - 1) * W;  // groups of the row's last segment; then come the next row's
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (i >= own) sc[i / 2] &= i & 1 ? 0xffffu : 0u, bi[i / 2] &= i & 1 ? 0xffffu : 0u;
          at = 0;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sc[i] = x.sc[i], bi[i] = x.bi[i];
      }
      uint32_t big[kPairs], odd = 0;  // times 2^133; odd: NaN where one is infinite or NaN, else 0
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        big[i] = bf16x2_mul(bf16x2_mul(sc[i], 0x7F007F00u), 0x42804280u);  // 2^127, 2^6
        odd = bf16x2_fma(big[i], 0u, odd);
      }
      const bool plain = __any_sync(0xffffffffu, (odd & 0x7fff7fffu) != 0);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const uint32_t v = plain ? sc[i] : big[i];
        if (W || 2 * i < p.seg_words) sts32(out + 2 * i * (kTileRows * 4), __byte_perm(v, bi[i], 0x5410));
        if (W > 1 || (W == 0 && 2 * i + 1 < p.seg_words))
          sts32(out + (2 * i + 1) * (kTileRows * 4), __byte_perm(v, bi[i], 0x7632));
      }
      if (lane == 0) ctl->plain[stage][row0 / 32] = plain;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->w_full[stage]);
      if (++stage == (uint32_t)p.stages) stage = 0, ph ^= 1u;
      return true;
    };
    const int64_t total = (int64_t)my_tiles * p.segs;
    enter_tile();
    Set x, y;
    if (total > 0) fetch(x);
    if (total > 1) fetch(y);
    for (int64_t left = total; left > 0; left -= 2) {
      if (!put(x)) break;
      if (left > 2) fetch(x);
      if (left == 1 || !put(y)) break;
      if (left > 3) fetch(y);
    }
  }
};

// 64 weights of a row into 32 words of A; sw: (scale, bias) of each 32.
template <int kBits, bool kScaled>
__device__ __forceinline__ void dequant_part(const uint4 (&x)[kBits / 2], const uint32_t (&sw)[2], uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t s2 = __byte_perm(sw[j], 0, 0x1010), b2 = __byte_perm(sw[j], 0, 0x3232);
    if constexpr (kBits == 4) {
      const uint32_t s129 = bf16x2_fma(s2, 0x3D803D80u, 0x80008000u);  // times 2^-4, plus -0
      unpack(x[j], [&](int e, uint32_t v) {
        uint32_t y[4];
        if constexpr (kScaled)
          dequant4_scaled(v, s2, s129, b2, y);
        else
          dequant4(v, s2, b2, y);
#pragma unroll
        for (int f = 0; f < 4; ++f) r[16 * j + 4 * e + f] = y[f];
      });
    } else {
#pragma unroll
      for (int o = 0; o < 2; ++o)
        unpack(x[2 * j + o], [&](int e, uint32_t v) {
          uint32_t y[2];
          if constexpr (kScaled)
            dequant8_scaled(v, s2, b2, y);
          else
            dequant8(v, s2, b2, y);
          r[16 * j + 8 * o + 2 * e] = y[0], r[16 * j + 8 * o + 2 * e + 1] = y[1];
        });
    }
  }
}

// Warps that sum: four per 32 columns of the accumulator at most
constexpr int sum_groups(int np) { return np > 32 ? np / 32 : 1; }
constexpr int first_dequant_warp(int np) { return kSumWarp + 4 * sum_groups(np); }
constexpr int tc_threads(int np) { return 32 * (first_dequant_warp(np) + 4 * kGroups); }

template <int kBits, int NP, bool kStream>
__global__ void __launch_bounds__(tc_threads(NP), 1)
    logits_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ TcArgs p) {
  constexpr int kSegK = seg_k(kBits), kUnits = kSegK / kUnitK, kASlots = a_slots(kBits), kScaleBytes = scale_bytes(kBits);
  constexpr uint32_t kHUnit = NP * kUnitK * 2, kHSeg = kUnits * kHUnit;  // bytes of a unit (two blocks of 64 columns) and a segment of h
  constexpr int kAccSegs = kAccK / kSegK;           // segments per set of accumulators
  // A parity wait is sound only for a waiter that sees every phase of its barrier, so no slot of a ring changes
  // hands: the slots of A and the stages of weights are multiples of the groups that take turns on them.
  constexpr int kLoadWarps = 4 * (sum_groups(NP) + kGroups);
  constexpr int kSums = sum_groups(NP), kCols = NP / kSums, kFirstDequantWarp = first_dequant_warp(NP);
  static_assert(2 * NP <= kTmemA && kTmemA + kTmemACols <= 512 && kASlots % kGroups == 0, "tensor memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const LogitsArgs& a = p.a;
  uint8_t* const ring = smem;
  uint8_t* const hbuf = ring + p.stages * kBoxBytes;
  uint8_t* const sring = hbuf + (kStream ? p.hslots : p.segs) * kHSeg;  // scale words, by ring stage
  TcCtl* const ctl = reinterpret_cast<TcCtl*>(sring + p.stages * kScaleBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = blockIdx.y * NP;

  // Tiles blockIdx.x, blockIdx.x + gridDim.x, ...
  const int my_tiles = (p.tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  // Resident h, by the warps that sum and dequantise, a thread always the same 16-byte pieces; rows past M stay as
  // they are, which their own columns of the accumulators get to see and nobody else.  Asked for before any weights:
  // behind them it came 5000 clocks later, and no product starts without it.
  auto each_piece = [&](auto f) {  // f(address in shared memory, row, piece of the row)
    const int live = min(NP, a.M - m0), per_row = p.units * (kUnitK / 8);
    const int w = warp - kSumWarp, split = max(1, kLoadWarps / live);  // warps to a row, or rows to a warp
    const int part = live < kLoadWarps ? w / live : 0;
    if (part >= split) return;
    for (int m = live < kLoadWarps ? w % live : w; m < live; m += kLoadWarps)
      for (int k = part * 32 + lane; k < per_row; k += split * 32)
        f(smem_u32(hbuf) + (k >> 3) * (NP * 128) + m * 128 + (((k ^ m) & 7) << 4), m, k);
  };
  grid_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&ctl->w_full[i], 1 + 4), mbar_init(&ctl->w_empty[i], 4);
    for (int i = 0; i < kASlots; ++i) mbar_init(&ctl->a_full[i], 4), mbar_init(&ctl->a_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->d_full[i], 1), mbar_init(&ctl->d_empty[i], 4 * kSums);
    for (int i = 0; i < kMaxH; ++i) mbar_init(&ctl->h_full[i], 1), mbar_init(&ctl->h_empty[i], 1);
    mbar_init(&ctl->h_ready, kLoadWarps);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<1>(&ctl->tmem_base, 512);
    tmem_relinquish<1>();
  }
  if constexpr (!kStream) {
    grid_wait();  // set up; from here on memory is read (streamed: h's image waits, and this kernel for that one)
    if (warp >= kSumWarp)
      each_piece([&](uint32_t at, int m, int k) {
        if (!in_bounds(a.status, at + 15 - smem_u32(hbuf), p.segs * kHSeg)) return;
        if (8 * k < a.d && in_bounds(a.status, (int64_t)(m0 + m) * a.ld_h + 8 * k + 7, h_size(a)))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(a.h + (int64_t)(m0 + m) * a.ld_h + 8 * k)
                       : "memory");
        else
          st_shared_v4(at, 0u, 0u, 0u, 0u);
      });
  }
  prefetch_scales(p, blockIdx.x, threadIdx.x - 32);  // the same goes for the first tile's scales
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if constexpr (!kStream) {
    if (warp >= kSumWarp) {  // resident h is here: into the dequantised order
      asm volatile("cp.async.wait_all;" ::: "memory");
      each_piece([&](uint32_t at, int, int) {
        if (!in_bounds(a.status, at + 15 - smem_u32(hbuf), p.segs * kHSeg)) return;
        const uint4 x = reorder_pairs<kBits>(lds128(at));
        st_shared_v4(at, x.x, x.y, x.z, x.w);
      });
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->h_ready);
    }
  }
  if (warp == 0) {
    // ---- TMA: the whole warp walks the loop and one elected lane issues, as below
    const bool leader = elect_one();
    uint32_t it = 0;          // segments issued
    uint32_t st = 0, ph = 1;  // weight ring: stage, parity of its release
    bool ok = true;
    int row0 = blockIdx.x * p.rows;
    for (int i = 0; ok && i < my_tiles; ++i, row0 += gridDim.x * p.rows) {
      for (int seg = 0; seg < p.segs; ++seg) {
        ok = in_bounds(a.status, st, p.stages) && wait_warp(ctl, &ctl->w_empty[st], ph, a.status);
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(&ctl->w_full[st], 128 * p.rows);
          tma_load_2d(&map_w, smem_u32(&ctl->w_full[st]), ring + st * kBoxBytes, seg * 128, row0);
        }
        ++it;
        if (++st == (uint32_t)p.stages) st = 0, ph ^= 1u;
      }
    }
    if (!ok && leader) {  // let the loads in flight land before the CTA can exit
      const uint32_t k0 = it > (uint32_t)p.stages ? it - p.stages : 0;
      for (uint32_t k = k0; k < it; ++k) drain_bar(&ctl->w_full[k % p.stages], (k / p.stages) & 1u);
    }
  } else if (warp == kHWarp) {
    // ---- streamed h
    if constexpr (kStream) {
      const bool leader = elect_one();
      grid_wait();  // the kernel that writes the image is done
      const uint8_t* const image = p.image + (int64_t)blockIdx.y * p.segs * kHSeg;
      uint32_t it = 0, hs = 0, hp = 1;  // segments issued; slot, parity of its release
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const uint8_t* src = image;
        for (int seg = 0; seg < p.segs; ++seg, ++it, src += kHSeg) {
          ok = in_bounds(a.status, hs, p.hslots) && in_bounds(a.status, src + kHSeg - 1 - p.image, p.image_bytes) &&
               wait_warp(ctl, &ctl->h_empty[hs], hp, a.status);
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(&ctl->h_full[hs], kHSeg);
            bulk_load(src, kHSeg, hbuf + hs * kHSeg, &ctl->h_full[hs]);
          }
          if (++hs == (uint32_t)p.hslots) hs = 0, hp ^= 1u;
        }
      }
      if (!ok && leader) {  // loads in flight
        const uint32_t k0 = it > (uint32_t)p.hslots ? it - p.hslots : 0;
        for (uint32_t k = k0; k < it; ++k) drain_bar(&ctl->h_full[k % p.hslots], (k / p.hslots) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---- MMA.  The whole warp walks the loop, so that addresses and descriptors stay in uniform registers, and
    // one elected lane issues: with a single thread in the loop a product took 109 clocks to issue.
    const bool leader = elect_one();
    const uint32_t idesc = make_idesc_bf16(kTileRows, NP, 0, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t desc0 = smem_desc_sw128(smem_u32(hbuf), 16, 1024);
    uint32_t slot = 0, ap = 0;  // segment's place in tensor memory, parity
    uint32_t db = 0, dp = 1;    // set of accumulators, parity of its release
    uint32_t hs = 0, hp = 0;    // streamed h: ring slot and parity
    bool ok = kStream || wait_warp(ctl, &ctl->h_ready, 0, a.status);
    for (int i = 0; ok && i < my_tiles; ++i) {
      int j = 0;  // segments in the accumulators
      for (int seg = 0; seg < p.segs; ++seg) {
        // all the waits polled at once: one after the other, each costs its 90 clocks even when there is nothing to
        // wait for
        bool ready = poll_bar(&ctl->a_full[slot], ap);
        if (j == 0) ready = poll_bar(&ctl->d_empty[db], dp) && ready;
        if constexpr (kStream) ready = poll_bar(&ctl->h_full[hs], hp) && ready;
        if (!__all_sync(0xffffffffu, ready)) {
          if (j == 0) ok = wait_warp(ctl, &ctl->d_empty[db], dp, a.status);
          ok = ok && wait_warp(ctl, &ctl->a_full[slot], ap, a.status);
          if constexpr (kStream) ok = ok && wait_warp(ctl, &ctl->h_full[hs], hp, a.status);
        }
        ok = ok && in_bounds(a.status, slot, kASlots) && in_bounds(a.status, kStream ? hs : seg, kStream ? p.hslots : p.segs);
        if (!ok) break;
        tc_fence_after();
        const bool last = j == kAccSegs - 1 || seg + 1 == p.segs;
        if (leader) {
          const uint64_t desc = desc0 + (uint64_t)((kStream ? hs : (uint32_t)seg) * (kHSeg >> 4));
          const uint32_t at = tm + kTmemA + slot * (kSegK / 2), dt = tm + db * NP;
#pragma unroll
          for (int kk = 0; kk < kSegK / 16; ++kk)
            umma_bf16_ta(dt, at + kk * 8, desc + ((kk >> 2) * (kHUnit / 2) + (kk & 3) * 32) / 16, idesc,
                         (kk | j) != 0 ? 1u : 0u);
          umma_commit(&ctl->a_empty[slot]);
          if constexpr (kStream) umma_commit(&ctl->h_empty[hs]);
          if (last) umma_commit(&ctl->d_full[db]);
        }
        __syncwarp();
        ++j;
        if (last) {
          j = 0;
          db ^= 1u;
          dp ^= db ^ 1u;  // after both sets
        }
        if (++slot == kASlots) slot = 0, ap ^= 1u;
        if constexpr (kStream)
          if (++hs == (uint32_t)p.hslots) hs = 0, hp ^= 1u;
      }
    }
    if (leader) {  // every issued MMA has finished before tensor memory is released
      umma_commit(&ctl->drain);
      drain_bar(&ctl->drain, 0);
    }
  } else if (warp == 3) {
    // ---- nothing to do
  } else if (warp < kSumWarp) {
    // ---- scales and biases
    const ScaleRole<kSegK> role{p, ctl, smem_u32(sring), my_tiles, (warp - kScaleWarp) * 32, lane};
    if (!p.word_groups)
      role.template run<0, false>();
    else if (kBits == 4 && p.seg_words == 8)
      p.wide_scales ? role.template run<kSegK / 32, true>() : role.template run<kSegK / 32, false>();
    else if (p.seg_words == 4)
      p.wide_scales ? role.template run<4, true>() : role.template run<4, false>();
    else if (p.seg_words == 2)
      p.wide_scales ? role.template run<2, true>() : role.template run<2, false>();
    else
      role.template run<1, true>();
  } else if (warp < kFirstDequantWarp) {
    // ---- sums and output
    const int q = warp & 3, n0 = (warp - kSumWarp) / 4 * kCols;
    bool ok = true;
    float acc[kCols];  // columns n0 on
    const float inv_cap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;
    const int chunks = (p.segs + kAccSegs - 1) / kAccSegs;
    uint32_t db = 0, dp = 0;  // set and parity
    for (int i = 0; ok && i < my_tiles; ++i) {
#pragma unroll
      for (int n = 0; n < kCols; ++n) acc[n] = 0.f;
      for (int c = 0; c < chunks; ++c) {
        ok = wait_warp(ctl, &ctl->d_full[db], dp, a.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int n = 0; n < kCols; n += 16) {
          uint32_t r[16];
          tmem_ld16(tmem + db * NP + n0 + n + ((uint32_t)(32 * q) << 16), r);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[n + e] += __uint_as_float(r[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->d_empty[db]);
        db ^= 1u;
        dp ^= db ^ 1u;
      }
      if (!ok) break;
      const int row = 32 * q + lane;
      const int64_t v = (int64_t)(blockIdx.x + i * gridDim.x) * p.rows + row;
      if (row < p.rows && v < a.V) {
        const int64_t at = (int64_t)(m0 + n0) * a.ld_out + v;
        float* f32 = static_cast<float*>(a.out) + at;
        uint16_t* b16 = static_cast<uint16_t*>(a.out) + at;
        const int n_live = a.M - m0 - n0;
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          if (n >= n_live || !in_bounds(a.status, at + n * a.ld_out, out_size(a))) break;
          float x = acc[n];
          if (a.softcap > 0.f) x = softcap_of(x, a.softcap, inv_cap);
          if (a.out_bf16) {
            *b16 = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
            b16 += a.ld_out;
          } else {
            *f32 = x;
            f32 += a.ld_out;
          }
        }
      }
    }
  } else {
    // ---- dequantisation
    const int wg = (warp - kFirstDequantWarp) >> 2, q = warp & 3, row = 32 * q + lane;
    // segments wg, wg + kGroups, ...
    constexpr int kParts = kSegK / 64, kVec = 8 / kParts;  // pieces of 64 columns, their 16-byte vectors
    const uint32_t swz = (uint32_t)(row & 7) << 4;
    const uint32_t wrow = smem_u32(ring) + row * 128, srow = smem_u32(sring) + row * 4;
    const uint32_t trow = tmem + kTmemA + ((uint32_t)(32 * q) << 16);
    uint32_t stage = wg, wph = 0;  // weight ring
    uint32_t slot = wg, aph = 0;   // place in tensor memory
    bool ok = true;
    for (int64_t left = (int64_t)my_tiles * p.segs - wg; left > 0; left -= kGroups) {
      ok = in_bounds(a.status, stage, p.stages) && in_bounds(a.status, slot, kASlots) &&
           in_bounds(a.status, (kSegK / 32 - 1) >> p.shift, kSegK / 32) && wait_warp(ctl, &ctl->w_full[stage], wph, a.status);
      if (!ok) break;
      const uint32_t wst = wrow + stage * kBoxBytes, sst = srow + stage * kScaleBytes;
      const bool plain = (lds32(smem_u32(ctl->plain[stage])) >> (8 * q) & 1u) != 0;
      const uint32_t dst = trow + slot * (kSegK / 2);
      // The stage is given back behind the tensor-memory stores that take what the weights became: a release right
      // behind the loads does not hold them back, and the next box landed first.
      auto load = [&](int part, uint4 (&x)[kVec], uint32_t (&y)[2]) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = lds128(wst + (((part * kVec + i) << 4) ^ swz));
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = lds32(sst + ((part * 2 + i) >> p.shift) * (kTileRows * 4));
      };
      auto store = [&](int part, const uint32_t (&r)[32]) {
        if (part == 0) {
          ok = wait_warp(ctl, &ctl->a_empty[slot], aph ^ 1u, a.status);
          if (!ok) return;
          tc_fence_after();
        }
        tmem_st(dst + part * 32, r);
      };
      if (__builtin_expect(!plain, 1)) {
        uint4 w[2][kVec];  // this piece and the next
        uint32_t sw[2][2];
        load(0, w[0], sw[0]);
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (part + 1 < kParts) load(part + 1, w[(part + 1) & 1], sw[(part + 1) & 1]);
          uint32_t r[32];
          dequant_part<kBits, true>(w[part & 1], sw[part & 1], r);
          store(part, r);
          if (!ok) break;
        }
      } else {  // apart and rolled up: inside the loop above it cost 10 of 78 us
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          uint4 w[kVec];
          uint32_t sw[2], r[32];
          load(part, w, sw);
          dequant_part<kBits, false>(w, sw, r);
          store(part, r);
          if (!ok) break;
        }
      }
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->w_empty[stage]);
        mbar_arrive(&ctl->a_full[slot]);
      }
      slot += kGroups;
      if (slot >= kASlots) slot -= kASlots, aph ^= 1u;
      stage += kGroups;
      if (stage >= (uint32_t)p.stages) stage -= p.stages, wph ^= 1u;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

// h for the streamed form: per m tile of `rows` rows and block of 64 columns the block as shared memory holds it
// (128-byte swizzled rows), 16-byte pieces in the dequantised order, zero where h has no element.
template <int kBits>
__global__ void __launch_bounds__(256) h_image_kernel(LogitsArgs a, int rows, int blocks, int64_t pieces, uint4* image, int64_t size) {
  // set up while the kernel before it in the stream ends; the products' kernel may be set up once that one has
  grid_wait();
  grid_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int row = (int)(i / 8 % rows);
  const int64_t blk = i / 8 / rows % blocks, m = i / 8 / rows / blocks * rows + row;
  const int64_t k = blk * 64 + (int)((i ^ row) & 7) * 8;
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  if (m < a.M && k < a.d && in_bounds(a.status, m * a.ld_h + k + 7, h_size(a))) x = reorder_pairs<kBits>(__ldg(reinterpret_cast<const uint4*>(a.h + m * a.ld_h + k)));
  if (in_bounds(a.status, i, size)) image[i] = x;
}

constexpr int kMinStages = 6;  // of weights, beside resident or streamed h
constexpr int stage_bytes(int bits) { return kBoxBytes + scale_bytes(bits); }
int64_t units_of(int64_t d, int bits) { return cdiv(d, seg_k(bits)) * (seg_k(bits) / kUnitK); }
int rows_per_pass(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }
// A pass's rows, beside at least kMinStages of weights.  (With three stages beside them, 13 rows of d 3840 took
// 36.4 us resident and 34.7 streamed; 42 rows of d 768, V 48710, which fit beside six: 13.1 resident, 16.6 streamed.)
bool resident(int bits, int64_t M, int64_t d) {
  return units_of(d, bits) * (rows_per_pass(M) * kUnitK * 2) <= kSmemLimit - kCtlBytes - kMinStages * stage_bytes(bits);
}

template <int kBits, int NP, bool kStream>
cudaError_t launch_np(const LogitsArgs& a, int sms, void* workspace, cudaStream_t st) {
  constexpr int kHUnit = NP * kUnitK * 2, kSegK = seg_k(kBits), kUnits = kSegK / kUnitK;
  TcArgs p;
  p.a = a;
  const int64_t row_bytes = (int64_t)a.d * kBits / 8;
  // Tiles of as many rows as deal the vocabulary out evenly in the fewest rounds of 128 rows: with 128 in every
  // one, V = 32000 on 152 SMs takes two rounds of which the second is 64% full.  A multiple of 8, so that a
  // tile's scales start on 16 bytes.
  const int64_t rounds = cdiv(a.V, (int64_t)kTileRows * sms);
  p.rows = (int)std::min<int64_t>(kTileRows, cdiv(cdiv(a.V, rounds * sms), 8) * 8);
  p.tiles = (int)cdiv(a.V, p.rows);
  p.segs = (int)cdiv(a.d, kSegK);
  p.units = p.segs * kUnits;
  p.ngroups = a.d / a.group;
  // A scale word per group where groups of a power of two columns fit a segment; else one per 32 columns
  // (or per segment, for groups of whole segments), the group's repeated.
  const int per = a.group / 32;
  p.shift = 0;
  if (a.group % kSegK == 0)
    while (32 << p.shift < kSegK) ++p.shift;
  else if ((per & (per - 1)) == 0)
    while (1 << p.shift < per) ++p.shift;
  p.seg_words = (kSegK / 32) >> p.shift;
  const uint32_t repeat = (uint32_t)(per >> p.shift);  // words per group
  p.gmul = repeat > 1 ? (uint32_t)(((1ull << 32) + repeat - 1) / repeat) : 0u;
  p.word_groups = repeat == 1;
  p.prefetch_scales = aligned16(a.scales) && aligned16(a.biases);
  p.wide_scales = p.word_groups && p.ngroups % p.seg_words == 0 && p.prefetch_scales;
  static_assert(kMaxStages % kGroups == 0 && kMinStages % kGroups == 0, "weight ring");
  const int fixed = kCtlBytes, stage = stage_bytes(kBits);
  p.hslots = kStream ? std::min(kMaxH, (kSmemLimit - fixed - kMinStages * stage) / (kUnits * kHUnit)) : 0;
  const int h_bytes = (kStream ? p.hslots : p.segs) * kUnits * kHUnit;
  p.stages = std::min(kMaxStages, (kSmemLimit - fixed - h_bytes) / stage) / kGroups * kGroups;
  p.image = static_cast<const uint8_t*>(workspace);
  p.image_bytes = kStream ? (int64_t)logits_tc_workspace(kBits, a.M, a.d) : 0;
  const int smem = p.stages * stage + h_bytes + fixed + 1024;
  CUtensorMap mw;
  if (!encode_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq, row_bytes, a.V, row_bytes, 128, p.rows)) return cudaErrorNotSupported;
  static std::atomic<int> done[64];
  auto kernel = logits_tc_kernel<kBits, NP, kStream>;
  if (cudaError_t e = opt_in_smem(kernel, kSmemLimit + 1024, done)) return e;
  const int mt = (int)cdiv(a.M, NP);
  if constexpr (kStream) {
    const int blocks = p.units * 2;
    const int64_t pieces = (int64_t)mt * blocks * NP * 8;
    if (cudaError_t e = launch_dependent(h_image_kernel<kBits>, dim3((unsigned)cdiv(pieces, 256)), 256, 0, st, a, NP, blocks,
                                         pieces, static_cast<uint4*>(workspace), p.image_bytes / 16))
      return e;
  }
  return launch_dependent(kernel, dim3((unsigned)std::min(p.tiles, sms), (unsigned)mt), tc_threads(NP), (size_t)smem, st, mw, p);
}

template <int kBits>
cudaError_t launch_bits(const LogitsArgs& a, int sms, void* workspace, cudaStream_t st) {
  const bool whole = resident(kBits, a.M, a.d);
  switch (rows_per_pass(a.M)) {
    case 16: return whole ? launch_np<kBits, 16, false>(a, sms, workspace, st) : launch_np<kBits, 16, true>(a, sms, workspace, st);
    case 32: return whole ? launch_np<kBits, 32, false>(a, sms, workspace, st) : launch_np<kBits, 32, true>(a, sms, workspace, st);
    default: return whole ? launch_np<kBits, 64, false>(a, sms, workspace, st) : launch_np<kBits, 64, true>(a, sms, workspace, st);
  }
}

}  // namespace

size_t logits_tc_workspace(int bits, int64_t M, int64_t d) {
  if (resident(bits, M, d)) return 0;
  const int rows = rows_per_pass(M);
  return (size_t)(cdiv(M, rows) * rows * units_of(d, bits) * kUnitK * 2);
}

cudaError_t launch_logits_tc(const LogitsArgs& a, int bits, int sms, void* workspace, cudaStream_t st) {
  return bits == 4 ? launch_bits<4>(a, sms, workspace, st) : launch_bits<8>(a, sms, workspace, st);
}

}  // namespace orpo
