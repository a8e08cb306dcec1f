// decode_logits.cu — logits of a few rows under the quantised head (orpo_head_logits_q).
//
//   z[m, v] = sum_j h[m, j] W[v, j],  W[v, j] = bf16(scale q + bias),  logits = softcap(z)
//
// Every weight is used for M rows only, so the call is bound by reading the quantised weights once.
//
// Generic kernel: a warp owns one vocabulary row and a tile of 8 rows of h.  Lane l takes the
// 8-weight slices l, l + 32, ... of the row (one 4- or 8-byte word of q, one scale and bias: a group
// is a multiple of 8 columns), so any d that is a multiple of 8 works; the lanes' fp32 sums are
// added in a fixed shuffle order.
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "decode_logits.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr int kRowsTile = 8;

// ---------------------------------------------------------------- streaming kernel
//
// A warp multiplies 16 vocabulary rows with 8 NT rows of h by mma m16n8k16 (weights as A, h as B).
// The order of k inside a product is free as long as A and B agree, so a thread takes the 16 bytes
// that its quad's quarter of a 64-byte row segment holds, exactly as they lie in memory: 32 4-bit or
// 16 8-bit weights of row g and as many of row g + 8 (g = lane / 4).  h is laid out once per CTA in
// shared memory in the matching fragment order, so a fragment of B is one conflict-free 16-byte load.
// Weights go from global memory to registers, kStages segments ahead of their use (about 100 KB in
// flight per SM), and are used once: no shared memory, no barrier after the prologue.
// The partial sum of a segment starts from zero and is added to the running sum in fp32, so the
// matrix unit's truncating adds span at most 128 products.
constexpr int kStreamWarps = 16;
constexpr int kStreamThreads = 32 * kStreamWarps;
constexpr int kSegBytes = 64;  // bytes of a row per segment: 128 4-bit or 64 8-bit weights

struct StreamArgs {
  LogitsArgs a;
  int row_bytes;   // d * bits / 8
  int segs;        // segments per row
  int panel_segs;  // segments of h that fit in shared memory (segs: the whole row)
  int ngroups;     // d / group
  uint32_t gmul;   // ceil(2^31 / (group / weights per thread and segment))
  int tiles;       // ceil(V / 16)
};

struct Stage {
  uint4 w0, w1;             // 16 bytes of rows g and g + 8
  uint16_t s0, b0, s1, b1;  // their scales and biases
};

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int kBits, int NT, int kStages>
__global__ void __launch_bounds__(kStreamThreads, 1) logits_stream_kernel(StreamArgs p) {
  constexpr int kFrags = kBits == 4 ? 4 : 2;           // 16-byte B fragments per segment and 8 rows of h
  constexpr int kPerThread = kBits == 4 ? 32 : 16;     // weights of a row per thread and segment
  constexpr int kSegK = 4 * kPerThread;                // weights of a row per segment
  extern __shared__ __align__(16) uint4 hs[];          // [panel_segs][kFrags][NT][32]
  const LogitsArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.y * (8 * NT);
  const int first = warp * gridDim.x + blockIdx.x, step = kStreamWarps * gridDim.x;

  auto load = [&](Stage& st, int tile, int seg) {
    const int64_t r0 = min((int64_t)tile * 16 + g, (int64_t)a.V - 1), r1 = min((int64_t)tile * 16 + g + 8, (int64_t)a.V - 1);
    const int off = seg * kSegBytes + t * 16;
    st.w0 = st.w1 = make_uint4(0u, 0u, 0u, 0u);
    st.s0 = st.b0 = st.s1 = st.b1 = 0;
    if (off < p.row_bytes) {
      st.w0 = ldg_stream(a.wq + r0 * p.row_bytes + off);
      st.w1 = ldg_stream(a.wq + r1 * p.row_bytes + off);
      const int gi = (int)(((uint64_t)(uint32_t)(seg * 4 + t) * p.gmul) >> 31);
      st.s0 = __ldg(a.scales + r0 * p.ngroups + gi);
      st.b0 = __ldg(a.biases + r0 * p.ngroups + gi);
      st.s1 = __ldg(a.scales + r1 * p.ngroups + gi);
      st.b1 = __ldg(a.biases + r1 * p.ngroups + gi);
    }
  };

  auto fill = [&](int seg0, int nseg) {  // h, segments [seg0, seg0 + nseg), into fragment order
    const int n = nseg * kFrags * NT * 32;
    for (int i = threadIdx.x; i < n; i += kStreamThreads) {
      const int l = i & 31, nt = (i >> 5) % NT, j = (i >> 5) / NT % kFrags, s = (i >> 5) / NT / kFrags;
      const int m = m0 + nt * 8 + (l >> 2);
      const int k = (seg0 + s) * kSegK + (l & 3) * kPerThread + j * 8;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (m < a.M && k < a.d) x = __ldg(reinterpret_cast<const uint4*>(a.h + (int64_t)m * a.ld_h + k));
      uint4 f;
      if constexpr (kBits == 4)
        f = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                       __byte_perm(x.y, x.w, 0x7632));
      else
        f = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x5410),
                       __byte_perm(x.z, x.w, 0x7632));
      hs[i] = f;
    }
  };

  auto segment = [&](const Stage& st, int pseg, float (&acc)[NT][4]) {
    float c[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
    const uint32_t s0 = st.s0 * 0x10001u, b0 = st.b0 * 0x10001u, s1 = st.s1 * 0x10001u, b1 = st.b1 * 0x10001u;
    const uint32_t w0[4] = {st.w0.x, st.w0.y, st.w0.z, st.w0.w}, w1[4] = {st.w1.x, st.w1.y, st.w1.z, st.w1.w};
    const uint4* frag = hs + pseg * (kFrags * NT * 32) + lane;
#pragma unroll
    for (int j = 0; j < kFrags; ++j) {
      uint32_t x[4], y[4];  // rows g and g + 8: the pairs of two products
      if constexpr (kBits == 4) {
        dequant4(w0[j], s0, b0, x);
        dequant4(w1[j], s1, b1, y);
      } else {
        uint32_t u[2];
        dequant8(w0[2 * j], s0, b0, u), x[0] = u[0], x[1] = u[1];
        dequant8(w0[2 * j + 1], s0, b0, u), x[2] = u[0], x[3] = u[1];
        dequant8(w1[2 * j], s1, b1, u), y[0] = u[0], y[1] = u[1];
        dequant8(w1[2 * j + 1], s1, b1, u), y[2] = u[0], y[3] = u[1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 f = frag[(j * NT + nt) * 32];
        mma16816(c[nt], x[0], y[0], x[1], y[1], f.x, f.y);
        mma16816(c[nt], x[2], y[2], x[3], y[3], f.z, f.w);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] += c[nt][i];
  };

  auto finish = [&](int tile, float (&acc)[NT][4]) {
    const int v = tile * 16 + g;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + nt * 8 + 2 * t + (i & 1), vi = v + (i >> 1) * 8;
        if (m < a.M && vi < a.V) store_logit(a, m, vi, acc[nt][i]);
        acc[nt][i] = 0.f;
      }
  };

  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
  Stage st[kStages];

  if (p.panel_segs == p.segs) {  // all of h is resident: the warp's tiles are one stream of segments
    int lt = first, ls = 0;  // next segment to load
    auto advance = [&](Stage& s) {
      if (lt < p.tiles) load(s, lt, ls);
      if (++ls == p.segs) ls = 0, lt += step;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) advance(st[i]);
    fill(0, p.segs);
    __syncthreads();
    int tile = first, seg = 0;
    while (tile < p.tiles) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        if (tile < p.tiles) {
          segment(st[i], seg, acc);
          advance(st[i]);
          if (++seg == p.segs) {
            finish(tile, acc);
            seg = 0, tile += step;
          }
        }
      }
    }
    return;
  }
  // h in panels: every tile of the CTA passes over each panel, which is then replaced
  const int rounds = (p.tiles - (int)blockIdx.x + step - 1) / step;  // of warp 0, the most of any warp
  for (int r = 0; r < rounds; ++r) {
    const int tile = first + r * step;
    for (int s0 = 0; s0 < p.segs; s0 += p.panel_segs) {
      const int n = min(p.panel_segs, p.segs - s0);
      __syncthreads();
      fill(s0, n);
      __syncthreads();
      if (tile >= p.tiles) continue;
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        if (i < n) load(st[i], tile, s0 + i);
      for (int s = 0; s < n; s += kStages) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
          if (s + i < n) {
            segment(st[i], s + i, acc);
            if (s + i + kStages < n) load(st[i], tile, s0 + s + i + kStages);
          }
        }
      }
    }
    if (tile < p.tiles) finish(tile, acc);
  }
}

constexpr int kStreamSmem = 200 << 10;  // most shared memory for h

template <int kBits, int NT, int kStages>
cudaError_t launch_stream(const LogitsArgs& a, int sms, cudaStream_t st) {
  constexpr int kFrags = kBits == 4 ? 4 : 2, kPerThread = kBits == 4 ? 32 : 16;
  constexpr int kSegSmem = kFrags * NT * 32 * 16;
  static std::atomic<int> done[64];
  auto kernel = logits_stream_kernel<kBits, NT, kStages>;
  if (cudaError_t e = opt_in_smem(kernel, kStreamSmem, done)) return e;
  StreamArgs p;
  p.a = a;
  p.row_bytes = a.d * kBits / 8;
  p.segs = (int)cdiv(p.row_bytes, kSegBytes);
  p.panel_segs = std::min(p.segs, kStreamSmem / kSegSmem);
  p.ngroups = a.d / a.group;
  const uint32_t per = (uint32_t)(a.group / kPerThread);
  p.gmul = (uint32_t)(((1ull << 31) + per - 1) / per);
  p.tiles = (int)cdiv(a.V, 16);
  const dim3 grid((unsigned)std::min(p.tiles, sms), (unsigned)cdiv(a.M, 8 * NT));
  kernel<<<grid, kStreamThreads, p.panel_segs * kSegSmem, st>>>(p);
  return cudaGetLastError();
}

template <int kBits>
__global__ void __launch_bounds__(256) logits_generic_kernel(LogitsArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int m0 = blockIdx.y * kRowsTile;
  if (v >= a.V) return;
  const uint8_t* row = a.wq + v * ((int64_t)a.d * kBits / 8);
  const int64_t g0 = v * (a.d / a.group);
  float acc[kRowsTile] = {};
  for (int c = lane; c < a.d / 8; c += 32) {
    uint2 raw = make_uint2(0u, 0u);
    if constexpr (kBits == 4)
      raw.x = __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    else
      raw = __ldg(reinterpret_cast<const uint2*>(row) + c);
    const int64_t gi = g0 + (8 * c) / a.group;
    const float sc = dq_bf16_to_float(__ldg(a.scales + gi)), bi = dq_bf16_to_float(__ldg(a.biases + gi));
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t q = kBits == 4 ? (raw.x >> (4 * e)) & 15u : ((e < 4 ? raw.x : raw.y) >> (8 * (e & 3))) & 255u;
      w[e] = __uint_as_float(dq_pack2(0.f, fmaf(sc, (float)q, bi)) & 0xffff0000u);
    }
#pragma unroll
    for (int m = 0; m < kRowsTile; ++m) {
      if (m0 + m < a.M) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.h + (int64_t)(m0 + m) * a.ld_h) + c);
        const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[m] = fmaf(__uint_as_float(p[e] << 16), w[2 * e], acc[m]);
          acc[m] = fmaf(__uint_as_float(p[e] & 0xffff0000u), w[2 * e + 1], acc[m]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kRowsTile; ++m) {
    float s = acc[m];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == m && m0 + m < a.M) store_logit(a, m0 + m, (int)v, s);
  }
}

template <int kBits>
cudaError_t launch_stream_rows(const LogitsArgs& a, int sms, cudaStream_t st) {
  if (a.M <= 8) return launch_stream<kBits, 1, 5>(a, sms, st);
  if (a.M <= 16) return launch_stream<kBits, 2, 5>(a, sms, st);
  return launch_stream<kBits, 4, 4>(a, sms, st);
}

cudaError_t launch_generic(const LogitsArgs& a, int bits, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv(a.V, 8), (unsigned)cdiv(a.M, kRowsTile));
  if (bits == 4)
    logits_generic_kernel<4><<<grid, 256, 0, st>>>(a);
  else
    logits_generic_kernel<8><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace orpo

using namespace orpo;

extern "C" size_t orpo_head_logits_q_workspace_bytes(int64_t M, int64_t d, int bits) {
  if (M < 1 || M > kMaxRows || d < 8 || d >= (1 << 20) || (bits != 4 && bits != 8)) return 0;
  return logits_tc_workspace(bits, M, d);
}

extern "C" int orpo_head_logits_q(const void* h, int64_t ld_h, const uint8_t* wq, const void* scales,
                                  const void* biases, int bits, int group, int64_t M, int64_t V, int64_t d,
                                  float softcap, void* logits, int64_t ld_logits, int logits_bf16, void* workspace,
                                  size_t ws_bytes, int32_t* status, void* stream) {
  if (M < 0 || M > kMaxRows || V < 1 || V > kMaxRows || d < 8 || d >= (1 << 20)) return ORPO_ERR_SHAPE;
  if (M == 0) return ORPO_OK;
  if (ld_h < d || ld_logits < V || ld_h > (1ll << 40) || ld_logits > (1ll << 40)) return ORPO_ERR_SHAPE;
  if (!h || !logits || !status) return ORPO_ERR_NULL;
  const QuantW q{wq, scales, biases, bits, group};
  if (int e = check_quant(&q, d)) return e;
  const uintptr_t out_align = logits_bf16 ? 1 : 3;
  if (d % 8 != 0 || ld_h % 8 != 0 || !aligned16(h) || (reinterpret_cast<uintptr_t>(logits) & out_align))
    return ORPO_ERR_ALIGN;
  if (!isfinite(softcap)) return ORPO_ERR_ARG;
  if (const size_t need = logits_tc_workspace(bits, M, d)) {
    if (!workspace) return ORPO_ERR_NULL;
    if (!aligned16(workspace)) return ORPO_ERR_ALIGN;
    if (ws_bytes < need) return ORPO_ERR_WORKSPACE;
  }
  int sms = 0;
  if (int e = device_check(&sms)) return e;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LogitsArgs a{static_cast<const uint16_t*>(h), ld_h, wq, static_cast<const uint16_t*>(scales),
               static_cast<const uint16_t*>(biases), group, (int)M, (int)V, (int)d, softcap > 0.f ? softcap : 0.f,
               logits, ld_logits, logits_bf16 != 0, status};
  // The streaming kernel wants 16-byte pieces of a row that lie in one group.
  const int per_thread = bits == 4 ? 32 : 16;
  const bool streamed = d % per_thread == 0 && group % per_thread == 0 && aligned16(wq);
  const bool tensor = streamed && group % 32 == 0 && getenv("ORPO_LOGITS_STREAM") == nullptr;
  // rows of h in launches of at most 65535 tiles
  const int64_t chunk = 65535ll * kRowsTile;
  for (int64_t m = 0; m < M; m += chunk) {
    a.h = static_cast<const uint16_t*>(h) + m * ld_h;
    a.out = static_cast<uint8_t*>(logits) + m * ld_logits * (logits_bf16 ? 2 : 4);
    a.M = (int)std::min(chunk, M - m);
    prof_begin(K_LOGITS, st);
    const cudaError_t e = tensor     ? launch_logits_tc(a, bits, sms, workspace, st)
                          : streamed ? (bits == 4 ? launch_stream_rows<4>(a, sms, st) : launch_stream_rows<8>(a, sms, st))
                                   : launch_generic(a, bits, st);
    prof_end(K_LOGITS, st);
    if (e != cudaSuccess) return ORPO_ERR_CUDA;
  }
  return ORPO_OK;
}
