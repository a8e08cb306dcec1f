// decode_logits.cu — logits of a few rows under the quantised head (orpo_head_logits_q).
//
//   z[m, v] = sum_j h[m, j] W[v, j],  W[v, j] = bf16(scale q + bias),  logits = softcap(z)
//
// Every weight is used for M rows only, so the call is bound by reading the quantised weights once.
// Groups that are a multiple of 32 columns, at 16-byte aligned weights, take the tensor-core kernel
// (decode_logits_tc.cu); the kernel here takes the rest.
//
// Generic kernel: a warp owns one vocabulary row and a tile of 8 rows of h.  Lane l takes the
// 8-weight slices l, l + 32, ... of the row (one 4- or 8-byte word of q, one scale and bias: a group
// is a multiple of 8 columns), so any d that is a multiple of 8 works; the lanes' fp32 sums are
// added in a fixed shuffle order.  Bound by its instructions (dequantisation, loads of h,
// conversions, products): 0.66 ms for one row at d 2560, V 262144, 4 bits, where the tensor-core kernel takes
// 0.065 ms.
#include <math.h>

#include <algorithm>

#include "../../include/orpo_decode.h"
#include "decode_logits.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace orpo {
namespace {

constexpr int kRowsTile = 8;

template <int kBits>
__global__ void __launch_bounds__(256) logits_generic_kernel(LogitsArgs a) {
  grid_trigger();
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int m0 = blockIdx.y * kRowsTile;
  if (v >= a.V) return;
  const uint8_t* row = a.wq + v * ((int64_t)a.d * kBits / 8);
  const int64_t g0 = v * (a.d / a.group);
  float acc[kRowsTile] = {};
  for (int c = lane; c < a.d / 8; c += 32) {
    if (!in_bounds(a.status, v * (a.d / 8) + c, (int64_t)a.V * (a.d / 8))) break;
    uint2 raw = make_uint2(0u, 0u);
    if constexpr (kBits == 4)
      raw.x = __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    else
      raw = __ldg(reinterpret_cast<const uint2*>(row) + c);
    const int64_t gi = g0 + (8 * c) / a.group;
    if (!in_bounds(a.status, gi, scales_size(a))) break;
    // (scale, scale) and (bias, bias); product and sum round once, as in the tensor-core kernel
    const uint32_t s2 = __ldg(a.scales + gi) * 0x10001u, b2 = __ldg(a.biases + gi) * 0x10001u;
    float w[8];
    if constexpr (kBits == 4) {
      uint32_t p[4];  // (0, 4), (1, 5), (2, 6), (3, 7)
      dequant4(raw.x, s2, b2, p);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __uint_as_float(p[e] << 16), w[e + 4] = __uint_as_float(p[e] & 0xffff0000u);
    } else {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        uint32_t p[2];  // (0, 2), (1, 3)
        dequant8(o ? raw.y : raw.x, s2, b2, p);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[4 * o + e] = __uint_as_float(p[e] << 16), w[4 * o + e + 2] = __uint_as_float(p[e] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int m = 0; m < kRowsTile; ++m) {
      if (m0 + m < a.M && in_bounds(a.status, (int64_t)(m0 + m) * a.ld_h + 8 * c + 7, h_size(a))) {
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

cudaError_t launch_generic(const LogitsArgs& a, int bits, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv(a.V, 8), (unsigned)cdiv(a.M, kRowsTile));
  return launch_dependent(bits == 4 ? logits_generic_kernel<4> : logits_generic_kernel<8>, grid, 256, 0, st, a);
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
  // The tensor-core kernel wants 32 columns with one scale and rows of whole 16-byte pieces (d is a multiple of
  // the group).  It is the faster one at every size measured, from 14.5 -> 7 us for one row at d 256, V 4096.
  const bool tensor = group % 32 == 0 && aligned16(wq);
  // rows of h in launches of at most 65535 tiles
  const int64_t chunk = 65535ll * kRowsTile;
  for (int64_t m = 0; m < M; m += chunk) {
    a.h = static_cast<const uint16_t*>(h) + m * ld_h;
    a.out = static_cast<uint8_t*>(logits) + m * ld_logits * (logits_bf16 ? 2 : 4);
    a.M = (int)std::min(chunk, M - m);
    prof_begin(K_LOGITS, st);
    const cudaError_t e = tensor ? launch_logits_tc(a, bits, sms, workspace, st) : launch_generic(a, bits, st);
    prof_end(K_LOGITS, st);
    if (e != cudaSuccess) return ORPO_ERR_CUDA;
  }
  return ORPO_OK;
}
