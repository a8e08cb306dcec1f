// decode_logits.cuh — what the kernels of orpo_head_logits_q share: arguments, the softcap and store of
// one logit, and the dequantisation of packed weights into bf16 pairs.
#pragma once

#include <stdint.h>

#include "bounds.cuh"
#include "ptx.cuh"

namespace orpo {

struct LogitsArgs {
  const uint16_t* h;
  int64_t ld_h;
  const uint8_t* wq;
  const uint16_t* scales;
  const uint16_t* biases;
  int group;
  int M, V, d;
  float softcap;
  void* out;
  int64_t ld_out;
  int out_bf16;
  int32_t* status;
};

// Elements from the first to the last of h, of the logits, and values of scales or biases (for the bounds-checked build).
__device__ __forceinline__ int64_t h_size(const LogitsArgs& a) { return (int64_t)(a.M - 1) * a.ld_h + a.d; }
__device__ __forceinline__ int64_t out_size(const LogitsArgs& a) { return (int64_t)(a.M - 1) * a.ld_out + a.V; }
__device__ __forceinline__ int64_t scales_size(const LogitsArgs& a) { return (int64_t)a.V * (a.d / a.group); }

// cap tanh(z / cap), inv = 1 / cap: the series for small |z / cap| (no cancellation), else by ex2; both are
// computed and one taken, so that lanes do not part
__device__ __forceinline__ float softcap_of(float z, float cap, float inv) {
  const float u = z * inv;
  float q;
  const float s = tanh_small(u), e = tanh_exp(u, &q);
  return cap * (fabsf(u) < kTanhSmall ? s : e);
}

__device__ __forceinline__ void store_logit(const LogitsArgs& a, int m, int v, float z) {
  const float x = a.softcap > 0.f ? softcap_of(z, a.softcap, 1.f / a.softcap) : z;
  const int64_t at = (int64_t)m * a.ld_out + v;
  if (!in_bounds(a.status, at, out_size(a))) return;
  if (a.out_bf16)
    static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
  else
    static_cast<float*>(a.out)[at] = x;
}

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (x & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}

constexpr uint32_t k128x2 = 0x43004300u;  // (128, 128) in bf16

// Eight 4-bit values -> bf16(s q + b) as the pairs (0,4), (1,5), (2,6), (3,7).  0x4300 | q is the
// bf16 value 128 + q, and subtracting 128 is exact; the product and sum round once.
__device__ __forceinline__ void dequant4(uint32_t w, uint32_t s, uint32_t b, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = bf16x2_fma(bf16x2_sub(and_or(w >> (4 * i), 0x000F000Fu, k128x2), k128x2), s, b);
}

// Four 8-bit values -> bf16(s q + b) as the pairs (0,2), (1,3).  The low seven bits make 128 + low as
// above; the high bit, shifted into bit 14, is the bf16 value 2 or 0 and adds 64 times itself.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t b, uint32_t (&p)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = w >> (8 * i);
    const uint32_t low = bf16x2_sub(and_or(x, 0x007F007Fu, k128x2), k128x2);
    const uint32_t q = bf16x2_fma((x << 7) & 0x40004000u, 0x42804280u, low);  // 64 * (2 or 0) + low
    p[i] = bf16x2_fma(q, s, b);
  }
}

// The same results in 9 instructions per 8 4-bit weights instead of 15 (5 instead of 13 per 4 8-bit
// weights).  The bf16 with the bit pattern q, 0 <= q < 256, is q 2^-133 exactly: subnormals and the first
// normal binade are one linear scale.  So the masked bits are an operand as they stand, with the scale
// multiplied by 2^133 (exact while |s| < 2^-5, s133), or by 2^129 for a nibble left in bits 4..7
// (s129); bf16 fma takes subnormal operands at full rate, and product and sum still round once.
__device__ __forceinline__ void dequant4_scaled(uint32_t w, uint32_t s133, uint32_t s129, uint32_t b, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8;
  p[0] = bf16x2_fma(w & 0x000F000Fu, s133, b);
  p[1] = bf16x2_fma(w & 0x00F000F0u, s129, b);
  p[2] = bf16x2_fma(v & 0x000F000Fu, s133, b);
  p[3] = bf16x2_fma(v & 0x00F000F0u, s129, b);
}
__device__ __forceinline__ void dequant8_scaled(uint32_t w, uint32_t s133, uint32_t b, uint32_t (&p)[2]) {
  p[0] = bf16x2_fma(w & 0x00FF00FFu, s133, b);
  p[1] = bf16x2_fma((w >> 8) & 0x00FF00FFu, s133, b);
}

// Tensor-core kernel (decode_logits_tc.cu), its workspace, and a cudaErrorNotSupported when a tensor map
// cannot be made.
size_t logits_tc_workspace(int bits, int64_t M, int64_t d);
cudaError_t launch_logits_tc(const LogitsArgs& a, int bits, int sms, void* workspace, cudaStream_t st);

}  // namespace orpo
