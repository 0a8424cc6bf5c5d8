// Device helpers of the kernels that read and write KV caches: eight bf16 values of a
// 16-byte word, FP8 E4M3 pairs, and the Walsh-Hadamard transform and quantiser of a
// Turbo8 row held eight elements a lane.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace q35 {

// Eight bf16 values of a 16-byte word as floats, and back (round to nearest even).
__device__ __forceinline__ void unpack8(const uint4 u, float* x) {
  x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
  x[4] = bf16lo(u.z); x[5] = bf16hi(u.z); x[6] = bf16lo(u.w); x[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)to_bf16(x[2 * i]) | ((uint32_t)to_bf16(x[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two floats as E4M3 codes (round to nearest even, saturated), and back (exact).
__device__ __forceinline__ uint32_t e4m3_pair(float x0, float x1) {  // x0 in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
__device__ __forceinline__ float2 e4m3_pair_value(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// The orthonormal Walsh-Hadamard transform (Sylvester order) of a row of 8 * LPR elements,
// lane l of each LPR lanes holding elements [8 l, 8 l + 8): butterflies over the index's
// low bits inside the lane, then over the lane bits, scaled by 1 / sqrt(8 LPR). Bits in
// rising order, as in the layer forwards, so the rows come out the same bit for bit.
template <int LPR>
__device__ __forceinline__ void wht8(float (&x)[8], uint32_t lane) {
#pragma unroll
  for (int hb = 1; hb < 8; hb <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!(e & hb)) {
        const float u = x[e], w = x[e + hb];
        x[e] = u + w;
        x[e + hb] = u - w;
      }
#pragma unroll
  for (uint32_t m = 1; m < LPR; m <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_xor_sync(0xffffffffu, x[e], m);
      x[e] = (lane & m) ? o - x[e] : x[e] + o;
    }
  const float norm = rsqrtf((float)(8 * LPR));
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= norm;
}

// The same transform, four lanes a row: lane l of each four holds pieces i < D / 32 of eight
// elements, [32 i + 8 l, 32 i + 8 l + 8). Index bits 3 and 4 lie on the lanes, all others inside a
// lane, so a row of 256 costs a warp 16 shuffles (40 with 32 lanes a row).
template <int D>
__device__ __forceinline__ void wht_quad(float (&x)[D / 4], uint32_t lane) {
  constexpr int N = D / 4;
#pragma unroll
  for (int hb = 1; hb < 8; hb <<= 1)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!(e & hb)) {
        const float u = x[e], w = x[e + hb];
        x[e] = u + w;
        x[e + hb] = u - w;
      }
#pragma unroll
  for (uint32_t m = 1; m < 4; m <<= 1) {
    const float s = lane & m ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = fmaf(x[e], s, __shfl_xor_sync(0xffffffffu, x[e], m));
  }
#pragma unroll
  for (int hb = 8; hb < N; hb <<= 1)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!(e & hb)) {
        const float u = x[e], w = x[e + hb];
        x[e] = u + w;
        x[e + hb] = u - w;
      }
  const float norm = rsqrtf((float)D);
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] *= norm;
}

// Quantise a piece of eight elements, a group of 16 on two lanes: scale = bf16(amax / 448),
// code = E4M3(x / scale); a zero group keeps scale 0 and codes 0. The quotient is
// x * (1 / scale) with one residual correction (Markstein 1990: q + (x - q s) / s). x and
// scale have 8 significant bits and a border between codes 5, so a quotient that is not on a
// border is at least 2^-13 away from it, and one that is comes out exact: the codes are
// those of the rounded quotient. Scales near the ends of the range take the division.
__device__ __forceinline__ uint2 quant8(const float* x, uint16_t& scale) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  scale = to_bf16(amax / 448.f);
  const float sc = bf16f(scale);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (sc > 1e-30f && sc < 1e30f) {
    const float r = __frcp_rn(sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q0 = x[2 * i] * r, q1 = x[2 * i + 1] * r;
      q0 = fmaf(fmaf(-q0, sc, x[2 * i]), r, q0);
      q1 = fmaf(fmaf(-q1, sc, x[2 * i + 1]), r, q1);
      c[i] = e4m3_pair(q0, q1);
    }
  } else if (sc != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3_pair(x[2 * i] / sc, x[2 * i + 1] / sc);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// Eight codes times their scale (exact).
__device__ __forceinline__ void dequant_codes8(uint2 c, float sc, float* x) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 f = e4m3_pair_value((e < 4 ? c.x : c.y) >> (8 * (e % 4)));
    x[e] = f.x * sc;
    x[e + 1] = f.y * sc;
  }
}

}  // namespace q35
