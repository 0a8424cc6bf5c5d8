// Device helpers of the kernels that read and write KV caches: eight bf16 values of a
// 16-byte word, FP8 E4M3 pairs, and the Walsh-Hadamard transform and quantiser of a
// Turbo8 row held eight elements a lane, or by four lanes in pieces of sixteen.
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

// u - w in pairs.
__device__ __forceinline__ float2 sub2(float2 u, float2 w) { return __ffma2_rn(w, make_float2(-1.f, -1.f), u); }

// The same transform, four lanes a row: lane l of each four holds pieces i < D / 64 of sixteen
// elements, [64 i + 16 l, 64 i + 16 l + 16), in pairs (eight a piece). Index bits 4 and 5 lie on the lanes, all
// others inside a lane, so a row of 256 costs a warp 16 shuffles (40 with 32 lanes a row); sums
// and differences are taken two at a time.
template <int D>
__device__ __forceinline__ void wht_quad(float2 (&x)[D / 8], uint32_t lane) {
  constexpr int N = D / 8;
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = make_float2(x[k].x + x[k].y, x[k].x - x[k].y);
#pragma unroll
  for (int hb = 1; hb < 8; hb <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (!(k & hb)) {
        const float2 u = x[k], w = x[k + hb];
        x[k] = __fadd2_rn(u, w);
        x[k + hb] = sub2(u, w);
      }
#pragma unroll
  for (uint32_t m = 1; m < 4; m <<= 1) {
    const float s = lane & m ? -1.f : 1.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, x[k].x, m), __shfl_xor_sync(0xffffffffu, x[k].y, m));
      x[k] = __ffma2_rn(x[k], make_float2(s, s), o);
    }
  }
#pragma unroll
  for (int hb = 8; hb < N; hb <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (!(k & hb)) {
        const float2 u = x[k], w = x[k + hb];
        x[k] = __fadd2_rn(u, w);
        x[k + hb] = sub2(u, w);
      }
  const float norm = rsqrtf((float)D);
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = __fmul2_rn(x[k], make_float2(norm, norm));
}

// 16 bytes, loaded where the call stands.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
// 32 bytes of a lane, in one access where the address is a multiple of 32 (wide), else in two.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Quantise a group of sixteen bf16 values (in pairs): scale = bf16(amax / 448), code = E4M3(x / scale); a
// zero group keeps scale 0 and codes 0, and so does one without a number (the layer forwards' maxima skip NaN); one with
// an infinity gets that as its scale. Neither quotient needs a division:
//  - amax has 8 significant bits and 448 = 7 * 64, so amax / 448 is never on a border between two bf16 values (9
//    bits times 7 has more than 8) and at least 2^-12 away from one: the product with 1 / 448 rounds alike;
//  - x / scale as q = x r with r near 1 / scale and one residual correction, q + (x - q scale) r (Markstein 1990).
//    x and scale have 8 bits and a border between codes 5: a quotient that is not on a border is at least
//    2^-13 away from it, and one that is comes out exact. Scales near the ends of the range take the division.
__device__ __forceinline__ uint4 quant16(const uint32_t (&w)[8], uint16_t& scale) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  const float amax = fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);  // 0 if none is a number
  scale = to_bf16(amax * (1.0f / 448.0f));
  const float sc = bf16f(scale);
  uint32_t c[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (sc > 1e-30f && sc < 1e30f) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sc));
    const float2 r2 = make_float2(r, r), s2 = make_float2(-sc, -sc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = make_float2(bf16lo(w[i]), bf16hi(w[i]));
      float2 q = __fmul2_rn(x, r2);
      q = __ffma2_rn(__ffma2_rn(q, s2, x), r2, q);
      c[i] = e4m3_pair(q.x, q.y);
    }
  } else if (sc != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = e4m3_pair(bf16lo(w[i]) / sc, bf16hi(w[i]) / sc);
  }
  return make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16), c[6] | (c[7] << 16));
}
// Sixteen codes times their scale (exact), in pairs.
__device__ __forceinline__ void dequant16(uint4 c, float sc, float2* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 2 ? c.x : i < 4 ? c.y : i < 6 ? c.z : c.w;
    x[i] = __fmul2_rn(e4m3_pair_value(w >> (16 * (i % 2))), make_float2(sc, sc));
  }
}

}  // namespace q35
