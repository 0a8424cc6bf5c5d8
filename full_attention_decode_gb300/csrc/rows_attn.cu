// Attention of drafted trees and of rows that see a sliding window (rows_ops.h).
#include "rows_ops.h"

#include "cache_ops.cuh"
#include "turbo8.cuh"

namespace q35c {
using namespace q35;
namespace {

// A warp a (row, q-head), token after token.
template <int D, bool T8>
__global__ void __launch_bounds__(128) rows_kernel(const __grid_constant__ RowsAttend a) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch();
  const uint32_t item = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (item >= a.r.n_rows * a.H) return;
  const uint32_t r = item / a.H, h = item % a.H, g = h / (a.H / a.c.Hkv);
  uint32_t seq, pos, index, left;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos, index, left);
  if (kind != kRowOk) {
    if (kind == kRowBad && lane == 0) set_status(a.status, kStatusRange);
    return;
  }
  uint32_t line[kMaxNodes / 32] = {};
  if (a.parent) {
    bool bad = index >= kMaxNodes || index > r;  // the latter: row starts that fall below 0
    for (int32_t i = (int32_t)index; !bad;) {
#pragma unroll
      for (uint32_t w = 0; w < kMaxNodes / 32; ++w)
        if (i / 32 == (int32_t)w) line[w] |= 1u << (i % 32);
      const int32_t p = a.parent[r - index + i];
      if (p == -1) break;
      bad = p < 0 || p >= i;
      i = p;
    }
    if (bad) {
      if (lane == 0) set_status(a.status, kStatusRange);
      return;
    }
  }
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  float buf[E];
  const uint16_t* qs = a.q + ((size_t)r * a.H + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = bf16f(qs[e]);
  auto rotate = [&](float (&x)[E]) {
#pragma unroll
    for (int hb = 1; hb < E; hb <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (!(e & hb)) {
          const float u = x[e], w = x[e + hb];
          x[e] = u + w;
          x[e + hb] = u - w;
        }
    for (uint32_t b = 1; b < 32; b <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = __shfl_xor_sync(0xffffffffu, x[e], b);
        x[e] = lane & b ? y - x[e] : x[e] + y;
      }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= rsqrtf((float)D);
  };
  if (T8) rotate(q);
  const float scale = 1.4426950408889634f / sqrtf((float)D);
  const uint32_t base = pos - (a.parent ? index : 0), low = a.parent || pos < a.window ? 0 : pos - a.window + 1;
  for (uint32_t t = 0; t <= pos; ++t) {
    if (a.parent) {
      const uint32_t i = t - base;
      if (t >= base && !(line[i / 32] >> (i % 32) & 1)) continue;
    } else if (t < low && t >= a.n_first) {
      t = low - 1;
      continue;
    }
    size_t row;
    if (!cache_row(a.c, seq, t, row)) {
      if (lane == 0) set_status(a.status, kStatusRange);
      continue;
    }
    const size_t at = (row * a.c.Hkv + g) * D + lane * E;
    const auto load = [&](const uint8_t* x, const uint16_t* sc) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if constexpr (T8) {
          const float2 v = e4m3_pair_value(x[at + e]);
          buf[e] = v.x * bf16f(sc[row * a.c.sstride + g * (D / 16) + (lane * E + e) / 16]);
        } else {
          buf[e] = bf16f(reinterpret_cast<const uint16_t*>(x)[at + e]);
        }
    };
    load(a.c.k, a.c.ks);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], buf[e], s);
    s = warp_sum(s) * scale;
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - mn), p = s == -INFINITY ? 0.f : exp2f(s - mn);
    load(a.c.v, a.c.vs);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, buf[e], o[e] * f);
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = l == 0.f ? 0.f : o[e] / l;
  if (T8) rotate(o);
  uint16_t* out = a.out + ((size_t)r * a.H + h) * D + lane * E;
  const uint16_t* gate = a.gate ? a.gate + ((size_t)r * a.H + h) * a.gate_stride + lane * E : nullptr;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = to_bf16(gate ? o[e] * sigmoidf_(bf16f(gate[e])) : o[e]);
}

}  // namespace

size_t rows_work_bytes(uint32_t n_rows, uint32_t H, uint32_t Hkv, uint32_t D) {
  return ((size_t)n_rows * H + kMaxCtas * 128) * (D + 8) * 4 + (size_t)n_rows * Hkv * 16;
}
cudaError_t rows_attend_attributes() { return cudaSuccess; }

cudaError_t rows_attend(const RowsAttend& a, cudaStream_t st) {
  const dim3 grid((a.r.n_rows * a.H + 3) / 4);
  const bool t8 = a.c.ks != nullptr;
#define CALL(DD)                                                        \
  return t8 ? launch_early(rows_kernel<DD, true>, grid, 128, 0, st, a)  \
            : launch_early(rows_kernel<DD, false>, grid, 128, 0, st, a)
  switch (a.c.D) {
    case 64: CALL(64);
    case 128: CALL(128);
    case 256: CALL(256);
  }
#undef CALL
  return cudaErrorInvalidValue;
}

}  // namespace q35c
