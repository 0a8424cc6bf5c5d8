// Rows normed, rotated by position and appended to a cache, and accepted rows of a tree moved
// together (rows_ops.h).
#include "rows_ops.h"

#include "cache_ops.cuh"
#include "turbo8.cuh"

#include <algorithm>

namespace q35c {
using namespace q35;
namespace {

constexpr uint32_t kThreads = 256;

// ------------------------------------------------------------------ rotated append

// Eight of the sixteen values of a group, the others in the neighbouring lane, as quant16 does it.
__device__ __forceinline__ uint2 quant8(const uint32_t (&w)[4], uint16_t& scale) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  float amax = fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  scale = to_bf16(amax * (1.0f / 448.0f));
  const float sc = bf16f(scale);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (sc > 1e-30f && sc < 1e30f) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sc));
    const float2 r2 = make_float2(r, r), s2 = make_float2(-sc, -sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = make_float2(bf16lo(w[i]), bf16hi(w[i]));
      float2 q = __fmul2_rn(x, r2);
      q = __ffma2_rn(__ffma2_rn(q, s2, x), r2, q);
      c[i] = e4m3_pair(q.x, q.y);
    }
  } else if (sc != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3_pair(bf16lo(w[i]) / sc, bf16hi(w[i]) / sc);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// bf16(RMSNorm(x) w) of a head's row, eight dims a lane, then RoPE on its first R dims in halves: dim i < R / 2
// turns with dim i + R / 2 by the angle whose (cos, sin) is cs[i]. swap: a row in shared memory, for the other half's
// values. The roundings are the layer forwards'.
template <int LPR>
__device__ __forceinline__ void norm_rotate(float (&x)[8], const uint16_t* w, const float2* cs, float* swap, uint32_t l,
                                            uint32_t R, float eps) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
#pragma unroll
  for (uint32_t m = 1; m < LPR; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (w) {  // null for a row that is not normed: teams of one warp differ
    float g[8];
    unpack8(*reinterpret_cast<const uint4*>(w + 8 * l), g);
    const float inv = rsqrtf(s / (float)(8 * LPR) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = round_bf16(x[e] * inv * g[e]);
  }
  const uint32_t half = R / 2;
  if (8 * l < R)
#pragma unroll
    for (int e = 0; e < 8; ++e) swap[8 * l + e] = x[e];
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t d = 8 * l + e;
    if (d < R) {
      const float2 c = cs[d < half ? d : d - half];
      x[e] = round_bf16(d < half ? x[e] * c.x - swap[d + half] * c.y : x[e] * c.x + swap[d - half] * c.y);
    }
  }
  __syncwarp();
}

// A CTA takes a row: the angles once for all heads, then a team of D / 8 lanes a head's row, q-heads, then k, then v.
template <int D, bool T8>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeAppend a) {
  constexpr uint32_t LPR = D / 8, TEAMS = kThreads / LPR;
  __shared__ float2 cs[D / 2];
  __shared__ float swap[TEAMS][D];
  const uint32_t r = blockIdx.x, l = threadIdx.x % LPR, team = threadIdx.x / LPR, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  uint32_t seq, pos;
  size_t row = 0;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
  const bool ok = kind == kRowOk && cache_row(a.c, seq, pos, row);
  if (!ok) {
    if (kind != kRowSkip && threadIdx.x == 0) set_status(a.status, kStatusRange);
    return;
  }
  const int32_t p = a.rope_pos ? a.rope_pos[r] : (int32_t)pos;
  for (uint32_t i = threadIdx.x; i < a.R / 2; i += kThreads) {
    float sn, c;
    sincosf((float)p * a.inv_freq[i], &sn, &c);
    cs[i] = make_float2(c, sn);
  }
  __syncthreads();
  const uint32_t nq = a.q ? a.H : 0, slots = nq + 2 * a.c.Hkv;
  for (uint32_t s0 = 0; s0 < slots; s0 += TEAMS) {
    const uint32_t s = s0 + team;
    const bool in = s < slots, is_q = s < nq, is_v = s >= nq + a.c.Hkv;
    const uint32_t g = is_q ? s : is_v ? s - nq - a.c.Hkv : s - nq;
    const uint16_t* src = is_q ? a.q + ((size_t)r * a.H + g) * a.q_stride : (is_v ? a.v : a.k) + ((size_t)r * a.c.Hkv + g) * D;
    float x[8] = {};
    if (in) unpack8(*reinterpret_cast<const uint4*>(src + 8 * l), x);
    const bool turns = in && !is_v;
    norm_rotate<LPR>(x, !turns ? nullptr : is_q ? a.q_norm : a.k_norm, cs, swap[team], l, turns ? a.R : 0, a.eps);
    if (in && is_q) *reinterpret_cast<uint4*>(a.q_out + ((size_t)r * a.H + g) * D + 8 * l) = pack8(x);
    if (in && !is_q && !is_v && a.k_out)
      *reinterpret_cast<uint4*>(a.k_out + ((size_t)r * a.c.Hkv + g) * D + 8 * l) = pack8(x);
    if (!a.to_cache) continue;
    const size_t at = (row * a.c.Hkv + g) * D + 8 * l;
    if constexpr (T8) {
      wht8<LPR>(x, lane);
      const uint4 u = pack8(x);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint16_t sc;
      const uint2 codes = quant8(w, sc);
      if (in && !is_q) {
        *reinterpret_cast<uint2*>((is_v ? a.c.v : a.c.k) + at) = codes;
        if (l % 2 == 0) (is_v ? a.c.vs : a.c.ks)[row * a.c.sstride + g * (D / 16) + l / 2] = sc;
      }
    } else if (in && !is_q) {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at) = pack8(x);
    }
  }
}

// ------------------------------------------------------------------ accepted rows moved together

constexpr uint32_t kFlight = 8;  // entries of a thread in flight

// A sequence a CTA column: rows pos + path[i] to pos + i, path rising, so path[i] >= i and no entry's source is
// written before it is read as long as one thread takes all entries of a 16-byte column in order: kFlight are
// loaded, then stored.
__global__ void __launch_bounds__(kThreads) keep_kernel(const __grid_constant__ Keep a) {
  __shared__ size_t from[kMaxNodes], to[kMaxNodes];
  pdl_wait();
  pdl_launch();
  const uint32_t b = blockIdx.x, tid = threadIdx.x;
  int64_t r0 = b, r1 = (int64_t)b + 1;
  if (a.r.row_start) {
    r0 = a.r.row_start[b];
    r1 = a.r.row_start[b + 1];
  }
  r0 = max(r0, (int64_t)0);
  r1 = min(r1, (int64_t)a.r.n_rows);
  if (r1 <= r0) return;
  const int64_t n = r1 - r0, pos = a.r.pos[b];
  bool bad = n > (int64_t)kMaxNodes || pos < 0;
  if (!bad && tid < n) {
    const int64_t p = a.path[r0 + tid], before = tid ? a.path[r0 + tid - 1] : -1;
    size_t x = 0, y = 0;
    bad = p <= before || p < 0 || pos + p >= (int64_t)a.c.capacity;
    if (!bad) bad = !cache_row(a.c, b, (uint32_t)(pos + p), x) || !cache_row(a.c, b, (uint32_t)pos + tid, y);
    from[tid] = x;
    to[tid] = y;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(a.status, kStatusRange);
    return;
  }
  const uint32_t row = a.c.Hkv * a.c.D * (a.c.ks ? 1 : 2) / 16, sc = a.c.ks ? a.c.sstride * 2 / 16 : 0;
  const uint32_t pieces = 2 * (row + sc), i = blockIdx.y * kThreads + tid;
  if (i < pieces) {
    uint8_t* base;
    uint32_t piece, stride;
    if (i < 2 * row) {
      base = i < row ? a.c.k : a.c.v;
      piece = i < row ? i : i - row;
      stride = row;
    } else {
      const uint32_t j = i - 2 * row;
      base = reinterpret_cast<uint8_t*>(j < sc ? a.c.ks : a.c.vs);
      piece = j < sc ? j : j - sc;
      stride = sc;
    }
    uint4* at = reinterpret_cast<uint4*>(base) + piece;
    for (uint32_t e0 = 0; e0 < n; e0 += kFlight) {
      uint4 x[kFlight];
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k)
        if (e0 + k < n && from[e0 + k] != to[e0 + k]) x[k] = at[from[e0 + k] * stride];
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k)
        if (e0 + k < n && from[e0 + k] != to[e0 + k]) at[to[e0 + k] * stride] = x[k];
    }
  }
  // Bounds: a block that gets a row of a later block takes that block's in (they hold the row).
  if (a.bounds && i < a.c.Hkv * a.c.D) {
    const uint32_t g = i / a.c.D, d = i % a.c.D;
    for (uint32_t e = 0; e < n; ++e) {
      const size_t x = from[e] >> a.blk_shift, y = to[e] >> a.blk_shift;
      if (x == y) continue;
      const uint16_t* src = a.bounds + (x * a.c.Hkv + g) * 2 * a.c.D + d;
      uint16_t* dst = a.bounds + (y * a.c.Hkv + g) * 2 * a.c.D + d;
      dst[0] = to_bf16(fminf(bf16f(dst[0]), bf16f(src[0])));
      dst[a.c.D] = to_bf16(fmaxf(bf16f(dst[a.c.D]), bf16f(src[a.c.D])));
    }
  }
}

}  // namespace

cudaError_t rope_append(const RopeAppend& a, cudaStream_t st) {
  const bool t8 = a.c.ks != nullptr;
#define CALL(DD)                                                                                       \
  return t8 ? launch_early(rope_kernel<DD, true>, dim3(a.r.n_rows), kThreads, 0, st, a)                \
            : launch_early(rope_kernel<DD, false>, dim3(a.r.n_rows), kThreads, 0, st, a)
  switch (a.c.D) {
    case 64: CALL(64);
    case 128: CALL(128);
    case 256: CALL(256);
  }
#undef CALL
  return cudaErrorInvalidValue;
}

cudaError_t keep(const Keep& a, cudaStream_t st) {
  const uint32_t row = a.c.Hkv * a.c.D * (a.c.ks ? 1 : 2) / 16, sc = a.c.ks ? a.c.sstride * 2 / 16 : 0;
  const uint32_t pieces = std::max(2 * (row + sc), a.bounds ? a.c.Hkv * a.c.D : 0u);
  return launch_early(keep_kernel, dim3(a.r.n_seqs, (pieces + kThreads - 1) / kThreads), kThreads, 0, st, a);
}

}  // namespace q35c
