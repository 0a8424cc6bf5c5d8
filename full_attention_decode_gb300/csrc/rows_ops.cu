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

// bf16(RMSNorm(x) w) of a head's row (wht_quad's layout: four lanes, pieces of sixteen dims in pairs), then RoPE on its first R
// dims in halves: dim i < R / 2 turns with dim i + R / 2 by the angle whose (cos, sin) is cs[i]. The other half's
// values are bf16 by then and come through the team's row of shared memory. The roundings are the layer forwards'.
template <int D>
__device__ __forceinline__ void norm_rotate(float2 (&x)[D / 8], const uint16_t* w, const float2* cs, uint16_t* swap, uint32_t l,
                                            uint32_t R, float eps) {
  constexpr int P = D / 64;
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < D / 8; ++k) s2 = __ffma2_rn(x[k], x[k], s2);
  float s = s2.x + s2.y;
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  if (w) {  // null for a row that is not normed: teams of a warp differ
    const float inv = rsqrtf(s / (float)D + eps);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint4* g4 = reinterpret_cast<const uint4*>(w + 64 * i + 16 * l);
      const uint4 ga = g4[0], gb = g4[1];
      const uint32_t g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float2& v = x[8 * i + k];
        v = make_float2(round_bf16(v.x * inv * bf16lo(g[k])), round_bf16(v.y * inv * bf16hi(g[k])));
      }
    }
  }
  const uint32_t half = R / 2;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t d0 = 64 * i + 16 * l;
    if (d0 < R) {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 q = __float22bfloat162_rn(x[8 * i + k]);
        u[k] = *reinterpret_cast<const uint32_t*>(&q);
      }
      reinterpret_cast<uint4*>(swap + d0)[0] = make_uint4(u[0], u[1], u[2], u[3]);
      reinterpret_cast<uint4*>(swap + d0)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t d = 64 * i + 16 * l + 8 * h;
      float2* v = x + 8 * i + 4 * h;
      if (d < R && half % 8 == 0) {  // eight dims on one side, their partners side by side
        const bool low = d < half;
        const uint32_t first = low ? d : d - half;
        const float4* c4 = reinterpret_cast<const float4*>(cs + first);
        const uint4 o = *reinterpret_cast<const uint4*>(swap + (low ? d + half : first));
        const uint32_t other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 c = c4[k];  // cos, sin of two dims
          const float a = low ? -c.y : c.y, b = low ? -c.w : c.w;
          v[k] = make_float2(round_bf16(v[k].x * c.x + bf16lo(other[k]) * a), round_bf16(v[k].y * c.z + bf16hi(other[k]) * b));
        }
      } else if (d < R) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& y = e & 1 ? v[e / 2].y : v[e / 2].x;
          if (d + e < half) y = round_bf16(y * cs[d + e].x - bf16f(swap[d + e + half]) * cs[d + e].y);
          else if (d + e < R) y = round_bf16(y * cs[d + e - half].x + bf16f(swap[d + e - half]) * cs[d + e - half].y);
        }
      }
    }
  __syncwarp();
}

constexpr uint32_t kTeams = kThreads / 4;
constexpr uint32_t kRopeRows = 8;  // rows of a CTA at most

// A CTA takes a few rows: their places and angles once for all heads, then four lanes a head's row, q-heads, then k, then v.
// Bound by the instructions of norm, rotation and quantiser and, as a team's items after its first are fetched where they are used, by
// their loads' latency where there are many rows (five prompts of 700 to 4097 tokens into Turbo8, 24 heads of 256: 86 us, 99 with the
// rows read back by qwen35_cache_read; a warp a head's row with its own angles 159 with it), by the launch and the chain of loads of the
// place where there are few (8 rows: 6.0 us a call, 2.5 of them on the GPU).
template <int D, bool T8>
__global__ void __launch_bounds__(kThreads, 2) rope_kernel(const __grid_constant__ RopeAppend a, uint32_t rows) {
  constexpr int P = D / 64;
  __shared__ __align__(16) float2 cs[kRopeRows][D / 2];
  __shared__ __align__(16) uint16_t swap[kTeams][D + 8];
  __shared__ size_t place[kRopeRows];
  __shared__ int32_t turn[kRopeRows];
  __shared__ bool ok[kRopeRows];
  const uint32_t r0 = blockIdx.x * rows, tid = threadIdx.x, l = tid & 3, team = tid / 4, lane = tid & 31;
  pdl_wait();
  pdl_launch();
  const uint32_t nq = a.q ? a.H : 0, slots = nq + 2 * a.c.Hkv, items = min(rows, a.r.n_rows - r0) * slots;
  uint32_t u[P][8];
  const uint16_t* w = nullptr;
  uint32_t r = 0, slot = 0, g = 0;
  bool is_q = false, is_v = false, in = false;
  const auto fetch = [&](uint32_t item) {
    in = item < items;
    r = in ? item / slots : 0;
    slot = in ? item % slots : 0;
    is_q = slot < nq;
    is_v = slot >= nq + a.c.Hkv;
    g = is_q ? slot : is_v ? slot - nq - a.c.Hkv : slot - nq;
    w = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
    const size_t row = r0 + r;
    const uint16_t* src = is_q ? a.q + (row * a.H + g) * a.q_stride : (is_v ? a.v : a.k) + (row * a.c.Hkv + g) * D;
    const bool wide = is_q ? a.wide_q : a.wide_kv;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in) load32(src + 64 * i + 16 * l, wide, u[i]);
  };
  fetch(team);  // on their way while the places are looked up
  if (tid < min(rows, a.r.n_rows - r0)) {
    uint32_t seq, pos;
    size_t row = 0;
    const RowKind kind = locate(a.r, a.c.capacity, r0 + tid, seq, pos);
    ok[tid] = kind == kRowOk && cache_row(a.c, seq, pos, row);
    if (!ok[tid] && kind != kRowSkip) set_status(a.status, kStatusRange);
    place[tid] = row;
    turn[tid] = !ok[tid] ? 0 : a.rope_pos ? a.rope_pos[r0 + tid] : (int32_t)pos;
  }
  __syncthreads();
  const uint32_t half = a.R / 2;
  for (uint32_t i = tid; i < min(rows, a.r.n_rows - r0) * half; i += kThreads) {
    float sn, c;
    sincosf((float)turn[i / half] * a.inv_freq[i % half], &sn, &c);
    cs[i / half][i % half] = make_float2(c, sn);
  }
  __syncthreads();
  for (uint32_t item = team; item - team < items; item += kTeams) {  // whole CTAs
    if (item != team) fetch(item);
    float2 x[D / 8];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[8 * i + k] = in ? make_float2(bf16lo(u[i][k]), bf16hi(u[i][k])) : make_float2(0.f, 0.f);
    const bool go = in && ok[r];
    norm_rotate<D>(x, in ? w : nullptr, cs[r], swap[team], l, in && !is_v ? a.R : 0, a.eps);
    const size_t row = r0 + r;
    const auto store = [&](uint16_t* to, bool wide) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __nv_bfloat162 q = __float22bfloat162_rn(x[8 * i + k]);
          y[k] = *reinterpret_cast<const uint32_t*>(&q);
        }
        store32(to + 64 * i + 16 * l, wide, y);
      }
    };
    if (go && is_q) store(a.q_out + (row * a.H + g) * D, a.wide_out);
    if (go && !is_q && !is_v && a.k_out) store(a.k_out + (row * a.c.Hkv + g) * D, a.wide_out);
    if (!a.to_cache) continue;
    const size_t at = go ? (place[r] * a.c.Hkv + g) * D : 0;
    if constexpr (T8) {
      if (__all_sync(0xffffffffu, !go || is_q)) continue;
      wht_quad<D>(x, lane);
      uint32_t* sc = reinterpret_cast<uint32_t*>((is_v ? a.c.vs : a.c.ks) + (go ? place[r] : 0) * a.c.sstride + (go && !is_q ? g : 0) * (D / 16));
#pragma unroll
      for (int i = 0; i < P; ++i) {
        uint32_t y[8];
        uint16_t s;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __nv_bfloat162 q = __float22bfloat162_rn(x[8 * i + k]);
          y[k] = *reinterpret_cast<const uint32_t*>(&q);
        }
        const uint4 codes = quant16(y, s);
        const uint32_t two = s | (uint32_t)__shfl_xor_sync(0xffffffffu, (uint32_t)s, 1) << 16;  // two groups' scales as one word
        if (go && !is_q) {
          *reinterpret_cast<uint4*>((is_v ? a.c.v : a.c.k) + at + 64 * i + 16 * l) = codes;
          if (l % 2 == 0) sc[2 * i + l / 2] = two;
        }
      }
    } else if (go && !is_q) {
      store(reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at, a.wide_cache);
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
  // A row a CTA while one wave of two CTAs an SM takes all, then as many as keep it one wave, which share the places' latency:
  // 64 rows (bf16, 24 heads of 256) by 1, 2 and 8 a CTA take 5.8, 6.2 and 10.6 us, 608 rows 9.3, 6.6 and 11.0, 8192 rows 105, 67 and 55.
  const uint32_t rows = std::min((a.r.n_rows + 303) / 304, kRopeRows);
  const dim3 grid((a.r.n_rows + rows - 1) / rows);
#define CALL(DD)                                                                         \
  return t8 ? launch_early(rope_kernel<DD, true>, grid, kThreads, 0, st, a, rows)        \
            : launch_early(rope_kernel<DD, false>, grid, kThreads, 0, st, a, rows)
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
