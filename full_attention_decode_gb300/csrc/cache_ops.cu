// Cache rows written and read, and block selection (cache_ops.h).
#include "cache_ops.cuh"
#include "turbo8.cuh"

#include <algorithm>

namespace q35c {
using namespace q35;
namespace {

constexpr uint32_t kThreads = 256;

// ------------------------------------------------------------------ rows in and out

// LPR = D / 8 lanes per (row, kv-head), eight elements a lane: 16-byte loads at every head
// dim. Turbo8: r = bf16(WHT(x)), then codes and scales (quant8).
template <int D, bool T8>
__global__ void __launch_bounds__(kThreads) append_kernel(const Append a) {
  constexpr int LPR = D / 8;
  const size_t item = (blockIdx.x * (size_t)kThreads + threadIdx.x) / LPR;
  const uint32_t lane = threadIdx.x & 31, l = lane % LPR;
  const uint32_t r = (uint32_t)(item / a.c.Hkv), g = (uint32_t)(item % a.c.Hkv);
  uint32_t seq = 0, pos = 0;
  size_t row = 0;
  RowKind kind = r < a.r.n_rows ? locate(a.r, a.c.capacity, r, seq, pos) : kRowSkip;
  if (kind == kRowOk && !cache_row(a.c, seq, pos, row)) kind = kRowBad;
  if (kind == kRowBad) set_status(a.status, kStatusRange);
  const bool ok = kind == kRowOk;
  const size_t src = item * D + 8 * l, dst = (row * a.c.Hkv + g) * D + 8 * l;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (ok) u = *reinterpret_cast<const uint4*>((p ? a.v : a.k) + src);
    uint8_t* to = p ? a.c.v : a.c.k;
    if constexpr (T8) {
      float x[8];
      unpack8(u, x);
      wht8<LPR>(x, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = round_bf16(x[e]);
      uint16_t sc;
      const uint2 codes = quant8(x, sc);
      if (ok) {
        *reinterpret_cast<uint2*>(to + dst) = codes;
        if (l % 2 == 0) (p ? a.c.vs : a.c.ks)[row * a.c.sstride + (g * D + 8 * l) / 16] = sc;
      }
    } else if (ok) {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(to) + dst) = u;
    }
  }
}

// The key bounds: the first row of each (sequence, block) of the call folds the block's
// rows; a block whose first token is among them starts anew.
template <int D>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const Append a) {
  constexpr int LPR = D / 8;
  const size_t item = (blockIdx.x * (size_t)kThreads + threadIdx.x) / LPR;
  const uint32_t l = threadIdx.x % LPR;
  const uint32_t r = (uint32_t)(item / a.c.Hkv), g = (uint32_t)(item % a.c.Hkv);
  uint32_t seq, pos;
  size_t row;
  if (r >= a.r.n_rows || locate(a.r, a.c.capacity, r, seq, pos) != kRowOk || !cache_row(a.c, seq, pos, row)) return;
  const uint32_t S = 1u << a.blk_shift, first = a.r.row_start ? (uint32_t)a.r.row_start[seq] : r;
  if (r != first && pos % S != 0) return;
  uint32_t last = a.r.row_start ? (uint32_t)a.r.row_start[seq + 1] : r + 1;  // rows [r, last) of the block
  last = min(min(last, a.r.n_rows), r + (S - pos % S));
  last = min(last, r + (a.c.capacity - pos));
  uint16_t* b = a.bounds + (((row >> a.blk_shift) * a.c.Hkv + g) * 2) * D + 8 * l;
  float lo[8], hi[8], x[8];
  if (pos % S == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = INFINITY;
      hi[e] = -INFINITY;
    }
  } else {
    unpack8(*reinterpret_cast<const uint4*>(b), lo);
    unpack8(*reinterpret_cast<const uint4*>(b + D), hi);
  }
  for (uint32_t i = r; i < last; ++i) {
    unpack8(*reinterpret_cast<const uint4*>(a.k + ((size_t)i * a.c.Hkv + g) * D + 8 * l), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = fminf(lo[e], x[e]);
      hi[e] = fmaxf(hi[e], x[e]);
    }
  }
  *reinterpret_cast<uint4*>(b) = pack8(lo);
  *reinterpret_cast<uint4*>(b + D) = pack8(hi);
}

template <int D, bool T8>
__global__ void __launch_bounds__(kThreads) read_kernel(const Read a) {
  constexpr int LPR = D / 8;
  const size_t item = (blockIdx.x * (size_t)kThreads + threadIdx.x) / LPR;
  const uint32_t lane = threadIdx.x & 31, l = lane % LPR;
  const uint32_t r = (uint32_t)(item / a.c.Hkv), g = (uint32_t)(item % a.c.Hkv);
  uint32_t seq = 0, pos = 0;
  size_t row = 0;
  RowKind kind = r < a.r.n_rows ? locate(a.r, a.c.capacity, r, seq, pos) : kRowSkip;
  if (kind == kRowOk && !cache_row(a.c, seq, pos, row)) kind = kRowBad;
  if (kind == kRowBad) set_status(a.status, kStatusRange);
  const bool ok = kind == kRowOk;
  const size_t dst = item * D + 8 * l, src = (row * a.c.Hkv + g) * D + 8 * l;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint8_t* from = p ? a.c.v : a.c.k;
    uint16_t* to = p ? a.v : a.k;
    if constexpr (T8) {
      uint2 codes = make_uint2(0u, 0u);
      float sc = 0.f;
      if (ok) {
        codes = *reinterpret_cast<const uint2*>(from + src);
        sc = bf16f((p ? a.c.vs : a.c.ks)[row * a.c.sstride + (g * D + 8 * l) / 16]);
      }
      float x[8];
      dequant_codes8(codes, sc, x);
      wht8<LPR>(x, lane);
      if (ok) *reinterpret_cast<uint4*>(to + dst) = pack8(x);
    } else if (ok) {
      *reinterpret_cast<uint4*>(to + dst) =
          *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(from) + src);
    }
  }
}

uint32_t item_blocks(const Rows& r, const Cache& c) {
  const size_t lanes = (size_t)r.n_rows * c.Hkv * (c.D / 8);
  return (uint32_t)((lanes + kThreads - 1) / kThreads);
}

// ------------------------------------------------------------------ selection

// A float's bits in an order that unsigned comparison follows; NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) x = -INFINITY;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return u >> 63 ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ bool forced(const Select& a, uint32_t j, uint32_t n) {
  return j < a.n_first || (uint64_t)j + a.n_last >= n;
}

// Scores of the blocks a row sees: s_j = sum_d Q+_d hi_jd + Q-_d lo_jd with Q+ and Q- the sums
// over the group's heads of q's positive and negative parts, the sum over the heads of the
// largest q.k a key inside the bounds could have. One CTA per (row, kv-head) and
// gridDim.x-th part of the blocks; LPR lanes a block.
template <int D>
__global__ void __launch_bounds__(kThreads) score_kernel(const Select a) {
  constexpr int LPR = D / 8, PER = kThreads / LPR;
  const uint32_t r = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31, l = lane % LPR;
  uint32_t seq, pos;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
  if (kind != kRowOk) {
    if (kind == kRowBad) set_status(a.status, kStatusRange);
    return;
  }
  const uint32_t n = (pos >> a.blk_shift) + 1;
  if (n <= a.n_select) return;  // every block is taken
  float up[8], dn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) up[e] = dn[e] = 0.f;
  const uint32_t group = a.H / a.c.Hkv;
  for (uint32_t h = 0; h < group; ++h) {
    float x[8];
    unpack8(*reinterpret_cast<const uint4*>(a.q + ((size_t)r * a.H + g * group + h) * D + 8 * l), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      up[e] += fmaxf(x[e], 0.f);
      dn[e] += fminf(x[e], 0.f);
      if (x[e] != x[e]) up[e] = x[e];
    }
  }
  float* out = a.scores + ((size_t)r * a.c.Hkv + g) * a.nblk;
  float most = 0.f;
  for (uint32_t j0 = blockIdx.x * PER; j0 < n; j0 += gridDim.x * PER) {
    const uint32_t j = j0 + threadIdx.x / LPR;
    size_t row = 0;
    const bool in = j < n, here = in && cache_row(a.c, seq, j << a.blk_shift, row);
    if (in && !here) set_status(a.status, kStatusRange);
    float s = 0.f, t = 0.f;
    if (here) {
      const uint16_t* b = a.bounds + (((row >> a.blk_shift) * a.c.Hkv + g) * 2) * D + 8 * l;
      float lo[8], hi[8];
      unpack8(*reinterpret_cast<const uint4*>(b), lo);
      unpack8(*reinterpret_cast<const uint4*>(b + D), hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = fmaf(up[e], hi[e], s);
        t = fmaf(up[e], fabsf(hi[e]), t);
        s = fmaf(dn[e], lo[e], s);
        t = fmaf(-dn[e], fabsf(lo[e]), t);
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (in && l == 0) out[j] = forced(a, j, n) ? INFINITY : here ? s : -INFINITY;
    if (here && !forced(a, j, n)) most = t > most || t != t ? t : most;
  }
  // a NaN or an infinity: no bound on the rounding, every score is formed again
  const bool wild = !(most < INFINITY);
  most = wild ? INFINITY : most;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) atomicMax(reinterpret_cast<int*>(a.most) + (size_t)r * a.c.Hkv + g, __float_as_int(most));
}

// Block j's score in 64 bits, by one warp (the same value in every lane).
template <int D>
__device__ double exact_score(const Select& a, uint32_t r, uint32_t g, uint32_t seq, uint32_t j) {
  const uint32_t lane = threadIdx.x & 31, group = a.H / a.c.Hkv;
  size_t row;
  if (!cache_row(a.c, seq, j << a.blk_shift, row)) return -INFINITY;
  const uint16_t* b = a.bounds + (((row >> a.blk_shift) * a.c.Hkv + g) * 2) * D;
  double s = 0.0;
  for (uint32_t d = lane; d < D; d += 32) {
    double up = 0.0, dn = 0.0;
    for (uint32_t h = 0; h < group; ++h) {
      const double x = bf16f(a.q[((size_t)r * a.H + g * group + h) * D + d]);
      if (x > 0.0 || x != x) up += x;
      else dn += x;
    }
    s += up * (double)bf16f(b[D + d]) + dn * (double)bf16f(b[d]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <typename F>
__device__ __forceinline__ uint32_t block_count(uint32_t n, F&& is, uint32_t* tmp) {
  uint32_t c = 0;
  for (uint32_t j = threadIdx.x; j < n; j += kThreads) c += is(j) ? 1u : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = c;
  __syncthreads();
  c = 0;
  for (uint32_t w = 0; w < kThreads / 32; ++w) c += tmp[w];
  return c;
}

// One CTA per (row, kv-head): the k-th largest of the 32-bit scores (radix selection, a byte a
// pass), then which blocks the exact scores choose. Every s_j is within E of the exact t_j
// (E = 48 2^-24 max_j sum|terms|: at most 15 additions in Q+-, 16 multiply-adds and 5
// additions round). The k-th largest t is then within E of the k-th largest s, T: s_j > T + 2E
// is in, s_j < T - 2E is out, and only what lies between is scored again in 64 bits.
template <int D>
__global__ void __launch_bounds__(kThreads) choose_kernel(const Select a) {
  __shared__ uint32_t hist[256], tmp[kThreads / 32], s_pick[2], s_base[2];
  const uint32_t r = blockIdx.y, g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t seq, pos;
  if (locate(a.r, a.c.capacity, r, seq, pos) != kRowOk) return;
  const uint32_t n = (pos >> a.blk_shift) + 1, K = a.n_select;
  const size_t item = (size_t)r * a.c.Hkv + g;
  int32_t* out = a.blocks + item * K;
  if (n <= K) {
    for (uint32_t i = tid; i < K; i += kThreads) out[i] = i < n ? (int32_t)i : -1;
    return;
  }
  const float* s = a.scores + item * a.nblk;
  double* t = a.exact + item * a.nblk;
  uint32_t prefix = 0, mask = 0, left = K;  // the left-th largest among keys with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (uint32_t j = tid; j < n; j += kThreads) {
      const uint32_t key = order_key(s[j]);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t b = 255, c = 0;
      while (b > 0 && c + hist[b] < left) c += hist[b--];
      s_pick[0] = b;
      s_pick[1] = left - c;
    }
    __syncthreads();
    prefix |= s_pick[0] << shift;
    mask |= 255u << shift;
    left = s_pick[1];
    __syncthreads();
  }
  const float T = key_value(prefix), E = 48.f * 5.9604645e-8f * a.most[item];
  float lo = -INFINITY, hi = INFINITY;
  if (E < INFINITY) {
    lo = isinf(T) ? T : __fadd_rd(T, -2.f * E);
    hi = isinf(T) ? T : __fadd_ru(T, 2.f * E);
  }
  const auto value = [&](uint32_t j) { return key_value(order_key(s[j])); };
  const auto sure = [&](uint32_t j) { return value(j) > hi; };
  const auto maybe = [&](uint32_t j) { return value(j) >= lo && value(j) <= hi; };
  const uint32_t n_sure = block_count(n, sure, tmp), n_maybe = block_count(n, maybe, tmp), need = K - n_sure;
  unsigned long long bar = 0;  // what lies between is in from this key up, `ties` of the equal ones
  uint32_t ties = need;
  const bool again = n_maybe != need;
  if (again) {
    for (uint32_t j0 = 0; j0 < n; j0 += kThreads) {
      unsigned m = __ballot_sync(0xffffffffu, j0 + tid < n && maybe(j0 + tid));
      while (m) {
        const uint32_t j = j0 + warp * 32 + (__ffs(m) - 1);
        m &= m - 1;
        const double x = forced(a, j, n) ? (double)INFINITY : exact_score<D>(a, r, g, seq, j);
        if (lane == 0) t[j] = x;
      }
    }
    __syncthreads();
    for (int bit = 63; bit >= 0; --bit) {  // the need-th largest key, bit by bit
      const unsigned long long c = bar | (1ull << bit);
      if (block_count(n, [&](uint32_t j) { return maybe(j) && order_key(t[j]) >= c; }, tmp) >= need) bar = c;
    }
    ties = need - block_count(n, [&](uint32_t j) { return maybe(j) && order_key(t[j]) > bar; }, tmp);
  }
  // in index order, the lower of equal ones first
  if (tid < 2) s_base[tid] = 0;
  __syncthreads();
  for (uint32_t j0 = 0; j0 < n; j0 += kThreads) {
    const uint32_t j = j0 + tid;
    bool in = false, eq = false;
    if (j < n) {
      in = sure(j);
      if (maybe(j)) {
        if (!again) in = true;
        else if (order_key(t[j]) > bar) in = true;
        else eq = order_key(t[j]) == bar;
      }
    }
    const unsigned me = __ballot_sync(0xffffffffu, eq), below = (1u << lane) - 1u;
    if (lane == 0) tmp[warp] = __popc(me);
    __syncthreads();
    uint32_t rank = s_base[0] + __popc(me & below);
    for (uint32_t w = 0; w < warp; ++w) rank += tmp[w];
    if (eq && rank < ties) in = true;
    uint32_t n_eq = 0;
    for (uint32_t w = 0; w < kThreads / 32; ++w) n_eq += tmp[w];
    __syncthreads();
    const unsigned mi = __ballot_sync(0xffffffffu, in);
    if (lane == 0) tmp[warp] = __popc(mi);
    __syncthreads();
    uint32_t at = s_base[1] + __popc(mi & below), n_in = 0;
    for (uint32_t w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += tmp[w];
      n_in += tmp[w];
    }
    if (in && at < K) out[at] = (int32_t)j;
    __syncthreads();
    if (tid == 0) {
      s_base[0] += n_eq;
      s_base[1] += n_in;
    }
    __syncthreads();
  }
}

}  // namespace

#define Q35C_BY_DIM(D, call)                 \
  switch (D) {                               \
    case 64: { call(64); } break;            \
    case 128: { call(128); } break;          \
    case 256: { call(256); } break;          \
    default: return cudaErrorInvalidValue;   \
  }

cudaError_t append(const Append& a, cudaStream_t st) {
  const uint32_t blocks = item_blocks(a.r, a.c);
  const bool t8 = a.c.ks != nullptr;
#define CALL(DD)                                                         \
  if (t8) append_kernel<DD, true><<<blocks, kThreads, 0, st>>>(a);       \
  else append_kernel<DD, false><<<blocks, kThreads, 0, st>>>(a);         \
  if (a.bounds) bounds_kernel<DD><<<blocks, kThreads, 0, st>>>(a)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
  return cudaGetLastError();
}

cudaError_t read(const Read& a, cudaStream_t st) {
  const uint32_t blocks = item_blocks(a.r, a.c);
  const bool t8 = a.c.ks != nullptr;
#define CALL(DD)                                                    \
  if (t8) read_kernel<DD, true><<<blocks, kThreads, 0, st>>>(a);    \
  else read_kernel<DD, false><<<blocks, kThreads, 0, st>>>(a)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
  return cudaGetLastError();
}

cudaError_t select(const Select& a, cudaStream_t st) {
  const size_t items = (size_t)a.r.n_rows * a.c.Hkv;
  cudaError_t e = cudaMemsetAsync(a.most, 0, items * 4, st);
  if (e != cudaSuccess) return e;
  const uint32_t per = kThreads / (a.c.D / 8);
  const uint32_t parts = (uint32_t)std::min<size_t>((a.nblk + per - 1) / per, std::max<size_t>(1, 1216 / items));
  const dim3 sg(parts, a.c.Hkv, a.r.n_rows), cg(a.c.Hkv, a.r.n_rows);
#define CALL(DD)                                       \
  score_kernel<DD><<<sg, kThreads, 0, st>>>(a);        \
  choose_kernel<DD><<<cg, kThreads, 0, st>>>(a)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
  return cudaGetLastError();
}

}  // namespace q35c
