// Tokens sampled from bf16 logits (rows_ops.h).
//
// bf16 logits take at most 2^16 values, so a row is a histogram: counts are whole numbers, a token's weight
// 2^-y, y = (largest - logit) log2(e) / temperature, is that of its value, and the cuts of top-k, top-p and
// min-p are places in the line of values from the largest down, with the lower indexes of equal ones first. Weights
// are whole multiples of 2^-44 (2^-48 accurate before that rounding), so every sum of them is exact and the same in any
// order: what is chosen is what 64-bit arithmetic chooses.
//
// A row is taken by a cluster of kSampleCtas CTAs, each with a part of the tokens: its own histogram in shared memory
// (16-bit counts), read by all through distributed shared memory: a CTA adds up an equal part of the values.
#include <cooperative_groups.h>

#include <cmath>

#include "common.cuh"
#include "rows_ops.h"

namespace q35c {
using namespace q35;
namespace cg = cooperative_groups;
namespace {

constexpr uint32_t kThreads = 512;
constexpr uint32_t kKeyCount = 65536, kBins = kKeyCount / kSampleCtas;  // values of a CTA at most
constexpr uint32_t kSmem = kKeyCount * 2 + kBins * (4 + 8);
constexpr int kOne = 44;  // the largest weight is 2^kOne: kMaxVocab < 2^19 of them fit 64 bits

struct Table {
  unsigned long long t[64];  // 2^63 2^(-i / 64)
};
struct Args {
  Sample s;
  Table table;
};

// A bf16 value's place in an order that unsigned comparison follows; both zeros are one value.
__device__ __forceinline__ uint32_t key_of(uint32_t u) {
  if ((u & 0x7fffu) == 0) u = 0;
  return u & 0x8000u ? 0xffffu & ~u : u | 0x8000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x8000u ? k & 0x7fffu : 0xffffu & ~k) << 16);
}
__device__ __forceinline__ bool is_nan(uint32_t u) { return (u & 0x7fffu) > 0x7f80u; }

// 2^-y as m 2^-(63 + n), m to 2^-48: n whole, 2^(-i / 64) from the table, e^-z for the rest z < 2^-6 ln 2 by its
// series to z^5 / 120 (the next term is below 2^-48 of it).
__device__ __forceinline__ unsigned long long weight(const Table& tab, double y, uint32_t& n) {
  n = 64;
  if (!(y < 63.0)) return 0;
  n = (uint32_t)y;
  const unsigned long long f = __double2ull_rd((y - (double)n) * 18446744073709551616.0);  // in 2^-64
  constexpr unsigned long long kLn2 = 12786308645202655660ull, kAll = ~0ull;                // ln 2 in 2^-64
  const unsigned long long z = __umul64hi(f << 6, kLn2) >> 6;
  unsigned long long e = kAll - z / 5;
  e = kAll - __umul64hi(z / 4, e);
  e = kAll - __umul64hi(z / 3, e);
  e = kAll - __umul64hi(z / 2, e);
  e = kAll - __umul64hi(z, e);
  return __umul64hi(tab.t[f >> 58], e);
}
__device__ __forceinline__ unsigned long long fixed(unsigned long long m, uint32_t n) {  // in 2^-kOne, rounded
  const uint32_t s = 63 - kOne + n;
  return s > 63 ? 0 : (m + (1ull << (s - 1))) >> s;
}

// A place in the line of tokens: how many lie before it and what they weigh.
struct Place {
  unsigned long long weight;
  uint32_t count;
};

struct Shared {
  unsigned long long warp_w[kThreads / 32];
  uint32_t warp_c[kThreads / 32];
  uint32_t least, most;           // this CTA's keys
  Place total;                    // of this CTA's values
  unsigned long long cut;         // what the kept tokens weigh (written by the CTA that finds it)
  unsigned long long floor_w;     // this CTA's weight of values that min-p keeps
  uint32_t key;                   // the chosen value, from the CTA that finds it
  uint32_t nth;                   // which of its tokens
  uint32_t token;
};

__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ Args g) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Shared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(sm);  // two 16-bit counts a word
  unsigned long long* wt = reinterpret_cast<unsigned long long*>(sm + kKeyCount * 2);  // [kBins], from the largest value down
  uint32_t* cnt = reinterpret_cast<uint32_t*>(sm + kKeyCount * 2 + kBins * 8);
  const Sample& a = g.s;
  const cg::cluster_group cl = cg::this_cluster();
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = cl.block_rank(), r = blockIdx.x / kSampleCtas;
  for (uint32_t i = tid; i < kKeyCount * 2 / 16; i += kThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) {
    sh.least = kKeyCount;
    sh.most = 0;
  }
  pdl_wait();
  pdl_launch();
  __syncthreads();

  // ---- this CTA's tokens: eights of 16 aligned bytes, `lead` of the first eight before the row's first token
  const uint16_t* x = a.logits + (size_t)r * a.row_stride;
  const uint32_t lead = (uint32_t)((uintptr_t)x / 2 % 8), eights = (lead + a.vocab + 7) / 8;
  const uint32_t part = (eights + kSampleCtas - 1) / kSampleCtas, t0 = min(eights, me * part), t1 = min(eights, t0 + part);
  // the tokens of an eight, in order
  const auto tokens = [&](uint32_t t, auto&& use) {
    const int32_t i0 = (int32_t)(8 * t) - (int32_t)lead;
    if (i0 >= 0 && (uint32_t)i0 + 8 <= a.vocab) {
      const uint4 u = *reinterpret_cast<const uint4*>(x + i0);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        use(w[i] & 0xffffu, i0 + 2 * i);
        use(w[i] >> 16, i0 + 2 * i + 1);
      }
    } else {
      for (int32_t i = max(i0, 0); i < min(i0 + 8, (int32_t)a.vocab); ++i) use(x[i], i);
    }
  };
  uint32_t least = kKeyCount, most = 0;
#pragma unroll 4
  for (uint32_t t = t0 + tid; t < t1; t += kThreads)
    tokens(t, [&](uint32_t u, int32_t) {
      if (is_nan(u)) return;
      const uint32_t k = key_of(u);
      least = min(least, k);
      most = max(most, k);
      atomicAdd(hist + (k >> 1), k & 1 ? 65536u : 1u);
    });
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    atomicMin(&sh.least, least);
    atomicMax(&sh.most, most);
  }
  cl.sync();

  // ---- the values between the row's least and largest, an equal part a CTA, from the largest down
  for (uint32_t c = 0; c < kSampleCtas; ++c) {
    const Shared* o = cl.map_shared_rank(&sh, c);
    least = min(least, o->least);
    most = max(most, o->most);
  }
  if (least == kKeyCount) {  // no number among them
    if (me == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
    cl.sync();
    return;
  }
  const float temperature = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(temperature > 0.f);
  const double rate = greedy ? 0.0 : 1.4426950408889634 / (double)temperature;
  const double largest = (double)key_value(most);
  const auto octaves = [&](uint32_t k) { return k == most ? 0.0 : (largest - (double)key_value(k)) * rate; };
  const uint32_t n = most - least + 1, each = (n + kSampleCtas - 1) / kSampleCtas;
  const uint32_t b0 = min(n, me * each), bins = min(n, b0 + each) - b0;  // value b of this CTA: key most - b0 - b
  for (uint32_t b = tid; b < bins; b += kThreads) {
    const uint32_t k = most - b0 - b;
    uint32_t c = 0;
#pragma unroll
    for (uint32_t o = 0; o < kSampleCtas; ++o) c += cl.map_shared_rank(hist, o)[k >> 1] >> (k & 1 ? 16 : 0) & 0xffffu;
    cnt[b] = c;
    uint32_t e = 64;
    unsigned long long m = 0;
    if (c) m = weight(g.table, octaves(k), e);
    wt[b] = fixed(m, e);
  }
  __syncthreads();

  // ---- each thread a run of values: what lies before it in the row's line
  const uint32_t run = (bins + kThreads - 1) / kThreads, v0 = min(bins, tid * run), v1 = min(bins, v0 + run);
  const int64_t k64 = greedy ? 1 : a.top_k ? a.top_k[r] : 0;
  const float min_p = a.min_p && a.min_p[r] > 0.f ? fminf(a.min_p[r], 1.f) : 0.f;
  const unsigned long long floor_w = min_p > 0.f ? __double2ull_ru((double)min_p * (double)(1ull << kOne)) : 0;
  Place mine = {0, 0};
  unsigned long long over = 0;
  for (uint32_t b = v0; b < v1; ++b) {
    const unsigned long long w = wt[b] * cnt[b];
    mine.count += cnt[b];
    mine.weight += w;
    if (wt[b] >= floor_w) over += w;
  }
  Place at = mine;  // inclusive sums of the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long w = __shfl_up_sync(0xffffffffu, at.weight, o);
    const uint32_t c = __shfl_up_sync(0xffffffffu, at.count, o);
    if (lane >= (uint32_t)o) {
      at.weight += w;
      at.count += c;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) over += __shfl_xor_sync(0xffffffffu, over, o);
  if (lane == 31) {
    sh.warp_w[warp] = at.weight;
    sh.warp_c[warp] = at.count;
  }
  if (tid == 0) sh.floor_w = 0;
  __syncthreads();
  if (lane == 0) atomicAdd(&sh.floor_w, over);
  at.weight -= mine.weight;
  at.count -= mine.count;
  Place all = {0, 0};
  for (uint32_t w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      at.weight += sh.warp_w[w];
      at.count += sh.warp_c[w];
    }
    all.weight += sh.warp_w[w];
    all.count += sh.warp_c[w];
  }
  if (tid == 0) sh.total = all;
  cl.sync();
  Place row = {0, 0};
  unsigned long long row_floor = 0;
  for (uint32_t c = 0; c < kSampleCtas; ++c) {
    const Shared* o = cl.map_shared_rank(&sh, c);
    const Place p = o->total;
    if (c < me) {
      at.weight += p.weight;
      at.count += p.count;
    }
    row.weight += p.weight;
    row.count += p.count;
    row_floor += o->floor_w;
  }

  // ---- the cuts: what the kept tokens weigh. The thread whose run holds a cut tells all CTAs.
  const auto tell = [&](unsigned long long w) {
    for (uint32_t c = 0; c < kSampleCtas; ++c) cl.map_shared_rank(&sh, c)->cut = w;
  };
  unsigned long long kept = row.weight;
  if (k64 > 0 && k64 < (int64_t)row.count) {
    const uint32_t k = (uint32_t)k64;
    if (at.count < k && k <= at.count + mine.count) {
      Place p = at;
      for (uint32_t b = v0; b < v1; ++b) {
        const uint32_t take = min(cnt[b], k - p.count);
        p.weight += wt[b] * take;
        p.count += take;
      }
      tell(p.weight);
    }
    cl.sync();
    kept = sh.cut;
    cl.sync();
  }
  const float top_p = a.top_p ? a.top_p[r] : 1.f;
  if (top_p < 1.f) {
    // tokens with less than `limit` before them, the first always
    const double limit = fmax((double)top_p, 0.0) * (double)kept;
    const unsigned long long need = max(1ull, __double2ull_ru(limit));  // the least sum that is not below the limit
    if (at.weight < need && need <= at.weight + mine.weight) {
      unsigned long long p = at.weight;
      for (uint32_t b = v0; b < v1 && p < need; ++b)
        if (cnt[b] && wt[b]) p += wt[b] * min((unsigned long long)cnt[b], (need - p + wt[b] - 1) / wt[b]);
      tell(p);
    }
    cl.sync();
    kept = min(kept, sh.cut);
    cl.sync();
  }
  kept = min(kept, row_floor);

  // ---- the token with u of that before it
  const float u = a.u[r];
  unsigned long long goal = u > 0.f ? __double2ull_rd((double)u * (double)kept) : 0;
  goal = min(goal, kept - 1);
  if (at.weight <= goal && goal < at.weight + mine.weight) {
    unsigned long long p = at.weight;
    uint32_t b = v0;
    while (goal - p >= wt[b] * cnt[b]) p += wt[b] * cnt[b], ++b;
    const uint32_t key = most - b0 - b, nth = (uint32_t)((goal - p) / wt[b]);
    for (uint32_t c = 0; c < kSampleCtas; ++c) {
      Shared* o = cl.map_shared_rank(&sh, c);
      o->key = key;
      o->nth = nth;
    }
    if (a.prob) {
      uint32_t e;
      const unsigned long long m = weight(g.table, octaves(key), e);
      a.prob[r] = ldexpf((float)m, kOne - 63 - (int)e) / (float)kept;
    }
  }
  cl.sync();
  // ---- its index: the nth token of that value, in the CTA that holds it
  const uint32_t key = sh.key;
  uint32_t nth = sh.nth, here = 0;
  for (uint32_t c = 0; c <= me; ++c) {
    here = cl.map_shared_rank(hist, c)[key >> 1] >> (key & 1 ? 16 : 0) & 0xffffu;
    if (c < me) {
      if (nth < here) here = kKeyCount;  // an earlier CTA's
      if (here == kKeyCount) break;
      nth -= here;
    }
  }
  if (here != kKeyCount && nth < here) {
    const uint32_t per = (part + kThreads - 1) / kThreads;  // eights of a thread, in order
    const uint32_t e0 = min(t1, t0 + tid * per), e1 = min(t1, e0 + per);
    uint32_t found = 0;
    for (uint32_t t = e0; t < e1; ++t) tokens(t, [&](uint32_t u, int32_t) { found += !is_nan(u) && key_of(u) == key; });
    uint32_t before = found;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= (uint32_t)o) before += y;
    }
    if (lane == 31) sh.warp_c[warp] = before;
    __syncthreads();
    before -= found;
    for (uint32_t w = 0; w < warp; ++w) before += sh.warp_c[w];
    if (before <= nth && nth < before + found)
      for (uint32_t t = e0; t < e1; ++t)
        tokens(t, [&](uint32_t u, int32_t i) {
          if (!is_nan(u) && key_of(u) == key && before++ == nth) a.token[r] = i;
        });
  }
  cl.sync();  // no CTA leaves while another reads its counts
}

}  // namespace

cudaError_t sample_attributes() {
  return cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t sample(const Sample& s, cudaStream_t st) {
  static const Table table = [] {
    Table t;
    for (int i = 0; i < 64; ++i) t.t[i] = (unsigned long long)std::ldexp(std::exp2(-i / 64.0), 63);
    return t;
  }();
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(s.n_rows * kSampleCtas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  c.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kSampleCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, sample_kernel, Args{s, table});
}

}  // namespace q35c
