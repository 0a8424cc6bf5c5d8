// Tokens sampled from bf16 logits (rows_ops.h).
//
// bf16 logits take at most 2^16 values, so a row is a histogram: counts are whole numbers, a token's weight
// 2^-y, y = (largest - logit) log2(e) / temperature, is that of its value, and the cuts of top-k, top-p and
// min-p are places in the line of values from the largest down, with the lower indexes of equal ones first. Weights
// are whole multiples of 2^-44 (2^-40 of themselves accurate before that rounding), so every sum of them is exact and the
// same in any order. No sort: the 64-bit pipe and the order of sums stay out of it.
//
// A row is taken by a cluster of CTAs, each with a part of the tokens and a histogram of it in shared memory (16-bit counts).
// The values come in runs of 128 (a sign and an exponent). Each run that holds a token is added up over the CTAs, through
// distributed shared memory, and weighed by one of them; all read all runs' sums, so all know where the cuts lie without
// asking; the run that a cut lies in is then added up again value by value. Bound by the shared-memory additions of the counting
// and a chain of reads and barriers: a row of 248320 takes 18 us (its bytes 0.1), 64 rows 47 us. The simplest form,
// whose CTAs read one another's runs, took 36 and 170.
#include <cooperative_groups.h>

#include <cmath>
#include <utility>

#include "common.cuh"
#include "rows_ops.h"

namespace q35c {
using namespace q35;
namespace cg = cooperative_groups;
namespace {

constexpr uint32_t kThreads = 1024;
constexpr uint32_t kKeyCount = 65536, kRun = 128, kRuns = kKeyCount / kRun;
constexpr uint32_t kSmem = kKeyCount * 2;
constexpr int kOne = 44;  // the largest weight is 2^kOne: kMaxVocab < 2^19 of them fit 64 bits
typedef unsigned long long u64;

struct Table {
  u64 t[64];  // 2^63 2^(-i / 64)
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

// How a row weighs its values. y = (largest - value) rate in two 32-bit numbers each (TwoSum, Knuth, and products with
// their errors by fma): 2^-46 of it; values and rate over and times two, so that no difference overflows.
struct Scale {
  float half_largest, rate, rate_low;  // rate: 2 log2(e) / temperature
  uint32_t most;                       // the largest value's key
};
__device__ __forceinline__ Scale scale_of(uint32_t most, float temperature) {
  Scale c;
  c.most = most;
  c.half_largest = 0.5f * key_value(most);
  constexpr float kHi = 2.88539004f, kLo = 3.8519259822532e-08f;  // 2 log2(e)
  c.rate = c.rate_low = 0.f;
  if (temperature > 0.f && temperature < INFINITY) {
    c.rate = kHi / temperature;
    c.rate_low = (fmaf(-c.rate, temperature, kHi) + kLo) / temperature;
    if (!(fabsf(c.rate_low) < INFINITY)) c.rate_low = 0.f;
  }
  return c;
}
// 2^-y of key k's value as m 2^-(63 + n): n whole, 2^(-i / 64) from the table, e^-z for the rest z < 2^-6 ln 2 by its
// series to z^5 / 120 (the next term is below 2^-48 of it).
__device__ __forceinline__ u64 weight(const Table& tab, const Scale& c, uint32_t k, uint32_t& n) {
  const float a = c.half_largest, b = -0.5f * key_value(k), s = a + b, t = s - a;
  const float low = (a - (s - t)) + (b - t);
  const float y = s * c.rate;
  n = 64;
  if (k == c.most) {
    n = 0;
    return 1ull << 63;
  }
  if (!(y < 63.f)) return 0;
  const float err = fmaf(s, c.rate, -y) + fmaf(s, c.rate_low, low * c.rate);
  const float whole = floorf(y);
  long long f = (long long)__float2ull_rn((y - whole) * 9223372036854775808.f) + __float2ll_rn(err * 9223372036854775808.f);
  int w = (int)whole;
  if (f < 0) {  // in 2^-63, to [0, 2^63): below 0, or past it as an unsigned number
    const bool past = y - whole > 0.5f;
    w += past ? 1 : -1;
    f = past ? (long long)((u64)f - (1ull << 63)) : (long long)((u64)f + (1ull << 63));
    if (w < 0) w = 0, f = 0;
  }
  n = (uint32_t)w;
  const u64 g = (u64)f << 1;                                     // in 2^-64
  constexpr u64 kLn2 = 12786308645202655660ull, kAll = ~0ull;  // ln 2 in 2^-64
  const u64 z = __umul64hi(g << 6, kLn2) >> 6;
  u64 e = kAll - z / 5;
  e = kAll - __umul64hi(z / 4, e);
  e = kAll - __umul64hi(z / 3, e);
  e = kAll - __umul64hi(z / 2, e);
  e = kAll - __umul64hi(z, e);
  return __umul64hi(tab.t[g >> 58], e);
}
__device__ __forceinline__ u64 fixed(u64 m, uint32_t n) {  // in 2^-kOne, rounded
  const uint32_t s = 63 - kOne + n;
  return s > 63 ? 0 : (m + (1ull << (s - 1))) >> s;
}
// floor(p x), or ceil, for p in [0, 1]: exact.
__device__ __forceinline__ u64 share(float p, u64 x, bool up) {
  const uint32_t b = __float_as_uint(p), e = b >> 23;
  if (!(p > 0.f)) return 0;
  if (p >= 1.f) return x;
  const u64 m = (b & 0x7fffffu) | (e ? 0x800000u : 0u), hi = __umul64hi(m, x), lo = m * x;
  const uint32_t s = 150 - (e ? e : 1);  // p = m 2^-s, s >= 24
  u64 q, rest;
  if (s < 64) {
    q = lo >> s | hi << (64 - s);
    rest = lo << (64 - s);
  } else {
    q = s < 128 ? hi >> (s - 64) : 0;
    rest = lo | (s < 128 ? (s > 64 ? hi << (128 - s) : 0) : hi);
  }
  return q + (up && rest != 0);
}

// What other CTAs need is pushed to them: a store into another CTA's shared memory waits for nothing, a load takes a microsecond.
struct Shared {
  u64 mine_weight[kRuns];  // of the runs that are this CTA's (run % CTAs)
  uint32_t mine_count[kRuns];
  uint32_t used[kRuns];  // runs of this CTA that hold a token in any
  uint32_t list[kRuns], listed;  // those, in no order
  u64 mine_floor;        // of those runs' values that min-p keeps
  uint32_t found[kRuns]; // runs that hold a token of this CTA
  uint32_t word[8 * kRun / 2];  // each CTA's counts of the run that was searched last
  // the row's, written by all CTAs
  u64 run_weight[kRuns];
  uint32_t run_count[kRuns];
  u64 floor_weight;
  uint32_t least, most;
  u64 before_weight;  // of the run that is searched
  uint32_t before_count;
  u64 warp_w[32];
  uint32_t warp_c[32];
  uint32_t fine[kRun];  // the row's counts of a run's values, from its largest down
  u64 fine_w[kRun];     // and their weights
  uint32_t run;
  u64 place;    // what a search found
  uint32_t key, nth;
};

template <uint32_t C>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ Args g) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Shared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(sm);  // two 16-bit counts a word
  const Sample& a = g.s;
  const cg::cluster_group cl = cg::this_cluster();
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = cl.block_rank(), r = blockIdx.x / C;
  for (uint32_t i = tid; i < kKeyCount * 2 / 16; i += kThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < kRuns) {
    sh.mine_weight[tid] = sh.run_weight[tid] = 0;
    sh.mine_count[tid] = sh.run_count[tid] = 0;
    sh.used[tid] = sh.found[tid] = 0;
  }
  if (tid == 0) {
    sh.least = kKeyCount;
    sh.most = 0;
    sh.mine_floor = sh.floor_weight = 0;
    sh.listed = 0;
  }
  auto begun = cl.barrier_arrive();  // the other CTAs may write here
  pdl_wait();
  pdl_launch();
  const float temperature = a.temperature ? a.temperature[r] : 1.f;
  const float u = a.u[r], top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
  const bool greedy = !(temperature > 0.f);
  const int32_t top_k = greedy ? 1 : a.top_k ? a.top_k[r] : 0;
  __syncthreads();

  // ---- this CTA's tokens: eights of 16 aligned bytes, `lead` of the first eight before the row's first token
  const uint16_t* x = a.logits + (size_t)r * a.row_stride;
  const uint32_t lead = (uint32_t)((uintptr_t)x / 2 % 8), eights = (lead + a.vocab + 7) / 8;
  const uint32_t part = (eights + C - 1) / C, t0 = min(eights, me * part), t1 = min(eights, t0 + part);
  // the tokens of an eight, in order
  const auto tokens = [&](uint32_t t, auto&& use) {
    const int32_t i0 = (int32_t)(8 * t) - (int32_t)lead;
    if (i0 >= 0 && (uint32_t)i0 + 8 <= a.vocab) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + i0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
  const auto add = [&](uint32_t k) { atomicAdd(hist + (k >> 1), k & 1 ? 65536u : 1u); };
  constexpr uint32_t kAhead = 4;  // eights of a thread in flight
  for (uint32_t b = t0 + tid; b < t1; b += kAhead * kThreads) {
    uint4 v[kAhead];
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      const uint32_t t = b + i * kThreads;
      const int32_t i0 = (int32_t)(8 * t) - (int32_t)lead;
      // an eight that is not wholly the row's, or none: zeros, which are counted one by one
      v[i] = t < t1 && i0 >= 0 && (uint32_t)i0 + 8 <= a.vocab ? *reinterpret_cast<const uint4*>(x + i0) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t low = 0xffffffffu, high = 0;  // sizes, two a word
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        low = __vminu2(low, w[j] & 0x7fff7fffu);
        high = __vmaxu2(high, w[j] & 0x7fff7fffu);
      }
      if ((low & 0xffffu) && low >> 16 && (high & 0xffffu) <= 0x7f80u && high >> 16 <= 0x7f80u) {  // no zero, no NaN: two keys at once
        uint32_t kmin = 0xffffffffu, kmax = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t k2 = w[j] ^ ((w[j] >> 15 & 0x00010001u) * 0x7fffu | 0x80008000u);
          kmin = __vminu2(kmin, k2);
          kmax = __vmaxu2(kmax, k2);
          add(k2 & 0xffffu);
          add(k2 >> 16);
        }
        least = min(least, min(kmin & 0xffffu, kmin >> 16));
        most = max(most, max(kmax & 0xffffu, kmax >> 16));
      } else if (b + i * kThreads < t1) {
        tokens(b + i * kThreads, [&](uint32_t y, int32_t) {
          if (is_nan(y)) return;
          const uint32_t k = key_of(y);
          least = min(least, k);
          most = max(most, k);
          add(k);
        });
      }
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  cl.barrier_wait(std::move(begun));
  if (lane < C) {  // a warp tells CTA `lane`
    Shared* o = cl.map_shared_rank(&sh, lane);
    atomicMin(&o->least, least);
    atomicMax(&o->most, most);
  }
  __syncthreads();
  for (uint32_t i = tid; i < kKeyCount * 2 / 16; i += kThreads) {
    const uint4 v = reinterpret_cast<const uint4*>(sm)[i];
    if (v.x | v.y | v.z | v.w) sh.found[i * 8 / kRun] = 1;
  }
  __syncthreads();
  if (tid < kRuns && sh.found[tid]) cl.map_shared_rank(&sh, tid % C)->used[tid] = 1;
  cl.sync();
  least = sh.least;
  most = sh.most;
  if (least == kKeyCount) {  // no number among them
    if (me == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
    return;  // no CTA reads another's memory any more
  }

  // ---- this CTA's runs: half a run a warp, two values a lane
  const Scale scale = scale_of(most, greedy ? 0.f : temperature);
  const u64 floor_w = min_p > 0.f ? share(fminf(min_p, 1.f), 1ull << kOne, true) : 0;
  u64 over = 0;
  if (tid < kRuns && sh.used[tid]) sh.list[atomicAdd(&sh.listed, 1u)] = tid;
  __syncthreads();
  for (uint32_t unit = warp; unit < 2 * sh.listed; unit += kThreads / 32) {
    const uint32_t q = sh.list[unit / 2], word = q * (kRun / 2) + unit % 2 * 32 + lane;
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (uint32_t c = 0; c < C; ++c) {
      const uint32_t y = cl.map_shared_rank(hist, c)[word];
      c0 += y & 0xffffu;
      c1 += y >> 16;
    }
    u64 w = 0;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t n = i ? c1 : c0;
      uint32_t e;
      const u64 m = n ? weight(g.table, scale, 2 * word + i, e) : 0, y = n ? fixed(m, e) : 0;
      w += y * n;
      if (y >= floor_w) over += y * n;
    }
    const uint32_t n = __reduce_add_sync(0xffffffffu, c0 + c1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    if (lane == 0) {
      atomicAdd(&sh.mine_weight[q], w);
      atomicAdd(&sh.mine_count[q], n);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) over += __shfl_xor_sync(0xffffffffu, over, o);
  if (lane == 0 && over) atomicAdd(&sh.mine_floor, over);
  __syncthreads();
  if (tid < kRuns) {  // thread i: run i / C of this CTA's, to CTA i % C
    const uint32_t q = tid / C * C + me;
    if (sh.mine_count[q]) {
      Shared* o = cl.map_shared_rank(&sh, tid % C);
      o->run_weight[q] = sh.mine_weight[q];
      o->run_count[q] = sh.mine_count[q];
    }
    if (tid < C) atomicAdd(&cl.map_shared_rank(&sh, tid)->floor_weight, sh.mine_floor);
  }
  cl.sync();

  // ---- the row's runs, from the largest values down: thread i has run kRuns - 1 - i; what lies before each
  u64 mine_w = 0;
  uint32_t mine_c = 0;
  if (tid < kRuns) {
    mine_w = sh.run_weight[kRuns - 1 - tid];
    mine_c = sh.run_count[kRuns - 1 - tid];
  }
  u64 at_w = mine_w;
  uint32_t at_c = mine_c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, at_w, o);
    const uint32_t c = __shfl_up_sync(0xffffffffu, at_c, o);
    if (lane >= (uint32_t)o) {
      at_w += w;
      at_c += c;
    }
  }
  if (lane == 31) {
    sh.warp_w[warp] = at_w;
    sh.warp_c[warp] = at_c;
  }
  __syncthreads();
  u64 row_w = 0;
  uint32_t row_c = 0;
  for (uint32_t w = 0; w < kRuns / 32; ++w) {
    if (w < warp) {
      at_w += sh.warp_w[w];
      at_c += sh.warp_c[w];
    }
    row_w += sh.warp_w[w];
    row_c += sh.warp_c[w];
  }
  at_w -= mine_w;  // before this run
  at_c -= mine_c;

  // A search: the thread whose run holds the place says so, the run's counts are added up over the CTAs and weighed, and
  // warp 0 walks its values, four a lane from the largest down: find(weight and count before the value, its weight and count,
  // its key).
  const auto search = [&](bool here, auto&& find) {
    if (here) {
      sh.run = kRuns - 1 - tid;
      sh.before_weight = at_w;
      sh.before_count = at_c;
    }
    if (tid < kRun) sh.fine[tid] = 0;
    __syncthreads();
    const uint32_t q = sh.run;
    if (tid < 64 * C) {
      const uint32_t h = cl.map_shared_rank(hist, tid / 64)[q * 64 + tid % 64], k = 2 * (tid % 64);
      sh.word[tid] = h;
      if (h & 0xffffu) atomicAdd(&sh.fine[kRun - 1 - k], h & 0xffffu);
      if (h >> 16) atomicAdd(&sh.fine[kRun - 2 - k], h >> 16);
    }
    __syncthreads();
    if (tid < kRun) {
      uint32_t e;
      const u64 m = sh.fine[tid] ? weight(g.table, scale, q * kRun + kRun - 1 - tid, e) : 0;
      sh.fine_w[tid] = m ? fixed(m, e) : 0;
    }
    if (tid < kRun) named_barrier(1, kRun);  // the warps that weighed; warp 0 goes on alone
    if (warp == 0) {
      u64 w[4], sum = 0;
      uint32_t c[4], n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = sh.fine[4 * lane + i];
        w[i] = sh.fine_w[4 * lane + i];
        sum += w[i] * c[i];
        n += c[i];
      }
      u64 bw = sum;
      uint32_t bc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, bw, o);
        const uint32_t z = __shfl_up_sync(0xffffffffu, bc, o);
        if (lane >= (uint32_t)o) {
          bw += y;
          bc += z;
        }
      }
      bw += sh.before_weight - sum;
      bc += sh.before_count - n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        find(bw, bc, w[i], c[i], q * kRun + kRun - 1 - (4 * lane + i));
        bw += w[i] * c[i];
        bc += c[i];
      }
    }
    __syncthreads();
  };

  // ---- the cuts: what the kept tokens weigh
  u64 kept = row_w;
  if (top_k > 0 && (uint32_t)top_k < row_c) {
    const uint32_t k = (uint32_t)top_k;
    search(at_c < k && k <= at_c + mine_c, [&](u64 bw, uint32_t bc, u64 w, uint32_t c, uint32_t) {
      if (bc < k && k <= bc + c) sh.place = bw + w * (k - bc);
    });
    kept = sh.place;
  }
  if (top_p < 1.f) {
    // tokens with less than top_p of the sum before them, the first always: the least sum that is not below it
    const u64 need = max(1ull, share(top_p, kept, true));
    search(at_w < need && need <= at_w + mine_w, [&](u64 bw, uint32_t, u64 w, uint32_t c, uint32_t) {
      if (bw < need && need <= bw + w * c) sh.place = bw + w * ((need - bw + w - 1) / w);
    });
    kept = min(kept, sh.place);
  }
  kept = min(kept, sh.floor_weight);

  // ---- the token with u of that before it
  const u64 goal = min(share(u, kept, false), kept - 1);
  search(at_w <= goal && goal < at_w + mine_w, [&](u64 bw, uint32_t, u64 w, uint32_t c, uint32_t key) {
    if (bw <= goal && goal < bw + w * c) {
      sh.key = key;
      sh.nth = (uint32_t)((goal - bw) / w);
    }
  });
  // ---- its index: the nth token of that value, in the CTA that holds it
  auto read = cl.barrier_arrive();  // this CTA reads no other's counts any more
  const uint32_t key = sh.key;
  if (a.prob && me == C - 1 && tid == kThreads - 1) {  // 53 bits, rounded once
    uint32_t e;
    const u64 m = weight(g.table, scale, key, e);
    a.prob[r] = (float)(ldexp((double)m, kOne - 63 - (int)e) / (double)kept);
  }
  uint32_t nth = sh.nth, before = 0, here = 0;
  for (uint32_t c = 0; c <= me; ++c) {
    before += here;
    here = sh.word[c * (kRun / 2) + (key % kRun) / 2] >> (key & 1 ? 16 : 0) & 0xffffu;
  }
  if (before <= nth && nth < before + here) {
    nth -= before;
    // each warp a stretch of eights, its lanes side by side: counted, then looked through by the warp that has the token
    const uint32_t per = (part + kThreads / 32 - 1) / (kThreads / 32), e0 = min(t1, t0 + warp * per), e1 = min(t1, e0 + per);
    const uint32_t bits = key & 0x8000u ? key & 0x7fffu : 0xffffu & ~key, two = bits | bits << 16;
    // which tokens of an eight are of that value
    const auto which = [&](uint32_t t) {
      const int32_t i0 = (int32_t)(8 * t) - (int32_t)lead;
      uint32_t is = 0;
      if (t < e1 && bits && i0 >= 0 && (uint32_t)i0 + 8 <= a.vocab) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + i0);
        const uint32_t w[4] = {v.x ^ two, v.y ^ two, v.z ^ two, v.w ^ two};
#pragma unroll
        for (int i = 0; i < 4; ++i) is |= (uint32_t)((w[i] & 0xffffu) == 0) << 2 * i | (uint32_t)(w[i] >> 16 == 0) << (2 * i + 1);
      } else if (t < e1) {  // an end, or either zero
        tokens(t, [&](uint32_t v, int32_t i) { is |= (uint32_t)(!is_nan(v) && key_of(v) == key) << (i - i0); });
      }
      return is;
    };
    uint32_t found = 0;
#pragma unroll 4
    for (uint32_t t = e0 + lane; t - lane < e1; t += 32) found += __popc(which(t));
    found = __reduce_add_sync(0xffffffffu, found);
    if (lane == 0) sh.warp_c[warp] = found;
    __syncthreads();
    uint32_t ahead = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_c[lane] : 0u);
    if (ahead <= nth && nth < ahead + found)
      for (uint32_t t = e0 + lane; t - lane < e1; t += 32) {
        uint32_t is = which(t), n = __popc(is), upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= (uint32_t)o) upto += y;
        }
        const uint32_t rank = ahead + upto - n;
        if (rank <= nth && nth < rank + n) {
          for (uint32_t k = rank; k < nth; ++k) is &= is - 1;
          a.token[r] = (int32_t)(8 * t) - (int32_t)lead + __ffs(is) - 1;
        }
        ahead += __shfl_sync(0xffffffffu, upto, 31);
        if (nth < ahead) break;
      }
  }
  cl.barrier_wait(std::move(read));  // and none leaves while another reads its own
}

template <uint32_t C>
cudaError_t launch(const Args& g, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(g.s.n_rows * C);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  c.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, sample_kernel<C>, g);
}

}  // namespace

cudaError_t sample_attributes() {
  const cudaError_t e = cudaFuncSetAttribute(sample_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(sample_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t sample(const Sample& s, cudaStream_t st) {
  static const Table table = [] {
    Table t;
    for (int i = 0; i < 64; ++i) t.t[i] = (u64)std::ldexp(std::exp2(-i / 64.0), 63);
    return t;
  }();
  // Eight CTAs a row while the clusters of all rows find room at once, or where four could not count the tokens in 16 bits;
  // otherwise four. Of 248320 tokens 1 row takes 18.8 us with eight, 22.5 with four; 8 rows 19.9 and 24.8; 16 rows 35.5 and 25.7; 64
  // rows 82.8 and 49.0.
  return s.n_rows <= 8 || s.vocab > 4 * (kMaxVocab / 8) ? launch<8>({s, table}, st) : launch<4>({s, table}, st);
}

}  // namespace q35c
