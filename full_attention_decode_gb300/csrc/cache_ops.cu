// Cache rows written and read, and block selection (cache_ops.h).
#include "cache_ops.cuh"
#include "turbo8.cuh"

#include <algorithm>

namespace q35c {
using namespace q35;
namespace {

constexpr uint32_t kThreads = 256;

// ------------------------------------------------------------------ rows in and out

// A (row, kv-head) item of a call: where its cache row is. Every lane of a team asks.
struct Item {
  bool ok;
  uint32_t g;
  size_t row;
};
__device__ __forceinline__ Item find_item(const Rows& w, const Cache& c, size_t item, int* status) {
  Item x = {false, 0, 0};
  const uint32_t r = (uint32_t)(item / c.Hkv);
  x.g = (uint32_t)(item % c.Hkv);
  if (r >= w.n_rows) return x;
  uint32_t seq, pos;
  const RowKind kind = locate(w, c.capacity, r, seq, pos);
  x.ok = kind == kRowOk && cache_row(c, seq, pos, x.row);
  if (!x.ok && kind != kRowSkip) set_status(status, kStatusRange);
  return x;
}

// A bf16 row: D / 8 lanes an item, 16 bytes a lane.
template <int D>
__device__ __forceinline__ void append_plain(const Append& a, uint32_t block) {
  constexpr int LPR = D / 8;
  const size_t item = (block * (size_t)kThreads + threadIdx.x) / LPR;
  const uint32_t l = threadIdx.x % LPR;
  if (item >= (size_t)a.r.n_rows * a.c.Hkv) return;
  const size_t src = item * D + 8 * l;  // on its way while the cache row is looked up
  const uint4 k = load16(a.k + src), v = load16(a.v + src);
  const Item x = find_item(a.r, a.c, item, a.status);
  if (!x.ok) return;
  const size_t dst = (x.row * a.c.Hkv + x.g) * D + 8 * l;
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.c.k) + dst) = k;
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.c.v) + dst) = v;
}

// A Turbo8 row: four lanes an item and K or V, D / 4 elements a lane (wht_quad's layout).
struct QuadItem {
  size_t item;
  uint32_t l;
  bool is_v;
};
__device__ __forceinline__ QuadItem quad_item(uint32_t block) {  // a warp's eight fours: eight items' K or V
  const size_t team = (block * (size_t)kThreads + threadIdx.x) / 4;
  return {team / 16 * 8 + team % 8, threadIdx.x & 3, (team & 8) != 0};
}

template <int D>
__device__ __forceinline__ void append_turbo8(const Append& a, uint32_t block) {
  constexpr int P = D / 64;  // pieces of sixteen elements
  const QuadItem t = quad_item(block);
  const uint32_t lane = threadIdx.x & 31;
  const bool in = t.item < (size_t)a.r.n_rows * a.c.Hkv;
  const uint16_t* src = (t.is_v ? a.v : a.k) + t.item * D + 16 * t.l;
  uint32_t u[P][8] = {};
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (in) load32(src + 64 * i, a.wide, u[i]);
  const Item w = find_item(a.r, a.c, t.item, a.status);  // while the rows are on their way
  float2 x[D / 8];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) x[8 * i + k] = make_float2(bf16lo(u[i][k]), bf16hi(u[i][k]));
  wht_quad<D>(x, lane);
  uint8_t* to = (t.is_v ? a.c.v : a.c.k) + (w.row * a.c.Hkv + w.g) * D + 16 * t.l;
  uint32_t* sc = reinterpret_cast<uint32_t*>((t.is_v ? a.c.vs : a.c.ks) + w.row * a.c.sstride + w.g * (D / 16));
#pragma unroll
  for (int i = 0; i < P; ++i) {
    uint16_t s;
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 q = __float22bfloat162_rn(x[8 * i + k]);
      r[k] = *reinterpret_cast<const uint32_t*>(&q);
    }
    const uint4 codes = quant16(r, s);
    if (w.ok) *reinterpret_cast<uint4*>(to + 64 * i) = codes;
    // two groups' scales as one word
    const uint32_t two = s | (uint32_t)__shfl_xor_sync(0xffffffffu, (uint32_t)s, 1) << 16;
    if (w.ok && t.l % 2 == 0) sc[2 * i + t.l / 2] = two;
  }
}

// The key bounds of spans of rows. A run is the call's rows of one block of one sequence; who has the span with
// its first row folds it, starting anew if that is the block's first token. A dimension in which every value was NaN (lo
// is still above hi) gets NaN for its bounds, which later rows' values replace. WIDE: a CTA a (span, kv-head), its
// teams of D / 8 lanes taking a run's rows in turn; otherwise a team alone, sixteen rows in flight (fold_wide).
template <int D, bool WIDE>
__device__ __forceinline__ void append_bounds(const Append& a, uint32_t span, uint32_t g, uint32_t span_rows) {
  constexpr int LPR = D / 8, TEAMS = WIDE ? kThreads / LPR : 1;
  __shared__ float part[2][WIDE ? TEAMS : 1][WIDE ? D : 1];
  const uint32_t l = threadIdx.x % LPR, team = WIDE ? threadIdx.x / LPR : 0, S = 1u << a.blk_shift;
  const uint32_t end = min(a.r.n_rows, (span + 1) * span_rows);
  for (uint32_t r = span * span_rows; r < end;) {
    uint32_t seq, pos;
    size_t row;
    const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
    if (kind != kRowOk || !cache_row(a.c, seq, pos, row)) {  // reported by the row's writer
      ++r;
      continue;
    }
    // the rows of this sequence from r on that lie in its block
    int64_t last = a.r.row_start ? a.r.row_start[seq + 1] : (int64_t)r + 1;
    last = min(min(last, (int64_t)a.r.n_rows), (int64_t)r + (S - pos % S));
    last = min(last, (int64_t)r + (a.c.capacity - pos));
    const uint32_t stop = (uint32_t)max(last, (int64_t)r + 1);
    const bool fresh = pos % S == 0;
    if (!fresh && a.r.row_start && (int64_t)r != a.r.row_start[seq]) {  // its first row is in an earlier span
      r = stop;
      continue;
    }
    uint16_t* b = a.bounds + (((row >> a.blk_shift) * a.c.Hkv + g) * 2) * D;
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = INFINITY;
      hi[e] = -INFINITY;
    }
    if (!fresh && team == 0) {
      unpack8(*reinterpret_cast<const uint4*>(b + 8 * l), lo);
      unpack8(*reinterpret_cast<const uint4*>(b + D + 8 * l), hi);
    }
    const uint16_t* src = a.k + (size_t)g * D + 8 * l;
#pragma unroll WIDE ? 4 : 16
    for (uint32_t i = r + team; i < stop; i += TEAMS) {
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(src + (size_t)i * a.c.Hkv * D), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = fminf(lo[e], x[e]);
        hi[e] = fmaxf(hi[e], x[e]);
      }
    }
    if constexpr (WIDE) {
      const uint32_t used = min(stop - r, (uint32_t)TEAMS);
      if (team < used)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          part[0][team][8 * l + e] = lo[e];
          part[1][team][8 * l + e] = hi[e];
        }
      __syncthreads();
      for (uint32_t d = threadIdx.x; d < D; d += kThreads) {
        float x = part[0][0][d], y = part[1][0][d];
        for (uint32_t t = 1; t < used; ++t) {
          x = fminf(x, part[0][t][d]);
          y = fmaxf(y, part[1][t][d]);
        }
        b[d] = to_bf16(x > y ? NAN : x);
        b[D + d] = to_bf16(x > y ? NAN : y);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lo[e] > hi[e]) lo[e] = hi[e] = NAN;
      *reinterpret_cast<uint4*>(b + 8 * l) = pack8(lo);
      *reinterpret_cast<uint4*>(b + D + 8 * l) = pack8(hi);
    }
    r = stop;
  }
}

// bound_ctas CTAs bring the bounds up to date, the first of every 2^period_shift CTAs until there are enough; the others
// write rows. A bounds' CTA has the longest chain of loads, so it is a little ahead of the rows that it shares: those
// find the keys in the L2 (32768 rows, blocks of 16: 57 us; all bounds first: 61 us).
template <int D, bool T8>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Append a, uint32_t bound_ctas,
                                                          uint32_t period_shift, uint32_t span_rows) {
  pdl_wait();
  pdl_launch();
  const uint32_t turn = blockIdx.x >> period_shift;
  if (turn >= bound_ctas || turn << period_shift != blockIdx.x) {
    const uint32_t block = blockIdx.x - min(turn + 1, bound_ctas);
    if constexpr (T8) append_turbo8<D>(a, block);
    else append_plain<D>(a, block);
  } else if (a.wide_bounds) {
    append_bounds<D, true>(a, turn / a.c.Hkv, turn % a.c.Hkv, span_rows);
  } else {
    const uint32_t team = turn * (kThreads / (D / 8)) + threadIdx.x / (D / 8);
    append_bounds<D, false>(a, team / a.c.Hkv, team % a.c.Hkv, span_rows);
  }
}

template <int D, bool T8>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Read a) {
  pdl_wait();
  pdl_launch();
  if constexpr (T8) {
    constexpr int P = D / 64;
    const QuadItem t = quad_item(blockIdx.x);
    const Item w = find_item(a.r, a.c, t.item, a.status);
    const uint8_t* from = (t.is_v ? a.c.v : a.c.k) + (w.row * a.c.Hkv + w.g) * D + 16 * t.l;
    const uint16_t* sc = (t.is_v ? a.c.vs : a.c.ks) + w.row * a.c.sstride + w.g * (D / 16) + t.l;
    float2 x[D / 8];
    uint4 codes[P];
    uint16_t s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      codes[i] = w.ok ? *reinterpret_cast<const uint4*>(from + 64 * i) : make_uint4(0u, 0u, 0u, 0u);
      s[i] = w.ok ? sc[4 * i] : 0;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) dequant16(codes[i], bf16f(s[i]), x + 8 * i);
    wht_quad<D>(x, threadIdx.x & 31);
    uint16_t* to = (t.is_v ? a.v : a.k) + t.item * D + 16 * t.l;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 q = __float22bfloat162_rn(x[8 * i + k]);
        u[k] = *reinterpret_cast<const uint32_t*>(&q);
      }
      if (w.ok) store32(to + 64 * i, a.wide, u);
    }
  } else {
    constexpr int LPR = D / 8;
    const size_t item = (blockIdx.x * (size_t)kThreads + threadIdx.x) / LPR;
    const uint32_t l = threadIdx.x % LPR;
    const Item w = find_item(a.r, a.c, item, a.status);
    if (!w.ok) return;
    const size_t dst = item * D + 8 * l, src = (w.row * a.c.Hkv + w.g) * D + 8 * l;
    const uint4 k = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.c.k) + src);
    const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.c.v) + src);
    *reinterpret_cast<uint4*>(a.k + dst) = k;
    *reinterpret_cast<uint4*>(a.v + dst) = v;
  }
}

// CTAs that cover a call's rows: D / 8 lanes an item (K and V in turn), or four lanes for each of K and V
// in whole warps of eight items.
uint32_t row_ctas_of(const Rows& r, const Cache& c, bool t8) {
  const size_t items = (size_t)r.n_rows * c.Hkv;
  const size_t lanes = t8 ? (items + 7) / 8 * 64 : items * (c.D / 8);
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

constexpr uint32_t kSelWarps = kThreads / 32;
constexpr uint32_t kMine = 8;      // scores a thread holds in registers: 2048 blocks a CTA
constexpr uint32_t kKeys = 16384;  // and all of a CTA in shared memory
constexpr uint32_t kClose = 256;  // blocks scored again side by side
constexpr uint32_t kAhead = 8;     // blocks of a lane in flight
constexpr uint32_t kRing = kAhead * 2 * kThreads * 16;  // their bytes
constexpr uint32_t kSteps = 4;     // of eight bits each
constexpr uint32_t kInf = 0xff800000u;  // the key of +infinity

// Sums over the group's heads of q's positive and negative parts, eight dims a lane.
template <int D>
__device__ __forceinline__ void signed_sums(const Select& a, uint32_t r, uint32_t g, uint32_t l, float (&up)[8],
                                            float (&dn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) up[e] = dn[e] = 0.f;
  const uint32_t group = a.H / a.c.Hkv;
#pragma unroll 4
  for (uint32_t h = 0; h < group; ++h) {
    float x[8];
    unpack8(*reinterpret_cast<const uint4*>(a.q + ((size_t)r * a.H + g * group + h) * D + 8 * l), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      up[e] += x[e] > 0.f || x[e] != x[e] ? x[e] : 0.f;
      dn[e] += x[e] < 0.f ? x[e] : 0.f;
    }
  }
}

// Scores of blocks [j0, j1): s_j = sum_d Q+_d hi_jd + Q-_d lo_jd, with Q+ and Q- the sums over the
// group's heads of q's positive and negative parts: the sum over the heads of the largest q.k that a key
// inside the bounds could have. The bytes of the bounds bound it: a team of LPR lanes takes a block, each lane
// copies its own 32 bytes of kAhead blocks ahead (64 KB a CTA in flight, two CTAs an
// SM: 25.5 us for 16 sequences of 16K-64K tokens; four blocks in registers, 32 KB: 26.5 us; three CTAs of 80
// registers: 31.6 us) and waits for nobody else. Returns (in every thread) sum_d Q+_d max_j|hi_jd| + |Q-_d| max_j|lo_jd|, which bounds every block's sum
// of absolute terms; infinity where an infinity or NaN leaves no bound.
template <int D>
__device__ __forceinline__ float score_blocks(const Select& a, uint32_t r, uint32_t g, uint32_t seq, uint32_t n,
                                              uint32_t j0, uint32_t j1, float* out, uint4* ring, float* tmp) {
  constexpr int LPR = D / 8, PER = kThreads / LPR;
  const uint32_t l = threadIdx.x % LPR, team = threadIdx.x / LPR;
  const uint32_t mine = j0 + team < j1 ? (j1 - j0 - team + PER - 1) / PER : 0;  // blocks of this team
  const uint32_t all = (j1 - j0 + PER - 1) / PER;                               // and of the one with the most
  unsigned long long found = 0;  // where a block's bounds are, plus one: LPR blocks looked up at a time
  uint32_t have = 0;             // bit k % kAhead: the block there has bounds
  const auto fetch = [&](uint32_t k) {
    if (k % LPR == 0) {
      size_t row = 0;
      found = 0;
      if (k + l < mine) {
        if (cache_row(a.c, seq, (j0 + (k + l) * PER + team) << a.blk_shift, row)) found = (row >> a.blk_shift) + 1;
        else set_status(a.status, kStatusRange);
      }
    }
    const unsigned long long at = __shfl_sync(0xffffffffu, found, k % LPR, LPR);
    have &= ~(1u << (k % kAhead));
    if (at) {
      have |= 1u << (k % kAhead);
      const uint16_t* b = a.bounds + (((at - 1) * a.c.Hkv + g) * 2) * D + 8 * l;
      const uint32_t to = smem_addr(ring + (k % kAhead) * 2 * kThreads + threadIdx.x);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(b) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kThreads * 16), "l"(b + D) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float up[8], dn[8], mh[8], ml[8];
#pragma unroll 1
  for (uint32_t k = 0; k < kAhead; ++k) fetch(k);
  signed_sums<D>(a, r, g, l, up, dn);
#pragma unroll
  for (int e = 0; e < 8; ++e) mh[e] = ml[e] = 0.f;
  bool wild = false;
#pragma unroll 1
  for (uint32_t k = 0; k < all; ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const uint4* from = ring + (k % kAhead) * 2 * kThreads + threadIdx.x;
    const bool in = have >> (k % kAhead) & 1;
    float lo[8], hi[8], c[4] = {0.f, 0.f, 0.f, 0.f};  // four short chains: less rounding, no waiting
    unpack8(in ? from[0] : make_uint4(0u, 0u, 0u, 0u), lo);
    unpack8(in ? from[kThreads] : make_uint4(0u, 0u, 0u, 0u), hi);
    fetch(k + kAhead);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e & 1] = fmaf(up[e], hi[e], c[e & 1]);
      c[2 + (e & 1)] = fmaf(dn[e], lo[e], c[2 + (e & 1)]);
      mh[e] = fmaxf(mh[e], fabsf(hi[e]));
      ml[e] = fmaxf(ml[e], fabsf(lo[e]));
    }
    float s = (c[0] + c[1]) + (c[2] + c[3]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const uint32_t j = j0 + k * PER + team;
    if (in) wild |= !(fabsf(s) < INFINITY);
    if (k < mine && l == 0) __stcg(out + j, forced(a, j, n) ? INFINITY : in ? s : -INFINITY);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float most = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) most += up[e] * mh[e] - dn[e] * ml[e];
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) most += __shfl_xor_sync(0xffffffffu, most, o);
  if (wild || !(most < INFINITY)) most = INFINITY;
  most = warp_max(most);
  if (threadIdx.x % 32 == 0) tmp[threadIdx.x / 32] = most;
  __syncthreads();
  most = tmp[0];
  for (uint32_t w = 1; w < kSelWarps; ++w) most = fmaxf(most, tmp[w]);
  return most;
}

// A sum as two 32-bit numbers: TwoSum (Knuth) of hi and x, its error into lo.
__device__ __forceinline__ void add_exactly(float& hi, float& lo, float x) {
  const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
  hi = t;
}

// Block j's score again, by one warp (the same in every lane): sum over the heads of q hi where q is not negative
// and q lo where it is. A product of two bf16 values is exact in 32 bits unless it leaves their range.
// WIDE: in 64 bits. Otherwise as a sum of two 32-bit numbers, within 2^-37 of the sum of absolute terms (at most 40
// additions one after the other keep lo below 40 2^-24 of it, so each of lo's 40 roundings is below 40 2^-48), NaN
// where a product leaves the range: this GPU's 64-bit pipe takes 60 cycles an instruction, and a score there 5 us.
template <int D, bool WIDE>
__device__ double score_again(const Select& a, uint32_t r, uint32_t g, uint32_t seq, uint32_t j) {
  const uint32_t l = (threadIdx.x & 31) % (D / 8), group = a.H / a.c.Hkv;
  size_t row;
  if (!cache_row(a.c, seq, j << a.blk_shift, row)) return -INFINITY;
  const uint16_t* b = a.bounds + (((row >> a.blk_shift) * a.c.Hkv + g) * 2) * D + 8 * l;
  const uint16_t* q = a.q + ((size_t)r * a.H + g * group) * D + 8 * l;
  float lo[8], hi[8];
  unpack8(*reinterpret_cast<const uint4*>(b), lo);
  unpack8(*reinterpret_cast<const uint4*>(b + D), hi);
  if constexpr (WIDE) {
    double c[8] = {};
#pragma unroll 2
    for (uint32_t h = 0; h < group; ++h) {
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(q + (size_t)h * D), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] += (double)x[e] * (double)(x[e] < 0.f ? lo[e] : hi[e]);
    }
    double s = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s != s ? -(double)INFINITY : s > 1e300 ? 1e300 : s;  // infinity stays below the blocks that always come first
  } else {
    float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
    bool out = false;
#pragma unroll 4
    for (uint32_t h = 0; h < group; ++h) {
      float x[8];
      unpack8(*reinterpret_cast<const uint4*>(q + (size_t)h * D), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = x[e] < 0.f ? lo[e] : hi[e], p = __fmul_rn(x[e], y);
        out |= !(fabsf(p) < 1e30f) || (fabsf(p) < 1e-30f && x[e] != 0.f && y != 0.f);
        add_exactly(s[e & 3], t[e & 3], p);
      }
    }
#pragma unroll
    for (int e = 1; e < 4; ++e) {
      add_exactly(s[0], t[0], s[e]);
      t[0] = __fadd_rn(t[0], t[e]);
    }
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) {
      const float s2 = __shfl_xor_sync(0xffffffffu, s[0], o), t2 = __shfl_xor_sync(0xffffffffu, t[0], o);
      add_exactly(s[0], t[0], s2);
      t[0] = __fadd_rn(t[0], t2);
    }
    return __any_sync(0xffffffffu, out) ? (double)NAN : (double)s[0] + (double)t[0];
  }
}

// The scores of an item, spread over one CTA: warp w has blocks [w span, (w + 1) span), lane l every 32nd
// of them from l. Their order keys are in registers (the first kMine of a thread) for the counts,
// and in shared memory (the first kKeys of the item) for what runs once, whose code should be short;
// others are read again.
struct Scores {
  const float* s;
  uint32_t* keys;         // a thread reads what it wrote
  uint32_t n, base, end;  // base: this thread's first block; end: of its warp
  uint32_t key[kMine];

  __device__ __forceinline__ uint32_t load(uint32_t j) const { return j < end ? order_key(__ldcg(s + j)) : 0u; }
  __device__ void place(const float* scores, uint32_t count, uint32_t* shared) {
    const uint32_t span = (count + kThreads - 1) / kThreads * 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s = scores;
    keys = shared;
    n = count;
    end = (uint32_t)min((uint64_t)(warp + 1) * span, (uint64_t)count);
    base = warp * span + lane;
  }
  __device__ void take() {
#pragma unroll
    for (uint32_t i = 0; i < kMine; ++i) key[i] = load(base + 32 * i);
#pragma unroll
    for (uint32_t i = 0; i < kMine; ++i)
      if (base + 32 * i < min(end, kKeys)) keys[base + 32 * i] = key[i];
    for (uint32_t j = base + 32 * kMine; j < min(end, kKeys); j += 32) keys[j] = load(j);
  }
  // f(key) for this thread's blocks (a key of 0 stands for no block: a score's key is above it)
  template <typename F>
  __device__ __forceinline__ void count(F&& f) const {
    const uint32_t w0 = base - (threadIdx.x & 31);
#pragma unroll
    for (uint32_t i = 0; i < kMine; ++i)
      if (w0 + 32 * i < end) f(key[i]);
    for (uint32_t j = base + 32 * kMine; j < end; j += 32) f(j < kKeys ? keys[j] : load(j));
  }
  // f(block, key) in order; every lane of a warp is called equally often
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll 1
    for (uint32_t j0 = base - lane; j0 < end; j0 += 32) {
      const uint32_t j = j0 + lane;
      f(j, j >= end ? 0u : j < kKeys ? keys[j] : load(j));
    }
  }
};

// Sum over the CTA (the same in every thread); tmp: [2][kSelWarps], turn: alternates between calls.
__device__ __forceinline__ uint32_t cta_sum(uint32_t x, uint32_t* tmp, uint32_t& turn) {
  x = __reduce_add_sync(0xffffffffu, x);
  uint32_t* t = tmp + turn * kSelWarps;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) t[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (uint32_t w = 0; w < kSelWarps; ++w) x += t[w];
  return x;
}

// The n_close blocks whose keys lie in [klo, khi], scored again: the `need` largest of them (the lower
// index of equal ones) get the score +infinity, the others -infinity. Up to kClose of them are listed in close_j
// and ranked side by side, by two 32-bit numbers each, and where those leave the last that is in within 2^-36 most
// of the first that is out, by 64-bit ones.
template <int D>
__device__ __forceinline__ void decide(const Select& a, uint32_t r, uint32_t g, uint32_t seq, uint32_t n, size_t item,
                                       uint32_t klo, uint32_t khi, uint32_t n_close, uint32_t need, float most,
                                       uint32_t* tmp, const uint32_t* close_j) {
  __shared__ double close_t[kClose], s_edge[2];
  __shared__ bool s_nan;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* s = a.scores + item * a.nblk;
  if (n_close <= kClose) {
    if (tid == 0) s_nan = false;
    __syncthreads();
#pragma unroll 1
    for (int wide = 0; wide < 2; ++wide) {
      for (uint32_t i = warp; i < n_close; i += kSelWarps) {
        const uint32_t j = close_j[i];
        double x = INFINITY;
        if (!forced(a, j, n)) x = wide ? score_again<D, true>(a, r, g, seq, j) : score_again<D, false>(a, r, g, seq, j);
        if (lane == 0) close_t[i] = x;
        if (lane == 0 && x != x) s_nan = true;
      }
      __syncthreads();
      uint32_t rank = 0;
      if (tid < n_close) {  // as integers: the order of the bits
        const unsigned long long x = order_key(close_t[tid]);
        for (uint32_t i = 0; i < n_close; ++i) {
          const unsigned long long y = order_key(close_t[i]);
          rank += y > x || (y == x && close_j[i] < close_j[tid]);
        }
        if (rank == need - 1) s_edge[0] = close_t[tid];
        if (rank == need) s_edge[1] = close_t[tid];
      }
      __syncthreads();
      if (wide || (!s_nan && s_edge[0] - s_edge[1] > (double)most * 0x1p-36)) {
        if (tid < n_close) __stcg(s + close_j[tid], rank < need ? INFINITY : -INFINITY);
        break;
      }
    }
    __syncthreads();
    return;
  }
  const auto close = [&](uint32_t j) {
    if (j >= n) return false;
    const uint32_t k = order_key(__ldcg(s + j));
    return k >= klo && k <= khi;
  };
  const auto score = [&](uint32_t j) {
    return forced(a, j, n) ? (double)INFINITY : score_again<D, true>(a, r, g, seq, j);
  };
  // many equal or unbounded scores: all of them in 64 bits, then bisection of those bits
  double* t = a.exact + item * a.nblk;
  uint32_t turn = 0;
  __syncthreads();
  for (uint32_t j0 = warp * 32; j0 < n; j0 += kThreads) {
    unsigned m = __ballot_sync(0xffffffffu, close(j0 + lane));
    while (m) {
      const uint32_t j = j0 + (__ffs(m) - 1);
      m &= m - 1;
      const double x = score(j);
      if (lane == 0) __stcg(t + j, x);
    }
  }
  __syncthreads();
  const auto count = [&](unsigned long long from, bool above) {
    uint32_t c = 0;
    for (uint32_t j = tid; j < n; j += kThreads)
      if (close(j)) {
        const unsigned long long x = order_key(__ldcg(t + j));
        c += above ? x > from : x >= from;
      }
    return cta_sum(c, tmp, turn);
  };
  unsigned long long bar = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const unsigned long long c = bar | (1ull << bit);
    if (count(c, false) >= need) bar = c;
  }
  const uint32_t ties = need - count(bar, true);
  // the first `ties` of those on the bar, in index order: one warp counts
  if (warp == 0) {
    uint32_t seen = 0;
    for (uint32_t j0 = 0; j0 < n; j0 += 32) {
      const uint32_t j = j0 + lane;
      const bool c = close(j);
      const unsigned long long x = c ? order_key(__ldcg(t + j)) : 0ull;
      const unsigned eq = __ballot_sync(0xffffffffu, c && x == bar);
      const bool in = x > bar || (x == bar && seen + __popc(eq & ((1u << lane) - 1u)) < ties);
      if (c) __stcg(s + j, in ? INFINITY : -INFINITY);
      seen += __popc(eq);
    }
  }
  __syncthreads();
}

// Which blocks the exact scores choose, given 32-bit ones. Every s_j is within E of the exact t_j
// (E = (group + 13) 2^-24 most + (D + 1) 2^-149: group - 1 additions in Q+-, 4 multiply-adds and 2 + 5 additions round
// one after the other, and the rounding of `most` itself is covered by the rest; where products leave 32 bits at the
// lower end, each of the 2 D multiply-adds loses up to 2^-150 besides, and so may E). The K-th largest t is then within E
// of the K-th largest s, T: s_j > T + 2E is in, s_j < T - 2E is out, and only what lies between is scored again. T is
// found from the scores' bits, eight a step, until a step leaves exactly K. This part is latency (one CTA an item, a
// few barriers, code that runs once): bisection and a barrier for each count took 0.6 us more of a
// selection's 8.5 (64K tokens), keys from shared memory alone, with shorter code, 0.4 us more.
template <int D>
__device__ void choose(const Select& a, uint32_t r, uint32_t g, uint32_t seq, uint32_t n, size_t item, float most) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t tmp[2 * kSelWarps], range[3 * kSelWarps], close_j[kClose];
  __shared__ __align__(16) uint32_t s_bins[kSteps][256];
  const uint32_t K = a.n_select, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* out = a.blocks + item * K;
  uint32_t turn = 0;
  Scores sc;
  sc.place(a.scores + item * a.nblk, n, keys);
  sc.take();
  for (uint32_t i = threadIdx.x; i < kSteps * 256; i += kThreads) s_bins[0][i] = 0;
  // the finite scores' range: the first step over all 32 bits would only find it
  uint32_t low = 0xffffffffu, high = 0, n_forced = 0;
  sc.count([&](uint32_t k) {
    low = k ? min(low, k) : low;
    high = k < kInf ? max(high, k) : high;
    n_forced += k >= kInf;
  });
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    range[warp] = low;
    range[kSelWarps + warp] = high;
  }
  n_forced = cta_sum(n_forced, tmp, turn);
  uint32_t at_low = n, at_high = n_forced;
  for (uint32_t w = 0; w < kSelWarps; ++w) {
    low = min(low, range[w]);
    high = max(high, range[kSelWarps + w]);
  }
  ++high;  // below kInf: only what is infinite is from here up
  if (n_forced >= K) {
    low = kInf;
    high = kInf + 1;
    at_low = n_forced;
  }
  // low: the largest tried value with at least K keys from it up (at_low); high: the smallest with fewer (at_high).
  // A step cuts what lies between into 256: one count of all bins where a bisection takes eight
  for (uint32_t step = 0; step < kSteps && at_low != K && high - low > 1; ++step) {
    const uint32_t bits = 32 - __clz(high - low - 1), shift = bits > 8 ? bits - 8 : 0;
    uint32_t* bins = s_bins[step];
    sc.count([&](uint32_t k) {
      if (k >= low && k < high) atomicAdd(bins + ((k - low) >> shift), 1u);
    });
    __syncthreads();
    // every warp for itself: eight bins a lane, the keys above them, and the bin that reaches K
    const uint4 c0 = reinterpret_cast<const uint4*>(bins)[2 * lane], c1 = reinterpret_cast<const uint4*>(bins)[2 * lane + 1];
    const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    uint32_t up = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7])), mine = up;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_down_sync(0xffffffffu, up, o);
      up += lane + o < 32 ? x : 0u;
    }
    uint32_t above = at_high + up - mine, b = 0, to = 0;
    const unsigned here = __ballot_sync(0xffffffffu, above < K && above + mine >= K);
    bool found = false;
#pragma unroll
    for (int e = 7; e >= 0; --e)
      if (!found) {
        to = above + c[e];
        found = to >= K;
        if (found) b = 8 * lane + e;
        else above = to;
      }
    const int src = __ffs(here) - 1;
    at_high = __shfl_sync(0xffffffffu, above, src);
    at_low = __shfl_sync(0xffffffffu, to, src);
    b = __shfl_sync(0xffffffffu, b, src);
    high = (uint32_t)min((uint64_t)high, low + ((uint64_t)(b + 1) << shift));
    low += b << shift;
  }
  uint32_t kth = 0xffffffffu;  // the smallest key from low up: the K-th largest's
  sc.count([&](uint32_t k) { kth = k >= low ? min(kth, k) : kth; });
  kth = __reduce_min_sync(0xffffffffu, kth);
  if (lane == 0) range[2 * kSelWarps + warp] = kth;
  __syncthreads();
  for (uint32_t w = 0; w < kSelWarps; ++w) kth = min(kth, range[2 * kSelWarps + w]);
  const float T = key_value(kth), E = fmaf((float)(a.H / a.c.Hkv + 13) * 0x1p-24f, most, (D + 1) * 0x1p-149f);
  uint32_t klo = 1, khi = 0xffffffffu;  // keys above khi are in, below klo out
  if (E < INFINITY) {
    klo = order_key(isinf(T) ? T : __fadd_rd(T, -2.f * E));
    khi = order_key(isinf(T) ? T : __fadd_ru(T, 2.f * E));
  }
  uint32_t c1 = 0, c2 = 0;
  sc.count([&](uint32_t k) {
    c1 += k > khi;
    c2 += k >= klo && k <= khi;
  });
  // over the CTA, and over the warps before this one: where its blocks go in the list
  c1 = __reduce_add_sync(0xffffffffu, c1);
  c2 = __reduce_add_sync(0xffffffffu, c2);
  if (lane == 0) {
    tmp[warp] = c1;
    tmp[kSelWarps + warp] = c2;
  }
  __syncthreads();
  uint32_t n_sure = 0, n_close = 0, at = 0;
#pragma unroll
  for (uint32_t w = 0; w < kSelWarps; ++w) {
    const uint32_t x = tmp[w], y = tmp[kSelWarps + w];
    at += w < warp ? x + y : 0u;
    n_sure += x;
    n_close += y;
  }
  const uint32_t need = K - n_sure;
  uint32_t cut = klo;  // in from this key up
  if (n_close != need) {
    if (n_close <= kClose) {  // a list of them, in any order
      // counted in `range`, which nobody reads any more (another warp may still read the sums in tmp)
      if (threadIdx.x == 0) range[0] = 0;
      __syncthreads();
      sc.each([&](uint32_t j, uint32_t k) {
        if (k >= klo && k <= khi) close_j[atomicAdd(range, 1u)] = j;
      });
      __syncthreads();
    }
    decide<D>(a, r, g, seq, n, item, klo, khi, n_close, need, most, tmp, close_j);
    sc.take();
    cut = min(khi, kInf - 1) + 1;
    uint32_t n_in = 0;
    sc.count([&](uint32_t k) { n_in += k >= cut; });
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    __syncthreads();
    if (lane == 0) tmp[warp] = n_in;
    __syncthreads();
    at = 0;
    for (uint32_t w = 0; w < warp; ++w) at += tmp[w];
  }
  // in index order: a warp's blocks are neighbours, so places come from ballots and the counts of the warps before
  sc.each([&](uint32_t j, uint32_t k) {
    const unsigned m = __ballot_sync(0xffffffffu, k >= cut);
    const uint32_t to = at + __popc(m & ((1u << lane) - 1u));
    if (k >= cut && to < K) out[to] = (int32_t)j;
    at += __popc(m);
  });
}

// CTA x of a (row, kv-head) scores the x-th `part` of its blocks; the last of them to finish chooses.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const __grid_constant__ Select a, uint32_t part) {
  extern __shared__ __align__(16) uint32_t keys[];  // the bounds in flight, then choose()'s keys
  __shared__ float tmp[kSelWarps];
  __shared__ uint32_t s_last;
  pdl_wait();
  pdl_launch();
  const uint32_t r = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  uint32_t seq, pos;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
  if (kind != kRowOk) {
    if (kind == kRowBad) set_status(a.status, kStatusRange);
    return;
  }
  const uint32_t n = (pos >> a.blk_shift) + 1, K = a.n_select;
  const size_t item = (size_t)r * a.c.Hkv + g;
  if (n <= K) {  // every block is taken
    if (blockIdx.x == 0)
      for (uint32_t i = tid; i < K; i += kThreads) {
        size_t row;
        if (i < n && !cache_row(a.c, seq, i << a.blk_shift, row)) set_status(a.status, kStatusRange);
        a.blocks[item * K + i] = i < n ? (int32_t)i : -1;
      }
    return;
  }
  const uint32_t parts = (n + part - 1) / part;
  if (blockIdx.x >= parts) return;
  float* most = a.most + item * gridDim.x;
  float m = score_blocks<D>(a, r, g, seq, n, blockIdx.x * part, min(n, (blockIdx.x + 1) * part),
                            a.scores + item * a.nblk, reinterpret_cast<uint4*>(keys), tmp);
  __syncthreads();
  if (parts > 1) {
    if (tid == 0) {
      // the barrier has put the CTA's scores before this; the count's release and acquire put them before the
      // last one's reads
      __stcg(most + blockIdx.x, m);
      const uint32_t had = count_up(a.tickets + item);
      s_last = had == parts - 1;
      if (had > parts - 1) set_status(a.status, kStatusInvalid);
      if (had == parts - 1) a.tickets[item] = 0;
    }
    __syncthreads();
    if (!s_last) return;
    m = 0.f;
    for (uint32_t p = tid % 32; p < parts; p += 32) m = fmaxf(m, __ldcg(most + p));
    m = warp_max(m);
  }
  choose<D>(a, r, g, seq, n, item, m);
}

}  // namespace

#define Q35C_BY_DIM(D, call)                 \
  switch (D) {                               \
    case 64: { call(64); } break;            \
    case 128: { call(128); } break;          \
    case 256: { call(256); } break;          \
    default: return cudaErrorInvalidValue;   \
  }

// Whether a CTA folds a block's bounds, or a team of D / 8 lanes. A CTA ends a block sooner, teams keep more blocks in
// flight. us of an append of 4 heads of 256 (Turbo8 | bf16), by a CTA and by teams:
//             300 rows                2 688 rows in 3 prompts   32 768 rows
//   block 16  3.6, 4.0 | 3.4, 4.1     12.0, 6.9 | 9.0, 7.4      106, 55 | 75, 45
//         32  3.6, 4.2 | 3.7, 5.2     9.5, 8.0 | 7.9, 10.1      73, 54 | 56, 46
//         64  3.6, 5.4 | 4.0, 8.5     8.5, 10.0 | 8.3, 13.0     64, 54 | 49, 50
//        128  3.8, 8.4 | 5.3, 15.0    7.5, 13.8 | 9.1, 19.2     59, 58 | 47, 63
// so by a CTA from 128 tokens on, and from 32 on while such CTAs are few (folds: 40, 336 and 4 096 at blocks of 32).
bool fold_wide(uint32_t blk_shift, uint32_t folds) { return blk_shift >= 7 || (blk_shift >= 5 && folds <= 512); }

cudaError_t append(const Append& args, cudaStream_t st) {
  Append a = args;
  const bool t8 = a.c.ks != nullptr;
  const uint32_t rows = row_ctas_of(a.r, a.c, t8);
  const uint32_t span = a.r.row_start ? 1u << a.blk_shift : 1u;  // rows of a bounds CTA: about one block's
  const uint32_t folds = (a.r.n_rows + span - 1) / span * a.c.Hkv;
  a.wide_bounds = fold_wide(a.blk_shift, folds);
  const uint32_t teams = a.wide_bounds ? 1 : kThreads / (a.c.D / 8);
  const uint32_t bounds = a.bounds ? (folds + teams - 1) / teams : 0, grid = rows + bounds;
  uint32_t shift = 0;
  while (bounds && (grid / bounds) >> (shift + 1)) ++shift;
#define CALL(DD)                                                               \
  return t8 ? launch_early(append_kernel<DD, true>, dim3(grid), kThreads, 0, st, a, bounds, shift, span)   \
            : launch_early(append_kernel<DD, false>, dim3(grid), kThreads, 0, st, a, bounds, shift, span)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
}

cudaError_t read(const Read& a, cudaStream_t st) {
  const bool t8 = a.c.ks != nullptr;
  const uint32_t grid = row_ctas_of(a.r, a.c, t8);
#define CALL(DD)                                                   \
  return t8 ? launch_early(read_kernel<DD, true>, dim3(grid), kThreads, 0, st, a)     \
            : launch_early(read_kernel<DD, false>, dim3(grid), kThreads, 0, st, a)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
}

cudaError_t select_attributes() {
  const auto allow = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)std::max(kKeys * 4, kRing)) == cudaSuccess;
  };
  return allow(select_kernel<64>) && allow(select_kernel<128>) && allow(select_kernel<256>) ? cudaSuccess
                                                                                            : cudaGetLastError();
}

cudaError_t select(const Select& a, cudaStream_t st) {
  // Blocks of a CTA: whole passes of the teams, and no more CTAs than a.ctas if the sequences were all as long as
  // the capacity (parts of one size, so that a long sequence is not the last to finish)
  const uint32_t pass = kThreads / (a.c.D / 8) * 4, items = a.r.n_rows * a.c.Hkv;
  const uint32_t parts = std::max(1u, std::min((a.nblk + pass - 1) / pass, a.ctas / items));
  const uint32_t part = ((a.nblk + parts - 1) / parts + pass - 1) / pass * pass;
  const dim3 grid((a.nblk + part - 1) / part, a.c.Hkv, a.r.n_rows);
  const uint32_t smem = std::max(std::min(a.nblk, kKeys) * 4, kRing);
#define CALL(DD) return launch_early(select_kernel<DD>, grid, kThreads, smem, st, a, part)
  Q35C_BY_DIM(a.c.D, CALL)
#undef CALL
}

}  // namespace q35c
