// Attention of new tokens over a KV cache (cache_ops.h): one launch for any number of
// rows, split over the cache's length and joined.
//
// An item is a kv-head of one row, or of as many neighbouring rows of a sequence as
// its group of q-heads leaves room for in eight columns (a group of 1: 8 rows, of 4: 2;
// only without a list of blocks, which every row has of its own): softmax(q K^T /
// sqrt D) V for the columns, (row, q-head) pairs. The bytes of K and V bound it: each is read once
// for all columns, by asynchronous copies into shared memory, and the products run on
// matrix instructions with the tokens as their rows (M = 16) and the columns as
// theirs (N = 8), one instruction per 16 tokens x 16 dims:
//   S^T [16 tokens x 8] += K [16 x 16 dims] Q^T [16 dims x 8], D / 16 times;
//   O^T [16 dims x 8] += V^T [16 dims x 16 tokens] P^T [16 tokens x 8], D / 16 times.
// A warp works alone: it has its own ring of K and V tiles of 16 tokens, its own running
// maximum, sum and output, and meets the other warps only at the end of an item.
//
// The work of a call is the line of all items' 16-token tiles; every CTA takes an equal
// stretch of it, whatever the sequences' lengths. An item that lies in several CTAs is joined by
// the last of them to finish, in the order of the CTAs, so equal calls give equal bits.
//
// Roundings. bf16 K, V and q enter the products exactly, the weights P as hi + lo bf16
// (2^-16 relative). Turbo8 codes enter as f16 (exact); the K scales multiply the fp32
// products of their 16 dims; the rotated q enters as hi + lo f16 over the power of two of
// its largest value (2^-22 of a value or 2^-25 of the largest, where the rotation's own
// sums end too).
// A token's V scales enter as f16 over 2^E, E the exponent of the token's largest (exact
// down to 2^-17 of that one, lost below 2^-25), and E goes into the exponent of the token's
// weight: the weights that multiply V are 2^((x - m) + E - M), M the running maximum of
// (x - m) + E, so a token counts by what it adds and not by its neighbours' sizes, and E is
// added where large scores have cancelled. m, which the softmax's sum refers to, follows the
// scores only when one lies 32 octaves above it: 32 bits have room for that, and the lanes
// exchange one maximum a tile (128K tokens: 68 us; one power of two a tile, which lost
// tokens beside larger ones: 64).
// Those weights are rounded to f16 (2^-11), up to 2^13 so that f16 holds 2^-27 of the largest
// in full and what lies 2^-38 below is lost, and rounded again with the scale (2^-11): next
// to the codes' own 2^-4 and the output's 2^-8 these are small (error against 64 bits 0.00171
// at 128K, of fp32 weights 0.00169), and a second f16 for their rest (2^-21) takes 73 us.
#include "cache_ops.cuh"
#include "turbo8.cuh"

#include <algorithm>

namespace q35c {
using namespace q35;
namespace {

constexpr int kWarps = 8;  // of a CTA, one CTA an SM (16 warps of 128 registers for Turbo8: 84 us where 8 took 73)
constexpr int kAttnThreads = 32 * kWarps;

constexpr int kMl = 48;  // a warp's maxima, sums and (T8) maxima of V's weights, 16 columns each
constexpr float kUp = 13.f;  // T8: the largest weight of V is 2^kUp
constexpr float kFar = 32.f;  // T8: how far a score may lie above what the sum refers to

// A ring slot: K or V of 16 tokens. Rows are padded by 16 bytes, which puts eight rows'
// 16-byte pieces in different banks.
template <int D, bool T8>
struct Slot {
  static constexpr int row = T8 ? D + 16 : 2 * D + 16;
  static constexpr int scales = T8 ? D / 16 * 2 : 0;  // a token's scales
  static constexpr int bytes = 16 * (row + scales);
  // slots of a warp, what shared memory holds up to 4 (K and V of two tiles)
  static constexpr int n = D == 256 && !T8 ? 3 : 4;
};
// Shared memory of a CTA: the rings (reused to join the warps), Q's fragments and (T8)
// the rotated q, the warps' maxima and sums, T8's transposed V scales, then the rows' first tiles.
template <int D, int NT, bool T8>
struct Smem {
  using S = Slot<D, T8>;
  static constexpr int ring = kWarps * S::n * S::bytes;
  static constexpr int join = kWarps * 8 * NT * (D + 4) * 4;
  static constexpr int weights = 24576;  // the parts' weights, behind their sums
  static constexpr int parts = weights + 8 * NT * (int)kMaxCtas * 4;
  static constexpr int big = ring > join ? (ring > parts ? ring : parts) : join > parts ? join : parts;
  static constexpr int qf = big;                                    // fragments, 8 or (T8) 16 bytes a lane
  static constexpr int qs = qf + (D / 16) * NT * 32 * (T8 ? 16 : 8);  // [8 NT][D] fp32
  static constexpr int ml = qs + (T8 ? 8 * NT * D * 4 : 0);           // [warps + 1][3][16]
  static constexpr int vsc = ml + (kWarps + 1) * kMl * 4;
  static constexpr int scale_row = D / 8 + 4;  // words, padded
  static constexpr int misc = vsc + (T8 ? kWarps * scale_row * 16 : 0);
  static constexpr int first = misc + 256;  // [n_rows + 1]
  static_assert(kWarps <= 16 && 2 * kMaxSeqs * 4 + 4 <= big, "misc, the rows' places");
  // misc: words 0-15 and 40-55 the warps' sums, 16 a flag, 20-35 (T8) q's powers of two
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {  // the low 16 bits' codes
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
  return h2;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to 2^-22 relative; 0 below 2^-126
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]
// The maximum over the eight lanes of a column.
__device__ __forceinline__ float col_max(float x) {
#pragma unroll
  for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
  return x;
}
// What is subtracted for a maximum: 0 where there is nothing yet.
__device__ __forceinline__ float finite_or_0(float mx) { return mx == -INFINITY ? 0.f : mx; }
__device__ __forceinline__ float rescale(float from, float to) { return from == -INFINITY ? 0.f : ex2(from - to); }

// One item's stretch in a CTA: rows row .. row + rows - 1, the last at position pos.
struct Segment {
  uint32_t row, rows, g, seq, pos;
  uint32_t tiles;   // the item's tiles
  uint32_t t0, t1;  // this CTA's
  size_t row0;         // contiguous: the sequence's first cache row
  const int32_t* tab;  // paged: its table
};

// The first token of a tile and where its tokens lie: rows of tokens 0-7 and 8-15 (a page holds at least 8
// tokens), and how many tokens the item's last row sees from the tile's first on, up to 32.
struct Tile {
  size_t row[2];
  uint32_t token, seen;
  bool in[2];
};
__device__ __forceinline__ Tile lane_of(const Tile& t, uint32_t src) {
  Tile x;
  x.row[0] = __shfl_sync(0xffffffffu, (unsigned long long)t.row[0], src);
  x.row[1] = __shfl_sync(0xffffffffu, (unsigned long long)t.row[1], src);
  x.token = __shfl_sync(0xffffffffu, t.token, src);
  const uint32_t f = __shfl_sync(0xffffffffu, t.seen | (t.in[0] ? 256u : 0u) | (t.in[1] ? 512u : 0u), src);
  x.seen = f & 255u;
  x.in[0] = f & 256u;
  x.in[1] = f & 512u;
  return x;
}

constexpr uint32_t kNo0 = 64, kNo1 = 128;  // tokens 0-7, 8-15 lie in no block of the pool

template <int D, int NT, bool T8>
struct Attention {
  using S = Slot<D, T8>;
  using M = Smem<D, NT, T8>;
  const Attend& a;
  uint8_t* sm;
  uint32_t warp, lane, group;
  uint32_t pack;  // the most rows of an item
  uint32_t ring;  // this warp's slots
  float m[NT][2], l[NT][2], o[D / 16][NT][4];  // l refers to m, the scores' maximum (T8: or up to kFar below it)
  float mv[NT][2];  // T8: the maximum of V's weights, relative to m, which o refers to
  uint32_t later[NT][2];  // tokens of the item's last row that this column's row does not see
  float qscale[NT][2];  // log2(e) / sqrt(D), with T8's power of two of q

  // ---- where a tile's tokens are
  __device__ Tile tile(const Segment& s, uint32_t t) const {
    Tile x;
    x.token = x.seen = 0;
    x.in[0] = x.in[1] = false;
    x.row[0] = x.row[1] = 0;
    if (t >= s.t1) return x;
    uint64_t token = (uint64_t)t * 16;
    if (a.blocks) {
      const uint32_t per = a.blk_shift - 4;
      const int32_t b = a.blocks[((size_t)s.row * a.c.Hkv + s.g) * a.n_blocks + (t >> per)];
      if (b < 0) return x;
      token = ((uint64_t)(uint32_t)b << a.blk_shift) + (t & ((1u << per) - 1u)) * 16;
    }
    if (token > s.pos) return x;
    x.token = (uint32_t)token;
    x.seen = min(32u, s.pos - x.token + 1);
    if (s.tab) {
      const uint32_t sh = a.c.bt_shift, mask = (1u << sh) - 1u, t8 = x.token + (x.seen > 8 ? 8 : 0);
      const uint32_t b0 = (uint32_t)s.tab[x.token >> sh], b1 = (uint32_t)s.tab[t8 >> sh];
      x.in[0] = b0 < a.c.num_blocks;
      x.in[1] = b1 < a.c.num_blocks;
      x.row[0] = ((size_t)b0 << sh) | (x.token & mask);
      x.row[1] = ((size_t)b1 << sh) | ((x.token + 8) & mask);
      if (!x.in[0] || !x.in[1]) set_status(a.status, kStatusRange);
    } else {
      x.in[0] = x.in[1] = true;
      x.row[0] = s.row0 + x.token;
      x.row[1] = x.row[0] + 8;
    }
    return x;
  }

  // ---- K (p = 0) or V of a tile into a slot. Tokens no row sees read as zero; so do the V rows of
  // tokens that only later rows of the item see (add_tail): their weight is 0 in the earlier rows' columns,
  // and 0 times an infinity would spoil them. Their V scales are loaded: add_tail's weights need the exponents.
  __device__ void load(const Segment& s, const Tile& x, int p, uint32_t slot) const {
    const uint32_t last = s.pos + 1 - (p ? s.rows - 1 : 0);  // tokens below it
    const uint32_t seen = x.seen ? min(16u, last > x.token ? last - x.token : 0u) : 0u;
    constexpr int C = (T8 ? D : 2 * D) / 16, R = 32 / C > 0 ? 32 / C : 1;  // 16-byte pieces of a row, rows a pass
    const uint8_t* base = p ? a.c.v : a.c.k;
    const uint32_t stride = a.c.Hkv * D * (T8 ? 1 : 2), r0 = lane / C, c = lane % C;
    const uint32_t dst = ring + slot * S::bytes, to = dst + r0 * S::row + c * 16;
    const uint32_t within = r0 * stride + s.g * D * (T8 ? 1 : 2) + c * 16;
    const uint8_t* p0 = base + x.row[0] * stride + within;
    const uint8_t* p1 = base + x.row[1] * stride + within;
    const bool full = seen == 16 && x.in[0] && x.in[1];
    if (full) {
#pragma unroll
      for (int i = 0; i < 8 / R; ++i) {
        cp16(to + i * R * S::row, p0);
        cp16(to + (8 + i * R) * S::row, p1);
        p0 += R * stride;
        p1 += R * stride;
      }
    } else {  // the last tile of an item
#pragma unroll 1
      for (int i = 0; i < 16 / R; ++i) {
        const uint32_t r = i * R + r0;
        const bool in = r < seen && (r & 8 ? x.in[1] : x.in[0]);
        const uint8_t* src = r & 8 ? p1 + (i * R - 8) * (int)stride : p0 + i * R * stride;
        cp16(to + i * R * S::row, in ? src : base, in);
      }
    }
    if constexpr (T8) {
      constexpr int SB = S::scales, P = SB >= 16 ? SB / 16 : 1;  // pieces of a token's scales
      const uint8_t* sbase = reinterpret_cast<const uint8_t*>(p ? a.c.vs : a.c.ks);
      const uint32_t r = lane / P, c2 = lane % P;
      if (r < 16) {
        const bool in = r < x.seen && (r & 8 ? x.in[1] : x.in[0]);
        const size_t row = (r & 8 ? x.row[1] : x.row[0]) + (r & 7);
        const uint8_t* src = sbase + (row * a.c.sstride + s.g * (D / 16)) * 2 + c2 * 16;
        const uint32_t sto = dst + 16 * S::row + r * SB + c2 * 16;
        if constexpr (SB >= 16) cp16(sto, in ? src : sbase, in);
        else cp8(sto, in ? src : sbase, in);
      }
    }
  }

  // ---- q of an item as B fragments, [k-step][n-tile][lane]; column c: row c / group, head c % group
  __device__ __forceinline__ const uint16_t* q_at(const Segment& s, uint32_t col) const {
    return a.q + ((size_t)(s.row + col / group) * a.H + s.g * group + col % group) * D;
  }
  // What a thread holds of q between its loads, which go ahead of the first copies, and their use.
  static constexpr int kFrag = (D / 16) * NT * 32;  // fragments
  static constexpr int kQ = T8 ? (8 * NT * (D / 8) + kAttnThreads - 1) / kAttnThreads
                               : (kFrag + kAttnThreads - 1) / kAttnThreads;
  struct QRegs {
    uint4 u[kQ];  // T8: eight elements; bf16: a fragment's two words
  };
  __device__ QRegs fetch_q(const Segment& s) const {
    const uint32_t cols = group * s.rows;
    QRegs q;
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
      const uint32_t i = threadIdx.x + k * kAttnThreads;
      q.u[k] = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (T8) {
        const uint32_t h = i / (D / 8), c = i % (D / 8);
        if (h < cols) q.u[k] = *reinterpret_cast<const uint4*>(q_at(s, h) + 8 * c);
      } else {
        const uint32_t ln = i & 31, nt = (i >> 5) % NT, kk = (i >> 5) / NT, col = 8 * nt + ln / 4, c = ln % 4;
        if (i < kFrag && col < cols) {
          const uint16_t* x = q_at(s, col) + 16 * kk + 2 * c;
          q.u[k].x = *reinterpret_cast<const uint32_t*>(x);
          q.u[k].y = *reinterpret_cast<const uint32_t*>(x + 8);
        }
      }
    }
    return q;
  }
  __device__ void put_q(const QRegs& q) {
    constexpr int LPR = D / 8;
    float* qs = reinterpret_cast<float*>(sm + M::qs);
    int* qe = reinterpret_cast<int*>(sm + M::misc) + 20;
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
      const uint32_t i = threadIdx.x + k * kAttnThreads;
      if constexpr (T8) {
        if (i < 8 * NT * LPR) {  // whole warps
          const uint32_t h = i / LPR, c = i % LPR;
          float x[8];
          unpack8(q.u[k], x);
          wht8<LPR>(x, lane);
          float mx = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
          for (int w = 1; w < LPR; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          // the largest |x| 2^-e is in [1, 2): no larger than it need be, so that products with keys of up to
          // 2^118 stay in 32 bits
          const int e2 = min(max((int)((__float_as_uint(mx) >> 23) & 255) - 127, -126), 126);
          const float f = mx > 0.f ? pow2(-e2) : 1.f;
          if (c == 0) qe[h] = mx > 0.f ? e2 : 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) qs[h * D + 8 * c + e] = x[e] * f;
        }
      } else {
        if (i < kFrag) *reinterpret_cast<uint2*>(sm + M::qf + i * 8) = make_uint2(q.u[k].x, q.u[k].y);
      }
    }
    __syncthreads();
    if constexpr (T8) {
      for (uint32_t i = threadIdx.x; i < kFrag; i += kAttnThreads) {
        const uint32_t ln = i & 31, nt = (i >> 5) % NT, kk = (i >> 5) / NT, c = ln % 4;
        // a code word of 4 dims feeds both halves of the k-step: dims 4c, 4c+1 | 4c+2, 4c+3
        const float4 x = *reinterpret_cast<const float4*>(qs + (8 * nt + ln / 4) * D + 16 * kk + 4 * c);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float u = j ? x.z : x.x, v = j ? x.w : x.y;
          hi[j] = pack_f16(u, v);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
          lo[j] = pack_f16(u - f.x, v - f.y);
        }
        *reinterpret_cast<uint4*>(sm + M::qf + i * 16) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
      }
      __syncthreads();
    }
    const float sl2 = 1.4426950408889634f / sqrtf((float)D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) qscale[nt][j] = T8 ? sl2 * pow2(qe[8 * nt + 2 * (lane % 4) + j]) : sl2;
  }

  // ---- one tile: scores from its K slot
  __device__ void scores(uint32_t slot, float (&s)[NT][4]) const {
    const uint32_t k = ring + slot * S::bytes, r8 = lane & 7, q4 = lane >> 3;
    const uint32_t at = k + (r8 + (q4 & 1) * 8) * S::row + (q4 >> 1) * 16;
    if constexpr (T8) {
      const uint8_t* sc = sm + (k - smem_addr(sm)) + 16 * S::row;
      const uint32_t r = lane >> 2;
      uint32_t s0[D / 32], s1[D / 32];  // the scales of tokens r and r + 8, two a word
#pragma unroll
      for (int i = 0; i < D / 32; i += 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(sc + r * S::scales + i * 4);
        const uint2 v = *reinterpret_cast<const uint2*>(sc + (r + 8) * S::scales + i * 4);
        s0[i] = u.x;
        s0[i + 1] = u.y;
        s1[i] = v.x;
        s1[i + 1] = v.y;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
      for (int g2 = 0; g2 < D / 32; ++g2) {  // two groups of 16 dims
        uint32_t w[4];
        ldsm4(w, at + g2 * 32);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w0 = w[2 * j], w1 = w[2 * j + 1];  // tokens 0-7, 8-15
          const uint32_t A[4] = {e4m3_to_f16x2(w0), e4m3_to_f16x2(w1), e4m3_to_f16x2(w0 >> 16), e4m3_to_f16x2(w1 >> 16)};
          const float f0 = j ? bf16hi(s0[g2]) : bf16lo(s0[g2]), f1 = j ? bf16hi(s1[g2]) : bf16lo(s1[g2]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 b = *reinterpret_cast<const uint4*>(sm + M::qf + (((2 * g2 + j) * NT + nt) * 32 + lane) * 16);
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma<true>(c, A, b.x, b.y);
            mma<true>(c, A, b.z, b.w);
            s[nt][0] = fmaf(c[0], f0, s[nt][0]);
            s[nt][1] = fmaf(c[1], f0, s[nt][1]);
            s[nt][2] = fmaf(c[2], f1, s[nt][2]);
            s[nt][3] = fmaf(c[3], f1, s[nt][3]);
          }
        }
      }
    } else {
      float c[2][NT][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[j][nt][i] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t A[4];
        ldsm4(A, at + kk * 32);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 b = *reinterpret_cast<const uint2*>(sm + M::qf + ((kk * NT + nt) * 32 + lane) * 8);
          mma<false>(c[kk & 1][nt], A, b.x, b.y);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = c[0][nt][i] + c[1][nt][i];
    }
  }

  // ---- T8: a tile's V scales, each token's over 2^e (e: the exponent of its largest), as f16 pairs of tokens: word
  // (c, g, h) has tokens 2c + 8h and 2c + 8h + 1 of dims group g; those of tokens from `all` on, which not every
  // row of the item sees, are 0. e0, e1: of the tokens of this lane's scores.
  __device__ void v_scales(uint32_t slot, uint32_t all, int& e0, int& e1) const {
    const uint8_t* sc = sm + (ring - smem_addr(sm)) + slot * S::bytes + 16 * S::row;
    uint16_t* t = reinterpret_cast<uint16_t*>(sm + M::vsc + warp * M::scale_row * 16);
    constexpr int PER = D / 32;  // scales a lane: half a token's
    const uint32_t tok = lane >> 1, g0 = (lane & 1) * PER;
    float f[PER], mx = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(sc + tok * S::scales + (g0 + i) * 2);
      f[i] = bf16lo(u);
      f[i + 1] = bf16hi(u);
      mx = fmaxf(mx, fmaxf(fabsf(f[i]), fabsf(f[i + 1])));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126);
    const float k = pow2(-e);
    uint16_t* to = t + ((tok & 7) >> 1) * M::scale_row * 2 + g0 * 4 + (tok >> 3) * 2 + (tok & 1);
#pragma unroll
    for (int i = 0; i < PER; ++i) to[i * 4] = tok < all ? __half_as_ushort(__float2half_rn(f[i] * k)) : 0;
    e0 = __shfl_sync(0xffffffffu, e, lane >> 2 << 1);
    e1 = __shfl_sync(0xffffffffu, e, (lane >> 2 << 1) + 16);
    __syncwarp();
  }

  // ---- one tile: weights from the scores, then the output from its V slot; the last row sees `seen` tokens
  // from the tile's first on, those in a block outside the pool left out. e0, e1: v_scales'
  __device__ __forceinline__ void accumulate(uint32_t slot, float (&s)[NT][4], uint32_t seen, uint32_t rows, int& e0,
                                             int& e1) {
    const uint32_t r = lane >> 2, seen0 = seen & kNo0 ? 0 : seen & 63u, seen1 = seen & kNo1 ? 0 : seen & 63u;
    if constexpr (T8) v_scales(slot, max(seen & 63u, rows - 1) - (rows - 1), e0, e1);
    uint32_t ph[NT][2], pl[NT][2];
    bool grew = false, far = false;
    float corr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[nt][j] = r + later[nt][j] >= seen0 ? -INFINITY : s[nt][j] * qscale[nt][j];
        s[nt][2 + j] = r + 8 + later[nt][j] >= seen1 ? -INFINITY : s[nt][2 + j] * qscale[nt][j];
        far |= fmaxf(s[nt][j], s[nt][2 + j]) > m[nt][j] + kFar;
      }
    if constexpr (T8) {
      if (__any_sync(0xffffffffu, far))  // the first tile, as a rule
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mx = col_max(fmaxf(s[nt][j], s[nt][2 + j])), down = m[nt][j] - mx;
            if (mx > m[nt][j] + kFar) {
              l[nt][j] *= ex2(down);
              mv[nt][j] += down;
              m[nt][j] = mx;
            }
          }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mn, mu;
        if constexpr (T8) {
          mu = finite_or_0(m[nt][j]);
          const float x0 = s[nt][j] - mu, x1 = s[nt][2 + j] - mu;
          l[nt][j] += ex2(x0) + ex2(x1);
          s[nt][j] = x0 + (float)e0;
          s[nt][2 + j] = x1 + (float)e1;
        }
        float& top = T8 ? mv[nt][j] : m[nt][j];
        mn = fmaxf(top, col_max(fmaxf(s[nt][j], s[nt][2 + j])));
        mu = finite_or_0(mn);
        corr[nt][j] = top == mn ? 1.f : ex2(top - mu);
        grew |= top != mn;
        top = mn;
        const float ref = T8 ? mu - kUp : mu;
        s[nt][j] = ex2(s[nt][j] - ref);
        s[nt][2 + j] = ex2(s[nt][2 + j] - ref);
        if constexpr (!T8) l[nt][j] = l[nt][j] * corr[nt][j] + (s[nt][j] + s[nt][2 + j]);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // tokens 0-7, 8-15: [token][head] to [head][token]
        const float u = s[nt][2 * h], v = s[nt][2 * h + 1];
        if constexpr (T8) {
          ph[nt][h] = transpose8x8(pack_f16(u, v));
        } else {
          const uint32_t hi = pack_bf16(u, v);
          ph[nt][h] = transpose8x8(hi);
          pl[nt][h] = transpose8x8(pack_bf16(u - bf16lo(hi), v - bf16hi(hi)));
        }
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[d][nt][0] *= corr[nt][0];
          o[d][nt][1] *= corr[nt][1];
          o[d][nt][2] *= corr[nt][0];
          o[d][nt][3] *= corr[nt][1];
        }
    }
    const uint32_t v = ring + slot * S::bytes, r8 = lane & 7, q4 = lane >> 3;
    if constexpr (T8) {
      // matrices: tokens 0-7 and 8-15 of a group of 16 dims, then of the next
      const uint32_t at = v + (r8 + (q4 & 1) * 8) * S::row + (q4 >> 1) * 16;
      const uint32_t* t = reinterpret_cast<const uint32_t*>(sm + M::vsc + warp * M::scale_row * 16) + (lane & 3) * M::scale_row;
#pragma unroll
      for (int g2 = 0; g2 < D / 32; ++g2) {
        uint32_t w[4];
        ldsm4t(w, at + g2 * 32);
        const uint4 c4 = *reinterpret_cast<const uint4*>(t + g2 * 4);  // two groups' scales of tokens 2c.. and 2c + 8..
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int g = 2 * g2 + j;
          // (dims 2r, 2r+1 of token 2c, then of 2c+1) -> (tokens 2c, 2c+1 of dim 2r, then of 2r+1)
          const uint32_t w0 = __byte_perm(w[2 * j], 0u, 0x3120), w1 = __byte_perm(w[2 * j + 1], 0u, 0x3120);
          const uint32_t A[4] = {e4m3_to_f16x2(w0), e4m3_to_f16x2(w0 >> 16), e4m3_to_f16x2(w1), e4m3_to_f16x2(w1 >> 16)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<true>(o[g][nt], A, hmul2(ph[nt][0], j ? c4.z : c4.x), hmul2(ph[nt][1], j ? c4.w : c4.y));
        }
      }
      __syncwarp();  // the transposed scales are free
    } else {
      const uint32_t at = v + (r8 + (q4 >> 1) * 8) * S::row + (q4 & 1) * 16;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t A[4];
        ldsm4t(A, at + d * 32);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma<false>(o[d][nt], A, ph[nt][0], ph[nt][1]);
          mma<false>(o[d][nt], A, pl[nt][0], pl[nt][1]);
        }
      }
    }
  }

  // ---- the tokens of a tile that the item's first row does not see (the call's own later rows: at most
  // seven): their V from the cache, weight times value in the columns that see them
  __device__ void add_tail(const Segment& sg, uint32_t t, const float (&p)[NT][4], int e0, int e1) {
    const Tile x = tile(sg, t);
    const uint32_t first = sg.pos + 2 - sg.rows, r = lane >> 2;  // the first such token
    for (uint32_t k = first > x.token ? first - x.token : 0u; k < min(x.seen, 16u); ++k) {
      if (!(k & 8 ? x.in[1] : x.in[0])) continue;
      const size_t row = (k & 8 ? x.row[1] : x.row[0]) + (k & 7);
      const size_t at = (row * a.c.Hkv + sg.g) * D;
      const int ev = T8 ? __shfl_sync(0xffffffffu, k & 8 ? e1 : e0, (k & 7) * 4) : 0;
      float w[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float lo = __shfl_sync(0xffffffffu, p[nt][j], (k & 7) * 4 + (lane & 3));
          const float hi = __shfl_sync(0xffffffffu, p[nt][2 + j], (k & 7) * 4 + (lane & 3));
          w[nt][j] = k & 8 ? hi : lo;
        }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const uint32_t d0 = 16 * d + (T8 ? 2 * r : r), d1 = 16 * d + (T8 ? 2 * r + 1 : r + 8);
        float v0, v1;
        if constexpr (T8) {
          const float sc = bf16f(a.c.vs[row * a.c.sstride + sg.g * (D / 16) + d]) * pow2(-ev);
          const float2 v = e4m3_pair_value(*reinterpret_cast<const uint16_t*>(a.c.v + at + d0));
          v0 = v.x * sc;
          v1 = v.y * sc;
        } else {
          v0 = bf16f(reinterpret_cast<const uint16_t*>(a.c.v)[at + d0]);
          v1 = bf16f(reinterpret_cast<const uint16_t*>(a.c.v)[at + d1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (w[nt][j] != 0.f) {
              o[d][nt][j] = fmaf(w[nt][j], v0, o[d][nt][j]);
              o[d][nt][2 + j] = fmaf(w[nt][j], v1, o[d][nt][2 + j]);
            }
      }
    }
  }

  // ---- this warp's tiles of a segment, t0 + warp, t0 + warp + kWarps, ...: K and V of each in turn through the
  // ring, S::n half-tiles ahead. One loop for the start, where q is put in place, and the rest, so that the copies'
  // code is there once: an SM runs it cold, and what it fetches shows in the small calls.
  __device__ __forceinline__ void walk(const Segment& s, const QRegs& q) {
    const uint32_t first = s.t0 + warp;
    const int halves = first < s.t1 ? 2 * (int)((s.t1 - first + kWarps - 1) / kWarps) : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
        mv[nt][j] = -INFINITY;
        later[nt][j] = s.rows - 1 - min((8 * nt + 2 * (lane & 3) + j) / group, s.rows - 1);
      }
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][nt][i] = 0.f;
    float sc[NT][4];
    uint32_t slot = 0;                          // the slot that is read now and refilled then
    uint32_t seen = 0, seen1 = 0, seen2 = 0;    // of the tile that is read, the last one copied, the one before; with
                                                // a bit for each half in a block outside the pool
    Tile found, ahead;  // each lane: a tile's place, 32 tiles looked up at a time; the tile that is being copied
    found.seen = ahead.seen = 0;
#pragma unroll 1
    for (int h = -S::n; h < max(halves, 1); ++h) {
      if (h == 0) put_q(q);
      if (h >= 0 && h < halves) {
        cp_wait<S::n - 1>();
        __syncwarp();
        if (!(h & 1)) {
          seen = seen2;  // the copies are one tile ahead
          if (seen) scores(slot, sc);
        } else if (seen) {
          int e0 = 0, e1 = 0;
          accumulate(slot, sc, seen, s.rows, e0, e1);
          if ((seen & 63u) < 16 + s.rows - 1 && s.rows > 1) add_tail(s, first + (h >> 1) * kWarps, sc, e0, e1);
        }
        __syncwarp();  // this half-tile has been read by every lane
      }
      const int c = h + S::n;  // the half-tile to copy
      if (!(c & 1)) {
        const uint32_t i = c >> 1;
        if (i % 32 == 0) found = tile(s, first + (i + lane) * kWarps);
        ahead = lane_of(found, i % 32);
        seen2 = seen1;
        seen1 = ahead.seen ? ahead.seen | (ahead.in[0] ? 0u : kNo0) | (ahead.in[1] ? 0u : kNo1) : 0u;
      }
      if (c < halves) load(s, ahead, c & 1, slot);
      cp_commit();
      slot = slot + 1 == S::n ? 0 : slot + 1;
    }
    cp_wait<0>();
  }
  // T8: the largest of the warps' maxima in column h, and of V's relative to it (warps without a tile have -infinity)
  __device__ __forceinline__ static float2 tops(const float* ml, uint32_t h) {
    float m[kWarps], v[kWarps], mx = -INFINITY, vx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      m[w] = ml[w * kMl + h];
      v[w] = ml[w * kMl + 32 + h];
      mx = fmaxf(mx, m[w]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) vx = fmaxf(vx, v[w] + (m[w] - finite_or_0(mx)));
    return make_float2(mx, vx);
  }
  // ---- the warps' outputs added up: sum [cols][D + 4] at sm, M, L and (T8) V's maximum at ml[kWarps]
  __device__ void join_warps(uint32_t cols, uint32_t warps) {
    float* ml = reinterpret_cast<float*>(sm + M::ml);
    float* red = reinterpret_cast<float*>(sm);
    const uint32_t r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        if (r == 0) {
          ml[warp * kMl + 8 * nt + 2 * c + j] = m[nt][j];
          ml[warp * kMl + 16 + 8 * nt + 2 * c + j] = x;
          if (T8) ml[warp * kMl + 32 + 8 * nt + 2 * c + j] = mv[nt][j];
        }
      }
    __syncthreads();  // the rings are free too
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t h = 8 * nt + 2 * c + j;
        float f, mx = -INFINITY;
        if constexpr (T8) {
          const float2 top = tops(ml, h);
          f = rescale(mv[nt][j] + (m[nt][j] - finite_or_0(top.x)), top.y);
        } else {
          for (uint32_t w = 0; w < warps; ++w) mx = fmaxf(mx, ml[w * kMl + h]);
          f = rescale(m[nt][j], mx);
        }
        if (h < cols && warp < warps) {
          float* to = red + (warp * cols + h) * (D + 4);
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const uint32_t d0 = 16 * d + (T8 ? 2 * r : r), d1 = 16 * d + (T8 ? 2 * r + 1 : r + 8);
            to[d0] = o[d][nt][j] * f;
            to[d1] = o[d][nt][2 + j] * f;
          }
        }
      }
    if (threadIdx.x < 8 * NT) {
      const uint32_t h = threadIdx.x;
      float mx = -INFINITY, sum = 0.f;
      for (uint32_t w = 0; w < warps; ++w) mx = fmaxf(mx, ml[w * kMl + h]);
      for (uint32_t w = 0; w < warps; ++w) sum += ml[w * kMl + 16 + h] * rescale(ml[w * kMl + h], mx);
      ml[kWarps * kMl + h] = mx;
      ml[kWarps * kMl + 16 + h] = sum;
      if (T8) ml[kWarps * kMl + 32 + h] = tops(ml, h).y;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < cols * (D / 4); i += kAttnThreads) {
      float* at = red + (i / (D / 4)) * (D + 4) + 4 * (i % (D / 4));
      float4 x = *reinterpret_cast<float4*>(at);
#pragma unroll 4
      for (uint32_t w = 1; w < warps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(at + w * cols * (D + 4));
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      *reinterpret_cast<float4*>(at) = x;
    }
    __syncthreads();
  }

  // ---- sum [cols][D + 4] over L: rotated back, gated, rounded, stored. A thread has kOut pieces of eight dims;
  // their gates are fetched ahead.
  static constexpr int kOut = (8 * NT * (D / 8) + kAttnThreads - 1) / kAttnThreads;
  struct Gates {
    uint4 u[kOut];
  };
  __device__ __forceinline__ size_t head_of(const Segment& s, uint32_t col) const {
    return (size_t)(s.row + col / group) * a.H + s.g * group + col % group;
  }
  __device__ Gates fetch_gates(const Segment& s) const {
    Gates z;
#pragma unroll
    for (int k = 0; k < kOut; ++k) {
      const uint32_t i = threadIdx.x + k * kAttnThreads, h = i / (D / 8), c = i % (D / 8);
      z.u[k] = make_uint4(0u, 0u, 0u, 0u);
      if (a.gate && h < group * s.rows)
        z.u[k] = *reinterpret_cast<const uint4*>(a.gate + head_of(s, h) * a.gate_stride + 8 * c);
    }
    return z;
  }
  __device__ void store(const Segment& s, const Gates& gates) {
    const float* red = reinterpret_cast<const float*>(sm);
    const float* ml = reinterpret_cast<const float*>(sm + M::ml) + kWarps * kMl;
    constexpr int LPR = D / 8;
#pragma unroll
    for (int k = 0; k < kOut; ++k) {
      const uint32_t i = threadIdx.x + k * kAttnThreads, h = i / LPR, c = i % LPR;
      if (i >= 8 * NT * LPR) break;  // whole warps
      float x[8] = {};
      if (h < group * s.rows) {
        const float L = ml[16 + h], inv = L == 0.f ? 0.f : 1.0f / L;
        // T8: times 2^(V's maximum - kUp), in two steps: it may be 2^-140 where the sums are large
        const float up = !T8 ? 1.f : L == 0.f ? 0.f : ex2(0.5f * (ml[32 + h] - kUp));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = red[h * (D + 4) + 8 * c + e] * inv;
          if (T8) x[e] = x[e] * up * up;
        }
      }
      if constexpr (T8) wht8<LPR>(x, lane);
      if (h < group * s.rows) {
        if (a.gate) {
          float z[8];
          unpack8(gates.u[k], z);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= sigmoidf_(z[e]);
        }
        *reinterpret_cast<uint4*>(a.out + head_of(s, h) * D + 8 * c) = pack8(x);
      }
    }
  }

  // ---- a split item's part of this CTA (slot 0: the item began in an earlier CTA)
  __device__ float* part(uint32_t cta, uint32_t slot) const {
    return a.parts + ((size_t)cta * 2 + slot) * (group * pack * (D + 4));
  }
  // Part: for each column D sums, M, L, (T8) V's maximum and padding.
  __device__ void store_part(uint32_t slot, uint32_t cols) {
    const float* red = reinterpret_cast<const float*>(sm);
    const float* ml = reinterpret_cast<const float*>(sm + M::ml) + kWarps * kMl;
    float* to = part(blockIdx.x, slot);
    for (uint32_t i = threadIdx.x; i < cols * (D / 4); i += kAttnThreads) {
      const uint32_t at = (i / (D / 4)) * (D + 4) + 4 * (i % (D / 4));
      __stcg(reinterpret_cast<float4*>(to + at), *reinterpret_cast<const float4*>(red + at));
    }
    if (threadIdx.x < cols)
      __stcg(reinterpret_cast<float4*>(to + threadIdx.x * (D + 4) + D),
             make_float4(ml[threadIdx.x], ml[16 + threadIdx.x], T8 ? ml[32 + threadIdx.x] : 0.f, 0.f));
  }
  // The parts of CTAs c0 .. c1 added up, as join_warps leaves its sums: a thread has four dims of a column and,
  // where there are fewer such columns than threads, every subs-th part. The order is fixed by c0 and c1.
  __device__ void join_parts(uint32_t c0, uint32_t c1, uint32_t ncol) {
    float* red = reinterpret_cast<float*>(sm);  // [subs][ncol][D + 4]
    float* ml = reinterpret_cast<float*>(sm + M::ml) + kWarps * kMl;
    float* wt = reinterpret_cast<float*>(sm + M::weights);  // [ncol][parts]
    const uint32_t n = c1 - c0 + 1, cols = ncol * (D / 4), subs = max(1u, kAttnThreads / cols);
    // Parts of a thread in flight, in its own slots of what the ring leaves: all of them in one wait where 38 CTAs share an
    // item, and less code than sixteen in registers (32 sequences 126 us, was 128; 32 chosen blocks 11.5, was 11.8).
    constexpr int B = (M::big - M::parts) / (kAttnThreads * 16);
    uint4* stage = reinterpret_cast<uint4*>(sm + M::parts) + threadIdx.x;
    const size_t step = 2 * (size_t)(group * pack * (D + 4));
    // every thread takes the same rounds (the first has a barrier in it): columns of a stride of the threads, B parts each
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t i0 = 0, k0 = 0; i0 < cols * subs;) {
      const uint32_t i = i0 + threadIdx.x, sub = i / cols, col = i % cols, h = col / (D / 4);
      const uint32_t at = h * (D + 4) + 4 * (col % (D / 4));
      const bool mine = i < cols * subs;
      const float* p0 = part(c0, 1) + at;  // CTA c0's part, then slot 0 of each CTA
      const float* p = part(c0, 0) + at;
      const uint32_t left = mine && k0 + sub < n ? min((n - k0 - sub + subs - 1) / subs, (uint32_t)B) : 0;
#pragma unroll 4
      for (uint32_t k = 0; k < left; ++k) {
        const uint32_t c = k0 + sub + k * subs;
        cp16(smem_addr(stage + k * kAttnThreads), c ? p + c * step : p0);
      }
      cp_commit();
      if (i0 == 0 && k0 == 0) {  // the weights, their loads in the same wait as the first parts'
        for (uint32_t hh = warp; hh < ncol; hh += kWarps) {
          float mx = -INFINITY, sum = 0.f, vx = -INFINITY;
          constexpr int U = (kMaxCtas + 31) / 32;
          float2 z[U];
          float zv[U];  // T8: V's maximum
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t c = c0 + lane + 32 * u;
            z[u] = make_float2(-INFINITY, 0.f);
            zv[u] = -INFINITY;
            if (c <= c1) {
              const float* from = part(c, c == c0) + hh * (D + 4) + D;
              z[u] = __ldcg(reinterpret_cast<const float2*>(from));
              if (T8) zv[u] = __ldcg(from + 2);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) mx = fmaxf(mx, z[u].x);
          mx = warp_max(mx);
          if constexpr (T8) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              zv[u] += z[u].x - finite_or_0(mx);
              vx = fmaxf(vx, zv[u]);
            }
            vx = warp_max(vx);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t c = lane + 32 * u;
            const float f = rescale(z[u].x, mx);
            if (c < n) wt[hh * n + c] = T8 ? rescale(zv[u], vx) : f;
            sum += z[u].y * f;
          }
          sum = warp_sum(sum);
          if (lane == 0) {
            ml[hh] = mx;
            ml[16 + hh] = sum;
            if (T8) ml[32 + hh] = vx;
          }
        }
        __syncthreads();
      }
      cp_wait<0>();
#pragma unroll 4
      for (uint32_t k = 0; k < left; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(stage + k * kAttnThreads);
        const float f = wt[h * n + k0 + sub + k * subs];
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      k0 += B * subs;
      if (k0 >= n) {
        if (mine) *reinterpret_cast<float4*>(red + sub * ncol * (D + 4) + at) = x;
        x = make_float4(0.f, 0.f, 0.f, 0.f);
        k0 = 0;
        i0 += kAttnThreads;
      }
    }
    __syncthreads();
    if (subs > 1) {
      for (uint32_t col = threadIdx.x; col < cols; col += kAttnThreads) {
        float* at = red + (col / (D / 4)) * (D + 4) + 4 * (col % (D / 4));
        float4 x = *reinterpret_cast<float4*>(at);
        for (uint32_t s = 1; s < subs; ++s) {
          const float4 y = *reinterpret_cast<const float4*>(at + s * ncol * (D + 4));
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        *reinterpret_cast<float4*>(at) = x;
      }
      __syncthreads();
    }
  }
};

// The tiles of the item that begins with row r, of its tokens or of its listed blocks, with the item's rows
// and last position; 0 for a row that is skipped or inside an item.
__device__ __forceinline__ uint32_t row_tiles(const Attend& a, const Rows& at, uint32_t pack, uint32_t r, bool report,
                                              uint32_t& seq, uint32_t& rows, uint32_t& last) {
  uint32_t pos, index, left;
  const RowKind kind = locate(at, a.c.capacity, r, seq, pos, index, left);
  if (kind == kRowBad && report) set_status(a.status, kStatusRange);
  if (kind != kRowOk || index % pack != 0) return 0;
  rows = min(min(pack, left), a.c.capacity - pos);
  last = pos + rows - 1;
  return a.blocks ? a.n_blocks << (a.blk_shift - 4) : last / 16 + 1;
}

template <int D, int NT, bool T8>
__global__ void __launch_bounds__(kAttnThreads, 1) attend_kernel(const __grid_constant__ Attend a) {
  extern __shared__ __align__(128) uint8_t sm[];
  using A = Attention<D, NT, T8>;
  using M = Smem<D, NT, T8>;
  uint32_t* first = reinterpret_cast<uint32_t*>(sm + M::first);  // [n_rows + 1]: tiles before a row (of one head)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + M::misc);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = a.H / a.c.Hkv;
  const uint32_t pack = a.blocks || group > 8 ? 1 : 8 / group;
  pdl_wait();
  pdl_launch();
  // where the rows are, in shared memory (the ring is empty): one round trip for all searches
  Rows rows_here = a.r;
  {
    int32_t* pos = reinterpret_cast<int32_t*>(sm);
    int32_t* start = pos + kMaxSeqs;
    for (uint32_t i = tid; i < a.r.n_seqs; i += kAttnThreads) pos[i] = a.r.pos[i];
    if (a.r.row_start)
      for (uint32_t i = tid; i <= a.r.n_seqs; i += kAttnThreads) start[i] = a.r.row_start[i];
    rows_here.pos = pos;
    if (a.r.row_start) rows_here.row_start = start;
    __syncthreads();
  }
  // the line of all items: prefix sums of the rows' tiles with kLead before each item's, or (whole) of ones.
  // kLead stands for what an item's beginning and end cost a CTA that has another item too: about two
  // rounds of its warps (32 sequences of 1K-16K: 128 us, without it 134; 128K tokens in Turbo8 66 and 71).
  constexpr uint32_t kLead = 2 * kWarps;
  uint32_t most = 0, items = 0;
  uint32_t total = 0, per = 0;
  bool whole = false;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t base = 0;
    for (uint32_t r0 = 0; r0 < a.r.n_rows; r0 += kAttnThreads) {
      const uint32_t r = r0 + tid;
      uint32_t seq, rows, last, v = 0;
      if (r < a.r.n_rows) v = row_tiles(a, rows_here, pack, r, blockIdx.x == 0, seq, rows, last);
      most = max(most, v);
      items += v > 0;
      v = whole ? v > 0 : v ? v + kLead : 0;
      uint32_t x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= (uint32_t)o) x += y;
      }
      if (lane == 31) misc[warp] = x;
      __syncthreads();
      uint32_t before = base;
#pragma unroll
      for (uint32_t w = 0; w < kWarps; ++w) {
        before += w < warp ? misc[w] : 0;
        base += misc[w];
      }
      if (r < a.r.n_rows) first[r] = before + x - v;
      if (r == a.r.n_rows - 1) first[r + 1] = before + x;
      __syncthreads();
    }
    total = base * a.c.Hkv;
    if (total == 0) return;
    if (whole) {
      per = 1;
      break;
    }
    // An equal stretch for every CTA, whole rounds of the warps, or at least kLeast tiles where there is less
    // (512 tokens of 4 heads on 64 CTAs: 9.9 us, on 16 CTAs of a whole round 11.6). Few items of up to kShort rounds go
    // to a CTA each instead: a split's hand-over and join take 4 us or more (6.4 for 32 parts), a round of one CTA 1.5 to 2.5.
    constexpr uint32_t kShort = 2, kLeast = 2;
    most = __reduce_max_sync(0xffffffffu, most);
    items = __reduce_add_sync(0xffffffffu, items);
    if (lane == 0) {
      misc[warp] = most;
      misc[40 + warp] = items;
    }
    __syncthreads();
    most = items = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
      most = max(most, misc[w]);
      items += misc[40 + w];
    }
    __syncthreads();
    whole = items * a.c.Hkv <= gridDim.x && most <= kShort * kWarps;
    per = max((total + gridDim.x - 1) / gridDim.x, kLeast);
    if (per > kWarps / 2) per = (per + kWarps - 1) / kWarps * kWarps;
    if (!whole) break;
  }
  __syncthreads();  // the ring is free
  const uint64_t w64 = (uint64_t)blockIdx.x * per;
  if (w64 >= total) return;
  const uint32_t w0 = (uint32_t)w64, w1 = min(total, w0 + per);
  uint32_t row = 0;
  {
    uint32_t lo = 0, hi = a.r.n_rows;  // first[lo] Hkv <= w0 < first[hi] Hkv
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (first[mid] * a.c.Hkv <= w0) lo = mid;
      else hi = mid;
    }
    row = lo;
  }
  A at{a, sm, warp, lane, group, pack};
  at.ring = smem_addr(sm) + warp * A::S::n * A::S::bytes;
  for (uint32_t w = w0; w < w1;) {
    Segment s;
    while (first[row + 1] * a.c.Hkv <= w) ++row;
    s.row = row;
    s.tiles = row_tiles(a, a.r, pack, row, false, s.seq, s.rows, s.pos);
    s.row0 = (size_t)s.seq * a.c.capacity;
    s.tab = a.c.btab ? a.c.btab + (size_t)s.seq * (a.c.capacity >> a.c.bt_shift) : nullptr;
    const uint32_t in_row = w - first[row] * a.c.Hkv, length = s.tiles + kLead;
    uint32_t c0 = 0, c1 = 0, used = 1;  // the CTAs the item's tiles lie in, the line this CTA has of it
    s.t0 = 0;
    s.t1 = s.tiles;
    if (whole) {
      s.g = in_row;
    } else {
      s.g = in_row / length;
      const uint32_t at0 = in_row % length;
      used = min(length - at0, w1 - w);
      s.t0 = max(at0, kLead) - kLead;
      s.t1 = max(at0 + used, kLead) - kLead;
      c0 = (w - at0 + kLead) / per;
      c1 = (w - at0 + length - 1) / per;
    }
    if (s.t0 == s.t1) {
      w += used;
      continue;
    }
    const typename A::QRegs q = at.fetch_q(s);
    at.walk(s, q);
    const uint32_t cols = group * s.rows;
    const typename A::Gates gates = at.fetch_gates(s);
    at.join_warps(cols, min(kWarps, s.t1 - s.t0));
    bool finish = true;
    if (c0 != c1) {
      at.store_part(blockIdx.x == c0 ? 1 : 0, cols);
      __syncthreads();
      if (tid == 0) {
        // One item at most begins in CTA c0 and goes on behind it: its counter. The barrier has put the CTA's part
        // before this, and the count's release and acquire put it before the last one's reads.
        const uint32_t had = count_up(a.tickets + c0);
        misc[16] = had == c1 - c0;
        if (had > c1 - c0) set_status(a.status, kStatusInvalid);
        if (had == c1 - c0) a.tickets[c0] = 0;
      }
      __syncthreads();
      finish = misc[16] != 0;
      if (finish) at.join_parts(c0, c1, cols);
    }
    if (finish) at.store(s, gates);
    __syncthreads();
    w += used;
  }
}

template <int D, int NT, bool T8>
cudaError_t launch(const Attend& a, cudaStream_t st) {
  const uint32_t bytes = Smem<D, NT, T8>::first + (a.r.n_rows + 1) * 4;
  const uint64_t most = (uint64_t)a.r.n_rows * a.c.Hkv *
                        (a.blocks ? (uint64_t)a.n_blocks << (a.blk_shift - 4) : (a.c.capacity + 15) / 16);
  const uint32_t grid = (uint32_t)std::min<uint64_t>(std::min(a.sms, kMaxCtas), most);
  return launch_early(attend_kernel<D, NT, T8>, dim3(grid), kAttnThreads, bytes, st, a);
}
template <int D>
cudaError_t launch_for(const Attend& a, cudaStream_t st) {
  if (a.H / a.c.Hkv <= 8) return a.c.ks ? launch<D, 1, true>(a, st) : launch<D, 1, false>(a, st);
  return a.c.ks ? launch<D, 2, true>(a, st) : launch<D, 2, false>(a, st);
}

template <int D, int NT, bool T8>
bool allow() {
  constexpr int bytes = Smem<D, NT, T8>::first + (kMaxQueries + 1) * 4;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  return cudaFuncSetAttribute(attend_kernel<D, NT, T8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
         cudaSuccess;
}
template <int D>
bool allow_dim() {
  return allow<D, 1, false>() && allow<D, 1, true>() && allow<D, 2, false>() && allow<D, 2, true>();
}

}  // namespace

cudaError_t attend_attributes() {
  return allow_dim<64>() && allow_dim<128>() && allow_dim<256>() ? cudaSuccess : cudaGetLastError();
}

cudaError_t attend(const Attend& a, cudaStream_t st) {
  switch (a.c.D) {
    case 64: return launch_for<64>(a, st);
    case 128: return launch_for<128>(a, st);
    case 256: return launch_for<256>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace q35c
