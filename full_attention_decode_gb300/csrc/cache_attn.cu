// Attention of new tokens over a KV cache (cache_ops.h): one launch for any number of
// rows, split over the cache's length and joined.
//
// Per (row, kv-head), an item, softmax(q K^T / sqrt D) V for the kv-head's group of up to
// 16 q-heads. The bytes of K and V bound it: each is read once for the whole group, by
// asynchronous copies into shared memory, and the products run on matrix instructions
// with the tokens as their rows (M = 16), the heads as their columns (N = 8), so that a
// group of 4 costs one instruction per 16 tokens x 16 dims:
//   S^T [16 tokens x 8 heads] += K [16 x 16 dims] Q^T [16 dims x 8], D / 16 times;
//   O^T [16 dims x 8 heads] += V^T [16 dims x 16 tokens] P^T [16 tokens x 8], D / 16 times.
// A warp works alone: it has its own ring of K and V tiles of 16 tokens, its own running
// maximum, sum and output, and meets the other warps only at the end of an item.
//
// The work of a call is the line of all items' 16-token tiles; every CTA takes an equal
// stretch of it, whatever the sequences' lengths. An item that lies in several CTAs is joined by
// the last of them to finish, in the order of the CTAs, so equal calls give equal bits.
//
// Roundings: bf16 K, V and q enter the products exactly, the weights P as hi + lo bf16
// (2^-16 relative). Turbo8 codes enter as f16 (exact); the K scales multiply the fp32
// products of their 16 dims; the rotated q enters as hi + lo f16 (2^-21); V = code * scale is
// rounded to f16 (2^-12 relative: 12 bits to 11) with its tile's largest scale taken out as a power
// of two, which is put into the weights, and those are rounded to f16 (2^-12).
#include "cache_ops.cuh"
#include "turbo8.cuh"

#include <algorithm>

namespace q35c {
using namespace q35;
namespace {

#ifndef ATT_WARPS
#define ATT_WARPS 8
#endif
constexpr int kWarps = ATT_WARPS, kCtasPerSm = 8 / kWarps;
constexpr int kAttnThreads = 32 * kWarps;

// A ring slot: K or V of 16 tokens. Rows are padded by 16 bytes, which puts eight rows'
// 16-byte pieces in different banks.
template <int D, bool T8>
struct Slot {
  static constexpr int row = T8 ? D + 16 : 2 * D + 16;
  static constexpr int scales = T8 ? D / 16 * 2 : 0;  // a token's scales
  static constexpr int bytes = 16 * (row + scales);
  static constexpr int n = D == 256 && !T8 ? 3 : 4;  // slots of a warp
};
// Shared memory of a CTA: the rings (reused to join the warps), Q's fragments, the warps'
// maxima and sums, T8's transposed V scales, then the rows' first tiles.
template <int D, int NT, bool T8>
struct Smem {
  using S = Slot<D, T8>;
  static constexpr int ring = kWarps * S::n * S::bytes;
  static constexpr int join = kWarps * 8 * NT * (D + 4) * 4;
  static constexpr int weights = 24576;  // the parts' weights, behind their sums
  static constexpr int parts = weights + 8 * NT * (int)kMaxCtas * 4;
  static constexpr int big = ring > join ? (ring > parts ? ring : parts) : join > parts ? join : parts;
  static constexpr int qf = big;                                    // fragments, 8 or (T8) 16 bytes a lane
  static constexpr int ml = qf + (D / 16) * NT * 32 * (T8 ? 16 : 8);  // [warps + 1][2][16]
  static constexpr int vsc = ml + (kWarps + 1) * 2 * 16 * 4;
  static constexpr int misc = vsc + (T8 ? kWarps * (D / 16) * 32 : 0);
  static constexpr int first = misc + 128;  // [n_rows + 1]
};

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
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]
__device__ __forceinline__ float rescale(float from, float to) { return from == -INFINITY ? 0.f : exp2f(from - to); }

// One item's stretch in a CTA.
struct Segment {
  uint32_t row, g, seq, pos;
  uint32_t tiles;   // the item's tiles
  uint32_t t0, t1;  // this CTA's
};

// The first token of a tile and where its tokens lie: rows of tokens 0-7 and 8-15 (a
// page holds at least 8 tokens), and how many of the 16 the row sees.
struct Tile {
  size_t row[2];
  uint32_t token, seen;
  bool in[2];
};

template <int D, int NT, bool T8>
struct Attention {
  using S = Slot<D, T8>;
  using M = Smem<D, NT, T8>;
  const Attend& a;
  uint8_t* sm;
  uint32_t warp, lane, group;
  uint32_t ring;  // this warp's slots
  float m[NT][2], l[NT][2], o[D / 16][NT][4];
  float qscale[NT][2];  // log2(e) / sqrt(D), with T8's power of two of q

  // ---- where a tile's tokens are
  __device__ Tile tile(const Segment& s, uint32_t t) const {
    Tile x;
    x.seen = 0;
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
    x.seen = min(16u, s.pos - x.token + 1);
    bool ok = true;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (8u * h < x.seen) {
        x.in[h] = cache_row(a.c, s.seq, x.token + 8 * h, x.row[h]);
        ok = ok && x.in[h];
      }
    if (!ok) set_status(a.status, kStatusRange);
    return x;
  }

  // ---- K (p = 0) or V of a tile into a slot; tokens the row does not see read as zero
  __device__ void load(const Segment& s, const Tile& x, int p, uint32_t slot) const {
    constexpr int C = (T8 ? D : 2 * D) / 16, R = 32 / C > 0 ? 32 / C : 1;  // 16-byte pieces of a row, rows a pass
    const uint8_t* base = p ? a.c.v : a.c.k;
    const uint32_t dst = ring + slot * S::bytes;
    const size_t stride = (size_t)a.c.Hkv * D * (T8 ? 1 : 2);
    const uint32_t r0 = lane / C, c = lane % C;
#pragma unroll
    for (int i = 0; i < 16 / R; ++i) {
      const uint32_t r = i * R + r0, h = (i * R) / 8;
      const bool in = r < x.seen && x.in[h];
      const uint8_t* src = base + (x.row[h] + (r & 7)) * stride + (size_t)s.g * D * (T8 ? 1 : 2) + c * 16;
      cp16(dst + r * S::row + c * 16, in ? src : base, in);
    }
    if constexpr (T8) {
      constexpr int SB = S::scales, P = SB >= 16 ? SB / 16 : 1;  // pieces of a token's scales
      const uint8_t* sbase = reinterpret_cast<const uint8_t*>(p ? a.c.vs : a.c.ks);
      const uint32_t r = lane / P, c2 = lane % P;
      if (r < 16) {
        const bool in = r < x.seen && (r & 8 ? x.in[1] : x.in[0]);
        const size_t row = (r & 8 ? x.row[1] : x.row[0]) + (r & 7);
        const uint8_t* src = sbase + (row * a.c.sstride + s.g * (D / 16)) * 2 + c2 * 16;
        const uint32_t to = dst + 16 * S::row + r * SB + c2 * 16;
        if constexpr (SB >= 16) cp16(to, in ? src : sbase, in);
        else cp8(to, in ? src : sbase, in);
      }
    }
  }

  // ---- q of an item as B fragments, [k-step][n-tile][lane]
  __device__ void load_q(const Segment& s) {
    float* qs = reinterpret_cast<float*>(sm);  // [8 NT][D] (the ring is empty)
    const uint16_t* q = a.q + ((size_t)s.row * a.H + s.g * group) * D;
    constexpr int LPR = D / 8;
    int* qe = reinterpret_cast<int*>(sm + M::misc) + 8;  // [16]
    for (uint32_t i = threadIdx.x; i < 8 * NT * LPR; i += kAttnThreads) {
      const uint32_t h = i / LPR, c = i % LPR;
      float x[8] = {};
      if (h < group) unpack8(*reinterpret_cast<const uint4*>(q + h * D + 8 * c), x);
      if constexpr (T8) {
        wht8<LPR>(x, lane);
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (int w = 1; w < LPR; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        // |x| 2^-e below 2^15: e = exponent - 14
        const int e2 = min(max((int)((__float_as_uint(mx) >> 23) & 255) - 127 - 14, -100), 100);
        const float f = mx > 0.f ? pow2(-e2) : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
        if (c == 0) qe[h] = mx > 0.f ? e2 : 0;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) qs[h * D + 8 * c + e] = x[e];
    }
    __syncthreads();
    constexpr int N = (D / 16) * NT;
    for (uint32_t i = threadIdx.x; i < N * 32; i += kAttnThreads) {
      const uint32_t ln = i & 31, nt = (i >> 5) % NT, kk = (i >> 5) / NT;
      const float* x = qs + (8 * nt + ln / 4) * D + 16 * kk;
      const uint32_t c = ln % 4;
      if constexpr (T8) {
        // a code word of 4 dims feeds both halves of the k-step: dims 4c, 4c+1 | 4c+2, 4c+3
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float u = x[4 * c + 2 * j], v = x[4 * c + 2 * j + 1];
          hi[j] = pack_f16(u, v);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
          lo[j] = pack_f16(u - f.x, v - f.y);
        }
        *reinterpret_cast<uint4*>(sm + M::qf + i * 16) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
      } else {
        *reinterpret_cast<uint2*>(sm + M::qf + i * 8) =
            make_uint2(pack_bf16(x[2 * c], x[2 * c + 1]), pack_bf16(x[2 * c + 8], x[2 * c + 9]));
      }
    }
    const float sl2 = 1.4426950408889634f / sqrtf((float)D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) qscale[nt][j] = T8 ? sl2 * pow2(qe[8 * nt + 2 * (lane % 4) + j]) : sl2;
    __syncthreads();  // the ring is free
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

  // ---- T8: a tile's V scales, divided by 2^e, transposed to [dims group][token] f16; returns e
  __device__ int v_scales(uint32_t slot) const {
    const uint8_t* sc = sm + (ring - smem_addr(sm)) + slot * S::bytes + 16 * S::row;
    uint16_t* t = reinterpret_cast<uint16_t*>(sm + M::vsc + warp * (D / 16) * 32);
    constexpr int PER = D / 32;  // scales a lane: half a token's
    const uint32_t tok = lane >> 1, g0 = (lane & 1) * PER;
    float f[PER], mx = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(sc + tok * S::scales + (g0 + i) * 2);
      f[i] = bf16lo(u);
      f[i + 1] = bf16hi(u);
      mx = fmaxf(mx, fmaxf(f[i], f[i + 1]));
    }
    mx = warp_max(mx);
    const int e = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -60), 60) : -60;
    const float k = pow2(-e);
#pragma unroll
    for (int i = 0; i < PER; ++i) t[(g0 + i) * 16 + tok] = __half_as_ushort(__float2half_rn(f[i] * k));
    __syncwarp();
    return e;
  }

  // ---- one tile: weights from the scores, then the output from its V slot
  __device__ void accumulate(uint32_t slot, float (&s)[NT][4], uint32_t seen) {
    const uint32_t r = lane >> 2;
    int ev = 0;
    if constexpr (T8) ev = v_scales(slot);
    uint32_t ph[NT][2], pl[NT][2];
    bool grew = false;
    float corr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x0 = s[nt][j] * qscale[nt][j], x1 = s[nt][2 + j] * qscale[nt][j];
        if (T8) {
          x0 += (float)ev;
          x1 += (float)ev;
        }
        if (r >= seen) x0 = -INFINITY;
        if (r + 8 >= seen) x1 = -INFINITY;
        float mx = fmaxf(x0, x1);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m[nt][j], mx), mu = mn == -INFINITY ? 0.f : mn;
        corr[nt][j] = m[nt][j] == mn ? 1.f : exp2f(m[nt][j] - mu);
        grew |= m[nt][j] != mn;
        m[nt][j] = mn;
        s[nt][j] = exp2f(x0 - mu);
        s[nt][2 + j] = exp2f(x1 - mu);
        const float sum = s[nt][j] + s[nt][2 + j];
        l[nt][j] = l[nt][j] * corr[nt][j] + (T8 ? sum * pow2(-ev) : sum);
      }
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
      const uint8_t* t = sm + M::vsc + warp * (D / 16) * 32 + (lane & 3) * 4;
#pragma unroll
      for (int g2 = 0; g2 < D / 32; ++g2) {
        uint32_t w[4];
        ldsm4t(w, at + g2 * 32);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int g = 2 * g2 + j;
          const uint32_t c0 = *reinterpret_cast<const uint32_t*>(t + g * 32);       // tokens 2c, 2c+1
          const uint32_t c1 = *reinterpret_cast<const uint32_t*>(t + g * 32 + 16);  // tokens 2c+8, 2c+9
          // (dims 2r, 2r+1 of token 2c, then of 2c+1) -> (tokens 2c, 2c+1 of dim 2r, then of 2r+1)
          const uint32_t w0 = __byte_perm(w[2 * j], 0u, 0x3120), w1 = __byte_perm(w[2 * j + 1], 0u, 0x3120);
          const uint32_t A[4] = {hmul2(e4m3_to_f16x2(w0), c0), hmul2(e4m3_to_f16x2(w0 >> 16), c0),
                                 hmul2(e4m3_to_f16x2(w1), c1), hmul2(e4m3_to_f16x2(w1 >> 16), c1)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<true>(o[g][nt], A, ph[nt][0], ph[nt][1]);
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

  // ---- the segment's tiles t0 + warp, t0 + warp + kWarps, ...
  __device__ void walk(const Segment& s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][nt][i] = 0.f;
    // slots hold K and V of tiles in turn; half-tile i of this warp: tile i / 2, V if odd.
    // The copies run S::n half-tiles ahead; `ahead` is the tile they are at.
    const uint32_t first = s.t0 + warp;
    if (first >= s.t1) return;
    const uint32_t n = (s.t1 - first + kWarps - 1) / kWarps, halves = 2 * n;
    Tile ahead = tile(s, first), next = tile(s, first + kWarps);
    uint32_t issued = 0, islot = 0;
    auto issue = [&]() {
      if (issued < halves) {
        load(s, ahead, issued & 1, islot);
        if (issued & 1) {  // the next tile's place, one tile before its copies
          ahead = next;
          next = tile(s, first + (issued / 2 + 2) * kWarps);
        }
      }
      cp_commit();
      ++issued;
      islot = islot + 1 == S::n ? 0 : islot + 1;
    };
    for (int i = 0; i < S::n; ++i) issue();
    uint32_t slot = 0;
    auto done = [&]() {  // this half-tile has been read by every lane
      __syncwarp();
      issue();
      slot = slot + 1 == S::n ? 0 : slot + 1;
    };
    for (uint32_t tick = 0; tick < n; ++tick) {
      const uint32_t seen = seen_of(s, first + tick * kWarps);
      float sc[NT][4];
      cp_wait<S::n - 1>();
      __syncwarp();
      if (seen) scores(slot, sc);
      done();
      cp_wait<S::n - 1>();
      __syncwarp();
      if (seen) accumulate(slot, sc, seen);
      done();
    }
    cp_wait<0>();
  }
  // How many tokens of a tile the row sees.
  __device__ uint32_t seen_of(const Segment& s, uint32_t t) const {
    uint64_t token = (uint64_t)t * 16;
    if (a.blocks) {
      const uint32_t per = a.blk_shift - 4;
      const int32_t b = a.blocks[((size_t)s.row * a.c.Hkv + s.g) * a.n_blocks + (t >> per)];
      if (b < 0) return 0;
      token = ((uint64_t)(uint32_t)b << a.blk_shift) + (t & ((1u << per) - 1u)) * 16;
    }
    return token > s.pos ? 0u : (uint32_t)min((uint64_t)16, s.pos - token + 1);
  }

  // ---- the warps' outputs added up: sum [group][D + 4] at sm, M and L at ml[kWarps]
  __device__ void join_warps() {
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
          ml[warp * 32 + 8 * nt + 2 * c + j] = m[nt][j];
          ml[warp * 32 + 16 + 8 * nt + 2 * c + j] = x;
        }
      }
    __syncthreads();  // the rings are free too
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t h = 8 * nt + 2 * c + j;
        float mx = -INFINITY;
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * 32 + h]);
        const float f = rescale(m[nt][j], mx);
        if (h < group) {
          float* to = red + (warp * group + h) * (D + 4);
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
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * 32 + h]);
      for (int w = 0; w < kWarps; ++w) sum += ml[w * 32 + 16 + h] * rescale(ml[w * 32 + h], mx);
      ml[kWarps * 32 + h] = mx;
      ml[kWarps * 32 + 16 + h] = sum;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < group * (D / 4); i += kAttnThreads) {
      float* at = red + (i / (D / 4)) * (D + 4) + 4 * (i % (D / 4));
      float4 x = *reinterpret_cast<float4*>(at);
      for (int w = 1; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(at + w * group * (D + 4));
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      *reinterpret_cast<float4*>(at) = x;
    }
    __syncthreads();
  }

  // ---- sum [group][D + 4] over L: rotated back, gated, rounded, stored
  __device__ void store(const Segment& s) {
    const float* red = reinterpret_cast<const float*>(sm);
    const float* L = reinterpret_cast<const float*>(sm + M::ml) + kWarps * 32 + 16;
    constexpr int LPR = D / 8;
    for (uint32_t i = threadIdx.x; i < 8 * NT * LPR; i += kAttnThreads) {
      const uint32_t h = i / LPR, c = i % LPR;
      float x[8] = {};
      if (h < group) {
        const float inv = L[h] == 0.f ? 0.f : 1.0f / L[h];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = red[h * (D + 4) + 8 * c + e] * inv;
      }
      if constexpr (T8) wht8<LPR>(x, lane);
      if (h < group) {
        const size_t hh = (size_t)s.row * a.H + s.g * group + h;
        if (a.gate) {
          float z[8];
          unpack8(*reinterpret_cast<const uint4*>(a.gate + hh * a.gate_stride + 8 * c), z);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= sigmoidf_(z[e]);
        }
        *reinterpret_cast<uint4*>(a.out + hh * D + 8 * c) = pack8(x);
      }
    }
    __syncthreads();
  }

  // ---- a split item's part of this CTA (slot 0: the item began in an earlier CTA)
  __device__ float* part(uint32_t cta, uint32_t slot) const {
    return a.parts + ((size_t)cta * 2 + slot) * (group * (D + 4));
  }
  // Part: group rows of D sums, M, L and two words of padding.
  __device__ void store_part(uint32_t slot) {
    const float* red = reinterpret_cast<const float*>(sm);
    const float* ml = reinterpret_cast<const float*>(sm + M::ml) + kWarps * 32;
    float* to = part(blockIdx.x, slot);
    for (uint32_t i = threadIdx.x; i < group * (D / 4); i += kAttnThreads) {
      const uint32_t at = (i / (D / 4)) * (D + 4) + 4 * (i % (D / 4));
      __stcg(reinterpret_cast<float4*>(to + at), *reinterpret_cast<const float4*>(red + at));
    }
    if (threadIdx.x < group)
      __stcg(reinterpret_cast<float4*>(to + threadIdx.x * (D + 4) + D),
             make_float4(ml[threadIdx.x], ml[16 + threadIdx.x], 0.f, 0.f));
  }
  // The parts of CTAs c0 .. c1 added up, as join_warps leaves its sums: a thread has four dims of a head and,
  // where there are fewer such columns than threads, every subs-th part. The order is fixed by c0 and c1.
  __device__ void join_parts(uint32_t c0, uint32_t c1) {
    float* red = reinterpret_cast<float*>(sm);  // [subs][group][D + 4]
    float* ml = reinterpret_cast<float*>(sm + M::ml) + kWarps * 32;
    float* wt = reinterpret_cast<float*>(sm + M::weights);  // [group][parts]
    const uint32_t n = c1 - c0 + 1;
    for (uint32_t h = warp; h < group; h += kWarps) {
      float mx = -INFINITY, sum = 0.f;
      constexpr int U = (kMaxCtas + 31) / 32;
      float2 x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = c0 + lane + 32 * i;
        x[i] = make_float2(-INFINITY, 0.f);
        if (c <= c1) x[i] = __ldcg(reinterpret_cast<const float2*>(part(c, c == c0) + h * (D + 4) + D));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) mx = fmaxf(mx, x[i].x);
      mx = warp_max(mx);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = lane + 32 * i;
        const float f = rescale(x[i].x, mx);
        if (c < n) wt[h * n + c] = f;
        sum += x[i].y * f;
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        ml[h] = mx;
        ml[16 + h] = sum;
      }
    }
    __syncthreads();
    const uint32_t cols = group * (D / 4), subs = max(1u, kAttnThreads / cols);
    for (uint32_t i = threadIdx.x; i < cols * subs; i += kAttnThreads) {
      const uint32_t sub = i / cols, col = i % cols, h = col / (D / 4), at = h * (D + 4) + 4 * (col % (D / 4));
      const float* w = wt + h * n;
      const float* p0 = part(c0, 1) + at;  // CTA c0's part, then slot 0 of each CTA
      const float* p = part(c0, 0) + at;
      const size_t step = 2 * (size_t)(group * (D + 4));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t k0 = sub; k0 < n; k0 += 16 * subs) {
        float4 y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t c = k0 + k * subs;
          y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < n) y[k] = __ldcg(reinterpret_cast<const float4*>(c ? p + c * step : p0));
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t c = k0 + k * subs;
          const float f = c < n ? w[c] : 0.f;
          x.x = fmaf(y[k].x, f, x.x);
          x.y = fmaf(y[k].y, f, x.y);
          x.z = fmaf(y[k].z, f, x.z);
          x.w = fmaf(y[k].w, f, x.w);
        }
      }
      *reinterpret_cast<float4*>(red + sub * group * (D + 4) + at) = x;
    }
    __syncthreads();
    if (subs > 1) {
      for (uint32_t col = threadIdx.x; col < cols; col += kAttnThreads) {
        float* at = red + (col / (D / 4)) * (D + 4) + 4 * (col % (D / 4));
        float4 x = *reinterpret_cast<float4*>(at);
        for (uint32_t s = 1; s < subs; ++s) {
          const float4 y = *reinterpret_cast<const float4*>(at + s * group * (D + 4));
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

// Tiles of a row: of its tokens, or of its listed blocks; 0 for a row that is skipped.
__device__ __forceinline__ uint32_t row_tiles(const Attend& a, uint32_t r, bool report) {
  uint32_t seq, pos;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
  if (kind == kRowBad && report) set_status(a.status, kStatusRange);
  if (kind != kRowOk) return 0;
  return a.blocks ? a.n_blocks << (a.blk_shift - 4) : pos / 16 + 1;
}

template <int D, int NT, bool T8>
__global__ void __launch_bounds__(kAttnThreads, kCtasPerSm) attend_kernel(const __grid_constant__ Attend a) {
  extern __shared__ __align__(128) uint8_t sm[];
  using A = Attention<D, NT, T8>;
  using M = Smem<D, NT, T8>;
  uint32_t* first = reinterpret_cast<uint32_t*>(sm + M::first);  // [n_rows + 1]: tiles before a row (of one head)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + M::misc);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the line of all items: prefix sums of the rows' tiles
  uint32_t base = 0;
  for (uint32_t r0 = 0; r0 < a.r.n_rows; r0 += kAttnThreads) {
    const uint32_t r = r0 + tid;
    const uint32_t v = r < a.r.n_rows ? row_tiles(a, r, blockIdx.x == 0) : 0;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= (uint32_t)o) x += y;
    }
    if (lane == 31) misc[warp] = x;
    __syncthreads();
    uint32_t before = base;
    for (uint32_t w = 0; w < warp; ++w) before += misc[w];
    if (r < a.r.n_rows) first[r] = before + x - v;
    for (uint32_t w = 0; w < (uint32_t)kWarps; ++w) base += misc[w];
    __syncthreads();
  }
  if (tid == 0) first[a.r.n_rows] = base;
  __syncthreads();
  const uint32_t total = base * a.c.Hkv;
  if (total == 0) return;
  // an equal stretch for every CTA, whole rounds of the warps
  uint32_t per = (total + gridDim.x - 1) / gridDim.x;
  per = (per + kWarps - 1) / kWarps * kWarps;
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
  A at{a, sm, warp, lane, a.H / a.c.Hkv};
  at.ring = smem_addr(sm) + warp * Slot<D, T8>::n * Slot<D, T8>::bytes;
  for (uint32_t w = w0; w < w1;) {
    Segment s;
    while (first[row + 1] * a.c.Hkv <= w) ++row;
    s.row = row;
    s.tiles = first[row + 1] - first[row];
    const uint32_t in_row = w - first[row] * a.c.Hkv;
    s.g = in_row / s.tiles;
    s.t0 = in_row % s.tiles;
    s.t1 = min(s.tiles, s.t0 + (w1 - w));
    locate(a.r, a.c.capacity, row, s.seq, s.pos);
    at.load_q(s);
    at.walk(s);
    at.join_warps();
    const uint32_t i0 = w - s.t0, i1 = i0 + s.tiles;  // the item on the line
    const uint32_t c0 = i0 / per, c1 = (i1 - 1) / per;
    if (c0 == c1) {
      at.store(s);
    } else {
      at.store_part(blockIdx.x == c0 ? 1 : 0);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        // one item at most begins in CTA c0 and goes on behind it: its counter
        const uint32_t had = atomicAdd(a.tickets + c0, 1u);
        misc[7] = had == c1 - c0;
        if (had > c1 - c0) set_status(a.status, kStatusInvalid);
        if (had == c1 - c0) a.tickets[c0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (misc[7]) {
        at.join_parts(c0, c1);
        at.store(s);
      }
    }
    __syncthreads();
    w += s.t1 - s.t0;
  }
}

template <int D, int NT, bool T8>
cudaError_t launch(const Attend& a, cudaStream_t st) {
  const uint32_t bytes = Smem<D, NT, T8>::first + (a.r.n_rows + 1) * 4;
  cudaError_t e =
      cudaFuncSetAttribute(attend_kernel<D, NT, T8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  const uint64_t most = (uint64_t)a.r.n_rows * a.c.Hkv *
                        (a.blocks ? (uint64_t)a.n_blocks << (a.blk_shift - 4) : (a.c.capacity + 15) / 16);
  const uint32_t grid = (uint32_t)std::min<uint64_t>(std::min(a.sms * kCtasPerSm, kMaxCtas), (most + kWarps - 1) / kWarps);
  attend_kernel<D, NT, T8><<<grid, kAttnThreads, bytes, st>>>(a);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_for(const Attend& a, cudaStream_t st) {
  if (a.H / a.c.Hkv <= 8) return a.c.ks ? launch<D, 1, true>(a, st) : launch<D, 1, false>(a, st);
  return a.c.ks ? launch<D, 2, true>(a, st) : launch<D, 2, false>(a, st);
}

}  // namespace

cudaError_t attend(const Attend& a, cudaStream_t st) {
  switch (a.c.D) {
    case 64: return launch_for<64>(a, st);
    case 128: return launch_for<128>(a, st);
    case 256: return launch_for<256>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace q35c
