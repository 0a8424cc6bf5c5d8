// Attention of new tokens over a KV cache (cache_ops.h).
#include "cache_ops.cuh"
#include "turbo8.cuh"

namespace q35c {
using namespace q35;
namespace {

// One CTA per (row, kv-head), LPR = D / 8 lanes a token with eight dims a lane; each such
// group of lanes keeps its own running maximum, sum and output, joined at the end.
template <int D, int HPG, bool T8>
__global__ void __launch_bounds__(128) attend_kernel(const Attend a) {
  constexpr int LPR = D / 8, TEAMS = 128 / LPR;
  __shared__ float qs[HPG][D];
  __shared__ float sm[TEAMS][HPG], sl[TEAMS][HPG];
  __shared__ float so[D];
  const uint32_t r = blockIdx.y, g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, l = lane % LPR, team = tid / LPR;
  const uint32_t group = a.H / a.c.Hkv;
  uint32_t seq, pos;
  const RowKind kind = locate(a.r, a.c.capacity, r, seq, pos);
  if (kind != kRowOk) {
    if (kind == kRowBad) set_status(a.status, kStatusRange);
    return;
  }
  for (uint32_t h = team; h < (HPG + TEAMS - 1) / TEAMS * TEAMS; h += TEAMS) {
    float x[8] = {};
    if (h < group) unpack8(*reinterpret_cast<const uint4*>(a.q + ((size_t)r * a.H + g * group + h) * D + 8 * l), x);
    if (T8) wht8<LPR>(x, lane);
    if (h < HPG)
      for (int e = 0; e < 8; ++e) qs[h][8 * l + e] = x[e];
  }
  __syncthreads();
  const float sl2 = 1.4426950408889634f / sqrtf((float)D);
  float m[HPG], s[HPG], o[HPG][8];
#pragma unroll
  for (int h = 0; h < HPG; ++h) {
    m[h] = -INFINITY;
    s[h] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[h][e] = 0.f;
  }
  const uint64_t n = a.blocks ? (uint64_t)a.n_blocks << a.blk_shift : (uint64_t)pos + 1;
  const int32_t* list = a.blocks ? a.blocks + ((size_t)r * a.c.Hkv + g) * a.n_blocks : nullptr;
  for (uint64_t i0 = 0; i0 < n; i0 += TEAMS) {
    const uint64_t i = i0 + team;
    bool in = i < n;
    uint64_t t = i;
    if (list && in) {
      const int32_t b = list[i >> a.blk_shift];
      in = b >= 0;
      t = ((uint64_t)(uint32_t)b << a.blk_shift) + (i & ((1u << a.blk_shift) - 1u));
    }
    in = in && t <= pos;
    size_t row = 0;
    if (in && !cache_row(a.c, seq, (uint32_t)t, row)) {
      set_status(a.status, kStatusRange);
      in = false;
    }
    float k[8] = {}, v[8] = {};
    if (in) {
      const size_t at = (row * a.c.Hkv + g) * D + 8 * l;
      if constexpr (T8) {
        const size_t sat = row * a.c.sstride + (g * D + 8 * l) / 16;
        dequant_codes8(*reinterpret_cast<const uint2*>(a.c.k + at), bf16f(a.c.ks[sat]), k);
        dequant_codes8(*reinterpret_cast<const uint2*>(a.c.v + at), bf16f(a.c.vs[sat]), v);
      } else {
        unpack8(*reinterpret_cast<const uint4*>(a.c.k + 2 * at), k);
        unpack8(*reinterpret_cast<const uint4*>(a.c.v + 2 * at), v);
      }
    }
#pragma unroll
    for (int h = 0; h < HPG; ++h) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x = fmaf(qs[h][8 * l + e], k[e], x);
#pragma unroll
      for (int w = 1; w < LPR; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      if (in) {
        x *= sl2;
        const float mn = fmaxf(m[h], x), c = m[h] == mn ? 1.f : exp2f(m[h] - mn), p = exp2f(x - mn);
        m[h] = mn;
        s[h] = s[h] * c + p;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[h][e] = o[h][e] * c + p * v[e];
      }
    }
  }
#pragma unroll
  for (int h = 0; h < HPG; ++h)
    if (l == 0) {
      sm[team][h] = m[h];
      sl[team][h] = s[h];
    }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HPG; ++h) {
    if ((uint32_t)h >= group) break;
    float mx = -INFINITY, sum = 0.f;
    for (int t = 0; t < TEAMS; ++t) mx = fmaxf(mx, sm[t][h]);
    for (int t = 0; t < TEAMS; ++t) sum += sl[t][h] > 0.f ? sl[t][h] * exp2f(sm[t][h] - mx) : 0.f;
    const float c = s[h] > 0.f ? exp2f(m[h] - mx) / sum : 0.f;
    for (int t = 0; t < TEAMS; ++t) {  // in order of the teams
      if ((int)team == t)
#pragma unroll
        for (int e = 0; e < 8; ++e) so[8 * l + e] = (t ? so[8 * l + e] : 0.f) + o[h][e] * c;
      __syncthreads();
    }
    if (tid < 32) {
      float x[8] = {};
      for (int e = 0; e < 8; ++e) x[e] = so[8 * l + e];
      if (T8) wht8<LPR>(x, lane);
      if (lane < LPR) {
        const size_t hh = (size_t)r * a.H + g * group + h;
        if (a.gate) {
          float z[8];
          unpack8(*reinterpret_cast<const uint4*>(a.gate + hh * a.gate_stride + 8 * l), z);
          for (int e = 0; e < 8; ++e) x[e] *= sigmoidf_(z[e]);
        }
        *reinterpret_cast<uint4*>(a.out + hh * D + 8 * l) = pack8(x);
      }
    }
    __syncthreads();
  }
}

template <int D, int HPG>
void launch(const Attend& a, cudaStream_t st) {
  const dim3 grid(a.c.Hkv, a.r.n_rows);
  if (a.c.ks) attend_kernel<D, HPG, true><<<grid, 128, 0, st>>>(a);
  else attend_kernel<D, HPG, false><<<grid, 128, 0, st>>>(a);
}
template <int D>
void launch_for(const Attend& a, cudaStream_t st) {
  const uint32_t group = a.H / a.c.Hkv;
  if (group <= 1) launch<D, 1>(a, st);
  else if (group <= 4) launch<D, 4>(a, st);
  else launch<D, 16>(a, st);
}

}  // namespace

cudaError_t attend(const Attend& a, cudaStream_t st) {
  switch (a.c.D) {
    case 64: launch_for<64>(a, st); break;
    case 128: launch_for<128>(a, st); break;
    case 256: launch_for<256>(a, st); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace q35c
