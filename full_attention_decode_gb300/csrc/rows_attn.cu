// Attention of drafted trees and of rows that see a sliding window (rows_ops.h): any number
// of rows a sequence, one pass over K and V for up to 128 (row, q-head) pairs.
//
// An item is a kv-head of a block of a sequence's rows: 128 / group rows, whose (row, q-head) pairs are the
// M = 128 rows of the products (TMEM's lanes); the tokens come in tiles of 64:
//   S [128 x 64] = Q [128 x D] K^T,  P = 2^(S - m),  O [128 x D] += P [128 x 64] V,
// on the fifth-generation tensor cores: Q, K and V in shared memory (V as it lies, rows along the inner
// dimension), S and O in tensor memory, P written back there as the second product's first factor (Turbo8: over its S, as q's
// upper part lies there too). A decode row of 4
// q-heads leaves most of M empty; what bounds the call is the bytes of K and V all the same: a tile of D = 256
// is 64 KB, 1.5 us of an SM's share of the memory, its products 1 us.
//
// Roles of a CTA's 17 warps: 0-7 are the softmax, two threads a row with 32 of a tile's 64 tokens each, which
// exchange their maxima; 8-15 fill a ring of K and V tiles, 16-byte pieces by asynchronous copies (pages as small as 8
// tokens, rows outside as zeros), Turbo8's as they lie and then as f16; one thread of warp 16 issues the products. The softmax
// of a tile runs under the product of the tile before and the scores of the next (two S, two P; Turbo8 with one S and two P beside it: 16 trees 168 us where 157).
//
// The line of all items' tiles is cut into equal stretches, one CTA an SM. A stretch leaves its sums and maxima in the
// scratch, and an item's parts are added up in the order of the CTAs, so equal calls give equal bits. Few columns are
// joined by the last of the item's CTAs; those of a block of many rows, and of many items, by a second launch, spread over the GPU: one
// CTA that joined a block of 128 columns would read 2.5 MB.
//
// What bounds it (152 SMs, 16 q-heads over 4 kv-heads of 256). One token a sequence through windows of 4096, 32 sequences: 76 us,
// 5.4 TB/s, 412 MB of K and V in pieces of 16 bytes. A tree of 64 nodes over 8191 tokens: 31 us, 273 TFLOP/s, where
// seven tiles a CTA share with the way in and the join. Turbo8, 16 trees: 157 us, the chain of loader, products and softmax a
// tile, 3.3 us, with K and V in one place each beside q's lower part: shared memory's data path is busy half of the time, the issue
// slots 40%, the tensor cores a third. With one f16 of q and of K it took 139: q's lower part costs 6 us, K's second part 4, two halves of a
// tile ahead instead of three 1.5, the way of q into tensor memory 4, the wait for P's product before the next S over it the rest.
// (K's second part in a place of its own, written in a second pass 174 us, held in registers 269.)
//
// Roundings. bf16: Q, K, V exactly, P as hi + lo bf16 (2^-16). Turbo8: the rotated q as hi + lo f16 over the power of two of its
// largest value (2^-22 of a value or 2^-25 of the largest); K's codes times scale / 2^E, E the exponent of the token's largest
// scale, exactly, as two f16 (a product of 4 and 8 bits has 12, f16 11), lo times the second left out (at most 2^-11 2^-7 of a term); V's as
// one f16 (2^-11); 2^E of K multiplies the score in fp32, E of V goes into the weight's exponent: weights of V are
// 2^((x - m) + E - R) in f16, R following the largest within 2^4, so a token counts by what it adds. l refers to m alone.
//
// A tile that not every row of the item sees to its end may hold anything where it is not seen, and 0 times infinity would
// spoil the rows that do not: V's infinities and NaN are taken out of such tiles (Turbo8: of all) on their way in, and
// added by plain arithmetic for the rows that see them (`mend`). Other bf16 tiles go in as they lie; where a stretch's sums
// are no numbers then, they are put right at its end (`put_infinities`), so it does not matter where in a tile a token lies.
#include "rows_ops.h"

#include "cache_ops.cuh"
#include "tcgen05.cuh"
#include "turbo8.cuh"

#include <algorithm>
#include <type_traits>

namespace q35c {
using namespace q35;
namespace {

constexpr uint32_t kM = 128, kTile = 64, kOctets = kTile / 8;
constexpr uint32_t kSoft = 256;  // threads of the softmax
constexpr uint32_t kLoaders = 8, kLoadThreads = 32 * kLoaders, kRowsThreads = kSoft + kLoadThreads + 32;
// Registers of a thread: as launched (what 17 warps leave, five of them on one scheduler), then shared out anew where
// one role needs more.
constexpr int kRegsLaunch = 96;
constexpr int kRegsSoft = 112, kRegsLoad = 80;
static_assert(8 * (kRegsSoft + kRegsLoad) <= 16 * kRegsLaunch, "no more than the block was launched with");
constexpr uint32_t kHalf = kTile / 2;  // tokens of a thread
// What an item's beginning and end cost a CTA, in tiles (1, 2, 4, 6: 64 nodes over 8191 tokens 35.1, 33.5, 30.9, 31.3 us, 16
// Turbo8 trees 164, 160, 156, 159, 32 rows through windows of 4096 79.8, 78.8, 76.7, 77.7, of 128 -, 15.2, 18.7, 18.5), and the tiles of
// a stretch at least (1, 2, 3: a row through a window of 512 13.0, 13.5, 14.2, eight nodes over 1000 tokens 14.0, 14.7, 15.9).
constexpr uint32_t kLead = 4, kLeast = 1;
// How far a score may lie above what P and l refer to before O, in tensor memory, is read, scaled and written back: weights up to
// 2^8 cost bf16's hi + lo and fp32 sums no digit, and after an item's first tiles nearly none moves them.
constexpr float kSlack = 8.f;
constexpr float kSlack8 = 4.f, kUp8 = 11.f;  // Turbo8's weights of V: at most 2^(kUp8 + kSlack8) in f16

// Q (Turbo8: its lower part), then the ring of K (even slots; Turbo8: two parts) and V tiles as the products take them; Turbo8:
// then `raw` halves of tiles as they lie in the cache, on their way. (Loads into registers instead hang on the L1, which has a
// few KB beside this: 16 trees 174 us.)
template <int D, bool T8>
struct Ring {
  static constexpr uint32_t bytes = kTile * D * 2;  // K or V of a tile
  static constexpr uint32_t k_bytes = (T8 ? 2 : 1) * bytes;
  static constexpr uint32_t slots = T8 ? (D == 256 ? 2 : 4) : D == 256 ? 4 : 8;
  static constexpr uint32_t slab = kTile * 128, q_slab = kM * 128;  // 64 dims of all rows
  static constexpr uint32_t q = kM * D * 2;
  static constexpr uint32_t raw = T8 ? (D == 256 ? 2 : 6) : 0, raw_bytes = kTile * (D + D / 8);  // codes, then scales
  static constexpr uint32_t places = slots / 2 * (k_bytes + bytes), all = q + places + raw * raw_bytes;
  static __device__ __forceinline__ uint32_t at(uint32_t slot) { return slot / 2 * (k_bytes + bytes) + slot % 2 * k_bytes; }
  static constexpr uint32_t info = D == 256 ? 4 : 8;  // tiles whose notes are kept: the ring's and two of the softmax's
  static_assert(slots / 2 + 2 <= info, "notes");
};

// A row of the call as every CTA keeps it: position, sequence, which of its sequence's rows it is, and how many rows the
// block has that begins with it. Positions of more rows than shared memory has room for (a.near) are looked up again.
struct RowNote {
  uint32_t pos, bits;
  __device__ __forceinline__ uint32_t seq() const { return bits & 4095u; }
  __device__ __forceinline__ uint32_t index() const { return bits >> 12 & 2047u; }
  __device__ __forceinline__ uint32_t rows() const { return bits >> 23 & 255u; }
  __device__ __forceinline__ bool ok() const { return bits >> 31; }
};
static_assert(kMaxSeqs <= 4096 && kMaxQueries <= 2048, "bits of a row's note");
// Behind the prefix sums [n_rows + 1]: bits [n_rows], positions [n_rows].
struct RowNotes {
  uint32_t *bits, *pos;
  __device__ __forceinline__ RowNotes(const RowsAttend& a, const uint32_t* first)
      : bits(const_cast<uint32_t*>(first) + a.r.n_rows + 1), pos(a.near ? bits + a.r.n_rows : nullptr) {}
  __device__ __forceinline__ void put(uint32_t r, const RowNote& x) {
    bits[r] = x.bits;
    if (pos) pos[r] = x.pos;
  }
  __device__ __forceinline__ RowNote without_pos(uint32_t r) const { return {0, bits[r]}; }
  __device__ __forceinline__ RowNote get(const RowsAttend& a, uint32_t r) const {
    RowNote x = without_pos(r);
    x.pos = pos ? pos[r] : (uint32_t)a.r.pos[x.seq()] + x.index();
    return x;
  }
};
constexpr uint32_t rows_bytes(uint32_t n_rows, bool near) { return ((near ? 3 : 2) * n_rows + 1) * 4; }

// A block of rows and the tokens it sees: octets of eight tokens, nA first ones, then from b8 on.
struct Block {
  uint32_t row, rows, seq, index, pos, last;  // pos, last: positions of the first and the last row
  uint32_t nA, b8, octets;
  uint32_t from;  // the first token behind nA's that a row sees
  __device__ __forceinline__ uint32_t token(uint32_t o) const { return o < nA ? 8 * o : b8 + 8 * (o - nA); }
  __device__ __forceinline__ uint32_t tiles() const { return (octets + kOctets - 1) / kOctets; }
};
__device__ __forceinline__ Block block_of(const RowsAttend& a, uint32_t row, uint32_t rows, const RowNote& n) {
  Block b;
  b.row = row;
  b.rows = rows;
  b.seq = n.seq();
  b.index = n.index();
  b.pos = n.pos;
  b.last = n.pos + rows - 1;
  b.nA = b.b8 = b.from = 0;
  if (!a.parent) {
    b.from = b.pos + 1 > a.window ? b.pos + 1 - a.window : 0;
    b.b8 = b.from & ~7u;
    b.nA = a.n_first / 8 + (a.n_first % 8 != 0);
    if (b.nA > b.b8 / 8) b.nA = b.b8 = b.from = 0;  // the first tokens reach the window
  }
  b.octets = b.nA + (b.last - b.b8) / 8 + 1;
  return b;
}
// A CTA's stretch of an item.
struct Stretch {
  Block b;
  uint32_t g, t0, t1, c0, c1;
  // tiles of which every row of the block sees every token: [0, whole0) and [whole1, whole2)
  uint32_t whole0, whole1, whole2;
  __device__ __forceinline__ bool whole(uint32_t t) const { return t < whole0 || (t >= whole1 && t < whole2); }
};
__device__ __forceinline__ void set_whole(const RowsAttend& a, Stretch& s) {
  const Block& b = s.b;
  s.whole0 = 0;
  if (a.parent) {
    s.whole1 = 0;
    s.whole2 = (b.pos - b.index) / kTile;
  } else {
    if (b.nA) s.whole0 = a.n_first / kTile;
    // octets behind the first tokens' that lie in the last row's window and not behind the first row's position
    const uint32_t low = b.last + 1 > a.window ? b.last + 1 - a.window : 0, from = max(low, b.b8);
    const uint32_t o1 = b.nA + (from - b.b8 + 7) / 8, o2 = b.pos + 1 > b.b8 ? b.nA + (b.pos + 1 - b.b8) / 8 : 0;
    s.whole1 = (o1 + kOctets - 1) / kOctets;
    s.whole2 = o2 / kOctets;
  }
}
// A warp's way along the line: its CTA's part is [w, w1), cut into stretches. In shared memory, one for each warp: the
// registers are the loops'.
struct Walk {
  uint32_t w, w1, row, more;
  Stretch s;
};
__device__ __forceinline__ bool next(const RowsAttend& a, const uint32_t* first, uint32_t per, Walk& k, uint32_t lane) {
  __syncwarp();
  if (lane == 0) {
    const RowNotes notes(a, first);
    const uint32_t Hkv = a.c.Hkv, w1 = k.w1;
    uint32_t w = k.w, row = k.row, more = 0;
    while (w < w1 && !more) {
      while (first[row + 1] * Hkv <= w) ++row;
      const RowNote note = notes.get(a, row);
      const Block b = block_of(a, row, note.rows(), note);
      const uint32_t length = b.tiles() + kLead, in = w - first[row] * Hkv;
      const uint32_t at = in % length, used = min(length - at, w1 - w);
      k.s.b = b;
      k.s.g = in / length;
      k.s.t0 = max(at, kLead) - kLead;
      k.s.t1 = max(at + used, kLead) - kLead;
      k.s.c0 = (w - at + kLead) / per;
      k.s.c1 = (w - at + length - 1) / per;
      set_whole(a, k.s);
      w += used;
      more = k.s.t0 != k.s.t1;
    }
    k.w = w;
    k.row = row;
    k.more = more;
  }
  __syncwarp();
  return k.more;
}

// Shared memory behind Q and the ring.
template <uint32_t kInfo>
struct NotesOf {
  uint64_t full[8], empty[8], s_full[2], s_free[2], p_full[2], v_notes[kInfo], q_full;
  uint32_t tmem, last;
  uint32_t sums[kRowsThreads / 32];
  uint32_t valid[kInfo];             // octets of the tile that hold tokens
  uint32_t ahead[8];                 // Turbo8: of the tiles that are on their way
  alignas(16) uint8_t dirty[kInfo][kLoaders];  // V held something that is no number (a loader warp each)
  alignas(16) float k_scale[kInfo][kTile], v_exp[kInfo][kTile];  // Turbo8: 2^E of K's tokens, E of V's
  float q_scale[kM];
  alignas(16) float2 top[2][2][kM];  // a row's two threads' maxima
  float sum[kM];         // the second thread's sum
  int32_t parent[kMaxNodes];
  Walk walk[kRowsThreads / 32];
  int32_t pos[32], start[33];  // few rows: where they are
};

template <int D>
using Notes = NotesOf<Ring<D, false>::info>;

struct Work {  // the scratch
  // Sums of an item's first stretch and of the one that a CTA goes on with: [D / 8][columns][8], so that a
  // thread's 32 bytes lie beside its neighbours'. Items lie one behind another: block's rows x H columns.
  float* nat;
  float* cont;     // [CTAs][D / 8][128][8]
  float4* nat_ml;  // m, l, R of a column; l < 0: a row that is skipped
  float4* cont_ml;
  uint32_t* rec;   // [n_rows][Hkv]: the CTAs of the row's item, the block's rows, the row's place in it
};
__host__ __device__ inline Work work_of(uint8_t* p, uint32_t n_rows, uint32_t H, uint32_t D) {
  Work w;
  w.nat = reinterpret_cast<float*>(p);
  w.cont = w.nat + (size_t)n_rows * H * D;
  w.nat_ml = reinterpret_cast<float4*>(w.cont + (size_t)kMaxCtas * kM * D);
  w.cont_ml = w.nat_ml + (size_t)n_rows * H;
  w.rec = reinterpret_cast<uint32_t*>(w.cont_ml + kMaxCtas * kM);
  return w;
}
constexpr uint32_t kRecOk = 1u << 30;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// Arrive on bar when this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
  return h2;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 16-byte piece j of row r in a slab.
__device__ __forceinline__ uint32_t sw(uint32_t r, uint32_t j) { return r * 128 + ((j ^ (r & 7)) << 4); }
__device__ __forceinline__ uint32_t bits_below(int64_t n) { return n <= 0 ? 0u : n >= 8 ? 0xffu : (1u << n) - 1u; }

// One arrival for a warp, behind everything its lanes have done. (Each lane's own arrival is a turn at the barrier's word.)
__device__ __forceinline__ void arrive_warp(uint64_t* bar, uint32_t lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Bounded waits of one thread: after one has run out no other waits.
struct Waiter {
  uint64_t limit;
  int* status;
  bool dead;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!dead && !mbar_wait(bar, parity, limit)) {
      set_status(status, kStatusTimeout);
      dead = true;
    }
  }
};

// Where a half-tile h (2 n for tile n's K, 2 n + 1 for its V; n counts the CTA's tiles) lies in the ring.
template <int D, bool T8>
struct Place {
  uint32_t slot, turn;
  __device__ __forceinline__ explicit Place(uint32_t h) : slot(h % Ring<D, T8>::slots), turn(h / Ring<D, T8>::slots) {}
};

// ------------------------------------------------------------------ loaders

// Where the octets of four tiles lie, an octet a lane. A lookup is made four tiles ahead; nothing looks at it before.
struct Found {
  uint32_t row;  // a row is 128 bytes of K and V at least: no memory holds 2^32
  bool in;
};
__device__ __forceinline__ uint32_t look_up(const RowsAttend& a, const Block& b, uint32_t t, uint32_t lane) {
  const uint32_t o = t * kOctets + lane;
  if (!a.c.btab || o >= b.octets) return 0;
  return (uint32_t)a.c.btab[(size_t)b.seq * (a.c.capacity >> a.c.bt_shift) + (b.token(o) >> a.c.bt_shift)];
}
__device__ __forceinline__ Found found(const RowsAttend& a, const Block& b, uint32_t t, uint32_t lane, uint32_t block) {
  const uint32_t o = t * kOctets + lane, token = b.token(o);
  Found f = {b.seq * a.c.capacity + token, o < b.octets};
  if (a.c.btab) {
    if (f.in && block >= a.c.num_blocks) {
      set_status(a.status, kStatusRange);
      f.in = false;
    }
    f.row = block << a.c.bt_shift | (token & ((1u << a.c.bt_shift) - 1u));
  }
  return f;
}
// Rows of the octet at token t that are loaded: [lo, hi).
__device__ __forceinline__ void octet_rows(const RowsAttend& a, const Block& b, uint32_t o, uint32_t& lo, uint32_t& hi) {
  const uint32_t t = b.token(o);
  lo = 0;
  hi = min(8u, b.last - t + 1);
  if (o < b.nA) hi = min(8u, a.n_first - t);
  else if (b.from > t) lo = b.from - t;
}
__device__ __forceinline__ bool not_a_number_bf16(uint32_t w) {  // in either half, infinities too
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D>
__device__ __forceinline__ void load_plain(const RowsAttend& a, const uint32_t* first, uint32_t per, Walk& walk, uint8_t* ring,
                                           Notes<D>& sh, uint32_t tid, Waiter& wait) {
  constexpr uint32_t C = D / 8, STEP = kLoadThreads / C, J = kTile / STEP;  // pieces of a row, rows of a pass, passes
  const uint32_t warp = tid / 32, lane = tid % 32, r0 = tid / C, c = tid % C, q0 = warp * 32 / C / 8;
  const uint32_t to = (c / 8) * Ring<D, false>::slab + sw(r0, c % 8);  // STEP is a multiple of 8: piece j lies STEP * 128 behind
  static_assert(STEP % 8 == 0, "the swizzle of a thread's rows");
  const uint32_t stride = a.c.Hkv * D;
  const Stretch& s = walk.s;
  uint32_t n = 0, then = 0;
  Found now = {0, false};
  struct Pieces {  // the thread's, of a tile: their rows, which are there; the tile's octets, and whether it is seen to its end
    uint32_t row[J], in, valid;
    bool full;
  };
  const auto places = [&](uint32_t t) {
    Pieces x;
    const uint32_t i = (t - s.t0) % 4;
    if (i == 0) {
      now = found(a, s.b, t, lane, then);
      then = look_up(a, s.b, t + 4, lane);
    }
    x.full = s.whole(t);
    x.valid = __ballot_sync(0xffffffffu, now.in) >> (8 * i) & 0xffu;
    uint32_t rows = 0xffu;  // lane % 8's octet: rows of it that are loaded
    if (!x.full) {
      uint32_t lo, hi;
      octet_rows(a, s.b, t * kOctets + lane % 8, lo, hi);
      rows = bits_below(hi) & ~bits_below(lo);
    }
    if (!(x.valid >> (lane % 8) & 1)) rows = 0;
    x.in = 0;
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      const uint32_t q = q0 + j * STEP / 8;  // a warp's rows lie in one octet
      x.row[j] = __shfl_sync(0xffffffffu, now.row, 8 * i + q) + r0 % 8;
      x.in |= (__shfl_sync(0xffffffffu, rows, q) >> (r0 % 8) & 1u) << j;
    }
    return x;
  };
  const auto put = [&](const Pieces& x, uint32_t n, bool v) {
    const Place<D, false> at(2 * n + v);
    if (at.turn) wait(&sh.empty[at.slot], (at.turn - 1) & 1);
    uint8_t* slot = ring + Ring<D, false>::at(at.slot);
    const uint16_t* base = reinterpret_cast<const uint16_t*>(v ? a.c.v : a.c.k) + s.g * D + 8 * c;
    if (!v || x.full) {
      const uint32_t dst = smem_addr(slot) + to;
#pragma unroll
      for (uint32_t j = 0; j < J; ++j) cp16(dst + j * STEP * 128, x.in >> j & 1 ? base + (size_t)x.row[j] * stride : base, x.in >> j & 1);
      cp_arrive(&sh.full[at.slot]);
    } else {
      uint4 u[J];
#pragma unroll
      for (uint32_t j = 0; j < J; ++j) u[j] = x.in >> j & 1 ? load16(base + (size_t)x.row[j] * stride) : make_uint4(0u, 0u, 0u, 0u);
      bool bad = false;
#pragma unroll
      for (uint32_t j = 0; j < J; ++j) {
        uint32_t* w = &u[j].x;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
          if (not_a_number_bf16(w[e])) {
            bad = true;
            if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
            if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
          }
        *reinterpret_cast<uint4*>(slot + to + j * STEP * 128) = u[j];
      }
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) sh.dirty[n % Ring<D, false>::info][warp] = bad;
      tm_fence_shared();
      mbar_arrive(&sh.full[at.slot]);
    }
    if (!v && tid == 0) {  // an arrival that the notes are released by
      sh.valid[n % Ring<D, false>::info] = x.valid;
      mbar_arrive(&sh.full[at.slot]);
    }
  };
  // K of tile n + 1 before V of tile n: K's place is free as soon as its scores are there, V's only after its softmax (32 rows through
  // windows of 4096: 78 us, V of a tile straight after its K 89)
  while (next(a, first, per, walk, lane)) {
    then = look_up(a, s.b, s.t0, lane);
    Pieces x = places(s.t0);
    put(x, n, false);
#pragma unroll 1
    for (uint32_t t = s.t0; t < s.t1; ++t, ++n) {
      Pieces y = x;
      if (t + 1 < s.t1) {
        y = places(t + 1);
        put(y, n + 1, false);
      }
      put(x, n, true);
      x = y;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Turbo8: sixteen codes and their scale a piece. A thread copies the pieces that it will turn into f16 itself, Ring::raw halves
// of tiles ahead; its warp's rows' scales come with them. So only the warp waits. The order is K of tile 0, then K of tile n + 1
// and V of tile n in turn: K's place is free as soon as tile n's scores are there, V's only after its softmax.
template <int D>
struct LoadTurbo8 {
  using R = Ring<D, true>;
  static constexpr uint32_t C = D / 16, STEP = kLoadThreads / C, J = kTile / STEP;
  static constexpr uint32_t RW = 32 / C, S = D == 256 ? 2 : 1;  // a warp's rows of a pass; lanes that copy a row's scales
  const RowsAttend& a;
  uint8_t* ring;
  Notes<D>& sh;
  uint32_t tid, warp, lane, r0, c;
  Waiter& wait;
  const uint32_t* first;
  uint32_t per;
  Walk& walk;
  const Stretch& s;
  Found now;
  // the tile that is copied next, into a stage; how many there were
  uint32_t then, t, stage, tiles;
  bool more;
  struct Pieces {  // the thread's, of a tile: which are there (bit 31: the scales), their rows, the kv-head
    uint32_t in, row[J], scale_row, g;
  } kp, vp;

  __device__ __forceinline__ uint8_t* raw(uint32_t st) const { return ring + R::places + st * R::raw_bytes; }
  __device__ __forceinline__ void begin() {
    more = next(a, first, per, walk, lane);
    if (!more) return;
    t = s.t0;
    then = look_up(a, s.b, t, lane);
  }
  __device__ __forceinline__ void places() {
    const uint32_t i = (t - s.t0) % 4;
    if (i == 0) {
      now = found(a, s.b, t, lane, then);
      then = look_up(a, s.b, t + 4, lane);
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, now.in) >> (8 * i) & 0xffu;
    if (tid == 0) sh.ahead[tiles % 8] = valid;
    uint32_t rows = 0xffu;  // lane % 8's octet: rows of it that are loaded
    if (!s.whole(t)) {
      uint32_t lo, hi;
      octet_rows(a, s.b, t * kOctets + lane % 8, lo, hi);
      rows = bits_below(hi) & ~bits_below(lo);
    }
    if (!(valid >> (lane % 8) & 1)) rows = 0;
    kp.in = 0;
    kp.g = s.g;
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      const uint32_t q = warp * RW / 8 + j * STEP / 8;  // a warp's rows lie in one octet
      kp.row[j] = __shfl_sync(0xffffffffu, now.row, 8 * i + q) + r0 % 8;
      kp.in |= (__shfl_sync(0xffffffffu, rows, q) >> (r0 % 8) & 1u) << j;
    }
    const uint32_t r = scale_of();
    kp.scale_row = __shfl_sync(0xffffffffu, now.row, 8 * i + r / 8) + r % 8;
    kp.in |= (__shfl_sync(0xffffffffu, rows, r / 8) >> (r % 8) & (lane < 8 * S ? 1u : 0u)) << 31;
  }
  // The row of the tile whose scales the lane copies, 16 bytes of them or (D = 64) 8: one of its warp's eight.
  __device__ __forceinline__ uint32_t scale_of() const {
    const uint32_t k = lane / S % 8;
    return warp * RW + k % RW + k / RW * STEP;
  }
  __device__ __forceinline__ void copy(const Pieces& x, const uint8_t* codes, const uint16_t* scales) {
    codes += x.g * D + 16 * c;
    scales += x.g * C + lane % S * 8;
    const uint32_t to = smem_addr(raw(stage));
#pragma unroll
    for (uint32_t j = 0; j < J; ++j)
      cp16(to + (j * kLoadThreads + tid) * 16, x.in >> j & 1 ? codes + (size_t)x.row[j] * (a.c.Hkv * D) : codes, x.in >> j & 1);
    if (lane < 8 * S) {
      const bool here = x.in >> 31;
      const uint16_t* from = here ? scales + (size_t)x.scale_row * a.c.sstride : scales;
      const uint32_t dst = to + kTile * D + scale_of() * (D / 8) + lane % S * 16;
      if constexpr (D != 64) cp16(dst, from, here);
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(from), "r"(here ? 8 : 0) : "memory");
    }
  }
  __device__ __forceinline__ void copied() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + 1 == R::raw ? 0 : stage + 1;
  }
  __device__ __forceinline__ void copy_k() {  // of the next tile, if there is one
    vp = kp;
    if (more) {
      places();
      copy(kp, a.c.k, a.c.ks);
      ++tiles;
      if (++t == s.t1) begin();
    }
    copied();
  }
  __device__ __forceinline__ void copy_v(bool any) {  // of the tile before that
    if (any) copy(vp, a.c.v, a.c.vs);
    copied();
  }
  // A half of tile n into the ring, as f16 over 2^E. A code has 4 bits and a scale 8, their product 12, one more than f16: K goes in as
  // two, with the scale's upper seven bits and with its last. K's arrival releases its scales and what octets are there, V's exponents have a
  // barrier of their own: they are known before their place in the ring is free.
  template <uint32_t V>
  __device__ __forceinline__ void put(uint32_t n, uint32_t st) {
    const uint8_t* from = raw(st);
    uint32_t sc[J], mx[(J + 1) / 2], f[J], last[J], bad = 0;
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) sc[j] = *reinterpret_cast<const uint16_t*>(from + kTile * D + (r0 + j * STEP) * (D / 8) + 2 * c);
    // a token's largest scale, two pieces at once, from the lanes that have them; those that are no numbers do not count
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      uint32_t m = sc[j] & 0x7fffu;
      if (m >= 0x7f80u) {
        m = 0;
        bad = 1;
      }
      mx[j / 2] = j % 2 ? mx[j / 2] | m << 16 : m;
    }
#pragma unroll
    for (uint32_t m = 1; m < C; m <<= 1)
#pragma unroll
      for (uint32_t j = 0; j < (J + 1) / 2; ++j) mx[j] = __vmaxu2(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], m));
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      const int e = min(max((int)(mx[j / 2] >> (j % 2 ? 23 : 7) & 255u) - 127, -126), 126);
      if (c == 0) {
        if (V) sh.v_exp[n % R::info][r0 + j * STEP] = (float)e;
        else sh.k_scale[n % R::info][r0 + j * STEP] = pow2(e);
      }
      const bool number = (sc[j] & 0x7f80u) != 0x7f80u;
      const float full = bf16f(sc[j]);
      if (V) {
        const float y = number ? full * pow2(-e) : 0.f;
        f[j] = pack_f16(y, y);
      } else {
        const float seven = number ? bf16f(sc[j] & 0xfffeu) : full, rest = number ? full - seven : 0.f;
        f[j] = pack_f16(seven * pow2(-e), seven * pow2(-e));
        last[j] = pack_f16(rest * pow2(-e), rest * pow2(-e));
      }
    }
    if (V) arrive_warp(&sh.v_notes[n % R::info], lane);
    const Place<D, true> at(2 * n + V);
    if (at.turn) wait(&sh.empty[at.slot], (at.turn - 1) & 1);
    uint8_t* slab = ring + R::at(at.slot) + (c / 4) * R::slab;
    const uint32_t j8 = (c % 4) * 2;
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(from + (j * kLoadThreads + tid) * 16);
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
      if (V) {
        uint32_t nan = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // codes 0x7f and 0xff
        if (nan) {
          bad = 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] &= ~__vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        }
      }
      const uint32_t r = r0 + j * STEP;
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        uint32_t x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = e4m3_to_f16x2(w[2 * h + i / 2] >> (16 * (i % 2)));
          y[i] = hmul2(x[i], f[j]);
        }
        *reinterpret_cast<uint4*>(slab + sw(r, j8 + h)) = make_uint4(y[0], y[1], y[2], y[3]);
        if (!V) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = hmul2(x[i], last[j]);
          *reinterpret_cast<uint4*>(slab + R::bytes + sw(r, j8 + h)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
    if (V) {
      const bool any = __any_sync(0xffffffffu, bad);
      if (lane == 0) sh.dirty[n % R::info][warp] = any;
    }
    if (!V && tid == 0) sh.valid[n % R::info] = sh.ahead[n % 8];
    tm_fence_shared();
    arrive_warp(&sh.full[at.slot], lane);
  }
  __device__ __forceinline__ void run() {
    constexpr uint32_t N = R::raw;  // halves on their way: K0, K1, V0, K2, V1, ...
    stage = tiles = 0;
    begin();
    copy_k();
#pragma unroll 1
    for (uint32_t i = 1; i < N; ++i) {
      if (i % 2) copy_k();
      else copy_v(i / 2 - 1 < tiles);
    }
    uint32_t st = 0, q = 0;  // the half that is put: its stage, its number
    const auto landed = [&] {
      asm volatile("cp.async.wait_group %0;" ::"n"(N - 1) : "memory");
      __syncwarp();
    };
    const auto done = [&] {  // a half, and half q + N after it
      __syncwarp();          // its scales have been read
      st = st + 1 == N ? 0 : st + 1;
      if ((q + N) % 2) copy_k();
      else copy_v((q + N) / 2 - 1 < tiles);
      ++q;
    };
    landed();
    if (tiles) put<0>(0, st);
    done();
#pragma unroll 1
    for (uint32_t n = 0; n < tiles; ++n) {
      landed();
      if (n + 1 < tiles) put<0>(n + 1, st);
      done();
      landed();
      put<1>(n, st);
      done();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// ------------------------------------------------------------------ the join

// Columns' parts added up. A lane has eight dims, so D / 8 lanes a column and 256 / D columns a warp; `teams` warps of a
// CTA, one of them `team`, take a column's parts in turn. Little code on purpose: it runs once, as fast as its instructions come
// (32 dims a lane, four columns a warp, unrolled: 16 Turbo8 trees 168 us, with this 144).
// Column c = row H + head of the output, whose item lies in CTAs c0 .. c0 + n - 1 (0: none) and has `cols` columns from
// `first` on, this one the col-th. sync: of the CTA's eight warps, which come here together; sums theirs.
template <int D>
constexpr uint32_t kJoinColumns = 256 / D;
__device__ __forceinline__ void load_part(const float* p, bool wide, float (&x)[8]) {  // written by other SMs: from the L2
  if (wide) {
    asm volatile("ld.relaxed.gpu.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
  } else {
    const float4 u = __ldcg(reinterpret_cast<const float4*>(p)), v = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  }
}
template <int D, bool T8, typename Sync>
__device__ __forceinline__ void join_columns(const RowsAttend& a, const Work& work, uint32_t warp, uint32_t teams, uint32_t lane,
                                             uint32_t c, uint32_t c0, uint32_t n, uint32_t cols, uint32_t col, size_t first,
                                             float (*sums)[8][32], Sync&& sync) {
  constexpr uint32_t L = D / 8;
  const uint32_t piece = lane % L, team = warp % teams, most = __reduce_max_sync(0xffffffffu, n);
  uint4 gate = make_uint4(0, 0, 0, 0);
  if (a.gate && n && team == 0) gate = *reinterpret_cast<const uint4*>(a.gate + (size_t)c * a.gate_stride + 8 * piece);
  const auto ml = [&](uint32_t k) { return __ldcg(k ? work.cont_ml + (size_t)(c0 + k) * kM + col : work.nat_ml + first + col); };
  // the largest maximum and (T8) V's relative to it, the sum: a part each of the column's lanes, in rounds
  const float4 mine = piece < n ? ml(piece) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  bool ok = n > 0;
  float M = -INFINITY, V = -INFINITY, l = 0.f;
#pragma unroll 1
  for (uint32_t k = piece; k < n; k += L) {
    const float4 x = k < L ? mine : ml(k);
    if (x.y < 0.f) ok = false;
    M = fmaxf(M, x.x);
  }
#pragma unroll
  for (uint32_t w = 1; w < L; w <<= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    ok &= __shfl_xor_sync(0xffffffffu, ok, w);
  }
  const float mu = finite_or_0(M);
  const auto exponent = [&](const float4& x) { return T8 ? x.z + (finite_or_0(x.x) - mu) : x.x - mu; };  // of its sums O
#pragma unroll 1
  for (uint32_t k = piece; k < n; k += L) {
    const float4 x = k < L ? mine : ml(k);
    if (T8) V = fmaxf(V, exponent(x));
    l += x.x == -INFINITY ? x.y : x.y * ex2(x.x - mu);  // no score that is a number: 0 of no token, or NaN
  }
#pragma unroll
  for (uint32_t w = 1; w < L; w <<= 1) {
    if (T8) V = fmaxf(V, __shfl_xor_sync(0xffffffffu, V, w));
    l += __shfl_xor_sync(0xffffffffu, l, w);
  }
  const float down = T8 ? finite_or_0(V) : 0.f;
  const auto factor = [&](const float4& y) {
    if (y.x == -INFINITY || (T8 && y.z == -INFINITY)) return 0.f;
    return fmaxf(ex2(exponent(y) - down), 1.4e-45f);  // an infinity counts, however small its weight
  };
  const float own = factor(mine);
  float x[8] = {};
#pragma unroll 4
  for (uint32_t k = team; k < most; k += teams) {
    float f = __shfl_sync(0xffffffffu, own, min(k, L - 1), L), u[8] = {};
    if (k < n) {
      load_part((k ? work.cont + (size_t)(c0 + k) * kM * D + (piece * kM + col) * 8 : work.nat + first * D + (piece * cols + col) * 8),
                a.wide, u);
      if (k >= L) f = factor(ml(k));
      if (f != 0.f)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(u[e], f, x[e]);
    }
  }
  if (teams > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][e][lane] = x[e];
    sync();
    if (team) return;
#pragma unroll 1
    for (uint32_t k = 1; k < teams; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += sums[warp + k][e][lane];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l, up = T8 ? ex2(0.5f * down) : 1.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = l == 0.f ? 0.f : T8 ? x[e] * inv * up * up : x[e] * inv;
  if constexpr (T8) {  // rotated back: dim 8 piece + e
#pragma unroll
    for (int hb = 1; hb < 8; hb <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(e & hb)) {
          const float u = x[e], w = x[e + hb];
          x[e] = u + w;
          x[e + hb] = u - w;
        }
#pragma unroll 1
    for (uint32_t w = 1; w < L; w <<= 1) {
      const float sign = lane & w ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], sign, __shfl_xor_sync(0xffffffffu, x[e], w));
    }
    const float norm = rsqrtf((float)D);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= norm;
  }
  if (!ok) return;
  if (a.gate) {
    float g[8];
    unpack8(gate, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= sigmoidf_(g[e]);
  }
  *reinterpret_cast<uint4*>(a.out + (size_t)c * D + 8 * piece) = pack8(x);
}

// ------------------------------------------------------------------ softmax

// V's elements of a half of a tile (tokens j0 ..) that are no numbers, which the loaders took out: weight w[j] times each
// for the rows that see it (bit j of vis). Runs after the tile's product; rare, so plain and slow.
template <int D, bool T8>
__device__ __noinline__ void mend(const RowsAttend& a, const Block& b, uint32_t g, uint32_t t, uint32_t j0, uint32_t valid,
                                  uint32_t vis, const float* w, uint32_t o_col) {
#pragma unroll 1
  for (uint32_t j = 0; j < kHalf; ++j) {
    const uint32_t q = (j0 + j) / 8;
    if (!(valid >> q & 1)) continue;
    const uint32_t tok = b.token(t * kOctets + q) + j % 8;
    const bool see = vis >> j & 1;
    size_t row;
    if (!__any_sync(0xffffffffu, see) || tok > b.last || !cache_row(a.c, b.seq, tok, row)) continue;
    const size_t at = (row * a.c.Hkv + g) * D;
#pragma unroll 1
    for (uint32_t d = 0; d < D; ++d) {
      float x;
      if constexpr (T8) x = e4m3_pair_value(a.c.v[at + d]).x * bf16f(a.c.vs[row * a.c.sstride + g * (D / 16) + d / 16]);
      else x = bf16f(reinterpret_cast<const uint16_t*>(a.c.v)[at + d]);
      if (fabsf(x) < INFINITY) continue;
      const float o = __uint_as_float(tm_ld1(o_col + d));
      tm_st1(o_col + d, __float_as_uint(see ? fmaf(w[j], x, o) : o));
      tm_stored();
    }
  }
}

// O of a stretch over a bf16 cache where infinities among V that its tiles hold as they lie have left NaN (hi and lo of a
// weight times one, and 0 or less times one): every infinity and NaN among the values that a row sees is added to it, whatever its
// weight, the first in the NaN's place. A warp's 32 rows and its half of O's columns, D / 64 a lane as V is looked through, eight
// tokens at a time (the CTA's other warps wait meanwhile, so a long stretch must not take their time limit); a column that every
// row holds for good is passed over. Rare, so plain.
template <int D>
__device__ __noinline__ void put_infinities(const RowsAttend& a, const Stretch& st, uint32_t half, bool live, uint32_t p,
                                            uint64_t line0, uint64_t line1, uint32_t o_col) {
  constexpr uint32_t K = D / 64;
  struct alignas(2 * K) Values {
    uint16_t v[K];
  };
  const Block& b = st.b;
  const uint32_t lane = threadIdx.x % 32, c0 = half * (D / 2);
  constexpr uint32_t kNone = 0x7fc00001u;  // a NaN that is the sum's own; the matrix unit's is 0x7fffffff
  uint32_t held = 0;  // two bits a column of the lane: what all rows have there, 1 and 2 an infinity of a sign, 3 NaN
  const auto sees = [&](uint32_t tok) {
    if (!live) return false;
    if (a.parent) {
      const uint32_t start = b.pos - b.index, off = tok - start;
      return tok < start || (off < 64 ? line0 >> off & 1 : off < 128 && (line1 >> (off - 64) & 1));
    }
    return tok <= p && ((uint64_t)tok + a.window > p || tok < a.n_first);
  };
#pragma unroll 1
  for (uint32_t o = st.t0 * kOctets; o < min(st.t1 * kOctets, b.octets); ++o) {
    const uint32_t t0 = b.token(o);
    size_t row;
    if (!cache_row(a.c, b.seq, t0, row)) continue;  // pages hold whole octets
    const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v) + (row * a.c.Hkv + st.g) * D + c0 + lane * K;
    Values x[8];
    uint32_t seen = 0;
    bool any = false;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const bool one = __any_sync(0xffffffffu, sees(t0 + j));  // so the token is in the cache
      seen |= (uint32_t)one << j;
      x[j] = one ? *reinterpret_cast<const Values*>(v + (size_t)j * a.c.Hkv * D) : Values{};
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
#pragma unroll
      for (uint32_t e = 0; e < K; ++e) any |= (x[j].v[e] & 0x7f80u) == 0x7f80u && (held >> (2 * e) & 3u) != 3u;
    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll 1
    for (uint32_t j = 0; j < 8; ++j) {
      if (!(seen >> j & 1)) continue;
      const bool see = sees(t0 + j);
      const Values u8 = *reinterpret_cast<const Values*>(v + (size_t)j * a.c.Hkv * D);
#pragma unroll
      for (uint32_t e = 0; e < K; ++e) {
        const float x = bf16f(u8.v[e]);
        const uint32_t has = held >> (2 * e) & 3u, want = x != x ? 3u : x > 0.f ? 1u : 2u;
        uint32_t who = __ballot_sync(0xffffffffu, !(fabsf(x) < INFINITY) && has != 3u && has != want);
        while (who) {
          const uint32_t from = __ffs(who) - 1, col = o_col + c0 + from * K + e;
          who &= who - 1;
          const float y = __shfl_sync(0xffffffffu, x, from);
          uint32_t u = tm_ld1(col);
          if (see && u != kNone) {
            const float o = __uint_as_float(u), sum = o == o ? o + y : y;
            u = sum == sum ? __float_as_uint(sum) : kNone;
          }
          tm_st1(col, u);
          tm_stored();
          const bool nan = __all_sync(0xffffffffu, !live || u == kNone);
          const bool same = __all_sync(0xffffffffu, !live || __uint_as_float(u) == y);
          if (lane == from) held = (held & ~(3u << (2 * e))) | (nan ? 3u : !same ? 0u : y > 0.f ? 1u : 2u) << (2 * e);
        }
      }
    }
  }
}

// Thread tid of 256: row (TMEM lane) tid % 128, half tid / 128 of each tile's tokens and of O's columns.
template <int D, bool T8>
struct Softmax {
  const RowsAttend& a;
  uint8_t* q_sm;
  Notes<D>& sh;
  uint32_t tid, lane, tmem, group;  // tmem: the warp's lanes of it
  Waiter& wait;
  float scale;
  uint32_t row, half, pair;  // pair: the barrier of the warp and its other half
  // the thread's row
  uint32_t p;             // its position
  bool live, skip;        // it is one of the block's; it is skipped
  uint64_t line0, line1;  // tree: the nodes that it sees
  float m, l, R;

  __device__ __forceinline__ uint32_t s_col(uint32_t n) const { return tmem + (n & 1) * kTile + half * kHalf; }
  // Turbo8: over the S that it is made of, beside q's upper part
  __device__ __forceinline__ uint32_t p_col(uint32_t n) const { return tmem + (T8 ? 0 : 128) + (n & 1) * 64 + half * (kHalf / 2); }
  __device__ __forceinline__ uint32_t o_col() const { return tmem + 256; }

  // Each thread copies the pieces that it goes on with: four lanes a column, sixteen dims of each 64 a lane.
  __device__ __forceinline__ void put_q(const Block& b, uint32_t g) {
    constexpr uint32_t P = D / 64;
    // Turbo8: a warp and its other half take the columns of their lanes of tensor memory
    constexpr uint32_t STEP = T8 ? 8 : kSoft / 4, TIMES = kM * 4 / kSoft;
    const uint32_t cols = b.rows * group, l4 = tid & 3, from = T8 ? row / 32 * 32 + 16 * half + lane / 4 : tid / 4;
    const auto piece = [&](uint32_t col, uint32_t i) {
      return reinterpret_cast<uint4*>(q_sm + i / 2 * Ring<D, T8>::q_slab + sw(col, 2 * l4 + i % 2));
    };
    for (uint32_t k = 0, col = from; k < TIMES && col < cols; ++k, col += STEP) {
      const uint16_t* q = a.q + ((size_t)(b.row + col / group) * a.H + g * group + col % group) * D + 16 * l4;
#pragma unroll
      for (uint32_t i = 0; i < 2 * P; ++i) cp16(smem_addr(piece(col, i)), q + 64 * (i / 2) + 8 * (i % 2), true);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (T8) {
      // The rotated q over the power of two of its largest value, as hi + lo f16: hi through this memory into tensor memory, a thread
      // half of its row, then lo in its place. Meanwhile lo lies where O will (registers that went to local memory, and barriers
      // of all 256 threads: chunks of 100 to 257 rows 70 us, with this 68).
      constexpr uint32_t W = 16, N = D == 256 ? 2 : 1;  // words at once, times (D = 64: half of them are lo)
      const uint32_t aside = o_col() + half * (D / 2);
      if (row / 32 * 32 < cols) {
#pragma unroll 1
        for (uint32_t k = 0; k < TIMES && from - lane / 4 + STEP * k < cols; ++k) {
          const uint32_t col = from + STEP * k;
          float2 x[D / 8];
          float mx = 0.f;
#pragma unroll
          for (uint32_t i = 0; i < 2 * P; ++i) {
            const uint4 u = col < cols ? *piece(col, i) : make_uint4(0u, 0u, 0u, 0u);
            x[4 * i] = make_float2(bf16lo(u.x), bf16hi(u.x));
            x[4 * i + 1] = make_float2(bf16lo(u.y), bf16hi(u.y));
            x[4 * i + 2] = make_float2(bf16lo(u.z), bf16hi(u.z));
            x[4 * i + 3] = make_float2(bf16lo(u.w), bf16hi(u.w));
          }
          wht_quad<D>(x, lane);
#pragma unroll
          for (uint32_t i = 0; i < D / 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int e2 = min(max((int)((__float_as_uint(mx) >> 23) & 255) - 127, -126), 126);
          const float f = pow2(-e2);
          if (l4 == 0 && col < cols) sh.q_scale[col] = pow2(e2);
#pragma unroll
          for (uint32_t n = 0; n < N; ++n) {
            uint32_t lo[W] = {};
#pragma unroll
            for (uint32_t i = 0; i < 2 * P / N; ++i) {
              uint32_t hi[4];
#pragma unroll
              for (uint32_t j = 0; j < 4; ++j) {
                const float2 y = x[4 * (i + n * (2 * P / N)) + j];
                const float u = y.x * f, v = y.y * f;
                hi[j] = pack_f16(u, v);
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
                lo[4 * i + j] = pack_f16(u - back.x, v - back.y);
              }
              if (col < cols) *piece(col, i + n * (2 * P / N)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            }
            tm_st16(aside + W * (N * k + n), lo);
          }
        }
        named_barrier(pair, 64);
#pragma unroll 1
        for (uint32_t w = half * (D / 4); w < (half + 1) * (D / 4); w += W) {
          uint32_t r[W];
#pragma unroll
          for (uint32_t k = 0; k < W / 4; ++k) {
            const uint32_t j = w / 4 + k;
            const uint4 u = *reinterpret_cast<const uint4*>(q_sm + j / 8 * Ring<D, T8>::q_slab + sw(row, j % 8));
            r[4 * k] = u.x, r[4 * k + 1] = u.y, r[4 * k + 2] = u.z, r[4 * k + 3] = u.w;
          }
          tm_st16(tmem + 128 + w, r);
        }
        tm_stored();
        named_barrier(pair, 64);
#pragma unroll 1
        for (uint32_t k = 0; k < TIMES && from - lane / 4 + STEP * k < cols; ++k) {
          const uint32_t col = from + STEP * k;
#pragma unroll
          for (uint32_t n = 0; n < N; ++n) {
            uint32_t lo[W];
            tm_ld16(aside + W * (N * k + n), lo);
            tm_loaded(lo);
#pragma unroll
            for (uint32_t i = 0; i < 2 * P / N; ++i)
              if (col < cols) *piece(col, i + n * (2 * P / N)) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          }
        }
      }
      tm_before_sync();
    }
    tm_fence_shared();
    arrive_warp(&sh.q_full, lane);
  }

  __device__ __forceinline__ void begin(const Block& b) {
    const uint32_t r = row / group;
    live = row < b.rows * group;
    p = b.pos + r;
    skip = false;
    line0 = line1 = 0;
    if (a.parent) {
      const uint32_t nodes = b.index + b.rows;  // at most kMaxNodes
      if (tid < nodes) sh.parent[tid] = a.parent[b.row - b.index + tid];
      named_barrier(1, kSoft);
      if (live) {
        for (int32_t i = (int32_t)(b.index + r);;) {
          if (i < 64) line0 |= 1ull << i;
          else line1 |= 1ull << (i & 63);
          const int32_t up = sh.parent[i];
          if (up == -1) break;
          if (up < 0 || up >= i) {
            skip = true;
            set_status(a.status, kStatusRange);
            break;
          }
          i = up;
        }
      }
    }
    if (T8 || a.parent) named_barrier(1, kSoft);  // q's scales are there; the next block's parents may come
    m = R = -INFINITY;
    l = 0.f;
  }

  // Tokens of the thread's half of tile t that its row sees, of those that are there.
  __device__ __forceinline__ uint32_t seen(const Block& b, uint32_t t, uint32_t valid) const {
    uint32_t bits = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < kHalf / 8; ++i) {
      const uint32_t q = half * (kHalf / 8) + i;
      if (!(valid >> q & 1)) continue;
      const int64_t t0 = b.token(t * kOctets + q);
      uint32_t x;
      if (a.parent) {
        const int64_t off = t0 - (int64_t)(b.pos - b.index);
        x = bits_below(-off);
        if (off > -8 && off < 128) {
          const uint64_t w = off < 0 ? line0 << -off : off < 64 ? line0 >> off | (off ? line1 << (64 - off) : 0) : line1 >> (off - 64);
          x |= (uint32_t)w & 0xffu;
        }
      } else {
        x = bits_below((int64_t)p + 1 - t0) & (~bits_below((int64_t)p + 1 - (int64_t)a.window - t0) | bits_below((int64_t)a.n_first - t0));
      }
      bits |= (x & 0xffu) << (8 * i);
    }
    return bits;
  }

  __device__ __forceinline__ void rescale_o(float f) {
#pragma unroll 1
    for (uint32_t c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
      uint32_t r[32];
      tm_ld32(o_col() + c, r);
      tm_loaded(r);
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
      tm_st32(o_col() + c, r);
    }
    tm_stored();
  }

  __device__ __forceinline__ void tile(const Stretch& st, uint32_t t, uint32_t n) {
    const bool busy = row - lane % 32 < st.b.rows * group;
    const bool all = st.whole(t);
    const Place<D, T8> pv(2 * n + 1);
    wait(&sh.s_full[n & 1], (n >> 1) & 1);
    tm_after_sync();
    const uint32_t valid = sh.valid[n % Ring<D, T8>::info];
    if (T8) wait(&sh.v_notes[n % Ring<D, T8>::info], n / Ring<D, T8>::info & 1);
    float s[kHalf];
    uint32_t vis = ~0u;
    if (busy) {
      uint32_t r[32];
      tm_ld32(s_col(n), r);
      tm_loaded(r);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r[i]);
      tm_before_sync();
    }
    if (!T8) arrive_warp(&sh.s_free[n & 1], lane);
    if (busy) {
      if constexpr (T8) {
        const float sc = scale * (live ? sh.q_scale[row] : 0.f);
#pragma unroll
        for (uint32_t j = 0; j < kHalf; j += 4) {
          const float4 k = *reinterpret_cast<const float4*>(&sh.k_scale[n % Ring<D, T8>::info][half * kHalf + j]);
          s[j] = s[j] * sc * k.x;
          s[j + 1] = s[j + 1] * sc * k.y;
          s[j + 2] = s[j + 2] * sc * k.z;
          s[j + 3] = s[j + 3] * sc * k.w;
        }
      }
      if (!all || valid != 0xffu) {
        vis = live && !skip ? seen(st.b, t, valid) : 0;
#pragma unroll
        for (uint32_t j = 0; j < kHalf; ++j) s[j] = vis >> j & 1 ? s[j] : -INFINITY;
      }
      // the largest score, and (T8) with V's exponent, of both threads of the row
      float2 top = make_float2(-INFINITY, -INFINITY);
      {
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (uint32_t j = 0; j < kHalf; j += 4) {
          float4 e;
          if (T8) e = *reinterpret_cast<const float4*>(&sh.v_exp[n % Ring<D, T8>::info][half * kHalf + j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = fmaxf(x[i], s[j + i]);
            if (T8) y[i] = fmaxf(y[i], s[j + i] + (i == 0 ? e.x : i == 1 ? e.y : i == 2 ? e.z : e.w));
          }
        }
        top.x = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (T8) top.y = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      }
      sh.top[n & 1][half][row] = top;
      named_barrier(pair, 64);
      if (T8) tm_after_sync();  // both halves of S have been loaded: P may come
      const float2 other = sh.top[n & 1][half ^ 1][row];
      top.x = fmaxf(top.x, other.x);
      top.y = fmaxf(top.y, other.y);
      float f = 1.f, sums[4] = {0.f, 0.f, 0.f, 0.f};  // f: what O is multiplied by
      if constexpr (T8) {
        const float mn = fmaxf(m, top.x), down = m - finite_or_0(mn);
        if (mn != m) {
          l *= m == -INFINITY ? 0.f : ex2(down);
          R += m == -INFINITY ? 0.f : down;  // R is relative to m, the sums O are not
          m = mn;
        }
        const float mu = finite_or_0(m), want = top.y - mu - kUp8;
        if (want > R && (want > R + kSlack8 || R == -INFINITY)) {
          f = R == -INFINITY ? 0.f : ex2(R - want);
          R = want;
        }
        const float ref = finite_or_0(R);
#pragma unroll
        for (uint32_t j = 0; j < kHalf; j += 4) {
          const float4 e = *reinterpret_cast<const float4*>(&sh.v_exp[n % Ring<D, T8>::info][half * kHalf + j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float d = s[j + i] - mu;
            sums[i] += ex2(d);
            s[j + i] = ex2(d + (i == 0 ? e.x : i == 1 ? e.y : i == 2 ? e.z : e.w) - ref);
          }
        }
      } else {
        const float mx = top.x * scale;
        if (mx > m && (mx > m + kSlack || m == -INFINITY)) {
          f = m == -INFINITY ? 0.f : ex2(m - mx);
          l *= f;
          m = mx;
        }
        const float ref = finite_or_0(m);
#pragma unroll
        for (uint32_t j = 0; j < kHalf; ++j) {
          s[j] = ex2(fmaf(s[j], scale, -ref));
          sums[j % 4] += s[j];
        }
      }
      l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
      if (!live) f = 1.f;  // whatever its scores are
      if (t != st.t0 && __any_sync(0xffffffffu, f != 1.f)) {
        const Place<D, T8> before(2 * n - 1);
        wait(&sh.empty[before.slot], before.turn & 1);
        tm_after_sync();
        rescale_o(f);
      }
      // bf16: the product that read this P two tiles ago was issued before these scores', whose arrival covers it
      uint32_t h[16];
      if constexpr (T8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = pack_f16(s[2 * i], s[2 * i + 1]);
        tm_st16(p_col(n), h);
      } else {
        uint32_t lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float u = s[2 * i], v = s[2 * i + 1];
          h[i] = pack_bf16(u, v);
          lo[i] = pack_bf16(u - bf16lo(h[i]), v - bf16hi(h[i]));
        }
        tm_st16(p_col(n), h);
        tm_st16(p_col(n) + 32, lo);
      }
      tm_stored();
      tm_before_sync();
    }
    bool dirty = false;
    // Before the arrival: behind it the slot may be filled again. Turbo8: of all warps, whether they have columns or not. With one place for V
    // its arrival says that the product of the tile before is complete; without that a wait for this tile's product, which tells phases
    // by their parity, could take the one before for it, and the next item's q would lie in O before O is made.
    if (T8 || (busy && !all)) wait(&sh.full[pv.slot], pv.turn & 1);
    if (busy && (T8 || !all)) {  // bf16: the other tiles have not been looked through
      const uint2 u = *reinterpret_cast<const uint2*>(sh.dirty[n % Ring<D, T8>::info]);
      dirty = (u.x | u.y) != 0;
    }
    arrive_warp(&sh.p_full[n & 1], lane);
    if (dirty) {
      wait(&sh.empty[pv.slot], pv.turn & 1);
      float w[kHalf];
#pragma unroll
      for (uint32_t j = 0; j < kHalf; ++j) w[j] = s[j];
#pragma unroll 1
      for (uint32_t h = 0; h < 2; ++h) {  // one thread of a row after the other
        tm_after_sync();
        if (half == h) mend<D, T8>(a, st.b, st.g, t, half * kHalf, valid, live ? vis : 0, w, o_col());
        tm_before_sync();
        named_barrier(pair, 64);
      }
      tm_after_sync();
    }
  }

  // a.here: the last of an item's CTAs adds its parts up. One item at most begins in CTA c0 and goes on behind it: its ticket.
  __device__ void finish(const Stretch& st) {
    const Work work = work_of(a.work, a.r.n_rows, a.H, D);
    const uint32_t cols = st.b.rows * group, n = st.c1 - st.c0 + 1;
    if (n > 1) {
      named_barrier(1, kSoft);  // the CTA's part lies before this, and the count's release and acquire put it before the last one's reads
      if (tid == 0) {
        const uint32_t had = count_up(a.tickets + st.c0);
        sh.last = had + 1 == n;
        if (had >= n) set_status(a.status, kStatusInvalid);
        if (had + 1 >= n) a.tickets[st.c0] = 0;
      }
    }
    named_barrier(1, kSoft);
    if (n > 1 && !sh.last) return;
    float(*sums)[8][32] = reinterpret_cast<float(*)[8][32]>(q_sm);  // the products are done with Q
    // as many warps a column as there are: at most eight columns, 256 / D of them a warp
    const uint32_t fours = (cols + kJoinColumns<D> - 1) / kJoinColumns<D>, teams = fours > 4 ? 1 : fours > 2 ? 2 : fours > 1 ? 4 : 8;
    const uint32_t col = tid / 32 / teams * kJoinColumns<D> + lane / (D / 8), r = st.b.row + col / group;
    const bool in = col < cols;
    join_columns<D, T8>(a, work, tid / 32, teams, lane, in ? r * a.H + st.g * group + col % group : 0, st.c0, in ? n : 0, cols,
                        in ? col : 0, (size_t)st.b.row * a.H + st.g * cols, sums, [] { named_barrier(1, kSoft); });
    named_barrier(1, kSoft);  // the sums are free
  }

  // The sums of a stretch, the last of whose tiles is tile n of the CTA.
  __device__ __forceinline__ void store(const Stretch& st, uint32_t n) {
    const Place<D, T8> pv(2 * n + 1);
    wait(&sh.empty[pv.slot], pv.turn & 1);
    tm_after_sync();
    const uint32_t cols = st.b.rows * group;
    if (row - lane % 32 >= cols) return;
    if (half) sh.sum[row] = l;
    named_barrier(pair, 64);
    const Work work = work_of(a.work, a.r.n_rows, a.H, D);
    const bool nat = st.c0 == blockIdx.x;
    const size_t first = nat ? (size_t)st.b.row * a.H + st.g * cols : (size_t)blockIdx.x * kM;
    const uint32_t wide = nat ? cols : kM;
    float* to = (nat ? work.nat : work.cont) + first * D + row * 8;
    float2 odd[2] = {};  // NaN of an infinity or a NaN
    const auto write = [&] {
#pragma unroll 1
      for (uint32_t c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
        uint32_t r[32];
        tm_ld32(o_col() + c, r);
        tm_loaded(r);
        if (live) {
#pragma unroll
          for (uint32_t i = 0; i < 32; i += 8) {
            const uint32_t w[8] = {r[i], r[i + 1], r[i + 2], r[i + 3], r[i + 4], r[i + 5], r[i + 6], r[i + 7]};
            store32(to + (c + i) * (size_t)wide, a.wide, w);
          }
          if (!T8)
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 2)
              odd[i / 2 % 2] = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(0.f, 0.f), odd[i / 2 % 2]);
        }
      }
    };
    write();
    if constexpr (!T8) {
      const bool number = live && !skip && l == l;  // else the row is NaN by its scores, or not written
      const float all = (odd[0].x + odd[0].y) + (odd[1].x + odd[1].y);
      if (__any_sync(0xffffffffu, number && all != all)) {
        put_infinities<D>(a, st, half, number, p, line0, line1, o_col());
        write();
      }
    }
    if (live && !half) (nat ? work.nat_ml : work.cont_ml)[first + row] = make_float4(m, skip ? -1.f : l + sh.sum[row], R, 0.f);
    tm_before_sync();
  }
};

// ------------------------------------------------------------------ products

// A warp forms and waits, one lane issues.
template <int D, bool T8>
__device__ __forceinline__ void issue(const RowsAttend& a, const uint32_t* first, uint32_t per, Walk& walk, uint32_t lane, uint32_t q, uint32_t ring, Notes<D>& sh, uint32_t tmem, Waiter& wait) {
  constexpr uint32_t kQK = tm_idesc(!T8, false, kM, kTile), kPV = tm_idesc(!T8, true, kM, D);
  const uint64_t dq = tm_desc(q, 16, 1024);
  const Stretch& s = walk.s;
  uint32_t n = 0, items = 0;
  const auto values = [&](uint32_t i, bool add) {  // O += P V of tile i
    const Place<D, T8> v(2 * i + 1);
    wait(&sh.full[v.slot], v.turn & 1);
    wait(&sh.p_full[i & 1], (i >> 1) & 1);
    tm_after_sync();
    tm_fence_shared();
    const uint32_t p = tmem + (T8 ? 0 : 128) + (i & 1) * 64;
    const uint64_t dv = tm_desc(ring + Ring<D, T8>::at(v.slot), Ring<D, T8>::slab, 1024);
    if (elect_one()) {
#pragma unroll
      for (uint32_t k = 0; k < kTile / 16; ++k) {
        const uint64_t b = dv + k * 2048 / 16;
        tm_mma_ta(tmem + 256, p + 8 * k, b, kPV, add || k);
        if (!T8) tm_mma_ta(tmem + 256, p + 32 + 8 * k, b, kPV, true);
      }
      tm_commit(&sh.empty[v.slot]);
    }
    __syncwarp();
  };
  while (next(a, first, per, walk, lane)) {
    wait(&sh.q_full, items++ & 1);
    for (uint32_t t = s.t0; t < s.t1; ++t, ++n) {
      const Place<D, T8> k(2 * n);
      wait(&sh.full[k.slot], k.turn & 1);
      if (!T8) {
        if (n >= 2) wait(&sh.s_free[n & 1], ((n - 2) >> 1) & 1);
      } else if (t - s.t0 >= 2) {  // P of the tile before the last lay there; an item's first two tiles come after q, and that after all
        const Place<D, T8> v(2 * n - 3);
        wait(&sh.empty[v.slot], v.turn & 1);
      }
      tm_after_sync();
      tm_fence_shared();
      const uint64_t dk = tm_desc(ring + Ring<D, T8>::at(k.slot), 16, 1024);
      const uint32_t to = tmem + (n & 1) * kTile;
      const auto q_at = [](uint32_t i) { return ((i / 4) * Ring<D, T8>::q_slab + (i % 4) * 32) / 16; };  // descriptors count in 16 bytes
      const auto k_at = [](uint32_t i) { return ((i / 4) * Ring<D, T8>::slab + (i % 4) * 32) / 16; };
      if (elect_one()) {
        if constexpr (T8) {  // the small terms first: q's lower part and the scales' last bits
#pragma unroll
          for (uint32_t i = 0; i < D / 16; ++i) tm_mma(to, dq + q_at(i), dk + k_at(i), kQK, i != 0);
#pragma unroll
          for (uint32_t i = 0; i < D / 16; ++i) tm_mma_ta(to, tmem + 128 + 8 * i, dk + Ring<D, T8>::bytes / 16 + k_at(i), kQK, true);
#pragma unroll
          for (uint32_t i = 0; i < D / 16; ++i) tm_mma_ta(to, tmem + 128 + 8 * i, dk + k_at(i), kQK, true);
        } else {
#pragma unroll
          for (uint32_t i = 0; i < D / 16; ++i) tm_mma(to, dq + q_at(i), dk + k_at(i), kQK, i != 0);
        }
        tm_commit(&sh.s_full[n & 1]);
        mbar_arrive(&sh.s_full[n & 1]);  // passes the loaders' notes on
        tm_commit(&sh.empty[k.slot]);
      }
      __syncwarp();
      if (t != s.t0) values(n - 1, t - 1 != s.t0);
    }
    values(n - 1, s.t1 - 1 != s.t0);
  }
  if (n) {  // every product is complete before the tensor memory goes
    const Place<D, T8> last(2 * n - 1);
    wait(&sh.empty[last.slot], last.turn & 1);
  }
}

// ------------------------------------------------------------------ the kernel

template <int N>
__device__ __forceinline__ void set_registers() {
  if constexpr (N > kRegsLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, bool T8>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ RowsAttend a) {
  extern __shared__ uint8_t raw[];
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* q_sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  uint8_t* ring = q_sm + Ring<D, T8>::q;
  Notes<D>& sh = *reinterpret_cast<Notes<D>*>(q_sm + Ring<D, T8>::all);
  uint32_t* first = reinterpret_cast<uint32_t*>(&sh + 1);  // [n_rows + 1]
  RowNotes notes(a, first);
  if (tid == 0) {
    for (uint32_t i = 0; i < Ring<D, T8>::slots; ++i) {
      mbar_init(&sh.full[i], T8 ? kLoaders : kLoadThreads + (i % 2 == 0));
      mbar_init(&sh.empty[i], 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 2);
      mbar_init(&sh.s_free[i], kSoft / 32);
      mbar_init(&sh.p_full[i], kSoft / 32);
    }
    if (T8)
      for (uint32_t i = 0; i < Ring<D, T8>::info; ++i) mbar_init(&sh.v_notes[i], kLoaders);
    mbar_init(&sh.q_full, kSoft / 32);
    mbar_fence_init();
  }
  constexpr uint32_t kIssuer = kRowsThreads / 32 - 1;
  if (warp == kIssuer) tm_alloc(&sh.tmem, 512);
  tm_before_sync();
  __syncthreads();
  tm_after_sync();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_launch();

  // ---- the rows' places, looked up in shared memory, and the line of tiles
  const uint32_t group = a.H / a.c.Hkv, RB = kM / group;
  // Row r's note, and its tiles if a block begins with it.
  const auto row_tiles = [&](const Rows& here, uint32_t r) {
    uint32_t seq = 0, pos = 0, index = 0, left = 1, v = 0;
    RowKind kind = locate(here, a.c.capacity, r, seq, pos, index, left);
    if (kind == kRowOk && (index > r || (a.parent && index >= kMaxNodes))) kind = kRowBad;
    if (kind == kRowBad && blockIdx.x == 0) set_status(a.status, kStatusRange);
    RowNote x = {pos, seq | min(index, 2047u) << 12 | (uint32_t)(kind == kRowOk) << 31};
    if (kind == kRowOk && index % RB == 0) {
      uint32_t rows = min(min(min(RB, left), a.r.n_rows - r), a.c.capacity - pos);
      if (a.parent) rows = min(rows, kMaxNodes - index);
      v = block_of(a, r, rows, x).tiles() + kLead;
      x.bits |= rows << 23;
    }
    notes.put(r, x);
    return v;
  };
  Rows here = a.r;
  uint32_t base = 0;
  if (a.r.n_rows <= 32 && a.r.n_seqs <= 32) {
    // Few rows: every warp looks them up for itself, the same values into the same places, and goes on without the others
    if (lane < a.r.n_seqs) sh.pos[lane] = a.r.pos[lane];
    if (a.r.row_start) {
      if (lane < a.r.n_seqs) sh.start[lane] = a.r.row_start[lane];
      if (lane == 0) sh.start[a.r.n_seqs] = a.r.row_start[a.r.n_seqs];
      here.row_start = sh.start;
    }
    here.pos = sh.pos;
    __syncwarp();
    const uint32_t v = lane < a.r.n_rows ? row_tiles(here, lane) : 0;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= (uint32_t)o) x += y;
    }
    if (lane < a.r.n_rows) first[lane] = x - v;
    base = __shfl_sync(0xffffffffu, x, 31);
    if (lane == 0) first[a.r.n_rows] = base;
    __syncwarp();
  } else {
    int32_t* pos = reinterpret_cast<int32_t*>(ring);  // which is empty
    int32_t* start = pos + kMaxSeqs;
    for (uint32_t i = tid; i < a.r.n_seqs; i += kRowsThreads) pos[i] = a.r.pos[i];
    if (a.r.row_start)
      for (uint32_t i = tid; i <= a.r.n_seqs; i += kRowsThreads) start[i] = a.r.row_start[i];
    here.pos = pos;
    if (a.r.row_start) here.row_start = start;
    __syncthreads();
    for (uint32_t r0 = 0; r0 < a.r.n_rows; r0 += kRowsThreads) {
      const uint32_t r = r0 + tid, v = r < a.r.n_rows ? row_tiles(here, r) : 0;
      uint32_t x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= (uint32_t)o) x += y;
      }
      if (lane == 31) sh.sums[warp] = x;
      __syncthreads();
      uint32_t before = base;
#pragma unroll
      for (uint32_t w = 0; w < kRowsThreads / 32; ++w) {
        before += w < warp ? sh.sums[w] : 0;
        base += sh.sums[w];
      }
      if (r < a.r.n_rows) first[r] = before + x - v;
      if (r == a.r.n_rows - 1) first[r + 1] = before + x;
      __syncthreads();
    }
  }
  const uint32_t total = base * a.c.Hkv, per = max((total + gridDim.x - 1) / gridDim.x, kLeast);
  const Work work = work_of(a.work, a.r.n_rows, a.H, D);
  // every row's record for the join
  for (uint32_t i = blockIdx.x * kRowsThreads + tid; i < a.r.n_rows * a.c.Hkv; i += gridDim.x * kRowsThreads) {
    const uint32_t r = i / a.c.Hkv, g = i % a.c.Hkv;
    const RowNote x = notes.without_pos(r);
    const uint32_t off = x.index() % RB;
    const RowNote start = notes.without_pos(off <= r ? r - off : r);
    uint32_t rec = 0;
    if (x.ok() && off <= r && start.seq() == x.seq() && off < start.rows()) {
      const uint32_t b = r - off, length = first[b + 1] - first[b], w = first[b] * a.c.Hkv + g * length;
      rec = (w + kLead) / per | ((w + length - 1) / per) << 8 | off << 16 | (start.rows() - 1u) << 23 | kRecOk;
    }
    work.rec[i] = rec;
  }
  const uint64_t w64 = (uint64_t)blockIdx.x * per;
  Walk& walk = sh.walk[warp];
  if (lane == 0) {
    walk.w = (uint32_t)min(w64, (uint64_t)total);
    walk.w1 = (uint32_t)min(w64 + per, (uint64_t)total);
    uint32_t lo = 0, hi = a.r.n_rows;  // first[lo] Hkv <= w < first[hi] Hkv, if there is anything
    while (walk.w < walk.w1 && hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (first[mid] * a.c.Hkv <= walk.w) lo = mid;
      else hi = mid;
    }
    walk.row = lo;
  }
  Waiter wait{a.wait_ns, a.status, false};
  if (tid < kSoft) {
    set_registers<kRegsSoft>();
    Softmax<D, T8> x{a, q_sm, sh, tid, lane, tmem + ((32 * (warp % 4)) << 16), group, wait,
                     1.4426950408889634f / sqrtf((float)D), tid % kM, tid / kM, 2 + warp % 4};
    const Stretch& s = walk.s;
    uint32_t n = 0;
    while (next(a, first, per, walk, lane)) {
      x.put_q(s.b, s.g);
      x.begin(s.b);
      for (uint32_t t = s.t0; t < s.t1; ++t, ++n) x.tile(s, t, n);
      x.store(s, n - 1);
      if (a.here) x.finish(s);
    }
  } else if (warp == kIssuer) {
    issue<D, T8>(a, first, per, walk, lane, smem_addr(q_sm), smem_addr(ring), sh, tmem, wait);
  } else if (warp < kIssuer) {
    set_registers<kRegsLoad>();
    const uint32_t i = tid - kSoft;
    if constexpr (T8) {
      LoadTurbo8<D> x{a, ring, sh, i, i / 32, lane, i / (D / 16), i % (D / 16), wait, first, per, walk, walk.s, {0, false}};
      x.run();
    } else {
      load_plain<D>(a, first, per, walk, ring, sh, i, wait);
    }
  }
  tm_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    tm_after_sync();
    tm_free(tmem, 512);
  }
}

// Registers that leave it room beside a CTA of rows_kernel, so it waits for that on the SM.
template <int D, bool T8>
__global__ void __launch_bounds__(256, 5) join_kernel(const __grid_constant__ RowsAttend a, uint32_t teams) {
  __shared__ float sums[8][8][32];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t group = a.H / a.c.Hkv, c = (blockIdx.x * (8 / teams) + warp / teams) * kJoinColumns<D> + lane / (D / 8);
  const uint32_t r = c / a.H, h = c % a.H;
  const bool in = r < a.r.n_rows;
  const Work work = work_of(a.work, a.r.n_rows, a.H, D);
  pdl_wait();
  pdl_launch();
  const uint32_t rec = in ? work.rec[r * a.c.Hkv + h / group] : 0;
  const uint32_t c0 = rec & 255u, n = rec & kRecOk ? (rec >> 8 & 255u) - c0 + 1 : 0, off = rec >> 16 & 127u;
  const uint32_t cols = ((rec >> 23 & 127u) + 1) * group;
  join_columns<D, T8>(a, work, warp, teams, lane, c, c0, n, cols, off * group + h % group,
                      in ? (size_t)(r - off) * a.H + h / group * cols : 0, sums, [] { __syncthreads(); });
}

constexpr uint32_t kSmemMost = 227 * 1024;
template <int D, bool T8>
constexpr uint32_t smem_of(uint32_t n_rows, bool near) {
  return 1024 + Ring<D, T8>::all + sizeof(Notes<D>) + rows_bytes(n_rows, near);
}
template <int D, bool T8>
bool allow() {
  static_assert(smem_of<D, T8>(kMaxQueries, T8 && D == 256 ? false : true) <= kSmemMost, "shared memory of a CTA");
  return cudaFuncSetAttribute(rows_kernel<D, T8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) == cudaSuccess;
}

template <int D, bool T8>
cudaError_t launch(RowsAttend& a, cudaStream_t st) {
  static_assert(2 * kMaxSeqs * 4 + 4 <= Ring<64, true>::all - Ring<64, true>::q, "the rows' places");
  a.near = smem_of<D, T8>(a.r.n_rows, true) <= kSmemMost;
  cudaError_t e =
      launch_early(rows_kernel<D, T8>, dim3(std::min(a.sms, kMaxCtas)), kRowsThreads, smem_of<D, T8>(a.r.n_rows, a.near), st, a);
  if (e != cudaSuccess) return e;
  if (a.here) return cudaSuccess;
  // Up to eight warps a column, as long as the SMs hold all CTAs at once, four each (64 nodes over 8191 tokens, one after another:
  // 31.9 us, half as many warps 35.0, twice as many 34.1).
  const uint32_t warps = (a.r.n_rows * a.H + kJoinColumns<D> - 1) / kJoinColumns<D>;
  uint32_t teams = 8;
  while (teams > 1 && warps * teams > 32 * a.sms) teams /= 2;
  return launch_early(join_kernel<D, T8>, dim3((warps * teams + 7) / 8), 256, 0, st, a, teams);
}

}  // namespace

size_t rows_work_bytes(uint32_t n_rows, uint32_t H, uint32_t Hkv, uint32_t D) {
  return ((size_t)n_rows * H + kMaxCtas * kM) * (D * 4 + 16) + (size_t)n_rows * Hkv * 4;
}
cudaError_t rows_attend_attributes() {
  return allow<64, false>() && allow<64, true>() && allow<128, false>() && allow<128, true>() && allow<256, false>() &&
                 allow<256, true>()
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t rows_attend(const RowsAttend& args, cudaStream_t st) {
  RowsAttend a = args;
  // Eight columns, one for each warp of the softmax, are joined where their last part is made, as long as an SM has few items; more
  // columns, and the many items of an SM, by CTAs of their own. Single rows (bf16, 4 kv-heads of 256) through windows of 64 and 512, here and by a
  // second launch: 8 rows 12.7, 15.1 and 14.9, 16.4 us, 64 rows 23.2, 25.3 and 45.0, 46.5, 128 rows (3.4 items an SM) 39.7, 39.1 and 80.0, 78.0, 1024
  // rows 245, 227 and 517, 494; one kv-head of 64, windows of 64: 256 rows 18.8, 19.9, 512 rows 32.0, 30.1.
  a.here = a.H / a.c.Hkv * (a.r.row_start ? a.r.n_rows : 1) <= 8 && a.r.n_rows * a.c.Hkv < 3 * a.sms;
  const bool t8 = a.c.ks != nullptr;
#define CALL(DD) return t8 ? launch<DD, true>(a, st) : launch<DD, false>(a, st)
  switch (a.c.D) {
    case 64: CALL(64);
    case 128: CALL(128);
    case 256: CALL(256);
  }
#undef CALL
  return cudaErrorInvalidValue;
}

}  // namespace q35c
