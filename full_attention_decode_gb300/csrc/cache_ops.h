// Operators on KV caches by themselves (outside a layer forward): rows written to a
// cache and read back, blocks of a cache chosen by their key bounds, and the attention
// of new tokens over the cache. Launchers called by the C ABI (abi.cu); every argument
// has been checked there, what lies in device memory is checked by the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace q35c {

constexpr uint32_t kMaxSeqs = 4096;       // sequences of a call
constexpr uint32_t kMaxRows = 1u << 20;   // rows of an append or a read
constexpr uint32_t kMaxQueries = 2048;    // rows of a selection or an attention
constexpr uint32_t kMaxGroup = 16;        // q-heads of a kv-head
constexpr uint32_t kMaxSelect = 65536;    // blocks of a list

// The cache arrays of a batch: contiguous rows [n_seqs][capacity][Hkv][D], or pools of
// num_blocks blocks of 2^bt_shift rows with tables [n_seqs][capacity >> bt_shift].
struct Cache {
  uint8_t* k;
  uint8_t* v;
  uint16_t* ks;  // Turbo8 scales [rows][sstride], or null: bf16 rows
  uint16_t* vs;
  const int32_t* btab;
  uint32_t bt_shift, num_blocks, capacity, Hkv, D, sstride;
};

// The rows of a call: sequence b's are [row_start[b], row_start[b + 1]) at positions
// pos[b], pos[b] + 1, ...; row_start null: row b is sequence b's.
struct Rows {
  const int32_t* row_start;
  const int32_t* pos;
  uint32_t n_seqs, n_rows;
};

struct Append {
  Cache c;
  Rows r;
  const uint16_t* k;  // [n_rows][Hkv][D]
  const uint16_t* v;
  uint16_t* bounds;  // [rows >> blk_shift][Hkv][2][D], or null
  uint32_t blk_shift;
  bool wide;         // k and v are 32-byte aligned
  bool wide_bounds;  // set by append(): a CTA folds a block's bounds, not a team
  int* status;
};
cudaError_t append(const Append& a, cudaStream_t st);

struct Read {
  Cache c;
  Rows r;
  uint16_t* k;  // [n_rows][Hkv][D]
  uint16_t* v;
  bool wide;  // k and v are 32-byte aligned
  int* status;
};
cudaError_t read(const Read& a, cudaStream_t st);

struct Select {
  Cache c;
  Rows r;
  const uint16_t* bounds;
  const uint16_t* q;  // [n_rows][H][D]
  int32_t* blocks;    // [n_rows][Hkv][n_select]
  float* scores;      // work [n_rows * Hkv][nblk]
  double* exact;      // work, the same shape
  float* most;        // work [n_rows * Hkv][parts]: bounds of the blocks' sums of absolute terms
  uint32_t* tickets;  // [n_rows * Hkv], zero between calls
  uint32_t ctas;      // CTAs that fill the GPU
  uint32_t H, blk_shift, nblk, n_select, n_first, n_last;
  int* status;
};
cudaError_t select(const Select& a, cudaStream_t st);
cudaError_t select_attributes();  // once per device, before the first select
constexpr uint32_t kMaxItems = kMaxQueries * 8;  // of 8 kv-heads
constexpr uint32_t kMaxParts = 2048;   // parts of all items: at most one an item, or this many

struct Attend {
  Cache c;
  Rows r;
  const uint16_t* q;     // [n_rows][H][D]
  const uint16_t* gate;  // [n_rows][H] values of D, gate_stride apart, or null
  const int32_t* blocks; // [n_rows][Hkv][n_blocks], or null: every token
  uint16_t* out;         // [n_rows][H][D]
  uint32_t* tickets;     // [kMaxCtas], zero between calls
  float* parts;          // work [kMaxCtas][2][columns of an item][D + 4]
  uint32_t sms;          // of the GPU
  uint32_t H, gate_stride, n_blocks, blk_shift;
  int* status;
};
constexpr uint32_t kMaxCtas = 160;  // one on each SM of the largest sm_103 part
// Tiles of 16 tokens that a call's rows and kv-heads may have in all.
constexpr uint64_t kMaxTiles = 1ull << 31;
cudaError_t attend(const Attend& a, cudaStream_t st);
cudaError_t attend_attributes();  // once per device, before the first attend

}  // namespace q35c
