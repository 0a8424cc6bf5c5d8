// Operators of a drafting serving loop beside those of cache_ops.h: rows normed and rotated
// on their way into a cache, the attention of drafted trees and of rows that see a sliding
// window, accepted rows moved together, and tokens sampled from logits. Launchers called by the
// C ABI (abi.cu); every argument has been checked there, what lies in device memory is checked
// by the kernels.
#pragma once

#include "cache_ops.h"

namespace q35c {

constexpr uint32_t kMaxNodes = 128;  // rows of a sequence's tree

struct RopeAppend {
  Cache c;
  Rows r;
  const int32_t* rope_pos;  // [n_rows], or null: the row's position in the cache
  const uint16_t* q;        // [n_rows][H] values of D, q_stride apart, or null
  const uint16_t* k;        // [n_rows][Hkv][D]
  const uint16_t* v;
  const uint16_t* q_norm;  // [D], or null: no norm
  const uint16_t* k_norm;
  uint16_t* q_out;  // [n_rows][H][D]
  uint16_t* k_out;  // [n_rows][Hkv][D], or null
  uint32_t H, q_stride, R;
  bool to_cache;  // else q_out and k_out alone
  bool wide_q, wide_kv, wide_out, wide_cache;  // rows are 32-byte aligned
  float eps;
  int* status;
  float inv_freq[128];
};
cudaError_t rope_append(const RopeAppend& a, cudaStream_t st);

struct Keep {
  Cache c;
  Rows r;               // a sequence's rows: the entries of its path
  const int32_t* path;  // [n_rows]
  uint16_t* bounds;     // as Append's, or null
  uint32_t blk_shift;
  int* status;
};
cudaError_t keep(const Keep& a, cudaStream_t st);

struct RowsAttend {
  Cache c;
  Rows r;
  const int32_t* parent;  // [n_rows]: a tree; null: a window
  uint32_t window, n_first;
  const uint16_t* q;     // [n_rows][H][D]
  const uint16_t* gate;  // as Attend's
  uint16_t* out;         // [n_rows][H][D]
  uint32_t* tickets;     // [kMaxCtas], zero between calls
  bool here;             // set by rows_attend(): the parts are added up by the last CTA of an item, not by a second launch
  bool near;             // set by rows_attend(): the rows' positions lie in shared memory
  uint8_t* work;         // rows_work_bytes
  bool wide;             // it is 32-byte aligned
  uint32_t sms;          // of the GPU
  uint32_t H, gate_stride;
  uint64_t wait_ns;
  int* status;
};
size_t rows_work_bytes(uint32_t n_rows, uint32_t H, uint32_t Hkv, uint32_t D);
cudaError_t rows_attend_attributes();  // once per device, before the first rows_attend
cudaError_t rows_attend(const RowsAttend& a, cudaStream_t st);

struct Sample {
  const uint16_t* logits;  // [n_rows] values of vocab, row_stride apart (0: all rows are one)
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* prob;
  uint32_t n_rows, vocab;
  uint64_t row_stride;
};
constexpr uint32_t kMaxVocab = 8 * 65520;  // eight CTAs a row at most; counts of a CTA's part fit 16 bits
constexpr uint32_t kMaxSampleRows = 65536;
cudaError_t sample(const Sample& a, cudaStream_t st);
cudaError_t sample_attributes();  // once per device, before the first sample

}  // namespace q35c
