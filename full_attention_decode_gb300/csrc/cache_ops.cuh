// Where a call's rows and a cache's tokens are (device side of cache_ops.h). Whatever
// the arrays in device memory hold, no address outside the cache is formed: a position
// outside [0, capacity) or a table entry outside the pool makes the caller skip the access
// and set the range status. Row starts that fall or lie below 0 leave a row with a position of one of the
// sequences from its pos on, or with none; which one is not said, and nothing reports it.
#pragma once

#include "cache_ops.h"
#include "common.cuh"

namespace q35c {

constexpr int kStatusInvalid = 1;  // QWEN35_ERR_INVALID_ARGUMENT

enum RowKind { kRowOk = 0, kRowSkip = 1, kRowBad = 2 };

// Row r's sequence and position, which of the sequence's rows it is and how many are left from
// it on; kRowSkip for a row no sequence has.
__device__ __forceinline__ RowKind locate(const Rows& w, uint32_t capacity, uint32_t r, uint32_t& seq, uint32_t& pos,
                                          uint32_t& index, uint32_t& left) {
  int64_t i = 0;
  index = 0;
  left = 1;
  if (!w.row_start) {
    seq = r;
  } else {
    if ((int64_t)r < w.row_start[0] || (int64_t)r >= w.row_start[w.n_seqs]) return kRowSkip;
    uint32_t lo = 0, hi = w.n_seqs;  // row_start[lo] <= r < row_start[hi]
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (w.row_start[mid] <= (int64_t)r) lo = mid;
      else hi = mid;
    }
    seq = lo;
    i = (int64_t)r - w.row_start[lo];
    index = (uint32_t)i;
    left = (uint32_t)(min((int64_t)w.row_start[lo + 1], (int64_t)w.n_rows) - r);
  }
  const int64_t p = (int64_t)w.pos[seq] + i;
  if (w.pos[seq] < 0 || i < 0 || p >= (int64_t)capacity) return kRowBad;
  pos = (uint32_t)p;
  return kRowOk;
}
__device__ __forceinline__ RowKind locate(const Rows& w, uint32_t capacity, uint32_t r, uint32_t& seq, uint32_t& pos) {
  uint32_t index, left;
  return locate(w, capacity, r, seq, pos, index, left);
}

// The cache row of token t (< capacity) of a sequence; false for a block outside the pool.
__device__ __forceinline__ bool cache_row(const Cache& c, uint32_t seq, uint32_t t, size_t& row) {
  if (!c.btab) {
    row = (size_t)seq * c.capacity + t;
    return true;
  }
  const uint32_t blk = (uint32_t)c.btab[(size_t)seq * (c.capacity >> c.bt_shift) + (t >> c.bt_shift)];
  if (blk >= c.num_blocks) return false;
  row = ((size_t)blk << c.bt_shift) | (t & ((1u << c.bt_shift) - 1u));
  return true;
}

// Launch with programmatic serialisation: the kernel may be scheduled while the one before it in the stream ends;
// it begins with pdl_wait(), so it sees everything that one wrote.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, uint32_t threads, uint32_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// One more at *p, and how many there were: what this CTA wrote before (a barrier puts its threads' writes
// before the counting thread's) is seen by who counts after it.
__device__ __forceinline__ uint32_t count_up(uint32_t* p) {
  uint32_t had;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(had) : "l"(p) : "memory");
  return had;
}

}  // namespace q35c
