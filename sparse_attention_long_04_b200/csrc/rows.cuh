// Which sequence, position and cache row a query row or a logical key has: the geometry of
// decode (one new token per sequence) and of chunks (several new tokens per sequence, packed by
// cu_seqlens, over the same paged caches).
#pragma once
#include "sm100.cuh"

namespace dsa {

// Where the new tokens and the cached keys live.
struct PagedSeqs {
  int32_t chunk;               // 1: rows packed by cu_seqlens; 0: row b is sequence b
  int32_t batch;
  const int32_t* cu_seqlens;   // chunk: [batch + 1]
  const int32_t* seq_lens;     // [batch] context lengths, new tokens included
  const int32_t* block_table;  // [batch, max_blocks] or null (sequence b at b * max_seqlen)
  int32_t max_blocks;
  int32_t max_seqlen;
  int64_t num_kv_rows;
};

// Largest b with cu[b] <= row (empty sequences are passed over).
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int batch, int row) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// The same for a row that every lane of a (converged) warp asks for: 32 sequences a step instead of
// one, since each step is a trip to L2.
__device__ __forceinline__ int seq_of_warp_row(const int32_t* cu, int batch, int row) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool at = lane * step < n && cu[lo + lane * step] <= row;
    const int k = max(__popc(__ballot_sync(0xffffffffu, at)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Sequence of `row`, the same in all lanes of a converged warp, and its position; a context above max_seqlen (a caller error) is taken as
// max_seqlen and *bad set.  A position below 0 (more new tokens than context, or a row behind the
// last sequence) has no keys.
__device__ __forceinline__ void paged_row(const PagedSeqs& s, int row, int* b, int* pos,
                                          bool* bad) {
  int len, ahead;
  if (s.chunk) {
    *b = seq_of_warp_row(s.cu_seqlens, s.batch, row);
    ahead = s.cu_seqlens[*b + 1] - row;            // this row and the new tokens behind it
  } else {
    *b = row;
    ahead = 1;
  }
  len = s.seq_lens[*b];
  *bad = len > s.max_seqlen || len < ahead || ahead < 1;
  *pos = ahead < 1 ? -1 : min(len, s.max_seqlen) - ahead;
}

// Cache row of logical key `pos` of sequence b, -1 when its page lies outside the caches.
__device__ __forceinline__ int64_t paged_phys(const PagedSeqs& s, int b, int pos) {
  int64_t r;
  if (s.block_table != nullptr) {
    const int64_t blk = __ldg(s.block_table + static_cast<int64_t>(b) * s.max_blocks + pos / 64);
    if (blk < 0) return -1;
    r = blk * 64 + pos % 64;
  } else {
    r = static_cast<int64_t>(b) * s.max_seqlen + pos;
  }
  return r < s.num_kv_rows ? r : -1;
}

}  // namespace dsa
