// kv_common.cuh -- what the kernels of the INT8 paged KV cache share: the
// device view of a cache and of a batch of sequences, the checks of what the
// host cannot see (offsets, lengths, page numbers), and the search that finds
// a packed row's sequence.
#pragma once

#include "device.cuh"
#include "kernels.h"

namespace w8a8 {

// One sequence of a batch as a kernel uses it; q == 0 when it is skipped.
struct KvSeq {
  int32_t row0;  // its first packed row
  int32_t q;     // its new tokens
  int32_t n;     // its tokens, the new ones included
  __device__ __forceinline__ int32_t pos0() const { return n - q; }  // position of the first new token
};

// Sequence b, checked against the call's limits (`len_limit`: the largest
// kv_len accepted). A sequence outside them is recorded and skipped.
__device__ __forceinline__ KvSeq load_seq(const KvSeqs &s, int32_t b, int32_t len_limit, int32_t *status) {
  KvSeq r;
  const int32_t s0 = __ldg(s.seq_start + b), s1 = __ldg(s.seq_start + b + 1);
  r.n = __ldg(s.kv_len + b);
  r.row0 = s0;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= s.tokens && s1 - s0 <= s.max_q && r.n >= 0 && r.n <= len_limit;
  r.q = ok ? s1 - s0 : 0;
  if (!ok) {
    r.n = 0;
    record_error(status, W8A8_ERR_BAD_SEQUENCE);
  }
  return r;
}

// Page `i` of sequence b, or -1 (recorded) when the entry is outside the cache.
__device__ __forceinline__ int32_t load_page(const int32_t *table_row, int32_t i, int64_t num_pages, int32_t *status) {
  const int32_t p = __ldg(table_row + i);
  if (p >= 0 && p < num_pages) return p;
  record_error(status, W8A8_ERR_BAD_PAGE);
  return -1;
}

// How many of f(0) .. f(n - 1), which do not descend, are <= x; called by a
// whole warp, 32 values a step. For values that do descend the result is some
// number in [0, n], and the caller's own check of the sequence finds it.
template <typename F>
__device__ __forceinline__ int32_t warp_count_le(F f, int32_t n, int64_t x) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = n;
  while (lo < hi) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step - 1;
    const bool le = i < hi && f(static_cast<int32_t>(i)) <= x;
    const int32_t c = __popc(__ballot_sync(0xFFFFFFFFu, le));
    lo += c * step;
    hi = min(hi, lo + step - 1);
    if (lo > n) lo = n;
  }
  return lo;
}

// clamp(rne(x * r), -127, 127) as the low byte of an int (0 for a NaN product).
__device__ __forceinline__ int quant_sym(float x, float r) {
  return min(max(rne_s32(__fmul_rn(x, r)), -127), 127);
}

}  // namespace w8a8
