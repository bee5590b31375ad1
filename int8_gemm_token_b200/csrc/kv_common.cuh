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

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kGran = 16;  // a page holds whole granules of keys

// Four int8 codes (bytes e0..e3 of w) as two bf16 pairs, exactly.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t &p01, uint32_t &p23) {
  const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140), b = __byte_perm(w, 0x43434343u, 0x4342);
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p01) : "r"(a & 0xFF7FFF7Fu), "r"(a & 0xFF80FF80u));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p23) : "r"(b & 0xFF7FFF7Fu), "r"(b & 0xFF80FF80u));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The key tiles (of `tile` keys) that queries at positions first .. last - 1
// see: [0, n1) for the prefix and [t0, ...) up to their own positions, both
// cut at the sequence's n keys; tile number x of the walk is tile(x).
struct TileWalk {
  int n1, t0, count;
  __device__ __forceinline__ int tile(int x) const { return x < n1 ? x : t0 + (x - n1); }
};

__device__ __forceinline__ TileWalk tile_walk(int tile, int prefix, int n, int first, int last, int window) {
  TileWalk w;
  w.n1 = (max(min(prefix, n), 0) + tile - 1) / tile;
  w.t0 = max((window > 0 ? max(0, first - window + 1) : 0) / tile, w.n1);
  w.count = w.n1 + max(0, (max(min(last, n), 0) + tile - 1) / tile - w.t0);
  return w;
}

// Whether some query of a sequence of n keys, whose first query is at position
// `first`, sees a key of the granule that begins at `key` (a tile of a walk
// may begin in front of the window's edge or end behind the prefix). The page
// of any other granule is not looked at: its entry may say anything.
__device__ __forceinline__ bool granule_seen(int key, int prefix, int n, int first, int window) {
  return key < n && (key < prefix || window == 0 || key + kGran > first - window + 1);
}

// Final values of neighbouring output elements.
__device__ __forceinline__ void store_out2(const KvAttnArgs &a, int64_t elem, float y0, float y1) {
  const uint32_t b = pack_bf16x2(y0, y1);
  if (!a.r_out) {
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + elem) = b;
    return;
  }
  const uint2 q = quant8_asym_sat(make_uint4(b, 0, 0, 0), __ldg(a.r_out), __ldg(a.z_out));
  *reinterpret_cast<uint16_t *>(static_cast<int8_t *>(a.out) + elem) = static_cast<uint16_t>(q.x);
}
__device__ __forceinline__ void store_out4(const KvAttnArgs &a, int64_t elem, const float (&y)[4]) {
  const uint2 b = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  if (!a.r_out) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + elem) = b;
    return;
  }
  const uint2 q = quant8_asym_sat(make_uint4(b.x, b.y, 0, 0), __ldg(a.r_out), __ldg(a.z_out));
  *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(a.out) + elem) = q.x;
}

}  // namespace w8a8
