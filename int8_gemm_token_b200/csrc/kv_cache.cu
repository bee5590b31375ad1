// kv_cache.cu -- writing and reading the INT8 paged KV cache.
//
// What it computes (include/w8a8.h, w8a8_kv_append and w8a8_kv_gather): the
// position rotation of new keys and queries, the symmetric absmax int8
// quantization of new keys and values with one scale for each page and head
// (LLM.int8() summary §一.1), and value = scale * code back.
//
// How (sm_100a): both are HBM streams with a data-dependent address, so the
// work is cut where the addresses are: a UNIT is one page of one head of k or
// of v, held by one group of threads that reads its new tokens once into
// registers (rotated there), reduces their absmax, settles the page's scale
// and writes the codes. Nothing is read twice and no atomic is needed: a page
// and head belong to one group.
//   Few new tokens a sequence (at most kFewTokens: decode steps): the group
//   is one warp per (sequence, head, k or v), which walks the one or two
//   pages its tokens touch.
//   Many: the group is 2 threads per token of a page (a warp for pages of 16,
//   a block of 64 to 256 threads for the larger), so that a thread holds 64
//   values whatever the page, all its loads in flight at once. Packed rows
//   are cut into pages of their sequences by a search over
//   f(b) = seq_start[b] / page + 2 b, which leaves each sequence room for
//   the pages its tokens can touch (at most q / page + 2).
// Within a group, D / 16 neighbouring threads hold one token: each takes the
// two 8-element chunks of which one holds the first and one the second
// elements of its pairs (or both whole pairs when interleaved), so a rotation
// needs no exchange. Query rows are rotated by warps of their own, 4 passes
// over the heads of a row at a time.
//   The read-back takes a warp per (granule of 16 positions, head), whose
// codes of k and of v are each one run of 16 D bytes.
//
// Measured (device time, back to back over buffers larger than L2 together):
// the append of 8192 tokens of 8 heads of 128 with 32 query heads rotated
// moves 190 MB in 38.8 us, 4.9 TB/s; at that point the SMs issue in 61 % of
// cycles and DRAM is 46 % busy, so what is left is latency between a row's
// loads and the work on them. Five prompts of up to 1531 tokens with pages of
// 16: 28.6 us. A step of 32 tokens x 32 heads: 3.5 us, a launch and five dependent
// loads. The read-back of 32768 tokens of 8 heads moves 201 MB in 35 us,
// 5.7 TB/s, 0.87 of what a copy reaches.
#include "kv_common.cuh"

namespace w8a8 {

namespace {

constexpr int kThreads = 256;
constexpr int kFewTokens = 8;

// 8 bf16 as fp32.
__device__ __forceinline__ void widen8(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ void load8f(const float *p, float *x) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The two 8-element chunks of unit u (of D / 16): pairs lie across them
// (halves of the rotated part) or inside them (interleaved, and the part that
// is not rotated).
__device__ __forceinline__ void unit_chunks(int u, int rot, bool interleaved, int &c0, int &c1) {
  const int nr = rot >> 4;  // units of the rotated part
  if (!interleaved && u < nr) {
    c0 = u;
    c1 = u + nr;
  } else {
    c0 = 2 * u;
    c1 = c0 + 1;
  }
}

// Rotates the 16 values of unit u (x[0..7] of chunk c0, x[8..15] of c1) with
// the 8 angles of the unit; products and sums rounded one by one.
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&c)[8], const float (&s)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
      x[8 + i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    }
  }
}

__device__ __forceinline__ uint2 codes8(const float *x, float r) {
  return make_uint2(low_bytes4(quant_sym(x[0], r), quant_sym(x[1], r), quant_sym(x[2], r), quant_sym(x[3], r)),
                    low_bytes4(quant_sym(x[4], r), quant_sym(x[5], r), quant_sym(x[6], r), quant_sym(x[7], r)));
}

// Codes of a page re-rounded for its larger scale: clamp(rne(code * ratio), -127, 127).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  return low_bytes4(
      quant_sym(static_cast<float>(sext_byte<0>(w)), ratio), quant_sym(static_cast<float>(sext_byte<1>(w)), ratio),
      quant_sym(static_cast<float>(sext_byte<2>(w)), ratio), quant_sym(static_cast<float>(sext_byte<3>(w)), ratio));
}

// One unit: tokens [lo, hi) (positions) of sequence `seq`, all in page index
// `pi`, head h of k (which == 0) or v. G threads (a warp or the block) of
// which this is thread `tid`; PASSES * (G / U) covers the tokens of a page.
template <int D, int G, int PASSES>
__device__ __forceinline__ void append_unit(const KvAppendArgs &a, const KvSeq &seq, const int32_t *table_row, int pi,
                                            int lo, int hi, int h, int which, int tid, float *s_red) {
  constexpr int U = D / 16, TP = G / U;  // threads of a token, tokens of a pass
  const KvRows &src = which ? a.v : a.k;
  const int u = tid % U, tok = tid / U;
  const bool turn = a.cos != nullptr && which == 0;
  const bool il = a.interleaved != 0;
  const int rot = turn ? a.rot : 0;
  int c0, c1;
  unit_chunks(u, rot, il, c0, c1);
  uint4 raw[PASSES][2];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int pos = lo + p * TP + tok;
    raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    if (tok < TP && pos < hi) {
      const uint16_t *row = src.p + (seq.row0 + pos - seq.pos0()) * src.token_stride + h * src.head_stride;
      raw[p][0] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c0));
      raw[p][1] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c1));
    }
  }
  const int32_t page = load_page(table_row, pi, a.c.pages, a.status);
  if (page < 0) return;  // uniform over the group: every thread read the same entry
  int8_t *codes = (which ? a.c.v : a.c.k) + ((static_cast<int64_t>(page) * a.c.heads + h) << a.c.page_shift) * D;
  float *scale = (which ? a.c.vs : a.c.ks) + static_cast<int64_t>(page) * a.c.heads + h;
  const int old = lo & (a.c.page - 1);  // tokens that lie in the page already
  const float s_old = old > 0 ? *scale : 0.0f;
  // More than 2 passes hold their rows as bf16 and form the fp32 values twice,
  // for the absmax and for the codes: 80 registers and 24 warps an SM, where
  // holding the values takes 115 and 16 (a prompt of 8192 tokens, 8 heads and
  // 32 query heads of 128: 39.1 us against 40.8; five prompts of up to 1531
  // with pages of 16: 28.8 against 30.8). 1 or 2 passes keep them: a step of
  // few tokens is bound by its latency (3.5 us; forming them again, 4.0).
  const auto values = [&](int p, float(&x)[16]) {
    const int pos = lo + p * TP + tok;
    widen8(raw[p][0], x);
    widen8(raw[p][1], x + 8);
    if (16 * u < rot && tok < TP && pos < hi) {
      float cs[8], sn[8];
      const int64_t at = static_cast<int64_t>(pos) * (a.rot >> 1) + 8 * u;
      load8f(a.cos + at, cs);
      load8f(a.sin + at, sn);
      rotate16(x, cs, sn, il);
    }
  };
  constexpr bool kKeep = PASSES <= 2;
  float x[kKeep ? PASSES : 1][16];
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    float(&y)[16] = x[kKeep ? p : 0];
    values(p, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
    if constexpr (!kKeep) {
#pragma unroll
      for (int i = 0; i < 2; ++i)  // the compiler is not to keep the values either
        asm volatile("" : "+r"(raw[p][i].x), "+r"(raw[p][i].y), "+r"(raw[p][i].z), "+r"(raw[p][i].w));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if constexpr (G > 32) {
    if ((tid & 31) == 0) s_red[tid >> 5] = amax;
    __syncthreads();  // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < G / 32; ++w) amax = fmaxf(amax, s_red[w]);
  } else {
    __syncwarp();
  }
  float S = fmaxf(s_old, __fdiv_rn(amax, 127.0f));
  float r = S > 0.0f ? __fdiv_rn(1.0f, S) : 0.0f;
  if (isinf(r)) S = r = 0.0f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int pos = lo + p * TP + tok;
    if (tok < TP && pos < hi) {
      float(&y)[16] = x[kKeep ? p : 0];
      if constexpr (!kKeep) values(p, y);
      int8_t *row = codes + (pos & (a.c.page - 1)) * D;
      *reinterpret_cast<uint2 *>(row + 8 * c0) = codes8(y, r);
      *reinterpret_cast<uint2 *>(row + 8 * c1) = codes8(y + 8, r);
    }
  }
  if (old > 0 && S != s_old) {
    const float ratio = S > 0.0f ? __fdiv_rn(s_old, S) : 0.0f;
    for (int i = tid; i < old * U; i += G) {
      uint4 *w = reinterpret_cast<uint4 *>(codes) + i;
      const uint4 v = *w;
      *w = make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
    }
  }
  if (tid == 0 && (old == 0 || S != s_old)) *scale = S;
}

// Rotation of a part of the query rows by one warp: of the `w`-th (row, block
// of kQueryPasses * 32 / (D / 16) heads).
constexpr int kQueryPasses = 4;

template <int D>
__host__ __device__ constexpr int query_heads() { return kQueryPasses * (32 / (D / 16)); }

template <int D>
__device__ __forceinline__ void rotate_query_rows(const KvAppendArgs &a, int64_t w) {
  constexpr int U = D / 16, HP = 32 / U;  // lanes of a head, heads of a pass
  const int lane = threadIdx.x & 31;
  const int blocks = (a.q_heads + query_heads<D>() - 1) / query_heads<D>();
  const int64_t t = w / blocks;
  const int h0 = static_cast<int>(w - t * blocks) * query_heads<D>();
  if (t >= a.s.tokens) return;
  const int u = lane % U, hl = lane / U;
  const bool il = a.interleaved != 0;
  int c0, c1;
  unit_chunks(u, a.rot, il, c0, c1);
  uint4 raw[kQueryPasses][2];
#pragma unroll
  for (int p = 0; p < kQueryPasses; ++p) {
    const int h = h0 + p * HP + hl;
    raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    if (hl < HP && h < a.q_heads) {
      const uint16_t *row = a.q.p + t * a.q.token_stride + h * a.q.head_stride;
      raw[p][0] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c0));
      raw[p][1] = __ldg(reinterpret_cast<const uint4 *>(row + 8 * c1));
    }
  }
  const int32_t *next = a.s.seq_start + 1;
  const int32_t b = warp_count_le([&](int32_t i) { return static_cast<int64_t>(__ldg(next + i)); }, a.s.batch, t);
  if (b >= a.s.batch) return;  // behind the last sequence
  const KvSeq seq = load_seq(a.s, b, a.len_limit, a.status);
  const int64_t i = t - seq.row0;
  if (i < 0 || i >= seq.q) return;
  const int64_t pos = seq.pos0() + i;
  const bool turn = a.cos != nullptr && 16 * u < a.rot && pos >= 0;
  float cs[8], sn[8];
  if (turn) {
    const int64_t at = pos * (a.rot >> 1) + 8 * u;
    load8f(a.cos + at, cs);
    load8f(a.sin + at, sn);
  }
#pragma unroll
  for (int p = 0; p < kQueryPasses; ++p) {
    const int h = h0 + p * HP + hl;
    if (hl >= HP || h >= a.q_heads) continue;
    uint16_t *out = a.q_out + (t * a.q_heads + h) * D;
    if (pos < 0) raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    float x[16];
    widen8(raw[p][0], x);
    widen8(raw[p][1], x + 8);
    if (turn) rotate16(x, cs, sn, il);
    *reinterpret_cast<uint4 *>(out + 8 * c0) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                          pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    *reinterpret_cast<uint4 *>(out + 8 * c1) = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]),
                                                          pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15]));
  }
}

// Few new tokens a sequence: warps [0, batch * heads * 2) one (sequence,
// head, k or v) each, the following warps a block of heads of a query row each.
template <int D>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const __grid_constant__ KvAppendArgs a) {
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int lane = threadIdx.x & 31;
  int64_t w = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  const int64_t units = static_cast<int64_t>(a.s.batch) * a.c.heads * 2;
  if (w >= units) {
    if (a.q_out) rotate_query_rows<D>(a, w - units);
    return;
  }
  const int which = static_cast<int>(w & 1);
  w >>= 1;
  const int h = static_cast<int>(w % a.c.heads), b = static_cast<int>(w / a.c.heads);
  const KvSeq seq = load_seq(a.s, b, a.len_limit, a.status);
  if (seq.q == 0) return;
  const int32_t *row = a.s.table + b * a.s.table_ld;
  constexpr int TP = 32 / (D / 16), PASSES = (kFewTokens + TP - 1) / TP;
  for (int lo = max(seq.pos0(), 0); lo < seq.n;) {
    const int pi = lo >> a.c.page_shift;
    const int hi = min(seq.n, (pi + 1) << a.c.page_shift);
    append_unit<D, 32, PASSES>(a, seq, row, pi, lo, hi, h, which, lane, nullptr);
    lo = hi;
  }
}

// Many new tokens: units [0, tiles * heads * 2) are a page of a head of k or
// v each, for G threads (units whose page does not exist are skipped); the
// warps that follow them have query rows. (24 warps an SM: at 20, pages of 16
// lose 9 % and pages of 64 gain 1 %.)
template <int D, int G>
__global__ void __launch_bounds__(G > 32 ? G : kThreads, 768 / (G > 32 ? G : kThreads))
    append_pages_kernel(const __grid_constant__ KvAppendArgs a, int64_t tiles) {
  constexpr int BLOCK = G > 32 ? G : kThreads;
  __shared__ float s_red[BLOCK / 32];
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int64_t units = tiles * a.c.heads * 2;
  const int64_t unit = (blockIdx.x * static_cast<int64_t>(BLOCK) + threadIdx.x) / G;
  if (blockIdx.x == 0 && threadIdx.x < 32)  // every sequence is checked, the search may not come upon a bad one
    for (int32_t i = threadIdx.x; i < a.s.batch; i += 32) load_seq(a.s, i, a.len_limit, a.status);
  if (unit >= units) {
    if (a.q_out) rotate_query_rows<D>(a, (unit - units) * (G / 32) + (threadIdx.x % G) / 32);
    return;
  }
  const int64_t per = a.c.heads * 2;
  const int64_t tile = unit / per;
  const int which = static_cast<int>(unit & 1), h = static_cast<int>((unit % per) >> 1);
  const int shift = a.c.page_shift;
  const auto f = [&](int32_t i) { return static_cast<int64_t>(__ldg(a.s.seq_start + i) >> shift) + 2 * int64_t(i); };
  const int32_t b = warp_count_le(f, a.s.batch, tile) - 1;
  if (b < 0) return;
  const KvSeq seq = load_seq(a.s, b, a.len_limit, a.status);
  if (seq.q == 0) return;
  const int start = max(seq.pos0(), 0);
  const int64_t pi = (start >> shift) + (tile - f(b));
  // (where the starts descend, the search may end at a sequence whose slots lie behind this one)
  if (tile < f(b) || start >= seq.n || pi > ((seq.n - 1) >> shift)) return;
  const int lo = max(start, static_cast<int>(pi) << shift);
  const int hi = min(seq.n, static_cast<int>((pi + 1) << shift));
  constexpr int TP = G / (D / 16), PASSES = (G / 2 + TP - 1) / TP;
  append_unit<D, G, PASSES>(a, seq, a.s.table + b * a.s.table_ld, static_cast<int>(pi), lo, hi, h, which,
                            threadIdx.x % G, s_red);
}

cudaLaunchConfig_t pdl_config(int64_t blocks, int threads, cudaStream_t s, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int D>
int64_t query_warps(const KvAppendArgs &a) {
  return a.q_out ? a.s.tokens * ((a.q_heads + query_heads<D>() - 1) / query_heads<D>()) : 0;
}

// Threads of a page's unit (append_pages_kernel's G), and slots of pages.
int page_threads(const KvAppendArgs &a) { return 2 * a.c.page; }
int64_t page_slots(const KvAppendArgs &a) { return (a.s.tokens >> a.c.page_shift) + 2 * static_cast<int64_t>(a.s.batch); }
int page_block(const KvAppendArgs &a) { return page_threads(a) > 32 ? page_threads(a) : kThreads; }

template <int D>
int64_t append_blocks(const KvAppendArgs &a) {
  const int64_t heads = static_cast<int64_t>(a.c.heads) * 2;
  if (a.s.max_q <= kFewTokens) return (a.s.batch * heads + query_warps<D>(a) + kThreads / 32 - 1) / (kThreads / 32);
  return (page_slots(a) * heads * page_threads(a) + query_warps<D>(a) * 32 + page_block(a) - 1) / page_block(a);
}

template <int D, int G>
cudaError_t launch_pages_t(const KvAppendArgs &a, cudaStream_t s) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(append_blocks<D>(a), G > 32 ? G : kThreads, s, &attr);
  return cudaLaunchKernelEx(&cfg, append_pages_kernel<D, G>, a, page_slots(a));
}

template <int D>
cudaError_t launch_append_t(const KvAppendArgs &a, cudaStream_t s) {
  if (a.s.max_q <= kFewTokens) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(append_blocks<D>(a), kThreads, s, &attr);
    return cudaLaunchKernelEx(&cfg, append_few_kernel<D>, a);
  }
  switch (a.c.page) {
    case 16: return launch_pages_t<D, 32>(a, s);
    case 32: return launch_pages_t<D, 64>(a, s);
    case 64: return launch_pages_t<D, 128>(a, s);
    default: return launch_pages_t<D, 256>(a, s);
  }
}

// ------------------------------------------------------------------ gather
// scale * code of byte B of w: the sign-extended code plus 0x4B400000 is the
// bit pattern of 1.5 2^23 + code, from which 1.5 2^23 is subtracted exactly.
template <int B>
__device__ __forceinline__ float code_value(uint32_t w, float scale) {
  return __fmul_rn(scale, __fsub_rn(__int_as_float(sext_byte<B>(w) + 0x4B400000), 12582912.0f));
}

// 8 codes as values. (8 codes to a lane, not 16: a warp's 16-byte bf16 stores
// are then one run of 512 bytes; two stores of 16 bytes at a stride of 32 kept
// L1 76 % busy and cost 43 us for 32768 tokens of 8 x 128.)
template <bool BF16>
__device__ __forceinline__ void store_values(const uint2 &v, float scale, void *out, int64_t elem) {
  const float y[8] = {code_value<0>(v.x, scale), code_value<1>(v.x, scale), code_value<2>(v.x, scale),
                      code_value<3>(v.x, scale), code_value<0>(v.y, scale), code_value<1>(v.y, scale),
                      code_value<2>(v.y, scale), code_value<3>(v.y, scale)};
  if constexpr (BF16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + elem) = make_uint4(
        pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  } else {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + elem);
    o[0] = make_float4(y[0], y[1], y[2], y[3]);
    o[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

__device__ __forceinline__ bool gather_ok(const KvGatherArgs &a, int32_t r0, int32_t r1, int32_t first) {
  return r0 >= 0 && r1 >= r0 && r1 <= a.rows && first >= 0 &&
         static_cast<int64_t>(first) + (r1 - r0) <= static_cast<int64_t>(a.max_pages) << a.c.page_shift;
}

// Warp (slot, head): the slot's granule of a sequence, found as a page is in
// append_pages_kernel (f(b) = row_start[b] / 16 + 2 b).
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ KvGatherArgs a, int64_t warps) {
  constexpr int C = D / 8, N = D / 16;  // 8-code chunks of a row; of k or of v to a lane
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int lane = threadIdx.x & 31;
  const int64_t w = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  if (w >= warps) return;
  if (w == 0)  // as in append_pages_kernel
    for (int32_t i = lane; i < a.batch; i += 32)
      if (!gather_ok(a, __ldg(a.row_start + i), __ldg(a.row_start + i + 1), __ldg(a.first_pos + i)))
        record_error(a.status, W8A8_ERR_BAD_SEQUENCE);
  const int64_t slot = w / a.c.heads;
  const int h = static_cast<int>(w - slot * a.c.heads);
  const auto f = [&](int32_t i) { return static_cast<int64_t>(__ldg(a.row_start + i) / kGran) + 2 * int64_t(i); };
  const int32_t b = warp_count_le(f, a.batch, slot) - 1;
  if (b < 0) return;
  const int32_t r0 = __ldg(a.row_start + b), r1 = __ldg(a.row_start + b + 1), first = __ldg(a.first_pos + b);
  if (!gather_ok(a, r0, r1, first)) return;
  const int64_t granule = first / kGran + (slot - f(b));
  const int end = first + (r1 - r0);  // one past the last position
  // (the first as in append_pages_kernel; an empty range may begin inside a granule)
  if (slot < f(b) || r1 == r0 || granule * kGran >= end) return;
  const int key0 = static_cast<int>(granule) * kGran;
  const int32_t page = load_page(a.table + b * a.table_ld, key0 >> a.c.page_shift, a.c.pages, a.status);
  const int64_t block = static_cast<int64_t>(max(page, 0)) * a.c.heads + h;
  const int64_t src = ((block << a.c.page_shift) + (key0 & (a.c.page - 1))) * D;
  uint2 k[N], v[N];
  float ks = 0.0f, vs = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) k[i] = v[i] = make_uint2(0, 0);  // a page that does not exist reads as 0
  if (page >= 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = src + (i * 32 + lane) * 8;
      if (a.k_out) k[i] = __ldg(reinterpret_cast<const uint2 *>(a.c.k + at));
      if (a.v_out) v[i] = __ldg(reinterpret_cast<const uint2 *>(a.c.v + at));
    }
    ks = __ldg(a.c.ks + block);
    vs = __ldg(a.c.vs + block);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int idx = i * 32 + lane, pos = key0 + idx / C;
    if (pos < first || pos >= end) continue;
    const int64_t elem = (static_cast<int64_t>(r0 + pos - first) * a.c.heads + h) * D + 8 * (idx % C);
    if (a.k_out) store_values<BF16>(k[i], ks, a.k_out, elem);
    if (a.v_out) store_values<BF16>(v[i], vs, a.v_out, elem);
  }
}

int64_t gather_warps(const KvGatherArgs &a) { return (a.rows / kGran + 2 * static_cast<int64_t>(a.batch)) * a.c.heads; }

template <int D>
cudaError_t launch_gather_t(const KvGatherArgs &a, bool bf16_out, cudaStream_t s) {
  const int64_t warps = gather_warps(a);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config((warps + kThreads / 32 - 1) / (kThreads / 32), kThreads, s, &attr);
  if (bf16_out) return cudaLaunchKernelEx(&cfg, gather_kernel<D, true>, a, warps);
  return cudaLaunchKernelEx(&cfg, gather_kernel<D, false>, a, warps);
}

}  // namespace

bool kv_append_fits(const KvAppendArgs &a) {
  const int64_t blocks = a.c.d == 64 ? append_blocks<64>(a) : a.c.d == 96 ? append_blocks<96>(a) : append_blocks<128>(a);
  return blocks <= INT32_MAX;
}

bool kv_gather_fits(const KvGatherArgs &a) { return gather_warps(a) / (kThreads / 32) < INT32_MAX; }

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t s) {
  switch (a.c.d) {
    case 64: return launch_append_t<64>(a, s);
    case 96: return launch_append_t<96>(a, s);
    case 128: return launch_append_t<128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv_gather(const KvGatherArgs &a, bool bf16_out, cudaStream_t s) {
  switch (a.c.d) {
    case 64: return launch_gather_t<64>(a, bf16_out, s);
    case 96: return launch_gather_t<96>(a, bf16_out, s);
    case 128: return launch_gather_t<128>(a, bf16_out, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace w8a8
