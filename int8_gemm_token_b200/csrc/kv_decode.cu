// kv_decode.cu -- attention of few new tokens over the INT8 paged KV cache.
//
// What it computes (include/w8a8.h, w8a8_kv_attention): for each query row
// (new token i, head) the softmax-weighted sum of the cached values, one pass
// over the cache with a running maximum m and sum l:
//   m' = max(m, max_j s_j);  l = l 2^(m - m') + sum_j 2^(s_j - m');
//   o = o 2^(m - m') + sum_j 2^(s_j - m') v_j;  out = o / l
// with scores in units of log2.
//
// How: the bound is the cache's bytes from HBM, each used once for all the
// query rows of its kv head, so a warp takes 32 keys at a time and the rows
// (group * new tokens) are the narrow side of the products: S^T = K Q^T with
// 16 keys x 8 rows x 16 dims an instruction, and O^T = V^T P^T with 16 dims x
// 8 rows x 16 keys. Those shapes are mma.sync's; tcgen05 wants 128 rows of
// one operand in shared memory as fp16, which the int8 codes are not until a
// register has held them. Codes become fp16 in registers, exactly: the byte
// q + 128 under 0x64 is the bit pattern of 1024 + 128 + q, from which 1152 is
// subtracted (per four codes one xor, two byte permutes, two packed adds).
//   fp16 has the codes' bits to spare but not bf16's range, so what meets them
// is scaled by powers of two, exactly: a query row so that its largest
// element is in [2^14, 2^15) (elements below 2^-31 of it lose bits), and
// the weights 2^s_j times v's scale against a running reference of their own,
// apart from that of the scores:
//   w_j = 2^(s_j + log2 vs_j - mv + 7),  l = sum_j 2^(s_j - m) in fp32,
//   out = 2^(mv - m - 7) (sum_j w_j code_j) / l.
// w_j is rounded to fp16 once (2^-11). m and mv follow the maxima of s_j and of
// s_j + log2 vs_j only when these have outgrown them by 2^8, which a vote over
// the warp's elements finds; only then are maxima exchanged between lanes and
// the sums rescaled. So w_j stays below 2^15, fp16's largest power of two, and
// what fp16 cannot hold is below 2^-32 of the row's largest: l has every
// weight, and a long tail that the sums lacked would be missing from the output
// (2^18 keys of 2^-26 behind one of 1, in one piece: 0.4 % of it).
//   Both contractions may run over their axis in any order as long as both
// sides use the same one, so a lane reads its codes of K as 16 contiguous
// bytes of one key and those of V as the same dims of four keys (pairs of
// keys are interleaved by byte permutes), and w goes from the accumulator
// layout of the first product to the operand layout of the second by an 8x8
// transpose (movmatrix).
//   Loads are 16-byte cp.async into a ring of each warp's own, so a warp
// waits for nobody; the stages are swizzled so that both reads are free of
// bank conflicts (D = 128).
//
// Work: the key tiles (32 keys) of all segments -- (sequence, kv head, block
// of query rows) -- laid end to end, each with some units more for its start,
// are cut into equal pieces, whatever the lengths of the sequences, which only
// the device knows. A piece that holds all of a segment writes its output;
// parts go to the workspace (sums, references, sum of weights) and
// kv_join_kernel joins them in the order of the pieces. Every warp finds its
// piece by a scan over the sequences' lengths, and the join who has what: by
// the same scan, or, of many sequences, from what one warp left of it.
//   A piece is one warp's, so that warps start segments while others stream
// (kv_decode_kernel). Where segments are few and long it is that of a block of
// all an SM's warps, which deal its tiles out among them and join in shared
// memory, so that there are few parts (kv_decode_block_kernel). Where they are
// few and short a block has a segment, and there is nothing to join: one
// launch. The rules and what they measured stand at the host's choice below.
//
// Measured: 32 sequences x 32 heads x 4096 keys of 128 (1.07 GB of codes) alone
// in a profile 168 us, 6.4 TB/s, DRAM 79 % busy; the SMs issue in 57 % of cycles,
// the ALU pipe in 51 %, the tensor pipe is 20 % busy. Back to back for seconds
// the board is at its power cap and the time goes with the clock: 178.5 us at
// 1725 MHz on one, 191 at 1612 on another (0.308 s MHz both), 5.6 to 6.0 TB/s. 64
// sequences of 1 to 32768 keys, 8 heads for 32 (547 MB): 103 us, 5.3 TB/s.
// Scores by s8 products (codes as they lie, q as 22-bit fixed point in three
// int8 parts) need a sixth fewer instructions and measured 192 to 202 and
// 103.5 us where this took 189 to 193 and 102.7: instructions are not the limit.
// The smallest calls are their latency: one sequence of 512 keys 8.0 us.
#include "kv_common.cuh"

namespace w8a8 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;     // keys of a tile: two granules, each of one page
constexpr float kRescale = 8.0f;  // log2 of how far a maximum may outgrow its reference
constexpr float kLift = 7.0f;     // log2 of the largest fp16 power of two, less kRescale
// What a segment's start costs, in tiles, and units that a piece has at least:
// of a piece of one warp, and of all of an SM's warps.
constexpr int kSetup = 2, kMinUnits = 4;
constexpr int kBlockSetup = 12, kBlockMinUnits = 24;
constexpr int kJoinWarps = 4;

// 12 warps of 168 registers an SM with 8 query rows, 8 of 255 with 16 (twice
// the sums and queries in registers). Each has two stages of a tile: while one
// is computed with, the other's 8 KiB are in flight, 96 KiB an SM. (16 warps of
// 128 registers with tiles of 16 keys kept 128 KiB in flight and were slower:
// what is done once a tile, whatever its keys, cost them 100 of 450 instructions.)
constexpr int sm_warps(int nt) { return nt == 1 ? 12 : 8; }
constexpr int kStages = 2;

template <int D>
struct Cfg {
  static constexpr int kPitch = D == 64 ? 64 : 128;        // bytes of a key's row in a stage
  static constexpr int kStage = 2 * kTile * kPitch;        // K rows, then V rows
  static constexpr int kChunks = D / 16;
  static constexpr size_t kSmem = static_cast<size_t>(kWarps) * kStages * kStage;
  static_assert(sm_warps(1) / kWarps * (kSmem + 1024) <= 227 * 1024, "shared memory per SM");
};

// Byte offset of 16-byte chunk c of row r in a stage. D = 128 (and 96 in the
// same pitch): chunk bits 2..1 are flipped by ((r >> 2) ^ r) & 1 and by
// (r >> 1) & 1, which spreads both the two rows of a K read (same r >> 1) and
// the four rows of a V read (same r & 1) over all banks; D = 64: two rows
// share 128 bytes, chunks are flipped by (r >> 1) & 3.
template <int D>
__device__ __forceinline__ int stage_off(int r, int c) {
  if constexpr (D == 64)
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * 128 + ((c ^ (((((r >> 2) ^ r) & 1) << 2) | (((r >> 1) & 1) << 1))) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four int8 codes (bytes e0..e3 of w) as two fp16 pairs, exactly.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &p01, uint32_t &p23) {
  const uint32_t u = w ^ 0x80808080u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p01) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p23) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The dims of a head are cut into parts of 64 (and for D = 128 one of 128,
// for 96 one of 64 and one of 32) in which a lane's codes are contiguous.
// K: the words (4 dims) that lane quarter t holds of a row: word w of part
// [base, base + n) is dim base + (n / 4) t + 4 w.
template <int D>
__device__ __forceinline__ int k_dim(int t, int w) {
  if constexpr (D == 96) return w < 4 ? 16 * t + 4 * w : 64 + 8 * t + 4 * (w - 4);
  return (D / 4) * t + 4 * w;
}
// V: lane octet g holds in a row, for 16-dim tile i, dims v_dim and v_dim + 1
// (the tile's output rows g and g + 8).
template <int D>
__device__ __forceinline__ int v_dim(int g, int i) {
  if constexpr (D == 96) return i < 4 ? 8 * g + 2 * i : 64 + 4 * g + 2 * (i - 4);
  return (D / 8) * g + 2 * i;
}

template <int D>
__device__ __forceinline__ void load_k_words(const uint8_t *k, int r, int t, uint32_t (&w)[D / 16]) {
  if constexpr (D == 128) {
    const uint4 a = *reinterpret_cast<const uint4 *>(k + stage_off<D>(r, 2 * t));
    const uint4 b = *reinterpret_cast<const uint4 *>(k + stage_off<D>(r, 2 * t + 1));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(k + stage_off<D>(r, t));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if constexpr (D == 96) {
      const uint2 b = *reinterpret_cast<const uint2 *>(k + stage_off<D>(r, 4 + (t >> 1)) + 8 * (t & 1));
      w[4] = b.x, w[5] = b.y;
    }
  }
}

// The D / 8 bytes of row r that lane octet g holds, as words of 4 dims (2 tiles).
template <int D>
__device__ __forceinline__ void load_v_words(const uint8_t *v, int r, int g, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 a = *reinterpret_cast<const uint4 *>(v + stage_off<D>(r, g));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2 *>(v + stage_off<D>(r, g >> 1) + 8 * (g & 1));
    w[0] = a.x, w[1] = a.y;
    if constexpr (D == 96)
      w[2] = *reinterpret_cast<const uint32_t *>(v + stage_off<D>(r, 4 + (g >> 2)) + 4 * (g & 3));
  }
}

// ---------------------------------------------------------------- the cut
// Sequence b as the cut sees it: its segments (kv heads x blocks of query
// rows), each of SETUP + walk.count units (none without keys).
template <int SETUP>
struct SeqWork {
  KvSeq seq;
  int32_t prefix, segs;
  TileWalk walk;
  __device__ __forceinline__ uint32_t seg_units() const { return walk.count > 0 ? SETUP + walk.count : 0; }
  __device__ __forceinline__ uint32_t units() const { return segs * seg_units(); }
};

template <int ROWS, int SETUP>
__device__ __forceinline__ SeqWork<SETUP> seq_work(const KvAttnArgs &a, int32_t b, int32_t *status) {
  SeqWork<SETUP> w;
  w.prefix = a.prefix ? __ldg(a.prefix + b) : 0;
  w.seq = load_seq(a.s, b, a.s.max_kv, status);
  w.segs = (w.seq.q * a.group + ROWS - 1) / ROWS * a.c.heads;
  w.walk = tile_walk(kTile, w.prefix, w.seq.n, max(w.seq.pos0(), 0), w.seq.n, a.window);
  return w;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Units before sequence `b` (if it is one) and all units; called by a whole
// warp. Returns the lane's inclusive scan of the last 32 sequences. The one
// warp that is given `offsets` leaves the units before each sequence there,
// and all of them behind the last. (Fewer than 2^31 units in all: the host has
// checked it.)
template <int ROWS, int SETUP>
__device__ __forceinline__ uint32_t count_units(const KvAttnArgs &a, int32_t b, int32_t *status, uint32_t *offsets,
                                                uint32_t &before, uint32_t &all) {
  const int lane = threadIdx.x & 31;
  uint32_t sum = 0;
  before = all = 0;
  for (int32_t i0 = 0; i0 < a.s.batch; i0 += 32) {
    const int32_t i = i0 + lane;
    const uint32_t v = i < a.s.batch ? seq_work<ROWS, SETUP>(a, i, status).units() : 0;
    sum = warp_scan(v);
    if (b >= i0 && b < i0 + 32) before = all + __shfl_sync(0xFFFFFFFFu, sum - v, b - i0);
    if (offsets && i < a.s.batch) offsets[i] = all + sum - v;
    all += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  if (offsets && lane == 0) offsets[a.s.batch] = all;
  return sum;
}

// The sequence that unit `at` (of all) lies in, and the units before it.
template <int ROWS, int SETUP>
__device__ __forceinline__ int32_t find_unit(const KvAttnArgs &a, uint32_t at, uint32_t &before) {
  const int lane = threadIdx.x & 31;
  before = 0;
  for (int32_t i0 = 0; i0 < a.s.batch; i0 += 32) {
    const int32_t i = i0 + lane;
    const uint32_t v = i < a.s.batch ? seq_work<ROWS, SETUP>(a, i, nullptr).units() : 0;
    const uint32_t sum = warp_scan(v);
    const int32_t c = __popc(__ballot_sync(0xFFFFFFFFu, before + sum <= at));
    if (c < 32) {
      before += __shfl_sync(0xFFFFFFFFu, sum - v, c);
      return i0 + c;
    }
    before += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return a.s.batch;
}

// `all` units cut into at most `most` pieces whose sizes differ by at most one.
struct Cut {
  uint32_t pieces, size, more;  // the first `more` pieces have size + 1 units
  __device__ __forceinline__ Cut(uint32_t all, uint32_t most, uint32_t min_units) {
    pieces = max(1u, min((all + min_units - 1) / min_units, most));
    size = all / pieces;
    more = all - size * pieces;
  }
  __device__ __forceinline__ uint32_t begin(uint32_t p) const { return p * size + min(p, more); }
  __device__ __forceinline__ uint32_t piece_of(uint32_t unit) const {
    const uint32_t big = more * (size + 1);
    return unit < big ? unit / (size + 1) : more + (unit - big) / size;
  }
};

// Walks the parts of segments that units [begin, end) hold; by a whole warp.
template <int ROWS, int SETUP>
struct PieceWalk {
  uint32_t begin, at, end, before;  // `before`: units before sequence b
  int32_t b;
  SeqWork<SETUP> work;
  // the part
  int h, row0, x0, x1;
  bool first;  // its segment is the piece's first

  // `sum`: the lanes' scan from count_units
  __device__ __forceinline__ PieceWalk(const KvAttnArgs &a, const Cut &cut, uint32_t p, uint32_t sum) {
    begin = at = cut.begin(p);
    end = cut.begin(p + 1);
    if (a.s.batch <= 32) {  // the scan of the one round is at hand
      b = __popc(__ballot_sync(0xFFFFFFFFu, sum <= at));
      before = b > 0 ? __shfl_sync(0xFFFFFFFFu, sum, b - 1) : 0;
    } else {
      b = find_unit<ROWS, SETUP>(a, at, before);
    }
    work = seq_work<ROWS, SETUP>(a, b, nullptr);
  }
  __device__ __forceinline__ bool next(const KvAttnArgs &a) {
    while (at < end) {
      while (at >= before + work.units()) {  // on to the next sequence that has keys
        before += work.units();
        work = seq_work<ROWS, SETUP>(a, ++b, nullptr);
      }
      const uint32_t seg_units = work.seg_units();
      const int32_t seg = static_cast<int32_t>((at - before) / seg_units);
      const uint32_t seg0 = before + seg * seg_units, seg_end = min(seg0 + seg_units, end);
      x0 = max(static_cast<int>(at - seg0) - SETUP, 0);  // the tiles' units come after the start's
      x1 = static_cast<int>(seg_end - seg0) - SETUP;
      first = begin >= seg0;
      at = seg_end;
      if (x1 <= x0) continue;
      const int rbs = work.segs / a.c.heads;  // the row blocks of a head side by side: its keys stay in L2
      h = seg / rbs;
      row0 = (seg - h * rbs) * ROWS;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ bool whole() const { return x0 == 0 && x1 == work.walk.count; }
};

// A part of a segment in the workspace: slot 2 p of piece p where the segment
// is the piece's first, else 2 p + 1 (it is then its last). 8 NT rows x D
// sums, then 8 NT rows x (m, l, mv, unused).
template <int D, int NT>
constexpr int partial_floats() { return 8 * NT * (D + 4); }

// What a warp has of a segment: sums of 16-dim tile i and 8-row tile nt in the
// accumulator layout (element e: dim v_dim + (e >> 1), row 2 t + (e & 1)), and
// for rows 2 t + e the references and this lane's share of the weights' sum.
template <int D, int NT>
struct RowState {
  float acc[D / 16][NT][4];
  float m[NT][2], l[NT][2], mv[NT][2];
  // l over the lanes that share the rows
  __device__ __forceinline__ float sum(int nt, int e) const {
    float v = l[nt][e];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
};

// A row's share of a lane as a part (row r of 8 NT).
template <int D, int NT>
__device__ __forceinline__ void store_part(float *part, int r, const RowState<D, NT> &st, int nt, int e, float l) {
  const int g = (threadIdx.x & 31) >> 2;
  if (g == 0) *reinterpret_cast<float4 *>(part + 8 * NT * D + 4 * r) = make_float4(st.m[nt][e], l, st.mv[nt][e], 0.0f);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    *reinterpret_cast<float2 *>(part + r * D + v_dim<D>(g, i)) = make_float2(st.acc[i][nt][e], st.acc[i][nt][e + 2]);
}

// out = 2^(mv - m - kLift) sums / l; 0 where no key was seen
__device__ __forceinline__ float final_factor(float m, float l, float mv) {
  return l > 0.0f && mv != -INFINITY ? ex2(mv - m) * exp2f(-kLift) / l : 0.0f;
}

// Key tiles number x0 .. x1 - 1 (at least one) of the walk of sequence b, for
// query rows row0 .. of kv head h; by one warp with its ring of two stages.
template <int D, int NT>
__device__ __forceinline__ void attend(const KvAttnArgs &a, const KvSeq &seq, const TileWalk &walk, int32_t prefix,
                                       int32_t b, int h, int row0, int x0, int x1, uint8_t *ring,
                                       RowState<D, NT> &st) {
  using C = Cfg<D>;
  constexpr int KS = D / 16;   // contraction steps of the scores
  constexpr int MT = D / 16;   // 16-dim tiles of the output
  constexpr int ROWS = 8 * NT;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = seq.q * a.group;
  const int32_t *table_row = a.s.table + b * a.s.table_ld;
  const bool cap = a.softcap > 0.0f;
  // s = S * scale * log2(e), or with a cap c: z = S * scale / c, s = c log2(e) tanh(z)
  const float score_mul = cap ? a.scale / a.softcap : a.scale * kLog2e;
  const float cap2 = a.softcap * kLog2e;

  // this lane's query rows, asked for before the pages
  uint32_t qf[NT][KS][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + g;
    const int i = r / a.group, hq = h * a.group + (r - i * a.group);
    const uint16_t *q = a.q.p + (seq.row0 + i) * a.q.token_stride + hq * a.q.head_stride;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint2 v = make_uint2(0, 0);
      if (r < rows) v = __ldg(reinterpret_cast<const uint2 *>(q + k_dim<D>(t, k)));
      qf[nt][k][0] = v.x;
      qf[nt][k][1] = v.y;
    }
  }
  // positions of the first and last row (no row is hidden from keys at or before pos_min within the window)
  const int pos_min = seq.pos0() + row0 / a.group;
  const int pos_max = seq.pos0() + (min(row0 + ROWS, rows) - 1) / a.group;

  // Page, k's scale and log2 of v's scale of 32 granules (16 tiles), one to
  // a lane: of the window that is being computed and, fetched when it
  // begins, of the next.
  int page_c, page_n;
  float ks_c, vs_c, ks_n, vs_n;
  const auto fetch = [&](int x) {  // tiles x .. x + 15
    page_n = -1;
    ks_n = -1.0f;  // (no page, or none that is seen)
    vs_n = -INFINITY;
    const int key = walk.tile(x + (lane >> 1)) * kTile + (lane & 1) * kGran;
    if (x + (lane >> 1) >= x1 || !granule_seen(key, prefix, seq.n, max(seq.pos0(), 0), a.window)) return;
    page_n = load_page(table_row, key >> a.c.page_shift, a.c.pages, a.status);
    if (page_n < 0) return;
    const int64_t i = static_cast<int64_t>(page_n) * a.c.heads + h;
    ks_n = __ldg(a.c.ks + i);
    vs_n = log2f(__ldg(a.c.vs + i));
  };
  const auto load_tile = [&](int x, int win, int slot) {  // win: first tile of the window being computed
    if (x < x1) {
      const bool next = x >= win + 16;
      const int key0 = walk.tile(x) * kTile, y = 2 * (x - win) & 31;
      const uint32_t dst = smem_addr(ring + slot * C::kStage);
#pragma unroll
      for (int z = 0; z < 2; ++z) {  // a granule's rows are one run of kGran * D bytes
        const int page = __shfl_sync(0xFFFFFFFFu, next ? page_n : page_c, y + z);
        if (page < 0) continue;
        const int in_page = (key0 + z * kGran) & (a.c.page - 1);
        const int64_t src = (((static_cast<int64_t>(page) * a.c.heads + h) << a.c.page_shift) + in_page) * D + 16 * lane;
#pragma unroll
        for (int i = 0; i < C::kChunks / 2; ++i) {
          const int idx = i * 32 + lane, r = z * kGran + idx / C::kChunks, c = idx % C::kChunks;
          cp_async16(dst + stage_off<D>(r, c), a.c.k + src + 512 * i);
          cp_async16(dst + kTile * C::kPitch + stage_off<D>(r, c), a.c.v + src + 512 * i);
        }
      }
    }
    cp_async_commit();
  };

  fetch(x0);
  page_c = page_n, ks_c = ks_n, vs_c = vs_n;
  load_tile(x0, x0, 0);
  fetch(x0 + 16);

  // the query rows as the narrow operand of the scores, scaled into fp16's range, and as columns of S^T
  float slope[NT][2], mul[NT][2];
  int pos[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t big = 0;  // bits of the row's largest magnitude
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int z = 0; z < 2; ++z) big = max(big, max(qf[nt][k][z] & 0x7FFFu, (qf[nt][k][z] >> 16) & 0x7FFFu));
    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
    // 2^(14 - exponent of the largest) and back, exactly; a row of zeros stays one
    const int ex = min(max(static_cast<int>(big >> 7), 16), 254);
    const float up = __uint_as_float(static_cast<uint32_t>(min(127 + 127 + 14 - ex, 254)) << 23);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int z = 0; z < 2; ++z)
        qf[nt][k][z] = pack_f16x2(bf16_lo(qf[nt][k][z]) * up, bf16_hi(qf[nt][k][z]) * up);
    const float down = 1.0f / up;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mul[nt][e] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * t + e)) * score_mul;
      const int rc = row0 + nt * 8 + 2 * t + e;
      const int ic = rc / a.group;
      pos[nt][e] = rc < rows ? seq.pos0() + ic : -1;
      slope[nt][e] = a.slopes && rc < rows ? __ldg(a.slopes + h * a.group + (rc - ic * a.group)) * kLog2e : 0.0f;
    }
  }

  auto &acc = st.acc;
  auto &m = st.m, &l = st.l, &mv = st.mv;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) m[nt][e] = mv[nt][e] = -INFINITY, l[nt][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.0f;
  }

  float fv[NT][2], fv_log = NAN;  // 2^(m + log2 vs - mv + kLift) for log2 vs = fv_log
  const auto compute_tile = [&](int x, int slot, const float (&k_scale)[2], const float (&v_log)[2]) {
    const uint8_t *ks = ring + slot * C::kStage, *vs = ks + kTile * C::kPitch;
    const int key0 = walk.tile(x) * kTile;
    float s[2][NT][4];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[z][nt][e] = 0.0f;
      uint32_t w0[KS], w1[KS];
      load_k_words<D>(ks, z * kGran + g, t, w0);
      load_k_words<D>(ks, z * kGran + g + 8, t, w1);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a0, a1, a2, a3;
        codes_to_f16(w0[k], a0, a2);
        codes_to_f16(w1[k], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[z][nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[z][nt][e] *= k_scale[z] * mul[nt][e & 1];
    }
    // scores, in units of log2; element e of s[z][nt]: key 16 z + g + 8 (e >> 1), row 2 t + (e & 1)
    const bool whole = key0 + kTile - 1 <= pos_min && (a.window == 0 || key0 > pos_max - a.window) &&
                       k_scale[0] != -1.0f && k_scale[1] != -1.0f;
    if (cap) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[z][nt][e] = cap2 - __fdividef(2.0f * cap2, 1.0f + ex2(s[z][nt][e] * (2.0f * kLog2e)));
    }
    if (a.slopes || !whole) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + z * kGran + g + 8 * (e >> 1), at_q = pos[nt][e & 1];
            float v = s[z][nt][e] + slope[nt][e & 1] * static_cast<float>(j - at_q);
            if (!whole) {
              const bool seen = k_scale[z] != -1.0f && j < seq.n && at_q >= 0 &&
                                ((j <= at_q && (a.window == 0 || at_q - j < a.window)) || j < prefix);
              v = seen ? v : -INFINITY;
            }
            s[z][nt][e] = v;
          }
    }
    bool grew = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float t0 = fmaxf(s[0][nt][e], s[0][nt][e + 2]), t1 = fmaxf(s[1][nt][e], s[1][nt][e + 2]);
        grew = grew || fmaxf(t0, t1) > m[nt][e] + kRescale ||
               fmaxf(t0 + v_log[0], t1 + v_log[1]) > mv[nt][e] + kRescale;
      }
    if (__any_sync(0xFFFFFFFFu, grew)) {
      fv_log = NAN;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = -INFINITY, u = -INFINITY;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float top = fmaxf(s[z][nt][e], s[z][nt][e + 2]);
            v = fmaxf(v, top);
            u = fmaxf(u, top == -INFINITY ? top : top + v_log[z]);  // (a page no row sees may have any scale)
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, o));
          }
          if (v > m[nt][e]) {
            l[nt][e] *= ex2(m[nt][e] - v);
            m[nt][e] = v;
          }
          if (u > mv[nt][e]) {
            const float al = ex2(mv[nt][e] - u);
            mv[nt][e] = u;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              acc[i][nt][e] *= al;
              acc[i][nt][e + 2] *= al;
            }
          }
        }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (!(v_log[z] == fv_log)) {  // another page's scale, or new references
        fv_log = v_log[z];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (its exponent held in range: it passes 126 only where a page's scale is 2^100 times another's)
            const float f = m[nt][e] + fv_log - mv[nt][e] + kLift;
            fv[nt][e] = mv[nt][e] == -INFINITY ? 0.0f : ex2(f > 126.0f ? 126.0f : f);
          }
      }
      uint32_t ph[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[nt][e & 1] == -INFINITY ? 0.0f : m[nt][e & 1];  // a row that has seen no key yet
          w[e] = ex2(s[z][nt][e] - ref);
          l[nt][e & 1] += w[e];
        }
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] *= fv[nt][e & 1];
        } else {  // (a weight of 0 stays one whatever the scale of a page that the row does not see)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = w[e] > 0.0f ? w[e] * fv[nt][e & 1] : 0.0f;
        }
        ph[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        ph[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
      }
      uint32_t v0[D / 32], v1[D / 32], v2[D / 32], v3[D / 32];
      load_v_words<D>(vs, z * kGran + 2 * t, g, v0);
      load_v_words<D>(vs, z * kGran + 2 * t + 1, g, v1);
      load_v_words<D>(vs, z * kGran + 2 * t + 8, g, v2);
      load_v_words<D>(vs, z * kGran + 2 * t + 9, g, v3);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          codes_to_f16(__byte_perm(v0[w], v1[w], sel), a0, a1);
          codes_to_f16(__byte_perm(v2[w], v3[w], sel), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[2 * w + half][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
        }
      }
    }
  };

  int win = x0;
#pragma unroll 1
  for (int x = x0; x < x1; ++x) {
    if (x == win + 16) {
      win = x;
      page_c = page_n, ks_c = ks_n, vs_c = vs_n;
      fetch(x + 16);
    }
    const int slot = (x - x0) & 1, y = 2 * (x - win);
    cp_async_wait<0>();
    __syncwarp();  // every lane's copies of this tile have landed, and all have read the slot loaded next
    load_tile(x + 1, win, slot ^ 1);
    const float ks2[2] = {__shfl_sync(0xFFFFFFFFu, ks_c, y), __shfl_sync(0xFFFFFFFFu, ks_c, y + 1)};
    const float vs2[2] = {__shfl_sync(0xFFFFFFFFu, vs_c, y), __shfl_sync(0xFFFFFFFFu, vs_c, y + 1)};
    compute_tile(x, slot, ks2, vs2);
  }
  cp_async_wait<0>();
  __syncwarp();
}

// Four neighbouring dims of a row joined from parts.
struct Joined {
  float m = -INFINITY, l = 0.0f, mv = -INFINITY, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  __device__ __forceinline__ void add(const float4 &mlmv, const float4 &v) {
    const float m2 = fmaxf(m, mlmv.x), mv2 = fmaxf(mv, mlmv.z);
    if (m2 != -INFINITY) l = l * ex2(m - m2) + mlmv.y * ex2(mlmv.x - m2);
    if (mv2 != -INFINITY) {
      const float f0 = ex2(mv - mv2), f1 = ex2(mlmv.z - mv2);
      y[0] = y[0] * f0 + v.x * f1, y[1] = y[1] * f0 + v.y * f1, y[2] = y[2] * f0 + v.z * f1, y[3] = y[3] * f0 + v.w * f1;
    }
    m = m2;
    mv = mv2;
  }
  __device__ __forceinline__ void store(const KvAttnArgs &a, int64_t elem) {
    const float f = final_factor(m, l, mv);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= f;
    store_out4(a, elem, y);
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, sm_warps(NT) / kWarps)
    kv_decode_kernel(const __grid_constant__ KvAttnArgs a, float *__restrict__ partial, uint32_t *__restrict__ offsets) {
  constexpr int MT = D / 16, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait_prerequisite();
  pdl_launch_dependents();  // after the wait: the join may read the lengths before its own
  uint32_t all, before;
  const uint32_t p = warp * gridDim.x + blockIdx.x;  // few pieces spread over all SMs
  const uint32_t sum =
      count_units<ROWS, kSetup>(a, -1, p == 0 ? a.status : nullptr, p == 0 ? offsets : nullptr, before, all);
  if (all == 0) return;
  const Cut cut(all, gridDim.x * kWarps, kMinUnits);
  if (p >= cut.pieces) return;
  PieceWalk<ROWS, kSetup> w(a, cut, p, sum);
  while (w.next(a)) {
    RowState<D, NT> st;
    attend<D, NT>(a, w.work.seq, w.work.walk, w.work.prefix, w.b, w.h, w.row0, w.x0, w.x1,
                  smem + warp * (kStages * Cfg<D>::kStage), st);
    const int rows = w.work.seq.q * a.group;
    const bool whole = w.whole();
    float *out_p = partial + static_cast<int64_t>(2 * p + (w.first ? 0 : 1)) * partial_floats<D, NT>();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float l = st.sum(nt, e);
        const int r = nt * 8 + 2 * t + e;
        if (w.row0 + r >= rows) continue;
        if (whole) {
          const float f = final_factor(st.m[nt][e], l, st.mv[nt][e]);
          const int qi = (w.row0 + r) / a.group, hq = w.h * a.group + (w.row0 + r - qi * a.group);
          const int64_t elem = (static_cast<int64_t>(w.work.seq.row0 + qi) * a.q_heads + hq) * D;
#pragma unroll
          for (int i = 0; i < MT; ++i)
            store_out2(a, elem + v_dim<D>(g, i), st.acc[i][nt][e] * f, st.acc[i][nt][e + 2] * f);
        } else {
          store_part(out_p, r, st, nt, e, l);
        }
      }
  }
}

// Pieces of a block of all the SM's warps. per_segment: block (kv head and row
// block, sequence) has that segment; else the units are cut over the blocks.
template <int D, int NT>
__global__ void __launch_bounds__(32 * sm_warps(NT), 1)
    kv_decode_block_kernel(const __grid_constant__ KvAttnArgs a, float *__restrict__ partial,
                           uint32_t *__restrict__ offsets, int per_segment, int row_blocks) {
  using C = Cfg<D>;
  constexpr int ROWS = 8 * NT, F = partial_floats<D, NT>(), BW = sm_warps(NT);
  static_assert(F * sizeof(float) <= kStages * C::kStage, "a warp's sums fit its ring");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
  uint8_t *const ring = smem + warp * (kStages * C::kStage);
  pdl_wait_prerequisite();
  pdl_launch_dependents();  // after the wait: the join may read the lengths before its own

  // Tiles x0 .. x1 - 1 of a segment by the block; out_p: where the sums go, or nullptr for the output.
  const auto run = [&](const SeqWork<kBlockSetup> &work, int32_t b, int h, int row0, int x0, int x1, float *out_p) {
    const int rows = work.seq.q * a.group;
    const int per = (x1 - x0 + BW - 1) / BW, used = per > 0 ? (x1 - x0 + per - 1) / per : 0;
    if (warp < used) {
      RowState<D, NT> st;
      attend<D, NT>(a, work.seq, work.walk, work.prefix, b, h, row0, x0 + warp * per, min(x1, x0 + (warp + 1) * per),
                    ring, st);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          store_part(reinterpret_cast<float *>(ring), nt * 8 + 2 * t + e, st, nt, e, st.sum(nt, e));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += 32 * BW) {
      const int r = i / (D / 4), d = 4 * (i - r * (D / 4));
      if (row0 + r >= rows) continue;
      Joined y;
      for (int w = 0; w < used; ++w) {
        const float *part = reinterpret_cast<const float *>(smem + w * (kStages * C::kStage));
        y.add(*reinterpret_cast<const float4 *>(part + ROWS * D + 4 * r), *reinterpret_cast<const float4 *>(part + r * D + d));
      }
      if (out_p) {
        *reinterpret_cast<float4 *>(out_p + r * D + d) = make_float4(y.y[0], y.y[1], y.y[2], y.y[3]);
        if (d == 0) *reinterpret_cast<float4 *>(out_p + ROWS * D + 4 * r) = make_float4(y.m, y.l, y.mv, 0.0f);
      } else {
        const int qi = (row0 + r) / a.group, hq = h * a.group + (row0 + r - qi * a.group);
        y.store(a, (static_cast<int64_t>(work.seq.row0 + qi) * a.q_heads + hq) * D + d);
      }
    }
  };

  if (per_segment) {
    const int b = blockIdx.y, h = blockIdx.x / row_blocks, row0 = (blockIdx.x - h * row_blocks) * ROWS;
    const SeqWork<kBlockSetup> work = seq_work<ROWS, kBlockSetup>(a, b, a.status);
    if (row0 < work.seq.q * a.group) run(work, b, h, row0, 0, work.walk.count, nullptr);
    return;
  }
  uint32_t all, before;
  const uint32_t p = blockIdx.x;
  const bool first = p == 0 && warp == 0;
  const uint32_t sum =
      count_units<ROWS, kBlockSetup>(a, -1, first ? a.status : nullptr, first ? offsets : nullptr, before, all);
  if (all == 0) return;
  const Cut cut(all, gridDim.x, kBlockMinUnits);
  if (p >= cut.pieces) return;
  PieceWalk<ROWS, kBlockSetup> w(a, cut, p, sum);
  while (w.next(a)) {
    run(w.work, w.b, w.h, w.row0, w.x0, w.x1,
        w.whole() ? nullptr : partial + static_cast<int64_t>(2 * p + (w.first ? 0 : 1)) * F);
    __syncthreads();  // the rings hold the sums until all have been read
  }
}

// Joins the parts of each segment row; block (kv head and row, sequence). A
// segment that one piece holds is written already; one without keys is zeros.
template <int D, int NT, int SETUP>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const __grid_constant__ KvAttnArgs a,
                                                                  const float *partial, const uint32_t *offsets,
                                                                  uint32_t most_pieces, uint32_t min_units,
                                                                  int max_rows) {
  constexpr int ROWS = 8 * NT, F = partial_floats<D, NT>();
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float4 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int h = blockIdx.x / max_rows, row = blockIdx.x % max_rows;
  uint32_t before, all;
  if (offsets) {
    pdl_wait_prerequisite();
    before = offsets[b], all = offsets[a.s.batch];
  } else {  // the lengths: written before the kernel that this one follows passed its own wait
    count_units<ROWS, SETUP>(a, b, nullptr, nullptr, before, all);
  }
  const SeqWork<SETUP> work = seq_work<ROWS, SETUP>(a, b, nullptr);
  const Cut cut(all, most_pieces, min_units);
  const int rbs = work.segs / a.c.heads;
  const uint32_t s0 = before + (h * rbs + row / ROWS) * work.seg_units();
  uint32_t p0 = 0, p1 = 0;
  if (row < work.seq.q * a.group && work.walk.count > 0) {
    p0 = cut.piece_of(s0 + SETUP);
    p1 = cut.piece_of(s0 + work.seg_units() - 1);
  }
  pdl_launch_dependents();
  if (!offsets) pdl_wait_prerequisite();
  if (row >= work.seq.q * a.group || (work.walk.count > 0 && p0 == p1)) return;
  Joined y;
  if (work.walk.count > 0) {
    const int r = row % ROWS;
    constexpr int N = 4;  // parts in flight
    for (uint32_t q = p0 + warp; q <= p1; q += N * kJoinWarps) {
      float4 ml[N], v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t p = q + i * kJoinWarps;
        ml[i] = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p > p1) continue;
        const float *part = partial + static_cast<int64_t>(2 * p + (cut.begin(p) < s0 ? 1 : 0)) * F;
        ml[i] = *reinterpret_cast<const float4 *>(part + ROWS * D + 4 * r);
        if (4 * lane < D) v[i] = *reinterpret_cast<const float4 *>(part + r * D + 4 * lane);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) y.add(ml[i], v[i]);
    }
    if (4 * lane < D) *reinterpret_cast<float4 *>(&s_acc[warp][4 * lane]) = make_float4(y.y[0], y.y[1], y.y[2], y.y[3]);
    if (lane == 0) s_ml[warp] = make_float4(y.m, y.l, y.mv, 0.0f);
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (4 * lane < D) v = *reinterpret_cast<const float4 *>(&s_acc[w][4 * lane]);
      y.add(s_ml[w], v);
    }
  } else if (warp > 0) {
    return;
  }
  if (4 * lane >= D) return;
  const int qi = row / a.group, hq = h * a.group + (row - qi * a.group);
  y.store(a, (static_cast<int64_t>(work.seq.row0 + qi) * a.q_heads + hq) * D + 4 * lane);
}

bool wide_rows(const KvAttnArgs &a) { return static_cast<int64_t>(a.s.max_q) * a.group > 8; }

int row_blocks_of(const KvAttnArgs &a) {
  const int per = wide_rows(a) ? 16 : 8;
  return (a.s.max_q * a.group + per - 1) / per;
}

int64_t most_segments(const KvAttnArgs &a) { return static_cast<int64_t>(a.s.batch) * a.c.heads * row_blocks_of(a); }

// A block to a segment: no more segments than SMs, of at most kShortKeys keys
// (a window without a prefix bounds them too). Against pieces of warps, head
// dim 128, us a call: 8 segments of 8 rows x 512 keys 7.5 : 10.5, x 1024
// 10.1 : 10.7, x 2048 15.3 : 11.4; 128 segments x 1024 10.5 : 15.3; 64 of 16
// rows x 1024 15.5 : 17.0, x 2048 22.6 : 21.0.
constexpr int64_t kShortKeys = 1024;

bool block_segments(const KvAttnArgs &a, int num_sms) {
  const int64_t keys = a.window > 0 && !a.prefix && static_cast<int64_t>(a.window) + a.s.max_q < a.s.max_kv
                           ? static_cast<int64_t>(a.window) + a.s.max_q
                           : a.s.max_kv;
  return keys <= kShortKeys && most_segments(a) <= num_sms;
}

// Pieces of blocks: at most 8 rows, at most two segments an SM, and room for
// kBlockTiles key tiles an SM (8 a warp). Against pieces of warps: 128
// segments x 4096 keys 32 : 36, x 8192 50 : 67, but x 2048 21 : 17; with 16 rows
// 64 segments x 8192 49 : 39.
constexpr int64_t kBlockTiles = 100;

bool block_pieces(const KvAttnArgs &a, int num_sms) {
  const int64_t segs = most_segments(a);
  return !wide_rows(a) && segs <= 2 * num_sms && segs * (a.s.max_kv / kTile) >= kBlockTiles * num_sms;
}

// Sequences up to which each block of the join finds the units before its own
// by a scan, while the kernel before it ends; with more it reads what that
// kernel's first warp has left in the workspace, once it has ended. Scan : read,
// us a call, 4 kv heads of 4, 200 and 1500 keys: 64 sequences 15.7 28.1 : 16.2
// 27.0, 96 18.1 38.6 : 17.7 38.4, 128 22.9 48.0 : 20.8 46.6, 256 40 91 : 30 82,
// 1024 283 462 : 99 282 (the scan's cost grows with the square).
constexpr int32_t kScanSequences = 96;

// The parts in the workspace, two a piece; the units before each sequence follow them.
int64_t partials_floats(const KvAttnArgs &a, int num_sms) {
  const int64_t pieces = block_pieces(a, num_sms) ? num_sms : static_cast<int64_t>(num_sms) * sm_warps(wide_rows(a) ? 2 : 1);
  return 2 * pieces * (wide_rows(a) ? 16 : 8) * (a.c.d + 4);
}

template <int D, int NT>
cudaError_t launch_t(const KvAttnArgs &a, float *partial, int num_sms, cudaStream_t s) {
  using C = Cfg<D>;
  uint32_t *const offsets =
      a.s.batch > kScanSequences ? reinterpret_cast<uint32_t *>(partial + partials_floats(a, num_sms)) : nullptr;
  constexpr size_t kBlockSmem = C::kSmem / kWarps * sm_warps(NT);
  static_assert(kBlockSmem <= 227 * 1024, "shared memory per CTA");
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int row_blocks = row_blocks_of(a), max_rows = a.s.max_q * a.group;
  const dim3 join_grid(a.c.heads * max_rows, a.s.batch);
  const bool per_segment = block_segments(a, num_sms);
  if (per_segment || block_pieces(a, num_sms)) {
    cudaError_t e = ensure_kernel_smem<kv_decode_block_kernel<D, NT>>(static_cast<int>(kBlockSmem), true);
    if (e != cudaSuccess) return e;
    cfg.gridDim = per_segment ? dim3(a.c.heads * row_blocks, a.s.batch) : dim3(num_sms);
    cfg.blockDim = dim3(32 * sm_warps(NT));
    cfg.dynamicSmemBytes = kBlockSmem;
    e = cudaLaunchKernelEx(&cfg, kv_decode_block_kernel<D, NT>, a, partial, offsets, per_segment ? 1 : 0, row_blocks);
    if (e != cudaSuccess || per_segment) return e;
    cfg.gridDim = join_grid;
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT, kBlockSetup>, a, static_cast<const float *>(partial),
                              static_cast<const uint32_t *>(offsets), static_cast<uint32_t>(num_sms), static_cast<uint32_t>(kBlockMinUnits), max_rows);
  }
  cudaError_t e = ensure_kernel_smem<kv_decode_kernel<D, NT>>(static_cast<int>(C::kSmem), true);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(num_sms * (sm_warps(NT) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  const uint32_t warps = cfg.gridDim.x * kWarps;
  e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<D, NT>, a, partial, offsets);
  if (e != cudaSuccess) return e;
  cfg.gridDim = join_grid;
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT, kSetup>, a, static_cast<const float *>(partial),
                            static_cast<const uint32_t *>(offsets), warps, static_cast<uint32_t>(kMinUnits), max_rows);
}

template <int D>
cudaError_t launch_d(const KvAttnArgs &a, float *partial, int num_sms, cudaStream_t s) {
  return wide_rows(a) ? launch_t<D, 2>(a, partial, num_sms, s) : launch_t<D, 1>(a, partial, num_sms, s);
}

}  // namespace

bool kv_decode_fits(const KvAttnArgs &a) {  // all units in 31 bits
  const int64_t per = a.s.max_kv / kTile + 2 + kBlockSetup;
  return most_segments(a) <= INT32_MAX / per;
}

size_t kv_decode_workspace_bytes(const KvAttnArgs &a, int num_sms) {
  // None where a block has a segment. (The query knows no window and no
  // prefix: what it says is enough for any.)
  KvAttnArgs any = a;
  any.window = 0;
  if (block_segments(any, num_sms)) return 0;
  return static_cast<size_t>(partials_floats(a, num_sms)) * sizeof(float) +
         (a.s.batch > kScanSequences ? (a.s.batch + 1) * sizeof(uint32_t) : 0);
}

cudaError_t launch_kv_decode(const KvAttnArgs &a, void *workspace, int num_sms, cudaStream_t s) {
  float *partial = static_cast<float *>(workspace);
  switch (a.c.d) {
    case 64: return launch_d<64>(a, partial, num_sms, s);
    case 96: return launch_d<96>(a, partial, num_sms, s);
    case 128: return launch_d<128>(a, partial, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace w8a8
