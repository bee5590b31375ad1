// kv_prefill.cu -- attention of many new tokens over the INT8 paged KV cache,
// on the 5th-generation tensor cores.
//
// What it computes: as kv_decode.cu (one pass over the keys with a running
// maximum m and sum l), for chunks of prompts.
//
// How (sm_100a), two kernels:
//   kv_expand_kernel writes the sequences' codes as bf16 (exactly) into dense
//   [sequence][kv head][key][dim] matrices, 128-key tiles zero-padded, with
//   the scales of each granule of 16 keys beside them. Every key tile is used
//   by many query tiles; expanded once, it comes back through TMA in the
//   layout the MMAs read and no query tile converts anything. One of its
//   blocks lists the query blocks, those with the most key tiles first.
//   kv_prefill_kernel: persistent, one block per SM, which takes (query
//   block, kv head) items from that list. An item is 256 query rows in two
//   tiles of 128 = floor(128 / group) tokens x group heads, so that grouped
//   heads share their key tiles. Roles:
//     warps 0-3, 4-7  softmax of tile A and of tile B, one thread per row:
//                 S from TMEM (tcgen05.ld), maximum, 2^(s - m), row sum, and
//                 the weights times v's scale back into TMEM as the bf16 A
//                 operand of the second product (over S, which is dead by
//                 then); at the end O / l to global memory, through shared
//                 memory so that neighbouring lanes store neighbouring bytes;
//     warp 8      takes items and loads 128-byte-swizzled boxes of 64 dims by
//                 TMA: key tiles of K and V into a ring;
//     warp 9      MMA issuer: S = Q K^T (both K-major in shared memory) and
//                 O += P V (P in TMEM, V as an MN-major operand, so V needs
//                 no transpose). While one tile's softmax runs, the other
//                 tile's products do; the next item's first scores are
//                 computed while this one's output is written;
//     warp 10     loads the next item's query rows as soon as the last scores
//                 of this one are done, as boxes of floor(128 / group) tokens x
//                 group heads of the packed queries, which lie in shared
//                 memory in the row order of a tile.
//   The page scales never touch the operands: k's multiplies the scores (a
//   granule's maximum is scaled once, an element's factor is that of the
//   fused multiply-add before 2^x), v's multiplies the weights.
//   O is rescaled only when a row's maximum has grown by more than 2^8 since
//   its last reference (weights then stay below 2^8 and nothing is lost in
//   fp32); the softmax warps do it themselves between the products, since
//   S_w(j) complete implies O_w(j - 1) complete.
//   TMEM: S_A, S_B (128 columns each, fp32; P in their first 64), O_A, O_B.
//
// What bounds it: a pair of 128 x 128 tiles (head dim 128) takes 3450 cycles
// in the steady state, of which the products need 2060 (a k step of 16 of
// either takes 64 cycles) and the exponentials 2048 (16 a cycle); the rest is
// the chain scores -> softmax -> weights -> O -> next scores of one tile, which the
// other tile's work does not hide all of: TMEM has no room for a second
// buffer of scores beside both outputs. Tiles of 64 keys with two buffers: a
// 64-column product takes 48 cycles a k step instead of 32, 502 us at 8192
// against 445. Sixteen softmax warps: 96 registers each are too few for the
// row, slower. Some of the exponentials as polynomials on the FMA pipe:
// slower from the first element on.
// Measured (device time, both kernels, 32 heads of 128): a prompt of 2048 59 us;
// of 8192 (550 GFLOP) 449 us at 1965 MHz, 1.22 PFLOP/s and 0.73 of the rate of a
// large bf16 product in a short run, but 515 at the power cap's 1687 MHz after
// seconds (0.88 and 0.87 s MHz), 0.76 of what such a product keeps up there.
//   The weights are bf16 because they carry v's scales, whose range fp16 has
// only against a reference for each row, which kv_decode.cu keeps and which
// would cost this kernel a second running maximum. Against a 64-bit evaluation
// the output is off by 0.0023 to 0.0026 where its own rounding to bf16 is 0.0017.
#include <type_traits>

#include "kv_common.cuh"

namespace w8a8 {

namespace {

constexpr int kKeys = 128;             // keys of a tile
constexpr int kRows = 128;             // query rows of a tile = TMEM lanes
constexpr int kBox = kKeys * 128;      // bytes of a 64-dim box of 128 rows
constexpr int kSlots = 4;              // key tiles (K or V) in flight
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);  // softmax, key tiles, MMA, query rows, one idle
constexpr int kStageRow = 128;         // bytes of a row in a softmax warp's output staging (64 dims)
constexpr int kStage = 32 * kStageRow;
// Registers a thread: 168 at launch (65536 / 384); a softmax thread holds a
// whole row of 128 scores and wants more, the others few.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
static_assert(32 * kSoftmaxWarps * kSoftmaxRegs + 32 * 4 * kOtherRegs <= kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;        // S_A 0, S_B 128, O_A 256, O_B 384
constexpr float kRescale = 8.0f;       // log2 of how far a maximum may outgrow its reference

template <int D>
struct PCfg {
  static constexpr int kAtoms = D > 64 ? 2 : 1;       // 64-dim boxes of a row
  static constexpr int kPitch = 64 * kAtoms;          // elements of an expanded row
  static constexpr int kTile = kAtoms * kBox;         // bytes of a K, V or Q tile
  static constexpr size_t kSmem = static_cast<size_t>(2 + kSlots) * kTile + kSoftmaxWarps * kStage + 1024 + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

int64_t expanded_len(int32_t max_kv) { return (static_cast<int64_t>(max_kv) + kKeys - 1) / kKeys * kKeys; }

// ------------------------------------------------------------------ expansion
// Block (x > 0): 64 keys of one (kv head, sequence). Rows from the sequence's end to
// the end of its last 128-key tile are zeros (they meet weights of 0, and
// must not be NaN). A granule's scales: of its page; 0 past the end; -1 (k's)
// for a page that does not exist or of which no query sees a key there, and
// whose codes are then zeros.
constexpr int kExpandKeys = 64;
constexpr int kExpandThreads = 256;

// A query block, or a part of one: its first packed row, the position of that
// row's token, its tokens (of 2 floor(128 / group) at most), its sequence, the
// part [x0, x1) of the key tiles it walks, and where a part leaves its sums.
struct __align__(16) QueryBlock {
  int32_t row, pos, toks, b;
  int32_t n, prefix, x0, x1;
  int32_t slot;   // of parts: slot * kv heads + head in the workspace; -1: the block is whole
  int32_t parts;  // in the list of split blocks: how many, from `slot` on
  int32_t pad[2];
};

struct Expanded {
  uint16_t *k, *v;      // [sequence][head][len][pitch]
  float *ks, *vs;       // [sequence][head][len / 16]
  int64_t len;
  int32_t *counters;    // [0] entries listed, [1] items taken, [2] blocks split
  QueryBlock *blocks;   // blocks and parts, those with the most key tiles first
  QueryBlock *split;    // blocks in parts
  float *parts;         // [slot][kv head]: sums [2][128][D], then (maximum, sum of weights) [2][128][2]
  int32_t slots;        // query blocks there may be
  int32_t most_parts;   // parts there may be (0: blocks stay whole)
  int32_t sms;
};

// The list of query blocks, by one block of kExpandThreads threads: a counting
// sort by the number of key tiles, descending. Slot f(b) = seq_start[b] / T + b
// leaves sequence b room for its ceil(q / T) blocks of T tokens. The order of
// entries with equally many tiles is left open; it decides only where and when
// one runs.
//   Where there are few blocks (the host allows parts), one with many more key
// tiles than an even share of all of them over the SMs is split into parts of
// at most that share. Parts of split blocks are at most twice the SMs: each
// split block has more than a share, so ceil(count / share) < 2 count / share.
constexpr int kBins = 2048;
constexpr int kMinShare = 4, kMinOver = 8;

__device__ void list_query_blocks(const KvAttnArgs &a, const Expanded &x) {
  __shared__ int32_t s_bin[kBins], s_sum[kExpandThreads], s_count[2];  // split blocks; parts
  __shared__ unsigned long long s_all;                                 // tiles
  const int T = 2 * (kRows / a.group), tid = threadIdx.x;
  int shift = 0;
  while ((x.len / kKeys) >> shift >= kBins) ++shift;
  for (int i = tid; i < kBins; i += kExpandThreads) s_bin[i] = 0;
  if (tid < 2) s_count[tid] = 0;
  if (tid == 0) s_all = 0;
  __syncthreads();
  const auto block_of = [&](int32_t slot, QueryBlock &q) {
    int lo = 0, hi = a.s.batch;  // the last sequence whose slots begin at or before this one
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.s.seq_start + mid) / T + mid <= slot)
        lo = mid + 1;
      else
        hi = mid;
    }
    const int b = lo - 1;
    if (b < 0) return false;
    const KvSeq seq = load_seq(a.s, b, a.s.max_kv, a.status);
    const int64_t tok = static_cast<int64_t>(slot - (__ldg(a.s.seq_start + b) / T + b)) * T;
    if (tok < 0 || tok >= seq.q) return false;
    q.b = b;
    q.row = seq.row0 + static_cast<int>(tok);
    q.pos = seq.pos0() + static_cast<int>(tok);
    q.toks = min(T, seq.q - static_cast<int>(tok));
    q.n = seq.n;
    q.prefix = a.prefix ? __ldg(a.prefix + b) : 0;
    q.x0 = 0;
    q.x1 = tile_walk(kKeys, q.prefix, q.n, max(q.pos, 0), q.pos + q.toks, a.window).count;
    q.slot = -1;
    q.parts = 1;
    q.pad[0] = q.pad[1] = 0;
    return true;
  };
  // Each thread's first block is kept: where blocks may be split there are
  // hardly more of them than threads, and the search is most of the work.
  QueryBlock q0;
  const bool has0 = tid < x.slots && block_of(tid, q0);
  const auto each = [&](auto f) {
    if (has0) f(q0);
    QueryBlock q;
    for (int slot = tid + kExpandThreads; slot < x.slots; slot += kExpandThreads)
      if (block_of(slot, q)) f(q);
  };
  int share = INT32_MAX;
  if (x.most_parts > 0) {
    unsigned long long sum = 0;
    each([&](const QueryBlock &q) { sum += q.x1; });
    atomicAdd(&s_all, sum);
    __syncthreads();
    const int64_t all = static_cast<int64_t>(s_all) * a.c.heads;
    share = static_cast<int>(min(int64_t(INT32_MAX / 2), max(int64_t(kMinShare), (all + x.sms - 1) / x.sms)));
  }
  // (a part more costs about 4 tiles and the join as much: not for a few tiles over the share)
  const auto parts_of = [&](int count) {
    return share < INT32_MAX && count > share + max(kMinOver, share / 2) ? (count + share - 1) / share : 1;
  };
  const auto bin_of = [&](int tiles) { return kBins - 1 - min(tiles >> shift, kBins - 1); };
  each([&](const QueryBlock &q) {
    const int parts = parts_of(q.x1), per = (q.x1 + parts - 1) / parts;
    for (int i = 0; i < parts; ++i) atomicAdd(&s_bin[bin_of(min(per, q.x1 - i * per))], 1);
  });
  __syncthreads();
  // exclusive scan of the bins, kBins / kExpandThreads to a thread
  constexpr int PER = kBins / kExpandThreads;
  int sum = 0;
  for (int i = 0; i < PER; ++i) sum += s_bin[tid * PER + i];
  s_sum[tid] = sum;
  __syncthreads();
  for (int o = 1; o < kExpandThreads; o <<= 1) {
    const int v = tid >= o ? s_sum[tid - o] : 0;
    __syncthreads();
    s_sum[tid] += v;
    __syncthreads();
  }
  int at = s_sum[tid] - sum;
  for (int i = 0; i < PER; ++i) {
    const int c = s_bin[tid * PER + i];
    s_bin[tid * PER + i] = at;
    at += c;
  }
  if (tid == kExpandThreads - 1) {
    x.counters[0] = at;
    x.counters[1] = 0;
  }
  __syncthreads();
  each([&](QueryBlock q) {
    const int count = q.x1, parts = parts_of(count), per = (count + parts - 1) / parts;
    if (parts > 1) {
      q.slot = atomicAdd(&s_count[1], parts);
      q.parts = parts;
      x.split[atomicAdd(&s_count[0], 1)] = q;
    }
    const int slot0 = q.slot;
    for (int i = 0; i < parts; ++i) {
      if (parts > 1) q.slot = slot0 + i;
      q.x0 = i * per;
      q.x1 = min(count, q.x0 + per);
      x.blocks[atomicAdd(&s_bin[bin_of(q.x1 - q.x0)], 1)] = q;
    }
  });
  __syncthreads();
  if (tid == 0) x.counters[2] = s_count[0];
}

template <int D>
__global__ void __launch_bounds__(kExpandThreads, 6) kv_expand_kernel(const __grid_constant__ KvAttnArgs a,
                                                                   const __grid_constant__ Expanded x) {
  constexpr int CH = D / 8, PITCH = PCfg<D>::kPitch;  // 8 codes to a lane: its 16-byte stores make one run
  __shared__ int32_t s_page[kExpandKeys / kGran];
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0 && blockIdx.z == 0) list_query_blocks(a, x);
    return;
  }
  const int b = blockIdx.z, h = blockIdx.y, key0 = (blockIdx.x - 1) * kExpandKeys;
  const KvSeq seq = load_seq(a.s, b, a.s.max_kv, a.status);
  if (seq.q == 0 || key0 >= (seq.n + kKeys - 1) / kKeys * kKeys) return;
  const int32_t prefix = a.prefix ? __ldg(a.prefix + b) : 0;
  const TileWalk walk = tile_walk(kKeys, prefix, seq.n, max(seq.pos0(), 0), seq.n, a.window);
  if (key0 >= walk.n1 * kKeys && key0 < walk.t0 * kKeys) return;  // no query sees this tile
  const int64_t row0 = (static_cast<int64_t>(b) * a.c.heads + h) * x.len + key0;
  if (threadIdx.x < kExpandKeys / kGran) {
    const int key = key0 + threadIdx.x * kGran;
    int32_t page = -1;
    float ks = 0.0f, vs = 0.0f;
    if (key < seq.n) {
      if (granule_seen(key, prefix, seq.n, max(seq.pos0(), 0), a.window))
        page = load_page(a.s.table + b * a.s.table_ld, key >> a.c.page_shift, a.c.pages, a.status);
      ks = page < 0 ? -1.0f : __ldg(a.c.ks + static_cast<int64_t>(page) * a.c.heads + h);
      vs = page < 0 ? 0.0f : __ldg(a.c.vs + static_cast<int64_t>(page) * a.c.heads + h);
    }
    s_page[threadIdx.x] = page;
    const int64_t at = row0 / kGran + threadIdx.x;
    x.ks[at] = ks;
    x.vs[at] = vs;
  }
  __syncthreads();
  constexpr int N = (kExpandKeys * CH + kExpandThreads - 1) / kExpandThreads;
  uint2 kv[N][2];  // every load of the thread in flight before the first is used
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int i = n * kExpandThreads + threadIdx.x, r = i / CH, c = i - r * CH;
    kv[n][0] = kv[n][1] = make_uint2(0, 0);
    if (r >= kExpandKeys) continue;
    const int key = key0 + r;
    const int32_t page = s_page[r / kGran];
    if (page < 0 || key >= seq.n) continue;
    const int64_t src =
        (((static_cast<int64_t>(page) * a.c.heads + h) << a.c.page_shift) + (key & (a.c.page - 1))) * D + 8 * c;
    kv[n][0] = __ldg(reinterpret_cast<const uint2 *>(a.c.k + src));
    kv[n][1] = __ldg(reinterpret_cast<const uint2 *>(a.c.v + src));
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int i = n * kExpandThreads + threadIdx.x, r = i / CH, c = i - r * CH;
    if (r >= kExpandKeys) continue;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint4 o;
      codes_to_bf16(kv[n][z].x, o.x, o.y);
      codes_to_bf16(kv[n][z].y, o.z, o.w);
      *reinterpret_cast<uint4 *>((z ? x.v : x.k) + (row0 + r) * PITCH + 8 * c) = o;
    }
  }
}

// ------------------------------------------------------------------ attention
__device__ __forceinline__ void fma2(float &x0, float &x1, float c, float d) {  // x = x c + d, two at a time
  asm("{\n\t.reg .b64 a, b, e;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 e, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, e;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(c), "f"(d));
}
using Yes = std::true_type;
using No = std::false_type;

__device__ __forceinline__ void axpy2(float &y0, float &y1, float x0, float x1, float c) {  // y += x c, two at a time
  asm("{\n\t.reg .b64 a, b, e;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 e, {%0, %1};\n\t"
      "fma.rn.f32x2 e, a, b, e;\n\tmov.b64 {%0, %1}, e;\n\t}"
      : "+f"(y0), "+f"(y1)
      : "f"(x0), "f"(x1), "f"(c));
}
// Bits 0 .. n - 1 of a granule (n below 0 or past 16 taken as 0 or 16).
__device__ __forceinline__ uint32_t bits_below(int n) { return (1u << min(max(n, 0), 16)) - 1u; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void add2(float &x0, float &x1, float y0, float y1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}

// An item as its block's warps see it.
struct Item {
  QueryBlock q;
  int32_t h, pad[3];
};

// Floats of a part's sums and of its rows' (maximum, sum of weights).
template <int D>
constexpr int part_floats() { return 2 * kRows * (D + 2); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmOut,
                      const __grid_constant__ KvAttnArgs a, const __grid_constant__ Expanded x, uint64_t limit_ns) {
  using C = PCfg<D>;
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base;                                 // two tiles
  uint8_t *sKV = base + 2 * C::kTile;                 // ring of key tiles
  uint8_t *sStage = sKV + kSlots * C::kTile;          // [softmax warp] output staging
  Item *s_item = reinterpret_cast<Item *>(sStage + kSoftmaxWarps * kStage);  // [2]
  uint64_t *full_bar = reinterpret_cast<uint64_t *>(s_item + 2);
  uint64_t *empty_bar = full_bar + kSlots;
  uint64_t *s_bar = empty_bar + kSlots;  // [tile] scores are in TMEM
  uint64_t *p_bar = s_bar + 2;           // [tile][half of the keys] weights are (one arrival per softmax warp)
  uint64_t *o_bar = p_bar + 4;           // [tile] the output is final
  uint64_t *qfull_bar = o_bar + 2;       // [tile] query rows are in shared memory
  uint64_t *qempty_bar = qfull_bar + 2;  // [tile] their last product is complete
  uint64_t *ifull_bar = qempty_bar + 2;  // [2] an item is there
  uint64_t *iempty_bar = ifull_bar + 2;  // [2] every warp is done with it
  uint64_t *drain_bar = iempty_bar + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_bar + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(2 * sizeof(Item) + (2 * kSlots + 17) * 8 + 8 <= 512, "items, barriers and flags fit their reserve");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmQ);
    if (x.len > 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_bar[t], 1);
      mbar_init(&p_bar[2 * t], kSoftmaxWarps / 2);
      mbar_init(&p_bar[2 * t + 1], kSoftmaxWarps / 2);
      mbar_init(&o_bar[t], 1);
      mbar_init(&qfull_bar[t], 1);
      mbar_init(&qempty_bar[t], 1);
      mbar_init(&ifull_bar[t], 1);
      mbar_init(&iempty_bar[t], kSoftmaxWarps + 2);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const uint32_t tmem = *tmem_slot;
  const int tpt = kRows / a.group;  // tokens of a tile

  // Tokens of an item's tile A (t = 0) or B, the key tiles it walks (from
  // number x0 of the walk), and the walk. Both tiles walk from the block's
  // first key, so one walk is a prefix of the other.
  const auto toks_of = [&](const QueryBlock &q, int t) { return max(0, min(tpt, q.toks - t * tpt)); };
  const auto count_of = [&](const QueryBlock &q, int t) {
    const int toks = toks_of(q, t), last = q.pos + t * tpt + toks;  // one past its last position
    const int count = toks > 0 && last > 0 ? tile_walk(kKeys, q.prefix, q.n, max(q.pos, 0), last, a.window).count : 0;
    return max(0, min(count, q.x1) - q.x0);
  };
  const auto walk_of = [&](const QueryBlock &q) {
    return tile_walk(kKeys, q.prefix, q.n, max(q.pos, 0), q.n, a.window);
  };
  // The it-th item of this block (false: there are no more, or the kernel gave up).
  const auto take = [&](int it, Item &item, bool &ok) {
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&ifull_bar[it & 1], static_cast<uint32_t>(it >> 1) & 1u, abort_flag,
                                                   limit_ns))) {
      ok = false;
      return false;
    }
    item = s_item[it & 1];
    return item.q.toks > 0;
  };
  const auto done_with = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty_bar[it & 1]);
  };
  const auto fail = [&]() {
    record_error(a.status, W8A8_ERR_DEVICE_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps) {
      if (lane == 0) {
        // ------------------------------------------------ items, and their key tiles by TMA:
        // K(0), then V(j), K(j + 1) for j = 0, 1, ..., the order in which the MMAs use them
        bool ok = true;
        int i = 0;  // ring items loaded
        const int32_t items = x.counters[0] * a.c.heads;
        const auto load = [&](const CUtensorMap *map, int64_t key) {
          if (!ok) return;
          const int s = i % kSlots;
          if (!mbar_wait_bounded(&empty_bar[s], (static_cast<uint32_t>(i / kSlots) & 1u) ^ 1u, abort_flag, limit_ns)) {
            ok = false;
            return;
          }
          mbar_arrive_expect_tx(&full_bar[s], C::kTile);
#pragma unroll
          for (int c = 0; c < C::kAtoms; ++c)
            tma_load_2d(map, &full_bar[s], sKV + s * C::kTile + c * kBox, 64 * c, static_cast<int32_t>(key));
          ++i;
        };
        for (int it = 0; ok; ++it) {
          const int32_t n = atomicAdd(x.counters + 1, 1);
          Item item = {};
          if (n < items) {
            item.q = x.blocks[n / a.c.heads];
            item.h = n % a.c.heads;
          }
          if (!mbar_wait_bounded(&iempty_bar[it & 1], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, limit_ns)) {
            ok = false;
            break;
          }
          s_item[it & 1] = item;
          mbar_arrive(&ifull_bar[it & 1]);
          if (n >= items) break;
          const TileWalk walk = walk_of(item.q);
          const int most = max(count_of(item.q, 0), count_of(item.q, 1));
          const int64_t key0 = (static_cast<int64_t>(item.q.b) * a.c.heads + item.h) * x.len;
          const int x0 = item.q.x0;
          if (most > 0) load(&tmK, key0 + walk.tile(x0) * kKeys);
          for (int j = 0; j < most && ok; ++j) {
            load(&tmV, key0 + walk.tile(x0 + j) * kKeys);
            if (j + 1 < most) load(&tmK, key0 + walk.tile(x0 + j + 1) * kKeys);
          }
        }
        if (!ok) {
          fail();
          for (int n = max(0, i - kSlots); n < i; ++n)  // copies in flight land before the block leaves
            mbar_wait_bounded(&full_bar[n % kSlots], static_cast<uint32_t>(n / kSlots) & 1u, nullptr, limit_ns / 16 + 1);
        }
      }
    } else if (warp == kSoftmaxWarps + 1) {
      // ------------------------------------------------ MMA issuer
      // The whole warp walks the loop, so that every operand is warp-uniform,
      // and one elected lane issues.
      constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kKeys), kIdescO = idesc_bf16_f32_bt(kRows, D);
      const uint32_t q_lo = desc_lo_k_sw128(smem_addr(sQ)), k_lo = desc_lo_k_sw128(smem_addr(sKV)),
                     v_lo = desc_lo_mn_sw128(smem_addr(sKV), kBox);
      bool ok = true;
      int i = 0;                   // next ring item
      uint32_t steps_a = 0, steps_b = 0;  // score tiles issued of A and B
      const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity & 1u, abort_flag, limit_ns));
      };
      const auto wait_slot = [&]() {
        const int s = i % kSlots;
        wait(&full_bar[s], static_cast<uint32_t>(i / kSlots));
        ++i;
        return s;
      };
      const auto scores = [&](int t, int slot, bool last) {  // S_t = Q_t K^T; by the elected lane
        const uint32_t qa = q_lo + t * (C::kTile / 16), ka = k_lo + slot * (C::kTile / 16);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint32_t off = ((k >> 2) * kBox + (k & 3) * 32) / 16;
          mma_bf16(tmem + t * kKeys, qa + off, ka + off, kIdescS, k != 0);
        }
        mma_commit(&s_bar[t]);
        if (last) mma_commit(&qempty_bar[t]);
      };
      Item item;
      for (int it = 0; take(it, item, ok); ++it) {
        const int count_a = count_of(item.q, 0), count_b = count_of(item.q, 1), most = max(count_a, count_b);
        done_with(it);
        wait(&qfull_bar[0], static_cast<uint32_t>(it));
        wait(&qfull_bar[1], static_cast<uint32_t>(it));
        int slot = most > 0 ? wait_slot() : 0;
        tc_fence_after();
        if (ok && elect_one()) {
          // a tile without keys hands its query rows back at once
          if (count_a > 0) scores(0, slot, count_a == 1); else mbar_arrive(&qempty_bar[0]);
          if (count_b > 0) scores(1, slot, count_b == 1); else mbar_arrive(&qempty_bar[1]);
          if (most > 0) mma_commit(&empty_bar[slot]);
        }
        __syncwarp();
        for (int j = 0; j < most && ok; ++j) {
          const int v_slot = wait_slot();
          const int k_slot = j + 1 < most ? wait_slot() : 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int count = t ? count_b : count_a;
            if (!ok || j >= count) continue;
            const uint32_t parity = (t ? steps_b : steps_a) + static_cast<uint32_t>(j);
            const uint32_t va = v_lo + v_slot * (C::kTile / 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // 64 keys as soon as their weights are there
              wait(&p_bar[2 * t + half], parity);
              if (!ok) continue;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 4 * half; k < 4 * half + 4; ++k)
                  mma_bf16_ta(tmem + kOCol + t * 128, tmem + t * kKeys + 8 * k, va + 2048 / 16 * k, kIdescO, (j | k) != 0);
                if (half == 1) {
                  // the next scores overwrite the weights just read: the tensor core works in order
                  if (j + 1 < count)
                    scores(t, k_slot, j + 2 == count);
                  else
                    mma_commit(&o_bar[t]);
                }
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) {
            mma_commit(&empty_bar[v_slot]);
            if (j + 1 < most) mma_commit(&empty_bar[k_slot]);
          }
          __syncwarp();
        }
        steps_a += static_cast<uint32_t>(count_a);
        steps_b += static_cast<uint32_t>(count_b);
      }
      if (!ok && elect_one()) {
        fail();
        mma_commit(drain_bar);  // MMAs in flight finish before TMEM is freed
        mbar_wait_bounded(drain_bar, 0, nullptr, limit_ns / 16 + 1);
      }
      __syncwarp();
    } else if (warp == kSoftmaxWarps + 2) {
      // ------------------------------------------------ query rows
      bool ok = true;
      int it = 0;
      Item item;
      for (; take(it, item, ok); ++it) {
        done_with(it);
        if (lane == 0) {
          // Rows of tokens past the item's (another sequence's, or zeros past
          // the last) and the rows past floor(128 / group) x group are no
          // one's: their scores go nowhere.
          for (int t = 0; t < 2 && ok; ++t) {
            if (!mbar_wait_bounded(&qempty_bar[t], (static_cast<uint32_t>(it) & 1u) ^ 1u, abort_flag, limit_ns)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&qfull_bar[t], static_cast<uint32_t>(C::kAtoms * tpt * a.group * 128));
#pragma unroll
            for (int c = 0; c < C::kAtoms; ++c)
              tma_load_3d(&tmQ, &qfull_bar[t], sQ + t * C::kTile + c * kBox, 64 * c, item.h * a.group,
                          item.q.row + t * tpt);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        fail();
        for (int t = 0; t < 2; ++t)  // copies in flight land before the block leaves
          for (int n = max(0, it - 1); n <= it; ++n)
            mbar_wait_bounded(&qfull_bar[t], static_cast<uint32_t>(n) & 1u, nullptr, limit_ns / 16 + 1);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // -------------------------------------------------- softmax
    const int w = warp >> 2;  // query tile
    const int row = threadIdx.x & (kRows - 1), tok = row / a.group;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + static_cast<uint32_t>(w * kKeys);
    const uint32_t t_o = tmem + lanes + kOCol + static_cast<uint32_t>(w * 128);
    uint8_t *const stage = sStage + warp * kStage;
    const bool cap = a.softcap > 0.0f;
    const float mul = cap ? a.scale / a.softcap : a.scale * kLog2e;
    const float cap2 = a.softcap * kLog2e;
    const bool plain = !cap && !a.slopes && a.scale >= 0.0f;  // a granule's largest score is its largest product
    bool ok = true;
    uint32_t steps = 0, outs = 0;  // score tiles and outputs of this query tile so far
    Item item;
    for (int it = 0; take(it, item, ok); ++it) {
      const int toks = toks_of(item.q, w), count = count_of(item.q, w);
      const int n = item.q.n, prefix = item.q.prefix, x0 = item.q.x0;
      const int slot = item.q.slot < 0 ? -1 : item.q.slot * a.c.heads + item.h;
      const TileWalk walk = walk_of(item.q);
      const int row0 = item.q.row + w * tpt, h0 = item.h * a.group;
      const int pos_min = item.q.pos + w * tpt, pos_max = pos_min + toks - 1;
      const int64_t krow = (static_cast<int64_t>(item.q.b) * a.c.heads + item.h) * x.len;
      done_with(it);
      const bool real = tok < toks;
      const int pos = real ? pos_min + tok : -1;
      const float slope = a.slopes && real ? __ldg(a.slopes + h0 + row - tok * a.group) * kLog2e : 0.0f;
      float m = -INFINITY, l = 0.0f;
      const float *ks = x.ks + krow / kGran, *vs = x.vs + krow / kGran;
      for (int j = 0; j < count; ++j) {
        const int key0 = walk.tile(x0 + j) * kKeys;
        float kc[8], vc[8];  // scales of the tile's granules
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 k4 = *reinterpret_cast<const float4 *>(ks + key0 / kGran + 4 * e);
          const float4 v4 = *reinterpret_cast<const float4 *>(vs + key0 / kGran + 4 * e);
          kc[4 * e] = k4.x, kc[4 * e + 1] = k4.y, kc[4 * e + 2] = k4.z, kc[4 * e + 3] = k4.w;
          vc[4 * e] = v4.x, vc[4 * e + 1] = v4.y, vc[4 * e + 2] = v4.z, vc[4 * e + 3] = v4.w;
        }
        bool whole = key0 + kKeys - 1 <= pos_min && (a.window == 0 || key0 > pos_max - a.window);
#pragma unroll
        for (int g = 0; g < 8; ++g) whole = whole && kc[g] != -1.0f;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&s_bar[w], (steps + static_cast<uint32_t>(j)) & 1u, abort_flag,
                                                       limit_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the row's scores, all of them in flight at once
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tmem_ld_32x32b_x32(t_s, s0);
        tmem_ld_32x32b_x32(t_s + 32, s1);
        tmem_ld_32x32b_x32(t_s + 64, s2);
        tmem_ld_32x32b_x32(t_s + 96, s3);
        tmem_ld_wait();
        float top = -INFINITY;
        if (whole && plain) {
          const auto largest = [&](const uint32_t(&s)[32], int c) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float v = __uint_as_float(s[16 * g]), u = __uint_as_float(s[16 * g + 1]);
#pragma unroll
              for (int e = 2; e < 16; e += 4) {
                v = max3(v, __uint_as_float(s[16 * g + e]), __uint_as_float(s[16 * g + e + 1]));
                if (e + 2 < 16) u = max3(u, __uint_as_float(s[16 * g + e + 2]), __uint_as_float(s[16 * g + e + 3]));
              }
              kc[2 * c + g] *= mul;
              top = fmaxf(top, fmaxf(v, u) * kc[2 * c + g]);
            }
          };
          largest(s0, 0);
          largest(s1, 1);
          largest(s2, 2);
          largest(s3, 3);
        } else {  // element by element
          const float far = slope * static_cast<float>(key0 - pos);
          // keys key0 + e of this row: e <= hi and e >= lo, or e < pre
          const int hi = pos < 0 ? -1 : min(pos, n - 1) - key0;
          const int lo = a.window > 0 ? pos - a.window + 1 - key0 : -key0;
          const int pre = pos < 0 ? 0 : min(prefix, n) - key0;
          // CAP: tanh cap; BIAS: distance bias; MASK: some row of the tile does
          // not see some key (CAP decides about the other two as it goes)
          const auto finish = [&](auto cap_c, auto bias_c, auto mask_c, uint32_t(&s)[32], int c) {
            constexpr bool CAP = decltype(cap_c)::value, BIAS = decltype(bias_c)::value, MASK = decltype(mask_c)::value;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float k1 = kc[2 * c + g], f = k1 * mul;
              const int e0 = 32 * c + 16 * g;
              float y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(s[16 * g + i]);
              if constexpr (CAP) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  y[i] = cap2 - __fdividef(2.0f * cap2, 1.0f + ex2(y[i] * (f * (2.0f * kLog2e))));
              }
              if constexpr (BIAS) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float b0 = fmaf(slope, static_cast<float>(e0 + i), far);
                  float b1 = fmaf(slope, static_cast<float>(e0 + i + 1), far);
                  axpy2(b0, b1, y[i], y[i + 1], CAP ? 1.0f : f);
                  y[i] = b0, y[i + 1] = b1;
                }
              } else if constexpr (!CAP) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) mul_f32x2(y[i], y[i + 1], f, y[i], y[i + 1]);
              }
              if constexpr (MASK) {
                // bits of the granule's keys that this row sees
                uint32_t seen = (bits_below(hi + 1 - e0) & ~bits_below(lo - e0)) | bits_below(pre - e0);
                if (k1 == -1.0f) seen = 0;
                // a page of which this row sees nothing may hold anything: its weights are 0 times 0
                if (seen == 0) vc[2 * c + g] = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = (seen >> i) & 1u ? y[i] : -INFINITY;
              }
              float v = y[0], u = y[1];
#pragma unroll
              for (int i = 2; i < 16; i += 4) {
                v = max3(v, y[i], y[i + 1]);
                if (i + 2 < 16) u = max3(u, y[i + 2], y[i + 3]);
              }
              top = max3(top, v, u);
#pragma unroll
              for (int i = 0; i < 16; ++i) s[16 * g + i] = __float_as_uint(y[i]);
              kc[2 * c + g] = 1.0f;
            }
          };
          const auto finish_row = [&](auto cap_c, auto bias_c, auto mask_c) {
            finish(cap_c, bias_c, mask_c, s0, 0);
            finish(cap_c, bias_c, mask_c, s1, 1);
            finish(cap_c, bias_c, mask_c, s2, 2);
            finish(cap_c, bias_c, mask_c, s3, 3);
          };
          if (cap)
            finish_row(Yes(), Yes(), Yes());
          else if (a.slopes && whole)
            finish_row(No(), Yes(), No());
          else if (a.slopes)
            finish_row(No(), Yes(), Yes());
          else
            finish_row(No(), No(), Yes());
        }
        const bool grow = top > m + kRescale || (m == -INFINITY && top > m);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float fr = grow ? ex2(m - top) : 1.0f;
          if (grow) m = top;
          l *= fr;
          if (j > 0) {  // O_w(j - 1) is complete, O_w(j) waits for this warp
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(t_o + 16 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fr);
              tmem_st_32x32b_x16(t_o + 16 * c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.0f : -m;
        float l0 = 0.0f, l1 = 0.0f, l2 = 0.0f, l3 = 0.0f;
        // 32 weights, packed by two; stage by stage over a granule, so that the
        // steps of 16 independent elements overlap
        uint32_t p[32];
        const auto weights = [&](const uint32_t(&s)[32], int c) {
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const int g = 2 * c + h2;
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(s[16 * h2 + e]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) fma2(y[e], y[e + 1], kc[g], ref);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = ex2(y[e]);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              add2(l0, l1, y[e], y[e + 1]);
              add2(l2, l3, y[e + 2], y[e + 3]);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) mul_f32x2(y[e], y[e + 1], vc[g], y[e], y[e + 1]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) p[16 * (c & 1) + 8 * h2 + (e >> 1)] = pack_bf16x2(y[e], y[e + 1]);
          }
        };
        const auto hand_over = [&](int half) {  // the weights of 64 keys, over scores that have been read
          tmem_st_32x32b_x32(t_s + 32 * half, p);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_bar[2 * w + half]);
        };
        weights(s0, 0);
        weights(s1, 1);
        hand_over(0);
        weights(s2, 2);
        weights(s3, 3);
        hand_over(1);
        l += (l0 + l1) + (l2 + l3);
      }
      if (ok && count > 0)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&o_bar[w], outs & 1u, abort_flag, limit_ns));
      if (!ok) break;
      tc_fence_after();
      if (slot >= 0) {  // a part: its sums, maximum and sum of weights
        float *const part = x.parts + static_cast<int64_t>(slot) * part_floats<D>();
        *reinterpret_cast<float2 *>(part + 2 * kRows * D + (w * kRows + row) * 2) = make_float2(count > 0 ? m : -INFINITY, l);
        if (count > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(t_o + 16 * c, o);
            tmem_ld_wait();
            // dims by 4, rows side by side: a warp's stores are runs of 512 bytes
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4 *>(part + (static_cast<int64_t>(w * (D / 4) + 4 * c + e) * kRows + row) * 4) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        tc_fence_before();
        steps += static_cast<uint32_t>(count);
        outs += count > 0 ? 1u : 0u;
        continue;
      }
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const float r_out = a.r_out ? __ldg(a.r_out) : 0.0f;
      const int z_out = a.r_out ? __ldg(a.z_out) : 0;
      // 64 dims of the warp's 32 rows at a time through its staging (swizzled as
      // TMA would). bf16 rows of whole tokens that are all the item's leave as
      // one tensor store, which the warp does not wait for; others by
      // neighbouring lanes.
      const bool tensor_store = !a.r_out && 32 % a.group == 0 && (warp & 3) * 32 + 32 <= toks * a.group;
#pragma unroll
      for (int part = 0; part < C::kAtoms; ++part) {
        constexpr int kMost = 64;
        const int dims = D - kMost * part < kMost ? D - kMost * part : kMost;
        uint32_t o4[kMost / 16][16];
#pragma unroll
        for (int c = 0; c < kMost / 16; ++c) {
          if (16 * c >= dims) continue;
          if (count > 0) {
            tmem_ld_32x32b_x16(t_o + kMost * part + 16 * c, o4[c]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o4[c][e] = 0;
          }
        }
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kMost / 16; ++c) {
          if (16 * c >= dims) continue;
          const uint32_t(&o)[16] = o4[c];
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          uint8_t *const at = stage + lane * kStageRow;
          if (c == 0) {  // the staging's last store has read it
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
          *reinterpret_cast<uint4 *>(at + (((2 * c) ^ (lane & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4 *>(at + (((2 * c + 1) ^ (lane & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        if (tensor_store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmOut, stage, kMost * part, h0, row0 + (warp & 3) * (32 / a.group));
            bulk_commit_group();
          }
          continue;
        }
        __syncwarp();
        const int chunks = dims / 8;
#pragma unroll
        for (int k = 0; k < kMost / 8; ++k) {
          if (k >= chunks) continue;
          const int i = k * 32 + lane, r1 = i / chunks, c = i - r1 * chunks, r = (warp & 3) * 32 + r1;
          const int r_tok = r / a.group;
          if (r_tok >= toks) continue;
          const uint4 v = *reinterpret_cast<const uint4 *>(stage + r1 * kStageRow + ((c ^ (r1 & 7)) << 4));
          const int64_t elem =
              (static_cast<int64_t>(row0 + r_tok) * a.q_heads + h0 + r - r_tok * a.group) * D + kMost * part + 8 * c;
          if (!a.r_out)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + elem) = v;
          else
            *reinterpret_cast<uint2 *>(static_cast<int8_t *>(a.out) + elem) = quant8_asym_sat(v, r_out, z_out);
        }
        __syncwarp();
      }
      tc_fence_before();  // O has been read before this warp's next weights let it be overwritten
      steps += static_cast<uint32_t>(count);
      outs += count > 0 ? 1u : 0u;
    }
    if (lane == 0) bulk_wait_all();  // every store of this warp has completed before the block leaves
    __syncwarp();
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  __syncwarp();  // lanes of the producer and MMA warps reconverge before the CTA barrier
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of split blocks, in their order: a warp per 4 dims of 32
// neighbouring rows.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv_prefill_join_kernel(const __grid_constant__ KvAttnArgs a,
                                                                       const __grid_constant__ Expanded x) {
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int tpt = kRows / a.group, lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(x.counters[2]) * a.c.heads * (2 * kRows / 32) * (D / 4);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kJoinThreads / 32);
  for (int64_t u = blockIdx.x * static_cast<int64_t>(kJoinThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int d4 = static_cast<int>(u % (D / 4));
    const int64_t v = u / (D / 4);
    const int rows32 = static_cast<int>(v % (2 * kRows / 32)), h = static_cast<int>(v / (2 * kRows / 32) % a.c.heads);
    const QueryBlock &q = x.split[v / (2 * kRows / 32) / a.c.heads];
    const int w = rows32 / (kRows / 32), row = (rows32 % (kRows / 32)) * 32 + lane;  // tile and row in it
    const int tok = row / a.group;
    if (tok >= tpt || w * tpt + tok >= q.toks) continue;
    float m = -INFINITY, l = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < q.parts; ++i) {
      const float *part = x.parts + (static_cast<int64_t>(q.slot + i) * a.c.heads + h) * part_floats<D>();
      const float2 ml = *reinterpret_cast<const float2 *>(part + 2 * kRows * D + (w * kRows + row) * 2);
      if (ml.x == -INFINITY) continue;
      const float4 o = *reinterpret_cast<const float4 *>(part + (static_cast<int64_t>(w * (D / 4) + d4) * kRows + row) * 4);
      const float m2 = fmaxf(m, ml.x), f0 = ex2(m - m2), f1 = ex2(ml.x - m2);
      m = m2;
      l = l * f0 + ml.y * f1;
      y[0] = y[0] * f0 + o.x * f1, y[1] = y[1] * f0 + o.y * f1, y[2] = y[2] * f0 + o.z * f1, y[3] = y[3] * f0 + o.w * f1;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
    const int hq = h * a.group + row - tok * a.group;
    store_out4(a, (static_cast<int64_t>(q.row + w * tpt + tok) * a.q_heads + hq) * D + 4 * d4, y);
  }
}

int64_t query_block_slots(const KvAttnArgs &a) { return a.s.tokens / (2 * (kRows / a.group)) + a.s.batch; }

// Whether blocks may be split: where there are not many more items than SMs,
// and contexts longer than what a part has at least. Split : whole, us a call, 8
// kv heads of 4: 256 tokens behind 16384 keys 134 : 253, with eight prompts of
// 256 beside them 151 : 276, 512 behind 4096 73 : 81. Where nothing turns out
// to be worth splitting, the sum over all blocks and the join's launch cost
// 1 to 6: one prompt of 2048 51 : 48, eight of 512 in tables of 2048 54 : 48.
bool may_split(const KvAttnArgs &a, int num_sms) {
  return query_block_slots(a) * a.c.heads <= 4 * num_sms && expanded_len(a.s.max_kv) / kKeys > kMinShare + kMinOver;
}

int64_t part_bytes(const KvAttnArgs &a) { return int64_t(2) * kRows * (a.c.d + 2) * sizeof(float); }

Expanded expanded_of(const KvAttnArgs &a, void *workspace, int num_sms) {
  Expanded x;
  x.len = expanded_len(a.s.max_kv);
  x.slots = static_cast<int32_t>(query_block_slots(a));
  x.sms = num_sms;
  x.most_parts = may_split(a, num_sms) ? 2 * num_sms : 0;  // over all heads
  const int64_t keys = static_cast<int64_t>(a.s.batch) * a.c.heads * x.len;
  const int64_t pitch = a.c.d > 64 ? 128 : 64;
  x.k = static_cast<uint16_t *>(workspace);
  x.v = x.k + keys * pitch;
  x.ks = reinterpret_cast<float *>(x.v + keys * pitch);
  x.vs = x.ks + keys / kGran;
  x.parts = x.vs + keys / kGran;
  x.blocks = reinterpret_cast<QueryBlock *>(reinterpret_cast<char *>(x.parts) + x.most_parts * part_bytes(a));
  x.split = x.blocks + x.slots + x.most_parts;
  x.counters = reinterpret_cast<int32_t *>(x.split + (x.most_parts ? x.slots : 0));
  return x;
}

template <int D>
cudaError_t launch_t(const KvAttnArgs &a, void *workspace, int num_sms, cudaStream_t s) {
  using C = PCfg<D>;
  const Expanded x = expanded_of(a, workspace, num_sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  alignas(64) CUtensorMap tmQ, tmK = {}, tmV = {}, tmOut = {};  // K and V are not used where no sequence has a key
  // a stride of an axis of one element is never used, but must be one
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  if (!encode_tmap_3d_bf16(&tmQ, a.q.p, D, a.q_heads, static_cast<uint64_t>(a.s.tokens),
                           a.q_heads > 1 ? static_cast<uint64_t>(a.q.head_stride) * 2 : row,
                           a.s.tokens > 1 ? static_cast<uint64_t>(a.q.token_stride) * 2 : row, 64,
                           static_cast<uint32_t>(a.group), static_cast<uint32_t>(kRows / a.group)))
    return cudaErrorInvalidValue;
  if (!a.r_out && 32 % a.group == 0 &&
      !encode_tmap_3d_bf16(&tmOut, a.out, D, a.q_heads, static_cast<uint64_t>(a.s.tokens), row, row * a.q_heads, 64,
                           static_cast<uint32_t>(a.group), static_cast<uint32_t>(32 / a.group)))
    return cudaErrorInvalidValue;
  const uint64_t rows = static_cast<uint64_t>(a.s.batch) * a.c.heads * x.len;
  if (rows > 0 && (!encode_tmap_2d(&tmK, x.k, TmapType::kBF16, C::kPitch, rows, C::kPitch * 2, 64, kKeys, true) ||
                   !encode_tmap_2d(&tmV, x.v, TmapType::kBF16, C::kPitch, rows, C::kPitch * 2, 64, kKeys, true)))
    return cudaErrorInvalidValue;
  cfg.gridDim = dim3(static_cast<unsigned>(1 + x.len / kExpandKeys), a.c.heads, a.s.batch);
  cfg.blockDim = dim3(kExpandThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_expand_kernel<D>, a, x);
  if (e != cudaSuccess) return e;
  e = ensure_kernel_smem<kv_prefill_kernel<D>>(static_cast<int>(C::kSmem), false);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(x.slots + x.most_parts) * a.c.heads;
  cfg.gridDim = dim3(static_cast<unsigned>(items < num_sms ? items : num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<D>, tmQ, tmK, tmV, tmOut, a, x, kWaitLimitNs);
  if (e != cudaSuccess || x.most_parts == 0) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms) * 4);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_prefill_join_kernel<D>, a, x);
}

}  // namespace

bool kv_prefill_fits(const KvAttnArgs &a) {
  // rows of the expanded matrices are int32 tensor-map coordinates, items an int32 count
  const int64_t rows = static_cast<int64_t>(a.s.batch) * a.c.heads * expanded_len(a.s.max_kv);
  return rows <= INT32_MAX && query_block_slots(a) * a.c.heads <= INT32_MAX / 2;
}

size_t kv_prefill_workspace_bytes(const KvAttnArgs &a, int num_sms) {
  const Expanded x = expanded_of(a, nullptr, num_sms);
  return reinterpret_cast<uintptr_t>(x.counters) + 16;
}

cudaError_t launch_kv_prefill(const KvAttnArgs &a, void *workspace, int num_sms, cudaStream_t s) {
  switch (a.c.d) {
    case 64: return launch_t<64>(a, workspace, num_sms, s);
    case 96: return launch_t<96>(a, workspace, num_sms, s);
    case 128: return launch_t<128>(a, workspace, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace w8a8
