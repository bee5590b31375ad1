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
// one operand in shared memory as bf16, which the int8 codes are not until a
// register has held them. Codes become bf16 in registers, exactly:
// bf16(128 + (q & 127)) - bf16(128 or 256, by q's sign), both bit patterns
// made by masking a byte into 0x43xx.
//   Both contractions may run over their axis in any order as long as both
// sides use the same one, so a lane reads its codes of K as 16 contiguous
// bytes of one key and those of V as the same dims of four keys (pairs of
// keys are interleaved by byte permutes), and P goes from the accumulator
// layout of the first product to the operand layout of the second by an 8x8
// transpose (movmatrix). P times the page's v scale enters as bf16 high part
// plus bf16 low part.
//   Loads are 16-byte cp.async into a ring of each warp's own, so a warp
// waits for nobody; the stages are swizzled so that both reads are free of
// bank conflicts (D = 128).
#include "kv_common.cuh"

namespace w8a8 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;    // keys of a warp's tile
constexpr int kStages = 3;
constexpr int kPagesAhead = 16;  // tiles whose pages and scales a warp holds, two granules each, one per lane

template <int D>
struct Cfg {
  static constexpr int kPitch = D == 64 ? 64 : 128;        // bytes of a key's row in a stage
  static constexpr int kStage = 2 * kTile * kPitch;        // K rows, then V rows
  static constexpr int kChunks = D / 16;
  static constexpr size_t kSmem = static_cast<size_t>(kWarps) * kStages * kStage;
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

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// Partial results of a split: [sequence][kv head][row block][split] x (8 NT
// rows x D sums, then 8 NT rows x (maximum, sum)).
template <int D, int NT>
constexpr int partial_floats() { return 8 * NT * (D + 2); }

// Block (split, kv head and row block, sequence).
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    kv_decode_kernel(const __grid_constant__ KvAttnArgs a, float *__restrict__ partial) {
  using C = Cfg<D>;
  constexpr int KS = D / 16;   // contraction steps of the scores
  constexpr int MT = D / 16;   // 16-dim tiles of the output
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int b = blockIdx.z, h = blockIdx.y % a.c.heads, rb = blockIdx.y / a.c.heads;
  const int split = blockIdx.x, splits = gridDim.x;
  const KvSeq seq = load_seq(a.s, b, a.s.max_kv, a.status);
  const int rows = seq.q * a.group;  // query rows of this kv head
  const int row0 = rb * ROWS;
  if (row0 >= rows) return;
  const int32_t prefix = a.prefix ? __ldg(a.prefix + b) : 0;
  const TileWalk walk = tile_walk(kTile, prefix, seq.n, max(seq.pos0(), 0), seq.n, a.window);
  const int per = (walk.count + splits - 1) / splits;
  const int x0 = min(walk.count, split * per), x1 = min(walk.count, x0 + per);
  const int32_t *table_row = a.s.table + b * a.s.table_ld;
  uint8_t *ring = smem + warp * (kStages * C::kStage);

  // this lane's query rows as the narrow operand of the scores, and as columns of S^T
  uint32_t qf[NT][KS][2];
  float slope[NT][2];
  int pos[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + g;
    const bool ok = r < rows;
    const int i = r / a.group, hq = h * a.group + (r - i * a.group);
    const uint16_t *q = a.q.p + (seq.row0 + i) * a.q.token_stride + hq * a.q.head_stride;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint2 v = make_uint2(0, 0);
      if (ok) v = __ldg(reinterpret_cast<const uint2 *>(q + k_dim<D>(t, k)));
      qf[nt][k][0] = v.x;
      qf[nt][k][1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rc = row0 + nt * 8 + 2 * t + e;
      const int ic = rc / a.group;
      pos[nt][e] = rc < rows ? seq.pos0() + ic : -1;
      slope[nt][e] = a.slopes && rc < rows ? __ldg(a.slopes + h * a.group + (rc - ic * a.group)) * kLog2e : 0.0f;
    }
  }
  // positions of the block's first and last row (no row is hidden from keys at or before pos_min within the window)
  const int pos_min = seq.pos0() + row0 / a.group;
  const int pos_max = seq.pos0() + (min(row0 + ROWS, rows) - 1) / a.group;
  const bool cap = a.softcap > 0.0f;
  // s = S * scale * log2(e), or with a cap c: z = S * scale / c, s = c log2(e) tanh(z)
  const float mul = cap ? a.scale / a.softcap : a.scale * kLog2e;
  const float cap2 = a.softcap * kLog2e;

  float acc[MT][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) m[nt][e] = -INFINITY, l[nt][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.0f;
  }

  // pages and scales of the warp's next kPagesAhead tiles: lane 2 y + z holds granule z of tile y
  int page_l = -1;
  float ks_l = 0.0f, vs_l = 0.0f;
  const auto fetch_pages = [&](int xw) {
    page_l = -1;
    ks_l = vs_l = 0.0f;
    const int x = xw + (lane >> 1) * kWarps;
    if (x >= x1) return;
    const int key = walk.tile(x) * kTile + (lane & 1) * kGran;
    if (key >= seq.n) return;
    page_l = load_page(table_row, key >> a.c.page_shift, a.c.pages, a.status);
    if (page_l < 0) return;
    const int64_t at = static_cast<int64_t>(page_l) * a.c.heads + h;
    ks_l = __ldg(a.c.ks + at);
    vs_l = __ldg(a.c.vs + at);
  };
  const auto load_tile = [&](int x, int y, int stage) {  // tile x, the y-th of the fetched ones
    const uint32_t dst = smem_addr(ring + stage * C::kStage);
    const int key0 = walk.tile(x) * kTile;
    int64_t base[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int p = __shfl_sync(0xFFFFFFFFu, page_l, 2 * y + z);
      const int64_t blk = static_cast<int64_t>(p) * a.c.heads + h;
      base[z] = p < 0 ? -1 : ((blk << a.c.page_shift) + ((key0 + z * kGran) & (a.c.page - 1))) * D;
    }
#pragma unroll
    for (int i = 0; i < C::kChunks; ++i) {
      const int idx = i * 32 + lane, r = idx / C::kChunks, c = idx % C::kChunks;
      const int64_t bz = r >= kGran ? base[1] : base[0];
      if (bz >= 0) {
        const int64_t src = bz + (r & (kGran - 1)) * D + 16 * c;
        cp_async16(dst + stage_off<D>(r, c), a.c.k + src);
        cp_async16(dst + kTile * C::kPitch + stage_off<D>(r, c), a.c.v + src);
      }
    }
  };

  // The warp's tiles are x0 + warp, x0 + warp + kWarps, ... The pages of tile
  // number y (from 0) are fetched kPagesAhead at a time; loads run kStages - 1
  // tiles ahead, so the fetched window is refilled when its last tile is
  // loaded, and the scales of a loaded tile travel with it in registers.
  float ksc[kStages][2], vsc[kStages][2];
  int pgc[kStages][2];
  int y_load = 0;  // next tile to load, as a count of this warp's tiles
  const int ny = x1 - x0 > warp ? (x1 - x0 - warp + kWarps - 1) / kWarps : 0;
  const auto stage_tile = [&](int slot) {
    if (y_load < ny) {
      const int y = y_load % kPagesAhead;
      if (y == 0) fetch_pages(x0 + warp + y_load * kWarps);
      load_tile(x0 + warp + y_load * kWarps, y, slot);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        pgc[slot][z] = __shfl_sync(0xFFFFFFFFu, page_l, 2 * y + z);
        ksc[slot][z] = __shfl_sync(0xFFFFFFFFu, ks_l, 2 * y + z);
        vsc[slot][z] = __shfl_sync(0xFFFFFFFFu, vs_l, 2 * y + z);
      }
      ++y_load;
    }
    cp_async_commit();
  };

  const auto compute_tile = [&](int x, int slot) {
    const uint8_t *ks = ring + slot * C::kStage, *vs = ks + kTile * C::kPitch;
    const int key0 = walk.tile(x) * kTile;
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t w0[KS], w1[KS];
      load_k_words<D>(ks, mt * kGran + g, t, w0);
      load_k_words<D>(ks, mt * kGran + g + 8, t, w1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a0, a1, a2, a3;
        codes_to_bf16(w0[k], a0, a2);
        codes_to_bf16(w1[k], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(s[mt][nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
      }
    }
    // scores, in units of log2; element e of s[mt][nt]: key mt * 16 + g + 8 (e >> 1), row 2 t + (e & 1)
    const bool whole = key0 + kTile - 1 <= pos_min && (a.window == 0 || key0 > pos_max - a.window) &&
                       pgc[slot][0] >= 0 && pgc[slot][1] >= 0;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const float f = ksc[slot][mt] * mul;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[mt][nt][e] * f;
          if (cap) v = cap2 - __fdividef(2.0f * cap2, 1.0f + ex2(v * (2.0f * kLog2e)));
          s[mt][nt][e] = v;
        }
      }
    }
    if (a.slopes || !whole) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + mt * kGran + g + 8 * (e >> 1), p = pos[nt][e & 1];
            float v = s[mt][nt][e] + slope[nt][e & 1] * static_cast<float>(j - p);
            if (!whole) {
              const bool seen = pgc[slot][mt] >= 0 && j < seq.n && p >= 0 &&
                                ((j <= p && (a.window == 0 || p - j < a.window)) || j < prefix);
              v = seen ? v : -INFINITY;
            }
            s[mt][nt][e] = v;
          }
    }
    bool grew = false;
    float al[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        al[nt][e] = 1.0f;
        if (v > m[nt][e]) {
          al[nt][e] = ex2(m[nt][e] - v);
          m[nt][e] = v;
          grew = true;
        }
      }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] *= al[nt][0];
        l[nt][1] *= al[nt][1];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] *= al[nt][e & 1];
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[nt][e & 1] == -INFINITY ? 0.0f : m[nt][e & 1];  // a row that has seen no key yet
          p[e] = ex2(s[mt][nt][e] - ref);
          l[nt][e & 1] += p[e];
          // (not 0 times the scale of a page that no row sees, which may be anything)
          p[e] = whole || s[mt][nt][e] != -INFINITY ? p[e] * vsc[slot][mt] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t hi = pack_bf16x2(p[2 * k], p[2 * k + 1]);
          const uint32_t lo = pack_bf16x2(p[2 * k] - bf16_lo(hi), p[2 * k + 1] - bf16_hi(hi));
          ph[nt][k] = transpose8x8(hi);
          pl[nt][k] = transpose8x8(lo);
        }
      }
      uint32_t v0[D / 32], v1[D / 32], v2[D / 32], v3[D / 32];
      load_v_words<D>(vs, mt * kGran + 2 * t, g, v0);
      load_v_words<D>(vs, mt * kGran + 2 * t + 1, g, v1);
      load_v_words<D>(vs, mt * kGran + 2 * t + 8, g, v2);
      load_v_words<D>(vs, mt * kGran + 2 * t + 9, g, v3);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          codes_to_bf16(__byte_perm(v0[w], v1[w], sel), a0, a1);
          codes_to_bf16(__byte_perm(v2[w], v3[w], sel), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(acc[2 * w + half][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
            mma_bf16_16816(acc[2 * w + half][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
  };

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) stage_tile(i);
  for (int y = 0; y < ny; y += kStages) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (y + i < ny) {
        cp_async_wait<kStages - 2>();
        __syncwarp();  // every lane's copies of this tile have landed, and all have read the slot loaded next
        stage_tile((i + kStages - 1) % kStages);
        compute_tile(x0 + warp + (y + i) * kWarps, i);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // join the warps: sums of each row in shared memory, scaled to the row's maximum
  float *s_acc = reinterpret_cast<float *>(smem);               // [warp][row][D]
  float *s_ml = s_acc + kWarps * ROWS * D;                      // [warp][row](maximum, sum)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      const int r = nt * 8 + 2 * t + e;
      if (g == 0) {
        s_ml[(warp * ROWS + r) * 2] = m[nt][e];
        s_ml[(warp * ROWS + r) * 2 + 1] = v;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<float2 *>(s_acc + (warp * ROWS + r) * D + v_dim<D>(g, i)) =
            make_float2(acc[i][nt][e], acc[i][nt][e + 2]);
    }
  __syncthreads();
  const int row_blocks = gridDim.y / a.c.heads;
  float *out_p = partial +
                 (((static_cast<int64_t>(b) * a.c.heads + h) * row_blocks + rb) * splits + split) * partial_floats<D, NT>();
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    if (row0 + r >= rows) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[(w * ROWS + r) * 2]);
    float ll = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mm != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_ml[(w * ROWS + r) * 2] - mm);
        ll += f * s_ml[(w * ROWS + r) * 2 + 1];
        const float4 v = *reinterpret_cast<const float4 *>(s_acc + (w * ROWS + r) * D + d);
        y[0] += f * v.x, y[1] += f * v.y, y[2] += f * v.z, y[3] += f * v.w;
      }
    }
    if (splits == 1) {
      const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= inv;
      const int qi = (row0 + r) / a.group, hq = h * a.group + (row0 + r - qi * a.group);
      store_out4(a, (static_cast<int64_t>(seq.row0 + qi) * a.q_heads + hq) * D + d, y);
    } else {
      *reinterpret_cast<float4 *>(out_p + r * D + d) = make_float4(y[0], y[1], y[2], y[3]);
      if (d == 0) *reinterpret_cast<float2 *>(out_p + ROWS * D + 2 * r) = make_float2(mm, ll);
    }
  }
}

// Joins the splits: one warp per (row of a kv head, sequence).
template <int D, int NT>
__global__ void __launch_bounds__(128) kv_join_kernel(const __grid_constant__ KvAttnArgs a,
                                                      const float *__restrict__ partial, int splits, int row_blocks) {
  constexpr int ROWS = 8 * NT;
  pdl_launch_dependents();
  pdl_wait_prerequisite();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const KvSeq seq = load_seq(a.s, b, a.s.max_kv, nullptr);
  const int64_t id = blockIdx.x * 4 + (threadIdx.x >> 5);  // kv head, row
  const int h = static_cast<int>(id / (row_blocks * ROWS)), row = static_cast<int>(id % (row_blocks * ROWS));
  if (h >= a.c.heads || row >= seq.q * a.group) return;
  const int rb = row / ROWS, r = row % ROWS;
  const float *p = partial + ((static_cast<int64_t>(b) * a.c.heads + h) * row_blocks + rb) * splits * partial_floats<D, NT>();
  float mm = -INFINITY;
  for (int s = 0; s < splits; ++s) mm = fmaxf(mm, p[s * partial_floats<D, NT>() + ROWS * D + 2 * r]);
  float ll = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (mm != -INFINITY) {
    for (int s = 0; s < splits; ++s) {
      const float *ps = p + s * partial_floats<D, NT>();
      const float2 ml = *reinterpret_cast<const float2 *>(ps + ROWS * D + 2 * r);
      const float f = ex2(ml.x - mm);
      ll += f * ml.y;
      if (4 * lane < D) {
        const float4 v = *reinterpret_cast<const float4 *>(ps + r * D + 4 * lane);
        y[0] += f * v.x, y[1] += f * v.y, y[2] += f * v.z, y[3] += f * v.w;
      }
    }
  }
  if (4 * lane >= D) return;
  const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  const int qi = row / a.group, hq = h * a.group + (row - qi * a.group);
  store_out4(a, (static_cast<int64_t>(seq.row0 + qi) * a.q_heads + hq) * D + 4 * lane, y);
}

struct DecodePlan {
  int nt, row_blocks, splits;
  size_t bytes;
};

DecodePlan decode_plan(const KvAttnArgs &a, int num_sms) {
  DecodePlan p;
  const int64_t rows = static_cast<int64_t>(a.s.max_q) * a.group;
  p.nt = rows <= 8 ? 1 : 2;
  p.row_blocks = static_cast<int>((rows + 8 * p.nt - 1) / (8 * p.nt));
  const int64_t blocks = static_cast<int64_t>(a.s.batch) * a.c.heads * p.row_blocks;
  const int64_t most = (a.s.max_kv + kTile * kWarps - 1) / (kTile * kWarps);  // a tile for each warp of a split
  int64_t want = (num_sms + blocks - 1) / blocks;
  if (want > most) want = most;
  p.splits = static_cast<int>(want < 1 ? 1 : want);
  p.bytes = p.splits == 1 ? 0 : static_cast<size_t>(blocks) * p.splits * 8 * p.nt * (a.c.d + 2) * sizeof(float);
  return p;
}

template <int D, int NT>
cudaError_t launch_t(const KvAttnArgs &a, const DecodePlan &p, float *partial, cudaStream_t s) {
  constexpr size_t kJoin = static_cast<size_t>(kWarps) * 8 * NT * (D + 2) * sizeof(float);
  constexpr size_t kSmem = Cfg<D>::kSmem > kJoin ? Cfg<D>::kSmem : kJoin;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  cudaError_t e = ensure_kernel_smem<kv_decode_kernel<D, NT>>(static_cast<int>(kSmem), true);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.splits, a.c.heads * p.row_blocks, a.s.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<D, NT>, a, partial);
  if (e != cudaSuccess || p.splits == 1) return e;
  cfg.gridDim = dim3((a.c.heads * p.row_blocks * 8 * NT + 3) / 4, a.s.batch);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT>, a, static_cast<const float *>(partial), p.splits, p.row_blocks);
}

template <int D>
cudaError_t launch_d(const KvAttnArgs &a, const DecodePlan &p, float *partial, cudaStream_t s) {
  return p.nt == 1 ? launch_t<D, 1>(a, p, partial, s) : launch_t<D, 2>(a, p, partial, s);
}

}  // namespace

size_t kv_decode_workspace_bytes(const KvAttnArgs &a, int num_sms) { return decode_plan(a, num_sms).bytes; }

cudaError_t launch_kv_decode(const KvAttnArgs &a, void *workspace, int num_sms, cudaStream_t s) {
  const DecodePlan p = decode_plan(a, num_sms);
  float *partial = static_cast<float *>(workspace);
  switch (a.c.d) {
    case 64: return launch_d<64>(a, p, partial, s);
    case 96: return launch_d<96>(a, p, partial, s);
    case 128: return launch_d<128>(a, p, partial, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace w8a8
