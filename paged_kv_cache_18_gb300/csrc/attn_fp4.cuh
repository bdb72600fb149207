// attn_fp4.cuh -- what the two tensor-core kernels over the block-scaled 4-bit
// cache share (attn_fp4_warp.cu: a warp is a worker; attn_fp4_cta.cu: a CTA is):
// shared-memory loads, the f16 MMA, and the walk over the balanced partition.
#pragma once

#include <type_traits>

#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
constexpr int kWarps = 4;  // warps of a CTA
// Weights enter the MMAs in f16, against a reference per column that is raised
// when one exceeds 2^kSlack, to where the largest weight seen is 2^kHead: above 1,
// so that the weights of a long flat tail keep their bits (f16 holds 2^-14 of the
// largest at 11 bits, and drops what is below 2^-24 - kHead of it), and far enough
// below the slack that raising stays rare.
constexpr float kSlack = 14.f, kHeaviest = 16384.f, kHead = 6.f;
constexpr float kNothing = -3e38f;  // reference of a column that has seen no row: finite,
                                    // so that -inf scores still weigh 0 against it

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t perm(uint32_t a, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(d) : "r"(a), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t prmt2(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Key (row of the block) of MMA row g; row g + 8 is the key two after it.
__device__ __forceinline__ int key_of(int g) { return 4 * (g >> 1) + (g & 1); }

// d = a * b: the first product of a chain.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Scores of UB blocks that lie one after another (key tile, value tile) from
// shared address `blk`: S^T[16 keys x 8 NT] = K Q^T of each; `q(ks, nt, part, b0, b1)`
// gives the Q^T fragment of a k-step and tile.  Queries in PARTS f16 parts
// (split_row): the products with the small part have a sum of their own, so that
// the large one sees as few roundings as with one part.
// Lane (g, c) reads 32 dims of each panel of its two keys; k-step (panel, word w,
// half e) holds dims  panel + 8 WP c + 8 w + 4 e + {0, 1 | 2, 3}.
template <int D> struct Lanes {
  static constexpr int WP = Tile<D>::kPanel / 32;  // words (8 dims) of a lane in a panel
  static constexpr int KSP = 2 * WP;               // k-steps of a panel
};
template <int D, int NT, int UB, int PARTS = 1, typename Q>
__device__ __forceinline__ void block_scores(float (&sc)[UB][NT][4], uint32_t blk, int g, int c,
                                             const Q &q) {
  using TL = Tile<D>;
  constexpr int WP = Lanes<D>::WP, KSP = Lanes<D>::KSP;
  const int kk = key_of(g);
  float low[PARTS > 1 ? UB : 1][PARTS > 1 ? NT : 1][4];
#pragma unroll
  for (int pn = 0; pn < TL::kPanels; ++pn) {
    uint32_t w0[UB][WP], w1[UB][WP], s0[UB][2], s1[UB][2];
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      const uint32_t tile = blk + u * 2 * TL::kBytes;
      const uint32_t at = tile + pn * (kBlockSize * TL::kPanel / 2) + kk * (TL::kPanel / 2) +
                          c * (4 * WP);
      const uint32_t sat = tile + TL::kCodeBytes + kk * TL::kScales + c * (WP / 2) + pn * 8;
      if constexpr (WP == 4) {
        const uint4 x = lds128(at), y = lds128(at + TL::kPanel);
        w0[u][0] = x.x; w0[u][1] = x.y; w0[u][2] = x.z; w0[u][3] = x.w;
        w1[u][0] = y.x; w1[u][1] = y.y; w1[u][2] = y.z; w1[u][3] = y.w;
        const uint32_t a = e4m3x2_to_f16(lds16(sat));
        const uint32_t b = e4m3x2_to_f16(lds16(sat + 2 * TL::kScales));
        s0[u][0] = perm(a, 0x1010); s0[u][1] = perm(a, 0x3232);
        s1[u][0] = perm(b, 0x1010); s1[u][1] = perm(b, 0x3232);
      } else {
        const uint2 x = lds64(at), y = lds64(at + TL::kPanel);
        w0[u][0] = x.x; w0[u][1] = x.y;
        w1[u][0] = y.x; w1[u][1] = y.y;
        s0[u][0] = s0[u][1] = perm(e4m3x2_to_f16(lds8(sat)), 0x1010);
        s1[u][0] = s1[u][1] = perm(e4m3x2_to_f16(lds8(sat + 2 * TL::kScales)), 0x1010);
      }
    }
#pragma unroll
    for (int w = 0; w < WP; ++w) {
      uint32_t h0[UB][4], h1[UB][4];
#pragma unroll
      for (int u = 0; u < UB; ++u) {
        e2m1x8_to_f16(w0[u][w], h0[u]);
        e2m1x8_to_f16(w1[u][w], h1[u]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ks = pn * KSP + w * 2 + e;
        uint32_t a[UB][4];
#pragma unroll
        for (int u = 0; u < UB; ++u) {
          a[u][0] = mul2(h0[u][2 * e], s0[u][w >> 1]);
          a[u][1] = mul2(h1[u][2 * e], s1[u][w >> 1]);
          a[u][2] = mul2(h0[u][2 * e + 1], s0[u][w >> 1]);
          a[u][3] = mul2(h1[u][2 * e + 1], s1[u][w >> 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b0, b1;
          q(ks, nt, 0, b0, b1);
#pragma unroll
          for (int u = 0; u < UB; ++u) {
            if (ks == 0) mma_first(sc[u][nt], a[u], b0, b1);
            else Mma<__half>::run(sc[u][nt], a[u], b0, b1);
          }
          if constexpr (PARTS > 1) {
#pragma unroll
            for (int part = PARTS - 1; part > 0; --part) {
              q(ks, nt, part, b0, b1);
#pragma unroll
              for (int u = 0; u < UB; ++u) {
                if (ks == 0 && part == PARTS - 1) mma_first(low[u][nt], a[u], b0, b1);
                else Mma<__half>::run(low[u][nt], a[u], b0, b1);
              }
            }
          }
        }
      }
    }
  }
  if constexpr (PARTS > 1)
#pragma unroll
    for (int u = 0; u < UB; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][nt][e] += low[u][nt][e];
}

// Make the value scales of rows nv .. 15 of a block zero (tile: its key tile,
// the value tile follows): rows that are not there add nothing then, whatever
// their bytes are, their codes being finite.  Warp-collective; the caller
// fences before the next copy into the stage.
template <int D>
__device__ __forceinline__ void clear_value_scales(uint32_t tile, int nv, int lane) {
  using TL = Tile<D>;
  for (int w = lane; w < D / 4; w += 32) {
    const int keep = nv - 4 * (w & 3);  // of the four rows of this word
    if (keep >= 4) continue;
    const uint32_t at = tile + TL::kBytes + TL::kCodeBytes + 4 * w;
    const uint32_t left = keep <= 0 ? 0u : lds32(at) & ((1u << (8 * keep)) - 1u);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(left) : "memory");
  }
}

constexpr float kTiny = 1.17549435e-38f, kHuge = 3.4028234e38f;

// A query row as f16 operands: `f` holds PER = D / 32 dims of it a lane.  f16
// rows enter as they are, bf16 rows shifted by a power of two into f16 range
// (the largest magnitude in [2^14, 2^15)).  Returns the row's score factor,
// scale_log2 with the shift undone.  Warp-collective.
template <typename T, int WORDS>
__device__ __forceinline__ float convert_row(uint32_t (&f)[WORDS], float scale_log2) {
  if constexpr (std::is_same<T, __half>::value) {
    return scale_log2;
  } else {
    uint32_t top = 0;  // largest magnitude's bits
#pragma unroll
    for (int k = 0; k < WORDS; ++k) top = max(max(top, f[k] & 0x7fffu), f[k] >> 16 & 0x7fffu);
    top = __reduce_max_sync(kFull, top);
    const int ex = top > 0 ? static_cast<int>(top >> 7) - 126 : 15;
    const int qshift = max(-120, min(120, 15 - ex));
    const float up = __int_as_float((127 + qshift) << 23);
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
      float x, y;
      Mma<T>::unpack(f[k], x, y);
      f[k] = Mma<__half>::pack(x * up, y * up);
    }
    // (kept positive and finite: 0 and infinity would make NaN of masked scores)
    return fminf(fmaxf(scale_log2 * __int_as_float((127 - qshift) << 23), kTiny), kHuge);
  }
}

// float32 operands enter the f16 MMAs as two parts.
constexpr int kF32Parts = 2;

// Two float32 values as two f16 pairs: x = hi + lo to 2^-24 of x -- lo rounds what is
// left, at most 2^-12 of x, to 2^-12 of that -- or 2^-25 where lo is subnormal.  An
// infinity or NaN is the first part's alone.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&part)[kF32Parts]) {
  part[0] = Mma<__half>::pack(x, y);
  float hx, hy;
  Mma<__half>::unpack(part[0], hx, hy);
  part[1] = Mma<__half>::pack(isfinite(x) ? x - hx : 0.f, isfinite(y) ? y - hy : 0.f);
}

// A float32 query row as f16 operands in two parts: shifted by a power of two so that
// its largest magnitude lies in [2^14, 2^15), an element is off by at most 2^-24 of
// itself or 2^-39 of the largest.  Returns the row's score factor (convert_row).
// Warp-collective.
template <int PER>
__device__ __forceinline__ float split_row(const uint32_t (&f)[PER],
                                           uint32_t (&parts)[kF32Parts][PER / 2],
                                           float scale_log2) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) top = max(top, f[k] & 0x7fffffffu);
  top = __reduce_max_sync(kFull, top);
  const int ex = top > 0 ? static_cast<int>(top >> 23) - 126 : 15;
  const int qshift = max(-120, min(120, 15 - ex));
  const float up = __int_as_float((127 + qshift) << 23);
#pragma unroll
  for (int k = 0; k < PER; k += 2) {
    uint32_t part[kF32Parts];
    split_pair(__uint_as_float(f[k]) * up, __uint_as_float(f[k + 1]) * up, part);
#pragma unroll
    for (int j = 0; j < kF32Parts; ++j) parts[j][k / 2] = part[j];
  }
  return fminf(fmaxf(scale_log2 * __int_as_float((127 - qshift) << 23), kTiny), kHuge);
}

// The query rows of a piece: how many, the first one's flat index (of j = 0, its
// KV head's first query head), and column col's offset from it and query number.
__device__ __forceinline__ int rows_of(const AttnParams &p, int chunk) {
  return min(p.rows_per_cta, p.rows - chunk * p.rows_per_cta);
}
__device__ __forceinline__ int64_t first_row(const AttnParams &p, int b, int kvh) {
  return static_cast<int64_t>(b) * p.num_queries * p.num_heads + kvh * p.group;
}
__device__ __forceinline__ void map_columns(const AttnParams &p, int chunk, int columns, int *row,
                                            int *j_of) {
  for (int col = threadIdx.x & 31; col < columns; col += 32) {
    const int r = chunk * p.rows_per_cta + col;
    const int j = p.group == 1 ? r : r / p.group;
    row[col] = j * p.num_heads + r - j * p.group;
    j_of[col] = j;
  }
  __syncwarp();
}

// The fewest places of a worker: 8 contexts of 300 to 2000 rows, 8 KV heads, take
// 12.3 us at 4, 14.7 at 8, 17.4 at 16 (and 12.8 at 2).
constexpr int kMinPlaces = 4;

// The pieces of work of a worker (a CTA or a warp), in turn: one under the
// host's and the device's split partitions (cta_work), under the balanced one
// the parts of units in its range of the list of all places.
// Warp-collective; the warps of a CTA that is a worker walk alike.
struct Piece {
  int b, kvh, chunk, L;
  int blk_begin, blk_end;
  int split, item;  // of partial_index (CtaWork)
};
struct Pieces {
  int worker;
  int x, x1;  // balanced: the places still to do (the list has < 2^31)
  int base;   // first place of sequence `from`
  int from;   // first of the 32 sequences that were looked at last
  // the sequence that x was last found in, its first place and blocks
  int b, begin, nblk, L;

  // Blocks of sequence i (0 past the batch) and its places in the list.
  static __device__ __forceinline__ int blocks(const AttnParams &p, int i) {
    return i < p.batch ? seq_extent(p, i, false).nblk : 0;
  }
  static __device__ __forceinline__ int places(const AttnParams &p, int n) {
    return n > 0 ? p.num_kv_heads * p.row_chunks * (n + p.sk_weight) : 0;
  }
  // Inclusive sum over the lanes.
  static __device__ __forceinline__ int upto(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kFull, v, o);
      if ((threadIdx.x & 31) >= o) v += t;
    }
    return v;
  }

  __device__ __forceinline__ bool first(const AttnParams &p, int which, Piece *w) {
    worker = which;
    if (!p.stream_k) {
      const CtaWork k = cta_work(p);
      *w = Piece{k.b, k.kvh, k.chunk, k.ext.L, k.blk_begin, k.blk_end, k.split,
                 static_cast<int>(k.item)};
      x = x1 = 0;
      return k.active;
    }
    const int lane = threadIdx.x & 31;
    const bool report = blockIdx.x == 0 && threadIdx.x < 32;  // lengths out of range
    int total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 128) {
      int n[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) n[k] = blocks(p, b0 + 32 * k + lane);  // loads in flight together
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (report && b0 + 32 * k + lane < p.batch) seq_extent(p, b0 + 32 * k + lane, true);
        total += __reduce_add_sync(kFull, places(p, n[k]));
      }
    }
    // No worker without a few places: short batches are not cut to pieces, and
    // the slots of a unit's pieces are consecutive.
    const int workers = min(p.split_target, max(total / kMinPlaces, 1));
    if (worker >= workers) return false;
    const int each = total / workers, more = total - each * workers;  // (32-bit divisions)
    x = worker * each + min(worker, more);
    x1 = x + each + (worker < more ? 1 : 0);
    base = from = 0;
    begin = nblk = 0;
    return next(p, w);
  }

  __device__ __forceinline__ bool next(const AttnParams &p, Piece *w) {
    const int lane = threadIdx.x & 31;
    const int units = p.num_kv_heads * p.row_chunks;
    while (x < x1) {
      if (x >= begin + places(p, nblk)) {  // another sequence
        const int n = blocks(p, from + lane), mine = places(p, n);
        const int sum = __reduce_add_sync(kFull, mine);
        if (x >= base + sum) {  // past these 32
          base += sum;
          from += 32;
          continue;
        }
        const int to = upto(mine);
        const int at = __ffs(__ballot_sync(kFull, base + to > x)) - 1;
        b = from + at;
        begin = base + __shfl_sync(kFull, to - mine, at);
        nblk = __shfl_sync(kFull, n, at);
        L = seq_extent(p, b, false).L;
      }
      const int r = x - begin, len = nblk + p.sk_weight;
      const int u = r / len;
      const int lo = max(r - u * len - p.sk_weight, 0);
      const int end = min(x1, begin + (u + 1) * len);
      const int hi = end - begin - u * len - p.sk_weight;
      x = end;
      if (hi <= lo) continue;  // only the unit's fixed cost lies in this range
      w->b = b;
      w->kvh = p.row_chunks == 1 ? u : u / p.row_chunks;
      w->chunk = u - w->kvh * p.row_chunks;
      w->L = L;
      w->blk_begin = lo;
      w->blk_end = hi;
      w->split = 0;
      w->item = worker + b * units + u;
      // the merge kernel finds a unit's pieces by its first and last slot
      if (lane == 0) {
        if (lo == 0) p.split_info[2 * (b * units + u)] = w->item;
        if (hi == nblk) p.split_info[2 * (b * units + u) + 1] = w->item;
      }
      return true;
    }
    return false;
  }
};

}  // namespace fp4
}  // namespace pkv
