// attn_fp4.cu -- decode, causal and tree verification over the block-scaled
// 4-bit cache (fp4.cuh) on tensor cores, q and out bfloat16 or float16.
//
// One CTA serves one (sequence, KV head, row chunk, split) as the 16-bit
// kernel does (attn_mma.cuh): its four warps take every fourth block, each
// with its own ring of bulk copies (a tile is contiguous and its layout needs
// no swizzle, so the copies are plain 1-D ones).  Per 16-key block, keys on
// the MMA's M side and NT tiles of 8 query columns on N:
//   S^T = K Q^T,  online softmax over the keys (log2 units),  O^T += V^T P^T.
// Codes are widened to f16 pairs by the conversion unit and multiplied by
// their block scale there: code * scale has at most 6 significant bits, so the
// operands are exact; q enters as f16 after a power-of-two shift per row
// (undone in the score's factor) and the weights as f16 (2^-11 relative, below
// the output's own rounding); sums are float32.
//
// The order of keys and dims inside the MMAs is free, and chosen so that no
// operand is shuffled between lanes.  Lane (g, c) = (lane / 4, lane % 4):
//   scores   row g of M is key 4 (g / 2) + g % 2, row g + 8 the key two after
//            it; a lane reads 32 dims (c) of its two keys, 16 bytes each, two
//            scale blocks; k-step j takes 4 of them from each lane.
//   P.V      with those rows, movmatrix leaves lane (g, c) the weights of keys
//            4c .. 4c + 3, and it reads those keys' codes of 8 dims (word
//            g + 8 h): 16 bytes.  A nibble merge pairs two keys' codes of a
//            dim in one byte, which converts to one operand register.
#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
namespace {

constexpr int kLanes = 4;  // warps of a CTA, each a block lane
constexpr float kSlack = 8.f;  // log2: weights stay below 2^8 (as in attn_mma.cuh)

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

// Key (row of the block) of MMA row g; row g + 8 is the key two after it.
__device__ __forceinline__ int key_of(int g) { return 4 * (g >> 1) + (g & 1); }

// Head dim of element pair (row g, row g + 8) of O^T's m-tile mt: dims d, d + 1.
__device__ __forceinline__ int o_dim(int mt, int g) {
  return 8 * (g + 8 * (mt >> 2)) + 2 * (mt & 3);
}

// d = a * b: the first product of a chain.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The pieces of work of this CTA, in turn: one under the host's and the
// device's split partitions (cta_work), under the balanced one the parts of
// units in its range of the list (sk_begin, pkv_device.cuh).  Warp-collective;
// every warp walks alike.
struct Pieces {
  int x, x1;  // balanced: the places still to do (the list has < 2^31)
  int base;   // first place of sequence `from`
  int from;   // first of the 32 sequences that the lanes hold

  __device__ __forceinline__ int places(const AttnParams &p, int b, int *nblk) const {
    *nblk = b < p.batch ? seq_extent(p, b, false).nblk : 0;
    return *nblk > 0 ? p.num_kv_heads * p.row_chunks * (*nblk + p.sk_weight) : 0;
  }

  __device__ __forceinline__ bool first(const AttnParams &p, CtaWork *w) {
    if (!p.stream_k) {
      *w = cta_work(p);
      x = x1 = 0;
      return w->active;
    }
    const int lane = threadIdx.x & 31;
    const bool publish = blockIdx.x == 0 && threadIdx.x < 32;  // the list, for the merge kernel
    int total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int nblk;
      const int mine = places(p, b0 + lane, &nblk);
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += t;
      }
      if (publish && b0 + lane < p.batch) {
        seq_extent(p, b0 + lane, true);  // reports lengths out of range
        p.split_info[2 * (b0 + lane)] = total + upto - mine;
        p.split_info[2 * (b0 + lane) + 1] = nblk;
      }
      total += __shfl_sync(kFull, upto, 31);
    }
    if (publish && lane == 0) p.split_info[2 * p.batch] = total;
    x = static_cast<int>(sk_begin(total, p.split_target, blockIdx.x));
    x1 = static_cast<int>(sk_begin(total, p.split_target, blockIdx.x + 1));
    base = 0;
    from = 0;
    return next(p, w);
  }

  __device__ __forceinline__ bool next(const AttnParams &p, CtaWork *w) {
    const int lane = threadIdx.x & 31;
    const int units = p.num_kv_heads * p.row_chunks;
    while (x < x1) {
      int nblk;
      const int mine = places(p, from + lane, &nblk);
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += t;
      }
      const unsigned hit = __ballot_sync(kFull, base + upto > x);
      if (hit == 0u) {  // x lies past these 32 sequences
        base += __shfl_sync(kFull, upto, 31);
        from += 32;
        continue;
      }
      const int at = __ffs(hit) - 1;
      const int n = __shfl_sync(kFull, nblk, at);
      const int begin = base + __shfl_sync(kFull, upto - mine, at);
      const int r = x - begin, len = n + p.sk_weight;
      const int u = r / len;
      const int lo = max(r - u * len - p.sk_weight, 0);
      const int end = min(x1, begin + (u + 1) * len);
      const int hi = end - begin - u * len - p.sk_weight;
      x = end;
      if (hi <= lo) continue;  // only the unit's fixed cost lies in this range
      w->b = from + at;
      w->kvh = u / p.row_chunks;
      w->chunk = u - w->kvh * p.row_chunks;
      w->ns_b = 2;  // (always partials, for the merge kernel)
      w->split = 0;
      w->ext = seq_extent(p, w->b, false);
      w->blk_begin = lo;
      w->blk_end = hi;
      w->item = blockIdx.x + static_cast<int64_t>(w->b) * units + u;
      w->active = true;
      return true;
    }
    return false;
  }
};

// Resident CTAs a tile is compiled for.
template <int D, int NT> constexpr int min_ctas() {
  return D == 256 ? 2 : (NT == 1 ? 4 : (NT == 2 ? 3 : 2));
}

template <typename T, int D, int NT, int KB, int NS>
__global__ void __launch_bounds__(kLanes * 32, (min_ctas<D, NT>()))
    mma_kernel(const AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  using TL = Tile<D>;
  using MM = Mma<__half>;
  constexpr int PAIR = 2 * TL::kBytes;  // a block's key and value tiles
  constexpr int STAGE = KB * PAIR;      // a group of KB consecutive blocks
  constexpr int KS = D / 16;            // k-steps of the scores, m-tiles of O^T
  constexpr int NC = NT * 8;
  constexpr int WP = TL::kPanel / 32;   // words (8 dims) of a lane in a panel
  constexpr int KSP = 2 * WP;           // k-steps of a panel
  static_assert(2 * KB * NS <= 32 && 32 % KB == 0, "bad-block bits, table chunks");

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ uint64_t bars[kLanes * NS];
  // the epilogue's scratch follows the rings: the next piece's copies fly
  // while a piece is finished
  float *const red_o = reinterpret_cast<float *>(smem + kLanes * NS * STAGE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t my_bars = smem_u32(&bars[warp * NS]);
  const uint32_t my_stages = smem_u32(smem) + warp * NS * STAGE;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(my_bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();

  Pieces pieces;
  CtaWork wk;
  if (!pieces.first(p, &wk)) return;  // (the whole CTA agrees)

  // The ring runs on across pieces.  A warp's groups of a piece are number
  // warp, warp + kLanes, ... of it; `issue` copies group i of the piece `to`.
  int n_groups = 0, nspan = 0;  // of the piece whose copies are issued: mine, its blocks
  int stage_in = 0;             // stage that the next group goes to
  int stage_out = 0, phase = 0; // stage that is computed next, and its parity
  int in_flight = 0;
  uint32_t bad_ring = 0;        // 2 KB bits a stage
  const int32_t *table = nullptr;
  int tab_cur = 0, tab_next = 0;
  int head_off = 0;
  auto load_entries = [&](int chunk32) -> int {
    const int j = chunk32 * 32 + lane;
    const int blk = ((j / KB) * kLanes + warp) * KB + j % KB;
    return blk < nspan ? ld_keep(table + blk) : -1;
  };
  auto issue = [&](int i) {
    if (i > 0 && (i * KB) % 32 == 0) {
      tab_cur = tab_next;
      tab_next = load_entries(i * KB / 32 + 1);
    }
    const int v = __shfl_sync(kFull, tab_cur, (i * KB + (lane >> 1)) & 31);
    const int cnt = min(KB, nspan - (i * kLanes + warp) * KB);
    const bool mine = lane < 2 * cnt;
    const bool bad = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
    const uint32_t bits = __ballot_sync(kFull, mine && bad);
    const int sh = stage_in * 2 * KB;
    bad_ring = (bad_ring & ~(((1u << (2 * KB)) - 1u) << sh)) | (bits << sh);
    const uint32_t bar = my_bars + 8 * stage_in;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, cnt * PAIR);
      if (bits) record_error(p.err, PKV_DEVERR_BLOCK_ID);
    }
    if (mine) {
      const int64_t off =
          (static_cast<int64_t>(bad ? 0 : v) * p.num_kv_heads + head_off) * TL::kBytes;
      bulk_g2s(my_stages + stage_in * STAGE + lane * TL::kBytes,
               static_cast<const uint8_t *>((lane & 1) ? p.v_cache : p.k_cache) + off, TL::kBytes,
               bar);
    }
    stage_in = stage_in + 1 == NS ? 0 : stage_in + 1;
    ++in_flight;
  };
  bool dead = false;  // a copy never came: no more waits or copies, only barriers
  auto prologue = [&](const CtaWork &w) {
    nspan = max(w.blk_end - w.blk_begin, 0);
    const int groups = (nspan + KB - 1) / KB;
    n_groups = dead ? 0 : (groups > warp ? (groups - warp + kLanes - 1) / kLanes : 0);
    table = p.block_table + static_cast<int64_t>(w.b) * p.max_blocks_per_seq + w.blk_begin;
    head_off = w.kvh;
    tab_cur = load_entries(0);
    tab_next = load_entries(1);
    const int n = min(NS, n_groups);
    for (int i = 0; i < n; ++i) issue(i);
  };
  prologue(wk);

  // Byte offsets of this lane's pieces in a block's tiles.
  const int kk = key_of(g);
  const uint32_t k_off = kk * (TL::kPanel / 2) + c * (4 * WP);
  const uint32_t ks_off = TL::kCodeBytes + kk * TL::kScales + c * (WP / 2);
  const uint32_t v_off = TL::kBytes + g * 64 + c * 16;
  const uint32_t vs_off = TL::kBytes + TL::kCodeBytes + (g >> 1) * 16 + c * 4;

  for (bool more = true; more;) {
    const int b = wk.b, chunk = wk.chunk, L = wk.ext.L;
    const int mask_from = L - p.num_queries;  // first row some column may not see

    // Q^T operand fragments: k-step (panel, word w, half i) holds dims
    // panel + 8 WP c + 8 w + 4 i + {0, 1 | 2, 3} of column g, shifted by
    // 2^qshift into f16 range (the row's largest magnitude in [2^14, 2^15)).
    uint32_t qf[KS][NT][2];
    float colfac[NT][2];  // score factor of my two columns of each tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int64_t row = cta_row_index(p, b, wk.kvh, chunk, nt * 8 + g);
      const T *qrow = reinterpret_cast<const T *>(p.q) + (row < 0 ? 0 : row) * D;
      float qv[KS][4];
      float amax = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < KS / 2; ++k2) {
        const int pn = (2 * k2) / KSP, w = (2 * k2) % KSP / 2;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row >= 0)
          x = *reinterpret_cast<const uint4 *>(qrow + pn * TL::kPanel + (c * WP + w) * 8);
        Mma<T>::unpack(x.x, qv[2 * k2][0], qv[2 * k2][1]);
        Mma<T>::unpack(x.y, qv[2 * k2][2], qv[2 * k2][3]);
        Mma<T>::unpack(x.z, qv[2 * k2 + 1][0], qv[2 * k2 + 1][1]);
        Mma<T>::unpack(x.w, qv[2 * k2 + 1][2], qv[2 * k2 + 1][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(qv[2 * k2][e]), fabsf(qv[2 * k2 + 1][e])));
      }
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      const int ex = amax > 0.f ? ((__float_as_int(amax) >> 23) & 0xff) - 126 : 15;
      const int qshift = max(-120, min(120, 15 - ex));
      const float up = exp2f(static_cast<float>(qshift));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks][nt][0] = MM::pack(qv[ks][0] * up, qv[ks][1] * up);
        qf[ks][nt][1] = MM::pack(qv[ks][2] * up, qv[ks][3] * up);
      }
      // my score columns 2c, 2c + 1 were shifted by the lanes of groups 2c, 2c + 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sh = __shfl_sync(kFull, qshift, 4 * (2 * c + e));
        colfac[nt][e] = p.scale_log2 * exp2f(static_cast<float>(-sh));
      }
    }

    // Online-softmax state, per column of mine: the reference, a raw score (0
    // until a row is seen), the raw score that raises it, and the sum.  Weights
    // are 2^((s - m) colfac): the difference first, so that the largest score
    // has weight 1 however large it is.
    float o[KS][NT][4];
    float m[NT][2], raise[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = 0.f;
      raise[nt][0] = raise[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }

    const int n_here = n_groups;
    for (int i = 0; i < n_here; ++i) {
      // one decision per warp: its lanes then agree on every later shuffle
      if (!__all_sync(kFull, mbar_wait_bounded(my_bars + 8 * stage_out, phase))) {
        dead = true;
        if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        break;
      }
      const uint32_t tile = my_stages + stage_out * STAGE;
      const int blk0 = (i * kLanes + warp) * KB;  // of the piece
      const int key0 = (wk.blk_begin + blk0) * kBlockSize;
      const uint32_t bad = (bad_ring >> (stage_out * 2 * KB)) & ((1u << (2 * KB)) - 1u);
      // an edge group has rows that some column may not see, a bad block, or
      // fewer blocks (then a stage's rest is computed on whatever it holds,
      // finite or not, and masked out entirely)
      const bool edge = bad != 0u || key0 + KB * kBlockSize > mask_from || blk0 + KB > nspan;

      constexpr int NCH = NT == 1 ? 2 : 1;  // accumulator chains of a block's scores
      float sc[KB][NT][4];
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        float acc[NCH][NT][4];
#pragma unroll
        for (int pn = 0; pn < TL::kPanels; ++pn) {
          uint32_t w0[WP], w1[WP], s0[2], s1[2];
          const uint32_t at = tile + u * PAIR + k_off + pn * (kBlockSize * TL::kPanel / 2);
          const uint32_t sat = tile + u * PAIR + ks_off + pn * 8;
          if constexpr (WP == 4) {
            const uint4 x = lds128(at), y = lds128(at + TL::kPanel);
            w0[0] = x.x; w0[1] = x.y; w0[2] = x.z; w0[3] = x.w;
            w1[0] = y.x; w1[1] = y.y; w1[2] = y.z; w1[3] = y.w;
            const uint32_t a = e4m3x2_to_f16(lds16(sat));
            const uint32_t bq = e4m3x2_to_f16(lds16(sat + 2 * TL::kScales));
            s0[0] = perm(a, 0x1010); s0[1] = perm(a, 0x3232);
            s1[0] = perm(bq, 0x1010); s1[1] = perm(bq, 0x3232);
          } else {
            const uint2 x = lds64(at), y = lds64(at + TL::kPanel);
            w0[0] = x.x; w0[1] = x.y;
            w1[0] = y.x; w1[1] = y.y;
            s0[0] = s0[1] = perm(e4m3x2_to_f16(lds8(sat)), 0x1010);
            s1[0] = s1[1] = perm(e4m3x2_to_f16(lds8(sat + 2 * TL::kScales)), 0x1010);
          }
#pragma unroll
          for (int w = 0; w < WP; ++w) {
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(w0[w], h0);
            e2m1x8_to_f16(w1[w], h1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ks = pn * KSP + w * 2 + e;
              const uint32_t a[4] = {mul2(h0[2 * e], s0[w >> 1]), mul2(h1[2 * e], s1[w >> 1]),
                                     mul2(h0[2 * e + 1], s0[w >> 1]),
                                     mul2(h1[2 * e + 1], s1[w >> 1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (ks < NCH)
                  mma_first(acc[ks % NCH][nt], a, qf[ks][nt][0], qf[ks][nt][1]);
                else
                  MM::run(acc[ks % NCH][nt], a, qf[ks][nt][0], qf[ks][nt][1]);
              }
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[u][nt][e] = acc[0][nt][e];
            if (NCH == 2) sc[u][nt][e] += acc[NCH - 1][nt][e];
          }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * c + e;
            const int lim = cta_row_limit(p, L, chunk, col);
            const unsigned long long tm = cta_row_tree_mask(p, b, chunk, col);
#pragma unroll
            for (int u = 0; u < KB; ++u) {
              const bool none = ((bad >> (2 * u)) & 1u) || blk0 + u >= nspan;
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (!key_visible(p, key0 + u * kBlockSize + kk + 2 * r, L, none, lim, tm))
                  sc[u][nt][e + 2 * r] = -INFINITY;
            }
          }
      }
      // Online softmax against a per-column reference, raised to the exact
      // running maximum (rescaling l and O) only when a score exceeds it by
      // more than the slack; O / l does not depend on the reference.  A NaN
      // score never raises it and reaches O through its weight.
      float top[NT][2];
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
          for (int u = 1; u < KB; ++u) t = fmaxf(t, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
          top[nt][e] = t;
          above |= t > raise[nt][e];
        }
      if (__any_sync(kFull, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = top[nt][e];
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
            const bool none = raise[nt][e] == -INFINITY;  // nothing seen so far
            const float m_new = none ? (mx == -INFINITY ? 0.f : mx) : fmaxf(m[nt][e], mx);
            const float corr = none ? 0.f : ex2((m[nt][e] - m_new) * colfac[nt][e]);
            l[nt][e] *= corr;
            m[nt][e] = m_new;
            if (!none || mx != -INFINITY) raise[nt][e] = m_new + kSlack / colfac[nt][e];
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              o[mt][nt][e] *= corr;
              o[mt][nt][e + 2] *= corr;
            }
          }
      }
      uint32_t ph[KB][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < KB; ++u) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = ex2((sc[u][nt][e] - m[nt][e & 1]) * colfac[nt][e & 1]);
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          ph[u][nt][0] = movm_t(MM::pack(w[0], w[1]));
          ph[u][nt][1] = movm_t(MM::pack(w[2], w[3]));
        }
      // O^T += V^T P^T.
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        uint32_t m01 = kFull, m23 = kFull;
        if (edge) {
          // keys past the context (or of a bad block) get scale 0: their codes
          // are finite whatever they are, so they add nothing
          const bool none = ((bad >> (2 * u)) & 1u) || blk0 + u >= nspan;
          const int nv = none ? 0 : L - key0 - u * kBlockSize;
          m01 = (4 * c < nv ? 0x0000ffffu : 0u) | (4 * c + 1 < nv ? 0xffff0000u : 0u);
          m23 = (4 * c + 2 < nv ? 0x0000ffffu : 0u) | (4 * c + 3 < nv ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 w = lds128(tile + u * PAIR + v_off + h * 512);
          const uint32_t sw = lds32(tile + u * PAIR + vs_off + h * 64);
          const uint32_t s01 = e4m3x2_to_f16(sw) & m01, s23 = e4m3x2_to_f16(sw >> 16) & m23;
          constexpr uint32_t LOW = 0x0f0f0f0fu;
          uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, keys (0, 1) and (2, 3)
          e2m1x8_to_f16((w.x & LOW) | ((w.y << 4) & ~LOW), e01);
          e2m1x8_to_f16(((w.x >> 4) & LOW) | (w.y & ~LOW), o01);
          e2m1x8_to_f16((w.z & LOW) | ((w.w << 4) & ~LOW), e23);
          e2m1x8_to_f16(((w.z >> 4) & LOW) | (w.w & ~LOW), o23);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a[4] = {mul2(e01[j], s01), mul2(o01[j], s01), mul2(e23[j], s23),
                                   mul2(o23[j], s23)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              MM::run(o[h * 4 + j][nt], a, ph[u][nt][0], ph[u][nt][1]);
          }
        }
      }
      __syncwarp();  // the warp is done with this stage
      --in_flight;
      if (++stage_out == NS) {
        stage_out = 0;
        phase ^= 1;
      }
      if (i + NS < n_here) issue(i + NS);
    }

    // The next piece's first copies, then this piece's end.
    const CtaWork done = wk;
    more = pieces.next(p, &wk);
    if (more) prologue(wk);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        l[nt][e] = v;
      }
    constexpr int DP = D + 4;
    float *red_m = red_o + kLanes * NC * DP;
    float *red_l = red_m + kLanes * NC;
    float *wscale = red_l + kLanes * NC;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = nt * 8 + 2 * c + e;
        float *dst = red_o + (warp * NC + col) * DP;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
          *reinterpret_cast<float2 *>(dst + o_dim(mt, g)) =
              make_float2(o[mt][nt][e], o[mt][nt][e + 2]);
        if (g == 0) {
          red_m[warp * NC + col] =
              raise[nt][e] == -INFINITY ? -INFINITY : m[nt][e] * colfac[nt][e];
          red_l[warp * NC + col] = l[nt][e];
        }
      }
    __syncthreads();
    cta_epilogue<T, D, NC, kLanes, kLanes * 32>(p, red_m, red_l, red_o, wscale, done);
    __syncthreads();  // the scratch is free again
  }
  // After a time-out: give the copies in flight a bounded chance to land
  // before the shared memory is given up.
  while (dead && in_flight > 0) {
    mbar_wait_bounded(my_bars + 8 * stage_out, phase);
    --in_flight;
    if (++stage_out == NS) {
      stage_out = 0;
      phase ^= 1;
    }
  }
}

// Blocks of a group and ring depth (in groups) of each tile.
template <int D, int NT> constexpr int group_blocks() { return NT == 1 && D <= 128 ? 2 : 1; }
template <int D, int NT> constexpr int ring() { return group_blocks<D, NT>() == 2 ? 2 : 4; }

template <int D, int NT> constexpr size_t mma_smem() {
  constexpr int NC = NT * 8;
  constexpr size_t stages =
      size_t(kLanes) * ring<D, NT>() * group_blocks<D, NT>() * 2 * Tile<D>::kBytes;
  constexpr size_t red = (size_t(kLanes) * NC * (D + 4) + size_t(3 * kLanes + 2) * NC) * 4;
  constexpr size_t merge = (size_t(NC) * kMaxFusedSplits + NC) * 4;
  return stages + (red > merge ? red : merge) + 128;
}

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename T, int D, int NT>
cudaError_t mma_launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  constexpr int KB = group_blocks<D, NT>(), NS = ring<D, NT>();
  return launch_kernel(true, mma_kernel<T, D, NT, KB, NS>, grid, kLanes * 32, mma_smem<D, NT>(),
                       stream, p);
}

template <typename T, int D, int NT> bool take(KernelInfo *info, Launch *launch) {
  constexpr int KB = group_blocks<D, NT>(), NS = ring<D, NT>();
  info->func = reinterpret_cast<const void *>(&mma_kernel<T, D, NT, KB, NS>);
  info->threads = kLanes * 32;
  info->warps = kLanes;
  info->stages = NS;
  info->smem = mma_smem<D, NT>();
  info->warp_tiles = NT;
  info->blocks_per_iter = KB;
  *launch = &mma_launch_t<T, D, NT>;
  return true;
}

template <typename T, int D> bool pick_nt(int nt, KernelInfo *info, Launch *launch) {
  if constexpr (D == 256) return nt == 1 && take<T, D, 1>(info, launch);
  switch (nt) {
    case 1: return take<T, D, 1>(info, launch);
    case 2: return take<T, D, (D <= 128 ? 2 : 1)>(info, launch);
    case 3: return take<T, D, (D <= 128 ? 3 : 1)>(info, launch);
    default: return false;
  }
}

template <typename T> bool pick_d(int D, int nt, KernelInfo *info, Launch *launch) {
  switch (D) {
    case 64: return pick_nt<T, 64>(nt, info, launch);
    case 128: return pick_nt<T, 128>(nt, info, launch);
    case 256: return pick_nt<T, 256>(nt, info, launch);
    default: return false;
  }
}

bool pick(pkv_dtype q_dtype, int D, int nt, KernelInfo *info, Launch *launch) {
  switch (q_dtype) {
    case PKV_BF16: return pick_d<__nv_bfloat16>(D, nt, info, launch);
    case PKV_F16: return pick_d<__half>(D, nt, info, launch);
    default: return false;
  }
}

}  // namespace
}  // namespace fp4

int mma_fp4_max_tiles(int head_dim) { return head_dim <= 128 ? 3 : 1; }

bool mma_fp4_kernel_info(pkv_dtype q_dtype, int head_dim, int tiles, KernelInfo *info) {
  fp4::Launch launch = nullptr;
  return fp4::pick(q_dtype, head_dim, tiles, info, &launch);
}

cudaError_t mma_fp4_launch(pkv_dtype q_dtype, int head_dim, int tiles, const AttnParams &p,
                           dim3 grid, cudaStream_t stream) {
  KernelInfo info;
  fp4::Launch launch = nullptr;
  if (!fp4::pick(q_dtype, head_dim, tiles, &info, &launch)) return cudaErrorInvalidValue;
  return launch(p, grid, stream);
}

}  // namespace pkv
