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

template <typename T, int D, int NT, int KB, int NS>
__global__ void __launch_bounds__(kLanes * 32)
    mma_kernel(const AttnParams p) {
  static_assert(NS >= 2 * KB, "a pair of blocks in flight while a pair is computed");
  pdl_launch_dependents();
  pdl_wait();
  using TL = Tile<D>;
  using MM = Mma<__half>;
  constexpr int STAGE = 2 * TL::kBytes;
  constexpr int KS = D / 16;            // k-steps of the scores, m-tiles of O^T
  constexpr int NC = NT * 8;
  constexpr int WP = TL::kPanel / 32;   // words (8 dims) of a lane in a panel
  constexpr int KSP = 2 * WP;           // k-steps of a panel

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ uint64_t bars[kLanes * NS];
  __shared__ int s_lim[NC];                // causal visible-row limit per column
  __shared__ unsigned long long s_tm[NC];  // tree mask per column

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const CtaWork wk = cta_work(p);
  if (!wk.active) return;  // a split past its sequence's end (the whole CTA agrees)
  const int kvh = wk.kvh, chunk = wk.chunk, b = wk.b;
  const int L = wk.ext.L;
  const int blk_begin = wk.blk_begin;
  const int nspan = max(wk.blk_end - blk_begin, 0);
  const int n_my = nspan > warp ? (nspan - warp + kLanes - 1) / kLanes : 0;
  const int mask_from = L - p.num_queries;  // first row some column may not see

  const uint32_t my_bars = smem_u32(&bars[warp * NS]);
  const uint32_t my_stages = smem_u32(smem) + warp * NS * STAGE;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(my_bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();

  const int32_t *table =
      p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + blk_begin + warp;
  auto load_entries = [&](int chunk32) -> int {
    const int i = chunk32 * 32 + lane;
    return i < n_my ? ld_keep(table + static_cast<int64_t>(i) * kLanes) : -1;
  };
  int tab_cur = load_entries(0), tab_next = load_entries(1);
  uint32_t bad_mask = 0;
  auto issue = [&](int i) {
    if ((i & 31) == 0 && i > 0) {
      tab_cur = tab_next;
      tab_next = load_entries((i >> 5) + 1);
    }
    const int v = __shfl_sync(kFull, tab_cur, i & 31);
    const bool bad = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
    bad_mask = bad ? (bad_mask | (1u << (i & 31))) : (bad_mask & ~(1u << (i & 31)));
    if (lane == 0) {
      if (bad) record_error(p.err, PKV_DEVERR_BLOCK_ID);
      const int64_t off =
          (static_cast<int64_t>(bad ? 0 : v) * p.num_kv_heads + kvh) * TL::kBytes;
      const int s = i % NS;
      const uint32_t bar = my_bars + 8 * s, st = my_stages + s * STAGE;
      mbar_arrive_expect_tx(bar, STAGE);
      bulk_g2s(st, static_cast<const uint8_t *>(p.k_cache) + off, TL::kBytes, bar);
      bulk_g2s(st + TL::kBytes, static_cast<const uint8_t *>(p.v_cache) + off, TL::kBytes, bar);
    }
  };
  int issued = min(NS, n_my);
  for (int i = 0; i < issued; ++i) issue(i);

  for (int col = threadIdx.x; col < NC; col += kLanes * 32) {
    s_lim[col] = cta_row_limit(p, L, chunk, col);
    s_tm[col] = cta_row_tree_mask(p, b, chunk, col);
  }

  // Q^T operand fragments: k-step (panel, word w, half i) holds dims
  // panel + 8 WP c + 8 w + 4 i + {0, 1 | 2, 3} of column g, shifted by 2^qshift
  // into f16 range (the row's largest magnitude in [2^14, 2^15)).
  uint32_t qf[KS][NT][2];
  float colfac[NT][2];  // score factor of my two columns of each tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t row = cta_row_index(p, b, kvh, chunk, nt * 8 + g);
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

  float o[KS][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
  }
  __syncthreads();  // the columns' limits

  // Byte offsets of this lane's pieces in a tile.
  const int kk = key_of(g);
  const uint32_t k_off = kk * (TL::kPanel / 2) + c * (4 * WP);
  const uint32_t ks_off = TL::kCodeBytes + kk * TL::kScales + c * (WP / 2);
  const uint32_t v_off = TL::kBytes + g * 64 + c * 16;
  const uint32_t vs_off = TL::kBytes + TL::kCodeBytes + (g >> 1) * 16 + c * 4;

  bool timed_out = false;
  int landed = 0;
  for (int i0 = 0; i0 < n_my; i0 += KB) {
    bool ok = true;
    uint32_t tile[KB];
    int key0[KB];
    bool bad[KB];
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      const int i = i0 + u;
      const int s = i % NS;
      const bool has = KB == 1 || i < n_my;
      if (has && ok) {
        // one decision per warp: its lanes then agree on every later shuffle
        ok = __all_sync(kFull, mbar_wait_bounded(my_bars + 8 * s, (i / NS) & 1));
        if (ok) landed = i + 1;
      }
      // (a block past the end, in the last iteration, is computed on whatever
      // its stage holds -- finite or not -- and masked out entirely)
      tile[u] = my_stages + s * STAGE;
      key0[u] = (blk_begin + warp + i * kLanes) * kBlockSize;
      bad[u] = !has || ((bad_mask >> (i & 31)) & 1u);
    }
    if (!ok) {
      timed_out = true;
      break;
    }

    constexpr int NCH = NT * KB == 1 ? 4 : (NT * KB == 2 ? 2 : 1);  // accumulator chains
    float sc[KB][NT][4];
    bool above = false;  // some score exceeds its column's reference by > the slack
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      float acc[NCH][NT][4];
#pragma unroll
      for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[ch][nt][0] = acc[ch][nt][1] = acc[ch][nt][2] = acc[ch][nt][3] = 0.f;
#pragma unroll
      for (int pn = 0; pn < TL::kPanels; ++pn) {
        uint32_t w0[WP], w1[WP], s0[2], s1[2];
        const uint32_t at = tile[u] + k_off + pn * (kBlockSize * TL::kPanel / 2);
        if constexpr (WP == 4) {
          const uint4 x = lds128(at), y = lds128(at + TL::kPanel);
          w0[0] = x.x; w0[1] = x.y; w0[2] = x.z; w0[3] = x.w;
          w1[0] = y.x; w1[1] = y.y; w1[2] = y.z; w1[3] = y.w;
          const uint32_t a = e4m3x2_to_f16(lds16(tile[u] + ks_off + pn * 8));
          const uint32_t bq = e4m3x2_to_f16(lds16(tile[u] + ks_off + 2 * TL::kScales + pn * 8));
          s0[0] = perm(a, 0x1010); s0[1] = perm(a, 0x3232);
          s1[0] = perm(bq, 0x1010); s1[1] = perm(bq, 0x3232);
        } else {
          const uint2 x = lds64(at), y = lds64(at + TL::kPanel);
          w0[0] = x.x; w0[1] = x.y;
          w1[0] = y.x; w1[1] = y.y;
          s0[0] = s0[1] = perm(e4m3x2_to_f16(lds8(tile[u] + ks_off)), 0x1010);
          s1[0] = s1[1] = perm(e4m3x2_to_f16(lds8(tile[u] + ks_off + 2 * TL::kScales)), 0x1010);
        }
#pragma unroll
        for (int w = 0; w < WP; ++w) {
          uint32_t h0[4], h1[4];
          e2m1x8_to_f16(w0[w], h0);
          e2m1x8_to_f16(w1[w], h1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ks = pn * KSP + w * 2 + i;
            const uint32_t a[4] = {mul2(h0[2 * i], s0[w >> 1]), mul2(h1[2 * i], s1[w >> 1]),
                                   mul2(h0[2 * i + 1], s0[w >> 1]),
                                   mul2(h1[2 * i + 1], s1[w >> 1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              MM::run(acc[ks % NCH][nt], a, qf[ks][nt][0], qf[ks][nt][1]);
          }
        }
      }
      const bool need_mask = bad[u] || key0[u] + kBlockSize > mask_from;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float t = acc[0][nt][e];
#pragma unroll
          for (int ch = 1; ch < NCH; ++ch) t += acc[ch][nt][e];
          float v = t * colfac[nt][e & 1];
          if (need_mask) {
            const int col = nt * 8 + 2 * c + (e & 1);
            if (!key_visible(p, key0[u] + kk + (e & 2), L, bad[u], s_lim[col], s_tm[col]))
              v = -INFINITY;
          }
          sc[u][nt][e] = v;
          above |= v > m[nt][e & 1] + kSlack;
        }
      }
    }
    // Online softmax against a per-column reference m, raised to the exact
    // running maximum (rescaling l and O) only when a score exceeds it by more
    // than the slack; O / l does not depend on the reference.  A NaN score
    // never raises it and reaches O through its weight.
    if (__any_sync(kFull, above)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
          for (int u = 1; u < KB; ++u) mx = fmaxf(mx, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
          const float m_new = fmaxf(m[nt][e], mx);
          const float corr = ex2(m[nt][e] - (m_new == -INFINITY ? 0.f : m_new));
          l[nt][e] *= corr;
          m[nt][e] = m_new;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            o[mt][nt][e] *= corr;
            o[mt][nt][e + 2] *= corr;
          }
        }
    }
    uint32_t ph[KB][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m_use = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
        for (int u = 0; u < KB; ++u) {
          const float p0 = ex2(sc[u][nt][e] - m_use);
          const float p1 = ex2(sc[u][nt][e + 2] - m_use);
          l[nt][e] += p0 + p1;
          sc[u][nt][e] = p0;
          sc[u][nt][e + 2] = p1;
        }
      }
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        ph[u][nt][0] = movm_t(MM::pack(sc[u][nt][0], sc[u][nt][1]));
        ph[u][nt][1] = movm_t(MM::pack(sc[u][nt][2], sc[u][nt][3]));
      }
    }
    // O^T += V^T P^T.  Keys past the context (or of a bad block) get scale 0:
    // their codes are finite whatever they are, so they add nothing.
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      const int nvalid = bad[u] ? 0 : L - key0[u];
      uint32_t m01 = kFull, m23 = kFull;
      if (nvalid < kBlockSize) {
        m01 = (4 * c < nvalid ? 0x0000ffffu : 0u) | (4 * c + 1 < nvalid ? 0xffff0000u : 0u);
        m23 = (4 * c + 2 < nvalid ? 0x0000ffffu : 0u) | (4 * c + 3 < nvalid ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 w = lds128(tile[u] + v_off + h * 512);
        const uint32_t sw = lds32(tile[u] + vs_off + h * 64);
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
    __syncwarp();  // the warp is done with these stages
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      if (i0 + u + NS < n_my) {
        issue(i0 + u + NS);
        ++issued;
      }
    }
  }
  if (timed_out) {
    if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
    // give the copies in flight a bounded chance to land before their memory is reused
    for (int k = landed; k < issued; ++k) mbar_wait_bounded(my_bars + 8 * (k % NS), (k / NS) & 1);
  }

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
  __syncthreads();
  constexpr int DP = D + 4;
  float *red_o = reinterpret_cast<float *>(smem);
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
        red_m[warp * NC + col] = m[nt][e];
        red_l[warp * NC + col] = l[nt][e];
      }
    }
  __syncthreads();
  cta_epilogue<T, D, NC, kLanes, kLanes * 32>(p, red_m, red_l, red_o, wscale, wk);
}

template <int D, int NT, int NS> constexpr size_t mma_smem() {
  constexpr int NC = NT * 8;
  constexpr size_t stages = size_t(kLanes) * NS * 2 * Tile<D>::kBytes;
  constexpr size_t red = (size_t(kLanes) * NC * (D + 4) + size_t(3 * kLanes + 2) * NC) * 4;
  constexpr size_t merge = (size_t(NC) * kMaxFusedSplits + NC) * 4;
  constexpr size_t need = red > merge ? red : merge;
  return (need > stages ? need : stages) + 128;
}

// Blocks per iteration and ring depth of each tile.
template <int D, int NT> constexpr int blocks_per_iter() { return NT == 1 && D <= 128 ? 2 : 1; }
template <int D, int NT> constexpr int ring() { return D == 256 ? 3 : 4; }

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename T, int D, int NT>
cudaError_t mma_launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  constexpr int KB = blocks_per_iter<D, NT>(), NS = ring<D, NT>();
  return launch_kernel(true, mma_kernel<T, D, NT, KB, NS>, grid, kLanes * 32,
                       mma_smem<D, NT, NS>(), stream, p);
}

template <typename T, int D, int NT> bool take(KernelInfo *info, Launch *launch) {
  constexpr int KB = blocks_per_iter<D, NT>(), NS = ring<D, NT>();
  info->func = reinterpret_cast<const void *>(&mma_kernel<T, D, NT, KB, NS>);
  info->threads = kLanes * 32;
  info->warps = kLanes;
  info->stages = NS;
  info->smem = mma_smem<D, NT, NS>();
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
