// attn_fp4_warp.cu -- attention over the block-scaled 4-bit cache (fp4.cuh) on
// tensor cores, a warp being the worker: up to 16 query rows (8 at head_dim 256) a
// unit (sequence, KV head, row chunk).  q and out bfloat16 or float16.
//
// Each resident warp takes an equal share of the batch's blocks (the balanced
// partition) on its own: no barrier, no partner.  Against a CTA as the worker
// (attn_fp4_cta.cu) a piece costs its start and end once instead of four times,
// and nothing goes through shared memory but the copies: 40-head decode 70.5 us,
// CTAs 106.8; 2 contexts of 32768 and 65536 rows 29.7 and 38.0.
// Per group of KB blocks, keys on the MMA's M side and NT tiles of 8 query
// columns on N:
//   S^T = K Q^T,  online softmax over the keys (log2 units),  O^T += V^T P^T.
// The operands are those of the CTA kernel; for P.V a lane reads four keys' codes
// of 8 dims (word g + 8 h of the tile): 16 bytes.
//
// What bounds it: the 40-head decode step (32 contexts of 2048 rows, 377 MB of codes
// and scales) takes 70.5 us, 0.79 of the copy bandwidth: its loop spends 53 ns a
// block and SM where the bytes take 52, the rest is the call's start, the pieces'
// ends and the merge.  Per block 64 conversions, 64 f16 multiplies, 16 MMAs and
// about 110 other instructions.  Groups of four blocks share a wait, a vote and the
// copies' issue (one block: 96 us, two: 83 us, four: 77 us in an earlier form); two
// groups of four a ring (18 KB a warp, 12 warps an SM) hold more bytes in flight
// than the latency needs.  With two tiles groups of two leave registers to spare (16
// rows of 64 contexts of 2000 rows 51.7 us, groups of four 54.4), as they do at
// head_dim 256 (64 contexts of 1500 rows 31.9 us, one block 33.3).
#include "attn_fp4.cuh"

namespace pkv {
namespace fp4 {
namespace {

template <int D, int NT> struct WarpShape {
  static constexpr int KB = NT == 1 && D <= 128 ? 4 : 2;  // blocks of a group
  static constexpr int NS = 2;                            // groups in a ring
  // Compiled for 3 CTAs an SM, 2 where that would spill (two tiles at head_dim 128:
  // 16 rows of 64 contexts of 2000 rows 65.5 us at 3, 51.7 at 2).
  static constexpr int kMinCtas = D == 256 || (D == 128 && NT == 2) ? 2 : 3;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, (WarpShape<D, NT>::kMinCtas))
    warp_kernel(const AttnParams p) {
  pdl_wait();
  using TL = Tile<D>;
  using MM = Mma<__half>;
  using SH = WarpShape<D, NT>;
  constexpr int KB = SH::KB, NS = SH::NS;
  constexpr int NC = NT * 8;
  constexpr int PAIR = 2 * TL::kBytes;  // a block's key and value tiles
  constexpr int STAGE = KB * PAIR;
  constexpr int KS = D / 16;            // k-steps of the scores, m-tiles of O^T
  constexpr int WP = Lanes<D>::WP, KSP = Lanes<D>::KSP;
  static_assert((NS & (NS - 1)) == 0 && 2 * KB <= 32 && 32 % KB == 0, "ring, table chunks");

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ uint64_t bars[kWarps * NS];
  __shared__ int s_row[kWarps][NC], s_j[kWarps][NC];           // map_columns
  __shared__ __align__(16) uint8_t s_q[kWarps * D * 2];        // a query row in f16
  // the walk and the pieces: needed between pieces only, where registers are scarce
  __shared__ Pieces s_walk[kWarps];
  __shared__ Piece s_piece[kWarps][2];  // the one computed, the one after it

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t my_bars = smem_u32(&bars[warp * NS]);
  const uint32_t my_stages = smem_u32(smem) + warp * NS * STAGE;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(my_bars + 8 * s, 1);
    fence_mbar_init();
  }
  Piece wk;
  {
    Pieces walk;
    if (!walk.first(p, blockIdx.x * kWarps + warp, &wk)) return;
    if (lane == 0) {
      s_walk[warp] = walk;
      s_piece[warp][0] = wk;
    }
  }
  __syncwarp();

  // Copies.  The warp's ring runs on across pieces, group number t of all in
  // stage t % NS, so that the next piece's first copies fly while a piece is
  // finished.  Lanes 2u and 2u + 1 copy block u's key and value tile.  A block
  // id out of range is recorded, block 0 copied in its place, and from then on
  // every group of the piece looks its blocks up again.
  uint32_t turn = 0, turn_in = 0;  // groups computed and copied so far
  int i_in = 0, n_in = 0, nspan_in = 0;  // of the piece being copied: next group, groups, blocks
  const uint8_t *my_cache = nullptr;
  const int block_stride = p.num_kv_heads * TL::kBytes;
  int tab_cur = 0, tab_next = 0;
  bool ahead = false, more = false;     // the piece being copied is the next one; there is one
  bool bad_here = false, bad_next = false;  // bad blocks in the piece computed, in the next one
  auto groups_of = [&](int blocks) -> int { return (blocks + KB - 1) / KB; };
  auto load_entries = [&](int chunk32, const Piece &w) -> int {
    const int blk = chunk32 * 32 + lane;
    const int v = blk < nspan_in ? ld_keep(p.block_table +
                                           static_cast<int64_t>(w.b) * p.max_blocks_per_seq +
                                           w.blk_begin + blk)
                                 : 0;
    const bool bad = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
    if (bad) record_error(p.err, PKV_DEVERR_BLOCK_ID);
    const bool any = __any_sync(kFull, bad);
    if (ahead) bad_next |= any;
    else bad_here |= any;
    return bad ? 0 : v;
  };
  auto start_copies = [&](const Piece &w) {
    i_in = 0;
    nspan_in = max(w.blk_end - w.blk_begin, 0);
    n_in = groups_of(nspan_in);
    my_cache = static_cast<const uint8_t *>((lane & 1) ? p.v_cache : p.k_cache) +
               w.kvh * TL::kBytes;
    tab_cur = load_entries(0, w);
    tab_next = load_entries(1, w);
  };
  // A piece's query rows in registers, D / 32 dims a lane.  All are loaded
  // together, and for the first piece before the ring's copies, behind which
  // they would queue (5 us at the start of a call).
  constexpr int PER = D / 32, WORDS = PER / 2;
  uint32_t q_raw[NC][WORDS];
  auto load_rows = [&](const Piece &w) {
    const int n = rows_of(p, w.chunk);
    const T *base =
        static_cast<const T *>(p.q) + first_row(p, w.b, w.kvh) * D + lane * PER;
#pragma unroll
    for (int col = 0; col < NC; ++col) {
      if (col >= n) break;
      const uint32_t *src =
          reinterpret_cast<const uint32_t *>(base + s_row[warp][col] * static_cast<int64_t>(D));
#pragma unroll
      for (int e = 0; e < WORDS; ++e) q_raw[col][e] = __ldg(src + e);
    }
  };
  // Copy one more group, of the piece computed or of the one after it.
  auto copy_group = [&](int which) {
    if (i_in >= n_in) {
      if (ahead || !more) return;
      ahead = true;
      const Piece &w = s_piece[warp][which ^ 1];
      start_copies(w);
      if (i_in >= n_in) return;
    }
    const Piece &w = s_piece[warp][ahead ? which ^ 1 : which];
    if (i_in > 0 && (i_in * KB) % 32 == 0) {
      tab_cur = tab_next;
      tab_next = load_entries(i_in * KB / 32 + 1, w);
    }
    const uint32_t bar = my_bars + 8 * (turn_in % NS), tile = my_stages + (turn_in % NS) * STAGE;
    const int v = __shfl_sync(kFull, tab_cur, (i_in * KB + (lane >> 1)) & 31);
    const int cnt = min(KB, nspan_in - i_in * KB);
    if (lane == 0) mbar_arrive_expect_tx(bar, cnt * PAIR);
    if (lane < 2 * cnt)
      bulk_g2s(tile + lane * TL::kBytes, my_cache + static_cast<int64_t>(v) * block_stride,
               TL::kBytes, bar);
    ++i_in;
    ++turn_in;
  };
  map_columns(p, wk.chunk, NC, s_row[warp], s_j[warp]);
  load_rows(wk);
  start_copies(wk);

  // Byte offsets of this lane's pieces in a block's tiles.
  const uint32_t v_off = TL::kBytes + g * 64 + c * 16;
  const uint32_t vs_off = TL::kBytes + TL::kCodeBytes + (g >> 1) * 16 + c * 4;

  for (int which = 0;; which ^= 1) {
    // Piece s_piece[which] is computed (some of its copies are under way
    // already); the one after it is looked up.
    const Piece &cur = s_piece[warp][which];
    for (uint32_t k = turn_in - turn; k < NS && i_in < n_in; ++k) copy_group(which);
    {
      Pieces walk = s_walk[warp];
      more = walk.next(p, &wk);
      __syncwarp();
      if (more && lane == 0) {
        s_walk[warp] = walk;
        s_piece[warp][which ^ 1] = wk;
      }
      __syncwarp();
    }
    const int blk_begin = cur.blk_begin;
    const int nspan = max(cur.blk_end - blk_begin, 0);
    const int n_here = groups_of(nspan);
    const int mask_from = cur.L - p.num_queries;  // first row some column may not see

    // Q^T operand fragments (block_scores' order): the warp converts a row at a
    // time, the row's lanes pick their fragments up from shared memory.
    const int n_rows = rows_of(p, cur.chunk);
    const int64_t row0 = first_row(p, cur.b, cur.kvh);
    uint32_t qf[KS][NT][2];
    float colfac[NT][2];  // score factor of my two columns of each tile
    uint8_t *const mine = s_q + warp * D * 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      colfac[nt][0] = colfac[nt][1] = p.scale_log2;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[ks][nt][0] = qf[ks][nt][1] = 0u;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (nt * 8 + r >= n_rows) break;
        uint32_t(&f)[WORDS] = q_raw[nt * 8 + r];
        const float fac = convert_row<T>(f, p.scale_log2);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < WORDS; ++k)
          reinterpret_cast<uint32_t *>(mine + lane * (2 * PER))[k] = f[k];
        __syncwarp();
        if (g == r) {
#pragma unroll
          for (int k2 = 0; k2 < KS / 2; ++k2) {
            const int pn = (2 * k2) / KSP, w = (2 * k2) % KSP / 2;
            const uint4 x =
                *reinterpret_cast<const uint4 *>(mine + (pn * TL::kPanel + (c * WP + w) * 8) * 2);
            qf[2 * k2][nt][0] = x.x;
            qf[2 * k2][nt][1] = x.y;
            qf[2 * k2 + 1][nt][0] = x.z;
            qf[2 * k2 + 1][nt][1] = x.w;
          }
        }
        if (r == 2 * c) colfac[nt][0] = fac;
        if (r == 2 * c + 1) colfac[nt][1] = fac;
      }
    }
    auto q_frag = [&](int ks, int nt, int, uint32_t &b0, uint32_t &b1) {
      b0 = qf[ks][nt][0];
      b1 = qf[ks][nt][1];
    };

    // Online-softmax state, per column of mine: the reference, a raw score
    // (kNothing until a row is seen), and the sum.  Weights are 2^((s - m) factor):
    // the difference first, so that the largest score has weight 1 however
    // large it is.
    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNothing;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }

    for (int i = 0; i < n_here; ++i, ++turn) {
      const uint32_t bar = my_bars + 8 * (turn % NS);
      const uint32_t tile = my_stages + (turn % NS) * STAGE;
      // one decision per warp: its lanes then agree on every later shuffle
      if (!__all_sync(kFull, mbar_wait_bounded(bar, (turn / NS) & 1))) {
        // The copies in flight get a bounded chance to land before their memory
        // is given up.
        if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        for (; turn != turn_in; ++turn)
          mbar_wait_bounded(my_bars + 8 * (turn % NS), (turn / NS) & 1);
        return;
      }
      const int blk0 = i * KB;  // of the piece
      const int key0 = (blk_begin + blk0) * kBlockSize;
      // An edge group has rows that some column may not see, perhaps a bad
      // block, or fewer blocks than KB (then the rest of the stage is computed
      // on whatever it holds, and masked out).  The value scales of rows that
      // are not there become 0: their codes are finite whatever they are, so
      // they add nothing.
      const bool edge = bad_here || key0 + KB * kBlockSize > mask_from || blk0 + KB > nspan;
      uint32_t gone = 0;  // bit u: block u is not there
      if (edge) {
#pragma unroll
        for (int u = 0; u < KB; ++u) {
          bool none = blk0 + u >= nspan;
          if (bad_here && !none) {
            const int v =
                __ldg(p.block_table + static_cast<int64_t>(cur.b) * p.max_blocks_per_seq +
                      blk_begin + blk0 + u);
            none = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
          }
          gone |= none ? 1u << u : 0u;
          clear_value_scales<D>(tile + u * PAIR, none ? 0 : cur.L - key0 - u * kBlockSize, lane);
        }
        // these writes come before the next copy into the stage
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      float sc[KB][NT][4];
#pragma unroll
      for (int u = 0; u < KB; ++u)
        block_scores<D, NT, 1>(reinterpret_cast<float(&)[1][NT][4]>(sc[u]), tile + u * PAIR, g, c,
                               q_frag);
      if (edge) {
        const int kk = key_of(g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * c + e;
            const int j = s_j[warp][col];
            const int lim = mask_from + 1 + j;
            unsigned long long tm = 0;
            if (p.tree_mask != nullptr && col < n_rows)
              tm = __ldg(p.tree_mask + cur.b * p.mask_stride + j);
#pragma unroll
            for (int u = 0; u < KB; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (!key_visible(p, key0 + u * kBlockSize + kk + 2 * r, cur.L, (gone >> u) & 1u,
                                 lim, tm))
                  sc[u][nt][e + 2 * r] = -INFINITY;
          }
      }
      // Online softmax against a per-column reference, raised to the exact
      // running maximum (rescaling l and O) only when a score exceeds it by
      // more than the slack; O / l does not depend on the reference.  A NaN
      // score never raises it and reaches O through its weight.
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
          for (int u = 1; u < KB; ++u) t = fmaxf(t, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
          above |= (t - m[nt][e]) * colfac[nt][e] > kSlack;
        }
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
            const float m_new = fmaxf(m[nt][e], mx - __fdividef(kHead, colfac[nt][e]));
            const float corr = ex2((m[nt][e] - m_new) * colfac[nt][e]);
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
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 w = lds128(tile + u * PAIR + v_off + h * 512);
          const uint32_t sw = lds32(tile + u * PAIR + vs_off + h * 64);
          const uint32_t s01 = e4m3x2_to_f16(sw), s23 = e4m3x2_to_f16(sw >> 16);
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
      // (turn still counts this group: its stage is the one that is free)
      copy_group(which);
    }

    // The piece's end.
    float lse[NT][2];  // the reference in log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        l[nt][e] = v;
        lse[nt][e] = m[nt][e] * colfac[nt][e];
      }
    // (The next kernel is let in only here: earlier, its waiting CTAs would take
    // the places of this grid's last ones.)
    if (!more) pdl_launch_dependents();
    // The piece's partial and its log-sum-exp (a NaN sum as +inf, which makes the
    // merged row NaN).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = nt * 8 + 2 * c + e;
        if (col >= n_rows) continue;
        const float sum = l[nt][e];
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int64_t at = static_cast<int64_t>(cur.item) * p.rows_per_cta + col;
        float *dst = p.part_o + at * D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
          *reinterpret_cast<float2 *>(dst + 8 * (g + 8 * (mt >> 2)) + 2 * (mt & 3)) =
              make_float2(o[mt][nt][e] * inv, o[mt][nt][e + 2] * inv);
        if (g == 0)
          p.part_lse[at] = sum > 0.f ? lse[nt][e] + __log2f(sum)
                                     : (sum == 0.f ? -INFINITY : INFINITY);
      }
    if (!more) return;
    if (!ahead) {  // (the piece had no group)
      ahead = true;
      start_copies(s_piece[warp][which ^ 1]);
    }
    ahead = false;
    bad_here = bad_next;
    bad_next = false;
    const Piece &nx = s_piece[warp][which ^ 1];
    if (p.row_chunks > 1) map_columns(p, nx.chunk, NC, s_row[warp], s_j[warp]);
    load_rows(nx);
  }
}

template <int D, int NT> constexpr size_t warp_smem() {
  using SH = WarpShape<D, NT>;
  return size_t(kWarps) * SH::NS * SH::KB * 2 * Tile<D>::kBytes + 128;
}

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename T, int D, int NT>
cudaError_t launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  return launch_kernel(true, warp_kernel<T, D, NT>, grid, kWarps * 32, warp_smem<D, NT>(), stream,
                       p);
}

template <typename T, int D, int NT> bool take(KernelInfo *info, Launch *launch) {
  using SH = WarpShape<D, NT>;
  info->func = reinterpret_cast<const void *>(&warp_kernel<T, D, NT>);
  info->threads = kWarps * 32;
  info->warps = kWarps;
  info->stages = SH::NS;
  info->smem = warp_smem<D, NT>();
  info->warp_tiles = NT;
  info->blocks_per_iter = SH::KB;
  *launch = &launch_t<T, D, NT>;
  return true;
}

template <typename T> bool pick_d(int D, int nt, KernelInfo *info, Launch *launch) {
  switch (D) {
    case 64:
      return nt == 1 ? take<T, 64, 1>(info, launch) : nt == 2 && take<T, 64, 2>(info, launch);
    case 128:
      return nt == 1 ? take<T, 128, 1>(info, launch) : nt == 2 && take<T, 128, 2>(info, launch);
    case 256: return nt == 1 && take<T, 256, 1>(info, launch);
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

int warp_fp4_max_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }

bool warp_fp4_kernel_info(pkv_dtype q_dtype, int head_dim, int tiles, KernelInfo *info) {
  fp4::Launch launch = nullptr;
  return fp4::pick(q_dtype, head_dim, tiles, info, &launch);
}

cudaError_t warp_fp4_launch(pkv_dtype q_dtype, int head_dim, int tiles, const AttnParams &p,
                            dim3 grid, cudaStream_t stream) {
  KernelInfo info;
  fp4::Launch launch = nullptr;
  if (!fp4::pick(q_dtype, head_dim, tiles, &info, &launch)) return cudaErrorInvalidValue;
  return launch(p, grid, stream);
}

}  // namespace pkv
