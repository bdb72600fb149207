// attn_fp4_cta.cu -- attention over the block-scaled 4-bit cache (fp4.cuh) on
// tensor cores, a CTA being the worker: every split plan, float32 queries, and up
// to 64 query rows in one pass (32 at head_dim 256; float32: 48 and 16).
//
// Per group of 4 UW blocks (UW = 2 or 1), keys on the MMA's M side and NT tiles of
// 8 query columns on N:
//   warp w       S^T = K Q^T of its UW blocks, their softmax weights P^T (online
//                softmax, log2 units), which go to shared memory as operand
//                fragments;
//   one barrier
//   every warp   O^T += V^T P^T over all the group's blocks, for its quarter of the
//                dims.
// So every code is widened once in the CTA, and a warp's O^T is D / 64 m-tiles
// high: with 40 rows 40 registers a lane instead of 160, which leaves room for
// the warps that hide the conversions behind the MMAs of others.  (With a warp
// computing whole blocks for all columns, 20 and 40 rows took 51 and 90 us on the
// steps below.)  P^T is double-buffered and the reference of the online softmax is
// the CTA's, so the fast path needs no second barrier.
//
// Codes are widened to f16 pairs by the conversion unit and multiplied by
// their block scale there: code * scale has at most 6 significant bits, so the
// operands are exact; 16-bit q enters as f16 (convert_row), the weights as f16
// (2^-11 relative, below the output's own rounding); sums are float32.  A float32
// q row and its weights enter as sums of two f16 parts (split_pair: to 2^-24, what
// float32 itself rounds by), two MMAs for one; the small part of the scores, and each
// group's P.V, have a float32 sum of their own, the MMA's sums being rounded less
// well than float32's.  Against the CUDA-core kernel: GQA decode 267 -> 69 us, a ten-node
// tree 654 -> 85 (with three parts 78 and 137).
//
// The order of keys and dims inside the MMAs is free, and chosen so that no
// operand is shuffled between lanes: lane (g, c) = (lane / 4, lane % 4) of the
// scores holds keys 4 (g / 2) + g % 2 and the one two after it, and movmatrix
// then leaves it the weights of keys 4c .. 4c + 3 of a column; for P.V it reads
// those keys' codes of its D / 32 dims, and a nibble merge pairs two keys' codes
// of a dim in one byte, which converts to one operand register.
//
// What bounds it (D = 128, 16 sequences of 512 to 8192 rows, 8 KV heads, 81 MB): a
// block costs an SM 116 ns with 20 rows (41 us for the step) and 175 ns with 40
// (61 us), where its bytes take 52.  That is the time of its MMAs (16 a tile; one
// every two clocks) and of issuing the other instructions (370 and 560), added up:
// two or three CTAs an SM, one or two blocks a warp and group, rings of two to four
// groups all come within 2 %.  About 14 us a call are outside that loop: the
// first loads' chain, a piece's start and end, the merge.
#include "attn_fp4.cuh"

namespace pkv {
namespace fp4 {
namespace {

template <typename T, int D, int NT> struct CtaShape {
  static constexpr bool kF32 = std::is_same<T, float>::value;
  static constexpr int kParts = kF32 ? kF32Parts : 1;  // f16 parts of a query element, a weight
  // Blocks of a group that are a warp's: two, while their scores fit in registers
  // (20 rows 41.0 us, with one 42.6; 40 rows 61.7 both ways; float32, 20 rows, two
  // CTAs an SM with two 42.5, three with one 41.5).
  static constexpr int UW = NT <= (kF32 ? 2 : 4) ? 2 : 1;
  static constexpr int kGroup = UW * kWarps;               // blocks of a group
  static constexpr int NS = UW == 2 ? 2 : 4;               // groups in the ring
  static constexpr bool kRegQ = NT <= 2 && D <= 128 && !kF32;  // Q^T fragments in registers
  // Blocks whose scores are computed together, each Q^T fragment loaded once (20
  // rows 41.0 us, one at a time 44.3).
  static constexpr int UB = !kRegQ && NT <= 4 && D <= 128 ? UW : 1;
  static constexpr bool kRegFac = NT <= 4;    // score factors in registers
  // resident CTAs it is compiled for
  static constexpr int kMinCtas = D == 256 ? 1 : (NT >= (kF32 ? 4 : 6) ? 2 : 3);
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, (CtaShape<T, D, NT>::kMinCtas))
    cta_kernel(const AttnParams p) {
  pdl_wait();
  using TL = Tile<D>;
  using MM = Mma<__half>;
  using SH = CtaShape<T, D, NT>;
  constexpr int NS = SH::NS, UW = SH::UW, kGroup = SH::kGroup, PARTS = SH::kParts;
  constexpr bool F32 = SH::kF32;
  constexpr bool QR = SH::kRegQ;
  constexpr int NC = NT * 8;
  constexpr int PAIR = 2 * TL::kBytes;  // a block's key and value tiles
  constexpr int STAGE = kGroup * PAIR;
  constexpr int KS = D / 16;            // k-steps of the scores
  constexpr int MT = D / 64;            // m-tiles of O^T of a warp
  constexpr int KSP = Lanes<D>::KSP, WP = Lanes<D>::WP;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  const uint32_t ring = smem_u32(smem);
  const uint32_t q_smem = ring + NS * STAGE;           // [part][ks][nt][lane] fragments of Q^T
  constexpr int P_BLOCK = PARTS * NT * 256;
  uint8_t *const p_frags = smem + NS * STAGE + PARTS * KS * NT * 256;  // [2][block][part][nt][lane] of P^T
  __shared__ uint64_t bars[NS];
  __shared__ __align__(8) float s_fac[NC];             // score factor per column
  __shared__ int s_row[kWarps][NC], s_j[kWarps][NC];   // map_columns
  __shared__ float s_top[kWarps][NC], s_sum[kWarps][NC];
  __shared__ Piece s_piece[2];  // the piece computed and the one after it
  __shared__ int s_more, s_dead[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t bar0 = smem_u32(bars);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    s_dead[0] = s_dead[1] = 0;
  }
  Pieces walk;  // (goes on in warp 0 only)
  Piece wk;
  if (!walk.first(p, blockIdx.x, &wk)) return;  // (the whole CTA agrees)
  if (threadIdx.x == 0) s_piece[0] = wk;
  for (int k = threadIdx.x; k < PARTS * KS * NT * 32; k += kWarps * 32)  // columns without a row: 0
    if (k / 32 % NT * 8 + (k & 31) / 4 >= p.rows_per_cta)
      asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(q_smem + k * 8), "r"(0) : "memory");

  // A piece's query rows, every fourth by this warp, D / 32 dims a lane.  For
  // the first piece they are loaded before the ring's copies, behind which they
  // would queue (5 us at the start of a call).
  constexpr int PER = D / 32, WORDS = F32 ? PER : PER / 2, Q_ROWS = NC / kWarps;
  uint32_t q_raw[Q_ROWS][WORDS];
  auto load_rows = [&](const Piece &w) {
    const int n = rows_of(p, w.chunk);
    const T *base =
        static_cast<const T *>(p.q) + first_row(p, w.b, w.kvh) * D + lane * PER;
#pragma unroll
    for (int k = 0; k < Q_ROWS; ++k) {
      const int col = k * kWarps + warp;
      if (col >= n) break;
      const uint32_t *src =
          reinterpret_cast<const uint32_t *>(base + s_row[warp][col] * static_cast<int64_t>(D));
#pragma unroll
      for (int e = 0; e < WORDS; ++e) q_raw[k][e] = __ldg(src + e);
    }
  };
  map_columns(p, wk.chunk, NC, s_row[warp], s_j[warp]);
  load_rows(wk);
  __syncthreads();  // barriers, s_piece

  // Copies.  The warps take turns: warp t % 4 issues group number t of all, lanes
  // 2u and 2u + 1 the key and value tile of its block u; the ring runs on across
  // pieces, group t in stage t % NS.  A block id out of range is recorded, block 0
  // copied in its place, and from then on every block of the piece is looked up
  // again.
  uint32_t turn = 0, turn_in = 0;        // groups computed and copied so far
  int i_in = 0, n_in = 0, nspan_in = 0;  // of the piece being copied: next group, groups, blocks
  const uint8_t *my_cache = nullptr;
  const int block_stride = p.num_kv_heads * TL::kBytes;
  int tab_cur = 0, tab_next = 0;
  bool ahead = false, more = false;  // the piece being copied is the next one; there is one
  bool bad_here = false, bad_next = false;
  auto load_entries = [&](int chunk32, const Piece &w) -> int {
    const int blk = chunk32 * 32 + lane;
    const int v = blk < nspan_in ? ld_keep(p.block_table +
                                           static_cast<int64_t>(w.b) * p.max_blocks_per_seq +
                                           w.blk_begin + blk)
                                 : 0;
    const bool bad = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
    if (bad && warp == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID);
    const bool any = __any_sync(kFull, bad);
    if (ahead) bad_next |= any;
    else bad_here |= any;
    return bad ? 0 : v;
  };
  auto start_copies = [&](const Piece &w) {
    i_in = 0;
    nspan_in = max(w.blk_end - w.blk_begin, 0);
    n_in = (nspan_in + kGroup - 1) / kGroup;
    my_cache = static_cast<const uint8_t *>((lane & 1) ? p.v_cache : p.k_cache) +
               w.kvh * TL::kBytes;
    tab_cur = load_entries(0, w);
    tab_next = load_entries(1, w);
  };
  auto copy_group = [&](int which) {
    if (i_in >= n_in) {
      if (ahead || !more) return;
      ahead = true;
      start_copies(s_piece[which ^ 1]);
      if (i_in >= n_in) return;
    }
    if (i_in * kGroup % 32 == 0 && i_in > 0) {
      tab_cur = tab_next;
      tab_next = load_entries(i_in * kGroup / 32 + 1, s_piece[ahead ? which ^ 1 : which]);
    }
    if (turn_in % kWarps == static_cast<uint32_t>(warp)) {
      const uint32_t s = turn_in % NS;
      const int v = __shfl_sync(kFull, tab_cur, (i_in * kGroup + (lane >> 1)) & 31);
      const int cnt = min(kGroup, nspan_in - i_in * kGroup);
      if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * s, cnt * PAIR);
      if (lane < 2 * cnt)
        bulk_g2s(ring + s * STAGE + lane * TL::kBytes,
                 my_cache + static_cast<int64_t>(v) * block_stride, TL::kBytes, bar0 + 8 * s);
    }
    ++i_in;
    ++turn_in;
  };
  start_copies(wk);

  // This lane's dims of the values: D / 32 consecutive ones, part of a word.
  const int dim0 = warp * (D / 4) + g * (D / 32);
  const uint32_t v_off = TL::kBytes + (dim0 / 8) * 64 + c * 16;
  const uint32_t vs_off = TL::kBytes + TL::kCodeBytes + (dim0 / 16) * 16 + c * 4;
  const int v_byte = dim0 % 8 / 2;  // of its codes in a word

  for (int which = 0;; which ^= 1) {
    const Piece &cur = s_piece[which];
    for (uint32_t k = turn_in - turn; k < NS && i_in < n_in; ++k) copy_group(which);
    // Q^T operand fragments to shared memory; warp 0 looks up the next piece.
    const int n_rows = rows_of(p, cur.chunk);
    const int64_t row0 = first_row(p, cur.b, cur.kvh);
#pragma unroll
    for (int k = 0; k < Q_ROWS; ++k) {
      const int col = k * kWarps + warp;
      if (col >= n_rows) break;
      uint32_t parts[PARTS][PER / 2];
      float fac;
      if constexpr (F32) {
        fac = split_row<PER>(q_raw[k], parts, p.scale_log2);
      } else {
        fac = convert_row<T>(q_raw[k], p.scale_log2);
#pragma unroll
        for (int e = 0; e < WORDS; ++e) parts[0][e] = q_raw[k][e];
      }
      constexpr int HALVES = PER > 4 ? PER / 4 : 1;  // fragments of four dims (or a half)
#pragma unroll
      for (int e = 0; e < HALVES; ++e) {
        const int d = lane * PER + 4 * e, in = d % TL::kPanel;
        const int ks = d / TL::kPanel * KSP + in % (8 * WP) / 4, cq = in / (8 * WP);
        const uint32_t at =
            q_smem + (ks * NT + (col >> 3)) * 256 + ((col & 7) * 4 + cq) * 8 + d % 4 * 2;
        constexpr int PAIRS = PER / 2 / HALVES;
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int x = 0; x < PAIRS; ++x)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + part * (KS * NT * 256) + 4 * x),
                         "r"(parts[part][e * PAIRS + x])
                         : "memory");
      }
      if (lane == 0) s_fac[col] = fac;
    }
    if (lane == 0)
      for (int col = n_rows + warp; col < NC; col += kWarps) s_fac[col] = p.scale_log2;
    if (warp == 0) {
      const bool any = walk.next(p, &wk);
      if (lane == 0) {
        s_more = any;
        if (any) s_piece[which ^ 1] = wk;
      }
    }
    __syncthreads();
    more = s_more != 0;
    uint32_t qf[QR ? KS : 1][QR ? NT : 1][2];
    if constexpr (QR) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 x = lds64(q_smem + (ks * NT + nt) * 256 + lane * 8);
          qf[ks][nt][0] = x.x;
          qf[ks][nt][1] = x.y;
        }
    }
    auto q_frag = [&](int ks, int nt, int part, uint32_t &b0, uint32_t &b1) {
      if constexpr (QR) {
        b0 = qf[ks][nt][0];
        b1 = qf[ks][nt][1];
      } else {
        const uint2 x = lds64(q_smem + ((part * KS + ks) * NT + nt) * 256 + lane * 8);
        b0 = x.x;
        b1 = x.y;
      }
    };

    float fac[NT][2];  // score factors of my two columns of each tile
    auto load_factors = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 f = *reinterpret_cast<const float2 *>(&s_fac[nt * 8 + 2 * c]);
        fac[nt][0] = f.x;
        fac[nt][1] = f.y;
      }
    };
    if (SH::kRegFac) load_factors();

    const int blk_begin = cur.blk_begin;
    const int nspan = max(cur.blk_end - blk_begin, 0);
    const int n_here = (nspan + kGroup - 1) / kGroup;
    const int mask_from = cur.L - p.num_queries;  // first row some column may not see
    // This warp's first group at an edge: with rows that some column may not see,
    // or blocks that are not there.
    int edge_from = min(mask_from / kBlockSize - blk_begin, nspan) - (warp + 1) * UW;
    edge_from = mask_from < 0 || edge_from < 0 ? 0 : edge_from / kGroup + 1;
    if (bad_here) edge_from = 0;

    // Per column of mine: the CTA's reference, a raw score (kNothing, below every
    // score, until a row is seen), and this warp's part of the sum.  Weights are
    // 2^((s - m) factor): the difference first, so that the largest score has
    // weight 1 however large it is.
    float o[MT][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNothing;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
    }

    for (int i = 0; i < n_here; ++i, ++turn) {
      const uint32_t stage = ring + (turn % NS) * STAGE;
      const bool late =
          !__all_sync(kFull, mbar_wait_bounded(bar0 + 8 * (turn % NS), (turn / NS) & 1));
      if (late && lane == 0) {
        record_error(p.err, PKV_DEVERR_TIMEOUT);
        s_dead[turn & 1] = 1;
      }
      // This warp's blocks.
      const int blk = i * kGroup + warp * UW;
      const int key0 = (blk_begin + blk) * kBlockSize;
      const uint32_t tile = stage + warp * UW * PAIR;
      const bool edge = i >= edge_from || bad_here;
      uint32_t gone = 0;  // bit u: block u is not there
      if (edge) {
#pragma unroll
        for (int u = 0; u < UW; ++u) {
          bool none = blk + u >= nspan;
          if (bad_here && !none) {
            const int v =
                __ldg(p.block_table + static_cast<int64_t>(cur.b) * p.max_blocks_per_seq +
                      blk_begin + blk + u);
            none = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
          }
          gone |= none ? 1u << u : 0u;
          clear_value_scales<D>(tile + u * PAIR, none ? 0 : cur.L - key0 - u * kBlockSize, lane);
        }
        // (these writes come before the next copy into the stage)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      constexpr int UB = SH::UB;
      float sc[UW][NT][4];
      if (UW == 1 || blk < nspan) {
#pragma unroll
        for (int u = 0; u < UW; u += UB)
          block_scores<D, NT, UB, PARTS>(reinterpret_cast<float(&)[UB][NT][4]>(sc[u]),
                                         tile + u * PAIR, g, c, q_frag);
      }
      if (edge) {
        const int kk = key_of(g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * c + e;
            const int j = s_j[warp][col];
            unsigned long long tm = 0;
            if (p.tree_mask != nullptr && col < n_rows)
              tm = __ldg(p.tree_mask + cur.b * p.mask_stride + j);
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (!key_visible(p, key0 + u * kBlockSize + kk + 2 * r, cur.L, (gone >> u) & 1u,
                                 mask_from + 1 + j, tm))
                  sc[u][nt][e + 2 * r] = -INFINITY;
          }
      }
      if (!SH::kRegFac) load_factors();
      // Weights against the present reference; where one exceeds the slack the
      // whole CTA raises the reference and they are computed again.  (A NaN score
      // never raises it, and reaches O through its weight.)
      float sum[NT][2];
      uint8_t *const p_at =
          p_frags + (turn & 1) * (kGroup * P_BLOCK) + warp * UW * P_BLOCK + lane * 8;
      float heaviest = 0.f;
      auto weights = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
          for (int u = 0; u < UW; ++u) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = ex2((sc[u][nt][e] - m[nt][e & 1]) * fac[nt][e & 1]);
            sum[nt][0] += w[0] + w[2];
            sum[nt][1] += w[1] + w[3];
            heaviest = fmaxf(heaviest, fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])));
            if constexpr (F32) {
              uint32_t a[PARTS], b[PARTS];
              split_pair(w[0], w[1], a);
              split_pair(w[2], w[3], b);
#pragma unroll
              for (int k = 0; k < PARTS; ++k)
                *reinterpret_cast<uint2 *>(p_at + u * P_BLOCK + (k * NT + nt) * 256) =
                    make_uint2(movm_t(a[k]), movm_t(b[k]));
            } else {
              *reinterpret_cast<uint2 *>(p_at + u * P_BLOCK + nt * 256) =
                  make_uint2(movm_t(MM::pack(w[0], w[1])), movm_t(MM::pack(w[2], w[3])));
            }
          }
        }
      };
      auto top_of = [&](int nt, int e) -> float {
        float t = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
        for (int u = 1; u < UW; ++u) t = fmaxf(t, fmaxf(sc[u][nt][e], sc[u][nt][e + 2]));
        return t;
      };
      weights();
      if (__syncthreads_or(heaviest > kHeaviest || late)) {
        if (s_dead[turn & 1]) {  // (written before the barrier: the whole CTA agrees)
          // a copy never came: those in flight get a bounded chance to land
          // before their memory is given up
          for (; turn != turn_in; ++turn)
            mbar_wait_bounded(bar0 + 8 * (turn % NS), (turn / NS) & 1);
          return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = top_of(nt, e);
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
            if (g == 0) s_top[warp][nt * 8 + 2 * c + e] = mx;
          }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * c + e;
            float top = s_top[0][col];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_top[w][col]);
            const float m_new = fmaxf(m[nt][e], top - __fdividef(kHead, fac[nt][e]));
            const float corr = ex2((m[nt][e] - m_new) * fac[nt][e]);
            l[nt][e] *= corr;
            m[nt][e] = m_new;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[j][nt][e] *= corr;
              o[j][nt][e + 2] *= corr;
            }
          }
        weights();
        __syncthreads();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] += sum[nt][0];
        l[nt][1] += sum[nt][1];
      }
      // Every warp has passed the barrier, so the group before is done with:
      // its stage takes the next copies.  (NS groups in flight and this one.)
      if (turn_in - turn < NS) copy_group(which);
      // O^T += V^T P^T over the group, for this warp's dims.
      const uint8_t *const p_in = p_frags + (turn & 1) * (kGroup * P_BLOCK) + lane * 8;
      // (float32: the group's products have a sum of their own, so that a long
      // context is not a long chain of the MMA's roundings)
      float part_sum[F32 ? MT : 1][F32 ? NT : 1][4];
      auto add_block = [&](int u) {
        constexpr uint32_t LOW = 0x0f0f0f0fu;
        const uint4 w = lds128(stage + u * PAIR + v_off);
        const uint32_t sw = lds32(stage + u * PAIR + vs_off);
        const uint32_t s01 = e4m3x2_to_f16(sw), s23 = e4m3x2_to_f16(sw >> 16);
        uint32_t a[MT][4];
        if constexpr (MT == 4) {
          uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, keys (0, 1), (2, 3)
          e2m1x8_to_f16((w.x & LOW) | ((w.y << 4) & ~LOW), e01);
          e2m1x8_to_f16(((w.x >> 4) & LOW) | (w.y & ~LOW), o01);
          e2m1x8_to_f16((w.z & LOW) | ((w.w << 4) & ~LOW), e23);
          e2m1x8_to_f16(((w.z >> 4) & LOW) | (w.w & ~LOW), o23);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            a[j][0] = mul2(e01[j], s01);
            a[j][1] = mul2(o01[j], s01);
            a[j][2] = mul2(e23[j], s23);
            a[j][3] = mul2(o23[j], s23);
          }
        } else {
          // bytes of keys (0 | 2) in x and (1 | 3) in y: MT of each
          const uint32_t sel = MT == 2 ? (v_byte ? 0x7632u : 0x5410u)
                                       : static_cast<uint32_t>(v_byte | (v_byte + 4) << 4);
          const uint32_t x = prmt2(w.x, w.z, sel), y = prmt2(w.y, w.w, sel);
          uint32_t ev[4], od[4];  // even and odd dims: keys (0, 1) of each m-tile, then (2, 3)
          e2m1x8_to_f16((x & LOW) | ((y << 4) & ~LOW), ev);
          e2m1x8_to_f16(((x >> 4) & LOW) | (y & ~LOW), od);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            a[j][0] = mul2(ev[j], s01);
            a[j][1] = mul2(od[j], s01);
            a[j][2] = mul2(ev[MT + j], s23);
            a[j][3] = mul2(od[MT + j], s23);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int part = PARTS - 1; part >= 0; --part) {
            const uint2 b =
                *reinterpret_cast<const uint2 *>(p_in + u * P_BLOCK + (part * NT + nt) * 256);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              if constexpr (F32) {
                if (u == 0 && part == PARTS - 1) mma_first(part_sum[j][nt], a[j], b.x, b.y);
                else MM::run(part_sum[j][nt], a[j], b.x, b.y);
              } else {
                MM::run(o[j][nt], a[j], b.x, b.y);
              }
            }
          }
        }
      };
#pragma unroll
      for (int u = 0; u < 4; ++u) add_block(u);
      if constexpr (kGroup == 8)
        if (nspan - i * kGroup > 4) {  // (a piece's last group may be half empty)
#pragma unroll
          for (int u = 4; u < 8; ++u) add_block(u);
        }
      if constexpr (F32) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][nt][e] += part_sum[j][nt][e];
      }
    }

    // The piece's end: the warps' sums meet, and each writes its dims of the
    // rows -- normalised to the output where nothing else is to be merged, else
    // the piece's partial and its log-sum-exp (a NaN sum as +inf, which makes the
    // merged row NaN).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        if (g == 0) s_sum[warp][nt * 8 + 2 * c + e] = v;
      }
    __syncthreads();
    // (The next kernel is let in only here: earlier, its waiting CTAs would take
    // the places of this grid's last ones.)
    if (!more) pdl_launch_dependents();
    const bool direct = p.split_target == 0 && p.num_splits == 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = nt * 8 + 2 * c + e;
        if (col >= n_rows) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_sum[w][col];
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int64_t row = row0 + s_row[warp][col];
        if (direct) {
          T *dst = static_cast<T *>(p.out) + row * D + dim0;
          const float os = inv * p.out_scale;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const float x = o[j][nt][e] * os, y = o[j][nt][e + 2] * os;
            if constexpr (F32) reinterpret_cast<float2 *>(dst)[j] = make_float2(x, y);
            else reinterpret_cast<uint32_t *>(dst)[j] = Mma<T>::pack(x, y);
          }
        } else {
          const int64_t at = p.split_target == 0
                                 ? row * p.num_splits + cur.split
                                 : static_cast<int64_t>(cur.item) * p.rows_per_cta + col;
          float2 *dst = reinterpret_cast<float2 *>(p.part_o + at * D + dim0);
#pragma unroll
          for (int j = 0; j < MT; ++j)
            dst[j] = make_float2(o[j][nt][e] * inv, o[j][nt][e + 2] * inv);
          if (warp == 0 && g == 0)
            p.part_lse[at] = sum > 0.f ? m[nt][e] * s_fac[col] + __log2f(sum)
                                       : (sum == 0.f ? -INFINITY : INFINITY);
        }
      }
    if (!more) return;
    if (!ahead) {  // (the piece had no group)
      ahead = true;
      start_copies(s_piece[which ^ 1]);
    }
    ahead = false;
    bad_here = bad_next;
    bad_next = false;
    const Piece &nx = s_piece[which ^ 1];
    if (p.row_chunks > 1) map_columns(p, nx.chunk, NC, s_row[warp], s_j[warp]);
    load_rows(nx);
    // s_fac and the Q^T fragments are the finished piece's until every warp has
    // read the former for its log-sum-exps
    __syncthreads();
  }
}

template <typename T, int D, int NT> constexpr size_t cta_smem() {
  using SH = CtaShape<T, D, NT>;
  constexpr size_t stages = size_t(SH::NS) * SH::kGroup * 2 * Tile<D>::kBytes;
  return stages + size_t(SH::kParts) * NT * 256 * (D / 16 + 2 * SH::kGroup) + 128;
}

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename T, int D, int NT>
cudaError_t launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  return launch_kernel(true, cta_kernel<T, D, NT>, grid, kWarps * 32, cta_smem<T, D, NT>(), stream,
                       p);
}

template <typename T, int D, int NT> bool take(KernelInfo *info, Launch *launch) {
  info->func = reinterpret_cast<const void *>(&cta_kernel<T, D, NT>);
  info->threads = kWarps * 32;
  info->warps = kWarps;
  info->stages = CtaShape<T, D, NT>::NS;
  info->smem = cta_smem<T, D, NT>();
  info->warp_tiles = NT;
  info->blocks_per_iter = CtaShape<T, D, NT>::kGroup;
  *launch = &launch_t<T, D, NT>;
  return true;
}

// Tiles built: 1 to 6 and 8 at head_dim <= 128, 1, 2 and 4 at 256 (float32: 1 to 6,
// 1 and 2); another number takes the next one.  float32: 40 rows in one pass 84.5 us,
// in two 103; 48 rows 70.4 and 73.6.
template <typename T, int D> bool pick_nt(int nt, KernelInfo *info, Launch *launch) {
  if constexpr (std::is_same<T, float>::value && D <= 128) {
    return nt == 1   ? take<T, D, 1>(info, launch)
           : nt == 2 ? take<T, D, 2>(info, launch)
           : nt == 3 ? take<T, D, 3>(info, launch)
           : nt == 4 ? take<T, D, 4>(info, launch)
           : nt == 5 ? take<T, D, 5>(info, launch)
           : nt == 6 ? take<T, D, 6>(info, launch)
                     : false;
  } else if constexpr (std::is_same<T, float>::value) {
    return nt == 1 ? take<T, D, 1>(info, launch) : nt == 2 && take<T, D, 2>(info, launch);
  } else if constexpr (D == 256) {
    return nt == 1   ? take<T, D, 1>(info, launch)
           : nt == 2 ? take<T, D, 2>(info, launch)
           : nt <= 4 ? take<T, D, 4>(info, launch)
                     : false;
  } else {
    switch (nt) {
      case 1: return take<T, D, 1>(info, launch);
      case 2: return take<T, D, 2>(info, launch);
      case 3: return take<T, D, 3>(info, launch);
      case 4: return take<T, D, 4>(info, launch);
      case 5: return take<T, D, 5>(info, launch);
      case 6: return take<T, D, 6>(info, launch);
      case 7:
      case 8: return take<T, D, 8>(info, launch);
      default: return false;
    }
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
    case PKV_F32: return pick_d<float>(D, nt, info, launch);
    default: return false;
  }
}

}  // namespace
}  // namespace fp4

int cta_fp4_max_tiles(pkv_dtype q_dtype, int head_dim) {
  const int most = q_dtype == PKV_F32 ? 6 : 8;
  return head_dim <= 128 ? most : q_dtype == PKV_F32 ? 2 : 4;
}

bool cta_fp4_kernel_info(pkv_dtype q_dtype, int head_dim, int tiles, KernelInfo *info) {
  fp4::Launch launch = nullptr;
  return fp4::pick(q_dtype, head_dim, tiles, info, &launch);
}

cudaError_t cta_fp4_launch(pkv_dtype q_dtype, int head_dim, int tiles, const AttnParams &p,
                           dim3 grid, cudaStream_t stream) {
  KernelInfo info;
  fp4::Launch launch = nullptr;
  if (!fp4::pick(q_dtype, head_dim, tiles, &info, &launch)) return cudaErrorInvalidValue;
  return launch(p, grid, stream);
}

}  // namespace pkv
