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
#include <type_traits>

#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
namespace {

constexpr int kWarps = 4;  // warps of a CTA
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

// The pieces of work of a worker (a CTA or a warp), in turn: one under the
// host's and the device's split partitions (cta_work), under the balanced one
// the parts of units in its range of the list (sk_begin, pkv_device.cuh).
// Warp-collective; the warps of a CTA that is a worker walk alike.
// The walk's state and the pieces lie in shared memory, one copy a warp: they
// are needed between pieces only, where registers are scarce.
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
    const bool publish = blockIdx.x == 0 && threadIdx.x < 32;  // the list, for the merge kernel
    int total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 128) {
      int n[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) n[k] = blocks(p, b0 + 32 * k + lane);  // loads in flight together
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int mine = places(p, n[k]);
        if (publish) {
          const int i = b0 + 32 * k + lane, to = upto(mine);
          if (i < p.batch) {
            seq_extent(p, i, true);  // reports lengths out of range
            p.split_info[2 * i] = total + to - mine;
            p.split_info[2 * i + 1] = n[k];
          }
        }
        total += __reduce_add_sync(kFull, mine);
      }
    }
    if (publish && lane == 0) p.split_info[2 * p.batch] = total;
    x = static_cast<int>(sk_begin(total, p.split_target, worker));
    x1 = static_cast<int>(sk_begin(total, p.split_target, worker + 1));
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
      return true;
    }
    return false;
  }
};

// Tile shapes.  Query rows come in NT tiles of 8 columns; up to two tiles keep
// the Q^T fragments in registers, more in shared memory (their O^T fills the
// registers: D / 4 floats a tile and lane).  A group is the KB consecutive
// blocks that share a stage, a wait and a softmax step.
template <int D, int NT> struct Shape4 {
  static constexpr bool kSharedQ = NT >= 3;
  static constexpr int KB = D == 256 ? 1 : (NT == 1 ? 4 : (NT <= 3 ? 2 : 1));
  static constexpr int NS = KB == 1 ? 4 : 2;
  static constexpr int kMinCtas = D == 256 || NT >= 3 ? 2 : 3;
};

// TEAM: warps that share a piece, 4 (the CTA is the worker; the warps take its
// groups in turn and meet in shared memory at its end) or 1 (each warp is a
// worker of its own under the balanced partition; no barrier anywhere).
template <typename T, int D, int NT, int TEAM>
__global__ void __launch_bounds__(kWarps * 32, (Shape4<D, NT>::kMinCtas))
    mma_kernel(const AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  using TL = Tile<D>;
  using MM = Mma<__half>;
  using SH = Shape4<D, NT>;
  constexpr int KB = SH::KB, NS = SH::NS;
  constexpr bool QS = SH::kSharedQ;
  constexpr int PAIR = 2 * TL::kBytes;  // a block's key and value tiles
  constexpr int STAGE = KB * PAIR;
  constexpr int KS = D / 16;            // k-steps of the scores, m-tiles of O^T
  constexpr int WP = TL::kPanel / 32;   // words (8 dims) of a lane in a panel
  constexpr int KSP = 2 * WP;           // k-steps of a panel
  static_assert(!QS || TEAM == kWarps, "the Q^T fragments in shared memory are the CTA's");
  static_assert((NS & (NS - 1)) == 0 && 2 * KB <= 32 && 32 % KB == 0, "ring, table chunks");

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ uint64_t bars[kWarps * NS];
  constexpr int NC = NT * 8;
  __shared__ float s_fac[QS ? NC : 1];  // score factor per column
  // per warp and column: the query row's offset j Hq + h (of the sequence and KV
  // head's first), and j, the query's place among the Q
  __shared__ int s_row[kWarps][NC], s_j[kWarps][NC];
  __shared__ __align__(16) uint8_t s_q[QS ? 16 : kWarps * D * 2];  // a query row in f16

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int team_warp = TEAM == 1 ? 0 : warp;
  const uint32_t my_bars = smem_u32(&bars[warp * NS]);
  const uint32_t my_stages = smem_u32(smem) + warp * NS * STAGE;
  // behind the rings: Q^T fragments, then the accumulators that warps hand over
  const uint32_t q_smem = smem_u32(smem) + kWarps * NS * STAGE;
  float4 *const scratch = reinterpret_cast<float4 *>(
      smem + kWarps * NS * STAGE + (QS ? KS * NT * 256 : 0));
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) mbar_init(my_bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();

  __shared__ Pieces s_walk[kWarps];
  __shared__ Piece s_piece[kWarps][2];  // the one computed, the one whose copies are issued
  Piece wk;
  {
    Pieces walk;
    if (!walk.first(p, TEAM == 1 ? blockIdx.x * kWarps + warp : blockIdx.x, &wk))
      return;  // (the whole team agrees)
    if (lane == 0) {
      s_walk[warp] = walk;
      s_piece[warp][0] = wk;
    }
  }

  // Copies.  A warp's groups of a piece are number team_warp, team_warp + TEAM,
  // ... of it; its ring runs on across pieces, group number t of all in stage
  // t % NS, so that the next piece's first copies fly while a piece is
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
  bool dead = false;                    // a copy never came
  auto groups_of = [&](int blocks) -> int {
    const int groups = (blocks + KB - 1) / KB;
    return dead || groups <= team_warp ? 0 : (groups - team_warp + TEAM - 1) / TEAM;
  };
  auto load_entries = [&](int chunk32, const Piece &w) -> int {
    const int j = chunk32 * 32 + lane;
    const int blk = ((j / KB) * TEAM + team_warp) * KB + j % KB;
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
  // Query rows of a piece.
  auto rows_of = [&](const Piece &w) -> int {
    return min(p.rows_per_cta, p.rows - w.chunk * p.rows_per_cta);
  };
  auto first_row = [&](const Piece &w) -> int64_t {
    return static_cast<int64_t>(w.b) * p.num_queries * p.num_heads + w.kvh * p.group;
  };
  auto map_columns = [&](const Piece &w) {
    for (int col = lane; col < NC; col += 32) {
      const int r = w.chunk * p.rows_per_cta + col;
      const int j = p.group == 1 ? r : r / p.group;
      s_row[warp][col] = j * p.num_heads + r - j * p.group;
      s_j[warp][col] = j;
    }
    __syncwarp();
  };
  // A piece's query rows in registers: row k of this warp's (every row of its
  // own piece; of a CTA's, with the fragments in shared memory, every fourth),
  // D / 32 dims a lane.  All are loaded together, and for the first piece
  // before the ring's copies, behind which they would queue.
  constexpr int PER = D / 32, WORDS = PER / 2;
  constexpr int Q_STEP = QS ? kWarps : 1, Q_ROWS = NC / Q_STEP;
  uint32_t q_raw[Q_ROWS][WORDS];
  auto load_rows = [&](const Piece &w) {
    const int n = rows_of(w);
    const T *base = static_cast<const T *>(p.q) + first_row(w) * D + lane * PER;
#pragma unroll
    for (int k = 0; k < Q_ROWS; ++k) {
      const int col = k * Q_STEP + (QS ? warp : 0);
      if (col >= n) break;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(base + s_row[warp][col] * int64_t(D));
#pragma unroll
      for (int e = 0; e < WORDS; ++e) q_raw[k][e] = __ldg(src + e);
    }
  };
  // Copy one more group, of the piece computed or of the one after it.
  auto copy_group = [&](int which) {
    if (i_in >= n_in) {
      if (ahead || !more || dead) return;
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
    const int cnt = min(KB, nspan_in - (i_in * TEAM + team_warp) * KB);
    if (lane == 0) mbar_arrive_expect_tx(bar, cnt * PAIR);
    if (lane < 2 * cnt)
      bulk_g2s(tile + lane * TL::kBytes, my_cache + static_cast<int64_t>(v) * block_stride,
               TL::kBytes, bar);
    ++i_in;
    ++turn_in;
  };
  __syncwarp();  // s_piece
  map_columns(wk);
  load_rows(wk);
  start_copies(wk);
  if constexpr (QS) {  // columns without a row stay zero
    for (int k = threadIdx.x; k < KS * NT * 32; k += kWarps * 32)
      if (k / 32 % NT * 8 + (k & 31) / 4 >= p.rows_per_cta)
        asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(q_smem + k * 8), "r"(0) : "memory");
  }

  // Byte offsets of this lane's pieces in a block's tiles.
  const int kk = key_of(g);
  const uint32_t k_off = kk * (TL::kPanel / 2) + c * (4 * WP);
  const uint32_t ks_off = TL::kCodeBytes + kk * TL::kScales + c * (WP / 2);
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

    // Q^T operand fragments: k-step (panel, word w, half i) holds dims
    // panel + 8 WP c + 8 w + 4 i + {0, 1 | 2, 3} of column g.  f16 rows enter as
    // they are, bf16 rows shifted by a power of two into f16 range (the row's
    // largest magnitude in [2^14, 2^15)).  A warp converts a row at a time, each
    // lane D / 32 dims of it, and the row's lanes pick their fragments up from
    // shared memory.
    const int n_rows = rows_of(cur);
    const int64_t row0 = first_row(cur);
    auto convert = [&](uint32_t (&f)[WORDS]) -> float {  // returns the row's score factor
      if constexpr (std::is_same<T, __half>::value) {
        return p.scale_log2;
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
          f[k] = MM::pack(x * up, y * up);
        }
        return p.scale_log2 * __int_as_float((127 - qshift) << 23);
      }
    };
    uint32_t qf[QS ? 1 : KS][QS ? 1 : NT][2];
    float colfac[QS ? 1 : NT][2];  // score factor of my two columns of each tile
    if constexpr (QS) {
      static_assert(!QS || D <= 128, "a lane's dims are (part of) one fragment");
#pragma unroll
      for (int k = 0; k < Q_ROWS; ++k) {
        const int col = k * Q_STEP + warp;
        if (col >= n_rows) break;
        uint32_t(&f)[WORDS] = q_raw[k];
        const float fac = convert(f);
        // dims PER lane ...: lane c' = lane / 8 of the fragment's four, word and
        // half (D = 128), or half a fragment (D = 64)
        const int d = lane * PER;
        const int ks = d % (8 * WP) / 4, cq = d / (8 * WP);
        const uint32_t at = q_smem + (ks * NT + (col >> 3)) * 256 + ((col & 7) * 4 + cq) * 8 +
                            d % 4 * 2;
#pragma unroll
        for (int e = 0; e < WORDS; ++e)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4 * e), "r"(f[e]) : "memory");
        if (lane == 0) s_fac[col] = fac;
      }
      __syncthreads();
    } else {
      const uint32_t mine = smem_u32(s_q) + warp * D * 2;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        colfac[nt][0] = colfac[nt][1] = p.scale_log2;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qf[ks][nt][0] = qf[ks][nt][1] = 0u;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (nt * 8 + r >= n_rows) break;
          uint32_t(&f)[WORDS] = q_raw[nt * 8 + r];
          const float fac = convert(f);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < WORDS; ++k)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(mine + lane * (2 * PER) + 4 * k),
                         "r"(f[k])
                         : "memory");
          __syncwarp();
          if (g == r) {
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
              const int pn = (2 * k2) / KSP, w = (2 * k2) % KSP / 2;
              const uint4 x = lds128(mine + (pn * TL::kPanel + (c * WP + w) * 8) * 2);
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
    }
    auto factor = [&](int nt, int e) -> float {
      if constexpr (QS) return s_fac[nt * 8 + 2 * c + e];
      else return colfac[nt][e];
    };

    // Online-softmax state, per column of mine: the reference, a raw score
    // (-inf until a row is seen), and the sum.  Weights are 2^((s - m) factor):
    // the difference first, so that the largest score has weight 1 however
    // large it is.
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

    for (int i = 0; i < n_here; ++i, ++turn) {
      const uint32_t bar = my_bars + 8 * (turn % NS);
      const uint32_t tile = my_stages + (turn % NS) * STAGE;
      // one decision per warp: its lanes then agree on every later shuffle
      if (!__all_sync(kFull, mbar_wait_bounded(bar, (turn / NS) & 1))) {
        // From here on only barriers.  The copies in flight get a bounded
        // chance to land before their memory is given up.
        dead = true;
        if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
        for (; turn != turn_in; ++turn)
          mbar_wait_bounded(my_bars + 8 * (turn % NS), (turn / NS) & 1);
        i_in = n_in = 0;
        break;
      }
      const int blk0 = (i * TEAM + team_warp) * KB;  // of the piece
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
          const int nv = none ? 0 : cur.L - key0 - u * kBlockSize;
          for (int w = lane; w < D / 4; w += 32) {
            // rows 4 (w % 4) ... of one scale block
            const int keep = nv - 4 * (w & 3);
            if (keep >= 4) continue;
            const uint32_t at = tile + u * PAIR + TL::kBytes + TL::kCodeBytes + 4 * w;
            const uint32_t left = keep <= 0 ? 0u : lds32(at) & ((1u << (8 * keep)) - 1u);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(left) : "memory");
          }
        }
        // these writes come before the next copy into the stage
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // S^T = K Q^T, UB blocks at a time (all of the group where the Q^T
      // fragments come from shared memory, to load each once).
      constexpr int UB = QS ? KB : 1;
      float sc[KB][NT][4];
#pragma unroll
      for (int u0 = 0; u0 < KB; u0 += UB) {
#pragma unroll
        for (int pn = 0; pn < TL::kPanels; ++pn) {
          uint32_t w0[UB][WP], w1[UB][WP], s0[UB][2], s1[UB][2];
#pragma unroll
          for (int u = 0; u < UB; ++u) {
            const uint32_t blk = tile + (u0 + u) * PAIR;
            const uint32_t at = blk + k_off + pn * (kBlockSize * TL::kPanel / 2);
            const uint32_t sat = blk + ks_off + pn * 8;
            if constexpr (WP == 4) {
              const uint4 x = lds128(at), y = lds128(at + TL::kPanel);
              w0[u][0] = x.x; w0[u][1] = x.y; w0[u][2] = x.z; w0[u][3] = x.w;
              w1[u][0] = y.x; w1[u][1] = y.y; w1[u][2] = y.z; w1[u][3] = y.w;
              const uint32_t a = e4m3x2_to_f16(lds16(sat));
              const uint32_t bq = e4m3x2_to_f16(lds16(sat + 2 * TL::kScales));
              s0[u][0] = perm(a, 0x1010); s0[u][1] = perm(a, 0x3232);
              s1[u][0] = perm(bq, 0x1010); s1[u][1] = perm(bq, 0x3232);
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
                if constexpr (QS) {
                  const uint2 x = lds64(q_smem + (ks * NT + nt) * 256 + lane * 8);
                  b0 = x.x;
                  b1 = x.y;
                } else {
                  b0 = qf[ks][nt][0];
                  b1 = qf[ks][nt][1];
                }
#pragma unroll
                for (int u = 0; u < UB; ++u) {
                  if (ks == 0)
                    mma_first(sc[u0 + u][nt], a[u], b0, b1);
                  else
                    MM::run(sc[u0 + u][nt], a[u], b0, b1);
                }
              }
            }
          }
        }
      }
      if (edge) {
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
          // (-inf - -inf is NaN: not above)
          above |= (t - m[nt][e]) * factor(nt, e) > kSlack;
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
            const float m_new = fmaxf(m[nt][e], mx);
            const float corr =
                m[nt][e] == -INFINITY ? 0.f : ex2((m[nt][e] - m_new) * factor(nt, e));
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
          for (int e = 0; e < 4; ++e) {
            const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
            w[e] = ex2((sc[u][nt][e] - ref) * factor(nt, e & 1));
          }
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
    float lse[NT][2];  // the reference in log2 units, -inf while nothing was seen
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(kFull, v, 4);
        v += __shfl_xor_sync(kFull, v, 8);
        v += __shfl_xor_sync(kFull, v, 16);
        l[nt][e] = v;
        lse[nt][e] = m[nt][e] == -INFINITY ? -INFINITY : m[nt][e] * factor(nt, e);
      }
    if constexpr (TEAM > 1) {
      // The warps' states meet two by two: the lanes of all warps hold the same
      // elements, so a state is handed over lane by lane.
      constexpr int STATE = KS * NT + NT;  // float4s of a lane
      auto hand_over = [&](int slot) {
        float4 *to = scratch + slot * STATE * 32 + lane;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            to[(mt * NT + nt) * 32] =
                make_float4(o[mt][nt][0], o[mt][nt][1], o[mt][nt][2], o[mt][nt][3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          to[(KS * NT + nt) * 32] = make_float4(lse[nt][0], lse[nt][1], l[nt][0], l[nt][1]);
      };
      auto take_in = [&](int slot) {
        const float4 *from = scratch + slot * STATE * 32 + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 s = from[(KS * NT + nt) * 32];
          float f[2], t[2];  // factors of mine and of theirs
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float theirs = e ? s.y : s.x;
            const float top = fmaxf(lse[nt][e], theirs);
            const float ref = top == -INFINITY ? 0.f : top;
            f[e] = ex2(lse[nt][e] - ref);
            t[e] = ex2(theirs - ref);
            l[nt][e] = l[nt][e] * f[e] + (e ? s.w : s.z) * t[e];
            lse[nt][e] = top;
          }
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            const float4 x = from[(mt * NT + nt) * 32];
            o[mt][nt][0] = o[mt][nt][0] * f[0] + x.x * t[0];
            o[mt][nt][1] = o[mt][nt][1] * f[1] + x.y * t[1];
            o[mt][nt][2] = o[mt][nt][2] * f[0] + x.z * t[0];
            o[mt][nt][3] = o[mt][nt][3] * f[1] + x.w * t[1];
          }
        }
      };
      if (warp >= 2) hand_over(warp - 2);
      __syncthreads();
      if (warp < 2) take_in(warp);
      // (a slot of its own: the last reader may lag behind the next piece's first
      // writers, which the Q^T fragments' barrier holds back where there is one)
      constexpr int LAST = QS ? 1 : 2;
      if (warp == 1) hand_over(LAST);
      __syncthreads();
      if (warp == 0) take_in(LAST);
    }
    if (team_warp == 0) {
      // The rows: normalised to the output where nothing else is to be merged,
      // else the piece's partial and its log-sum-exp (a NaN sum as +inf, which
      // makes the merged row NaN).
      const bool direct = p.split_target == 0 && p.num_splits == 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = nt * 8 + 2 * c + e;
          if (col >= n_rows) continue;
          const int64_t row = row0 + s_row[warp][col];
          const float sum = l[nt][e];
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          if (direct) {
            T *dst = reinterpret_cast<T *>(p.out) + row * D;
            const float os = inv * p.out_scale;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
              *reinterpret_cast<uint32_t *>(dst + o_dim(mt, g)) =
                  Mma<T>::pack(o[mt][nt][e] * os, o[mt][nt][e + 2] * os);
          } else {
            const int64_t at = p.split_target == 0
                                   ? row * p.num_splits + cur.split
                                   : static_cast<int64_t>(cur.item) * p.rows_per_cta + col;
            float *dst = p.part_o + at * D;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
              *reinterpret_cast<float2 *>(dst + o_dim(mt, g)) =
                  make_float2(o[mt][nt][e] * inv, o[mt][nt][e + 2] * inv);
            if (g == 0)
              p.part_lse[at] = sum > 0.f ? lse[nt][e] + __log2f(sum)
                                         : (sum == 0.f ? -INFINITY : INFINITY);
          }
        }
    }
    if (!more) return;
    if (!ahead) {  // (the piece had no group of this warp's, or a copy never came)
      ahead = true;
      start_copies(s_piece[warp][which ^ 1]);
    }
    ahead = false;
    bad_here = bad_next;
    bad_next = false;
    if (p.row_chunks > 1) map_columns(s_piece[warp][which ^ 1]);
    load_rows(s_piece[warp][which ^ 1]);
  }
}

template <int D, int NT, int TEAM> constexpr size_t mma_smem() {
  using SH = Shape4<D, NT>;
  constexpr size_t stages = size_t(kWarps) * SH::NS * SH::KB * 2 * Tile<D>::kBytes;
  constexpr size_t q = SH::kSharedQ ? size_t(D / 16) * NT * 256 : 0;
  constexpr size_t scratch =
      TEAM == 1 ? 0 : size_t(SH::kSharedQ ? 2 : 3) * (D / 16 * NT + NT) * 32 * 16;
  return stages + q + scratch + 128;
}

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename T, int D, int NT, int TEAM>
cudaError_t mma_launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  return launch_kernel(true, mma_kernel<T, D, NT, TEAM>, grid, kWarps * 32,
                       mma_smem<D, NT, TEAM>(), stream, p);
}

template <typename T, int D, int NT, int TEAM> bool take(KernelInfo *info, Launch *launch) {
  using SH = Shape4<D, NT>;
  info->func = reinterpret_cast<const void *>(&mma_kernel<T, D, NT, TEAM>);
  info->threads = kWarps * 32;
  info->warps = kWarps;
  info->stages = SH::NS;
  info->smem = mma_smem<D, NT, TEAM>();
  info->warp_tiles = NT;
  info->blocks_per_iter = SH::KB;
  *launch = &mma_launch_t<T, D, NT, TEAM>;
  return true;
}

template <typename T, int D, int TEAM> bool pick_nt(int nt, KernelInfo *info, Launch *launch) {
  if (nt == 1) return take<T, D, 1, TEAM>(info, launch);
  if constexpr (D <= 128) {
    if (nt == 2) return take<T, D, 2, TEAM>(info, launch);
    if constexpr (TEAM == kWarps) {
      if (nt == 3) return take<T, D, 3, TEAM>(info, launch);
      if (nt == 4) return take<T, D, 4, TEAM>(info, launch);
      if (nt == 5) return take<T, D, 5, TEAM>(info, launch);
    }
  }
  return false;
}

template <typename T, int TEAM> bool pick_d(int D, int nt, KernelInfo *info, Launch *launch) {
  switch (D) {
    case 64: return pick_nt<T, 64, TEAM>(nt, info, launch);
    case 128: return pick_nt<T, 128, TEAM>(nt, info, launch);
    case 256: return pick_nt<T, 256, TEAM>(nt, info, launch);
    default: return false;
  }
}

bool pick(pkv_dtype q_dtype, int D, int nt, bool warp_workers, KernelInfo *info, Launch *launch) {
  switch (q_dtype) {
    case PKV_BF16:
      return warp_workers ? pick_d<__nv_bfloat16, 1>(D, nt, info, launch)
                          : pick_d<__nv_bfloat16, kWarps>(D, nt, info, launch);
    case PKV_F16:
      return warp_workers ? pick_d<__half, 1>(D, nt, info, launch)
                          : pick_d<__half, kWarps>(D, nt, info, launch);
    default: return false;
  }
}

}  // namespace
}  // namespace fp4

int mma_fp4_max_tiles(int head_dim) { return head_dim <= 128 ? 5 : 1; }

int mma_fp4_max_warp_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }

bool mma_fp4_kernel_info(pkv_dtype q_dtype, int head_dim, int tiles, bool warp_workers,
                         KernelInfo *info) {
  fp4::Launch launch = nullptr;
  return fp4::pick(q_dtype, head_dim, tiles, warp_workers, info, &launch);
}

cudaError_t mma_fp4_launch(pkv_dtype q_dtype, int head_dim, int tiles, const AttnParams &p,
                           dim3 grid, cudaStream_t stream) {
  KernelInfo info;
  fp4::Launch launch = nullptr;
  const bool warp_workers = p.stream_k && p.split_target > static_cast<int>(grid.x);
  if (!fp4::pick(q_dtype, head_dim, tiles, warp_workers, &info, &launch))
    return cudaErrorInvalidValue;
  return launch(p, grid, stream);
}

}  // namespace pkv
