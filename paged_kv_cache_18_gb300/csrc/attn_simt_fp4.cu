// attn_simt_fp4.cu -- CUDA-core attention over the block-scaled 4-bit cache
// (fp4.cuh): decode, causal verification and tree verification, q and out
// float32, bfloat16 or float16, all arithmetic in float32.
//
//   s_i = scale k_t <q, c^K_i>,   out = v_t sum_i softmax_i(s) c^V_i,
// c being code * block scale (exact in float32) and k_t, v_t the tensor scales.
//
// The work split is the other decode kernels' (one CTA per sequence, KV head,
// row chunk and split; each warp every W-th block with its own ring of bulk
// copies).  Scores: lane r + 16 h takes half h of key r's dims, one shuffle
// joins the halves, and the online softmax runs over the 16 keys of a block at
// once.  P.V: a lane owns D / 32 consecutive dims, the weights come by shuffle.
// Rows past the context are left out of both, so what they hold never matters.
// Its sums are the plain float32 ones of the formulas, and it is what kernel =
// PKV_KERNEL_SIMT asks for: the tensor-core kernels serve every type faster (float32
// GQA decode, 64 contexts of up to 4352 rows, 267 us here and 69 there).  Bound by
// the issue of its FMAs and shuffles, 450 instructions a block with one row and
// about 1100 with four.
#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;  // per warp

template <typename TQ, int D, int R>
__global__ void __launch_bounds__(kWarps * 32) simt_kernel(const AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  using TL = Tile<D>;
  constexpr int STAGE = 2 * TL::kBytes;
  constexpr int DL = D / 32;  // output dims of a lane

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ uint64_t bars[kWarps * kStages];
  __shared__ __align__(16) float qs[R][D];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int key = lane & 15, half = lane >> 4;
  const CtaWork wk = cta_work(p);
  if (!wk.active) return;  // a split past its sequence's end (the whole CTA agrees)
  const int kvh = wk.kvh, chunk = wk.chunk, b = wk.b;
  const int L = wk.ext.L;
  const int blk_begin = wk.blk_begin;
  const int nspan = max(wk.blk_end - blk_begin, 0);
  const int n_my = nspan > warp ? (nspan - warp + kWarps - 1) / kWarps : 0;

  const uint32_t my_bars = smem_u32(&bars[warp * kStages]);
  uint8_t *my_stages = smem + warp * kStages * STAGE;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(my_bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();

  const int32_t *table =
      p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + blk_begin + warp;
  uint32_t bad_mask = 0;
  auto issue = [&](int i) {
    const int v = __ldg(table + static_cast<int64_t>(i) * kWarps);
    const bool bad = v < 0 || static_cast<int64_t>(v) >= p.num_blocks;
    const int s = i % kStages;
    bad_mask = bad ? (bad_mask | (1u << s)) : (bad_mask & ~(1u << s));
    if (lane == 0) {
      if (bad) record_error(p.err, PKV_DEVERR_BLOCK_ID);
      const int64_t off = (static_cast<int64_t>(bad ? 0 : v) * p.num_kv_heads + kvh) * TL::kBytes;
      const uint32_t bar = my_bars + 8 * s, st = smem_u32(my_stages + s * STAGE);
      mbar_arrive_expect_tx(bar, STAGE);
      bulk_g2s(st, static_cast<const uint8_t *>(p.k_cache) + off, TL::kBytes, bar);
      bulk_g2s(st + TL::kBytes, static_cast<const uint8_t *>(p.v_cache) + off, TL::kBytes, bar);
    }
  };
  int issued = min(kStages, n_my);
  for (int i = 0; i < issued; ++i) issue(i);

  // query rows (while the first copies fly), their visibility, softmax states
  for (int e = threadIdx.x; e < R * D; e += kWarps * 32) {
    const int64_t row = cta_row_index(p, b, kvh, chunk, e / D);
    float x = 0.f;
    if (row >= 0) {
      const TQ v = reinterpret_cast<const TQ *>(p.q)[row * D + e % D];
      x = static_cast<float>(v);
    }
    qs[e / D][e % D] = x;
  }
  int lim[R];
  unsigned long long tm[R];
  float m[R], l[R], o[R][DL];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    lim[r] = cta_row_limit(p, L, chunk, r);
    tm[r] = cta_row_tree_mask(p, b, chunk, r);
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < DL; ++e) o[r][e] = 0.f;
  }
  __syncthreads();

  bool timed_out = false;
  int landed = 0;
  for (int i = 0; i < n_my; ++i) {
    const int s = i % kStages;
    if (!__all_sync(kFull, mbar_wait_bounded(my_bars + 8 * s, (i / kStages) & 1))) {
      timed_out = true;
      landed = i;
      break;
    }
    const uint8_t *kt = my_stages + s * STAGE, *vt = kt + TL::kBytes;
    const bool bad = (bad_mask >> s) & 1u;
    const int key0 = (blk_begin + warp + i * kWarps) * kBlockSize;
    const int nvalid = bad ? 0 : min(L - key0, kBlockSize);

    // Scores of this lane's key over its half of the dims: per scale block
    // sum code * q, then times the block's scale.
    float sc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) sc[r] = 0.f;
#pragma unroll 2
    for (int u = 0; u < TL::kScales / 2; ++u) {
      const int blk = half * (TL::kScales / 2) + u;
      const uint2 w = *reinterpret_cast<const uint2 *>(kt + TL::k_code(key, blk * 16));
      const float ks = e4m3_to_float(kt[TL::k_scale(key, blk)]);
      float kf[16];
      e2m1x8_to_float(w.x, 1.f, kf);
      e2m1x8_to_float(w.y, 1.f, kf + 8);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 q4 = *reinterpret_cast<const float4 *>(&qs[r][blk * 16 + e]);
          d = fmaf(q4.x, kf[e], d);
          d = fmaf(q4.y, kf[e + 1], d);
          d = fmaf(q4.z, kf[e + 2], d);
          d = fmaf(q4.w, kf[e + 3], d);
        }
        sc[r] = fmaf(d, ks, sc[r]);
      }
    }
    float pw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float t = sc[r] + __shfl_xor_sync(kFull, sc[r], 16);
      const float v =
          key_visible(p, key0 + key, L, bad, lim[r], tm[r]) ? t * p.scale_log2 : -INFINITY;
      float mx = v;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, k));
      const float m_new = fmaxf(m[r], mx);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float corr = ex2(m[r] - m_use);
      pw[r] = ex2(v - m_use);
      float sum = pw[r];
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) sum += __shfl_xor_sync(kFull, sum, k);
      l[r] = l[r] * corr + sum;
      m[r] = m_new;
#pragma unroll
      for (int e = 0; e < DL; ++e) o[r][e] *= corr;
    }
    // P.V over the rows that exist.
    const int d0 = lane * DL;
    for (int k = 0; k < nvalid; ++k) {
      const float vs = e4m3_to_float(vt[TL::v_scale(k, d0 / 16)]);
      const uint8_t *src = vt + TL::v_code(k, d0);
      uint32_t w;
      if (DL == 2) w = *src;
      else if (DL == 4) w = *reinterpret_cast<const uint16_t *>(src);
      else w = *reinterpret_cast<const uint32_t *>(src);
      float vf[8];
      e2m1x8_to_float(w, vs, vf);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float pk = __shfl_sync(kFull, pw[r], k);
#pragma unroll
        for (int e = 0; e < DL; ++e) o[r][e] = fmaf(pk, vf[e], o[r][e]);
      }
    }
    __syncwarp();
    if (i + kStages < n_my) {
      issue(i + kStages);
      ++issued;
    }
  }
  if (timed_out) {
    if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT);
    // give the copies in flight a bounded chance to land before their memory is reused
    for (int k = landed; k < issued; ++k)
      mbar_wait_bounded(my_bars + 8 * (k % kStages), (k / kStages) & 1);
  }

  __syncthreads();
  constexpr int DP = D + 4;
  float *red_o = reinterpret_cast<float *>(smem);
  float *red_m = red_o + kWarps * R * DP;
  float *red_l = red_m + kWarps * R;
  float *wscale = red_l + kWarps * R;
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < DL; ++e) red_o[(warp * R + r) * DP + lane * DL + e] = o[r][e];
    if (lane == 0) {
      red_m[warp * R + r] = m[r];
      red_l[warp * R + r] = l[r];
    }
  }
  __syncthreads();
  cta_epilogue<TQ, D, R, kWarps, kWarps * 32>(p, red_m, red_l, red_o, wscale, wk);
  // A partial whose sum is NaN (a NaN scale in the cache) has to reach the merged
  // row: its log-sum-exp is +inf, not that of a row that sees nothing.
  if (p.num_splits == 1 && p.split_target == 0) return;
  __syncthreads();
  const int64_t row = threadIdx.x < R ? cta_row_index(p, b, kvh, chunk, threadIdx.x) : -1;
  if (row < 0) return;
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += red_l[w * R + threadIdx.x];
  if (isnan(sum)) p.part_lse[partial_index(p, wk, row, threadIdx.x)] = INFINITY;
}

template <int D, int R> constexpr size_t simt_smem() {
  constexpr size_t stages = size_t(kWarps) * kStages * 2 * Tile<D>::kBytes;
  constexpr size_t red = (size_t(kWarps) * R * (D + 4) + size_t(3 * kWarps + 2) * R) * 4;
  constexpr size_t merge = (size_t(R) * kMaxFusedSplits + R) * 4;
  constexpr size_t need = red > merge ? red : merge;
  return (need > stages ? need : stages) + 128;
}

using Launch = cudaError_t (*)(const AttnParams &, dim3, cudaStream_t);

template <typename TQ, int D, int R>
cudaError_t simt_launch_t(const AttnParams &p, dim3 grid, cudaStream_t stream) {
  return launch_kernel(true, simt_kernel<TQ, D, R>, grid, kWarps * 32, simt_smem<D, R>(), stream,
                       p);
}

template <typename TQ, int D, int R> bool take(KernelInfo *info, Launch *launch) {
  info->func = reinterpret_cast<const void *>(&simt_kernel<TQ, D, R>);
  info->threads = kWarps * 32;
  info->warps = kWarps;
  info->stages = kStages;
  info->smem = simt_smem<D, R>();
  *launch = &simt_launch_t<TQ, D, R>;
  return true;
}

template <typename TQ, int D> bool pick_r(int r, KernelInfo *info, Launch *launch) {
  switch (r) {
    case 1: return take<TQ, D, 1>(info, launch);
    case 2: return take<TQ, D, 2>(info, launch);
    case 4: return take<TQ, D, 4>(info, launch);
    default: return false;
  }
}

template <typename TQ> bool pick_d(int D, int r, KernelInfo *info, Launch *launch) {
  switch (D) {
    case 64: return pick_r<TQ, 64>(r, info, launch);
    case 128: return pick_r<TQ, 128>(r, info, launch);
    case 256: return pick_r<TQ, 256>(r, info, launch);
    default: return false;
  }
}

bool pick(pkv_dtype q_dtype, int D, int r, KernelInfo *info, Launch *launch) {
  switch (q_dtype) {
    case PKV_F32: return pick_d<float>(D, r, info, launch);
    case PKV_BF16: return pick_d<__nv_bfloat16>(D, r, info, launch);
    case PKV_F16: return pick_d<__half>(D, r, info, launch);
    default: return false;
  }
}

}  // namespace
}  // namespace fp4

int simt_fp4_max_rows() { return 4; }

bool simt_fp4_kernel_info(pkv_dtype q_dtype, int head_dim, int rows, KernelInfo *info) {
  fp4::Launch launch = nullptr;
  return fp4::pick(q_dtype, head_dim, rows, info, &launch);
}

cudaError_t simt_fp4_launch(pkv_dtype q_dtype, int head_dim, int rows, const AttnParams &p,
                            dim3 grid, cudaStream_t stream) {
  KernelInfo info;
  fp4::Launch launch = nullptr;
  if (!fp4::pick(q_dtype, head_dim, rows, &info, &launch)) return cudaErrorInvalidValue;
  return launch(p, grid, stream);
}

}  // namespace pkv
