// merge_fp4.cu -- the split-K merge of the 4-bit cache's balanced partition: as
// attn_merge.cu's, for partials whose first and last slot the attention kernel
// published per unit (sequence, KV head, row chunk), split_info[2 U] and [2 U + 1];
// the slots between hold the unit's other pieces, [slot][column].
//
//   out = sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M),   M = max_s lse_s.
//
// WPR warps share a row: one where there are rows enough to fill the GPU, up to
// sixteen for a few rows of many pieces (two contexts of 32768 and 65536 rows: 64
// rows of up to 150 pieces).  The pieces a warp takes, eight at a time, are loaded
// together with their log-sum-exps, so a row costs two round trips (slots, then
// partials).  A dependent launch: it waits for the attention kernel's partials.
// Bound by those round trips: 3 to 5 us behind the attention kernel's end (the
// shared merge kernel, which looks the pieces up in the lengths, took 8).
#include <algorithm>

#include "attn_fp4.cuh"

namespace pkv {
namespace fp4 {
namespace {

constexpr int kInFlight = 8;

template <typename T, int D, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32) merge_kernel(const AttnParams p,
                                                                         int64_t nrows) {
  constexpr int ROWS = WPR == 1 ? 4 : 1;  // of a CTA
  constexpr int PER = D / 32;             // dims of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (WPR == 1 ? warp : 0);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= nrows) return;
  const int per_seq = p.num_queries * p.num_heads;
  const int b = static_cast<int>(row / per_seq);
  const int in = static_cast<int>(row - static_cast<int64_t>(b) * per_seq);
  const int j = in / p.num_heads, h = in - j * p.num_heads, kvh = h / p.group;
  const int r = j * p.group + h - kvh * p.group;  // within its KV head's rows
  const int chunk = r / p.rows_per_cta, col = r - chunk * p.rows_per_cta;
  const int unit = (b * p.num_kv_heads + kvh) * p.row_chunks + chunk;
  const int2 slots = *reinterpret_cast<const int2 *>(p.split_info + 2 * unit);
  const bool empty = seq_extent(p, b, false).nblk == 0;  // (nothing was published)
  int n = empty ? 0 : slots.y - slots.x + 1;
  // (slots that cannot be are those of a call whose copies never came: nothing is
  // read by them)
  const int64_t most = p.split_target + static_cast<int64_t>(p.batch) * p.num_kv_heads *
                                            p.row_chunks;
  if (!empty && (slots.x < 0 || n < 1 || slots.y >= most)) {
    record_error(p.err, PKV_DEVERR_TIMEOUT);
    n = 0;
  }

  float M = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  const int64_t first = static_cast<int64_t>(slots.x) * p.rows_per_cta + col;
  for (int s0 = WPR == 1 ? 0 : warp; s0 < n; s0 += WPR * kInFlight) {
    float lse[kInFlight], v[kInFlight][PER];
    float top = M;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int s = s0 + k * WPR;
      const int64_t at = first + static_cast<int64_t>(s) * p.rows_per_cta;
      lse[k] = s < n ? __ldcg(p.part_lse + at) : -INFINITY;
      const float2 *src = reinterpret_cast<const float2 *>(p.part_o + at * D + lane * PER);
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) {
        const float2 x = s < n ? __ldcg(src + e) : make_float2(0.f, 0.f);
        v[k][2 * e] = x.x;
        v[k][2 * e + 1] = x.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) top = fmaxf(top, lse[k]);
    if (top == -INFINITY) continue;  // nothing visible so far
    const float old = ex2(M - top);
    sum *= old;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= old;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const float w = ex2(lse[k] - top);
      sum += w;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
    }
    M = top;
  }
  if constexpr (WPR > 1) {
    __shared__ float s_max[WPR], s_sum[WPR], s_acc[WPR][D];
    if (lane == 0) {
      s_max[warp] = M;
      s_sum[warp] = sum;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) s_acc[warp][lane * PER + e] = acc[e];
    __syncthreads();
    if (warp * 32 >= D) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w) top = fmaxf(top, s_max[w]);
    const int d = threadIdx.x;
    float total = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float f = s_max[w] == -INFINITY ? 0.f : ex2(s_max[w] - top);
      total += f * s_sum[w];
      if (d < D) x = fmaf(f, s_acc[w][d], x);
    }
    const float inv = total > 0.f ? p.out_scale / total : 0.f;
    static_assert(D <= WPR * 32 || WPR == 1, "a thread a dim");
    static_cast<T *>(p.out)[row * D + d] = from_float<T>(x * inv);
  } else {
    const float inv = sum > 0.f ? p.out_scale / sum : 0.f;
    T *dst = static_cast<T *>(p.out) + row * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) dst[e] = from_float<T>(acc[e] * inv);
  }
}

template <typename T, int D>
cudaError_t merge_t(const AttnParams &p, int sm_count, cudaStream_t stream) {
  const int64_t nrows = static_cast<int64_t>(p.batch) * p.num_queries * p.num_heads;
  if (nrows > 0x7fffffffLL) return cudaErrorInvalidValue;
  // One warp a row from four warps an SM on (the pieces of many rows are few).
  if (nrows >= 4 * sm_count)
    return launch_kernel(true, merge_kernel<T, D, 1>,
                         dim3(static_cast<unsigned>((nrows + 3) / 4)), 128, 0, stream, p, nrows);
  return launch_kernel(true, merge_kernel<T, D, 16>, dim3(static_cast<unsigned>(nrows)), 512, 0,
                       stream, p, nrows);
}

template <typename T>
cudaError_t merge_d(int D, const AttnParams &p, int sm_count, cudaStream_t stream) {
  switch (D) {
    case 64: return merge_t<T, 64>(p, sm_count, stream);
    case 128: return merge_t<T, 128>(p, sm_count, stream);
    case 256: return merge_t<T, 256>(p, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace fp4

cudaError_t merge_fp4_launch(pkv_dtype dtype, int head_dim, const AttnParams &p, int sm_count,
                             cudaStream_t stream) {
  switch (dtype) {
    case PKV_BF16: return fp4::merge_d<__nv_bfloat16>(head_dim, p, sm_count, stream);
    case PKV_F16: return fp4::merge_d<__half>(head_dim, p, sm_count, stream);
    case PKV_F32: return fp4::merge_d<float>(head_dim, p, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
