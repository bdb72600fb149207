// commit_rows.cu -- keep the accepted path of a verified tree: in every given
// cache tensor, row L - Q + i of a sequence takes the contents of row
// L - Q + path[i], for i < n, and the sequence's length becomes L - Q + n.
//
// A path increases strictly, so path[i] >= i and a row that is written is
// never the source of a later one: a thread that moves one column of all the
// rows, in order and a few loads at a time, needs no second buffer, and no two
// threads touch the same bytes.  Bound by the latency of the chain
// (lengths and path) -> block table -> rows, not by its few bytes: one warp
// takes 32 columns of one (tensor, sequence), its lanes look the whole path's
// rows up at once, and all tensors of all layers go in one launch: 2.4 us for one
// layer's two caches, 3.5 us for 32 layers (16 sequences, 8 heads, five of ten rows
// kept; 0.7 us of bytes).
#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarpsPerCta = 4;
constexpr int kInFlight = 4;  // rows a thread loads before it stores them

// FP4_D = 0: plain rows, a lane's column being one 16-byte vector; else the
// 4-bit tiles of that head dim, a column being a 4-byte piece of the codes or
// one scale byte.
template <int FP4_D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    commit_kernel(const __grid_constant__ CommitList list, const CommitParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
  const int64_t per_seq = p.warps_per_seq;  // warps for the columns of one (tensor, sequence)
  const int64_t seq = w / per_seq;
  const int t = static_cast<int>(seq / p.batch);
  if (t >= list.count) return;
  const int b = static_cast<int>(seq - static_cast<int64_t>(t) * p.batch);
  const int64_t col = (w - seq * per_seq) * 32 + lane;
  const bool first_warp = w == seq * per_seq && t == 0;  // reports for its sequence

  // Lane i looks after path entries i and i + 32.
  const int L = __ldg(p.context_lens + b);
  const int n = __ldg(p.path_lens + b);
  int node[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    node[k] = i < p.max_path ? __ldg(p.path + static_cast<int64_t>(b) * p.max_path + i) : -1;
  }
  const int base = L - p.num_queries;
  const bool fits = base >= 0 && L <= p.max_blocks_per_seq * static_cast<int64_t>(kBlockSize);
  const bool counted = n >= 0 && n <= p.max_path && n <= p.num_queries;
  bool rising = counted;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    int before = __shfl_up_sync(kFull, node[k], 1);
    if (k == 1) {
      const int last = __shfl_sync(kFull, node[0], 31);
      if (lane == 0) before = last;
    } else if (lane == 0) {
      before = -1;
    }
    if (i < n && !(node[k] > before && node[k] < p.num_queries)) rising = false;
  }
  rising = __all_sync(kFull, rising);
  if (first_warp && lane == 0) {
    if (!fits) record_error(p.err, PKV_DEVERR_CONTEXT_LEN);
    else if (!rising) record_error(p.err, PKV_DEVERR_PATH);
    if (p.new_lens) p.new_lens[b] = fits && rising ? base + n : L;
  }
  if (!fits || !rising) return;

  // Physical rows of the moves: block * 16 + row, -1 for an entry to leave out.
  const int32_t *table = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
  auto slot = [&](int pos) -> int64_t {
    const int blk = __ldg(table + pos / kBlockSize);
    if (blk < 0 || blk >= p.num_blocks) return -1;
    return static_cast<int64_t>(blk) * kBlockSize + pos % kBlockSize;
  };
  int64_t src[2], dst[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    src[k] = dst[k] = -1;
    if (i < n && node[k] != i) {
      src[k] = slot(base + node[k]);
      dst[k] = slot(base + i);
      if (src[k] < 0 || dst[k] < 0) {
        if (first_warp) record_error(p.err, PKV_DEVERR_BLOCK_ID);
        src[k] = dst[k] = -1;
      }
    }
  }

  uint8_t *cache = static_cast<uint8_t *>(list.cache[t]);
  const bool live = col < p.columns;
  if constexpr (FP4_D == 0) {
    // column = (head, 16-byte vector); row r of block k is row (k heads + head) 16 + r
    const int head = live ? static_cast<int>(col / p.vec_per_row) : 0;
    const int64_t vec = live ? col - static_cast<int64_t>(head) * p.vec_per_row : 0;
    auto at = [&](int64_t s) -> uint4 * {
      const int64_t row = ((s / kBlockSize) * p.heads + head) * kBlockSize + s % kBlockSize;
      return reinterpret_cast<uint4 *>(cache) + row * p.vec_per_row + vec;
    };
    for (int i0 = 0; i0 < n; i0 += kInFlight) {
      uint4 v[kInFlight];
      int64_t to[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int i = i0 + u;
        const int64_t s = __shfl_sync(kFull, i < 32 ? src[0] : src[1], i & 31);
        to[u] = __shfl_sync(kFull, i < 32 ? dst[0] : dst[1], i & 31);
        if (i >= n) to[u] = -1;
        if (live && to[u] >= 0) v[u] = *at(s);
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u)
        if (live && to[u] >= 0) *at(to[u]) = v[u];
    }
  } else {
    using TL = fp4::Tile<FP4_D>;
    constexpr int WORDS = FP4_D / 8, PER = WORDS + TL::kScales;
    const bool values = t >= list.first_value;
    const int head = live ? static_cast<int>(col / PER) : 0;
    const int e = live ? static_cast<int>(col) - head * PER : 0;
    auto at = [&](int64_t s) -> uint8_t * {
      const int row = static_cast<int>(s % kBlockSize);
      const int off = e < WORDS
                          ? (values ? TL::v_code(row, e * 8) : TL::k_code(row, e * 8))
                          : (values ? TL::v_scale(row, e - WORDS) : TL::k_scale(row, e - WORDS));
      return cache + ((s / kBlockSize) * p.heads + head) * TL::kBytes + off;
    };
    for (int i0 = 0; i0 < n; i0 += kInFlight) {
      uint32_t v[kInFlight];
      int64_t to[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int i = i0 + u;
        const int64_t s = __shfl_sync(kFull, i < 32 ? src[0] : src[1], i & 31);
        to[u] = __shfl_sync(kFull, i < 32 ? dst[0] : dst[1], i & 31);
        if (i >= n) to[u] = -1;
        if (live && to[u] >= 0)
          v[u] = e < WORDS ? *reinterpret_cast<const uint32_t *>(at(s)) : *at(s);
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (!live || to[u] < 0) continue;
        if (e < WORDS) *reinterpret_cast<uint32_t *>(at(to[u])) = v[u];
        else *at(to[u]) = static_cast<uint8_t>(v[u]);
      }
    }
  }
}

}  // namespace

cudaError_t commit_launch(const CommitList &list, CommitParams p, int fp4_head_dim,
                          cudaStream_t stream) {
  p.warps_per_seq = (p.columns + 31) / 32;
  const int64_t warps = p.warps_per_seq * p.batch * list.count;
  const int64_t ctas = (warps + kWarpsPerCta - 1) / kWarpsPerCta;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(ctas);
  switch (fp4_head_dim) {
    case 0: commit_kernel<0><<<grid, kWarpsPerCta * 32, 0, stream>>>(list, p); break;
    case 64: commit_kernel<64><<<grid, kWarpsPerCta * 32, 0, stream>>>(list, p); break;
    case 128: commit_kernel<128><<<grid, kWarpsPerCta * 32, 0, stream>>>(list, p); break;
    case 256: commit_kernel<256><<<grid, kWarpsPerCta * 32, 0, stream>>>(list, p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace pkv
