// kv_fp4.cu -- rows into and out of the block-scaled 4-bit cache (fp4.cuh).
//
// Append, for 16 consecutive head dims x_0 .. x_15 of a new row and the tensor
// scale t, all in IEEE float32:
//   A = max |x_i|,  s = E4M3(min(A / t / 6, 448)),  code_i = E2M1(x_i / (s t)),
// both roundings to nearest even (6 is the largest code: the block's largest
// value lands on it), codes saturating; a block whose s is 0 or NaN (every
// value 0 or too small, or some value NaN) gets codes 0, so it reads back as
// zeros or NaN.  Load: out = (code * s) t, the product in brackets exact, one
// rounding to float32 and one to the output type.
//
// One thread takes one scale block of one (token, KV head): 16 elements on one
// side, 8 code bytes and a scale byte on the other; keys and values are
// separate halves of the grid.  Threads run over a row's blocks first for keys
// (the row's code bytes are contiguous), and over 4 blocks of 8 consecutive
// tokens for values, so that the 4-byte pieces of consecutive rows fill whole
// 32-byte sectors of the tile while each token's elements are still taken 128
// bytes (16-bit) at a time.  Bound by memory: 2.56 bytes an element at 16 bits.
#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
namespace {

template <typename T> struct Vec16;  // 16 elements in 16-byte vectors
template <> struct Vec16<float> { static constexpr int n = 4; };
template <> struct Vec16<__nv_bfloat16> { static constexpr int n = 2; };
template <> struct Vec16<__half> { static constexpr int n = 2; };

template <typename T>
__device__ __forceinline__ void load16(const T *src, float (&x)[16]) {
  uint4 w[Vec16<T>::n];
#pragma unroll
  for (int i = 0; i < Vec16<T>::n; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
  if constexpr (Vec16<T>::n == 4) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(reinterpret_cast<const uint32_t *>(w)[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      unpack2<T>(reinterpret_cast<const uint32_t *>(w)[i], x[2 * i], x[2 * i + 1]);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  return Mma<__nv_bfloat16>::pack(a, b);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  return Mma<__half>::pack(a, b);
}

template <typename T>
__device__ __forceinline__ void store16(T *dst, const float (&x)[16]) {
  uint32_t w[4 * Vec16<T>::n];
  if constexpr (Vec16<T>::n == 4) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], T{});
  }
#pragma unroll
  for (int i = 0; i < Vec16<T>::n; ++i)
    reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2],
                                                   w[4 * i + 3]);
}

// The work of one thread: which scale block of which row.
struct Item {
  bool values;   // of the value cache, else of the key cache
  int64_t token;
  int head, blk;
};
template <int D>
__device__ __forceinline__ Item item_of(int64_t i, int64_t tokens8, int heads) {
  constexpr int S = Tile<D>::kScales;  // 4, 8 or 16
  const int64_t half = tokens8 * heads * S;
  Item it;
  it.values = i >= half;
  if (!it.values) {
    it.blk = static_cast<int>(i % S);
    const int64_t r = i / S;
    it.head = static_cast<int>(r % heads);
    it.token = r / heads;
  } else {
    i -= half;
    const int low = static_cast<int>(i & 7), b4 = static_cast<int>((i >> 3) & 3);
    int64_t r = i >> 5;
    it.blk = static_cast<int>(r % (S / 4)) * 4 + b4;
    r /= S / 4;
    it.head = static_cast<int>(r % heads);
    it.token = (r / heads) * 8 + low;
  }
  return it;
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
    append_kernel(const T *__restrict__ k_new, const T *__restrict__ v_new,
                  uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache,
                  const int64_t *__restrict__ slots, int64_t num_tokens, int heads,
                  int64_t num_blocks, float k_scale, float v_scale, int32_t *err) {
  pdl_launch_dependents();  // as in kv_append_kernel
  using TL = Tile<D>;
  const int64_t tokens8 = (num_tokens + 7) / 8 * 8;
  const int64_t total = 2 * tokens8 * heads * TL::kScales;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const Item it = item_of<D>(i, tokens8, heads);
    if (it.token >= num_tokens) continue;
    const int64_t slot = __ldg(slots + it.token);
    if (slot < 0) continue;
    if (slot >= num_blocks * kBlockSize) {
      if (it.head == 0 && it.blk == 0) record_error(err, PKV_DEVERR_SLOT);
      continue;
    }
    float x[16];
    load16<T>((it.values ? v_new : k_new) + (it.token * heads + it.head) * D + it.blk * 16, x);
    // largest magnitude, by the bit patterns: a NaN is larger than anything
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    const float t = it.values ? v_scale : k_scale;
    const float ideal = __fdiv_rn(__fdiv_rn(__uint_as_float(top), t), 6.f);
    const uint32_t sbyte = __nv_cvt_float_to_fp8(ideal, __NV_SATFINITE, __NV_E4M3) & 0x7fu;
    const float f = __fmul_rn(e4m3_to_float(sbyte), t);
    float y[2][8];
    const bool live = f > 0.f;  // neither 0 nor NaN
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e >> 3][e & 7] = live ? __fdiv_rn(x[e], f) : 0.f;
    const uint32_t w0 = f32x8_to_e2m1(y[0]), w1 = f32x8_to_e2m1(y[1]);
    const int row = static_cast<int>(slot % kBlockSize);
    const int64_t tile = (slot / kBlockSize * heads + it.head) * TL::kBytes;
    if (it.values) {
      uint8_t *dst = v_cache + tile;
      *reinterpret_cast<uint32_t *>(dst + TL::v_code(row, it.blk * 16)) = w0;
      *reinterpret_cast<uint32_t *>(dst + TL::v_code(row, it.blk * 16 + 8)) = w1;
      dst[TL::v_scale(row, it.blk)] = static_cast<uint8_t>(sbyte);
    } else {
      uint8_t *dst = k_cache + tile;
      *reinterpret_cast<uint2 *>(dst + TL::k_code(row, it.blk * 16)) = make_uint2(w0, w1);
      dst[TL::k_scale(row, it.blk)] = static_cast<uint8_t>(sbyte);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
    load_kernel(T *__restrict__ k_out, T *__restrict__ v_out, const uint8_t *__restrict__ k_cache,
                const uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slots,
                int64_t num_tokens, int heads, int64_t num_blocks, float k_scale, float v_scale,
                int32_t *err) {
  using TL = Tile<D>;
  const int64_t tokens8 = (num_tokens + 7) / 8 * 8;
  const int64_t total = 2 * tokens8 * heads * TL::kScales;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const Item it = item_of<D>(i, tokens8, heads);
    if (it.token >= num_tokens) continue;
    const int64_t slot = __ldg(slots + it.token);
    float x[16];
    if (slot >= 0 && slot < num_blocks * kBlockSize) {
      const int row = static_cast<int>(slot % kBlockSize);
      const int64_t tile = (slot / kBlockSize * heads + it.head) * TL::kBytes;
      uint32_t w0, w1, sbyte;
      if (it.values) {
        const uint8_t *src = v_cache + tile;
        w0 = *reinterpret_cast<const uint32_t *>(src + TL::v_code(row, it.blk * 16));
        w1 = *reinterpret_cast<const uint32_t *>(src + TL::v_code(row, it.blk * 16 + 8));
        sbyte = src[TL::v_scale(row, it.blk)];
      } else {
        const uint8_t *src = k_cache + tile;
        const uint2 w = *reinterpret_cast<const uint2 *>(src + TL::k_code(row, it.blk * 16));
        w0 = w.x;
        w1 = w.y;
        sbyte = src[TL::k_scale(row, it.blk)];
      }
      const float s = e4m3_to_float(sbyte);
      e2m1x8_to_float(w0, s, x);
      e2m1x8_to_float(w1, s, x + 8);
      const float t = it.values ? v_scale : k_scale;
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= t;
    } else {  // padding (slot < 0) and slots past the cache read as zeros
      if (slot >= 0 && it.head == 0 && it.blk == 0) record_error(err, PKV_DEVERR_SLOT);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
    }
    store16<T>((it.values ? v_out : k_out) + (it.token * heads + it.head) * D + it.blk * 16, x);
  }
}

struct RowArgs {
  const void *k_new, *v_new;
  void *k_out, *v_out;
  void *k_cache, *v_cache;
  const int64_t *slots;
  int64_t num_tokens, num_blocks;
  int heads;
  float k_scale, v_scale;
  int32_t *err;
};

template <typename T, int D>
cudaError_t rows_t(bool append, const RowArgs &a, int sm_count, cudaStream_t stream) {
  const int64_t total = 2 * ((a.num_tokens + 7) / 8 * 8) * a.heads * Tile<D>::kScales;
  int64_t ctas = (total + 255) / 256;
  const int64_t cap = static_cast<int64_t>(sm_count) * 8;
  if (ctas > cap) ctas = cap;
  if (append) {
    append_kernel<T, D><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(
        static_cast<const T *>(a.k_new), static_cast<const T *>(a.v_new),
        static_cast<uint8_t *>(a.k_cache), static_cast<uint8_t *>(a.v_cache), a.slots,
        a.num_tokens, a.heads, a.num_blocks, a.k_scale, a.v_scale, a.err);
  } else {
    load_kernel<T, D><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(
        static_cast<T *>(a.k_out), static_cast<T *>(a.v_out),
        static_cast<const uint8_t *>(a.k_cache), static_cast<const uint8_t *>(a.v_cache), a.slots,
        a.num_tokens, a.heads, a.num_blocks, a.k_scale, a.v_scale, a.err);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t rows_d(bool append, int D, const RowArgs &a, int sm_count, cudaStream_t stream) {
  switch (D) {
    case 64: return rows_t<T, 64>(append, a, sm_count, stream);
    case 128: return rows_t<T, 128>(append, a, sm_count, stream);
    case 256: return rows_t<T, 256>(append, a, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t rows(bool append, pkv_dtype dtype, int D, const RowArgs &a, int sm_count,
                 cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  switch (dtype) {
    case PKV_F32: return rows_d<float>(append, D, a, sm_count, stream);
    case PKV_BF16: return rows_d<__nv_bfloat16>(append, D, a, sm_count, stream);
    case PKV_F16: return rows_d<__half>(append, D, a, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace fp4

cudaError_t append_fp4_launch(pkv_dtype src_dtype, const void *k_new, const void *v_new,
                              void *k_cache, void *v_cache, const int64_t *slots,
                              int64_t num_tokens, int num_kv_heads, int head_dim,
                              int64_t num_blocks, float k_scale, float v_scale, int32_t *err,
                              int sm_count, cudaStream_t stream) {
  const fp4::RowArgs a{k_new, v_new, nullptr, nullptr, k_cache, v_cache, slots, num_tokens,
                       num_blocks, num_kv_heads, k_scale, v_scale, err};
  return fp4::rows(true, src_dtype, head_dim, a, sm_count, stream);
}

cudaError_t load_fp4_launch(pkv_dtype out_dtype, void *k_out, void *v_out, const void *k_cache,
                            const void *v_cache, const int64_t *slots, int64_t num_tokens,
                            int num_kv_heads, int head_dim, int64_t num_blocks, float k_scale,
                            float v_scale, int32_t *err, int sm_count, cudaStream_t stream) {
  const fp4::RowArgs a{nullptr, nullptr, k_out, v_out, const_cast<void *>(k_cache),
                       const_cast<void *>(v_cache), slots, num_tokens, num_blocks, num_kv_heads,
                       k_scale, v_scale, err};
  return fp4::rows(false, out_dtype, head_dim, a, sm_count, stream);
}

}  // namespace pkv
