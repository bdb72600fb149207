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
// One thread takes two scale blocks (32 dims) of one (token, KV head): 64 bytes
// of 16-bit elements on one side, in whole 32-byte sectors, 16 code bytes and
// two scale bytes on the other.  Keys and values are the two rows of the grid.
// Threads run over a row's dims first for keys (a row's codes are contiguous),
// and over 8 consecutive tokens first for values, whose rows lie 4 bytes apart
// in the tile: 8 of them fill a sector.
//
// Bound by memory, 2.56 bytes an element at 16 bits, when the arithmetic stays
// short: an IEEE division for every element, and 64-bit index divisions, took
// three times as long as the bytes.  Quotients are therefore corrected products
// with a correctly rounded reciprocal (Markstein 1990): for r = RN(1 / f) and
// q = RN(x r), RN(q + r RN(x - q f)) is RN(x / f) unless f's significand is all
// ones or something leaves the range; those cases divide.  For 16-bit elements the
// product with the reciprocal alone gives the code wherever no element can lie that
// near a tie (clear_of_ties).
//
// Measured, bf16, head_dim 128, 8 heads: 8192 tokens appended in 10.7 us (33.5 MB read,
// 9.4 MB written: 0.59 of the copy bandwidth; 11.6 with every product corrected, 18
// with divisions and a thread a scale block), loaded in 8.3 us; 32768 loaded in 28.8 us
// (0.88); a few tokens in 2.3 us, a launch.
#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace fp4 {
namespace {

struct RowArgs {
  const void *k_rows, *v_rows;  // new rows, or rows to fill
  uint8_t *k_cache, *v_cache;
  const int64_t *slots;
  int64_t num_blocks;
  int num_tokens, heads;
  float k_scale, v_scale, k_inv, v_inv;  // tensor scales and their reciprocals
  int wide;                              // the rows are 32-byte aligned
  int32_t *err;
};

// 32 bytes of a row.
__device__ __forceinline__ void load32(const void *src, int wide, uint32_t *w) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  } else {
    const uint4 a = __ldg(static_cast<const uint4 *>(src));
    const uint4 b = __ldg(static_cast<const uint4 *>(src) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void *dst, int wide, const uint32_t *w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Whether the quotients by d may be corrected products.
__host__ __device__ __forceinline__ bool plain_divisor(float d) {
#ifdef __CUDA_ARCH__
  const uint32_t bits = __float_as_uint(d);
#else
  union { float f; uint32_t u; } x;
  x.f = d;
  const uint32_t bits = x.u;
#endif
  // 2^-40 <= d < 2^40, significand not all ones
  return (bits >> 23) - 87u < 80u && (bits & 0x7fffffu) != 0x7fffffu;
}
__device__ __forceinline__ float quotient(float x, float d, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, d, x), inv, q);
}

// Whether no 16-bit element lies so near a tie between two codes that its product
// with 1 / f could round to another code than the quotient by f.  The ties are f
// times an odd number up to 7 and a power of two.  The product and the quotient
// differ by less than 1.6 * 2^-23 of their value, 3.2 units of its last place, so the
// element that they could tell apart is within 4 units of the rounded tie; and an
// element has 11 significant bits (bfloat16 8), so its last 13 (16) are zero.
template <typename T> __device__ __forceinline__ bool clear_of_ties(float f) {
  if constexpr (Elt<T>::bytes == 4) return false;
  constexpr uint32_t LAST = std::is_same<T, __half>::value ? 0x1fffu : 0xffffu;
  uint32_t nearest = LAST;
#pragma unroll
  for (int odd = 1; odd <= 7; odd += 2)
    nearest = min(nearest, (__float_as_uint(__fmul_rn(f, float(odd))) + 4u) & LAST);
  return nearest > 8u;
}

// Scale byte and codes of one block: w holds its 16 elements (8 or 16 words).
template <typename T>
__device__ __forceinline__ uint32_t encode16(const uint32_t *w, float t, float t_inv,
                                             uint32_t (&codes)[2]) {
  // largest magnitude, by the bit patterns: a NaN is larger than anything
  float top;
  if constexpr (Elt<T>::bytes == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
    top = __uint_as_float(m);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    float a, b;
    unpack2<T>(max(m & 0xffffu, m >> 16), a, b);
    top = a;
  }
  const bool plain_top =
      plain_divisor(t) && (top == 0.f || (__float_as_uint(top) >> 23) - 87u < 80u);
  const float ideal = plain_top ? quotient(quotient(top, t, t_inv), 6.f, 1.f / 6.f)
                                : __fdiv_rn(__fdiv_rn(top, t), 6.f);
  const uint32_t sbyte = __nv_cvt_float_to_fp8(ideal, __NV_SATFINITE, __NV_E4M3) & 0x7fu;
  const float f = __fmul_rn(e4m3_to_float(sbyte), t);
  const bool live = f > 0.f;  // neither 0 nor NaN
  // a normal scale below the largest: |x / f| < 6.5
  const bool plain = plain_top && sbyte - 8u < 118u && plain_divisor(f);
  const float inv = __frcp_rn(f);
  const bool clear = plain && clear_of_ties<T>(f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8], y[8];
    if constexpr (Elt<T>::bytes == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[8 * h + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack2<T>(w[4 * h + i], x[2 * i], x[2 * i + 1]);
    }
    if (clear) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
    } else if (plain) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = copysignf(quotient(x[i], f, inv), x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = live ? __fdiv_rn(x[i], f) : 0.f;
    }
    codes[h] = f32x8_to_e2m1(y);
  }
  return sbyte;
}

// The 16 elements of a block (8 or 16 words) from its codes and scale byte.
template <typename T>
__device__ __forceinline__ void decode16(const uint32_t (&codes)[2], uint32_t sbyte, float t,
                                         uint32_t *w) {
  const float s = e4m3_to_float(sbyte);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8];
    e2m1x8_to_float(codes[h], s, x);  // exact
    if constexpr (Elt<T>::bytes == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 * h + i] = __float_as_uint(x[i] * t);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * h + i] = Mma<T>::pack(x[2 * i] * t, x[2 * i + 1] * t);
    }
  }
}

template <typename T, int D, bool APPEND>
__global__ void __launch_bounds__(256) rows_kernel(const RowArgs a) {
  if (APPEND) pdl_launch_dependents();  // as in kv_append_kernel
  using TL = Tile<D>;
  constexpr int P = D / 32;                   // threads of a row
  constexpr int WORDS = 8 * Elt<T>::bytes;    // words of 32 elements
  const bool values = blockIdx.y != 0;
  const unsigned per8 = 8u * P * a.heads;     // threads of 8 tokens
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  const unsigned chunk = i / per8, r = i - chunk * per8;
  const int head = r / (8 * P);
  const int pr = values ? (r >> 3) % P : r % P;
  const int token = static_cast<int>(chunk * 8 + (values ? r & 7 : r / P & 7));
  if (token >= a.num_tokens) return;
  const int64_t slot = __ldg(a.slots + token);
  T *row = static_cast<T *>(const_cast<void *>(values ? a.v_rows : a.k_rows)) +
           (static_cast<int64_t>(token) * a.heads + head) * D + pr * 32;
  const bool inside = slot >= 0 && slot < a.num_blocks * kBlockSize;
  uint32_t w[WORDS];
  if (APPEND) {  // (in flight together with the slot)
#pragma unroll
    for (int k = 0; k < WORDS / 8; ++k)
      load32(reinterpret_cast<const char *>(row) + 32 * k, a.wide, w + 8 * k);
  }
  if (slot >= 0 && !inside && head == 0 && pr == 0 && !values)
    record_error(a.err, PKV_DEVERR_SLOT);
  const int at = static_cast<int>(slot % kBlockSize);
  uint8_t *tile = (values ? a.v_cache : a.k_cache) +
                  (slot / kBlockSize * a.heads + head) * static_cast<int64_t>(TL::kBytes);
  const float t = values ? a.v_scale : a.k_scale;
  uint32_t codes[2][2];
  if (APPEND) {
    if (!inside) return;
    const float t_inv = values ? a.v_inv : a.k_inv;
    const uint32_t s0 = encode16<T>(w, t, t_inv, codes[0]);
    const uint32_t s1 = encode16<T>(w + WORDS / 2, t, t_inv, codes[1]);
    if (values) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint32_t *>(tile + TL::v_code(at, pr * 32 + 8 * k)) =
            codes[k >> 1][k & 1];
      tile[TL::v_scale(at, 2 * pr)] = static_cast<uint8_t>(s0);
      tile[TL::v_scale(at, 2 * pr + 1)] = static_cast<uint8_t>(s1);
    } else {
      *reinterpret_cast<uint4 *>(tile + TL::k_code(at, pr * 32)) =
          make_uint4(codes[0][0], codes[0][1], codes[1][0], codes[1][1]);
      *reinterpret_cast<uint16_t *>(tile + TL::k_scale(at, 2 * pr)) =
          static_cast<uint16_t>(s0 | s1 << 8);
    }
  } else {
    if (inside) {
      uint32_t s0, s1;
      if (values) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          codes[k >> 1][k & 1] =
              *reinterpret_cast<const uint32_t *>(tile + TL::v_code(at, pr * 32 + 8 * k));
        s0 = tile[TL::v_scale(at, 2 * pr)];
        s1 = tile[TL::v_scale(at, 2 * pr + 1)];
      } else {
        const uint4 c = *reinterpret_cast<const uint4 *>(tile + TL::k_code(at, pr * 32));
        codes[0][0] = c.x; codes[0][1] = c.y; codes[1][0] = c.z; codes[1][1] = c.w;
        s0 = *reinterpret_cast<const uint16_t *>(tile + TL::k_scale(at, 2 * pr));
        s1 = s0 >> 8;
      }
      decode16<T>(codes[0], s0, t, w);
      decode16<T>(codes[1], s1, t, w + WORDS / 2);
    } else {  // padding (slot < 0) and slots past the cache read as zeros
#pragma unroll
      for (int k = 0; k < WORDS; ++k) w[k] = 0u;
    }
#pragma unroll
    for (int k = 0; k < WORDS / 8; ++k)
      store32(reinterpret_cast<char *>(row) + 32 * k, a.wide, w + 8 * k);
  }
}

template <typename T, int D, bool APPEND>
cudaError_t rows_t(RowArgs a, int64_t num_tokens, cudaStream_t stream) {
  // thread numbers are 32-bit: long calls go in parts of at most 2^30 threads
  const int64_t per8 = int64_t(8) * (D / 32) * a.heads;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per8) * 8;
  for (int64_t t0 = 0; t0 < num_tokens; t0 += most) {
    RowArgs part = a;
    part.num_tokens = static_cast<int>(std::min(most, num_tokens - t0));
    const int64_t skip = t0 * a.heads * D * Elt<T>::bytes;
    part.k_rows = static_cast<const char *>(a.k_rows) + skip;
    part.v_rows = static_cast<const char *>(a.v_rows) + skip;
    part.slots = a.slots + t0;
    const int64_t threads = (part.num_tokens + 7) / 8 * per8;
    if (threads >= (int64_t(1) << 32)) return cudaErrorInvalidValue;
    rows_kernel<T, D, APPEND><<<dim3(static_cast<unsigned>((threads + 255) / 256), 2), 256, 0,
                                stream>>>(part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, bool APPEND>
cudaError_t rows_d(int D, const RowArgs &a, int64_t num_tokens, cudaStream_t stream) {
  switch (D) {
    case 64: return rows_t<T, 64, APPEND>(a, num_tokens, stream);
    case 128: return rows_t<T, 128, APPEND>(a, num_tokens, stream);
    case 256: return rows_t<T, 256, APPEND>(a, num_tokens, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <bool APPEND>
cudaError_t rows(pkv_dtype dtype, int D, const RowArgs &a, int64_t num_tokens,
                 cudaStream_t stream) {
  switch (dtype) {
    case PKV_F32: return rows_d<float, APPEND>(D, a, num_tokens, stream);
    case PKV_BF16: return rows_d<__nv_bfloat16, APPEND>(D, a, num_tokens, stream);
    case PKV_F16: return rows_d<__half, APPEND>(D, a, num_tokens, stream);
    default: return cudaErrorInvalidValue;
  }
}

RowArgs row_args(const void *k_rows, const void *v_rows, const void *k_cache, const void *v_cache,
                 const int64_t *slots, int num_kv_heads, int64_t num_blocks, float k_scale,
                 float v_scale, int32_t *err) {
  const int wide =
      ((reinterpret_cast<uintptr_t>(k_rows) | reinterpret_cast<uintptr_t>(v_rows)) & 31) == 0;
  return RowArgs{k_rows, v_rows, static_cast<uint8_t *>(const_cast<void *>(k_cache)),
                 static_cast<uint8_t *>(const_cast<void *>(v_cache)), slots, num_blocks, 0,
                 num_kv_heads, k_scale, v_scale, 1.f / k_scale, 1.f / v_scale, wide, err};
}

}  // namespace
}  // namespace fp4

cudaError_t append_fp4_launch(pkv_dtype src_dtype, const void *k_new, const void *v_new,
                              void *k_cache, void *v_cache, const int64_t *slots,
                              int64_t num_tokens, int num_kv_heads, int head_dim,
                              int64_t num_blocks, float k_scale, float v_scale, int32_t *err,
                              cudaStream_t stream) {
  return fp4::rows<true>(src_dtype, head_dim,
                         fp4::row_args(k_new, v_new, k_cache, v_cache, slots, num_kv_heads,
                                       num_blocks, k_scale, v_scale, err),
                         num_tokens, stream);
}

cudaError_t load_fp4_launch(pkv_dtype out_dtype, void *k_out, void *v_out, const void *k_cache,
                            const void *v_cache, const int64_t *slots, int64_t num_tokens,
                            int num_kv_heads, int head_dim, int64_t num_blocks, float k_scale,
                            float v_scale, int32_t *err, cudaStream_t stream) {
  return fp4::rows<false>(out_dtype, head_dim,
                          fp4::row_args(k_out, v_out, k_cache, v_cache, slots, num_kv_heads,
                                        num_blocks, k_scale, v_scale, err),
                          num_tokens, stream);
}

}  // namespace pkv
