// fp4.cuh -- the 4-bit cache format and its conversions.
//
// A value is  code * block scale * tensor scale:  the code is E2M1 (a sign and
// 0, 0.5, 1, 1.5, 2, 3, 4 or 6), the block scale is E4M3, one for every 16
// consecutive head dims of a row, and the tensor scale is one float per cache
// tensor: 4.5 bits a value.  code * block scale has at most 2 + 4 significant
// bits and lies in +-[2^-10, 2688], so it is exact in f16 and f32 alike.
//
// The tile of one (block, KV head) is 9 D contiguous bytes: the codes of its
// 16 rows (two to a byte, the even dim in the low nibble), then their scales.
//   keys    codes [D / P][16 rows][P / 2 bytes], P = min(D, 128);
//           scales [16 rows][D / 16]
//   values  codes [D / 8][16 rows][4 bytes];  scales [D / 16][16 rows]
// The two orders are those in which the tensor-core kernel's lanes take their
// fragments with 16-byte shared-memory loads free of bank conflicts: a lane of
// the scores reads 32 dims of one key, a lane of P.V four keys of 8 dims.
// Every byte belongs to one row, so rows are written without read-modify-write.
#pragma once

#include <cuda_fp8.h>

#include "pkv_device.cuh"

namespace pkv {
namespace fp4 {

__host__ __device__ constexpr int tile_bytes(int D) { return 9 * D; }

template <int D> struct Tile {
  static constexpr int kPanel = D < 128 ? D : 128;
  static constexpr int kPanels = D / kPanel;
  static constexpr int kCodeBytes = 8 * D;
  static constexpr int kBytes = 9 * D;
  static constexpr int kScales = D / 16;  // per row
  // Byte of dims d, d + 1 (d even) of a row, and of its scale for dims 16 blk ...
  static __device__ __forceinline__ int k_code(int row, int d) {
    return (d / kPanel) * (kBlockSize * kPanel / 2) + row * (kPanel / 2) + (d % kPanel) / 2;
  }
  static __device__ __forceinline__ int k_scale(int row, int blk) {
    return kCodeBytes + row * kScales + blk;
  }
  static __device__ __forceinline__ int v_code(int row, int d) {
    return (d / 8) * (kBlockSize * 4) + row * 4 + (d % 8) / 2;
  }
  static __device__ __forceinline__ int v_scale(int row, int blk) {
    return kCodeBytes + blk * kBlockSize + row;
  }
};

// Eight codes (one word) -> four pairs of f16, low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight floats -> eight codes in one word, round to nearest (ties to the even
// code), saturating at +-6; x[0] in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// Two E4M3 bytes -> a pair of f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(two));
  return h;
}
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __low2float(__half2(__nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(byte & 0xffu), __NV_E4M3)));
}

// Eight codes times one scale -> eight floats (exact).
__device__ __forceinline__ void e2m1x8_to_float(uint32_t w, float scale, float *f) {
  uint32_t h[4];
  e2m1x8_to_f16(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2<__half>(h[i], a, b);
    f[2 * i] = a * scale;
    f[2 * i + 1] = b * scale;
  }
}

}  // namespace fp4
}  // namespace pkv
