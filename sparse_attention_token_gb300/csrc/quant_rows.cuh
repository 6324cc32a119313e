// quant_rows.cuh -- layout of a row of the quantised latent cache.
//
// A row holds a token's 512 latent values c and 64 rotary values r.  2^E is the row's scale, a power
// of two, so every value that a code stands for is exact in bf16.
//
//   DSA_FP8_E4M3, 656 bytes   512 e4m3 codes of c / 2^E | 64 bf16 of r / 2^E | 2^E in fp32 | 12 zero bytes
//   DSA_FP4_E2M1, 416 bytes   512 4-bit codes | 64 bf16 of r / 2^E | 32 scale bytes of blocks of 16
//
// r is held in units of 2^E (exact: a power of two) so that one accumulator takes the products of both
// parts and 2^E is applied once to their sum.
//
// 4-bit codes: e2m1 of c / (2^E s), s = 2^k (1 + m / 8) the block's scale, -5 <= k, s <= 72.  A code of
// magnitude q stands for 2^E e4m3(q s): the eight values of a block are e4m3 numbers, which the tensor
// cores take as they are.  A 32-bit word holds eight values; nibble i's low three bits are the magnitude
// of value i (they are the selector of a byte permutation over a table of eight), the signs of values
// 0..3 are bits 7, 15, 23, 31 and those of values 4..7 bits 3, 11, 19, 27 (where one mask, or a shift and
// a mask, puts them on top of four bytes).  Scale byte i: 8 (k + 5) + m, and in its bit 7 bit i of E + 128
// (bytes 0..7; 0 in the others), so that a row is 13 sectors of 32 bytes and no more.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "dsa_indexer.h"

namespace dsa {
namespace quant {

constexpr int kRank = 512, kRope = 64;
constexpr int kRow8 = 656, kRow4 = 416;
constexpr int kRope8 = 512, kScale8 = 640;   // byte offsets in a row
constexpr int kRope4 = 256, kScale4 = 384;
constexpr int kMaxExp = 60;                  // |E| at most
constexpr float kTop8 = 448.f, kTop4 = 432.f;  // the largest |c| / 2^E of a row

__host__ __device__ inline int row_bytes(int format) {
  return format == DSA_FP8_E4M3 ? kRow8 : format == DSA_FP4_E2M1 ? kRow4 : 0;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two products, each rounded as by itself.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Two e4m3 codes of (lo, hi), nearest with ties to even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// The values of two e4m3 codes.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two e2m1 codes, the first in the low nibble, nearest with ties to even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void unpack_bf16(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// The eight e4m3 magnitudes that a block's codes 0, 0.5, 1, 1.5, 2, 3, 4, 6 stand for, code 0 in the
// lowest byte of .x.  For s = 2^k (1 + m / 8) they are those of m at k = -5 with their exponents
// raised by k + 5 (all but the zero are normal numbers down to k = -5, 0.5 s = 2^-6).
__device__ __forceinline__ uint2 levels_base(int m) {
  const float s = (1.f + 0.125f * m) * 0.03125f;
  return make_uint2(e4m3x2(0.f, 0.5f * s) | (e4m3x2(s, 1.5f * s) << 16),
                    e4m3x2(2.f * s, 3.f * s) | (e4m3x2(4.f * s, 6.f * s) << 16));
}
__device__ __forceinline__ uint2 levels_at(uint2 base, int scale_byte) {
  const uint32_t up = ((scale_byte >> 3) & 15) * 0x08080808u;
  return make_uint2(base.x + (up & 0xFFFFFF00u), base.y + up);
}
// Eight 4-bit codes as e4m3 codes: values 0..3 in .x, 4..7 in .y.
__device__ __forceinline__ uint2 codes4_to_e4m3(uint32_t w, uint2 levels) {
  const uint32_t sel = w & 0x77777777u;
  return make_uint2(__byte_perm(levels.x, levels.y, sel) | (w & 0x80808080u),
                    __byte_perm(levels.x, levels.y, sel >> 16) | ((w << 4) & 0x80808080u));
}

}  // namespace quant
}  // namespace dsa
