// pa_quant.cuh -- quantization of cache rows to FP8 (E4M3) and NVFP4 (E2M1 with E4M3 block scales):
// correctly rounded divisions by a pool's scale, the conversions and the row layout, shared by the
// kernels that write the paged cache.
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda_fp4.h>

#include "pa_common.cuh"

namespace pa {

// The correctly rounded quotient a / b is taken in one of three ways (the host picks per scale):
//   * b a normal power of two with a normal reciprocal: the product a * (1 / b), exact;
//   * b in [2^-100, 2^100]: Markstein's correction (P. Markstein, "Computation of elementary
//     functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): with
//     y = RN(1 / b), q = RN(a y) is within one ulp of a / b, the remainder r = a - b q is exact
//     (one fma), and RN(q + r y) is RN(a / b) whenever a and the quotient are normal numbers.  A
//     quotient that overflows (q infinite) stays infinite.  Where a or the quotient is subnormal
//     the result may be an ulp off, which changes no code derived from it: the quotient is then
//     below 2^-26 and rounds to the zero code of E4M3 and of E2M1 (its sign is a's), and a block
//     scale derived from it is the zero code;
//   * otherwise the correctly rounded division.
struct Fp8Scale {
  float sc;    // the pool's scale b
  float rcp;   // 1 / b when exact (a power of two), else 0
  float rcpn;  // RN(1 / b) when b and 1 / b are normal and b is not a power of two, else 0
};

__device__ __forceinline__ float markstein_quot(float a, float b, float y) {
  const float q = a * y;
  const float r = fmaf(-q, b, a);
  return fabsf(q) == INFINITY ? q : fmaf(r, y, q);
}

// The same for a quotient known to be finite (no infinite q to keep).
__device__ __forceinline__ float markstein_quot_finite(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

__device__ __forceinline__ float quot(float x, Fp8Scale s) {
  if (s.rcp != 0.f) return x * s.rcp;
  if (s.rcpn != 0.f) return markstein_quot(x, s.sc, s.rcpn);
  return __fdiv_rn(x, s.sc);
}

// Layout of an NVFP4 row.
struct Nvfp4Row {
  int log2_nb;   // blocks per row, head_dim / 16, as a power of two
  int code_off;  // byte offset of the block scales in a row: head_dim / 2
  int row;       // bytes per row (a multiple of 16)
};

// Nearest E2M1 codes of two values (never NaN here): the conversion instruction rounds to nearest
// with ties to the even mantissa bit, saturates at 6 and keeps the sign (a negative value that
// rounds to zero gives the negative-zero code); lo goes to the low nibble.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest) & 0xffu;
}

// Value of a non-negative, non-NaN E4M3 code (exact in fp32).
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t e = c >> 3, m = c & 7u;
  return e == 0 ? (float)m * 0.001953125f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

struct Nvfp4Block {
  uint2 codes;
  uint32_t scale;
};

// The value of each non-negative E4M3 scale code and its correctly rounded reciprocal (0 for the
// zero code), tabulated once per thread block.
struct E4m3Table {
  float val[128], rcp[128];
};

// How x / sc is divided (see Fp8Scale): the exact reciprocal of a normal power of two whose
// reciprocal is normal, else RN(1 / sc) for Markstein's correction when sc and 1 / sc are normal,
// else neither (the correctly rounded division).
inline Fp8Scale fp8_scale(float sc) {
  uint32_t b;
  std::memcpy(&b, &sc, 4);
  const uint32_t e = (b >> 23) & 0xffu;
  const bool pow2 = (b & 0x807fffffu) == 0 && e >= 1 && e <= 253;  // sc = 2^(e - 127), 1 / sc = 2^(127 - e)
  if (pow2) return {sc, 1.0f / sc, 0.f};
  const float y = 1.0f / sc;  // host IEEE division: correctly rounded
  const bool in_range = sc >= 0x1p-100f && sc <= 0x1p100f;
  return {sc, 0.f, in_range ? y : 0.f};
}

}  // namespace pa
