// A row of the 8-bit latent cache and its arithmetic, shared by the kernels that write, read and
// attend over it, and the 8-bit form of an indexer key.
//
// Layout of one row (D_QK latent dims, the first D_V of them values):
//   bytes [0, D_V)                     e4m3 codes of the D_V latent values
//   bytes [D_V, D_V + S)               fp32 scales, one per group of 128 values; S = 4 bytes a
//                                      group rounded up to 16 (unused scale slots are 0)
//   bytes [D_V + S, ...)               the D_QK - D_V rotary dims in bf16, unquantised
// 656 bytes at (576, 512), 208 at (160, 128): multiples of 16, so every part of every row is
// 16-byte aligned.
//
// Scales are powers of two: s = 2^e with the smallest e such that max|x| <= 448 s (1 for a group
// of zeros), e clamped to [-100, 119].  A code has 4 significant bits, so code * 2^e is exact in
// bf16 (and fp32): reading back and attending never round, and the only rounding of the format is
// x / s to the nearest e4m3 value (x / s itself is exact).  A floating-point code loses nothing
// to the coarser scale but up to one binade of its 18.  A group that holds an infinity or a NaN
// gets a NaN scale and zero codes, so that it reads back as NaN everywhere.
#pragma once
#include <cuda_fp8.h>

#include "sm100.cuh"

namespace dsa {

constexpr int kQ8Group = 128;       // values per scale
constexpr int kQ8ExpMin = -100, kQ8ExpMax = 119;

template <int D_QK, int D_V>
struct Q8Row {
  static_assert(D_V % kQ8Group == 0 && D_QK > D_V && (D_QK - D_V) % 8 == 0, "row dims");
  static constexpr int GROUPS = D_V / kQ8Group;
  static constexpr int ROPE = D_QK - D_V;
  static constexpr int SCALE_OFF = D_V;
  static constexpr int ROPE_OFF = D_V + (4 * GROUPS + 15) / 16 * 16;
  static constexpr int BYTES = ROPE_OFF + 2 * ROPE;
  static_assert(BYTES % 16 == 0, "16-byte rows");
};

// fp32 bits of 2^e, e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Exponent of the scale of a group whose largest |x| has the bf16 bits `amax` (finite):
// 448 = 1.75 * 2^8, so amax = (1 + m / 128) 2^E needs e = E - 8, one more when its mantissa is
// above 1.75 (m > 96).
__device__ __forceinline__ int q8_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 96u ? 1 : 0);
  return min(max(e, kQ8ExpMin), kQ8ExpMax);
}

// The e4m3 code nearest to y (ties to even, saturating at +-448; y is finite).
__device__ __forceinline__ uint32_t q8_code(float y) {
  return __nv_cvt_float_to_fp8(fminf(fmaxf(y, -448.f), 448.f), __NV_SATFINITE, __NV_E4M3);
}

// A token's indexer key, PER consecutive values a lane of a converged warp: returns its scale, amax /
// 448 in fp32 (1 for a key of zeros), and the lane's codes of x / scale (rounded to fp32 first, so
// that a code can be one step off the exact quotient's at a tie).  As in a latent group, a key that
// holds an infinity or a NaN gets a NaN scale and zero codes: its scores are NaN, not those of
// another key.
template <int PER>
__device__ __forceinline__ float q8_key(const float (&x)[PER], uint32_t* codes) {
  uint32_t top = 0;                                // largest magnitude (NaN above infinity)
#pragma unroll
  for (int i = 0; i < PER; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(0xffffffffu, top);
  const float amax = __uint_as_float(top);
  *codes = 0;
  if (top >= 0x7F800000u) return __uint_as_float(0x7FFFFFFFu);
  const float scale = amax > 0.f ? amax / 448.f : 1.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) *codes |= q8_code(x[i] / scale) << (8 * i);
  return scale;
}

// Two e4m3 codes (the low bytes of the halves of z) times a power of two, as two bf16.  A code's
// sign, 4 exponent and 3 mantissa bits belong in bits 15 and 10..4 of a bf16, where they are the
// code's value times 2^-120 (subnormal codes become bf16 subnormals); mul = 2^120 s in both
// halves undoes it exactly.  16 z puts the magnitude there and the sign at bit 11, and
// 240 (z & 0x80) adds what moves the sign on to bit 15.  The multiply-adds run on the FMA pipe:
// a form with shifts and logic alone, all on the half-rate integer pipe, took 16.6 cycles a
// scheduler for four codes of a warp, this one 11.
__device__ __forceinline__ uint32_t q8_expand2(uint32_t z, __nv_bfloat162 mul) {
  const uint32_t u = z * 16u + (z & 0x00800080u) * 240u;
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u), mul);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint2 q8_expand4(uint32_t w, __nv_bfloat162 mul) {
  return make_uint2(q8_expand2(__byte_perm(w, 0, 0x4140), mul),
                    q8_expand2(__byte_perm(w, 0, 0x4342), mul));
}

// Eight codes of a group with scale s as eight bf16.  2^120 s is a bf16 up to s = 2^7; larger
// scales (and the NaN scale) multiply in two steps.
__device__ __forceinline__ uint4 q8_expand8(uint2 c, float s) {
  const uint32_t sb = __float_as_uint(s);
  const bool big = sb > 0x43000000u;              // s > 2^7, or the NaN scale
  // the upper half of an fp32 power of two is its bf16
  const uint32_t mb = __byte_perm((big ? 0x43000000u : sb) + (120u << 23), 0, 0x3232);
  const __nv_bfloat162 mul = *reinterpret_cast<const __nv_bfloat162*>(&mb);
  uint2 e[2] = {q8_expand4(c.x, mul), q8_expand4(c.y, mul)};
  if (big) {
    const __nv_bfloat162 m2 = __float2bfloat162_rn(s * 0x1p-7f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&e[i].x), m2);
      const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&e[i].y), m2);
      e[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
  }
  return make_uint4(e[0].x, e[0].y, e[1].x, e[1].y);
}

}  // namespace dsa
