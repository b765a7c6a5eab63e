// codec_blocks.cuh -- encoders of one scale block, shared by the pack kernels
// and the fused KV append so that both write identical bytes.
//
// "DeepSeek-V4.1-Flash: Pushing the Limits of KV Cache Compression",
// section 2.4.4: OCP MXFP4 (E2M1 values, one E8M0 scale per 32) for the
// indexer keys and queries; E2M1 with one E4M3 scale per 16 channels and no
// global scale for the main KV latent.
#pragma once
#include "common.cuh"

namespace csa2 {

// One MXFP4 block: 32 bf16 values (16 words of bf16 pairs, element 2i in the
// low half) -> 16 bytes of E2M1 pairs (element 2i in the low nibble) and the
// E8M0 code. The shared exponent is floor(log2(amax)) - 2 (the largest E2M1
// magnitude is 6 = 1.5 * 2^2), clamped to the E8M0 range; values are scaled
// by its power of two and rounded to nearest-even E2M1, saturating.
// The shared exponent X of an MXFP4 block, from the largest magnitude bit
// pattern (sign cleared) among its bf16 values, and the scaling 2^-X as fp32.
__device__ __forceinline__ int mxfp4_exponent(uint32_t amax_bits, float& inv) {
  // floor(log2(amax)) is the unbiased exponent field for a normal amax;
  // subnormal or zero amax clamps to -127.
  const int exp_field = (int)(amax_bits >> 7);  // bf16 exponent field
  int X = exp_field == 0 ? -127 : (exp_field - 127) - 2;
  X = X < -127 ? -127 : (X > 127 ? 127 : X);
  // 2^-X as fp32 (X = 127 gives the subnormal 2^-127)
  inv = X == 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - X) << 23);
  return X;
}

// Four consecutive values of an MXFP4 block (two words of bf16 pairs), scaled
// by 2^-X and rounded to nearest-even E2M1, saturating: two bytes, element 0 in
// the low nibble.
__device__ __forceinline__ uint32_t encode_e2m1x4(uint32_t pair0, uint32_t pair1, float inv) {
  const float a0 = bf16_bits_to_f32(pair0 & 0xFFFFu) * inv;
  const float a1 = bf16_bits_to_f32(pair0 >> 16) * inv;
  const float a2 = bf16_bits_to_f32(pair1 & 0xFFFFu) * inv;
  const float a3 = bf16_bits_to_f32(pair1 >> 16) * inv;
  return cvt_e2m1x2(a0, a1) | (cvt_e2m1x2(a2, a3) << 8);
}

__device__ __forceinline__ void encode_mxfp4_block(const uint32_t (&w)[16], uint4& data, uint8_t& e8m0) {
  uint32_t amax_bits = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax_bits = max(amax_bits, (w[i] & 0x7FFFu));
    amax_bits = max(amax_bits, ((w[i] >> 16) & 0x7FFFu));
  }
  float inv;
  const int X = mxfp4_exponent(amax_bits, inv);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = encode_e2m1x4(w[4 * i], w[4 * i + 1], inv) | (encode_e2m1x4(w[4 * i + 2], w[4 * i + 3], inv) << 16);
  data = make_uint4(out[0], out[1], out[2], out[3]);
  e8m0 = (uint8_t)(X + 127);
}

// x / d rounded to nearest, from r = 1 / d rounded to nearest: the product x r
// is corrected once by its exact remainder (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990). The
// remainder is taken as q d - x, which keeps the sign of a zero. While x is
// finite, the quotient does not overflow and neither is near the subnormals, every
// step scales with powers of two, and over all significands of x and of an E4M3 d
// (6 has that of 1.5) the result is the rounded quotient: tests/test_quotient.py.
// No quotient overflows: x is at most 6.4 d unless d is the largest scale. Further
// down the quotient is off by some last bits, far below the lowest border of the
// codes made of it.
__device__ __forceinline__ float div_by(float x, float d, float r) {
  const float q = x * r;
  return __fmaf_rn(-__fmaf_rn(q, d, -x), r, q);
}

// One main-KV block: 16 values -> 8 bytes of E2M1 pairs and the E4M3 scale. The
// scale is amax / 6 rounded to nearest-even E4M3 (6 is the largest E2M1
// magnitude); each value is divided by the decoded scale and rounded to
// nearest-even E2M1, saturating. A zero scale stores zero codes.
__device__ __forceinline__ void encode_kv_fp4_values(const float (&f)[16], uint2& data, uint8_t& scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_abs3(amax, f[2 * i], f[2 * i + 1]);
  const bool finite = amax <= 3.402823466e38f;  // (an infinity has no remainder)
  const float q = finite ? div_by(amax, 6.0f, 1.0f / 6.0f) : amax;
  const uint32_t sc = cvt_e4m3x2(q, 0.0f) & 0xFFu;
  const float s = e4m3_to_f32(sc);
  uint32_t out[2] = {0, 0};
  if (s != 0.0f) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      if (finite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = div_by(f[8 * h + i], s, r);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(f[8 * h + i], s);
      }
      out[h] = cvt_e2m1x8(v);
    }
  }
  data = make_uint2(out[0], out[1]);
  scale = (uint8_t)sc;
}

// The same from 16 bf16 values (8 words of pairs, element 2i in the low half).
__device__ __forceinline__ void encode_kv_fp4_block(const uint32_t (&w)[8], uint2& data, uint8_t& scale) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
  encode_kv_fp4_values(f, data, scale);
}

}  // namespace csa2
