// attn_common.cuh -- what the attention kernels share: the fp16 instruction
// descriptor, exact FP4 / FP8 to fp16 conversion, the softmax's exponential and
// reductions across a warp.
#pragma once

#include "tc_common.cuh"

namespace csa2 {
namespace attn_tc {

// kind::f16 with fp16 A/B, fp32 accumulate; a_mn / b_mn select MN-major operands.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4)  // D format: f32 (A and B format fields 0: f16)
         | (a_mn & 1u) << 15 | (b_mn & 1u) << 16 | ((N >> 3) & 63u) << 17 | ((M >> 4) & 31u) << 24;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two E4M3 bytes (bits 0..7 and 8..15) to two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Two fp32 values to one fp16x2 word (`lo` in bits 0..15), round to nearest even.
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight E2M1 codes (the 32-bit w: channel i in bits 4i..4i+3) to eight exact
// fp16 values in four fp16x2 words (o0: channels 0, 1; ...; o3: 6, 7).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& o0, uint32_t& o1, uint32_t& o2, uint32_t& o3) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o0), "=r"(o1), "=r"(o2), "=r"(o3)
      : "r"(w));
}

// Transpose-reduce across a warp: lane L holds v[0..16) (one value per head);
// afterwards lane L returns the reduction over all 32 lanes of head L mod 16.
// v is overwritten.
template <bool kMax>
__device__ __forceinline__ float warp_transpose_reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int width = 8; width >= 1; width >>= 1) {
    const bool up = (lane & width) != 0;
#pragma unroll
    for (int i = 0; i < width; ++i) {
      const float keep = up ? v[i + width] : v[i];
      const float send = up ? v[i] : v[i + width];
      const float got = __shfl_xor_sync(0xffffffffu, send, width);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  const float o = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], o) : v[0] + o;
}

// 2^x (ex2.approx: relative error below 2^-22; +inf/-inf/NaN pass through).
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A hint: the cache line holding p is fetched into L2.
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace attn_tc
}  // namespace csa2
