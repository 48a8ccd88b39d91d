// Device-side helpers shared by the NVFP4 kernels (gfx950 / CDNA4).
//
// Format recap (picx.dev summary of arXiv 2609.04098, "Background", item 1):
// E2M1 values {0, .5, 1, 1.5, 2, 3, 4, 6} with a sign bit, one E4M3 scale per
// 16 values (blockmax / 6), one FP32 scale per tensor.  Dequantized values
// are E2M1 x E4M3 products: at most 6 significant bits between 2^-10 and
// 2688, which fp16 represents exactly (normal range 2^-14 .. 65504).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kBlock = 16;          // values per E4M3 block scale
constexpr float kE4M3Max = 448.0f;  // largest finite E4M3 (0x7E)
constexpr float kGlobalDiv = 2688.0f;  // 6 * 448

// E4M3 ("fn") byte -> fp32, exact (hardware conversion; subnormals kept).
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

// fp32 -> E4M3 byte, round-to-nearest-even.  Callers clamp to [0, 448]
// first: the hardware returns NaN (0x7F) for values rounding past 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float v) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false) & 0xFFu;
}

// Tensor scale from the absolute maximum: RN32(amax / 2688), 1.0 if zero.
// HIP's float division is correctly rounded (IEEE) by default.
__device__ __forceinline__ float tensor_scale_from_amax(float amax) {
  float g = amax / kGlobalDiv;
  return g == 0.0f ? 1.0f : g;
}

// Two fp32 values as bf16, round-to-nearest-even, a in the low half (NaN stays NaN).
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2v_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  float2v_t f;
  f[0] = a;
  f[1] = b;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}

// silu(z) = z / (1 + exp(-z)) with the hardware exp2 and reciprocal.  Both
// terms of the denominator carry a factor 2^-24, and so does z: with it the
// reciprocal stays a normal number down to results of 2^-126 (the hardware
// flushes subnormal reciprocals), at no more than one multiply.
__device__ __forceinline__ float silu(float z) {
  const float e = __builtin_amdgcn_exp2f(fmaf(-1.44269504088896340736f, z, -24.0f));
  return (z * 0x1p-24f) * __builtin_amdgcn_rcpf(e + 0x1p-24f);
}

// The largest i in 0 .. n - 1 for which before(i) holds, before(0) taken as
// true and before true up to some i only: the wave's lanes ask about 64
// places at a time.  All lanes of the wave must be active.
template <class F>
__device__ __forceinline__ int last_before(int n, F before) {
  const int lane = threadIdx.x & 63;
  int first = 0;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const bool yes = lane * step < n && before(first + lane * step);
    const int hits = max(__builtin_popcountll(__builtin_amdgcn_ballot_w64(yes)), 1);
    first += (hits - 1) * step;
    n = min(step, n - (hits - 1) * step);
  }
  return __builtin_amdgcn_readfirstlane(first);
}

// Row numbers of packed sequences that a call may use: cut off at 0 and T.
__device__ __forceinline__ int64_t row_clip(int32_t r, int64_t T) { return min(max((int64_t)r, (int64_t)0), T); }

// What a row of up to 256 finite values with the squared length `sum2` (as fp32 gives
// it, infinite on overflow) is multiplied by before it is used in place of its
// unit vector's numerator: 2^-70 from a length of 2^52 on.  Then neither its
// squared length (at most 2^124) nor a product of two such rows or their factors
// overflows or becomes subnormal, and its length stays past the least one that
// counts, 1e-6.  Exact but for values 2^-108 of the row.
__device__ __forceinline__ float large_row_scale(float sum2) { return sum2 < 0x1p104f ? 1.0f : 0x1p-70f; }

// Sum over the wave's 64 lanes, the same bits in every lane: each step adds
// the same two values in either order.
__device__ __forceinline__ float wave_sum64(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace nvfp4
