// The norms around a block, fused with what stands next to them.
//
//   add_rmsnorm    t = residual + scale x;  y = t / sqrt(mean(t^2) + eps) w
//   rmsnorm_gated  per group of a row: y = o / sqrt(mean(o^2) + eps) w silu(z),
//                  silu(z) = z / (1 + exp(-z))
//
// t goes out in the residual's type; y goes out in bf16 or fp32, or as NVFP4
// codes and block scales under a given tensor scale (what the projection that
// follows reads), or as both.  Everything between the loads and those stores
// is fp32: t is not rounded before its norm, y not before it is quantized.
//
// Both are HBM-bound: one pass, every value held in registers between its
// load and its stores.  A lane owns 16 consecutive values (one NVFP4 block, so
// quantize_block needs no exchange between lanes).  A lane's two 16-byte loads
// share cache lines with its neighbours' second ones, so they go through the
// caches: 32768 x 5120 bf16 takes 237 us (5.6 TB/s) against 277 with
// non-temporal loads and stores (fp32, where a lane has four: 431 against 842),
// the gated norm of 32768 x 4096 144 us (5.6 TB/s) against 150 (fp32: 236
// against 337); four or five times the values per lane took 295 us.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"
#include "nvfp4_quant_block.h"

namespace nvfp4 {
namespace {

// Vectors at any element's address: the memory path takes them.
typedef u32x4_t u32x4_at2 __attribute__((aligned(2)));
typedef floatx4_t floatx4_at4 __attribute__((aligned(4)));

// 16 values, bf16 or fp32.
template <bool kBf16>
__device__ __forceinline__ void load16(const void* base, int64_t at, float v[16]) {
  if constexpr (kBf16) {
    const u32x4_at2* p = reinterpret_cast<const u32x4_at2*>(reinterpret_cast<const uint16_t*>(base) + at);
    const u32x4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      v[8 + 2 * i] = __uint_as_float(b[i] << 16);
      v[9 + 2 * i] = __uint_as_float(b[i] & 0xFFFF0000u);
    }
  } else {
    const floatx4_at4* p = reinterpret_cast<const floatx4_at4*>(reinterpret_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx4_t t = p[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = t[e];
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void store16(void* base, int64_t at, const float v[16]) {
  if constexpr (kBf16) {
    u32x4_t a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      b[i] = pack_bf16(v[8 + 2 * i], v[9 + 2 * i]);
    }
    u32x4_at2* p = reinterpret_cast<u32x4_at2*>(reinterpret_cast<uint16_t*>(base) + at);
    p[0] = a;
    p[1] = b;
  } else {
    floatx4_at4* p = reinterpret_cast<floatx4_at4*>(reinterpret_cast<float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      floatx4_t t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = v[4 * i + e];
      p[i] = t;
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* p, int64_t at) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[at] << 16);
  return reinterpret_cast<const float*>(p)[at];
}
__device__ __forceinline__ void store_one(void* p, bool bf16, int64_t at, float v) {
  if (bf16)
    reinterpret_cast<uint16_t*>(p)[at] = (uint16_t)pack_bf16(v, 0.0f);
  else
    reinterpret_cast<float*>(p)[at] = v;
}

__device__ __forceinline__ void load_weight16(const float* w, int64_t at, float v[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const floatx4_t t = *reinterpret_cast<const floatx4_at4*>(w + at + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * i + e] = t[e];
  }
}

// y's destinations: values (or NULL) and NVFP4 codes with block scales (or NULL).
__device__ __forceinline__ void store_y(const NormOut& out, int64_t row, int64_t col, int64_t cols,
                                        const float y[16], float g, float r6) {
  if (out.y) {
    if (out.y_bf16)
      store16<true>(out.y, row * out.ldy + col, y);
    else
      store16<false>(out.y, row * out.ldy + col, y);
  }
  if (out.codes) {
    uint32_t w0, w1;
    const uint32_t s = quantize_block(y, g, r6, w0, w1);
    const int64_t b = (row * cols + col) / kBlock;
    u32x2_t c;
    c[0] = w0;
    c[1] = w1;
    __builtin_nontemporal_store(c, reinterpret_cast<u32x2_t*>(out.codes) + b);
    __builtin_nontemporal_store((uint8_t)s, out.scales + b);
  }
}

// Rows of up to 1,024 values: `lanes` (a power of two) lanes per row, a wave per
// workgroup; wider ones: the workgroup (lanes = blockDim.x, whole waves).
// kVec: lane l has the 16 consecutive values from 16 l; where less than 16 are
// left, the last 16 of the row, some of which the lane before it has too: both
// store the same bits, and since nothing is stored before the row's sum is
// known, neither loads what the other stored, in place either.  (With t out at
// once 32768 x 5120 takes 242 us in bf16 and 466 in fp32 instead of 237 and 431,
// 16,000 x 704 bf16 16.8 instead of 17.7.)  Rows of less than 16: value e is
// column e * lanes + l.
// 8,000 rows of 1,033 bf16 take 16 us, 22 with loads of single values; 30,000 of
// 100 take 8, 17 with a wave per row.
template <bool kXBf16, bool kRBf16, bool kVec>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(const void* x, int64_t ldx, const void* residual,
                                                           int64_t ldr, float scale, const float* __restrict__ w,
                                                           float eps, int64_t rows, int64_t cols, int lanes,
                                                           void* sum, int64_t lds, NormOut out) {
  const int tid = threadIdx.x, l = tid & (lanes <= 64 ? lanes - 1 : 1023);
  const int64_t row = lanes <= 64 ? (int)(blockIdx.x * 64 + tid) >> __builtin_ctz(lanes) : blockIdx.x;
  const bool live = 16 * l < cols && row < rows;
  const int col0 = min(16 * l, (int)cols - 16), before = 16 * l - col0;
  float t[16], ss = 0.0f;
  if constexpr (kVec) {
    if (live) {
      load16<kXBf16>(x, row * ldx + col0, t);
      if (residual) {
        float r[16];
        load16<kRBf16>(residual, row * ldr + col0, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) t[e] = fmaf(scale, t[e], r[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) t[e] *= scale;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = e < before ? ss : fmaf(t[e], t[e], ss);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int col = e * lanes + l;
      if (col < cols && row < rows) {
        const float r = residual ? load_one<kRBf16>(residual, row * ldr + col) : 0.0f;
        t[e] = fmaf(scale, load_one<kXBf16>(x, row * ldx + col), r);
        ss = fmaf(t[e], t[e], ss);
      }
    }
  }
  if (lanes >= 64) {
    __shared__ float part[16];
    ss = wave_sum64(ss);
    if (lanes > 64) {
      if ((tid & 63) == 0) part[tid >> 6] = ss;
      __syncthreads();
      ss = 0.0f;
      for (int i = 0; i < lanes / 64; ++i) ss += part[i];
    }
  } else {
    for (int m = 1; m < lanes; m <<= 1) ss += __shfl_xor(ss, m, 64);
  }
  const float rms = 1.0f / sqrtf(ss / (float)cols + eps);
  if constexpr (kVec) {
    if (live) {
      if (sum) store16<kRBf16>(sum, row * lds + col0, t);
      float wv[16];
      load_weight16(w, col0, wv);
#pragma unroll
      for (int e = 0; e < 16; ++e) t[e] = t[e] * rms * wv[e];
      const float g = out.codes ? *out.gs : 1.0f;
      store_y(out, row, col0, cols, t, g, __builtin_amdgcn_rcpf(6.0f * g));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int col = e * lanes + l;
      if (col < cols && row < rows) {
        if (sum) store_one(sum, kRBf16, row * lds + col, t[e]);
        store_one(out.y, out.y_bf16, row * out.ldy + col, t[e] * rms * w[col]);
      }
    }
  }
}

// One lane per 16 values; the group's lanes (group / 16, a power of two up to 64) are consecutive
// and add their squares with lane exchanges.  y may be in the place of o or z:
// a lane reads no value but those it writes.
template <bool kOBf16, bool kZBf16>
__global__ __launch_bounds__(256) void rmsnorm_gated_kernel(const void* o, int64_t ldo, const void* z, int64_t ldz,
                                                            const float* __restrict__ w, float eps, int64_t rows,
                                                            int64_t cols, int group, NormOut out) {
  const int64_t chunks = cols / 16;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / chunks, col = (i - row * chunks) * 16;
  // whole groups are past the end together: chunks is a multiple of the group's lanes
  const bool live = row < rows;
  float ov[16], zv[16], ss = 0.0f;
  if (live) {
    load16<kOBf16>(o, row * ldo + col, ov);
    load16<kZBf16>(z, row * ldz + col, zv);
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(ov[e], ov[e], ss);
  }
  for (int m = 1; m < group / 16; m <<= 1) ss += __shfl_xor(ss, m, 64);
  if (!live) return;
  const float rms = 1.0f / sqrtf(ss / (float)group + eps);
  float wv[16];
  load_weight16(w, col & (group - 1), wv);
#pragma unroll
  for (int e = 0; e < 16; ++e) ov[e] = ov[e] * rms * wv[e] * silu(zv[e]);
  const float g = out.codes ? *out.gs : 1.0f;
  store_y(out, row, col, cols, ov, g, __builtin_amdgcn_rcpf(6.0f * g));
}

template <bool kXBf16, bool kRBf16>
hipError_t launch_add_typed(bool vec, const void* x, int64_t ldx, const void* residual, int64_t ldr, float scale,
                            const float* w, float eps, int64_t rows, int64_t cols, void* sum, int64_t lds,
                            const NormOut& out, hipStream_t stream) {
  int lanes = 1;
  while (lanes < 64 && 16 * lanes < cols) lanes *= 2;
  if (16 * lanes < cols) lanes = (int)((cols + 16 * 64 - 1) / (16 * 64) * 64);
  const unsigned threads = lanes <= 64 ? 64u : (unsigned)lanes;
  const int64_t per = threads / lanes;
  const auto f = vec ? add_rmsnorm_kernel<kXBf16, kRBf16, true> : add_rmsnorm_kernel<kXBf16, kRBf16, false>;
  f<<<(unsigned)((rows + per - 1) / per), threads, 0, stream>>>(x, ldx, residual, ldr, scale, w, eps, rows, cols, lanes,
                                                                sum, lds, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm(const void* x, bool x_bf16, int64_t ldx, const void* residual, bool r_bf16,
                              int64_t ldr, float scale, const float* w, float eps, int64_t rows, int64_t cols,
                              void* sum, int64_t lds, const NormOut& out, hipStream_t stream) {
  const bool vec = cols >= 16;
  const auto f = x_bf16 ? (r_bf16 ? launch_add_typed<true, true> : launch_add_typed<true, false>)
                        : (r_bf16 ? launch_add_typed<false, true> : launch_add_typed<false, false>);
  return f(vec, x, ldx, residual, ldr, scale, w, eps, rows, cols, sum, lds, out, stream);
}

hipError_t launch_rmsnorm_gated(const void* o, bool o_bf16, int64_t ldo, const void* z, bool z_bf16, int64_t ldz,
                                const float* w, float eps, int64_t rows, int64_t cols, int group,
                                const NormOut& out, hipStream_t stream) {
  const unsigned grid = (unsigned)((rows * (cols / 16) + 255) / 256);
  const auto f = o_bf16 ? (z_bf16 ? rmsnorm_gated_kernel<true, true> : rmsnorm_gated_kernel<true, false>)
                        : (z_bf16 ? rmsnorm_gated_kernel<false, true> : rmsnorm_gated_kernel<false, false>);
  f<<<grid, 256, 0, stream>>>(o, ldo, z, ldz, w, eps, rows, cols, group, out);
  return hipGetLastError();
}

}  // namespace nvfp4
