// Norm of each query and key head with the rotation by position, in one pass:
//
//   y = x / sqrt(mean_head(x^2) + eps) w,
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot dims,
//
// in fp32, rounded to bf16 once.  The angles come as a table of cosines and
// sines: formed from a position in fp32 they would be off by 2^-24 of it.
//
// HBM-bound: every value is held in registers between its load and its store.
// A lane owns 16 values of a head, chosen so that it owns both values of its
// eight pairs 8 l .. 8 l + 7: no exchange but the sum of squares over the
// head's d / 16 lanes.  A wave takes heads of one token, so its cosines and
// sines are loaded once for all of them.  Measured: 32768 tokens of 28 heads of
// 256 in bf16 184 us, 0.95 GB at 5.2 TB/s, a large copy's rate (5.3); 4099 tokens of
// 40 heads of 128 from fp32 33 us, 3.9 TB/s; 64 tokens 3.8 us.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

// 8 values at a 16-byte aligned place, bf16 or fp32.
template <bool kBf16>
__device__ __forceinline__ void load8(const void* base, int64_t at, float v[8]) {
  if constexpr (kBf16) {
    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
    const floatx4_t* p = reinterpret_cast<const floatx4_t*>(reinterpret_cast<const float*>(base) + at);
    const floatx4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  u32x4_t a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = a;
}

// kLanes = d / 16 lanes per head, 64 / kLanes heads at a time; `waves` waves
// share a token's heads.
template <bool kBf16, int kLanes>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkNormRope a, int waves) {
  constexpr int kHeads = 64 / kLanes;
  const int lane = threadIdx.x & 63, l = lane & (kLanes - 1);
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = wave / waves;
  if (t >= a.T) return;
  const int half = a.rot / 2, pair0 = 8 * l;
  const bool turns = pair0 < half;
  // the places of the lane's two runs of 8 values
  const int at0 = a.adjacent ? 16 * l : turns ? 8 * l : 16 * l;
  const int at1 = a.adjacent || !turns ? at0 + 8 : half + 8 * l;

  bool known = true;
  float cs[8], sn[8];
  if (a.n_axes == 1) {
    const int pos = a.pos[t];
    known = (unsigned)pos < (unsigned)a.n_pos;
    if (turns && known) {
      load8<false>(a.table, (int64_t)pos * a.rot + pair0, cs);
      load8<false>(a.table, (int64_t)pos * a.rot + half + pair0, sn);
    }
  } else {
    int pos[4];
    for (int x = 0; x < 4; ++x) {
      pos[x] = a.pos[(int64_t)min(x, a.n_axes - 1) * a.T + t];
      known = known && (unsigned)pos[x] < (unsigned)a.n_pos;
    }
    if (turns && known) {
      const uint32_t axes = a.axis[pair0 / 16] >> (pair0 % 16 * 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int x = axes >> (2 * e) & 3;
        const int p = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
        cs[e] = a.table[(int64_t)p * a.rot + pair0 + e];
        sn[e] = a.table[(int64_t)p * a.rot + half + pair0 + e];
      }
    }
  }
  float qw[16], kw[16];
  load8<false>(a.q_w, at0, qw);
  load8<false>(a.q_w, at1, qw + 8);
  load8<false>(a.k_w, at0, kw);
  load8<false>(a.k_w, at1, kw + 8);

  for (int h = (int)(wave % waves) * kHeads + lane / kLanes; h < a.hq + a.hk; h += waves * kHeads) {
    const bool is_q = h < a.hq;
    const int64_t from = t * a.ldx + (is_q ? a.q_col + (int64_t)h * a.d : a.k_col + (int64_t)(h - a.hq) * a.d);
    uint16_t* to = is_q ? a.q + t * a.ldq + (int64_t)h * a.d : a.k + t * a.ldk + (int64_t)(h - a.hq) * a.d;
    float v[16], eps = a.eps;
    load8<kBf16>(a.x, from + at0, v);
    load8<kBf16>(a.x, from + at1, v + 8);
    const auto sum_squares = [&] {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) s = fmaf(v[e], v[e], s);
#pragma unroll
      for (int m = 1; m < kLanes; m <<= 1) s += __shfl_xor(s, m, 64);
      return s;
    };
    float ss = sum_squares();
    // Heads of finite values may have squares past fp32 (from 1.1e18 on, if all 256 are): they, and eps, are made smaller first.
    if (__builtin_amdgcn_ballot_w64(!(ss < 0x1p104f))) {
      const float by = large_row_scale(ss);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= by;
      eps = eps * by * by;
      ss = sum_squares();
    }
    const float rms = 1.0f / sqrtf(ss / (float)a.d + eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = v[e] * rms * (is_q ? qw[e] : kw[e]);
    if (turns) {
      if (a.adjacent) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = v[2 * e], y = v[2 * e + 1];
          v[2 * e] = fmaf(x, cs[e], -(y * sn[e]));
          v[2 * e + 1] = fmaf(y, cs[e], x * sn[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = v[e], y = v[8 + e];
          v[e] = fmaf(x, cs[e], -(y * sn[e]));
          v[8 + e] = fmaf(y, cs[e], x * sn[e]);
        }
      }
    }
    if (!known) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.0f;
    }
    store8(to + at0, v);
    store8(to + at1, v + 8);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRope& a, hipStream_t stream) {
  const int per = 64 / (a.d / 16);                       // heads of a wave at a time
  const int groups = (a.hq + a.hk + per - 1) / per;      // of a token
  // few tokens: a wave for each group of heads; many: one wave for all of a token's
  const int waves = (int)(a.T >= 4096 ? 1 : a.T * groups <= 4096 ? groups : (4096 + a.T - 1) / a.T);
  const unsigned grid = (unsigned)((a.T * waves + 3) / 4);
#define NVFP4_ROPE(L)                                                                                        \
  (a.x_bf16 ? qk_norm_rope_kernel<true, L><<<grid, 256, 0, stream>>>(a, waves)                               \
            : qk_norm_rope_kernel<false, L><<<grid, 256, 0, stream>>>(a, waves))
  if (a.d == 64)
    NVFP4_ROPE(4);
  else if (a.d == 128)
    NVFP4_ROPE(8);
  else
    NVFP4_ROPE(16);
#undef NVFP4_ROPE
  return hipGetLastError();
}

}  // namespace nvfp4
