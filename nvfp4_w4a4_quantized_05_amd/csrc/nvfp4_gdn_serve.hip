// Gated DeltaNet for serving: packed prompts, and one new token for each of
// many requests, with the fp32 states of the requests in a pool of slots.
//
// Per value head, S [d_k x d_v] = [128 x 128], q and k of unit length:
//     u_t = S_{t-1}^T k_t,  w_t = beta_t (v_t - u_t)
//     S_t = alpha_t S_{t-1} + k_t w_t^T,  o_t = S_t^T q_t / sqrt(128)
// with alpha_t = exp(g_t): the recurrence of nvfp4_gdn.hip (picx.dev summary
// page, "Gated DeltaNet Mechanics").
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kD = 128;
constexpr float kNormEps = 1e-6f;
constexpr float kRsqrtD = 0.08838834764831845f;  // 1 / sqrt(128)

template <bool kBf16>
__device__ __forceinline__ float load_val(const void* p, int64_t at) {
  if constexpr (kBf16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[at] << 16);
  return reinterpret_cast<const float*>(p)[at];
}
__device__ __forceinline__ float load_gate(const void* p, bool bf16, int64_t at) {
  return bf16 ? load_val<true>(p, at) : load_val<false>(p, at);
}
// 4 consecutive values, aligned to 4 values
template <bool kBf16>
__device__ __forceinline__ floatx4_t load_val4(const void* p, int64_t at) {
  if constexpr (kBf16) {
    const u32x2_t a = *reinterpret_cast<const u32x2_t*>(reinterpret_cast<const uint16_t*>(p) + at);
    floatx4_t f;
    f[0] = __uint_as_float(a[0] << 16);
    f[1] = __uint_as_float(a[0] & 0xFFFF0000u);
    f[2] = __uint_as_float(a[1] << 16);
    f[3] = __uint_as_float(a[1] & 0xFFFF0000u);
    return f;
  } else {
    return *reinterpret_cast<const floatx4_t*>(reinterpret_cast<const float*>(p) + at);
  }
}

__device__ __forceinline__ void store_o4(void* o, bool bf16, int64_t at, floatx4_t v) {
  if (bf16) {
    u32x2_t a;
    a[0] = pack_bf16(v[0], v[1]);
    a[1] = pack_bf16(v[2], v[3]);
    *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(o) + at) = a;
  } else {
    *reinterpret_cast<floatx4_t*>(reinterpret_cast<float*>(o) + at) = v;
  }
}

// One workgroup runs kCols columns of one head's state, a lane four columns
// and kRows rows of them.  A request's rows are t0 .. t1 - 1.
template <bool kXBf16, int kCols>
__device__ __forceinline__ void gdn_tokens(const GdnRows& in, int64_t t0, int64_t t1, int h, int part,
                                           const float* s_in, float* s_out, void* o, bool o_bf16, int64_t ldo) {
  constexpr int kLanes = kCols / 4, kGroups = 256 / kLanes, kRows = kD / kGroups;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cl = tid % kLanes, grp = tid / kLanes;
  const int col = part * kCols + cl * 4;       // first of the lane's columns
  const int r0 = grp * kRows;                  // first of its rows
  const int hk = h / (in.n_v / in.n_qk);
  __shared__ floatx4_t red[2][2][4][kLanes];

  floatx4_t S[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (s_in)
      S[r] = *reinterpret_cast<const floatx4_t*>(s_in + (int64_t)(r0 + r) * kD + col);
    else
      S[r] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t q_at = t * in.ldx + in.q_col + (int64_t)hk * kD, k_at = t * in.ldx + in.k_col + (int64_t)hk * kD;
    floatx4_t k[kRows / 4], q[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      k[i] = load_val4<kXBf16>(in.x, k_at + r0 + 4 * i);
      q[i] = load_val4<kXBf16>(in.x, q_at + r0 + 4 * i);
    }
    const float ka = load_val<kXBf16>(in.x, k_at + lane), kb = load_val<kXBf16>(in.x, k_at + 64 + lane);
    const float qa = load_val<kXBf16>(in.x, q_at + lane), qb = load_val<kXBf16>(in.x, q_at + 64 + lane);
    const floatx4_t v = load_val4<kXBf16>(in.x, t * in.ldx + in.v_col + (int64_t)h * kD + col);
    const float alpha = expf(load_gate(in.gates, in.gates_bf16, t * in.ldg + in.g_col + h));
    const float beta = load_gate(in.gates, in.gates_bf16, t * in.ldg + in.beta_col + h);
    const float rk = 1.0f / fmaxf(sqrtf(wave_sum64(fmaf(ka, ka, kb * kb))), kNormEps);
    const float rq = 1.0f / fmaxf(sqrtf(wave_sum64(fmaf(qa, qa, qb * qb))), kNormEps);
    const float kq = wave_sum64(fmaf(ka, qa, kb * qb)) * rk * rq;

    floatx4_t u = {0.0f, 0.0f, 0.0f, 0.0f}, sq = u;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = fmaf(S[r][e], k[r / 4][r % 4], u[e]);
        sq[e] = fmaf(S[r][e], q[r / 4][r % 4], sq[e]);
      }
    for (int m = kLanes; m < 64; m <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] += __shfl_xor(u[e], m, 64);
        sq[e] += __shfl_xor(sq[e], m, 64);
      }
    auto& buf = red[t & 1];
    if (lane < kLanes) {
      buf[0][wave][lane] = u;
      buf[1][wave][lane] = sq;
    }
    __syncthreads();
    u = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f}, sq = u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx4_t a = buf[0][i][cl], b = buf[1][i][cl];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] += a[e], sq[e] += b[e];
    }
    floatx4_t w, ov;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = beta * (v[e] - u[e] * rk);
      // S_t^T q = alpha S_{t-1}^T q + (k . q) w
      ov[e] = (alpha * sq[e] * rq + kq * w[e]) * kRsqrtD;
      w[e] *= rk;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] = fmaf(k[r / 4][r % 4], w[e], alpha * S[r][e]);
    if (grp == 0) store_o4(o, o_bf16, t * ldo + (int64_t)h * kD + col, ov);
  }
  if (s_out) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) *reinterpret_cast<floatx4_t*>(s_out + (int64_t)(r0 + r) * kD + col) = S[r];
  }
}

template <int kCols>
__device__ __forceinline__ void zero_rows(int64_t t0, int64_t t1, int h, int part, void* o, bool o_bf16, int64_t ldo) {
  for (int64_t t = t0 + threadIdx.x / (kCols / 4); t < t1; t += 256 / (kCols / 4))
    store_o4(o, o_bf16, t * ldo + (int64_t)h * kD + part * kCols + threadIdx.x % (kCols / 4) * 4,
             floatx4_t{0.0f, 0.0f, 0.0f, 0.0f});
}

// grid: requests x value heads x column parts, one row per request
template <bool kXBf16, int kCols>
__global__ __launch_bounds__(256) void gdn_decode_kernel(GdnRows in, float* states, const int32_t* slots,
                                                         int n_slots, void* o, bool o_bf16, int64_t ldo) {
  constexpr int kParts = kD / kCols;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts % in.n_v;
  const int64_t b = blockIdx.x / kParts / in.n_v;
  const int slot = slots ? slots[b] : (int)b;
  if (slot < 0 || slot >= n_slots) return zero_rows<kCols>(b, b + 1, h, part, o, o_bf16, ldo);
  float* s = states + ((int64_t)slot * in.n_v + h) * kD * kD;
  gdn_tokens<kXBf16, kCols>(in, b, b + 1, h, part, s, s, o, o_bf16, ldo);
}

}  // namespace

hipError_t launch_gdn_decode(const GdnRows& in, bool x_bf16, int64_t batch, float* states, const int32_t* slots,
                             int n_slots, void* o, bool o_bf16, int64_t ldo, hipStream_t stream) {
  constexpr int kCols = 64;
  const unsigned grid = (unsigned)(batch * in.n_v * (kD / kCols));
  const auto f = x_bf16 ? gdn_decode_kernel<true, kCols> : gdn_decode_kernel<false, kCols>;
  f<<<grid, 256, 0, stream>>>(in, states, slots, n_slots, o, o_bf16, ldo);
  return hipGetLastError();
}

}  // namespace nvfp4
