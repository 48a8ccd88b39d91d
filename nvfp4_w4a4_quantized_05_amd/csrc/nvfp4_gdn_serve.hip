// Gated DeltaNet for serving: one new token for each of many requests, whose
// fp32 states lie in a pool of slots (packed prompts: nvfp4_gdn_chunk.hip).
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

// One workgroup takes kCols columns of one request's head, a lane four columns
// and kRows rows of them.  HBM-bound: every state is read and written once,
// 128 KiB per request and head (the token's rows are under 2% of that), so all
// of a lane's state is asked for before anything else happens.  One reduction
// suffices, since
//     S_t^T q = alpha S_{t-1}^T q + (k . q) w
// needs only the old state, like u = S_{t-1}^T k: both sums meet in LDS once,
// then w, o and the new state follow.  The states stream past the caches (a
// model has dozens of layers' between two uses of one): non-temporal, 251
// requests x 32 heads take 178 us (5.9 TB/s) against 197 with plain accesses.
template <bool kXBf16, int kCols>
__global__ __launch_bounds__(256) void gdn_decode_kernel(GdnRows in, float* states, const int32_t* slots,
                                                         int n_slots, void* o, bool o_bf16, int64_t ldo) {
  constexpr int kParts = kD / kCols;
  constexpr int kLanes = kCols / 4, kGroups = 256 / kLanes, kRows = kD / kGroups;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts % in.n_v;
  const int64_t b = blockIdx.x / kParts / in.n_v;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cl = tid % kLanes, grp = tid / kLanes;
  const int col = part * kCols + cl * 4;  // first of the lane's columns
  const int r0 = grp * kRows;             // first of its rows
  const int hk = h / (in.n_v / in.n_qk);
  __shared__ floatx4_t red[2][4][kLanes];

  const int64_t o_at = b * ldo + (int64_t)h * kD + col;
  const int slot = slots ? slots[b] : (int)b;
  if (slot < 0 || slot >= n_slots) {  // an unused row of the batch
    if (grp == 0) store_o4(o, o_bf16, o_at, floatx4_t{0.0f, 0.0f, 0.0f, 0.0f});
    return;
  }
  floatx4_t* state = reinterpret_cast<floatx4_t*>(states + (((int64_t)slot * in.n_v + h) * kD + r0) * kD + col);
  floatx4_t S[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) S[r] = __builtin_nontemporal_load(state + r * (kD / 4));

  const int64_t q_at = b * in.ldx + in.q_col + (int64_t)hk * kD, k_at = b * in.ldx + in.k_col + (int64_t)hk * kD;
  floatx4_t k[kRows / 4], q[kRows / 4];
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i) {
    k[i] = load_val4<kXBf16>(in.x, k_at + r0 + 4 * i);
    q[i] = load_val4<kXBf16>(in.x, q_at + r0 + 4 * i);
  }
  float ka = load_val<kXBf16>(in.x, k_at + lane), kb = load_val<kXBf16>(in.x, k_at + 64 + lane);
  float qa = load_val<kXBf16>(in.x, q_at + lane), qb = load_val<kXBf16>(in.x, q_at + 64 + lane);
  const floatx4_t v = load_val4<kXBf16>(in.x, b * in.ldx + in.v_col + (int64_t)h * kD + col);
  const float alpha = expf(load_gate(in.gates, in.gates_bf16, b * in.ldg + in.g_col + h));
  const float beta = load_gate(in.gates, in.gates_bf16, b * in.ldg + in.beta_col + h);
  float k2 = wave_sum64(fmaf(ka, ka, kb * kb)), q2 = wave_sum64(fmaf(qa, qa, qb * qb));
  const float k_scale = large_row_scale(k2), q_scale = large_row_scale(q2);
  if (k_scale != 1.0f || q_scale != 1.0f) {  // the same in every lane
    ka *= k_scale, kb *= k_scale, qa *= q_scale, qb *= q_scale;
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) k[i][e] *= k_scale, q[i][e] *= q_scale;
    k2 = wave_sum64(fmaf(ka, ka, kb * kb));
    q2 = wave_sum64(fmaf(qa, qa, qb * qb));
  }
  const float rk = 1.0f / fmaxf(sqrtf(k2), kNormEps), rq = 1.0f / fmaxf(sqrtf(q2), kNormEps);
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
  if (lane < kLanes) {
    red[0][wave][lane] = u;
    red[1][wave][lane] = sq;
  }
  __syncthreads();
  u = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f}, sq = u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const floatx4_t x = red[0][i][cl], y = red[1][i][cl];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] += x[e], sq[e] += y[e];
  }
  floatx4_t w, ov;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = beta * (v[e] - u[e] * rk);
    ov[e] = (alpha * sq[e] * rq + kq * w[e]) * kRsqrtD;
    w[e] *= rk;
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) S[r][e] = fmaf(k[r / 4][r % 4], w[e], alpha * S[r][e]);
    __builtin_nontemporal_store(S[r], state + r * (kD / 4));
  }
  if (grp == 0) store_o4(o, o_bf16, o_at, ov);
}

// Below this many requests x value heads a head's columns are shared by two
// workgroups, to fill more CUs: 4 x 32 heads 7.7 -> 6.0 us, 16 x 32 13.4 -> 12.4;
// above, whole heads read longer runs: 64 x 32 51.2 -> 48.4 us, 251 x 32 191 -> 178.
constexpr int64_t kWholeHeads = 1024;

template <bool kXBf16, int kCols>
hipError_t launch_decode_cols(const GdnRows& in, int64_t batch, float* states, const int32_t* slots, int n_slots,
                              void* o, bool o_bf16, int64_t ldo, hipStream_t stream) {
  gdn_decode_kernel<kXBf16, kCols><<<(unsigned)(batch * in.n_v * (kD / kCols)), 256, 0, stream>>>(
      in, states, slots, n_slots, o, o_bf16, ldo);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdn_decode(const GdnRows& in, bool x_bf16, int64_t batch, float* states, const int32_t* slots,
                             int n_slots, void* o, bool o_bf16, int64_t ldo, hipStream_t stream) {
  const bool whole = batch * in.n_v >= kWholeHeads;
  const auto f = x_bf16 ? (whole ? launch_decode_cols<true, 128> : launch_decode_cols<true, 64>)
                        : (whole ? launch_decode_cols<false, 128> : launch_decode_cols<false, 64>);
  return f(in, batch, states, slots, n_slots, o, o_bf16, ldo, stream);
}

}  // namespace nvfp4
