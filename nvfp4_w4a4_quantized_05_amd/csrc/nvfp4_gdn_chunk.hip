// Gated DeltaNet over packed prompts, 64 tokens at a time on the matrix cores.
//
// The recurrence (per value head, S [d_k x d_v] = [128 x 128], |q| = |k| = 1)
//     w_t = beta_t (v_t - S_{t-1}^T k_t),  S_t = alpha_t S_{t-1} + k_t w_t^T,
//     o_t = S_t^T q_t / sqrt(128),         alpha_t = exp(g_t)
// is linear in S, so a chunk of C = 64 tokens can be written out.  With G_i the
// sum of the chunk's g up to token i, B_i = G_i - g_i the sum before it, and S
// the state at its start, S_{i-1} = e^{B_i} S + sum_{j<i} e^{B_i - G_j} k_j w_j^T, so
//     w_i + beta_i sum_{j<i} e^{B_i - G_j} (k_i . k_j) w_j = beta_i (v_i - e^{B_i} S^T k_i).
// With A_ij = beta_i e^{B_i - G_j} (k_i . k_j) for j < i and T = (I + A)^-1 diag(beta):
//     W  = T (V - diag(e^B) K S)                                    (64 x 128)
//     O  = (diag(e^G) Q S + P W) / sqrt(128),  P_ij = e^{G_i - G_j} (q_i . k_j), j <= i
//     S' = e^{G_C} S + K^T diag(e^{G_C - G_j}) W
// T and P do not depend on S.  One kernel makes them for every chunk at once;
// a second one walks the chunks of each sequence with S in registers.
//
// Precision.  q, k and v are bf16, so every product of two of them is exact in
// the matrix cores.  S, T, V - ... and W are fp32 and enter as the sum of three
// bf16 numbers (8 + 8 + 8 bits: exact), with the six largest of the nine
// products where both sides are split: the state is as exact as an fp32 sum.
// For O alone, whose result is bf16, S, W and P enter as two terms each (at
// most 2^-15 of S and 2^-16 of W and P off), with three of the four products
// of P and W: o is the 64-bit result rounded to bf16, but where that lies this
// close to the middle of two neighbours (0.0017 off it, 2-norm, relative, all
// of it that rounding; 0.0021 with P in one term).
// Decays inside a chunk are exponentials of differences of G, which is summed
// in fp64 and kept as two floats, so that a strong decay before both tokens
// does not cost the difference its digits.
//
// Infinities and NaN.  Token by token, one in q_t reaches o_t alone, one in k_t
// or a gate every output from t on, one in column c of v_t that column's; an
// earlier token's output is never touched.  In a product over a chunk it would
// be, by the zeros above the diagonals of T and P.  So a k, gate or v that is
// not finite is replaced by zero, and NaN put in where it belongs: in the row
// factor of Q S and the chunk's decay for k and gates, in the column's outputs
// and state for v.
#include <climits>

#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kD = 128;        // head dimension
constexpr int kC = 64;         // tokens per chunk
constexpr float kNormEps = 1e-6f;
constexpr float kRsqrtD = 0.08838834764831845f;  // 1 / sqrt(128)
// exp of less is 0 in fp32; keeps differences of G finite for alpha = 0
constexpr float kMinGate = -200.0f;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short shortx4_t __attribute__((ext_vector_type(4)));

// What the first kernel leaves for a chunk and value head, in the order the
// second one's lanes read it.  A 64 x 64 lower triangular matrix is kept as
// matrix-core A operands of 16 rows x 32 columns: rows 16 w .. + 15, columns
// 32 s .. + 31, s <= w / 2, a lane's eight columns being 32 s + 4 g + {0..3}
// and 32 s + 16 + 4 g + {0..3} (g = lane / 16): the order in which two
// 16 x 16 results lie in the lanes, so that results are operands as they are.
constexpr int kOperand = 1024;                     // bytes: 64 lanes x 8 bf16
constexpr int kBlocks = 6;                         // (w, s) with s <= w / 2
constexpr int kOffP = 3 * kBlocks * kOperand;      // after T's three terms
constexpr int kOffVec = kOffP + 2 * kBlocks * kOperand;  // after P's two: a, b, c [64] and e^{G_C}, fp32
constexpr int kUnitBytes = kOffVec + 1024;
// And for a chunk and q/k head: K, then Q, as operands of 16 tokens x 32
// columns, [32 columns][16 tokens], so that a load is 1 KiB in a row.  K's
// lanes are turned within each 16 (below) for reading it by columns.
constexpr int kHeadBytes = 2 * 16 * kOperand;
constexpr int kOffQ = 16 * kOperand;
// Place in a K operand of the lane that holds token m's columns 8 g .. + 7:
// the places of four neighbouring tokens' columns then lie in different LDS
// banks when they are read column by column.
__device__ __forceinline__ constexpr int k_place(int m, int g) { return 16 * g + ((m + 4 * g) & 15); }
__device__ __forceinline__ constexpr int block_of(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }

constexpr int kBufferFlags = 0x00020000;    // raw buffer, 32-bit data format
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every resource used here
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kBufferFlags);
}
__device__ __forceinline__ u32x4_t load16b(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t wave_off = 0) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, wave_off, 0));
}

__device__ __forceinline__ floatx4_t mfma_bf16(u32x4_t a, u32x4_t b, floatx4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// Behind the last matrix instructions of a step, with their A and B operands:
// keeps those registers taken for four more cycles of issue.  A vector
// instruction that wrote such a register right behind the matrix instruction
// was seen to change its operand on gfx950, and the compiler puts no wait
// states there.  A CPU test looks for closer ones in the compiled code.
__device__ __forceinline__ void hold(const u32x4_t& x) { __asm__ volatile("" ::"v"(x)); }
__device__ __forceinline__ void hold(const floatx4_t& x) { __asm__ volatile("" ::"v"(x)); }
template <class X, int N>
__device__ __forceinline__ void hold(const X (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) hold(x[i]);
}
template <class... X>
__device__ __forceinline__ void mfma_settle(const X&... x) {
  __builtin_amdgcn_sched_barrier(0);
  __asm__ volatile("s_nop 3");
  (hold(x), ...);
  __builtin_amdgcn_sched_barrier(0);
}

// a = hi + mid + lo exactly, each a bf16 (hi rounded to nearest); two values packed.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
  const uint32_t ma = __float_as_uint(ra) & 0xFFFF0000u, mb = __float_as_uint(rb) & 0xFFFF0000u;
  mid = __builtin_amdgcn_perm(mb, ma, 0x07060302u);
  lo = __builtin_amdgcn_perm(__float_as_uint(rb - __uint_as_float(mb)), __float_as_uint(ra - __uint_as_float(ma)),
                             0x07060302u);
}

// a as the sum of two bf16 numbers, both rounded to nearest (2^-16 of a off at most); two values packed.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

__device__ __forceinline__ u32x4_t join(u32x2_t a, u32x2_t b) {
  u32x4_t r;
  r[0] = a[0], r[1] = a[1], r[2] = b[0], r[3] = b[1];
  return r;
}

// Workspace place of a sequence's first chunk.  cu / 64 + s leaves room for
// one partial chunk per sequence, so places need no sum over sequences.
__device__ __forceinline__ int64_t first_place(int64_t start, int s) { return start / kC + s; }

// LDS writes made visible to the workgroup without waiting for loads from
// memory in flight (the next chunk's).
__device__ __forceinline__ void lds_barrier() {
  __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ---------------------------------------------------------------- chunk by chunk, independent of the state
//
// One workgroup per chunk and q/k head; it makes T, P and the row factors of
// each value head of the group.  Wave w owns token rows 16 w .. + 15.  The
// products k . k and q . k are formed transposed (rows j in the accumulators,
// columns i in the lanes), which is P's and T's operand order.  The inverse
// of I + A goes by blocks, in fp32: each wave substitutes forward through its
// 16 x 16 diagonal block, then blocks of 32 and of 64 are joined by
// -X_22 A_21 X_11 with fp32 matrix products.  (Summing powers of A instead
// would overflow for equal keys, whose inverse is harmless.)
// Bound by what it moves: 32,768 tokens with 16 / 32 heads take 196-202 us for
// 0.34 GB read and 0.79 GB written (5.6 TB/s; a plain copy of 2 GB 4.9).
constexpr int kKStride = kD + 8;   // bf16 per LDS row of K
constexpr int kXStride = kC + 4;   // floats per LDS row of A, T

__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void gdn_chunk_prepare_kernel(
    GdnRows in, const int32_t* __restrict__ cu, int n_seqs, int64_t T, uint8_t* __restrict__ ws,
    uint8_t* __restrict__ wsh, int split) {
  __shared__ __attribute__((aligned(16))) uint16_t kl[kC * kKStride];
  __shared__ __attribute__((aligned(16))) float X[kC * kXStride];
  // K is read only before the first head's gates; then its place takes four blocks of 16 x 16
  floatx4_t(&yb)[4][64] = *reinterpret_cast<floatx4_t(*)[4][64]>(kl);
  __shared__ float rk_l[kC], rq_l[kC], ghi_l[4][kC], glo_l[4][kC], alpha_l[4][kC], beta_l[4][kC];
  __shared__ int k_bad_l[kC];

  // `split` workgroups per chunk and q/k head share its value heads
  const int group = in.n_v / in.n_qk, heads = group / split;
  const int hk = blockIdx.x / split % in.n_qk, hv0 = blockIdx.x % split * heads;
  const int64_t place = blockIdx.x / split / in.n_qk;
  // the last sequence whose first place is not past this one
  const int s = last_before(n_seqs, [&](int i) { return first_place(row_clip(cu[i], T), i) <= place; });
  const int64_t start = row_clip(cu[s], T), end = row_clip(cu[s + 1], T);
  const int64_t t0 = start + (place - first_place(start, s)) * kC;
  if (place < first_place(start, s) || t0 >= end) return;
  const int rows = (int)min((int64_t)kC, end - t0);

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  const uint32_t ld = (uint32_t)in.ldx * 2;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(reinterpret_cast<const uint16_t*>(in.x) + t0 * in.ldx, (int64_t)rows * ld);
  u32x4_t kf[4], qf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = (uint32_t)(16 * w + m) * ld + (uint32_t)(hk * kD + 32 * i + 8 * g) * 2;
    const bool live = 16 * w + m < rows;
    kf[i] = load16b(rx, live ? at + (uint32_t)in.k_col * 2 : kOutside);
    qf[i] = load16b(rx, live ? at + (uint32_t)in.q_col * 2 : kOutside);
  }
  const auto length2 = [](const u32x4_t (&x)[4]) {  // of token 16 w + m: the four lanes that share it
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = __uint_as_float(x[i][e] << 16), x1 = __uint_as_float(x[i][e] & 0xFFFF0000u);
        sum = fmaf(x0, x0, fmaf(x1, x1, sum));
      }
    sum += __shfl_xor(sum, 16, 64);
    return sum + __shfl_xor(sum, 32, 64);
  };
  float k2 = length2(kf), q2 = length2(qf);
  const float k_scale = large_row_scale(k2), q_scale = large_row_scale(q2);
  if (__builtin_amdgcn_ballot_w64(k_scale != 1.0f || q_scale != 1.0f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kf[i][e] = pack_bf16(__uint_as_float(kf[i][e] << 16) * k_scale, __uint_as_float(kf[i][e] & 0xFFFF0000u) * k_scale);
        qf[i][e] = pack_bf16(__uint_as_float(qf[i][e] << 16) * q_scale, __uint_as_float(qf[i][e] & 0xFFFF0000u) * q_scale);
      }
    k2 = length2(kf);
    q2 = length2(qf);
  }
  const bool k_bad = !(k2 <= __FLT_MAX__);  // a value that is not finite: what large_row_scale leaves cannot overflow
  uint8_t* head = wsh + (place * in.n_qk + hk) * kHeadBytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) kf[i][e] = k_bad ? 0u : kf[i][e];
    if (hv0 == 0) {
      *reinterpret_cast<u32x4_t*>(head + (4 * i + w) * kOperand + k_place(m, g) * 16) = kf[i];
      *reinterpret_cast<u32x4_t*>(head + kOffQ + (4 * i + w) * kOperand + lane * 16) = qf[i];
    }
    *reinterpret_cast<u32x4_t*>(&kl[(16 * w + m) * kKStride + 32 * i + 8 * g]) = kf[i];
  }
  const float rk_i = 1.0f / fmaxf(sqrtf(k2), kNormEps);             // token i = 16 w + m
  const float rq_i = kRsqrtD / fmaxf(sqrtf(q2), kNormEps);
  if (g == 0) rk_l[16 * w + m] = rk_i, rq_l[16 * w + m] = rq_i, k_bad_l[16 * w + m] = k_bad;
  __syncthreads();

  // rows j = 16 tile + 4 g + e, column i, of the unit vectors' products (q's with 1 / sqrt(128))
  floatx4_t kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = qk[j] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (j > w) continue;
    u32x4_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const u32x4_t*>(&kl[(16 * j + m) * kKStride + 32 * i + 8 * g]);
      kk[j] = mfma_bf16(a[i], kf[i], kk[j]);
      qk[j] = mfma_bf16(a[i], qf[i], qk[j]);
    }
    mfma_settle(a, kf, qf);
    const floatx4_t rk = *reinterpret_cast<const floatx4_t*>(&rk_l[16 * j + 4 * g]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kk[j][e] *= rk[e] * rk_i;
      qk[j][e] *= rk[e] * rq_i;
    }
    __builtin_amdgcn_sched_barrier(0);  // one tile's operands at a time
  }

  for (int hv = 0; hv < heads; ++hv) {
    const int h = hk * group + hv0 + hv;
    const __amdgpu_buffer_rsrc_t unit = make_rsrc(ws + (place * in.n_v + h) * kUnitBytes, kUnitBytes);
    // the lane's number, unknown to the compiler anew for each head: else it
    // computes every LDS address before the loop and holds them (over 100 registers)
    int lane = tid & 63;
    __asm__ volatile("" : "+v"(lane));
    const int m = lane & 15, g = lane >> 4;
    if (hv % 4 == 0) {  // the next four heads' gates, one per wave, lane = token: running sums in fp64, base 2
      if (hv > 0) __syncthreads();
      float gate = 0.0f, beta = 0.0f;
      if (hv + w < heads && lane < rows) {
        const int64_t at = (t0 + lane) * in.ldg + h + w;
        if (in.gates_bf16) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(in.gates) + at;
          gate = __uint_as_float((uint32_t)p[in.g_col] << 16);
          beta = __uint_as_float((uint32_t)p[in.beta_col] << 16);
        } else {
          const float* p = reinterpret_cast<const float*>(in.gates) + at;
          gate = p[in.g_col];
          beta = p[in.beta_col];
        }
      }
      gate = gate < kMinGate ? kMinGate : gate;
      // the first token with a k or gate that is not finite: it and those behind it write nothing
      const uint64_t bad = __builtin_amdgcn_ballot_w64(k_bad_l[lane] || !(fabsf(gate) <= __FLT_MAX__) ||
                                                       !(fabsf(beta) <= __FLT_MAX__));
      const bool lost = bad && lane >= __builtin_ctzll(bad);
      if (lost) gate = beta = 0.0f;
      const double step = (double)gate * 1.4426950408889634;
      double sum = step;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_up(sum, o, 64);
        if (lane >= o) sum += up;
      }
      const float ghi = (float)sum;
      const float total = __shfl(ghi, 63, 64);
      ghi_l[w][lane] = ghi;
      glo_l[w][lane] = (float)(sum - (double)ghi);
      alpha_l[w][lane] = __builtin_amdgcn_exp2f((float)step);
      beta_l[w][lane] = beta;
      if (hv + w < heads) {
        // row factors: of K S, of Q S, and of the writes to the chunk's end
        float* vec = reinterpret_cast<float*>(ws + (place * in.n_v + h + w) * kUnitBytes + kOffVec);
        vec[lane] = __builtin_amdgcn_exp2f((float)(sum - step)) * rk_l[lane];
        vec[kC + lane] = lost ? __builtin_nanf("") : __builtin_amdgcn_exp2f(ghi) * rq_l[lane];
        vec[2 * kC + lane] = __builtin_amdgcn_exp2f((float)(__shfl(sum, 63, 64) - sum)) * rk_l[lane];
        if (lane == 0) vec[3 * kC] = bad ? __builtin_nanf("") : __builtin_amdgcn_exp2f(total);
      }
      __syncthreads();
    }
    const int hw = hv % 4;

    // A (fp32, to LDS) and P (two bf16 terms, out)
    const int i = 16 * w + m;
    const float alpha_i = alpha_l[hw][i], beta_i = beta_l[hw][i];
    const float bhi = i ? ghi_l[hw][max(i - 1, 0)] : 0.0f, blo = i ? glo_l[hw][max(i - 1, 0)] : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > (w | 1)) continue;
      floatx4_t p = {0.0f, 0.0f, 0.0f, 0.0f};
      if (j <= w) {
        const floatx4_t gh = *reinterpret_cast<const floatx4_t*>(&ghi_l[hw][16 * j + 4 * g]);
        const floatx4_t gl = *reinterpret_cast<const floatx4_t*>(&glo_l[hw][16 * j + 4 * g]);
        floatx4_t a;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = __builtin_amdgcn_exp2f((bhi - gh[e]) + (blo - gl[e]));  // e^{G_{i-1} - G_j}
          a[e] = beta_i * d * kk[j][e];
          p[e] = alpha_i * d * qk[j][e];
          if (j == w) {
            const int jj = 4 * g + e;  // j - 16 w; above the diagonal d may be infinite
            a[e] = jj < m ? a[e] : 0.0f;
            p[e] = jj < m ? p[e] : jj == m ? qk[j][e] : 0.0f;
          }
        }
        *reinterpret_cast<floatx4_t*>(&X[i * kXStride + 16 * j + 4 * g]) = a;
      }
      u32x2_t pp[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        split2(p[2 * e], p[2 * e + 1], hi, lo);
        pp[0][e] = hi;
        pp[1][e] = lo;
      }
#pragma unroll
      for (int term = 0; term < 2; ++term)
        __builtin_amdgcn_raw_buffer_store_b64(pp[term], unit, (uint32_t)(lane * 16 + (j & 1) * 8),
                                              kOffP + (term * kBlocks + block_of(w, j / 2)) * kOperand, 0);
    }
    __builtin_amdgcn_wave_barrier();  // the diagonal block is this wave's own

    // diagonal block w: lane m solves column m, x_r = [r = m] - sum_{k<r} A_rk x_k
    {
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float v = r == m ? 1.0f : 0.0f;
#pragma unroll
        for (int k4 = 0; k4 < r; k4 += 4) {
          const floatx4_t a = *reinterpret_cast<const floatx4_t*>(&X[(16 * w + r) * kXStride + 16 * w + k4]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k4 + e < r) v = fmaf(-a[e], x[k4 + e], v);
        }
        x[r] = v;
        if (r % 2) __asm__ volatile("" ::"v"(x[r]) : "memory");  // rows read a few ahead, not all 16 (160 registers)
      }
      __builtin_amdgcn_wave_barrier();  // all reads of the block before its inverse overwrites it
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (g == 0) X[(16 * w + r) * kXStride + 16 * w + m] = x[r];
    }
    __syncthreads();

    // blocks as matrix-core operands: A operand rows are read along, B operands down the columns
    auto a_op = [&](int r, int c) { return *reinterpret_cast<const floatx4_t*>(&X[(16 * r + m) * kXStride + 16 * c + 4 * g]); };
    auto b_op = [&](int r, int c) {
      floatx4_t b;
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = X[(16 * r + 4 * g + e) * kXStride + 16 * c + m];
      return b;
    };
    auto product = [&](floatx4_t a, floatx4_t b, floatx4_t acc) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
      mfma_settle(a, b);
      return acc;
    };
    auto put = [&](int r, int c, floatx4_t v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) X[(16 * r + 4 * g + e) * kXStride + 16 * c + m] = -v[e];
    };
    const floatx4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    if (w < 2) {  // blocks (1, 0) and (3, 2)
      const int c = 2 * w, r = c + 1;
      put(r, c, product(a_op(r, r), product(a_op(r, c), b_op(c, c), zero), zero));
    }
    __syncthreads();
    {  // blocks (2..3, 0..1): wave w has row 2 + w / 2, column w % 2
      const int r = 2 + w / 2, c = w & 1;
      floatx4_t y = zero;
      if (c == 0) y = product(a_op(r, 0), b_op(0, 0), y);
      y = product(a_op(r, 1), b_op(1, c), y);
      yb[w][lane] = y;
      __syncthreads();
      floatx4_t x = product(a_op(r, 2), yb[c][lane], zero);
      if (r == 3) x = product(a_op(3, 3), y, x);
      put(r, c, x);
    }
    __syncthreads();

    // T = (I + A)^-1 diag(beta), split in three, in operand order
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      if (sb > w / 2) continue;
      u32x4_t t[3];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = 2 * sb + half;
        floatx4_t v = zero;
        if (j <= w) {
          v = a_op(w, j);
          const floatx4_t b = *reinterpret_cast<const floatx4_t*>(&beta_l[hw][16 * j + 4 * g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= b[e];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi3, mid3, lo3;
          split3(v[2 * e], v[2 * e + 1], hi3, mid3, lo3);
          t[0][2 * half + e] = hi3;
          t[1][2 * half + e] = mid3;
          t[2][2 * half + e] = lo3;
        }
      }
#pragma unroll
      for (int term = 0; term < 3; ++term)
        __builtin_amdgcn_raw_buffer_store_b128(t[term], unit, (uint32_t)(lane * 16),
                                               (term * kBlocks + block_of(w, sb)) * kOperand, 0);
    }
    __syncthreads();  // X is free again
  }
}

// ---------------------------------------------------------------- the walk over a sequence's chunks
//
// One workgroup per sequence, value head and kT tiles of 16 state columns
// (columns do not meet); eight waves, two per SIMD.  Waves 0-3 carry the state from chunk to
// chunk, waves 4-7 make the outputs beside them.
//   State wave w holds state rows 32 w .. + 31 as two accumulators and
// multiplies them with its own 32 columns of K for all 64 tokens; the four
// waves' partial sums meet in LDS.  From there on it has token rows 16 w .. +
// 15: V - diag(a) K S, then (after an exchange) T times that, which is W, then
// (after another) the update of its state rows.  Three barriers a chunk.
//   Output wave w has token rows 16 w .. + 15: Q S from the state's terms that
// the state waves share, then P W.  It forms both transposed (rows = state
// columns, lanes = tokens), so that a lane holds four neighbours of a row of o.
// The output waves also bring V and the row factors to LDS.
//   Issuing loads bounds the walk as much as the chain of steps does (about 20
// cycles each on the path to the cache): a chunk takes 66.  Up to 128 registers
// two workgroups of one tile share a CU, which takes 16,384 tokens in 8 sequences (32 value
// heads) from 521 to 458 us; hence offsets that a wave has in common are kept in
// scalar registers.
//   Measured on 32,768 tokens, 32 value heads: 752-785 us in a kernel trace, 1.5
// a chunk (the whole call, untraced, takes 920-926 us, 720 of them the walk); the
// matrix cores are busy for 23% of it, and a state wave's own chain takes 1.1 us
// even without loads.
// Accumulator row 4 c + e of state tile t is row 32 w + 8 c + 4 t + e of S, so
// that a lane's rows of both tiles are eight neighbours.
constexpr int kCols = 16;
constexpr int kScanThreads = 512;
constexpr int kTStride = 40;  // bf16 per LDS row of a wave's K columns

template <int kT>
struct ScanShared {
  floatx4_t part[4][3][kT][64];  // K S: [token tile][its other waves][column tile][lane]
  u32x2_t rest[3][4][kT][64];    // V - diag(a) K S: [term][token tile][column tile][lane]
  u32x2_t wr[5][4][kT][64];      // W: three terms (scaled) for the state, two for o
  u32x4_t state[4][2][kT][64];   // S's first two terms: [32 rows][term][column tile][lane]
  uint16_t kt[4][kC * kTStride]; // [wave]: its 32 columns of K
  uint16_t v[kT][kC * kCols];    // V
  float vec[2][256];             // row factors a, b, c [64] and e^{G_C} (and as much that is not read)
  int lost[kT * kCols];          // a column's first token whose value is not finite
  float decay[kT][64][2];        // [column tile][lane][0]: e^{G_C}, NaN where the lane's column is lost
};

// One unit's rows and workspace, chunk by chunk; chunks past the end have
// empty resources (at chunk 0's address), and nothing uses what they load.
struct ChunkSource {
  const uint8_t* unit;   // of chunk 0
  const uint8_t* head;
  const uint16_t* v;     // first row's part of V
  uint16_t* o;
  int64_t unit_step, head_step, v_step, o_step;  // bytes, bytes, values, values per chunk
  uint32_t v_ld, o_ld;   // bytes per row
  int n_chunks, last_rows;
  __device__ __forceinline__ int rows(int c) const { return c < n_chunks - 1 ? kC : c < n_chunks ? last_rows : 0; }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t units(int c) const {
    return make_rsrc(unit + (c < n_chunks ? c : 0) * unit_step, c < n_chunks ? kUnitBytes : 0);
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t heads(int c) const {
    return make_rsrc(head + (c < n_chunks ? c : 0) * head_step, c < n_chunks ? kHeadBytes : 0);
  }
};

// kB: blocks of 32 columns that a wave's 16 rows of T and P have left of the
// diagonal: 1 for waves 0 and 1, 2 for waves 2 and 3.
template <int kB>
struct StateOperands {
  u32x4_t k[4];      // [t]: token tile (w + t) % 4
  u32x4_t t[3][kB];  // [term][32 columns]
};

template <int kB, int kT>
struct OutputOperands {
  u32x4_t q[4], p[2][kB];  // [32 columns], [term][32 columns]
  u32x4_t shared[kT];  // waves 0, 1: half a row of V's tile, row 32 w + lane / 2; wave 2: row factors
};

template <int kB, int kT>
__device__ __forceinline__ void scan_state(const ChunkSource& src, ScanShared<kT>& sh, int w, int lane,
                                           floatx4_t (&S)[kT][2]) {
  const int m = lane & 15, g = lane >> 4;
  const floatx4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  typedef __attribute__((address_space(3))) shortx4_t lds_shortx4_t;

  auto fetch_k = [&](int c, StateOperands<kB>& f) {
    const __amdgpu_buffer_rsrc_t r = src.heads(c);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      f.k[t] = load16b(r, (uint32_t)(k_place(m, g) * 16), (uint32_t)((4 * w + (w + t) % 4) * kOperand));
  };
  auto fetch_t = [&](int c, StateOperands<kB>& f) {
    const __amdgpu_buffer_rsrc_t r = src.units(c);
#pragma unroll
    for (int sb = 0; sb < kB; ++sb)
#pragma unroll
      for (int term = 0; term < 3; ++term)
        f.t[term][sb] = load16b(r, (uint32_t)(lane * 16), (uint32_t)((term * kBlocks + block_of(w, sb)) * kOperand));
  };

  // One chunk with its operands in f; those of chunk `next` are asked for in
  // pieces between the steps, so that the loads do not queue in front of one.
  auto chunk = [&](const StateOperands<kB>& f, int next, StateOperands<kB>& fn) {
    __builtin_amdgcn_sched_barrier(0);
    // K's columns, read back transposed below (this wave's own)
#pragma unroll
    for (int t = 0; t < 4; ++t) *reinterpret_cast<u32x4_t*>(&sh.kt[w][(16 * ((w + t) % 4) + m) * kTStride + 8 * g]) = f.k[t];
    floatx4_t own[kT];
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      u32x4_t sp[3];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi, mid, lo;
          split3(S[n][t][2 * e], S[n][t][2 * e + 1], hi, mid, lo);
          sp[0][2 * t + e] = hi;
          sp[1][2 * t + e] = mid;
          sp[2][2 * t + e] = lo;
        }
      floatx4_t ks[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) ks[t] = mfma_bf16(f.k[t], sp[0], zero);
#pragma unroll
      for (int term = 1; term < 3; ++term)
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = mfma_bf16(f.k[t], sp[term], ks[t]);
      mfma_settle(f.k, sp);
      sh.state[w][0][n][lane] = sp[0];
      sh.state[w][1][n][lane] = sp[1];
      __builtin_amdgcn_sched_barrier(0);
      // tile (w + t) % 4 goes to its wave; this wave's own is t = 0
#pragma unroll
      for (int t = 1; t < 4; ++t) sh.part[(w + t) % 4][t - 1][n][lane] = ks[t];
      own[n] = ks[0];
    }
    lds_barrier();

    const floatx4_t fa = *reinterpret_cast<const floatx4_t*>(&sh.vec[0][16 * w + 4 * g]);
    const floatx4_t fc = *reinterpret_cast<const floatx4_t*>(&sh.vec[0][2 * kC + 16 * w + 4 * g]);
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      floatx4_t kst = own[n];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const floatx4_t x = sh.part[w][i][n][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) kst[e] += x[e];
      }
      // lane 4 j + c of a group of 16 reads columns 4 c .. + 3 of row 4 g + j; the lanes get them back by column
      const u32x2_t vt = __builtin_bit_cast(
          u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4_t*)&sh.v[n][(16 * w + 4 * g + m / 4) * kCols + 4 * (m % 4)]));
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r[e] = fmaf(-fa[e], kst[e], __uint_as_float(e & 1 ? vt[e / 2] & 0xFFFF0000u : vt[e / 2] << 16));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, mid, lo;
        split3(r[2 * e], r[2 * e + 1], hi, mid, lo);
        sh.rest[0][w][n][lane][e] = hi;
        sh.rest[1][w][n][lane][e] = mid;
        sh.rest[2][w][n][lane][e] = lo;
      }
    }
    fetch_k(next, fn);
    lds_barrier();

    // W = T (V - ..): the six products of terms i, j with i + j <= 2
    floatx4_t wt[kT];
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      floatx4_t w0 = zero, w1 = zero;
      u32x4_t rv[3][kB];
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int sb = 0; sb < kB; ++sb)
          rv[term][sb] = join(sh.rest[term][2 * sb][n][lane], sh.rest[term][2 * sb + 1][n][lane]);
      int turn = 0;
#pragma unroll
      for (int order = 2; order >= 0; --order)
#pragma unroll
        for (int i = 0; i <= order; ++i)
#pragma unroll
          for (int sb = 0; sb < kB; ++sb) {  // two sums in turn: a product waits for the one before it
            floatx4_t& acc = turn++ % 2 ? w1 : w0;
            acc = mfma_bf16(f.t[i][sb], rv[order - i][sb], acc);
          }
      mfma_settle(f.t, rv);
#pragma unroll
      for (int e = 0; e < 4; ++e) wt[n][e] = w0[e] + w1[e];
    }
    u32x4_t kc[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // as above: lane 4 c + e gets column 8 c + 4 t + e of four token rows
          const uint16_t* at = &sh.kt[w][(32 * sb + 16 * half + 4 * g + m / 4) * kTStride + 8 * (m % 4) + 4 * t];
          const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4_t*)at));
          kc[t][sb][2 * half] = v[0];
          kc[t][sb][2 * half + 1] = v[1];
        }
#pragma unroll
    for (int n = 0; n < kT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = wt[n][2 * e], y = wt[n][2 * e + 1];
        uint32_t hi, mid, lo;
        split3(x * fc[2 * e], y * fc[2 * e + 1], hi, mid, lo);
        sh.wr[0][w][n][lane][e] = hi;
        sh.wr[1][w][n][lane][e] = mid;
        sh.wr[2][w][n][lane][e] = lo;
        split2(x, y, hi, lo);
        sh.wr[3][w][n][lane][e] = hi;
        sh.wr[4][w][n][lane][e] = lo;
      }
    fetch_t(next, fn);
    lds_barrier();

    // S' = e^{G_C} S + K^T (c W)
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      const float decay = sh.decay[n][lane][0];
      u32x4_t wv[3][2];
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) wv[i][sb] = join(sh.wr[i][2 * sb][n][lane], sh.wr[i][2 * sb + 1][n][lane]);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][t][e] *= decay;
#pragma unroll
        for (int term = 2; term >= 0; --term)
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) S[n][t] = mfma_bf16(kc[t][sb], wv[term][sb], S[n][t]);
      }
      mfma_settle(kc, wv);
    }
  };

  StateOperands<kB> f0, f1;
  fetch_k(0, f0);
  fetch_t(0, f0);
  int c = 0;
  for (; c + 1 < src.n_chunks; c += 2) {
    chunk(f0, c + 1, f1);
    chunk(f1, c + 2, f0);
  }
  if (c < src.n_chunks) chunk(f0, c + 1, f1);
}

template <int kB, int kT>
__device__ __forceinline__ void scan_output(const ChunkSource& src, ScanShared<kT>& sh, int w, int lane) {
  const int m = lane & 15, g = lane >> 4;
  auto fetch = [&](int c, OutputOperands<kB, kT>& f) {
    const __amdgpu_buffer_rsrc_t rh = src.heads(c), r = src.units(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.q[i] = load16b(rh, (uint32_t)(lane * 16), (uint32_t)(kOffQ + (4 * i + w) * kOperand));
#pragma unroll
    for (int term = 0; term < 2; ++term)
#pragma unroll
      for (int sb = 0; sb < kB; ++sb)
        f.p[term][sb] = load16b(r, (uint32_t)(lane * 16), (uint32_t)(kOffP + (term * kBlocks + block_of(w, sb)) * kOperand));
    if constexpr (kB == 1) {
      const __amdgpu_buffer_rsrc_t rv =
          make_rsrc(src.v + (c < src.n_chunks ? c : 0) * src.v_step, (int64_t)src.rows(c) * src.v_ld);
#pragma unroll
      for (int n = 0; n < kT; ++n)
        f.shared[n] = load16b(rv, (uint32_t)(32 * w + lane / 2) * src.v_ld + (lane & 1) * 16 + n * kCols * 2);
    } else {
      f.shared[0] = load16b(r, w == 2 ? (uint32_t)(kOffVec + lane * 16) : kOutside);
    }
  };
  // what all waves need of a chunk, between the third barrier of the one before and its own first
  auto share = [&](int c, OutputOperands<kB, kT>& f) {
    if constexpr (kB == 1) {
#pragma unroll
      for (int n = 0; n < kT; ++n) {
        u32x4_t& v = f.shared[n];
        uint32_t full = 0;  // the carry of an exponent of all ones
#pragma unroll
        for (int e = 0; e < 4; ++e) full |= (v[e] & 0x7F807F80u) + 0x00800080u;
        if (full & 0x80008000u)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t exponent = 0x7F80u << 16 * (e % 2);
            if ((v[e / 2] & exponent) == exponent) {
              v[e / 2] &= 0xFFFFu << 16 * (1 - e % 2);
              atomicMin(&sh.lost[n * kCols + 8 * (lane & 1) + e], c * kC + 32 * w + lane / 2);
            }
          }
        *reinterpret_cast<u32x4_t*>(&sh.v[n][512 * w + 8 * lane]) = v;
      }
    } else
      *reinterpret_cast<u32x4_t*>(&sh.vec[w - 2][4 * lane]) = f.shared[0];
  };
  auto chunk = [&](int c, const OutputOperands<kB, kT>& f, OutputOperands<kB, kT>& fn) {
    fetch(c + 1, fn);
    lds_barrier();
    const float b = sh.vec[0][kC + 16 * w + m];
    floatx4_t ov[kT];
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      ov[n] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
      u32x4_t st[2][4];
#pragma unroll
      for (int term = 1; term >= 0; --term)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st[term][i] = sh.state[i][term][n][lane];
          ov[n] = mfma_bf16(st[term][i], f.q[i], ov[n]);
        }
      mfma_settle(st, f.q);
      if (kB == 2 && w == 2)
        sh.decay[n][lane][0] = sh.lost[n * kCols + m] < (c + 1) * kC ? __builtin_nanf("") : sh.vec[0][3 * kC];
    }
    lds_barrier();
#pragma unroll
    for (int n = 0; n < kT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) ov[n][e] *= b;
    lds_barrier();
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(src.o + c * src.o_step, (int64_t)src.rows(c) * src.o_ld);
#pragma unroll
    for (int n = 0; n < kT; ++n) {
      u32x4_t wo[2][kB];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int sb = 0; sb < kB; ++sb) wo[i][sb] = join(sh.wr[3 + i][2 * sb][n][lane], sh.wr[3 + i][2 * sb + 1][n][lane]);
#pragma unroll
      for (int order = 1; order >= 0; --order)  // terms i of P and order - i of W, the small products first
#pragma unroll
        for (int i = 0; i <= order; ++i)
#pragma unroll
          for (int sb = 0; sb < kB; ++sb) ov[n] = mfma_bf16(wo[order - i][sb], f.p[i][sb], ov[n]);
      mfma_settle(wo, f.p);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c * kC + 16 * w + m >= sh.lost[n * kCols + 4 * g + e]) ov[n][e] = __builtin_nanf("");
      u32x2_t out;
      out[0] = pack_bf16(ov[n][0], ov[n][1]);
      out[1] = pack_bf16(ov[n][2], ov[n][3]);
      __builtin_amdgcn_raw_buffer_store_b64(out, ro, (uint32_t)(16 * w + m) * src.o_ld + 8 * g + n * kCols * 2, 0, 0);
    }
    share(c + 1, fn);
  };
  OutputOperands<kB, kT> f0, f1;
  fetch(0, f0);
  share(0, f0);
  int c = 0;
  for (; c + 1 < src.n_chunks; c += 2) {
    chunk(c, f0, f1);
    chunk(c + 1, f1, f0);
  }
  if (c < src.n_chunks) chunk(c, f0, f1);
}

// The sequence at place n by length, longest first (workgroups start in the
// order of their numbers, so the long ones are not left for the end); the
// n-th itself with more sequences than lanes, which level out anyway.
__device__ __forceinline__ int nth_longest(const int32_t* cu, int n_seqs, int64_t T, int n) {
  if (n_seqs < 2 || n_seqs > 64) return n;
  const int lane = threadIdx.x & 63;
  int len = -1, rank = 0;
  if (lane < n_seqs) len = (int)max(row_clip(cu[lane + 1], T) - row_clip(cu[lane], T), (int64_t)0);
  for (int j = 0; j < n_seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    rank += other > len || (other == len && j < lane);
  }
  return __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < n_seqs && rank == n));
}

template <int kT>
__global__ __launch_bounds__(kScanThreads) void gdn_chunk_scan_kernel(
    GdnRows in, const int32_t* __restrict__ cu, int n_seqs, int64_t T, const uint8_t* ws, const uint8_t* wsh,
    const float* s_in, float* s_out, const int32_t* __restrict__ slots, int n_slots,
    uint16_t* o, int64_t ldo) {
  constexpr int kParts = kD / (kT * kCols);
  __shared__ ScanShared<kT> sh;
  // the column parts of a unit run on one XCD and share its L2
  const int unit = (int)(blockIdx.x / (8 * kParts)) * 8 + blockIdx.x % 8;
  const int part = blockIdx.x / 8 % kParts;
  if (unit >= n_seqs * in.n_v) return;
  const int s = nth_longest(cu, n_seqs, T, unit / in.n_v), h = unit % in.n_v, hk = h / (in.n_v / in.n_qk);
  const int64_t start = row_clip(cu[s], T), end = max(row_clip(cu[s + 1], T), start);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = part * kT * kCols;
  const int slot = slots ? slots[s] : s;
  if (slot < 0 || slot >= n_slots) {
    for (int64_t t = start + tid / (kT * kCols); t < end; t += kScanThreads / (kT * kCols))
      o[t * ldo + h * kD + col + tid % (kT * kCols)] = 0;
    return;
  }
  ChunkSource src;
  const int64_t place = first_place(start, s);
  src.unit_step = (int64_t)in.n_v * kUnitBytes;
  src.unit = ws + place * src.unit_step + (int64_t)h * kUnitBytes;
  src.head_step = (int64_t)in.n_qk * kHeadBytes;
  src.head = wsh + place * src.head_step + (int64_t)hk * kHeadBytes;
  src.v_step = kC * in.ldx;
  src.v = reinterpret_cast<const uint16_t*>(in.x) + start * in.ldx + in.v_col + h * kD + col;
  src.o_step = kC * ldo;
  src.o = o + start * ldo + h * kD + col;
  src.n_chunks = (int)((end - start + kC - 1) / kC);
  src.last_rows = (int)(end - start - (int64_t)(src.n_chunks - 1) * kC);
  src.v_ld = (uint32_t)in.ldx * 2;
  src.o_ld = (uint32_t)ldo * 2;
  if (tid < kT * kCols) sh.lost[tid] = INT_MAX;
  __syncthreads();
  if (wave >= 6) return scan_output<2, kT>(src, sh, wave - 4, lane);
  if (wave >= 4) return scan_output<1, kT>(src, sh, wave - 4, lane);

  const int64_t at = ((int64_t)slot * in.n_v + h) * kD * kD + (32 * wave + 8 * (lane >> 4)) * kD + col + (lane & 15);
  floatx4_t S[kT][2];
#pragma unroll
  for (int n = 0; n < kT; ++n)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[n][t][e] = s_in ? s_in[at + (4 * t + e) * kD + n * kCols] : 0.0f;
  if (wave < 2)
    scan_state<1, kT>(src, sh, wave, lane, S);
  else
    scan_state<2, kT>(src, sh, wave, lane, S);
  if (s_out) {
#pragma unroll
    for (int n = 0; n < kT; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_out[at + (4 * t + e) * kD + n * kCols] = S[n][t][e];
  }
}

// ---------------------------------------------------------------- the same walk, one wave per 16 columns
//
// With many sequences the walk need not be split over waves: here a wave
// keeps all 128 rows of its 16 columns in registers (eight accumulators) and
// goes through a chunk alone.  What it multiplies comes out of one product in
// the lane order that the next one takes, so nothing is exchanged; the eight
// waves of a workgroup (the 128 columns of one unit) share the chunk's K, Q, T
// and P in LDS, two buffers deep, with one barrier a chunk.  Measured on 32,768
// tokens in 48 sequences, 32 value heads: 463-492 us; the matrix cores are busy
// for 43% of it.
constexpr int kWideWaves = 8;
constexpr int kWideThreads = 64 * kWideWaves;

constexpr int kWideUnitBytes = (kUnitBytes + kWideWaves * kOperand - 1) / (kWideWaves * kOperand) * (kWideWaves * kOperand);

struct WideShared {
  uint8_t head[2][kHeadBytes];                // [chunk parity]: K and Q
  uint8_t unit[2][kWideUnitBytes];            // T, P and the row factors as they lie in the workspace
  uint16_t v[kWideWaves][kC * kCols];         // [wave]: V's columns
};

__global__ __launch_bounds__(kWideThreads) void gdn_chunk_wide_kernel(
    GdnRows in, const int32_t* __restrict__ cu, int n_seqs, int64_t T, const uint8_t* ws, const uint8_t* wsh,
    const float* s_in, float* s_out, const int32_t* __restrict__ slots, int n_slots, uint16_t* o, int64_t ldo) {
  __shared__ __attribute__((aligned(16))) WideShared sh;
  typedef __attribute__((address_space(3))) shortx4_t lds_shortx4_t;
  const int h = blockIdx.x % in.n_v, hk = h / (in.n_v / in.n_qk);
  const int s = nth_longest(cu, n_seqs, T, blockIdx.x / in.n_v);
  const int64_t start = row_clip(cu[s], T), end = max(row_clip(cu[s + 1], T), start);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int col = kCols * w;
  const int slot = slots ? slots[s] : s;
  if (slot < 0 || slot >= n_slots) {
    for (int64_t t = start + tid / kD; t < end; t += kWideThreads / kD) o[t * ldo + h * kD + tid % kD] = 0;
    return;
  }
  const int n_chunks = (int)((end - start + kC - 1) / kC);
  const int64_t place = first_place(start, s);
  const uint32_t v_ld = (uint32_t)in.ldx * 2, o_ld = (uint32_t)ldo * 2;
  auto rows = [&](int c) { return max((int64_t)0, min((int64_t)kC, end - start - (int64_t)c * kC)); };
  auto units = [&](int c) {
    return make_rsrc(ws + ((place + (c < n_chunks ? c : 0)) * in.n_v + h) * kUnitBytes, c < n_chunks ? kUnitBytes : 0);
  };
  auto heads = [&](int c) {
    return make_rsrc(wsh + ((place + (c < n_chunks ? c : 0)) * in.n_qk + hk) * kHeadBytes, c < n_chunks ? kHeadBytes : 0);
  };

  // This wave's share of what goes to LDS: an eighth of K, Q, T, P and the row factors (what lies past the unit's end
  // loads as zeros), its columns of V.  No branches: a load in one makes its use wait for every load in flight.
  constexpr int kHeadShare = kHeadBytes / kOperand / kWideWaves, kUnitShare = kWideUnitBytes / kOperand / kWideWaves;
  u32x4_t sk[kHeadShare], st[kUnitShare], sv[2];
  auto stage = [&](int c) {
    const __amdgpu_buffer_rsrc_t rh = heads(c), ru = units(c);
#pragma unroll
    for (int i = 0; i < kHeadShare; ++i) sk[i] = load16b(rh, (uint32_t)((kHeadShare * w + i) * kOperand + lane * 16));
#pragma unroll
    for (int i = 0; i < kUnitShare; ++i) st[i] = load16b(ru, (uint32_t)((kUnitShare * w + i) * kOperand + lane * 16));
    const __amdgpu_buffer_rsrc_t rv =
        make_rsrc(reinterpret_cast<const uint16_t*>(in.x) + (start + (c < n_chunks ? (int64_t)c * kC : 0)) * in.ldx + in.v_col + h * kD + col,
                  rows(c) * v_ld);
#pragma unroll
    for (int i = 0; i < 2; ++i) sv[i] = load16b(rv, (uint32_t)(32 * i + lane / 2) * v_ld + (lane & 1) * 16);
  };
  auto put = [&](int c) {
    const int p = c & 1;
#pragma unroll
    for (int i = 0; i < kHeadShare; ++i)
      *reinterpret_cast<u32x4_t*>(&sh.head[p][(kHeadShare * w + i) * kOperand + lane * 16]) = sk[i];
#pragma unroll
    for (int i = 0; i < kUnitShare; ++i)
      *reinterpret_cast<u32x4_t*>(&sh.unit[p][(kUnitShare * w + i) * kOperand + lane * 16]) = st[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4_t*>(&sh.v[w][512 * i + 8 * lane]) = sv[i];
  };

  // row 4 c + e of accumulator S[i][t] is row 32 i + 8 c + 4 t + e of S
  const int64_t at = ((int64_t)slot * in.n_v + h) * kD * kD + 8 * g * kD + col + m;
  floatx4_t S[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][t][e] = s_in ? s_in[at + (32 * i + 4 * t + e) * kD] : 0.0f;

  const floatx4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  int lost = INT_MAX;  // the lane's column's first token whose V - diag(a) K S is not finite
  stage(0);
  put(0);
  for (int c = 0; c < n_chunks; ++c) {
    lds_barrier();
    stage(c + 1);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* k_lds = sh.head[c & 1];
    const uint8_t* q_lds = k_lds + kOffQ + lane * 16;
    const uint8_t* t_lds = sh.unit[c & 1] + lane * 16;
    const uint8_t* p_lds = t_lds + kOffP;
    const float* vec = reinterpret_cast<const float*>(sh.unit[c & 1] + kOffVec);

    // K S and Q S (the latter transposed: rows = state columns, lanes = tokens)
    floatx4_t ks[4] = {zero, zero, zero, zero}, qs[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4_t sp[3];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi, mid, lo;
          split3(S[i][t][2 * e], S[i][t][2 * e + 1], hi, mid, lo);
          sp[0][2 * t + e] = hi;
          sp[1][2 * t + e] = mid;
          sp[2][2 * t + e] = lo;
        }
      u32x4_t k[4], q[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        k[t] = *reinterpret_cast<const u32x4_t*>(k_lds + (4 * i + t) * kOperand + k_place(m, g) * 16);
        q[t] = *reinterpret_cast<const u32x4_t*>(q_lds + (4 * i + t) * kOperand);
      }
      // a product into an accumulator waits for the one before it: eight accumulators in turn
#pragma unroll
      for (int term = 0; term < 3; ++term) {
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = mfma_bf16(k[t], sp[term], ks[t]);
        if (term < 2)
#pragma unroll
          for (int t = 0; t < 4; ++t) qs[t] = mfma_bf16(sp[term], q[t], qs[t]);
      }
      mfma_settle(sp, k, q);
    }

    // V - diag(a) K S, split in three: [term][32 tokens]
    float nan = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const u32x2_t vt = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                         (lds_shortx4_t*)&sh.v[w][(16 * t + 4 * g + m / 4) * kCols + 4 * (m % 4)]));
      const floatx4_t fa = *reinterpret_cast<const floatx4_t*>(&vec[16 * t + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ks[t][e] = fmaf(-fa[e], ks[t][e], __uint_as_float(e & 1 ? vt[e / 2] & 0xFFFF0000u : vt[e / 2] << 16));
        nan = fmaf(ks[t][e], 0.0f, nan);
      }
    }
    if (__builtin_amdgcn_ballot_w64(nan != nan)) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(fabsf(ks[t][e]) <= __FLT_MAX__)) {
            lost = min(lost, c * kC + 16 * t + 4 * g + e);
            ks[t][e] = 0.0f;
          }
      lost = min(lost, __shfl_xor(lost, 16, 64));
      lost = min(lost, __shfl_xor(lost, 32, 64));
    }
    u32x4_t rv[3][2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, mid, lo;
        split3(ks[t][2 * e], ks[t][2 * e + 1], hi, mid, lo);
        rv[0][t / 2][2 * (t % 2) + e] = hi;
        rv[1][t / 2][2 * (t % 2) + e] = mid;
        rv[2][t / 2][2 * (t % 2) + e] = lo;
      }
    // W = T (V - ..), six products; then diag(c) W in three terms and W in two.  Two row tiles at a time, two sums each.
    u32x4_t wv[3][2], wo[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      floatx4_t acc[2][2] = {{zero, zero}, {zero, zero}};  // [tile][parity]
#pragma unroll
      for (int sb = 0; sb <= u; ++sb) {
        u32x4_t tf[2][3];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int term = 0; term < 3; ++term)
            tf[t][term] = *reinterpret_cast<const u32x4_t*>(t_lds + (term * kBlocks + block_of(2 * u + t, sb)) * kOperand);
        int n = 0;
#pragma unroll
        for (int order = 0; order < 3; ++order)
#pragma unroll
          for (int i = 0; i <= order; ++i, ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[t][n % 2] = mfma_bf16(tf[t][i], rv[order - i][sb], acc[t][n % 2]);
        mfma_settle(tf, rv);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const floatx4_t fc = *reinterpret_cast<const floatx4_t*>(&vec[2 * kC + 32 * u + 16 * t + 4 * g]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = acc[t][0][2 * e] + acc[t][1][2 * e], y = acc[t][0][2 * e + 1] + acc[t][1][2 * e + 1];
          uint32_t hi, mid, lo;
          split3(x * fc[2 * e], y * fc[2 * e + 1], hi, mid, lo);
          wv[0][u][2 * t + e] = hi;
          wv[1][u][2 * t + e] = mid;
          wv[2][u][2 * t + e] = lo;
          split2(x, y, hi, lo);
          wo[0][u][2 * t + e] = hi;
          wo[1][u][2 * t + e] = lo;
        }
      }
    }
    // O = b Q S + P W, transposed like Q S
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(o + (start + (int64_t)c * kC) * ldo + h * kD + col, rows(c) * o_ld);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float b = vec[kC + 16 * t + m];
#pragma unroll
      for (int e = 0; e < 4; ++e) qs[t][e] *= b;
    }
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      u32x4_t p[4][2];  // [row tile][term]
#pragma unroll
      for (int t = 2 * sb; t < 4; ++t)
#pragma unroll
        for (int term = 0; term < 2; ++term)
          p[t][term] = *reinterpret_cast<const u32x4_t*>(p_lds + (term * kBlocks + block_of(t, sb)) * kOperand);
      // terms i of P and order - i of W, the small products first
#pragma unroll
      for (int order = 1; order >= 0; --order)
#pragma unroll
        for (int i = 0; i <= order; ++i)
#pragma unroll
          for (int t = 2 * sb; t < 4; ++t) qs[t] = mfma_bf16(wo[order - i][sb], p[t][i], qs[t]);
      if (sb == 0)
        mfma_settle(p, wo);
      else
        mfma_settle(p[2], p[3], wo);
    }
    const bool any_lost = __builtin_amdgcn_ballot_w64(lost != INT_MAX) != 0;
    if (any_lost)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int from = __shfl(lost, 4 * g + e, 64);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (c * kC + 16 * t + m >= from) qs[t][e] = __builtin_nanf("");
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      u32x2_t out;
      out[0] = pack_bf16(qs[t][0], qs[t][1]);
      out[1] = pack_bf16(qs[t][2], qs[t][3]);
      __builtin_amdgcn_raw_buffer_store_b64(out, ro, (uint32_t)(16 * t + m) * o_ld + 8 * g, 0, 0);
    }

    // S' = e^{G_C} S + K^T (c W)
    const float decay = lost != INT_MAX ? __builtin_nanf("") : vec[3 * kC];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {  // four accumulators in turn
#pragma unroll
      for (int i = j; i < j + 2; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[i][t][e] *= decay;
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        u32x4_t kT[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // lane 4 c + e of a group of 16 gets column 8 c + 4 t + e of token rows 4 g .. + 3
              const uint8_t* from =
                  k_lds + (4 * (j + i) + 2 * sb + half) * kOperand + k_place(4 * g + m / 4, m % 4) * 16 + 8 * t;
              const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4_t*)from));
              kT[i][t][2 * half] = v[0];
              kT[i][t][2 * half + 1] = v[1];
            }
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) S[j + i][t] = mfma_bf16(kT[i][t], wv[term][sb], S[j + i][t]);
        mfma_settle(kT, wv);
      }
    }
    put(c + 1);
  }
  if (s_out) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_out[at + (32 * i + 4 * t + e) * kD] = S[i][t][e];
  }
}

// Places in the workspace: first_place() of the last sequence plus its chunks is at most this.
int64_t chunk_places(int64_t T, int64_t n_seqs) { return T / kC + n_seqs + 1; }

// From this many sequences x value heads on, one workgroup walks a whole unit.
// It needs two thirds of the CU time per chunk, but leaves a CU to each unit and
// takes 5.0 us a chunk instead of 1.4, so a few long units would be left over.
// The host does not know the lengths and takes them for about equal: one long
// sequence among short or empty ones takes that long a chunk here as well.
// Measured, split in two tiles / whole, 32 value heads: 32,768 tokens in 48
// sequences 922 / 680 us, in 20 (640 units) 811 / 752, in 16 (512) 806 / 820,
// 28,000 in 14 (448) 699 / 776, 16,384 in 8 (256) 424 / 654.
constexpr int64_t kWideUnits = 512;
// From this many on, a workgroup of the split form has two column tiles, which
// halves the loads of a chunk's operands but leaves a CU to one workgroup.
// Measured, one / two tiles, 32 value heads: 8,192 tokens in 4 sequences (128
// units) 224 / 242 us, 16,000 in 5 (160) 452 / 397, 3,000 in 6 (192) 83 / 89,
// 16,000 in 6 442 / 394, 30,000 in 6 802 / 717, 27,000 in 7 (224) 722 / 647, 16,384
// in 8 (256) 454 / 388, 8,191 in 12 (384) 240 / 221; 16,000 in 16 with 12 value
// heads (192) 170 / 166, 20,000 in 48 with 4 (192) 78 / 84.
constexpr int64_t kPairUnits = 192;
// Below this many chunks x q/k heads, the preparation takes one workgroup per
// value head instead of one per q/k head (which makes the group's K and Q
// products once): 300 tokens x 4 heads 11 -> 9 us.
constexpr int64_t kFewChunkHeads = 256;

}  // namespace

size_t gdn_prefill_workspace_bytes(int64_t T, int64_t n_seqs, int n_qk, int n_v) {
  return (size_t)(chunk_places(T, n_seqs) * ((int64_t)n_v * kUnitBytes + (int64_t)n_qk * kHeadBytes));
}

hipError_t launch_gdn_prefill(const GdnRows& in, const int32_t* cu, int n_seqs, int64_t T, const float* s_in,
                              float* s_out, const int32_t* slots, int n_slots, void* o, int64_t ldo, void* workspace,
                              hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* wsh = ws + chunk_places(T, n_seqs) * in.n_v * kUnitBytes;
  const int64_t chunk_heads = chunk_places(T, n_seqs) * in.n_qk;
  const int split = chunk_heads < kFewChunkHeads ? in.n_v / in.n_qk : 1;
  gdn_chunk_prepare_kernel<<<(unsigned)(chunk_heads * split), 256, 0, stream>>>(in, cu, n_seqs, T, ws, wsh, split);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t units = (int64_t)n_seqs * in.n_v;
  if (units >= kWideUnits)
    gdn_chunk_wide_kernel<<<(unsigned)units, kWideThreads, 0, stream>>>(
        in, cu, n_seqs, T, ws, wsh, s_in, s_out, slots, n_slots, static_cast<uint16_t*>(o), ldo);
  else if (units >= kPairUnits)
    gdn_chunk_scan_kernel<2><<<(unsigned)((units + 7) / 8 * 8 * (kD / (2 * kCols))), kScanThreads, 0, stream>>>(
        in, cu, n_seqs, T, ws, wsh, s_in, s_out, slots, n_slots, static_cast<uint16_t*>(o), ldo);
  else
    gdn_chunk_scan_kernel<1><<<(unsigned)((units + 7) / 8 * 8 * (kD / kCols)), kScanThreads, 0, stream>>>(
        in, cu, n_seqs, T, ws, wsh, s_in, s_out, slots, n_slots, static_cast<uint16_t*>(o), ldo);
  return hipGetLastError();
}

}  // namespace nvfp4
