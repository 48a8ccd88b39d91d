// Attention over the cache for many rows per sequence (nvfp4_attn.h): prompts, large trees.
#include "nvfp4_attn_rows.h"

namespace nvfp4 {
namespace {

// Many rows per sequence (prompts, large trees): the waves have 16 kNT rows each
// and share every step's keys, which the workgroup makes fp16 once, in LDS, in
// the order of the matrix instructions' operands (a lane's 16 bytes side by
// side: no bank conflicts, constant offsets).  In registers each wave would
// convert all of them itself, as many vector instructions as the softmax has.
// Wave t converts K's tile t and every fourth load of V.
//
// Bound by LDS, by instruction issue and by the waits of a lone wave on each SIMD: a
// prompt of 32768, E4M3, 24/4 heads of 256, takes 13.4 ms, 985 TFLOP/s of the 1530 of a
// library product.  Matrix instructions are busy for 42% of the cycles.  Each wave reads
// a whole step's operands for its 32 rows: at 128 B a clock the 16-byte accesses of 64 lanes
// take 52% of the cycles.  Heads of 128 (two waves a SIMD): 7 NVFP4 chunks of 1100 rows
// behind 6000, 32/8 heads, 2.05 ms, 965 TFLOP/s, 45% and 53%.
// 32x32x16 instructions took 10% fewer cycles at a lower clock, 14.25 ms.
//
// One barrier a step.  In step j the scores of step j + 1 are multiplied while
// step j's softmax is evaluated (neither waits for the other), then P V of step j;
// codes of K's step j + 2 and V's step j + 1 are asked for at its beginning and
// converted at its end, into the halves of the buffers that step j - 1 was the last
// to read.
template <bool kFp4, int kD, int kNT>
struct Many {
  using R = Rows<kFp4, kD, kNT>;
  using C = Codes<kFp4, kD>;
  static constexpr int kRows = 4 * R::kWaveRows;
  static constexpr int kMine = R::kVLoads < 4 ? 1 : R::kVLoads / 4;  // V loads of a wave
  struct Lds {
    u32x4_t k[2][4 * R::kFrags * 64], v[2][2 * R::kTiles * 64];  // operands of a step, 1 KiB each
    int nan[4];
  };
  struct State {
    RawK<kFp4, R::kLoads> rk;
    RawV<kFp4, kMine> rv;
    Pages p0, p1, p2;  // of steps k, k + 1, k + 2
    bool nan;          // whether this wave took NaN out of values
  };

  static __device__ __forceinline__ void store_k(const RawK<kFp4, R::kLoads>& r, int f, u32x4_t* to) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    to[(wave * R::kFrags + f) * 64 + lane] = __builtin_bit_cast(u32x4_t, C::key(r, f));
  }
  static __device__ __forceinline__ bool has_v() { return R::kVLoads >= 4 || (int)(threadIdx.x >> 6) < R::kVLoads; }
  static __device__ __forceinline__ void load_v(const Attn& a, int head, int step, int page, RawV<kFp4, kMine>& r) {
    if (has_v()) C::load_v(a, head, step, page, threadIdx.x >> 6, 4, r);
  }
  static __device__ __forceinline__ void store_v(const RawV<kFp4, kMine>& r, int i, int h, u32x4_t* to) {
    const int d = (threadIdx.x >> 6) + 4 * i, lane = threadIdx.x & 63;
    if (!has_v()) return;
    half8_t v0, v1;
    C::value(r, i, h, v0, v1);
    to[((kFp4 ? 2 * d : d) * 2 + h) * 64 + lane] = __builtin_bit_cast(u32x4_t, v0);
    if constexpr (kFp4) to[((2 * d + 1) * 2 + h) * 64 + lane] = __builtin_bit_cast(u32x4_t, v1);
  }

  // A step's scores and the largest of each row's.
  struct Found {
    typename R::Scores s;
    float top[kNT];
  };

  // Step k of the unit (the b-th, modulo 2), whose scores are in `now`; the next step's go to `next`.  `mine`: what
  // this wave has; `everyone`: positions that all rows of the workgroup see.  The parts between the scheduling barriers
  // hold matrix and vector instructions that do not wait for each other, and the LDS reads of the next part;
  // without the barriers the compiler asks for all of a step's operands at once, more than there are registers.
  static __device__ __forceinline__ void run_step(const Attn& a, const Unit& u, int head, R& w, State& st, Lds& lds,
                                                  int k, int end, const Reach& mine, int everyone, const int b,
                                                  Found& now, Found& next) {
    const int lane = threadIdx.x & 63, g = lane >> 4, wave = threadIdx.x >> 6;
    const int k1 = min(k + 1, end - 1), k2 = min(k + 2, end - 1), k3 = min(k + 3, end - 1);
    const half8_t* kf = reinterpret_cast<const half8_t*>(lds.k[b ^ 1]) + lane;
    const half8_t* vf = reinterpret_cast<const half8_t*>(lds.v[b]) + lane;
    constexpr int kPart = R::kFrags < 4 ? R::kFrags : 4, kParts = 4 * R::kFrags / kPart;  // K's operands at a time
    half8_t p[kNT][2], f[2][kPart];
#pragma unroll
    for (int i = 0; i < kPart; ++i) f[0][i] = kf[i * 64];
    if ((k + 1) * kStep > mine.all || !all_there(st.p0)) {
      w.hide(a, u.w.rows, k * kStep + 16 * g, st.p0.v >= 0, now.s);
      w.tops(0, 1, now.s, now.top);
    }
    w.raise_max(now.top, now.s);
    Pages e3;
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      if (x == 0) {
        C::load_k(a, head, k2, st.p2.k, wave, st.rk);
        load_v(a, head, k1, st.p1.v, st.rv);
        e3 = entries_of(a, u.seq, k3);
      }
      if (x + 1 < kParts) {
#pragma unroll
        for (int i = 0; i < kPart; ++i) f[(x + 1) & 1][i] = kf[((x + 1) * kPart + i) * 64];
      }
#pragma unroll
      for (int i = 0; i < kPart; ++i) {
        const int t = (x * kPart + i) / R::kFrags, q = (x * kPart + i) % R::kFrags;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
          next.s[nt][t] = mfma(f[x & 1][i], w.q[nt][q], q == 0 ? floatx4_t{0, 0, 0, 0} : next.s[nt][t]);
      }
      w.weights(x, kParts, now.s, p);
      __builtin_amdgcn_sched_barrier(0);
    }
    half8_t v[2][4];  // V's operands of two tiles of dims at a time
#pragma unroll
    for (int i = 0; i < 4; ++i) v[0][i] = vf[i * 64];
    w.add_sums(p);
    // values that some row of the workgroup does not see
    if (has_v() && ((k1 + 1) * kStep > everyone || !all_there(st.p1)))
      st.nan |= C::clear_v(st.rv, keys_there(a, u.w.rows, k1 * kStep + 16 * g, st.p1.v));
    constexpr int kPairs = R::kTiles / 2, kStores = R::kFrags + 2 * kMine;
#pragma unroll
    for (int x = 0; x < kPairs; ++x) {
      if (x + 1 < kPairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[(x + 1) & 1][i] = vf[(4 * (x + 1) + i) * 64];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w.add_value(2 * x + i / 2, i % 2, v[x & 1][i], p);
      w.tops(x, kPairs, next.s, next.top);
#pragma unroll
      for (int i = kStores * x / kPairs; i < kStores * (x + 1) / kPairs; ++i) {
        if (i < R::kFrags)
          store_k(st.rk, i, lds.k[b]);
        else
          store_v(st.rv, (i - R::kFrags) / 2, (i - R::kFrags) % 2, lds.v[b ^ 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    st.p0 = st.p1;
    st.p1 = st.p2;
    st.p2 = pages_of(a, k3, e3);
  }

  static __device__ __forceinline__ void run_unit(const Attn& a, const Unit& u, int k0, int k1, int slot, Lds& lds) {
    const int wave = uniform((int)threadIdx.x >> 6), n = threadIdx.x & 15;
    const int row0 = wave * R::kWaveRows, head = u.minor / a.parts;
    R w;
    const Reach mine = reach_of(a, u, kRows, row0, R::kWaveRows), whole = reach_of(a, u, kRows, 0, kRows);
    const int end = min(k1, whole.steps);
    // the page numbers are on their way while q is
    const int last = max(end - 1, k0);
    const Pages e0 = entries_of(a, u.seq, k0), e1 = entries_of(a, u.seq, min(k0 + 1, last)),
                e2 = entries_of(a, u.seq, min(k0 + 2, last));
    w.load_q(a, u, kRows, row0);
    if constexpr (kD != 128) w.pin_q();
    if (k0 < end) {
      State st;
      st.p0 = pages_of(a, k0, e0);
      st.p1 = pages_of(a, min(k0 + 1, end - 1), e1);
      st.p2 = pages_of(a, min(k0 + 2, end - 1), e2);
      RawK<kFp4, R::kLoads> rk1;
      C::load_k(a, head, k0, st.p0.k, wave, st.rk);
      load_v(a, head, k0, st.p0.v, st.rv);
      C::load_k(a, head, min(k0 + 1, end - 1), st.p1.k, wave, rk1);
#pragma unroll
      for (int f = 0; f < R::kFrags; ++f) store_k(st.rk, f, lds.k[0]);
      st.nan = has_v() && ((k0 + 1) * kStep > whole.all || !all_there(st.p0)) &&
               C::clear_v(st.rv, keys_there(a, u.w.rows, k0 * kStep + 16 * ((threadIdx.x & 63) >> 4), st.p0.v));
#pragma unroll
      for (int i = 0; i < 2 * kMine; ++i) store_v(st.rv, i / 2, i % 2, lds.v[0]);
#pragma unroll
      for (int f = 0; f < R::kFrags; ++f) store_k(rk1, f, lds.k[1]);
      __syncthreads();
      const half8_t* kf = reinterpret_cast<const half8_t*>(lds.k[0]) + (threadIdx.x & 63);
      Found s0, s1;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int f = 0; f < R::kFrags; ++f)
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            s0.s[nt][t] = mfma(kf[(t * R::kFrags + f) * 64], w.q[nt][f], f == 0 ? floatx4_t{0, 0, 0, 0} : s0.s[nt][t]);
        __builtin_amdgcn_sched_barrier(0);
      }
      w.tops(0, 1, s0.s, s0.top);
      __syncthreads();
      for (int k = k0;;) {
        run_step(a, u, head, w, st, lds, k, end, mine, whole.all, 0, s0, s1);
        if (++k >= end) break;
        run_step(a, u, head, w, st, lds, k, end, mine, whole.all, 1, s1, s0);
        if (++k >= end) break;
      }
      if ((threadIdx.x & 63) == 0) lds.nan[wave] = st.nan;
      __syncthreads();
      if (lds.nan[0] | lds.nan[1] | lds.nan[2] | lds.nan[3]) C::spread_nan(a, u, w, head, k0, end, 1, whole.all);
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const Sink<kFp4, kD> sink(a, u, kRows, row0 + 16 * nt + n, w.m[nt], w.total(nt), w.c1[nt], slot);
#pragma unroll
      for (int x = 0; x < R::kTiles / 2; ++x) sink.put(x, w.o[nt][2 * x], w.o[nt][2 * x + 1]);
    }
  }
};

template <bool kFp4, int kD, int kNT>
__global__ __launch_bounds__(256, kD == 128 ? 2 : 1) void attn_many_kernel(Attn a) {
  __shared__ typename Many<kFp4, kD, kNT>::Lds lds;
  run_range(a, xcd_order(blockIdx.x, a.ranges), [&](const Unit& u, int k0, int k1, int slot) { Many<kFp4, kD, kNT>::run_unit(a, u, k0, k1, slot, lds); });
}

}  // namespace

void launch_attn_many(const Attn& a, hipStream_t stream) {
  const int d = a.c.d;
  const auto f = a.c.fp4 ? (d == 64 ? attn_many_kernel<true, 64, 2> : d == 128 ? attn_many_kernel<true, 128, 2> : attn_many_kernel<true, 256, 2>)
                         : (d == 64 ? attn_many_kernel<false, 64, 2> : d == 128 ? attn_many_kernel<false, 128, 2> : attn_many_kernel<false, 256, 2>);
  f<<<a.ranges, 256, 0, stream>>>(a);
}

}  // namespace nvfp4
