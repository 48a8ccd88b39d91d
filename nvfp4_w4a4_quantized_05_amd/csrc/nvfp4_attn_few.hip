// Attention over the cache for few rows per sequence (nvfp4_attn.h): decode, small trees.
#include "nvfp4_attn_rows.h"

namespace nvfp4 {
namespace {

// Few rows per sequence (decode): the workgroup's four waves have the same 16
// kNT rows and every fourth step each, straight from memory to the matrix
// instructions; their results are joined through LDS.  A step's V is asked for
// at its beginning and the next step's K behind its scores.  Bound by HBM where there
// are keys enough: 64 tokens behind up to 16K, E4M3, 24/4 heads of 256, 184 us for
// 1.03 GB (5.6 TB/s); two behind 131072, NVFP4, 32/8 heads of 128, 61 us (5.1 TB/s).
//
// Where there are units enough, every wave has a range of its own instead (solo):
// a unit takes as long to begin and to end (6 us, waiting for lengths, page
// numbers, queries and the first keys, one after the other) as 200 keys take, and
// so four of them are begun at once.
template <bool kFp4, int kD, int kNT, bool kSolo>
struct Few {
  static constexpr int kBy = kSolo ? 1 : 4;  // steps from a wave's step to its next
  using R = Rows<kFp4, kD, kNT>;
  using C = Codes<kFp4, kD>;
  static constexpr int kRows = R::kWaveRows;
  struct Lds {
    floatx4_t sums[kSolo ? 1 : 4 * R::kTiles * 64];
    float ml[4][kNT][16][2];
  };
  struct Keys {
    RawK<kFp4, R::kLoads> t[4];
  };
  static __device__ __forceinline__ void load_keys(const Attn& a, int head, int step, const Pages& pg, Keys& k) {
#pragma unroll
    for (int t = 0; t < 4; ++t) C::load_k(a, head, step, pg.k, t, k.t[t]);
  }

  // Step `step`, whose keys are in k; those of `after` (its pages pg2) are asked for.  `whole`: every row sees all of it.
  // Returns whether NaN was taken out of its values.
  static __device__ __forceinline__ bool run_step(const Attn& a, const Unit& u, int head, R& w, Keys& k, int step,
                                                  const Pages& pg, bool whole, int after, const Pages& pg2) {
    const int g = (threadIdx.x & 63) >> 4;
    RawV<kFp4, R::kVLoads> rv;
    C::load_v(a, head, step, pg.v, 0, 1, rv);
    typename R::Scores s;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int f = 0; f < R::kFrags; ++f) {
        const half8_t k8 = C::key(k.t[t], f);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) s[nt][t] = mfma(k8, w.q[nt][f], f == 0 ? floatx4_t{0, 0, 0, 0} : s[nt][t]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    load_keys(a, head, after, pg2, k);
    half8_t p[kNT][2];
    if (!whole) w.hide(a, u.w.rows, step * kStep + 16 * g, pg.v >= 0, s);
    float top[kNT];
    w.tops(0, 1, s, top);
    w.raise_max(top, s);
    w.weights(0, 1, s, p);
    w.add_sums(p);
    bool nan = false;
    if (!whole) nan = C::clear_v(rv, keys_there(a, u.w.rows, step * kStep + 16 * g, pg.v));
#pragma unroll
    for (int d = 0; d < R::kVLoads; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        half8_t v0, v1;
        C::value(rv, d, h, v0, v1);
        w.add_value(kFp4 ? 2 * d : d, h, v0, p);
        if constexpr (kFp4) w.add_value(2 * d + 1, h, v1, p);
      }
      if (d % 2 == 1) __builtin_amdgcn_sched_barrier(0);
    }
    return nan;
  }

  static __device__ __forceinline__ void run_unit(const Attn& a, const Unit& u, int k0, int k1, int slot, Lds& lds) {
    const int wave = kSolo ? 0 : uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15;
    const int head = u.minor / a.parts;
    R w;
    const Reach reach = reach_of(a, u, kRows, 0, kRows);
    const int end = min(k1, reach.steps);
    int k = k0 + wave;
    const int last = max(end - 1, k0);
    const Pages e0 = entries_of(a, u.seq, min(k, last)), e1 = entries_of(a, u.seq, min(k + kBy, last));
    w.load_q(a, u, kRows, 0);
    bool nan = false;
    if (k < end) {
      Keys keys;
      Pages pg = pages_of(a, k, e0), pg2 = pages_of(a, min(k + kBy, end - 1), e1);
      load_keys(a, head, k, pg, keys);
      for (; k < end; k += kBy) {
        const Pages e = entries_of(a, u.seq, min(k + 2 * kBy, end - 1));
        nan |= run_step(a, u, head, w, keys, k, pg, (k + 1) * kStep <= reach.all && all_there(pg), min(k + kBy, end - 1), pg2);
        pg = pg2;
        pg2 = pages_of(a, min(k + 2 * kBy, end - 1), e);
      }
    }
    if (nan) C::spread_nan(a, u, w, head, k0 + wave, end, kBy, reach.all);
    if constexpr (kSolo) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const Sink<kFp4, kD> sink(a, u, kRows, 16 * nt + n, w.m[nt], w.total(nt), w.c1[nt], slot);
#pragma unroll
        for (int x = 0; x < R::kTiles / 2; ++x) sink.put(x, w.o[nt][2 * x], w.o[nt][2 * x + 1]);
      }
      return;
    }
    // four waves' results of the same rows; each wave adds up every fourth pair of tiles
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      if (lane < 16) {
        lds.ml[wave][nt][n][0] = w.m[nt];
        lds.ml[wave][nt][n][1] = w.total(nt);
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float m = -INFINITY, l = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) m = fmaxf(m, lds.ml[v][nt][n][0]);
#pragma unroll
      for (int v = 0; v < 4; ++v) l += lds.ml[v][nt][n][1] * rescale(lds.ml[v][nt][n][0], m, w.c1[nt]);
      const float f = rescale(w.m[nt], m, w.c1[nt]);
      const Sink<kFp4, kD> sink(a, u, kRows, 16 * nt + n, m, l, w.c1[nt], slot);
      constexpr int kPairs = R::kTiles / 2;
#pragma unroll
      for (int i = 0; i < R::kTiles; ++i) lds.sums[(wave * R::kTiles + i) * 64 + lane] = w.o[nt][i] * f;
      __syncthreads();
#pragma unroll
      for (int x0 = 0; x0 < kPairs; x0 += 4) {
        const int x = x0 + wave;
        if (x >= kPairs) break;
        floatx4_t t[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int i = 0; i < 2; ++i) t[i] += lds.sums[(v * R::kTiles + 2 * x + i) * 64 + lane];
        sink.put(x, t[0], t[1]);
      }
      __syncthreads();
    }
  }
};

template <bool kFp4, int kD, int kNT, bool kSolo>
__global__ __launch_bounds__(256, kD < 256 ? 2 : 1) void attn_few_kernel(Attn a) {
  using F = Few<kFp4, kD, kNT, kSolo>;
  __shared__ typename F::Lds lds;
  const int block = xcd_order(blockIdx.x, gridDim.x);
  run_range(a, kSolo ? 4 * block + uniform((int)threadIdx.x >> 6) : block,
            [&](const Unit& u, int k0, int k1, int slot) { F::run_unit(a, u, k0, k1, slot, lds); });
}

template <bool kFp4, int kD>
void launch_typed(const Attn& a, int nt, bool solo, hipStream_t stream) {
  if (solo)
    (nt == 1 ? attn_few_kernel<kFp4, kD, 1, true> : attn_few_kernel<kFp4, kD, 2, true>)<<<a.ranges / 4, 256, 0, stream>>>(a);
  else
    (nt == 1 ? attn_few_kernel<kFp4, kD, 1, false> : attn_few_kernel<kFp4, kD, 2, false>)<<<a.ranges, 256, 0, stream>>>(a);
}

}  // namespace

void launch_attn_few(const Attn& a, int nt, bool solo, hipStream_t stream) {
  const int d = a.c.d;
  const auto f = a.c.fp4 ? (d == 64 ? launch_typed<true, 64> : d == 128 ? launch_typed<true, 128> : launch_typed<true, 256>)
                         : (d == 64 ? launch_typed<false, 64> : d == 128 ? launch_typed<false, 128> : launch_typed<false, 256>);
  f(a, nt, solo, stream);
}

}  // namespace nvfp4
