// What the two attention kernels (nvfp4_attn.h) share: rows in tiles of 16, their softmax and results, and the
// codes of keys and values as operands.
#pragma once

#include "nvfp4_attn.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float max_over_g(float v) {  // over lanes n, n + 16, n + 32, n + 48
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ floatx4_t mfma(const half8_t& a, const half8_t& b, const floatx4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Pages of a step's keys: of the lane's K rows' block of 16 and of its own block g; -1 where there is none.
struct Pages {
  int k, v;
};
// They are asked for a step or more before they are needed: entries_of only loads (from within the table always),
// pages_of says what was found, once it has arrived.
__device__ __forceinline__ Pages entries_of(const Attn& a, int seq, int step) {
  const int lane = threadIdx.x & 63, last = a.r.max_pages - 1, shift = a.c.page_shift - 4;
  const int* row = a.r.table + (int64_t)seq * a.r.ld_table;
  const int k = (4 * step + ((lane & 15) >> 2)) >> shift, v = (4 * step + (lane >> 4)) >> shift;
  return {row[min(k, last)], row[min(v, last)]};
}
__device__ __forceinline__ Pages pages_of(const Attn& a, int step, const Pages& e) {
  const int lane = threadIdx.x & 63, shift = a.c.page_shift - 4;
  const int k = (4 * step + ((lane & 15) >> 2)) >> shift, v = (4 * step + (lane >> 4)) >> shift;
  return {k < a.r.max_pages && (unsigned)e.k < (unsigned)a.c.n_pages ? e.k : -1,
          v < a.r.max_pages && (unsigned)e.v < (unsigned)a.c.n_pages ? e.v : -1};
}
__device__ __forceinline__ Pages pages_now(const Attn& a, int seq, int step) {
  return pages_of(a, step, entries_of(a, seq, step));
}
__device__ __forceinline__ bool all_there(const Pages& p) { return __builtin_amdgcn_ballot_w64((p.k | p.v) < 0) == 0; }

// Sizes of a format's operands, and a wave's rows and results.
template <bool kFp4, int kD, int kNT>
struct Rows {
  static constexpr int kWaveRows = 16 * kNT;
  // K: a lane has kVals values of a row per load, dims 4 kVals c + kVals g and on
  static constexpr int kBytes = kFp4 && kD == 64 ? 8 : 16, kVals = kFp4 ? 2 * kBytes : kBytes;
  static constexpr int kLoads = kD / (4 * kVals), kFrags = kD / 32, kPerLoad = kVals / 8;
  // V: kTiles operands of 16 dims; NVFP4's come in pairs, dims d and d + 1
  static constexpr int kTiles = kD / 16, kVLoads = kFp4 ? kTiles / 2 : kTiles;
  typedef floatx4_t Scores[kNT][4];

  half8_t q[kNT][kFrags];
  floatx4_t o[kNT][kTiles];
  // The sum of a row's weights is one more result, with ones for V: no vector additions, no exchange between lanes.
  floatx4_t sum[kNT];
  // The running maximum is kept in the scores' own units, -inf before the first; c1 makes powers of two of them.
  // A weight is 2^(s c1 + off).  Where |m c1| passes kFar in a row of the wave, the rounding of off (2^-24 of it) would
  // reach a fp16 weight's own, and from 2^28 on more than fp16 holds (NaN, or no weight at all): the wave then takes m
  // off the scores first, exactly as far as weights go (`far`; 16 kNT subtractions more a step).
  float m[kNT], c1[kNT], off[kNT];
  bool far;
  float fate[kNT];                // 1, or NaN
  int limit[kNT];                 // positions the row may see
  uint64_t seen[kNT];             // tree: its mask

  __device__ __forceinline__ void load_q(const Attn& a, const Unit& u, int rows, int row0) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const float k_gs = *a.c.k_gs;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const RowOf r = row_of(a, u, rows, row0 + 16 * nt + n);
      const bool real = r.token >= 0;
      const int64_t row = u.w.rows.row0 + (real ? r.token : 0);
      const uint16_t* from = a.q + row * a.ldq + (int64_t)(real ? r.head : 0) * kD + kVals * g;
      u32x4_t x[kFrags];
      uint32_t top = 0;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        x[f] = u32x4_t{0, 0, 0, 0};
        if (real) x[f] = *reinterpret_cast<const u32x4_t*>(from + 4 * kVals * (f / kPerLoad) + 8 * (f % kPerLoad));
      }
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[f][i] & 0x7FFFu, x[f][i] >> 16 & 0x7FFFu));
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      const int exponent = max((int)(top >> 7), 1) - 127, shift = 14 - exponent;  // of the row's largest value
      const bool finite = top < 0x7F80u;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        half2_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[i] = two_fp16(ldexpf(finite ? __uint_as_float(x[f][i] << 16) : 0.0f, shift),
                          ldexpf(finite ? __uint_as_float(x[f][i] & 0xFFFF0000u) : 0.0f, shift));
        q[nt][f] = __builtin_bit_cast(half8_t, h);
      }
      // Kept normal and below 2^64: under the one all scores are 0 to any precision (but -inf times it is -inf still),
      // over the other any two that differ at all are further apart than weights can be.
      c1[nt] = fminf(fmaxf(ldexpf(a.scale * k_gs, a.power - shift), 0x1p-126f), 0x1p64f);
      fate[nt] = finite ? 1.0f : __builtin_nanf("");  // what is not finite in q makes the row NaN if it sees anything
      m[nt] = -INFINITY;
      off[nt] = kLift;
      sum[nt] = floatx4_t{0, 0, 0, 0};
      limit[nt] = real ? row_limit(a, u.w.rows, r.token) : 0;
      seen[nt] = a.tree && real ? a.tree[row] : 0;
#pragma unroll
      for (int d = 0; d < kTiles; ++d) o[nt][d] = floatx4_t{0, 0, 0, 0};
    }
    far = false;
  }

  // Part x of `parts` of the largest of each row's scores that the lane has.
  __device__ __forceinline__ void tops(int x, int parts, const Scores& s, float top[kNT]) const {
#pragma unroll
    for (int i = 16 * kNT * x / parts; i < 16 * kNT * (x + 1) / parts; ++i) {
      const int nt = i / 16, e = i % 16;
      top[nt] = e == 0 ? s[nt][0][0] : fmaxf(top[nt], s[nt][e / 4][e % 4]);
    }
  }
  // The running maximum after scores with the given tops; what it moves by is taken out of the sum and the result.
  __device__ __forceinline__ void raise_max(const float top[kNT], Scores& s) {
    bool lags = false;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) lags = lags || (top[nt] - m[nt]) * c1[nt] > kLag;
    if (__builtin_amdgcn_ballot_w64(lags)) {
      bool past = false;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const float now = fmaxf(m[nt], max_over_g(top[nt])), f = rescale(m[nt], now, c1[nt]);
        m[nt] = now;
        sum[nt] *= f;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) o[nt][d] *= f;
        const float at = now == -INFINITY ? 0.0f : now * c1[nt];
        off[nt] = kLift - at;
        past = past || fabsf(at) > kFar;
      }
      far = __builtin_amdgcn_ballot_w64(past) != 0;
    }
    if (far) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const float base = fmaxf(m[nt], -0x1p100f);  // before the first: -inf less it is -inf still
        off[nt] = kLift;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[nt][e / 4][e % 4] -= base;
      }
    }
  }

  // q to accumulation registers, where matrix instructions can read it, and for good: left to itself the compiler
  // keeps its parts apart and puts them together again in every step.
  __device__ __forceinline__ void pin_q() {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int f = 0; f < kFrags; ++f) asm volatile("" : "+a"(q[nt][f]));
  }

  // Scores of keys key .. key + 15 that their row does not see become -inf.
  __device__ __forceinline__ void hide(const Attn& a, const SeqRows& sr, int key, bool has_page, Scores& s) const {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const uint32_t bits = seen_bits(a, sr, limit[nt], seen[nt], key, has_page);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[nt][e / 4][e % 4] = bits >> e & 1 ? s[nt][e / 4][e % 4] : -INFINITY;
    }
  }

  // Part x of `parts` of the rows' weights of the lane's 16 keys, under the running maximum.
  __device__ __forceinline__ void weights(int x, int parts, const Scores& s, half8_t p[kNT][2]) {
#pragma unroll
    for (int i = 8 * kNT * x / parts; i < 8 * kNT * (x + 1) / parts; ++i) {
      const int nt = i / 8, e = i % 8 * 2;
      const float v = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4], c1[nt], off[nt]));
      const float y = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4 + 1], c1[nt], off[nt]));
      const half2_t h = two_fp16(v, y);
      p[nt][e / 8][e % 8] = h[0];
      p[nt][e / 8][e % 8 + 1] = h[1];
    }
  }

  __device__ __forceinline__ void add_sums(const half8_t p[kNT][2]) {
    const half8_t one = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) sum[nt] = mfma(one, p[nt][h], sum[nt]);
  }
  // Operand h of V's tile d (keys 8 h .. 8 h + 7 of the lane's) times the weights.
  __device__ __forceinline__ void add_value(int d, int h, const half8_t& v, const half8_t p[kNT][2]) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) o[nt][d] = mfma(v, p[nt][h], o[nt][d]);
  }
  // Results of tile d that see a NaN of V become NaN; v: the tile's operands of keys 8 h .. as they were stored.
  __device__ __forceinline__ void spread_nan(int d, const half8_t v[2], const uint32_t bits[kNT]) {
    half8_t bad[2];
#pragma unroll
    for (int e = 0; e < 16; ++e) bad[e / 8][e % 8] = v[e / 8][e % 8] == v[e / 8][e % 8] ? (_Float16)0 : (_Float16)1;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      floatx4_t found = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        half8_t see;
#pragma unroll
        for (int e = 0; e < 8; ++e) see[e] = bits[nt] >> (8 * h + e) & 1 ? (_Float16)1 : (_Float16)0;
        found = mfma(bad[h], see, found);
      }
      floatx4_t more;
#pragma unroll
      for (int i = 0; i < 4; ++i) more[i] = found[i] > 0.0f ? __builtin_nanf("") : 0.0f;
      o[nt][d] += more;
    }
  }

  // The sum of row n's weights; NaN where the row is.
  __device__ __forceinline__ float total(int nt) const { return sum[nt][0] == 0.0f ? 0.0f : sum[nt][0] * fate[nt]; }
};

// Where a row's results go: to the output if its unit is whole (slot < 0), else to the workspace.
template <bool kFp4, int kD>
struct Sink {
  uint16_t* to;
  float* part;
  float f;
  // Row rho (of `rows`), its maximum m, sum l and factor of the scores c1.
  __device__ __forceinline__ Sink(const Attn& a, const Unit& u, int rows, int rho, float m, float l, float c1, int slot) {
    const int g = (threadIdx.x & 63) >> 4;
    const RowOf r = row_of(a, u, rows, rho);
    to = nullptr;
    part = nullptr;
    if (r.token < 0) return;
    if (slot < 0) {
      f = l == 0.0f ? 0.0f : *a.c.v_gs / l;  // a row that sees nothing is zeros
      to = a.o + (u.w.rows.row0 + r.token) * a.ldo + (int64_t)r.head * kD;
    } else {
      float* base = a.part + (int64_t)slot * (rows * (kD + kPartMore));
      part = base + rho * kD;
      if (g == 0) {
        float* more = base + rows * kD + kPartMore * rho;
        more[0] = m;
        more[1] = l;
        more[2] = c1;
      }
    }
  }
  // Tiles 2 x and 2 x + 1: the lane's eight values are two runs of four dims.
  __device__ __forceinline__ void put(int x, const floatx4_t& t0, const floatx4_t& t1) const {
    const int g = (threadIdx.x & 63) >> 4, d0 = kFp4 ? 32 * x + 8 * g : 32 * x + 4 * g, d1 = kFp4 ? d0 + 4 : d0 + 16;
    const floatx4_t v0 = kFp4 ? floatx4_t{t0[0], t1[0], t0[1], t1[1]} : t0;
    const floatx4_t v1 = kFp4 ? floatx4_t{t0[2], t1[2], t0[3], t1[3]} : t1;
    if (to) {
      u32x2_t b;
      b[0] = pack_bf16(v0[0] * f, v0[1] * f);
      b[1] = pack_bf16(v0[2] * f, v0[3] * f);
      *reinterpret_cast<u32x2_t*>(to + d0) = b;
      b[0] = pack_bf16(v1[0] * f, v1[1] * f);
      b[1] = pack_bf16(v1[2] * f, v1[3] * f);
      *reinterpret_cast<u32x2_t*>(to + d1) = b;
    } else if (part) {
      *reinterpret_cast<floatx4_t*>(part + d0) = v0;
      *reinterpret_cast<floatx4_t*>(part + d1) = v1;
    }
  }
};

// Codes of a lane: of `kN` loads of K rows or V lines, with NVFP4's scales.
template <bool kFp4, int kN>
struct RawK {
  u32x4_t x[kN];
  uint32_t sc[kFp4 ? kN : 1];
};
template <bool kFp4, int kN>
struct RawV {
  u32x4_t x[kN], sc[kFp4 ? kN : 1];
};

// The place of (page, head) in the cache's arrays, in units of a head's page.
__device__ __forceinline__ int64_t unit_of(const Attn& a, int page, int head) {
  return (int64_t)((uint64_t)(uint32_t)max(page, 0) * (uint32_t)a.c.hk + (uint32_t)head);
}

template <bool kFp4, int kD>
struct Codes {
  using R = Rows<kFp4, kD, 1>;

  // The lane's part of the row of K's tile t.
  static __device__ __forceinline__ void load_k(const Attn& a, int head, int step, int page, int t,
                                                RawK<kFp4, R::kLoads>& r) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, ps = 1 << a.c.page_shift;
    const int krow = (step * kStep + 16 * (n >> 2) + (n & 3)) & (ps - 1);
    const int64_t row = (unit_of(a, page, head) << a.c.page_shift) + krow + 4 * t;
    const uint8_t* at = a.c.k + row * code_bytes<kFp4>(kD) + R::kBytes * g;
#pragma unroll
    for (int c = 0; c < R::kLoads; ++c) {
      if constexpr (R::kBytes == 16) {
        r.x[c] = *reinterpret_cast<const u32x4_t*>(at + 64 * c);
      } else {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at + 32 * c);
        r.x[c][0] = v[0];
        r.x[c][1] = v[1];
      }
      if constexpr (kFp4) {
        const uint8_t* from = a.c.k_scales + row * (kD / 16) + (4 * R::kVals * c + R::kVals * g) / 16;
        r.sc[c] = R::kVals == 32 ? *reinterpret_cast<const uint16_t*>(from) : *from;
      }
    }
  }
  // Operand f of them.
  static __device__ __forceinline__ half8_t key(const RawK<kFp4, R::kLoads>& r, int f) {
    const int c = f / R::kPerLoad, i = f % R::kPerLoad;
    if constexpr (kFp4) {
      const half2_t sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.sc[c], 1.0f, false);
      const half2_t s2 = {sc[i / 2], sc[i / 2]};
      return half8_of_e2m1(r.x[c][i], s2);
    } else {
      return half8_of_e4m3(r.x[c][2 * i], r.x[c][2 * i + 1]);
    }
  }

  // V's loads first, first + by, ...
  template <int kN>
  static __device__ __forceinline__ void load_v(const Attn& a, int head, int step, int page, int first, int by,
                                                RawV<kFp4, kN>& r) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, ps = 1 << a.c.page_shift;
    const int vrow = (step * kStep + 16 * g) & (ps - 1);
    const int64_t unit = unit_of(a, page, head);
    const uint8_t* at = a.c.v + ((unit * code_bytes<kFp4>(kD) + 16 * first + n) << a.c.page_shift) + vrow;
    const uint8_t* sc = kFp4 ? a.c.v_scales + ((unit * (kD / 16) + 2 * first + (n >> 3)) << a.c.page_shift) + vrow : nullptr;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      r.x[i] = *reinterpret_cast<const u32x4_t*>(at + 16 * by * i * ps);
      if constexpr (kFp4) r.sc[i] = *reinterpret_cast<const u32x4_t*>(sc + 2 * by * i * ps);
    }
  }
  // Codes (scales) behind the first `keep` of the lane's 16 keys, and NaN among the others, become zeros; whether
  // there was such a NaN in any lane.
  template <int kN>
  static __device__ __forceinline__ bool clear_v(RawV<kFp4, kN>& r, int keep) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      u32x4_t& x = kFp4 ? r.sc[kFp4 ? i : 0] : r.x[i];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x[w] &= kept_bytes(keep, w);
        const uint32_t nan = nan_bytes(x[w]);
        bad |= nan;
        x[w] &= ~((nan >> 7) * 0xFFu);
      }
    }
    return __builtin_amdgcn_ballot_w64(bad != 0) != 0;
  }
  // What clear_v took out of the steps k, k + by, ... before `end`: the results that see it become NaN.  The codes
  // are read once more, of the steps that not every row sees all of (`all`: positions that every row sees).
  template <int kNT>
  static __device__ __forceinline__ void spread_nan(const Attn& a, const Unit& u, Rows<kFp4, kD, kNT>& w, int head, int k,
                                                 int end, int by, int all) {
    for (; k < end; k += by) {
      const Pages pg = pages_now(a, u.seq, k);
      if ((k + 1) * kStep <= all && all_there(pg)) continue;
      const int keep = keys_there(a, u.w.rows, k * kStep + 16 * ((threadIdx.x & 63) >> 4), pg.v), key = k * kStep + 16 * ((threadIdx.x & 63) >> 4);
      uint32_t bits[kNT];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) bits[nt] = seen_bits(a, u.w.rows, w.limit[nt], w.seen[nt], key, pg.v >= 0) & ((1u << keep) - 1u);
#pragma unroll
      for (int d = 0; d < R::kVLoads; ++d) {
        RawV<kFp4, 1> r;
        half8_t v[2][2];
        load_v(a, head, k, pg.v, d, 0, r);
        u32x4_t& x = kFp4 ? r.sc[0] : r.x[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] &= kept_bytes(keep, i);  // keys that are not there may hold anything
        value(r, 0, 0, v[0][0], v[1][0]);
        value(r, 0, 1, v[0][1], v[1][1]);
        w.spread_nan(kFp4 ? 2 * d : d, v[0], bits);
        if constexpr (kFp4) w.spread_nan(2 * d + 1, v[1], bits);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // Operand h (keys 8 h .. 8 h + 7 of the lane's) of load i: v0, and in NVFP4 v1 of the next dim.
  template <int kN>
  static __device__ __forceinline__ void value(const RawV<kFp4, kN>& r, int i, int h, half8_t& v0, half8_t& v1) {
    if constexpr (kFp4) {
      half2_t sc[4];
      sc[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.sc[i][2 * h], 1.0f, false);
      sc[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.sc[i][2 * h], 1.0f, true);
      sc[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.sc[i][2 * h + 1], 1.0f, false);
      sc[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.sc[i][2 * h + 1], 1.0f, true);
      half8s_of_pairs(r.x[i][2 * h], r.x[i][2 * h + 1], sc, v0, v1);
    } else {
      v0 = half8_of_e4m3(r.x[i][2 * h], r.x[i][2 * h + 1]);
    }
  }
};

}  // namespace
}  // namespace nvfp4
