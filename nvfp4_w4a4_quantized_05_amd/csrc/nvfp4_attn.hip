// Attention of new tokens over a paged, quantised key/value cache (layout:
// nvfp4_kv.h): one token per request, trees of drafted tokens, or prompts.
//
//   o_r = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q_r . k_p - max),
//
// over the positions p that row r sees: those up to its own, or, with a tree
// mask, the context and the new tokens whose bit is set.
//
// One pass over K and V with the running maximum and sum of the softmax.  The
// codes go from memory to registers, are made fp16 there (exact for E4M3, and
// for E2M1 x E4M3) and multiplied with fp16 16x16x32 matrix instructions; the
// tensor scales are applied to the scores and to the result.
//
//  * S^T = K Q^T, 64 keys a step: tile t (0 .. 3) of 16 keys has as its row m
//    the key 16 (m / 4) + 4 t + m % 4 of the step.  Then lane (n, g) = (lane %
//    16, lane / 16) holds for query row n the scores of keys 16 g .. 16 g + 15,
//    in order, which is what the second product's operand wants of it:
//  * O^T = V^T P^T: no score leaves its lane.  The row's maximum, sum and
//    rescaling factor are values of the lane.
//  * q is scaled by a power of two that brings the row's largest value to
//    [2^14, 2^15): fp16 then holds every bf16 value down to 2^-31 of it exactly.
//  * P is rounded to fp16 (11 bits; bf16's 8 would cost the result more than
//    its own rounding), times 2^7: with the running maximum allowed to lag by up to
//    2^8 behind, its largest value is 2^15, and values are normal down to
//    2^-21 of the row's maximum, below that off by 2^-32 of it.
//  * What is not finite in V reaches only the rows that see it: where a step
//    hides keys from some rows, a lane looks for NaN codes, and if there are any the
//    step's second product is done with those as zeros and a third product of
//    what is seen and what is NaN says where the result is NaN.
//
// Work: the steps of all (sequence, tile of rows, head) are laid end to end and
// cut into equal ranges, one per workgroup, so that one long sequence among
// short ones, or one request alone, still fills the GPU.  Every workgroup finds
// its place from the lengths by itself.  A unit cut by a range's end leaves its
// maximum, sum and unscaled result in the workspace, and a second kernel joins
// them, in order.
#include "nvfp4_kv.h"

namespace nvfp4 {
namespace {

constexpr int kStep = 64;      // keys per step
constexpr float kLag = 8.0f;   // log2: how far the running maximum may lag behind
constexpr float kLift = 7.0f;  // log2: P is stored times 2^7
constexpr float kNoMax = -0x1p100f;

struct Attn {
  KvCache c;
  KvRows r;
  const uint16_t* q;
  int64_t ldq;
  int group;        // query heads per key/value head
  float scale;      // times log2(e)
  const uint64_t* tree;
  uint16_t* o;
  int64_t ldo;
  float* part;      // [2 x ranges][rows x (d + 2)]
  int ranges;       // workgroups
  int least;        // steps of a range, at least
  int tokens, parts;  // tokens per tile of rows; tiles that a token's heads take
};

__device__ __forceinline__ int64_t scan64(int64_t v) {  // inclusive, over the wave
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int64_t o = __shfl_up(v, m, 64);
    v += lane >= m ? o : 0;
  }
  return v;
}

// sum over r < n of (a r + b) / m, rounded down, for a, b >= 0.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// A sequence's share of the work.  Its tiles of rows (`tokens` tokens each) take
// (first + r tokens) / 64 steps per head, r the tile: with first = context +
// tokens + 63 that is what the tile's last token sees, rounded up (for the last
// tile that may be a step more than there is).
struct SeqWork {
  SeqRows rows;
  int64_t first;
  int slope;
  int tiles;
  int minor;  // heads x parts, which share a tile's number of steps
  __device__ __forceinline__ int64_t before(int64_t r) const {  // steps of the tiles before r
    return minor * (r == 1 || slope == 0 ? r * (first / kStep) : floor_sum(r, kStep, slope, first));
  }
  __device__ __forceinline__ int64_t steps(int64_t r) const { return (first + r * slope) / kStep; }
  __device__ __forceinline__ int64_t total() const { return before(tiles); }
};

__device__ __forceinline__ int64_t cache_rows(const Attn& a) { return (int64_t)a.r.max_pages << a.c.page_shift; }

__device__ __forceinline__ SeqWork seq_work(const Attn& a, int i) {
  SeqWork w;
  w.rows = seq_rows(a.r, i);
  const int64_t most = cache_rows(a);
  if (a.tree) {
    w.first = min(max((int64_t)w.rows.kv, (int64_t)1), max(most, (int64_t)1)) + kStep - 1;
    w.slope = 0;
  } else {
    w.first = min(max((int64_t)w.rows.kv - w.rows.n, (int64_t)0), most) + a.tokens + kStep - 1;
    w.slope = a.tokens;
  }
  w.tiles = (w.rows.n + a.tokens - 1) / a.tokens;
  w.minor = a.c.hk * a.parts;
  return w;
}

// All sequences' steps, and with `find` the sequence that holds step `pos`
// (pos < total) and the steps before it.  Every lane of the wave gets the same.
__device__ __forceinline__ int64_t total_steps(const Attn& a) {
  const int lane = threadIdx.x & 63;
  int64_t sum = 0;
  for (int i = lane; i < a.r.n_seqs; i += 64) sum += seq_work(a, i).total();
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 64);
  return sum;
}

__device__ __forceinline__ int find_seq(const Attn& a, int64_t pos, int64_t& before) {
  const int lane = threadIdx.x & 63;
  before = 0;
  for (int i0 = 0; i0 < a.r.n_seqs; i0 += 64) {
    const int64_t mine = i0 + lane < a.r.n_seqs ? seq_work(a, i0 + lane).total() : 0;
    const int64_t upto = before + scan64(mine);
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > pos);
    if (past) {
      const int at = __builtin_ctzll(past);
      before = __shfl(upto - mine, at, 64);
      return __builtin_amdgcn_readfirstlane(i0 + at);
    }
    before = __shfl(upto, 63, 64);
  }
  return -1;
}

// A unit of work: one tile of one sequence's rows and one (head, part).
struct Unit {
  int seq;
  SeqWork w;
  int tile, minor;
  int64_t start, steps;  // its place among all steps
};

__device__ __forceinline__ Unit unit_at(const Attn& a, int64_t pos) {
  Unit u;
  int64_t before;
  u.seq = find_seq(a, pos, before);
  u.w = seq_work(a, u.seq);
  const int64_t x = pos - before;
  u.tile = u.w.tiles == 1 ? 0 : last_before(u.w.tiles, [&](int r) { return u.w.before(r) <= x; });
  u.steps = u.w.steps(u.tile);
  const int64_t y = x - u.w.before(u.tile);
  u.minor = (int)(y / u.steps);
  u.start = pos - y % u.steps;
  return u;
}

// The unit behind u (there is one).
__device__ __forceinline__ void next_unit(const Attn& a, Unit& u) {
  u.start += u.steps;
  if (++u.minor < u.w.minor) return;
  u.minor = 0;
  if (++u.tile == u.w.tiles) {
    u.tile = 0;
    do u.w = seq_work(a, ++u.seq);
    while (u.w.tiles == 0 && u.seq + 1 < a.r.n_seqs);
  }
  u.steps = u.w.steps(u.tile);
}

// Row `rho` of a unit's tile: its token and query head, or token -1.
struct RowOf {
  int token, head;
};
__device__ __forceinline__ RowOf row_of(const Attn& a, const Unit& u, int rows, int rho) {
  const int wide = a.parts == 1 ? a.group : rows;
  const int h = (u.minor % a.parts) * rows + rho % wide;
  const int token = u.tile * a.tokens + rho / wide;
  const bool real = rho < a.tokens * wide && h < a.group && token < u.w.rows.n;
  return {real ? token : -1, (u.minor / a.parts) * a.group + h};
}

// Positions that a row of token j sees at the most: [0, limit).
__device__ __forceinline__ int64_t row_limit(const Attn& a, const SeqRows& s, int64_t most, int token) {
  const int64_t end = a.tree ? (int64_t)s.kv : min((int64_t)s.kv, (int64_t)s.kv - s.n + token + 1);
  return max(min(end, most), (int64_t)0);
}

__device__ __forceinline__ float max_over_g(float v) {  // over lanes n, n + 16, n + 32, n + 48
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_g(float v) {
  v += __shfl_xor(v, 32, 64);
  return v + __shfl_xor(v, 16, 64);
}

__device__ __forceinline__ floatx4_t mfma(const half8_t& a, const half8_t& b, const floatx4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ half2_t two_fp16(float a, float b) {  // round to nearest even
  float2v_t f;
  f[0] = a;
  f[1] = b;
  return __builtin_convertvector(f, half2_t);
}

// Eight E4M3 codes as fp16.
__device__ __forceinline__ half8_t half8_of_e4m3(uint32_t lo, uint32_t hi) {
  half2_t h[4];
  h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false);
  h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true);
  h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false);
  h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true);
  return __builtin_bit_cast(half8_t, h);
}

// Eight E2M1 codes of one block times its scale.
__device__ __forceinline__ half8_t half8_of_e2m1(uint32_t codes, half2_t s) {
  half2_t h[4];
  h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s;
  h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s;
  h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s;
  h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s;
  return __builtin_bit_cast(half8_t, h);
}

// Eight bytes of V codes (keys 0 .. 7, dims d and d + 1) times the keys' scales
// (two scales per s): the operands of dim d and of dim d + 1.
__device__ __forceinline__ void half8s_of_pairs(uint32_t lo, uint32_t hi, const half2_t s[4], half8_t& even,
                                                half8_t& odd) {
  uint32_t p[8];
  p[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 0));
  p[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 1));
  p[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 2));
  p[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 3));
  p[4] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(hi, 1.0f, 0));
  p[5] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(hi, 1.0f, 1));
  p[6] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(hi, 1.0f, 2));
  p[7] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(hi, 1.0f, 3));
  half2_t e[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u)) * s[i];
    o[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u)) * s[i];
  }
  even = __builtin_bit_cast(half8_t, e);
  odd = __builtin_bit_cast(half8_t, o);
}

// kSplit: the workgroup's four waves have the same 16 kNT rows and every fourth
// step each, and are joined through LDS; else 16 kNT rows each and every step.
template <bool kFp4, int kD, int kNT, bool kSplit>
struct Kernel {
  static constexpr int kWaveRows = 16 * kNT, kRows = kSplit ? kWaveRows : 4 * kWaveRows;
  // K: a lane has kVals values of a row per load, dims 4 kVals c + kVals g and on
  static constexpr int kBytes = kFp4 && kD == 64 ? 8 : 16, kVals = kFp4 ? 2 * kBytes : kBytes;
  static constexpr int kLoads = kD / (4 * kVals), kFrags = kD / 32, kPerLoad = kVals / 8;
  // V: kTiles operands of 16 dims; NVFP4's come in pairs, dims d and d + 1
  static constexpr int kTiles = kD / 16, kVLoads = kFp4 ? kTiles / 2 : kTiles;

  struct Wave {
    half8_t q[kNT][kFrags];
    floatx4_t o[kNT][kTiles];
    float m[kNT], l[kNT], c1[kNT];  // running maximum, the lane's part of the sum, factor of the scores (log2)
    int64_t limit[kNT];             // positions the row may see
    uint64_t seen[kNT];             // tree: its mask
  };

  // Pages of a step's keys: of the lane's K rows' block of 16 and of its own block g.
  struct Pages {
    int k, v;
  };
  static __device__ __forceinline__ Pages pages_of(const Attn& a, int seq, int64_t key0) {
    const int lane = threadIdx.x & 63;
    return {page_of(a.r, a.c, seq, key0 + 16 * ((lane & 15) >> 2)), page_of(a.r, a.c, seq, key0 + 16 * (lane >> 4))};
  }

  // Bits of the lane's 16 keys from position `key` on that row nt sees.
  static __device__ __forceinline__ uint32_t seen_bits(const Attn& a, const Wave& w, int nt, const SeqRows& s,
                                                       int64_t key, bool has_page) {
    const auto below = [&](int64_t end) {
      const int n = (int)min(max(end - key, (int64_t)0), (int64_t)16);
      return (1u << n) - 1u;
    };
    uint32_t bits = below(w.limit[nt]);
    if (a.tree) {
      const int64_t ctx = (int64_t)s.kv - s.n, b = key - ctx;
      const uint64_t drafts = b >= 0 ? (b < 64 ? w.seen[nt] >> b : 0) : (b > -16 ? w.seen[nt] << -b : 0);
      bits &= below(ctx) | (uint32_t)drafts;
    }
    return has_page ? bits : 0u;
  }

  // One step: keys key0 .. key0 + 63.  kMasked: some row does not see all of them.
  template <bool kMasked>
  static __device__ __forceinline__ void step(const Attn& a, Wave& w, const Unit& u, int64_t key0, Pages pg) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int head = u.minor / a.parts, ps = 1 << a.c.page_shift;
    const int krow = (int)(key0 + 16 * (n >> 2) + (n & 3)) & (ps - 1), vrow = (int)(key0 + 16 * g) & (ps - 1);
    const int64_t kunit = (int64_t)max(pg.k, 0) * a.c.hk + head, vunit = (int64_t)max(pg.v, 0) * a.c.hk + head;

    // ---- scores
    floatx4_t s[kNT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) s[nt][t] = floatx4_t{0, 0, 0, 0};
      const int64_t row = kunit * ps + krow + 4 * t;
      const uint8_t* at = a.c.k + row * code_bytes<kFp4>(kD) + kBytes * g;
#pragma unroll
      for (int c = 0; c < kLoads; ++c) {
        uint32_t x[4];
        if constexpr (kBytes == 16) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = v[i];
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at + 32 * c);
          x[0] = v[0];
          x[1] = v[1];
        }
        half2_t sc = {0, 0};
        if constexpr (kFp4) {
          const uint8_t* from = a.c.k_scales + row * (kD / 16) + (4 * kVals * c + kVals * g) / 16;
          const uint32_t b = kVals == 32 ? *reinterpret_cast<const uint16_t*>(from) : *from;
          sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b, 1.0f, false);
        }
#pragma unroll
        for (int f = 0; f < kPerLoad; ++f) {
          half8_t k8;
          if constexpr (kFp4) {
            const half2_t s2 = {sc[f / 2], sc[f / 2]};
            k8 = half8_of_e2m1(x[f], s2);
          } else {
            k8 = half8_of_e4m3(x[2 * f], x[2 * f + 1]);
          }
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) s[nt][t] = mfma(k8, w.q[nt][kPerLoad * c + f], s[nt][t]);
        }
      }
    }

    // ---- softmax: the lane has row n's scores of keys key0 + 16 g + 4 t + i
    half8_t p[kNT][2];
    uint32_t bits[kNT];
    const int64_t key = key0 + 16 * g;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      if constexpr (kMasked) bits[nt] = seen_bits(a, w, nt, u.w.rows, key, pg.v >= 0);
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if constexpr (kMasked) s[nt][e / 4][e % 4] = bits[nt] >> e & 1 ? s[nt][e / 4][e % 4] : -INFINITY;
        top = fmaxf(top, s[nt][e / 4][e % 4]);
      }
      top *= w.c1[nt];
      if (__builtin_amdgcn_ballot_w64(top > w.m[nt] + kLag)) {
        const float now = fmaxf(w.m[nt], max_over_g(top)), f = __builtin_amdgcn_exp2f(w.m[nt] - now);
        w.m[nt] = now;
        w.l[nt] *= f;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) w.o[nt][d] *= f;
      }
      const float off = kLift - w.m[nt];
      half2_t h[8];
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float x = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4], w.c1[nt], off));
        float y = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4 + 1], w.c1[nt], off));
        if constexpr (kMasked) {
          x = bits[nt] >> e & 1 ? x : 0.0f;
          y = bits[nt] >> (e + 1) & 1 ? y : 0.0f;
        }
        sum += x + y;
        h[e / 2] = two_fp16(x, y);
      }
      w.l[nt] += sum;
      p[nt][0] = __builtin_bit_cast(half8_t, *(const half2_t(*)[4])h);
      p[nt][1] = __builtin_bit_cast(half8_t, *(const half2_t(*)[4])(h + 4));
    }

    // ---- result
    uint32_t keep[4];  // bytes of the lane's 16 keys that exist
    bool nan = false;
    if constexpr (kMasked) {
      const int64_t end = min((int64_t)u.w.rows.kv, cache_rows(a));
      const int have = pg.v >= 0 ? (int)min(max(end - key, (int64_t)0), (int64_t)16) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = min(max(have - 4 * i, 0), 4);
        keep[i] = b == 4 ? ~0u : (1u << (8 * b)) - 1u;
      }
    }
    const auto load = [&](const uint8_t* from) {
      u32x4_t x = *reinterpret_cast<const u32x4_t*>(from);
      if constexpr (kMasked) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] &= keep[i];
      }
      return x;
    };
    u32x4_t codes[kVLoads], scales[kFp4 ? kVLoads : 1];
#pragma unroll
    for (int d = 0; d < kVLoads; ++d) {
      codes[d] = load(a.c.v + (vunit * code_bytes<kFp4>(kD) + 16 * d + n) * ps + vrow);
      if constexpr (kFp4) scales[d] = load(a.c.v_scales + (vunit * (kD / 16) + 2 * d + (n >> 3)) * ps + vrow);
      if constexpr (kMasked) {
        const u32x4_t x = kFp4 ? scales[kFp4 ? d : 0] : codes[d];
#pragma unroll
        for (int i = 0; i < 4; ++i) nan = nan || (((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u);
      }
    }
    const auto operand = [&](int d, int h, half8_t& v0, half8_t& v1) {  // of keys 8 h .. 8 h + 7
      if constexpr (kFp4) {
        half2_t sc[4];
        sc[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales[d][2 * h], 1.0f, false);
        sc[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales[d][2 * h], 1.0f, true);
        sc[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales[d][2 * h + 1], 1.0f, false);
        sc[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales[d][2 * h + 1], 1.0f, true);
        half8s_of_pairs(codes[d][2 * h], codes[d][2 * h + 1], sc, v0, v1);
      } else {
        v0 = half8_of_e4m3(codes[d][2 * h], codes[d][2 * h + 1]);
      }
    };
    if (kMasked && __builtin_amdgcn_ballot_w64(nan)) {
      for (int nt = 0; nt < kNT; ++nt) {
        half8_t see[2];
#pragma unroll
        for (int e = 0; e < 16; ++e) see[e / 8][e % 8] = bits[nt] >> e & 1 ? (_Float16)1 : (_Float16)0;
#pragma unroll
        for (int d = 0; d < kVLoads; ++d) {
          floatx4_t found[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            half8_t v[2], bad[2];
            operand(d, h, v[0], v[1]);
#pragma unroll
            for (int x = 0; x < (kFp4 ? 2 : 1); ++x) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const bool is = !(v[x][e] == v[x][e]);
                bad[x][e] = is ? (_Float16)1 : (_Float16)0;
                v[x][e] = is ? (_Float16)0 : v[x][e];
              }
              found[x] = mfma(bad[x], see[h], found[x]);
              const int at = kFp4 ? 2 * d + x : d;
              w.o[nt][at] = mfma(v[x], p[nt][h], w.o[nt][at]);
            }
          }
#pragma unroll
          for (int x = 0; x < (kFp4 ? 2 : 1); ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (found[x][i] > 0.0f) w.o[nt][kFp4 ? 2 * d + x : d][i] = __builtin_nanf("");
        }
      }
      return;
    }
#pragma unroll
    for (int d = 0; d < kVLoads; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        half8_t v0, v1;
        operand(d, h, v0, v1);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          if constexpr (kFp4) {
            w.o[nt][2 * d] = mfma(v0, p[nt][h], w.o[nt][2 * d]);
            w.o[nt][2 * d + 1] = mfma(v1, p[nt][h], w.o[nt][2 * d + 1]);
          } else {
            w.o[nt][d] = mfma(v0, p[nt][h], w.o[nt][d]);
          }
        }
      }
    }
  }

  static __device__ __forceinline__ void load_q(const Attn& a, Wave& w, const Unit& u, int row0) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const float k_gs = *a.c.k_gs;
    const int64_t most = cache_rows(a);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const RowOf r = row_of(a, u, kRows, row0 + 16 * nt + n);
      const bool real = r.token >= 0;
      const int64_t row = u.w.rows.row0 + (real ? r.token : 0);
      const uint16_t* from = a.q + row * a.ldq + (int64_t)(real ? r.head : 0) * kD;
      u32x4_t x[kFrags];
      uint32_t top = 0;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        x[f] = u32x4_t{0, 0, 0, 0};
        if (real)
          x[f] = *reinterpret_cast<const u32x4_t*>(from + 4 * kVals * (f / kPerLoad) + kVals * g + 8 * (f % kPerLoad));
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[f][i] & 0x7FFFu, x[f][i] >> 16 & 0x7FFFu));
      }
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
        w.q[nt][f] = __builtin_bit_cast(half8_t, h);
      }
      // what is not finite in q makes every score of the row NaN
      w.c1[nt] = finite ? ldexpf(a.scale * k_gs, -shift) : __builtin_nanf("");
      w.m[nt] = kNoMax;
      w.l[nt] = 0.0f;
      w.limit[nt] = real ? row_limit(a, u.w.rows, most, r.token) : 0;
      w.seen[nt] = a.tree && real ? a.tree[row] : 0;
#pragma unroll
      for (int d = 0; d < kTiles; ++d) w.o[nt][d] = floatx4_t{0, 0, 0, 0};
    }
  }

  // The eight values of row n that lane (n, g) has of tiles 2 x and 2 x + 1:
  // two runs of four dims, at dims d0 and d1.
  static __device__ __forceinline__ void runs_of(int x, int g, int& d0, int& d1) {
    d0 = kFp4 ? 32 * x + 8 * g : 32 * x + 4 * g;
    d1 = kFp4 ? d0 + 4 : d0 + 16;
  }
  static __device__ __forceinline__ void in_order(const floatx4_t& a, const floatx4_t& b, floatx4_t r[2]) {
    if constexpr (kFp4) {
      r[0] = floatx4_t{a[0], b[0], a[1], b[1]};
      r[1] = floatx4_t{a[2], b[2], a[3], b[3]};
    } else {
      r[0] = a;
      r[1] = b;
    }
  }

  // Row rho's pair x of tiles, with its maximum m and sum l: to the output if
  // the unit is whole (slot < 0), else to the workspace.
  static __device__ __forceinline__ void emit(const Attn& a, const Unit& u, int rho, int x, const floatx4_t& t0,
                                              const floatx4_t& t1, float m, float l, int64_t slot) {
    const int g = (threadIdx.x & 63) >> 4;
    const RowOf r = row_of(a, u, kRows, rho);
    if (r.token < 0) return;
    int d[2];
    runs_of(x, g, d[0], d[1]);
    floatx4_t v[2];
    in_order(t0, t1, v);
    if (slot < 0) {
      const float f = l == 0.0f ? 0.0f : *a.c.v_gs / l;  // a row that sees nothing is zeros
      uint16_t* to = a.o + (u.w.rows.row0 + r.token) * a.ldo + (int64_t)r.head * kD;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x2_t b;
        b[0] = pack_bf16(v[i][0] * f, v[i][1] * f);
        b[1] = pack_bf16(v[i][2] * f, v[i][3] * f);
        *reinterpret_cast<u32x2_t*>(to + d[i]) = b;
      }
      return;
    }
    float* part = a.part + slot * (kRows * (kD + 2));
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<floatx4_t*>(part + rho * kD + d[i]) = v[i];
    if (x == 0 && g == 0) {
      part[kRows * kD + 2 * rho] = m;
      part[kRows * kD + 2 * rho + 1] = l;
    }
  }

  // Steps [k0, k1) of unit u.
  static __device__ __forceinline__ void run_unit(const Attn& a, const Unit& u, int64_t k0, int64_t k1, int64_t slot,
                                                  floatx4_t* lds) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 15;
    const int row0 = kSplit ? 0 : wave * kWaveRows;
    Wave w;
    load_q(a, w, u, row0);
    // the wave's first and last token, and from them the steps it has
    const int wide = a.parts == 1 ? a.group : kRows;
    const SeqRows& s = u.w.rows;
    const int64_t most = cache_rows(a);
    const int t0 = u.tile * a.tokens + row0 / wide;
    const int t1 = min(min(u.tile * a.tokens + (row0 + kWaveRows - 1) / wide, (u.tile + 1) * a.tokens - 1), s.n - 1);
    const int64_t reach = t0 > t1 ? 0 : row_limit(a, s, most, t1);
    const int64_t all = a.tree ? min((int64_t)s.kv - s.n, most) : row_limit(a, s, most, t0);  // every row sees these
    const int64_t end = min(k1, (reach + kStep - 1) / kStep), by = kSplit ? 4 : 1;
    int64_t k = k0 + (kSplit ? wave : 0);
    Pages next = k < end ? pages_of(a, u.seq, k * kStep) : Pages{-1, -1};
    for (; k < end; k += by) {
      const Pages pg = next;
      if (k + by < end) next = pages_of(a, u.seq, (k + by) * kStep);
      if ((k + 1) * kStep <= all && __builtin_amdgcn_ballot_w64(pg.k < 0 || pg.v < 0) == 0)
        step<false>(a, w, u, k * kStep, pg);
      else
        step<true>(a, w, u, k * kStep, pg);
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) w.l[nt] = sum_over_g(w.l[nt]);
    if constexpr (!kSplit) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int x = 0; x < kTiles / 2; ++x)
          emit(a, u, row0 + 16 * nt + n, x, w.o[nt][2 * x], w.o[nt][2 * x + 1], w.m[nt], w.l[nt], slot);
    } else {
      // four waves' results of the same rows: four pairs of tiles at a time, each wave adds up one pair
      float* ml = reinterpret_cast<float*>(lds + 4 * 8 * 64);  // [wave][nt][16][2]
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        if (lane < 16) {
          ml[((wave * kNT + nt) * 16 + n) * 2] = w.m[nt];
          ml[((wave * kNT + nt) * 16 + n) * 2 + 1] = w.l[nt];
        }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float m = kNoMax, l = 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) m = fmaxf(m, ml[((v * kNT + nt) * 16 + n) * 2]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float* at = ml + ((v * kNT + nt) * 16 + n) * 2;
          l += at[1] * __builtin_amdgcn_exp2f(at[0] - m);
        }
        const float f = __builtin_amdgcn_exp2f(w.m[nt] - m);
        constexpr int kPairs = kTiles / 2, kAtOnce = kPairs < 4 ? kPairs : 4;
#pragma unroll
        for (int x0 = 0; x0 < kPairs; x0 += kAtOnce) {
#pragma unroll
          for (int i = 0; i < 2 * kAtOnce; ++i) lds[(wave * 8 + i) * 64 + lane] = w.o[nt][2 * x0 + i] * f;
          __syncthreads();
          if (wave < kAtOnce) {
            floatx4_t t[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
              for (int i = 0; i < 2; ++i) t[i] += lds[(v * 8 + 2 * wave + i) * 64 + lane];
            emit(a, u, 16 * nt + n, x0 + wave, t[0], t[1], m, l, slot);
          }
          __syncthreads();
        }
      }
    }
  }
};

template <bool kFp4, int kD, int kNT, bool kSplit>
__global__ __launch_bounds__(256) void attn_kernel(Attn a) {
  using K = Kernel<kFp4, kD, kNT, kSplit>;
  __shared__ floatx4_t lds[kSplit ? 4 * 8 * 64 + 4 * kNT * 16 / 2 : 1];
  // neighbouring ranges on one XCD (workgroups go round the eight in turn): they share keys
  const int w = (int)(blockIdx.x & 7) * (a.ranges / 8) + (int)(blockIdx.x >> 3);
  const int64_t total = total_steps(a);
  const int64_t each = max((total + a.ranges - 1) / a.ranges, (int64_t)a.least);
  int64_t pos = w * each;
  const int64_t end = min(pos + each, total);
  if (pos >= end) return;
  Unit u = unit_at(a, pos);
  while (true) {
    const int64_t k0 = pos - u.start, k1 = min(u.steps, end - u.start);
    // a unit that is cut: its part behind the cut at the range's beginning, or before the one at its end
    const int64_t slot = k0 > 0 ? 2 * (int64_t)w : k1 < u.steps ? 2 * (int64_t)w + 1 : -1;
    K::run_unit(a, u, k0, k1, slot, lds);
    pos = u.start + k1;
    if (pos >= end) return;
    next_unit(a, u);
  }
}

// The first range that begins inside a unit joins the unit's parts: the end of
// the range before, its own, and those behind it up to the unit's end.  One
// row at a time; kD / 4 lanes share a row's values, the workgroup's 1024 / kD
// such groups its parts.
template <int kD>
__global__ __launch_bounds__(256) void attn_join_kernel(Attn a, int rows) {
  constexpr int kLanes = kD / 4, kGroups = 256 / kLanes;
  const int w = blockIdx.x + 1;
  const int64_t total = total_steps(a);
  const int64_t each = max((total + a.ranges - 1) / a.ranges, (int64_t)a.least);
  const int64_t pos = w * each;
  if (pos >= total) return;
  const Unit u = unit_at(a, pos);
  if (u.start == pos || u.start < pos - each) return;  // no cut here, or one before it in the same unit
  const int last = (int)((u.start + u.steps - 1) / each);  // the range of its last step
  const int n_parts = last - w + 2;
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int64_t size = (int64_t)rows * (kD + 2);
  const auto part = [&](int i) { return a.part + (i == 0 ? 2 * (int64_t)(w - 1) + 1 : 2 * (int64_t)(w + i - 1)) * size; };
  __shared__ float tops[4], ls[kGroups];
  __shared__ floatx4_t sums[256];
  for (int rho = blockIdx.y; rho < rows; rho += gridDim.y) {
    const RowOf r = row_of(a, u, rows, rho);
    if (r.token < 0) continue;
    // the maximum, and the sum under it, over all parts
    float m = kNoMax;
    for (int i = threadIdx.x; i < n_parts; i += 256) m = fmaxf(m, part(i)[(int64_t)rows * kD + 2 * rho]);
#pragma unroll
    for (int b = 32; b > 0; b >>= 1) m = fmaxf(m, __shfl_xor(m, b, 64));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    floatx4_t o = {0, 0, 0, 0};
    float l = 0.0f;
#pragma unroll 4
    for (int i = grp; i < n_parts; i += kGroups) {
      const float* p = part(i);
      const float f = __builtin_amdgcn_exp2f(p[(int64_t)rows * kD + 2 * rho] - m);
      l += p[(int64_t)rows * kD + 2 * rho + 1] * f;
      o += *reinterpret_cast<const floatx4_t*>(p + (int64_t)rho * kD + 4 * lane) * f;
    }
    sums[threadIdx.x] = o;
    if (lane == 0) ls[grp] = l;
    __syncthreads();
    if (grp == 0) {
      float sum = ls[0];
#pragma unroll
      for (int i = 1; i < kGroups; ++i) {
        o += sums[i * kLanes + lane];
        sum += ls[i];
      }
      const float f = sum == 0.0f ? 0.0f : *a.c.v_gs / sum;
      u32x2_t b;
      b[0] = pack_bf16(o[0] * f, o[1] * f);
      b[1] = pack_bf16(o[2] * f, o[3] * f);
      *reinterpret_cast<u32x2_t*>(a.o + (u.w.rows.row0 + r.token) * a.ldo + (int64_t)r.head * kD + 4 * lane) = b;
    }
    __syncthreads();
  }
}

// How a call is laid out: by the rows that a sequence has on average for each
// key/value head, which the host knows, so that no kernel waits for lengths.
struct Plan {
  int nt;
  bool split;
  int rows, ranges, least;
};

Plan plan_of(int64_t T, int n_seqs, int group, int d) {
  const int64_t rows = (T * group + n_seqs - 1) / n_seqs;
  if (rows <= 16) return {1, true, 16, 512, 4};
  if (rows <= 32) return {2, true, 32, 512, 4};
  return {2, false, 128, 512, 4};
}

template <bool kFp4, int kD>
void launch_typed(const Plan& p, const Attn& a, hipStream_t stream) {
  const auto f = p.nt == 1 ? attn_kernel<kFp4, kD, 1, true>
                           : p.split ? attn_kernel<kFp4, kD, 2, true> : attn_kernel<kFp4, kD, 2, false>;
  f<<<(unsigned)p.ranges, 256, 0, stream>>>(a);
  attn_join_kernel<kD><<<dim3((unsigned)p.ranges - 1, 16), 256, 0, stream>>>(a, p.rows);
}

}  // namespace

size_t attn_cached_workspace_bytes(int64_t T, int n_seqs, int hq, int hk, int d) {
  const Plan p = plan_of(T, n_seqs, hq / hk, d);
  return (size_t)2 * p.ranges * p.rows * (d + 2) * sizeof(float);
}

hipError_t launch_attn_cached(const KvCache& c, const KvRows& r, const void* q, int64_t ldq, int hq, float scale,
                              const uint64_t* tree, void* o, int64_t ldo, void* workspace, hipStream_t stream) {
  const int group = hq / c.hk;
  const Plan p = plan_of(r.T, r.n_seqs, group, c.d);
  const Attn a{c,      r,       static_cast<const uint16_t*>(q), ldq, group, scale * 1.44269504088896340736f, tree,
               static_cast<uint16_t*>(o), ldo, static_cast<float*>(workspace), p.ranges, p.least,
               group <= p.rows ? p.rows / group : 1, group <= p.rows ? 1 : (group + p.rows - 1) / p.rows};
  if (c.fp4)
    c.d == 64 ? launch_typed<true, 64>(p, a, stream)
              : c.d == 128 ? launch_typed<true, 128>(p, a, stream) : launch_typed<true, 256>(p, a, stream);
  else
    c.d == 64 ? launch_typed<false, 64>(p, a, stream)
              : c.d == 128 ? launch_typed<false, 128>(p, a, stream) : launch_typed<false, 256>(p, a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
