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
// Work: the keys of all (sequence, tile of rows, head) are laid end to end and
// cut into equal ranges, one per workgroup, so that one long sequence among
// short ones, or one request alone, still fills the GPU.  Every workgroup finds
// its place from the lengths by itself.  A unit cut by a range's end leaves its
// maximum, sum and unscaled result in the workspace, and a second kernel joins
// them, in order.
#include "nvfp4_kv.h"

namespace nvfp4 {
namespace {

constexpr int kStep = 64;      // keys per step
constexpr int kRanges = 256;   // workgroups, one for each CU
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
  float* part;      // [2 kRanges][rows x (d + 2)]
  int least;        // keys of a range, at least
  int start;        // what beginning and ending a unit takes, in keys
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

// a / b for 0 <= a < 2^62, b > 0 and quotients below 2^52: the quotient of the doubles is off by one at most.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  int64_t q = (int64_t)((double)a / (double)b);
  const int64_t r = a - q * b;
  return r < 0 ? q - 1 : r >= b ? q + 1 : q;
}

// A sequence's share of the work, counted in keys.  Its tiles of rows (`tokens`
// tokens each) count first + r slope keys per head, r the tile: what the tile's
// last token sees (or somewhat more in the last tile), and what beginning and
// ending a unit takes, so that a range of many short units is no longer than others.
// Step k of a unit belongs to the range that holds its key 64 k.
struct SeqWork {
  SeqRows rows;
  int64_t first;
  int slope;
  int tiles;
  int minor;  // heads x parts, which share a tile's count
  __device__ __forceinline__ int64_t before(int64_t r) const {  // keys of the tiles before r
    return minor * (r * first + r * (r - 1) / 2 * slope);
  }
  __device__ __forceinline__ int64_t keys(int64_t r) const { return first + r * slope; }
  __device__ __forceinline__ int64_t total() const { return before(tiles); }
};

// Values that are the same in every lane, told to the compiler: they then live
// in scalar registers, and branches on them are branches of the wave.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// Positions that the page table has room for, and that fit the kernels' ints.
__device__ __forceinline__ int cache_rows(const Attn& a) {
  return (int)min((int64_t)a.r.max_pages << a.c.page_shift, (int64_t)INT32_MAX - 127);
}

__device__ __forceinline__ SeqWork seq_work(const Attn& a, int i) {
  SeqWork w;
  w.rows = seq_rows(a.r, i);
  const int most = cache_rows(a);
  if (a.tree) {
    w.first = min(max(w.rows.kv, 1), most) + a.start;
    w.slope = 0;
  } else {
    w.first = min(max((int64_t)w.rows.kv - w.rows.n, (int64_t)0), (int64_t)most) + a.tokens + a.start;
    w.slope = a.tokens;
  }
  w.tiles = (w.rows.n + a.tokens - 1) / a.tokens;
  w.minor = a.c.hk * a.parts;
  return w;
}

// How the keys of all sequences are cut into ranges.
struct Cut {
  int64_t total, each;  // keys in all; keys of a range
  int64_t mine;         // the lane's sequence's (of the first 64)
};
__device__ __forceinline__ Cut cut_of(const Attn& a) {
  const int lane = threadIdx.x & 63;
  Cut c;
  c.mine = lane < a.r.n_seqs ? seq_work(a, lane).total() : 0;
  int64_t sum = c.mine;
  for (int i = lane + 64; i < a.r.n_seqs; i += 64) sum += seq_work(a, i).total();
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 64);
  c.total = uniform(sum);
  c.each = max((c.total + kRanges - 1) / kRanges, (int64_t)a.least);
  return c;
}

// The sequence that holds key `pos` (below the total), and the keys before it.
__device__ __forceinline__ int find_seq(const Attn& a, const Cut& c, int64_t pos, int64_t& before) {
  const int lane = threadIdx.x & 63;
  before = 0;
  for (int i0 = 0; i0 < a.r.n_seqs; i0 += 64) {
    const int64_t mine = i0 == 0 ? c.mine : i0 + lane < a.r.n_seqs ? seq_work(a, i0 + lane).total() : 0;
    const int64_t upto = before + scan64(mine);
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > pos);
    if (past) {
      const int at = __builtin_ctzll(past);
      before = uniform(__shfl(upto - mine, at, 64));
      return uniform(i0 + at);
    }
    before = uniform(__shfl(upto, 63, 64));
  }
  return 0;
}

// A unit of work: one tile of one sequence's rows and one (head, part).
struct Unit {
  int seq;
  SeqWork w;
  int tile, minor;
  int64_t start, keys;  // its place among all keys
};

__device__ __forceinline__ void take_seq(const Attn& a, Unit& u, int seq) {
  u.seq = seq;
  u.w = seq_work(a, seq);
  u.w.rows.row0 = uniform(u.w.rows.row0);
  u.w.rows.n = uniform(u.w.rows.n);
  u.w.rows.kv = uniform(u.w.rows.kv);
  u.w.first = uniform(u.w.first);
  u.w.tiles = uniform(u.w.tiles);
}

__device__ __forceinline__ Unit unit_at(const Attn& a, const Cut& c, int64_t pos) {
  Unit u;
  int64_t before;
  const int seq = find_seq(a, c, pos, before);
  take_seq(a, u, seq);
  const int64_t x = pos - before;
  u.tile = u.w.tiles == 1 ? 0 : last_before(u.w.tiles, [&](int r) { return u.w.before(r) <= x; });
  u.keys = uniform(u.w.keys(u.tile));
  const int64_t y = uniform(x - u.w.before(u.tile));
  u.minor = uniform((int)quotient(y, u.keys));
  u.start = pos - (y - (int64_t)u.minor * u.keys);
  return u;
}

// The unit behind u (there is one).
__device__ __forceinline__ void next_unit(const Attn& a, Unit& u) {
  u.start += u.keys;
  if (++u.minor < u.w.minor) return;
  u.minor = 0;
  if (++u.tile == u.w.tiles) {
    u.tile = 0;
    do take_seq(a, u, u.seq + 1);
    while (u.w.tiles == 0 && u.seq + 1 < a.r.n_seqs);
  }
  u.keys = uniform(u.w.keys(u.tile));
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
__device__ __forceinline__ int row_limit(const Attn& a, const SeqRows& s, int token) {
  const int64_t end = a.tree ? (int64_t)s.kv : min((int64_t)s.kv, (int64_t)s.kv - s.n + token + 1);
  return (int)max(min(end, (int64_t)cache_rows(a)), (int64_t)0);
}

// What a wave with rows row0 .. row0 + count - 1 of the tile has to do.
struct Reach {
  int all;    // every row of it sees the positions below
  int steps;  // steps up to the last position that one of them sees
};
__device__ __forceinline__ Reach reach_of(const Attn& a, const Unit& u, int rows, int row0, int count) {
  const int wide = a.parts == 1 ? a.group : rows;
  const SeqRows& s = u.w.rows;
  const int first = u.tile * a.tokens, last = min(first + a.tokens, s.n) - 1;
  const int t0 = first + row0 / wide, t1 = min(first + (row0 + count - 1) / wide, last);
  Reach r;
  r.all = a.tree ? (int)min((int64_t)s.kv - s.n, (int64_t)cache_rows(a)) : row_limit(a, s, t0);
  r.steps = t0 > t1 ? 0 : (row_limit(a, s, t1) + kStep - 1) / kStep;
  return r;
}

__device__ __forceinline__ float max_over_g(float v) {  // over lanes n, n + 16, n + 32, n + 48
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
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
template <bool kFp4, int kD, int kNT, bool kPin>
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
  float m[kNT], c1[kNT];          // running maximum, factor of the scores (log2)
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
        // to an accumulation register, where matrix instructions can read it, and for good: left to itself the
        // compiler keeps its parts apart and puts them together again in every step
        if constexpr (kPin) asm volatile("" : "+a"(q[nt][f]));
      }
      c1[nt] = ldexpf(a.scale * k_gs, -shift);
      fate[nt] = finite ? 1.0f : __builtin_nanf("");  // what is not finite in q makes the row NaN if it sees anything
      m[nt] = kNoMax;
      sum[nt] = floatx4_t{0, 0, 0, 0};
      limit[nt] = real ? row_limit(a, u.w.rows, r.token) : 0;
      seen[nt] = a.tree && real ? a.tree[row] : 0;
#pragma unroll
      for (int d = 0; d < kTiles; ++d) o[nt][d] = floatx4_t{0, 0, 0, 0};
    }
  }

  // Bits of the lane's 16 keys from position `key` on that row n of tile nt sees.
  __device__ __forceinline__ uint32_t seen_bits(const Attn& a, int nt, const SeqRows& s, int key, bool has_page) const {
    const auto below = [&](int64_t end) { return (1u << (int)min(max(end - key, (int64_t)0), (int64_t)16)) - 1u; };
    uint32_t bits = below(limit[nt]);
    if (a.tree) {
      const int64_t ctx = (int64_t)s.kv - s.n, b = key - ctx;
      const uint64_t drafts = b >= 0 ? (b < 64 ? seen[nt] >> b : 0) : (b > -16 ? seen[nt] << -b : 0);
      bits &= below(ctx) | (uint32_t)drafts;
    }
    return has_page ? bits : 0u;
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
  __device__ __forceinline__ void raise_max(const float top[kNT]) {
    bool lags = false;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) lags = lags || top[nt] * c1[nt] > m[nt] + kLag;
    if (__builtin_amdgcn_ballot_w64(lags)) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const float now = fmaxf(m[nt], max_over_g(top[nt] * c1[nt])), f = __builtin_amdgcn_exp2f(m[nt] - now);
        m[nt] = now;
        sum[nt] *= f;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) o[nt][d] *= f;
      }
    }
  }

  // Scores of keys key .. key + 15 that their row does not see become -inf.
  __device__ __forceinline__ void hide(const Attn& a, const SeqRows& sr, int key, bool has_page, Scores& s) const {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const uint32_t bits = seen_bits(a, nt, sr, key, has_page);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[nt][e / 4][e % 4] = bits >> e & 1 ? s[nt][e / 4][e % 4] : -INFINITY;
    }
  }

  // Part x of `parts` of the rows' weights of the lane's 16 keys, under the running maximum.
  __device__ __forceinline__ void weights(int x, int parts, const Scores& s, half8_t p[kNT][2]) {
#pragma unroll
    for (int i = 8 * kNT * x / parts; i < 8 * kNT * (x + 1) / parts; ++i) {
      const int nt = i / 8, e = i % 8 * 2;
      const float off = kLift - m[nt];
      const float v = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4], c1[nt], off));
      const float y = __builtin_amdgcn_exp2f(fmaf(s[nt][e / 4][e % 4 + 1], c1[nt], off));
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
  // Row rho (of `rows`), its maximum m and sum l.
  __device__ __forceinline__ Sink(const Attn& a, const Unit& u, int rows, int rho, float m, float l, int slot) {
    const int g = (threadIdx.x & 63) >> 4;
    const RowOf r = row_of(a, u, rows, rho);
    to = nullptr;
    part = nullptr;
    if (r.token < 0) return;
    if (slot < 0) {
      f = l == 0.0f ? 0.0f : *a.c.v_gs / l;  // a row that sees nothing is zeros
      to = a.o + (u.w.rows.row0 + r.token) * a.ldo + (int64_t)r.head * kD;
    } else {
      float* base = a.part + (int64_t)slot * (rows * (kD + 2));
      part = base + rho * kD;
      if (g == 0) {
        base[rows * kD + 2 * rho] = m;
        base[rows * kD + 2 * rho + 1] = l;
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

// How many of a lane's 16 keys of a step are there.
__device__ __forceinline__ int keys_there(const Attn& a, const SeqRows& s, int step, int page) {
  const int exist = min(s.kv, cache_rows(a)), key = step * kStep + 16 * ((threadIdx.x & 63) >> 4);
  return page < 0 ? 0 : min(max(exist - key, 0), 16);
}

template <bool kFp4, int kD>
struct Codes {
  using R = Rows<kFp4, kD, 1, false>;

  // The lane's part of the row of K's tile t.
  static __device__ __forceinline__ void load_k(const Attn& a, int head, int step, int page, int t,
                                                RawK<kFp4, R::kLoads>& r) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, ps = 1 << a.c.page_shift;
    const int krow = (step * kStep + 16 * (n >> 2) + (n & 3)) & (ps - 1);
    const int64_t row = ((int64_t)max(page, 0) * a.c.hk + head) * ps + krow + 4 * t;
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
    const int64_t unit = (int64_t)max(page, 0) * a.c.hk + head;
    const uint8_t* at = a.c.v + (unit * code_bytes<kFp4>(kD) + 16 * first + n) * ps + vrow;
    const uint8_t* sc = kFp4 ? a.c.v_scales + (unit * (kD / 16) + 2 * first + (n >> 3)) * ps + vrow : nullptr;
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
        const int b = min(max(keep - 4 * w, 0), 4);
        x[w] &= b == 4 ? ~0u : (1u << (8 * b)) - 1u;
        const uint32_t nan = ((x[w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // top bit of a NaN byte
        bad |= nan;
        x[w] &= ~((nan >> 7) * 0xFFu);
      }
    }
    return __builtin_amdgcn_ballot_w64(bad != 0) != 0;
  }
  // What clear_v took out of the steps k, k + by, ... before `end`: the results that see it become NaN.  The codes
  // are read once more, of the steps that not every row sees all of (`all`: positions that every row sees).
  template <int kNT, bool kPin>
  static __device__ __forceinline__ void spread_nan(const Attn& a, const Unit& u, Rows<kFp4, kD, kNT, kPin>& w, int head, int k,
                                                 int end, int by, int all) {
    for (; k < end; k += by) {
      const Pages pg = pages_now(a, u.seq, k);
      if ((k + 1) * kStep <= all && all_there(pg)) continue;
      const int keep = keys_there(a, u.w.rows, k, pg.v), key = k * kStep + 16 * ((threadIdx.x & 63) >> 4);
      uint32_t bits[kNT];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) bits[nt] = w.seen_bits(a, nt, u.w.rows, key, pg.v >= 0) & ((1u << keep) - 1u);
#pragma unroll
      for (int d = 0; d < R::kVLoads; ++d) {
        RawV<kFp4, 1> r;
        half8_t v[2][2];
        load_v(a, head, k, pg.v, d, 0, r);
        u32x4_t& x = kFp4 ? r.sc[0] : r.x[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // keys that are not there may hold anything
          const int b = min(max(keep - 4 * i, 0), 4);
          x[i] &= b == 4 ? ~0u : (1u << (8 * b)) - 1u;
        }
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

// Few rows per sequence (decode): the workgroup's four waves have the same 16
// kNT rows and every fourth step each, straight from memory to the matrix
// instructions; their results are joined through LDS.
template <bool kFp4, int kD, int kNT>
struct Few {
  using R = Rows<kFp4, kD, kNT, false>;
  using C = Codes<kFp4, kD>;
  static constexpr int kRows = R::kWaveRows;
  struct Lds {
    floatx4_t sums[4 * 8 * 64];
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
    w.raise_max(top);
    w.weights(0, 1, s, p);
    w.add_sums(p);
    bool nan = false;
    if (!whole) nan = C::clear_v(rv, keys_there(a, u.w.rows, step, pg.v));
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
    const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15;
    const int head = u.minor / a.parts;
    R w;
    const Reach reach = reach_of(a, u, kRows, 0, kRows);
    const int end = min(k1, reach.steps);
    int k = k0 + wave;
    const int last = max(end - 1, k0);
    const Pages e0 = entries_of(a, u.seq, min(k, last)), e1 = entries_of(a, u.seq, min(k + 4, last));
    w.load_q(a, u, kRows, 0);
    bool nan = false;
    if (k < end) {
      Keys keys;
      Pages pg = pages_of(a, k, e0), pg2 = pages_of(a, min(k + 4, end - 1), e1);
      load_keys(a, head, k, pg, keys);
      for (; k < end; k += 4) {
        const Pages e = entries_of(a, u.seq, min(k + 8, end - 1));
        nan |= run_step(a, u, head, w, keys, k, pg, (k + 1) * kStep <= reach.all && all_there(pg), min(k + 4, end - 1), pg2);
        pg = pg2;
        pg2 = pages_of(a, min(k + 8, end - 1), e);
      }
    }
    if (nan) C::spread_nan(a, u, w, head, k0 + wave, end, 4, reach.all);
    // four waves' results of the same rows: four pairs of tiles at a time, each wave adds up one pair
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
      float m = kNoMax, l = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) m = fmaxf(m, lds.ml[v][nt][n][0]);
#pragma unroll
      for (int v = 0; v < 4; ++v) l += lds.ml[v][nt][n][1] * __builtin_amdgcn_exp2f(lds.ml[v][nt][n][0] - m);
      const float f = __builtin_amdgcn_exp2f(w.m[nt] - m);
      const Sink<kFp4, kD> sink(a, u, kRows, 16 * nt + n, m, l, slot);
      constexpr int kPairs = R::kTiles / 2, kAtOnce = kPairs < 4 ? kPairs : 4;
#pragma unroll
      for (int x0 = 0; x0 < kPairs; x0 += kAtOnce) {
#pragma unroll
        for (int i = 0; i < 2 * kAtOnce; ++i) lds.sums[(wave * 8 + i) * 64 + lane] = w.o[nt][2 * x0 + i] * f;
        __syncthreads();
        if (wave < kAtOnce) {
          floatx4_t t[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int i = 0; i < 2; ++i) t[i] += lds.sums[(v * 8 + 2 * wave + i) * 64 + lane];
          sink.put(x0 + wave, t[0], t[1]);
        }
        __syncthreads();
      }
    }
  }
};

// Many rows per sequence (prompts, large trees): the waves have 16 kNT rows each
// and share every step's keys, which the workgroup makes fp16 once, in LDS, in
// the order of the matrix instructions' operands (a lane's 16 bytes side by
// side: no bank conflicts, constant offsets).  In registers each wave would
// convert all of them itself, as many vector instructions as the softmax has.
// Wave t converts K's tile t and every fourth load of V.
//
// One barrier a step.  In step j the scores of step j + 1 are multiplied while
// step j's softmax is evaluated (neither waits for the other), then P V of step j;
// codes of K's step j + 2 and V's step j + 1 are asked for at its beginning and
// converted at its end, into the halves of the buffers that step j - 1 was the last
// to read.
template <bool kFp4, int kD, int kNT>
struct Many {
  using R = Rows<kFp4, kD, kNT, true>;
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
    w.raise_max(now.top);
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
      st.nan |= C::clear_v(st.rv, keys_there(a, u.w.rows, k1, st.p1.v));
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
               C::clear_v(st.rv, keys_there(a, u.w.rows, k0, st.p0.v));
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
      const Sink<kFp4, kD> sink(a, u, kRows, row0 + 16 * nt + n, w.m[nt], w.total(nt), slot);
#pragma unroll
      for (int x = 0; x < R::kTiles / 2; ++x) sink.put(x, w.o[nt][2 * x], w.o[nt][2 * x + 1]);
    }
  }
};

// The workgroup's range, unit by unit: run(unit, first step, step behind the last, slot of its part or -1).
template <class Run>
__device__ __forceinline__ void run_range(const Attn& a, Run run) {
  // neighbouring ranges on one XCD (workgroups go round the eight in turn): they share keys
  const int w = (int)(blockIdx.x & 7) * (kRanges / 8) + (int)(blockIdx.x >> 3);
  const Cut c = cut_of(a);
  int64_t pos = w * c.each;
  const int64_t end = min(pos + c.each, c.total);
  if (pos >= end) return;
  Unit u = unit_at(a, c, pos);
  while (true) {
    const int64_t from = pos - u.start, to = min(u.keys, end - u.start);
    // a unit that is cut: its part behind the cut at the range's beginning, or before the one at its end
    const int slot = from > 0 ? 2 * w : to < u.keys ? 2 * w + 1 : -1;
    run(u, (int)((from + kStep - 1) / kStep), (int)((to + kStep - 1) / kStep), slot);
    pos = u.start + to;
    if (pos >= end) return;
    next_unit(a, u);
  }
}

template <bool kFp4, int kD, int kNT>
__global__ __launch_bounds__(256) void attn_few_kernel(Attn a) {
  __shared__ typename Few<kFp4, kD, kNT>::Lds lds;
  run_range(a, [&](const Unit& u, int k0, int k1, int slot) { Few<kFp4, kD, kNT>::run_unit(a, u, k0, k1, slot, lds); });
}

template <bool kFp4, int kD, int kNT>
__global__ __launch_bounds__(256) void attn_many_kernel(Attn a) {
  __shared__ typename Many<kFp4, kD, kNT>::Lds lds;
  run_range(a, [&](const Unit& u, int k0, int k1, int slot) { Many<kFp4, kD, kNT>::run_unit(a, u, k0, k1, slot, lds); });
}

// A unit that is cut `cuts` times has cuts + 1 parts: the end of one range, whole
// ranges, and the beginning of the last.  Its rows are joined by the workgroups
// of its cuts (blockIdx.x + 1 is the range that begins there; blockIdx.y shares
// the rows out further).  kD / 4 lanes share a row's values.  With few parts each
// such group of lanes joins a row of its own, else the groups share a row's parts.
// (With one workgroup per row and cut, most of which found nothing to do, joining took as long as
// the attention itself: 10.6 us of 24 for one request, 33 of 130 for 16 trees.)
template <int kD>
__global__ __launch_bounds__(256) void attn_join_kernel(Attn a, int rows) {
  constexpr int kLanes = kD / 4, kGroups = 256 / kLanes, kFewParts = 16;
  const int w = blockIdx.x + 1;
  const Cut c = cut_of(a);
  const int64_t pos = w * c.each;
  if (pos >= c.total) return;
  const Unit u = unit_at(a, c, pos);
  if (u.start == pos) return;  // between two units
  const int first = (int)quotient(u.start, c.each) + 1, cuts = (int)quotient(u.start + u.keys - 1, c.each) - first + 1;
  const int share = (w - first) * gridDim.y + blockIdx.y, shares = cuts * gridDim.y;
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int64_t size = (int64_t)rows * (kD + 2);
  const float* parts = a.part + (2 * (int64_t)first - 1) * size;  // of the range before: slot 2 (first - 1) + 1
  const auto part = [&](int i) { return parts + (i == 0 ? 0 : 2 * i - 1) * size; };
  const float v_gs = *a.c.v_gs;
  const auto put = [&](const RowOf& r, const floatx4_t& o, float l) {
    const float f = l == 0.0f ? 0.0f : v_gs / l;  // a row that sees nothing is zeros
    u32x2_t b;
    b[0] = pack_bf16(o[0] * f, o[1] * f);
    b[1] = pack_bf16(o[2] * f, o[3] * f);
    *reinterpret_cast<u32x2_t*>(a.o + (u.w.rows.row0 + r.token) * a.ldo + (int64_t)r.head * kD + 4 * lane) = b;
  };
  // Parts first, first + by, ... of row rho, under their own maximum.
  const auto join = [&](int rho, int from, int by, float& m, float& l, floatx4_t& o) {
    m = kNoMax;
    l = 0.0f;
    o = floatx4_t{0, 0, 0, 0};
#pragma unroll 4
    for (int i = from; i <= cuts; i += by) m = fmaxf(m, part(i)[rows * kD + 2 * rho]);
#pragma unroll 4
    for (int i = from; i <= cuts; i += by) {
      const float* p = part(i);
      const float f = __builtin_amdgcn_exp2f(p[rows * kD + 2 * rho] - m);
      l += p[rows * kD + 2 * rho + 1] * f;
      o += *reinterpret_cast<const floatx4_t*>(p + rho * kD + 4 * lane) * f;
    }
  };
  float m, l;
  floatx4_t o;
  if (cuts < kFewParts) {
    for (int rho = share * kGroups + grp; rho < rows; rho += shares * kGroups) {
      const RowOf r = row_of(a, u, rows, rho);
      if (r.token < 0) continue;
      join(rho, 0, 1, m, l, o);
      put(r, o, l);
    }
    return;
  }
  __shared__ float ml[2][kGroups];
  __shared__ floatx4_t sums[256];
  for (int rho = share; rho < rows; rho += shares) {
    const RowOf r = row_of(a, u, rows, rho);
    if (r.token < 0) continue;
    join(rho, grp, kGroups, m, l, o);
    sums[threadIdx.x] = o;
    if (lane == 0) {
      ml[0][grp] = m;
      ml[1][grp] = l;
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int i = 1; i < kGroups; ++i) m = fmaxf(m, ml[0][i]);
      l = 0.0f;
      o = floatx4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[0][i] - m);
        l += ml[1][i] * f;
        o += sums[i * kLanes + lane] * f;
      }
      put(r, o, l);
    }
    __syncthreads();
  }
}

// How a call is laid out: by the rows that a sequence has on average for each
// key/value head, which the host knows, so that no kernel waits for lengths.
struct Plan {
  int nt;
  bool split;
  int rows, least, start;
};

Plan plan_of(int64_t T, int n_seqs, int group, int d) {
  const int64_t rows = (T * group + n_seqs - 1) / n_seqs;
  if (rows <= 16) return {1, true, 16, 256, 256};
  if (rows <= 32) return {2, true, 32, 256, 256};
  return {2, false, 128, 256, 512};
}

template <bool kFp4, int kD>
void launch_typed(const Plan& p, const Attn& a, hipStream_t stream) {
  const auto f = p.nt == 1 ? attn_few_kernel<kFp4, kD, 1>
                           : p.split ? attn_few_kernel<kFp4, kD, 2> : attn_many_kernel<kFp4, kD, 2>;
  f<<<kRanges, 256, 0, stream>>>(a);
  attn_join_kernel<kD><<<dim3(kRanges - 1, p.split ? 1 : 8), 256, 0, stream>>>(a, p.rows);
}

}  // namespace

size_t attn_cached_workspace_bytes(int64_t T, int n_seqs, int hq, int hk, int d) {
  const Plan p = plan_of(T, n_seqs, hq / hk, d);
  return (size_t)2 * kRanges * p.rows * (d + 2) * sizeof(float);
}

hipError_t launch_attn_cached(const KvCache& c, const KvRows& r, const void* q, int64_t ldq, int hq, float scale,
                              const uint64_t* tree, void* o, int64_t ldo, void* workspace, hipStream_t stream) {
  const int group = hq / c.hk;
  const Plan p = plan_of(r.T, r.n_seqs, group, c.d);
  const Attn a{c,      r,       static_cast<const uint16_t*>(q), ldq, group, scale * 1.44269504088896340736f, tree,
               static_cast<uint16_t*>(o), ldo, static_cast<float*>(workspace), p.least, p.start,
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
