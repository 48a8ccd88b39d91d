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
//    hides keys from some rows, NaN codes are taken as zeros, and if there were
//    any, the unit's steps of that kind are read once more behind the last one and a
//    product of what is seen and what is NaN says which results are NaN.
//
// Work: the keys of all (sequence, tile of rows, head) are laid end to end and
// cut into equal ranges, one per workgroup (or per wave, for many short
// sequences), so that one long sequence among short ones, or one request alone,
// still fills the GPU.  Every range finds its place from the lengths by itself.  A
// unit cut by a range's end leaves its maximum, sum and unscaled result in the
// workspace, and a second kernel joins them, in order.
#pragma once

#include "nvfp4_kv.h"

namespace nvfp4 {

// The unit that a range's beginning cuts, for the joining of its parts.
struct Joint {
  int64_t row0;  // of its sequence
  int n;         // its sequence's rows
  int tile, minor;
  int first;     // the first range that begins within it
  int cuts;      // ranges that do; 0: this one begins between two units, or not at all
  int unused;
};

struct Attn {
  KvCache c;
  KvRows r;
  const uint16_t* q;
  int64_t ldq;
  int group;        // query heads per key/value head
  float scale;      // of the scores, times log2(e): scale * 2^power, scale in [0.7, 1.5), as the product with the
  int power;        // tensor scale may be no fp32 number where the scores themselves are
  const uint64_t* tree;
  uint16_t* o;
  int64_t ldo;
  float* part;      // [2 ranges][rows x (d + kPartMore)]
  Joint* joints;    // [ranges]
  int least;        // keys of a range, at least
  int start;        // what beginning and ending a unit takes, in keys
  int ranges;       // of workgroups, or (solo) of waves; a multiple of 32
  int tokens, parts;  // tokens per tile of rows; tiles that a token's heads take
};

// The kernels for few and for many rows per sequence (16 nt and 128 rows of a tile).
void launch_attn_few(const Attn& a, int nt, bool solo, hipStream_t stream);
void launch_attn_many(const Attn& a, hipStream_t stream);

namespace {

constexpr int kStep = 64;      // keys per step
constexpr int kCus = 256;
constexpr float kLag = 8.0f;   // log2: how far the running maximum may lag behind
constexpr float kLift = 7.0f;  // log2: P is stored times 2^7
constexpr float kFar = 4096.0f;  // log2: from here on weights are formed from differences of scores
constexpr int kPartMore = 3;    // of a row's part, beside its values: maximum, sum, factor of the scores

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
    w.first = (int64_t)min(max(w.rows.kv, 1), most) + a.start;
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
  int64_t mine;         // of the lane's share of the sequences, `chunk` neighbours
  int chunk;
};
__device__ __forceinline__ Cut cut_of(const Attn& a) {
  const int lane = threadIdx.x & 63;
  Cut c;
  c.chunk = (a.r.n_seqs + 63) / 64;
  c.mine = lane * c.chunk < a.r.n_seqs ? seq_work(a, lane * c.chunk).total() : 0;
  if (c.chunk > 1) {
#pragma unroll 4
    for (int i = lane * c.chunk + 1; i < min((lane + 1) * c.chunk, a.r.n_seqs); ++i) c.mine += seq_work(a, i).total();
  }
  int64_t sum = c.mine;
  if (a.r.n_seqs > 1) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 64);
  }
  c.total = uniform(sum);
  c.each = max((c.total + a.ranges - 1) / a.ranges, (int64_t)a.least);
  return c;
}

// The first lane whose keys, in order behind `before`, go past `pos`, and the keys before it; -1 where none does.
__device__ __forceinline__ int find_lane(int64_t mine, int64_t pos, int64_t& before) {
  const int64_t upto = before + scan64(mine);
  const uint64_t past = __builtin_amdgcn_ballot_w64(upto > pos);
  const int at = past ? __builtin_ctzll(past) : 63;
  before = uniform(__shfl(past ? upto - mine : upto, at, 64));
  return past ? uniform(at) : -1;
}

// The sequence that holds key `pos` (below the total), and the keys before it.
__device__ __forceinline__ int find_seq(const Attn& a, const Cut& c, int64_t pos, int64_t& before) {
  before = 0;
  if (a.r.n_seqs == 1) return 0;
  const int first = max(find_lane(c.mine, pos, before), 0) * c.chunk, end = min(first + c.chunk, a.r.n_seqs);
  if (c.chunk == 1) return first;
  for (int i0 = first; i0 < end; i0 += 64) {
    const int i = i0 + (threadIdx.x & 63);
    const int at = find_lane(i < end ? seq_work(a, i).total() : 0, pos, before);
    if (at >= 0) return i0 + at;
  }
  return end - 1;
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
__device__ __forceinline__ RowOf row_of(const Attn& a, int tile, int minor, int n, int rows, int rho) {
  const int wide = a.parts == 1 ? a.group : rows;
  const int h = (minor % a.parts) * rows + rho % wide;
  const int token = tile * a.tokens + rho / wide;
  const bool real = rho < a.tokens * wide && h < a.group && token < n;
  return {real ? token : -1, (minor / a.parts) * a.group + h};
}
__device__ __forceinline__ RowOf row_of(const Attn& a, const Unit& u, int rows, int rho) {
  return row_of(a, u.tile, u.minor, u.w.rows.n, rows, rho);
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

// What weights under the maximum `from` are multiplied by to be under `to`; c1: the factor of the scores.
__device__ __forceinline__ float rescale(float from, float to, float c1) {
  return from == to ? 1.0f : __builtin_amdgcn_exp2f((from - to) * c1);
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

// Bits of the 16 keys from position `key` on that a row sees, which may see `limit` positions and has tree mask `tree`.
__device__ __forceinline__ uint32_t seen_bits(const Attn& a, const SeqRows& s, int limit, uint64_t tree, int key,
                                              bool has_page) {
  const auto below = [&](int64_t end) { return (1u << (int)min(max(end - key, (int64_t)0), (int64_t)16)) - 1u; };
  uint32_t bits = below(limit);
  if (a.tree) {
    const int64_t ctx = (int64_t)s.kv - s.n, b = key - ctx;
    const uint64_t drafts = b >= 0 ? (b < 64 ? tree >> b : 0) : (b > -16 ? tree << -b : 0);
    bits &= below(ctx) | (uint32_t)drafts;
  }
  return has_page ? bits : 0u;
}

// How many of the 16 keys from position `key` on are there.
__device__ __forceinline__ int keys_there(const Attn& a, const SeqRows& s, int key, int page) {
  return page < 0 ? 0 : min(max(min(s.kv, cache_rows(a)) - key, 0), 16);
}

// The bytes of word w (four keys) of the first `keep` keys.
__device__ __forceinline__ uint32_t kept_bytes(int keep, int w) {
  const int b = min(max(keep - 4 * w, 0), 4);
  return b == 4 ? ~0u : (1u << (8 * b)) - 1u;
}
// Top bit of every byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Neighbouring ranges go to one XCD (workgroups go round the eight in turn): they share keys.
__device__ __forceinline__ int xcd_order(int block, int blocks) { return (block & 7) * (blocks / 8) + (block >> 3); }

// Range w, unit by unit: run(unit, first step, step behind the last, slot of its part or -1).
template <class Run>
__device__ __forceinline__ void run_range(const Attn& a, int w, Run run) {
  const Cut c = cut_of(a);
  int64_t pos = w * c.each;
  const int64_t end = min(pos + c.each, c.total);
  const bool one = (threadIdx.x & 63) == 0;
  if (pos >= end) {
    if (one) a.joints[w].cuts = 0;
    return;
  }
  Unit u = unit_at(a, c, pos);
  if (one) {
    const int first = (int)quotient(u.start, c.each) + 1;
    const int cuts = u.start == pos ? 0 : (int)quotient(u.start + u.keys - 1, c.each) - first + 1;
    a.joints[w] = {u.w.rows.row0, u.w.rows.n, u.tile, u.minor, first, cuts, 0};
  }
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

}  // namespace
}  // namespace nvfp4
