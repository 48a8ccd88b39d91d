// Rows of keys and values into a paged, quantised cache, and back out of it
// (layout: nvfp4_kv.h).
//
//   E4M3   code = E4M3 round-to-nearest-even of x / gs, exact real quotient,
//          saturated at 448
//   NVFP4  nvfp4_quantize's block of 16 dims under the tensor scale gs
//
// Both are HBM-bound.  A workgroup takes 16 neighbouring positions of one
// sequence that lie in one page, of one head and of K or V; a thread takes 16
// dims of one position (a whole NVFP4 block).  K goes straight to its place, 8
// or 16 bytes a thread.  V is turned over in LDS, so that where all 16 positions
// are the call's, 16 bytes go out at once; at the ends of a sequence's rows, and
// for single tokens, only the bytes of its own positions are written.
// Measured, 32768 rows of 4 heads of 256, bf16: write NVFP4 47 us (172 MB at 3.7
// TB/s; the exact rounding keeps vector instructions busy for 64% of the cycles, LDS
// 27%), E4M3 56 us (201 MB at 3.6 TB/s; 50%, LDS 44%: the byte stores that turn v over
// meet in one bank); read NVFP4 32 us (5.3 TB/s, a large copy's rate).
#include "nvfp4_kv.h"
#include "nvfp4_quant_block.h"

namespace nvfp4 {
namespace {

template <bool kBf16>
__device__ __forceinline__ void load16(const void* base, int64_t at, float v[16]) {
  if constexpr (kBf16) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t a = p[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] = __uint_as_float(a[i] << 16);
        v[8 * h + 2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    }
  } else {
    const floatx4_t* p = reinterpret_cast<const floatx4_t*>(reinterpret_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx4_t t = p[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = t[e];
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void store16(void* base, int64_t at, const float v[16]) {
  if constexpr (kBf16) {
    u32x4_t* p = reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
      p[h] = a;
    }
  } else {
    floatx4_t* p = reinterpret_cast<floatx4_t*>(reinterpret_cast<float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      floatx4_t t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = v[4 * i + e];
      p[i] = t;
    }
  }
}

// A value that the E4M3 converter rounds as the exact quotient x / g (r an
// approximate 1 / g).  E4M3's decision points have at most 4 fraction bits, so
// between two neighbouring values m of that kind the code is constant; the
// approximate quotient rounded to 4 fraction bits is one of the two around the
// exact one, and fma(|m|, g, -|x|), the exact difference rounded once, says on
// which side of it that lies.  m moved by 2^-7 of itself to that side stays
// inside the interval; on m itself the converter's tie to even is right.  Past
// 448 the moved value is 451.5, which still rounds to 448.
__device__ __forceinline__ float settle_e4m3(float x, float g, float r) {
  const float y = fminf(fmaxf(x * r, -kE4M3Max), kE4M3Max);
  const float m = __uint_as_float((__float_as_uint(y) + 0x40000u) & 0xFFF80000u);
  const float d = fmaf(fabsf(m), g, -fabsf(x));
  return m * (d > 0.0f ? 1.0f - 0x1p-7f : d < 0.0f ? 1.0f + 0x1p-7f : 1.0f);
}

__device__ __forceinline__ bool all_finite(const float v[16]) {
  bool ok = true;
#pragma unroll
  for (int e = 0; e < 16; ++e) ok = ok && fabsf(v[e]) < INFINITY;
  return ok;
}

// 16 codes of E4M3: finite values saturate, what is not finite becomes NaN.
__device__ __forceinline__ u32x4_t encode_e4m3(const float v[16], float g) {
  const float r = __builtin_amdgcn_rcpf(g);
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(settle_e4m3(v[4 * i], g, r), settle_e4m3(v[4 * i + 1], g, r), 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(settle_e4m3(v[4 * i + 2], g, r), settle_e4m3(v[4 * i + 3], g, r), c, true);
    w[i] = (uint32_t)c;
  }
  if (!all_finite(v)) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (!(fabsf(v[e]) < INFINITY)) w[e / 4] = (w[e / 4] & ~(0xFFu << (e % 4 * 8))) | 0x7Fu << (e % 4 * 8);
  }
  return w;
}

// The block of 16 positions that a workgroup takes: sequence i's rows stand at
// positions kv - n .. kv - 1, in at most n / 16 + 2 blocks of 16.  With places
// cu[i] / 16 + 2 i for the first of them no two sequences' blocks meet, and
// the sequence of a place is found by search, without a sum over the lengths.
// Without cu it is place i.
struct Place {
  int seq;
  int64_t pos0;        // the block's first position (a multiple of 16; may be negative)
  int64_t row0;        // packed row that would stand there
  int64_t lo, hi;      // the call's positions, cut to the block
};

__device__ __forceinline__ Place place_of(const KvRows& r, int b) {
  int i = b;
  int64_t first = b;
  if (r.cu) {
    const auto start = [&](int s) { return row_clip(r.cu[s], r.T) / 16 + 2 * (int64_t)s; };
    i = last_before(r.n_seqs, [&](int s) { return start(s) <= b; });
    first = start(i);
  }
  const SeqRows s = seq_rows(r, i);
  const int64_t p0 = (int64_t)s.kv - s.n;
  Place p;
  p.seq = i;
  p.pos0 = ((p0 >> 4) + (b - first)) * 16;
  p.row0 = s.row0 + (p.pos0 - p0);
  p.lo = max(p0, p.pos0);
  p.hi = min((int64_t)s.kv, p.pos0 + 16);  // lo >= hi: nothing
  return p;
}

// The place that workgroup x takes.  Workgroups go round the eight XCDs in turn; eight neighbouring places go to one of
// them, since up to eight (a page of 128 rows) share lines of V, which one L2 then puts together.
__device__ __forceinline__ int place_index() {
  const int x = blockIdx.x, base = x & ~63;
  return base + 64 <= (int)gridDim.x ? base + (x & 7) * 8 + (x >> 3 & 7) : x;
}

// Threads: kD, thread (j, l) = (t / (kD / 16), t % (kD / 16)): position j of
// the block, dims 16 l .. 16 l + 15.  blockIdx: block, head, K or V.
template <bool kFp4, bool kBf16, int kD>
__global__ __launch_bounds__(kD) void kv_write_kernel(KvCache c, KvRows r, const void* k, int64_t ldk, const void* v,
                                                      int64_t ldv) {
  constexpr int kL = kD / 16;
  const Place p = place_of(r, place_index());
  if (p.lo >= p.hi) return;
  const int h = blockIdx.y, t = threadIdx.x, j = t / kL, l = t % kL;
  const bool is_v = blockIdx.z, live = p.pos0 + j >= p.lo && p.pos0 + j < p.hi;
  float x[16];
  if (live) load16<kBf16>(is_v ? v : k, (p.row0 + j) * (is_v ? ldv : ldk) + h * kD + 16 * l, x);
  const int page = page_of(r, c, p.seq, p.pos0);  // while the row is on its way
  if (page < 0) return;  // before position 0 too
  const int ps = 1 << c.page_shift, row = (int)p.pos0 & (ps - 1);
  const int64_t unit = (int64_t)page * c.hk + h;  // (page, head)
  const float g = is_v ? *c.v_gs : *c.k_gs;
  u32x4_t w = {0, 0, 0, 0};
  uint32_t scale = 0;
  if (live) {
    if constexpr (kFp4) {
      uint32_t w0, w1;
      scale = quantize_block(x, g, __builtin_amdgcn_rcpf(6.0f * g), w0, w1);
      const bool ok = all_finite(x);
      w[0] = ok ? w0 : 0u;
      w[1] = ok ? w1 : 0u;
      scale = ok ? scale : 0x7Fu;  // the block reads as NaN
    } else {
      w = encode_e4m3(x, g);
    }
  }
  if (!is_v) {
    if (!live) return;
    uint8_t* to = c.k + (unit * ps + row + j) * code_bytes<kFp4>(kD);
    if constexpr (kFp4) {
      u32x2_t w2;
      w2[0] = w[0];
      w2[1] = w[1];
      reinterpret_cast<u32x2_t*>(to)[l] = w2;
      c.k_scales[(unit * ps + row + j) * kL + l] = (uint8_t)scale;
    } else {
      reinterpret_cast<u32x4_t*>(to)[l] = w;
    }
    return;
  }
  // V: lines of 16 positions, one per dim (pair of dims), then one per scale
  constexpr int kCodes = code_bytes<kFp4>(kD), kLines = kCodes + (kFp4 ? kL : 0), kPer = kCodes / kL;
  __shared__ u32x4_t lines[kLines];
  uint8_t* s = reinterpret_cast<uint8_t*>(lines);
#pragma unroll
  for (int e = 0; e < kPer; ++e) s[(kPer * l + e) * 16 + j] = (uint8_t)(w[e / 4] >> (e % 4 * 8));
  if constexpr (kFp4) s[(kCodes + l) * 16 + j] = (uint8_t)scale;
  __syncthreads();
  const bool whole = p.hi - p.lo == 16;
  for (int i = t; i < kLines; i += kD) {
    uint8_t* to = (i < kCodes ? c.v + (unit * kCodes + i) * ps : c.v_scales + (unit * kL + (i - kCodes)) * ps) + row;
    if (whole) {
      *reinterpret_cast<u32x4_t*>(to) = lines[i];
    } else {
      for (int e = (int)(p.lo - p.pos0); e < (int)(p.hi - p.pos0); ++e) to[e] = s[i * 16 + e];
    }
  }
}

template <bool kFp4>
__device__ __forceinline__ void decode16(const u32x4_t& w, uint32_t scale, float g, float v[16]) {
  if constexpr (kFp4) {
    const float sc = e4m3_to_f32(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0);
      const float2v_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
      const float2v_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2);
      const float2v_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[8 * i + e] = a[e] * sc * g;  // E2M1 * E4M3 is exact: one rounding
        v[8 * i + 2 + e] = b[e] * sc * g;
        v[8 * i + 4 + e] = c[e] * sc * g;
        v[8 * i + 6 + e] = d[e] * sc * g;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2v_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const float2v_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = a[0] * g;
      v[4 * i + 1] = a[1] * g;
      v[4 * i + 2] = b[0] * g;
      v[4 * i + 3] = b[1] * g;
    }
  }
}

// The same threads and blocks; rows without a page, or before position 0, are zeros.
template <bool kFp4, bool kBf16, int kD>
__global__ __launch_bounds__(kD) void kv_read_kernel(KvCache c, KvRows r, void* k, int64_t ldk, void* v, int64_t ldv) {
  constexpr int kL = kD / 16, kCodes = code_bytes<kFp4>(kD), kLines = kCodes + (kFp4 ? kL : 0), kPer = kCodes / kL;
  const Place p = place_of(r, place_index());
  if (p.lo >= p.hi) return;
  const int page = page_of(r, c, p.seq, p.pos0);
  const int h = blockIdx.y, t = threadIdx.x, j = t / kL, l = t % kL;
  const int ps = 1 << c.page_shift, row = (int)p.pos0 & (ps - 1);
  const int64_t unit = (int64_t)page * c.hk + h;
  const bool is_v = blockIdx.z, live = p.pos0 + j >= p.lo && p.pos0 + j < p.hi;
  const float g = is_v ? *c.v_gs : *c.k_gs;
  u32x4_t w = {0, 0, 0, 0};
  uint32_t scale = 0;
  if (is_v) {
    __shared__ u32x4_t lines[kLines];
    if (page >= 0) {
      for (int i = t; i < kLines; i += kD)
        lines[i] = *reinterpret_cast<const u32x4_t*>(
            (i < kCodes ? c.v + (unit * kCodes + i) * ps : c.v_scales + (unit * kL + (i - kCodes)) * ps) + row);
    }
    __syncthreads();
    if (!live) return;
    if (page >= 0) {
      const uint8_t* s = reinterpret_cast<const uint8_t*>(lines);
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[e / 4] |= (uint32_t)s[(kPer * l + e) * 16 + j] << (e % 4 * 8);
      if constexpr (kFp4) scale = s[(kCodes + l) * 16 + j];
    }
  } else {
    if (!live) return;
    if (page >= 0) {
      const uint8_t* from = c.k + (unit * ps + row + j) * kCodes;
      if constexpr (kFp4) {
        const u32x2_t w2 = reinterpret_cast<const u32x2_t*>(from)[l];
        w[0] = w2[0];
        w[1] = w2[1];
        scale = c.k_scales[(unit * ps + row + j) * kL + l];
      } else {
        w = reinterpret_cast<const u32x4_t*>(from)[l];
      }
    }
  }
  float x[16];
  decode16<kFp4>(w, scale, g, x);
  store16<kBf16>(is_v ? v : k, (p.row0 + j) * (is_v ? ldv : ldk) + h * kD + 16 * l, x);
}

dim3 places(const KvCache& c, const KvRows& r) {
  return dim3((unsigned)(r.cu ? r.T / 16 + 2 * (int64_t)r.n_seqs : r.n_seqs), (unsigned)c.hk, 2);
}

// kernel<fp4, bf16, d> for the cache's format and head size.
#define NVFP4_KV_LAUNCH(KERNEL, ...)                                                        \
  do {                                                                                      \
    const auto f64 = c.fp4 ? (bf16 ? KERNEL<true, true, 64> : KERNEL<true, false, 64>)      \
                           : (bf16 ? KERNEL<false, true, 64> : KERNEL<false, false, 64>);   \
    const auto f128 = c.fp4 ? (bf16 ? KERNEL<true, true, 128> : KERNEL<true, false, 128>)   \
                            : (bf16 ? KERNEL<false, true, 128> : KERNEL<false, false, 128>); \
    const auto f256 = c.fp4 ? (bf16 ? KERNEL<true, true, 256> : KERNEL<true, false, 256>)   \
                            : (bf16 ? KERNEL<false, true, 256> : KERNEL<false, false, 256>); \
    (c.d == 64 ? f64 : c.d == 128 ? f128 : f256)<<<places(c, r), c.d, 0, stream>>>(__VA_ARGS__); \
  } while (0)

}  // namespace

hipError_t launch_kv_cache_write(const KvCache& c, const KvRows& r, const void* k, int64_t ldk, const void* v,
                                 int64_t ldv, bool bf16, hipStream_t stream) {
  NVFP4_KV_LAUNCH(kv_write_kernel, c, r, k, ldk, v, ldv);
  return hipGetLastError();
}

hipError_t launch_kv_cache_read(const KvCache& c, const KvRows& r, void* k, int64_t ldk, void* v, int64_t ldv,
                                bool bf16, hipStream_t stream) {
  NVFP4_KV_LAUNCH(kv_read_kernel, c, r, k, ldk, v, ldv);
  return hipGetLastError();
}

}  // namespace nvfp4
