// Short causal convolution per channel, with SiLU, over packed sequences or
// one row for each of many requests:
//
//   y_t = silu(sum_{i < W} w[c][i] x_{t - W + 1 + i}),  silu(v) = v / (1 + exp(-v))
//
// where the rows before a sequence's first are the last W - 1 inputs of its
// request, kept oldest first in a slot of the state pool (zeros without a
// pool), and the slot gets the sequence's own last W - 1 inputs.  Sums are
// fp32 in tap order; x, y and the pool are bf16 or fp32.
//
// HBM-bound (2 values moved for 2 W + 4 flops).  Packed form: a lane owns
// kVec neighbouring channels and walks kRows rows with the last W - 1 inputs
// in registers, so a row is read once but for the W - 1 rows above a tile.
// The tile that holds a sequence's first row also takes every row whose
// window reaches into the pool's slot (W - 1 rows, also past the tile's end)
// and updates the slot: one thread reads and writes each value of it.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

// Vectors at any element's address: the memory path takes them.
typedef u32x4_t u32x4_at2 __attribute__((aligned(2)));
typedef floatx4_t floatx4_at4 __attribute__((aligned(4)));

// kVec neighbouring channels of a row: one, or 16 bytes (8 bf16, 4 fp32).
template <bool kBf16, int kVec>
struct Row {
  float v[kVec];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (kVec == 1) {
      if constexpr (kBf16)
        v[0] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[at] << 16);
      else
        v[0] = reinterpret_cast<const float*>(base)[at];
    } else if constexpr (kBf16) {
      const u32x4_t a = *reinterpret_cast<const u32x4_at2*>(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    } else {
      const floatx4_t a = *reinterpret_cast<const floatx4_at4*>(reinterpret_cast<const float*>(base) + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a[e];
    }
  }
  static __device__ __forceinline__ void store_one(void* base, int64_t at, float x) {
    if constexpr (kBf16)
      reinterpret_cast<uint16_t*>(base)[at] = (uint16_t)pack_bf16(x, 0.0f);
    else
      reinterpret_cast<float*>(base)[at] = x;
  }
  // all but the first `before`
  __device__ __forceinline__ void store(void* base, int64_t at, int before) const {
    if constexpr (kVec == 1) {
      store_one(base, at, v[0]);
    } else if (before) {
#pragma unroll
      for (int e = 1; e < kVec; ++e)
        if (e >= before) store_one(base, at + e, v[e]);
    } else if constexpr (kBf16) {
      u32x4_t a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      __builtin_nontemporal_store(a, reinterpret_cast<u32x4_at2*>(reinterpret_cast<uint16_t*>(base) + at));
    } else {
      floatx4_t a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = v[e];
      __builtin_nontemporal_store(a, reinterpret_cast<floatx4_at4*>(reinterpret_cast<float*>(base) + at));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = 0.0f;
  }
};

// y of one row from its window (win[W - 1] is the row itself).
template <bool kBf16, int kVec, int kW>
__device__ __forceinline__ Row<kBf16, kVec> conv_row(const Row<kBf16, kVec> (&win)[kW], const float (&w)[kVec][kW]) {
  Row<kBf16, kVec> y;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kW; ++i) s = fmaf(w[e][i], win[i].v[e], s);
    y.v[e] = silu(s);
  }
  return y;
}

template <int kVec, int kW>
__device__ __forceinline__ void load_weights(const float* w, int64_t c, float (&out)[kVec][kW]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e)
#pragma unroll
    for (int i = 0; i < kW; ++i) out[e][i] = w[(c + e) * kW + i];
}

constexpr int kConvThreads = 256;
// Where less than kVec channels are left, a lane takes the last kVec of the
// row and leaves the first `before` to the lane before it (it loads them, also
// from a slot that that lane is writing, and stores nothing of them): 9,000
// rows of 4,895 bf16 take 39 us, 55 with a channel per lane.
// Rows per tile and rows loaded at once.  On 32768 x 8192 bf16: 209 us (5.1
// TB/s, a plain copy of that size reads and writes 4.9-5.0), against 222-227
// with 64 rows, 232 with 8, and 298 / 219 with 128 / 512 threads.  fp32: 407 us
// (5.3 TB/s) with 16 bytes a lane, 505-765 with 32.
constexpr int kRows = 16, kAhead = 8;

// Tiles along x of a grid: a launch takes less than 2^32 threads along one
// dimension, so those of 2^26 rows and more go on along z.
constexpr int64_t kTilesX = (int64_t)1 << 22;

// Packed sequences: grid (tiles of kRows rows, channel blocks, kTilesX tiles).
template <bool kBf16, int kVec, int kW>
__global__ __launch_bounds__(kConvThreads) void conv_silu_kernel(
    const void* __restrict__ x, int64_t ldx, int64_t channels, const float* __restrict__ w, const int32_t* __restrict__ cu,
    int n_seqs, int64_t T, void* state, const int32_t* __restrict__ slots, int n_slots, void* __restrict__ y,
    int64_t ldy) {
  using R = Row<kBf16, kVec>;
  const int64_t t0 = (blockIdx.z * kTilesX + blockIdx.x) * kRows;
  if (t0 >= T) return;
  const int64_t t1 = min(t0 + kRows, T);
  // the last sequence that starts at or before t0 (cut off or not): no earlier one has a row in the tile
  const int first = last_before(n_seqs, [&](int i) { return cu[i] <= t0; });
  const int64_t mine0 = ((int64_t)blockIdx.y * kConvThreads + threadIdx.x) * kVec;
  if (mine0 >= channels) return;
  const int64_t c = min(mine0, channels - kVec);
  const int before = (int)(mine0 - c);
  float wt[kVec][kW];
  load_weights<kVec, kW>(w, c, wt);

  for (int s = first; s < n_seqs; ++s) {
    const int64_t start = row_clip(cu[s], T), end = row_clip(cu[s + 1], T);
    if (start >= t1) break;
    if (end <= start) continue;
    const bool mine = start >= t0;  // this tile holds the first row
    int64_t t = mine ? start : max(t0, min(start + kW - 1, end));
    const int64_t stop = mine ? min(end, max(t1, start + kW - 1)) : min(end, t1);
    if (t >= stop) continue;
    const int slot = state ? (slots ? slots[s] : s) : 0;
    if (slot < 0 || slot >= n_slots) {  // a skipped sequence: zeros
      R z;
      z.zero();
      for (; t < stop; ++t) z.store(y, t * ldy + c, before);
      continue;
    }
    R win[kW];
    if (mine) {
      R old[kW - 1];
#pragma unroll
      for (int i = 0; i < kW - 1; ++i) {
        if (state) old[i].load(state, ((int64_t)slot * (kW - 1) + i) * channels + c); else old[i].zero();
        win[i] = old[i];
      }
      if (state) {  // the last W - 1 inputs of [old; this sequence]
        const int64_t len = end - start;
#pragma unroll
        for (int i = 0; i < kW - 1; ++i) {
          const int64_t r = len - (kW - 1) + i;
          R nw;
          if (r >= 0) {
            nw.load(x, (start + r) * ldx + c);
          } else {
            nw = old[0];
#pragma unroll
            for (int j = 1; j < kW - 1; ++j)
              if (j == len + i) nw = old[j];
          }
          nw.store(state, ((int64_t)slot * (kW - 1) + i) * channels + c, before);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kW - 1; ++i) win[i].load(x, (t - (kW - 1) + i) * ldx + c);
    }
    auto row = [&](const R& next, int64_t at) {
      win[kW - 1] = next;
      conv_row<kBf16, kVec, kW>(win, wt).store(y, at * ldy + c, before);
#pragma unroll
      for (int i = 0; i < kW - 1; ++i) win[i] = win[i + 1];
    };
    for (; t + kAhead <= stop; t += kAhead) {
      R next[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) next[j].load(x, (t + j) * ldx + c);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) row(next[j], t + j);
    }
    for (; t < stop; ++t) {
      R next;
      next.load(x, t * ldx + c);
      row(next, t);
    }
  }
}

// One row for each request: grid (requests, channel blocks).
template <bool kBf16, int kVec, int kW>
__global__ __launch_bounds__(kConvThreads) void conv_silu_step_kernel(
    const void* __restrict__ x, int64_t ldx, int64_t channels, const float* __restrict__ w, void* state,
    const int32_t* __restrict__ slots, int n_slots, void* __restrict__ y, int64_t ldy) {
  using R = Row<kBf16, kVec>;
  const int64_t mine0 = ((int64_t)blockIdx.y * kConvThreads + threadIdx.x) * kVec;
  if (mine0 >= channels) return;
  const int64_t c = min(mine0, channels - kVec);
  const int before = (int)(mine0 - c);
  const int64_t b = blockIdx.x;
  const int slot = state ? (slots ? slots[b] : (int)b) : 0;
  if (slot < 0 || slot >= n_slots) {
    R z;
    z.zero();
    z.store(y, b * ldy + c, before);
    return;
  }
  float wt[kVec][kW];
  load_weights<kVec, kW>(w, c, wt);
  R win[kW];
  win[kW - 1].load(x, b * ldx + c);
#pragma unroll
  for (int i = 0; i < kW - 1; ++i) {
    if (state) win[i].load(state, ((int64_t)slot * (kW - 1) + i) * channels + c); else win[i].zero();
  }
  conv_row<kBf16, kVec, kW>(win, wt).store(y, b * ldy + c, before);
  if (state) {
#pragma unroll
    for (int i = 0; i < kW - 1; ++i) win[i + 1].store(state, ((int64_t)slot * (kW - 1) + i) * channels + c, before);
  }
}

template <bool kBf16, int kVec, int kW>
hipError_t launch_conv_typed(const void* x, int64_t ldx, int64_t channels, const float* w, const int32_t* cu,
                             int n_seqs, int64_t T, void* state, const int32_t* slots, int n_slots, void* y,
                             int64_t ldy, hipStream_t stream) {
  const unsigned blocks = (unsigned)((channels + kConvThreads * kVec - 1) / (kConvThreads * kVec));
  if (cu) {
    const int64_t tiles = (T + kRows - 1) / kRows;
    const dim3 grid((unsigned)(tiles < kTilesX ? tiles : kTilesX), blocks, (unsigned)((tiles + kTilesX - 1) / kTilesX));
    conv_silu_kernel<kBf16, kVec, kW><<<grid, kConvThreads, 0, stream>>>(x, ldx, channels, w, cu, n_seqs, T, state,
                                                                         slots, n_slots, y, ldy);
  } else {
    const dim3 grid((unsigned)T, blocks);
    conv_silu_step_kernel<kBf16, kVec, kW><<<grid, kConvThreads, 0, stream>>>(x, ldx, channels, w, state, slots,
                                                                              n_slots, y, ldy);
  }
  return hipGetLastError();
}

template <bool kBf16, int kVec>
hipError_t launch_conv_width(int width, const void* x, int64_t ldx, int64_t channels, const float* w,
                             const int32_t* cu, int n_seqs, int64_t T, void* state, const int32_t* slots,
                             int n_slots, void* y, int64_t ldy, hipStream_t stream) {
  const auto f = width == 2   ? launch_conv_typed<kBf16, kVec, 2>
                 : width == 3 ? launch_conv_typed<kBf16, kVec, 3>
                              : launch_conv_typed<kBf16, kVec, 4>;
  return f(x, ldx, channels, w, cu, n_seqs, T, state, slots, n_slots, y, ldy, stream);
}

}  // namespace

hipError_t launch_conv_silu(const void* x, bool bf16, int64_t ldx, int64_t channels, const float* w, int width,
                            const int32_t* cu, int n_seqs, int64_t T, void* state, const int32_t* slots, int n_slots,
                            void* y, int64_t ldy, hipStream_t stream) {
  const auto f = bf16 ? (channels >= 8 ? launch_conv_width<true, 8> : launch_conv_width<true, 1>)
                      : (channels >= 4 ? launch_conv_width<false, 4> : launch_conv_width<false, 1>);
  return f(width, x, ldx, channels, w, cu, n_seqs, T, state, slots, n_slots, y, ldy, stream);
}

}  // namespace nvfp4
