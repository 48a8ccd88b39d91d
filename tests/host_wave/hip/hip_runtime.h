// What the kernels take from HIP and from gfx950, for a build of their sources
// by a host compiler: the lanes of a workgroup are run in turn, each on a stack of
// its own, up to the next place where the wave's lanes exchange values or the
// workgroup's waves wait for each other.  Every array of a call ends at an
// unmapped page, so an access out of bounds ends the call with its address.
//
// Not shown by such a run: races (one order of the lanes is taken), registers,
// what the compiler makes of the source for the GPU, and shared arrays' own bounds.
#pragma once

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#define __device__
#define __host__
#define __global__
#define __shared__ static
#define __forceinline__ inline
#define __launch_bounds__(...)

typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};

namespace host {

constexpr int kMost = 1024, kStack = 128 << 10;
enum State { kRuns, kAtWave, kAtBarrier, kDone };
struct Lane {
  void* sp;
  State state;
};
extern Lane lanes[kMost];
extern int lane_now;                  // of the workgroup
extern uint64_t slot[3][kMost];       // what the lanes give at this exchange and at the next
extern uint64_t given[3][kMost / 64]; // which lanes of a wave gave something
extern int turn[kMost];               // exchanges of a lane so far, modulo 3
void wait(State s);                   // back when the others have come here too
void launch(dim3 grid, dim3 block, void (*body)(void*), void* args);

// A lane's value to the wave; then each lane may look at any other's.
struct Wave {
  const uint64_t* of;
  uint64_t who;
};
inline Wave exchange(uint64_t v) {
  const int t = turn[lane_now], wave = lane_now / 64;
  turn[lane_now] = (t + 1) % 3;
  slot[t][lane_now] = v;
  given[t][wave] |= 1ull << (lane_now % 64);
  wait(kAtWave);
  given[(t + 2) % 3][wave] = 0;  // of the exchange before, which all have left
  return {slot[t] + 64 * wave, given[t][wave]};
}

template <class T>
uint64_t bits(T v) {
  uint64_t b = 0;
  memcpy(&b, &v, sizeof v);
  return b;
}
template <class T>
T value(uint64_t b) {
  T v;
  memcpy(&v, &b, sizeof v);
  return v;
}
template <class T>
T shuffle(T v, int from) {
  const Wave w = exchange(bits(v));
  if (!(w.who >> (from & 63) & 1)) fprintf(stderr, "host_wave: a value of a lane that is not there\n"), abort();
  return value<T>(w.of[from & 63]);
}

inline float e4m3(uint32_t b) {
  const int e = b >> 3 & 15, m = b & 7;
  const float v = (b & 127) == 127 ? NAN : e ? ldexpf(1.0f + m / 8.0f, e - 7) : ldexpf((float)m, -9);
  return b & 128 ? -v : v;
}
inline float e2m1(uint32_t c) {
  constexpr float v[8] = {0, 0.5f, 1, 1.5f, 2, 3, 4, 6};
  return c & 8 ? -v[c & 7] : v[c & 7];
}
// The code of the nearest of n values, ties to the even code (values past the last: the last, or `past`).
template <class F>
uint32_t nearest(float v, uint32_t n, F of, uint32_t sign) {
  const float a = fabsf(v);
  uint32_t c = 0;
  while (c + 1 < n && of(c + 1) <= a) ++c;
  if (c + 1 < n && (a - of(c) > of(c + 1) - a || (a - of(c) == of(c + 1) - a && c % 2))) ++c;
  return c | (signbit(v) ? sign : 0);
}
inline uint32_t to_e4m3(float v) { return fabsf(v) <= 464.0f ? nearest(v, 127, e4m3, 128) : 127; }
inline uint32_t to_e2m1(float v) { return nearest(v, 8, e2m1, 8); }

}  // namespace host

#define HOST_INDEX(NAME)                 \
  struct NAME##_t {                      \
    unsigned x, y, z;                    \
  };                                     \
  extern NAME##_t NAME;
HOST_INDEX(threadIdx)
HOST_INDEX(blockIdx)
HOST_INDEX(blockDim)
HOST_INDEX(gridDim)

template <class... P, class... A>
void host_launch(void (*kernel)(P...), dim3 grid, dim3 block, A... args) {
  auto run = [&] { kernel(args...); };
  host::launch(grid, block, [](void* p) { (*static_cast<decltype(run)*>(p))(); }, &run);
}

inline int min(int a, int b) { return a < b ? a : b; }
inline int max(int a, int b) { return a > b ? a : b; }
inline uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
inline int64_t min(int64_t a, int64_t b) { return a < b ? a : b; }
inline int64_t max(int64_t a, int64_t b) { return a > b ? a : b; }

inline void __syncthreads() { host::wait(host::kAtBarrier); }
inline uint32_t __float_as_uint(float v) { return (uint32_t)host::bits(v); }
inline float __uint_as_float(uint32_t v) { return host::value<float>(v); }
template <class T>
T __shfl(T v, int from, int = 64) {
  return host::shuffle(v, from);
}
template <class T>
T __shfl_xor(T v, int m, int = 64) {
  return host::shuffle(v, (host::lane_now & 63) ^ m);
}
template <class T>
T __shfl_up(T v, int m, int = 64) {
  const int l = host::lane_now & 63;
  return host::shuffle(v, l >= m ? l - m : l);
}

namespace host {
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
struct Two {
  uint32_t v[2];
  uint32_t operator[](int i) const { return v[i]; }
};
inline uint64_t ballot(bool b) {
  const Wave w = exchange(b);
  uint64_t r = 0;
  for (int i = 0; i < 64; ++i) r |= (w.who >> i & 1 && w.of[i] ? 1ull : 0) << i;
  return r;
}
inline int first_lane(int v) {
  const Wave w = exchange((uint32_t)v);
  return (int)w.of[__builtin_ctzll(w.who)];
}
// The lanes' rows of `width`: the odd ones of a and the even ones of b change places.
inline Two swap_rows(uint32_t a, uint32_t b, int width) {
  const Wave w = exchange((uint64_t)b << 32 | a);
  const int l = lane_now & 63;
  if (l / width % 2) return {{(uint32_t)(w.of[l - width] >> 32), b}};
  return {{a, (uint32_t)w.of[l + width]}};
}
// D = A B + C: lane (n, g) has row (column) n of A (B), 8 g .. 8 g + 7 of what is summed over, and column n, rows 4 g .. of D.
inline f4 mfma_16x16x32(const h8& a, const h8& b, f4 c) {
  uint64_t part[4];
  h8 at[64][2];
  for (int half = 0; half < 2; ++half) {
    memcpy(part, &a, 16);
    memcpy(part + 2, &b, 16);
    const uint64_t first = half == 0 ? part[0] : part[1], second = half == 0 ? part[2] : part[3];
    const Wave w = exchange(first);
    for (int i = 0; i < 64; ++i) memcpy(reinterpret_cast<char*>(&at[i][0]) + 8 * half, w.of + i, 8);
    const Wave x = exchange(second);
    for (int i = 0; i < 64; ++i) memcpy(reinterpret_cast<char*>(&at[i][1]) + 8 * half, x.of + i, 8);
  }
  const int n = lane_now & 15, g = (lane_now & 63) >> 4;
  for (int r = 0; r < 4; ++r) {
    float s = c[r];
    for (int k = 0; k < 32; ++k) s += (float)at[4 * g + r + 16 * (k / 8)][0][k % 8] * (float)at[n + 16 * (k / 8)][1][k % 8];
    c[r] = s;
  }
  return c;
}
inline h2 two_fp8(int w, float scale, bool high) {
  const uint32_t b = (uint32_t)w >> (high ? 16 : 0);
  return h2{(_Float16)(e4m3(b & 255) * scale), (_Float16)(e4m3(b >> 8 & 255) * scale)};
}
inline h2 two_fp4(uint32_t w, float scale, int byte) {
  const uint32_t b = w >> (8 * byte);
  return h2{(_Float16)(e2m1(b & 15) * scale), (_Float16)(e2m1(b >> 4 & 15) * scale)};
}
inline f2 two_f32_fp8(int w, bool high) {
  const uint32_t b = (uint32_t)w >> (high ? 16 : 0);
  return f2{e4m3(b & 255), e4m3(b >> 8 & 255)};
}
inline f2 two_f32_fp4(uint32_t w, float scale, int byte) {
  const uint32_t b = w >> (8 * byte);
  return f2{e2m1(b & 15) * scale, e2m1(b >> 4 & 15) * scale};
}
inline int two_to_fp8(float a, float b, int old, bool high) {
  const uint32_t v = to_e4m3(a) | to_e4m3(b) << 8;
  return (int)(high ? ((uint32_t)old & 0xFFFFu) | v << 16 : ((uint32_t)old & 0xFFFF0000u) | v);
}
inline uint32_t two_to_fp4(uint32_t old, float a, float b, float scale, int byte) {
  const uint32_t v = to_e2m1(a / scale) | to_e2m1(b / scale) << 4;
  return (old & ~(255u << (8 * byte))) | v << (8 * byte);
}
inline uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  const uint64_t all = (uint64_t)hi << 32 | lo;
  uint32_t r = 0;
  for (int i = 0; i < 4; ++i) r |= (uint32_t)(all >> (8 * (sel >> (8 * i) & 7)) & 255) << (8 * i);
  return r;
}
}  // namespace host

#define __builtin_amdgcn_exp2f exp2f
#define __builtin_amdgcn_rcpf(x) (1.0f / (x))
#define __builtin_amdgcn_ballot_w64 host::ballot
#define __builtin_amdgcn_readfirstlane host::first_lane
#define __builtin_amdgcn_permlane32_swap(a, b, x, y) host::swap_rows(a, b, 32)
#define __builtin_amdgcn_permlane16_swap(a, b, x, y) host::swap_rows(a, b, 16)
#define __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, x, y, z) host::mfma_16x16x32(a, b, c)
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 host::two_fp8
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp4 host::two_fp4
#define __builtin_amdgcn_cvt_f32_fp8(w, byte) host::e4m3((uint32_t)(w) >> (8 * (byte)) & 255)
#define __builtin_amdgcn_cvt_pk_fp8_f32 host::two_to_fp8
#define __builtin_amdgcn_cvt_pk_f32_fp8 host::two_f32_fp8
#define __builtin_amdgcn_cvt_scalef32_pk_f32_fp4 host::two_f32_fp4
#define __builtin_amdgcn_cvt_scalef32_pk_fp4_f32 host::two_to_fp4
#define __builtin_amdgcn_perm host::perm
#define __builtin_amdgcn_sched_barrier(x)
