// Attention over the cache (nvfp4_attn.h): the layout of a call, and the joining of parts.
#include "nvfp4_attn.h"

#include <cmath>

namespace nvfp4 {
namespace {

// A unit that is cut `cuts` times has cuts + 1 parts: the end of one range, whole
// ranges, and the beginning of the last.  Its rows are joined by the workgroups
// of its cuts (blockIdx.x + 1 is the range that begins there and has said so; blockIdx.y shares
// the rows out further).  kD / 4 lanes share a row's values.  With few parts each
// such group of lanes joins a row of its own, else the groups share a row's parts.
// (With one workgroup per row and cut, most of which found nothing to do, joining took as long as
// the attention itself: 10.6 us of 24 for one request, 33 of 130 for 16 trees.  Finding the cut units
// from the lengths once more, as the attention does, 8 us of 92 for 600 tokens behind 200.)
template <int kD>
__global__ __launch_bounds__(256) void attn_join_kernel(Attn a, int rows) {
  constexpr int kLanes = kD / 4, kGroups = 256 / kLanes, kFewParts = 16;
  const int w = blockIdx.x + 1;
  const Joint u = a.joints[w];
  if (u.cuts == 0) return;
  const int first = u.first, cuts = u.cuts;
  const int share = (w - first) * gridDim.y + blockIdx.y, shares = cuts * gridDim.y;
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int64_t size = (int64_t)rows * (kD + kPartMore);
  const float* parts = a.part + (2 * (int64_t)first - 1) * size;  // of the range before: slot 2 (first - 1) + 1
  const auto part = [&](int i) { return parts + (i == 0 ? 0 : 2 * i - 1) * size; };
  const float v_gs = *a.c.v_gs;
  const auto put = [&](const RowOf& r, const floatx4_t& o, float l) {
    const float f = l == 0.0f ? 0.0f : v_gs / l;  // a row that sees nothing is zeros
    u32x2_t b;
    b[0] = pack_bf16(o[0] * f, o[1] * f);
    b[1] = pack_bf16(o[2] * f, o[3] * f);
    *reinterpret_cast<u32x2_t*>(a.o + (u.row0 + r.token) * a.ldo + (int64_t)r.head * kD + 4 * lane) = b;
  };
  // Parts first, first + by, ... of row rho, under their own maximum.
  const auto join = [&](int rho, int from, int by, float& m, float& l, floatx4_t& o) {
    m = -INFINITY;
    l = 0.0f;
    o = floatx4_t{0, 0, 0, 0};
    const int more = rows * kD + kPartMore * rho;
#pragma unroll 4
    for (int i = from; i <= cuts; i += by) m = fmaxf(m, part(i)[more]);
#pragma unroll 4
    for (int i = from; i <= cuts; i += by) {
      const float* p = part(i);
      const float f = rescale(p[more], m, p[more + 2]);
      l += p[more + 1] * f;
      o += *reinterpret_cast<const floatx4_t*>(p + rho * kD + 4 * lane) * f;
    }
  };
  float m, l;
  floatx4_t o;
  if (cuts < kFewParts) {
    for (int rho = share * kGroups + grp; rho < rows; rho += shares * kGroups) {
      const RowOf r = row_of(a, u.tile, u.minor, u.n, rows, rho);
      if (r.token < 0) continue;
      join(rho, 0, 1, m, l, o);
      put(r, o, l);
    }
    return;
  }
  __shared__ float ml[2][kGroups];
  __shared__ floatx4_t sums[256];
  for (int rho = share; rho < rows; rho += shares) {
    const RowOf r = row_of(a, u.tile, u.minor, u.n, rows, rho);
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
      const float c1 = part(0)[rows * kD + kPartMore * rho + 2];
      l = 0.0f;
      o = floatx4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float f = rescale(ml[0][i], m, c1);
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
  bool split, solo;
  int rows, least, start, ranges;
};

Plan plan_of(int64_t T, int n_seqs, int hk, int group, int d) {
  // Two workgroups on a CU where their registers allow it, so that one multiplies while the other waits or evaluates
  // its softmax.  One -> two, us: seven chunks of 1100 rows behind 6000, d 128, 2360 -> 2045 (NVFP4), 2228 -> 1990 (E4M3);
  // d 64, 2015 -> 1473, 1621 -> 1259; 64 tokens behind 8200, d 128, 84.0 -> 74.3, 108.1 -> 103.5; trees of 5, d 128,
  // 55 -> 42; two tokens behind 131072, E4M3, d 128, 105.2 -> 106.6, the only one that lost.
  const int ranges = d < 256 ? 2 * kCus : kCus;
  const int64_t rows = (T * group + n_seqs - 1) / n_seqs;
  if (rows <= 32) {
    const int nt = rows <= 16 ? 1 : 2;
    // A range for every wave, where there are units enough (a quarter as many with 32 rows, whose sums are joined for
    // longer).  Workgroups -> waves, us, E4M3, 24/4 heads of 256: 64 tokens behind 100, 27.8 -> 28.0, behind 1000,
    // 51.3 -> 35.6, behind 3000, 101.5 -> 85.9, behind 8200, 196.0 -> 194.7; 600 behind 200, 131 -> 85; 16 trees of 5
    // (32 rows) behind 4100, 73.5 -> 54.1.  Behind 500 these lose, 31.7 -> 43.5, but the host does not know the lengths.
    // Fewer units lose, or gain little: 16 tokens behind 1000, 23.5 -> 28.4, one, 18.1 -> 24.9, 32, 34.8 -> 32.9.
    const bool solo = (int64_t)n_seqs * hk * (nt == 1 ? 1 : 4) >= ranges;
    return {nt, true, solo, 16 * nt, 256, solo ? 192 : 256, solo ? 4 * ranges : ranges};
  }
  return {2, false, false, 128, 256, 512, ranges};
}

size_t part_bytes(const Plan& p, int d) { return (size_t)2 * p.ranges * p.rows * (d + kPartMore) * sizeof(float); }

Attn attn_of(const Plan& p, const KvCache& c, const KvRows& r, const void* q, int64_t ldq, int group, float scale,
             const uint64_t* tree, void* o, int64_t ldo, void* workspace) {
  int power;
  const float mantissa = std::frexp(scale, &power) * 1.44269504088896340736f;
  return {c,      r,       static_cast<const uint16_t*>(q), ldq, group, mantissa, power, tree,
          static_cast<uint16_t*>(o), ldo, static_cast<float*>(workspace),
          reinterpret_cast<Joint*>(static_cast<char*>(workspace) + part_bytes(p, c.d)), p.least, p.start, p.ranges,
          group <= p.rows ? p.rows / group : 1, group <= p.rows ? 1 : (group + p.rows - 1) / p.rows};
}

}  // namespace

size_t attn_cached_workspace_bytes(int64_t T, int n_seqs, int hq, int hk, int d) {
  const Plan p = plan_of(T, n_seqs, hk, hq / hk, d);
  return part_bytes(p, d) + p.ranges * sizeof(Joint);
}

hipError_t launch_attn_cached(const KvCache& c, const KvRows& r, const void* q, int64_t ldq, int hq, float scale,
                              const uint64_t* tree, void* o, int64_t ldo, void* workspace, hipStream_t stream) {
  const int group = hq / c.hk;
  const Plan p = plan_of(r.T, r.n_seqs, c.hk, group, c.d);
  const Attn a = attn_of(p, c, r, q, ldq, group, scale, tree, o, ldo, workspace);
  if (p.split)
    launch_attn_few(a, p.nt, p.solo, stream);
  else
    launch_attn_many(a, stream);
  const auto join = c.d == 64 ? attn_join_kernel<64> : c.d == 128 ? attn_join_kernel<128> : attn_join_kernel<256>;
  join<<<dim3(p.ranges - 1, p.split ? 2 * p.nt : 8), 256, 0, stream>>>(a, p.rows);
  return hipGetLastError();
}

}  // namespace nvfp4
