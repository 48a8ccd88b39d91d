// What the kernels of the paged, quantised key/value cache share: where the
// rows of packed sequences stand, and where a position lies in the cache.
//
// Row j of sequence i (n rows of the packed rows) stands at position
// kv_lens[i] - n + j.  Position p lies in page table[i][p / page], row
// p % page.  A page holds, per key/value head, K as [row][dim] and V as
// [dim][row]: a lane of the attention's matrix instructions takes 8 or 16
// neighbouring dims of one key, and 16 neighbouring keys of one dim of V, so in
// both a lane's operand is 16 bytes that it loads straight into registers.
//   E4M3:   one byte per value, value = code * gs
//   NVFP4:  a byte holds the codes of dims 2 b (low nibble) and 2 b + 1 of one
//           key, value = E2M1(code) * E4M3(scale) * gs, one scale byte per 16
//           dims of a key: K scales [row][dim / 16], V codes [dim / 2][row],
//           V scales [dim / 16][row]
// A token's bytes are its own in every array, so tokens are written one by one.
#pragma once

#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

// One sequence's rows: its packed rows [row0, row0 + n) and its length.
struct SeqRows {
  int64_t row0;
  int n;
  int kv;
};

__device__ __forceinline__ SeqRows seq_rows(const KvRows& r, int i) {
  if (!r.cu) return {i, 1, r.kv_lens[i]};
  const int64_t a = row_clip(r.cu[i], r.T), b = row_clip(r.cu[i + 1], r.T);
  return {a, (int)max(b - a, (int64_t)0), r.kv_lens[i]};
}

// The page of a position, or -1 where there is none.
__device__ __forceinline__ int page_of(const KvRows& r, const KvCache& c, int i, int64_t pos) {
  const int64_t slot = pos >> c.page_shift;
  if (pos < 0 || slot >= r.max_pages) return -1;
  const int p = r.table[(int64_t)i * r.ld_table + slot];
  return (unsigned)p < (unsigned)c.n_pages ? p : -1;
}

// Bytes of a head's row of codes, and of its scales (0 in E4M3).
template <bool kFp4>
__host__ __device__ constexpr int code_bytes(int d) {
  return kFp4 ? d / 2 : d;
}

}  // namespace
}  // namespace nvfp4
