// Host-side launchers behind the C ABI.  Arguments are already validated by
// nvfp4_api.cpp; each launcher only enqueues kernels and returns the launch
// status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

hipError_t launch_quantize(const void* x, bool in_bf16, int64_t rows, int64_t cols, int64_t ldx,
                           uint8_t* codes, uint8_t* scales, float* global_scale, bool from_amax,
                           hipStream_t stream);

constexpr int kMaxModules = 64;

// Tensor scales of the weight's output columns.  Column range s (s = 0 ..
// n - 1) is [end[s - 1], end[s]) with end[-1] = 0 and end[n - 1] = N; its
// tensor scale is gs[s] (device).  A plain GEMM is the case n = 1.  Passed
// to the kernels by value (kernel arguments).
struct ColScales {
  const float* gs;
  int n;
  int end[kMaxModules];
  // Gated DeltaNet gate columns (both ranges empty in a plain GEMM).  With
  // v = acc * RN32(g_a g_w): columns [decay_lo, decay_hi) become the decay
  // gate -exp(a_log[j]) softplus(v + dt_bias[j]), j = col - decay_lo, and
  // columns [write_lo, write_hi) the write strength sigmoid(v).
  int decay_lo, decay_hi, write_lo, write_hi;
  const float* a_log;
  const float* dt_bias;
};

// Output of the SwiGLU + quantize epilogue: h = silu(gate) * up of a GEMM
// whose weight rows are [gate (F rows); up (F rows)], quantized with the
// given tensor scale into codes [M x F/2] and scales [M x F/16], and
// optionally written in fp32 to h [M x ldh].
struct SwigluOut {
  const float* gs;
  uint8_t* codes;
  uint8_t* scales;
  float* h;
  int64_t ldh;
  int F;
};

hipError_t launch_gemm_swiglu_quantize(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                                       const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                                       int64_t M, int64_t F, int64_t K, const SwigluOut& out, hipStream_t stream);

// Tail split of the large-tile GEMM.  Its workgroups take 256 x 256 output
// tiles, one per CU at a time, so a tile count just above a multiple of 256
// leaves the last round almost empty (4096 x 12384 has 784 tiles: 3 full
// rounds and 16 tiles).  Tiles 0 .. full - 1 are done whole; each of the
// `tail` remaining tiles is split over K into `splits` parts whose fp32
// partial sums go to the workspace, and a second kernel adds the parts in
// part order and writes the output.  splits == 0: no split.
struct SplitTail {
  int full;
  int tail;
  int splits;
  float* part;  // [tail x splits x 64 x 256 x 4] fp32 partial sums (workspace)
};

// The split for a shape on the large-tile kernel (splits == 0 when the last
// round is more than a quarter full, or K is too short to split), and the
// workspace bytes it needs (0 without a split).
SplitTail gemm_split_plan(int64_t M, int64_t N, int64_t K);
size_t gemm_split_workspace_bytes(int64_t M, int64_t N, int64_t K);

// The GEMM; `workspace` (16-byte aligned, workspace_bytes) lets it split the
// last round's tiles when gemm_split_workspace_bytes() > 0 and the
// large-tile kernel runs; NULL / 0 runs without.
hipError_t launch_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                       const uint8_t* w_codes, const uint8_t* w_scales, const ColScales& cs,
                       int64_t M, int64_t N, int64_t K, void* y, bool out_bf16, int64_t ldy,
                       hipStream_t stream, void* workspace = nullptr, size_t workspace_bytes = 0);

// Decode GEMM with the activation quantization done inside the kernel (bf16
// X, given tensor scale).  Only for shapes where quantize_gemm_fused_fits();
// W pointers 16 / 8 byte aligned, X rows 16 byte aligned.
bool quantize_gemm_fused_fits(int64_t M, int64_t N, int64_t K, bool in_bf16);
hipError_t launch_quantize_gemm_fused(const void* x, bool in_bf16, int64_t ldx, const float* a_gs,
                                      const uint8_t* w_codes, const uint8_t* w_scales, const ColScales& cs,
                                      int64_t M, int64_t N, int64_t K, void* y, bool out_bf16, int64_t ldy,
                                      hipStream_t stream);

// The allocation-free quantize + GEMM keeps the quantized activations in a
// static device array of this many bytes per GPU (nvfp4_noalloc.hip).
constexpr size_t kNoAllocScratchBytes = (size_t)4 << 20;

// Device address of that array on the current device, looked up with
// hipGetSymbolAddress on the first call per device and kept.
hipError_t no_alloc_scratch(void** ptr);

hipError_t launch_harmonize(uint8_t* scales, const float* module_gs, const int64_t* module_rows,
                            int32_t n_modules, int64_t K, float* shared_gs, uint32_t* counters,
                            hipStream_t stream);

// Gated DeltaNet recurrence over T >= 1 tokens, the columns of each value
// head's state (head dimension 128) split over workgroups; arguments as
// nvfp4_gdn_recurrence, already checked.
hipError_t launch_gdn_recurrence(const float* x, int64_t ldx, int64_t q_col, int64_t k_col, int64_t v_col,
                                 int64_t g_col, int64_t b_col, int64_t T, int n_qk, int n_v, const float* s_in,
                                 float* s_out, float* o, int64_t ldo, float* norms, const int* snap_steps,
                                 int n_snaps, float* snaps, hipStream_t stream);

// S_0 of a recurrence over no tokens: s_out = s_in, or zeros when s_in is
// NULL ([n_v x 128 x 128] fp32; s_in may equal s_out).
hipError_t launch_gdn_start_state(const float* s_in, float* s_out, int n_v, hipStream_t stream);

// Where the rows of a Gated DeltaNet call lie: q, k (n_qk heads) and v (n_v
// heads of 128) at columns of x, log-decay gates and write strengths (n_v
// each) at columns of gates, one row per token.
struct GdnRows {
  const void* x;
  int64_t ldx, q_col, k_col, v_col;
  const void* gates;
  bool gates_bf16;
  int64_t ldg, g_col, beta_col;
  int n_qk, n_v;
};

// One token for each of `batch` requests; the request's state slot is
// updated in place.  Arguments as nvfp4_gdn_decode, already checked.
hipError_t launch_gdn_decode(const GdnRows& in, bool x_bf16, int64_t batch, float* states, const int32_t* slots,
                             int n_slots, void* o, bool o_bf16, int64_t ldo, hipStream_t stream);

// Packed prompts (bf16 rows); arguments as nvfp4_gdn_prefill, already
// checked; workspace of gdn_prefill_workspace_bytes().
size_t gdn_prefill_workspace_bytes(int64_t T, int64_t n_seqs, int n_qk, int n_v);
hipError_t launch_gdn_prefill(const GdnRows& in, const int32_t* cu, int n_seqs, int64_t T, const float* s_in,
                              float* s_out, const int32_t* slots, int n_slots, void* o, int64_t ldo, void* workspace,
                              hipStream_t stream);

// Causal convolution + SiLU; cu NULL: one row per request.  Arguments as
// nvfp4_conv_silu, already checked.
hipError_t launch_conv_silu(const void* x, bool bf16, int64_t ldx, int64_t channels, const float* w, int width,
                            const int32_t* cu, int n_seqs, int64_t T, void* state, const int32_t* slots, int n_slots,
                            void* y, int64_t ldy, hipStream_t stream);

// Where a norm's y goes: values (bf16 or fp32) if y, NVFP4 codes and block
// scales under tensor scale *gs if codes.
struct NormOut {
  void* y;
  bool y_bf16;
  int64_t ldy;
  const float* gs;
  uint8_t* codes;
  uint8_t* scales;
};

// Columns of an add_rmsnorm row: one workgroup holds it, 16 values per lane.
constexpr int64_t kMaxNormCols = 16384;

hipError_t launch_add_rmsnorm(const void* x, bool x_bf16, int64_t ldx, const void* residual, bool r_bf16,
                              int64_t ldr, float scale, const float* w, float eps, int64_t rows, int64_t cols,
                              void* sum, int64_t lds, const NormOut& out, hipStream_t stream);
hipError_t launch_rmsnorm_gated(const void* o, bool o_bf16, int64_t ldo, const void* z, bool z_bf16, int64_t ldz,
                                const float* w, float eps, int64_t rows, int64_t cols, int group,
                                const NormOut& out, hipStream_t stream);

// Norm of each query and key head, then the rotation of its first `rot` dims:
// pair p by the angle whose cosine and sine are columns p and rot / 2 + p of
// row pos[axis(p)] of the table.  Arguments as nvfp4_qk_norm_rope, checked.
struct QkNormRope {
  const void* x;
  bool x_bf16;
  int64_t ldx, q_col, k_col;
  int64_t T;
  int hq, hk, d, rot;
  const float* q_w;
  const float* k_w;
  float eps;
  const float* table;
  int n_pos;
  const int32_t* pos;  // [n_axes x T]
  int n_axes;
  uint32_t axis[8];  // two bits per pair, pair 0 in the lowest
  bool adjacent;     // pairs (2 p, 2 p + 1) instead of (p, p + rot / 2)
  uint16_t* q;
  int64_t ldq;
  uint16_t* k;
  int64_t ldk;
};
hipError_t launch_qk_norm_rope(const QkNormRope& a, hipStream_t stream);

// A paged, quantised key/value cache (layout: nvfp4_kv.h).
struct KvCache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scales;  // NVFP4 only
  uint8_t* v_scales;
  const float* k_gs;
  const float* v_gs;
  bool fp4;
  int n_pages, page_shift, hk, d;
};

// The rows of a call and their sequences; cu NULL: row i is sequence i's only one.
struct KvRows {
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* kv_lens;
  const int32_t* cu;
  int n_seqs;
  int64_t T;
};

hipError_t launch_kv_cache_write(const KvCache& c, const KvRows& r, const void* k, int64_t ldk, const void* v,
                                 int64_t ldv, bool bf16, hipStream_t stream);
hipError_t launch_kv_cache_read(const KvCache& c, const KvRows& r, void* k, int64_t ldk, void* v, int64_t ldv,
                                bool bf16, hipStream_t stream);

// Attention over a cache; arguments as nvfp4_attn_cached, already checked;
// workspace of attn_cached_workspace_bytes().
size_t attn_cached_workspace_bytes(int64_t T, int n_seqs, int hq, int hk, int d);
hipError_t launch_attn_cached(const KvCache& c, const KvRows& r, const void* q, int64_t ldq, int hq, float scale,
                              const uint64_t* tree, void* o, int64_t ldo, void* workspace, hipStream_t stream);

}  // namespace nvfp4
