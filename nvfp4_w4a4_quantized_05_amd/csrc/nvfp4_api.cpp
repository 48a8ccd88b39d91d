// C ABI of the NVFP4 library: argument validation, then dispatch to the
// kernel launchers.  Every check runs before the first HIP call, so a bad
// argument never enqueues work (and the checks run on machines without a GPU).
#include "../../include/nvfp4.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "nvfp4_internal.h"

namespace {

thread_local int32_t g_last_hip_error = 0;

nvfp4_status_t hip_status(hipError_t e) {
  if (e == hipSuccess) return NVFP4_OK;
  g_last_hip_error = (int32_t)e;
  return NVFP4_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// Checks shared by nvfp4_gemm and nvfp4_gemm_segmented (the caller has
// filled the column scale table), then the launch.
nvfp4_status_t gemm_checked(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                            const uint8_t* w_codes, const uint8_t* w_scales, const nvfp4::ColScales& cs,
                            int64_t M, int64_t N, int64_t K, void* y, int32_t out_dtype, int64_t ldy,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_DTYPE;
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0 || ldy < N) return NVFP4_ERR_SHAPE;
  if (M > INT_MAX || N > INT_MAX || K > INT_MAX) return NVFP4_ERR_SHAPE;
  if (M == 0) return NVFP4_OK;
  if (!a_codes || !a_scales || !a_gs || !w_codes || !w_scales || !cs.gs || !y) return NVFP4_ERR_NULL;
  if (!aligned(a_gs, 4) || !aligned(cs.gs, 4) || !aligned(y, out_dtype == NVFP4_OUT_BF16 ? 2 : 4))
    return NVFP4_ERR_ALIGN;
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  if (tiles > (int64_t)INT_MAX) return NVFP4_ERR_SHAPE;
  const size_t need = nvfp4::gemm_split_workspace_bytes(M, N, K);
  if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (need > 0 && !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  return hip_status(nvfp4::launch_gemm(a_codes, a_scales, a_gs, w_codes, w_scales, cs, M, N, K, y,
                                       out_dtype == NVFP4_OUT_BF16, ldy, (hipStream_t)stream,
                                       need > 0 ? workspace : nullptr, need));
}


// Argument checks of nvfp4_quantize_gemm and its allocation-free variant
// (everything but the workspace), before any HIP call.
nvfp4_status_t quantize_gemm_checks(const void* x, int32_t in_dtype, int64_t ldx, const float* a_gs,
                                    const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs, int64_t M,
                                    int64_t N, int64_t K, void* y, int32_t out_dtype, int64_t ldy) {
  if (in_dtype != NVFP4_IN_F32 && in_dtype != NVFP4_IN_BF16) return NVFP4_ERR_DTYPE;
  if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_DTYPE;
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0 || ldx < K || ldy < N) return NVFP4_ERR_SHAPE;
  if (M > INT_MAX || N > INT_MAX || K > INT_MAX || M > INT64_MAX / ldx / 4) return NVFP4_ERR_SHAPE;
  if (M == 0) return NVFP4_OK;
  if (!x || !a_gs || !w_codes || !w_scales || !w_gs || !y) return NVFP4_ERR_NULL;
  const int64_t esize = in_dtype == NVFP4_IN_BF16 ? 2 : 4;
  if (!aligned(x, 16) || (ldx * esize) % 16 != 0 || !aligned(a_gs, 4) || !aligned(w_gs, 4) ||
      !aligned(y, out_dtype == NVFP4_OUT_BF16 ? 2 : 4))
    return NVFP4_ERR_ALIGN;
  if ((M * (K / 16) + 255) / 256 > (int64_t)INT_MAX) return NVFP4_ERR_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) > (int64_t)INT_MAX) return NVFP4_ERR_SHAPE;
  if (nvfp4_quantize_gemm_workspace_size(M, N, K, in_dtype, out_dtype) == 0 &&
      (!aligned(w_codes, 16) || !aligned(w_scales, 8)))
    return NVFP4_ERR_ALIGN;  // the one-kernel form reads W with 16- and 4-byte loads
  return NVFP4_OK;
}

// The launches of a checked quantize + GEMM: one kernel when `need` is 0,
// else the quantize kernel into ws (codes, then scales 256-byte aligned)
// and the GEMM from there.
nvfp4_status_t quantize_gemm_launch(const void* x, int32_t in_dtype, int64_t ldx, const float* a_gs,
                                    const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs, int64_t M,
                                    int64_t N, int64_t K, void* y, int32_t out_dtype, int64_t ldy, uint8_t* ws,
                                    size_t need, void* stream) {
  nvfp4::ColScales cs{};
  cs.gs = w_gs;
  cs.n = 1;
  cs.end[0] = (int)N;
  const bool in_bf16 = in_dtype == NVFP4_IN_BF16, out_bf16 = out_dtype == NVFP4_OUT_BF16;
  if (need == 0)  // one kernel: the decode GEMM quantizes the activations itself
    return hip_status(nvfp4::launch_quantize_gemm_fused(x, in_bf16, ldx, a_gs, w_codes, w_scales, cs, M, N, K, y,
                                                        out_bf16, ldy, (hipStream_t)stream));
  uint8_t* codes = ws;
  uint8_t* scales = codes + (M * (K / 2) + 255) / 256 * 256;
  const nvfp4_status_t st = hip_status(nvfp4::launch_quantize(x, in_bf16, M, K, ldx, codes, scales,
                                                              const_cast<float*>(a_gs), false, (hipStream_t)stream));
  if (st != NVFP4_OK) return st;
  return hip_status(nvfp4::launch_gemm(codes, scales, a_gs, w_codes, w_scales, cs, M, N, K, y, out_bf16, ldy,
                                       (hipStream_t)stream));
}

bool in_dtype_ok(int32_t d) { return d == NVFP4_IN_F32 || d == NVFP4_IN_BF16; }
int64_t in_size(int32_t d) { return d == NVFP4_IN_BF16 ? 2 : 4; }
// rows of ld values of 4 bytes can be addressed with 64-bit offsets
bool extent_ok(int64_t rows, int64_t ld) { return ld > 0 && rows <= INT64_MAX / ld / 4; }
bool row_aligned(const void* p, int64_t ld, int64_t esize) { return aligned(p, 16) && ld * esize % 16 == 0; }

// Memory that a call reads or writes: `rows` rows of `width` bytes, `step`
// bytes apart (step >= width); a plain array is one row, an absent one is at 0.
struct Span {
  uintptr_t at;
  uint64_t rows, width, step;
};
Span row_span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
  return {(uintptr_t)p, (uint64_t)rows, (uint64_t)(cols * esize), (uint64_t)(ld * esize)};
}
Span array_span(const void* p, uint64_t bytes) { return {(uintptr_t)p, 1, bytes, bytes}; }

bool overlap(const Span& a, const Span& b) {
  if (!a.at || !b.at || !a.rows || !b.rows || !a.width || !b.width) return false;
  if (a.at >= b.at + (b.rows - 1) * b.step + b.width || b.at >= a.at + (a.rows - 1) * a.step + a.width) return false;
  // rows of one step are apart as far as their columns are
  if (a.rows == 1 || b.rows == 1 || a.step != b.step) return true;
  const uint64_t d = b.at >= a.at ? (b.at - a.at) % a.step : (a.step - (a.at - b.at) % a.step) % a.step;
  return d < a.width || d + b.width > a.step;
}

// Whether what a call writes lies on anything else of it.  It may be one of
// `in_place` exactly, value by value.
bool clash(std::initializer_list<Span> written, std::initializer_list<Span> read,
           std::initializer_list<Span> in_place = {}) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* v = written.begin(); v != w; ++v)
      if (overlap(*w, *v)) return true;
    for (const Span& r : read)
      if (overlap(*w, r)) return true;
    for (const Span& r : in_place)
      if (overlap(*w, r) &&
          !(w->at == r.at && w->rows == r.rows && w->width == r.width && (w->rows == 1 || w->step == r.step)))
        return true;
  }
  return false;
}

// Shapes of the rows of nvfp4_gdn_prefill and nvfp4_gdn_decode.
nvfp4_status_t gdn_rows_shape(const nvfp4::GdnRows& in, int32_t gates_dtype) {
  constexpr int64_t kD = 128, kMaxLd = (int64_t)1 << 23;
  if (!in_dtype_ok(gates_dtype)) return NVFP4_ERR_DTYPE;
  if (in.ldx <= 0 || in.ldx >= kMaxLd || in.ldg <= 0 || in.ldg >= kMaxLd) return NVFP4_ERR_SHAPE;
  if (in.n_qk < 1 || in.n_v < 1 || in.n_v > 65535 || in.n_v % in.n_qk != 0) return NVFP4_ERR_SHAPE;
  const auto inside = [](int64_t col, int64_t width, int64_t ld) { return col >= 0 && col <= ld - width; };
  if (!inside(in.q_col, in.n_qk * kD, in.ldx) || !inside(in.k_col, in.n_qk * kD, in.ldx) ||
      !inside(in.v_col, in.n_v * kD, in.ldx) || !inside(in.g_col, in.n_v, in.ldg) ||
      !inside(in.beta_col, in.n_v, in.ldg))
    return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// x, its columns and gates aligned for the kernels' loads.
bool gdn_rows_aligned(const nvfp4::GdnRows& in, int64_t xsize) {
  const int64_t per = 16 / xsize;
  return row_aligned(in.x, in.ldx, xsize) && in.q_col % per == 0 && in.k_col % per == 0 && in.v_col % per == 0 &&
         aligned(in.gates, in.gates_bf16 ? 2 : 4);
}

// Whether o or the written states of a recurrence call lie on what it reads;
// `scratch` is written too.
bool gdn_clash(const nvfp4::GdnRows& in, int64_t xsize, int64_t rows, const Span& o, const Span& state_out,
               const Span& state_in, const Span& scratch, const Span& cu, const Span& slots) {
  const auto x = [&](int64_t col, int64_t heads) {
    return row_span(static_cast<const char*>(in.x) + col * xsize, in.x ? rows : 0, heads * 128, in.ldx, xsize);
  };
  const int64_t gsize = in.gates_bf16 ? 2 : 4;
  const auto gate = [&](int64_t col) {
    return row_span(static_cast<const char*>(in.gates) + col * gsize, in.gates ? rows : 0, in.n_v, in.ldg, gsize);
  };
  return clash({o, scratch}, {state_in}) ||
         clash({o, state_out, scratch},
               {x(in.q_col, in.n_qk), x(in.k_col, in.n_qk), x(in.v_col, in.n_v), gate(in.g_col), gate(in.beta_col), cu, slots},
               {state_in});
}

// Checks of a norm's destinations that nvfp4_add_rmsnorm and
// nvfp4_rmsnorm_gated share; `quant`: codes are asked for.
nvfp4_status_t norm_out_checks(const nvfp4::NormOut& out, int64_t rows, int64_t cols, bool& quant) {
  quant = out.gs || out.codes || out.scales;
  if (quant && (!out.gs || !out.codes || !out.scales)) return NVFP4_ERR_NULL;
  if (!quant && !out.y) return NVFP4_ERR_NULL;
  if (out.y && (out.ldy < cols || !extent_ok(rows, out.ldy))) return NVFP4_ERR_SHAPE;
  if (quant && cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (quant && (!aligned(out.codes, 8) || !aligned(out.gs, 4))) return NVFP4_ERR_ALIGN;
  if (out.y && !aligned(out.y, out.y_bf16 ? 2 : 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Whether what a norm writes (y, codes, scales and t) lies on anything else of
// it; a and b, its inputs, may be in the place of y or t.
bool norm_clash(const nvfp4::NormOut& out, int64_t rows, int64_t cols, const Span& t, const Span& w, const Span& a,
                const Span& b) {
  const Span gs = array_span(out.gs, 4);
  const Span codes = array_span(out.codes, (uint64_t)rows * cols / 2), scales = array_span(out.scales, (uint64_t)rows * cols / 16);
  return clash({row_span(out.y, rows, cols, out.ldy, out.y_bf16 ? 2 : 4), t, codes, scales}, {w, gs}, {a, b}) ||
         clash({codes, scales}, {a, b});
}

// Head sizes of the attention layer's calls.
bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

// A cache and the rows of a call on it, checked (but for alignment of what the
// call itself adds); `empty`: no rows, nothing to do.
nvfp4_status_t kv_checks(const nvfp4_kv_cache_t* cache, const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                         const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                         nvfp4::KvCache& c, nvfp4::KvRows& r, bool& empty) {
  empty = false;
  if (!cache) return NVFP4_ERR_NULL;
  if (cache->format != NVFP4_KV_E4M3 && cache->format != NVFP4_KV_NVFP4) return NVFP4_ERR_MODE;
  if (!head_dim_ok(cache->head_dim) || cache->n_kv_heads < 1 || cache->n_kv_heads > 4096 || cache->n_pages < 1)
    return NVFP4_ERR_SHAPE;
  const int32_t ps = cache->page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0) return NVFP4_ERR_SHAPE;
  if (max_pages < 1 || ld_table < max_pages || n_seqs < 1 || n_seqs > (1 << 20) || T < 0 || T >= (1 << 30))
    return NVFP4_ERR_SHAPE;
  if (ld_table > INT64_MAX / 4 / n_seqs || (!cu_seqlens && T != n_seqs)) return NVFP4_ERR_SHAPE;
  const bool fp4 = cache->format == NVFP4_KV_NVFP4;
  if (T == 0) {
    empty = true;
    return NVFP4_OK;
  }
  if (!cache->k || !cache->v || !cache->k_gs || !cache->v_gs || (fp4 && (!cache->k_scales || !cache->v_scales)) ||
      !page_table || !kv_lens)
    return NVFP4_ERR_NULL;
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || (fp4 && (!aligned(cache->k_scales, 16) || !aligned(cache->v_scales, 16))) ||
      !aligned(cache->k_gs, 4) || !aligned(cache->v_gs, 4) || !aligned(page_table, 4) || !aligned(kv_lens, 4) ||
      !aligned(cu_seqlens, 4))
    return NVFP4_ERR_ALIGN;
  c = {cache->k,    cache->v, cache->k_scales, cache->v_scales, cache->k_gs, cache->v_gs, fp4, cache->n_pages,
       __builtin_ctz((unsigned)ps), cache->n_kv_heads, cache->head_dim};
  r = {page_table, ld_table, max_pages, kv_lens, cu_seqlens, n_seqs, T};
  return NVFP4_OK;
}

// What those arguments span: k, v, k_scales, v_scales, k_gs, v_gs, page table, lengths, row numbers.
struct KvSpans {
  Span k, v, ks, vs, kg, vg, table, lens, cu;
};
KvSpans kv_spans(const nvfp4::KvCache& c, const nvfp4::KvRows& r) {
  const uint64_t values = (uint64_t)c.n_pages * c.hk * c.d << c.page_shift;
  return {array_span(c.k, c.fp4 ? values / 2 : values),
          array_span(c.v, c.fp4 ? values / 2 : values),
          array_span(c.fp4 ? c.k_scales : nullptr, values / 16),
          array_span(c.fp4 ? c.v_scales : nullptr, values / 16),
          array_span(c.k_gs, 4),
          array_span(c.v_gs, 4),
          row_span(r.table, r.n_seqs, r.max_pages, r.ld_table, 4),
          array_span(r.kv_lens, 4 * (uint64_t)r.n_seqs),
          array_span(r.cu, 4 * ((uint64_t)r.n_seqs + 1))};
}

// Shapes and places of the rows that nvfp4_kv_cache_write reads and _read writes.
nvfp4_status_t kv_row_checks(const nvfp4::KvCache& c, const nvfp4::KvRows& r, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, int32_t dtype) {
  const int64_t cols = (int64_t)c.hk * c.d, e = in_size(dtype);
  if (ldk < cols || ldv < cols || !extent_ok(r.T, ldk) || !extent_ok(r.T, ldv)) return NVFP4_ERR_SHAPE;
  if ((r.T / 16 + 2 * (int64_t)r.n_seqs) * cols >= ((int64_t)1 << 31)) return NVFP4_ERR_SHAPE;  // threads below 2^32
  if (!k || !v) return NVFP4_ERR_NULL;
  if (!row_aligned(k, ldk, e) || !row_aligned(v, ldv, e)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status_t nvfp4_quantize(const void* x, int32_t in_dtype, int64_t rows, int64_t cols,
                              int64_t ldx, uint8_t* codes, uint8_t* scales,
                              float* global_scale, int32_t mode, void* stream) {
  try {
    if (in_dtype != NVFP4_IN_F32 && in_dtype != NVFP4_IN_BF16) return NVFP4_ERR_DTYPE;
    if (mode != NVFP4_SCALE_GIVEN && mode != NVFP4_SCALE_FROM_AMAX) return NVFP4_ERR_MODE;
    if (rows < 0 || cols <= 0 || cols % 16 != 0 || ldx < cols) return NVFP4_ERR_SHAPE;
    if (rows > INT64_MAX / (ldx > 0 ? ldx : 1) / 4) return NVFP4_ERR_SHAPE;
    if (rows == 0) {  // nothing to encode; FROM_AMAX still writes g (1.0: no values, amax 0)
      if (mode == NVFP4_SCALE_GIVEN) return NVFP4_OK;
      if (!global_scale) return NVFP4_ERR_NULL;
      if (!aligned(global_scale, 4)) return NVFP4_ERR_ALIGN;
      return hip_status(nvfp4::launch_quantize(nullptr, in_dtype == NVFP4_IN_BF16, 0, cols, ldx, nullptr, nullptr,
                                               global_scale, true, (hipStream_t)stream));
    }
    if (!x || !codes || !scales || !global_scale) return NVFP4_ERR_NULL;
    const int64_t esize = in_dtype == NVFP4_IN_BF16 ? 2 : 4;
    if (!aligned(x, 16) || (ldx * esize) % 16 != 0 || !aligned(codes, 8) || !aligned(global_scale, 4))
      return NVFP4_ERR_ALIGN;
    if ((rows * (cols / 16) + 255) / 256 > (int64_t)INT_MAX) return NVFP4_ERR_SHAPE;
    return hip_status(nvfp4::launch_quantize(x, in_dtype == NVFP4_IN_BF16, rows, cols, ldx, codes,
                                             scales, global_scale, mode == NVFP4_SCALE_FROM_AMAX,
                                             (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

size_t nvfp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t out_dtype) {
  (void)out_dtype;
  if (M <= 0 || N <= 0 || K <= 0 || M > INT_MAX || N > INT_MAX || K > INT_MAX) return 0;
  return nvfp4::gemm_split_workspace_bytes(M, N, K);
}

nvfp4_status_t nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                          const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                          int64_t M, int64_t N, int64_t K, void* y, int32_t out_dtype,
                          int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    nvfp4::ColScales cs{};
    cs.gs = w_gs;
    cs.n = 1;
    cs.end[0] = (N > 0 && N <= INT_MAX) ? (int)N : 0;  // out-of-range N fails the shape check
    return gemm_checked(a_codes, a_scales, a_gs, w_codes, w_scales, cs, M, N, K, y, out_dtype, ldy,
                        workspace, workspace_bytes, stream);
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_gemm_segmented(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                                    const uint8_t* w_codes, const uint8_t* w_scales,
                                    const float* module_gs, const int64_t* module_rows, int32_t n_modules,
                                    int64_t M, int64_t K, void* y, int32_t out_dtype, int64_t ldy,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!module_rows) return NVFP4_ERR_NULL;
    if (n_modules < 1 || n_modules > nvfp4::kMaxModules) return NVFP4_ERR_SHAPE;
    nvfp4::ColScales cs{};
    cs.gs = module_gs;
    cs.n = n_modules;
    int64_t N = 0;
    for (int32_t i = 0; i < n_modules; ++i) {
      if (module_rows[i] < 0 || module_rows[i] > (int64_t)INT_MAX - N) return NVFP4_ERR_SHAPE;
      N += module_rows[i];
      cs.end[i] = (int)N;
    }
    return gemm_checked(a_codes, a_scales, a_gs, w_codes, w_scales, cs, M, N, K, y, out_dtype, ldy,
                        workspace, workspace_bytes, stream);
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_gemm_segmented_gates(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                                          const uint8_t* w_codes, const uint8_t* w_scales,
                                          const float* module_gs, const int64_t* module_rows, int32_t n_modules,
                                          int32_t decay_module, const float* a_log, const float* dt_bias,
                                          int32_t write_module, int64_t M, int64_t K, void* y, int32_t out_dtype,
                                          int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!module_rows) return NVFP4_ERR_NULL;
    if (n_modules < 1 || n_modules > nvfp4::kMaxModules) return NVFP4_ERR_SHAPE;
    if (decay_module < -1 || decay_module >= n_modules || write_module < -1 || write_module >= n_modules)
      return NVFP4_ERR_SHAPE;
    if (decay_module >= 0 && decay_module == write_module) return NVFP4_ERR_SHAPE;
    if (decay_module >= 0) {
      if (!a_log || !dt_bias) return NVFP4_ERR_NULL;
      if (!aligned(a_log, 4) || !aligned(dt_bias, 4)) return NVFP4_ERR_ALIGN;
    }
    nvfp4::ColScales cs{};
    cs.gs = module_gs;
    cs.n = n_modules;
    int64_t N = 0;
    for (int32_t i = 0; i < n_modules; ++i) {
      if (module_rows[i] < 0 || module_rows[i] > (int64_t)INT_MAX - N) return NVFP4_ERR_SHAPE;
      if (i == decay_module) cs.decay_lo = (int)N, cs.decay_hi = (int)(N + module_rows[i]);
      if (i == write_module) cs.write_lo = (int)N, cs.write_hi = (int)(N + module_rows[i]);
      N += module_rows[i];
      cs.end[i] = (int)N;
    }
    cs.a_log = a_log;
    cs.dt_bias = dt_bias;
    return gemm_checked(a_codes, a_scales, a_gs, w_codes, w_scales, cs, M, N, K, y, out_dtype, ldy,
                        workspace, workspace_bytes, stream);
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_gdn_recurrence(const float* x, int64_t ldx, int64_t q_col, int64_t k_col, int64_t v_col,
                                    int64_t g_col, int64_t beta_col, int64_t T, int32_t n_qk_heads,
                                    int32_t n_v_heads, const float* state_in, float* state_out, float* o,
                                    int64_t ldo, float* state_norms, const int32_t* snap_steps, int32_t n_snaps,
                                    float* snaps, void* stream) {
  try {
    constexpr int64_t kD = 128;
    // rows of fewer than 2^23 values: 64 rows of the chunk loads stay below 2^31 bytes
    if (T < 0 || T > INT_MAX || ldx <= 0 || ldx >= ((int64_t)1 << 23)) return NVFP4_ERR_SHAPE;
    if (n_qk_heads < 1 || n_v_heads < 1 || n_v_heads > 65535 || n_v_heads % n_qk_heads != 0) return NVFP4_ERR_SHAPE;
    if (q_col < 0 || q_col + n_qk_heads * kD > ldx || k_col < 0 || k_col + n_qk_heads * kD > ldx)
      return NVFP4_ERR_SHAPE;
    if (v_col < -1 || (v_col >= 0 && v_col + n_v_heads * kD > ldx)) return NVFP4_ERR_SHAPE;
    if (g_col < 0 || g_col + n_v_heads > ldx || beta_col < 0 || beta_col + n_v_heads > ldx) return NVFP4_ERR_SHAPE;
    if (o && ldo < n_v_heads * kD) return NVFP4_ERR_SHAPE;
    if (n_snaps < 0) return NVFP4_ERR_SHAPE;
    if (T == 0) {  // S_0 is the start state; nothing else has a row to write
      if (!state_out) return NVFP4_OK;
      if (!aligned(state_out, 4) || (state_in && !aligned(state_in, 4))) return NVFP4_ERR_ALIGN;
      return hip_status(nvfp4::launch_gdn_start_state(state_in, state_out, n_v_heads, (hipStream_t)stream));
    }
    if (!x || (n_snaps > 0 && (!snap_steps || !snaps))) return NVFP4_ERR_NULL;
    for (const void* p : {(const void*)x, (const void*)state_in, (const void*)state_out, (const void*)o,
                          (const void*)state_norms, (const void*)snap_steps, (const void*)snaps})
      if (p && !aligned(p, 4)) return NVFP4_ERR_ALIGN;
    return hip_status(nvfp4::launch_gdn_recurrence(x, ldx, q_col, k_col, v_col, g_col, beta_col, T, n_qk_heads,
                                                   n_v_heads, state_in, state_out, o, ldo, state_norms,
                                                   snap_steps, n_snaps > 0 ? n_snaps : 0, snaps,
                                                   (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_gemm_swiglu_quantize(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gs,
                                          const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                                          int64_t M, int64_t F, int64_t K, const float* h_gs, uint8_t* h_codes,
                                          uint8_t* h_scales, float* h, int64_t ldh, void* stream) {
  try {
    if (M < 0 || F <= 0 || K <= 0 || K % 128 != 0 || F % 64 != 0) return NVFP4_ERR_SHAPE;
    if (M > INT_MAX || F > INT_MAX / 2 || K > INT_MAX) return NVFP4_ERR_SHAPE;
    if (h && ldh < F) return NVFP4_ERR_SHAPE;
    // 32-bit buffer offsets of the streaming kernel
    if (M * (K / 2) >= ((int64_t)1 << 31) || 2 * F * (K / 2) >= ((int64_t)1 << 31)) return NVFP4_ERR_SHAPE;
    if (M == 0) return NVFP4_OK;
    if (!a_codes || !a_scales || !a_gs || !w_codes || !w_scales || !w_gs || !h_gs || !h_codes || !h_scales)
      return NVFP4_ERR_NULL;
    if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(a_scales, 8) || !aligned(w_scales, 8) ||
        !aligned(a_gs, 4) || !aligned(w_gs, 4) || !aligned(h_gs, 4) || !aligned(h_codes, 8) ||
        (h && (!aligned(h, 16) || ldh % 4 != 0)))
      return NVFP4_ERR_ALIGN;
    if (((M + 255) / 256) * ((2 * F + 255) / 256) > (int64_t)INT_MAX) return NVFP4_ERR_SHAPE;
    nvfp4::SwigluOut out{h_gs, h_codes, h_scales, h, ldh, (int)F};
    return hip_status(nvfp4::launch_gemm_swiglu_quantize(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, M, F, K,
                                                         out, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

size_t nvfp4_quantize_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t in_dtype, int32_t out_dtype) {
  (void)out_dtype;
  if (M <= 0 || N <= 0 || K <= 0 || K % 16 != 0 || M > INT_MAX || K > INT_MAX) return 0;
  if (nvfp4::quantize_gemm_fused_fits(M, N, K, in_dtype == NVFP4_IN_BF16)) return 0;
  const int64_t code_bytes = (M * (K / 2) + 255) / 256 * 256;  // scales start 256-byte aligned
  return (size_t)(code_bytes + M * (K / 16));
}

nvfp4_status_t nvfp4_quantize_gemm(const void* x, int32_t in_dtype, int64_t ldx, const float* a_gs,
                                   const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                                   int64_t M, int64_t N, int64_t K, void* y, int32_t out_dtype, int64_t ldy,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  try {
    const nvfp4_status_t st = quantize_gemm_checks(x, in_dtype, ldx, a_gs, w_codes, w_scales, w_gs, M, N, K, y,
                                                   out_dtype, ldy);
    if (st != NVFP4_OK || M == 0) return st;
    const size_t need = nvfp4_quantize_gemm_workspace_size(M, N, K, in_dtype, out_dtype);
    if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
    if (need > 0 && !workspace) return NVFP4_ERR_NULL;
    if (need > 0 && !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    return quantize_gemm_launch(x, in_dtype, ldx, a_gs, w_codes, w_scales, w_gs, M, N, K, y, out_dtype, ldy,
                                static_cast<uint8_t*>(workspace), need, stream);
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_quantize_gemm_no_alloc(const void* x, int32_t in_dtype, int64_t ldx, const float* a_gs,
                                            const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gs,
                                            int64_t M, int64_t N, int64_t K, void* y, int32_t out_dtype,
                                            int64_t ldy, void* stream) {
  try {
    const nvfp4_status_t st = quantize_gemm_checks(x, in_dtype, ldx, a_gs, w_codes, w_scales, w_gs, M, N, K, y,
                                                   out_dtype, ldy);
    if (st != NVFP4_OK || M == 0) return st;
    const size_t need = nvfp4_quantize_gemm_workspace_size(M, N, K, in_dtype, out_dtype);
    if (need > nvfp4::kNoAllocScratchBytes) return NVFP4_ERR_TOO_LARGE;
    void* scratch = nullptr;
    if (need > 0) {
      const hipError_t e = nvfp4::no_alloc_scratch(&scratch);
      if (e != hipSuccess) return hip_status(e);
    }
    return quantize_gemm_launch(x, in_dtype, ldx, a_gs, w_codes, w_scales, w_gs, M, N, K, y, out_dtype, ldy,
                                static_cast<uint8_t*>(scratch), need, stream);
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

size_t nvfp4_quantize_gemm_no_alloc_max_bytes(void) { return nvfp4::kNoAllocScratchBytes; }

nvfp4_status_t nvfp4_harmonize_fused_scales(uint8_t* scales, const float* module_gs,
                                            const int64_t* module_rows, int32_t n_modules,
                                            int64_t K, float* shared_gs, uint32_t* counters,
                                            void* stream) {
  try {
    if (!scales || !module_gs || !module_rows || !shared_gs) return NVFP4_ERR_NULL;
    if (n_modules < 1 || n_modules > nvfp4::kMaxModules) return NVFP4_ERR_SHAPE;
    if (K <= 0 || K % 16 != 0) return NVFP4_ERR_SHAPE;
    int64_t total = 0;
    for (int32_t i = 0; i < n_modules; ++i) {
      if (module_rows[i] < 0 || module_rows[i] > INT64_MAX / 2 - total) return NVFP4_ERR_SHAPE;
      total += module_rows[i];
    }
    if (total > INT64_MAX / (K / 16)) return NVFP4_ERR_SHAPE;
    if (!aligned(module_gs, 4) || !aligned(shared_gs, 4) || (counters && !aligned(counters, 4)))
      return NVFP4_ERR_ALIGN;
    // the shared scale is written while module scales are still being read
    const uintptr_t g0 = (uintptr_t)module_gs, g1 = g0 + 4u * (uintptr_t)n_modules;
    const uintptr_t s0 = (uintptr_t)shared_gs;
    if (s0 + 4 > g0 && s0 < g1) return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_harmonize(scales, module_gs, module_rows, n_modules, K, shared_gs,
                                              counters, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_gdn_prefill(const void* x, int64_t ldx, int64_t q_col, int64_t k_col, int64_t v_col,
                                 const void* gates, int32_t gates_dtype, int64_t ldg, int64_t g_col,
                                 int64_t beta_col, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                                 int32_t n_qk_heads, int32_t n_v_heads, const float* state_in, float* state_out,
                                 const int32_t* slots, int32_t n_slots, void* o, int64_t ldo, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  try {
    const nvfp4::GdnRows in{x,   ldx,   q_col,    k_col,      v_col,    gates, gates_dtype == NVFP4_IN_BF16,
                            ldg, g_col, beta_col, n_qk_heads, n_v_heads};
    const nvfp4_status_t st = gdn_rows_shape(in, gates_dtype);
    if (st != NVFP4_OK) return st;
    if (T < 0 || T > INT_MAX || n_seqs < 1 || n_seqs > (1 << 20) || n_slots < 0) return NVFP4_ERR_SHAPE;
    if (ldo < (int64_t)n_v_heads * 128 || ldo >= ((int64_t)1 << 23)) return NVFP4_ERR_SHAPE;
    // grid sizes (threads below 2^32)
    if ((int64_t)n_seqs * n_v_heads > (1 << 20) || (T / 64 + n_seqs + 1) * n_qk_heads >= (1 << 24))
      return NVFP4_ERR_SHAPE;
    if (!cu_seqlens || (T > 0 && (!x || !gates || !o))) return NVFP4_ERR_NULL;
    if ((T > 0 && !gdn_rows_aligned(in, 2)) || !row_aligned(o, ldo, 2) || !aligned(cu_seqlens, 4) ||
        !aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(slots, 4))
      return NVFP4_ERR_ALIGN;
    const size_t need = nvfp4::gdn_prefill_workspace_bytes(T, n_seqs, n_qk_heads, n_v_heads);
    if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
    if (need > 0 && !workspace) return NVFP4_ERR_NULL;
    if (need > 0 && !aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
    const uint64_t pool = (uint64_t)n_slots * n_v_heads * 128 * 128 * 4;
    if (gdn_clash(in, 2, T, row_span(o, T, (int64_t)n_v_heads * 128, ldo, 2), array_span(state_out, pool),
                  array_span(state_in, pool), array_span(workspace, need), array_span(cu_seqlens, 4 * ((uint64_t)n_seqs + 1)),
                  array_span(slots, 4 * (uint64_t)n_seqs)))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_gdn_prefill(in, cu_seqlens, n_seqs, T, state_in, state_out, slots, n_slots, o,
                                                ldo, workspace, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

size_t nvfp4_gdn_prefill_workspace_size(int64_t T, int32_t n_seqs, int32_t n_qk_heads, int32_t n_v_heads) {
  if (T < 0 || T > INT_MAX || n_seqs < 1 || n_seqs > (1 << 20) || n_qk_heads < 1 || n_v_heads < 1 ||
      n_v_heads > 65535 || n_v_heads % n_qk_heads != 0)
    return 0;
  return nvfp4::gdn_prefill_workspace_bytes(T, n_seqs, n_qk_heads, n_v_heads);
}

nvfp4_status_t nvfp4_gdn_decode(const void* x, int32_t x_dtype, int64_t ldx, int64_t q_col, int64_t k_col,
                                int64_t v_col, const void* gates, int32_t gates_dtype, int64_t ldg, int64_t g_col,
                                int64_t beta_col, int64_t batch, int32_t n_qk_heads, int32_t n_v_heads,
                                float* states, const int32_t* slots, int32_t n_slots, void* o, int32_t o_dtype,
                                int64_t ldo, void* stream) {
  try {
    if (!in_dtype_ok(x_dtype) || (o_dtype != NVFP4_OUT_F32 && o_dtype != NVFP4_OUT_BF16)) return NVFP4_ERR_DTYPE;
    const nvfp4::GdnRows in{x,   ldx,   q_col,    k_col,      v_col,    gates, gates_dtype == NVFP4_IN_BF16,
                            ldg, g_col, beta_col, n_qk_heads, n_v_heads};
    const nvfp4_status_t st = gdn_rows_shape(in, gates_dtype);
    if (st != NVFP4_OK) return st;
    if (batch < 0 || batch > (1 << 20) || batch * n_v_heads > (1 << 20) || n_slots < 0) return NVFP4_ERR_SHAPE;
    if (ldo < (int64_t)n_v_heads * 128 || !extent_ok(batch, ldo)) return NVFP4_ERR_SHAPE;
    if (batch == 0) return NVFP4_OK;
    if (!x || !gates || !states || !o) return NVFP4_ERR_NULL;
    if (!gdn_rows_aligned(in, in_size(x_dtype)) || !row_aligned(o, ldo, o_dtype == NVFP4_OUT_BF16 ? 2 : 4) ||
        !aligned(states, 16) || !aligned(slots, 4))
      return NVFP4_ERR_ALIGN;
    if (gdn_clash(in, in_size(x_dtype), batch,
                  row_span(o, batch, (int64_t)n_v_heads * 128, ldo, o_dtype == NVFP4_OUT_BF16 ? 2 : 4),
                  array_span(states, (uint64_t)n_slots * n_v_heads * 128 * 128 * 4), Span{}, Span{}, Span{},
                  array_span(slots, 4 * (uint64_t)batch)))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_gdn_decode(in, x_dtype == NVFP4_IN_BF16, batch, states, slots, n_slots, o,
                                               o_dtype == NVFP4_OUT_BF16, ldo, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_conv_silu(const void* x, int32_t dtype, int64_t ldx, int64_t channels, const float* w,
                               int32_t width, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T, void* state,
                               const int32_t* slots, int32_t n_slots, void* y, int64_t ldy, void* stream) {
  try {
    if (!in_dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
    if (width < 2 || width > 4 || channels < 1 || channels > (1 << 20) || n_slots < 0) return NVFP4_ERR_SHAPE;
    if (T < 0 || T > (cu_seqlens ? (int64_t)INT_MAX : (int64_t)1 << 22)) return NVFP4_ERR_SHAPE;
    if (cu_seqlens && (n_seqs < 1 || n_seqs > (1 << 20))) return NVFP4_ERR_SHAPE;
    if (ldx < channels || ldy < channels || !extent_ok(T, ldx) || !extent_ok(T, ldy)) return NVFP4_ERR_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!x || !w || !y) return NVFP4_ERR_NULL;
    const int64_t e = in_size(dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(state, e) || !aligned(w, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(slots, 4))
      return NVFP4_ERR_ALIGN;
    // neighbouring rows are read by other threads than the ones that write them
    if (clash({row_span(y, T, channels, ldy, e), array_span(state, (uint64_t)n_slots * (width - 1) * channels * e)},
              {row_span(x, T, channels, ldx, e), array_span(w, (uint64_t)channels * width * 4),
               array_span(cu_seqlens, cu_seqlens ? 4 * ((uint64_t)n_seqs + 1) : 0),
               array_span(slots, 4 * (uint64_t)(cu_seqlens ? n_seqs : T))}))
      return NVFP4_ERR_ALIAS;
    // without a pool every sequence starts at zeros and none is skipped
    return hip_status(nvfp4::launch_conv_silu(x, dtype == NVFP4_IN_BF16, ldx, channels, w, width, cu_seqlens,
                                              n_seqs, T, state, state ? slots : nullptr, state ? n_slots : 1, y, ldy,
                                              (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_add_rmsnorm(const void* x, int32_t x_dtype, int64_t ldx, const void* residual, int32_t r_dtype,
                                 int64_t ldr, float scale, const float* w, float eps, int64_t rows, int64_t cols,
                                 void* residual_out, int64_t ldro, void* y, int32_t y_dtype, int64_t ldy,
                                 const float* y_gs, uint8_t* y_codes, uint8_t* y_scales, void* stream) {
  try {
    if (!in_dtype_ok(x_dtype) || !in_dtype_ok(r_dtype)) return NVFP4_ERR_DTYPE;
    if (y_dtype != NVFP4_OUT_F32 && y_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_DTYPE;
    if (rows < 0 || rows > (1 << 22) || cols < 1 || cols > nvfp4::kMaxNormCols) return NVFP4_ERR_SHAPE;
    // grid size (threads below 2^32): a row of more than 15 x 1,024 columns takes 1,024
    if (rows == (1 << 22) && cols > 15 * 1024) return NVFP4_ERR_SHAPE;
    if (!(eps > 0.0f) || !std::isfinite(eps) || !std::isfinite(scale)) return NVFP4_ERR_SHAPE;
    if (ldx < cols || !extent_ok(rows, ldx)) return NVFP4_ERR_SHAPE;
    if (residual && (ldr < cols || !extent_ok(rows, ldr))) return NVFP4_ERR_SHAPE;
    if (residual_out && (ldro < cols || !extent_ok(rows, ldro))) return NVFP4_ERR_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!x || !w) return NVFP4_ERR_NULL;
    const nvfp4::NormOut out{y, y_dtype == NVFP4_OUT_BF16, ldy, y_gs, y_codes, y_scales};
    bool quant = false;
    const nvfp4_status_t st = norm_out_checks(out, rows, cols, quant);
    if (st != NVFP4_OK) return st;
    const int64_t xe = in_size(x_dtype), re = in_size(r_dtype);
    if (!aligned(x, xe) || !aligned(residual, re) || !aligned(residual_out, re) || !aligned(w, 4))
      return NVFP4_ERR_ALIGN;
    if (quant && (!row_aligned(x, ldx, xe) || (residual && !row_aligned(residual, ldr, re)) ||
                  (residual_out && !row_aligned(residual_out, ldro, re)) ||
                  (y && !row_aligned(y, ldy, out.y_bf16 ? 2 : 4)) || !aligned(w, 16)))
      return NVFP4_ERR_ALIGN;
    // a row is read whole before any of it is written
    if (norm_clash(out, rows, cols, row_span(residual_out, rows, cols, ldro, re), array_span(w, cols * 4),
                   row_span(x, rows, cols, ldx, xe), row_span(residual, rows, cols, ldr, re)))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_add_rmsnorm(x, x_dtype == NVFP4_IN_BF16, ldx, residual,
                                                r_dtype == NVFP4_IN_BF16, ldr, scale, w, eps, rows, cols,
                                                residual_out, ldro, out, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_rmsnorm_gated(const void* o, int32_t o_dtype, int64_t ldo, const void* z, int32_t z_dtype,
                                   int64_t ldz, const float* w, float eps, int64_t rows, int64_t cols, int32_t group,
                                   void* y, int32_t y_dtype, int64_t ldy, const float* y_gs, uint8_t* y_codes,
                                   uint8_t* y_scales, void* stream) {
  try {
    if (!in_dtype_ok(o_dtype) || !in_dtype_ok(z_dtype)) return NVFP4_ERR_DTYPE;
    if (y_dtype != NVFP4_OUT_F32 && y_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_DTYPE;
    if (group < 16 || group > 1024 || (group & (group - 1)) != 0) return NVFP4_ERR_SHAPE;
    if (rows < 0 || cols < 1 || cols % group != 0 || cols > INT_MAX || ldo < cols || ldz < cols)
      return NVFP4_ERR_SHAPE;
    if (rows > (((int64_t)1 << 35) - 1) / cols || !extent_ok(rows, ldo) || !extent_ok(rows, ldz)) return NVFP4_ERR_SHAPE;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return NVFP4_ERR_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!o || !z || !w) return NVFP4_ERR_NULL;
    const nvfp4::NormOut out{y, y_dtype == NVFP4_OUT_BF16, ldy, y_gs, y_codes, y_scales};
    bool quant = false;
    const nvfp4_status_t st = norm_out_checks(out, rows, cols, quant);
    if (st != NVFP4_OK) return st;
    if (!row_aligned(o, ldo, in_size(o_dtype)) || !row_aligned(z, ldz, in_size(z_dtype)) || !aligned(w, 16) ||
        (y && !row_aligned(y, ldy, out.y_bf16 ? 2 : 4)))
      return NVFP4_ERR_ALIGN;
    // a lane reads its values before it writes y there
    if (norm_clash(out, rows, cols, Span{}, array_span(w, group * 4), row_span(o, rows, cols, ldo, in_size(o_dtype)),
                   row_span(z, rows, cols, ldz, in_size(z_dtype))))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_rmsnorm_gated(o, o_dtype == NVFP4_IN_BF16, ldo, z, z_dtype == NVFP4_IN_BF16, ldz,
                                                  w, eps, rows, cols, group, out, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_qk_norm_rope(const void* x, int32_t x_dtype, int64_t ldx, int64_t q_col, int64_t k_col, int64_t T,
                                  int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const float* q_w,
                                  const float* k_w, float eps, const float* cos_sin, int32_t n_pos, int32_t rot,
                                  const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis, int32_t adjacent,
                                  void* q, int64_t ldq, void* k, int64_t ldk, void* stream) {
  try {
    if (!in_dtype_ok(x_dtype)) return NVFP4_ERR_DTYPE;
    if (adjacent != 0 && adjacent != 1) return NVFP4_ERR_MODE;
    if (!head_dim_ok(head_dim) || n_q_heads < 1 || n_q_heads > 4096 || n_kv_heads < 1 || n_kv_heads > 4096)
      return NVFP4_ERR_SHAPE;
    if (T < 0 || T > (1 << 25) || !(eps > 0.0f) || !std::isfinite(eps)) return NVFP4_ERR_SHAPE;
    if (rot < 16 || rot > head_dim || rot % 16 != 0 || n_pos < 1 || n_axes < 1 || n_axes > 4) return NVFP4_ERR_SHAPE;
    const int64_t q_cols = (int64_t)n_q_heads * head_dim, k_cols = (int64_t)n_kv_heads * head_dim;
    if (ldx <= 0 || q_col < 0 || q_col > ldx - q_cols || k_col < 0 || k_col > ldx - k_cols || ldq < q_cols || ldk < k_cols)
      return NVFP4_ERR_SHAPE;
    if (!extent_ok(T, ldx) || !extent_ok(T, ldq) || !extent_ok(T, ldk)) return NVFP4_ERR_SHAPE;
    nvfp4::QkNormRope a{x,       x_dtype == NVFP4_IN_BF16, ldx,       q_col,  k_col, T,      n_q_heads, n_kv_heads, head_dim,
                        rot,     q_w,                      k_w,       eps,    cos_sin, n_pos, positions, n_axes,     {},
                        adjacent == 1, static_cast<uint16_t*>(q), ldq, static_cast<uint16_t*>(k), ldk};
    if (n_axes > 1) {
      if (!pair_axis) return NVFP4_ERR_NULL;
      for (int p = 0; p < rot / 2; ++p) {
        if (pair_axis[p] >= n_axes) return NVFP4_ERR_SHAPE;
        a.axis[p / 16] |= (uint32_t)pair_axis[p] << (p % 16 * 2);
      }
    }
    if (T == 0) return NVFP4_OK;
    if (!x || !q_w || !k_w || !cos_sin || !positions || !q || !k) return NVFP4_ERR_NULL;
    const int64_t e = in_size(x_dtype);
    if (!row_aligned(x, ldx, e) || ldx % 8 != 0 || q_col % 8 != 0 || k_col % 8 != 0 || !aligned(q_w, 16) ||
        !aligned(k_w, 16) || !aligned(cos_sin, 16) || !aligned(positions, 4) || !row_aligned(q, ldq, 2) ||
        !row_aligned(k, ldk, 2))
      return NVFP4_ERR_ALIGN;
    const Span xq = row_span(static_cast<const char*>(x) + q_col * e, T, q_cols, ldx, e);
    const Span xk = row_span(static_cast<const char*>(x) + k_col * e, T, k_cols, ldx, e);
    const Span yq = row_span(q, T, q_cols, ldq, 2), yk = row_span(k, T, k_cols, ldk, 2);
    const Span qw = array_span(q_w, 4 * (uint64_t)head_dim), kw = array_span(k_w, 4 * (uint64_t)head_dim);
    const Span table = array_span(cos_sin, (uint64_t)n_pos * rot * 4), pos = array_span(positions, (uint64_t)n_axes * T * 4);
    // a head's lanes hold all of it before any of it is written; q and k of x are other waves' turns
    if (clash({yq, yk}, {qw, kw, table, pos}) || clash({yq}, {xk}, {xq}) || clash({yk}, {xq}, {xk})) return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_qk_norm_rope(a, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_kv_cache_write(const nvfp4_kv_cache_t* cache, const int32_t* page_table, int64_t ld_table,
                                    int32_t max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens,
                                    int32_t n_seqs, int64_t T, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                    int32_t dtype, void* stream) {
  try {
    if (!in_dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
    nvfp4::KvCache c;
    nvfp4::KvRows r;
    bool empty;
    nvfp4_status_t st = kv_checks(cache, page_table, ld_table, max_pages, kv_lens, cu_seqlens, n_seqs, T, c, r, empty);
    if (st != NVFP4_OK || empty) return st;
    st = kv_row_checks(c, r, k, ldk, v, ldv, dtype);
    if (st != NVFP4_OK) return st;
    const KvSpans s = kv_spans(c, r);
    const int64_t cols = (int64_t)c.hk * c.d, e = in_size(dtype);
    if (clash({s.k, s.v, s.ks, s.vs},
              {s.kg, s.vg, s.table, s.lens, s.cu, row_span(k, T, cols, ldk, e), row_span(v, T, cols, ldv, e)}))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_kv_cache_write(c, r, k, ldk, v, ldv, dtype == NVFP4_IN_BF16, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

nvfp4_status_t nvfp4_kv_cache_read(const nvfp4_kv_cache_t* cache, const int32_t* page_table, int64_t ld_table,
                                   int32_t max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens,
                                   int32_t n_seqs, int64_t T, void* k, int64_t ldk, void* v, int64_t ldv, int32_t dtype,
                                   void* stream) {
  try {
    if (dtype != NVFP4_OUT_F32 && dtype != NVFP4_OUT_BF16) return NVFP4_ERR_DTYPE;
    nvfp4::KvCache c;
    nvfp4::KvRows r;
    bool empty;
    nvfp4_status_t st = kv_checks(cache, page_table, ld_table, max_pages, kv_lens, cu_seqlens, n_seqs, T, c, r, empty);
    if (st != NVFP4_OK || empty) return st;
    st = kv_row_checks(c, r, k, ldk, v, ldv, dtype);
    if (st != NVFP4_OK) return st;
    const KvSpans s = kv_spans(c, r);
    const int64_t cols = (int64_t)c.hk * c.d, e = in_size(dtype);
    if (clash({row_span(k, T, cols, ldk, e), row_span(v, T, cols, ldv, e)},
              {s.k, s.v, s.ks, s.vs, s.kg, s.vg, s.table, s.lens, s.cu}))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_kv_cache_read(c, r, k, ldk, v, ldv, dtype == NVFP4_OUT_BF16, (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

size_t nvfp4_attn_cached_workspace_size(int64_t T, int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                        int32_t head_dim) {
  if (T <= 0 || T >= (1 << 30) || n_seqs < 1 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads > 4096 ||
      n_q_heads % n_kv_heads != 0 || !head_dim_ok(head_dim))
    return 0;
  return nvfp4::attn_cached_workspace_bytes(T, n_seqs, n_q_heads, n_kv_heads, head_dim);
}

nvfp4_status_t nvfp4_attn_cached(const nvfp4_kv_cache_t* cache, const int32_t* page_table, int64_t ld_table,
                                 int32_t max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t n_seqs,
                                 int64_t T, const void* q, int64_t ldq, int32_t n_q_heads, float scale,
                                 const uint64_t* tree, void* o, int64_t ldo, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  try {
    nvfp4::KvCache c;
    nvfp4::KvRows r;
    bool empty;
    const nvfp4_status_t st =
        kv_checks(cache, page_table, ld_table, max_pages, kv_lens, cu_seqlens, n_seqs, T, c, r, empty);
    if (st != NVFP4_OK) return st;
    if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % cache->n_kv_heads != 0) return NVFP4_ERR_SHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return NVFP4_ERR_SHAPE;
    const int64_t cols = (int64_t)n_q_heads * cache->head_dim;
    if (ldq < cols || ldo < cols || !extent_ok(T, ldq) || !extent_ok(T, ldo)) return NVFP4_ERR_SHAPE;
    if (empty) return NVFP4_OK;
    if (!q || !o) return NVFP4_ERR_NULL;
    if (!row_aligned(q, ldq, 2) || !row_aligned(o, ldo, 2) || !aligned(tree, 8)) return NVFP4_ERR_ALIGN;
    const size_t need = nvfp4::attn_cached_workspace_bytes(T, n_seqs, n_q_heads, c.hk, c.d);
    if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
    if (!workspace) return NVFP4_ERR_NULL;
    if (!aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
    const KvSpans s = kv_spans(c, r);
    if (clash({row_span(o, T, cols, ldo, 2), array_span(workspace, need)},
              {s.k, s.v, s.ks, s.vs, s.kg, s.vg, s.table, s.lens, s.cu, row_span(q, T, cols, ldq, 2),
               array_span(tree, 8 * (uint64_t)T)}))
      return NVFP4_ERR_ALIAS;
    return hip_status(nvfp4::launch_attn_cached(c, r, q, ldq, n_q_heads, scale, tree, o, ldo, workspace,
                                                (hipStream_t)stream));
  } catch (...) {
    return NVFP4_ERR_HIP;
  }
}

const char* nvfp4_status_string(int32_t status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_NULL: return "a required pointer is NULL";
    case NVFP4_ERR_SHAPE: return "invalid shape";
    case NVFP4_ERR_DTYPE: return "unknown dtype";
    case NVFP4_ERR_MODE: return "unknown scale mode";
    case NVFP4_ERR_ALIGN: return "misaligned pointer or row stride";
    case NVFP4_ERR_WORKSPACE: return "workspace too small";
    case NVFP4_ERR_HIP: return "HIP launch failed";
    case NVFP4_ERR_ALIAS: return "output overlaps an input that is still being read";
    case NVFP4_ERR_TOO_LARGE:
      return "the quantized activations need more than the static scratch of nvfp4_quantize_gemm_no_alloc "
             "(nvfp4_quantize_gemm_no_alloc_max_bytes())";
    default: return "unknown status";
  }
}

int32_t nvfp4_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
