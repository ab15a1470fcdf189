// C ABI of what a step has around the expert layer (RMS norm, balance loss of
// sequences, gradient norm): argument validation and the launches.
#include <string.h>

#include <algorithm>

#include "internal.h"

using moe::set_error;

#define REQUIRE(cond, code, ...)   \
  do {                             \
    if (!(cond)) {                 \
      set_error(__VA_ARGS__);      \
      return (code);               \
    }                              \
  } while (0)

static bool aligned(const void *p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

static moe_status_t cuda_status(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return MOE_OK;
  set_error("%s: %s", what, cudaGetErrorString(e));
  return MOE_ERR_CUDA;
}

static bool good_dtype(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }

// A leading dimension of `dtype` rows whose every row starts on 16 bytes.
static bool whole_rows(int64_t ld, int dtype) { return ld % (dtype == MOE_DTYPE_F32 ? 4 : 8) == 0; }

static moe_status_t check_norm(const char *who, int64_t rows, int cols, int stream_dtype,
                               const void *w, int w_dtype, float eps) {
  REQUIRE(rows >= 0 && cols > 0, MOE_ERR_INVALID_ARG, "%s: rows=%lld cols=%d", who, (long long)rows,
          cols);
  REQUIRE(good_dtype(stream_dtype) && good_dtype(w_dtype), MOE_ERR_INVALID_ARG,
          "%s: bad stream_dtype %d or w_dtype %d", who, stream_dtype, w_dtype);
  REQUIRE(eps > 0.0f && eps <= 1.0f, MOE_ERR_INVALID_ARG, "%s: eps=%g outside (0, 1]", who, eps);
  REQUIRE(cols % 8 == 0 && cols <= 16384, MOE_ERR_UNSUPPORTED,
          "%s: cols=%d is no multiple of 8 up to 16384", who, cols);
  REQUIRE(rows < (1ll << 31), MOE_ERR_UNSUPPORTED, "%s: rows of 2^31 and more", who);
  REQUIRE(w != nullptr, MOE_ERR_INVALID_ARG, "%s: null w", who);
  REQUIRE(aligned(w, 16), MOE_ERR_UNSUPPORTED, "%s: w must be 16-byte aligned", who);
  return MOE_OK;
}

// A matrix operand: given or not, its leading dimension and alignment.
static moe_status_t check_rows(const char *who, const char *name, const void *p, int64_t ld, int cols,
                               int dtype) {
  if (p == nullptr) return MOE_OK;
  REQUIRE(ld >= cols, MOE_ERR_INVALID_ARG, "%s: leading dimension of %s under %d", who, name, cols);
  REQUIRE(whole_rows(ld, dtype) && aligned(p, 16), MOE_ERR_UNSUPPORTED,
          "%s: rows of %s must start on 16 bytes", who, name);
  return MOE_OK;
}

#define CHECK(expr)                     \
  do {                                  \
    const moe_status_t st_ = (expr);    \
    if (st_ != MOE_OK) return st_;      \
  } while (0)

// ---------------------------------------------------------------- gradient clipping
static int64_t elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Elements of a chunk (a warp's piece): a step of the walk (1024 of fp32, 2048 of bf16) or two where
// there are few in all, so that every warp gets some; 8192 where each gets several, for fewer reads of
// the plan.  Clipping calls back to back, us a call, bf16 gradients written as bf16 / as fp32:
//   elements   chunks of 1024   of 2048       of 8192
//   1M           6.2 /  6.3     6.1 /  6.6    10.6 / 11.3
//   4M           9.0 / 11.0     7.9 / 10.6    10.8 / 13.2
//   16.8M       24.3 / 27.3    20.6 / 25.1    20.1 / 24.8
//   24M                        24.6 / 31.6    29.3 / 38.8 (one chunk for some warps, two for others)
//   32M         42.8 / 49.6    34.0 / 43.6    33.9 / 45.0
static int64_t chunk_elems(const moe_grad *grads, int n) {
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += std::max<int64_t>(0, grads[i].n);
  return all < (1ll << 21) ? 1024 : all < (1ll << 25) ? 2048 : 8192;
}

// Elements before the first where 8 of them start on their own size (16 or 32 bytes) in g and in
// out, or, if there is none (`apart`), where g starts on 16 bytes.
static int64_t peel(const moe_grad &t, bool *apart) {
  const int64_t gb = elem_bytes(t.g_dtype), ob = elem_bytes(t.out_dtype);
  const uintptr_t g = reinterpret_cast<uintptr_t>(t.g), out = reinterpret_cast<uintptr_t>(t.out);
  *apart = false;
  for (int64_t p = 0; p < 8; ++p)
    if ((g + p * gb) % (8 * gb) == 0 && (out + p * ob) % (8 * ob) == 0) return std::min(p, t.n);
  *apart = true;
  return std::min<int64_t>((16 - g % 16) % 16 / gb, t.n);
}

static moe_status_t check_grads(const char *who, const moe_grad *grads, int n) {
  REQUIRE(n >= 0 && (n == 0 || grads), MOE_ERR_INVALID_ARG, "%s: %d tensors", who, n);
  for (int i = 0; i < n; ++i) {
    const moe_grad &t = grads[i];
    REQUIRE(t.n >= 0 && good_dtype(t.g_dtype) && good_dtype(t.out_dtype), MOE_ERR_INVALID_ARG,
            "%s: tensor %d of %lld elements, types %d and %d", who, i, (long long)t.n, t.g_dtype,
            t.out_dtype);
    REQUIRE(t.n == 0 || (t.g && t.out), MOE_ERR_INVALID_ARG, "%s: tensor %d is null", who, i);
    REQUIRE(reinterpret_cast<uintptr_t>(t.g) % elem_bytes(t.g_dtype) == 0 &&
                reinterpret_cast<uintptr_t>(t.out) % elem_bytes(t.out_dtype) == 0,
            MOE_ERR_UNSUPPORTED, "%s: tensor %d is not aligned to its elements", who, i);
    REQUIRE(t.n == 0 || t.g != t.out || t.g_dtype == t.out_dtype, MOE_ERR_INVALID_ARG,
            "%s: tensor %d in place with another type", who, i);
  }
  return MOE_OK;
}

template <typename F>
static int64_t each_chunk(const moe_grad *grads, int n, F f) {
  const int64_t size = chunk_elems(grads, n);
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const moe_grad &t = grads[i];
    bool apart;
    const int64_t p = peel(t, &apart);
    const int kind = (t.g_dtype == MOE_DTYPE_F32 ? 1 : 0) | (t.out_dtype == MOE_DTYPE_F32 ? 2 : 0);
    for (int64_t lo = 0; lo < t.n;) {
      const int64_t hi = std::min(t.n, lo < p ? p : lo + size);
      f(chunks++, t, lo, hi, kind | (lo < p ? 4 : apart ? 4 | 8 : 0));
      lo = hi;
    }
  }
  return chunks;
}

extern "C" {

moe_status_t moe_rms_norm(const uint16_t *x, int64_t ldx, const void *residual, int64_t ld_res,
                          int stream_dtype, int64_t rows, int cols, const void *w, int w_dtype,
                          float eps, void *h, int64_t ldh, uint16_t *y, int64_t ldy, int codes,
                          uint8_t *q, int64_t ldq, void *scales, int64_t lds, size_t scales_bytes,
                          moe_stream_t stream) {
  const char *who = "moe_rms_norm";
  set_error("");
  CHECK(check_norm(who, rows, cols, stream_dtype, w, w_dtype, eps));
  REQUIRE(codes == MOE_CODES_NONE || codes == MOE_CODES_MX || codes == MOE_CODES_ACT8,
          MOE_ERR_INVALID_ARG, "%s: bad codes %d", who, codes);
  REQUIRE(codes != MOE_CODES_MX || cols % 128 == 0, MOE_ERR_UNSUPPORTED,
          "%s: block-scaled codes need cols in multiples of 128, not %d", who, cols);
  if (rows == 0) return MOE_OK;
  REQUIRE(x || residual, MOE_ERR_INVALID_ARG, "%s: neither x nor residual", who);
  REQUIRE(y || codes != MOE_CODES_NONE, MOE_ERR_INVALID_ARG, "%s: neither y nor codes", who);
  CHECK(check_rows(who, "x", x, ldx, cols, MOE_DTYPE_BF16));
  CHECK(check_rows(who, "residual", residual, ld_res, cols, stream_dtype));
  CHECK(check_rows(who, "h", h, ldh, cols, stream_dtype));
  CHECK(check_rows(who, "y", y, ldy, cols, MOE_DTYPE_BF16));
  if (codes != MOE_CODES_NONE) {
    REQUIRE(q && scales, MOE_ERR_INVALID_ARG, "%s: null q or scales", who);
    REQUIRE(ldq >= cols, MOE_ERR_INVALID_ARG, "%s: leading dimension of q under %d", who, cols);
    const int of = codes == MOE_CODES_MX ? 16 : 8;  // as the readers of these codes ask
    REQUIRE(ldq % of == 0 && aligned(q, of), MOE_ERR_UNSUPPORTED,
            "%s: rows of q must start on %d bytes", who, of);
  }
  if (codes == MOE_CODES_MX) {
    const size_t need = moe_mx_scale_bytes(rows, cols, MOE_MX_ROWS_PLAIN, 1);
    REQUIRE(scales_bytes >= need, MOE_ERR_INVALID_ARG, "%s: scales of %zu bytes < %zu", who,
            scales_bytes, need);
    REQUIRE(aligned(scales, 16), MOE_ERR_UNSUPPORTED, "%s: scales must be 16-byte aligned", who);
  } else if (codes == MOE_CODES_ACT8) {
    const int nb = (cols + 31) / 32;
    REQUIRE(lds >= nb, MOE_ERR_INVALID_ARG, "%s: leading dimension of scales under %d", who, nb);
    REQUIRE(scales_bytes >= ((size_t)(rows - 1) * (size_t)lds + nb) * 2, MOE_ERR_INVALID_ARG,
            "%s: scales of %zu bytes for %lld rows", who, scales_bytes, (long long)rows);
    REQUIRE(aligned(scales, 2), MOE_ERR_UNSUPPORTED, "%s: scales must be 2-byte aligned", who);
  }
  const moe::RmsNormArgs a = {x, ldx, residual, ld_res, stream_dtype, rows, cols, w, w_dtype, eps,
                              h, ldh, y, ldy, codes, q, ldq, scales, lds};
  return cuda_status(moe::launch_rms_norm(a, (cudaStream_t)stream), "moe_rms_norm launch");
}

size_t moe_rms_norm_bwd_workspace_bytes(int64_t rows, int cols) {
  if (rows < 0 || rows >= (1ll << 31) || cols <= 0 || cols > 16384) return 0;
  return std::max<size_t>(16, moe::rms_norm_bwd_workspace_bytes(rows, cols));
}

moe_status_t moe_rms_norm_bwd(const uint16_t *dy, int64_t ld_dy, const void *h, int64_t ldh,
                              int stream_dtype, int64_t rows, int cols, const void *w, int w_dtype,
                              float eps, const void *d_residual, int64_t ld_dres, void *dh,
                              int64_t ld_dh, uint16_t *dx, int64_t ld_dx, float *dw, int accumulate,
                              void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  const char *who = "moe_rms_norm_bwd";
  set_error("");
  CHECK(check_norm(who, rows, cols, stream_dtype, w, w_dtype, eps));
  if (rows > 0) {
    REQUIRE(dy && h && dh, MOE_ERR_INVALID_ARG, "%s: null pointer", who);
    CHECK(check_rows(who, "dy", dy, ld_dy, cols, MOE_DTYPE_BF16));
    CHECK(check_rows(who, "h", h, ldh, cols, stream_dtype));
    CHECK(check_rows(who, "d_residual", d_residual, ld_dres, cols, stream_dtype));
    CHECK(check_rows(who, "dh", dh, ld_dh, cols, stream_dtype));
    CHECK(check_rows(who, "dx", dx, ld_dx, cols, MOE_DTYPE_BF16));
  }
  REQUIRE(aligned(dw, 4), MOE_ERR_UNSUPPORTED, "%s: dw must be 4-byte aligned", who);
  if (dw != nullptr && rows > 0) {
    const size_t need = moe::rms_norm_bwd_workspace_bytes(rows, cols);
    REQUIRE(workspace && workspace_bytes >= need, MOE_ERR_INVALID_ARG,
            "%s: workspace of %zu bytes < %zu", who, workspace_bytes, need);
    REQUIRE(aligned(workspace, 16), MOE_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", who);
  }
  const moe::RmsNormBwdArgs a = {dy, ld_dy, h, ldh, stream_dtype, rows, cols, w, w_dtype, eps,
                                 d_residual, ld_dres, dh, ld_dh, dx, ld_dx, dw, accumulate};
  float *part = dw == nullptr ? nullptr : static_cast<float *>(workspace);
  if (rows == 0 && dw == nullptr) return MOE_OK;
  return cuda_status(moe::launch_rms_norm_bwd(a, part, (cudaStream_t)stream), "moe_rms_norm_bwd launch");
}

moe_status_t moe_mx_dequantize(const uint8_t *q, int64_t ldq, const uint8_t *sf, size_t sf_bytes,
                               int64_t rows, int cols, int fmt, uint16_t *x, int64_t ldx,
                               moe_stream_t stream) {
  const char *who = "moe_mx_dequantize";
  set_error("");
  REQUIRE(rows >= 0 && cols > 0, MOE_ERR_INVALID_ARG, "%s: rows=%lld cols=%d", who, (long long)rows,
          cols);
  REQUIRE(fmt == MOE_FP8_E4M3 || fmt == MOE_FP8_E5M2, MOE_ERR_INVALID_ARG, "%s: bad fmt %d", who, fmt);
  REQUIRE(cols % 128 == 0 && rows < (1ll << 31) - (1 << 20), MOE_ERR_UNSUPPORTED,
          "%s: cols=%d is no multiple of 128, or rows of 2^31 and more", who, cols);
  if (rows == 0) return MOE_OK;
  REQUIRE(q && sf && x, MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  REQUIRE(ldq >= cols, MOE_ERR_INVALID_ARG, "%s: leading dimension of q under %d", who, cols);
  REQUIRE(ldq % 8 == 0 && aligned(q, 8), MOE_ERR_UNSUPPORTED, "%s: rows of q must start on 8 bytes", who);
  CHECK(check_rows(who, "x", x, ldx, cols, MOE_DTYPE_BF16));
  REQUIRE(sf_bytes >= moe_mx_scale_bytes(rows, cols, MOE_MX_ROWS_PLAIN, 1), MOE_ERR_INVALID_ARG,
          "%s: sf of %zu bytes < %zu", who, sf_bytes,
          moe_mx_scale_bytes(rows, cols, MOE_MX_ROWS_PLAIN, 1));
  return cuda_status(moe::launch_mx_dequantize(q, ldq, sf, rows, cols, fmt, x, ldx, (cudaStream_t)stream),
                     "moe_mx_dequantize launch");
}

size_t moe_seq_aux_loss_workspace_bytes(int T, int E, int B) {
  if (T < 0 || E <= 0 || E > 256 || B <= 0) return 0;
  return moe::seq_aux_workspace_bytes(T, E, B);
}

static moe_status_t check_seq(const char *who, int T, int E, int k, int B, int score_fn,
                              const float *logits, int64_t ld, const int32_t *offsets, float coeff,
                              float z_coeff) {
  REQUIRE(T >= 0 && E > 0 && k > 0 && k <= E && B > 0, MOE_ERR_INVALID_ARG,
          "%s: T=%d E=%d k=%d B=%d", who, T, E, k, B);
  REQUIRE(E <= 256 && k <= 16 && T <= (1 << 30) && B <= 65536, MOE_ERR_UNSUPPORTED,
          "%s: needs E <= 256, k <= 16, T <= 2^30, B <= 65536", who);
  REQUIRE(score_fn == MOE_SCORE_SOFTMAX || score_fn == MOE_SCORE_SIGMOID, MOE_ERR_INVALID_ARG,
          "%s: bad score_fn %d", who, score_fn);
  REQUIRE(ld >= E, MOE_ERR_INVALID_ARG, "%s: ld_logits < E", who);
  REQUIRE(offsets && (T == 0 || logits), MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  REQUIRE(coeff - coeff == 0.0f && z_coeff - z_coeff == 0.0f, MOE_ERR_INVALID_ARG,
          "%s: coefficients must be finite", who);
  return MOE_OK;
}

moe_status_t moe_seq_aux_loss(const float *logits, int64_t ld_logits, int T, int E, int k,
                              int score_fn, const int32_t *topk_idx, const int32_t *seq_offsets, int B,
                              const uint8_t *token_mask, float coeff, float z_coeff, int32_t *counts,
                              int32_t *tokens, float *probs_mean, float *loss, float d_loss,
                              float *d_logits, int64_t ld_dlogits, int accumulate, void *workspace,
                              size_t workspace_bytes, moe_stream_t stream) {
  const char *who = "moe_seq_aux_loss";
  set_error("");
  CHECK(check_seq(who, T, E, k, B, score_fn, logits, ld_logits, seq_offsets, coeff, z_coeff));
  REQUIRE((T == 0 || topk_idx) && counts && tokens && probs_mean && loss, MOE_ERR_INVALID_ARG,
          "%s: null pointer", who);
  REQUIRE(d_logits == nullptr || ld_dlogits >= E, MOE_ERR_INVALID_ARG, "%s: ld_dlogits < E", who);
  REQUIRE(d_logits == nullptr || d_logits != logits, MOE_ERR_INVALID_ARG, "%s: d_logits are logits", who);
  REQUIRE(workspace && workspace_bytes >= moe::seq_aux_workspace_bytes(T, E, B), MOE_ERR_INVALID_ARG,
          "%s: workspace of %zu bytes < %zu", who, workspace_bytes,
          moe::seq_aux_workspace_bytes(T, E, B));
  REQUIRE(aligned(workspace, 4), MOE_ERR_UNSUPPORTED, "%s: workspace must be 4-byte aligned", who);
  const moe::SeqAuxArgs a = {logits, ld_logits, T, E, k, score_fn, topk_idx, seq_offsets, B, token_mask,
                             coeff, z_coeff, counts, tokens, probs_mean, loss, d_loss, d_logits,
                             ld_dlogits, accumulate};
  return cuda_status(moe::launch_seq_aux(a, workspace, (cudaStream_t)stream), "moe_seq_aux_loss launch");
}

moe_status_t moe_seq_aux_loss_bwd(const float *logits, int64_t ld_logits, int T, int E, int k,
                                  int score_fn, const int32_t *seq_offsets, int B,
                                  const uint8_t *token_mask, float coeff, float z_coeff,
                                  const int32_t *counts, const int32_t *tokens, float d_loss,
                                  float *d_logits, int64_t ld_dlogits, int accumulate,
                                  moe_stream_t stream) {
  const char *who = "moe_seq_aux_loss_bwd";
  set_error("");
  CHECK(check_seq(who, T, E, k, B, score_fn, logits, ld_logits, seq_offsets, coeff, z_coeff));
  REQUIRE(counts && tokens && (T == 0 || d_logits), MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  REQUIRE(ld_dlogits >= E, MOE_ERR_INVALID_ARG, "%s: ld_dlogits < E", who);
  REQUIRE(d_logits == nullptr || d_logits != logits, MOE_ERR_INVALID_ARG, "%s: d_logits are logits", who);
  const moe::SeqAuxArgs a = {logits, ld_logits, T, E, k, score_fn, nullptr, seq_offsets, B, token_mask,
                             coeff, z_coeff, const_cast<int32_t *>(counts), const_cast<int32_t *>(tokens),
                             nullptr, nullptr, d_loss, d_logits, ld_dlogits, accumulate};
  return cuda_status(moe::launch_seq_aux(a, nullptr, (cudaStream_t)stream), "moe_seq_aux_loss_bwd launch");
}

int64_t moe_clip_plan_chunks(const moe_grad *grads, int n) {
  set_error("");
  if (check_grads("moe_clip_plan_chunks", grads, n) != MOE_OK) return -1;
  return each_chunk(grads, n, [](int64_t, const moe_grad &, int64_t, int64_t, int) {});
}

moe_status_t moe_clip_plan(const moe_grad *grads, int n, void *plan, size_t plan_bytes) {
  set_error("");
  CHECK(check_grads("moe_clip_plan", grads, n));
  const int64_t chunks = moe_clip_plan_chunks(grads, n);
  REQUIRE(plan_bytes >= (size_t)chunks * sizeof(moe::ClipChunk) && (plan || chunks == 0),
          MOE_ERR_INVALID_ARG, "moe_clip_plan: %zu bytes for %lld chunks", plan_bytes, (long long)chunks);
  char *to = static_cast<char *>(plan);  // (of any alignment here)
  each_chunk(grads, n, [to](int64_t k, const moe_grad &t, int64_t lo, int64_t hi, int kind) {
    moe::ClipChunk c = {};
    c.g = static_cast<const char *>(t.g) + lo * elem_bytes(t.g_dtype);
    c.out = static_cast<char *>(t.out) + lo * elem_bytes(t.out_dtype);
    c.n = (int32_t)(hi - lo);
    c.kind = kind;
    memcpy(to + k * sizeof c, &c, sizeof c);
  });
  return MOE_OK;
}

size_t moe_clip_workspace_bytes(void) { return moe::kClipMaxBlocks * sizeof(double); }

static moe_status_t run_clip(const char *who, const void *plan, int64_t chunks, float scale,
                             float max_norm, bool write, float *norm, void *workspace,
                             size_t workspace_bytes, moe_stream_t stream) {
  set_error("");
  REQUIRE(chunks >= 0 && (chunks == 0 || plan) && norm && workspace, MOE_ERR_INVALID_ARG,
          "%s: null pointer, or %lld chunks", who, (long long)chunks);
  REQUIRE(scale > 0.0f && scale <= 3.402823466e38f, MOE_ERR_INVALID_ARG, "%s: scale=%g", who, scale);
  REQUIRE(!write || max_norm >= 0.0f, MOE_ERR_INVALID_ARG, "%s: max_norm=%g", who, max_norm);
  REQUIRE(workspace_bytes >= moe_clip_workspace_bytes(), MOE_ERR_INVALID_ARG,
          "%s: workspace of %zu bytes < %zu", who, workspace_bytes, moe_clip_workspace_bytes());
  REQUIRE(aligned(plan, 16) && aligned(workspace, 8) && aligned(norm, 4), MOE_ERR_UNSUPPORTED,
          "%s: plan must be 16-byte, workspace 8-byte, norm 4-byte aligned", who);
  return cuda_status(moe::launch_clip(static_cast<const moe::ClipChunk *>(plan), chunks, scale, max_norm,
                                      write, norm, static_cast<double *>(workspace),
                                      (cudaStream_t)stream),
                     who);
}

moe_status_t moe_grad_norm(const void *plan, int64_t chunks, float scale, float *norm, void *workspace,
                           size_t workspace_bytes, moe_stream_t stream) {
  return run_clip("moe_grad_norm", plan, chunks, scale, 0.0f, false, norm, workspace, workspace_bytes,
                  stream);
}

moe_status_t moe_clip_grads(const void *plan, int64_t chunks, float max_norm, float scale, float *norm,
                            void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  return run_clip("moe_clip_grads", plan, chunks, scale, max_norm, true, norm, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
