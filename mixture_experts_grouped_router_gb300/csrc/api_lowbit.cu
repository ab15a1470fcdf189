// C ABI of the low-bit operators (4-bit block-scaled formats, 8-bit activation
// checkpoints): argument validation and the launches.
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

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

// Rows and leading dimensions that the kernels index in 32 bits (offsets are 64).
static bool fits(int64_t rows, int64_t a, int64_t b = 0, int64_t c = 0, int64_t d = 0) {
  const int64_t most = (1ll << 31) - (1 << 20);
  return rows < most && a < most && b < most && c < most && d < most;
}

static bool good_fmt(int fmt) { return fmt == MOE_FP4_MX || fmt == MOE_FP4_NV; }

static bool good_map(int m) {
  return m == MOE_FP4_ROWS_GROUPED || m == MOE_FP4_ROWS_EXPERTS || m == MOE_FP4_ROWS_SWIGLU;
}

// Rows of a quantised matrix: groups, and what their map asks of them.
static moe_status_t check_rows(const char *who, int64_t rows, int cols, int fmt, int row_map,
                               const int32_t *offsets, int E) {
  REQUIRE(rows >= 0 && cols > 0 && E > 0, MOE_ERR_INVALID_ARG, "%s: rows=%lld cols=%d E=%d", who,
          (long long)rows, cols, E);
  REQUIRE(good_fmt(fmt), MOE_ERR_INVALID_ARG, "%s: bad fmt %d", who, fmt);
  REQUIRE(good_map(row_map), MOE_ERR_INVALID_ARG, "%s: bad row_map %d", who, row_map);
  REQUIRE(cols % 32 == 0, MOE_ERR_UNSUPPORTED, "%s: cols=%d is no multiple of 32", who, cols);
  REQUIRE(fits(rows + 128ll * E, 0), MOE_ERR_UNSUPPORTED, "%s: too many rows (2^31)", who);
  if (row_map == MOE_FP4_ROWS_GROUPED) {
    REQUIRE(E <= 256, MOE_ERR_UNSUPPORTED, "%s: E=%d > 256", who, E);
    REQUIRE(offsets != nullptr || rows == 0, MOE_ERR_INVALID_ARG,
            "%s: GROUPED needs group_offsets", who);
  } else {
    REQUIRE(rows % E == 0, MOE_ERR_INVALID_ARG, "%s: rows=%lld are no E=%d equal groups", who,
            (long long)rows, E);
    REQUIRE(row_map != MOE_FP4_ROWS_SWIGLU || rows / E % 64 == 0, MOE_ERR_UNSUPPORTED,
            "%s: SWIGLU needs 2F rows an expert, F a multiple of 32", who);
  }
  return MOE_OK;
}

extern "C" {

size_t moe_fp4_scale_bytes(int64_t rows, int cols, int fmt, int row_map, int E) {
  if (rows < 0 || cols <= 0 || E <= 0 || !good_fmt(fmt) || !good_map(row_map)) return 0;
  const int ac = moe::fp4_atom_cols(fmt);
  return (size_t)moe::fp4_atom_rows(rows, row_map, E) * (size_t)((cols + ac - 1) / ac) * 512u;
}

size_t moe_fp4_quantize_workspace_bytes(int64_t src_rows, int64_t rows) {
  if (src_rows < 0 || rows < 0) return 0;
  return moe::fp4_quantize_workspace_bytes(src_rows, rows);
}

moe_status_t moe_fp4_quantize(const uint16_t *x, int64_t ldx, int64_t src_rows,
                              const int32_t *row_index, int index_div, int64_t rows, int cols,
                              int fmt, int row_map, const int32_t *group_offsets, int E,
                              const float *scale, uint8_t *q, int64_t ldq, uint8_t *sf,
                              size_t sf_bytes, void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, moe_stream_t stream) {
  set_error("");
  const moe_status_t st =
      check_rows("moe_fp4_quantize", rows, cols, fmt, row_map, group_offsets, E);
  if (st != MOE_OK) return st;
  REQUIRE(ldx >= cols && ldq >= cols / 2, MOE_ERR_INVALID_ARG,
          "moe_fp4_quantize: leading dimension too small");
  REQUIRE(ldx % 8 == 0 && ldq % 16 == 0, MOE_ERR_UNSUPPORTED,
          "moe_fp4_quantize: ldx must be a multiple of 8, ldq of 16");
  REQUIRE(fits(src_rows, ldx, ldq), MOE_ERR_UNSUPPORTED,
          "moe_fp4_quantize: src_rows, ldx or ldq of 2^31 and more");
  REQUIRE(src_rows >= 0 && (row_index == nullptr ? src_rows >= rows : index_div > 0),
          MOE_ERR_INVALID_ARG, "moe_fp4_quantize: src_rows=%lld index_div=%d",
          (long long)src_rows, index_div);
  if (rows == 0) return MOE_OK;
  REQUIRE((x || src_rows == 0) && q && sf, MOE_ERR_INVALID_ARG, "moe_fp4_quantize: null pointer");
  REQUIRE(aligned(x, 16) && aligned(q, 16) && aligned(sf, 16) && aligned(workspace, 16),
          MOE_ERR_UNSUPPORTED, "moe_fp4_quantize: x, q, sf and workspace must be 16-byte aligned");
  REQUIRE(sf_bytes >= moe_fp4_scale_bytes(rows, cols, fmt, row_map, E), MOE_ERR_INVALID_ARG,
          "moe_fp4_quantize: sf of %zu bytes < %zu", sf_bytes,
          moe_fp4_scale_bytes(rows, cols, fmt, row_map, E));
  return cuda_status(
      moe::launch_fp4_quantize(x, ldx, src_rows, row_index, index_div, rows, cols, fmt, row_map,
                               group_offsets, E, scale, q, ldq, sf, workspace, workspace_bytes,
                               dev_status, (cudaStream_t)stream),
      "moe_fp4_quantize launch");
}

moe_status_t moe_fp4_dequantize(const uint8_t *q, int64_t ldq, const uint8_t *sf, size_t sf_bytes,
                                int64_t rows, int cols, int fmt, int row_map,
                                const int32_t *group_offsets, int E, const float *scale,
                                uint16_t *x, int64_t ldx, moe_stream_t stream) {
  set_error("");
  const moe_status_t st =
      check_rows("moe_fp4_dequantize", rows, cols, fmt, row_map, group_offsets, E);
  if (st != MOE_OK) return st;
  REQUIRE(ldx >= cols && ldq >= cols / 2, MOE_ERR_INVALID_ARG,
          "moe_fp4_dequantize: leading dimension too small");
  REQUIRE(ldx % 8 == 0 && ldq % 16 == 0, MOE_ERR_UNSUPPORTED,
          "moe_fp4_dequantize: ldx must be a multiple of 8, ldq of 16");
  REQUIRE(fits(0, ldx, ldq), MOE_ERR_UNSUPPORTED, "moe_fp4_dequantize: ldx or ldq of 2^31 and more");
  if (rows == 0) return MOE_OK;
  REQUIRE(x && q && sf, MOE_ERR_INVALID_ARG, "moe_fp4_dequantize: null pointer");
  REQUIRE(aligned(x, 16) && aligned(q, 16) && aligned(sf, 16), MOE_ERR_UNSUPPORTED,
          "moe_fp4_dequantize: x, q and sf must be 16-byte aligned");
  REQUIRE(sf_bytes >= moe_fp4_scale_bytes(rows, cols, fmt, row_map, E), MOE_ERR_INVALID_ARG,
          "moe_fp4_dequantize: sf of %zu bytes < %zu", sf_bytes,
          moe_fp4_scale_bytes(rows, cols, fmt, row_map, E));
  return cuda_status(moe::launch_fp4_dequantize(q, ldq, sf, rows, cols, fmt, row_map,
                                                group_offsets, E, scale, x, ldx,
                                                (cudaStream_t)stream),
                     "moe_fp4_dequantize launch");
}

moe_status_t moe_fp4_quantize_weights(const uint16_t *w, int E, int K, int N, int fmt, int row_map,
                                      const float *scale, uint8_t *q, uint8_t *sf,
                                      size_t sf_bytes, moe_stream_t stream) {
  set_error("");
  REQUIRE(row_map != MOE_FP4_ROWS_GROUPED, MOE_ERR_INVALID_ARG,
          "moe_fp4_quantize_weights: row_map must be EXPERTS or SWIGLU");
  REQUIRE(N > 0, MOE_ERR_INVALID_ARG, "moe_fp4_quantize_weights: N=%d", N);
  const moe_status_t st = check_rows("moe_fp4_quantize_weights", (int64_t)std::max(E, 0) * N, K,
                                     fmt, row_map, nullptr, E);
  if (st != MOE_OK) return st;
  REQUIRE(E <= 65535 && K <= 65535 * 64 && fits((int64_t)E * ((N + 127) / 128 * 128), 0),
          MOE_ERR_UNSUPPORTED,
          "moe_fp4_quantize_weights: E=%d K=%d", E, K);
  REQUIRE(w && q && sf, MOE_ERR_INVALID_ARG, "moe_fp4_quantize_weights: null pointer");
  REQUIRE(aligned(w, 2) && aligned(q, 16) && aligned(sf, 16), MOE_ERR_UNSUPPORTED,
          "moe_fp4_quantize_weights: q and sf must be 16-byte aligned");
  REQUIRE(sf_bytes >= moe_fp4_scale_bytes((int64_t)E * N, K, fmt, row_map, E),
          MOE_ERR_INVALID_ARG, "moe_fp4_quantize_weights: sf of %zu bytes < %zu", sf_bytes,
          moe_fp4_scale_bytes((int64_t)E * N, K, fmt, row_map, E));
  return cuda_status(moe::launch_fp4_quantize_weights(w, E, K, N, fmt, row_map, scale, q, sf,
                                                      (cudaStream_t)stream),
                     "moe_fp4_quantize_weights launch");
}

moe_status_t moe_fp4_arrange_scales(const uint8_t *scales, int64_t rows, int cols, int fmt,
                                    int row_map, int E, uint8_t *sf, size_t sf_bytes,
                                    moe_stream_t stream) {
  set_error("");
  REQUIRE(row_map != MOE_FP4_ROWS_GROUPED, MOE_ERR_INVALID_ARG,
          "moe_fp4_arrange_scales: row_map must be EXPERTS or SWIGLU");
  const moe_status_t st =
      check_rows("moe_fp4_arrange_scales", rows, cols, fmt, row_map, nullptr, E);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  REQUIRE(scales && sf, MOE_ERR_INVALID_ARG, "moe_fp4_arrange_scales: null pointer");
  REQUIRE(aligned(sf, 16), MOE_ERR_UNSUPPORTED,
          "moe_fp4_arrange_scales: sf must be 16-byte aligned");
  REQUIRE(sf_bytes >= moe_fp4_scale_bytes(rows, cols, fmt, row_map, E), MOE_ERR_INVALID_ARG,
          "moe_fp4_arrange_scales: sf of %zu bytes < %zu", sf_bytes,
          moe_fp4_scale_bytes(rows, cols, fmt, row_map, E));
  return cuda_status(moe::launch_fp4_arrange_scales(scales, rows, cols / moe::fp4_block(fmt), E,
                                                    row_map, sf, (cudaStream_t)stream),
                     "moe_fp4_arrange_scales launch");
}

moe_status_t moe_gmm_fp4(const uint8_t *A, int64_t lda, const uint8_t *sfa, const float *a_scale,
                         const uint8_t *B, int64_t ldb, int64_t stride_b, const uint8_t *sfb,
                         const float *b_scale, int fmt, const int32_t *group_offsets, int E,
                         int64_t rows_cap, int K, int N, int epilogue, void *C, int c_dtype,
                         int64_t ldc, uint8_t *Q2, int64_t ldq2, uint8_t *sf2, size_t sf2_bytes,
                         const float *q2_scale, int32_t *dev_status, moe_stream_t stream) {
  set_error("");
  REQUIRE(E > 0 && rows_cap >= 0 && K > 0 && N > 0, MOE_ERR_INVALID_ARG,
          "moe_gmm_fp4: E=%d rows_cap=%lld K=%d N=%d", E, (long long)rows_cap, K, N);
  REQUIRE(E <= 256, MOE_ERR_UNSUPPORTED, "moe_gmm_fp4: E=%d > 256", E);
  REQUIRE(good_fmt(fmt), MOE_ERR_INVALID_ARG, "moe_gmm_fp4: bad fmt %d", fmt);
  REQUIRE(epilogue == MOE_EPI_NONE || epilogue == MOE_EPI_SWIGLU_FWD, MOE_ERR_INVALID_ARG,
          "moe_gmm_fp4: bad epilogue %d", epilogue);
  REQUIRE(c_dtype == MOE_DTYPE_BF16 || c_dtype == MOE_DTYPE_F32, MOE_ERR_INVALID_ARG,
          "moe_gmm_fp4: bad c_dtype %d", c_dtype);
  REQUIRE(K % 32 == 0 && N % 8 == 0 && lda % 16 == 0 && ldb % 16 == 0 && stride_b % 16 == 0,
          MOE_ERR_UNSUPPORTED,
          "moe_gmm_fp4: K must be a multiple of 32, N of 8, lda, ldb and stride_b of 16 bytes");
  REQUIRE(lda >= K / 2 && ldb >= K / 2 && (E == 1 || stride_b >= (int64_t)N * ldb),
          MOE_ERR_INVALID_ARG, "moe_gmm_fp4: lda, ldb or stride_b too small");
  const bool swiglu = epilogue == MOE_EPI_SWIGLU_FWD;
  const int es = c_dtype == MOE_DTYPE_F32 ? 4 : 2;
  REQUIRE((C == nullptr && swiglu) || (ldc >= N && ldc * es % 16 == 0), MOE_ERR_INVALID_ARG,
          "moe_gmm_fp4: ldc=%lld (>= N=%d, rows of whole 16 bytes)", (long long)ldc, N);
  // padded row tiles are counted in 16 bits
  REQUIRE(rows_cap + 128ll * E < (1ll << 23), MOE_ERR_UNSUPPORTED,
          "moe_gmm_fp4: rows_cap=%lld E=%d: more than 2^23 padded rows", (long long)rows_cap, E);
  if (swiglu) {
    REQUIRE(N % 64 == 0, MOE_ERR_UNSUPPORTED, "moe_gmm_fp4: SWIGLU_FWD needs N = 2F, F %% 32 == 0");
    REQUIRE(c_dtype == MOE_DTYPE_BF16, MOE_ERR_INVALID_ARG, "moe_gmm_fp4: SWIGLU_FWD: H is bf16");
    REQUIRE(ldq2 >= N / 4 && ldq2 % 16 == 0, MOE_ERR_INVALID_ARG,
            "moe_gmm_fp4: ldq2=%lld (>= F / 2 = %d bytes, multiple of 16)", (long long)ldq2, N / 4);
  }
  if (rows_cap == 0) return MOE_OK;
  REQUIRE(A && sfa && B && sfb && group_offsets && (swiglu ? Q2 && sf2 : C != nullptr),
          MOE_ERR_INVALID_ARG, "moe_gmm_fp4: null pointer");
  REQUIRE(aligned(A, 16) && aligned(B, 16) && aligned(sfa, 16) && aligned(sfb, 16) &&
              aligned(C, 16) && aligned(Q2, 16) && aligned(sf2, 16),
          MOE_ERR_UNSUPPORTED, "moe_gmm_fp4: operands must be 16-byte aligned");
  REQUIRE(!swiglu || sf2_bytes >= moe_fp4_scale_bytes(rows_cap, N / 2, fmt, MOE_FP4_ROWS_GROUPED, E),
          MOE_ERR_INVALID_ARG, "moe_gmm_fp4: sf2 of %zu bytes < %zu", sf2_bytes,
          moe_fp4_scale_bytes(rows_cap, N / 2, fmt, MOE_FP4_ROWS_GROUPED, E));
  moe::GmmFp4Args a{A, lda, sfa, a_scale, B, ldb, stride_b, sfb, b_scale, fmt, group_offsets, E,
                    rows_cap, K, N, epilogue, C, c_dtype, ldc, Q2, ldq2, sf2, q2_scale,
                    dev_status, 0};
  return moe::launch_gmm_fp4(a, (cudaStream_t)stream);
}

moe_status_t moe_fp4_experts(const moe_fp4_weights *w, const moe_fp4_buffers *b,
                             const uint16_t *x, int64_t ldx, int T, const int32_t *sorted_to_flat,
                             int k, const int32_t *group_offsets, moe_stream_t stream) {
  set_error("");
  REQUIRE(w != nullptr && b != nullptr, MOE_ERR_INVALID_ARG, "moe_fp4_experts: null pointer");
  REQUIRE(w->E > 0 && w->d > 0 && w->f > 0 && T >= 0 && k > 0 && b->rows_cap >= 0,
          MOE_ERR_INVALID_ARG, "moe_fp4_experts: E=%d d=%d f=%d T=%d k=%d rows_cap=%lld", w->E,
          w->d, w->f, T, k, (long long)b->rows_cap);
  // everything is checked before the first launch: the three calls repeat only
  // what these do not cover
  REQUIRE(good_fmt(w->fmt), MOE_ERR_INVALID_ARG, "moe_fp4_experts: bad fmt %d", w->fmt);
  REQUIRE(w->d % 32 == 0 && w->f % 32 == 0 && w->E <= 256, MOE_ERR_UNSUPPORTED,
          "moe_fp4_experts: d=%d and f=%d must be multiples of 32, E=%d at most 256", w->d, w->f,
          w->E);
  REQUIRE(b->rows_cap + 128ll * w->E < (1ll << 23), MOE_ERR_UNSUPPORTED,
          "moe_fp4_experts: rows_cap=%lld E=%d: more than 2^23 padded rows",
          (long long)b->rows_cap, w->E);
  if (b->rows_cap == 0) return MOE_OK;
  REQUIRE(w->wi_q && w->wi_sf && w->wo_q && w->wo_sf && b->x_q && b->x_sf && b->act_q &&
              b->act_sf && b->y && (x || T == 0) && sorted_to_flat && group_offsets,
          MOE_ERR_INVALID_ARG, "moe_fp4_experts: null pointer");
  REQUIRE(aligned(w->wi_q, 16) && aligned(w->wi_sf, 16) && aligned(w->wo_q, 16) &&
              aligned(w->wo_sf, 16) && aligned(b->x_q, 16) && aligned(b->x_sf, 16) &&
              aligned(b->act_q, 16) && aligned(b->act_sf, 16) && aligned(b->y, 16) &&
              aligned(b->h, 16) && aligned(b->workspace, 16) && aligned(x, 16) && ldx % 8 == 0,
          MOE_ERR_UNSUPPORTED, "moe_fp4_experts: operands must be 16-byte aligned");
  REQUIRE(fits(T, ldx), MOE_ERR_UNSUPPORTED, "moe_fp4_experts: T or ldx of 2^31 and more");
  REQUIRE(ldx >= w->d, MOE_ERR_INVALID_ARG, "moe_fp4_experts: ldx=%lld < d", (long long)ldx);
  REQUIRE(b->x_sf_bytes >=
                  moe_fp4_scale_bytes(b->rows_cap, w->d, w->fmt, MOE_FP4_ROWS_GROUPED, w->E) &&
              b->act_sf_bytes >=
                  moe_fp4_scale_bytes(b->rows_cap, w->f, w->fmt, MOE_FP4_ROWS_GROUPED, w->E),
          MOE_ERR_INVALID_ARG, "moe_fp4_experts: scale buffers too small");
  cudaStream_t s = (cudaStream_t)stream;
  moe_status_t st = cuda_status(
      moe::launch_fp4_quantize(x, ldx, T, sorted_to_flat, k, b->rows_cap, w->d, w->fmt,
                               MOE_FP4_ROWS_GROUPED, group_offsets, w->E, w->x_scale, b->x_q,
                               w->d / 2, b->x_sf, b->workspace, b->workspace_bytes, b->dev_status,
                               s),
      "moe_fp4_experts: quantise");
  if (st != MOE_OK) return st;
  const int64_t d2 = w->d / 2, f2 = w->f / 2;
  moe::GmmFp4Args up{b->x_q, d2, b->x_sf, w->x_scale, w->wi_q, d2, 2ll * w->f * d2, w->wi_sf,
                     w->wi_scale, w->fmt, group_offsets, w->E, b->rows_cap, w->d, 2 * w->f,
                     MOE_EPI_SWIGLU_FWD, b->h, MOE_DTYPE_BF16, 2ll * w->f, b->act_q, f2, b->act_sf,
                     w->act_scale, b->dev_status, 1};
  st = moe::launch_gmm_fp4(up, s);
  if (st != MOE_OK) return st;
  moe::GmmFp4Args down{b->act_q, f2, b->act_sf, w->act_scale, w->wo_q, f2, (int64_t)w->d * f2,
                       w->wo_sf, w->wo_scale, w->fmt, group_offsets, w->E, b->rows_cap, w->f, w->d,
                       MOE_EPI_NONE, b->y, MOE_DTYPE_BF16, w->d, nullptr, 0, nullptr, nullptr,
                       b->dev_status, 1};
  return moe::launch_gmm_fp4(down, s);
}

// ------------------------------------------------- 8-bit activation checkpoints
static moe_status_t check_act8(const char *who, int64_t rows, int cols, const int32_t *offsets,
                               int E, int64_t ldq, int64_t need_q, int64_t lds, int64_t need_s) {
  REQUIRE(rows >= 0 && cols > 0 && (offsets == nullptr || E > 0), MOE_ERR_INVALID_ARG,
          "%s: rows=%lld cols=%d E=%d", who, (long long)rows, cols, E);
  REQUIRE(cols % 8 == 0, MOE_ERR_UNSUPPORTED, "%s: cols=%d is no multiple of 8", who, cols);
  REQUIRE(ldq >= need_q && lds >= need_s, MOE_ERR_INVALID_ARG,
          "%s: ldq=%lld (>= %lld) or lds=%lld (>= %lld) too small", who, (long long)ldq,
          (long long)need_q, (long long)lds, (long long)need_s);
  REQUIRE(ldq % 8 == 0, MOE_ERR_UNSUPPORTED, "%s: ldq must be a multiple of 8", who);
  REQUIRE(fits(rows, ldq, lds), MOE_ERR_UNSUPPORTED, "%s: rows, ldq or lds of 2^31 and more", who);
  return MOE_OK;
}

moe_status_t moe_act8_quantize(const uint16_t *x, int64_t ldx, int64_t rows, int cols,
                               const int32_t *group_offsets, int E, int8_t *q, int64_t ldq,
                               uint16_t *scales, int64_t lds, moe_stream_t stream) {
  set_error("");
  const moe_status_t st = check_act8("moe_act8_quantize", rows, cols, group_offsets, E, ldq, cols,
                                     lds, (cols + 31) / 32);
  if (st != MOE_OK) return st;
  REQUIRE(ldx >= cols, MOE_ERR_INVALID_ARG, "moe_act8_quantize: ldx too small");
  REQUIRE(ldx % 8 == 0 && fits(0, ldx), MOE_ERR_UNSUPPORTED,
          "moe_act8_quantize: ldx must be a multiple of 8 under 2^31");
  if (rows == 0) return MOE_OK;
  REQUIRE(x && q && scales, MOE_ERR_INVALID_ARG, "moe_act8_quantize: null pointer");
  REQUIRE(aligned(x, 16) && aligned(q, 8) && aligned(scales, 2), MOE_ERR_UNSUPPORTED,
          "moe_act8_quantize: x must be 16-byte, q 8-byte aligned");
  return cuda_status(moe::launch_act8_quantize(x, ldx, rows, cols, group_offsets, E, q, ldq,
                                               scales, lds, (cudaStream_t)stream),
                     "moe_act8_quantize launch");
}

moe_status_t moe_act8_dequantize(const int8_t *q, int64_t ldq, const uint16_t *scales, int64_t lds,
                                 int64_t rows, int cols, const int32_t *group_offsets, int E,
                                 uint16_t *x, int64_t ldx, moe_stream_t stream) {
  set_error("");
  const moe_status_t st = check_act8("moe_act8_dequantize", rows, cols, group_offsets, E, ldq,
                                     cols, lds, (cols + 31) / 32);
  if (st != MOE_OK) return st;
  REQUIRE(ldx >= cols, MOE_ERR_INVALID_ARG, "moe_act8_dequantize: ldx too small");
  REQUIRE(ldx % 8 == 0 && fits(0, ldx), MOE_ERR_UNSUPPORTED,
          "moe_act8_dequantize: ldx must be a multiple of 8 under 2^31");
  if (rows == 0) return MOE_OK;
  REQUIRE(x && q && scales, MOE_ERR_INVALID_ARG, "moe_act8_dequantize: null pointer");
  REQUIRE(aligned(x, 16) && aligned(q, 8) && aligned(scales, 2), MOE_ERR_UNSUPPORTED,
          "moe_act8_dequantize: x must be 16-byte, q 8-byte aligned");
  return cuda_status(moe::launch_act8_dequantize(q, ldq, scales, lds, rows, cols, group_offsets, E,
                                                 x, ldx, (cudaStream_t)stream),
                     "moe_act8_dequantize launch");
}

moe_status_t moe_act8_swiglu_fwd(const uint16_t *h, int64_t ldh, int64_t rows, int F,
                                 const int32_t *group_offsets, int E, uint16_t *act, int64_t lda,
                                 int8_t *q, int64_t ldq, uint16_t *scales, int64_t lds,
                                 moe_stream_t stream) {
  set_error("");
  const moe_status_t st = check_act8("moe_act8_swiglu_fwd", rows, F, group_offsets, E, ldq,
                                     2ll * F, lds, 2ll * ((F + 31) / 32));
  if (st != MOE_OK) return st;
  REQUIRE(ldh >= 2ll * F && lda >= F, MOE_ERR_INVALID_ARG,
          "moe_act8_swiglu_fwd: leading dimension too small");
  REQUIRE(ldh % 8 == 0 && lda % 8 == 0 && fits(0, ldh, lda), MOE_ERR_UNSUPPORTED,
          "moe_act8_swiglu_fwd: ldh and lda must be multiples of 8 under 2^31");
  if (rows == 0) return MOE_OK;
  REQUIRE(h && act && q && scales, MOE_ERR_INVALID_ARG, "moe_act8_swiglu_fwd: null pointer");
  REQUIRE(aligned(h, 16) && aligned(act, 16) && aligned(q, 8) && aligned(scales, 2),
          MOE_ERR_UNSUPPORTED, "moe_act8_swiglu_fwd: h and act must be 16-byte, q 8-byte aligned");
  return cuda_status(moe::launch_act8_swiglu_fwd(h, ldh, rows, F, group_offsets, E, act, lda, q,
                                                 ldq, scales, lds, (cudaStream_t)stream),
                     "moe_act8_swiglu_fwd launch");
}

moe_status_t moe_act8_swiglu_bwd(const int8_t *q, int64_t ldq, const uint16_t *scales, int64_t lds,
                                 const uint16_t *dact, int64_t ld_dact, int64_t rows, int F,
                                 const int32_t *group_offsets, int E, uint16_t *dh, int64_t ld_dh,
                                 uint16_t *act, int64_t lda, moe_stream_t stream) {
  set_error("");
  const moe_status_t st = check_act8("moe_act8_swiglu_bwd", rows, F, group_offsets, E, ldq,
                                     2ll * F, lds, 2ll * ((F + 31) / 32));
  if (st != MOE_OK) return st;
  REQUIRE(ld_dact >= F && ld_dh >= 2ll * F && (act == nullptr || lda >= F), MOE_ERR_INVALID_ARG,
          "moe_act8_swiglu_bwd: leading dimension too small");
  REQUIRE(ld_dact % 8 == 0 && ld_dh % 8 == 0 && (act == nullptr || lda % 8 == 0) &&
              fits(0, ld_dact, ld_dh, act == nullptr ? 0 : lda),
          MOE_ERR_UNSUPPORTED,
          "moe_act8_swiglu_bwd: ld_dact, ld_dh, lda must be multiples of 8 under 2^31");
  if (rows == 0) return MOE_OK;
  REQUIRE(q && scales && dact && dh, MOE_ERR_INVALID_ARG, "moe_act8_swiglu_bwd: null pointer");
  REQUIRE(aligned(dact, 16) && aligned(dh, 16) && aligned(act, 16) && aligned(q, 8) &&
              aligned(scales, 2),
          MOE_ERR_UNSUPPORTED,
          "moe_act8_swiglu_bwd: dact, dh and act must be 16-byte, q 8-byte aligned");
  return cuda_status(moe::launch_act8_swiglu_bwd(q, ldq, scales, lds, dact, ld_dact, rows, F,
                                                 group_offsets, E, dh, ld_dh, act, lda,
                                                 (cudaStream_t)stream),
                     "moe_act8_swiglu_bwd launch");
}

}  // extern "C"
