// The extern "C" boundary of the 4-bit operators and of the activation
// functions with 8-bit checkpoints (include/fp8q.h): argument checks, device
// check, workspace layout and dispatch.  No call allocates or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_common.cuh"
#include "fp4_internal.h"
#include "fp8_act.h"

namespace fp8q {
namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool valid_dtype(int d) { return d == FP8Q_DT_F32 || d == FP8Q_DT_BF16; }
bool valid_kind(int k) { return k == FP4Q_MXFP4 || k == FP4Q_NVFP4; }
int64_t dtype_size(int d) { return d == FP8Q_DT_BF16 ? 2 : 4; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA; }

int check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP8Q_ERR_CUDA;
  return fp8q_device_supported() == 1 ? FP8Q_OK : FP8Q_ERR_ARCH;
}

// A rows x cols matrix whose padded byte counts (4-byte elements, rows and
// columns rounded up to 128) fit in int64.
bool dims_ok(int64_t rows, int64_t cols) {
  constexpr int64_t kLim = INT64_MAX / 32;
  if (rows < 0 || cols < 0 || rows > kLim || cols > kLim) return false;
  return cols == 0 || rows + 128 <= kLim / (cols + 128);
}

// Row and column indexes of the activation kernels are 32-bit (offsets are not).
bool act_dims_ok(int64_t T, int64_t F) {
  return dims_ok(T, F) && T <= INT32_MAX / 4 && F <= INT32_MAX / 4;
}

// Matrix argument [rows, cols] with rows ld elements apart; `align` in bytes.
int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t align) {
  if (rows == 0 || cols == 0) return FP8Q_OK;
  if (p == nullptr || ld < cols) return FP8Q_ERR_INVALID_ARG;
  if (rows > 1 && !dims_ok(rows, ld)) return FP8Q_ERR_INVALID_ARG;
  return aligned(p, (uintptr_t)align) ? FP8Q_OK : FP8Q_ERR_MISALIGNED;
}

int check_operand(const fp4q_operand *op, int64_t rows, int64_t K) {
  if (op == nullptr || !valid_kind(op->kind) || op->reserved != 0) return FP8Q_ERR_INVALID_ARG;
  if ((op->kind == FP4Q_NVFP4) != (op->global_scale != nullptr)) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(op->global_scale, 4)) return FP8Q_ERR_MISALIGNED;
  if (rows > 0 && K > 0) {
    if (op->data == nullptr || op->scales == nullptr) return FP8Q_ERR_INVALID_ARG;
    if (!aligned(op->data, 16) || !aligned(op->scales, 16)) return FP8Q_ERR_MISALIGNED;
  }
  return FP8Q_OK;
}

bool linear_ok(int64_t M, int64_t N, int64_t K) {
  return dims_ok(M, K) && dims_ok(N, K) && dims_ok(M, N);
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

size_t data_bytes(int64_t rows, int64_t K) { return (size_t)(rows * fp4::row_bytes(K)); }

// A piece-by-piece workspace: take() hands out 256-byte aligned pieces.
struct Pieces {
  uint8_t *base;
  size_t used = 0;
  uint8_t *take(size_t bytes) {
    uint8_t *p = base == nullptr ? nullptr : base + used;
    used += round256(bytes);
    return p;
  }
};

// One matrix quantised in both orientations, in a workspace.
struct Both {
  fp4q_operand rows, cols;
  float *global;
  void lay_out(Pieces &ws, int kind, int64_t R, int64_t C) {
    global = reinterpret_cast<float *>(ws.take(sizeof(float)));
    const float *g = kind == FP4Q_NVFP4 ? global : nullptr;
    uint8_t *q = ws.take(data_bytes(R, C)), *qs = ws.take(fp4q_scale_bytes(kind, R, C));
    uint8_t *t = ws.take(data_bytes(C, R)), *ts = ws.take(fp4q_scale_bytes(kind, C, R));
    rows = fp4q_operand{q, qs, g, kind, 0};
    cols = fp4q_operand{t, ts, g, kind, 0};
  }
};

fp4::QuantArgs quant_args(const void *x, int64_t rows, int64_t cols, int64_t ld,
                          const float *amax, const fp4q_operand *q, const fp4q_operand *qt,
                          float *global) {
  fp4::QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.amax = amax;
  a.q = q == nullptr ? nullptr : const_cast<uint8_t *>(q->data);
  a.q_scales = q == nullptr ? nullptr : const_cast<uint8_t *>(q->scales);
  a.qt = qt == nullptr ? nullptr : const_cast<uint8_t *>(qt->data);
  a.qt_scales = qt == nullptr ? nullptr : const_cast<uint8_t *>(qt->scales);
  a.global_scale = global;
  return a;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" {

size_t fp4q_scale_bytes(int kind, int64_t rows, int64_t K) {
  if (!valid_kind(kind) || !dims_ok(rows, K)) return 0;
  return (size_t)((rows + 127) / 128 * fp4::num_atoms_k(kind, K) * 512);
}

int fp4_quantize(const void *x, int in_dtype, int64_t rows, int64_t cols, int64_t ld, int kind,
                 const float *amax, uint8_t *q, uint8_t *q_scales, uint8_t *qt,
                 uint8_t *qt_scales, float *global_scale, cudaStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_kind(kind) || !dims_ok(rows, cols))
    return FP8Q_ERR_INVALID_ARG;
  int rc = check_matrix(x, rows, cols, ld, dtype_size(in_dtype));
  if (rc != FP8Q_OK) return rc;
  const bool empty = rows == 0 || cols == 0;
  if ((q == nullptr) != (q_scales == nullptr) || (qt == nullptr) != (qt_scales == nullptr) ||
      (!empty && q == nullptr && qt == nullptr))
    return FP8Q_ERR_INVALID_ARG;
  if (kind == FP4Q_NVFP4 ? (amax == nullptr || global_scale == nullptr) : global_scale != nullptr)
    return FP8Q_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_scales, 16) || !aligned(qt, 16) || !aligned(qt_scales, 16) ||
      !aligned(amax, 4) || !aligned(global_scale, 4))
    return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp4_quantize %lldx%lld kind=%d q=%d qt=%d", (long long)rows, (long long)cols, kind,
           q != nullptr, qt != nullptr);
  if (empty)
    return kind == FP4Q_NVFP4 ? from_cuda(fp4::launch_global(amax, global_scale, stream)) : FP8Q_OK;
  const fp4q_operand a{q, q_scales, nullptr, kind, 0}, b{qt, qt_scales, nullptr, kind, 0};
  const fp4::QuantArgs args =
      quant_args(x, rows, cols, ld, amax, q ? &a : nullptr, qt ? &b : nullptr, global_scale);
  return from_cuda(fp4::launch_quantize(kind, in_dtype, &args, 1, stream));
}

int fp4_amax(const void *x, int in_dtype, int64_t rows, int64_t cols, int64_t ld, float *amax,
             cudaStream_t stream) {
  if (!valid_dtype(in_dtype) || !dims_ok(rows, cols) || amax == nullptr)
    return FP8Q_ERR_INVALID_ARG;
  int rc = check_matrix(x, rows, cols, ld, dtype_size(in_dtype));
  if (rc != FP8Q_OK) return rc;
  if (!aligned(amax, 4)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp4_amax %lldx%lld", (long long)rows, (long long)cols);
  return from_cuda(fp4::launch_amax_ld(x, in_dtype, rows, cols, ld, amax, stream));
}

int fp4_dequantize(const fp4q_operand *op, int64_t rows, int64_t K, void *y, int out_dtype,
                   cudaStream_t stream) {
  if (!valid_dtype(out_dtype) || !dims_ok(rows, K)) return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(op, rows, K);
  if (rc != FP8Q_OK) return rc;
  if ((rc = check_matrix(y, rows, K, K, 16)) != FP8Q_OK) return rc;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  if (rows == 0 || K == 0) return FP8Q_OK;
  log_line("fp4_dequantize %lldx%lld kind=%d", (long long)rows, (long long)K, op->kind);
  return from_cuda(fp4::launch_dequantize(op->kind, *op, rows, K, out_dtype, y, stream));
}

int fp4_gemm(const fp4q_operand *A, const fp4q_operand *B, void *C, int out_dtype, int64_t M,
             int64_t N, int64_t K, cudaStream_t stream) {
  if (!valid_dtype(out_dtype) || !linear_ok(M, N, K)) return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(A, M, K);
  if (rc != FP8Q_OK) return rc;
  if ((rc = check_operand(B, N, K)) != FP8Q_OK) return rc;
  if (A->kind != B->kind || !fp4::product_fits(A->kind, M, N, K)) return FP8Q_ERR_INVALID_ARG;
  if ((rc = check_matrix(C, M, N, N, 16)) != FP8Q_OK) return rc;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp4_gemm M=%lld N=%lld K=%lld kind=%d out=%d", (long long)M, (long long)N, (long long)K,
           A->kind, out_dtype);
  const fp4::Product d{*A, *B, C, M, N, K};
  return fp4::launch_products(A->kind, &d, 1, out_dtype, stream);
}

size_t fp4q_linear_workspace_size(int kind, int64_t M, int64_t N, int64_t K) {
  if (!valid_kind(kind) || !linear_ok(M, N, K)) return 0;
  Pieces ws{nullptr};
  ws.take(8);
  ws.take(data_bytes(M, K));
  ws.take(fp4q_scale_bytes(kind, M, K));
  return ws.used;
}

int fp4_linear(const void *x, int in_dtype, int64_t ldx, const fp4q_operand *w, int64_t M,
               int64_t N, int64_t K, const float *x_amax, void *y, int out_dtype,
               void *workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || !linear_ok(M, N, K))
    return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(w, N, K);
  if (rc != FP8Q_OK) return rc;
  if (!fp4::product_fits(w->kind, M, N, K)) return FP8Q_ERR_INVALID_ARG;
  if ((rc = check_matrix(x, M, K, ldx, dtype_size(in_dtype))) != FP8Q_OK) return rc;
  if ((rc = check_matrix(y, M, N, N, 16)) != FP8Q_OK) return rc;
  if (!aligned(x_amax, 4)) return FP8Q_ERR_MISALIGNED;
  const bool fused = M <= FP4Q_LINEAR_FUSED_ROWS;   // the product quantises x itself
  const bool find_amax = w->kind == FP4Q_NVFP4 && x_amax == nullptr;
  if ((!fused || find_amax) &&
      (workspace == nullptr || ws_bytes < fp4q_linear_workspace_size(w->kind, M, N, K)))
    return FP8Q_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  if (M == 0 || N == 0) return FP8Q_OK;
  log_line("fp4_linear M=%lld N=%lld K=%lld kind=%d out=%d amax=%d", (long long)M, (long long)N,
           (long long)K, w->kind, out_dtype, x_amax != nullptr);
  Pieces ws{static_cast<uint8_t *>(workspace)};
  float *words = reinterpret_cast<float *>(ws.take(8));
  fp4q_operand q{};
  q.kind = w->kind;
  q.data = ws.take(data_bytes(M, K));
  q.scales = ws.take(fp4q_scale_bytes(w->kind, M, K));
  q.global_scale = w->kind == FP4Q_NVFP4 ? words + 1 : nullptr;
  fp4::Product d{q, *w, y, M, N, K};
  if (K > 0) {
    if (find_amax) {
      if (fp4::launch_amax_ld(x, in_dtype, M, K, ldx, words, stream) != cudaSuccess)
        return FP8Q_ERR_CUDA;
      x_amax = words;
    }
    if (fused)
      return fp4::launch_split_quantizing(w->kind, x, in_dtype, ldx, x_amax, d, out_dtype, stream);
    float *global = w->kind == FP4Q_NVFP4 ? words + 1 : nullptr;
    const fp4::QuantArgs args = quant_args(x, M, K, ldx, x_amax, &q, nullptr, global);
    if (fp4::launch_quantize(w->kind, in_dtype, &args, 1, stream) != cudaSuccess)
      return FP8Q_ERR_CUDA;
  }
  return fp4::launch_products(w->kind, &d, 1, out_dtype, stream);
}

size_t fp4q_linear_train_workspace_size(int kind, int64_t M, int64_t N, int64_t K) {
  if (!valid_kind(kind) || !linear_ok(M, N, K)) return 0;
  Pieces ws{nullptr};
  ws.take(3 * sizeof(float));   // the amaxes
  Both b;
  b.lay_out(ws, kind, M, K);
  b.lay_out(ws, kind, N, K);
  b.lay_out(ws, kind, M, N);
  return ws.used;
}

int fp4_linear_train(const void *x, const void *w, const void *g, int in_dtype, int64_t M,
                     int64_t N, int64_t K, int kind, void *y, void *dx, void *dw, int out_dtype,
                     void *workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || !valid_kind(kind) ||
      !linear_ok(M, N, K) || !fp4::product_fits(kind, M, N, K) ||
      !fp4::product_fits(kind, M, K, N) || !fp4::product_fits(kind, N, K, M))
    return FP8Q_ERR_INVALID_ARG;
  const int64_t in = dtype_size(in_dtype);
  int rc;
  if ((rc = check_matrix(x, M, K, K, in)) != FP8Q_OK ||
      (rc = check_matrix(w, N, K, K, in)) != FP8Q_OK ||
      (rc = check_matrix(g, M, N, N, in)) != FP8Q_OK ||
      (rc = check_matrix(y, M, N, N, 16)) != FP8Q_OK ||
      (rc = check_matrix(dx, M, K, K, 16)) != FP8Q_OK ||
      (rc = check_matrix(dw, N, K, K, 16)) != FP8Q_OK)
    return rc;
  if (workspace == nullptr || ws_bytes < fp4q_linear_train_workspace_size(kind, M, N, K))
    return FP8Q_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp4_linear_train M=%lld N=%lld K=%lld kind=%d out=%d", (long long)M, (long long)N,
           (long long)K, kind, out_dtype);
  Pieces ws{static_cast<uint8_t *>(workspace)};
  float *amax = reinterpret_cast<float *>(ws.take(3 * sizeof(float)));
  Both bx, bw, bg;
  bx.lay_out(ws, kind, M, K);
  bw.lay_out(ws, kind, N, K);
  bg.lay_out(ws, kind, M, N);
  const struct {
    const void *p;
    int64_t rows, cols;
    const Both *to;
  } in_m[3] = {{x, M, K, &bx}, {w, N, K, &bw}, {g, M, N, &bg}};
  fp4::QuantArgs args[3];
  const void *src[3];
  int64_t size[3];
  int n = 0;
  for (const auto &m : in_m) {   // the empty ones have nothing to cast
    if (m.rows == 0 || m.cols == 0) continue;
    src[n] = m.p;
    size[n] = m.rows * m.cols;
    args[n] = quant_args(m.p, m.rows, m.cols, m.cols, amax + n, &m.to->rows, &m.to->cols,
                         kind == FP4Q_NVFP4 ? m.to->global : nullptr);
    ++n;
  }
  if (n > 0) {
    if (kind == FP4Q_NVFP4 &&
        fp4::launch_amax_group(src, size, n, in_dtype, amax, stream) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    if (fp4::launch_quantize(kind, in_dtype, args, n, stream) != cudaSuccess) return FP8Q_ERR_CUDA;
  }
  const fp4::Product prod[3] = {{bx.rows, bw.rows, y, M, N, K},
                                {bg.rows, bw.cols, dx, M, K, N},
                                {bg.cols, bx.cols, dw, N, K, M}};
  return fp4::launch_products(kind, prod, 3, out_dtype, stream);
}

int fp8_act_forward(int act, int dtype, int64_t T, int64_t F, const void *u, int64_t ldu,
                    const void *v, int64_t ldv, void *a, int64_t lda, uint8_t *u8,
                    float *u_scales, uint8_t *v8, float *v_scales, cudaStream_t stream) {
  if (act < FP8Q_ACT_SILU || act > FP8Q_ACT_GELU_TANH || !valid_dtype(dtype) || !act_dims_ok(T, F))
    return FP8Q_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const bool gated = v != nullptr;
  if (gated != (v8 != nullptr) || gated != (v_scales != nullptr)) return FP8Q_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_matrix(u, T, F, ldu, size)) != FP8Q_OK ||
      (gated && (rc = check_matrix(v, T, F, ldv, size)) != FP8Q_OK) ||
      (rc = check_matrix(a, T, F, lda, size)) != FP8Q_OK ||
      (rc = check_matrix(u8, T, F, F, 1)) != FP8Q_OK ||
      (rc = check_matrix(u_scales, T, F, F, 4)) != FP8Q_OK)
    return rc;
  if (!aligned(v_scales, 4)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  if (T == 0 || F == 0) return FP8Q_OK;
  log_line("fp8_act_forward act=%d %lldx%lld gated=%d", act, (long long)T, (long long)F, gated);
  act::ForwardArgs p{};
  p.T = T;
  p.F = F;
  p.u = u;
  p.v = v;
  p.ldu = ldu;
  p.ldv = ldv;
  p.a = a;
  p.lda = lda;
  p.u8 = u8;
  p.v8 = v8;
  p.u_scales = u_scales;
  p.v_scales = v_scales;
  return from_cuda(act::launch_forward(act, dtype, p, stream));
}

int fp8_act_backward(int act, int dtype, int64_t T, int64_t F, const uint8_t *u8,
                     const float *u_scales, const uint8_t *v8, const float *v_scales,
                     const void *da, int64_t ldda, void *du, int64_t lddu, void *dv,
                     int64_t lddv, void *a, int64_t lda, cudaStream_t stream) {
  if (act < FP8Q_ACT_SILU || act > FP8Q_ACT_GELU_TANH || !valid_dtype(dtype) || !act_dims_ok(T, F))
    return FP8Q_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  const bool gated = v8 != nullptr;
  if (gated != (v_scales != nullptr) || gated != (dv != nullptr)) return FP8Q_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_matrix(u8, T, F, F, 1)) != FP8Q_OK ||
      (rc = check_matrix(u_scales, T, F, F, 4)) != FP8Q_OK ||
      (rc = check_matrix(da, T, F, ldda, size)) != FP8Q_OK ||
      (rc = check_matrix(du, T, F, lddu, size)) != FP8Q_OK ||
      (gated && (rc = check_matrix(dv, T, F, lddv, size)) != FP8Q_OK) ||
      (a != nullptr && (rc = check_matrix(a, T, F, lda, size)) != FP8Q_OK))
    return rc;
  if (!aligned(v_scales, 4)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  if (T == 0 || F == 0) return FP8Q_OK;
  log_line("fp8_act_backward act=%d %lldx%lld gated=%d a=%d", act, (long long)T, (long long)F,
           gated, a != nullptr);
  act::BackwardArgs p{};
  p.T = T;
  p.F = F;
  p.u8 = u8;
  p.v8 = v8;
  p.u_scales = u_scales;
  p.v_scales = v_scales;
  p.da = da;
  p.ldda = ldda;
  p.du = du;
  p.lddu = lddu;
  p.dv = dv;
  p.lddv = lddv;
  p.a = a;
  p.lda = lda;
  return from_cuda(act::launch_backward(act, dtype, p, stream));
}

}  // extern "C"
