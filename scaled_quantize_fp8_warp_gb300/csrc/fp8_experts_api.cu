// The extern "C" boundary of the RMS norm and of the experts' operators
// (include/fp8q.h): argument checks, device check and dispatch.  No call
// allocates or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8_experts.h"
#include "fp8_norm.h"

namespace fp8q {
namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool valid_dtype(int d) { return d == FP8Q_DT_F32 || d == FP8Q_DT_BF16; }
int64_t dtype_size(int d) { return d == FP8Q_DT_BF16 ? 2 : 4; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA; }

int check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP8Q_ERR_CUDA;
  return fp8q_device_supported() == 1 ? FP8Q_OK : FP8Q_ERR_ARCH;
}

// Row and column indexes of the norm's kernels are 32-bit (offsets are not).
bool norm_dims_ok(int64_t T, int64_t C) {
  return T >= 0 && C >= 0 && T <= INT32_MAX / 4 && C <= INT32_MAX / 4;
}

// Matrix argument [rows, cols] with rows ld elements apart; `align` in bytes.
int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t align) {
  if (rows == 0 || cols == 0) return FP8Q_OK;
  if (p == nullptr || ld < cols || (rows > 1 && ld > INT64_MAX / 8 / rows)) return FP8Q_ERR_INVALID_ARG;
  return aligned(p, (uintptr_t)align) ? FP8Q_OK : FP8Q_ERR_MISALIGNED;
}

constexpr int64_t kMostRows = INT32_MAX - 1024;
// Longest contraction of a product: a tile of it takes some 0.4 s, a fifth of
// what a kernel waits for anything.
constexpr int64_t kMostContract = 1 << 27;

// Blocks of 128 rows; -1 for sizes that are refused.
int64_t blocks_of(int64_t rows, int64_t groups, bool ragged) {
  if (rows < 0 || rows > kMostRows || groups < 1 || groups > FP8Q_EXPERTS_MAX) return -1;
  if (!ragged && rows % groups != 0) return -1;
  const int64_t blocks = ragged ? rows / 128 + groups : groups * ((rows / groups + 127) / 128);
  return blocks <= kMostRows / 128 ? blocks : -1;
}

// Scale atoms of one orientation; -1 for sizes that are refused.
int64_t atoms_of(int64_t rows, int64_t cols, int64_t groups, bool ragged) {
  const int64_t blocks = blocks_of(rows, groups, ragged);
  if (blocks < 0 || cols < 0 || cols > kMostRows || cols % 16 != 0) return -1;
  const int64_t across = (cols + 127) / 128;
  return across == 0 || blocks <= INT32_MAX / across ? blocks * across : -1;
}

// An operand whose pairs in `need` (1: by rows, 2: transposed) must be there.
int check_operand(const fp8q_experts *op, int need) {
  if (op == nullptr || (op->format != FP8Q_E4M3 && op->format != FP8Q_E5M2)) return FP8Q_ERR_INVALID_ARG;
  const int64_t atoms = atoms_of(op->rows, op->cols, op->groups, op->offsets != nullptr);
  if (atoms < 0) return FP8Q_ERR_INVALID_ARG;
  // without rows or columns nothing is read or written through a pointer, and what
  // holds nothing may have any address: q of no rows is null beside scales that are not
  if (op->rows > 0 && op->cols > 0 &&
      ((op->q == nullptr) != (op->q_scales == nullptr) || (op->q_t == nullptr) != (op->qt_scales == nullptr) ||
       ((need & 1) && op->q == nullptr) || ((need & 2) && op->q_t == nullptr)))
    return FP8Q_ERR_INVALID_ARG;
  if (!aligned(op->offsets, 4) || !aligned(op->q, 16) || !aligned(op->q_scales, 16) ||
      !aligned(op->q_t, 16) || !aligned(op->qt_scales, 16))
    return FP8Q_ERR_MISALIGNED;
  return FP8Q_OK;
}

experts::Groups groups_of(const fp8q_experts &op) {
  experts::Groups g{};
  g.offsets = op.offsets;
  g.count = op.groups;
  g.rows = (int)op.rows;
  g.each = (int)(op.rows / op.groups);
  return g;
}

int64_t operand_blocks(const fp8q_experts &op) {
  return blocks_of(op.rows, op.groups, op.offsets != nullptr);
}
int64_t operand_atoms(const fp8q_experts &op) {
  return atoms_of(op.rows, op.cols, op.groups, op.offsets != nullptr);
}

experts::Side by_rows(const fp8q_experts &op) {
  return experts::Side{op.q, op.q_scales, op.rows, op.cols, (int)((op.cols + 127) / 128)};
}
experts::Side transposed(const fp8q_experts &op) {
  const int64_t blocks = operand_blocks(op);
  return experts::Side{op.q_t, op.qt_scales, op.cols, 128 * blocks, (int)blocks};
}

int run(const experts::ProductArgs &a, int out_dtype, const fp8q_experts &of_a, const fp8q_experts &of_b,
        cudaStream_t stream) {
  return experts::launch_product(a, out_dtype, operand_atoms(of_a), operand_atoms(of_b), stream);
}

// Rows of x times a weight per group, by rows (fprop) or transposed (dgrad).
int rows_product(const fp8q_experts *x, const fp8q_experts *w, bool dgrad, void *y, int out_dtype,
                 cudaStream_t stream) {
  if (!valid_dtype(out_dtype)) return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(x, 1);
  if (rc != FP8Q_OK) return rc;
  if ((rc = check_operand(w, dgrad ? 2 : 1)) != FP8Q_OK) return rc;
  if (w->offsets != nullptr || w->groups != x->groups) return FP8Q_ERR_INVALID_ARG;
  const int64_t N = w->rows / w->groups, K = w->cols, S = x->rows;
  const int64_t contract = dgrad ? N : K, result = dgrad ? K : N;
  if (N % 16 != 0 || x->cols != contract || contract > kMostContract ||
      (contract == 0 && S > 0 && result > 0))
    return FP8Q_ERR_INVALID_ARG;
  if (S > 0 && result > 0) {
    if (y == nullptr || result > INT64_MAX / 8 / S) return FP8Q_ERR_INVALID_ARG;
    if (!aligned(y, 16)) return FP8Q_ERR_MISALIGNED;
  }
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp8_experts_%s S=%lld N=%lld K=%lld E=%d out=%d", dgrad ? "dgrad" : "fprop", (long long)S,
           (long long)N, (long long)K, x->groups, out_dtype);
  if (S == 0 || result == 0) return FP8Q_OK;
  experts::ProductArgs a{};
  a.groups = groups_of(*x);
  a.by_rows = 1;
  a.a = dgrad ? transposed(*w) : by_rows(*w);
  a.b = by_rows(*x);
  a.a_row = dgrad ? 0 : (int)N;
  a.a_k = dgrad ? (int)((N + 127) / 128) : 0;
  a.a_block = dgrad ? 0 : (int)((N + 127) / 128);
  a.a_rows = (int)result;
  a.k = (int)contract;
  a.a_format = w->format;
  a.b_format = x->format;
  a.C = y;
  return run(a, out_dtype, *w, *x, stream);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" {

int fp8_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype,
                const void *weight, int w_dtype, const float *eps, int64_t T, int64_t C, void *h,
                int64_t ldh, void *y, int64_t ldy, int scaling, uint8_t *q, float *q_scales,
                float *rstd, cudaStream_t stream) {
  if (!valid_dtype(dtype) || !valid_dtype(w_dtype) || !norm_dims_ok(T, C)) return FP8Q_ERR_INVALID_ARG;
  if (eps == nullptr || !(*eps >= 0.0f) || *eps > 3.4028235e38f) return FP8Q_ERR_INVALID_ARG;
  // results of no elements may have any address: row scales of [T, 0] are not null beside a q that is
  if (T > 0 && C > 0 && ((residual == nullptr) != (h == nullptr) || (q == nullptr) != (q_scales == nullptr)))
    return FP8Q_ERR_INVALID_ARG;
  if (q != nullptr && scaling != FP8Q_SCALE_TILE_1x128 && scaling != FP8Q_SCALE_ROW)
    return FP8Q_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  int rc;
  if ((rc = check_matrix(x, T, C, ldx, size)) != FP8Q_OK ||
      (residual != nullptr && (rc = check_matrix(residual, T, C, ldr, size)) != FP8Q_OK) ||
      (h != nullptr && (rc = check_matrix(h, T, C, ldh, size)) != FP8Q_OK) ||
      (y != nullptr && (rc = check_matrix(y, T, C, ldy, size)) != FP8Q_OK) ||
      (rc = check_matrix(weight, T, C, C, dtype_size(w_dtype))) != FP8Q_OK)
    return rc;
  if (!aligned(q_scales, 4) || !aligned(rstd, 4)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp8_rmsnorm %lldx%lld residual=%d y=%d q=%d scaling=%d", (long long)T, (long long)C,
           residual != nullptr, y != nullptr, q != nullptr, scaling);
  if (T == 0 || C == 0) return FP8Q_OK;
  norm::ForwardArgs a{};
  a.T = T;
  a.C = C;
  a.x = x;
  a.residual = residual;
  a.ldx = ldx;
  a.ldr = ldr;
  a.weight = weight;
  a.w_bf16 = w_dtype == FP8Q_DT_BF16;
  a.eps = *eps;
  a.h = h;
  a.y = y;
  a.ldh = ldh;
  a.ldy = ldy;
  a.q = q;
  a.q_scales = q_scales;
  a.row_scale = scaling == FP8Q_SCALE_ROW;
  a.rstd = rstd;
  return from_cuda(norm::launch_forward(dtype, a, stream));
}

size_t fp8q_rmsnorm_backward_workspace_size(int64_t T, int64_t C) {
  if (!norm_dims_ok(T, C)) return 0;
  return ((size_t)norm::kPartials * (size_t)C * sizeof(float) + 255) & ~(size_t)255;
}

int fp8_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, int dtype,
                         const void *weight, int w_dtype, const float *rstd, const void *dresidual,
                         int64_t lddr, int64_t T, int64_t C, void *dx, int64_t lddx, void *dweight,
                         void *workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!valid_dtype(dtype) || !valid_dtype(w_dtype) || !norm_dims_ok(T, C)) return FP8Q_ERR_INVALID_ARG;
  const int64_t size = dtype_size(dtype);
  int rc;
  if ((rc = check_matrix(dy, T, C, lddy, size)) != FP8Q_OK ||
      (rc = check_matrix(h, T, C, ldh, size)) != FP8Q_OK ||
      (dresidual != nullptr && (rc = check_matrix(dresidual, T, C, lddr, size)) != FP8Q_OK) ||
      (rc = check_matrix(dx, T, C, lddx, size)) != FP8Q_OK ||
      (rc = check_matrix(weight, T, C, C, dtype_size(w_dtype))) != FP8Q_OK ||
      (rc = check_matrix(rstd, T, C, C, 4)) != FP8Q_OK)
    return rc;
  if (!aligned(dweight, (uintptr_t)dtype_size(w_dtype))) return FP8Q_ERR_MISALIGNED;
  if (dweight != nullptr && T > 0 && C > 0 &&
      (workspace == nullptr || ws_bytes < fp8q_rmsnorm_backward_workspace_size(T, C)))
    return FP8Q_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp8_rmsnorm_backward %lldx%lld dresidual=%d dweight=%d", (long long)T, (long long)C,
           dresidual != nullptr, dweight != nullptr);
  if (C == 0) return FP8Q_OK;
  norm::BackwardArgs a{};
  a.T = T;
  a.C = C;
  a.dy = dy;
  a.h = h;
  a.dresidual = dresidual;
  a.lddy = lddy;
  a.ldh = ldh;
  a.lddr = lddr;
  a.weight = weight;
  a.w_bf16 = w_dtype == FP8Q_DT_BF16;
  a.rstd = rstd;
  a.dx = dx;
  a.lddx = lddx;
  a.dweight = dweight;
  a.partial = static_cast<float *>(workspace);
  return from_cuda(norm::launch_backward(dtype, a, stream));
}

int64_t fp8q_experts_blocks(int64_t rows, int groups, int ragged) {
  const int64_t n = blocks_of(rows, groups, ragged != 0);
  return n < 0 ? 0 : n;
}

size_t fp8q_experts_scale_bytes(int64_t rows, int64_t cols, int groups, int ragged) {
  const int64_t n = atoms_of(rows, cols, groups, ragged != 0);
  return n < 0 ? 0 : (size_t)n * 512;
}

int fp8_quantize_experts(const void *x, int in_dtype, int64_t T, int64_t ld, const int32_t *index,
                         const fp8q_experts *out, cudaStream_t stream) {
  if (!valid_dtype(in_dtype) || T < 0 || T > kMostRows) return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(out, 0);
  if (rc != FP8Q_OK) return rc;
  const bool empty = out->rows == 0 || out->cols == 0;
  // an index of no rows may be null
  if ((!empty && out->q == nullptr && out->q_t == nullptr) ||
      (index == nullptr && out->rows > 0 && T != out->rows))
    return FP8Q_ERR_INVALID_ARG;
  if ((rc = check_matrix(x, T, out->cols, ld, dtype_size(in_dtype))) != FP8Q_OK) return rc;
  if (!aligned(index, 4)) return FP8Q_ERR_MISALIGNED;
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp8_quantize_experts %lld rows of %lldx%lld E=%d q=%d qt=%d", (long long)out->rows,
           (long long)T, (long long)out->cols, out->groups, out->q != nullptr, out->q_t != nullptr);
  if (empty) return FP8Q_OK;
  experts::CastArgs a{};
  a.x = x;
  a.T = T;
  a.ld = ld;
  a.index = index;
  a.groups = groups_of(*out);
  a.cols = (int)out->cols;
  a.blocks = (int)operand_blocks(*out);
  a.q = const_cast<uint8_t *>(out->q);
  a.q_scales = const_cast<uint8_t *>(out->q_scales);
  a.q_t = const_cast<uint8_t *>(out->q_t);
  a.qt_scales = const_cast<uint8_t *>(out->qt_scales);
  return from_cuda(experts::launch_cast(in_dtype, out->format, a, stream));
}

int fp8_experts_fprop(const fp8q_experts *x, const fp8q_experts *w, void *y, int out_dtype,
                      cudaStream_t stream) {
  return rows_product(x, w, false, y, out_dtype, stream);
}

int fp8_experts_dgrad(const fp8q_experts *g, const fp8q_experts *w, void *dx, int out_dtype,
                      cudaStream_t stream) {
  return rows_product(g, w, true, dx, out_dtype, stream);
}

int fp8_experts_wgrad(const fp8q_experts *g, const fp8q_experts *x, void *dw, int out_dtype,
                      cudaStream_t stream) {
  if (!valid_dtype(out_dtype)) return FP8Q_ERR_INVALID_ARG;
  int rc = check_operand(g, 2);
  if (rc != FP8Q_OK) return rc;
  if ((rc = check_operand(x, 2)) != FP8Q_OK) return rc;
  if (x->rows > kMostContract || g->rows != x->rows || g->groups != x->groups || (g->offsets == nullptr) != (x->offsets == nullptr))
    return FP8Q_ERR_INVALID_ARG;
  const int64_t N = g->cols, K = x->cols, E = x->groups;
  if (N > 0 && K > 0) {
    if (dw == nullptr || K > INT64_MAX / 8 / E / N) return FP8Q_ERR_INVALID_ARG;
    if (!aligned(dw, 16)) return FP8Q_ERR_MISALIGNED;
  }
  if ((rc = check_device()) != FP8Q_OK) return rc;
  log_line("fp8_experts_wgrad S=%lld N=%lld K=%lld E=%lld out=%d", (long long)x->rows, (long long)N,
           (long long)K, (long long)E, out_dtype);
  if (N == 0 || K == 0) return FP8Q_OK;
  if (x->rows == 0)
    return from_cuda(cudaMemsetAsync(dw, 0, (size_t)(E * N * K * dtype_size(out_dtype)), stream));
  experts::ProductArgs a{};
  a.groups = groups_of(*x);
  a.a_offsets = g->offsets != x->offsets ? g->offsets : nullptr;
  a.by_rows = 0;
  a.a = transposed(*g);
  a.b = transposed(*x);
  a.a_rows = (int)N;
  a.b_rows = (int)K;
  a.a_format = g->format;
  a.b_format = x->format;
  a.C = dw;
  return run(a, out_dtype, *g, *x, stream);
}

}  // extern "C"
