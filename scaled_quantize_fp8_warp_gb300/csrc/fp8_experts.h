// Host-side declarations of the experts' kernels, and where the groups of an
// operand lie.
#pragma once

#include "fp8q_internal.h"

namespace fp8q {
namespace experts {

// The groups of an operand's rows (fp8q_experts in include/fp8q.h).
struct Groups {
  const int32_t *offsets;   // null: equal groups of `each` rows
  int count;
  int rows;                 // S
  int each;
};

#ifdef __CUDACC__
// An offset is brought into [0, rows]: whatever it holds, rows stay inside the operand.
__device__ __forceinline__ int row_of(const Groups &g, int32_t offset) { return min(max(offset, 0), g.rows); }
// First row and number of rows of group e.
__device__ __forceinline__ int2 group_rows(const Groups &g, const int32_t *offsets, int e) {
  if (g.offsets == nullptr) return make_int2(e * g.each, g.each);
  const int a = row_of(g, offsets[e]), z = row_of(g, offsets[e + 1]);
  return make_int2(a, max(z - a, 0));
}
__device__ __forceinline__ int2 group_rows(const Groups &g, int e) { return group_rows(g, g.offsets, e); }

// First 128-row block of a group whose first row is `row`.
__device__ __forceinline__ int first_block(const Groups &g, int e, int row) {
  return g.offsets == nullptr ? e * ((g.each + 127) / 128) : row / 128 + e;
}
#endif

struct CastArgs {
  const void *x;
  int64_t T, ld;
  const int32_t *index;     // null: row r is row r of x
  Groups groups;
  int cols, blocks;         // C, NB
  uint8_t *q, *q_scales, *q_t, *qt_scales;   // either pair null
};

// A product per group.  by_rows: C [rows of B, rows of A] = B . A_e^T, group e
// owning rows of B and of C.  Otherwise C_e [rows of A, rows of B] = A_e . B_e^T,
// group e owning a stretch of the contraction.
struct Side {
  const uint8_t *data, *scales;
  int64_t rows, row_bytes;  // the whole matrix of bytes
  int atoms_k;              // scale atoms along K of one 128-row block of it
};
struct ProductArgs {
  Groups groups;            // of the rows of B (by_rows) or of the contraction
  const int32_t *a_offsets; // not by_rows: those of A's rows, where they lie elsewhere; null: B's
  int by_rows;
  Side a, b;
  int a_row, a_k, a_block;  // by_rows: group e's part of A starts at row a_row * e,
                            // K block a_k * e, 128-row block a_block * e
  int a_rows;               // rows of A in a group
  int b_rows;               // not by_rows: rows of B
  int k;                    // by_rows: the contraction
  int a_format, b_format;
  void *C;
};

cudaError_t launch_cast(int in_dtype, int format, const CastArgs &a, cudaStream_t stream);
// a_atoms, b_atoms: scale atoms of each side in all.
int launch_product(const ProductArgs &a, int out_dtype, int64_t a_atoms, int64_t b_atoms,
                   cudaStream_t stream);

// The same for few rows (by_rows): the contraction split over a cluster.
// split_for: CTAs that a tile's contraction is split over, 0 where this kernel
// does not serve the product.
int split_for(const ProductArgs &a);
int launch_split(const ProductArgs &a, int split, int out_dtype, int64_t a_atoms, int64_t b_atoms,
                 cudaStream_t stream);

}  // namespace experts
}  // namespace fp8q
