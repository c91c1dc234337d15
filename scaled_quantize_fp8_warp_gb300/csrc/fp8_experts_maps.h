// Tensor maps of the experts' operands.
#pragma once

#include "fp8_experts.h"

namespace fp8q {
namespace experts {

constexpr int kBK = 128;   // bytes = elements of K per stage of the products

// Boxes of `box_rows` rows x 128 bytes, 128-byte swizzled.
inline bool data_map(CUtensorMap *m, const Side &s, uint32_t box_rows) {
  return make_tmap_2d(m, s.data, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)s.row_bytes,
                      (uint64_t)s.rows, (uint64_t)s.row_bytes, kBK, box_rows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

// The scale atoms of a 128-row block as a row; boxes of one atom of each of
// `box_blocks` blocks.
inline bool scale_map(CUtensorMap *m, const Side &s, int64_t atoms, uint32_t box_blocks) {
  return make_tmap_2d(m, s.scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128 * (uint64_t)s.atoms_k,
                      (uint64_t)(atoms / s.atoms_k), 512 * (uint64_t)s.atoms_k, 128, box_blocks,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace experts
}  // namespace fp8q
