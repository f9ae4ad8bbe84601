// The 16-bit products' kernels for bfloat16.
#include "dense_kernels.h"

namespace moe {
hipError_t rows_product_bf16(const RowsProduct& a, RowsTile t, int split, hipStream_t s) { return rows_dt<T_BF16>(a, t, split, s); }
hipError_t cols_product_bf16(const ColsProduct& a, ColsTile t, int split, hipStream_t s) { return cols_dt<T_BF16>(a, t, split, s); }
}  // namespace moe
