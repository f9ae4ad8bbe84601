// The 16-bit products' kernels for half precision.
#include "dense_kernels.h"

namespace moe {
hipError_t rows_product_f16(const RowsProduct& a, RowsTile t, int split, hipStream_t s) { return rows_dt<T_F16>(a, t, split, s); }
hipError_t cols_product_f16(const ColsProduct& a, ColsTile t, int split, hipStream_t s) { return cols_dt<T_F16>(a, t, split, s); }
}  // namespace moe
