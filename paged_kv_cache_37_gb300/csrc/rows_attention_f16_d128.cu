// rows_attention_f16_d128.cu -- instances of rows_attention.cuh: f16 pools, head_dim 128.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_f16_d128(int n_rows, bool f32, bool paged) { return pick<__half, 128>(n_rows, f32, paged); }

}  // namespace rows
}  // namespace pkv
