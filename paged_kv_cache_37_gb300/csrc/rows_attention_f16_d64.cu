// rows_attention_f16_d64.cu -- instances of rows_attention.cuh: f16 pools, head_dim 64.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_f16_d64(int n_rows, bool f32, bool paged) { return pick<__half, 64>(n_rows, f32, paged); }

}  // namespace rows
}  // namespace pkv
