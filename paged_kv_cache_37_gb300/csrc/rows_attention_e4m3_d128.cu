// rows_attention_e4m3_d128.cu -- instances of rows_attention.cuh: e4m3 pools, head_dim 128.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_e4m3_d128(int n_rows, bool f32, bool paged) { return pick<uint8_t, 128>(n_rows, f32, paged); }

}  // namespace rows
}  // namespace pkv
