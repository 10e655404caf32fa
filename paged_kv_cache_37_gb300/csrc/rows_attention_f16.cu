// rows_attention_f16.cu -- instances of rows_attention.cuh over f16 pools.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_f16(int head_dim, int n_rows, bool f32) {
    return head_dim == 64 ? pick<__half, 64>(n_rows, f32) : pick<__half, 128>(n_rows, f32);
}

}  // namespace rows
}  // namespace pkv
