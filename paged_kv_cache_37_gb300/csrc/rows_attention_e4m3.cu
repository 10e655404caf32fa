// rows_attention_e4m3.cu -- instances of rows_attention.cuh over e4m3 pools.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_e4m3(int head_dim, int n_rows, bool f32) {
    return head_dim == 64 ? pick<uint8_t, 64>(n_rows, f32) : pick<uint8_t, 128>(n_rows, f32);
}

}  // namespace rows
}  // namespace pkv
