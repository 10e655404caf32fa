// rows_attention_f16_d64_window.cu -- instances of rows_attention.cuh: fp16 pools, head_dim 64, a window with sinks.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_f16_d64_window(int n_rows, bool f32, bool paged) {
    return pick<__half, 64, kMaskWindow>(n_rows, f32, paged);
}

}  // namespace rows
}  // namespace pkv
