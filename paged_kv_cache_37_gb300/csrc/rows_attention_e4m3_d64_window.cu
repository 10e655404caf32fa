// rows_attention_e4m3_d64_window.cu -- instances of rows_attention.cuh: e4m3 pools, head_dim 64, a window with sinks.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_e4m3_d64_window(int n_rows, bool f32, bool paged) {
    return pick<uint8_t, 64, kMaskWindow>(n_rows, f32, paged);
}

}  // namespace rows
}  // namespace pkv
