// rows_attention_e4m3_d128_tree.cu -- instances of rows_attention.cuh: e4m3 pools, head_dim 128, a tree of drafts.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_e4m3_d128_tree(int n_rows, bool f32, bool paged) {
    return pick<uint8_t, 128, kMaskTree>(n_rows, f32, paged);
}

}  // namespace rows
}  // namespace pkv
