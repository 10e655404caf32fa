// rows_attention_f16_d64_tree.cu -- instances of rows_attention.cuh: fp16 pools, head_dim 64, a tree of drafts.
#include "rows_attention.cuh"

namespace pkv {
namespace rows {

Kernel kernel_f16_d64_tree(int n_rows, bool f32, bool paged) {
    return pick<__half, 64, kMaskTree>(n_rows, f32, paged);
}

}  // namespace rows
}  // namespace pkv
