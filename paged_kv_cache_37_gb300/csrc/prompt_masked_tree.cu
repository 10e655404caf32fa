// prompt_masked_tree.cu -- instances of prompt_masked.cuh: a tree of drafts.
#include "prompt_masked.cuh"

namespace pkv {
namespace prompt_masked {

Kernels tree_kernels(int D, bool q8, bool split) {
    return D == 64 ? kernels_of<kMaskTree, 64>(q8, split) : kernels_of<kMaskTree, 128>(q8, split);
}

}  // namespace prompt_masked
}  // namespace pkv
