// prompt_masked_tree.cu -- instances of prompt_masked.cuh: a tree of drafts.
#include "prompt_masked.cuh"

namespace pkv {
namespace prompt_masked {

Kernels tree_kernels(int D, bool q8, bool split, bool dual) {
    return D == 64 ? kernels_of<kMaskTree, 64>(q8, split, dual) : kernels_of<kMaskTree, 128>(q8, split, dual);
}

}  // namespace prompt_masked
}  // namespace pkv
