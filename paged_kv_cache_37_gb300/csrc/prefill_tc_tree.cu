// prefill_tc_tree.cu -- instances of prefill_tc.cuh: a tree of drafts.
#include "prefill_tc.cuh"

namespace pkv {
namespace prefill_tc {

Kernels tree_kernels(int D, bool q8, bool split) {
    return D == 64 ? masked<kMaskTree, 64>(q8, split) : masked<kMaskTree, 128>(q8, split);
}

}  // namespace prefill_tc
}  // namespace pkv
