// prompt_masked_window.cu -- instances of prompt_masked.cuh: a window with sinks.
#include "prompt_masked.cuh"

namespace pkv {
namespace prompt_masked {

Kernels window_kernels(int D, bool q8, bool split) {
    return D == 64 ? kernels_of<kMaskWindow, 64>(q8, split) : kernels_of<kMaskWindow, 128>(q8, split);
}

}  // namespace prompt_masked
}  // namespace pkv
