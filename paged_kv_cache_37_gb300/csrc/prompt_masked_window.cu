// prompt_masked_window.cu -- instances of prompt_masked.cuh: a window with sinks.
#include "prompt_masked.cuh"

namespace pkv {
namespace prompt_masked {

Kernels window_kernels(int D, bool q8, bool split, bool dual) {
    return D == 64 ? kernels_of<kMaskWindow, 64>(q8, split, dual) : kernels_of<kMaskWindow, 128>(q8, split, dual);
}

}  // namespace prompt_masked
}  // namespace pkv
