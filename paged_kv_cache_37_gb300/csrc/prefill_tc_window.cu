// prefill_tc_window.cu -- instances of prefill_tc.cuh: a window with sinks.
#include "prefill_tc.cuh"

namespace pkv {
namespace prefill_tc {

Kernels window_kernels(int D, bool q8, bool split) {
    return D == 64 ? masked<kMaskWindow, 64>(q8, split) : masked<kMaskWindow, 128>(q8, split);
}

}  // namespace prefill_tc
}  // namespace pkv
