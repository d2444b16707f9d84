// window_tc_kernel instantiation for head_dim 64, int8 cache.
#include "window_tc.cuh"

namespace pkv {
WindowFn window_tc_fn_d64_int8(size_t* smem, int* threads) {
    *smem = window_tc_smem<64, true>();
    *threads = TcTraits<64, true>::kThreads;
    return window_tc_kernel<64, true>;
}
}  // namespace pkv
