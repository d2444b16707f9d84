// window_tc_kernel instantiation for head_dim 128, int8 cache.
#include "window_tc.cuh"

namespace pkv {
WindowFn window_tc_fn_d128_int8(size_t* smem, int* threads) {
    *smem = window_tc_smem<128, true>();
    *threads = TcTraits<128, true>::kThreads;
    return window_tc_kernel<128, true>;
}
}  // namespace pkv
