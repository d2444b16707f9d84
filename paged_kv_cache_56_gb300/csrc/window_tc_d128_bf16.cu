// window_tc_kernel instantiation for head_dim 128, bf16 cache.
#include "window_tc.cuh"

namespace pkv {
WindowFn window_tc_fn_d128_bf16(size_t* smem, int* threads) {
    *smem = window_tc_smem<128, false>();
    *threads = TcTraits<128, false>::kThreads;
    return window_tc_kernel<128, false>;
}
}  // namespace pkv
