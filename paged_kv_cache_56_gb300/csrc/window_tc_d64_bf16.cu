// window_tc_kernel instantiation for head_dim 64, bf16 cache.
#include "window_tc.cuh"

namespace pkv {
WindowFn window_tc_fn_d64_bf16(size_t* smem, int* threads) {
    *smem = window_tc_smem<64, false>();
    *threads = TcTraits<64, false>::kThreads;
    return window_tc_kernel<64, false>;
}
}  // namespace pkv
