// window_rows_kernel instantiations for head_dim 128, bf16 cache.
#include "window_rows.cuh"

namespace pkv {
WindowFn window_rows_fn_d128_bf16(int nt, bool hook) { return window_rows_pick<128, false>(nt, hook); }
}  // namespace pkv
