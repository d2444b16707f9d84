// window_rows_kernel instantiations for head_dim 64, bf16 cache.
#include "window_rows.cuh"

namespace pkv {
WindowFn window_rows_fn_d64_bf16(int nt, bool hook) { return window_rows_pick<64, false>(nt, hook); }
}  // namespace pkv
