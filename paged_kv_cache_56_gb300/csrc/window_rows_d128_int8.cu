// window_rows_kernel instantiations for head_dim 128, int8 cache.
#include "window_rows.cuh"

namespace pkv {
WindowFn window_rows_fn_d128_int8(int nt, bool hook) { return window_rows_pick<128, true>(nt, hook); }
}  // namespace pkv
