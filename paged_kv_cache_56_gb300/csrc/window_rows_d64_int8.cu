// window_rows_kernel instantiations for head_dim 64, int8 cache.
#include "window_rows.cuh"

namespace pkv {
WindowFn window_rows_fn_d64_int8(int nt, bool hook) { return window_rows_pick<64, true>(nt, hook); }
}  // namespace pkv
