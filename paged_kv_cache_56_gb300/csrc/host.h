// Host-side helpers shared by the library's translation units: descriptor
// checks, kernel launches and tensor maps.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include <atomic>
#include <cstdint>
#include <utility>

#include "../../include/pkv.h"

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_desc(const pkv_cache_desc* c);

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

extern std::atomic<int> g_pdl;
extern std::atomic<int> g_skip_copy;  // pkv_debug_skip_copy

// Launches with the programmatic-stream-serialization attribute when enabled
// (pkv_set_programmatic_launch), plainly otherwise.
template <typename... Params, typename... Args>
int launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    if (g_pdl.load(std::memory_order_relaxed)) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

// Checks a cache and a batch descriptor and fills the kernels' views of them.
// A batch without sequences or rows passes with its arrays unlooked at.
struct BatchView;
struct CacheView;
int check_batch(const pkv_cache_desc* c, const pkv_batch_desc* batch, BatchView* bt, CacheView* cv);

// cuTensorMapEncodeTiled, or nullptr if the driver does not offer it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Tensor map of a pool for box_rows x 128-byte boxes (kept per thread).
int pool_tensor_map(const void* pool, int32_t num_blocks, int32_t rows, int32_t row_bytes, CUtensorMap* out,
                    int32_t box_rows = 16);

}  // namespace pkv
