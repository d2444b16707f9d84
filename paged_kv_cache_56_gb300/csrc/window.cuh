// Attention of a batch's new tokens over the paged cache, causal, with an
// optional sliding window and a few first tokens that stay visible
// (pkv_window_attention): what its kernels share.
//
// Row r of (sequence b, kv head) is query head r % G of the group, of new
// token r / G: its position is p = ctx - n + r / G and it sees the tokens
//   t <= p  and  (p - t < window  or  t < sinks).
// The rows of a tile see one stretch of tokens up to the last row's position
// and, before it, the sinks; a tile's keys are walked as 16-token tiles of
// that list, so tokens between the sinks and the window are neither read nor
// looked up in the block table.
#pragma once

#include "batch.cuh"

namespace pkv {

struct WindowParams {
    CUtensorMap tm_k;  // the pools, as in DecodeParams
    CUtensorMap tm_v;
    // window_tc_kernel:
    CUtensorMap tm_q;    // q as [tokens][Hkv][G][D], boxes of 128 rows x 64 elements
    CUtensorMap tm_out;  // out likewise, boxes of 32 rows
    CUtensorMap tm_ws;   // ws_o, boxes of 32 rows x one split x 32 elements
    BatchView bt;
    CacheView c;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    float* ws_o;        // [rows][max_splits][D] partial outputs; rows: of q, of all heads
    float* ws_ml;       // [rows][max_splits][2]     (window_tc_kernel: of the items that are split)
    int32_t* ws_count;  // arrivals at each (sequence, kv head, row tile)
    int32_t window;     // INT32_MAX: none
    int32_t sinks;
    int32_t split_tiles;  // 16-token tiles a split (0: no split)
    int32_t max_splits;
    int32_t row_tiles;  // row tiles of max_tokens tokens
    int32_t item_tiles;   // window_tc_kernel: row tiles that the batch can have; the list of those it
    int32_t split_items;  // has, with each kv head, ends in this many that are split
    float qscale;       // sm_scale * log2(e)
    int32_t skip_copy;  // pkv_debug_skip_copy (-1: off)
};

// The 16-token tiles that rows of positions p_first .. p_last see, as a list.
struct KeyTiles {
    int nsink;  // leading tiles of sinks, tiles 0 .. nsink-1 of the context
    int lo;     // then the context's tiles lo ..
    int n;      // tiles in all
    __device__ __forceinline__ int tile(int k) const { return k < nsink ? k : k - nsink + lo; }
};

// `unit`: tokens a tile of the list is aligned to (16, or the block size).
__device__ __forceinline__ KeyTiles key_tiles(int p_first, int p_last, int window, int sinks, int unit) {
    KeyTiles kt;
    const int lo = max(0, p_first - window + 1);
    const int s = min(sinks, lo);
    kt.lo = lo / unit;
    kt.nsink = (s + unit - 1) / unit;
    if (kt.nsink >= kt.lo && s > 0) kt.nsink = kt.lo = 0;  // no gap
    kt.n = kt.nsink + p_last / unit - kt.lo + 1;
    return kt;
}

// Registers a thread that window_tc_kernel is launched with.
constexpr int kTcLaunchRegsBf16 = 168;
constexpr int kTcLaunchRegsInt8 = 128;

using WindowFn = void (*)(WindowParams);

size_t window_rows_smem(int d, bool int8);

}  // namespace pkv
