// A batch of sequences that each bring n_b new tokens (pkv_batch_desc), as the
// chunk kernels see it. Row token_starts[b] + i of the token arrays is token
// ctx_lens[b] - n_b + i of sequence b.
#pragma once

#include <cstdint>

#include "kernels.cuh"

namespace pkv {

constexpr int kErrBatch = 32;

struct BatchView {
    const int32_t* starts;   // [B + 1]
    const int32_t* tables;   // [B][max_blocks]
    const int32_t* ctx;      // [B]
    const int32_t* slots;    // [B] (INT8)
    int32_t B, max_blocks, num_tokens, max_tokens;
};

// The cache as the chunk kernels see it.
struct CacheView {
    void* k_pool;
    void* v_pool;
    float* scales;
    uint16_t* k_tail;
    uint16_t* v_tail;
    int32_t* err;
    int32_t num_blocks, Hq, Hkv, bs, max_slots;
};

struct SeqRange {
    int row0;  // first row of the sequence in the token arrays
    int n;     // its rows (0 where the batch's arrays do not hold together)
    int ctx;   // its tokens in the cache, the new ones included
    bool bad;  // the context length does not hold its rows: n is kept, the rows have no tokens
};

// Sequence b of the batch, its lengths checked. `reporter`: one thread of the grid.
__device__ __forceinline__ SeqRange seq_range(const BatchView& bt, int b, int bs, int32_t* err, bool reporter) {
    SeqRange s;
    s.row0 = bt.starts[b];
    const int end = bt.starts[b + 1];
    s.ctx = bt.ctx[b];
    s.n = end - s.row0;
    s.bad = false;
    if (s.row0 < 0 || end < s.row0 || end > bt.num_tokens || s.n > bt.max_tokens) {
        if (reporter) report(err, kErrBatch);
        s.n = 0;
        s.row0 = 0;
    }
    if (s.n > 0 && (s.ctx < s.n || int64_t(s.ctx) > int64_t(bt.max_blocks) * bs)) {
        if (reporter) report(err, kErrCtxLen);
        s.bad = true;
    }
    return s;
}

}  // namespace pkv
