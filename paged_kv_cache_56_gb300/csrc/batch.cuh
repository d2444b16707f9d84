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

// Work of ragged sequences as one list: sequence 0's count(0) items, then
// sequence 1's, and so on. Finds item `item`; every lane of the warp calls it
// and gets the same answer. b == -1: past the end.
struct WorkItem {
    int b, i;
};
template <class Count>
__device__ __forceinline__ WorkItem locate(int item, int B, Count count) {
    const int lane = int(threadIdx.x) & 31;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int mine = b0 + lane < B ? count(b0 + lane) : 0;
        int upto = mine;  // items of this lane's sequence and those before it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += x;
        }
        const uint32_t past = __ballot_sync(kFull, item < upto);
        if (past) {
            const int l = __ffs(past) - 1;
            return WorkItem{b0 + l, item - __shfl_sync(kFull, upto - mine, l)};
        }
        item -= __shfl_sync(kFull, upto, 31);
    }
    return WorkItem{-1, 0};
}

// The same list for a warp that looks up many items, near each other: it knows how
// many there are and keeps the 32 sequences around the item before, so that a walk
// through the list reads each sequence's lengths once or twice, not once an item.
template <class Count>
struct ListCursor {
    Count count;
    int B, b0;               // the group of sequences b0 .. b0 + 31: a lane has one
    int mine, upto, sum;     // its items, those up to its end, the group's
    long long before, total; // items before the group; of all sequences
    __device__ __forceinline__ void load(int b) {
        const int lane = int(threadIdx.x) & 31;
        b0 = b;
        mine = b + lane < B ? count(b + lane) : 0;
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += x;
        }
        sum = __shfl_sync(kFull, upto, 31);
    }
    __device__ __forceinline__ ListCursor(int B_, Count count_) : count(count_), B(B_) {
        const int lane = int(threadIdx.x) & 31, end = (B - 1) / 32 * 32;  // begins at the last group
        before = 0;
#pragma unroll 4
        for (int b = 0; b < end; b += 32) before += count(b + lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
        load(end);
        total = before + sum;
    }
    // Item `item` < total; b == -1 if the lengths have changed meanwhile.
    __device__ __forceinline__ WorkItem find(long long item) {
        while (item < before && b0 > 0) {
            load(b0 - 32);
            before -= sum;
        }
        while (item >= before + sum && b0 + 32 < B) {
            before += sum;
            load(b0 + 32);
        }
        const int at = int(item - before);
        const uint32_t past = __ballot_sync(kFull, at < upto);
        if (at < 0 || !past) return WorkItem{-1, 0};
        const int l = __ffs(past) - 1;
        return WorkItem{b0 + l, at - __shfl_sync(kFull, upto - mine, l)};
    }
};

// Reports what is wrong with the batch's lengths: one CTA a launch.
__device__ __forceinline__ void check_lengths(const BatchView& bt, int bs, int32_t* err) {
    for (int b = int(threadIdx.x); b < bt.B; b += int(blockDim.x)) (void)seq_range(bt, b, bs, err, true);
}

}  // namespace pkv
