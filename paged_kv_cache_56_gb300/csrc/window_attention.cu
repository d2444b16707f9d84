// Entry points of the windowed attention: argument checks, the choice of the
// kernel and of the split, and the launch.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "host.h"
#include "window.cuh"

namespace pkv {

WindowFn window_rows_fn_d64_bf16(int nt, bool hook);
WindowFn window_rows_fn_d64_int8(int nt, bool hook);
WindowFn window_rows_fn_d128_bf16(int nt, bool hook);
WindowFn window_rows_fn_d128_int8(int nt, bool hook);
WindowFn window_tc_fn_d64_bf16(size_t* smem, int* threads);
WindowFn window_tc_fn_d128_bf16(size_t* smem, int* threads);
WindowFn window_tc_fn_d64_int8(size_t* smem, int* threads);
WindowFn window_tc_fn_d128_int8(size_t* smem, int* threads);

int prepare_kernel(const void* f, size_t smem, int threads, int launch_regs, int* ctas) {
    struct Entry {
        const void* fn;
        int dev;
        int ctas;
    };
    static std::mutex mu;
    static Entry seen[256];
    static int n = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (seen[i].fn == f && seen[i].dev == dev) {
            *ctas = seen[i].ctas;
            return PKV_OK;
        }
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess ||
        cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, int(cudaSharedmemCarveoutMaxShared)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, f, threads, smem) != cudaSuccess)
        return PKV_ERR_CUDA;
    // the warpgroups of window_tc_kernel and prompt_kernel share out the registers that the block was
    // launched with, and would wait forever for more than that
    cudaFuncAttributes at;
    if (launch_regs > 0 && (cudaFuncGetAttributes(&at, f) != cudaSuccess || at.numRegs != launch_regs))
        return PKV_ERR_CUDA;
    if (n < 256) seen[n++] = Entry{f, dev, *ctas};
    return PKV_OK;
}

int sm_count(int* out) {
    static std::atomic<int> known[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return PKV_ERR_CUDA;
        known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return PKV_OK;
}

int encode_map(CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box, CUtensorMap* out) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    return enc && enc(out, type, rank, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_ERR_CUDA;
}

int rows_tensor_map(int group, int kv_heads, int head_dim, int tokens, const void* base, int64_t stride, int rows,
                    CUtensorMap* out) {
    const cuuint64_t g = cuuint64_t(group), d = cuuint64_t(head_dim);
    const cuuint64_t dims[4] = {d, g, cuuint64_t(kv_heads), cuuint64_t(tokens)};
    const cuuint64_t strides[3] = {d * 2, g * d * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[4] = {64, cuuint32_t(g), 1, cuuint32_t(rows / g)};
    return encode_map(CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, out);
}

namespace {

constexpr int kMaxSplits = 128;  // the merge holds 16 rows' weights of every split in a CTA's rings
// Arrival counters at the front of every workspace, whatever the call, so
// that calls of other shapes may share it: each leaves its counters at zero
// and no call's partial results lie on another's counters. A batch of more
// row tiles than this fills the GPU without splits and is not split.
constexpr int kCounters = 16384;

struct Plan {
    WindowFn fn;
    size_t smem;
    int threads;
    bool tc;          // window_tc_kernel
    int row_tiles;    // row tiles of max_tokens tokens
    int key_tiles;    // most 16-token tiles that one row tile sees
    int64_t n;        // tc: items (row tile, kv head), as many as the batch is likely to have
    int64_t most;     // ... as it can have
    int64_t split_items;  // ... the last ones, that split_tokens > 0 splits
    int ctas_per_sm;
};

// Most 16-token tiles in the list of keys (in units of `unit` tokens) that
// `span` tokens in a row see.
int most_key_tiles(const pkv_cache_desc* c, const pkv_batch_desc* bt, int window, int sinks, int span, int unit) {
    const int64_t all = int64_t(bt->max_blocks) * c->block_size / kTile;
    if (window <= 0) return int(all);
    const int64_t seen = (int64_t(window) + span + unit - 2) / unit + 1 + (int64_t(sinks) + unit - 1) / unit;
    return int(std::min(all, seen * (unit / kTile)));
}

int make_plan(const pkv_cache_desc* c, const pkv_batch_desc* bt, int window, int sinks, Plan* pl, bool hook = false) {
    const bool int8 = c->dtype == PKV_DTYPE_INT8;
    const int g = c->num_q_heads / c->num_kv_heads;
    const int64_t rows = int64_t(bt->max_tokens) * g;
    // The row kernel reads each key once for up to 16 rows and is bound by that;
    // more rows would have it read them again, and the tensor cores take over.
    // Measured, 16 sequences of 7000 tokens, 8 kv heads, d = 128, bf16 / INT8, us:
    //   rows              16          32          64
    //   row kernel      82 /  68   136 / 135   278 / 259
    //   tensor cores    88 / 121    88 / 121    88 / 121
    // and 64 sequences of 1000 tokens: 62 / 57 against 64 / 80 with 16 rows, 81 / 85
    // against 64 / 80 with 32.
    pl->tc = rows > 16;
    if (pl->tc) {
        if (c->head_dim == 128)
            pl->fn = int8 ? window_tc_fn_d128_int8(&pl->smem, &pl->threads) : window_tc_fn_d128_bf16(&pl->smem, &pl->threads);
        else
            pl->fn = int8 ? window_tc_fn_d64_int8(&pl->smem, &pl->threads) : window_tc_fn_d64_bf16(&pl->smem, &pl->threads);
        pl->row_tiles = int((rows + 255) / 256);
        // One CTA a SM walks through the items, so all but the last n % SMs of them
        // keep every SM busy as they are; those are split. (Ragged batches: the rows of
        // num_tokens, and half a row tile more a sequence, or one a sequence.)
        int sms = 0;
        const int st = sm_count(&sms);
        if (st != PKV_OK) return st;
        const int64_t tiles = int64_t(pl->row_tiles) * bt->B;
        pl->n = std::min(tiles, std::max<int64_t>(bt->B, (bt->num_tokens * int64_t(g) + 128 * int64_t(bt->B) + 255) / 256)) *
                c->num_kv_heads;
        pl->most = std::min(tiles, bt->num_tokens * int64_t(g) / 256 + bt->B) * c->num_kv_heads;
        pl->split_items = pl->n < sms ? pl->most : pl->n % sms;
        pl->key_tiles = most_key_tiles(c, bt, window, sinks, int(std::min<int64_t>(256 / g, bt->max_tokens)), c->block_size);
        return prepare_kernel(reinterpret_cast<const void*>(pl->fn), pl->smem, pl->threads, int8 ? kTcLaunchRegsInt8 : kTcLaunchRegsBf16,
                              &pl->ctas_per_sm);
    }
    // up to 8 rows in tiles of 16 (the first of these): 81 / 66 us against 78 / 50 us
    const int nt = rows <= 8 ? 1 : 2;
    if (c->head_dim == 128) pl->fn = int8 ? window_rows_fn_d128_int8(nt, hook) : window_rows_fn_d128_bf16(nt, hook);
    else pl->fn = int8 ? window_rows_fn_d64_int8(nt, hook) : window_rows_fn_d64_bf16(nt, hook);
    if (!pl->fn) return PKV_ERR_UNSUPPORTED;
    pl->smem = window_rows_smem(c->head_dim, int8);
    pl->threads = kThreads;
    pl->row_tiles = int((rows + 8 * nt - 1) / (8 * nt));
    pl->key_tiles = most_key_tiles(c, bt, window, sinks, std::max(1, 8 * nt / g), kTile);
    return prepare_kernel(reinterpret_cast<const void*>(pl->fn), pl->smem, pl->threads, 0, &pl->ctas_per_sm);
}

int max_splits_of(const pkv_cache_desc* c, const pkv_batch_desc* bt, const Plan& pl, int split_tokens) {
    if (split_tokens <= 0) return 1;
    const int64_t split = pl.tc ? pl.split_items : int64_t(bt->B) * c->num_kv_heads * pl.row_tiles;
    if (split == 0 || split > kCounters) return 1;
    const int tiles = split_tokens / kTile;
    return std::min(kMaxSplits, (pl.key_tiles + tiles - 1) / tiles);
}

struct Workspace {
    size_t ml, o, total;
};

Workspace workspace_of(const pkv_cache_desc* c, const pkv_batch_desc* bt, const Plan& pl, int max_splits) {
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Workspace w;
    const size_t rows = pl.tc ? size_t(pl.split_items) * 256 : size_t(bt->num_tokens) * c->num_q_heads;
    w.ml = up(rows * max_splits * 8);
    w.o = rows * max_splits * c->head_dim * 4;
    w.total = max_splits > 1 ? size_t(kCounters) * 4 + w.ml + w.o : 0;
    return w;
}

int check_window(const pkv_cache_desc* c, const pkv_batch_desc* batch, int window, int sinks, int split_tokens,
                 BatchView* bt, CacheView* cv) {
    const int st = check_batch(c, batch, bt, cv);
    if (st != PKV_OK) return st;
    if (window < 0 || sinks < 0 || split_tokens < 0 || split_tokens % kTile) return PKV_ERR_INVALID;
    return PKV_OK;
}

// ... of the partial outputs: [rows][splits][d] fp32, boxes of 32 rows x 32 elements.
int partials_tensor_map(const pkv_cache_desc* c, int64_t rows, int splits, const void* base, CUtensorMap* out) {
    const cuuint64_t d = cuuint64_t(c->head_dim);
    const cuuint64_t dims[3] = {d, cuuint64_t(splits), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {d * 4, cuuint64_t(splits) * d * 4};
    const cuuint32_t box[3] = {32, 1, 32};
    return encode_map(CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, out);
}

bool is_empty(const pkv_batch_desc* b) { return b->B == 0 || b->num_tokens == 0 || b->max_tokens == 0; }

}  // namespace

size_t window_rows_smem(int d, bool int8) {
    if (d == 64)
        return int8 ? DecodeTraits<64, true>::kAlignSlack + size_t(kWarps) * DecodeTraits<64, true>::kStages * DecodeTraits<64, true>::kStageBytes
                    : DecodeTraits<64, false>::kAlignSlack + size_t(kWarps) * DecodeTraits<64, false>::kStages * DecodeTraits<64, false>::kStageBytes;
    return int8 ? DecodeTraits<128, true>::kAlignSlack + size_t(kWarps) * DecodeTraits<128, true>::kStages * DecodeTraits<128, true>::kStageBytes
                : DecodeTraits<128, false>::kAlignSlack + size_t(kWarps) * DecodeTraits<128, false>::kStages * DecodeTraits<128, false>::kStageBytes;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_window_split_tokens(const pkv_cache_desc* c, const pkv_batch_desc* batch, int32_t window, int32_t sinks) {
    BatchView bt;
    CacheView cv;
    int st = check_window(c, batch, window, sinks, 0, &bt, &cv);
    if (st != PKV_OK) return st;
    if (is_empty(batch)) return 0;
    Plan pl;
    int sms = 0;
    if ((st = make_plan(c, batch, window, sinks, &pl)) != PKV_OK || (st = sm_count(&sms)) != PKV_OK) return st;
    if (pl.tc) {
        // The last r items in s parts each take ceil(r s / SMs) rounds of (key tiles / s
        // + o) tiles' time, where o stands for an item's beginning and end: 2.5, or with
        // the partial rows written, read back and merged 5.5 and as much again for 256
        // rows as there are parts, measured over items of 8 to 250 tiles and 24 to 256
        // rows. The s that makes it least. (In quarters of a tile.)
        const int64_t r = pl.n < sms ? pl.n : pl.split_items, tiles = (pl.key_tiles + 7) / 8;
        const int64_t rows = std::min<int64_t>(256, int64_t(batch->max_tokens) * (c->num_q_heads / c->num_kv_heads));
        int64_t best = 0, split = 1;
        for (int64_t s = 1; s <= std::min<int64_t>(tiles / 2, kMaxSplits); ++s) {
            const int64_t o = s > 1 ? 22 + s * std::max<int64_t>(1, rows / 64) : 10;
            const int64_t cost = (r * s + sms - 1) / sms * (4 * ((tiles + s - 1) / s) + o);
            if (s == 1 || cost < best) {
                best = cost;
                split = s;
            }
        }
        return split <= 1 ? 0 : int((tiles + split - 1) / split * 128);
    }
    const int64_t units = int64_t(batch->B) * c->num_kv_heads * pl.row_tiles;
    const int64_t splits = int64_t(sms) * pl.ctas_per_sm / units;
    if (splits <= 1) return 0;
    // at least two tiles a warp: shorter splits spend their time on the start and the merge
    const int64_t tiles = std::max<int64_t>((pl.key_tiles + splits - 1) / splits, 2 * kWarps);
    return tiles >= pl.key_tiles ? 0 : int(tiles * kTile);
}

size_t pkv_window_ws_bytes(const pkv_cache_desc* c, const pkv_batch_desc* batch, int32_t window, int32_t sinks,
                           int32_t split_tokens) {
    BatchView bt;
    CacheView cv;
    Plan pl;
    if (check_window(c, batch, window, sinks, split_tokens, &bt, &cv) != PKV_OK || is_empty(batch) ||
        make_plan(c, batch, window, sinks, &pl) != PKV_OK)
        return 0;
    return workspace_of(c, batch, pl, max_splits_of(c, batch, pl, split_tokens)).total;
}

int pkv_window_attention(const pkv_cache_desc* c, const pkv_batch_desc* batch, const void* q, int64_t q_stride,
                         int32_t window, int32_t sinks, float sm_scale, int32_t split_tokens, void* ws,
                         size_t ws_bytes, void* out, int64_t out_stride, void* stream) {
    WindowParams p;
    int st = check_window(c, batch, window, sinks, split_tokens, &p.bt, &p.c);
    if (st != PKV_OK) return st;
    if (!(sm_scale >= 0.f) || sm_scale > 3.0e38f) return PKV_ERR_INVALID;
    if (is_empty(batch)) return PKV_OK;
    const int64_t row = int64_t(c->num_q_heads) * c->head_dim;
    if (!q || !out || !aligned16(q) || !aligned16(out) || q_stride < row || out_stride < row ||
        ((q_stride | out_stride) & 7))
        return PKV_ERR_INVALID;
    if (q == out && q_stride != out_stride) return PKV_ERR_INVALID;
    Plan pl;
    p.skip_copy = g_skip_copy.load(std::memory_order_relaxed);
    if ((st = make_plan(c, batch, window, sinks, &pl, p.skip_copy >= 0)) != PKV_OK) return st;
    const int splits = max_splits_of(c, batch, pl, split_tokens);
    // window_tc_kernel's planner and warps without rows wait for as long as an item
    // takes, a second at most; 2^25 tokens take about half of that
    const int parts = pl.tc && pl.split_items < pl.most ? 1 : splits;
    if (pl.tc && (pl.key_tiles + parts - 1) / parts > (1 << 25) / kTile) return PKV_ERR_UNSUPPORTED;
    const Workspace w = workspace_of(c, batch, pl, splits);
    if (w.total > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < w.total)) return PKV_ERR_INVALID;

    const bool int8 = c->dtype == PKV_DTYPE_INT8;
    const int32_t row_bytes = c->head_dim * (int8 ? 1 : 2);
    if (pl.tc) {
        const int32_t rows = c->num_kv_heads * c->block_size;
        if (!int8) {
            if ((st = pool_tensor_map(c->k_pool, c->num_blocks, rows, row_bytes, &p.tm_k, c->block_size)) != PKV_OK) return st;
            if ((st = pool_tensor_map(c->v_pool, c->num_blocks, rows, row_bytes, &p.tm_v, c->block_size)) != PKV_OK) return st;
        }
        if ((st = rows_tensor_map(c->num_q_heads / c->num_kv_heads, c->num_kv_heads, c->head_dim, batch->num_tokens, q, q_stride, 128, &p.tm_q)) != PKV_OK) return st;
        if ((st = rows_tensor_map(c->num_q_heads / c->num_kv_heads, c->num_kv_heads, c->head_dim, batch->num_tokens, out, out_stride, 32, &p.tm_out)) != PKV_OK) return st;
    } else if (row_bytes >= 128) {
        const int32_t rows = c->num_kv_heads * c->block_size;
        if ((st = pool_tensor_map(c->k_pool, c->num_blocks, rows, row_bytes, &p.tm_k)) != PKV_OK) return st;
        if ((st = pool_tensor_map(c->v_pool, c->num_blocks, rows, row_bytes, &p.tm_v)) != PKV_OK) return st;
    } else {
        std::memset(&p.tm_k, 0, sizeof(p.tm_k));
        std::memset(&p.tm_v, 0, sizeof(p.tm_v));
    }
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    auto* bytes = static_cast<uint8_t*>(ws);
    p.ws_count = splits > 1 ? reinterpret_cast<int32_t*>(bytes) : nullptr;
    p.ws_ml = splits > 1 ? reinterpret_cast<float*>(bytes + kCounters * 4) : nullptr;
    p.ws_o = splits > 1 ? reinterpret_cast<float*>(bytes + kCounters * 4 + w.ml) : nullptr;
    p.window = window > 0 ? window : 0x7FFFFFFF;
    p.sinks = window > 0 ? sinks : 0;
    p.split_tiles = splits > 1 ? split_tokens / kTile : 0;
    p.max_splits = splits;
    p.row_tiles = pl.row_tiles;
    // never 0 or infinite: a hidden token's score is -infinity, and 0 times that is
    // not a number, nor is an infinite scale times a score of 0
    p.qscale = std::min(std::max(sm_scale * 1.4426950408889634f, 1e-37f), 3.4e38f);
    // window_tc_kernel: the row tiles of all sequences are one list
    p.item_tiles = p.split_items = 0;
    int64_t gx = int64_t(pl.row_tiles) * splits;
    if (pl.tc) {
        p.split_items = splits > 1 ? int(pl.split_items) : 0;
        if (splits > 1 && (st = partials_tensor_map(c, pl.split_items * 256, splits, p.ws_o, &p.tm_ws)) != PKV_OK) return st;
        gx = pl.most + int64_t(p.split_items) * (splits - 1);
        p.item_tiles = int(pl.most / c->num_kv_heads);
    }
    if (gx > 0x7FFFFFFF) return PKV_ERR_INVALID;
    // A CTA drops items that the batch does not have at 0.4 us each, while its other
    // warps wait: 2^27 items on 152 SMs are 0.35 s of the second that they do.
    if (pl.tc && gx > int64_t(1) << 27) return PKV_ERR_UNSUPPORTED;
    const dim3 grid(unsigned(gx), pl.tc ? 1u : unsigned(c->num_kv_heads), pl.tc ? 1u : unsigned(batch->B));
    return launch(pl.fn, grid, dim3(unsigned(pl.threads)), pl.smem, static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
