// Rows of the paged cache read back in token order (pkv_gather_kv), and the
// checks that the chunk entry points share.
//
// One CTA per (16 tokens, sequence), or several if that is few: their K and V rows
// of every kv head, 256 rows at a time. A thread first works out where one row lies and goes to --
// the divisions and the block table are paid once a row -- then the CTA moves
// the rows, 8 elements a thread and several loads in flight: consecutive
// threads take consecutive elements of the output, so that writes are whole
// lines and reads whole rows of a block. Bound by memory: every cached byte is
// read once and every output byte written once. Measured: 8 contexts of 30000 to
// 32768 tokens, 8 kv heads, d = 128, INT8 -> bf16, 1.55 GB in 250 us, 6.2 TB/s (a
// plain copy: 6.7); with the divisions in the copying loop 401 us.
#include <algorithm>

#include "batch.cuh"
#include "host.h"

namespace pkv {

struct GatherParams {
    BatchView bt;
    CacheView c;
    const int32_t* first;
    void* k_out;
    void* v_out;
    int64_t out_stride;
    int32_t ragged;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 16;

struct GatherRow {
    const uint8_t* src;  // nullptr: left out
    float scale;         // of a row of codes
    uint16_t v;          // to v_out
    uint16_t codes;      // INT8 codes; otherwise bf16 values (a bf16 pool, or the tail)
    int64_t dst;         // element offset in the outputs
};

template <int D, bool INT8, bool F32>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
    constexpr int CH = D / 8;  // pieces of 8 elements a row
    __shared__ int s_id[kGatherTokens];  // block of each token; -1: from the tail; -2: left out
    __shared__ GatherRow s_row[kGatherThreads];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    // one CTA a sequence at most, or the x-th of all sequences' CTAs and one
    // more that checks the lengths
    WorkItem it{int(blockIdx.x), 0};
    if (p.ragged) {
        if (blockIdx.x == gridDim.x - 1) {
            if (blockIdx.y == 0) check_lengths(p.bt, p.c.bs, p.c.err);
            return;
        }
        it = locate(int(blockIdx.x), p.bt.B, [&](int s) {
            return (seq_range(p.bt, s, p.c.bs, nullptr, false).n + kGatherTokens - 1) / kGatherTokens;
        });
        if (it.b < 0) return;
    }
    const int b = it.b;
    const SeqRange sq = seq_range(p.bt, b, p.c.bs, p.c.err, !p.ragged && tid == 0 && blockIdx.y == 0);
    const int i0 = it.i * kGatherTokens;
    if (i0 >= sq.n || (sq.bad && !p.first)) return;
    const int t_first = p.first ? p.first[b] : sq.ctx - sq.n;
    // with `first` the rows may be any range inside the context
    if (p.first && (t_first < 0 || sq.ctx < 0 || int64_t(sq.ctx) > int64_t(p.bt.max_blocks) * p.c.bs ||
                    int64_t(t_first) + sq.n > sq.ctx)) {
        if (tid == 0 && i0 == 0) report(p.c.err, kErrCtxLen);
        return;
    }
    const int m = min(kGatherTokens, sq.n - i0), Hkv = p.c.Hkv, bs = p.c.bs;
    const int slot = INT8 ? p.bt.slots[b] : 0;
    const int nfull = INT8 ? sq.ctx / bs * bs : sq.ctx;
    if (tid < m) {
        const int t = t_first + i0 + tid;
        int id = -1;
        if (t < nfull) {
            id = p.bt.tables[size_t(b) * p.bt.max_blocks + t / bs];
            if (id < 0 || id >= p.c.num_blocks) {
                report(p.c.err, kErrBlockId);
                id = -2;
            }
        } else if (slot < 0 || slot >= p.c.max_slots) {
            report(p.c.err, kErrSlot);
            id = -2;
        }
        s_id[tid] = id;
    }

    // rows in the order (token, kv head) of the outputs, all of K, then all of V
    const int per = m * Hkv;
    for (int r0 = int(blockIdx.y) * kGatherThreads; r0 < 2 * per; r0 += int(gridDim.y) * kGatherThreads) {
        const int rows = min(kGatherThreads, 2 * per - r0);
        __syncthreads();
        if (tid < rows) {
            const int kv = r0 + tid >= per, e = r0 + tid - kv * per, tl = e / Hkv, h = e % Hkv;
            const int id = s_id[tl], off = (t_first + i0 + tl) % bs;
            GatherRow r;
            r.src = nullptr;
            r.scale = 0.f;
            r.v = uint16_t(kv);
            r.codes = INT8 && id >= 0;
            r.dst = int64_t(sq.row0 + i0 + tl) * p.out_stride + h * D;
            if (id >= 0) {
                r.src = static_cast<const uint8_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                        ((size_t(id) * Hkv + h) * bs + off) * D * (INT8 ? 1 : 2);
                if (INT8) r.scale = __ldg(p.c.scales + (size_t(id) * Hkv + h) * 2 + kv);
            } else if (INT8 && id == -1) {
                r.src = reinterpret_cast<const uint8_t*>((kv ? p.c.v_tail : p.c.k_tail) +
                                                         ((size_t(slot) * Hkv + h) * bs + off) * D);
            }
            s_row[tid] = r;
        }
        __syncthreads();
        constexpr int NB = 8;  // loads in flight a thread
#pragma unroll 1
        for (int i = tid; i < rows * CH; i += NB * kGatherThreads) {
            uint4 w[NB];
#pragma unroll
            for (int u = 0; u < NB; ++u) {
                const int e = i + u * kGatherThreads;
                if (e >= rows * CH) break;
                const GatherRow& r = s_row[e / CH];
                if (!r.src) continue;
                if (INT8 && r.codes) {
                    const uint2 x = __ldg(reinterpret_cast<const uint2*>(r.src + e % CH * 8));
                    w[u].x = x.x;
                    w[u].y = x.y;
                } else {
                    w[u] = ldg128(r.src + e % CH * 16);
                }
            }
#pragma unroll
            for (int u = 0; u < NB; ++u) {
                const int e = i + u * kGatherThreads;
                if (e >= rows * CH) break;
                const GatherRow& r = s_row[e / CH];
                if (!r.src) continue;
                void* out = r.v ? p.v_out : p.k_out;
                const int64_t at = r.dst + e % CH * 8;
                if (!F32 && (!INT8 || !r.codes)) {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = w[u];
                    continue;
                }
                float2 x[4];
                if (INT8 && r.codes) {
                    s8x4_to_f4(w[u].x, x[0], x[1]);
                    s8x4_to_f4(w[u].y, x[2], x[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = make_float2(x[k].x * r.scale, x[k].y * r.scale);
                } else {
                    x[0] = bf16x2_to_f2(w[u].x);
                    x[1] = bf16x2_to_f2(w[u].y);
                    x[2] = bf16x2_to_f2(w[u].z);
                    x[3] = bf16x2_to_f2(w[u].w);
                }
                if (F32) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
                    o[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
                    o[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
                        make_uint4(f2_to_bf16x2(x[0].x, x[0].y), f2_to_bf16x2(x[1].x, x[1].y),
                                   f2_to_bf16x2(x[2].x, x[2].y), f2_to_bf16x2(x[3].x, x[3].y));
                }
            }
        }
    }
}

int check_batch(const pkv_cache_desc* c, const pkv_batch_desc* batch, BatchView* bt, CacheView* cv) {
    const int st = check_desc(c);
    if (st != PKV_OK) return st;
    if (!batch || batch->B < 0 || batch->num_tokens < 0 || batch->max_tokens < 0) return PKV_ERR_INVALID;
    *bt = BatchView{batch->token_starts, batch->block_tables, batch->ctx_lens, batch->slots, batch->B,
                    batch->max_blocks, batch->num_tokens, batch->max_tokens};
    *cv = CacheView{c->k_pool, c->v_pool, c->scales, static_cast<uint16_t*>(c->k_tail),
                    static_cast<uint16_t*>(c->v_tail), c->err_word, c->num_blocks, c->num_q_heads, c->num_kv_heads,
                    c->block_size, c->max_slots};
    if (batch->B == 0 || batch->num_tokens == 0 || batch->max_tokens == 0) return PKV_OK;
    if (!batch->token_starts || !batch->block_tables || !batch->ctx_lens) return PKV_ERR_INVALID;
    if (c->dtype == PKV_DTYPE_INT8 && !batch->slots) return PKV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(batch->token_starts) | reinterpret_cast<uintptr_t>(batch->block_tables) |
         reinterpret_cast<uintptr_t>(batch->ctx_lens) | reinterpret_cast<uintptr_t>(batch->slots)) & 3u)
        return PKV_ERR_INVALID;
    if (batch->B > 65535 || c->num_kv_heads > 65535 || batch->max_blocks <= 0) return PKV_ERR_INVALID;
    if (int64_t(batch->max_blocks) * c->block_size >= (int64_t(1) << 31) - 65536) return PKV_ERR_INVALID;
    if (batch->max_tokens > batch->num_tokens) return PKV_ERR_INVALID;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_gather_kv(const pkv_cache_desc* c, const pkv_batch_desc* batch, const int32_t* first, void* k_out,
                             void* v_out, int64_t out_stride, int32_t out_dtype, void* stream) {
    GatherParams p;
    const int st = check_batch(c, batch, &p.bt, &p.c);
    if (st != PKV_OK) return st;
    if (out_dtype != PKV_OUT_BF16 && out_dtype != PKV_OUT_FP32) return PKV_ERR_INVALID;
    if (batch->B == 0 || batch->num_tokens == 0 || batch->max_tokens == 0) return PKV_OK;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return PKV_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(first) & 3u) return PKV_ERR_INVALID;
    const bool f32 = out_dtype == PKV_OUT_FP32;
    if (out_stride < int64_t(c->num_kv_heads) * c->head_dim || out_stride % (f32 ? 4 : 8)) return PKV_ERR_INVALID;
    p.first = first;
    p.k_out = k_out;
    p.v_out = v_out;
    p.out_stride = out_stride;
    const int64_t most = (batch->max_tokens - 1) / kGatherTokens + 1;
    p.ragged = most > 1;
    const int64_t gx = std::min(most * batch->B, batch->num_tokens / kGatherTokens + int64_t(batch->B)) + p.ragged;
    // Many heads are several times 256 rows: other CTAs', where one for all does not
    // fill the GPU (4 fit on an SM). 16 contexts of 40 tokens, 32 kv heads, INT8:
    // 17.0 us -> 7.0 us; 8 of 300 tokens 17.4 -> 12.9; 8 of 1000, where one CTA for
    // all does fill it, 38.
    const int64_t rounds = (2 * kGatherTokens * int64_t(c->num_kv_heads) + kGatherThreads - 1) / kGatherThreads;
    const dim3 grid(unsigned(gx), unsigned(std::max<int64_t>(1, std::min(rounds, 152 * 4 / gx))));
    const bool int8 = c->dtype == PKV_DTYPE_INT8;
    void (*fn)(GatherParams) = nullptr;
    if (c->head_dim == 128)
        fn = int8 ? (f32 ? gather_kernel<128, true, true> : gather_kernel<128, true, false>)
                  : (f32 ? gather_kernel<128, false, true> : gather_kernel<128, false, false>);
    else
        fn = int8 ? (f32 ? gather_kernel<64, true, true> : gather_kernel<64, true, false>)
                  : (f32 ? gather_kernel<64, false, true> : gather_kernel<64, false, false>);
    return launch(fn, grid, dim3(kGatherThreads), 0, static_cast<cudaStream_t>(stream), p);
}
