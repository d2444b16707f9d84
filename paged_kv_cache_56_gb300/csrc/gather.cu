// Rows of the paged cache read back in token order (pkv_gather_kv), and the
// checks that the chunk entry points share.
//
// One CTA per (16 tokens, sequence): their K and V rows of every kv head. A
// thread moves 16 elements at a time -- 16 bytes of an INT8 row, 32 of a bf16
// one -- with several loads in flight; consecutive threads take consecutive
// elements of the output rows, so that the writes are whole lines and the
// reads whole rows of a block. Bound by memory: every cached byte is read
// once and every output byte written once.
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
};

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 16;

// 16 values as two bf16 pairs of words each, stored as bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void store16(void* out, int64_t at, const float (&x)[16]) {
    if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            o[e] = make_uint4(f2_to_bf16x2(x[8 * e], x[8 * e + 1]), f2_to_bf16x2(x[8 * e + 2], x[8 * e + 3]),
                              f2_to_bf16x2(x[8 * e + 4], x[8 * e + 5]), f2_to_bf16x2(x[8 * e + 6], x[8 * e + 7]));
    }
}

__device__ __forceinline__ void bf16x8_to_f(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_f2(u[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}

template <int D, bool INT8, bool F32>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
    constexpr int PR = D / 16;
    __shared__ int s_id[kGatherTokens];  // block of each token; -1: from the tail; -2: left out
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x;
    const SeqRange sq = seq_range(p.bt, b, p.c.bs, p.c.err, tid == 0 && blockIdx.x == 0);
    const int i0 = int(blockIdx.x) * kGatherTokens;
    if (i0 >= sq.n || (sq.bad && !p.first)) return;
    const int t_first = p.first ? p.first[b] : sq.ctx - sq.n;
    // with `first` the rows may be any range inside the context
    if (p.first && (t_first < 0 || sq.ctx < 0 || int64_t(sq.ctx) > int64_t(p.bt.max_blocks) * p.c.bs ||
                    int64_t(t_first) + sq.n > sq.ctx)) {
        if (tid == 0 && blockIdx.x == 0) report(p.c.err, kErrCtxLen);
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
    __syncthreads();

    constexpr int NB = 4;  // loads of 16 elements in flight a thread
    const int items = 2 * m * Hkv * PR;
    for (int i = tid; i < items; i += NB * kGatherThreads) {
        uint4 w[NB][2];
        float sc[NB];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            const int e = i + u * kGatherThreads;
            if (e >= items) continue;
            const int c = e % PR, h = e / PR % Hkv, tl = e / (PR * Hkv) % m, kv = e / (PR * Hkv * m);
            const int id = s_id[tl], off = (t_first + i0 + tl) % bs;
            if (id >= 0) {
                const size_t row = (size_t(id) * Hkv + h) * bs + off;
                const uint8_t* pool = static_cast<const uint8_t*>(kv ? p.c.v_pool : p.c.k_pool);
                if (INT8) {
                    w[u][0] = ldg128(pool + row * D + c * 16);
                    sc[u] = __ldg(p.c.scales + (size_t(id) * Hkv + h) * 2 + kv);
                } else {
                    w[u][0] = ldg128(pool + (row * D + c * 16) * 2);
                    w[u][1] = ldg128(pool + (row * D + c * 16) * 2 + 16);
                }
            } else if (INT8 && id == -1) {
                const uint16_t* r = (kv ? p.c.v_tail : p.c.k_tail) + ((size_t(slot) * Hkv + h) * bs + off) * D + c * 16;
                w[u][0] = ldg128(r);
                w[u][1] = ldg128(r + 8);
            }
        }
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            const int e = i + u * kGatherThreads;
            if (e >= items) continue;
            const int c = e % PR, h = e / PR % Hkv, tl = e / (PR * Hkv) % m, kv = e / (PR * Hkv * m);
            const int id = s_id[tl];
            if (id == -2) continue;
            float x[16];
            if (INT8 && id >= 0) {
                const uint32_t q[4] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 lo, hi;
                    s8x4_to_f4(q[k], lo, hi);
                    x[4 * k] = lo.x * sc[u];
                    x[4 * k + 1] = lo.y * sc[u];
                    x[4 * k + 2] = hi.x * sc[u];
                    x[4 * k + 3] = hi.y * sc[u];
                }
            } else {
                bf16x8_to_f(w[u][0], x);
                bf16x8_to_f(w[u][1], x + 8);
            }
            store16<F32>(kv ? p.v_out : p.k_out, int64_t(sq.row0 + i0 + tl) * p.out_stride + h * D + c * 16, x);
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
    const dim3 grid(unsigned((batch->max_tokens - 1) / kGatherTokens + 1), unsigned(batch->B));
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
