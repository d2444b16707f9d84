// Entry point of the attention of whole prompts: argument checks and the launch.
#include <algorithm>

#include "host.h"
#include "prompt.cuh"

using namespace pkv;

extern "C" int pkv_prompt_attention(const pkv_cache_desc* c, const pkv_batch_desc* batch, const void* q, int64_t q_stride,
                                    const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t window,
                                    int32_t sinks, float sm_scale, void* out, int64_t out_stride, void* stream) {
    PromptParams p;
    CacheView cv;
    int st = check_batch(c, batch, &p.bt, &cv);
    if (st != PKV_OK) return st;
    if (window < 0 || sinks < 0 || !(sm_scale >= 0.f) || sm_scale > 3.0e38f) return PKV_ERR_INVALID;
    if (batch->B == 0 || batch->num_tokens == 0 || batch->max_tokens == 0) return PKV_OK;
    const int d = c->head_dim, hq = c->num_q_heads, hkv = c->num_kv_heads, g = hq / hkv;
    const int64_t q_row = int64_t(hq) * d, kv_row = int64_t(hkv) * d;
    if (!q || !k || !v || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        q_stride < q_row || out_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
        ((q_stride | k_stride | v_stride | out_stride) & 7))
        return PKV_ERR_INVALID;
    if (q == out && q_stride != out_stride) return PKV_ERR_INVALID;
    // an item takes half of the second that others wait for it at 2^25 keys
    if (batch->max_tokens > 1 << 25) return PKV_ERR_UNSUPPORTED;
    void (*const fn)(PromptParams) = d == 128 ? prompt_kernel<128> : prompt_kernel<64>;
    const size_t smem = d == 128 ? PromptTraits<128>::kSmem : PromptTraits<64>::kSmem;
    int ctas = 0;
    if ((st = prepare_kernel(reinterpret_cast<const void*>(fn), smem, kPrThreads, kPrLaunchRegs, &ctas)) != PKV_OK) return st;
    if ((st = rows_tensor_map(g, hkv, d, batch->num_tokens, q, q_stride, 128, &p.tm_q)) != PKV_OK) return st;
    if ((st = rows_tensor_map(1, hkv, d, batch->num_tokens, k, k_stride, 128, &p.tm_k)) != PKV_OK) return st;
    if ((st = rows_tensor_map(1, hkv, d, batch->num_tokens, v, v_stride, 128, &p.tm_v)) != PKV_OK) return st;
    if ((st = rows_tensor_map(g, hkv, d, batch->num_tokens, out, out_stride, 32, &p.tm_out)) != PKV_OK) return st;
    p.out = static_cast<uint16_t*>(out);
    p.out_stride = out_stride;
    p.err = c->err_word;
    p.skip_copy = g_skip_copy.load(std::memory_order_relaxed);
    p.Hq = hq;
    p.Hkv = hkv;
    p.window = window > 0 ? window : 0x7FFFFFFF;
    p.sinks = window > 0 ? sinks : 0;
    // never 0 or infinite: a hidden token's score is -infinity, and 0 times that is
    // not a number, nor is an infinite scale times a score of 0
    p.qscale = std::min(std::max(sm_scale * 1.4426950408889634f, 1e-37f), 3.4e38f);
    // items of a kv head, as many as the batch can have
    const int64_t longest = (int64_t(batch->max_tokens) * g + 2 * kPrRows - 1) / (2 * kPrRows);
    const int64_t tiles = std::min(longest * batch->B, batch->num_tokens * int64_t(g) / (2 * kPrRows) + batch->B);
    const int64_t items = tiles * hkv;
    // A CTA drops items that the batch does not have at 0.4 us each, while its other
    // warps wait: 2^27 items on 152 SMs are 0.35 s of the second that they do.
    if (items > int64_t(1) << 27) return PKV_ERR_UNSUPPORTED;
    p.item_tiles = int(tiles);
    return launch(fn, dim3(unsigned(items)), dim3(kPrThreads), smem, static_cast<cudaStream_t>(stream), p);
}
