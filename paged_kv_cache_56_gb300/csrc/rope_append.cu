// Rotary turn of a batch's new q and k rows fused with the write of k and v
// into the paged cache (pkv_rope_append).
//
// One CTA per (chunk of CT tokens aligned to the cache's blocks, kv head,
// sequence): it turns the chunk's rows of the kv head and of its group of
// query heads, so q, k and v are read once and the cache is written once. In
// INT8 mode CT is the block size and the CTA that holds a full block
// quantizes it from registers: the block's bf16 rows never go to memory.
//
// Angles. The position is an integer p, so only the fraction of p * f / 2 pi
// matters. f / 2 pi modulo 1 is held as a 64-bit binary fraction u (from the
// fp64 frequency: off by less than 2^-52 of a turn), p * u wraps modulo 2^64
// exactly, and its top 32 bits are the angle in turns to 2^-33 -- no large
// angle ever meets a floating-point reduction, and no table of sines over all
// positions is read from memory. sincospi of that fraction is fp32, computed
// once a (token, pair) and used by the group's G + 1 heads.
//
// Bound by memory: 2 * (Hq + Hkv + Hkv) * d bytes read a token, and as much
// written (the INT8 cache half of its part).
#include "batch.cuh"
#include "host.h"

namespace pkv {

struct RopeParams {
    BatchView bt;
    CacheView c;
    const double* inv_freq;
    const int32_t* positions;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t half;  // rotary_dim / 2 (0: nothing turns)
    int32_t interleaved;
    float scale;
};

constexpr int kRopeThreads = 256;

// 16 elements of a row: two 16-byte chunks, at element offsets lo and hi.
struct Pair16 {
    uint4 a, b;
};

// Element offsets of a row's i-th pair of 16-byte chunks: with the halves
// layout the two chunks that turn together, otherwise 16 elements in a row.
__device__ __forceinline__ void pair_offsets(int i, int half, bool interleaved, int& lo, int& hi) {
    if (!interleaved && i < half / 8) {
        lo = i * 8;
        hi = half + i * 8;
    } else {
        lo = i * 16;
        hi = lo + 8;
    }
}

// Turns the i-th pair of chunks of a row; cs: (cos, sin) of the row's pairs.
__device__ __forceinline__ void turn(Pair16& w, int i, int half, bool interleaved, const float2* cs) {
    if (i >= half / 8) return;
    uint32_t x[4] = {w.a.x, w.a.y, w.a.z, w.a.w}, y[4] = {w.b.x, w.b.y, w.b.z, w.b.w};
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = bf16x2_to_f2(x[e]), r = bf16x2_to_f2(y[e]);
            const float2 c0 = cs[i * 8 + e], c1 = cs[i * 8 + 4 + e];
            x[e] = f2_to_bf16x2(p.x * c0.x - p.y * c0.y, p.y * c0.x + p.x * c0.y);
            y[e] = f2_to_bf16x2(r.x * c1.x - r.y * c1.y, r.y * c1.x + r.x * c1.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = bf16x2_to_f2(x[e]), r = bf16x2_to_f2(y[e]);
            const float2 c0 = cs[i * 8 + 2 * e], c1 = cs[i * 8 + 2 * e + 1];
            x[e] = f2_to_bf16x2(p.x * c0.x - r.x * c0.y, p.y * c1.x - r.y * c1.y);
            y[e] = f2_to_bf16x2(r.x * c0.x + p.x * c0.y, r.y * c1.x + p.y * c1.y);
        }
    }
    w.a = make_uint4(x[0], x[1], x[2], x[3]);
    w.b = make_uint4(y[0], y[1], y[2], y[3]);
}

__device__ __forceinline__ float absmax8(const uint4& w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_f2(x[e]);
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    return m;
}

// Eight codes clamp(rint(x / scale)): the cache's quantizer (see quantize_slab).
__device__ __forceinline__ uint2 codes8(const uint4& w, float scale) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_f2(x[e]);
        const int q0 = min(127, max(-127, __float2int_rn(__fdiv_rn(f.x, scale))));
        const int q1 = min(127, max(-127, __float2int_rn(__fdiv_rn(f.y, scale))));
        out[e >> 1] |= ((uint32_t(q0) & 0xFFu) | ((uint32_t(q1) & 0xFFu) << 8)) << (16 * (e & 1));
    }
    return make_uint2(out[0], out[1]);
}

template <int D, bool INT8, int CT>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
    constexpr int PR = D / 16;                             // chunk pairs a row
    constexpr int HT = kRopeThreads / 2;                   // threads for K, and for V
    constexpr int NI = (CT * PR + HT - 1) / HT;            // chunk pairs a thread holds of K or V
    __shared__ float2 cs[CT * (D / 2)];
    __shared__ unsigned long long s_turns[D / 2];
    __shared__ float s_max[kRopeThreads / 32];
    pdl_wait();
    pdl_launch_dependents();

    const int kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int G = p.c.Hq / p.c.Hkv;
    const SeqRange sq = seq_range(p.bt, b, p.c.bs, p.c.err, tid == 0 && kvh == 0 && blockIdx.x == 0);
    if (sq.n == 0 || sq.bad) return;
    const int start = sq.ctx - sq.n;                       // first new token
    const int chunk0 = start / CT, last = (sq.ctx - 1) / CT;
    const int chunk = chunk0 + int(blockIdx.x);
    if (chunk > last) return;

    if (tid < p.half) {
        // turns a position, modulo 1, in units of 2^-64
        double u = p.inv_freq[tid] * 0.15915494309189535;  // 1 / (2 pi)
        u -= floor(u);
        s_turns[tid] = static_cast<unsigned long long>(u * 18446744073709551616.0);
    }

    const int slot = INT8 ? p.bt.slots[b] : 0;
    const bool slot_ok = !INT8 || (slot >= 0 && slot < p.c.max_slots);
    const int32_t* table = p.bt.tables + size_t(b) * p.bt.max_blocks;
    const bool inter = p.interleaved != 0;

    // INT8: the CTA of a block that earlier tokens began reads their rows from
    // the tail; if the last block is another one and partly filled, its rows
    // go to the same tail. So that CTA writes them too, after its reads, and
    // the last block's own CTA leaves them.
    const bool from_tail = INT8 && start % CT != 0;
    const bool last_partial = INT8 && sq.ctx % CT != 0;
    const int jobs = (from_tail && last_partial && chunk == chunk0 && last > chunk0) ? 2 : 1;
    const bool leave_kv = from_tail && last_partial && chunk == last && last > chunk0;

    for (int job = 0; job < jobs; ++job) {
        const int base = (job == 0 ? chunk : last) * CT;
        const int t0 = max(start, base), t1 = min(sq.ctx, base + CT);  // new tokens of the chunk
        const int m = t1 - t0;
        __syncthreads();  // the turns; the previous job's use of cs
        for (int i = tid; i < m * p.half; i += kRopeThreads) {
            const int tok = t0 + i / p.half, j = i % p.half;
            const int row = sq.row0 + tok - start;
            const int pos = p.positions ? p.positions[row] : tok;
            const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(pos)) * s_turns[j];
            float sn, cn;
            // the top half as a signed number of half turns, in [-1, 1)
            sincospif(float(int32_t(a >> 32)) * 4.656612873077393e-10f, &sn, &cn);
            cs[(tok - base) * p.half + j] = make_float2(cn * p.scale, sn * p.scale);
        }
        __syncthreads();

        // ---- K and V: half of the threads each
        if (!(leave_kv && job == 0)) {
            const int kv = tid / HT, th = tid % HT;
            const bool full = INT8 && base + CT <= sq.ctx;
            int id = -1;
            if (!INT8 || full) {
                id = table[base / p.c.bs];
                if (id < 0 || id >= p.c.num_blocks) {
                    if (tid == 0) report(p.c.err, kErrBlockId);
                    id = -1;
                }
            }
            if (INT8 && !slot_ok && (!full || start > base) && tid == 0) report(p.c.err, kErrSlot);
            const bool write = INT8 && !full ? slot_ok : id >= 0 && (slot_ok || start <= base);
            uint16_t* tail = kv ? p.c.v_tail : p.c.k_tail;
            const uint16_t* src = kv ? p.v : p.k;
            const int64_t stride = kv ? p.v_stride : p.k_stride;
            if (write) {
                Pair16 w[NI];
                const size_t tail0 = (size_t(slot) * p.c.Hkv + kvh) * p.c.bs;
#pragma unroll
                for (int u = 0; u < NI; ++u) {
                    const int i = th + u * HT, tl = i / PR, tok = base + tl;
                    int lo, hi;
                    pair_offsets(i % PR, p.half, inter, lo, hi);
                    w[u].a = w[u].b = make_uint4(0u, 0u, 0u, 0u);
                    if (CT * PR % HT != 0 && i >= CT * PR) continue;
                    if (tok >= t0 && tok < t1) {
                        const uint16_t* r = src + int64_t(sq.row0 + tok - start) * stride + kvh * D;
                        w[u].a = ldg128(r + lo);
                        w[u].b = ldg128(r + hi);
                    } else if (full && tok < t0) {
                        const uint16_t* r = tail + (tail0 + tl) * D;
                        w[u].a = ldcg128(r + lo);
                        w[u].b = ldcg128(r + hi);
                    }
                }
                float mx = 0.f;
#pragma unroll
                for (int u = 0; u < NI; ++u) {
                    const int i = th + u * HT, tl = i / PR, tok = base + tl;
                    if (kv == 0 && tok >= t0 && tok < t1) turn(w[u], i % PR, p.half, inter, cs + tl * p.half);
                    if (full) mx = fmaxf(mx, fmaxf(absmax8(w[u].a), absmax8(w[u].b)));
                }
                if (full) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                    if ((tid & 31) == 0) s_max[tid >> 5] = mx;
                    __syncthreads();  // `full` and `write` are the CTA's
                    mx = 0.f;
#pragma unroll
                    for (int x = 0; x < HT / 32; ++x) mx = fmaxf(mx, s_max[kv * (HT / 32) + x]);
                    const float scale = mx < 1e-6f ? 1.0f : __fdiv_rn(mx, 127.0f);
                    int8_t* dst = static_cast<int8_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                  (size_t(id) * p.c.Hkv + kvh) * CT * D;
#pragma unroll
                    for (int u = 0; u < NI; ++u) {
                        const int i = th + u * HT, tl = i / PR;
                        if (CT * PR % HT != 0 && i >= CT * PR) continue;
                        int lo, hi;
                        pair_offsets(i % PR, p.half, inter, lo, hi);
                        *reinterpret_cast<uint2*>(dst + tl * D + lo) = codes8(w[u].a, scale);
                        *reinterpret_cast<uint2*>(dst + tl * D + hi) = codes8(w[u].b, scale);
                    }
                    if (th == 0) p.c.scales[(size_t(id) * p.c.Hkv + kvh) * 2 + kv] = scale;
                } else {
                    // rows of the pool block, or of the tail
                    uint16_t* dst = INT8 ? tail + tail0 * D
                                         : static_cast<uint16_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                               ((size_t(id) * p.c.Hkv + kvh) * p.c.bs + base % p.c.bs) * D;
#pragma unroll
                    for (int u = 0; u < NI; ++u) {
                        const int i = th + u * HT, tl = i / PR, tok = base + tl;
                        if (tok < t0 || tok >= t1) continue;
                        int lo, hi;
                        pair_offsets(i % PR, p.half, inter, lo, hi);
                        *reinterpret_cast<uint4*>(dst + tl * D + lo) = w[u].a;
                        *reinterpret_cast<uint4*>(dst + tl * D + hi) = w[u].b;
                    }
                }
            }
        }

        // ---- the group's queries
        if (job == 0 && p.q) {
            constexpr int NB = 4;  // chunk pairs in flight a thread
            const int items = m * G * PR;
            for (int i0 = tid; i0 < items; i0 += NB * kRopeThreads) {
                Pair16 w[NB];
#pragma unroll
                for (int u = 0; u < NB; ++u) {
                    const int i = i0 + u * kRopeThreads;
                    if (i >= items) continue;
                    const int tok = t0 + i / (G * PR), h = i / PR % G;
                    int lo, hi;
                    pair_offsets(i % PR, p.half, inter, lo, hi);
                    const uint16_t* r = p.q + int64_t(sq.row0 + tok - start) * p.q_stride + (kvh * G + h) * D;
                    w[u].a = ldcg128(r + lo);
                    w[u].b = ldcg128(r + hi);
                }
#pragma unroll
                for (int u = 0; u < NB; ++u) {
                    const int i = i0 + u * kRopeThreads;
                    if (i >= items) continue;
                    const int tok = t0 + i / (G * PR), h = i / PR % G;
                    int lo, hi;
                    pair_offsets(i % PR, p.half, inter, lo, hi);
                    turn(w[u], i % PR, p.half, inter, cs + (tok - base) * p.half);
                    uint16_t* r = p.q_out + int64_t(sq.row0 + tok - start) * p.q_out_stride + (kvh * G + h) * D;
                    *reinterpret_cast<uint4*>(r + lo) = w[u].a;
                    *reinterpret_cast<uint4*>(r + hi) = w[u].b;
                }
            }
        }
    }
}

__global__ void empty_kernel() {}

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_rope_append(const pkv_cache_desc* c, const pkv_batch_desc* batch, const pkv_rope* rope, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               void* q_out, int64_t q_out_stride, void* stream) {
    RopeParams p;
    int st = check_batch(c, batch, &p.bt, &p.c);
    if (st != PKV_OK) return st;
    const int d = c->head_dim;
    p.half = 0;
    p.interleaved = 0;
    p.scale = 1.f;
    p.inv_freq = nullptr;
    p.positions = nullptr;
    if (rope) {
        if (rope->rotary_dim < 0 || rope->rotary_dim > d) return PKV_ERR_INVALID;
        if (rope->rotary_dim % 16) return PKV_ERR_UNSUPPORTED;
        if (rope->rotary_dim > 0 && (!rope->inv_freq || (reinterpret_cast<uintptr_t>(rope->inv_freq) & 7u)))
            return PKV_ERR_INVALID;
        if (reinterpret_cast<uintptr_t>(rope->positions) & 3u) return PKV_ERR_INVALID;
        if (!(rope->scale == rope->scale)) return PKV_ERR_INVALID;
        p.half = rope->rotary_dim / 2;
        p.interleaved = rope->interleaved;
        p.scale = rope->scale;
        p.inv_freq = rope->inv_freq;
        p.positions = rope->positions;
    }
    if (batch->B == 0 || batch->num_tokens == 0 || batch->max_tokens == 0) return PKV_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || (q && (!q_out || !aligned16(q) || !aligned16(q_out))))
        return PKV_ERR_INVALID;
    const int64_t kv_row = int64_t(c->num_kv_heads) * d, q_row = int64_t(c->num_q_heads) * d;
    if (k_stride < kv_row || v_stride < kv_row || ((k_stride | v_stride) & 7)) return PKV_ERR_INVALID;
    if (q && (q_stride < q_row || q_out_stride < q_row || ((q_stride | q_out_stride) & 7))) return PKV_ERR_INVALID;
    if (q && q == q_out && q_stride != q_out_stride) return PKV_ERR_INVALID;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    const bool int8 = c->dtype == PKV_DTYPE_INT8;
    const int ct = int8 ? c->block_size : 16;
    // the most aligned chunks that max_tokens tokens in a row can touch
    const unsigned chunks = unsigned((batch->max_tokens + ct - 2) / ct + 1);
    const dim3 grid(chunks, unsigned(c->num_kv_heads), unsigned(batch->B));
    void (*fn)(RopeParams) = nullptr;
    if (d == 128)
        fn = !int8 ? rope_append_kernel<128, false, 16>
                   : ct == 16 ? rope_append_kernel<128, true, 16> : rope_append_kernel<128, true, 64>;
    else
        fn = !int8 ? rope_append_kernel<64, false, 16>
                   : ct == 16 ? rope_append_kernel<64, true, 16> : rope_append_kernel<64, true, 64>;
    auto s = static_cast<cudaStream_t>(stream);
    if ((st = launch(fn, grid, dim3(kRopeThreads), 0, s, p)) != PKV_OK) return st;
    if (g_pdl.load(std::memory_order_relaxed) && batch->max_tokens > 1) {
        empty_kernel<<<1, 1, 0, s>>>();
        return cuda_status(cudaGetLastError());
    }
    return PKV_OK;
}
