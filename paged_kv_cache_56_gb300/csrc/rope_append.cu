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
// matters. f / 2 pi modulo 1 is held as a 64-bit binary fraction u -- the fp64
// frequency's significand times 1 / 2 pi in integers, since fp64 arithmetic
// runs at a 64th of the integer rate here -- p * u wraps modulo 2^64
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
    int32_t heads;  // kv heads a CTA
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

// (cos, sin) of a token's pairs in shared memory: pair 8 i + k at k * (half / 8)
// + i, so that threads of neighbouring i read neighbouring entries; tokens are
// half + 8 entries apart, which puts two tokens' entries in different banks.
__device__ __forceinline__ int cs_stride(int half) { return half + 8; }

// Turns the i-th pair of chunks of a row; cs: its token's entries.
__device__ __forceinline__ void turn(Pair16& w, int i, int half, bool interleaved, const float2* cs) {
    const int n = half / 8;
    if (i >= n) return;
    uint32_t x[4] = {w.a.x, w.a.y, w.a.z, w.a.w}, y[4] = {w.b.x, w.b.y, w.b.z, w.b.w};
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = bf16x2_to_f2(x[e]), r = bf16x2_to_f2(y[e]);
            const float2 c0 = cs[e * n + i], c1 = cs[(e + 4) * n + i];
            x[e] = f2_to_bf16x2(p.x * c0.x - p.y * c0.y, p.y * c0.x + p.x * c0.y);
            y[e] = f2_to_bf16x2(r.x * c1.x - r.y * c1.y, r.y * c1.x + r.x * c1.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = bf16x2_to_f2(x[e]), r = bf16x2_to_f2(y[e]);
            const float2 c0 = cs[2 * e * n + i], c1 = cs[(2 * e + 1) * n + i];
            x[e] = f2_to_bf16x2(p.x * c0.x - r.x * c0.y, p.y * c1.x - r.y * c1.y);
            y[e] = f2_to_bf16x2(r.x * c0.x + p.x * c0.y, r.y * c1.x + p.y * c1.y);
        }
    }
    w.a = make_uint4(x[0], x[1], x[2], x[3]);
    w.b = make_uint4(y[0], y[1], y[2], y[3]);
}

// f / (2 pi) modulo 1 in units of 2^-64: the significand (53 bits, put to the
// top of 64) times 1 / (2 pi) = 0x28BE60DB9391054A / 2^64, shifted to the
// frequency's exponent. Zero and subnormal frequencies are 0 turns; for
// frequencies of 2^k >= 1 radian a position the lowest k bits are unknown.
__device__ __forceinline__ unsigned long long turns_of(double f) {
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(f));
    const int e = int((bits >> 52) & 0x7FF);
    if (e == 0) return 0;
    const unsigned long long m = (bits << 11) | 0x8000000000000000ull;  // |f| = m * 2^(e - 1086)
    const unsigned long long inv = 0x28BE60DB9391054Aull;
    const unsigned long long hi = __umul64hi(m, inv), lo = m * inv;
    // |f| / (2 pi) = (hi:lo) * 2^(e - 1150); wanted: its fraction in 64 bits
    const int right = 1086 - e;  // of hi:lo, to leave the fraction's 64 bits below 2^0
    unsigned long long u;
    if (right >= 128) u = 0;
    else if (right >= 64) u = hi >> (right - 64);
    else if (right > 0) u = (hi << (64 - right)) | (lo >> right);
    else if (right > -64) u = lo << -right;
    else u = 0;
    return bits >> 63 ? 0ull - u : u;
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

// Eight codes clamp(rint(x / scale)) as the cache's quantizer defines them (see
// quantize_slab), inv = 1 / scale. x * inv is off by at most 127 * 2^-22 < 4e-5
// from the rounded quotient, so away from a tie it rounds to the same integer;
// within 1e-4 of one the division decides (one value in 5000).
__device__ __forceinline__ int code1(float x, float scale, float inv) {
    const float t = x * inv;
    int q = __float2int_rn(t);
    if (fabsf(t - float(q)) > 0.4999f) q = __float2int_rn(__fdiv_rn(x, scale));
    return min(127, max(-127, q));
}
__device__ __forceinline__ uint2 codes8(const uint4& w, float scale, float inv) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_f2(x[e]);
        const int q0 = code1(f.x, scale, inv), q1 = code1(f.y, scale, inv);
        out[e >> 1] |= ((uint32_t(q0) & 0xFFu) | ((uint32_t(q1) & 0xFFu) << 8)) << (16 * (e & 1));
    }
    return make_uint2(out[0], out[1]);
}

template <int D, bool INT8, int CT>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
    constexpr int PR = D / 16;                             // chunk pairs a row
    constexpr int HT = kRopeThreads / 2;                   // threads for K, and for V
    constexpr int NI = (CT * PR + HT - 1) / HT;            // chunk pairs a thread holds of K or V
    constexpr int NB = 4;                                  // chunk pairs of q in flight a thread
    __shared__ float2 cs[CT * (D / 2 + 8)];
    __shared__ unsigned long long s_turns[D / 2];
    __shared__ float s_max[kRopeThreads / 32];
    pdl_wait();
    pdl_launch_dependents();

    const int b = blockIdx.z, tid = threadIdx.x, half = p.half;
    const int G = p.c.Hq / p.c.Hkv, lgG = 31 - __clz(G);   // 1, 2, 4 or 8
    const SeqRange sq = seq_range(p.bt, b, p.c.bs, p.c.err, tid == 0 && blockIdx.y == 0 && blockIdx.x == 0);
    if (sq.n == 0 || sq.bad) return;
    const int start = sq.ctx - sq.n;                       // first new token
    const int chunk0 = start / CT, last = (sq.ctx - 1) / CT;
    const int chunk = chunk0 + int(blockIdx.x);
    if (chunk > last) return;
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
    const int kv = tid / HT, th = tid % HT;  // half of the threads take K, half V
    const int kvh0 = int(blockIdx.y) * p.heads, kvh1 = min(p.c.Hkv, kvh0 + p.heads);

    for (int job = 0; job < jobs; ++job) {
        const int base = (job == 0 ? chunk : last) * CT;
        const int t0 = max(start, base), t1 = min(sq.ctx, base + CT);  // new tokens of the chunk
        const int m = t1 - t0, rows = m << lgG;
        const bool do_kv = !(leave_kv && job == 0), do_q = job == 0 && p.q;
        const bool full = INT8 && base + CT <= sq.ctx;
        int id = -1;
        if (do_kv && (!INT8 || full)) id = table[base / p.c.bs];

        Pair16 w[NI], x[NB];
        const auto load_kv = [&](int kvh) {
            const uint16_t* src = kv ? p.v : p.k;
            const int64_t stride = kv ? p.v_stride : p.k_stride;
            const uint16_t* tail = (kv ? p.c.v_tail : p.c.k_tail) + (size_t(slot) * p.c.Hkv + kvh) * p.c.bs * D;
#pragma unroll
            for (int u = 0; u < NI; ++u) {
                const int i = th + u * HT, tl = i / PR, tok = base + tl;
                int lo, hi;
                pair_offsets(i % PR, half, inter, lo, hi);
                w[u].a = w[u].b = make_uint4(0u, 0u, 0u, 0u);
                if (CT * PR % HT != 0 && i >= CT * PR) continue;
                if (tok >= t0 && tok < t1) {
                    const uint16_t* r = src + int64_t(sq.row0 + tok - start) * stride + kvh * D;
                    w[u].a = ldg128(r + lo);
                    w[u].b = ldg128(r + hi);
                } else if (full && slot_ok && tok < t0) {
                    w[u].a = ldcg128(tail + tl * D + lo);
                    w[u].b = ldcg128(tail + tl * D + hi);
                }
            }
        };
        // q rows (token, head of the group), NB of a thread's chunk pairs from i0 on
        const auto load_q = [&](int kvh, int i0) {
#pragma unroll
            for (int u = 0; u < NB; ++u) {
                const int i = i0 + u * kRopeThreads, r = i / PR;
                if (r >= rows) break;
                int lo, hi;
                pair_offsets(i % PR, half, inter, lo, hi);
                const uint16_t* at = p.q + int64_t(sq.row0 + t0 - start + (r >> lgG)) * p.q_stride +
                                     (kvh * G + (r & (G - 1))) * D;
                x[u].a = ldcg128(at + lo);  // q may be turned in place
                x[u].b = ldcg128(at + hi);
            }
        };
        // the first head's rows are under way while the angles are worked out
        if (do_kv) load_kv(kvh0);
        if (do_q) load_q(kvh0, tid);
        __syncthreads();  // the previous job's use of cs
        if (half > 0) {
            if (job == 0) {
                if (tid < half) s_turns[tid] = turns_of(p.inv_freq[tid]);
                __syncthreads();
            }
            int tl = tid / half, j = tid % half;
            const int dt = kRopeThreads / half, dj = kRopeThreads % half;
            for (; tl < m; tl += dt, j += dj) {
                if (j >= half) {
                    j -= half;
                    if (++tl >= m) break;
                }
                const int row = sq.row0 + t0 + tl - start;
                const int pos = p.positions ? p.positions[row] : t0 + tl;
                const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(pos)) * s_turns[j];
                float sn, cn;
                // the top half as a signed number of half turns, in [-1, 1)
                sincospif(float(int32_t(a >> 32)) * 4.656612873077393e-10f, &sn, &cn);
                cs[(t0 + tl - base) * cs_stride(half) + (j % 8) * (half / 8) + j / 8] = make_float2(cn * p.scale, sn * p.scale);
            }
        }
        if (do_kv && (!INT8 || full) && (id < 0 || id >= p.c.num_blocks)) {
            if (tid == 0) report(p.c.err, kErrBlockId);
            id = -1;
        }
        if (INT8 && do_kv && !slot_ok && (!full || start > base) && tid == 0) report(p.c.err, kErrSlot);
        const bool write = do_kv && (INT8 && !full ? slot_ok : id >= 0 && (slot_ok || start <= base));
        __syncthreads();

        for (int kvh = kvh0; kvh < kvh1; ++kvh) {
            if (kvh > kvh0) {
                if (do_kv) load_kv(kvh);
                if (do_q) load_q(kvh, tid);
            }
            // ---- K and V
            if (write) {
                float mx = 0.f;
#pragma unroll
                for (int u = 0; u < NI; ++u) {
                    const int i = th + u * HT, tl = i / PR, tok = base + tl;
                    if (kv == 0 && tok >= t0 && tok < t1) turn(w[u], i % PR, half, inter, cs + tl * cs_stride(half));
                    if (full) mx = fmaxf(mx, fmaxf(absmax8(w[u].a), absmax8(w[u].b)));
                }
                if (full) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                    if ((tid & 31) == 0) s_max[tid >> 5] = mx;
                    __syncthreads();  // `full` and `write` are the CTA's
                    mx = 0.f;
#pragma unroll
                    for (int k = 0; k < HT / 32; ++k) mx = fmaxf(mx, s_max[kv * (HT / 32) + k]);
                    const float scale = mx < 1e-6f ? 1.0f : __fdiv_rn(mx, 127.0f), inv = __fdiv_rn(1.0f, scale);
                    int8_t* dst = static_cast<int8_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                  (size_t(id) * p.c.Hkv + kvh) * CT * D;
#pragma unroll
                    for (int u = 0; u < NI; ++u) {
                        const int i = th + u * HT, tl = i / PR;
                        if (CT * PR % HT != 0 && i >= CT * PR) continue;
                        int lo, hi;
                        pair_offsets(i % PR, half, inter, lo, hi);
                        *reinterpret_cast<uint2*>(dst + tl * D + lo) = codes8(w[u].a, scale, inv);
                        *reinterpret_cast<uint2*>(dst + tl * D + hi) = codes8(w[u].b, scale, inv);
                    }
                    if (th == 0) p.c.scales[(size_t(id) * p.c.Hkv + kvh) * 2 + kv] = scale;
                    if (kvh + 1 < kvh1) __syncthreads();  // s_max
                } else {
                    // rows of the pool block, or of the tail
                    uint16_t* dst = INT8 ? (kv ? p.c.v_tail : p.c.k_tail) + (size_t(slot) * p.c.Hkv + kvh) * p.c.bs * D
                                         : static_cast<uint16_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                               ((size_t(id) * p.c.Hkv + kvh) * p.c.bs + base % p.c.bs) * D;
#pragma unroll
                    for (int u = 0; u < NI; ++u) {
                        const int i = th + u * HT, tl = i / PR, tok = base + tl;
                        if (tok < t0 || tok >= t1) continue;
                        int lo, hi;
                        pair_offsets(i % PR, half, inter, lo, hi);
                        *reinterpret_cast<uint4*>(dst + tl * D + lo) = w[u].a;
                        *reinterpret_cast<uint4*>(dst + tl * D + hi) = w[u].b;
                    }
                }
            }

            // ---- the group's queries
            if (do_q) {
                for (int i0 = tid;;) {
#pragma unroll
                    for (int u = 0; u < NB; ++u) {
                        const int i = i0 + u * kRopeThreads, r = i / PR;
                        if (r >= rows) break;
                        int lo, hi;
                        pair_offsets(i % PR, half, inter, lo, hi);
                        turn(x[u], i % PR, half, inter, cs + (t0 - base + (r >> lgG)) * cs_stride(half));
                        uint16_t* at = p.q_out + int64_t(sq.row0 + t0 - start + (r >> lgG)) * p.q_out_stride +
                                       (kvh * G + (r & (G - 1))) * D;
                        *reinterpret_cast<uint4*>(at + lo) = x[u].a;
                        *reinterpret_cast<uint4*>(at + hi) = x[u].b;
                    }
                    i0 += NB * kRopeThreads;
                    if (i0 / PR >= rows) break;
                    load_q(kvh, i0);
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
    // Angles are worked out once a CTA: where there are CTAs enough for several
    // waves (8 fit on an SM) a CTA takes several kv heads.
    p.heads = 1;
    while (p.heads < 4 && p.heads * 2 <= c->num_kv_heads &&
           int64_t(chunks) * batch->B * c->num_kv_heads / (p.heads * 2) >= 152 * 8 * 2)
        p.heads *= 2;
    const dim3 grid(chunks, unsigned((c->num_kv_heads + p.heads - 1) / p.heads), unsigned(batch->B));
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
