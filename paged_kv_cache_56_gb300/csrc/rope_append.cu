// Rotary turn of a batch's new q and k rows fused with the write of k and v
// into the paged cache (pkv_rope_append).
//
// One CTA per (chunk of 16 tokens, aligned to the cache's blocks, group of kv
// heads); a thread has one token and one pair of 16-byte chunks of a row -- the
// eight pairs of elements that turn by the same angles in every head -- so it
// works out its eight angles once, keeps their sines and cosines in registers
// and walks through the heads, four rows in flight. In INT8 mode a block
// of 64 tokens is a cluster of four CTAs, and a full block is quantized from registers: its bf16 rows
// never go to memory, and the only shared memory is the block's maximum.
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
// written (the INT8 cache half of its part). Measured, d = 128, 8 kv heads:
// 30718 tokens of 16 query heads, bf16, 503 MB in 82 us, 6.1 TB/s (a plain copy:
// 6.7); 12535 tokens of 32 query heads, INT8, 282 MB in 53 us, 5.4 TB/s -- the
// quantizer's arithmetic and its block maximum (a barrier a head) leave half of
// the issue slots and a part of the loads idle; 128 single tokens 8.6 us (bf16 5.7),
// launch and the chain lengths -> rows -> maximum -> codes.
//
// Layout: with a token a thread the angles are worked out once and stay in
// registers (shared-memory tables: 131 us for the bf16 case), consecutive lanes
// read whole 256-byte rows, and a block's rows meet in one CTA or cluster for its
// maximum.
#include <algorithm>

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
    int32_t heads;   // kv heads a CTA
    int32_t groups;  // CTAs a chunk: neighbours in the grid, as their rows are in memory
    int32_t ragged;
    float scale;
};

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

// Turns a pair of chunks by the thread's eight angles, two pairs of elements at
// a time in packed fp32.
struct Angles {
    float2 c[4], s[4];  // of pairs 2e and 2e + 1
};
template <bool INTER>
__device__ __forceinline__ void turn_pairs(Pair16& w, const Angles& an) {
    uint32_t x[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t a = INTER ? x[2 * e] : x[e], b = INTER ? x[2 * e + 1] : x[e + 4];
        // (p, q): the first and second elements of the two pairs
        const float2 p = INTER ? make_float2(__uint_as_float(a << 16), __uint_as_float(b << 16)) : bf16x2_to_f2(a);
        const float2 q = INTER ? make_float2(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u))
                               : bf16x2_to_f2(b);
        const float2 ns = make_float2(-an.s[e].x, -an.s[e].y);
        const float2 u = __ffma2_rn(p, an.c[e], __fmul2_rn(q, ns)), v = __ffma2_rn(q, an.c[e], __fmul2_rn(p, an.s[e]));
        x[INTER ? 2 * e : e] = INTER ? f2_to_bf16x2(u.x, v.x) : f2_to_bf16x2(u.x, u.y);
        x[INTER ? 2 * e + 1 : e + 4] = INTER ? f2_to_bf16x2(u.y, v.y) : f2_to_bf16x2(v.x, v.y);
    }
    w.a = make_uint4(x[0], x[1], x[2], x[3]);
    w.b = make_uint4(x[4], x[5], x[6], x[7]);
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

// Sine and cosine of a / 2^32 turns. The nearest quarter turn is taken off in
// integers; on the rest, |x| <= pi/4, the Taylor sums through x^9 and x^8 are
// off by less than x^11/11! < 2e-9 and x^10/10! < 3e-8, fp32's own rounding.
__device__ __forceinline__ void sincos_turn(uint32_t a, float& sn, float& cn) {
    const uint32_t quarter = (a + 0x20000000u) >> 30;
    const float x = float(int32_t(a - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(y, s, 1.f / 120.f);
    s = fmaf(y, s, -1.f / 6.f);
    s = fmaf(x * y, s, x);
    float c = fmaf(y, 1.f / 40320.f, -1.f / 720.f);
    c = fmaf(y, c, 1.f / 24.f);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.f);
    // a quarter turn on: (sin, cos) -> (cos, -sin)
    const bool odd = quarter & 1u;
    const float u = odd ? c : s, v = odd ? s : c;
    sn = (quarter & 2u) ? -u : u;
    cn = ((quarter + 1u) & 2u) ? -v : v;
}

// Two floats to the same place of another CTA of the cluster's shared memory, and
// the meeting after which what was stored before it is there.
__device__ __forceinline__ void st_cluster_f2(uint32_t addr, uint32_t cta, float x, float y) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(addr),
                 "r"(cta), "f"(x), "f"(y)
                 : "memory");
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Largest |x| of eight bf16 values, as bf16 pairs (not-a-numbers do not count).
__device__ __forceinline__ __nv_bfloat162 absmax8(const uint4& w, __nv_bfloat162 m) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[e])));
    return m;
}

// Eight codes rint(x / scale) as the cache's quantizer defines them (see
// quantize_slab), with the quotient rounded to fp32 first. inv is the rounded
// reciprocal; from q = x * inv, q + (x - q * scale) * inv is within an ulp and,
// by Markstein's theorem (a quotient within an ulp, a correctly rounded
// reciprocal, the remainder by a fused multiply-add), the same step again gives
// the correctly rounded quotient. Ties are common here (bf16 over bf16 * 127),
// so that a branch for them would be taken by most warps. |q| <= 127 but for
// rounding, so no code passes +-127. Not-a-numbers become 0.
__device__ __forceinline__ uint2 codes8(const uint4& w, float scale, float inv) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    const float2 i2 = make_float2(inv, inv), ns = make_float2(-scale, -scale);
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int n[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 f = bf16x2_to_f2(x[2 * h + e]);
            float2 q = __fmul2_rn(f, i2);
            q = __ffma2_rn(__ffma2_rn(q, ns, f), i2, q);
            q = __ffma2_rn(__ffma2_rn(q, ns, f), i2, q);
            n[2 * e] = __float2int_rn(q.x);
            n[2 * e + 1] = __float2int_rn(q.y);
        }
        uint32_t upper;
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(upper) : "r"(n[3]), "r"(n[2]));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(out[h]) : "r"(n[1]), "r"(n[0]), "r"(upper));
    }
    return make_uint2(out[0], out[1]);
}

constexpr int kRopeTokens = 16;  // of a CTA

// PARTS: CTAs a chunk of kRopeTokens * PARTS tokens, a cluster.
template <int D, bool INT8, int PARTS>
__device__ __forceinline__ void rope_append(const RopeParams& p) {
    constexpr int CT = kRopeTokens * PARTS;
    constexpr int PR = D / 16;               // chunk pairs a row
    constexpr int THREADS = kRopeTokens * PR, WARPS = THREADS / 32;
    constexpr int NB = 2;                    // query rows in flight
    __shared__ unsigned long long s_turns[D / 2];
    __shared__ __align__(16) float s_max[2][PARTS * WARPS][2];  // of every warp of the chunk: K's and V's, of two heads in turn
    pdl_wait();
    pdl_launch_dependents();

    const int tid = threadIdx.x, half = p.half;
    const int bx = int(blockIdx.x) / PARTS, part = int(blockIdx.x) % PARTS;
    const int G = p.c.Hq / p.c.Hkv;
    if (tid < half) s_turns[tid] = turns_of(__ldg(p.inv_freq + tid));
    // one chunk a sequence at most: item x is sequence x; otherwise the x-th of
    // the chunks of all sequences, and one more CTA that checks the lengths
    const int item = bx / p.groups, group = bx % p.groups;
    WorkItem it{item, 0};
    if (p.ragged) {
        if (bx == int(gridDim.x) / PARTS - 1) {
            if (part == 0) check_lengths(p.bt, p.c.bs, p.c.err);
            return;
        }
        it = locate(item, p.bt.B, [&](int s) {
            const SeqRange r = seq_range(p.bt, s, p.c.bs, nullptr, false);
            return r.n == 0 || r.bad ? 0 : (r.ctx - 1) / CT - (r.ctx - r.n) / CT + 1;
        });
        if (it.b < 0) return;
    }
    const int b = it.b;
    const SeqRange sq = seq_range(p.bt, b, p.c.bs, p.c.err, !p.ragged && group == 0 && part == 0 && tid == 0);
    if (sq.n == 0 || sq.bad) return;
    const int start = sq.ctx - sq.n;                       // first new token
    const int chunk0 = start / CT, last = (sq.ctx - 1) / CT;
    const int chunk = chunk0 + it.i;
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
    const int kvh0 = group * p.heads, kvh1 = min(p.c.Hkv, kvh0 + p.heads);
    const int tl = part * kRopeTokens + tid / PR, pr = tid % PR;  // this thread's token of the chunk, chunk pair of a row
    if constexpr (PARTS > 1) {
        // tokens that are neither new nor in a block that fills; the cluster's other
        // CTAs meet this one's only over a block that does
        const auto idle = [&](int base) {
            const int t0 = base + part * kRopeTokens;
            return base + CT > sq.ctx && (t0 + kRopeTokens <= start || t0 >= sq.ctx);
        };
        if (idle(chunk * CT) && (jobs == 1 || idle(last * CT))) return;
    }
    int lo, hi;
    pair_offsets(pr, half, inter, lo, hi);
    const bool turns = pr < half / 8;
    const auto turn = [&](Pair16& w, const Angles& an) {
        if (!turns) return;
        if (inter) turn_pairs<true>(w, an);
        else turn_pairs<false>(w, an);
    };

    int turn_no = 0;  // heads whose maximum has been taken
    for (int job = 0; job < jobs; ++job) {
        const int base = (job == 0 ? chunk : last) * CT, tok = base + tl;
        const bool fresh = tok >= start && tok < sq.ctx;   // this thread's token is a new one
        const int64_t row = sq.row0 + tok - start;
        const bool do_kv = !(leave_kv && job == 0), do_q = job == 0 && p.q;
        const bool full = INT8 && base + CT <= sq.ctx;
        int id = -1;
        if (do_kv && (!INT8 || full)) id = table[base / p.c.bs];

        Pair16 w[2], x[NB];  // K and V of a head; query rows
        const auto load_kv = [&](int h) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                w[kv].a = w[kv].b = make_uint4(0u, 0u, 0u, 0u);
                if (fresh) {
                    const uint16_t* r = (kv ? p.v + row * p.v_stride : p.k + row * p.k_stride) + h * D;
                    w[kv].a = ldg128(r + lo);
                    w[kv].b = ldg128(r + hi);
                } else if (full && slot_ok) {  // an earlier token of the block
                    const uint16_t* r = (kv ? p.c.v_tail : p.c.k_tail) + ((size_t(slot) * p.c.Hkv + h) * CT + tl) * D;
                    w[kv].a = ldcg128(r + lo);
                    w[kv].b = ldcg128(r + hi);
                }
            }
        };
        const uint16_t* q_in = p.q + row * p.q_stride;
        uint16_t* q_to = p.q_out + row * p.q_out_stride;
        const auto load_q = [&](int h) {
#pragma unroll
            for (int u = 0; u < NB; ++u) {
                if (h + u >= kvh1 * G) break;
                x[u].a = ldcg128(q_in + (h + u) * D + lo);  // q may be turned in place
                x[u].b = ldcg128(q_in + (h + u) * D + hi);
            }
        };
        // the first rows are under way while the angles are worked out
        if (do_kv) load_kv(kvh0);
        if (do_q && fresh) load_q(kvh0 * G);
        if (job == 0) __syncthreads();  // s_turns

        Angles an;
        if (turns && fresh) {
            const int pos = p.positions ? p.positions[row] : tok;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(pos));
                sincos_turn(uint32_t(at * s_turns[pr * 8 + 2 * e] >> 32), an.s[e].x, an.c[e].x);
                sincos_turn(uint32_t(at * s_turns[pr * 8 + 2 * e + 1] >> 32), an.s[e].y, an.c[e].y);
                an.s[e] = __fmul2_rn(an.s[e], make_float2(p.scale, p.scale));
                an.c[e] = __fmul2_rn(an.c[e], make_float2(p.scale, p.scale));
            }
        }
        if (do_kv && (!INT8 || full) && (id < 0 || id >= p.c.num_blocks)) {
            if (tid == 0) report(p.c.err, kErrBlockId);
            id = -1;
        }
        if (INT8 && do_kv && !slot_ok && (!full || start > base) && tid == 0) report(p.c.err, kErrSlot);
        const bool write = do_kv && (INT8 && !full ? slot_ok : id >= 0 && (slot_ok || start <= base));

        // Neighbouring CTAs (clusters) take the two halves in opposite order: one's
        // arithmetic on K and V beside the other's stream of queries
        for (int turn_of = 0; turn_of < 2; ++turn_of) {
        // ---- K and V rows, a head at a time
        if (turn_of == (bx & 1) && write) {
            if (PARTS > 1 && full) cluster_meet();  // every CTA has begun
            for (int kvh = kvh0; kvh < kvh1; ++kvh) {
                if (kvh > kvh0) load_kv(kvh);
                if (fresh) turn(w[0], an);
                if (full) {  // (`full` and `write` are the cluster's)
                    float mx[2];
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const __nv_bfloat162 top = absmax8(w[kv].b, absmax8(w[kv].a, __floats2bfloat162_rn(0.f, 0.f)));
                        mx[kv] = fmaxf(__low2float(top), __high2float(top));
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv) mx[kv] = fmaxf(mx[kv], __shfl_xor_sync(kFull, mx[kv], o));
                    // two buffers in turn: a CTA is at most one meeting ahead of another
                    float(*top)[2] = s_max[turn_no++ & 1];
                    if constexpr (PARTS > 1) {
                        if ((tid & 31) < PARTS)  // one lane for each CTA of the cluster
                            st_cluster_f2(smem_addr(top[part * WARPS + (tid >> 5)]), uint32_t(tid & 31), mx[0], mx[1]);
                        cluster_meet();
                    } else {
                        if ((tid & 31) == 0) *reinterpret_cast<float2*>(top[tid >> 5]) = make_float2(mx[0], mx[1]);
                        __syncthreads();
                    }
                    float m[2] = {0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < PARTS * WARPS; ++k) {
                        const float2 v = *reinterpret_cast<const float2*>(top[k]);
                        m[0] = fmaxf(m[0], v.x);
                        m[1] = fmaxf(m[1], v.y);
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const float scale = m[kv] < 1e-6f ? 1.0f : __fdiv_rn(m[kv], 127.0f), inv = __fdiv_rn(1.0f, scale);
                        int8_t* dst = static_cast<int8_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                      ((size_t(id) * p.c.Hkv + kvh) * CT + tl) * D;
                        *reinterpret_cast<uint2*>(dst + lo) = codes8(w[kv].a, scale, inv);
                        *reinterpret_cast<uint2*>(dst + hi) = codes8(w[kv].b, scale, inv);
                        if (tid == 0 && part == 0) p.c.scales[(size_t(id) * p.c.Hkv + kvh) * 2 + kv] = scale;
                    }
                } else if (fresh) {
                    // rows of the pool block, or of the tail
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        uint16_t* dst = INT8 ? (kv ? p.c.v_tail : p.c.k_tail) + ((size_t(slot) * p.c.Hkv + kvh) * CT + tl) * D
                                             : static_cast<uint16_t*>(kv ? p.c.v_pool : p.c.k_pool) +
                                                   ((size_t(id) * p.c.Hkv + kvh) * p.c.bs + tok % p.c.bs) * D;
                        *reinterpret_cast<uint4*>(dst + lo) = w[kv].a;
                        *reinterpret_cast<uint4*>(dst + hi) = w[kv].b;
                    }
                }
            }
        }

        // ---- the groups' queries, NB rows in flight
        if (turn_of != (bx & 1) && do_q && fresh) {
            for (int h = kvh0 * G; h < kvh1 * G; h += NB) {
                if (h > kvh0 * G) load_q(h);
#pragma unroll
                for (int u = 0; u < NB; ++u) {
                    if (h + u >= kvh1 * G) break;
                    turn(x[u], an);
                    *reinterpret_cast<uint4*>(q_to + (h + u) * D + lo) = x[u].a;
                    *reinterpret_cast<uint4*>(q_to + (h + u) * D + hi) = x[u].b;
                }
            }
        }
        }
    }
}

template <int D, bool INT8>
__global__ void __launch_bounds__(D, (INT8 ? 768 : 896) / D) rope_append_kernel(const __grid_constant__ RopeParams p) {
    rope_append<D, INT8, 1>(p);
}

// INT8 blocks of 64 tokens: a cluster of four CTAs, which exchange their rows'
// maxima. (One CTA of 4 D threads took 18.6 us for 128 single tokens and 67.5 us
// for 11200 tokens in chunks of 700: its threads sit idle in a step, and two of
// them fill an SM.)
template <int D>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(D, 768 / D)
rope_append_cluster_kernel(const __grid_constant__ RopeParams p) {
    rope_append<D, true, 4>(p);
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
    const int ct = int8 ? c->block_size : kRopeTokens, parts = ct / kRopeTokens;
    // the most aligned chunks that max_tokens tokens in a row can touch
    const unsigned chunks = unsigned((batch->max_tokens + ct - 2) / ct + 1);
    // Angles are worked out once a CTA, so it takes as many kv heads as leave
    // CTAs for a wave or two (7 of 128 threads fit on an SM). Of a chunk with few
    // tokens most threads are idle and a CTA's time is its loads' latency, so that one
    // wave is better: 128 single tokens of 32 kv heads, two waves -> one, bf16 13.3 us
    // -> 7.9 us, INT8 16.5 -> 11.9; but clusters of four, of which three CTAs end at
    // once, 19.4 -> 35.9.
    const int64_t enough = batch->max_tokens <= kRopeTokens && parts == 1 ? 152 * 6 : 152 * 7 * 2;
    const int64_t real = std::min<int64_t>(int64_t(chunks) * batch->B, batch->num_tokens / ct + 2 * int64_t(batch->B));
    p.heads = 1;
    while (p.heads * 2 <= c->num_kv_heads && real * parts * c->num_kv_heads / (p.heads * 2) >= enough) p.heads *= 2;
    // chunks of all sequences: no more than B times the longest's, nor than
    // the tokens fill, two begun ones a sequence
    p.ragged = chunks > 1;
    const int64_t gx = p.ragged ? real : batch->B;
    p.groups = (c->num_kv_heads + p.heads - 1) / p.heads;
    if ((gx * p.groups + 1) * parts > 0x7FFFFFFF) return PKV_ERR_INVALID;
    const dim3 grid(unsigned((gx * p.groups + p.ragged) * parts));
    void (*fn)(RopeParams) = nullptr;
    if (d == 128)
        fn = !int8 ? rope_append_kernel<128, false> : parts == 1 ? rope_append_kernel<128, true> : rope_append_cluster_kernel<128>;
    else
        fn = !int8 ? rope_append_kernel<64, false> : parts == 1 ? rope_append_kernel<64, true> : rope_append_cluster_kernel<64>;
    auto s = static_cast<cudaStream_t>(stream);
    if ((st = launch(fn, grid, dim3(unsigned(d)), 0, s, p)) != PKV_OK) return st;
    if (g_pdl.load(std::memory_order_relaxed) && batch->max_tokens > 1) {
        empty_kernel<<<1, 1, 0, s>>>();
        return cuda_status(cudaGetLastError());
    }
    return PKV_OK;
}
