// Windowed attention for many query rows (prompts and chunks) on the tensor
// cores of sm_103a (tcgen05, accumulators in tensor memory).
//
// One CTA per (split, 256 rows, kv head, sequence): two tiles of 128 rows, a
// row a (token, query head of the group), so that a kv head's whole group
// shares each K and V tile that the CTA loads. Keys come in tiles of 128
// tokens, gathered block by block through the block table.
//
//   warps 0-3, 4-7: softmax of row tile 0 and 1, one row a thread -- no shuffle
//                   anywhere; scores from tensor memory, weights back to it
//   then            the loader: one warp of tensor copies (bf16 cache), or four
//                   warps that turn int8 codes into bf16 (an integer up to 128
//                   is exact in bf16) on their way to shared memory; the
//                   block's scales go to the scores' and weights' columns
//   last warp       one thread that issues the multiplies
//
//   S_i = Q_i K^T   128 x 128 x D, operands in shared memory
//   O_i += P_i V    128 x D x 128, P_i in tensor memory over the scores it came
//                   from; V as it lies in the cache (MN-major B)
// The two row tiles take turns: while one's softmax runs the tensor core works
// for the other. S_i of the next key tile is issued right behind O_i += P_i V,
// so one commit tells the softmax both that its scores are there and that O_i
// may be corrected.
//
// The running maximum is a reference that follows the true one only when that
// is more than 2^8 ahead, so O_i is rarely rescaled. Weights are kept in units
// of 2^-24 (an exponent bias, free), so that neither they times V nor their
// sum leaves fp32 for any bf16 V. Weights are rounded to bf16 for the multiply
// (half a step, 2^-8 of each weight, as the outputs are); their sum is fp32.
#pragma once

#include "ptx_tc.cuh"
#include "window.cuh"

namespace pkv {

constexpr int kTcRows = 128;   // rows of a row tile
constexpr int kTcKeys = 128;   // tokens of a key tile
constexpr float kTcShift = 24.f;
constexpr float kTcAhead = 8.f;

template <int D, bool INT8>
struct TcTraits {
    // warps: softmax 0-7, the loader(s), the multiplies, INT8: the copies of codes
    static constexpr int kLoadWarps = INT8 ? 4 : 2;
    static constexpr int kMmaWarp = 8 + kLoadWarps;
    static constexpr int kThreads = (kMmaWarp + 1 + INT8) * 32;
    static constexpr int kTileBytes = kTcKeys * D * 2;          // one K or V tile (bf16) = one row tile of Q
    static constexpr int kStages = D == 128 ? 4 : 6;
    static constexpr int kRawStages = INT8 ? 2 : 0;             // int8 tiles on their way to bf16
    static constexpr int kRawBytes = kTcKeys * D;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + kRawStages * kRawBytes;
    static constexpr int kSlab = kTcKeys * 128;                 // 64 of a tile's D columns
};

// Barriers of a CTA.
template <int STAGES>
struct TcBars {
    uint64_t q_full;
    uint64_t kv_full[STAGES];
    uint64_t kv_empty[STAGES];
    uint64_t raw_full[2];   // INT8: codes to convert; bf16 [0]: a V tile whose dead rows have to be cleared first
    uint64_t raw_empty[2];
    uint64_t s_full[2];     // S_i is there and O_i += P_i V of the tile before is done
    uint64_t p_full[2];     // P_i is there, O_i corrected
    uint64_t drain;
};

template <bool V>
struct Const {
    static constexpr bool value = V;
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// Four int8 codes -> bf16, exact: a code with bit pattern s:m (one and seven
// bits) is (128 + m) - (s ? 256 : 128), and 0x4300 | m, 0x4300 | s << 7 are
// those numbers' bf16 patterns.
__device__ __forceinline__ void s8_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140), b = __byte_perm(w, 0x43434343u, 0x4342);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a & 0xFF7FFF7Fu), "r"(a & 0xFF80FF80u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b & 0xFF7FFF7Fu), "r"(b & 0xFF80FF80u));
}

template <int D, bool INT8>
__global__ void __launch_bounds__(TcTraits<D, INT8>::kThreads, 1)
window_tc_kernel(const __grid_constant__ WindowParams p) {
    using T = TcTraits<D, INT8>;
    constexpr int STAGES = T::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ TcBars<STAGES> bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_last;
    __shared__ uint32_t s_bad[8];          // units of a key tile that are not there, by tile % 8
    __shared__ float2 s_sc[INT8 ? 8 : 1][8];  // (K, V) scales of a key tile's units

    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.max_splits;
    const int j = int(blockIdx.x) % S, rt = p.row_tiles - 1 - int(blockIdx.x) / S;  // the longest first
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.c.Hq / p.c.Hkv, bs = p.c.bs;
    const SeqRange sq = seq_range(p.bt, b, bs, p.c.err, tid == 0 && blockIdx.x == 0 && kvh == 0);
    const int r_first = rt * 2 * kTcRows, r_end = min(sq.n * G, r_first + 2 * kTcRows);
    if (r_first >= r_end) return;
    const int nrow = r_end - r_first, nq = nrow > kTcRows ? 2 : 1;
    if (sq.bad) {
        if (j == 0)
            for (int e = tid; e < nrow * D; e += T::kThreads) {
                const int r = r_first + e / D;
                p.out[int64_t(sq.row0 + r / G) * p.out_stride + (kvh * G + r % G) * D + e % D] = 0;
            }
        return;
    }
    const int pos0 = sq.ctx - sq.n;
    const int p_first = pos0 + r_first / G, p_last = pos0 + (r_end - 1) / G;
    const KeyTiles kt = key_tiles(p_first, p_last, p.window, p.sinks, bs);  // in blocks
    const int U = kTcKeys / bs, lg = bs == 16 ? 4 : 6;                        // blocks a key tile
    const int tiles = (kt.n + U - 1) / U;
    int per = tiles;
    if (p.split_tiles > 0) per = max(p.split_tiles * kTile / kTcKeys, (tiles + S - 1) / S);
    const int ns = (tiles + per - 1) / per;
    if (j >= ns) return;
    const int k0 = j * per, n = min(tiles, k0 + per) - k0;  // this split's key tiles

    uint8_t* q_smem = smem + ((1024u - (smem_addr(smem) & 1023u)) & 1023u);
    const uint32_t q_addr = smem_addr(q_smem), kv_addr = q_addr + 2 * T::kTileBytes;
    const uint32_t bar0 = smem_addr(&bars);
    const auto bar = [&](const uint64_t* x) {
        return bar0 + uint32_t(reinterpret_cast<const uint8_t*>(x) - reinterpret_cast<const uint8_t*>(&bars));
    };
    constexpr int kMmaWarp = T::kMmaWarp;
    if (tid == 0) {
        mbar_init(bar(&bars.q_full), 1);
        mbar_init(bar(&bars.drain), 1);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(&bars.kv_full[s]), INT8 ? T::kLoadWarps * 32 : 1);
            mbar_init(bar(&bars.kv_empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(&bars.raw_full[i]), 1);
            mbar_init(bar(&bars.raw_empty[i]), T::kLoadWarps * 32);
            mbar_init(bar(&bars.s_full[i]), 1);
            mbar_init(bar(&bars.p_full[i]), kTcRows);
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const auto s_col = [&](int i) { return tmem + uint32_t(i) * 128u; };
    const auto o_col = [&](int i) { return tmem + 256u + uint32_t(i) * 128u; };
    // Waits for a phase; after about a second without it a role gives up (and
    // so, one after the other, do those that wait for it).
    const auto wait = [&](const uint64_t* x, uint32_t parity) { return wait_phase(bar(x), parity & 1u); };
    // ... for a whole warp, which it leaves converged
    const auto wait_warp = [&](const uint64_t* x, uint32_t parity) {
        return __all_sync(kFull, wait_phase(bar(x), parity & 1u)) != 0;
    };
    // tokens that no row of the CTA sees: their V rows count as zero
    const int dead_lo = max(0, p_first - p.window + 1);
    const auto dead = [&](int t) { return t > p_last || (t < dead_lo && t >= p.sinks); };
    const int32_t* table = p.bt.tables + size_t(b) * p.bt.max_blocks;
    // INT8: tokens from nfull on are in the slot's bf16 tail
    const int nfull = INT8 ? sq.ctx / bs * bs : sq.ctx;
    const int slot = INT8 ? p.bt.slots[b] : 0;

    if (warp < 8) {
        // ================= softmax of row tile i, a row a thread =================
        const int i = warp >> 2, row = r_first + tid;  // tid < 256: rows of the CTA in order
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_addr = s_col(i) + lane_base, o_addr = o_col(i) + lane_base;
        const bool have = row < r_end;
        const int hi = have ? pos0 + row / G : -1;
        const int lo = max(0, hi - p.window + 1);
        // the row tile's first and last position
        const int pf = pos0 + (r_first + i * kTcRows) / G;
        const int pl = pos0 + (min(r_end, r_first + (i + 1) * kTcRows) - 1) / G;
        const float scale = p.qscale;
        float m_ref = -INFINITY;  // reference of the exponent, in score units
        float2 l2 = make_float2(0.f, 0.f);
        bool ok = true;
        if (i < nq) {
            for (int jj = 0; jj < n; ++jj) {
                if (!(ok = wait_warp(&bars.s_full[i], jj))) break;
                tc_fence_after();
                const int u0 = (k0 + jj) * U;  // first block of the tile in the list
                const uint32_t bad = s_bad[jj & 7];
                const int t_first = kt.tile(u0) << lg;
                const bool masked = bad != 0 || u0 < kt.nsink || t_first + kTcKeys - 1 > pf || t_first < pl - p.window + 1;
                // One pass: weights against the reference as it stands, and the true
                // maximum beside them. Where a row's maximum is too far ahead (its
                // first tile, and rarely later) the reference follows, the sums and
                // O_i are rescaled, and the pass is made again: the weights wait in
                // registers (w), so the scores are still there. 16 columns at a time,
                // one chunk's load in flight while the other is worked on.
                uint32_t w[8][8];
                float2 sum;
                for (;;) {
                    const float neg = (m_ref == -INFINITY ? 0.f : -m_ref * scale) - kTcShift;
                    float mx = -INFINITY, my = -INFINITY;
                    sum = make_float2(0.f, 0.f);
                    const auto chunk = [&](auto hide, uint32_t (&r)[16], int c) {
                        const int col = c * 16, u = col >> lg;
                        if constexpr (hide.value) {
                            const int t0 = (kt.tile(u0 + u) << lg) + (col & (bs - 1));
                            // bit e: this row sees token t0 + e
                            const auto below = [](int x) { return (1u << min(16, max(0, x))) - 1u; };
                            uint32_t see = below(hi - t0 + 1) & (below(p.sinks - t0) | ~below(lo - t0));
                            if ((bad >> u) & 1u) see = 0u;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (!((see >> e) & 1u)) r[e] = 0xFF800000u;
                        }
                        float2 sc = make_float2(1.f, 1.f);  // INT8: the block's K and V scales
                        if (INT8) sc = s_sc[jj & 7][u];
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float2 x0 = make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                            float2 x1 = make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
                            if (INT8) {
                                x0 = mul2(x0, make_float2(sc.x, sc.x));
                                x1 = mul2(x1, make_float2(sc.x, sc.x));
                            }
                            mx = fmaxf(fmaxf(mx, x0.x), x1.x);
                            my = fmaxf(fmaxf(my, x0.y), x1.y);
                            x0 = __ffma2_rn(x0, make_float2(scale, scale), make_float2(neg, neg));
                            x1 = __ffma2_rn(x1, make_float2(scale, scale), make_float2(neg, neg));
                            x0 = make_float2(fast_exp2(x0.x), fast_exp2(x0.y));
                            x1 = make_float2(fast_exp2(x1.x), fast_exp2(x1.y));
                            sum = __fadd2_rn(sum, __fadd2_rn(x0, x1));
                            if (INT8) {
                                x0 = mul2(x0, make_float2(sc.y, sc.y));
                                x1 = mul2(x1, make_float2(sc.y, sc.y));
                            }
                            w[c][e / 2] = f2_to_bf16x2(x0.x, x0.y);
                            w[c][e / 2 + 1] = f2_to_bf16x2(x1.x, x1.y);
                        }
                    };
                    const auto pass = [&](auto hide) {
                        uint32_t ra[16], rb[16];
                        tmem_ld_start(ra, s_addr);
#pragma unroll
                        for (int c = 0; c < 8; c += 2) {
                            tmem_ld_wait(ra);
                            tmem_ld_start(rb, s_addr + c * 16 + 16);
                            chunk(hide, ra, c);
                            tmem_ld_wait(rb);
                            if (c < 6) tmem_ld_start(ra, s_addr + c * 16 + 32);
                            chunk(hide, rb, c + 1);
                        }
                    };
                    if (masked) pass(Const<true>{});
                    else pass(Const<false>{});
                    mx = fmaxf(mx, my);
                    const bool up = (mx - m_ref) * scale > kTcAhead;  // false while nothing has been seen
                    if (!__any_sync(kFull, up)) break;
                    const float f = up ? fast_exp2((m_ref - mx) * scale) : 1.f;
                    if (up) m_ref = mx;
                    l2.x *= f;
                    l2.y *= f;
                    if (jj > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld(o, o_addr + c);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st(o_addr + c, o);
                        }
                    }
                }
                l2 = __fadd2_rn(l2, sum);
#pragma unroll
                for (int c = 0; c < 8; ++c) tmem_st(s_addr + c * 8, w[c]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(&bars.p_full[i]));
            }
            if (ok) ok = wait_warp(&bars.s_full[i], n);  // the last O_i += P_i V
            tc_fence_after();
        }
        // ---- write the row
        if (i < nq && ok) {
            const float l = l2.x + l2.y;
            const int64_t tok = sq.row0 + (have ? row / G : 0);
            const int head = kvh * G + (have ? row % G : 0);
            const float f = ns > 1 ? 1.f : (l > 0.f ? 1.f / l : 0.f);
            const size_t at = (size_t(tok) * p.c.Hq + head) * S + j;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld(o, o_addr + c);
                if (!have) {
                } else if (ns > 1) {
                    float4* dst = reinterpret_cast<float4*>(p.ws_o + at * D + c);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        dst[e / 4] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                 __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.out_stride + head * D + c);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = f2_to_bf16x2(__uint_as_float(o[e + 2 * k]) * f, __uint_as_float(o[e + 2 * k + 1]) * f);
                        dst[e / 8] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            if (ns > 1 && have) {
                p.ws_ml[at * 2] = m_ref == -INFINITY ? -1e30f : m_ref * scale;
                p.ws_ml[at * 2 + 1] = l;
            }
        }
        if (!ok && lane == 0) report(p.c.err, kErrTimeout);
    } else if (warp < kMmaWarp) {
        if constexpr (!INT8) {
            // ================= loaders: tensor copies through the block table =================
            // One warp for K (and Q), one for V: copies of 16 rows x 128 bytes are issued
            // one by one, and a single warp's issue would not keep up with the multiplies.
            // The ids come one tile ahead, so their latency is off the path.
            const int role = warp - 8;  // 0: K, 1: V
            const CUtensorMap* tm = role ? &p.tm_v : &p.tm_k;
            const bool leader = elect_one();
            if (leader) {
                prefetch_tensormap(tm);
                if (role == 0) {
                    prefetch_tensormap(&p.tm_q);
                    mbar_arrive_expect_tx(bar(&bars.q_full), uint32_t(nq) * T::kTileBytes);
                    for (int i = 0; i < nq; ++i)
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_4d(q_addr + i * T::kTileBytes + h * T::kSlab, &p.tm_q, h * 64, 0, kvh,
                                        sq.row0 + (r_first + i * kTcRows) / G, bar(&bars.q_full));
                }
            }
            __syncwarp();
            const auto entry = [&](int tile) {  // lane u: the table's entry for unit u of a tile
                const int u = tile * U + lane;
                return lane < U && u < kt.n ? table[kt.tile(u)] : -1;
            };
            bool ok = true;
            uint32_t raw_phase = 0;
            int jj = 0, next = entry(k0);
            for (; jj < n; ++jj) {
                const int tile = k0 + jj, it = 2 * jj + role, s = it % STAGES;
                const int got = next, u = tile * U + lane;
                if (jj + 1 < n) next = entry(tile + 1);
                const bool there = got >= 0 && got < p.c.num_blocks;
                const int id = there ? got : p.c.num_blocks;  // behind the pool: the copy fills zeros
                bool fix = false;
                if (role == 0) {
                    if (lane < U && u < kt.n && !there) report(p.c.err, kErrBlockId);
                    const uint32_t missing = __ballot_sync(kFull, lane < U && !there);
                    if (lane == 0) s_bad[jj & 7] = missing;
                } else {
                    const int t0 = kt.tile(u) << lg;
                    fix = __any_sync(kFull, there && (t0 + bs - 1 > p_last || (t0 < dead_lo && t0 + bs > p.sinks)));
                }
                if (it >= STAGES && !(ok = wait_warp(&bars.kv_empty[s], it / STAGES - 1))) break;
                const uint32_t full = fix ? bar(&bars.raw_full[0]) : bar(&bars.kv_full[s]);
                const uint32_t dst = kv_addr + uint32_t(s) * T::kTileBytes;
                if (leader) mbar_arrive_expect_tx(full, T::kTileBytes);
                __syncwarp();
#pragma unroll
                for (int x = 0; x < kTcKeys / 16; ++x) {
                    if (x >= U) break;
                    const int uid = __shfl_sync(kFull, id, x);
                    if (leader) {
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(dst + uint32_t(h * T::kSlab + x * bs * 128), tm, h * 128, kvh * bs, uid, full);
                    }
                }
                if (fix) {
                    // clear the rows of V that no row of the CTA sees
                    if (!(ok = wait_warp(&bars.raw_full[0], raw_phase))) break;
                    ++raw_phase;
                    for (int x = 0; x < U && tile * U + x < kt.n; ++x) {
                        const int t0 = kt.tile(tile * U + x) << lg;
                        for (int e = lane; e < bs * (D / 8); e += 32) {
                            const int rr = e / (D / 8), ch = e % (D / 8);
                            if (dead(t0 + rr))
                                sts128(dst + uint32_t((ch / 8) * T::kSlab + (x * bs + rr) * 128 + (ch % 8) * 16),
                                       make_uint4(0u, 0u, 0u, 0u));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (leader) mbar_arrive(bar(&bars.kv_full[s]));
                }
            }
            if (!ok) {
                // let the copies in flight land before the CTA ends
                for (int x = max(0, jj - STAGES / 2); x < jj; ++x) {
                    const int it = 2 * x + role;
                    (void)wait_warp(&bars.kv_full[it % STAGES], it / STAGES);
                }
                if (lane == 0) report(p.c.err, kErrTimeout);
            }
        } else {
            // ================= INT8: codes (or tail rows) to bf16 tiles, 128 threads =================
            constexpr int CPR = D / 16;               // 16-element chunks a row
            constexpr int NC = kTcKeys * CPR / 128;   // chunks a thread
            const int th = tid - 256;
            const uint32_t raw0 = kv_addr + STAGES * T::kTileBytes;
            bool ok = true;
            for (int it = 0; it < 2 * n; ++it) {
                const int tile = k0 + it / 2, s = it % STAGES, rs = it % 2;
                ok = wait_warp(&bars.raw_full[rs], it / 2) && (it < STAGES || wait_warp(&bars.kv_empty[s], it / STAGES - 1));
                if (!ok) break;
                const uint32_t raw = raw0 + uint32_t(rs) * T::kRawBytes, dst = kv_addr + uint32_t(s) * T::kTileBytes;
                const uint32_t bad = s_bad[(it / 2) & 7];
                const int u0 = tile * U, t0 = kt.tile(u0) * bs;
                // a plain tile: every block is in the pool and (V) some row sees every token
                const bool plain = bad == 0 && u0 >= kt.nsink && t0 + kTcKeys <= min(nfull, p_last + 1) && t0 >= dead_lo;
                const uint16_t* tail = it % 2 ? p.c.v_tail : p.c.k_tail;
                uint4 w[NC];  // all loads first: shared memory's latency is paid once a tile
#pragma unroll
                for (int q = 0; q < NC; ++q) w[q] = lds128(raw + uint32_t(th + q * 128) * 16u);
                mbar_arrive(bar(&bars.raw_empty[rs]));
#pragma unroll
                for (int q = 0; q < NC; ++q) {
                    const int x = th + q * 128, row = x / CPR, c = x % CPR;
                    const uint32_t at = dst + uint32_t(row * 128 + (c / 4) * T::kSlab);
                    const uint32_t ca = uint32_t((2 * c) % 8), sw = uint32_t(row & 7);
                    uint4 lo, hi;
                    s8_to_bf16(w[q].x, lo.x, lo.y);
                    s8_to_bf16(w[q].y, lo.z, lo.w);
                    s8_to_bf16(w[q].z, hi.x, hi.y);
                    s8_to_bf16(w[q].w, hi.z, hi.w);
                    if (!plain) {
                        const int u = row >> lg, t = (kt.tile(u0 + u) << lg) + (row & (bs - 1));
                        if (((bad >> u) & 1u) || (it % 2 && dead(t))) {
                            lo = hi = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t >= nfull) {
                            const uint16_t* r = tail + ((size_t(slot) * p.c.Hkv + kvh) * bs + (t - nfull)) * D + c * 16;
                            lo = ldcg128(r);
                            hi = ldcg128(r + 8);
                        }
                    }
                    // the two slabs' threads take the halves in opposite order: different banks
                    const bool second = c >= 4;
                    sts128(at + (((ca + second) ^ sw) << 4), second ? hi : lo);
                    sts128(at + (((ca + !second) ^ sw) << 4), second ? lo : hi);
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(&bars.kv_full[s]));
            }
            if (!ok && lane == 0) report(p.c.err, kErrTimeout);
        }
    } else if (INT8 && warp == kMmaWarp + 1) {
        // ================= INT8: queries, codes and scales =================
        if (lane == 0) {
            prefetch_tensormap(&p.tm_q);
            mbar_arrive_expect_tx(bar(&bars.q_full), uint32_t(nq) * T::kTileBytes);
            for (int i = 0; i < nq; ++i)
                for (int h = 0; h < D / 64; ++h)
                    tma_load_4d(q_addr + i * T::kTileBytes + h * T::kSlab, &p.tm_q, h * 64, 0, kvh,
                                sq.row0 + (r_first + i * kTcRows) / G, bar(&bars.q_full));
        }
        const uint32_t raw0 = kv_addr + STAGES * T::kTileBytes;
        const uint32_t bytes = uint32_t(bs) * D;  // a block's rows of one kv head lie in a row
        bool ok = true;
        int issued = 0, id = -1;  // lane u: the pool block of unit u, or -1
        for (int it = 0; it < 2 * n; ++it) {
            const int tile = k0 + it / 2, rs = it % 2;
            if (it % 2 == 0) {
                id = -1;
                bool miss = false;
                if (lane < U) {
                    const int u = tile * U + lane, t0 = kt.tile(u) * bs;
                    float2 sc = make_float2(1.f, 1.f);
                    if (u >= kt.n) {
                        miss = true;
                    } else if (t0 >= nfull) {
                        miss = slot < 0 || slot >= p.c.max_slots;
                        if (miss) report(p.c.err, kErrSlot);
                    } else {
                        id = table[t0 / bs];
                        if (id < 0 || id >= p.c.num_blocks) {
                            report(p.c.err, kErrBlockId);
                            id = -1;
                            miss = true;
                        } else {
                            sc = __ldcg(reinterpret_cast<const float2*>(p.c.scales) + size_t(id) * p.c.Hkv + kvh);
                        }
                    }
                    s_sc[(it / 2) & 7][lane] = sc;
                }
                const uint32_t missing = __ballot_sync(kFull, miss);
                if (lane == 0) s_bad[(it / 2) & 7] = missing;
            }
            if (it >= 2) ok = wait_warp(&bars.raw_empty[rs], it / 2 - 1);
            if (!ok) break;
            const uint32_t have = __ballot_sync(kFull, id >= 0);
            const uint32_t full = bar(&bars.raw_full[rs]);
            if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(__popc(have)) * bytes);
            __syncwarp();
            if (id >= 0)
                bulk_g2s(raw0 + uint32_t(rs) * T::kRawBytes + uint32_t(lane) * bytes,
                         static_cast<const uint8_t*>(it % 2 ? p.c.v_pool : p.c.k_pool) +
                             (size_t(id) * p.c.Hkv + kvh) * bytes, bytes, full);
            issued = it + 1;
        }
        if (!ok) {  // let the copies in flight land before the CTA ends
            for (int it = max(0, issued - 2); it < issued; ++it) (void)wait(&bars.raw_full[it % 2], it / 2);
            if (lane == 0) report(p.c.err, kErrTimeout);
        }
    } else if (warp == kMmaWarp) {
        // ================= the multiplies =================
        // The whole warp walks through the loop, so that addresses and descriptors
        // stay warp-uniform; one thread issues. A step along K is an addition to a
        // descriptor's address field (16-byte units).
        constexpr uint32_t kDescS = mma_desc_bf16(kTcKeys, false), kDescO = mma_desc_bf16(D, true);
        constexpr uint64_t kTile16 = T::kTileBytes / 16;
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(kFull, tmem, 0);
        const uint64_t dq = smem_desc(q_addr, 16), dk = smem_desc(kv_addr, 16), dv = smem_desc(kv_addr, T::kSlab);
        const auto issue_s = [&](int i, int stage) {
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    constexpr uint64_t kSlab16 = T::kSlab / 16;
                    const uint64_t off = uint64_t(ks / 4) * kSlab16 + uint64_t(ks % 4) * 2u;
                    mma_ss(tm + uint32_t(i) * 128u, dq + uint64_t(i) * kTile16 + off, dk + uint64_t(stage) * kTile16 + off,
                           kDescS, ks > 0);
                }
            }
        };
        const auto commit = [&](const uint64_t* x) {
            if (leader) mma_commit(bar(x));
        };
        bool ok = wait_warp(&bars.q_full, 0) && wait_warp(&bars.kv_full[0], 0);
        if (ok) {
            tc_fence_after();
            for (int i = 0; i < nq; ++i) {
                issue_s(i, 0);
                commit(&bars.s_full[i]);
            }
            commit(&bars.kv_empty[0]);
        }
        for (int jj = 0; jj < n && ok; ++jj) {
            const int iv = 2 * jj + 1, ik = 2 * jj + 2, sv = iv % STAGES, sk = ik % STAGES;
            ok = wait_warp(&bars.kv_full[sv], iv / STAGES);
            for (int i = 0; i < nq && ok; ++i) {
                if (!(ok = wait_warp(&bars.p_full[i], jj))) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kTcKeys / 16; ++ks)
                        mma_ts(tm + 256u + uint32_t(i) * 128u, tm + uint32_t(i) * 128u + uint32_t(ks) * 8u,
                               dv + uint64_t(sv) * kTile16 + uint64_t(ks) * 128u, kDescO, jj > 0 || ks > 0);
                }
                if (i == nq - 1) commit(&bars.kv_empty[sv]);
                if (jj + 1 < n) {
                    if (i == 0 && !(ok = wait_warp(&bars.kv_full[sk], ik / STAGES))) break;
                    tc_fence_after();
                    issue_s(i, sk);
                }
                commit(&bars.s_full[i]);
                if (i == nq - 1 && jj + 1 < n) commit(&bars.kv_empty[sk]);
            }
        }
        if (!ok) {
            commit(&bars.drain);
            (void)wait_warp(&bars.drain, 0);
            if (lane == 0) report(p.c.err, kErrTimeout);
        }
    }

    // ---- the last split of the row tile to arrive merges all of them
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    if (ns == 1) return;
    int32_t* cnt = p.ws_count + (size_t(b) * p.c.Hkv + kvh) * p.row_tiles + rt;
    if (tid == 0) s_last = atom_add_acq_rel_gpu(cnt, 1) == ns - 1;
    __syncthreads();
    if (!s_last) return;
    // a warp a row: the splits' weights in its lanes, then D elements
    for (int r = warp; r < nrow; r += T::kThreads / 32) {
        const int rr = r_first + r;
        const size_t tok = sq.row0 + rr / G, head = kvh * G + rr % G, at = (tok * p.c.Hq + head) * S;
        const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + at;
        float mm = -1e30f;
        for (int q = lane; q < ns; q += 32) mm = fmaxf(mm, __ldcg(ml + q).x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(kFull, mm, off));
        float acc[D / 32], L = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
        for (int q = 0; q < ns; ++q) {
            const float2 x = __ldcg(ml + q);
            const float c = fast_exp2(x.x - mm);
            L += c * x.y;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] += c * __ldcg(p.ws_o + (at + q) * D + e * 32 + lane);
        }
        const float f = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            reinterpret_cast<__nv_bfloat16*>(p.out)[int64_t(tok) * p.out_stride + head * D + e * 32 + lane] =
                __float2bfloat16_rn(acc[e] * f);
    }
    if (tid == 0) *cnt = 0;  // ready for the next call
}

template <int D, bool INT8>
constexpr size_t window_tc_smem() { return TcTraits<D, INT8>::kSmem; }

}  // namespace pkv
