// Windowed attention for many query rows (prompts and chunks) on the tensor
// cores of sm_103a (tcgen05, accumulators in tensor memory).
//
// A work item is (split, 256 rows, kv head, sequence): two tiles of 128 rows, a
// row a (token, query head of the group), so that a kv head's whole group
// shares each K and V tile that the CTA loads. Keys come in tiles of 128
// tokens, gathered block by block through the block table. There is one CTA a
// SM; it walks from item to item, taking the grid's next one from the hardware
// (launch cancellation) while it works, so that an item's first loads and
// scores overlap the end of the item before. Long items are first in the grid.
//
//   warps 0-3, 4-7: softmax of row tile 0 and 1, one row a thread -- no shuffle
//                   anywhere; scores from tensor memory, weights back to it
//   bf16: 8, 9      the loaders of K and V: tensor copies of 16 (64) rows x 128 bytes
//   INT8: 8-11      int8 codes to bf16 (an integer up to 128 is exact in bf16), from
//                   shared memory to shared memory; the block's K scale goes to the
//                   score's factor, the V scale into the weight's exponent
//   then            one warp whose elected thread issues the multiplies, one that
//                   schedules the items and loads Q, INT8: one that copies the codes
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
// is more than 2^12 ahead, so O_i is rarely rescaled; it begins as the first
// tile's maximum (a reference of 1, without that tile's second pass, measured 5%
// slower: more tiles go beyond it later, and a tile that does costs its warp two
// passes). Weights are kept in units of 2^-40 (an exponent bias, free): 2^12 of
// them times the largest V and 2^28 tokens stay in fp32, one times a V of 2^-60
// leaves 26 bits. Weights are rounded to bf16 for the multiply
// (half a step, 2^-8 of each weight, as the outputs are); their sum is fp32.
//
// Measured, d = 128, 8 kv heads (4 d flops a visible pair and head): causal
// prompts of 7400 to 8000 tokens, 16 query heads, bf16, 1.0 TF in 707 us, 1415
// TF/s (cuBLAS: 1969), 745 to 755 us at the clocks that a long run settles at;
// prompts of 5000 to 8192 tokens, window 1024, 32 query heads, 211 GF in 197 to
// 201 us; chunks of 100 to 512 tokens, window 4096, INT8, 161 GF in 193 us. The
// INT8 kernel of d = 128 spills 17 words. A key tile of an item takes about 3400 cycles, its multiplies 2048
// of them. They read 192 KB of shared memory for it (Q and K at 128 bytes a cycle,
// all that it has; V at 64) and the copies write another 64 KB, 2048 cycles too;
// what is above that is the chain from scores to weights (without the loads from
// tensor memory: 644 us). Scores in halves of 64 tokens, the first issued before
// O_i += P_i V so that the softmax starts earlier, read Q twice as often: 823 us.
// With windows the tiles at both ends, half masked but multiplied whole, and the
// items' ends come to that (ten tiles an item). INT8: the conversion stores as
// much to shared memory again, and 328 items on 152 SMs fill two rounds and a
// sixth, whose items are split. Of other forms, two threads a row, exponentials
// in polynomials, and scores in two buffers of 32 columns were slower or the same.
//
// Work list: a CTA counts the batch's row tiles once and walks along the list (3 of
// 65535 sequences with tokens: 1.75 ms a call, of which 0.4 us for each item of the
// grid that the batch does not have; searched from the front for every item, 3 of
// 16000 took 142 ms).
#pragma once

#include "ptx_tc.cuh"
#include "window.cuh"

namespace pkv {

constexpr int kTcRows = 128;   // rows of a row tile
constexpr int kTcKeys = 128;   // tokens of a key tile
constexpr float kTcShift = 40.f;
constexpr float kTcAhead = 12.f;

template <int D, bool INT8>
struct TcTraits {
    static constexpr int kLoadWarps = INT8 ? 4 : 2;
    static constexpr int kMmaWarp = 8 + kLoadWarps;
    static constexpr int kPlanWarp = kMmaWarp + 1;
    static constexpr int kThreads = INT8 ? 512 : 384;           // whole warpgroups
    // Registers a thread once the warpgroups have shared them out: softmax (two),
    // loaders (bf16: with the multiplies and the plan), INT8: multiplies and plan.
    // Their sum is what the block is launched with.
    static constexpr int kLaunchRegs = INT8 ? kTcLaunchRegsInt8 : kTcLaunchRegsBf16;
    static constexpr int kSoftmaxRegs = INT8 ? 168 : 200;
    static constexpr int kLoadRegs = 104;
    static constexpr int kRestRegs = INT8 ? 72 : 0;
    static_assert(256 * kSoftmaxRegs + 128 * (kLoadRegs + kRestRegs) == kThreads * kLaunchRegs, "register split");
    static constexpr int kTileBytes = kTcKeys * D * 2;          // one K or V tile (bf16) = one row tile of Q
    static constexpr int kStages = D == 64 ? 6 : INT8 ? 3 : 4;
    static constexpr int kRawStages = INT8 ? 2 : 0;             // codes of a K and a V tile on their way to bf16
    static constexpr int kRawBytes = kTcKeys * D;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 8 * 4096 + kRawStages * kRawBytes;
    static constexpr int kSlab = kTcKeys * 128;                 // 64 of a tile's D columns
};

// Barriers of a CTA.
template <int STAGES>
struct TcBars {
    uint64_t q_full, q_empty;
    uint64_t kv_full[STAGES];
    uint64_t kv_empty[STAGES];
    uint64_t raw_full[2];    // INT8: codes of a K, V tile; bf16 [0]: a V tile whose dead rows have to be cleared first
    uint64_t raw_empty[2];
    uint64_t s_full[2];      // S_i is there and O_i += P_i V of the tile before is done
    uint64_t p_full[2];      // P_i is there, O_i corrected
    uint64_t o_full[2];      // O_i is complete
    uint64_t item_full[2];   // an item's description is there
    uint64_t item_empty[2];  // every warp has taken it
    uint64_t merge;          // the softmax warps, around the merge of splits
    uint64_t next;           // the answer about the next item is there
    uint64_t drain;
};

// A work item, as the planning warp describes it to the others.
struct TcItem {
    int kind;          // 0: attention; 1: rows of a sequence with a bad length, zero; 2: the end
    int b, kvh, j;     // sequence, kv head, split
    int ns;            // splits of this row tile
    int at;            // its place among the row tiles that are split
    int row0, pos0;    // the sequence's first row, and its position
    int r_first, r_end;
    int p_first, p_last;
    KeyTiles kt;       // in blocks
    int k0, n;         // this split's key tiles
    int nfull, slot;   // INT8: tokens from nfull on are in the slot's bf16 tail
};

// f(0), f(1), ... f(N - 1) with the argument a constant.
template <int V>
struct Index {
    static constexpr int value = V;
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(const F& f) {
    if constexpr (I < N) {
        f(Index<I>{});
        each<N, I + 1>(f);
    }
}

template <bool V>
struct Const {
    static constexpr bool value = V;
};

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
    __shared__ TcItem s_item[2];
    __shared__ __align__(16) uint4 s_next;
    __shared__ uint32_t s_tmem;
    __shared__ int s_last;
    // Splits that another CTA may wait for (see the end): items up to s_settled have
    // arrived, those up to s_published were described to the other warps.
    __shared__ int s_settled, s_published;
    // units of a key tile that are not there, by tile % 8; INT8, [1]: or whose V is zero
    __shared__ uint32_t s_bad[1 + INT8][8];
    __shared__ float2 s_sc[INT8 ? 8 : 1][8];   // units' K scale times p.qscale, log2 of the V scale

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.c.Hq / p.c.Hkv, lgG = 31 - __clz(G), bs = p.c.bs, lg = bs == 16 ? 4 : 6, U = kTcKeys >> lg;  // U: blocks a key tile
    const int S = p.max_splits;
    uint8_t* q_smem = smem + ((1024u - (smem_addr(smem) & 1023u)) & 1023u);
    const uint32_t q_addr = smem_addr(q_smem), kv_addr = q_addr + 2 * T::kTileBytes;
    const uint32_t stage0 = kv_addr + STAGES * T::kTileBytes;  // 4 KB a softmax warp, for its output rows
    const uint32_t raw0 = stage0 + 8 * 4096;                   // INT8: codes of a K and a V tile
    const uint32_t bar0 = smem_addr(&bars);
    const auto bar = [&](const uint64_t* x) {
        return bar0 + uint32_t(reinterpret_cast<const uint8_t*>(x) - reinterpret_cast<const uint8_t*>(&bars));
    };
    if (tid == 0) {
        mbar_init(bar(&bars.q_full), 1);
        mbar_init(bar(&bars.q_empty), 1);
        mbar_init(bar(&bars.next), 1);
        mbar_init(bar(&bars.merge), 8);
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
            mbar_init(bar(&bars.o_full[i]), 1);
            mbar_init(bar(&bars.item_full[i]), 1);
            mbar_init(bar(&bars.item_empty[i]), 8 + T::kLoadWarps + 1 + INT8);
        }
        fence_mbar_init();
        s_settled = s_published = 0;
    }
    if (warp == T::kMmaWarp) tmem_alloc(smem_addr(&s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // Waits for a phase, a whole warp, which it leaves converged. After about a
    // second without it a role gives up, and so, one after the other, do those
    // that wait for it.
    const auto wait = [&](const uint64_t* x, uint32_t parity) {
        return __all_sync(kFull, wait_phase(bar(x), parity & 1u)) != 0;
    };
    pdl_wait();
    pdl_launch_dependents();

    // A split of a row tile arrives (one thread): true for the last one, which leaves
    // the counter ready for the next call.
    const auto arrive = [&](int at, int ns) {
        const bool last = atom_add_acq_rel_gpu(p.ws_count + at, 1) == ns - 1;
        if (last) p.ws_count[at] = 0;
        return last;
    };
    bool ok = true;
    // The q-th item of this CTA (every warp but the planner's): false at the end.
    const auto take = [&](int q) {
        ok = wait(&bars.item_full[q & 1], q >> 1);
        return ok && s_item[q & 1].kind != 2;
    };
    // Its description is no longer needed.
    const auto release = [&](int q) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&bars.item_empty[q & 1]));
    };

    if (warp < 8) reg_inc<T::kSoftmaxRegs>();
    else if (warp < 12) reg_dec<T::kLoadRegs>();
    else reg_dec<INT8 ? T::kRestRegs : 24>();  // (bf16 has no such warps)

    if (warp < 8) {
        // ================= softmax of row tile i, a row a thread =================
        const int i = warp >> 2;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + uint32_t(i) * 128u + lane_base, o_addr = tmem + 256u + uint32_t(i) * 128u + lane_base;
        const float scale = p.qscale;
        int tiles = 0, mine = 0, done = 0;  // key tiles of the CTA and of this row tile, items of this row tile
        int merges = 0;
        const auto meet = [&](int phase) {  // the eight softmax warps
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(&bars.merge));
            return wait(&bars.merge, phase);
        };
        for (int q = 0; take(q); release(q++)) {
            const TcItem& im = s_item[q & 1];
            const int row = im.r_first + tid;  // tid < 256: rows of the item in order
            const bool have = row < im.r_end;
            if (im.kind == 1) {
                for (int e = tid; e < (im.r_end - im.r_first) * D; e += 256) {
                    const int r = im.r_first + e / D;
                    p.out[int64_t(im.row0 + (r >> lgG)) * p.out_stride + (im.kvh * G + (r & (G - 1))) * D + e % D] = 0;
                }
                continue;
            }
            const KeyTiles kt = im.kt;
            const int n = im.n, k0 = im.k0;
            const bool used = im.r_first + i * kTcRows < im.r_end;
            float m_ref = -INFINITY;  // reference of the exponent (base 2)
            float2 l2 = make_float2(0.f, 0.f);
            if (used) {
                const int hi = have ? im.pos0 + (row >> lgG) : -1;
                const int lo = max(0, hi - p.window + 1);
                // the row tile's first and last position
                const int pf = im.pos0 + ((im.r_first + i * kTcRows) >> lgG);
                const int pl = im.pos0 + ((min(im.r_end, im.r_first + (i + 1) * kTcRows) - 1) >> lgG);
                for (int jj = 0; jj < n; ++jj) {
                    if (!(ok = wait(&bars.s_full[i], mine + jj))) break;
                    tc_fence_after();
                    const int u0 = (k0 + jj) * U;  // first block of the tile in the list
                    const int slot = (tiles + jj) & 7;
                    const uint32_t bad = s_bad[0][slot];
                    const int t_first = kt.tile(u0) << lg;
                    const bool masked =
                        bad != 0 || u0 < kt.nsink || t_first + kTcKeys - 1 > pf || t_first < pl - p.window + 1;
                    // One pass: weights against the reference as it stands, and the true
                    // maximum beside them. Where a row's maximum is too far ahead (its
                    // first tile, and rarely later) the reference follows, the sums and
                    // O_i are rescaled, and the pass is made again: the weights wait in
                    // registers (w), so the scores are still there. 16 columns at a time,
                    // one chunk's load in flight while the other is worked on.
                    uint32_t w[8][8];
                    float2 sum;
                    // INT8: the columns' factors, read here at once: beside the multiplies
                    // and the conversion a shared-memory load in the pass takes long
                    float2 sc[INT8 ? 8 : 1];
                    if (INT8) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) sc[c] = lds64(smem_addr(&s_sc[slot][(c * 16) >> lg]));
                    }
                    for (;;) {
                        const float neg = (m_ref == -INFINITY ? 0.f : -m_ref) - kTcShift;
                        float mx = -INFINITY;
                        sum = make_float2(0.f, 0.f);
                        const auto chunk = [&](auto hide, uint32_t (&r)[16], int c) {
                            const int col = c * 16, u = col >> lg;
                            if constexpr (hide.value) {
                                const int t0 = (kt.tile(u0 + u) << lg) + (col & (bs - 1));
                                // bit e: this row sees token t0 + e
                                const auto below = [](int x) { return (1u << min(16, max(0, x))) - 1u; };
                                uint32_t see = below(hi - t0 + 1) & (below(p.sinks - t0) | ~below(lo - t0));
                                if ((bad >> u) & 1u) see = 0u;
                                if (__all_sync(kFull, (see & 0xFFFFu) == 0u)) {  // nothing for the whole warp
#pragma unroll
                                    for (int e = 0; e < 8; ++e) w[c][e] = 0u;
                                    return;
                                }
                                if (!__all_sync(kFull, (see & 0xFFFFu) == 0xFFFFu)) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        if (!((see >> e) & 1u)) r[e] = 0xFF800000u;
                                }
                            }
                            // INT8: a score is its K scale times the column, a weight its V
                            // scale times the softmax weight, by way of the exponent
                            const float a = INT8 ? sc[INT8 ? c : 0].x : scale, b = INT8 ? neg + sc[INT8 ? c : 0].y : neg;
                            const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
                            float mc = -INFINITY, md = -INFINITY;
                            float2 part = make_float2(0.f, 0.f);
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                float2 x0 = make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                                float2 x1 = make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
                                mc = fmaxf(fmaxf(mc, x0.x), x1.x);
                                md = fmaxf(fmaxf(md, x0.y), x1.y);
                                x0 = __ffma2_rn(x0, a2, b2);
                                x1 = __ffma2_rn(x1, a2, b2);
                                x0 = make_float2(fast_exp2(x0.x), fast_exp2(x0.y));
                                x1 = make_float2(fast_exp2(x1.x), fast_exp2(x1.y));
                                part = __fadd2_rn(part, __fadd2_rn(x0, x1));
                                w[c][e / 2] = f2_to_bf16x2(x0.x, x0.y);
                                w[c][e / 2 + 1] = f2_to_bf16x2(x1.x, x1.y);
                            }
                            mx = fmaxf(mx, fmaxf(mc, md) * a);
                            if (INT8) {
                                const float vi = fast_exp2(-sc[INT8 ? c : 0].y);
                                sum = __ffma2_rn(part, make_float2(vi, vi), sum);
                            } else {
                                sum = __fadd2_rn(sum, part);
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
                        const bool up = mx - m_ref > kTcAhead;  // false while nothing has been seen
                        if (!__any_sync(kFull, up)) break;
                        const float f = up ? fast_exp2(m_ref - mx) : 1.f;
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
                if (ok) ok = wait(&bars.o_full[i], done);
                mine += n;
                ++done;
            }
            tiles += n;
            if (!ok) break;
            // ---- write the row
            const float l = l2.x + l2.y;
            if (used) {
                tc_fence_after();
                const float f = im.ns > 1 ? 1.f : l > 0.f ? 1.f / l : 0.f;
                // Rows lie far apart, a thread's own would be written a piece of a line at
                // a time: the warp's 32 rows pass through shared memory, 128 bytes of each
                // at a time (32 fp32 partials or 64 bf16 outputs), chunks swizzled by row,
                // and leave as a tensor copy, which nobody waits for -- stores would go
                // out at an SM's 43 bytes a cycle (a 9-tile item: 2.0 us against 1.4 us).
                // The output's last rows share their box with the next sequence's, and
                // leave as stores of whole lines.
                const uint32_t st = stage0 + uint32_t(warp) * 4096u;
                const uint32_t mine_at = st + uint32_t(lane) * 128u, mine_sw = uint32_t(lane & 7);
                const bool partial = im.ns > 1;
                const int steps = partial ? D / 32 : D / 64;
                const int first = im.r_first + warp * 32, rows = min(32, im.r_end - first);
                for (int c = 0; c < steps; ++c) {
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                    if (partial) {
                        uint32_t o[32];
                        tmem_ld(o, o_addr + c * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sts128(mine_at + ((uint32_t(e) ^ mine_sw) << 4), make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t o[32];
                            tmem_ld(o, o_addr + c * 64 + h * 32);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t x[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    x[k] = f2_to_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * f, __uint_as_float(o[8 * e + 2 * k + 1]) * f);
                                sts128(mine_at + ((uint32_t(h * 4 + e) ^ mine_sw) << 4), make_uint4(x[0], x[1], x[2], x[3]));
                            }
                        }
                    }
                    if (partial || rows == 32) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (partial) tma_store_3d(&p.tm_ws, st, c * 32, im.j, im.at * 256 + warp * 32);
                            else tma_store_4d(&p.tm_out, st, c * 64, 0, im.kvh, im.row0 + (first >> lgG));
                            bulk_commit();
                        }
                    } else {
                        __syncwarp();
#pragma unroll 1
                        for (int r = lane / 8; r < rows; r += 4) {  // four rows at a time
                            const int rr = first + r, ch = lane % 8;
                            const uint4 v = lds128(st + uint32_t(r) * 128u + ((uint32_t(ch) ^ uint32_t(r & 7)) << 4));
                            *reinterpret_cast<uint4*>(p.out + int64_t(im.row0 + (rr >> lgG)) * p.out_stride +
                                                      (im.kvh * G + (rr & (G - 1))) * D + c * 64 + ch * 8) = v;
                        }
                    }
                }
                if (im.ns > 1 && have) {
                    reinterpret_cast<float2*>(p.ws_ml)[size_t(im.at * 256 + tid) * S + im.j] =
                        make_float2(m_ref == -INFINITY ? -1e30f : m_ref, l);
                }
                tc_fence_before();  // O_i has been read before the next item's P_i is announced
            }
            if (im.ns == 1) continue;

            // ---- the last split of the row tile to arrive merges all of them
            if (lane == 0) bulk_wait();  // this warp's partials are written
            if (!(ok = meet(merges++))) break;
            if (tid == 0) {
                s_last = arrive(im.at, im.ns);
                s_settled = q + 1;
            }
            if (!(ok = meet(merges++))) break;
            if (!s_last) continue;
            // Latency counts here: a warp takes eight rows at a time, whose partials (16 bytes
            // a lane) of two splits are in flight, and a lane has those rows' weights of one
            // split in 32.
            const int rows = im.r_end - im.r_first, parts = im.ns;
            const int head0 = im.kvh * G, row0 = im.row0;
            const size_t place0 = size_t(im.at) * 256;  // of the item's first row in the workspace
            const auto ml = [&](int r, int x) {
                return __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + (place0 + min(r, rows - 1)) * S + x);
            };
            constexpr int E = D / 32;  // elements a lane
            // the warp's rows are warp * 8 .. + 7 of every 64; this lane has one's statistics
            float mm = -1e30f, L = 0.f;
#pragma unroll 4
            for (int x = 0; x < parts; ++x) {
                const float2 v = ml(lane / 8 * 64 + warp * 8 + lane % 8, x);
                const float up = fmaxf(mm, v.x);
                L = L * fast_exp2(mm - up) + v.y * fast_exp2(v.x - up);
                mm = up;
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            for (int g = warp * 8; g < rows; g += 64) {
                float acc[8][E];
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
                for (int x0 = 0; x0 < parts; x0 += 32) {
                    float wr[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float m = __shfl_sync(kFull, mm, g / 64 * 8 + r), f = __shfl_sync(kFull, inv, g / 64 * 8 + r);
                        wr[r] = x0 + lane < parts ? fast_exp2(ml(g + r, x0 + lane).x - m) * f : 0.f;
                    }
                    for (int x = 0; x < min(32, parts - x0); x += 2) {
                        float v[2][8][E];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                const float* o = p.ws_o + ((place0 + min(g + r, rows - 1)) * S + min(x0 + x + h, parts - 1)) * D + lane * E;
                                if constexpr (E == 4) {
                                    const float4 f = __ldcg(reinterpret_cast<const float4*>(o));
                                    v[h][r][0] = f.x; v[h][r][1] = f.y; v[h][r][2] = f.z; v[h][r][3] = f.w;
                                } else {
                                    const float2 f = __ldcg(reinterpret_cast<const float2*>(o));
                                    v[h][r][0] = f.x; v[h][r][1] = f.y;
                                }
                            }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                const float w = __shfl_sync(kFull, wr[r], x + h);  // (behind the last: 0)
#pragma unroll
                                for (int e = 0; e < E; ++e) acc[r][e] += w * v[h][r][e];
                            }
                    }
                }
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (g + r >= rows) break;
                    const int rr = im.r_first + g + r;
                    uint16_t* at = p.out + int64_t(row0 + (rr >> lgG)) * p.out_stride + (head0 + (rr & (G - 1))) * D + lane * E;
#pragma unroll
                    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(at + e) = f2_to_bf16x2(acc[r][e], acc[r][e + 1]);
                }
            }
        }
        if (lane == 0) {
            bulk_wait();
            if (!ok) report(p.c.err, kErrTimeout);
        }
    } else if (warp < T::kMmaWarp) {
        int tiles = 0;  // key tiles of the items before
        if constexpr (!INT8) {
            // ================= loaders: tensor copies through the block table =================
            // One warp for K, one for V: copies of 16 rows x 128 bytes are issued one by
            // one, and a single warp's issue would not keep up with the multiplies. The
            // ids come one tile ahead, so their latency is off the path.
            const int role = warp - 8;  // 0: K, 1: V
            const CUtensorMap* tm = role ? &p.tm_v : &p.tm_k;
            const bool leader = elect_one();
            if (leader) prefetch_tensormap(tm);
            __syncwarp();
            uint32_t raw_phase = 0;
            for (int q = 0; ok && take(q); release(q++)) {
                const TcItem& im = s_item[q & 1];
                if (im.kind == 1) continue;
                const KeyTiles kt = im.kt;
                const int n = im.n, k0 = im.k0, p_last = im.p_last, y = im.kvh * bs;
                const int dead_lo = max(0, im.p_first - p.window + 1);
                const int32_t* table = p.bt.tables + size_t(im.b) * p.bt.max_blocks;
                const auto entry = [&](int tile) {  // lane u: the table's entry for unit u of a tile
                    const int u = tile * U + lane;
                    return lane < U && u < kt.n ? table[kt.tile(u)] : -1;
                };
                int next = entry(k0), jj = 0;
                for (; jj < n; ++jj) {
                    const int tile = k0 + jj, it = 2 * (tiles + jj) + role, s = it % STAGES;
                    const int got = next, u = tile * U + lane;
                    if (jj + 1 < n) next = entry(tile + 1);
                    const bool there = got >= 0 && got < p.c.num_blocks;
                    const int id = there ? got : p.c.num_blocks;  // behind the pool: the copy fills zeros
                    bool fix = false;
                    if (role == 0) {
                        if (lane < U && u < kt.n && !there) report(p.c.err, kErrBlockId);
                        const uint32_t missing = __ballot_sync(kFull, lane < U && !there);
                        if (lane == 0) s_bad[0][(tiles + jj) & 7] = missing;
                    } else {
                        const int t0 = kt.tile(u) << lg;
                        fix = __any_sync(kFull, there && (t0 + bs - 1 > p_last || (t0 < dead_lo && t0 + bs > p.sinks)));
                    }
                    if (it >= STAGES && !(ok = wait(&bars.kv_empty[s], it / STAGES - 1))) break;
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
                                tma_load_3d(dst + uint32_t(h * T::kSlab + x * bs * 128), tm, h * 128, y, uid, full);
                        }
                    }
                    if (fix) {
                        // clear the rows of V that no row of the item sees
                        if (!(ok = wait(&bars.raw_full[0], raw_phase))) break;
                        ++raw_phase;
                        for (int x = 0; x < U && tile * U + x < kt.n; ++x) {
                            const int t0 = kt.tile(tile * U + x) << lg;
                            for (int e = lane; e < bs * (D / 8); e += 32) {
                                const int rr = e / (D / 8), ch = e % (D / 8);
                                if (t0 + rr > p_last || (t0 + rr < dead_lo && t0 + rr >= p.sinks))
                                    sts128(dst + uint32_t((ch / 8) * T::kSlab + (x * bs + rr) * 128 + (ch % 8) * 16),
                                           make_uint4(0u, 0u, 0u, 0u));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader) mbar_arrive(bar(&bars.kv_full[s]));
                    }
                }
                tiles += ok ? n : jj;
            }
            if (!ok) {
                // let the copies in flight land before the CTA ends
                for (int x = max(0, tiles - STAGES / 2); x < tiles; ++x) {
                    const int it = 2 * x + role;
                    (void)wait(&bars.kv_full[it % STAGES], it / STAGES);
                }
                if (lane == 0) report(p.c.err, kErrTimeout);
            }
        } else {
            // ================= INT8: codes (or tail rows) to bf16 tiles, 128 threads =================
            constexpr int CPR = D / 16;               // 16-element chunks a row
            constexpr int NC = kTcKeys * CPR / 128;   // chunks a thread
            constexpr int kStep = 128 / CPR;          // rows from a thread's chunk to its next
            // A thread's chunk c of rows row0 + k * kStep. Eight neighbouring threads have
            // four chunks of two rows in the same slab: their swizzled 16-byte stores fall
            // in different banks.
            const int c = D == 128 ? (lane & 3) + ((lane >> 3) & 1) * 4 : lane & 3;
            const int row0 = (warp - 8) * (32 / CPR) + (D == 128 ? ((lane >> 2) & 1) + (lane >> 4) * 2 : lane >> 2);
            for (int q = 0; ok && take(q); release(q++)) {
                const TcItem& im = s_item[q & 1];
                if (im.kind == 1) continue;
                const KeyTiles kt = im.kt;
                const int n = im.n, k0 = im.k0, p_last = im.p_last, nfull = im.nfull;
                const int dead_lo = max(0, im.p_first - p.window + 1);
                for (int x = 0; x < 2 * n; ++x) {  // K and V tiles in turn
                    const int tile = k0 + x / 2, v = x % 2, it = 2 * tiles + x, s = it % STAGES;
                    if (!(ok = wait(&bars.raw_full[v], it / 2))) break;
                    const uint32_t raw = raw0 + uint32_t(v) * T::kRawBytes + uint32_t(row0 * D + c * 16);
                    uint4 w[NC];
                    each<NC>([&](auto k) { w[k.value] = lds128_at<k.value * kStep * D>(raw); });
                    const uint32_t bad = s_bad[v][(it / 2) & 7];
                    const int u0 = tile * U, t0 = kt.tile(u0) << lg;
                    // a plain tile: every block is in the pool and (V) some row sees every token
                    const bool plain = bad == 0 && u0 >= kt.nsink && t0 + kTcKeys <= min(nfull, p_last + 1) && t0 >= dead_lo;
                    if (it >= STAGES && !(ok = wait(&bars.kv_empty[s], it / STAGES - 1))) break;
                    mbar_arrive(bar(&bars.raw_empty[v]));
                    const uint32_t dst = kv_addr + uint32_t(s) * T::kTileBytes + uint32_t((c / 4) * T::kSlab + row0 * 128);
                    const uint32_t ca = uint32_t((2 * c) % 8), sw = uint32_t(row0 & 7);
                    const uint32_t a0 = dst + ((ca ^ sw) << 4), a1 = dst + (((ca + 1) ^ sw) << 4);
                    const auto convert = [&](const uint4& x, uint4& lo, uint4& hi) {
                        s8_to_bf16(x.x, lo.x, lo.y);
                        s8_to_bf16(x.y, lo.z, lo.w);
                        s8_to_bf16(x.z, hi.x, hi.y);
                        s8_to_bf16(x.w, hi.z, hi.w);
                    };
                    if (plain) {
                        each<NC>([&](auto k) {
                            uint4 lo, hi;
                            convert(w[k.value], lo, hi);
                            sts128_at<k.value * kStep * 128>(a0, lo);
                            sts128_at<k.value * kStep * 128>(a1, hi);
                        });
                    } else {
#pragma unroll 1
                        for (int k = 0; k < NC; ++k) {
                            const int row = row0 + k * kStep, u = row >> lg;
                            const int t = (kt.tile(u0 + u) << lg) + (row & (bs - 1));
                            uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                            if (((bad >> u) & 1u) || (v && (t > p_last || (t < dead_lo && t >= p.sinks)))) {
                            } else if (t >= nfull) {
                                const uint16_t* r = (v ? p.c.v_tail : p.c.k_tail) +
                                                    ((size_t(im.slot) * p.c.Hkv + im.kvh) * bs + (t - nfull)) * D + c * 16;
                                lo = ldcg128(r);
                                hi = ldcg128(r + 8);
                            } else {
                                uint4 x = w[0];
#pragma unroll
                                for (int e = 1; e < NC; ++e)
                                    if (e == k) x = w[e];
                                convert(x, lo, hi);
                            }
                            sts128(a0 + uint32_t(k * kStep * 128), lo);
                            sts128(a1 + uint32_t(k * kStep * 128), hi);
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(bar(&bars.kv_full[s]));
                }
                tiles += n;
            }
            if (!ok && lane == 0) report(p.c.err, kErrTimeout);
        }
    } else if (warp == T::kMmaWarp) {
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
        int tiles = 0, mine[2] = {0, 0}, items = 0;
        for (int q = 0; ok && take(q); release(q++)) {
            const TcItem& im = s_item[q & 1];
            if (im.kind == 1) continue;
            const int n = im.n;
            const int nq = im.r_end - im.r_first > kTcRows ? 2 : 1;
            const int first = 2 * tiles, sf = first % STAGES;
            ok = wait(&bars.q_full, items) && wait(&bars.kv_full[sf], first / STAGES);
            if (!ok) break;
            tc_fence_after();
            for (int i = 0; i < nq; ++i) {
                issue_s(i, sf);
                commit(&bars.s_full[i]);
            }
            commit(&bars.kv_empty[sf]);
            if (n == 1) commit(&bars.q_empty);
            for (int jj = 0; jj < n && ok; ++jj) {
                const int iv = 2 * (tiles + jj) + 1, ik = iv + 1, sv = iv % STAGES, sk = ik % STAGES;
                ok = wait(&bars.kv_full[sv], iv / STAGES);
                for (int i = 0; i < nq && ok; ++i) {
                    if (!(ok = wait(&bars.p_full[i], mine[i] + jj))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < kTcKeys / 16; ++ks)
                            mma_ts(tm + 256u + uint32_t(i) * 128u, tm + uint32_t(i) * 128u + uint32_t(ks) * 8u,
                                   dv + uint64_t(sv) * kTile16 + uint64_t(ks) * 128u, kDescO, jj > 0 || ks > 0);
                    }
                    if (i == nq - 1) commit(&bars.kv_empty[sv]);
                    if (jj + 1 < n) {
                        if (i == 0 && !(ok = wait(&bars.kv_full[sk], ik / STAGES))) break;
                        tc_fence_after();
                        issue_s(i, sk);
                        commit(&bars.s_full[i]);
                        if (i == nq - 1) {
                            commit(&bars.kv_empty[sk]);
                            if (jj + 2 == n) commit(&bars.q_empty);  // the last use of Q
                        }
                    } else {
                        commit(&bars.o_full[i]);
                    }
                }
            }
            tiles += n;
            mine[0] += n;
            if (nq == 2) mine[1] += n;
            ++items;
        }
        if (!ok) {
            commit(&bars.drain);
            (void)wait(&bars.drain, 0);
            if (lane == 0) report(p.c.err, kErrTimeout);
        }
    } else if (INT8 && warp == T::kPlanWarp + 1) {
        // ================= INT8: blocks of codes, and their scales =================
        const uint32_t bytes = uint32_t(bs) * D;  // a block's rows of one kv head lie in a row
        int tiles = 0;
        for (int q = 0; ok && take(q); release(q++)) {
            const TcItem& im = s_item[q & 1];
            if (im.kind == 1) continue;
            const KeyTiles kt = im.kt;
            const int n = im.n, k0 = im.k0, kvh = im.kvh, nfull = im.nfull;
            const int32_t* table = p.bt.tables + size_t(im.b) * p.bt.max_blocks;
            const bool slot_ok = im.slot >= 0 && im.slot < p.c.max_slots;
            // lane u: the table's entry for unit u of a tile (looked at one tile later)
            const auto entry = [&](int tile) {
                const int u = tile * U + lane;
                return lane < U && u < kt.n ? table[kt.tile(u)] : -1;
            };
            int next = entry(k0), jj = 0;
            for (; jj < n; ++jj) {
                const int tile = k0 + jj, u = tile * U + lane, slot = (tiles + jj) & 7;
                int id = next;
                next = entry(tile + 1);
                bool miss = lane < U;
                if (lane < U && u < kt.n) {
                    if ((kt.tile(u) << lg) >= nfull) {
                        miss = !slot_ok;
                        if (miss) report(p.c.err, kErrSlot);
                        id = -1;
                    } else {
                        miss = id < 0 || id >= p.c.num_blocks;
                        if (miss) {
                            report(p.c.err, kErrBlockId);
                            id = -1;
                        }
                    }
                } else {
                    id = -1;
                }
                const uint32_t missing = __ballot_sync(kFull, miss);
                const uint32_t total = uint32_t(__popc(__ballot_sync(kFull, id >= 0))) * bytes;
                float2 sc = make_float2(1.f, 1.f);
                if (id >= 0) sc = __ldcg(reinterpret_cast<const float2*>(p.c.scales) + size_t(id) * p.c.Hkv + kvh);
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    if (tiles + jj > 0 && !(ok = wait(&bars.raw_empty[v], tiles + jj - 1))) {
                        if (v) (void)wait(&bars.raw_full[0], tiles + jj);  // (this tile's K is not among `tiles`)
                        break;
                    }
                    if (v == 0) {
                        // K: never 0: a hidden token's score is -infinity, and 0 times that is not
                        // a number. V scales below 2^-60 are taken for zero, by way of zero rows:
                        // 2^-40 and the scale in one exponent leave a weight 26 bits above fp32's
                        // smallest (a block's quantizer gives 1e-6 / 127 at the least).
                        const bool zero = !(sc.y >= 0x1p-60f);
                        const uint32_t zeros = __ballot_sync(kFull, zero);
                        if (lane < U) s_sc[slot][lane] = make_float2(fmaxf(sc.x * p.qscale, 1e-37f), zero ? 0.f : __log2f(sc.y));
                        if (lane == 0) {
                            s_bad[0][slot] = missing;
                            s_bad[INT8][slot] = missing | zeros;
                        }
                    }
                    __syncwarp();
                    const uint32_t full = bar(&bars.raw_full[v]);
                    if (lane == 0) mbar_arrive_expect_tx(full, total);
                    __syncwarp();
                    if (id >= 0)
                        bulk_g2s(raw0 + uint32_t(v) * T::kRawBytes + uint32_t(lane) * bytes,
                                 static_cast<const uint8_t*>(v ? p.c.v_pool : p.c.k_pool) + (size_t(id) * p.c.Hkv + kvh) * bytes,
                                 bytes, full);
                    __syncwarp();
                }
                if (!ok) break;
            }
            tiles += ok ? n : jj;
        }
        if (!ok) {  // let the copies in flight land before the CTA ends
            for (int v = 0; v < 2; ++v)
                if (tiles > 0) (void)wait(&bars.raw_full[v], tiles - 1);
            if (lane == 0) report(p.c.err, kErrTimeout);
        }
    } else if (warp == T::kPlanWarp) {
        // ================= items and queries =================
        const bool leader = elect_one();
        if (leader) prefetch_tensormap(&p.tm_q);
        int cx = blockIdx.x;
        // (row tile, kv head) of all sequences in a list, the row tiles from the last one
        // on: later rows see more keys. The list's last split_items are split. The grid
        // has a CTA for each item that the host's bounds allow; behind the batch's own
        // they have none, and are asked for and dropped.
        const auto row_tiles = [&](int s) {
            const SeqRange r = seq_range(p.bt, s, bs, nullptr, false);
            return int((int64_t(r.n) * G + 2 * kTcRows - 1) / (2 * kTcRows));
        };
        ListCursor<decltype(row_tiles)> list(p.bt.B, row_tiles);
        const int list_tiles = int(list.total < p.item_tiles ? list.total : p.item_tiles);
        const int items = list_tiles * p.c.Hkv, whole = max(0, items - p.split_items);
        if (cx == 0)
            for (int b = lane; b < p.bt.B; b += 32) (void)seq_range(p.bt, b, bs, p.c.err, true);
        int published = 0, loaded = 0, round = 0;
        // The grid's cx-th CTA's item; false: it has none.
        const auto describe = [&](TcItem& x) {
            const bool split = cx >= whole;
            const int at = split ? (cx - whole) / S : 0, j = split ? (cx - whole) % S : 0;
            const int item = split ? whole + at : cx, kvh = item % p.c.Hkv;
            if (item >= items) return false;
            const WorkItem wi = list.find(list_tiles - 1 - item / p.c.Hkv);
            if (wi.b < 0) return false;
            const SeqRange sq = seq_range(p.bt, wi.b, bs, nullptr, false);
            x.kind = sq.bad ? 1 : 0;
            x.b = wi.b;
            x.kvh = kvh;
            x.at = at;
            x.j = j;
            x.row0 = sq.row0;
            x.pos0 = sq.ctx - sq.n;
            x.r_first = wi.i * 2 * kTcRows;
            x.r_end = min(sq.n * G, x.r_first + 2 * kTcRows);
            x.p_first = x.pos0 + (x.r_first >> lgG);
            x.p_last = x.pos0 + ((x.r_end - 1) >> lgG);
            x.kt = key_tiles(max(0, x.p_first), max(0, x.p_last), p.window, p.sinks, bs);
            const int all = (x.kt.n + U - 1) / U;
            int per = all;
            if (split) per = max(p.split_tiles * kTile / kTcKeys, (all + S - 1) / S);
            x.ns = (all + per - 1) / per;
            x.k0 = j * per;
            x.n = min(all, x.k0 + per) - x.k0;
            x.nfull = INT8 ? sq.ctx / bs * bs : sq.ctx;
            x.slot = INT8 ? p.bt.slots[wi.b] : 0;
            return sq.bad ? j == 0 : j < x.ns;
        };
        TcItem x;
        for (;; ++round) {
            if (describe(x)) {
                const int s = published & 1;
                if (published >= 2 && !(ok = wait(&bars.item_empty[s], (published >> 1) - 1))) {
                    if (lane == 0 && x.kind == 0 && x.ns > 1) (void)arrive(x.at, x.ns);
                    break;
                }
                if (lane == 0) {
                    s_item[s] = x;
                    mbar_arrive(bar(&bars.item_full[s]));
                }
                ++published;
                if (x.kind == 0) {
                    if (loaded > 0 && !(ok = wait(&bars.q_empty, loaded - 1))) break;
                    // (the test hook leaves one item of the first CTA without its queries)
                    if (leader && !(blockIdx.x == 0 && loaded == p.skip_copy)) {
                        const int nq = x.r_end - x.r_first > kTcRows ? 2 : 1;
                        mbar_arrive_expect_tx(bar(&bars.q_full), uint32_t(nq) * T::kTileBytes);
                        for (int i = 0; i < nq; ++i)
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_4d(q_addr + i * T::kTileBytes + h * T::kSlab, &p.tm_q, h * 64, 0, x.kvh,
                                            x.row0 + ((x.r_first + i * kTcRows) >> lgG), bar(&bars.q_full));
                    }
                    __syncwarp();
                    ++loaded;
                }
            }
            // ask for the CTA that the grid would start next, an item ahead and no more
            if (leader) {
                fence_proxy_async_smem();  // the answer before has been read
                mbar_arrive_expect_tx(bar(&bars.next), 16);
                next_cta(smem_addr(&s_next), bar(&bars.next));
            }
            __syncwarp();
            // (nobody else will take that CTA's item: its answer is waited for twice as long)
            if (!(ok = wait(&bars.next, round) || wait(&bars.next, round))) break;
            const bool more = next_cta_read(smem_addr(&s_next), cx);
            __syncwarp();
            if (!more) break;
        }
        if (ok) {
            const int s = published & 1;
            if (published >= 2) ok = wait(&bars.item_empty[s], (published >> 1) - 1);
            if (ok && lane == 0) {
                s_item[s].kind = 2;
                mbar_arrive(bar(&bars.item_full[s]));
            }
        }
        if (!ok) {
            // let the copies in flight land before the CTA ends
            if (loaded > 0) (void)wait(&bars.q_full, loaded - 1);
            if (lane == 0) report(p.c.err, kErrTimeout);
        }
        if (lane == 0) s_published = published;
    }

    // bf16: a V tile that was on its way to be cleared lands too, by its barrier's open
    // phase (here, since a second wait in the loaders' code costs prompts 1 to 2%)
    if (!INT8 && warp == 9 && !ok)
        for (uint32_t x = 0; x < 2; ++x) (void)wait(&bars.raw_full[0], x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // After a wait that ran out, the splits that this CTA took and did not finish arrive
    // all the same, so that the counters are back at zero when the call ends (its outputs
    // mean nothing, the next call's do). Described ones that have not arrived are the
    // last two at most: the softmax gives an item back after it has arrived.
    if (tid == 0)
        for (int q = max(s_settled, s_published - 2); q < s_published; ++q) {
            const TcItem& im = s_item[q & 1];
            if (im.kind == 0 && im.ns > 1) (void)arrive(im.at, im.ns);
        }
    if (warp == T::kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool INT8>
constexpr size_t window_tc_smem() { return TcTraits<D, INT8>::kSmem; }

}  // namespace pkv
