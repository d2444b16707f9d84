// Windowed attention for few query rows (decode steps, drafted tokens): one
// CTA per (split, row tile, kv head, sequence), 8 * NT rows a tile.
//
// Bound by memory: every visible K and V byte is read once per kv head. The
// rows of the whole GQA group and of all new tokens are the N dimension of
// mma.m16n8k16 (tokens are M), so further rows cost arithmetic that the loads
// hide, not traffic. Four warps, each with its own ring of 16-token tiles
// filled by the TMA engine, as in the decode kernel, whose tile arithmetic
// (operand runs, f16 codes, power-of-two units of the accumulators) this is
// with NT column tiles and a per-row mask. The mask is applied only to tiles
// that some row does not see whole; tokens that no row of the tile sees count
// as zero rows of V, so what lies behind the context cannot leak in.
//
// Measured, d = 128, 8 kv heads: 16 sequences of 6000 to 8000 tokens with 2 to 6
// new ones and 2 query heads a group, bf16, 453 MB in 77 us, 5.9 TB/s (a plain
// copy: 6.7); 64 sequences, one new token, window 2048, 4 heads a group, INT8,
// 250 MB in 54 us, 4.6 TB/s: four CTAs a SM hold all of it at once (608 places
// for 512 CTAs), so every CTA pays its start -- lengths, block ids, scales, first
// tiles, each load waiting for the one before, about 7 us -- before the stream
// and the merge behind it, and the SMs with three CTAs wait for those with four.
// Splits that even this out cost more in merging than they gain (58 us).
// With 16 rows a tile over INT8 (d = 128) 49 words spill under the 168 registers of
// three CTAs an SM, and issue bounds it: 16 sequences of 7000 tokens 68 us, 34 by bytes.
#pragma once

#include "window.cuh"

namespace pkv {

constexpr int kSegTiles = 256;  // tiles whose block ids and scales are held at a time

template <int D, int NT>
struct RowsState {
    float m[NT][2], md[NT][2], l[NT][2];
    float acc[NT][D / 16][4];
};

// What the columns (rows of the problem) 2t, 2t+1 of each column tile see.
template <int NT>
struct RowsMask {
    int hi[NT][2];  // position; -1: no row
    int lo[NT][2];  // first token of the window
    int sinks;
    int dead_lo, dead_hi;  // tokens in [sinks, dead_lo) and above dead_hi are seen by no row
};

// One 16-token tile at token tok. any: some of it is there. MASKED: some row may
// not see all of it (two copies of the code: most tiles are seen whole, and as a
// condition inside the mask's instructions are issued for them too, predicated
// off). The other arguments are those of mma_tile.
template <int D, bool I8, bool SHIFT, bool HALVES, int NT, bool MASKED, class Rows>
__device__ __forceinline__ void rows_tile(const Rows& K, const Rows& V, int tok, bool any, float ksc, float vmul, float delta, const uint32_t (&qf)[NT][D / 16][2],
                                          const float (&hs)[NT][2], const RowsMask<NT>& mk, int g, int t,
                                          RowsState<D, NT>& st) {
    using Gm = Geom<D, I8>;
    constexpr bool F16 = I8;
    float s[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
    {
        float s2[4] = {0.f, 0.f, 0.f, 0.f};  // NT == 1: a second accumulator chain
        uint32_t k0[Gm::kKW], k1[Gm::kKW];
        const auto kc = [t](int c) { return k_chunk<Gm::kKB, HALVES>(t, c); };
        load_run<Gm::kKB>(K, g, kc, k0);
        load_run<Gm::kKB>(K, g + 8, kc, k1);
#pragma unroll
        for (int ks = 0; ks < Gm::kSteps; ++ks) {
            uint32_t a0, a1, a2, a3;
            if (I8) {
                s8_pairs(k0[ks], a0, a2);
                s8_pairs(k1[ks], a1, a3);
            } else {
                a0 = k0[2 * ks]; a2 = k0[2 * ks + 1];
                a1 = k1[2 * ks]; a3 = k1[2 * ks + 1];
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                if (NT == 1 && (ks & 1)) mma16816<F16>(s2, a0, a1, a2, a3, qf[x][ks][0], qf[x][ks][1]);
                else mma16816<F16>(s[x], a0, a1, a2, a3, qf[x][ks][0], qf[x][ks][1]);
            }
        }
        if (NT == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][i] += s2[i];
        }
    }
    uint32_t b0[NT], b1[NT], b0l[NT], b1l[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const float f0 = ksc * hs[x][0], f1 = ksc * hs[x][1];
        s[x][0] *= f0; s[x][1] *= f1; s[x][2] *= f0; s[x][3] *= f1;
        if (MASKED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tt = tok + g + (i >> 1) * 8;
                const bool see = any && tt <= mk.hi[x][i & 1] && (tt >= mk.lo[x][i & 1] || tt < mk.sinks);
                if (!see) s[x][i] = -INFINITY;
            }
        }
        float mx0 = fmaxf(s[x][0], s[x][2]), mx1 = fmaxf(s[x][1], s[x][3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, off));
        }
        mx0 = fmaxf(mx0, st.m[x][0]);
        mx1 = fmaxf(mx1, st.m[x][1]);
        if (__any_sync(kFull, (mx0 > st.m[x][0]) | (mx1 > st.m[x][1]))) {
            const float c0 = fast_exp2(st.m[x][0] - mx0), c1 = fast_exp2(st.m[x][1] - mx1);
            st.m[x][0] = mx0;
            st.m[x][1] = mx1;
            if (SHIFT) {
                st.md[x][0] = mx0 - delta;
                st.md[x][1] = mx1 - delta;
            }
            st.l[x][0] *= c0;
            st.l[x][1] *= c1;
#pragma unroll
            for (int m = 0; m < Gm::kSteps; ++m) {
                st.acc[x][m][0] *= c0; st.acc[x][m][1] *= c1; st.acc[x][m][2] *= c0; st.acc[x][m][3] *= c1;
            }
        }
        const float r0 = SHIFT ? st.md[x][0] : st.m[x][0], r1 = SHIFT ? st.md[x][1] : st.m[x][1];
        const float p0 = fast_exp2(s[x][0] - r0), p1 = fast_exp2(s[x][1] - r1);
        const float p2 = fast_exp2(s[x][2] - r0), p3 = fast_exp2(s[x][3] - r1);
        st.l[x][0] += p0 + p2;
        st.l[x][1] += p1 + p3;
        const float x0 = p0 * vmul, x1 = p1 * vmul, x2 = p2 * vmul, x3 = p3 * vmul;
        const uint32_t w01 = pack2<F16>(x0, x1), w23 = pack2<F16>(x2, x3);
        b0[x] = movmatrix_t(w01);
        b1[x] = movmatrix_t(w23);
        if (!F16) {  // the weights' rounding residuals, as in the decode kernel
            const float2 h01 = bf16x2_to_f2(w01), h23 = bf16x2_to_f2(w23);
            b0l[x] = movmatrix_t(pack2<false>(x0 - h01.x, x1 - h01.y));
            b1l[x] = movmatrix_t(pack2<false>(x2 - h23.x, x3 - h23.y));
        }
    }
    uint32_t v0[Gm::kVW], v1[Gm::kVW], v2[Gm::kVW], v3[Gm::kVW];
    const auto vc = [g](int c) { return v_chunk<Gm::kVB, HALVES>(g, c); };
    load_run<Gm::kVB>(V, 2 * t, vc, v0);
    load_run<Gm::kVB>(V, 2 * t + 1, vc, v1);
    load_run<Gm::kVB>(V, 2 * t + 8, vc, v2);
    load_run<Gm::kVB>(V, 2 * t + 9, vc, v3);
    if (MASKED) {
        const auto dead = [&](int i) {
            const int tt = tok + i;
            return !any || tt > mk.dead_hi || (tt < mk.dead_lo && tt >= mk.sinks);
        };
        const bool d0 = dead(2 * t), d1 = dead(2 * t + 1), d2 = dead(2 * t + 8), d3 = dead(2 * t + 9);
#pragma unroll
        for (int i = 0; i < Gm::kVW; ++i) {
            if (d0) v0[i] = 0u;
            if (d1) v1[i] = 0u;
            if (d2) v2[i] = 0u;
            if (d3) v3[i] = 0u;
        }
    }
    if (I8) {
#pragma unroll
        for (int j = 0; j < Gm::kVW; ++j) {
            uint32_t r01[4], r23[4];
            s8_interleave(v0[j], v1[j], r01);
            s8_interleave(v2[j], v3[j], r23);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma16816<true>(st.acc[x][2 * j], r01[0], r01[1], r23[0], r23[1], b0[x], b1[x]);
                mma16816<true>(st.acc[x][2 * j + 1], r01[2], r01[3], r23[2], r23[3], b0[x], b1[x]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < Gm::kVW; ++j) {
            const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632);
            const uint32_t a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma16816<false>(st.acc[x][j], a0, a1, a2, a3, b0[x], b1[x]);
                mma16816<false>(st.acc[x][j], a0, a1, a2, a3, b0l[x], b1l[x]);
            }
        }
    }
}

// HOOK: the test build of pkv_debug_skip_copy, which leaves one tile's copies unissued.
template <int D, bool INT8, int NT, bool HOOK>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kMinCtas : 3)
window_rows_kernel(const __grid_constant__ WindowParams p) {
    using T = DecodeTraits<D, INT8>;
    using Gm = Geom<D, INT8>;
    constexpr int STAGES = T::kStages;
    constexpr bool HALVES = T::kHalves;
    constexpr int R = 8 * NT;  // rows a tile
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t s_id[kSegTiles];
    __shared__ float2 s_sc[INT8 ? kSegTiles : 1];
    __shared__ float s_ml[kWarps][R][2];
    __shared__ int s_ev[kWarps];
    __shared__ __align__(8) uint64_t s_bar[kWarps * STAGES];
    __shared__ int s_last;
    static_assert(R * D * 4 <= STAGES * T::kStageBytes, "a warp's output tile fits its ring");

    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int j = int(blockIdx.x) % p.max_splits, rt = int(blockIdx.x) / p.max_splits;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.c.Hq / p.c.Hkv, lgG = 31 - __clz(G), bs = p.c.bs, lg = bs == 16 ? 4 : 6;
    const SeqRange sq = seq_range(p.bt, b, bs, p.c.err, tid == 0 && blockIdx.x == 0 && kvh == 0);
    const int r_first = rt * R, r_end = min(sq.n * G, r_first + R);
    if (r_first >= r_end) return;
    // output element e (row e / D of the tile, dim e % D)
    auto out_at = [&](int e) {
        const int r = r_first + e / D;
        return p.out + int64_t(sq.row0 + (r >> lgG)) * p.out_stride + (kvh * G + (r & (G - 1))) * D + e % D;
    };
    const int nrow = r_end - r_first;
    if (sq.bad) {
        if (j == 0)
            for (int e = tid; e < nrow * D; e += kThreads) *out_at(e) = 0;
        return;
    }
    const int pos0 = sq.ctx - sq.n;
    const int p_first = pos0 + (r_first >> lgG), p_last = pos0 + ((r_end - 1) >> lgG);
    const KeyTiles kt = key_tiles(p_first, p_last, p.window, p.sinks, kTile);
    int per = kt.n;
    if (p.split_tiles > 0) per = max(p.split_tiles, (kt.n + p.max_splits - 1) / p.max_splits);
    const int ns = (kt.n + per - 1) / per;
    if (j >= ns) return;
    const int k0 = j * per, k1 = min(kt.n, k0 + per);
    const int nfull = INT8 ? (sq.ctx >> lg) << lg : sq.ctx;
    // tiles of the list that lie in the pool come first, those of the tail last
    const int fullt = nfull / kTile;
    const int kpool = !INT8 ? k1 : min(k1, max(k0, fullt < kt.nsink ? fullt : kt.nsink + max(0, fullt - kt.lo)));
    const int slot = INT8 ? p.bt.slots[b] : 0;
    const int32_t* table = p.bt.tables + size_t(b) * p.bt.max_blocks;

    uint8_t* stages = smem + (T::kSwz ? (1024u - (smem_addr(smem) & 1023u)) & 1023u : 0u);
    const uint32_t bar0 = smem_addr(s_bar), stage0 = smem_addr(stages);
    auto bar_of = [&](int s) { return bar0 + uint32_t(warp * STAGES + s) * 8u; };
    auto stage_of = [&](int s) { return stage0 + uint32_t(warp * STAGES + s) * T::kStageBytes; };
    if (lane == 0)
        for (int s = 0; s < STAGES; ++s) mbar_init(bar_of(s), 1);
    fence_mbar_init();
    if (T::kSwz && tid == 0) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
    }

    // ---- this lane's rows
    uint32_t qw[NT][D / 8];
    RowsMask<NT> mk;
    mk.sinks = p.sinks;
    mk.dead_hi = p_last;
    mk.dead_lo = max(0, p_first - p.window + 1);
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const int r = r_first + x * 8 + g;
        const bool have = r < r_end;
        const uint16_t* qrow = p.q + int64_t(sq.row0 + (have ? (r >> lgG) : 0)) * p.q_stride + (kvh * G + (have ? (r & (G - 1)) : 0)) * D;
        load_q_words<D, 8, HALVES>(qrow, have ? g : 8, t, qw[x]);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int rr = r_first + x * 8 + 2 * t + jj;
            mk.hi[x][jj] = rr < r_end ? pos0 + (rr >> lgG) : -1;
            mk.lo[x][jj] = max(0, mk.hi[x][jj] - p.window + 1);
        }
    }

    RowsState<D, NT> st;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        st.m[x][0] = st.m[x][1] = st.md[x][0] = st.md[x][1] = -1e30f;
        st.l[x][0] = st.l[x][1] = 0.f;
#pragma unroll
        for (int m = 0; m < D / 16; ++m) st.acc[x][m][0] = st.acc[x][m][1] = st.acc[x][m][2] = st.acc[x][m][3] = 0.f;
    }
    auto is_masked = [&](int tok) {
        return tok + kTile - 1 > p_first || !(tok >= p_last - p.window + 1 || tok + kTile <= p.sinks);
    };
    const uint64_t pol = l2_policy_evict_first();
    auto issue = [&](int k, int seg, int s) {
        if (HOOK && k - k0 == p.skip_copy && warp == 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0) return;
        const int tok = kt.tile(k) * kTile;
        const int id = s_id[k - seg];
        const uint32_t bar = bar_of(s);
        if (id < 0) {
            mbar_arrive(bar);
            return;
        }
        mbar_arrive_expect_tx(bar, T::kStageBytes);
        if constexpr (T::kSwz) {
            const int y = kvh * bs + (tok & (bs - 1));
#pragma unroll
            for (int h = 0; h < T::kRowBytes / 128; ++h) {
                tma_load_3d(stage_of(s) + h * 2048, &p.tm_k, h * 128, y, id, bar, pol);
                tma_load_3d(stage_of(s) + T::kTileBytes + h * 2048, &p.tm_v, h * 128, y, id, bar, pol);
            }
        } else {
            const size_t row = (size_t(id) * p.c.Hkv + kvh) * bs + (tok & (bs - 1));
            bulk_g2s(stage_of(s), static_cast<const uint8_t*>(p.c.k_pool) + row * T::kRowBytes, T::kTileBytes, bar, pol);
            bulk_g2s(stage_of(s) + T::kTileBytes, static_cast<const uint8_t*>(p.c.v_pool) + row * T::kRowBytes,
                     T::kTileBytes, bar, pol);
        }
    };
    // exponent of a V scale, as in the decode kernel
    auto v_exp = [](float v) {
        const uint32_t u = __float_as_uint(v);
        return u ? min(121, max(-40, int((u >> 23) & 0xFFu) - 127)) : kExpNone;
    };

    uint32_t qf[NT][D / 16][2];
    float hs[NT][2];
    int kk = 0;  // tiles this warp has consumed
    bool timed_out = false;
    int ew = kExpNone;  // INT8: the accumulators' units are 2^(ew - 14); none yet: plain
    for (int seg = k0;; seg += kSegTiles) {
        const int seg_end = min(kpool, seg + kSegTiles);
        if (seg > k0) __syncthreads();  // the last segment's ids are no longer read
        // ids first, so that the copies start without waiting for the scales
        for (int k = seg + tid; k < seg_end; k += kThreads) {
            int id = table[(kt.tile(k) * kTile) >> lg];
            if (id < 0 || id >= p.c.num_blocks) {
                report(p.c.err, kErrBlockId);
                id = -1;
            }
            s_id[k - seg] = id;
        }
        __syncthreads();
        if (lane == 0)
            for (int s = 0; s < STAGES; ++s) {
                const int k = seg + warp + s * kWarps;
                if (k < seg_end) issue(k, seg, (kk + s) % STAGES);
            }
        // the scales' loads fly while the tail is worked on
        static_assert(kSegTiles == 2 * kThreads, "two scales a thread");
        float2 sc[2];
        if (INT8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // (a block that is not there: block 0's, dropped when they are used)
                const int k = seg + tid + u * kThreads, id = k < seg_end ? max(0, s_id[k - seg]) : 0;
                sc[u] = __ldcg(reinterpret_cast<const float2*>(p.c.scales) + size_t(id) * p.c.Hkv + kvh);
            }
        }
        if (seg == k0) {
            // ---- INT8: the partly filled last block, from the slot's bf16 tail, in
            // plain units, while the ring's first copies fly
            if (INT8 && k1 > kpool) {
                const bool ok = slot >= 0 && slot < p.c.max_slots;
                if (!ok && tid == 0) report(p.c.err, kErrSlot);
                const int k = kpool + kWarps - 1 - warp;  // at most bs / 16 <= kWarps tail tiles
                if (ok && k < k1) {
                    uint32_t qb[NT][D / 16][2];
                    float hb[NT][2];
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        (void)q_frags<D, false>(qw[x], qb[x]);
                        hb[x][0] = hb[x][1] = p.qscale;
                    }
                    const int tok = kt.tile(k) * kTile;
                    const size_t rbase = (size_t(slot) * p.c.Hkv + kvh) * bs + (tok - nfull);
                    const GmemRows kr{reinterpret_cast<const uint8_t*>(p.c.k_tail + rbase * D), D * 2};
                    const GmemRows vr{reinterpret_cast<const uint8_t*>(p.c.v_tail + rbase * D), D * 2};
                    rows_tile<D, false, INT8, false, NT, true>(kr, vr, tok, true, 1.f, 1.f, 0.f, qb, hb, mk,
                                                         g, t, st);
                }
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const int qe = q_frags<D, INT8>(qw[x], qf[x]);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int eh = __shfl_sync(kFull, qe, ((2 * t + jj) & 7) * 4);
                    hs[x][jj] = p.qscale * ldexpf(1.0f, -eh);
                }
            }
        }
        float delta = 0.f;
        if (INT8) {
            int ev = kExpNone;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = seg + tid + u * kThreads;
                if (k < seg_end) {
                    if (s_id[k - seg] < 0) sc[u] = make_float2(0.f, 0.f);
                    s_sc[k - seg] = sc[u];
                    ev = max(ev, v_exp(sc[u].y));
                }
            }
            ev = __reduce_max_sync(kFull, ev);
            if (lane == 0) s_ev[warp] = ev;
            __syncthreads();  // the scales
            int e = ew;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) e = max(e, s_ev[w]);
            const int from = ew == kExpNone ? 14 : ew, to = e == kExpNone ? 14 : e;
            ew = e;
            delta = float(14 - to);
            // the state's units follow (a state far below the new unit flushes to zero)
            const float f = exp2i(min(127, max(-126, from - to)));
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                st.md[x][0] = st.m[x][0] - delta;
                st.md[x][1] = st.m[x][1] - delta;
                if (from != to) {
                    st.l[x][0] *= f;
                    st.l[x][1] *= f;
#pragma unroll
                    for (int m = 0; m < D / 16; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) st.acc[x][m][i] *= f;
                }
            }
        }
        for (int k = seg + warp; k < seg_end; k += kWarps, ++kk) {
            const int s = kk % STAGES;
            if (!wait_phase(bar_of(s), uint32_t(kk / STAGES) & 1u)) {
                // drain this warp's copies in flight (each wait again bounded)
                if (lane == 0) report(p.c.err, kErrTimeout);
                timed_out = true;
                for (int q = 0; q < STAGES && k + q * kWarps < seg_end; ++q)
                    (void)wait_phase(bar_of((kk + q) % STAGES), uint32_t((kk + q) / STAGES) & 1u);
                break;
            }
            const int tok = kt.tile(k) * kTile;
            const bool any = s_id[k - seg] >= 0;
            const bool masked = !any || is_masked(tok);
            float ksc = 1.f, vmul = 1.f;
            if (INT8) {
                const float2 sc = s_sc[k - seg];
                ksc = sc.x;
                vmul = sc.y;
            }
            if constexpr (T::kSwz) {
                const SwzRows kr{stage_of(s)}, vr{stage_of(s) + T::kTileBytes};
                if (masked) rows_tile<D, INT8, INT8, HALVES, NT, true>(kr, vr, tok, any, ksc, vmul, delta, qf, hs, mk, g, t, st);
                else rows_tile<D, INT8, INT8, HALVES, NT, false>(kr, vr, tok, any, ksc, vmul, delta, qf, hs, mk, g, t, st);
            } else {
                const SmemRows kr{stage_of(s), Gm::kRow}, vr{stage_of(s) + T::kTileBytes, Gm::kRow};
                if (masked) rows_tile<D, INT8, INT8, false, NT, true>(kr, vr, tok, any, ksc, vmul, delta, qf, hs, mk, g, t, st);
                else rows_tile<D, INT8, INT8, false, NT, false>(kr, vr, tok, any, ksc, vmul, delta, qf, hs, mk, g, t, st);
            }
            __syncwarp();
            const int nxt = k + STAGES * kWarps;
            if (lane == 0 && nxt < seg_end) {
                fence_proxy_async_smem();
                issue(nxt, seg, s);
            }
        }
        if (__syncthreads_or(timed_out) || seg_end >= kpool) break;
        // the next segment's first copies overwrite stages that were just read
        fence_proxy_async_smem();
    }

    // ---- merge the warps (plain units) and write
    const float units = INT8 && ew != kExpNone ? exp2i(ew - 14) : 1.f;
    float* mo = reinterpret_cast<float*>(stages + size_t(warp) * STAGES * T::kStageBytes);
    auto mo_of = [&](int w) { return reinterpret_cast<const float*>(stages + size_t(w) * STAGES * T::kStageBytes); };
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            st.l[x][0] += __shfl_xor_sync(kFull, st.l[x][0], off);
            st.l[x][1] += __shfl_xor_sync(kFull, st.l[x][1], off);
        }
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int r = x * 8 + 2 * t + jj;
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                const int d0 = HALVES ? (m >> 2) * (D / 2) + g * 8 + 2 * (m & 3) : g * (D / 8) + 2 * m;
                mo[r * D + d0] = st.acc[x][m][jj] * units;
                mo[r * D + d0 + 1] = st.acc[x][m][2 + jj] * units;
            }
            if (g == 0) {
                s_ml[warp][r][0] = st.m[x][jj];
                s_ml[warp][r][1] = st.l[x][jj] * units;
            }
        }
    }
    __syncthreads();
    // the warps' factors of each row, over its sum unless partial
    const bool partial = ns > 1;
    auto row_at = [&](int r) {  // of row r of the tile: its number among all rows and heads
        const int rr = r_first + r;
        return size_t(sq.row0 + (rr >> lgG)) * p.c.Hq + kvh * G + (rr & (G - 1));
    };
    if (tid < nrow) {
        float mm = -1e30f, L = 0.f, c[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][tid][0]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            c[w] = fast_exp2(s_ml[w][tid][0] - mm);
            L += s_ml[w][tid][1] * c[w];
        }
        const float f = partial ? 1.f : L > 0.f ? 1.f / L : 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_ml[w][tid][0] = c[w] * f;
        if (partial) reinterpret_cast<float2*>(p.ws_ml)[row_at(tid) * p.max_splits + j] = make_float2(mm, L);
    }
    __syncthreads();
    for (int e = tid * 4; e < nrow * D; e += kThreads * 4) {
        const int r = e / D, dim = e % D;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(mo_of(w) + e);
            const float c = s_ml[w][r][0];
            o.x += x.x * c; o.y += x.y * c; o.z += x.z * c; o.w += x.w * c;
        }
        if (partial)
            *reinterpret_cast<float4*>(p.ws_o + (row_at(r) * p.max_splits + j) * D + dim) = o;
        else
            *reinterpret_cast<uint2*>(out_at(e)) = make_uint2(f2_to_bf16x2(o.x, o.y), f2_to_bf16x2(o.z, o.w));
    }
    if (!partial) return;

    // ---- the last split of the row tile to arrive merges all of them
    int32_t* cnt = p.ws_count + (size_t(b) * p.c.Hkv + kvh) * p.row_tiles + rt;
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel_gpu(cnt, 1) == ns - 1;
    __syncthreads();
    if (!s_last) return;
    float* wsm = reinterpret_cast<float*>(stages);  // [rows][ns] weights, over the row's sum
    static_assert(R * 8 <= kThreads, "eight threads a row");
    {
        const int r = tid >> 3, sub = tid & 7;
        const bool have = r < nrow;
        const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row_at(have ? r : 0) * p.max_splits;
        float mm = -1e30f, L = 0.f;
        for (int q = sub; q < ns; q += 8) mm = fmaxf(mm, __ldcg(ml + q).x);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(kFull, mm, off));
        for (int q = sub; q < ns; q += 8) {
            const float2 v = __ldcg(ml + q);
            const float c = fast_exp2(v.x - mm);
            if (have) wsm[r * ns + q] = c;
            L += c * v.y;
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) L += __shfl_xor_sync(kFull, L, off);
        if (have && sub == 0) s_ml[0][r][0] = L > 0.f ? 1.f / L : 0.f;
    }
    __syncthreads();
    for (int e = tid * 4; e < nrow * D; e += kThreads * 4) {
        const int r = e / D, dim = e % D;
        const float* o = p.ws_o + row_at(r) * p.max_splits * D + dim;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = 0; q < ns; ++q) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(o + size_t(q) * D));
            const float c = wsm[r * ns + q];
            acc.x += x.x * c; acc.y += x.y * c; acc.z += x.z * c; acc.w += x.w * c;
        }
        const float f = s_ml[0][r][0];
        *reinterpret_cast<uint2*>(out_at(e)) = make_uint2(f2_to_bf16x2(acc.x * f, acc.y * f), f2_to_bf16x2(acc.z * f, acc.w * f));
    }
    if (tid == 0) *cnt = 0;  // ready for the next call
}

template <int D, bool INT8>
WindowFn window_rows_pick(int nt, bool hook) {
    if constexpr (D == 64) {
        if (hook) return nt == 1 ? window_rows_kernel<D, INT8, 1, true> : nullptr;
    }
    if (hook) return nullptr;
    return nt == 1 ? window_rows_kernel<D, INT8, 1, false> : window_rows_kernel<D, INT8, 2, false>;
}

}  // namespace pkv
