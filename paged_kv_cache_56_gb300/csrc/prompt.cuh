// Attention of whole prompts from their rows (pkv_prompt_attention), on the tensor
// cores of sm_103a (tcgen05, accumulators in tensor memory).
//
// A work item is (256 rows, kv head, sequence), a row a (token, query head of the
// group), so that a kv head's whole group shares each K and V tile. Two CTAs, a
// cluster, have 128 of the rows each and multiply as one (cta_group::2, M = 256):
// of a tile of 128 keys each loads half -- 64 rows of K, half of V's columns.
// There is one pair for each two SMs; it walks from item to item, taking the grid's
// next one from the hardware (launch cancellation). Long items are first in the grid.
//
//   warps 0-7: softmax; warps w and w + 4 have the same 32 rows, a row a thread
//              each, and take the key tiles in turn; scores from tensor memory, weights back
//   warp 8     the loader of Q, K and V
//   warp 9     items               } of the first
//   warp 10    issues S = Q K^T    } CTA, for both
//   warp 11    issues O += P V     }
//
//   S = Q K^T   256 x 128 x D, operands in shared memory
//   O += P V    256 x D x 128, P in tensor memory over the scores it came from
// Tensor memory holds O and three S: the scores of the next two tiles are worked
// out while the softmax has this one, so that neither waits for the other's
// latency, and the next item's first scores come during the end of the one before.
//
// The reference of a row's exponents is its first visible tile's maximum. It follows
// only when a tile's weights sum to more than 2^13: their sum, which is needed anyway,
// shows it, so that no maximum is taken after the first tile. Then (rarely) the
// tile's maximum becomes the reference and O is rescaled. The two warps of a row have one
// reference: a tile is weighed ahead against the last one known, and again if the tile
// before, the other warp's, turns out to have raised it. Weights are kept
// in units of 2^-40 (an exponent bias, free) and rounded to bf16 for the multiply
// (2^-8 of each weight, as the outputs are); their sum is fp32.
#pragma once

#include "ptx_tc.cuh"
#include "window.cuh"

namespace pkv {

constexpr int kPrRows = 128;  // rows of a CTA
constexpr int kPrKeys = 128;  // tokens of a key tile
constexpr int kPrScores = 3;  // tiles of scores in tensor memory
constexpr float kPrShift = 40.f;
constexpr float kPrMost = 0x1p-27f;  // 2^13 in units of 2^-40
constexpr int kPrThreads = 384;
constexpr int kPrLaunchRegs = 168;

struct PromptParams {
    CUtensorMap tm_q;    // q as [tokens][Hkv][G][D], boxes of 128 rows x 64 elements
    CUtensorMap tm_k;    // k as [tokens][Hkv][1][D], boxes of 64 rows x 64 elements
    CUtensorMap tm_v;    // v likewise, boxes of 128 rows x D / 2 elements
    CUtensorMap tm_out;  // out as q, boxes of 32 rows x 64 elements
    BatchView bt;
    uint16_t* out;
    int64_t out_stride;
    int32_t* err;
    int32_t Hq, Hkv;
    int32_t window;      // INT32_MAX: none
    int32_t sinks;
    int32_t item_tiles;  // row tiles (of 256) that the batch can have
    float qscale;        // sm_scale * log2(e)
};

template <int D>
struct PromptTraits {
    static constexpr int kQBytes = kPrRows * D * 2;     // a CTA's rows of Q
    static constexpr int kTileBytes = kPrKeys * D;      // a CTA's half of a K or V tile
    static constexpr int kStages = D == 64 ? 6 : 4;     // of K, and of V
    static constexpr int kOutBytes = 32 * D;            // a softmax warp's rows on their way out
    static constexpr int kData = 2 * kQBytes + 2 * kStages * kTileBytes + 8 * kOutBytes;
    static constexpr int kSmem = kData + 3072;          // and PromptShared
    static constexpr int kSoftmaxRegs = 200, kRestRegs = 104;
    static_assert(256 * kSoftmaxRegs + 128 * kRestRegs == kPrThreads * kPrLaunchRegs, "register split");
};

// Barriers, at the same places in both CTAs. Those marked 0 are used in the first CTA only.
template <int STAGES>
struct PromptBars {
    uint64_t q_full[2], q_empty[2];  // full: 0
    uint64_t k_full[STAGES], k_empty[STAGES];
    uint64_t v_full[STAGES], v_empty[STAGES];
    uint64_t fix;                    // a V tile whose dead rows have to be cleared first
    uint64_t s_full[kPrScores];      // scores are there
    uint64_t p_full[kPrScores];      // 0: weights are there, O corrected, in both CTAs
    uint64_t pv_done[kPrScores];     // O += P V of the weights there is done
    uint64_t o_full;                 // O is complete
    uint64_t item_full[2];           // an item's description is there
    uint64_t item_empty[2];          // 0: every warp of both CTAs has taken it
    uint64_t settled[4][4];          // warps w, w + 4: a tile's references are settled (tiles in turn)
    uint64_t sum_there[4];           // ... the sums of the one are there for the other
    uint64_t o_read[4];              // ... O has been read
    uint64_t mail[2];                // (second CTA) an item's description has come
    uint64_t next;                   // 0: the answer about the next item is there
    uint64_t drain[2];
};

struct PromptItem {
    int kind;  // 0: attention; 1: rows of a sequence with earlier tokens, zero; 2: the end
    int kvh, row0, n;    // kv head; the sequence's first row, its rows (tokens)
    int r_first, r_end;  // of the pair
    KeyTiles kt;
};

template <int STAGES>
struct alignas(16) PromptShared {
    PromptBars<STAGES> bars;
    PromptItem item[2];
    uint4 next;
    float ref[2][kPrRows];  // the rows' references, as the last tile that raised them left them (items in turn)
    int raised[2][4];       // that tile, of each 32 rows
    float2 sum[kPrRows];    // the rows' sums over the tiles of the warp that has not the item's last one, and their reference
    uint32_t tmem;
};

template <bool V>
struct PromptConst {
    static constexpr bool value = V;
};

// wait_phase for barriers on which the other CTA arrives.
__device__ __forceinline__ bool wait_phase_cluster(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait_cluster(bar, parity, 0u)) return true;
    uint64_t t0;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (;;) {
        if (mbar_try_wait_cluster(bar, parity, 2000u)) return true;
        uint64_t t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > 1000000000ull) return false;
    }
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrThreads, 1)
prompt_kernel(const __grid_constant__ PromptParams p) {
    using T = PromptTraits<D>;
    constexpr int STAGES = T::kStages, kLoadWarp = 8, kPlanWarp = 9, kScoreWarp = 10, kValueWarp = 11;
    extern __shared__ __align__(1024) uint8_t smem_1024[];  // (aligned as the swizzles need it)
    static_assert(sizeof(PromptShared<STAGES>) <= size_t(T::kSmem - T::kData), "shared memory");
    PromptShared<STAGES>& sh = *reinterpret_cast<PromptShared<STAGES>*>(smem_1024 + T::kData);
    PromptBars<STAGES>& bars = sh.bars;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int G = p.Hq / p.Hkv, lgG = 31 - __clz(G);
    const uint32_t q_addr = smem_addr(smem_1024), k_addr = q_addr + 2 * T::kQBytes, v_addr = k_addr + STAGES * T::kTileBytes;
    const uint32_t out0 = v_addr + STAGES * T::kTileBytes;
    const uint32_t bar0 = smem_addr(&bars);
    const auto bar = [&](const uint64_t* x) {
        return bar0 + uint32_t(reinterpret_cast<const uint8_t*>(x) - reinterpret_cast<const uint8_t*>(&bars));
    };
    // the same barrier of the first CTA, for arrivals
    const uint32_t lead0 = cluster_addr(bar0, 0);
    const auto lead = [&](const uint64_t* x) { return bar(x) - bar0 + lead0; };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(&bars.q_full[i]), 2);
            mbar_init(bar(&bars.q_empty[i]), 1);
            mbar_init(bar(&bars.item_full[i]), 1);
            mbar_init(bar(&bars.item_empty[i]), 2 * (8 + 1) + 2);
            mbar_init(bar(&bars.drain[i]), 1);
            mbar_init(bar(&bars.mail[i]), 1);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(&bars.k_full[s]), 2);
            mbar_init(bar(&bars.k_empty[s]), 1);
            mbar_init(bar(&bars.v_full[s]), 2);
            mbar_init(bar(&bars.v_empty[s]), 1);
        }
        for (int i = 0; i < kPrScores; ++i) {
            mbar_init(bar(&bars.s_full[i]), 1);
            mbar_init(bar(&bars.pv_done[i]), 1);
            mbar_init(bar(&bars.p_full[i]), 8);
        }
        for (int i = 0; i < 4; ++i) {
            for (int t = 0; t < 4; ++t) mbar_init(bar(&bars.settled[i][t]), 1);
            mbar_init(bar(&bars.sum_there[i]), 1);
            mbar_init(bar(&bars.o_read[i]), 1);
            sh.raised[0][i] = sh.raised[1][i] = -1;
        }
        mbar_init(bar(&bars.fix), 1);
        mbar_init(bar(&bars.o_full), 1);
        mbar_init(bar(&bars.next), 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == kScoreWarp) tmem_alloc_pair(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are there, too
    tc_fence_after();
    const uint32_t tmem = sh.tmem, tm_s = tmem + 128u;  // O, then the tiles of scores
    // Waits for a phase, a whole warp, which it leaves converged. After about a
    // second without it a role gives up, and so, one after the other, do those
    // that wait for it. (Every copy has landed long before that.)
    const auto wait = [&](const uint64_t* x, uint32_t parity) {
        return __all_sync(kFull, wait_phase(bar(x), parity & 1u)) != 0;
    };
    pdl_wait();
    pdl_launch_dependents();

    bool ok = true;
    // The q-th item of this pair (every warp but the planner's): false at the end.
    const auto take = [&](int q) {
        ok = wait(&bars.item_full[q & 1], q >> 1);
        return ok && sh.item[q & 1].kind != 2;
    };
    // Its description is no longer needed.
    const auto release = [&](int q) {
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(lead(&bars.item_empty[q & 1]));
    };

    if (warp < 8) reg_inc<T::kSoftmaxRegs>();
    else reg_dec<T::kRestRegs>();

    if (warp < 8) {
        // ================= softmax: 32 rows of every second tile =================
        const int quad = warp & 3, team = warp >> 2, mine = quad * 32 + lane;
        const uint32_t lane_base = uint32_t(quad * 32) << 16, o_addr = tmem + lane_base;
        const float scale = p.qscale;
        int g = 0, items = 0, full = 0;  // tiles and items so far; items that have rows of this warp
        bool unread = false;             // the other warp may still be reading O of the last one
        for (int q = 0; take(q); release(q++)) {
            const PromptItem& im = sh.item[q & 1];
            const int first = im.r_first + int(rank) * kPrRows + quad * 32;  // of this warp
            const int rows = min(32, im.r_end - first);                      // (none: <= 0)
            const bool have = lane < rows;
            const int kvh = im.kvh, row0 = im.row0;
            if (im.kind == 1) {
                for (int e = lane; e < rows * (D / 2); e += 32) {
                    const int r = first + e / (D / 2);
                    p.out[int64_t(row0 + (r >> lgG)) * p.out_stride + (kvh * G + (r & (G - 1))) * D + team * (D / 2) + e % (D / 2)] = 0;
                }
                continue;
            }
            const KeyTiles kt = im.kt;
            const int n = kt.n;
            const int hi = have ? (first + lane) >> lgG : -1, lo = max(0, hi - p.window + 1);
            const int pf = first >> lgG, pl = (first + rows - 1) >> lgG;  // the warp's first and last position
            float m_ref = have ? -INFINITY : INFINITY;  // reference of the exponent (base 2); no row: weights of 0
            float2 l2 = make_float2(0.f, 0.f);          // sum of this thread's tiles
            float* const ref = sh.ref[items & 1];
            volatile int* const raised = &sh.raised[items & 1][quad];
            // Tile g's reference is settled: the other warp's next tile may be weighed against it.
            const auto settle = [&](int tile) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(&bars.settled[quad][tile & 3]));
            };
            // The reference that the tile before left (`raised` by the other warp).
            const auto follow = [&](int tile) {
                if (!(ok = wait(&bars.settled[quad][tile & 3], tile >> 2))) return false;
                if (*raised != tile) return false;
                const float to = ref[mine], f = to > m_ref ? fast_exp2(m_ref - to) : 1.f;
                m_ref = to;
                l2.x *= f;
                l2.y *= f;
                return true;
            };
            for (int jj = 0; jj < n; ++jj, ++g) {
                if ((g & 1) != team) continue;
                const int b = g % kPrScores;
                if (!(ok = wait(&bars.s_full[b], g / kPrScores))) break;
                tc_fence_after();
                if (rows > 0) {
                    const uint32_t s_addr = tm_s + uint32_t(b) * 128u + lane_base;
                    const int t0 = kt.tile(jj) * kPrKeys;
                    const bool masked = jj < kt.nsink || t0 + kPrKeys - 1 > pf || t0 < pl - p.window + 1;
                    // Hidden ones of 16 scores from column c on become -infinity; true: all 32 rows' are hidden.
                    const auto hide = [&](uint32_t (&r)[16], int c) {
                        const int tc = t0 + c;
                        // bit e: this row sees token tc + e
                        const auto below = [](int x) { return (1u << min(16, max(0, x))) - 1u; };
                        const uint32_t see = below(hi - tc + 1) & (below(p.sinks - tc) | ~below(lo - tc));
                        if (__all_sync(kFull, (see & 0xFFFFu) == 0u)) return true;
                        if (!__all_sync(kFull, (see & 0xFFFFu) == 0xFFFFu)) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (!((see >> e) & 1u)) r[e] = 0xFF800000u;
                        }
                        return false;
                    };
                    // 16 scores to weights and their sum.
                    const auto weights = [&](const uint32_t (&r)[16], uint32_t* to, float neg) {
                        const float2 a2 = make_float2(scale, scale), b2 = make_float2(neg, neg);
                        float2 part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float2 x0 = make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                            float2 x1 = make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
                            x0 = __ffma2_rn(x0, a2, b2);
                            x1 = __ffma2_rn(x1, a2, b2);
                            x0 = make_float2(fast_exp2(x0.x), fast_exp2(x0.y));
                            x1 = make_float2(fast_exp2(x1.x), fast_exp2(x1.y));
                            part = __fadd2_rn(part, __fadd2_rn(x0, x1));
                            to[e / 2] = f2_to_bf16x2(x0.x, x0.y);
                            to[e / 2 + 1] = f2_to_bf16x2(x1.x, x1.y);
                        }
                        return part;
                    };
                    float2 sum = make_float2(0.f, 0.f);
                    // Weighed ahead of the tile before, against the reference as it is known; again where
                    // that tile, or this one's sum, asks for another one.
                    bool anew = jj == 0, ahead = true;
                    if (jj > 0 && __any_sync(kFull, m_ref == -INFINITY)) {  // (not without any)
                        (void)follow(g - 1);
                        anew = __any_sync(kFull, m_ref == -INFINITY);
                        ahead = false;
                    }
                    if (!ok) break;
                    if (!anew) {
                        // 16 columns at a time, one chunk's load in flight while the other is worked on
                        uint32_t w[2][32];
                        const auto weigh = [&](auto hidden) {
                            const float neg = -m_ref - kPrShift;
                            const auto chunk = [&](uint32_t (&r)[16], uint32_t* to, int c) {
                                if constexpr (hidden.value) {
                                    if (hide(r, c)) {
#pragma unroll
                                        for (int e = 0; e < 8; ++e) to[e] = 0u;
                                        return;
                                    }
                                }
                                sum = __fadd2_rn(sum, weights(r, to, neg));
                            };
                            uint32_t ra[16], rb[16];
                            tmem_ld_start(ra, s_addr);
#pragma unroll
                            for (int c = 0; c < 128; c += 32) {
                                tmem_ld_wait(ra);
                                tmem_ld_start(rb, s_addr + uint32_t(c + 16));
                                chunk(ra, w[c / 64] + c % 64 / 2, c);
                                tmem_ld_wait(rb);
                                if (c < 96) tmem_ld_start(ra, s_addr + uint32_t(c + 32));
                                chunk(rb, w[c / 64] + c % 64 / 2 + 8, c + 16);
                            }
                        };
                        if (masked) weigh(PromptConst<true>{});
                        else weigh(PromptConst<false>{});
                        anew = (ahead && follow(g - 1)) || __any_sync(kFull, sum.x + sum.y > kPrMost);
                        if (!ok) break;
                        if (!anew) {
                            settle(g);
                            tmem_st(s_addr, w[0]);
                            tmem_st(s_addr + 32u, w[1]);
                        }
                    }
                    if (anew) {
                        // The tile's maximum becomes the reference where it is larger; O follows.
                        // (Rolled up: code that runs once an item is fetched anew each time.)
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 128; c += 16) {
                            uint32_t r[16];
                            tmem_ld_start(r, s_addr + uint32_t(c));
                            tmem_ld_wait(r);
                            if (masked && hide(r, c)) continue;
#pragma unroll
                            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, __uint_as_float(r[e]));
                        }
                        const float to = fmaxf(m_ref, mx * scale), f = to > m_ref ? fast_exp2(m_ref - to) : 1.f;
                        m_ref = ref[mine] = to;
                        l2.x *= f;
                        l2.y *= f;
                        if (lane == 0) *raised = g;
                        if (jj > 0 && __any_sync(kFull, f != 1.f)) {
                            if (!(ok = wait(&bars.pv_done[(g - 1) % kPrScores], (g - 1) / kPrScores))) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld_start(o, o_addr + uint32_t(c));
                                tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st(o_addr + uint32_t(c), o);
                            }
                        }
                        settle(g);
                        // weights over scores that have been read
                        const float neg = (m_ref == -INFINITY ? 0.f : -m_ref) - kPrShift;
                        sum = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int c = 0; c < 128; c += 16) {
                            uint32_t r[16], x[8];
                            tmem_ld_start(r, s_addr + uint32_t(c));
                            tmem_ld_wait(r);
                            if (masked && hide(r, c)) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) x[e] = 0u;
                            } else {
                                sum = __fadd2_rn(sum, weights(r, x, neg));
                            }
                            tmem_st(s_addr + uint32_t(c / 2), x);
                        }
                    }
                    l2 = __fadd2_rn(l2, sum);
                    tmem_wait_st();
                } else {
                    settle(g);
                }
                // the first weights are for an O that begins anew
                if (jj == 0 && unread) {
                    if (!(ok = wait(&bars.o_read[quad], full - 1))) break;
                    unread = false;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(lead(&bars.p_full[b]));
            }
            if (!ok) break;
            // ---- The warp that has the last tile writes the rows; the other goes on to the next
            // item, whose first tile it has.
            const bool last = ((g - 1) & 1) == team;
            if (rows > 0 && !last) {
                sh.sum[mine] = make_float2(l2.x + l2.y, m_ref);
                if (lane == 0) bulk_wait_read();  // (of an item whose rows this warp wrote: the space is the other's now)
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(&bars.sum_there[quad]));
                unread = true;
                ++full;
                ++items;
                continue;
            }
            if (!(ok = wait(&bars.o_full, items++))) break;
            if (rows <= 0) continue;
            if (!(ok = wait(&bars.sum_there[quad], full++))) break;
            tc_fence_after();
            const float2 other = sh.sum[mine];
            const float l = l2.x + l2.y + (m_ref > other.y ? other.x * fast_exp2(other.y - m_ref) : other.x), f = l > 0.f ? 1.f / l : 0.f;
            // The rows pass through shared memory, chunks swizzled by row, and leave as tensor
            // copies, which nobody waits for. A sequence's last rows share their box with the
            // next one's, and leave as stores of whole lines.
            const uint32_t st = out0 + uint32_t(quad * 2 * T::kOutBytes);
            const uint32_t mine_at = st + uint32_t(lane * 128), sw = uint32_t(lane & 7);
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
                uint32_t o[32];
                tmem_ld(o, o_addr + uint32_t(h * 32));
                if (h == D / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(&bars.o_read[quad]));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = f2_to_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * f, __uint_as_float(o[8 * e + 2 * k + 1]) * f);
                    sts128(mine_at + uint32_t(h / 2 * 4096) + ((uint32_t(h % 2 * 4 + e) ^ sw) << 4), make_uint4(x[0], x[1], x[2], x[3]));
                }
            }
            if (rows == 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_store_4d(&p.tm_out, st + uint32_t(c * 4096), c * 64, 0, kvh, row0 + (first >> lgG));
                    bulk_commit();
                }
            } else {
                __syncwarp();
                constexpr int CH = D / 8;  // 16-byte chunks of a row
#pragma unroll 1
                for (int e = lane; e < rows * CH; e += 32) {
                    const int r = e / CH, ch = e % CH, rr = first + r;
                    const uint4 v = lds128(st + uint32_t(ch / 8 * 4096 + r * 128) + ((uint32_t(ch % 8) ^ uint32_t(r & 7)) << 4));
                    *reinterpret_cast<uint4*>(p.out + int64_t(row0 + (rr >> lgG)) * p.out_stride +
                                              (kvh * G + (rr & (G - 1))) * D + ch * 8) = v;
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            bulk_wait();
            if (!ok) report(p.err, kErrTimeout);
        }
    } else if (warp == kLoadWarp) {
        // ================= Q, this CTA's half of K's rows and of V's columns =================
        const bool leader = elect_one();
        if (leader) {
            prefetch_tensormap(&p.tm_q);
            prefetch_tensormap(&p.tm_k);
            prefetch_tensormap(&p.tm_v);
        }
        __syncwarp();
        int it = 0, loaded = 0, fixed = 0;
        for (int q = 0; ok && take(q); release(q++)) {
            const PromptItem& im = sh.item[q & 1];
            if (im.kind == 1) continue;
            const KeyTiles kt = im.kt;
            const int kvh = im.kvh, row0 = im.row0, r_first = im.r_first, n = im.n, qs = loaded & 1;
            if (loaded >= 2 && !(ok = wait(&bars.q_empty[qs], (loaded >> 1) - 1))) break;
            if (leader) {
                mbar_arrive_expect_tx_peer(lead(&bars.q_full[qs]), T::kQBytes);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_4d_pair(q_addr + uint32_t(qs * T::kQBytes + h * kPrRows * 128), &p.tm_q, h * 64, 0, kvh,
                                     row0 + ((r_first + int(rank) * kPrRows) >> lgG), lead(&bars.q_full[qs]));
            }
            __syncwarp();
            ++loaded;
            for (int jj = 0; jj < kt.n; ++jj, ++it) {
                const int s = it % STAGES, t0 = kt.tile(jj) * kPrKeys;
                if (it >= STAGES && !(ok = wait(&bars.k_empty[s], it / STAGES - 1))) break;
                if (leader) {
                    mbar_arrive_expect_tx_peer(lead(&bars.k_full[s]), T::kTileBytes);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_4d_pair(k_addr + uint32_t(s * T::kTileBytes + h * 64 * 128), &p.tm_k, h * 64, 0, kvh,
                                         row0 + t0 + int(rank) * 64, lead(&bars.k_full[s]));
                }
                __syncwarp();
                if (it >= STAGES && !(ok = wait(&bars.v_empty[s], it / STAGES - 1))) break;
                // V's rows behind the sequence's end are another's, or nobody's: cleared, since
                // their weight of zero would not hide a not-a-number
                const bool fix = t0 + kPrKeys > n;
                const uint32_t dst = v_addr + uint32_t(s * T::kTileBytes);
                if (leader) {
                    if (fix) mbar_arrive_expect_tx(bar(&bars.fix), T::kTileBytes);
                    else mbar_arrive_expect_tx_peer(lead(&bars.v_full[s]), T::kTileBytes);
                    tma_load_4d_pair(dst, &p.tm_v, int(rank) * (D / 2), 0, kvh, row0 + t0,
                                     fix ? cluster_addr(bar(&bars.fix), rank) : lead(&bars.v_full[s]));
                }
                __syncwarp();
                if (fix) {
                    if (!(ok = wait(&bars.fix, fixed))) break;
                    ++fixed;
                    for (int e = (n - t0) * (D / 16) + lane; e < kPrKeys * (D / 16); e += 32)
                        sts128(dst + uint32_t(e * 16), make_uint4(0u, 0u, 0u, 0u));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (leader) mbar_arrive_release_cluster(lead(&bars.v_full[s]));
                }
            }
        }
        if (!ok && lane == 0) report(p.err, kErrTimeout);
    } else if (warp == kScoreWarp) {
        if (rank == 0) {
            // ================= S = Q K^T of both CTAs, up to three tiles ahead =================
            // (In the two issuing warps the whole warp walks through the loop, so that
            // addresses and descriptors stay warp-uniform; one thread issues. A step along
            // K is an addition to a descriptor's address field, in 16-byte units.)
            constexpr uint32_t kDesc = mma_desc_bf16(kPrKeys, false, 256);
            const bool leader = elect_one();
            const uint32_t tm = __shfl_sync(kFull, tm_s, 0);
            const uint64_t dq = smem_desc(q_addr, 16), dk = smem_desc(k_addr, 16);
            int g = 0, used = 0;
            for (int q = 0; ok && take(q); release(q++)) {
                const PromptItem& im = sh.item[q & 1];
                if (im.kind == 1) continue;
                const int n = im.kt.n, qs = used & 1;
                if (!(ok = wait(&bars.q_full[qs], used >> 1))) break;
                for (int jj = 0; jj < n; ++jj, ++g) {
                    const int s = g % STAGES, b = g % kPrScores;
                    // the weights that were there have been used
                    if (g >= kPrScores && !(ok = wait(&bars.pv_done[b], g / kPrScores - 1))) break;
                    if (!(ok = wait(&bars.k_full[s], g / STAGES))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            mma_ss_pair(tm + uint32_t(b) * 128u, dq + uint64_t((qs * T::kQBytes + (ks / 4) * kPrRows * 128 + (ks % 4) * 32) / 16),
                                        dk + uint64_t((s * T::kTileBytes + (ks / 4) * 64 * 128 + (ks % 4) * 32) / 16), kDesc, ks > 0);
                        mma_commit_pair(bar(&bars.s_full[b]));
                        mma_commit_pair(bar(&bars.k_empty[s]));
                        if (jj + 1 == n) mma_commit_pair(bar(&bars.q_empty[qs]));
                    }
                    __syncwarp();
                }
                ++used;
            }
            if (!ok) {
                if (leader) mma_commit_pair(bar(&bars.drain[0]));
                (void)wait(&bars.drain[0], 0);
                if (lane == 0) report(p.err, kErrTimeout);
            }
        }
    } else if (warp == kValueWarp) {
        if (rank == 0) {
            // ================= O += P V of both CTAs =================
            constexpr uint32_t kDesc = mma_desc_bf16(D, true, 256);
            const bool leader = elect_one();
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            const uint64_t dv = D == 128 ? smem_desc(v_addr, 16) : smem_desc_64b(v_addr);
            int g = 0;
            for (int q = 0; ok && take(q); release(q++)) {
                const PromptItem& im = sh.item[q & 1];
                if (im.kind == 1) continue;
                const int n = im.kt.n;
                for (int jj = 0; jj < n; ++jj, ++g) {
                    const int s = g % STAGES, b = g % kPrScores;
                    if (!(ok = wait(&bars.v_full[s], g / STAGES) && wait(&bars.p_full[b], g / kPrScores))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < kPrKeys / 16; ++ks)
                            mma_ts_pair(tm, tm + 128u + uint32_t(b) * 128u + uint32_t(ks) * 8u,
                                        dv + uint64_t((s * T::kTileBytes + ks * 16 * D) / 16), kDesc, jj > 0 || ks > 0);
                        mma_commit_pair(bar(&bars.pv_done[b]));
                        mma_commit_pair(bar(&bars.v_empty[s]));
                        if (jj + 1 == n) mma_commit_pair(bar(&bars.o_full));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                if (leader) mma_commit_pair(bar(&bars.drain[1]));
                (void)wait(&bars.drain[1], 0);
                if (lane == 0) report(p.err, kErrTimeout);
            }
        }
    } else if (warp == kPlanWarp) {
        if (rank == 0) {
            // ================= items, for both CTAs =================
            const bool leader = elect_one();
            int cx = int(blockIdx.x) / 2;
            // (row tile, kv head) of all sequences in a list, the row tiles from the last one
            // on: later rows see more keys. The grid has a pair for each item that the
            // host's bounds allow; behind the batch's own they have none, and are asked for
            // and dropped.
            const auto range = [&](int s, int32_t* err) { return seq_range(p.bt, s, 1 << 16, err, err != nullptr); };
            const auto row_tiles = [&](int s) { return int((int64_t(range(s, nullptr).n) * G + 2 * kPrRows - 1) / (2 * kPrRows)); };
            ListCursor<decltype(row_tiles)> list(p.bt.B, row_tiles);
            const int list_tiles = int(list.total < p.item_tiles ? list.total : p.item_tiles);
            const int items = list_tiles * p.Hkv;
            if (cx == 0)
                for (int b = lane; b < p.bt.B; b += 32) {
                    const SeqRange r = range(b, p.err);
                    if (r.n > 0 && r.ctx != r.n) report(p.err, kErrCtxLen);
                }
            int published = 0, round = 0;
            // The grid's cx-th pair's item; false: it has none.
            const auto describe = [&](PromptItem& x) {
                if (cx >= items) return false;
                const WorkItem wi = list.find(list_tiles - 1 - cx / p.Hkv);
                if (wi.b < 0) return false;
                const SeqRange sq = range(wi.b, nullptr);
                x.kind = sq.ctx != sq.n ? 1 : 0;
                x.kvh = cx % p.Hkv;
                x.row0 = sq.row0;
                x.n = sq.n;
                x.r_first = wi.i * 2 * kPrRows;
                x.r_end = min(sq.n * G, x.r_first + 2 * kPrRows);
                x.kt = key_tiles(x.r_first >> lgG, (x.r_end - 1) >> lgG, p.window, p.sinks, kPrKeys);
                return true;
            };
            const auto publish = [&](const PromptItem& x) {
                const int s = published & 1;
                if (published >= 2 && !(ok = wait(&bars.item_empty[s], (published >> 1) - 1))) return false;
                if (lane == 0) {
                    sh.item[s] = x;
                    mbar_arrive(bar(&bars.item_full[s]));
                    // and to the other CTA, whose planner passes it on: a wait that
                    // sees another CTA's stores takes long
                    const uint32_t to = cluster_addr(smem_addr(&sh.item[s]), 1);
                    const int words[] = {x.kind, x.kvh, x.row0, x.n, x.r_first, x.r_end, x.kt.nsink, x.kt.lo, x.kt.n};
                    static_assert(sizeof(words) == sizeof(PromptItem), "an item's words");
#pragma unroll
                    for (int e = 0; e < int(sizeof(words) / 4); ++e) st_cluster_u32(to + 4u * e, uint32_t(words[e]));
                    mbar_arrive_release_cluster(cluster_addr(bar(&bars.mail[s]), 1));
                }
                __syncwarp();
                ++published;
                return true;
            };
            PromptItem x;
            for (;; ++round) {
                if (describe(x) && !publish(x)) break;
                // ask for the pair that the grid would start next, an item ahead and no more
                if (leader) {
                    fence_proxy_async_smem();  // the answer before has been read
                    mbar_arrive_expect_tx(bar(&bars.next), 16);
                    next_cta(smem_addr(&sh.next), bar(&bars.next));
                }
                __syncwarp();
                // (nobody else will take that pair's item: its answer is waited for twice as long)
                if (!(ok = wait(&bars.next, round) || wait(&bars.next, round))) break;
                const bool more = next_cta_read(smem_addr(&sh.next), cx);
                cx /= 2;
                __syncwarp();
                if (!more) break;
            }
            if (ok) {
                x = PromptItem{};
                x.kind = 2;
                (void)publish(x);
            }
            if (!ok && lane == 0) report(p.err, kErrTimeout);
        } else {
            for (int q = 0;; ++q) {
                if (!__all_sync(kFull, wait_phase_cluster(bar(&bars.mail[q & 1]), uint32_t(q >> 1) & 1u))) break;
                const int kind = sh.item[q & 1].kind;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(&bars.item_full[q & 1]));
                if (kind == 2) break;
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // neither CTA ends while the other may use its shared memory
    tc_fence_after();
    if (warp == kScoreWarp) tmem_dealloc_pair(tmem, 512);
}

}  // namespace pkv
