// Attention of whole prompts from their rows (pkv_prompt_attention), on the tensor
// cores of sm_103a (tcgen05, accumulators in tensor memory).
//
// A work item is (256 rows, kv head, sequence): two tiles of 128 rows, a row a
// (token, query head of the group), so that a kv head's whole group shares each
// K and V tile that the CTA loads. Keys come in tiles of 128 tokens, tensor
// copies of 128 rows x 64 elements. There is one CTA a SM; it walks from item to
// item, taking the grid's next one from the hardware (launch cancellation) while
// it works. Within a sequence the items with the most keys come first; the last sequence is
// first in the grid, whatever its length, so a batch packed by ascending length begins with its
// longest items (32 of 16 to 4096 tokens 298.5 us, by descending length 301.8).
//
//   warps 0-3, 4-7: softmax of row tile 0 and 1, one row a thread; scores from
//                   tensor memory, weights back to it
//   warp 8          the loader of K and V
//   warp 9          items, and their queries
//   warp 10         one thread issues the multiplies
//
//   S_i = Q_i K^T   128 x 128 x D, operands in shared memory
//   O_i += P_i V    128 x D x 128, P_i in tensor memory over the scores it came from
// The two row tiles take turns: while one's softmax runs the tensor core works
// for the other. S_i of the next key tile, or of the next item, is issued right
// behind O_i += P_i V, so one commit tells the softmax both that its scores are
// there and that O_i may be corrected.
//
// The reference of a row's exponents is the maximum of its first visible tile. That
// a tile's scores are far above it shows in the sum of the weights, which is needed
// anyway: only above 2^20 (in fp32) the tile's maximum becomes the reference, O_i
// and the sum are rescaled and the tile is weighed again. So no maximum is taken after
// the first tile (with one in the pass: 622 us against 595, below). References of 2^28 and more
// leave the plain path, as their rounding would show in the exponents. Tiles that hide
// something from some row of a warp take a path that is rolled up and skips what nobody
// sees. Weights are kept in units of 2^-40 (an exponent bias, free): the largest, 2^20
// of them, stays below 1, one times a V of 2^-60 leaves 26 bits. They are rounded to bf16 for the multiply (half a step, 2^-8 of
// each weight, as the outputs are); their sum is fp32.
//
// Measured, d = 128: prompts of 7400 to 8000 tokens, 16 query and 8 kv heads, 1.0 TF in
// 595 to 600 us, 1670 TF/s, 640 us once the GPU has come to its power limit (cuBLAS:
// 1897 and 1699); one of 16384 tokens, 32 and 8 heads, 2.2 TF in 1250 us, 1760 TF/s;
// of 5000 to 8192 tokens, window 1024, 211 GF in 181 us; 32 of 16 to 4096 tokens,
// 422 GF in 303 us (with inputs that are not in L2 644, 189 and 325 us); d = 64, two of
// 8000, 16 and 8 heads, 250 to 253 us, 1040 TF/s, of 5000 to 8192 with 32 and 8, window
// 1024, 146 us, 720. One prompt by itself, d = 128, 16 / 32 query heads over 8, us in a graph:
//   tokens        128          512        1024        2048      4096
//   us        10.8/10.9    14.9/15.4   20.4/20.6   30.7/40.1   68/92
//   floor      0.2/0.4      0.9/1.5     2.3/4.5     9.1/18     36/73
// No item is spread over several CTAs, so the longest item's chain is the time while there are
// fewer items than SMs (2048 tokens: 128, of up to 16 key tiles, where an even share is 7). 16
// prompts of 1 to 512 tokens, 32 heads, 28.8 us (floor 6.8). A key tile of both row tiles takes
// 2650 cycles, its multiplies 2048 by themselves and 2440 beside the softmax (they read 192
// KB of shared memory, at 128 bytes a cycle at most). A tile's chain is 930 cycles of
// softmax (a warp's 128 exponentials a thread take 512 of them), 190 until the weights
// are announced, 200 until they are seen, 1220 of multiplies. An item's beginning and
// end cost some 4000 cycles beside that, so windows (ten tiles an item) and short
// prompts are further from the floor. Without the softmax the first case takes 549 us.
// Other forms, the first case and the windowed one: a pair of CTAs with one row tile
// each (cta_group::2, three tiles of scores ahead) 600 and 213 us; the multiplies of
// each row tile by a warp of its own 824 and 222 (they interleave, and both end late);
// outputs by four more warps 669 and 193 (registers); K waited for before O += P V
// instead of behind it 644 to 660 and 190; three stages of K and V or four, the same; hidden
// scores selected in the plain tile's pass, without branches 609 and 184 (short
// prompts 6% faster, d = 64 4% slower), with branches 673 and 199: a branch between two
// chunks keeps one's end from overlapping the next one's beginning.
#pragma once

#include "ptx_tc.cuh"
#include "window.cuh"

namespace pkv {

constexpr int kPrRows = 128;  // rows of a row tile
constexpr int kPrKeys = 128;  // tokens of a key tile
constexpr float kPrShift = 40.f;
constexpr float kPrAhead = 12.f;
constexpr float kPrMost = 0x1p-20f;  // 2^20 in units of 2^-40
constexpr float kPrLarge = 0x1p28f;  // references whose rounding an exponent must not see
constexpr int kPrThreads = 384;
constexpr int kPrLaunchRegs = 168;

struct PromptParams {
    CUtensorMap tm_q;    // q as [tokens][Hkv][G][D], boxes of 128 rows x 64 elements
    CUtensorMap tm_k;    // k, v as [tokens][Hkv][1][D], boxes of 128 rows x 64 elements
    CUtensorMap tm_v;
    CUtensorMap tm_out;  // out as q, boxes of 32 rows
    BatchView bt;
    uint16_t* out;
    int64_t out_stride;
    int32_t* err;
    int32_t Hq, Hkv;
    int32_t window;      // INT32_MAX: none
    int32_t sinks;
    int32_t item_tiles;  // items of a kv head that the batch can have
    int32_t skip_copy;   // pkv_debug_skip_copy (-1: off)
    float qscale;        // sm_scale * log2(e)
};

template <int D>
struct PromptTraits {
    static constexpr int kTileBytes = kPrKeys * D * 2;  // one K or V tile = one row tile of Q
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kOutBytes = 32 * D * 2;        // a softmax warp's rows on their way out
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 8 * kOutBytes;
    static constexpr int kSlab = kPrKeys * 128;         // 64 of a tile's D columns
    static constexpr int kSoftmaxRegs = 200, kRestRegs = 104;
    static_assert(256 * kSoftmaxRegs + 128 * kRestRegs == kPrThreads * kPrLaunchRegs, "register split");
};

template <int STAGES>
struct PromptBars {
    uint64_t q_full, q_empty;
    uint64_t kv_full[STAGES];
    uint64_t kv_empty[STAGES];
    uint64_t fix;            // a V tile whose dead rows have to be cleared first
    uint64_t s_full[2];      // S_i is there and O_i += P_i V of the tile before is done
    uint64_t p_full[2];      // P_i is there, O_i corrected (four warps)
    uint64_t o_full[2];      // O_i is complete
    uint64_t item_full[2];   // an item's description is there
    uint64_t item_empty[2];  // every warp has taken it
    uint64_t next;           // the answer about the next item is there
    uint64_t drain;
};

struct PromptItem {
    int kind;  // 0: attention; 1: rows of a sequence with earlier tokens, zero; 2: the end
    int kvh, row0, n;    // kv head; the sequence's first row, its rows (tokens)
    int r_first, r_end;
    KeyTiles kt;
};

template <int V>
struct PromptCount {
    static constexpr int value = V;
};

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    using T = PromptTraits<D>;
    constexpr int STAGES = T::kStages, kMmaWarp = 10, kPlanWarp = 9, kLoadWarp = 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PromptBars<STAGES> bars;
    __shared__ PromptItem s_item[2];
    __shared__ __align__(16) uint4 s_next;
    __shared__ uint32_t s_tmem;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hq / p.Hkv, lgG = 31 - __clz(G);
    uint8_t* q_smem = smem + ((1024u - (smem_addr(smem) & 1023u)) & 1023u);
    const uint32_t q_addr = smem_addr(q_smem), kv_addr = q_addr + 2 * T::kTileBytes;
    const uint32_t stage0 = kv_addr + STAGES * T::kTileBytes;  // kOutBytes a softmax warp, for its output rows
    const uint32_t bar0 = smem_addr(&bars);
    const auto bar = [&](const uint64_t* x) {
        return bar0 + uint32_t(reinterpret_cast<const uint8_t*>(x) - reinterpret_cast<const uint8_t*>(&bars));
    };
    if (tid == 0) {
        mbar_init(bar(&bars.q_full), 1);
        mbar_init(bar(&bars.q_empty), 1);
        mbar_init(bar(&bars.fix), 1);
        mbar_init(bar(&bars.next), 1);
        mbar_init(bar(&bars.drain), 1);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(&bars.kv_full[s]), 1);
            mbar_init(bar(&bars.kv_empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(&bars.s_full[i]), 1);
            mbar_init(bar(&bars.p_full[i]), 4);
            mbar_init(bar(&bars.o_full[i]), 1);
            mbar_init(bar(&bars.item_full[i]), 1);
            mbar_init(bar(&bars.item_empty[i]), 8 + 2);
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), 512);
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
    else reg_dec<T::kRestRegs>();

    if (warp < 8) {
        // ================= softmax of row tile i, a row a thread =================
        const int i = warp >> 2;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + uint32_t(i) * 128u + lane_base, o_addr = tmem + 256u + uint32_t(i) * 128u + lane_base;
        const float scale = p.qscale;
        int mine = 0, done = 0;  // key tiles and items of this row tile
        for (int q = 0; take(q); release(q++)) {
            const PromptItem& im = s_item[q & 1];
            const int row = im.r_first + tid;  // tid < 256: rows of the item in order
            const bool have = row < im.r_end;
            if (im.kind == 1) {
                for (int e = tid; e < (im.r_end - im.r_first) * D; e += 256) {
                    const int r = im.r_first + e / D;
                    p.out[int64_t(im.row0 + (r >> lgG)) * p.out_stride + (im.kvh * G + (r & (G - 1))) * D + e % D] = 0;
                }
                continue;
            }
            if (im.r_first + i * kPrRows >= im.r_end) continue;
            const KeyTiles kt = im.kt;
            const int n = kt.n;
            float m_ref = have ? -INFINITY : INFINITY;  // reference of the exponent (base 2); no row: weights of 0
            bool odd = true;  // some row of the warp has no reference yet, or one of 2^28 and more
            float2 l2 = make_float2(0.f, 0.f);
            const int hi = have ? row >> lgG : -1, lo = max(0, hi - p.window + 1);
            // the warp's first and last position, and where their windows begin
            const int w_first = im.r_first + warp * 32, w_rows = min(32, im.r_end - w_first);
            const int pf = w_first >> lgG, pl = (w_first + w_rows - 1) >> lgG, wf = pf - p.window + 1, wl = pl - p.window + 1;
            for (int jj = 0; jj < n; ++jj) {
                if (!(ok = wait(&bars.s_full[i], mine + jj))) break;
                tc_fence_after();
                if (w_rows > 0) {
                    const int t0 = kt.tile(jj) * kPrKeys;
                    const bool masked = jj < kt.nsink || t0 + kPrKeys - 1 > pf || t0 < wl;
                    float2 sum = make_float2(0.f, 0.f);
                    // `count` scores to weights, into `to`, and their sum.
                    const auto weights = [&](const uint32_t* r, auto count, uint32_t* to, float mul, float neg) {
                        const float2 a2 = make_float2(mul, mul), b2 = make_float2(neg, neg);
                        float2 part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < count.value; e += 4) {
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
                        sum = __fadd2_rn(sum, part);
                    };
                    // 32 scores from column c on, hidden ones -infinity; false: no row of the warp sees any.
                    const auto scores = [&](uint32_t (&r)[32], int c) {
                        const int tc = t0 + c;
                        if (masked && (tc > pl || (tc + 31 < wf && tc >= p.sinks))) return false;
                        tmem_ld(r, s_addr + uint32_t(c));
                        if (masked && !(tc + 31 <= pf && (tc >= wl || tc + 31 < p.sinks))) {
                            // bit e: this row sees token tc + e
                            const auto below = [](int x) { return x >= 32 ? 0xFFFFFFFFu : (1u << max(0, x)) - 1u; };
                            const uint32_t see = below(hi - tc + 1) & (below(p.sinks - tc) | ~below(lo - tc));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((see >> e) & 1u)) r[e] = 0xFF800000u;
                        }
                        return true;
                    };
                    // The tile's maximum becomes the reference of a row that has none, and of one that it
                    // is more than 2^12 above (`all`: that it is above); O follows.
                    const auto raise = [&](bool all) {
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32) {
                            uint32_t r[32];
                            if (!scores(r, c)) continue;
#pragma unroll
                            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(r[e]));
                        }
                        mx *= scale;
                        const bool up = mx > m_ref && (all || mx - m_ref > kPrAhead);
                        const float f = up ? fast_exp2(m_ref - mx) : 1.f;
                        if (up) m_ref = mx;
                        odd = __any_sync(kFull, fabsf(m_ref) >= kPrLarge && m_ref < INFINITY);
                        l2.x *= f;
                        l2.y *= f;
                        if (jj > 0 && __any_sync(kFull, up)) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld(o, o_addr + uint32_t(c));
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st(o_addr + uint32_t(c), o);
                            }
                        }
                    };
                    // Weights over scores that have been read, rolled up: for what is not the plain tile.
                    // A score's exponent is score * scale - reference, in one rounding: up to half a step of
                    // the reference above 0. From 2^28 on that is 16 and more, from 2^31 on the weight overflows.
                    // There products are rounded as the reference was, and lie 32 or more apart or are the same.
                    const auto large = [&]() { return __any_sync(kFull, fabsf(m_ref) >= kPrLarge && fabsf(m_ref) < INFINITY); };
                    const auto weigh_in_place = [&]() {
                        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
                        const bool rounded = large();
                        const float mul = rounded ? 1.f : scale, neg = (rounded ? 0.f : -ref) - kPrShift;
                        sum = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32) {
                            uint32_t r[32], x[16];
                            if (scores(r, c)) {
                                if (rounded) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        r[e] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(r[e]), scale), -ref));
                                }
                                weights(r, PromptCount<32>{}, x, mul, neg);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = 0u;
                            }
                            tmem_st(s_addr + uint32_t(c / 2), x);
                        }
                    };
                    bool slow = masked;
                    if (masked || odd) {
                        raise(false);
                        slow |= large();
                    }
                    if (slow) {
                        weigh_in_place();
                    } else {
                        // 16 columns at a time, one chunk's load in flight while the other is worked on
                        const float neg = (m_ref == -INFINITY ? 0.f : -m_ref) - kPrShift;
                        uint32_t w[2][32], ra[16], rb[16];
                        tmem_ld_start(ra, s_addr);
#pragma unroll
                        for (int c = 0; c < 128; c += 32) {
                            tmem_ld_wait(ra);
                            tmem_ld_start(rb, s_addr + uint32_t(c + 16));
                            weights(ra, PromptCount<16>{}, w[c / 64] + c % 64 / 2, scale, neg);
                            tmem_ld_wait(rb);
                            if (c < 96) tmem_ld_start(ra, s_addr + uint32_t(c + 32));
                            weights(rb, PromptCount<16>{}, w[c / 64] + c % 64 / 2 + 8, scale, neg);
                        }
                        if (__any_sync(kFull, sum.x + sum.y > kPrMost)) {
                            raise(true);
                            weigh_in_place();
                        } else {
                            tmem_st(s_addr, w[0]);
                            tmem_st(s_addr + 32u, w[1]);
                        }
                    }
                    l2 = __fadd2_rn(l2, sum);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(&bars.p_full[i]));
            }
            if (ok) ok = wait(&bars.o_full[i], done);
            mine += n;
            ++done;
            if (!ok) break;
            // ---- write the rows: the warp's 32 pass through shared memory, 128 bytes of each at a
            // time, chunks swizzled by row, and leave as tensor copies, which nobody waits for. A
            // sequence's last rows share their box with the next one's, and leave as
            // stores of whole lines. (Rolled up: code that runs once an item is fetched anew.)
            tc_fence_after();
            const float l = l2.x + l2.y, f = l > 0.f ? 1.f / l : 0.f;
            const uint32_t st = stage0 + uint32_t(warp * T::kOutBytes);
            const uint32_t mine_at = st + uint32_t(lane) * 128u, sw = uint32_t(lane & 7);
            const int first = im.r_first + warp * 32, rows = min(32, im.r_end - first);
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld(o, o_addr + uint32_t(c));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = f2_to_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * f, __uint_as_float(o[8 * e + 2 * k + 1]) * f);
                    sts128(mine_at + uint32_t(c / 64 * 4096) + ((uint32_t(c % 64 / 8 + e) ^ sw) << 4), make_uint4(x[0], x[1], x[2], x[3]));
                }
            }
            if (rows == 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_store_4d(&p.tm_out, st + uint32_t(c * 4096), c * 64, 0, im.kvh, im.row0 + (first >> lgG));
                    bulk_commit();
                }
            } else {
                __syncwarp();
                constexpr int CH = D / 8;  // 16-byte chunks of a row
#pragma unroll 1
                for (int e = lane; e < rows * CH; e += 32) {
                    const int r = e / CH, ch = e % CH, rr = first + r;
                    const uint4 v = lds128(st + uint32_t(ch / 8 * 4096 + r * 128) + ((uint32_t(ch % 8) ^ uint32_t(r & 7)) << 4));
                    *reinterpret_cast<uint4*>(p.out + int64_t(im.row0 + (rr >> lgG)) * p.out_stride +
                                              (im.kvh * G + (rr & (G - 1))) * D + ch * 8) = v;
                }
                __syncwarp();
            }
            tc_fence_before();  // O_i has been read before the next item's P_i is announced
        }
        if (lane == 0) {
            bulk_wait();
            if (!ok) report(p.err, kErrTimeout);
        }
    } else if (warp == kLoadWarp) {
        // ================= K and V tiles =================
        const bool leader = elect_one();
        if (leader) {
            prefetch_tensormap(&p.tm_k);
            prefetch_tensormap(&p.tm_v);
        }
        __syncwarp();
        int tiles = 0, fixed = 0, jj = 0, v = 0;  // tiles: of the items before
        bool fixing = false;
        for (int q = 0; ok && take(q); release(q++)) {
            const PromptItem& im = s_item[q & 1];
            if (im.kind == 1) continue;
            const KeyTiles kt = im.kt;
            const int kvh = im.kvh, row0 = im.row0, n = im.n;
            for (jj = 0; jj < kt.n && ok; ++jj) {
                const int t0 = kt.tile(jj) * kPrKeys;
                for (v = 0; v < 2; ++v) {
                    const int it = 2 * (tiles + jj) + v, s = it % STAGES;
                    if (it >= STAGES && !(ok = wait(&bars.kv_empty[s], it / STAGES - 1))) break;
                    // V: rows behind the sequence's end are another's, or nobody's: cleared,
                    // since their weight of zero would not hide a not-a-number
                    fixing = v && t0 + kPrKeys > n;
                    const uint32_t full = fixing ? bar(&bars.fix) : bar(&bars.kv_full[s]);
                    const uint32_t dst = kv_addr + uint32_t(s) * T::kTileBytes;
                    if (leader) {
                        mbar_arrive_expect_tx(full, T::kTileBytes);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_4d(dst + uint32_t(h * T::kSlab), v ? &p.tm_v : &p.tm_k, h * 64, 0, kvh, row0 + t0, full);
                    }
                    __syncwarp();
                    if (fixing) {
                        if (!(ok = wait(&bars.fix, fixed))) break;
                        ++fixed;
                        fixing = false;
                        for (int e = (n - t0) * (D / 8) + lane; e < kPrKeys * (D / 8); e += 32) {
                            const int rr = e / (D / 8), ch = e % (D / 8);
                            sts128(dst + uint32_t((ch / 8) * T::kSlab + rr * 128 + (ch % 8) * 16), make_uint4(0u, 0u, 0u, 0u));
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader) mbar_arrive(bar(&bars.kv_full[s]));
                    }
                }
                if (!ok) break;
            }
            if (ok) {
                tiles += kt.n;
                jj = v = 0;
            }
        }
        if (!ok) {
            // let the copies in flight land before the CTA ends
            const int upto = 2 * (tiles + jj) + v;
            for (int it = max(0, upto - STAGES); it < upto; ++it) (void)wait(&bars.kv_full[it % STAGES], it / STAGES);
            if (fixing) (void)wait(&bars.fix, fixed);
            if (lane == 0) report(p.err, kErrTimeout);
        }
    } else if (warp == kMmaWarp) {
        // ================= the multiplies =================
        // The whole warp walks through the loop, so that addresses and descriptors
        // stay warp-uniform; one thread issues. A step along K is an addition to a
        // descriptor's address field (16-byte units).
        constexpr uint32_t kDescS = mma_desc_bf16(kPrKeys, false), kDescO = mma_desc_bf16(D, true);
        constexpr uint64_t kTile16 = T::kTileBytes / 16;
        // One thread: what it does between two groups of multiplies shows, since no more than
        // about four of them wait in the tensor core's queue.
        if (elect_one()) {
            const uint64_t dq = smem_desc(q_addr, 16), dk = smem_desc(kv_addr, 16), dv = smem_desc(kv_addr, T::kSlab);
            const uint32_t tm = tmem;
            const auto issue_s = [&](int i, int stage) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    constexpr uint64_t kSlab16 = T::kSlab / 16;
                    const uint64_t off = uint64_t(ks / 4) * kSlab16 + uint64_t(ks % 4) * 2u;
                    mma_ss(tm + uint32_t(i) * 128u, dq + uint64_t(i) * kTile16 + off, dk + uint64_t(stage) * kTile16 + off,
                           kDescS, ks > 0);
                }
                mma_commit(bar(&bars.s_full[i]));
            };
            const auto wait1 = [&](const uint64_t* x, uint32_t parity) { return wait_phase(bar(x), parity & 1u); };
            const auto there = [&](const uint64_t* x, uint32_t parity) { return mbar_try_wait(bar(x), parity & 1u); };
            int tiles = 0, mine[2] = {0, 0}, items = 0;
            uint32_t begun = 0;  // row tiles whose first scores of the next item have been issued
            for (int q = 0; ok; ++q) {
                if (!(ok = wait1(&bars.item_full[q & 1], q >> 1))) break;
                const PromptItem& im = s_item[q & 1];
                const int kind = im.kind, n = im.kt.n, nq = im.r_end - im.r_first > kPrRows ? 2 : 1;
                if (kind == 2) break;
                if (kind == 0) {
                    const int first = 2 * tiles, sf = first % STAGES;
                    if (!(ok = wait1(&bars.q_full, items) && wait1(&bars.kv_full[sf], first / STAGES))) break;
                    tc_fence_after();
                    for (int i = 0; i < nq; ++i)
                        if (!((begun >> i) & 1u)) issue_s(i, sf);
                    begun = 0;
                    mma_commit(bar(&bars.kv_empty[sf]));
                    if (n == 1) mma_commit(bar(&bars.q_empty));
                    for (int jj = 0; jj < n && ok; ++jj) {
                        const int iv = 2 * (tiles + jj) + 1, ik = iv + 1, sv = iv % STAGES, sk = ik % STAGES;
                        ok = wait1(&bars.kv_full[sv], iv / STAGES);
                        for (int i = 0; i < nq && ok; ++i) {
                            if (!(ok = wait1(&bars.p_full[i], mine[i] + jj))) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < kPrKeys / 16; ++ks)
                                mma_ts(tm + 256u + uint32_t(i) * 128u, tm + uint32_t(i) * 128u + uint32_t(ks) * 8u,
                                       dv + uint64_t(sv) * kTile16 + uint64_t(ks) * 128u, kDescO, jj > 0 || ks > 0);
                            if (jj + 1 < n) {
                                if (i == 0 && !(ok = wait1(&bars.kv_full[sk], ik / STAGES))) break;
                                tc_fence_after();
                                if (i == nq - 1) mma_commit(bar(&bars.kv_empty[sv]));
                                issue_s(i, sk);
                                if (i == nq - 1) {
                                    mma_commit(bar(&bars.kv_empty[sk]));
                                    if (jj + 2 == n) mma_commit(bar(&bars.q_empty));  // the last use of Q
                                }
                            } else {
                                mma_commit(bar(&bars.o_full[i]));
                                if (i == nq - 1) mma_commit(bar(&bars.kv_empty[sv]));
                                // (not waited for: the other row tile's O goes first)
                                if (there(&bars.item_full[(q + 1) & 1], (q + 1) >> 1)) {
                                    const PromptItem& nx = s_item[(q + 1) & 1];
                                    if (nx.kind == 0 && nx.r_end - nx.r_first > i * kPrRows && there(&bars.q_full, items + 1) &&
                                        there(&bars.kv_full[sk], ik / STAGES)) {
                                        tc_fence_after();
                                        issue_s(i, sk);
                                        begun |= 1u << i;
                                    }
                                }
                            }
                        }
                    }
                    tiles += n;
                    mine[0] += n;
                    if (nq == 2) mine[1] += n;
                    ++items;
                }
                if (ok) mbar_arrive(bar(&bars.item_empty[q & 1]));
            }
            if (!ok) {
                mma_commit(bar(&bars.drain));
                (void)wait1(&bars.drain, 0);
                report(p.err, kErrTimeout);
            }
        }
        __syncwarp();
    } else if (warp == kPlanWarp) {
        // ================= items and queries =================
        const bool leader = elect_one();
        if (leader) prefetch_tensormap(&p.tm_q);
        int cx = blockIdx.x;
        // (row tile, kv head) of all sequences in a list, the row tiles from the last one
        // on: later rows see more keys. The grid has a CTA for each item that the
        // host's bounds allow; behind the batch's own they have none, and are asked for
        // and dropped.
        // (the context only says that there are no earlier tokens: it need not fit a block table)
        const auto range = [&](int s) {
            const int begin = p.bt.starts[s], end = p.bt.starts[s + 1];
            if (begin < 0 || end < begin || end > p.bt.num_tokens || end - begin > p.bt.max_tokens) return SeqRange{0, 0, 0, true};
            return SeqRange{begin, end - begin, p.bt.ctx[s], false};
        };
        const auto row_tiles = [&](int s) { return int((int64_t(range(s).n) * G + 2 * kPrRows - 1) / (2 * kPrRows)); };
        ListCursor<decltype(row_tiles)> list(p.bt.B, row_tiles);
        const int list_tiles = int(list.total < p.item_tiles ? list.total : p.item_tiles);
        const int items = list_tiles * p.Hkv;
        if (cx == 0)
            for (int b = lane; b < p.bt.B; b += 32) {
                const SeqRange r = range(b);
                if (r.bad) report(p.err, kErrBatch);
                else if (r.n > 0 && r.ctx != r.n) report(p.err, kErrCtxLen);
            }
        int published = 0, loaded = 0, round = 0;
        // The grid's cx-th CTA's item; false: it has none.
        const auto describe = [&](PromptItem& x) {
            if (cx >= items) return false;
            const WorkItem wi = list.find(list_tiles - 1 - cx / p.Hkv);
            if (wi.b < 0) return false;
            const SeqRange sq = range(wi.b);
            x.kind = sq.ctx != sq.n ? 1 : 0;
            x.kvh = cx % p.Hkv;
            x.row0 = sq.row0;
            x.n = sq.n;
            x.r_first = wi.i * 2 * kPrRows;
            x.r_end = min(sq.n * G, x.r_first + 2 * kPrRows);
            x.kt = key_tiles(x.r_first >> lgG, (x.r_end - 1) >> lgG, p.window, p.sinks, kPrKeys);
            return true;
        };
        PromptItem x;
        for (;; ++round) {
            if (describe(x)) {
                const int s = published & 1;
                if (published >= 2 && !(ok = wait(&bars.item_empty[s], (published >> 1) - 1))) break;
                if (lane == 0) {
                    s_item[s] = x;
                    mbar_arrive(bar(&bars.item_full[s]));
                }
                ++published;
                if (x.kind == 0) {
                    // its place is free only behind the last scores of the item before: to L2 meanwhile
                    if (leader && loaded > 0) {
                        for (int i = 0; i < 2; ++i)
                            for (int h = 0; h < D / 64; ++h)
                                if (x.r_first + i * kPrRows < x.r_end)
                                    tma_prefetch_4d(&p.tm_q, h * 64, 0, x.kvh, x.row0 + ((x.r_first + i * kPrRows) >> lgG));
                    }
                    if (loaded > 0 && !(ok = wait(&bars.q_empty, loaded - 1))) break;
                    // (the test hook leaves one item of the first CTA without its queries)
                    if (leader && !(blockIdx.x == 0 && loaded == p.skip_copy)) {
                        const int nq = x.r_end - x.r_first > kPrRows ? 2 : 1;
                        mbar_arrive_expect_tx(bar(&bars.q_full), uint32_t(nq) * T::kTileBytes);
                        for (int i = 0; i < nq; ++i)
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_4d(q_addr + i * T::kTileBytes + h * T::kSlab, &p.tm_q, h * 64, 0, x.kvh,
                                            x.row0 + ((x.r_first + i * kPrRows) >> lgG), bar(&bars.q_full));
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
            if (lane == 0) report(p.err, kErrTimeout);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace pkv
