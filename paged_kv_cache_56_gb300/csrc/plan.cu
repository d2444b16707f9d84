// Batches planned on the GPU (pkv_plan_batch, pkv_commit_batch,
// pkv_release_batch): block lists, lengths and a ring of free blocks in device
// memory.
//
// A plan is two prefix sums over the batch's entries -- new tokens, and blocks
// that an entry's list lacks -- and then copies: the padded tables, and for each
// new token its block, offset, slot and index. Every CTA works out the sums over
// all entries by itself (an entry is 16 bytes in L2), so that one launch is
// enough: a CTA then makes its share of the copies, entries taken from the
// front of the list on. All CTAs come to the same verdict about the batch, so that all
// of them make the plan or none does. New ids go into the pool's lists by the CTA
// that copies that part of the table; numbers that others still read (held,
// the ring's front) are changed by the CTA that is last to arrive. A thread's first
// word of a list is read before the sums are there (its place depends on the slot alone).
//
// Bound by latency: launch, slots -> lengths -> sums (two barriers) -> lists, and where
// blocks are taken ring -> lists, a fence, the arrivals and the last CTA's pass. In a graph, us:
//                                                        all held   blocks taken
//   4 entries                                               5.1          -
//   144 entries, 128 single tokens, tables of 1024          5.4      7.5 (9 blocks)
//   512 entries of 1 to 200 tokens, the same (2.9 MB)       6.6      9.1 (1271)
//   1024 single tokens, the same                           10.8     13.6 (68)
//   4096 single tokens, tables of 64                       18.7     24.7 (262)
// (0.4 us of the third are bytes at the memory's rate.) Commit 1.9 to 2.3; release of 144
// entries with 17975 blocks 6.4, of 512 with 119586 8.0. Steps that go on, plan and commit of 128
// sequences, 8 of which need a block: 10.4 for both. Called one by one from Python 10 to 16 us: the
// call. Entries are taken 512 at a time, by every CTA, and twice when there are more than 512.
#include <algorithm>

#include "batch.cuh"
#include "host.h"

namespace pkv {

constexpr int kErrOom = 64;
constexpr int kPlanThreads = 512;
constexpr int kMaxPoolSlots = 65536;

struct PoolView {
    int32_t* tables;
    int32_t* lens;
    int32_t* held;
    int32_t* ring;
    int32_t* state;
    int32_t* err;
    int32_t max_slots, max_blocks, num_blocks, bs, lg, int8;  // lg: bs = 1 << lg
};

struct PlanParams {
    PoolView pool;
    pkv_plan out;
    const int32_t* slots;
    const int32_t* counts;
    int32_t B;
    int32_t rows;  // rows of the token arrays (0: none of them is wanted)
    int32_t wide;  // tables are copied four entries at a time
};

// An entry of the batch: its new tokens and the blocks it takes (release: gives back).
struct Entry {
    int slot, len, held, n, move;
};

template <bool RELEASE>
__device__ __forceinline__ Entry load_entry(const PlanParams& p, int e, int& bad) {
    Entry x{-1, 0, 0, 0, 0};
    if (e >= p.B) return x;
    x.slot = p.slots[e];
    if (x.slot == -1) return x;
    if (x.slot < 0 || x.slot >= p.pool.max_slots) {
        bad |= kErrSlot;
        x.slot = -1;
        return x;
    }
    x.n = RELEASE ? 0 : p.counts ? p.counts[e] : 1;
    x.len = p.pool.lens[x.slot];
    x.held = p.pool.held[x.slot];
    if (x.held < 0 || x.held > p.pool.max_blocks || x.len < 0 || int64_t(x.len) > int64_t(x.held) * p.pool.bs) {
        bad |= kErrCtxLen;
        x.held = x.len = x.n = 0;
        return x;
    }
    if (RELEASE) {
        x.move = x.held;
        return x;
    }
    if (x.n < 0 || x.n > p.out.max_tokens) {
        bad |= kErrBatch;
        x.n = 0;
        return x;
    }
    const int64_t blocks = (int64_t(x.len) + x.n + p.pool.bs - 1) >> p.pool.lg;
    if (blocks > p.pool.max_blocks) {
        bad |= kErrCtxLen;
        x.n = 0;
        return x;
    }
    x.move = max(0, int(blocks) - x.held);
    return x;
}

struct PlanShared {
    Entry entry[kPlanThreads];
    long long start[kPlanThreads + 1];  // first row of a tile's entries
    long long off[kPlanThreads + 1];    // blocks taken before
    long long warp[2][kPlanThreads / 32];
    uint32_t seen[kMaxPoolSlots / 32];  // slots of the batch so far
    int bad, last;
};

template <bool RELEASE>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ PlanShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const PoolView& pool = p.pool;
    const int N = pool.num_blocks;
    for (int i = tid; i < (pool.max_slots + 31) / 32; i += kPlanThreads) sh.seen[i] = 0u;
    if (tid == 0) sh.bad = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();

    // Sums over a tile of entries: start[i], off[i] of entry i, and the tile's at [512].
    const auto scan = [&](const Entry& x, long long row0, long long off0) {
        long long a = x.n, b = x.move;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, a, o), v = __shfl_up_sync(kFull, b, o);
            if (lane >= o) {
                a += u;
                b += v;
            }
        }
        if (lane == 31) {
            sh.warp[0][warp] = a;
            sh.warp[1][warp] = b;
        }
        __syncthreads();
        constexpr int W = kPlanThreads / 32;
        long long a0 = lane < W ? sh.warp[0][lane] : 0, b0 = lane < W ? sh.warp[1][lane] : 0;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, a0, o), v = __shfl_up_sync(kFull, b0, o);
            if (lane >= o) {
                a0 += u;
                b0 += v;
            }
        }
        a0 = row0 + (warp > 0 ? __shfl_sync(kFull, a0, warp - 1) : 0);  // (of the warps before)
        b0 = off0 + (warp > 0 ? __shfl_sync(kFull, b0, warp - 1) : 0);
        sh.entry[tid] = x;
        sh.start[tid] = a0 + a - x.n;
        sh.off[tid] = b0 + b - x.move;
        if (tid == kPlanThreads - 1) {
            sh.start[kPlanThreads] = a0 + a;
            sh.off[kPlanThreads] = b0 + b;
        }
        __syncthreads();
    };

    // ---- this CTA's share of the tables (in words of one or four entries), entries and rows
    const int G = gridDim.x, cta = blockIdx.x, mb = pool.max_blocks, vec = p.wide ? 4 : 1, wpr = mb / vec;  // words a row
    const long long words = (long long)p.B * wpr;
    const long long w0 = words * cta / G, w1 = words * (cta + 1) / G;
    const int e0 = int((long long)p.B * cta / G), e1 = int((long long)p.B * (cta + 1) / G);
    const int r0 = int((long long)p.rows * cta / G), r1 = int((long long)p.rows * (cta + 1) / G);
    // A thread's first word of a list is on its way before the batch has been looked at: whatever
    // the verdict, it lies inside the lists.
    const auto entry_of = [&](long long w) {
        return words <= 0x7FFFFFFF ? int(uint32_t(w) / uint32_t(wpr)) : int(w / wpr);
    };
    int4 ahead = make_int4(-1, -1, -1, -1);
    if (!RELEASE && w0 + tid < w1) {
        const int e = entry_of(w0 + tid), slot = p.slots[e];
        const int32_t* list = pool.tables + size_t(slot) * mb + size_t(w0 + tid - (long long)e * wpr) * vec;
        if (slot >= 0 && slot < pool.max_slots) {
            if (p.wide) ahead = *reinterpret_cast<const int4*>(list);
            else ahead.x = *list;
        }
    }

    // ---- what the batch needs, and whether it can be had
    const int tiles = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int head = pool.state[0], free = pool.state[1];
    int bad = 0;
    long long total_n = 0, total_move = 0;
    for (int t = 0; t < tiles; ++t) {
        const Entry x = load_entry<RELEASE>(p, t * kPlanThreads + tid, bad);
        if (x.slot >= 0 && (atomicOr(&sh.seen[x.slot >> 5], 1u << (x.slot & 31)) >> (x.slot & 31)) & 1u) bad |= kErrSlot;
        if (tiles == 1) {
            scan(x, 0, 0);
        } else {
            total_n += x.n;
            total_move += x.move;
        }
    }
    if (tiles == 1) {
        total_n = sh.start[kPlanThreads];
        total_move = sh.off[kPlanThreads];
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total_n += __shfl_xor_sync(kFull, total_n, o);
            total_move += __shfl_xor_sync(kFull, total_move, o);
        }
        if (lane == 0) {
            sh.warp[0][warp] = total_n;
            sh.warp[1][warp] = total_move;
        }
        __syncthreads();
        total_n = total_move = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            total_n += sh.warp[0][w];
            total_move += sh.warp[1][w];
        }
        __syncthreads();
    }
    if (bad) atomicOr(&sh.bad, bad);
    __syncthreads();
    bad = sh.bad;
    if (head < 0 || head >= N || free < 0 || free > N) bad |= kErrCtxLen;
    if (RELEASE) {
        if (total_move + free > N) bad |= kErrCtxLen;
    } else {
        if (total_n > p.out.num_tokens) bad |= kErrBatch;
        if (total_move > free) bad |= kErrOom;
    }
    if (bad && blockIdx.x == 0 && tid == 0) report(pool.err, bad);
    if (RELEASE && bad) return;

    // the i-th id from the ring's front (plan: taken) or end (release: given back)
    const auto place = [&](long long i) {
        i += (long long)head + (RELEASE ? free : 0);  // < 2 N
        return int(i < N ? i : i - N);
    };
    if (bad) {
        for (long long w = w0 * vec + tid; w < w1 * vec; w += kPlanThreads) p.out.block_tables[w] = -1;
        for (int e = e0 + tid; e < e1; e += kPlanThreads) {
            p.out.token_starts[e + 1] = p.out.ctx_lens[e] = 0;
            if (p.out.fill_blocks) p.out.fill_blocks[e] = -1;
        }
        if (cta == 0 && tid == 0) p.out.token_starts[0] = 0;
    } else {
        long long row0 = 0, off0 = 0;
        for (int t = 0; t < tiles; ++t) {
            const int first = t * kPlanThreads, end = min(p.B, first + kPlanThreads);
            if (tiles > 1) {
                int ignored = 0;
                scan(load_entry<RELEASE>(p, first + tid, ignored), row0, off0);
            }
            // tables
            const long long wa = max(w0, (long long)first * wpr), wb = min(w1, (long long)end * wpr);
            for (long long w = wa + tid; w < wb; w += kPlanThreads) {
                const int e = entry_of(w), c0 = int(w - (long long)e * wpr) * vec;
                const Entry x = sh.entry[e - first];
                const long long off = sh.off[e - first];
                int32_t* list = pool.tables + size_t(max(0, x.slot)) * mb + c0;
                if (RELEASE) {
                    for (int v = 0; v < vec; ++v) {
                        if (c0 + v >= x.move) break;
                        pool.ring[place(off + c0 + v)] = list[v];
                        list[v] = -1;
                    }
                    continue;
                }
                const int have = x.held + x.move;
                int4 id = make_int4(-1, -1, -1, -1);
                if (c0 + vec <= x.held) {
                    if (w == w0 + tid) id = ahead;
                    else if (p.wide) id = *reinterpret_cast<const int4*>(list);
                    else id.x = *list;
                } else if (c0 < have) {
                    int y[4] = {-1, -1, -1, -1};
                    for (int v = 0; v < vec; ++v) {
                        const int c = c0 + v;
                        if (c < x.held) y[v] = list[v];
                        else if (c < have) list[v] = y[v] = pool.ring[place(off + c - x.held)];
                    }
                    id = make_int4(y[0], y[1], y[2], y[3]);
                }
                if (p.wide) *reinterpret_cast<int4*>(p.out.block_tables + w * 4) = id;
                else p.out.block_tables[w] = id.x;
            }
            if (!RELEASE) {
                // a block of entry i: held before, or taken now
                const auto block = [&](int i, int c) {
                    const Entry& x = sh.entry[i];
                    return c < x.held ? pool.tables[size_t(x.slot) * mb + c] : pool.ring[place(sh.off[i] + c - x.held)];
                };
                for (int e = max(e0, first) + tid; e < min(e1, end); e += kPlanThreads) {
                    const Entry& x = sh.entry[e - first];
                    const int ctx = x.len + x.n;
                    p.out.token_starts[e + 1] = int(sh.start[e - first + 1]);
                    p.out.ctx_lens[e] = ctx;
                    if (p.out.fill_blocks)
                        p.out.fill_blocks[e] = x.n > 0 && (ctx & (pool.bs - 1)) == 0 ? block(e - first, (ctx >> pool.lg) - 1) : -1;
                }
                if (cta == 0 && tid == 0 && t == 0) p.out.token_starts[0] = 0;
                const int ra = max(r0, int(sh.start[0])), rb = min(r1, int(sh.start[kPlanThreads]));
                for (int r = ra + tid; r < rb; r += kPlanThreads) {
                    int lo = 0, hi = kPlanThreads - 1;  // the last entry that starts at or before r
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) / 2;
                        if (sh.start[mid] <= r) lo = mid;
                        else hi = mid - 1;
                    }
                    const Entry& x = sh.entry[lo];
                    const int pos = x.len + r - int(sh.start[lo]);
                    if (p.out.block_ids) p.out.block_ids[r] = block(lo, pos >> pool.lg);
                    if (p.out.offsets) p.out.offsets[r] = pos & (pool.bs - 1);
                    if (p.out.token_slots) p.out.token_slots[r] = x.slot;
                    if (p.out.positions) p.out.positions[r] = pos;
                }
            }
            row0 = sh.start[kPlanThreads];
            off0 = sh.off[kPlanThreads];
            __syncthreads();
        }
    }
    if (!RELEASE) {
        for (int r = max(r0, bad ? 0 : int(total_n)) + tid; r < r1; r += kPlanThreads) {
            if (p.out.block_ids) p.out.block_ids[r] = -1;
            if (p.out.offsets) p.out.offsets[r] = 0;
            if (p.out.token_slots) p.out.token_slots[r] = -1;
            if (p.out.positions) p.out.positions[r] = 0;
        }
    }
    if (bad || (total_move == 0 && !RELEASE)) return;

    // ---- the last CTA, when nobody reads them any more: the numbers that change
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        sh.last = atomicAdd(&pool.state[2], 1) == G - 1;
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    for (int e = tid; e < p.B; e += kPlanThreads) {
        int ignored = 0;
        const Entry x = load_entry<RELEASE>(p, e, ignored);
        if (x.slot < 0) continue;
        if (RELEASE) pool.held[x.slot] = pool.lens[x.slot] = 0;
        else if (x.move) pool.held[x.slot] = x.held + x.move;
    }
    if (tid == 0) {
        if (!RELEASE) pool.state[0] = int((head + total_move) % N);
        pool.state[1] = int(RELEASE ? free + total_move : free - total_move);
        pool.state[2] = 0;
    }
}

struct CommitParams {
    PoolView pool;
    const int32_t* slots;
    const int32_t* accepted;
    const int32_t* starts;
    const int32_t* ctx;
    int32_t B;
};

__global__ void __launch_bounds__(256) commit_kernel(const __grid_constant__ CommitParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int e = int(blockIdx.x * blockDim.x + threadIdx.x);
    if (e >= p.B) return;
    const int n = p.starts[e + 1] - p.starts[e], slot = p.slots[e];
    if (n <= 0) return;
    if (slot < 0 || slot >= p.pool.max_slots) {
        report(p.pool.err, kErrSlot);
        return;
    }
    const int keep = p.accepted ? p.accepted[e] : n, bs = p.pool.bs;
    const int64_t ctx = p.ctx[e], before = ctx - n, end = before + keep;
    const bool fine = keep >= 0 && keep <= n && before >= 0 && p.pool.lens[slot] == before &&
                      ctx <= int64_t(p.pool.held[slot]) * bs && !(p.pool.int8 && end % bs != 0 && end / bs != ctx / bs);
    if (fine) p.pool.lens[slot] = int(end);
    else report(p.pool.err, kErrCtxLen);
}

__global__ void after_plan_kernel() {}

int check_pool(const pkv_seq_pool* pool, PoolView* v) {
    if (!pool || !pool->tables || !pool->lens || !pool->held || !pool->ring || !pool->state) return PKV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(pool->tables) | reinterpret_cast<uintptr_t>(pool->lens) |
         reinterpret_cast<uintptr_t>(pool->held) | reinterpret_cast<uintptr_t>(pool->ring) |
         reinterpret_cast<uintptr_t>(pool->state) | reinterpret_cast<uintptr_t>(pool->err_word)) & 3u)
        return PKV_ERR_INVALID;
    if (pool->max_slots <= 0 || pool->max_blocks <= 0 || pool->num_blocks <= 0) return PKV_ERR_INVALID;
    if ((pool->block_size != 16 && pool->block_size != 64) || pool->max_slots > kMaxPoolSlots) return PKV_ERR_UNSUPPORTED;
    if (int64_t(pool->max_blocks) * pool->block_size >= (int64_t(1) << 31) - 65536) return PKV_ERR_INVALID;
    *v = PoolView{pool->tables, pool->lens, pool->held, pool->ring, pool->state, pool->err_word,
                  pool->max_slots, pool->max_blocks, pool->num_blocks, pool->block_size, pool->block_size == 16 ? 4 : 6, pool->int8};
    return PKV_OK;
}

// CTAs for this many 4-byte words of output: about four a thread, two CTAs a SM at most.
unsigned plan_grid(int64_t words) {
    return unsigned(std::clamp<int64_t>((words + kPlanThreads * 4 - 1) / (kPlanThreads * 4), 1, 2 * 152));
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_plan_batch(const pkv_seq_pool* pool, const int32_t* slots, const int32_t* counts, int32_t B, const pkv_plan* plan,
                   void* stream) {
    PlanParams p;
    int st = check_pool(pool, &p.pool);
    if (st != PKV_OK) return st;
    if (!plan || B < 0 || B > 65535 || plan->num_tokens < 0 || plan->max_tokens < 0 || plan->max_tokens > plan->num_tokens)
        return PKV_ERR_INVALID;
    if (plan->num_tokens >= 0x7FFF0000) return PKV_ERR_INVALID;  // a CTA's row counters would wrap
    if (B == 0) return PKV_OK;
    if (!slots || !plan->token_starts || !plan->block_tables || !plan->ctx_lens) return PKV_ERR_INVALID;
    if (!aligned4(slots) || !aligned4(counts) || !aligned4(plan->token_starts) || !aligned4(plan->block_tables) ||
        !aligned4(plan->ctx_lens) || !aligned4(plan->fill_blocks) || !aligned4(plan->block_ids) ||
        !aligned4(plan->offsets) || !aligned4(plan->token_slots) || !aligned4(plan->positions))
        return PKV_ERR_INVALID;
    p.out = *plan;
    p.slots = slots;
    p.counts = counts;
    p.B = B;
    const int arrays = (plan->block_ids != nullptr) + (plan->offsets != nullptr) + (plan->token_slots != nullptr) +
                       (plan->positions != nullptr);
    p.rows = arrays ? plan->num_tokens : 0;
    p.wide = pool->max_blocks % 4 == 0 && aligned16(pool->tables) && aligned16(plan->block_tables);
    const dim3 grid(plan_grid(int64_t(B) * pool->max_blocks + int64_t(p.rows) * arrays));
    auto s = static_cast<cudaStream_t>(stream);
    if ((st = launch(plan_kernel<false>, grid, dim3(kPlanThreads), 0, s, p)) != PKV_OK) return st;
    if (g_pdl.load(std::memory_order_relaxed)) {
        after_plan_kernel<<<1, 1, 0, s>>>();
        return cuda_status(cudaGetLastError());
    }
    return PKV_OK;
}

int pkv_commit_batch(const pkv_seq_pool* pool, const int32_t* slots, const int32_t* accepted, int32_t B,
                     const pkv_plan* plan, void* stream) {
    CommitParams p;
    const int st = check_pool(pool, &p.pool);
    if (st != PKV_OK) return st;
    if (!plan || B < 0 || B > 65535) return PKV_ERR_INVALID;
    if (B == 0) return PKV_OK;
    if (!slots || !plan->token_starts || !plan->ctx_lens || !aligned4(slots) || !aligned4(accepted) ||
        !aligned4(plan->token_starts) || !aligned4(plan->ctx_lens))
        return PKV_ERR_INVALID;
    p.slots = slots;
    p.accepted = accepted;
    p.starts = plan->token_starts;
    p.ctx = plan->ctx_lens;
    p.B = B;
    return launch(commit_kernel, dim3(unsigned(B + 255) / 256), dim3(256), 0, static_cast<cudaStream_t>(stream), p);
}

int pkv_release_batch(const pkv_seq_pool* pool, const int32_t* slots, int32_t B, void* stream) {
    PlanParams p;
    const int st = check_pool(pool, &p.pool);
    if (st != PKV_OK) return st;
    if (B < 0 || B > 65535) return PKV_ERR_INVALID;
    if (B == 0) return PKV_OK;
    if (!slots || !aligned4(slots)) return PKV_ERR_INVALID;
    p.out = pkv_plan{};
    p.slots = slots;
    p.counts = nullptr;
    p.B = B;
    p.rows = 0;
    p.wide = 0;
    return launch(plan_kernel<true>, dim3(plan_grid(int64_t(B) * pool->max_blocks)), dim3(kPlanThreads), 0,
                  static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
