// Rotary positions on three axes of a batch's tokens, from their sequences'
// segments of text and of t x h x w grids (pkv_axis_positions).
//
// A CTA has up to kPosTokens new tokens of one sequence. It walks through the sequence's
// segments a tile of 256 at a time: two prefix sums (tokens, positions) give
// each segment's first token and base, and the CTA's tokens that fall into the
// tile find their segment by bisection in shared memory. It ends with the tile that
// holds its last token, or with the list; tokens behind that are text.
//
// Bound by latency: 3.0 us in a graph for 128 single tokens behind 24 segments, 4.9 us
// for 53600 tokens of 8 prompts with 48 segments (0.65 MB; 0.1 us at the memory's rate):
// launch, lengths -> number of segments -> segments -> two sums, then eight
// steps of the bisection a token.
#include "batch.cuh"
#include "host.h"

namespace pkv {

constexpr int kErrSegment = 128;
constexpr int kPosThreads = 256;
constexpr int kPosTokens = 1024;
constexpr int kMaxContext = 0x7FFF0000;  // as any cache's: a CTA's token counters pass it without wrapping

struct PositionParams {
    const int32_t* starts;
    const int32_t* ctx;
    const int4* segments;
    const int32_t* num_segments;
    const int32_t* rows;
    int32_t* out;
    int64_t axis_stride;
    int32_t* err;
    int32_t num_tokens, max_tokens, num_rows, max_segments;
};

__device__ __forceinline__ int to_position(long long x) { return int(min(x, 0x7FFFFFFFll)); }

__global__ void __launch_bounds__(kPosThreads) positions_kernel(const __grid_constant__ PositionParams p) {
    __shared__ int4 s_seg[kPosThreads];
    __shared__ long long s_first[kPosThreads + 1], s_base[kPosThreads + 1], s_warp[2][kPosThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
    const bool reporter = blockIdx.x == 0 && tid == 0;
    const int row0 = p.starts[b], end = p.starts[b + 1], n = end - row0, ctx = p.ctx[b];
    if (row0 < 0 || end < row0 || end > p.num_tokens || n > p.max_tokens) {
        if (reporter) report(p.err, kErrBatch);
        return;
    }
    if (n == 0) return;
    if (ctx < n || ctx >= kMaxContext) {
        if (reporter) report(p.err, kErrCtxLen);
        return;
    }
    const int r = p.rows ? p.rows[b] : b;
    if (r < 0 || r >= p.num_rows) {
        if (reporter) report(p.err, kErrSlot);
        return;
    }
    const int count = p.num_segments[r];
    if (count < 0 || count > p.max_segments) {
        if (reporter) report(p.err, kErrSegment);
        return;
    }
    const long long chunk = (long long)blockIdx.x * kPosTokens;
    if (chunk >= n) return;
    const int t0 = ctx - n + int(chunk), t1 = t0 + min(ctx - t0, kPosTokens);  // this CTA's tokens
    const auto write = [&](int tok, long long x, long long y, long long z) {
        int32_t* o = p.out + row0 + (tok - (ctx - n));
        o[0] = to_position(x);
        o[p.axis_stride] = to_position(y);
        o[2 * p.axis_stride] = to_position(z);
    };
    long long first = 0, base = 0;  // of the tile
    for (int s0 = 0; s0 < count && first < t1; s0 += kPosThreads) {
        int4 g = make_int4(0, 0, 0, 0);
        if (s0 + tid < count) g = p.segments[size_t(r) * p.max_segments + s0 + tid];
        long long tokens = 0, moves = 0;
        if (g.y == 0 && g.z == 0) {
            const bool fine = g.x >= 0 && g.w >= 0;
            tokens = moves = fine ? g.x : 0;
            if (!fine) report(p.err, kErrSegment);  // (any CTA: the first one ends with its own last token)
        } else {
            const long long area = (long long)g.y * g.z, frames = ((long long)g.x - 1) * g.w;
            const bool fine = g.x >= 0 && g.y > 0 && g.z > 0 && g.w >= 0 && area <= 0x7FFFFFFF &&
                              area * g.x <= 0x7FFFFFFF && frames <= 0x7FFFFFFF;
            if (!fine) report(p.err, kErrSegment);
            if (fine && g.x > 0) {
                tokens = area * g.x;
                moves = max(frames, (long long)max(g.y, g.z) - 1) + 1;
            }
        }
        long long a = tokens, m = moves;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, a, o), v = __shfl_up_sync(kFull, m, o);
            if (lane >= o) {
                a += u;
                m += v;
            }
        }
        if (lane == 31) {
            s_warp[0][warp] = a;
            s_warp[1][warp] = m;
        }
        __syncthreads();
        long long a0 = first, m0 = base;
        for (int w = 0; w < warp; ++w) {
            a0 += s_warp[0][w];
            m0 += s_warp[1][w];
        }
        s_seg[tid] = g;
        s_first[tid] = a0 + a - tokens;
        s_base[tid] = m0 + m - moves;
        if (tid == kPosThreads - 1) {
            s_first[kPosThreads] = a0 + a;
            s_base[kPosThreads] = m0 + m;
        }
        __syncthreads();
        const int ta = int(max((long long)t0, s_first[0])), tb = int(min((long long)t1, s_first[kPosThreads]));
        for (int tok = ta + tid; tok < tb; tok += kPosThreads) {
            int lo = 0, hi = kPosThreads - 1;  // the last segment that starts at or before tok
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_first[mid] <= tok) lo = mid;
                else hi = mid - 1;
            }
            const int4 s = s_seg[lo];
            const int i = tok - int(s_first[lo]);
            const long long at = s_base[lo];
            if (s.y == 0) {
                write(tok, at + i, at + i, at + i);
            } else {
                const int area = s.y * s.z, f = i / area, rest = i - f * area, y = rest / s.z;
                write(tok, at + (long long)f * s.w, at + y, at + rest - y * s.z);
            }
        }
        first = s_first[kPosThreads];
        base = s_base[kPosThreads];
        __syncthreads();
    }
    // (`first` may be any 64-bit number: the list's tokens need not fit a context)
    for (int tok = int(min((long long)t1, max((long long)t0, first))) + tid; tok < t1; tok += kPosThreads) {
        const long long x = base + (tok - first);
        write(tok, x, x, x);
    }
}

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_axis_positions(const pkv_batch_desc* batch, const int32_t* segments, const int32_t* num_segments,
                                  int32_t num_rows, int32_t max_segments, const int32_t* rows, int32_t* positions,
                                  int64_t axis_stride, int32_t* err_word, void* stream) {
    if (!batch || batch->B < 0 || batch->B > 65535 || batch->num_tokens < 0 || batch->max_tokens < 0 ||
        batch->max_tokens > batch->num_tokens || num_rows < 0 || max_segments < 0 || max_segments > 1 << 30)
        return PKV_ERR_INVALID;
    if (batch->B == 0 || batch->num_tokens == 0 || batch->max_tokens == 0) return PKV_OK;
    if (!batch->token_starts || !batch->ctx_lens || !num_segments || !positions || (max_segments > 0 && !segments))
        return PKV_ERR_INVALID;
    if (!aligned16(segments) || ((reinterpret_cast<uintptr_t>(batch->token_starts) | reinterpret_cast<uintptr_t>(batch->ctx_lens) |
                                  reinterpret_cast<uintptr_t>(num_segments) | reinterpret_cast<uintptr_t>(rows) |
                                  reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(err_word)) & 3u))
        return PKV_ERR_INVALID;
    if (axis_stride < batch->num_tokens || num_rows == 0 || (!rows && num_rows < batch->B)) return PKV_ERR_INVALID;
    PositionParams p;
    p.starts = batch->token_starts;
    p.ctx = batch->ctx_lens;
    p.segments = reinterpret_cast<const int4*>(segments);
    p.num_segments = num_segments;
    p.rows = rows;
    p.out = positions;
    p.axis_stride = axis_stride;
    p.err = err_word;
    p.num_tokens = batch->num_tokens;
    p.max_tokens = batch->max_tokens;
    p.num_rows = num_rows;
    p.max_segments = max_segments;
    const dim3 grid(unsigned((int64_t(batch->max_tokens) + kPosTokens - 1) / kPosTokens), unsigned(batch->B));
    return launch(positions_kernel, grid, dim3(kPosThreads), 0, static_cast<cudaStream_t>(stream), p);
}
