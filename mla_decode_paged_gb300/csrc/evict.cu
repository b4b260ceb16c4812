// Eviction from the paged cache by accumulated attention weight.
//
// What it computes: request r of L tokens keeps n = min(L, max(budget, 0))
// of them: its last min(recent, n), its first min(sinks, the rest), and for
// the remaining m the tokens in between with the largest weights (NaN as
// -inf, equal weights by the lowest position).  Kept tokens stay in order;
// the page list becomes every request's kept rows, then the freed rows.
//
// The m-th largest weight is found by radix selection on an order-preserving
// 32-bit key (11 + 11 + 10 bits, a shared histogram a pass), then one pass
// in position order places every token by a block scan.
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;

struct EvictArgs {
    const int32_t *pages, *indptr, *budgets;
    const float *weights;
    int64_t num_pages;
    int R, budget, recent, sinks;
    int32_t *pages_out, *indptr_out;
    float *weights_out;
};

// Larger weight <=> larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
    w = w != w ? __int_as_float(0xff800000) : w + 0.f;
    const uint32_t u = __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int kept_tokens(const EvictArgs &a, int r, int len) {
    const int b = a.budgets ? __ldg(a.budgets + r) : a.budget;
    return b < 0 ? 0 : b < len ? b : len;
}

// Sum of v over the block, to every thread.
__device__ long long block_sum(long long v, long long *red) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    long long t = red[threadIdx.x & 31];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    return t;
}

// Exclusive prefix sum over the block of v; the block's sum in *total.
__device__ uint32_t block_scan(uint32_t v, uint32_t *red, uint32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    uint32_t w = red[lane], s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return x - v + __shfl_sync(0xffffffffu, s - w, warp);
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t red[32];
    __shared__ long long red64[32];
    __shared__ uint32_t pick[2];
    const int r = blockIdx.x, tid = threadIdx.x;

    // Kept and freed tokens of the requests before this one, kept of all.
    long long kept_before = 0, len_before = 0, kept_total = 0;
    for (int i = tid; i < a.R; i += kThreads) {
        int base;
        const int len = request_len(a.indptr, i, a.num_pages, &base), k = kept_tokens(a, i, len);
        kept_total += k;
        if (i < r) {
            kept_before += k;
            len_before += len;
        }
    }
    kept_before = block_sum(kept_before, red64);
    len_before = block_sum(len_before, red64);
    kept_total = block_sum(kept_total, red64);
    int base;
    const int len = request_len(a.indptr, r, a.num_pages, &base);
    const int kept = kept_tokens(a, r, len);
    if (tid == 0) {
        if (r == 0) a.indptr_out[0] = 0;
        a.indptr_out[r + 1] = (int32_t)(kept_before + kept);
    }
    const int recent = a.recent < kept ? a.recent : kept;
    const int sinks = a.sinks < kept - recent ? a.sinks : kept - recent;
    const int lo = sinks, hi = len - recent;   // the tokens that may go
    int m = kept - recent - sinks;             // how many of them stay
    const float *w = a.weights + base;

    // The m-th largest key T of [lo, hi), and how many keys equal to T stay.
    uint32_t T = 0, ties = 0;
    const bool all = m >= hi - lo;
    if (m > 0 && !all) {
        uint32_t need = (uint32_t)m, mask = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024u : 2048u;
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kThreads) {
                const uint32_t key = weight_key(__ldg(w + i));
                if ((key & mask) == T) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            // Bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t.
            const uint32_t b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
            const uint32_t n1 = hist[b1], n0 = hist[b0];
            uint32_t total;
            const uint32_t above = block_scan(n1 + n0, red, &total);
            if (above < need && need <= above + n1) {
                pick[0] = b1;
                pick[1] = need - above;
            } else if (above + n1 < need && need <= above + n1 + n0) {
                pick[0] = b0;
                pick[1] = need - above - n1;
            }
            __syncthreads();
            T |= pick[0] << shift;
            need = pick[1];
            mask |= (bins - 1) << shift;
        }
        ties = need;
    }

    // Placement, in position order.
    long long out_kept = kept_before, out_freed = kept_total + (len_before - kept_before);
    uint32_t ties_seen = 0;
    for (int c = 0; c < len; c += kThreads) {
        const int i = c + tid;
        uint32_t sure = 0, tie = 0;
        float wi = 0.f;
        if (i < len) {
            wi = __ldg(w + i);
            if (i < lo || i >= hi || all) sure = 1;
            else if (m > 0) {
                const uint32_t key = weight_key(wi);
                sure = key > T;
                tie = key == T;
            }
        }
        uint32_t total;
        const uint32_t before = block_scan(sure | tie << 16, red, &total);
        const uint32_t sure_before = before & 0xffff, tie_before = ties_seen + (before >> 16);
        const uint32_t ties_chunk0 = ties_seen < ties ? ties_seen : ties;
        const uint32_t ties_here = tie_before < ties ? tie_before : ties;
        const uint32_t rank = sure_before + ties_here - ties_chunk0;   // kept tokens of this chunk before i
        const bool keep = sure || (tie && tie_before < ties);
        if (i < len) {
            const long long at = keep ? out_kept + rank : out_freed + (tid - rank);
            if (at < a.num_pages) {
                a.pages_out[at] = __ldg(a.pages + base + i);
                a.weights_out[at] = keep ? wi : 0.f;
            }
        }
        ties_seen += total >> 16;
        const uint32_t ties_now = ties_seen < ties ? ties_seen : ties;
        const uint32_t chunk_kept = (total & 0xffff) + ties_now - ties_chunk0;
        const int n = len - c < kThreads ? len - c : kThreads;
        out_kept += chunk_kept;
        out_freed += n - (int)chunk_kept;
    }
}

}  // namespace

cudaError_t kv_evict_launch(const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R, const float *weights,
                            const int32_t *budgets, int budget, int recent, int sinks, int32_t *pages_out,
                            int32_t *indptr_out, float *weights_out, cudaStream_t st) {
    if (R == 0) return cudaMemsetAsync(indptr_out, 0, sizeof(int32_t), st);
    EvictArgs a = {};
    a.pages = pages;
    a.indptr = indptr;
    a.budgets = budgets;
    a.weights = weights;
    a.num_pages = num_pages;
    a.R = R;
    a.budget = budget;
    a.recent = recent;
    a.sinks = sinks;
    a.pages_out = pages_out;
    a.indptr_out = indptr_out;
    a.weights_out = weights_out;
    evict_kernel<<<R, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t evict_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
