// How a persistent grid shares a ragged batch's token tiles: equal, contiguous
// ranges of them, walked by every role of a block on its own.
//
// The arguments' struct A has the page list's indptr and num_pages, the
// requests R and the shares of the grid `virt`.
#pragma once

#include "common.cuh"

namespace mla {

// A CTA's (a pair's) tiles of TOKENS in order; every role, a whole warp, walks
// them on its own (uniform loads).
template <int TOKENS>
struct Walk {
    int r, t, ntiles, len, base, left, unit;
    bool first;     // the tile is its unit's first in this CTA

    // `start`: this CTA's first request, its first tile there, tiles in all (find_start).
    template <class A>
    __device__ void init(const A &a, const int (&start)[3]) {
        r = start[0];
        t = start[1];
        left = start[2];
        unit = 0;
        first = true;
        if (left > 0) open(a);
    }
    template <class A>
    __device__ void open(const A &a) {
        len = request_len(a.indptr, r, a.num_pages, &base);
        ntiles = (len + TOKENS - 1) / TOKENS;
    }
    __device__ bool valid() const { return left > 0; }
    __device__ bool last() const { return left == 1 || t + 1 == ntiles; }
    // Past n tiles, or past the last.
    template <class A>
    __device__ __forceinline__ void skip(const A &a, int n) {
        if (left > n && t + n < ntiles) {
            t += n;
            left -= n;
            first = false;
            return;
        }
#pragma unroll 1
        for (int k = 0; k < n && left > 0; ++k) next(a);
    }
    template <class A>
    __device__ void next(const A &a) {
        --left;
        first = false;
        if (++t < ntiles || left <= 0) return;
        t = 0;
        first = true;
        ++unit;
        ++r;        // at least one more tile is to come, so a request with tokens follows
        open(a);
        // Empty requests are passed over 32 at a time: one by one 2^24 of them
        // took 3.5 s, more than the roles wait for each other.
        while (ntiles == 0 && r + 1 < a.R) {
            const int mine = r + 1 + (threadIdx.x & 31);
            int b = 0;
            const int n = mine < a.R ? request_len(a.indptr, mine, a.num_pages, &b) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
            if (some == 0) {
                r = min(r + 32, a.R - 1);
                continue;
            }
            const int src = __ffs(some) - 1;
            r += 1 + src;
            len = __shfl_sync(0xffffffffu, n, src);
            base = __shfl_sync(0xffffffffu, b, src);
            ntiles = (len + TOKENS - 1) / TOKENS;
        }
    }
};

// Share v's range of the batch's tiles -> start.  Run by all THREADS of the
// block (it passes a barrier before it reads start); start[0] and start[1] are
// 0 before.  Requests that share entries (a bad indptr only) count up to what
// the page list could hold.
template <int TOKENS, int THREADS, class A>
__device__ void find_start(const A &a, int (&start)[3], int v) {
    __shared__ long long part[THREADS / 32 + 1];
    __shared__ uint32_t part32[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto tiles_of = [&](int r) {
        int base;
        return (request_len(a.indptr, r, a.num_pages, &base) + TOKENS - 1) / TOKENS;
    };
    const int64_t most = a.num_pages / TOKENS + a.R;     // tiles
    // Shares that differ by one at most, the larger ones first.
    const auto range = [&](uint32_t total, uint32_t &lo, uint32_t &n) {
        const uint32_t each = total / (uint32_t)a.virt, more = total - each * a.virt;
        lo = each * v + min((uint32_t)v, more);
        n = each + ((uint32_t)v < more ? 1 : 0);
    };
    if (a.R <= THREADS && most * a.R < INT32_MAX) {      // in one step, in 32 bits
        const uint32_t n = tid < a.R ? tiles_of(tid) : 0;
        uint32_t incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        if (lane == 31) part32[warp] = incl;
        __syncthreads();
        const uint32_t w = lane < THREADS / 32 ? part32[lane] : 0;
        const uint32_t at = incl - n + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
        uint32_t lo, count;
        range(min(__reduce_add_sync(0xffffffffu, w), (uint32_t)most), lo, count);
        if (tid == 0) start[2] = (int)count;
        if (at <= lo && lo < at + n) {
            start[0] = tid;
            start[1] = (int)(lo - at);
        }
        __syncthreads();
        return;
    }
    int mine = 0;
    long long sum = 0;
    for (int r = tid; r < a.R; r += THREADS) {
        const int n = tiles_of(r);
        if (r == tid) mine = n;
        sum += n;
    }
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < THREADS / 32; ++w) total += part[w];
    uint32_t first, count;
    range((uint32_t)min(total, (long long)most), first, count);
    const int64_t lo = first;
    if (tid == 0) start[2] = (int)count;
    int64_t before = 0;   // tiles of the requests before this chunk
    for (int r0 = 0; r0 < a.R && before <= lo; r0 += THREADS) {
        const int r = r0 + tid;
        const int n = r0 == 0 ? mine : r < a.R ? tiles_of(r) : 0;
        int incl = n;
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        __syncthreads();
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        int64_t at = before;
        int64_t all = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) at += part[w];
            all += part[w];
        }
        at += incl - n;
        if (n > 0 && at <= lo && lo < at + n) {
            start[0] = r;
            start[1] = (int)(lo - at);
        }
        before += all;
    }
    __syncthreads();
}

}  // namespace mla
