// The tokens that each query row attends to: the blocks of best score, as a
// page list a row.
//
// What it computes: row b = r * qlen + tq sees the first n tokens of request
// r, in nb = ceil(n / block) blocks of `block` tokens, of which k = min(nb,
// topk) stay: the last min(recent, k), the first min(sinks, the rest), and
// for the remaining m the blocks in between with the largest maximum of their
// tokens' scores (NaN as -inf, equal ones by the lowest position).  The rows
// of pages of the kept blocks' tokens are written one list after another, in
// order, with an indptr; -1 behind them.  How many tokens a row keeps does
// not depend on its scores (only its last block may be cut short, and with
// blocks of more than one token that stays).
//
// Bound by the 4 bytes a score that are read for many long rows, by the chain
// of dependent steps for one: 64 requests of 1K to 8K tokens 8.6 us, one of
// 128K 14, 512 rows of 4K to 32K by blocks of 64 19 (2.5 TB/s).
//
// Design: a cluster of thread blocks per row, as many of them as it takes to
// hold it (the others end at once), each with a contiguous slice of its token
// blocks: 8,192 or 16,384 keys (order-preserving 32-bit images of the scores), formed in
// shared memory from coalesced reads, then up to 32 neighbours in a thread's
// registers, so that one prefix sum over the threads places what stays (with
// 32 lanes of a warp side by side every key needed its ballots: three times
// the instructions).  A longer slice is taken in rounds of that size, read
// again for every step.  The m-th largest key: a histogram of the first 11
// bits, summed over the cluster through distributed shared memory, names the
// bin that holds it; one warp finds it bit by bit among that bin's keys, up
// to 1,024 of them.  More take another histogram, of the next 11 bits, and
// the same search, then one of the last 10, unless all of them are equal.
// (First digits of 12 bits: a row of 32K 13.7 us and not 12.1, as twice the
// bins have to be summed over the cluster.)  The kept blocks are listed in shared memory and their tokens' pages copied from
// there, coalesced.
//
// A row's place in the output is the sum of the kept tokens of the rows
// before it: each cluster sums over all of them up to 1,024 rows, a small
// kernel writes the indptr first for more.
#include <algorithm>
#include <atomic>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kBins = 2048;
constexpr int kLong = 8192, kShort = 4096;     // token blocks a thread block holds, of 512 and more threads (or twice these), of 256
constexpr int kCand = 1024, kFew = 512;    // keys of a bin, of a row, that one warp searches
constexpr int kCounted = 1024;     // rows whose kept tokens every cluster counts itself

struct SelectArgs {
    const float *scores;
    const int32_t *pages, *indptr;
    int64_t num_pages, capacity;
    uint32_t over_qlen;             // 2^32 / qlen, rounded up
    int R, qlen, topk, log_block, recent, sinks;
    bool causal, scanned;           // scanned: indptr_out is there
    int32_t *pages_out, *indptr_out;
};

// A query row: its request and place there, its first entry, the tokens it
// sees, their blocks, the blocks and tokens it keeps.
struct Row {
    int r, tq, base, seen, blocks, kept, tokens;
};
__device__ __forceinline__ Row row_of(const SelectArgs &a, int b) {
    Row x;
    x.r = a.qlen == 1 ? b : (int)__umulhi((uint32_t)b, a.over_qlen);       // b below 2^24
    x.tq = b - x.r * a.qlen;
    int begin = a.indptr[x.r], end = a.indptr[x.r + 1];
    if (begin < 0 || end < begin || end > a.num_pages) {        // as request_len does
        flag(MLA_DEV_BAD_INDPTR);
        begin = end = 0;
    }
    x.base = begin;
    x.seen = a.causal ? max(0, end - begin - a.qlen + x.tq + 1) : end - begin;
    x.blocks = (x.seen + (1 << a.log_block) - 1) >> a.log_block;
    x.kept = min(x.blocks, a.topk);
    // Where some stay, the last one does: all whole but that.
    x.tokens = x.kept == 0 ? 0 : x.seen - ((x.blocks - x.kept) << a.log_block);
    return x;
}

// Where key i of a round lies: eight neighbours and a gap, so that threads
// that read their neighbours fall in different banks.
__host__ __device__ constexpr int place(int i) { return i + (i >> 3); }

template <int THREADS, int ROUND, bool CLUSTER>
struct __align__(16) Shared {
    uint32_t key[place(ROUND)];     // a round's keys; then the blocks that stay, in order
    uint32_t hist[kBins];
    uint32_t sums[CLUSTER ? kBins : 4];     // of this block's share of the bins, over the cluster
    uint32_t cand[kCand], all[CLUSTER ? kCand : 4];     // keys of the m-th largest's bin: this block's, the cluster's
    uint32_t red[2][32], scan[2][32];
    uint32_t least, most;           // of this block's keys of that bin
    uint32_t ncand;
    uint32_t sum[2];                // this block's sure blocks and ties, for the cluster
    uint32_t pick[4];
};

// Thread blocks that share a row of so many tokens, as a power of two up to log_cs.
__device__ __forceinline__ int blocks_for(int tokens, int log_cs, int slice) {
    int le = 0;
#pragma unroll 1
    while (le < log_cs && (tokens >> le) > slice) ++le;
    return le;
}

// The need-th largest of the n keys at p (zeros do not count), which agree
// with T above their lowest `bits` bits (run by a warp): a value T that
// exactly `need` of them reach, and true, or the key itself, how many of it
// belong to them, and false.
template <int N>
__device__ __forceinline__ bool search(const uint32_t *p, uint32_t n, int bits, uint32_t &T, uint32_t &need) {
    const int lane = threadIdx.x & 31;
    uint32_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane + 32 * i < n ? p[lane + 32 * i] : 0;
    if (bits == 32) {       // the bits that all of them share
        uint32_t ones = ~0u, any = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ones &= x[i] != 0 ? x[i] : ~0u;
            any |= x[i];
        }
        ones = __reduce_and_sync(0xffffffffu, ones);
        any = __reduce_or_sync(0xffffffffu, any);
        bits = 32 - __clz(ones ^ any);
        T = bits < 32 ? any & ~((1u << bits) - 1) : 0;
    }
#pragma unroll 1
    for (int bit = bits - 1; bit >= 0; --bit) {
        const uint32_t t = T | 1u << bit;
        uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < N; ++i) c[i & 3] += x[i] >= t;
        const uint32_t all = __reduce_add_sync(0xffffffffu, (c[0] + c[1]) + (c[2] + c[3]));
        if (all < need) continue;
        T = t;
        if (all == need) return true;
    }
    uint32_t above = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) above += x[i] > T;
    need -= __reduce_add_sync(0xffffffffu, above);
    return false;
}

// Sum of x over the threads before this one and over all of the block's, by
// way of `totals`, which is free again after the block's next barrier but one.
// (Not inlined, as what else is run more than once: SMs of one GPC that start
// together wait for each other's instructions.)
template <int THREADS>
__device__ __noinline__ uint2 block_sums(uint32_t x, uint32_t *totals) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) totals[warp] = incl;
    __syncthreads();
    const uint32_t t = lane < THREADS / 32 ? totals[lane] : 0;
    return make_uint2(incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0), __reduce_add_sync(0xffffffffu, t));
}

// Lanes that differ in bit S: the maxima of the 16 >> S values that both hold, half of them in each.
template <int S>
__device__ __forceinline__ void halve(float (&v)[16]) {
    const bool up = threadIdx.x >> S & 1;
#pragma unroll
    for (int i = 0; i < 8 >> S; ++i) {
        const float keep = up ? v[i + (8 >> S)] : v[i], give = up ? v[i] : v[i + (8 >> S)];
        v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 1 << S));
    }
}

// Keys of the token blocks r0 .. s1 - 1 of a row, a round at most, into their
// places: those of lo .. hi - 1, of `seen` tokens at w; 0 elsewhere, up to
// `held` places.
template <int THREADS, int ROUND, bool BLOCKED>
__device__ __noinline__ void load_keys(uint32_t *key, const float *w, int r0, int s1, int lo, int hi, int seen, int held,
                                       int lb) {
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int f0 = max(lo - r0, 0), f1 = min(hi - r0, min(ROUND, s1 - r0));
    __syncthreads();        // the histogram's zeros; the round before has been read
    if (!BLOCKED) {
        const float *from = w + r0 + tid;
        uint32_t *to = key + place(tid);
        const uint32_t width = max(f1 - f0, 0);
#pragma unroll 1
        for (int i0 = tid - f0; i0 < held - f0; i0 += 8 * THREADS, from += 8 * THREADS, to += 8 * place(THREADS)) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (uint32_t)(i0 + THREADS * j) < width ? from[THREADS * j] : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t x = weight_key(v[j]);
                if (i0 + THREADS * j < held - f0) to[place(THREADS) * j] = (uint32_t)(i0 + THREADS * j) < width ? x : 0;
            }
        }
    } else {
        // Block maxima (NaN ignored: as -inf).  A warp holds 16 chunks of 32
        // tokens, one a register.  Each of up to four steps joins lanes that
        // differ in one bit and leaves either with half of the chunks, so that
        // 16 maxima cost 15 exchanges; further bits of larger blocks are joined
        // one by one (a join of every chunk on its own: 512 rows by blocks of
        // 16 51 us).
#pragma unroll 1
        for (int i = tid; i < held; i += THREADS) key[place(i)] = 0;
        __syncthreads();
        const int t1 = min((r0 + f1) << lb, seen);
        const int to_last = lb < 5 ? 32 : 1 << (9 - lb);       // the last of the bits joined one by one
        // Chunks chunk .. chunk + kept - 1 end up in this lane (kept 0: in another too, which writes).
        const int each = max(16 >> lb, 1), chunk = __brev(lane) >> 28 & ~(each - 1), off = lb < 5 ? lane >> lb << lb : 0;
        const int kept = lb >= 5 && (lane & 32 - to_last) != 0 ? 0 : each;
#pragma unroll 1
        for (int t0 = ((r0 + f0) << lb) + 32 * 16 * warp; t0 < t1; t0 += 32 * 16 * kWarps) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int t = t0 + 32 * k + lane;
                v[k] = t < t1 ? w[t] : -INFINITY;
            }
            halve<0>(v);
            if (lb >= 2) halve<1>(v);
            if (lb >= 3) halve<2>(v);
            if (lb >= 4) halve<3>(v);
#pragma unroll 1
            for (int d = 16; d >= to_last; d >>= 1) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], d));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = t0 + 32 * (chunk + k) + off;
                if (k < kept && t < t1) key[place((t >> lb) - r0)] = weight_key(v[k]);
            }
        }
    }
    __syncthreads();
}

// 2^log_cs blocks (a cluster) per row.
template <int THREADS, int ROUND, bool CLUSTER, bool BLOCKED>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (BLOCKED ? 4 : 5) : 1024 / THREADS) select_kernel(const SelectArgs a, int log_cs) {
    constexpr int kWarps = THREADS / 32, kOwn = kBins / THREADS;       // bins a thread sums
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared<THREADS, ROUND, CLUSTER> &sh = *reinterpret_cast<Shared<THREADS, ROUND, CLUSTER> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = CLUSTER ? block_rank() : 0;
    const int rows = a.R * a.qlen, b = CLUSTER ? blockIdx.x >> log_cs : blockIdx.x, lb = BLOCKED ? a.log_block : 0;
    grid_wait();
    const Row row = row_of(a, b);
    const uint32_t my_tokens = !a.scanned && tid < rows ? (uint32_t)row_of(a, tid).tokens : 0;      // its loads beside the row's
    // The blocks past those that hold the row end (a cluster barrier waits for
    // running threads only).
    const int le = CLUSTER ? blocks_for(row.seen, log_cs, ROUND) : 0;
    const uint32_t E = 1u << le;
    if (rank >= E) return;
    const bool one = !CLUSTER || le == 0;
    const int recent = min(a.recent, row.kept), sinks = min(a.sinks, row.kept - recent);
    const int lo = sinks, hi = row.blocks - recent;     // the blocks that may go
    const int m = row.kept - recent - sinks;            // how many of them stay
    const bool select = m > 0 && m < hi - lo;           // the same in every block of the cluster
    const float *w = a.scores + (int64_t)row.tq * a.num_pages + row.base;

    // This block's slice, in rounds.  Key 0: none that may go.
    const int slice = (((row.blocks + (int)E - 1) >> le) + 31) / 32 * 32;
    const int s0 = (int)min((int64_t)slice * rank, (int64_t)row.blocks), s1 = min(slice, row.blocks - s0) + s0;
    const int rounds = (s1 - s0 + ROUND - 1) / ROUND;
    // A round's keys are `per` neighbours in each thread, as few as hold the longest round.
    const int longest = min(s1 - s0, ROUND), per = max(1, (longest + THREADS - 1) / THREADS);
    const int held = THREADS * per;     // places of a round's keys; those past the round hold 0
    const auto load = [&](int q) { load_keys<THREADS, ROUND, BLOCKED>(sh.key, w, s0 + q * ROUND, s1, lo, hi, row.seen, held, lb); };
#pragma unroll 1
    for (int i = tid; i < kBins; i += THREADS) {
        sh.hist[i] = 0;
        if (CLUSTER) sh.sums[i] = 0;
    }
    if (tid == 0) {
        sh.ncand = 0;
        sh.least = ~0u;
        sh.most = 0;
    }
    if (!one) cluster_arrive();     // waited for before the first sums are added to
    if (select && rounds > 0) load(0);

    // The m-th largest key T of [lo, hi), and how many keys equal to T stay.
    uint32_t T = 0, ties = 0;
    bool tied = false;              // some of the equal keys go
    if (!select && !one) cluster_wait();
    if (select) {
        uint32_t need = (uint32_t)m;
        bool found = false;         // the keys that begin with T's digits so far all stay
        const bool few = BLOCKED && one && longest <= kFew;     // one warp searches them all
        if (few) {
            if (warp == 0) {
                // (to where they lie without gaps)
#pragma unroll 1
                for (int i = lane; i < kFew; i += 32) sh.cand[i] = i < held ? sh.key[place(i)] : 0;
                __syncwarp();
                found = search<kFew / 32>(sh.cand, kFew, 32, T, need);
                if (lane == 0) sh.pick[0] = T, sh.pick[1] = need, sh.pick[3] = found;
            }
            __syncthreads();
            T = sh.pick[0];
            need = sh.pick[1];
            found = sh.pick[3] != 0;
        }
#pragma unroll 1
        for (int digit = few ? 3 : 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const uint32_t mask = digit == 2 ? 1023u : 2047u;
            const uint32_t top_bits = digit == 0 ? 0u : digit == 1 ? 0xffe00000u : 0xfffffc00u;     // found so far
            if (digit > 0) {
                // Too many keys in T's bin for one warp.
                if (!one) cluster_sync();       // all have read the sums
                else __syncthreads();
#pragma unroll 1
                for (int i = tid; i < kBins; i += THREADS) {
                    sh.hist[i] = 0;
                    if (CLUSTER) sh.sums[i] = 0;
                }
                if (!one) cluster_sync();
                else __syncthreads();
            }
#pragma unroll 1
            for (int q = 0; q < rounds; ++q) {
                if (rounds > 1) load(q);
                const uint32_t *from = sh.key + place(tid);
                if (digit == 0) {
                    // Without a condition before them additions of 1 to the
                    // same bin are joined by the hardware (8,192 scores, many
                    // of them 0, in 360 cycles and not one by one); key 0
                    // falls in a bin that no score's key does.
#pragma unroll 4
                    for (int i = 0; i < per; ++i) atomicAdd(&sh.hist[from[place(THREADS) * i] >> 21], 1u);
                } else {
#pragma unroll 1
                    for (int i = 0; i < per; ++i) {
                        const uint32_t x = from[place(THREADS) * i];
                        if (x != 0 && ((x ^ T) & top_bits) == 0) atomicAdd(&sh.hist[x >> shift & mask], 1u);
                    }
                }
            }
            __syncthreads();
            // Bins from the top: thread t holds the kOwn from kBins - 1 - kOwn * t down, summed over the cluster.
            const uint32_t top = kBins - 1 - kOwn * tid, low = top - (kOwn - 1);
            Bins<kOwn> bin = local_bins<kOwn>(sh.hist + low);
            if constexpr (CLUSTER) if (!one) {
                // Bins in use lie together: each block sums every 2^le-th thread's.
                const uint32_t owner = tid & (E - 1);
                uint32_t *at = sh.sums + (tid >> le) * kOwn;
                if (digit == 0) cluster_wait();
#pragma unroll
                for (int j = 0; j < kOwn; ++j)
                    if (bin.n[j]) remote_add(at + j, owner, bin.n[j]);
                cluster_sync();
                bin = remote_bins<kOwn>(at, owner);
            }
            uint32_t sum = 0;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) sum += bin.n[j];
            uint32_t above = block_sums<THREADS>(sum, sh.scan[0]).x;
            if (above < need && need <= above + sum) {
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    const uint32_t n = bin.n[kOwn - 1 - j];
                    if (above < need && need <= above + n) sh.pick[0] = top - j, sh.pick[1] = need - above, sh.pick[2] = n;
                    above += n;
                }
            }
            __syncthreads();
            T |= sh.pick[0] << shift;
            need = sh.pick[1];
            const uint32_t n = sh.pick[2];
            found = need == n;
            if (found || digit == 2) break;
            if (n <= kCand) {
                // The bin's keys, in no order, and the search among them.
#pragma unroll 1
                for (int q = 0; q < rounds; ++q) {
                    if (rounds > 1) load(q);
                    const uint32_t *from = sh.key + place(tid);
                    uint32_t in = 0;
#pragma unroll 4
                    for (int i = 0; i < per; ++i) in |= (uint32_t)((from[place(THREADS) * i] ^ T) >> shift == 0) << i;
                    const uint32_t mine = __popc(in);
                    uint32_t end = mine, at = 0;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, end, d);
                        if (lane >= d) end += y;
                    }
                    if (lane == 31 && end > 0) at = atomicAdd(&sh.ncand, end);
                    at = __shfl_sync(0xffffffffu, at, 31) + end - mine;
#pragma unroll 1
                    for (uint32_t i = 0; i < mine; ++i, in &= in - 1) sh.cand[at + i] = from[place(THREADS) * (__ffs(in) - 1)];
                }
                if (one) __syncthreads();
                else cluster_sync();
                if (CLUSTER && !one) {
                    // Every block's, one after another: a warp copies a block's.
                    const uint32_t mine = lane < E ? remote(&sh.ncand, lane) : 0;
#pragma unroll 1
                    for (uint32_t r = warp; r < E; r += kWarps) {
                        const uint32_t first = __reduce_add_sync(0xffffffffu, lane < r ? mine : 0);
                        const uint32_t count = __shfl_sync(0xffffffffu, mine, r);
#pragma unroll 2
                        for (uint32_t i = lane; i < count; i += 32) sh.all[first + i] = remote(&sh.cand[i], r);
                    }
                    __syncthreads();
                }
                if (warp == 0) {
                    const uint32_t *p = CLUSTER && !one ? sh.all : sh.cand;
                    found = n <= 256 ? search<8>(p, n, shift, T, need) : search<kCand / 32>(p, n, shift, T, need);
                    if (lane == 0) sh.pick[0] = T, sh.pick[1] = need, sh.pick[3] = found;
                }
                __syncthreads();
                T = sh.pick[0];
                need = sh.pick[1];
                found = sh.pick[3] != 0;
                break;
            }
            if (digit == 0 && one && rounds == 1) {
                // All equal, as scores that no head likes are?
                uint32_t least = ~0u, most = 0;
                const uint32_t *from = sh.key + place(tid);
#pragma unroll 1
                for (int i = 0; i < per; ++i) {
                    const uint32_t x = from[place(THREADS) * i];
                    if ((x ^ T) >> 21 == 0) {
                        least = min(least, x);
                        most = max(most, x);
                    }
                }
                least = __reduce_min_sync(0xffffffffu, least);
                most = __reduce_max_sync(0xffffffffu, most);
                if (lane == 0) {
                    atomicMin(&sh.least, least);
                    atomicMax(&sh.most, most);
                }
                __syncthreads();
                if (sh.least == sh.most) {
                    T = sh.least;
                    break;
                }
            }
        }
        ties = need;
        tied = !found;
    }

    // Kept tokens of the rows before this one, and of all.
    uint32_t before = 0, all_tokens = 0;
    if (a.scanned) {
        before = (uint32_t)a.indptr_out[b];
        all_tokens = (uint32_t)a.indptr_out[rows];
    } else {
        before = tid < b ? my_tokens : 0;
        all_tokens = my_tokens;
#pragma unroll 1
        for (int i = tid + THREADS; i < rows; i += THREADS) {
            const uint32_t n = (uint32_t)row_of(a, i).tokens;
            before += i < b ? n : 0;
            all_tokens += n;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        all_tokens = __reduce_add_sync(0xffffffffu, all_tokens);
        if (lane == 0) sh.red[0][warp] = before, sh.red[1][warp] = all_tokens;
    }

    // A block outside [lo, hi), or any when all stay, is sure; between, those
    // above T are, and those equal to T are ties (sure too when all of them
    // stay).  Bits of this thread's keys of a round; their counts (at most
    // ROUND each in a block), summed over the threads.
    const bool all = m >= hi - lo;
    uint32_t sure = 0, tie = 0;
    const auto upto = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
    const auto mark = [&](int q, int buffer) {
        const int e0 = tid * per, i0 = s0 + q * ROUND + e0, n = min(s1, s0 + (q + 1) * ROUND) - i0;
        const uint32_t valid = upto(min(n, per)), inside = upto(hi - i0) & ~upto(lo - i0);
        sure = all ? valid : valid & ~inside;
        tie = 0;
        if (select) {
            uint32_t ge = 0, eq = 0;
#pragma unroll 4
            for (int j = 0; j < per; ++j) {
                const uint32_t x = sh.key[place(e0 + j)];
                ge |= (uint32_t)(x >= T) << j;
                eq |= (uint32_t)(x == T) << j;
            }
            sure |= ge & valid;         // (a key outside is 0)
            if (tied) {
                tie = eq & valid & inside;
                sure &= ~tie;
            }
        }
        return block_sums<THREADS>((uint32_t)__popc(sure) | (uint32_t)__popc(tie) << 16, sh.scan[buffer]);
    };
    uint2 at = make_uint2(0, 0);
    uint32_t block_kept = 0, block_ties = 0;        // sure blocks and ties of the thread blocks before this one
    if (one && rounds > 1) {
        __syncthreads();        // nothing needs the sums; every round's are formed below
    } else {
#pragma unroll 1
        for (int q = 0; q < max(rounds, 1); ++q) {
            if (rounds > 1 && select) load(q);
            else if (q > 0) __syncthreads();
            at = mark(q, 1);
            block_kept += at.y & 0xffff;
            block_ties += at.y >> 16;
        }
    }
    if (!one && tid == 0) sh.sum[0] = block_kept, sh.sum[1] = block_ties;
    block_kept = block_ties = 0;
    if (!a.scanned) {
        // (written before the barrier above)
        before = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[0][lane] : 0);
        all_tokens = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[1][lane] : 0);
        if (tid == 0 && rank == 0) {
            if (b == 0) a.indptr_out[0] = 0;
            a.indptr_out[b + 1] = (int32_t)(before + row.tokens);
        }
    }
    if (!one) {
        cluster_sync();
        if (lane < rank) {
            block_kept = remote(&sh.sum[0], lane);
            block_ties = remote(&sh.sum[1], lane);
        }
        block_kept = __reduce_add_sync(0xffffffffu, block_kept);
        block_ties = __reduce_add_sync(0xffffffffu, block_ties);
        cluster_arrive();       // the last of the others' shared memory has been read
    }

    // Placement, in position order.  Places past the output (only requests
    // that share entries, a bad indptr, make them) are dropped.
    const int32_t *pages = a.pages + row.base;
    const uint32_t limit = (uint32_t)a.capacity;
#pragma unroll 1
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) {
            if (select) load(q);
            else __syncthreads();
            at = mark(q, 1);
            __syncthreads();        // the keys have been read
        }
        // kept blocks of the row before this round: the sure ones and the ties among the first `ties`
        const uint32_t first = block_kept + min(block_ties, ties);
        const uint32_t tie_at = block_ties + (at.x >> 16);
        uint32_t put = block_kept + (at.x & 0xffff) + min(tie_at, ties) - first;
        block_kept += at.y & 0xffff;
        block_ties += at.y >> 16;
        const uint32_t n = (block_kept + min(block_ties, ties) - first) << lb;      // tokens
        int32_t *list = reinterpret_cast<int32_t *>(sh.key);
        // Of this thread's ties those among the first `ties`.
        const uint32_t mine = __popc(tie), past = tie_at + mine > ties ? min(mine, tie_at + mine - ties) : 0;
#pragma unroll 1
        for (uint32_t i = 0; i < past; ++i) tie &= ~(0x80000000u >> __clz(tie));
        const uint32_t keep = sure | tie;
        const int i0 = s0 + q * ROUND + tid * per;
#pragma unroll 2
        for (int j = 0; j < per; ++j)
            if (keep >> j & 1) list[put++] = i0 + j;
        __syncthreads();
        const uint32_t to = before + (first << lb);
#pragma unroll 1
        for (uint32_t x0 = tid; x0 < n; x0 += 4 * THREADS) {     // four loads, then their stores
            int32_t page[4];
            uint32_t some = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = x0 + j * THREADS;
                if (x >= n) break;
                const int i = (list[x >> lb] << lb) + (int)(x & ((1u << lb) - 1));
                if (i >= row.seen || to + x >= limit) continue;
                some |= 1u << j;
                page[j] = pages[i];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (some >> j & 1) a.pages_out[to + x0 + j * THREADS] = page[j];
        }
    }
    if (rank == 0)
#pragma unroll 1
        for (uint64_t i = all_tokens + ((uint64_t)b * THREADS + tid); i < limit; i += (uint64_t)rows * THREADS) a.pages_out[i] = -1;
    if (!one) cluster_wait();                  // no block ends while another may read its shared memory
}

// indptr_out of all rows, by one block.
__global__ void __launch_bounds__(1024) indptr_kernel(const SelectArgs a) {
    __shared__ uint32_t red[32];
    __shared__ uint32_t total;
    const int rows = a.R * a.qlen, tid = threadIdx.x;
    uint32_t carry = 0;
    grid_wait();
    if (tid == 0) a.indptr_out[0] = 0;
    for (int b0 = 0; b0 < rows; b0 += 1024) {
        const uint32_t n = b0 + tid < rows ? (uint32_t)row_of(a, b0 + tid).tokens : 0;
        const uint32_t at = carry + block_scan<32>(n, red) + n;
        if (b0 + tid < rows) a.indptr_out[b0 + tid + 1] = (int32_t)at;
        if (tid == 1023) total = at;
        __syncthreads();
        carry = total;
    }
}

__global__ void __launch_bounds__(256) empty_kernel(const SelectArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at == 0) a.indptr_out[0] = 0;
    for (int64_t i = at; i < a.capacity; i += (int64_t)gridDim.x * 256) a.pages_out[i] = -1;
}

template <int THREADS, int ROUND, bool CLUSTER, bool BLOCKED>
cudaError_t launch_kernel(SelectArgs a, int log_cs, cudaStream_t st) {
    constexpr int smem = sizeof(Shared<THREADS, ROUND, CLUSTER>);
    cudaError_t e = smem_attr_once<select_kernel<THREADS, ROUND, CLUSTER, BLOCKED>>(smem);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> wide{0};     // devices where clusters of 16 have been allowed
    if (log_cs > 3) {
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        if (!(bit & wide.load(std::memory_order_acquire))) {
            e = cudaFuncSetAttribute(select_kernel<THREADS, ROUND, CLUSTER, BLOCKED>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_release);
        }
    }
    const int rows = a.R * a.qlen;
    a.scanned = rows > kCounted;
    if (a.scanned) {
        e = launch_early(indptr_kernel, 1, 1024, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows << log_cs, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;    // it calls grid_wait()
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << log_cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = log_cs > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<THREADS, ROUND, CLUSTER, BLOCKED>, a, log_cs);
}

template <int THREADS, int ROUND, bool CLUSTER>
cudaError_t launch(const SelectArgs &a, int log_cs, cudaStream_t st) {
    return a.log_block > 0 ? launch_kernel<THREADS, ROUND, CLUSTER, true>(a, log_cs, st)
                           : launch_kernel<THREADS, ROUND, CLUSTER, false>(a, log_cs, st);
}

}  // namespace

// Arguments checked by mla_index_select.
cudaError_t index_select_launch(const float *scores, const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R,
                                int qlen, int topk, int block, int recent, int sinks, bool causal, int32_t *pages_out,
                                int64_t capacity, int32_t *indptr_out, int sms, cudaStream_t st) {
    SelectArgs a = {};
    a.scores = scores;
    a.pages = pages;
    a.indptr = indptr;
    a.num_pages = num_pages;
    a.capacity = capacity;
    a.R = R;
    a.qlen = qlen;
    a.topk = topk;
    while ((1 << a.log_block) < block) ++a.log_block;
    a.recent = recent;
    a.sinks = sinks;
    a.over_qlen = qlen > 1 ? (uint32_t)((0x100000000ull + qlen - 1) / qlen) : 0;
    a.causal = causal;
    a.pages_out = pages_out;
    a.indptr_out = indptr_out;
    const int64_t rows = (int64_t)R * qlen;
    if (rows == 0) {
        empty_kernel<<<(unsigned)std::min<int64_t>((capacity + 255) / 256 + 1, sms), 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    // The lengths are on the device: the rule goes by their mean.  More rows
    // than SMs that fit half a round of 256 threads take these.  Longer ones
    // take blocks of 16,384, in clusters that hold the mean (512 rows of 8K to
    // 16K 34 us, in clusters with rounds of 8,192 57; 300 of 40K to 128K 160
    // and 330; but 256 of 128 to 128K 119 and 89, where the longest go by
    // rounds).  Up to as many rows as SMs share a thread block's round, of
    // 16,384 too (100 rows of 16K 12 us, in clusters 16), or a cluster's, and
    // few rows take the blocks that half the SMs hold.
    const int64_t mean = (num_pages + R - 1) / R, blocks = mean >> a.log_block;
    int log_cs = 0;
    if (rows > sms) {
        if (blocks <= kShort / 2) return launch<256, kShort, false>(a, 0, st);
        if (blocks <= kLong) return launch<512, kLong, true>(a, 0, st);
        while (log_cs < 4 && (blocks >> log_cs) > 2 * kLong) ++log_cs;
        return launch<512, 2 * kLong, true>(a, log_cs, st);
    }
    if (blocks > kLong && blocks <= 2 * kLong) return launch<1024, 2 * kLong, false>(a, 0, st);
    while (log_cs < 4 && ((blocks >> log_cs) > kLong || (rows << (log_cs + 1)) <= sms / 2)) ++log_cs;
    return log_cs == 0 ? launch<1024, kLong, false>(a, 0, st) : launch<512, kLong, true>(a, log_cs, st);
}

cudaError_t index_select_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
