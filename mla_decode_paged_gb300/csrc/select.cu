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
// of dependent steps for one.
//
// Design: a cluster of thread blocks per row, as many of them as it takes to
// hold it (the others end at once), each with a contiguous slice of its token
// blocks: 8,192 keys (order-preserving 32-bit images of the scores), formed in
// shared memory from coalesced reads, then 8 or 16 neighbours in a thread's
// registers, so that one prefix sum over the threads places what stays (with
// 32 lanes of a warp side by side every key needed its ballots: three times
// the instructions).  A longer slice is taken in rounds of that size, read
// again for every step.  The m-th largest key: a histogram of the first 11
// bits, summed over the cluster through distributed shared memory, names the
// bin that holds it; one warp finds it bit by bit among that bin's keys, up
// to 1,024 of them.  More (many equal scores, mostly) take two more
// histograms, of 11 and 10 bits, unless all of them are equal.  The kept
// blocks are listed in shared memory and their tokens' pages copied from
// there, coalesced.
//
// A row's place in the output is the sum of the kept tokens of the rows
// before it: each cluster sums over all of them where they are no more than
// a block's threads, a small kernel writes the indptr first where they are.
#include <algorithm>
#include <atomic>

#include <cuda_runtime.h>

#include "cluster.cuh"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kBins = 2048;
constexpr int kRound = 8192;       // token blocks a thread block holds
constexpr int kCand = 1024;        // keys that one warp searches

struct SelectArgs {
    const float *scores;
    const int32_t *pages, *indptr;
    int64_t num_pages, capacity;
    int R, qlen, topk, log_block, recent, sinks;
    bool causal, scanned;           // scanned: indptr_out is there
    int32_t *pages_out, *indptr_out;
};

// A query row: its first entry, the tokens it sees, their blocks, the blocks and tokens it keeps.
struct Row {
    int base, seen, blocks, kept, tokens;
};
__device__ __forceinline__ Row row_of(const SelectArgs &a, int b) {
    Row x;
    const int r = b / a.qlen, tq = b - r * a.qlen;
    const int len = request_len(a.indptr, r, a.num_pages, &x.base);
    x.seen = a.causal ? max(0, len - a.qlen + tq + 1) : len;
    x.blocks = (x.seen + (1 << a.log_block) - 1) >> a.log_block;
    x.kept = min(x.blocks, a.topk);
    x.tokens = x.kept == x.blocks ? x.seen : (x.kept << a.log_block) - ((x.blocks << a.log_block) - x.seen);
    return x;
}

template <int THREADS>
struct __align__(16) Shared {
    uint32_t key[kRound];           // a round's keys (place); then the blocks that stay, in order
    uint32_t hist[kBins];
    uint32_t sums[kBins];           // of this block's share of the bins, over the cluster
    uint32_t cand[kCand], all[kCand];   // keys of the m-th largest's bin: this block's, the cluster's
    uint32_t red[2][32], scan[32], totals[32];
    uint32_t least, most;           // of this block's keys of that bin
    uint32_t ncand;
    uint32_t sum[2];                // this block's sure blocks and ties, for the cluster
    uint32_t pick[4];
};

// Where key i of a round lies: a thread's PER neighbours in vectors of four,
// their order turned by the thread so that eight threads' vectors fall in
// different banks.
template <int PER>
__device__ __forceinline__ int place(int i) {
    const int t = i / PER, c = i / 4 % (PER / 4);
    return t * PER + ((c ^ (PER == 16 ? t >> 1 & 3 : t >> 2 & 1)) << 2) + (i & 3);
}

// Blocks it takes to hold a row's tokens, as a power of two up to log_cs.
__device__ __forceinline__ int blocks_for(int tokens, int log_cs) {
    int le = 0;
    while (le < log_cs && (tokens >> le) > kRound) ++le;
    return le;
}

// The need-th largest of the n keys at p, which agree above their lowest 21
// bits (run by a warp): a value T that exactly `need` of them reach, and
// true, or the key itself, how many of it belong to them, and false.
template <int N>
__device__ bool search(const uint32_t *p, uint32_t n, uint32_t &T, uint32_t &need) {
    const int lane = threadIdx.x & 31;
    uint32_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane + 32 * i < n ? p[lane + 32 * i] : 0;
    for (int bit = 20; bit >= 0; --bit) {
        const uint32_t t = T | 1u << bit;
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) c += x[i] >= t;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c < need) continue;
        T = t;
        if (c == need) return true;
    }
    uint32_t above = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) above += x[i] > T;
    need -= __reduce_add_sync(0xffffffffu, above);
    return false;
}

// 2^log_cs blocks (a cluster) per row.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 1) select_kernel(const SelectArgs a, int log_cs) {
    constexpr int kWarps = THREADS / 32, kPer = kRound / THREADS, kOwn = kBins / THREADS;   // keys of a thread; bins it sums
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared<THREADS> &sh = *reinterpret_cast<Shared<THREADS> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = block_rank();
    const int rows = a.R * a.qlen, b = blockIdx.x >> log_cs, lb = a.log_block;
    const Row row = row_of(a, b);
    const uint32_t my_tokens = !a.scanned && tid < rows ? (uint32_t)row_of(a, tid).tokens : 0;
    // The blocks past those that hold the row end (a cluster barrier waits for
    // running threads only).
    const int le = blocks_for(row.seen, log_cs);
    const uint32_t E = 1u << le;
    if (rank >= E) return;
    const bool one = le == 0;
    const int recent = min(a.recent, row.kept), sinks = min(a.sinks, row.kept - recent);
    const int lo = sinks, hi = row.blocks - recent;     // the blocks that may go
    const int m = row.kept - recent - sinks;            // how many of them stay
    const bool select = m > 0 && m < hi - lo;           // the same in every block of the cluster
    const float *w = a.scores + (int64_t)(b % a.qlen) * a.num_pages + row.base;

    // This block's slice, in rounds.  Key 0: none that may go.
    const int slice = (((row.blocks + (int)E - 1) >> le) + 31) / 32 * 32;
    const int s0 = (int)min((int64_t)slice * rank, (int64_t)row.blocks), s1 = min(slice, row.blocks - s0) + s0;
    const int rounds = (s1 - s0 + kRound - 1) / kRound;
    uint32_t key[kPer];
    const auto load = [&](int q) {
        const int r0 = s0 + q * kRound, n = min(kRound, s1 - r0), f0 = max(lo - r0, 0), f1 = min(hi - r0, n);
        if (rounds > 1) __syncthreads();    // the round before has been read
        if (lb == 0) {
            float v[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = tid + THREADS * j;
                v[j] = i >= f0 && i < f1 ? __ldg(w + r0 + i) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = tid + THREADS * j;
                sh.key[place<kPer>(i)] = i >= f0 && i < f1 ? weight_key(v[j]) : 0;
            }
        } else {
            // Block maxima: warps take 32 tokens in turn, eight of these reads
            // in flight; the lanes of a block join by shuffles.
            for (int i = tid; i < kRound; i += THREADS) sh.key[i] = 0;
            __syncthreads();
            const int t1 = min((r0 + f1) << lb, row.seen);
            for (int at = ((r0 + f0) << lb) + 32 * warp; at < t1; at += 32 * 8 * kWarps) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int t = at + 32 * kWarps * k + lane;
                    v[k] = t < t1 ? __ldg(w + t) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int t = at + 32 * kWarps * k + lane;
                    if (t - lane >= t1) break;
                    uint32_t x = t < t1 ? weight_key(v[k]) : 0;
                    if (lb >= 5) {
                        x = __reduce_max_sync(0xffffffffu, x);
                        if (lane == 0) atomicMax(&sh.key[place<kPer>((t >> lb) - r0)], x);
                    } else {
                        for (int d = 1; d < 1 << lb; d <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if ((t & ((1 << lb) - 1)) == 0 && t < t1) sh.key[place<kPer>((t >> lb) - r0)] = x;
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kPer / 4; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sh.key + place<kPer>(tid * kPer + 4 * c));
            key[4 * c] = v.x, key[4 * c + 1] = v.y, key[4 * c + 2] = v.z, key[4 * c + 3] = v.w;
        }
    };
    for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<uint4 *>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
    if (!one)
        for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<uint4 *>(sh.sums)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        sh.ncand = 0;
        sh.least = ~0u;
        sh.most = 0;
    }
    if (!one) cluster_arrive();     // waited for before the first sums are added to
    if (select && rounds > 0) load(0);      // (its barriers order the zeros above, too)

    // The m-th largest key T of [lo, hi), and how many keys equal to T stay.
    uint32_t T = 0, ties = 0;
    bool tied = false;              // some of the equal keys go
    if (!one) cluster_wait();
    if (select) {
        uint32_t need = (uint32_t)m;
        bool found = false;         // the keys that begin with T's digits so far all stay
        for (int digit = 0; digit < 3; ++digit) {
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const uint32_t mask = digit == 2 ? 1023u : 2047u;
            const uint32_t top_bits = digit == 0 ? 0u : digit == 1 ? 0xffe00000u : 0xfffffc00u;     // found so far
            if (digit > 0) {
                // Too many keys in T's bin for one warp.
                __syncthreads();
                for (int i = tid; i < kBins; i += THREADS) sh.hist[i] = 0;
                if (!one) {
                    cluster_sync();         // all have read the sums
                    for (int i = tid; i < kBins; i += THREADS) sh.sums[i] = 0;
                    cluster_sync();
                }
                __syncthreads();
            }
            for (int q = 0; q < rounds; ++q) {
                if (rounds > 1) load(q);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (key[j] != 0 && ((key[j] ^ T) & top_bits) == 0) atomicAdd(&sh.hist[key[j] >> shift & mask], 1u);
            }
            __syncthreads();
            // Bins from the top: thread t holds the kOwn from kBins - 1 - kOwn * t down, summed over the cluster.
            const uint32_t top = kBins - 1 - kOwn * tid, low = top - (kOwn - 1);
            Bins<kOwn> bin = local_bins<kOwn>(sh.hist + low);
            if (!one) {
                const uint32_t share = kBins >> le, owner = low >> (11 - le);       // a block's bins; these bins' block
                uint32_t *at = sh.sums + (low & (share - 1));
#pragma unroll
                for (int j = 0; j < kOwn; ++j)
                    if (bin.n[j]) remote_add(at + j, owner, bin.n[j]);
                cluster_sync();
                bin = remote_bins<kOwn>(at, owner);
            }
            uint32_t sum = 0;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) sum += bin.n[j];
            uint32_t incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            if (lane == 31) sh.scan[warp] = incl;
            __syncthreads();
            uint32_t above = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[lane] : 0);
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const uint32_t n = bin.n[kOwn - 1 - j];
                if (above < need && need <= above + n) {
                    sh.pick[0] = top - j;
                    sh.pick[1] = need - above;
                    sh.pick[2] = n;
                }
                above += n;
            }
            __syncthreads();
            T |= sh.pick[0] << shift;
            need = sh.pick[1];
            const uint32_t n = sh.pick[2];
            found = need == n;
            if (found || digit == 2) break;
            if (digit > 0) continue;
            if (n <= kCand) {
                // The bin's keys, in no order, and the search among them.
                for (int q = 0; q < rounds; ++q) {
                    if (rounds > 1) load(q);
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if ((key[j] ^ T) >> 21 == 0) sh.cand[atomicAdd(&sh.ncand, 1u)] = key[j];
                }
                if (one) __syncthreads();
                else cluster_sync();
                if (warp == 0) {
                    const uint32_t *p = sh.cand;
                    if (!one) {
                        // Every block's, one after another.
                        const uint32_t mine = lane < E ? remote(&sh.ncand, lane) : 0;
                        uint32_t ends = mine;
#pragma unroll
                        for (int d = 1; d < 16; d <<= 1) {
                            const uint32_t y = __shfl_up_sync(0xffffffffu, ends, d);
                            if (lane >= d) ends += y;
                        }
                        for (uint32_t i0 = 0; i0 < n; i0 += 32) {
                            const uint32_t i = i0 + lane;
                            uint32_t r = 0;         // the block of the i-th: those that end before it
#pragma unroll
                            for (int d = 0; d < 16; ++d) r += d < (int)E && __shfl_sync(0xffffffffu, ends, d) <= i;
                            const uint32_t from = __shfl_sync(0xffffffffu, ends - mine, r & 31);
                            if (i < n) sh.all[i] = remote(&sh.cand[i - from], r);
                        }
                        __syncwarp();
                        p = sh.all;
                    }
                    found = n <= 256 ? search<8>(p, n, T, need) : search<kCand / 32>(p, n, T, need);
                    if (lane == 0) {
                        sh.pick[0] = T;
                        sh.pick[1] = need;
                        sh.pick[3] = found;
                    }
                }
                __syncthreads();
                T = sh.pick[0];
                need = sh.pick[1];
                found = sh.pick[3] != 0;
                break;
            }
            if (one && rounds == 1) {
                // All equal, as scores that no head likes are?
                uint32_t least = ~0u, most = 0;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if ((key[j] ^ T) >> 21 == 0) {
                        least = min(least, key[j]);
                        most = max(most, key[j]);
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
    uint32_t before, all_tokens;
    if (a.scanned) {
        before = (uint32_t)__ldg(a.indptr_out + b);
        all_tokens = (uint32_t)__ldg(a.indptr_out + rows);
    } else {
        const uint32_t x = __reduce_add_sync(0xffffffffu, tid < b ? my_tokens : 0);
        const uint32_t y = __reduce_add_sync(0xffffffffu, my_tokens);
        if (lane == 0) {
            sh.red[0][warp] = x;
            sh.red[1][warp] = y;
        }
    }

    // A block outside [lo, hi), or any when all stay, is sure; between, those
    // above T are, and those equal to T are ties (sure too when all of them
    // stay).  Bits of this thread's keys.
    const bool all = m >= hi - lo;
    uint32_t sure = 0, tie = 0;
    const auto upto = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
    const auto mark = [&](int q) {
        const int i0 = s0 + q * kRound + tid * kPer, n = min(s1, s0 + (q + 1) * kRound) - i0;      // keys of the round here
        const uint32_t valid = upto(min(n, kPer)), inside = upto(hi - i0) & ~upto(lo - i0);
        sure = all ? valid : valid & ~inside;
        tie = 0;
        if (select) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (key[j] >= T) sure |= 1u << j;
                if (key[j] == T) tie |= 1u << j;
            }
            tie &= valid & inside;
            sure &= valid;
            if (tied) sure &= ~tie;
            else tie = 0;
        }
        return (uint32_t)__popc(sure) | (uint32_t)__popc(tie) << 16;     // at most kRound each in a block's round
    };
    // Prefix over the block's threads of such counts, and their sum.
    const auto scan = [&](uint32_t x, uint32_t &total) {
        uint32_t incl = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) sh.totals[warp] = incl;
        __syncthreads();
        const uint32_t t = lane < kWarps ? sh.totals[lane] : 0;
        total = __reduce_add_sync(0xffffffffu, t);
        return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
    };
    uint32_t total, at = 0;
    uint32_t block_kept = 0, block_ties = 0;        // sure blocks and ties of the thread blocks before this one
    if (rounds <= 1) {
        at = scan(rounds > 0 ? mark(0) : 0, total);
        if (!one && tid == 0) sh.sum[0] = total & 0xffff, sh.sum[1] = total >> 16;
    } else {
        uint32_t sum = 0, nties = 0;
        for (int q = 0; q < rounds; ++q) {
            if (select) load(q);
            __syncthreads();
            scan(mark(q), total);
            sum += total & 0xffff;
            nties += total >> 16;
        }
        if (!one && tid == 0) sh.sum[0] = sum, sh.sum[1] = nties;
    }
    if (!a.scanned) {
        // (written before the barrier in scan)
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
    }

    // Placement, in position order.  Places past the output (only requests
    // that share entries, a bad indptr, make them) are dropped.
    const int32_t *pages = a.pages + row.base;
    const int64_t limit = a.capacity;
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) {
            if (select) load(q);
            __syncthreads();
            at = scan(mark(q), total);
        }
        // kept blocks of the row before this round: the sure ones and the ties among the first `ties`
        const uint32_t first = block_kept + min(block_ties, ties);
        uint32_t tie_at = block_ties + (at >> 16);
        uint32_t put = block_kept + (at & 0xffff) + min(tie_at, ties) - first;
        block_kept += total & 0xffff;
        block_ties += total >> 16;
        const uint32_t n = (block_kept + min(block_ties, ties) - first) << lb;      // tokens
        const int i0 = s0 + q * kRound + tid * kPer;
        if (rounds > 1) __syncthreads();
        int32_t *list = reinterpret_cast<int32_t *>(sh.key);       // the keys are in registers
        uint32_t keep = sure | tie;
        while (keep) {
            const int j = __ffs(keep) - 1;
            keep &= keep - 1;
            if ((tie >> j & 1) && tie_at++ >= ties) continue;
            list[put++] = i0 + j;
        }
        __syncthreads();
        const uint32_t to = before + (first << lb);
        for (uint32_t x = tid; x < n; x += THREADS) {
            const int i = (list[x >> lb] << lb) + (int)(x & ((1u << lb) - 1));
            if (i < row.seen && to + x < limit) a.pages_out[to + x] = __ldg(pages + i);
        }
    }
    if (rank == 0)
        for (int64_t i = all_tokens + ((int64_t)b * THREADS + tid); i < limit; i += (int64_t)rows * THREADS)
            a.pages_out[i] = -1;
    if (!one) cluster_sync();                  // no block ends while another may read its shared memory
}

// indptr_out of all rows, by one block.
__global__ void __launch_bounds__(1024) indptr_kernel(const SelectArgs a) {
    __shared__ uint32_t red[32];
    __shared__ uint32_t total;
    const int rows = a.R * a.qlen, tid = threadIdx.x;
    uint32_t carry = 0;
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

template <int THREADS>
cudaError_t launch(SelectArgs a, int log_cs, cudaStream_t st) {
    constexpr int smem = sizeof(Shared<THREADS>);
    cudaError_t e = smem_attr_once<select_kernel<THREADS>>(smem);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> wide{0};     // devices where clusters of 16 have been allowed
    if (log_cs > 3) {
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        if (!(bit & wide.load(std::memory_order_acquire))) {
            e = cudaFuncSetAttribute(select_kernel<THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_release);
        }
    }
    const int rows = a.R * a.qlen;
    a.scanned = rows > THREADS;
    if (a.scanned) {
        indptr_kernel<<<1, 1024, 0, st>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows << log_cs, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log_cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = log_cs > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, select_kernel<THREADS>, a, log_cs);
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
    a.causal = causal;
    a.pages_out = pages_out;
    a.indptr_out = indptr_out;
    const int64_t rows = (int64_t)R * qlen;
    if (rows == 0) {
        empty_kernel<<<(unsigned)std::min<int64_t>((capacity + 255) / 256 + 1, sms), 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    // The lengths are on the device: a cluster holds a row of the mean length
    // in one round, and a few rows take the blocks that half the SMs hold.
    const int64_t mean = (num_pages + R - 1) / R;
    int log_cs = 0;
    while (log_cs < 4 && ((mean >> a.log_block >> log_cs) > kRound || (rows << (log_cs + 1)) <= sms / 2)) ++log_cs;
    return log_cs == 0 && rows <= sms ? launch<1024>(a, log_cs, st) : launch<512>(a, log_cs, st);
}

cudaError_t index_select_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
