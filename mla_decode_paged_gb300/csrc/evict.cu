// Eviction from the paged cache by accumulated attention weight.
//
// What it computes: request r of L tokens keeps n = min(L, max(budget, 0))
// of them: its last min(recent, n), its first min(sinks, the rest), and for
// the remaining m the tokens in between with the largest weights (NaN as
// -inf, equal weights by the lowest position).  Kept tokens stay in order;
// the page list becomes every request's kept rows, then the freed rows.
//
// Bound by the 16 bytes a token that are read and written for many long
// requests, by the chain of dependent steps for one.
//
// Design: a cluster of blocks per request, as many of them as it takes to
// hold it (the others end at once), each with a contiguous slice of its
// tokens and every warp with a contiguous part of that, whose keys
// (order-preserving 32-bit images of the weights) stay in registers: 8,192
// tokens a block.  A longer slice is taken in rounds of that
// size, read again for every step.  The m-th largest key is found by radix
// selection, 11 + 11 + 10 bits, ended by the digits whose keys all stay: every
// block counts its slice into a shared histogram, adds the bins that are not
// empty to their sums over the cluster, which the blocks hold in equal shares,
// and reads these through distributed shared memory (reading all histograms in
// every block instead took 11,500 cycles a digit with 16 blocks; a histogram
// per digit: none is reused).  What each warp keeps is counted
// by ballots, the offsets of warps and blocks are exchanged once, and the
// tokens are placed by the ballots again.
//
// Measured: 12.8 us for one request of 128K tokens, 8.7 for 64 of 1K to 8K, 77
// for 256 of 128 to 128K (log-uniform, 5.0 M tokens, 1.0 TB/s: its counts and
// placements are bound by instructions, and by how many clusters an SM holds).
// Every cluster sums over all requests for its place in the outputs, in one
// step up to a block's threads, in a loop above: quadratic, so mla_kv_evict
// takes 65,536 requests at most (of 100 tokens each: 1,024 in 26.5 us, 8,192
// in 218, 16,384 in 527, 65,536 in 5,165, of which the sums are about two thirds).
#include <atomic>

#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {
namespace {

constexpr int kBins = 2048, kDigits = 3;
constexpr int kRound = 8192;       // tokens a block holds
constexpr int kClasses = 6;        // powers of two of blocks, 0 to 4, and more than one round
constexpr int kInOrder = 32;       // clusters that all run at once

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

// The weight of a key, where the key tells it (not of NaN or -inf, nor of a zero).
__device__ __forceinline__ float key_weight(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
constexpr uint32_t kKeyZero = 0x80000000u, kKeyLowest = ~0xff800000u;     // no key is below kKeyLowest

__device__ __forceinline__ int kept_tokens(const EvictArgs &a, int r, int len) {
    const int b = a.budgets ? __ldg(a.budgets + r) : a.budget;
    return b < 0 ? 0 : b < len ? b : len;
}

template <int WARPS>
struct __align__(16) Shared {
    uint32_t hist[kDigits][kBins];
    uint32_t sums[kDigits][kBins];  // of this block's share of the bins, over the cluster
    uint32_t red[3][WARPS];
    uint32_t classes[WARPS][kClasses];     // a warp's requests by the blocks they take
    int own[4];                             // the cluster's request, its tokens, first entry, kept tokens
    uint32_t scan[WARPS];
    uint32_t warp_kept[WARPS], warp_ties[WARPS];
    uint32_t totals[2];             // this block's sure tokens and ties, for the cluster
    uint32_t pick[3];
};

__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// All running blocks of the cluster, their shared-memory writes before it
// visible after it.  Both halves are for whole warps: lanes that took a
// branch before them meet first.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// What is at `p`'s place in the shared memory of block `rank`.
__device__ __forceinline__ uint32_t remote(const uint32_t *p, uint32_t rank) {
    uint32_t addr, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// A thread's bins.
template <int N>
struct Bins {
    static_assert(N == 2 || N == 4, "one vector");
    uint32_t n[N];
};
template <int N>
__device__ __forceinline__ Bins<N> local_bins(const uint32_t *p) {
    Bins<N> b;
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        b.n[0] = v.x, b.n[1] = v.y, b.n[2] = v.z, b.n[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        b.n[0] = v.x, b.n[1] = v.y;
    }
    return b;
}
template <int N>
__device__ __forceinline__ Bins<N> remote_bins(const uint32_t *p, uint32_t rank) {
    uint32_t addr;
    Bins<N> b;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    if constexpr (N == 4)
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b.n[0]), "=r"(b.n[1]), "=r"(b.n[2]), "=r"(b.n[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(b.n[0]), "=r"(b.n[1]) : "r"(addr) : "memory");
    return b;
}

// Adds v at `p`'s place in the shared memory of block `rank`.
__device__ __forceinline__ void remote_add(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tred.relaxed.cluster.shared::cluster.add.u32 [a], %2;\n\t}" ::"r"(
            smem_u32(p)),
        "r"(rank), "r"(v)
        : "memory");
}

// Exclusive prefix sum of v over the block's threads.
template <int WARPS>
__device__ uint32_t block_scan(uint32_t v, uint32_t *red) {
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
    const uint32_t w = lane < WARPS ? red[lane] : 0;
    uint32_t s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    return x - v + __shfl_sync(0xffffffffu, s - w, warp);
}

// Blocks it takes to hold a request, as a power of two; above log_cs where a
// cluster of 2^log_cs needs more than one round for it.
__device__ __forceinline__ int blocks_for(int len, int log_cs) {
    int le = 0;
    while (le <= log_cs && (len >> le) > kRound) ++le;
    return le;
}

// 2^log_cs blocks (a cluster) per request.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_kernel(const EvictArgs a, int log_cs) {
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    constexpr int kSteps = kRound / THREADS, kOwn = kBins / THREADS;    // tokens a thread holds; bins it sums
    __shared__ Shared<kWarps> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1, rank = block_rank();
    // The cluster's request.  Clusters start in order of their number: with
    // more of them than run at once, the requests of most blocks go first.
    int r = blockIdx.x >> log_cs, len, base, kept;
    uint32_t sums[3] = {0, 0, 0};   // kept and all tokens of the requests before it, kept of all (mod 2^32)
    if (a.R <= kThreads) {
        int my_base = 0, my_len = 0, my_kept = 0;
        if (tid < a.R) {
            my_len = request_len(a.indptr, tid, a.num_pages, &my_base);
            my_kept = kept_tokens(a, tid, my_len);
        }
        int place = tid;
        if (log_cs > 0 && a.R > kInOrder) {
            const int mine = tid < a.R ? blocks_for(my_len, log_cs) : -1;
            uint32_t same = 0;
#pragma unroll
            for (int c = 0; c < kClasses; ++c) {
                const uint32_t m = __ballot_sync(0xffffffffu, mine == c);
                if (mine == c) same = m;
                if (lane == 0) sh.classes[warp][c] = __popc(m);
            }
            __syncthreads();
            place = __popc(same & below);
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int c = 0; c < kClasses; ++c)
                    if (c > mine || (c == mine && w < warp)) place += sh.classes[w][c];
        }
        if (tid < a.R && place == r) {
            sh.own[0] = tid;
            sh.own[1] = my_len;
            sh.own[2] = my_base;
            sh.own[3] = my_kept;
        }
        __syncthreads();
        r = sh.own[0];
        len = sh.own[1];
        base = sh.own[2];
        kept = sh.own[3];
        sums[0] = tid < r ? my_kept : 0;
        sums[1] = tid < r ? my_len : 0;
        sums[2] = my_kept;
    } else {
        len = request_len(a.indptr, r, a.num_pages, &base);
        kept = kept_tokens(a, r, len);
    }
    // The blocks past those that hold the request end (a cluster barrier
    // waits for running threads only).
    const int le = min(blocks_for(len, log_cs), log_cs);
    const uint32_t E = 1u << le;
    if (rank >= E) return;
    const bool one = le == 0;
    const int recent = a.recent < kept ? a.recent : kept;
    const int sinks = a.sinks < kept - recent ? a.sinks : kept - recent;
    const int lo = sinks, hi = len - recent;        // the tokens that may go
    const int m = kept - recent - sinks;            // how many of them stay
    const float *w = a.weights + base;

    // This block's slice, in rounds; a warp's part of a round, whole groups of
    // 32 tokens.  Key 0: no token that may go.
    const int slice = (((len + (int)E - 1) >> le) + 31) / 32 * 32;
    const int s0 = (int)min((int64_t)slice * rank, (int64_t)len), s1 = min(slice, len - s0) + s0;
    const int rounds = (s1 - s0 + kRound - 1) / kRound;
    uint32_t key[kSteps];
    uint32_t valid = 0, free = 0;   // a bit a step: a token, one that may go
    int first = 0, steps = 0;
    const auto fetch = [&](int q) {                 // weights into key, as they are
        const int q0 = s0 + q * kRound, q1 = min(q0 + kRound, s1);
        const int part = ((q1 - q0 + kWarps - 1) / kWarps + 31) / 32 * 32;
        first = q0 + warp * part + lane;
        steps = part / 32;
        valid = free = 0;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int i = first + 32 * j;
            key[j] = 0;
            if (j < steps && i < q1) {
                key[j] = __float_as_uint(__ldg(w + i));
                valid |= 1u << j;
                if (i >= lo && i < hi) free |= 1u << j;
            }
        }
    };
    const auto convert = [&] {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) key[j] = weight_key(__uint_as_float(key[j]));
    };
    const auto load = [&](int q) {
        fetch(q);
        convert();
    };
    // On their way during the sums over the requests.
    if (rounds > 0) {
        fetch(0);
        const int line = first - lane + 32 * lane;      // 32 rows of the page list, read at the placement
        if (lane < steps && line < s1) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.pages + base + line));
    }
    for (int i = tid; i < kDigits * kBins / 4; i += kThreads)
        reinterpret_cast<uint4 *>(&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    if (!one) {
        for (int i = tid; i < kDigits * kBins / 4; i += kThreads)
            reinterpret_cast<uint4 *>(&sh.sums[0][0])[i] = make_uint4(0, 0, 0, 0);
        cluster_arrive();       // waited for before the first sums are added to
    }
    if (a.R > kThreads)
        for (int i = tid; i < a.R; i += kThreads) {
            int at;
            const int n = request_len(a.indptr, i, a.num_pages, &at), k = kept_tokens(a, i, n);
            sums[2] += k;
            if (i < r) {
                sums[0] += k;
                sums[1] += n;
            }
        }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const uint32_t s = __reduce_add_sync(0xffffffffu, sums[j]);
        if (lane == 0) sh.red[j][warp] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) sums[j] = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[j][lane] : 0);
    if (tid == 0 && rank == 0) {
        if (r == 0) a.indptr_out[0] = 0;
        a.indptr_out[r + 1] = (int32_t)(sums[0] + kept);
    }
    if (rounds > 0) convert();

    // The m-th largest key T of [lo, hi), and how many keys equal to T stay.
    uint32_t T = 0, ties = 0;
    const bool select = m > 0 && m < hi - lo;       // the same in every block of the cluster
    bool tied = false;                              // some of the equal keys go
    if (!select && !one) cluster_wait();
    if (select) {
        uint32_t need = (uint32_t)m;
        bool found = false;                         // the keys that begin with T's digits so far all stay
#pragma unroll
        for (int digit = 0; digit < kDigits; ++digit) {
            if (found) break;
            const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
            const uint32_t bins = digit == 2 ? 1024u : 2048u;
            const int above_bits = digit == 0 ? 0 : digit == 1 ? 21 : 10;   // bits below the digits found
            uint32_t *hist = sh.hist[digit];
            for (int q = 0; q < rounds; ++q) {
                if (rounds > 1) load(q);
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
                    if (j < steps && (free >> j & 1) && (digit == 0 || (key[j] ^ T) >> above_bits == 0))
                        atomicAdd(&hist[(key[j] >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            // Bins from the top: thread t holds the kOwn from kBins - 1 - kOwn * t down, summed over the cluster.
            const uint32_t top = kBins - 1 - kOwn * tid, low = top - (kOwn - 1);
            uint32_t sum = 0;
            Bins<kOwn> bin = local_bins<kOwn>(hist + low);
            if (!one) {
                const uint32_t share = kBins >> le, owner = low >> (11 - le);       // a block's bins; these bins' block
                uint32_t *at = sh.sums[digit] + (low & (share - 1));
                if (digit == 0) cluster_wait();
#pragma unroll
                for (int j = 0; j < kOwn; ++j)
                    if (bin.n[j]) remote_add(at + j, owner, bin.n[j]);
                cluster_sync();
                bin = remote_bins<kOwn>(at, owner);
            }
#pragma unroll
            for (int j = 0; j < kOwn; ++j) sum += bin.n[j];
            uint32_t above = block_scan<kWarps>(sum, sh.scan);
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
            found = need == sh.pick[2];
        }
        ties = need;
        tied = !found;
    }

    // A token outside [lo, hi), or any when all stay, is sure; between, those
    // above T are, and those equal to T are ties (sure too when all of them stay).
    const bool all = m >= hi - lo;
    uint32_t sure = 0, tie = 0;     // a bit a step
    const auto count = [&](uint32_t &nsure, uint32_t &nties) {
        sure = all ? valid : valid & ~free;
        tie = 0;
        if (select) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                if (key[j] >= T) sure |= free & 1u << j;
                if (tied && key[j] == T) tie |= free & 1u << j;
            }
            sure &= ~tie;
        }
        nsure += __reduce_add_sync(0xffffffffu, __popc(sure));
        if (tied) nties += __reduce_add_sync(0xffffffffu, __popc(tie));
    };
    // Sums over the block (k, t) and over the warps before this one (kb, tb) of what every warp counted.
    const auto exchange = [&](uint32_t nsure, uint32_t nties, uint32_t &k, uint32_t &t, uint32_t &kb, uint32_t &tb) {
        __syncthreads();
        if (lane == 0) {
            sh.warp_kept[warp] = nsure;
            sh.warp_ties[warp] = nties;
        }
        __syncthreads();
        k = lane < kWarps ? sh.warp_kept[lane] : 0;
        t = lane < kWarps ? sh.warp_ties[lane] : 0;
        kb = __reduce_add_sync(0xffffffffu, lane < warp ? k : 0);
        tb = __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
        k = __reduce_add_sync(0xffffffffu, k);
        t = __reduce_add_sync(0xffffffffu, t);
    };
    uint32_t nsure = 0, nties = 0, k, t, kb, tb;
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) load(q);
        count(nsure, nties);
    }
    exchange(nsure, nties, k, t, kb, tb);
    uint32_t block_kept = 0, block_ties = 0;        // sure tokens and ties of the blocks before this one
    if (!one) {
        if (tid == 0) {
            sh.totals[0] = k;
            sh.totals[1] = t;
        }
        cluster_sync();
        if (lane < rank) {
            block_kept = remote(&sh.totals[0], lane);
            block_ties = remote(&sh.totals[1], lane);
        }
        block_kept = __reduce_add_sync(0xffffffffu, block_kept);
        block_ties = __reduce_add_sync(0xffffffffu, block_ties);
    }

    // Placement, in position order.  Places past the page list (only a bad
    // indptr makes them) are dropped.
    const uint32_t out_kept = sums[0], out_freed = sums[2] + (sums[1] - sums[0]);
    const uint32_t limit = (uint32_t)a.num_pages;
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) {
            load(q);
            nsure = nties = 0;
            count(nsure, nties);
            exchange(nsure, nties, k, t, kb, tb);
        }
        uint32_t kept_at = block_kept + kb, ties_at = block_ties + tb;
        block_kept += k;
        block_ties += t;
        const int32_t *pages = a.pages + base + first;
#pragma unroll
        for (int j0 = 0; j0 < kSteps; j0 += 8) {
            if (j0 >= steps) break;
            int32_t page[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) page[j] = (valid >> (j0 + j) & 1) ? __ldg(pages + 32 * (j0 + j)) : 0;
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
                const int j = j0 + jj;
                if (j >= steps) break;
                const uint32_t ms = __ballot_sync(0xffffffffu, sure >> j & 1);
                // kept tokens of the request before this one: the sure ones and the ties among the first `ties`
                uint32_t rank_i = kept_at + __popc(ms & below);
                bool keep = sure >> j & 1;
                if (tied) {
                    const uint32_t mt = __ballot_sync(0xffffffffu, tie >> j & 1);
                    const uint32_t tie_rank = ties_at + __popc(mt & below);
                    keep = keep || ((tie >> j & 1) && tie_rank < ties);
                    rank_i += min(tie_rank, ties);
                    ties_at += __popc(mt);
                }
                kept_at += __popc(ms);
                const uint32_t i = first + 32 * j;
                const uint32_t at = keep ? out_kept + rank_i : out_freed + (i - rank_i);
                float wi = 0.f;
                if (keep) {
                    wi = key_weight(key[j]);
                    if (key[j] == kKeyZero || key[j] == kKeyLowest) wi = (valid >> j & 1) ? __ldg(w + i) : 0.f;
                }
                if ((valid >> j & 1) && at < limit) {
                    a.pages_out[at] = page[jj];
                    a.weights_out[at] = wi;
                }
            }
        }
    }
    if (!one) cluster_sync();                  // no block ends while another may read its shared memory
}

template <int THREADS>
cudaError_t launch(const EvictArgs &a, int log_cs, cudaStream_t st) {
    static std::atomic<unsigned long long> wide{0};     // devices where clusters of 16 have been allowed
    if (log_cs > 3) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        if (!(bit & wide.load(std::memory_order_acquire))) {
            e = cudaFuncSetAttribute(evict_kernel<THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R << log_cs, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log_cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<THREADS>, a, log_cs);
}

}  // namespace

cudaError_t kv_evict_launch(const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R, const float *weights,
                            const int32_t *budgets, int budget, int recent, int sinks, int32_t *pages_out,
                            int32_t *indptr_out, float *weights_out, int sms, cudaStream_t st) {
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
    // The lengths are on the device.  A cluster holds a request of the mean
    // length in one round.  Fewer blocks take a long request in rounds (one of
    // 128K: 136 us with 1, 75 with 2, 42 with 4, 25 with 8, 12.8 with 16); more
    // mostly end unused, and each costs its launch (64 requests of 1K to 8K:
    // 9.2 us with 1, 10.5 with 2, 15 with 4, 17 with 8; 128 of 8K to 32K: 44
    // with 2, 34 with 4, 40 with 8; 256 of 128 to 128K: 96 with 2, 77 with 4,
    // 74 with 8, 114 with 16).  A few requests take the blocks that half the
    // SMs hold: these cost nothing (8 of 4K: 7.4 us with 1 to 8, 10 with 16),
    // and one request may be much longer than the mean (15 of 1K and one of
    // 128K: 47 us with 4, 82 with the mean's 2).
    const int64_t mean = (num_pages + R - 1) / R;
    int log_cs = 0;
    while (log_cs < 4 && ((mean >> log_cs) > kRound || ((int64_t)R << (log_cs + 1)) <= sms / 2)) ++log_cs;
    // One block a request and an SM for each: 1,024 threads (64 of 1K to 8K
    // 8.7 us, 9.2 with 512; 63 of 1K and one of 128K 133 and 147).  Elsewhere
    // two blocks of 512 an SM (256 of 512 to 2K 9.9, 12.2 with 1,024; one of
    // 128K 12.8 and 13.7; 128 of 8K to 32K 34 and 57).
    return log_cs == 0 && R <= sms ? launch<1024>(a, log_cs, st) : launch<512>(a, log_cs, st);
}

cudaError_t evict_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
