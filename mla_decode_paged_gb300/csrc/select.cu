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
// Design: a cluster of blocks per row, as many of them as it takes to hold it
// (the others end at once), each with a contiguous slice of its token blocks
// and every warp with a contiguous part of that, whose keys (order-preserving
// 32-bit images of the scores) stay in registers: 8,192 a block.  A longer
// slice is taken in rounds of that size, read again for every step.  Blocks
// of more than one token get their keys first, in shared memory, from
// coalesced reads of 32 tokens a warp.  The m-th largest key is found by
// radix selection, 11 + 11 + 10 bits, ended by the digits whose keys all
// stay, over histograms summed through distributed shared memory.  What each
// warp keeps is counted by ballots, the offsets of warps and blocks are
// exchanged once, and the kept are placed by the ballots again.
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

constexpr int kBins = 2048, kDigits = 3;
constexpr int kRound = 8192;       // token blocks a block holds

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

template <int WARPS>
struct __align__(16) Shared {
    uint32_t hist[kDigits][kBins];
    uint32_t sums[kDigits][kBins];  // of this block's share of the bins, over the cluster
    uint32_t red[2][WARPS];
    uint32_t scan[WARPS];
    uint32_t warp_kept[WARPS], warp_ties[WARPS];
    uint32_t totals[2];             // this block's sure blocks and ties, for the cluster
    uint32_t pick[3];
};

// A round's keys, and the blocks that stay in order (BLOCKED only).
struct Held {
    uint32_t key[kRound];
    int32_t kept[kRound];
};

template <int THREADS, bool BLOCKED>
constexpr int smem_bytes() {
    return sizeof(Shared<THREADS / 32>) + (BLOCKED ? sizeof(Held) : 0);
}

// Blocks it takes to hold a row's tokens, as a power of two up to log_cs.
__device__ __forceinline__ int blocks_for(int tokens, int log_cs) {
    int le = 0;
    while (le < log_cs && (tokens >> le) > kRound) ++le;
    return le;
}

// 2^log_cs blocks (a cluster) per row.
template <int THREADS, bool BLOCKED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(const SelectArgs a, int log_cs) {
    constexpr int kWarps = THREADS / 32;
    constexpr int kSteps = kRound / THREADS, kOwn = kBins / THREADS;    // keys a thread holds; bins it sums
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared<kWarps> &sh = *reinterpret_cast<Shared<kWarps> *>(smem_raw);
    Held &held = *reinterpret_cast<Held *>(smem_raw + sizeof(Shared<kWarps>));      // BLOCKED only
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1, rank = block_rank();
    const int rows = a.R * a.qlen, b = blockIdx.x >> log_cs, lb = a.log_block;
    const Row row = row_of(a, b);
    // The blocks past those that hold the row end (a cluster barrier waits for
    // running threads only).
    const int le = blocks_for(row.seen, log_cs);
    const uint32_t E = 1u << le;
    if (rank >= E) return;
    const bool one = le == 0;
    const int recent = min(a.recent, row.kept), sinks = min(a.sinks, row.kept - recent);
    const int lo = sinks, hi = row.blocks - recent;     // the blocks that may go
    const int m = row.kept - recent - sinks;            // how many of them stay
    const float *w = a.scores + (int64_t)(b % a.qlen) * a.num_pages + row.base;

    // This block's slice, in rounds; a warp's part of a round, whole groups of
    // 32.  Key 0: none that may go.
    const int slice = (((row.blocks + (int)E - 1) >> le) + 31) / 32 * 32;
    const int s0 = (int)min((int64_t)slice * rank, (int64_t)row.blocks), s1 = min(slice, row.blocks - s0) + s0;
    const int rounds = (s1 - s0 + kRound - 1) / kRound;
    uint32_t key[kSteps];
    uint32_t valid = 0, free = 0;   // a bit a step: a block, one that may go
    int first = 0, steps = 0, round0 = 0;
    const auto place = [&](int q) {
        round0 = s0 + q * kRound;
        const int q1 = min(round0 + kRound, s1);
        const int part = ((q1 - round0 + kWarps - 1) / kWarps + 31) / 32 * 32;
        first = round0 + warp * part + lane;
        steps = part / 32;
        valid = free = 0;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int i = first + 32 * j;
            if (j < steps && i < q1) {
                valid |= 1u << j;
                if (i >= lo && i < hi) free |= 1u << j;
            }
        }
        return q1;
    };
    const auto load = [&](int q) {
        const int q1 = place(q);
        if (!BLOCKED) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) key[j] = (free >> j & 1) ? __float_as_uint(__ldg(w + first + 32 * j)) : 0;
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (free >> j & 1) key[j] = weight_key(__uint_as_float(key[j]));
        } else {
            // The round's block maxima: warps take 32 tokens in turn, eight of
            // these reads in flight; the lanes of a block join by shuffles.
            __syncthreads();
            for (int i = tid; i < q1 - round0; i += THREADS) held.key[i] = 0;
            __syncthreads();
            const int t0 = max(round0, lo) << lb, t1 = min(min(q1, hi) << lb, row.seen);
            for (int at = t0 + 32 * warp; at < t1; at += 32 * 8 * kWarps) {
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
                        if (lane == 0) atomicMax(&held.key[(t >> lb) - round0], x);
                    } else {
                        for (int d = 1; d < 1 << lb; d <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if ((t & ((1 << lb) - 1)) == 0 && t < t1) held.key[(t >> lb) - round0] = x;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kSteps; ++j) key[j] = (free >> j & 1) ? held.key[first + 32 * j - round0] : 0;
        }
    };
    const bool select = m > 0 && m < hi - lo;       // the same in every block of the cluster
    if (select && rounds > 0) load(0);
    else if (rounds > 0) place(0);
    for (int i = tid; i < kDigits * kBins / 4; i += THREADS)
        reinterpret_cast<uint4 *>(&sh.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    if (!one) {
        for (int i = tid; i < kDigits * kBins / 4; i += THREADS)
            reinterpret_cast<uint4 *>(&sh.sums[0][0])[i] = make_uint4(0, 0, 0, 0);
        cluster_arrive();       // waited for before the first sums are added to
    }
    // Kept tokens of the rows before this one, and of all.
    uint32_t before = 0, all_tokens = 0;
    if (a.scanned) {
        before = (uint32_t)__ldg(a.indptr_out + b);
        all_tokens = (uint32_t)__ldg(a.indptr_out + rows);
        __syncthreads();        // the histograms' zeros
    } else {
        const uint32_t t = tid < rows ? (uint32_t)row_of(a, tid).tokens : 0;
        const uint32_t x = __reduce_add_sync(0xffffffffu, tid < b ? t : 0), y = __reduce_add_sync(0xffffffffu, t);
        if (lane == 0) {
            sh.red[0][warp] = x;
            sh.red[1][warp] = y;
        }
        __syncthreads();
        before = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[0][lane] : 0);
        all_tokens = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red[1][lane] : 0);
        if (tid == 0 && rank == 0) {
            if (b == 0) a.indptr_out[0] = 0;
            a.indptr_out[b + 1] = (int32_t)(before + row.tokens);
        }
    }

    // The m-th largest key T of [lo, hi), and how many keys equal to T stay.
    uint32_t T = 0, ties = 0;
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
                    if ((free >> j & 1) && (digit == 0 || (key[j] ^ T) >> above_bits == 0))
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

    // A block outside [lo, hi), or any when all stay, is sure; between, those
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
    const auto again = [&](int q) {
        if (select) load(q);
        else place(q);
    };
    uint32_t nsure = 0, nties = 0, k, t, kb, tb;
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) again(q);
        count(nsure, nties);
    }
    exchange(nsure, nties, k, t, kb, tb);
    uint32_t block_kept = 0, block_ties = 0;        // sure blocks and ties of the thread blocks before this one
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

    // Placement, in position order.  Places past the output (only requests
    // that share entries, a bad indptr, make them) are dropped.
    const int32_t *pages = a.pages + row.base;
    const int64_t limit = a.capacity;
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1) {
            again(q);
            nsure = nties = 0;
            count(nsure, nties);
            exchange(nsure, nties, k, t, kb, tb);
        }
        uint32_t kept_at = block_kept + kb, ties_at = block_ties + tb;
        // kept blocks of the row before this round: the sure ones and the ties among the first `ties`
        const uint32_t round_first = block_kept + min(block_ties, ties);
        const uint32_t round_kept = k + (min(block_ties + t, ties) - min(block_ties, ties));
        block_kept += k;
        block_ties += t;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if (j >= steps) break;
            const uint32_t ms = __ballot_sync(0xffffffffu, sure >> j & 1);
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
            if (!keep) continue;
            const int i = first + 32 * j;
            if (BLOCKED) {
                held.kept[rank_i - round_first] = i;
            } else {
                const uint32_t at = before + rank_i;
                if (at < limit) a.pages_out[at] = __ldg(pages + i);
            }
        }
        if (BLOCKED) {
            __syncthreads();
            const uint32_t n = round_kept << lb, to = before + (round_first << lb);
            for (uint32_t x = tid; x < n; x += THREADS) {
                const int i = (held.kept[x >> lb] << lb) + (int)(x & ((1u << lb) - 1));
                if (i < row.seen && to + x < limit) a.pages_out[to + x] = __ldg(pages + i);
            }
            __syncthreads();
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

template <int THREADS, bool BLOCKED>
cudaError_t launch(SelectArgs a, int log_cs, cudaStream_t st) {
    constexpr int smem = smem_bytes<THREADS, BLOCKED>();
    cudaError_t e = smem_attr_once<select_kernel<THREADS, BLOCKED>>(smem);
    if (e != cudaSuccess) return e;
    static std::atomic<unsigned long long> wide{0};     // devices where clusters of 16 have been allowed
    if (log_cs > 3) {
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        if (!(bit & wide.load(std::memory_order_acquire))) {
            e = cudaFuncSetAttribute(select_kernel<THREADS, BLOCKED>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<THREADS, BLOCKED>, a, log_cs);
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
    while (log_cs < 4 && ((mean >> log_cs) > kRound || (rows << (log_cs + 1)) <= sms / 2)) ++log_cs;
    const bool wide = log_cs == 0 && rows <= sms;       // one block a row and an SM for each
    if (block > 1) return wide ? launch<1024, true>(a, log_cs, st) : launch<512, true>(a, log_cs, st);
    return wide ? launch<1024, false>(a, log_cs, st) : launch<512, false>(a, log_cs, st);
}

cudaError_t index_select_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
