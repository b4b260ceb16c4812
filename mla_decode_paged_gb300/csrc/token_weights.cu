// Attention weight received by each cached token in one decode step --
// tcgen05 tensor-memory kernel (sm_103a).
//
// What it computes, for token j of request r at entry i = indptr[r] + j of
// the page list:
//   out[i] = decay * weights[i] + sum_{t, h} exp(sc * <q[t, h], K_j> - lse[t, h])
// over r's query rows t that see token j and heads h with lse[t, h] > -inf,
// K_j the e4m3 cache row of pages[i] and sc = scale * q_scale * kv_scale.
// The LSE is given, so one pass over the scores does: no running maximum,
// and a token's sum needs no other token.
//
// Bound by the cache rows (576 bytes a token) up to about 160 query rows a
// request, by the tensor cores above.
//
// Design: one persistent CTA per SM walks a contiguous range of the batch's
// 128-token tiles (equal shares; a request's query is prepared once per CTA
// that meets it).  Tokens are the MMA's M dimension: S[tok, n] = K[tok, :] .
// Q'[n, :] as 18 kind::f8f6f4 MMAs over the e4m3 rows as they are stored, so
// a token is a TMEM lane, one thread sums its row of scores, and no sum
// crosses threads (equal inputs give equal bits).  A bf16 query row is two
// e4m3 terms, q * 2^e = hi + lo / 16 (exact except below 2^-21 of the row's
// largest element), two columns of the same MMA; an fp8 query is one.
//   warps 0..7   two warpgroups take the tiles in turn: scores from TMEM,
//                exponentials, the sum, the output
//   warp 8       MMA issuer (D double-buffered in TMEM, so the next tile's
//                MMAs overlap this tile's exponentials)
//   warps 9..13  producers: one 128- or 64-byte column block each, a
//                gather4 (four cache rows) a lane and tile, two 72 KB stages
//   warps 14..17 convert the next request's query rows once the last MMA on
//                the previous ones has completed
// Up to 64 rows (128 of an fp8 query) fit one CTA's Q' buffer.  Up to 128
// bf16 rows take a pair of CTAs: each holds half of Q' and a 128-token tile
// of its own, and cta_group::2 MMAs give both their tokens' scores with all
// rows, so a cache row still crosses L2 once.  (Two CTAs reading every tile
// for half of the rows each took 213 us against 121 us for 32 x 96 heads, 32K
// tokens: L2 then delivers the cache twice.)  Both CTAs' copies count at CTA
// 0's barriers (a warp of CTA 1 that passed its tiles' arrival on: 164 us to
// 128), and each converts its half of the query only (from both: 128 to 121).
// More rows are cut into groups on neighbouring CTAs (pairs), each writing
// its partial sums to the workspace, joined in group order by a small kernel.
//
// Measured (12 heads, bf16 query): 64 requests of 1K to 8K tokens, one row
// each, in 35 us, 5.0 TB/s of cache rows; 128 of 4K to 32K, four rows each,
// in 257 us, 5.65 TB/s (250 on another GPU; loads alone top out at 5.3 to 5.7
// at this random order of 576-byte rows); 32 of 32K, 96 heads, in 123 us, 5.0
// TB/s: two stages' copies do not cover their latency and the MMAs' 1,940
// cycles.  With an fp8 query, one column a row, 34.4, 246 and 114 us.  Four
// rows of 96 heads (three groups) over 8 requests of 4K to 32K: 61 us, fp8 51,
// where the bytes would take 10 and the MMAs 25 and 12.
// A new request costs the conversion of its query, about 3,400 cycles for 16
// rows (100 requests of 384 rows and 9 to 65 tokens: 58 us; fp8, copied as it
// is, 29).
#include <climits>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "tc.cuh"
#include "tile_walk.cuh"

namespace mla {
namespace {

constexpr int kEpiWarps = 8, kMmaWarp = 8, kProdWarp0 = 9, kProdWarps = 5, kPrepWarp0 = 14, kPrepWarps = 4;
constexpr int kThreads = (kPrepWarp0 + kPrepWarps) * 32;
constexpr int kStages = 2, kTile = 128, kAhead = 8;
constexpr int kLatBlock = (kTile / 8) * 1024;              // one 128-byte column block of a stage
constexpr int kRopeOff = 4 * kLatBlock;
constexpr int kStageBytes = kRopeOff + (kTile / 8) * 512;  // 73,728
constexpr int kOffQ = kStages * kStageBytes;
constexpr long long kTileCycles = 1 << 16;      // more than a tile takes (some 4,700 where it takes longest)

struct TokenArgs {
    const void *q;
    int64_t q_row_stride, pool_rows, num_pages;
    const int32_t *pages, *indptr;
    const float *lse, *weights;
    float *out;             // the result, or (groups > 1) the groups' partial sums
    int64_t group_stride;
    int R, qlen, heads, causal, groups, virt;
    float sc_hi, sc_lo;     // sc * log2(e) as two floats
    float decay;
};

// A query row's constants: with acc = hi + lo / 16, the exponent (base 2) is
// (acc * c.x - c.z) + (acc * c.y - c.w), its two halves each a float pair.
constexpr int kConstBufs = 3;   // a unit's constants outlive two more units' (one-tile units in flight)

// NP columns of Q' in a CTA, TERMS of them per query row; PAIR: two CTAs'
// columns make the MMA's N (CTA 0's first), two tiles its M.
template <int NP, int TERMS, bool PAIR>
struct Cfg {
    static constexpr int NQ = NP / TERMS;               // query rows in this CTA's Q'
    static constexpr int Rows = PAIR ? 2 * NQ : NQ;     // query rows of the MMA
    static constexpr int N = PAIR ? 2 * NP : NP;
    static constexpr int Tokens = PAIR ? 2 * kTile : kTile;
    static constexpr int QLatBlock = (NP / 8) * 1024;
    static constexpr int QRope = 4 * QLatBlock;
    static constexpr int OffMisc = kOffQ + NP * MLA_D_QK;
    static constexpr uint32_t TmemCols = 2 * N <= 64 ? 64 : 2 * N <= 128 ? 128 : 2 * N <= 256 ? 256 : 512;
    // Instruction descriptor: e4m3 operands, f32 sums, M = 128 or 256.
    static constexpr uint32_t Idesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)((PAIR ? 256 : 128) >> 4) << 24);
};

template <class C>
struct Misc {
    float4 c[kConstBufs][C::Rows];
    int vis[kConstBufs][C::Rows];   // tokens of the request that the row counts (0: a skipped row)
    int all_vis[kConstBufs];    // smallest of them over the real rows
    uint64_t kv_full[kStages], kv_empty[kStages], d_full[2], d_free[2], q_ready, q_free, fin;
    uint32_t tmem;
    int abort_flag;
    int issued[kProdWarps];     // PAIR: tiles whose copies each producer has issued
    int start[3];               // this CTA's first request, its first tile there, tiles in all
};

// ------------------------------------------------------------------ producers

// The place of `p` in the shared memory of the pair's block `rank`.
__device__ __forceinline__ uint32_t in_block(const void *p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ int load_in_block(const int *p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(in_block(p, rank)) : "memory");
    return v;
}

// tc::gather4_hint whose bytes count at a barrier of either CTA of the pair
// (`bar`: its shared::cluster address).
__device__ __forceinline__ void gather4_pair(void *dst, const CUtensorMap *map, int x, const int (&rows)[4],
                                             uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(rows[0]), "r"(rows[1]), "r"(rows[2]), "r"(rows[3]), "r"(bar), "l"(policy)
        : "memory");
}

constexpr int part_bytes(int part) { return part < 4 ? 32 * 512 : 32 * 256; }      // of a producer and tile

template <class C, bool PAIR>
__device__ void producer(const TokenArgs &a, const CUtensorMap *mlat, const CUtensorMap *mrope, uint8_t *sm,
                         Misc<C> &ms, int rank) {
    const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) - kProdWarp0;
    Walk<C::Tokens> w;
    w.init(a, ms.start);
    const uint64_t pol = tc::l2_policy(true);   // the rows stream through L2; the query and the outputs stay
    // The page indices of this lane's four tokens; how many of them the request has.
    const auto load = [&](int (&rows)[4]) {
        const int tok0 = w.t * C::Tokens + rank * kTile + 4 * lane;
        const int n = w.valid() ? min(max(w.len - tok0, 0), 4) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = i < n ? __ldg(a.pages + (int64_t)w.base + tok0 + i) : -1;
        return n;
    };
    // Past the request the copy fills zeros (row -1).
    const auto check = [&](int (&rows)[4], int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n && (rows[i] < 0 || rows[i] >= a.pool_rows)) {
                flag(MLA_DEV_BAD_PAGE);
                rows[i] = 0;
            }
    };
    // The page list, contiguous over a CTA's tiles, is brought to L2 kAhead
    // tiles before its indices are read: an index that misses L2 waits behind
    // the stream of rows for several thousand cycles.
    const auto ahead = [&](int tiles) {
        const int64_t at = (int64_t)w.base + (int64_t)(w.t + tiles) * C::Tokens + rank * kTile + 32 * lane;
        if (lane < 5 && at < a.num_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.pages + at));
    };
    if (part == 4 && w.valid())
        for (int k = 1; k < kAhead; ++k) ahead(k);
    int rows[4], it = 0;
    {
        const int n = load(rows);
        check(rows, n);
    }
    bool ok = true;
    while (w.valid()) {
        if (part == 4) ahead(kAhead);
        // The next tile's indices are on their way while this one's copies are issued.
        int next[4];
        w.next(a);
        const int n = load(next);
        const int s = it % kStages;
        if (!(ok = warp_wait(&ms.kv_empty[s], ((it / kStages) & 1) ^ 1, &ms.abort_flag))) break;
        // A pair's tiles are both counted by CTA 0's barrier.
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&ms.kv_full[s], (PAIR ? 2 : 1) * part_bytes(part));
        __syncwarp();
        uint8_t *st = sm + s * kStageBytes;
        const int g8 = lane >> 1, half = lane & 1;
        void *dst = st + (part < 4 ? part * kLatBlock + g8 * 1024 + half * 512 : kRopeOff + g8 * 512 + half * 256);
        const CUtensorMap *map = part < 4 ? mlat : mrope;
        if (PAIR) gather4_pair(dst, map, part * 128, rows, in_block(&ms.kv_full[s], 0), pol);
        else tc::gather4_hint(dst, map, part * 128, rows[0], rows[1], rows[2], rows[3], &ms.kv_full[s], pol);
        ++it;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = next[i];
        check(rows, n);
    }
    if (PAIR) {
        if (lane == 0) ms.issued[part] = it;        // see land
    } else if (!ok) {       // flagged: let the copies in flight land before the CTA ends
        for (int k = it < kStages ? 0 : it - kStages; k < it; ++k) mbar_wait(&ms.kv_full[k % kStages], (k / kStages) & 1);
    }
}

// A pair that gave up (flagged): run by one thread of CTA 0 once neither CTA
// issues any more, lets the copies of both land.  The barriers' last phases
// may lack a producer's arrival or one CTA's bytes, which never come.
template <class C>
__device__ void land(Misc<C> &ms) {
    int most = 0;
    for (int j = 0; j < kProdWarps; ++j) most = max(most, max(ms.issued[j], load_in_block(&ms.issued[j], 1)));
    for (int k = max(most - kStages, 0); k < most; ++k) {
        uint64_t *bar = &ms.kv_full[k % kStages];
        for (int j = 0; j < kProdWarps; ++j) {
            const bool here = k < ms.issued[j], there = k < load_in_block(&ms.issued[j], 1);
            if (!here)
                mbar_arrive_expect_tx(bar, there ? part_bytes(j) : 0);
            else if (!there)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                             "r"(part_bytes(j))
                             : "memory");
        }
        mbar_wait(bar, (k / kStages) & 1);
    }
}

// ------------------------------------------------------------------ MMA issuer

// Run by the whole warp, its arguments the same in every lane; `one` set in
// the lane that issues (a branch around it would keep the descriptors out of
// the uniform registers).
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                    uint32_t one) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(one));
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(one));
}

// Arrive on `bar` (PAIR: in both CTAs) once this thread's MMAs so far have completed.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        tc::commit(bar);
}

// Arrive on CTA 0's `bar`, from either CTA of a pair.  RELAXED: where only
// TMEM reads (fenced by the caller) go before it; a release at cluster scope
// would wait for this thread's global stores, several thousand cycles under
// the stream of rows.
template <bool PAIR, bool RELAXED = false>
__device__ __forceinline__ void arrive_lead(uint64_t *bar, int rank) {
    if (!PAIR || rank == 0)
        mbar_arrive(bar);
    else if (RELAXED)
        asm volatile(
            "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
            "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
            "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
            : "memory");
}

// mbar_wait for what the other CTA has written too.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t par) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(par)
            : "memory");
        if (ok) return true;
        if (clock64() - t0 > kWaitCycles) {
            flag(MLA_DEV_TIMEOUT);
            return false;
        }
    }
}

template <bool PAIR>
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t par) {
    return PAIR ? mbar_wait_cluster(bar, par) : mbar_wait(bar, par);
}

// CTA 0 issues a pair's; its last commit, to `fin` in both CTAs, is waited for
// by CTA 1 at the kernel's end.
template <int NP, int TERMS, bool PAIR>
__device__ void mma_issuer(const TokenArgs &a, uint8_t *sm, Misc<Cfg<NP, TERMS, PAIR>> &ms, int rank) {
    using C = Cfg<NP, TERMS, PAIR>;
    const uint32_t base = smem_u32(sm), tm = ms.tmem;
    const uint32_t one = tc::elect_one();
    const uint64_t lat0 = tc::sdesc(base, 16, 1024, tc::kSw128), rope0 = tc::sdesc(base + kRopeOff, 16, 512, tc::kSw64);
    const uint64_t q0 = tc::sdesc(base + kOffQ, 16, 1024, tc::kSw128);
    const uint64_t qr0 = tc::sdesc(base + kOffQ + C::QRope, 16, 512, tc::kSw64);
    Walk<C::Tokens> w;
    w.init(a, ms.start);
    if (PAIR && rank > 0) return;
    for (int it = 0; w.valid(); ++it, w.next(a)) {
        const int s = it % kStages, d = it & 1;
        const bool ready = !aborted(&ms.abort_flag) && (!w.first || wait_pair<PAIR>(&ms.q_ready, w.unit & 1)) &&
                           wait_pair<PAIR>(&ms.d_free[d], ((it >> 1) & 1) ^ 1) &&
                           wait_pair<PAIR>(&ms.kv_full[s], (it / kStages) & 1);
        if (!warp_agrees(ready, &ms.abort_flag)) break;
        tc::fence_after();
        // Column blocks of 128 bytes, 32 bytes a step (an address counts 16).
        const uint32_t dt = tm + d * C::N;
        const uint64_t lat = lat0 + s * (kStageBytes >> 4), rope = rope0 + s * (kStageBytes >> 4);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            mma<PAIR>(dt, lat + (j >> 2) * (kLatBlock >> 4) + (j & 3) * 2,
                      q0 + (j >> 2) * (C::QLatBlock >> 4) + (j & 3) * 2, C::Idesc, j > 0, one);
#pragma unroll
        for (int j = 0; j < 2; ++j) mma<PAIR>(dt, rope + j * 2, qr0 + j * 2, C::Idesc, true, one);
        if (one) {
            commit<PAIR>(&ms.kv_empty[s]);
            commit<PAIR>(&ms.d_full[d]);
            if (w.last()) commit<PAIR>(&ms.q_free);
        }
        __syncwarp();
    }
    // Every MMA issued must be complete before TMEM is released.
    if (one) commit<PAIR>(&ms.fin);
    __syncwarp();
    mbar_wait(&ms.fin, 0);
}

// ------------------------------------------------------------------ query

// Byte offset of column d of Q' row n.
template <class C>
__device__ __forceinline__ uint32_t q_offset(int n, int d) {
    return d < 512 ? kOffQ + (d >> 7) * C::QLatBlock + (n >> 3) * 1024 + tc::sw128(n, d & 127)
                   : kOffQ + C::QRope + (n >> 3) * 512 + tc::sw64(n, d - 512);
}

// The constants of request r's rows [grp * Rows, ...) and the rows as the B
// operand, a warp a row; a pair's CTAs take half of them each and write the
// constants to both.
template <int NP, int TERMS, bool PAIR>
__device__ void prep_unit(const TokenArgs &a, uint8_t *sm, Misc<Cfg<NP, TERMS, PAIR>> &ms, int r, int len, int grp,
                          int unit, int rank) {
    using C = Cfg<NP, TERMS, PAIR>;
    constexpr int NQ = C::NQ;
    const int lane = threadIdx.x & 31, pw = (threadIdx.x >> 5) - kPrepWarp0, buf = unit % kConstBufs;
    const int rows_total = a.qlen * a.heads;
    if (pw == 0) {
        int least = INT_MAX;
        for (int n = lane; n < C::Rows; n += 32) {
            const int rho = grp * C::Rows + n;
            int vis = 0;
            if (rho < rows_total) {
                const int t = rho / a.heads;
                const float lse = __ldg(a.lse + ((int64_t)r * a.qlen) * a.heads + rho);
                vis = a.causal ? max(0, len - a.qlen + t + 1) : len;
                if (lse == -INFINITY) vis = 0;
                least = min(least, vis);
            }
            ms.vis[buf][n] = vis;
        }
        for (int d = 16; d >= 1; d >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, d));
        if (lane == 0) ms.all_vis[buf] = least;
    }
    // Lane i: the LSE of the warp's i-th row.
    float lses = -INFINITY;
    static_assert(NQ <= 32 * kPrepWarps, "a lane per row of a warp");
    {
        const int rho = grp * C::Rows + rank * NQ + pw + kPrepWarps * lane;
        if (pw + kPrepWarps * lane < NQ && rho < rows_total) lses = __ldg(a.lse + (int64_t)r * rows_total + rho);
    }
    // Four rows' loads in flight a warp.
    constexpr int kBatch = 4, kVecs = TERMS == 1 ? 2 : 3;   // 16-byte vectors of a row a lane
    static_assert(NQ % (kBatch * kPrepWarps) == 0, "whole batches");
#pragma unroll 1
    for (int i0 = 0; i0 < NQ / kPrepWarps; i0 += kBatch) {
        uint4 v[kBatch][kVecs];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int rho = grp * C::Rows + rank * NQ + pw + kPrepWarps * (i0 + i);
            const int t = rho / a.heads, h = rho - t * a.heads;
            const uint8_t *src = static_cast<const uint8_t *>(a.q) +
                                 (((int64_t)r * a.qlen + t) * a.q_row_stride + (int64_t)h * MLA_D_QK) * TERMS;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int ch = lane + 32 * j;
                v[i][j] = rho < rows_total && ch < MLA_D_QK * TERMS / 16 ? __ldg(reinterpret_cast<const uint4 *>(src) + ch)
                                                                         : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int n = pw + kPrepWarps * (i0 + i), row = rank * NQ + n;     // of this CTA's Q', of the group
            float back = 1.f;                   // 2^-e
            if (TERMS == 1) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int ch = lane + 32 * j;
                    if (ch < MLA_D_QK / 16) *reinterpret_cast<uint4 *>(sm + q_offset<C>(n, ch * 16)) = v[i][j];
                }
            } else {
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const uint32_t x[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[e])), fabsf(bf16_hi(x[e]))));
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                // amax = f * 2^(ex - 127), 1 <= f < 2: scaled by 2^e into [128, 256).
                const int ex = min(max((int)(__float_as_uint(amax) >> 23), 40), 254);
                const float up = __uint_as_float((uint32_t)(127 + 134 - ex) << 23);
                back = __uint_as_float((uint32_t)(127 + ex - 134) << 23);
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int ch = lane + 32 * j;
                    if (ch >= MLA_D_QK / 8) continue;
                    const uint32_t x[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // hi is x rounded to 4 bits; the difference, at most 4 bits more, and 16 times it are exact.
                        const float2 f = make_float2(bf16_lo(x[e]) * up, bf16_hi(x[e]) * up);
                        const __nv_fp8x2_storage_t h8 = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                        const float2 hf = unpack_f16x2(e4m3x2_to_f16x2(h8));
                        const __nv_fp8x2_storage_t l8 = __nv_cvt_float2_to_fp8x2(
                            make_float2((f.x - hf.x) * 16.f, (f.y - hf.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
                        if (e & 1) {
                            hi[e >> 1] |= (uint32_t)h8 << 16;
                            lo[e >> 1] |= (uint32_t)l8 << 16;
                        } else {
                            hi[e >> 1] = h8;
                            lo[e >> 1] = l8;
                        }
                    }
                    *reinterpret_cast<uint2 *>(sm + q_offset<C>(n, ch * 8)) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(sm + q_offset<C>(NQ + n, ch * 8)) = make_uint2(lo[0], lo[1]);
                }
            }
            // lse * log2(e) as a float pair (log2(e) itself as one).
            const float lse = __shfl_sync(0xffffffffu, lses, i0 + i);
            float4 c = make_float4(0.f, 0.f, INFINITY, 0.f);   // a row that counts nothing: 2^-inf
            if (lse != -INFINITY) {
                constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLo = 1.92596299112661746e-8f;
                c.x = a.sc_hi * back;
                c.y = a.sc_lo * back;
                c.z = lse * kLog2e;
                c.w = isinf(c.z) ? 0.f : fmaf(lse, kLog2e, -c.z) + lse * kLog2eLo;
            }
            if (lane == 0) {
                ms.c[buf][row] = c;
                if (PAIR)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(in_block(&ms.c[buf][row], rank ^ 1)),
                                 "f"(c.x), "f"(c.y), "f"(c.z), "f"(c.w)
                                 : "memory");
            }
        }
    }
}

// This CTA's rows of a request into L2, ahead of their conversion.
template <class C, int TERMS>
__device__ void prefetch_rows(const TokenArgs &a, int r, int grp, int rank) {
    const int rows_total = a.qlen * a.heads;
    const uint64_t keep = tc::l2_policy_last();
    for (int row = threadIdx.x - kPrepWarp0 * 32; row < C::NQ; row += kPrepWarps * 32) {
        const int rho = grp * C::Rows + rank * C::NQ + row;
        if (rho >= rows_total) break;
        const int t = rho / a.heads, h = rho - t * a.heads;
        tc::bulk_prefetch_l2(static_cast<const uint8_t *>(a.q) +
                                 (((int64_t)r * a.qlen + t) * a.q_row_stride + (int64_t)h * MLA_D_QK) * TERMS,
                             MLA_D_QK * TERMS, keep);
    }
}

// ------------------------------------------------------------------ scores

// One token's sum over the query rows; MASK: rows count tokens below their
// vis only.  HALVES blocks of NP columns, each its rows' hi then lo terms.
// Eight rows' scores leave TMEM while the eight before are summed.  A loop,
// not unrolled over all rows: 96 rows of straight code per warp do not stay
// in the instruction cache.
template <int NP, int TERMS, int HALVES, bool MASK>
__device__ __forceinline__ float token_sum(uint32_t taddr, const float4 *c, const int *vis, int j) {
    constexpr int NQ = NP / TERMS, kGroups = NQ * HALVES / 8;
    static_assert(kGroups % 2 == 0, "groups in pairs");
    float sum[2] = {0.f, 0.f};
    float acc[2][8], lo[2][8];
    const auto load = [&](int b, int g) {
        const uint32_t at = taddr + g * 8 + (HALVES == 2 && g >= kGroups / 2 ? NP - NQ : 0);
        tc::ld8(at, acc[b]);
        if (TERMS == 2) tc::ld8(at + NQ, lo[b]);
    };
    const auto add = [&](int b, int g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 k = c[8 * g + i];
            const float x = TERMS == 2 ? fmaf(lo[b][i], 0.0625f, acc[b][i]) : acc[b][i];
            const float p = tc::exp2_approx(fmaf(x, k.x, -k.z) + fmaf(x, k.y, -k.w));
            sum[i & 1] += !MASK || j < vis[8 * g + i] ? p : 0.f;
        }
    };
    load(0, 0);
    tc::wait_ld();
#pragma unroll 1
    for (int g = 0; g < kGroups; g += 2) {
        load(1, g + 1);
        add(0, g);
        tc::wait_ld();
        if (g + 2 < kGroups) load(0, g + 2);
        add(1, g + 1);
        tc::wait_ld();
    }
    return sum[0] + sum[1];
}

template <int NP, int TERMS, bool PAIR>
__device__ void epilogue(const TokenArgs &a, Misc<Cfg<NP, TERMS, PAIR>> &ms, int grp, int rank) {
    using C = Cfg<NP, TERMS, PAIR>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, wq = warp & 3;
    const uint32_t taddr = ms.tmem + wg * C::N + ((uint32_t)(32 * wq) << 16);
    float *out = a.out + (int64_t)grp * a.group_stride;
    Walk<C::Tokens> w;
    w.init(a, ms.start);
    for (int it = 0; w.valid(); ++it, w.next(a)) {
        if ((it & 1) != wg) continue;
        const int j0 = w.t * C::Tokens + rank * kTile, j = j0 + 32 * wq + lane, buf = w.unit % kConstBufs;
        const int64_t i = (int64_t)w.base + j;
        const bool real = j < w.len;
        float old = 0.f;
        if (a.decay != 0.f && real) old = a.weights[i] * a.decay;
        if (!warp_wait(&ms.d_full[wg], (it >> 1) & 1, &ms.abort_flag)) break;
        tc::fence_after();
        const bool whole = ms.all_vis[buf] >= min(j0 + kTile, w.len);
        constexpr int kHalves = PAIR ? 2 : 1;
        const float sum = whole ? token_sum<NP, TERMS, kHalves, false>(taddr, ms.c[buf], ms.vis[buf], j)
                                : token_sum<NP, TERMS, kHalves, true>(taddr, ms.c[buf], ms.vis[buf], j);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead<PAIR, true>(&ms.d_free[wg], rank);
        if (real) out[i] = old + sum;
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        tc::tmem_alloc(dst, cols);
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
    else tc::tmem_free(base, cols);
}

// All threads of the CTA, or of both.  (The cluster barrier is for whole
// warps: lanes that took a branch before it meet first.)
template <bool PAIR>
__device__ __forceinline__ void sync_all() {
    __syncwarp();
    if (PAIR)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
}

template <int NP, int TERMS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    token_weights_kernel(const __grid_constant__ CUtensorMap mlat, const __grid_constant__ CUtensorMap mrope,
                         const TokenArgs a) {
    using C = Cfg<NP, TERMS, PAIR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<C> &ms = *reinterpret_cast<Misc<C> *>(sm + C::OffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // A pair's blocks are neighbours (a cluster), and so are a tile's row groups.
    const int rank = PAIR ? blockIdx.x & 1 : 0, unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, grp = unit % a.groups;
    if (tid == 0) {
        const int more = PAIR && rank == 0;         // CTA 0 also hears of CTA 1's
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ms.kv_full[s], kProdWarps);
            mbar_init(&ms.kv_empty[s], 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(&ms.d_full[d], 1);
            mbar_init(&ms.d_free[d], 4 + 4 * more);
        }
        mbar_init(&ms.q_ready, kPrepWarps + kPrepWarps * more);
        mbar_init(&ms.q_free, 1);
        mbar_init(&ms.fin, 1);
        ms.abort_flag = 0;
        ms.start[0] = ms.start[1] = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc<PAIR>(&ms.tmem, C::TmemCols);
    tc::fence_before();
    sync_all<PAIR>();
    tc::fence_after();
    find_start<C::Tokens, kThreads>(a, ms.start, unit / a.groups);
    if (warp < kEpiWarps) {
        epilogue<NP, TERMS, PAIR>(a, ms, grp, rank);
    } else if (warp == kMmaWarp) {
        mma_issuer<NP, TERMS, PAIR>(a, sm, ms, rank);
    } else if (warp < kPrepWarp0) {
        producer<C, PAIR>(a, &mlat, &mrope, sm, ms, rank);
    } else {
        Walk<C::Tokens> w;
        w.init(a, ms.start);
        int tiles = 0;      // of the request before this one, here
        for (; w.valid(); w.next(a), ++tiles) {
            if (!w.first) continue;
            // The last of all the MMAs of the request before: a wait for its
            // tiles, not for one (2,048 query rows of 2^30 tokens take seconds).
            if (w.unit > 0 &&
                !warp_wait_long(&ms.q_free, (w.unit - 1) & 1, &ms.abort_flag, kWaitCycles + tiles * kTileCycles))
                break;
            tiles = 0;
            prep_unit<NP, TERMS, PAIR>(a, sm, ms, w.r, w.len, grp, w.unit, rank);
            tc::fence_async_smem();     // generic-proxy writes -> tensor-core reads
            __syncwarp();
            if (lane == 0) {
                if (PAIR) asm volatile("fence.acq_rel.cluster;" ::: "memory");      // the constants in the other CTA
                arrive_lead<PAIR>(&ms.q_ready, rank);
            }
            // The next request's (a few empty ones passed over), if this CTA gets to it.
            if (w.left > w.ntiles - w.t) {
                int r = w.r + 1, base;
                const int end = min(a.R, r + 32);
                while (r < end && request_len(a.indptr, r, a.num_pages, &base) == 0) ++r;
                if (r < end) prefetch_rows<C, TERMS>(a, r, grp, rank);
            }
        }
    }
    // Neither CTA of a pair ends while the other may still reach it.
    tc::fence_before();
    sync_all<PAIR>();
    if (PAIR) {
        // CTA 0's commits have completed there; those to this CTA's barriers land before it ends.
        if (rank > 0 && warp == kMmaWarp) mbar_wait(&ms.fin, 0);
        if ((ms.abort_flag || load_in_block(&ms.abort_flag, rank ^ 1)) && tid == 0 && rank == 0) land(ms);
        sync_all<PAIR>();
    }
    tc::fence_after();
    if (warp == kMmaWarp) tmem_free<PAIR>(ms.tmem, C::TmemCols);
}

// out[i] = decay * weights[i] + the groups' partial sums, in group order.
__global__ void __launch_bounds__(256) join_kernel(const TokenArgs a, const float *__restrict__ parts, float *out,
                                                   float decay) {
    int base;
    const int len = request_len(a.indptr, blockIdx.x, a.num_pages, &base);
    // 64 bits: a step of the grid past the last token may pass 32.
    for (int64_t j = blockIdx.y * 256 + threadIdx.x; j < len; j += gridDim.y * 256) {
        const int64_t i = base + j;
        float sum = parts[i];
        for (int g = 1; g < a.groups; ++g) sum += parts[i + g * a.group_stride];
        out[i] = decay == 0.f ? sum : fmaf(a.weights[i], decay, sum);
    }
}

// The cache as [pool_rows, 576] bytes, read in rows of `cols` bytes.
bool encode_rows(CUtensorMap *m, const void *kv, int64_t pool_rows, cuuint32_t cols, CUtensorMapSwizzle swz) {
    const cuuint64_t dim[2] = {(cuuint64_t)MLA_D_QK, (cuuint64_t)pool_rows}, stride[1] = {(cuuint64_t)MLA_D_QK};
    const cuuint32_t box[2] = {cols, 1}, es[2] = {1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(kv), dim, stride, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a request's query rows are laid out: `groups` of CTAs (or pairs), np
// columns of Q' in each CTA.
struct Shape {
    int groups, np;
    bool pair;
};

// The fewest groups of at most 128 columns a CTA, each as narrow as that
// allows (steps of 32 columns); bf16 rows above one CTA's 64 take pairs.
Shape shape(int rows, int terms) {
    Shape s;
    s.pair = terms == 2 && rows > 64;
    const int most = (s.pair ? 256 : 128) / terms;
    s.groups = (rows + most - 1) / most;
    const int n = (rows + s.groups - 1) / s.groups * terms;     // columns of a group
    s.np = ((s.pair ? (n + 1) / 2 : n) + 31) / 32 * 32;
    return s;
}

template <int NP, int TERMS, bool PAIR>
cudaError_t launch(const CUtensorMap &ml, const CUtensorMap &mr, const TokenArgs &a, cudaStream_t st) {
    using C = Cfg<NP, TERMS, PAIR>;
    constexpr int smem = C::OffMisc + sizeof(Misc<C>) + 1024;
    static_assert(smem <= 226 * 1024, "shared memory of one CTA");
    cudaError_t e = smem_attr_once<token_weights_kernel<NP, TERMS, PAIR>>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.virt * a.groups * (PAIR ? 2 : 1), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, token_weights_kernel<NP, TERMS, PAIR>, ml, mr, a);
}

cudaError_t launch_shape(const Shape &s, bool q8, const CUtensorMap &ml, const CUtensorMap &mr, const TokenArgs &a,
                         cudaStream_t st) {
    if (s.pair) return s.np <= 96 ? launch<96, 2, true>(ml, mr, a, st) : launch<128, 2, true>(ml, mr, a, st);
    switch (s.np) {
        case 32: return q8 ? launch<32, 1, false>(ml, mr, a, st) : launch<32, 2, false>(ml, mr, a, st);
        case 64: return q8 ? launch<64, 1, false>(ml, mr, a, st) : launch<64, 2, false>(ml, mr, a, st);
        case 96: return q8 ? launch<96, 1, false>(ml, mr, a, st) : launch<96, 2, false>(ml, mr, a, st);
        default: return q8 ? launch<128, 1, false>(ml, mr, a, st) : launch<128, 2, false>(ml, mr, a, st);
    }
}

}  // namespace

int64_t token_weights_workspace(int rows, bool q8, int64_t num_pages) {
    const int groups = shape(rows, q8 ? 1 : 2).groups;
    return groups > 1 ? (int64_t)groups * num_pages * 4 : 0;
}

cudaError_t token_weights_launch(const void *q, int64_t q_row_stride, const void *kv, int64_t pool_rows,
                                 const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R, int qlen,
                                 int heads, double sc, const float *lse, float decay, const float *weights, float *out,
                                 bool causal, bool q8, void *workspace, int sms, cudaStream_t st) {
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    CUtensorMap ml, mr;
    if (!encode_rows(&ml, kv, pool_rows, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_rows(&mr, kv, pool_rows, 64, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    TokenArgs a = {};
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.pool_rows = pool_rows;
    a.num_pages = num_pages;
    a.pages = pages;
    a.indptr = indptr;
    a.lse = lse;
    a.weights = weights;
    a.R = R;
    a.qlen = qlen;
    a.heads = heads;
    a.causal = causal;
    const double sc2 = sc * 1.4426950408889634;
    a.sc_hi = (float)sc2;
    a.sc_lo = (float)(sc2 - (double)a.sc_hi);
    const Shape s = shape(qlen * heads, q8 ? 1 : 2);
    a.groups = s.groups;
    const int ctas = a.groups * (s.pair ? 2 : 1);
    a.virt = sms / ctas < 1 ? 1 : sms / ctas;
    a.out = a.groups > 1 ? static_cast<float *>(workspace) : out;
    a.group_stride = num_pages;
    a.decay = a.groups > 1 ? 0.f : decay;
    cudaError_t e = launch_shape(s, q8, ml, mr, a, st);
    if (e != cudaSuccess || a.groups == 1) return e;
    const int chunks = (sms * 8 + R - 1) / R;
    join_kernel<<<dim3(R, chunks < 65535 ? chunks : 65535), 256, 0, st>>>(a, static_cast<const float *>(workspace), out,
                                                                         decay);
    return cudaGetLastError();
}

cudaError_t token_weights_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
