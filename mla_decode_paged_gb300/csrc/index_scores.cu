// A cheap score of every cached token for every query row: what a sparse
// attention picks its tokens by -- tcgen05 kernel (sm_103a).
//
// What it computes, for token j of request r at entry i = indptr[r] + j of
// the page list and query row t = r * qlen + tq:
//   out[tq, i] = sum_h ws[t, h] * max(0, <q[t, h], K_i>),  ws = weights * q_scales * scale
// with K_i the 128 e4m3 codes of row pages[i] of the index cache; -inf where
// row tq does not see the token.
//
// Bound by DRAM up to about 128 heads x rows a request (128 bytes a token,
// and 4 a row of output), by the epilogue's two operations a token, head and
// row above.  Rows of 128 bytes from random places come at 5.6 TB/s at most
// (plain 16-byte loads of as many in flight as the SMs hold).  32 requests of
// 32K tokens, 64 heads: 30.6 us (4.7 TB/s); 128 x 4 rows of 4K to 32K, 32
// heads: 75 (4.9; without the sums 65); 64 requests of 1K to 8K, 64 heads: 13;
// 256 x 8 rows of 128 to 128K 161 with 12 heads (5.1), 292 with 32, 538 with 64
// (1.2 PFLOP/s: the sums, and the tiles walked twice above 256 columns).
//
// Design: one persistent CTA per SM walks a contiguous range of the batch's
// 128-token tiles.  Tokens are the MMA's M dimension, heads of some query
// rows its N (a row's heads padded to 16 columns): a token is a TMEM lane, one
// thread sums its heads, and no sum crosses threads (equal inputs give equal
// bits).  A cache row is 128 bytes, one swizzled row of the operand, so a
// gather4 fetches four tokens whole.
//   warps 0..15   four warpgroups take the tiles in turn: the sums, the output
//                 (two: 106 us for the 128 x 4 rows)
//   warp 16       MMA issuer; four accumulators in TMEM up to 128 columns, two above
//   warps 17..20  producers, a tile in four each: a gather4 a lane (the lanes'
//                 copies are issued one by one: two warps 106 us, six 76)
//   warp 21       a request's query by TMA and its weights, two requests deep
// Rows whose heads exceed 256 columns are cut into groups on neighbouring
// CTAs, which read the same tiles at about the same time.
#include <cuda_runtime.h>

#include "common.cuh"
#include "tc.cuh"
#include "tile_walk.cuh"
#include "vec8.cuh"

namespace mla {
namespace {

constexpr int kMmaWarp = 16, kProdWarp0 = 17, kProdWarps = 4, kPrepWarp = 21;
constexpr int kThreads = (kPrepWarp + 1) * 32;
constexpr int kTile = 128, kRow = MLA_D_INDEX, kStages = 8, kAhead = 8;
constexpr int kStageBytes = kTile * kRow;
constexpr int kCols = 256;                          // columns of a group, at most
constexpr int kTmemCols = 512;                      // four tiles of up to 128 columns in flight, or two
constexpr int kQBufs = 2, kConstBufs = 8;           // requests' queries; their weights (six requests' may be in flight)
constexpr int kOffQ = kStages * kStageBytes, kOffMisc = kOffQ + kQBufs * kCols * kRow;
constexpr long long kTileCycles = 1 << 16;          // more than a tile takes

struct ScoreArgs {
    const float *weights, *q_scales;
    const int32_t *pages, *indptr;
    float *out;
    int64_t pool_rows, num_pages;
    int R, qlen, heads, causal, groups, virt;
    int rows, hp;           // query rows of a group; a row's columns
    int bufs;               // accumulators: 4, or 2 where rows * hp exceeds 128
    float scale;
};

struct Misc {
    float4 w[kConstBufs][kCols / 4];
    uint64_t kv_full[kStages], kv_empty[kStages], d_full[4], d_free[4], q_full[kQBufs], q_free[kQBufs], fin;
    uint32_t tmem;
    int abort_flag;
    int start[3];
};

__device__ void producer(const ScoreArgs &a, const CUtensorMap *mk, uint8_t *sm, Misc &ms) {
    const int lane = threadIdx.x & 31, pw = (threadIdx.x >> 5) - kProdWarp0;
    Walk<kTile> w;
    w.init(a, ms.start);
    const uint64_t pol = tc::l2_policy(true);
    const auto load = [&](int (&rows)[4]) {     // the page indices of this lane's four tokens
        const int tok0 = w.t * kTile + 4 * lane;
        const int n = w.valid() ? min(max(w.len - tok0, 0), 4) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = i < n ? a.pages[(int64_t)w.base + tok0 + i] : -1;
        return n;
    };
    // The page list is brought to L2 kAhead tiles before its indices are read.
    const auto ahead = [&](int tiles) {
        const int64_t at = (int64_t)w.base + (int64_t)(w.t + tiles) * kTile + 32 * lane;
        if (lane < 5 && at < a.num_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.pages + at));
    };
    int it = pw;
    w.skip(a, pw);
    if (w.valid())
        for (int k = kProdWarps; k < kAhead; k += kProdWarps) ahead(k);
    int rows[4];
    int n = load(rows);
    bool ok = true;
    int mine = -1;      // the newest tile whose copies this warp has issued
    while (w.valid()) {
        ahead(kAhead);
        const int now = it, s = now % kStages;
        // The next tile's indices are on their way while this one's copies are issued.
        w.skip(a, kProdWarps);
        it += kProdWarps;
        int next[4];
        const int nn = load(next);
        // Past the request the copy fills zeros (row -1).
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n && (rows[i] < 0 || rows[i] >= a.pool_rows)) {
                flag(MLA_DEV_BAD_PAGE);
                rows[i] = 0;
            }
        if (!(ok = warp_wait(&ms.kv_empty[s], ((now / kStages) & 1) ^ 1, &ms.abort_flag))) break;
        if (lane == 0) mbar_arrive_expect_tx(&ms.kv_full[s], kStageBytes);
        __syncwarp();
        tc::gather4_hint(sm + s * kStageBytes + lane * 4 * kRow, mk, 0, rows[0], rows[1], rows[2], rows[3],
                         &ms.kv_full[s], pol);
        mine = now;
        n = nn;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = next[i];
    }
    if (!ok)        // flagged: let this warp's copies in flight land before the CTA ends
        for (int k = mine; k >= 0 && k > mine - kStages; k -= kProdWarps)
            mbar_wait(&ms.kv_full[k % kStages], (k / kStages) & 1);
}

__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                    uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(one));
}

__device__ void mma_issuer(const ScoreArgs &a, uint8_t *sm, Misc &ms) {
    const uint32_t base = smem_u32(sm), tm = ms.tmem;
    const uint32_t one = tc::elect_one();
    const uint32_t idesc = tc::idesc_e4m3(a.rows * a.hp, false, false);
    const uint64_t k0 = tc::sdesc(base, 16, 1024, tc::kSw128), q0 = tc::sdesc(base + kOffQ, 16, 1024, tc::kSw128);
    Walk<kTile> w;
    w.init(a, ms.start);
    const int log_bufs = a.bufs >> 1, cols = kTmemCols >> log_bufs;
    for (int it = 0; w.valid(); ++it, w.next(a)) {
        const int s = it % kStages, d = it & (a.bufs - 1), b = w.unit % kQBufs;
        if (w.first && !warp_wait(&ms.q_full[b], (w.unit / kQBufs) & 1, &ms.abort_flag)) break;
        if (!warp_wait(&ms.d_free[d], ((it >> log_bufs) & 1) ^ 1, &ms.abort_flag)) break;
        if (!warp_wait(&ms.kv_full[s], (it / kStages) & 1, &ms.abort_flag)) break;
        tc::fence_after();
        const uint64_t kd = k0 + s * (kStageBytes >> 4), qd = q0 + b * ((kCols * kRow) >> 4);
#pragma unroll
        for (int j = 0; j < kRow / 32; ++j) mma(tm + d * cols, kd + 2 * j, qd + 2 * j, idesc, j > 0, one);
        if (one) {
            tc::commit(&ms.kv_empty[s]);
            tc::commit(&ms.d_full[d]);
            if (w.last()) tc::commit(&ms.q_free[b]);
        }
        __syncwarp();
    }
    // Every MMA issued must be complete before TMEM is released.
    if (one) tc::commit(&ms.fin);
    __syncwarp();
    mbar_wait(&ms.fin, 0);
}

// The requests' queries and weights.
__device__ void prepare(const ScoreArgs &a, const CUtensorMap *mq, uint8_t *sm, Misc &ms, int grp) {
    const int lane = threadIdx.x & 31;
    const int tq0 = grp * a.rows, rows = min(a.rows, a.qlen - tq0);
    Walk<kTile> w;
    w.init(a, ms.start);
    long long pending = 0;      // tiles of the requests that the wait may have to outlast
    int last = 0, issued = 0;
    bool ok = true;
    for (int tiles = 0; w.valid(); w.next(a), ++tiles) {
        if (!w.first) continue;
        pending = last + tiles;
        last = tiles;
        tiles = 0;
        const int u = w.unit, b = u % kQBufs;
        const int64_t row0 = (int64_t)w.r * a.qlen + tq0;
        // All MMAs of the request two before: a wait for tiles, not for one.
        if (!(ok = warp_wait_long(&ms.q_free[b], ((u / kQBufs) & 1) ^ 1, &ms.abort_flag,
                                  kWaitCycles + pending * kTileCycles)))
            break;
        if (lane == 0) {
            mbar_arrive_expect_tx(&ms.q_full[b], rows * a.heads * kRow);
            for (int tq = 0; tq < rows; ++tq)
                tc::tma_2d(sm + kOffQ + (b * kCols + tq * a.hp) * kRow, mq, 0, (int)((row0 + tq) * a.heads), &ms.q_full[b]);
        }
        __syncwarp();
        // (Their readers are done, too: see kConstBufs.)
        float *to = reinterpret_cast<float *>(ms.w[u % kConstBufs]);
        float c[kCols / 32];
        int tq = 0, h = lane;       // of column lane + 32 k
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k, h += 32) {
            if (h >= a.hp) h -= a.hp, ++tq;
            if (h >= a.hp) h -= a.hp, ++tq;
            c[k] = 0.f;
            if (tq < rows && h < a.heads) {
                const int64_t at = (row0 + tq) * a.heads + h;
                c[k] = a.weights[at] * (a.q_scales ? a.q_scales[at] : 1.f) * a.scale;
            }
        }
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) to[lane + 32 * k] = c[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.q_full[b]);
        issued = u + 1;
    }
    if (!ok)        // flagged: the copies in flight land before the CTA ends
        for (int u = max(issued - kQBufs, 0); u < issued; ++u) mbar_wait(&ms.q_full[u % kQBufs], (u / kQBufs) & 1);
}

// Warpgroup wg takes the tiles of accumulator wg, or with two accumulators
// half of the query rows of accumulator wg & 1's.
__device__ void epilogue(const ScoreArgs &a, Misc &ms, int grp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, wq = warp & 3;
    const int log_bufs = a.bufs >> 1, d = wg & (a.bufs - 1), cols = kTmemCols >> log_bufs, steps = a.hp / 16;
    const int all = min(a.rows, a.qlen - grp * a.rows), half = (all + 1) / 2;
    const int first = a.bufs == 4 || wg < 2 ? 0 : half, rows = a.bufs == 4 ? all : wg < 2 ? half : all - half;
    const uint32_t taddr = ms.tmem + d * cols + first * a.hp + ((uint32_t)(32 * wq) << 16);
    const int tq0 = grp * a.rows + first, chunks = rows * steps;
    Walk<kTile> w;
    w.init(a, ms.start);
    w.skip(a, d);
    for (int it = 0; w.valid(); ++it, w.skip(a, a.bufs)) {      // every bufs-th tile
        const int j = w.t * kTile + 32 * wq + lane;
        float *out = a.out + (int64_t)tq0 * a.num_pages + w.base + j;
        if (!warp_wait(&ms.d_full[d], it & 1, &ms.abort_flag)) break;
        tc::fence_after();
        const float4 *c = ms.w[w.unit % kConstBufs] + first * (a.hp / 4);
        float sum[4] = {0, 0, 0, 0};
        int step = 0, seen = a.causal ? w.len - a.qlen + tq0 + 1 : w.len;       // tokens that the row sees
        // 16 heads' columns of this token; a row's last ones end its sum.  (Two
        // columns an instruction: 76 us for 128 x 4 rows and not 74.)
        const auto add = [&](const float (&x)[16]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 ws = *c++;
                sum[0] = fmaf(max_nan(x[4 * i], 0.f), ws.x, sum[0]);
                sum[1] = fmaf(max_nan(x[4 * i + 1], 0.f), ws.y, sum[1]);
                sum[2] = fmaf(max_nan(x[4 * i + 2], 0.f), ws.z, sum[2]);
                sum[3] = fmaf(max_nan(x[4 * i + 3], 0.f), ws.w, sum[3]);
            }
            if (++step < steps) return;
            if (j < w.len) *out = j < seen ? (sum[0] + sum[2]) + (sum[1] + sum[3]) : -INFINITY;
            out += a.num_pages;
            sum[0] = sum[1] = sum[2] = sum[3] = 0;
            step = 0;
            if (a.causal) ++seen;
        };
        float x[2][16];
        if (chunks > 0) tc::ld16(taddr, x[0]);
        tc::wait_ld();
#pragma unroll 1
        for (int g = 0; g < chunks; g += 2) {
            // The next columns leave TMEM while these are summed.
            if (g + 1 < chunks) tc::ld16(taddr + 16 * (g + 1), x[1]);
            add(x[0]);
            tc::wait_ld();
            if (g + 1 >= chunks) break;
            if (g + 2 < chunks) tc::ld16(taddr + 16 * (g + 2), x[0]);
            add(x[1]);
            tc::wait_ld();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.d_free[d]);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    index_scores_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq, const ScoreArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(sm + kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, grp = blockIdx.x % a.groups;
    if (tid == 0) {
        tc::prefetch_map(&mk);
        tc::prefetch_map(&mq);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ms.kv_full[s], 1);
            mbar_init(&ms.kv_empty[s], 1);
        }
        for (int d = 0; d < 4; ++d) {
            mbar_init(&ms.d_full[d], 1);
            mbar_init(&ms.d_free[d], a.bufs == 4 ? 4 : 8);      // warps that read it
        }
        for (int b = 0; b < kQBufs; ++b) {
            mbar_init(&ms.q_full[b], 2);        // the copies' and the weights'
            mbar_init(&ms.q_free[b], 1);
        }
        mbar_init(&ms.fin, 1);
        ms.abort_flag = 0;
        ms.start[0] = ms.start[1] = 0;
        mbar_fence_init();
    }
    // Columns that no copy fills hold zeros: their weights are 0, but a NaN code would stay.
    const int rows = min(a.rows, a.qlen - grp * a.rows);
    if (a.hp != a.heads || rows < a.rows) {
#pragma unroll 1
        for (int i = tid; i < kQBufs * kCols * (kRow / 16); i += kThreads) {
            const int n = i / (kRow / 16) % kCols, tq = n / a.hp;
            if (n - tq * a.hp >= a.heads || tq >= rows) *reinterpret_cast<uint4 *>(sm + kOffQ + 16 * i) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_async_smem();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&ms.tmem, kTmemCols);
    tc::fence_before();
    grid_wait();
    find_start<kTile, kThreads>(a, ms.start, blockIdx.x / a.groups);
    tc::fence_after();
    if (warp < kMmaWarp) epilogue(a, ms, grp);
    else if (warp == kMmaWarp) mma_issuer(a, sm, ms);
    else if (warp < kPrepWarp) producer(a, &mk, sm, ms);
    else prepare(a, &mq, sm, ms, grp);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kMmaWarp) tc::tmem_free(ms.tmem, kTmemCols);
}

// [rows, 128] bytes, read `box` rows at a time.
bool encode(CUtensorMap *m, const void *p, int64_t rows, int box_rows) {
    const cuuint64_t dim[2] = {(cuuint64_t)kRow, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)kRow};
    const cuuint32_t box[2] = {(cuuint32_t)kRow, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dim, stride, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Arguments checked by mla_index_scores.
cudaError_t index_scores_launch(const void *q, const float *weights, const float *q_scales, const void *k,
                                int64_t pool_rows, const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R,
                                int qlen, int heads, float scale, float *out, bool causal, int sms, cudaStream_t st) {
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    CUtensorMap mk, mq;
    if (!encode(&mk, k, pool_rows, 1) || !encode(&mq, q, (int64_t)R * qlen * heads, heads)) return cudaErrorInvalidValue;
    ScoreArgs a = {};
    a.weights = weights;
    a.q_scales = q_scales;
    a.pages = pages;
    a.indptr = indptr;
    a.out = out;
    a.pool_rows = pool_rows;
    a.num_pages = num_pages;
    a.R = R;
    a.qlen = qlen;
    a.heads = heads;
    a.causal = causal;
    a.scale = scale;
    // The fewest groups of whole rows that fit a group's columns, of even size.
    a.hp = (heads + 15) / 16 * 16;
    const int most = kCols / a.hp;
    a.groups = (qlen + most - 1) / most;
    a.rows = (qlen + a.groups - 1) / a.groups;
    a.bufs = a.rows * a.hp <= kTmemCols / 4 ? 4 : 2;
    a.virt = sms / a.groups < 1 ? 1 : sms / a.groups;
    constexpr int smem = kOffMisc + sizeof(Misc) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = smem_attr_once<index_scores_kernel>(smem);
    if (e != cudaSuccess) return e;
    return launch_early(index_scores_kernel, a.virt * a.groups, kThreads, smem, st, mk, mq, a);
}

cudaError_t index_scores_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
