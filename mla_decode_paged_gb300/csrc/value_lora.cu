// W_UV projection and sigmoid gate with one low-rank adapter per request --
// two kernels: the requests' low-rank products, then the projection.
//
// What it computes, for row t (request r = t / qlen), head h, output v, with
// a = adapters[r] (-1: no adapter):
//   val = sum_c latent[t, h, c] w_uv[h, v, c]
//         + lora_scale[a] * sum_k (sum_c latent[t, h, c] A[a, k, c]) B[a, h, v, k]
//   out[t, h*128 + v] = lengths[r] > 0 ? bf16(val * sigmoid(gate)) : 0
//
// Bound by bytes: the latent (1 KB a row and head), W_UV (128 KB a head), A
// and B of every adapter in use; at a few rows by the two launches.
//
//   shrink: the (row, head) pairs of a request share A: T = latent A^T *
//     lora_scale.  Few pairs: warp MMAs on fragments loaded straight from
//     global memory (a lane's 16 bytes are two k-steps' worth: the products'
//     order over k is free), eight warps of 64 latent columns each, joined in
//     shared memory.  Many: tcgen05 MMAs, 48 pairs (M, the rows past them
//     whatever follows in shared memory: unused lanes) times A (N), two
//     blocks an SM.
//     T goes to the workspace as two bf16 terms, hi + lo (2^-17 of the
//     product; one term would add 2^-9, as much as the output's own rounding).
//   project: a persistent block per head (as many as fit), W_UV[h] (M = 128
//     outputs) staying in shared memory, over the head's tiles of rows (N):
//     tcgen05 MMAs into TMEM, the next tile's latents and products in flight
//     during this one.  Meanwhile the 16 warps form B T by warp MMAs into a
//     float32 tile, reading B[a, h] once per request of the tile (every
//     column of a warp MMA is a row of its own, so rows of other requests
//     need no mask), four requests' loads in flight a warp.  The epilogue
//     adds the two and gates.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "tc.cuh"

namespace mla {
namespace {

struct LoraArgs {
    const __nv_bfloat16 *latent, *gate, *a, *b;
    const int32_t *lengths, *adapters;
    const float *scale;
    __nv_bfloat16 *t;       // [S * H, 2, rank]: hi, lo
    __nv_bfloat16 *out;
    int S, qlen, H, rank, n;
};

// Request r's adapter, -1 for none (and, flagged, for an index outside).
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int r) {
    const int a = __ldg(p.adapters + r);
    if (a >= -1 && a < p.n) return a;
    flag(MLA_DEV_BAD_ADAPTER);
    return -1;
}

// Two values as bf16 pairs hi + lo; no lo beside an infinite hi (inf - inf).
__device__ __forceinline__ void two_terms(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(a, b);
    const float ha = bf16_lo(hi), hb = bf16_hi(hi);
    lo = pack_bf16x2(isinf(ha) ? 0.f : a - ha, isinf(hb) ? 0.f : b - hb);
}

// ------------------------------------------------------------------ shrink

constexpr int kShrinkWarps = 8;
constexpr int kNChunk = 8;              // n-tiles (of 8 ranks) whose sums a warp holds at once

// 16 (row, head) pairs per block.
__global__ void __launch_bounds__(kShrinkWarps * 32) shrink_kernel(const LoraArgs p, int tiles) {
    constexpr int kCols = kNChunk * 8 + 1;
    __shared__ float part[kShrinkWarps * 16 * kCols];
    asm volatile("griddepcontrol.launch_dependents;");
    const int r = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int a = adapter_of(p, r);
    if (a < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int pairs = p.qlen * p.H, m0 = tile * 16;
    const int64_t row0 = (int64_t)r * pairs;
    const float scale = __ldg(p.scale + a);
    const int c0 = warp * 64 + 8 * q;   // this lane's columns: c0 .. c0 + 7 and c0 + 32 ..
    uint4 x[2][2];                      // [32-column block][row g, g + 8]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = min(m0 + 8 * i + g, pairs - 1);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + (row0 + row) * MLA_D_LATENT + c0);
#pragma unroll
        for (int b = 0; b < 2; ++b) x[b][i] = __ldg(src + 4 * b);
    }
    const int ntiles = p.rank / 8;
    for (int n0 = 0; n0 < ntiles; n0 += kNChunk) {
        const int nn = min(kNChunk, ntiles - n0);
        float acc[kNChunk][4] = {};
        uint4 w[kNChunk][2];
#pragma unroll
        for (int n = 0; n < kNChunk; ++n)
            if (n < nn) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.a + ((int64_t)a * p.rank + 8 * (n0 + n) + g) * MLA_D_LATENT + c0);
                w[n][0] = __ldg(src);
                w[n][1] = __ldg(src + 4);
            }
#pragma unroll
        for (int n = 0; n < kNChunk; ++n)
            if (n < nn)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint4 u = x[b][0], v = x[b][1], k = w[n][b];
                    const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                    mma_bf16(acc[n], a0, k.x, k.y);
                    mma_bf16(acc[n], a1, k.z, k.w);
                }
        if (n0 > 0) __syncthreads();
#pragma unroll
        for (int n = 0; n < kNChunk; ++n)
            if (n < nn)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[(warp * 16 + g + 8 * (i >> 1)) * kCols + 8 * n + 2 * q + (i & 1)] = acc[n][i];
        __syncthreads();
        const int cols = 4 * nn;        // pairs of columns
        for (int e = threadIdx.x; e < 16 * cols; e += kShrinkWarps * 32) {
            const int row = e / cols, k = 2 * (e - row * cols);
            if (m0 + row >= pairs) break;
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int w8 = 0; w8 < kShrinkWarps; ++w8) {
                s[0] += part[(w8 * 16 + row) * kCols + k];
                s[1] += part[(w8 * 16 + row) * kCols + k + 1];
            }
            uint32_t hi, lo, *dst = reinterpret_cast<uint32_t *>(p.t + (row0 + m0 + row) * 2 * p.rank + 8 * n0 + k);
            two_terms(s[0] * scale, s[1] * scale, hi, lo);
            dst[0] = hi;
            dst[p.rank / 2] = lo;
        }
    }
}

// The shape both tcgen05 kernels share.
constexpr int kColBlocks = MLA_D_LATENT / 64;      // 128-byte column blocks of the K axis

// kind::f16: bf16 A and B (K-major), f32 D, M = 128.
constexpr uint32_t idesc_bf16(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16_tc(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate));
}

// D = A[128 x 512] B[N x 512]^T, both in 128B-swizzled column blocks.
__device__ __forceinline__ void mma_latent(uint32_t d_tmem, uint32_t a, uint32_t a_block, uint32_t b, uint32_t b_block,
                                           uint32_t idesc) {
#pragma unroll
    for (int j = 0; j < MLA_D_LATENT / 16; ++j) {
        const int kb = j >> 2, off = (j & 3) * 32;
        mma_bf16_tc(d_tmem, tc::sdesc(a + kb * a_block + off, 16, 1024, tc::kSw128),
                    tc::sdesc(b + kb * b_block + off, 16, 1024, tc::kSw128), idesc, j > 0);
    }
}

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

constexpr int kTcPairs = 48, kTcThreads = 128;
constexpr int kTcXBlock = kTcPairs * 128;

// The last block's reads of 128 rows of pairs, and of 16 of A where the rank
// ends at 8, stay inside too.
__host__ __device__ constexpr int shrink_tc_smem(int rank) {
    const int all = kColBlocks * (kTcXBlock + rank * 128) + (rank % 16 ? 1024 : 0), pairs = (kColBlocks - 1) * kTcXBlock + 128 * 128;
    return all > pairs ? all : pairs;
}

// 48 pairs per block: ma maps lora_a as [n * rank, 512], mx the latent as
// [S * H, 512].
__global__ void __launch_bounds__(kTcThreads)
    shrink_tc_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mx, const LoraArgs p,
                     int tiles) {
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ uint64_t full, done;
    __shared__ uint32_t tmem;
    asm volatile("griddepcontrol.launch_dependents;");
    const int r = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int a = adapter_of(p, r);
    if (a < 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = p.qlen * p.H, m0 = tile * kTcPairs;
    const int64_t row0 = (int64_t)r * pairs + m0;
    const int a_block = p.rank * 128, a_off = kColBlocks * kTcXBlock;
    if (tid == 0) {
        mbar_init(&full, 1);
        mbar_init(&done, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(&full, kColBlocks * (kTcXBlock + a_block));
        for (int kb = 0; kb < kColBlocks; ++kb) {
            tma_2d(sm + kb * kTcXBlock, &mx, 64 * kb, (int)row0, &full);
            tma_2d(sm + a_off + kb * a_block, &ma, 64 * kb, a * p.rank, &full);
        }
    }
    if (warp == 0) tc::tmem_alloc(&tmem, 128);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    bool ok = true, issued = false;
    if (tid == 0) {
        ok = mbar_wait(&full, 0);
        if (ok) {
            issued = true;
            tc::fence_after();
            mma_latent(tmem, smem_u32(sm), kTcXBlock, smem_u32(sm) + a_off, a_block, idesc_bf16((p.rank + 15) / 16 * 16));
            tc::commit(&done);
        }
    }
    ok = __syncthreads_and(ok);
    if (ok) ok = mbar_wait(&done, 0);
    ok = __syncthreads_and(ok);
    if (ok) {
        tc::fence_after();
        const int m = tid;      // TMEM lane = pair
        const float scale = __ldg(p.scale + a);
        uint4 *dst = reinterpret_cast<uint4 *>(p.t + (row0 + m) * 2 * p.rank);
        const int vecs = p.rank / 8;
        if (32 * warp < kTcPairs)
            for (int c = 0; c < p.rank; c += 16) {
                float d[16];
                tc::ld16(tmem + ((uint32_t)(32 * warp) << 16) + c, d);
                tc::wait_ld();
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) two_terms(d[8 * v + 2 * i] * scale, d[8 * v + 2 * i + 1] * scale, hi[i], lo[i]);
                    if (m < kTcPairs && m0 + m < pairs && c / 8 + v < vecs) {
                        dst[c / 8 + v] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        dst[vecs + c / 8 + v] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
    } else if (tid == 0) {
        // Flagged.  What is in flight finishes before TMEM is released.
        mbar_wait(&full, 0);
        if (issued) mbar_wait(&done, 0);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 128);
}

// ------------------------------------------------------------------ project

constexpr int kThreads = 512;                      // and a warp that issues copies and products
constexpr int kABlock = MLA_D_V * 128;             // one column block of W_UV[h]: 16 KB
constexpr int kBOff = kColBlocks * kABlock;
constexpr int kDStride = MLA_D_V + 4;              // float32 tile rows, a bank apart per row pair
constexpr int kBatch = 2;                          // items a warp expands at once

// NR rows a tile; two tiles' latents.
template <int NR>
struct Tile {
    static constexpr int kBBlock = NR * 128, kBBytes = kColBlocks * kBBlock;
    static constexpr int kDOff = kBOff + 2 * kBBytes;
    static constexpr int kSmem = kDOff + NR * kDStride * 4 + 1024;
    static constexpr int kRows = NR / 4;            // rows per thread in the epilogue
};

// N consecutive f32 TMEM columns of this warp's lanes.
template <int N>
__device__ __forceinline__ void ld_rows(uint32_t taddr, float (&v)[N]) {
    static_assert(N == 4 || N == 8, "rows of a 16- or 32-row tile");
    uint32_t r[8];
    if (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

// Up to eight rows [n0, e) of a tile that share a request, and B[a, h] of its
// adapter (null: none).
struct Item {
    const __nv_bfloat16 *b;
    int n0, e;
};

// 1 / (1 + e^-x); e^-x = inf gives 0.
__device__ __forceinline__ float sigmoid_f32(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x)));
    return r;
}

// The tile's items, one thread each; their number.
__device__ __forceinline__ int make_items(const LoraArgs &p, Item *items, int t0, int nrows, int h) {
    const int per = (p.qlen + 7) / 8;
    const int r0 = t0 / p.qlen, n = ((t0 + nrows - 1) / p.qlen - r0 + 1) * per;
    if (threadIdx.x < n) {
        const int i = threadIdx.x, r = r0 + i / per, first = r * p.qlen + i % per * 8;
        const int a = adapter_of(p, r);
        Item x;
        x.n0 = max(first, t0) - t0;
        x.e = min(min(first + 8, (r + 1) * p.qlen), t0 + nrows) - t0;
        x.b = a < 0 || x.e <= x.n0 ? nullptr : p.b + ((int64_t)a * p.H + h) * MLA_D_V * p.rank;
        items[i] = x;
    }
    return n;
}

// B[a, h] T of the tile's rows -> delta[row][v].  Warp w takes outputs
// 16 (w % 8) .. + 15 of every second item.
__device__ __forceinline__ void expand(const LoraArgs &p, float *delta, const Item *items, int nitems, int t0, int h) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int v0 = 16 * (warp & 7), rank = p.rank;
    const int b_lane = (v0 + g) * rank + 8 * q, t_row = p.H * 2 * rank;
    const __nv_bfloat16 *t_lane = p.t + ((int64_t)t0 * p.H + h) * 2 * rank + 8 * q;
    for (int i0 = warp >> 3; i0 < nitems; i0 += 2 * kBatch) {
        const __nv_bfloat16 *b[kBatch], *t[kBatch];
        int n0[kBatch], e[kBatch];
        float acc[kBatch][4] = {};
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + 2 * u;
            e[u] = n0[u] = 0;
            b[u] = nullptr;
            if (i < nitems) {
                const Item x = items[i];
                if (x.b) {
                    b[u] = x.b + b_lane;
                    n0[u] = x.n0;
                    e[u] = x.e;
                }
            }
            t[u] = t_lane + (int64_t)t_row * max(min(n0[u] + g, e[u] - 1), 0);    // columns past the request are not kept
        }
        for (int k = 0; k < rank; k += 32) {
            const bool in = k + 8 * q < rank;
            uint4 x[kBatch], y[kBatch], hi[kBatch], lo[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[u] = y[u] = hi[u] = lo[u] = make_uint4(0, 0, 0, 0);
                if (in && e[u]) {
                    x[u] = __ldg(reinterpret_cast<const uint4 *>(b[u] + k));
                    y[u] = __ldg(reinterpret_cast<const uint4 *>(b[u] + 8 * rank + k));
                    hi[u] = *reinterpret_cast<const uint4 *>(t[u] + k);
                    lo[u] = *reinterpret_cast<const uint4 *>(t[u] + rank + k);
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t a0[4] = {x[u].x, y[u].x, x[u].y, y[u].y}, a1[4] = {x[u].z, y[u].z, x[u].w, y[u].w};
                mma_bf16(acc[u], a0, hi[u].x, hi[u].y);
                mma_bf16(acc[u], a1, hi[u].z, hi[u].w);
                mma_bf16(acc[u], a0, lo[u].x, lo[u].y);
                mma_bf16(acc[u], a1, lo[u].z, lo[u].w);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int n = n0[u] + 2 * q;
            float *d = delta + n * kDStride + v0 + g;
            if (n < e[u]) {
                d[0] = acc[u][0];
                d[8] = acc[u][2];
            }
            if (n + 1 < e[u]) {
                d[kDStride] = acc[u][1];
                d[kDStride + 8] = acc[u][3];
            }
        }
    }
}

template <int NR>
__global__ void __launch_bounds__(kThreads + 32, 1)
    project_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ml, const LoraArgs p) {
    using T = Tile<NR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *delta = reinterpret_cast<float *>(sm + T::kDOff);
    __shared__ uint64_t full[2], done[2];
    __shared__ uint32_t tmem;
    __shared__ uint8_t active[NR], adapted[NR];
    __shared__ Item items[NR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, tiles = (p.S + NR - 1) / NR, step = gridDim.x;
    const bool issuer = tid == kThreads;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
        }
        mbar_fence_init();
    }
    if (warp == 0) tc::tmem_alloc(&tmem, 2 * NR);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t base = smem_u32(sm), tm = tmem;
    // Rows past S read as zeros (their outputs are not written).
    const auto fetch = [&](int tile, int s, uint32_t with) {
        mbar_arrive_expect_tx(&full[s], with + T::kBBytes);
        for (int kb = 0; kb < kColBlocks; ++kb)
            tma_3d(sm + kBOff + s * T::kBBytes + kb * T::kBBlock, &ml, 64 * kb, h, tile * NR, &full[s]);
    };
    if (issuer) {
        // Nothing here but the low-rank products is written by the kernel
        // before this one: W_UV and the latent are fetched at once.
        fetch(blockIdx.x, 0, kBOff);
        for (int kb = 0; kb < kColBlocks; ++kb) tma_2d(sm + kb * kABlock, &mw, 64 * kb, MLA_D_V * h, &full[0]);
        if (blockIdx.x + step < tiles) fetch(blockIdx.x + step, 1, 0);
    }
    bool ok = true;
    int issued = 0, it = 0;                         // issuer: tiles whose products are issued
    const auto multiply = [&](int n) {              // the n-th tile of this block
        ok = ok && mbar_wait(&full[n & 1], (n >> 1) & 1);
        if (!ok) return;
        tc::fence_after();
        mma_latent(tm + (n & 1) * NR, base, kABlock, base + kBOff + (n & 1) * T::kBBytes, T::kBBlock, idesc_bf16(NR));
        tc::commit(&done[n & 1]);
        ++issued;
    };
    for (int tile = blockIdx.x; tile < tiles; tile += step, ++it) {
        const int t0 = tile * NR, nrows = min(NR, p.S - t0);
        if (tid < NR) {
            const int r = (t0 + tid) / p.qlen;
            active[tid] = tid < nrows && __ldg(p.lengths + r) > 0;
            adapted[tid] = tid < nrows && adapter_of(p, r) >= 0;
        }
        const int nitems = make_items(p, items, t0, nrows, h);
        // This thread's gates (output v of rows first .. first + kRows - 1),
        // in flight during the products.
        const int v = 32 * (warp & 3) + lane, first = (warp >> 2) * T::kRows;
        const int64_t at = ((int64_t)(t0 + first) * p.H + h) * MLA_D_V + v;
        const int row_step = p.H * MLA_D_V;
        uint16_t gate[T::kRows];
#pragma unroll
        for (int i = 0; i < T::kRows; ++i)
            gate[i] = first + i < nrows
                          ? __ldg(reinterpret_cast<const uint16_t *>(p.gate) + at + (int64_t)i * row_step)
                          : 0;
        __syncthreads();
        if (it == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid < kThreads) expand(p, delta, items, nitems, t0, h);
        if (issuer) {
            if (it == 0) multiply(0);
            if (tile + step < tiles) multiply(it + 1);     // D and latents are double-buffered
        }
        __syncwarp();
        ok = __syncthreads_and(ok);
        if (ok) ok = mbar_wait(&done[it & 1], (it >> 1) & 1);
        ok = __syncthreads_and(ok);
        if (!ok) break;
        tc::fence_after();
        // The latents of this tile have been multiplied: their place takes the tile after the next.
        if (issuer && tile + 2 * step < tiles) fetch(tile + 2 * step, it & 1, 0);
        if (tid < kThreads) {
            float d[T::kRows];
            ld_rows<T::kRows>(tm + ((uint32_t)(32 * (warp & 3)) << 16) + (it & 1) * NR + first, d);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < T::kRows; ++i) {
                const int n = first + i;
                if (n >= nrows) break;
                float x = 0.f;      // a select, so that nothing of an empty request is seen
                if (active[n]) {
                    x = adapted[n] ? d[i] + delta[n * kDStride + v] : d[i];
                    x *= sigmoid_f32(__uint_as_float((uint32_t)gate[i] << 16));
                }
                p.out[at + (int64_t)i * row_step] = __float2bfloat16_rn(x);
            }
        }
        tc::fence_before();
        __syncthreads();            // the tile's shared arrays are read
    }
    if (!ok && issuer) {
        // Flagged.  What is in flight finishes (one more bounded wait each)
        // before TMEM is released and the CTA ends.
        for (int n = it; n < it + 2 && blockIdx.x + n * step < tiles; ++n) {
            mbar_wait(&full[n & 1], (n >> 1) & 1);
            if (n < issued) mbar_wait(&done[n & 1], (n >> 1) & 1);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tm, 2 * NR);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

bool encode_bf16(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dim, const cuuint64_t *stride,
                 const cuuint32_t *box) {
    const cuuint32_t es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dim, stride, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `map` over `rows` rows of the latent width, in boxes of box_rows.
bool encode_rows(CUtensorMap *m, const void *ptr, int64_t rows, int box_rows) {
    const cuuint64_t dim[2] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)rows};
    const cuuint64_t stride[1] = {(cuuint64_t)MLA_D_LATENT * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode_bf16(m, ptr, 2, dim, stride, box);
}

cudaError_t shrink(const LoraArgs &p, int R, int sms, cudaStream_t st) {
    const int pairs = p.qlen * p.H;
    // With more 16-pair blocks than the GPU holds at once, A's repeated reads
    // cost more than the taller tiles' start.
    if ((int64_t)R * ((pairs + 15) / 16) > 4 * (int64_t)sms && pairs > 16 && (int64_t)p.S * p.H <= INT32_MAX) {
        CUtensorMap ma, mx;
        if (!encode_rows(&ma, p.a, (int64_t)p.n * p.rank, p.rank) ||
            !encode_rows(&mx, p.latent, (int64_t)p.S * p.H, kTcPairs))
            return cudaErrorInvalidValue;
        cudaError_t e = smem_attr_once<shrink_tc_kernel>(shrink_tc_smem(MLA_MAX_LORA_RANK));
        if (e != cudaSuccess) return e;
        const int tiles = (pairs + kTcPairs - 1) / kTcPairs;
        shrink_tc_kernel<<<(unsigned)R * tiles, kTcThreads, shrink_tc_smem(p.rank), st>>>(ma, mx, p, tiles);
        return cudaGetLastError();
    }
    const int tiles = (pairs + 15) / 16;
    shrink_kernel<<<(unsigned)R * tiles, kShrinkWarps * 32, 0, st>>>(p, tiles);
    return cudaGetLastError();
}

template <int NR>
cudaError_t project(const CUtensorMap &mw, const LoraArgs &p, int sms, cudaStream_t st) {
    const cuuint64_t dim[3] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)p.H, (cuuint64_t)p.S};
    const cuuint64_t stride[2] = {(cuuint64_t)MLA_D_LATENT * 2, (cuuint64_t)p.H * MLA_D_LATENT * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)NR};
    CUtensorMap ml;
    if (!encode_bf16(&ml, p.latent, 3, dim, stride, box)) return cudaErrorInvalidValue;
    cudaError_t e = smem_attr_once<project_kernel<NR>>(Tile<NR>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min((p.S + NR - 1) / NR, std::max(1, sms / p.H)), p.H, 1);
    cfg.blockDim = dim3(kThreads + 32, 1, 1);
    cfg.dynamicSmemBytes = Tile<NR>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, project_kernel<NR>, mw, ml, p);
}

}  // namespace

int64_t value_lora_workspace(int64_t rows, int heads, int rank) { return rows * heads * rank * 4; }

cudaError_t value_lora_launch(const void *latent, const void *w_uv, const void *gate, const int32_t *lengths,
                              const void *lora_a, const void *lora_b, const int32_t *adapters, const float *lora_scale,
                              int num_adapters, int rank, int R, int qlen, int H, void *out, void *workspace, int sms,
                              cudaStream_t st) {
    if (!encode_fn()) return cudaErrorNotSupported;
    LoraArgs p = {};
    p.latent = static_cast<const __nv_bfloat16 *>(latent);
    p.gate = static_cast<const __nv_bfloat16 *>(gate);
    p.a = static_cast<const __nv_bfloat16 *>(lora_a);
    p.b = static_cast<const __nv_bfloat16 *>(lora_b);
    p.lengths = lengths;
    p.adapters = adapters;
    p.scale = lora_scale;
    p.t = static_cast<__nv_bfloat16 *>(workspace);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.S = R * qlen;
    p.qlen = qlen;
    p.H = H;
    p.rank = rank;
    p.n = num_adapters;
    CUtensorMap mw;
    if (!encode_rows(&mw, w_uv, (int64_t)H * MLA_D_V, MLA_D_V)) return cudaErrorInvalidValue;
    cudaError_t e = shrink(p, R, sms, st);
    if (e != cudaSuccess) return e;
    // 32-row tiles, unless 16-row ones leave no block of a head with two.
    if ((p.S + 15) / 16 <= std::max(1, sms / H)) return project<16>(mw, p, sms, st);
    return project<32>(mw, p, sms, st);
}

cudaError_t value_lora_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
