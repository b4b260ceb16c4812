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
// and B of every adapter in use; at a few rows by the two launches and the
// chain A -> T -> B T.
//
// Measured: 64 single-row requests of 12 heads, rank 16, in 6.8 us; 32 of 96
// heads, rank 32, in 9.5 (their bytes: 3.5); 256 requests of eight rows, 12
// heads, rank 64, in 27.6 (47.7 MB, 7.0): 8.8 until the last T, then six
// tiles a block of ~3,300 cycles, in which the ring's entries, the latents'
// products (their copies wait for the tile before) and the epilogue take
// about as long as each other.
//
//   shrink: the (row, head) pairs of a request share A: T = latent A^T *
//     lora_scale.  Few pairs: warp MMAs on fragments loaded straight from
//     global memory (a lane's 16 bytes are two k-steps' worth: the products'
//     order over k is free), eight warps of 64 latent columns each, joined in
//     shared memory.  Many: tcgen05 MMAs, 48 pairs (M, the rows past them
//     whatever follows in shared memory: unused lanes) times A (N), two
//     blocks an SM up to rank 64, one above.
//     T goes to the workspace as two bf16 terms, hi + lo (2^-17 of the
//     product; one term would add 2^-9, as much as the output's own rounding).
//   project: persistent blocks, each on one head: W_UV[h] (M = 128 outputs)
//     stays in shared memory over the head's tiles of rows (N), whose latents
//     stream past it into tcgen05 MMAs.  B[a, h] T in one of two ways.
//     One row a request: 16 warps form it by warp MMAs from global memory
//     into a float32 tile, an MMA's eight columns being rows that share an
//     adapter (32 requests of 96 heads on eight adapters 9.7 us, with a row an
//     MMA 12.3); the first ones' B is on its way while T is still formed.
//     More: through a ring, an entry being B[a, h] (M, by TMA) and the T rows
//     of up to eight rows of one request (its place in a 16-row window, N),
//     two MMAs per 16 ranks into 16 TMEM columns of its own, of which the
//     request's rows are added to the projection's.  (Added into the
//     projection's columns with the other rows zero, one tenant's infinite B
//     would be everyone's NaN.)
//       warps 0..7   epilogue: the sum from TMEM, gated, while the next
//                    tile's projection runs (its D is double-buffered)
//       warps 8..13  one ring slot each: T rows and B into it
//       warp 14      latents and W_UV, and their MMAs
//       warp 15      the entries' MMAs
#include <algorithm>

#include <cuda.h>
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
    uint64_t inv_qlen;
    int tile_rows;          // warp MMAs' kernel: rows of a tile
    int add_both;           // the ring's kernel: 1, two tiles' low-rank products fit TMEM
    int S, qlen, H, rank, n;
};

// t / qlen for 0 <= t < 2^29: with inv_qlen = ceil(2^35 / qlen) the quotient
// is too large by less than t / 2^35 < 1 / qlen.
__device__ __forceinline__ int request_of(const LoraArgs &p, int t) { return (int)((uint64_t)t * p.inv_qlen >> 35); }

// An adapter index; -1 for none and, flagged, for one outside.
__device__ __forceinline__ int valid_adapter(const LoraArgs &p, int a) {
    if (a >= -1 && a < p.n) return a;
    flag(MLA_DEV_BAD_ADAPTER);
    return -1;
}

// Request r's.
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int r) { return valid_adapter(p, __ldg(p.adapters + r)); }

// Two values as bf16 pairs hi + lo; no lo beside an infinite hi (inf - inf).
__device__ __forceinline__ void two_terms(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(a, b);
    const float ha = bf16_lo(hi), hb = bf16_hi(hi);
    lo = pack_bf16x2(isinf(ha) ? 0.f : a - ha, isinf(hb) ? 0.f : b - hb);
}

// N 4-byte words, 4 N bytes aligned.
template <int N>
struct Words {
    uint32_t w[N];
};

// Read-only loads that stay where they are: ahead of what follows them.
template <int N>
__device__ __forceinline__ Words<N> load_now(const void *p) {
    static_assert(N == 2 || N == 4, "8 or 16 bytes");
    Words<N> x;
    if constexpr (N == 4)
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(x.w[0]), "=r"(x.w[1]) : "l"(p));
    return x;
}

__device__ __forceinline__ int load_int(const int *p) {
    int x;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x) : "l"(p));
    return x;
}

template <int N>
__device__ __forceinline__ Words<N> load_words(const void *p) {
    Words<N> x;
    if constexpr (N == 4) {
        const uint4 v = *static_cast<const uint4 *>(p);
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else {
        const uint2 v = *static_cast<const uint2 *>(p);
        x.w[0] = v.x, x.w[1] = v.y;
    }
    return x;
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
    const int index = __ldg(p.adapters + r);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int pairs = p.qlen * p.H, m0 = tile * 16;
    const int64_t row0 = (int64_t)r * pairs;
    const int c0 = warp * 64 + 8 * q;   // this lane's columns: c0 .. c0 + 7 and c0 + 32 ..
    Words<4> x[2][2];                   // [32-column block][row g, g + 8], on its way with the index
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = min(m0 + 8 * i + g, pairs - 1);
        const __nv_bfloat16 *src = p.latent + (row0 + row) * MLA_D_LATENT + c0;
#pragma unroll
        for (int b = 0; b < 2; ++b) x[b][i] = load_now<4>(src + 32 * b);
    }
    const int a = valid_adapter(p, index);
    if (a < 0) return;
    const float scale = __ldg(p.scale + a);
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
                    const Words<4> u = x[b][0], v = x[b][1];
                    const uint4 k = w[n][b];
                    const uint32_t a0[4] = {u.w[0], v.w[0], u.w[1], v.w[1]}, a1[4] = {u.w[2], v.w[2], u.w[3], v.w[3]};
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

// Run by a whole warp, its arguments the same in every lane; `one` (0 or 1)
// set in the lane that issues.  A branch around it instead would keep the
// descriptors out of the uniform registers.
__device__ __forceinline__ void mma_bf16_tc(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                            uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(one));
}

// D (+)= A[128 x 64 (kb1 - kb0)] B[N x ..]^T: column blocks kb0 .. kb1 - 1 of
// the latent's, both 128B-swizzled.
__device__ __forceinline__ void mma_latent(uint32_t d_tmem, uint32_t a, uint32_t a_block, uint32_t b, uint32_t b_block,
                                           uint32_t idesc, uint32_t one, int kb0 = 0, int kb1 = kColBlocks) {
    const uint64_t ad = tc::sdesc(a, 16, 1024, tc::kSw128), bd = tc::sdesc(b, 16, 1024, tc::kSw128);
#pragma unroll
    for (int j = 4 * kb0; j < 4 * kb1; ++j)
        mma_bf16_tc(d_tmem, ad + (j >> 2) * (a_block >> 4) + (j & 3) * 2, bd + (j >> 2) * (b_block >> 4) + (j & 3) * 2,
                    idesc, j > 0, one);
}

constexpr int kTcPairs = 48, kTcThreads = 128, kParts = 4;
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
    __shared__ uint64_t full[kParts], done;     // a part: column blocks that arrive and are multiplied together
    __shared__ uint32_t tmem;
    asm volatile("griddepcontrol.launch_dependents;");
    const int r = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int index = load_int(p.adapters + r);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int pairs = p.qlen * p.H, m0 = tile * kTcPairs;
    const int64_t row0 = (int64_t)r * pairs + m0;
    const int a_block = p.rank * 128, a_off = kColBlocks * kTcXBlock;
    if (tid == 0) {
        for (int i = 0; i < kParts; ++i) mbar_init(&full[i], 1);
        mbar_init(&done, 1);
        mbar_fence_init();
    }
    if (warp == 1) tc::tmem_alloc(&tmem, 128);
    const int a = valid_adapter(p, index);
    if (tid == 0 && a >= 0)
        for (int i = 0; i < kParts; ++i) {
            constexpr int kPer = kColBlocks / kParts;
            mbar_arrive_expect_tx(&full[i], kPer * (kTcXBlock + a_block));
            for (int kb = i * kPer; kb < (i + 1) * kPer; ++kb) {
                tc::tma_2d(sm + kb * kTcXBlock, &mx, 64 * kb, (int)row0, &full[i]);
                tc::tma_2d(sm + a_off + kb * a_block, &ma, 64 * kb, a * p.rank, &full[i]);
            }
        }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (a < 0) {
        if (warp == 1) tc::tmem_free(tmem, 128);
        return;
    }
    bool ok = true;
    if (warp == 0) {
        const uint32_t one = tc::elect_one(), idesc = idesc_bf16((p.rank + 15) / 16 * 16);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            constexpr int kPer = kColBlocks / kParts;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[i], 0));
            if (!ok) break;
            tc::fence_after();
            mma_latent(tmem, smem_u32(sm), kTcXBlock, smem_u32(sm) + a_off, a_block, idesc, one, i * kPer, (i + 1) * kPer);
        }
        if (one) tc::commit(&done);     // of those issued
        __syncwarp();
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
                __syncwarp();       // lanes past the pairs store nothing
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
        for (int i = 0; i < kParts; ++i) mbar_wait(&full[i], 0);
        mbar_wait(&done, 0);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_free(tmem, 128);
}

// ------------------------------------------------------------------ project

constexpr int kABlock = MLA_D_V * 128;             // one column block of W_UV[h]: 16 KB
constexpr int kXOff = kColBlocks * kABlock;        // the tile's latents

// --------------------------------- project: B T by warp MMAs (one row a request)

constexpr int kFewThreads = 512;                   // and a warp that issues copies and products
constexpr int kBatch = 4;                          // items a warp expands at once
constexpr int kDStride = MLA_D_V + 4;              // float32 tile rows, a bank apart per row pair

// A row of T, hi and lo, in shared memory (its 16 bytes more spread rows over the banks).
__host__ __device__ constexpr int t_stride(int rank) { return 2 * rank + 8; }

// NR rows a tile; two tiles' latents.
template <int NR>
struct FewTile {
    static constexpr int kBBlock = NR * 128, kBBytes = kColBlocks * kBBlock;
    static constexpr int kDOff = kXOff + 2 * kBBytes;
    static constexpr int kTOff = kDOff + NR * kDStride * 4;         // the rows' T
    static constexpr int kSmem = kTOff + NR * t_stride(MLA_MAX_LORA_RANK) * 2 + 1024;
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

// Up to eight rows of a tile that share an adapter, and its B[a, h].
struct Item {
    const __nv_bfloat16 *b;
    int n;
    uint8_t row[8];     // past the n-th: the first again
};

// Run by a warp, lane i with row i's adapter (-1: none): the tile's items; their number.
__device__ __forceinline__ int make_items(const LoraArgs &p, Item *items, int a, int h) {
    const uint32_t lane = threadIdx.x & 31, below = (1u << lane) - 1;
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    const int before = __popc(same & below);
    const bool lead = a >= 0 && before % 8 == 0;
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    if (lead) {
        Item x;
        x.b = p.b + ((int64_t)a * p.H + h) * MLA_D_V * p.rank;
        x.n = min(8, __popc(same) - before);
        uint32_t rest = same & ~below;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            x.row[c] = (uint8_t)(c < x.n ? __ffs(rest) - 1 : lane);
            rest &= rest - 1;
        }
        items[__popc(leads & below)] = x;
    }
    return __popc(leads);
}

// B[a, h] T of the tile's items -> delta[row][v], T staged in `ts`.  Warp w
// takes outputs 16 (w % 8) .. + 15 of every second item, BATCH items at once,
// 8 W ranks a step: a lane's W words of B and of T are W / 2 k-steps' worth.
// FIRST: T is waited for once the first items' B is on its way.
template <int W, int BATCH, bool FIRST>
__device__ __forceinline__ void expand(const LoraArgs &p, float *delta, __nv_bfloat16 *ts, const Item *items,
                                       int nitems, int nrows, int t0, int h) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int v0 = 16 * (warp & 7), rank = p.rank, stride = t_stride(rank);
    const int b_lane = (v0 + g) * rank + 2 * W * q;
    Words<W> x[BATCH], y[BATCH];
    const auto load = [&](int i0, int k) {
        const bool in = k + 2 * W * q < rank;
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            x[u] = y[u] = {};
            if (in && i0 + 2 * u < nitems) {
                const __nv_bfloat16 *b = items[i0 + 2 * u].b + b_lane + k;
                x[u] = load_now<W>(b);
                y[u] = load_now<W>(b + 8 * rank);
            }
        }
    };
    const int first = warp >> 3;
    load(first, 0);
    if (FIRST) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int row = warp; row < nrows; row += kFewThreads / 32)
        if (lane < rank / 4)
            reinterpret_cast<uint4 *>(ts + row * stride)[lane] =
                reinterpret_cast<const uint4 *>(p.t + ((int64_t)(t0 + row) * p.H + h) * 2 * rank)[lane];
    asm volatile("bar.sync 1, %0;" ::"n"(kFewThreads) : "memory");
    for (int i0 = first; i0 < nitems; i0 += 2 * BATCH) {
        float acc[BATCH][4] = {};
        for (int k = 0; k < rank; k += 8 * W) {
            if (i0 > first || k > 0) load(i0, k);
            const bool in = k + 2 * W * q < rank;
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                if (i0 + 2 * u >= nitems) break;
                Words<W> hi = {}, lo = {};
                if (in) {
                    const __nv_bfloat16 *s = ts + items[i0 + 2 * u].row[g] * stride + k + 2 * W * q;
                    hi = load_words<W>(s);
                    lo = load_words<W>(s + rank);
                }
#pragma unroll
                for (int j = 0; j < W; j += 2) {
                    const uint32_t a[4] = {x[u].w[j], y[u].w[j], x[u].w[j + 1], y[u].w[j + 1]};
                    mma_bf16(acc[u], a, hi.w[j], hi.w[j + 1]);
                    mma_bf16(acc[u], a, lo.w[j], lo.w[j + 1]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            if (i0 + 2 * u >= nitems) break;
            const Item &it = items[i0 + 2 * u];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (2 * q + c < it.n) {
                    float *d = delta + it.row[2 * q + c] * kDStride + v0 + g;
                    d[0] = acc[u][c];
                    d[8] = acc[u][2 + c];
                }
        }
    }
}

// NR rows a tile at most, p.tile_rows of them.
template <int NR>
__global__ void __launch_bounds__(kFewThreads + 32, 1)
    project_few_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ml, const LoraArgs p) {
    using T = FewTile<NR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *delta = reinterpret_cast<float *>(sm + T::kDOff);
    __nv_bfloat16 *ts = reinterpret_cast<__nv_bfloat16 *>(sm + T::kTOff);
    __shared__ uint64_t full[2], done[2];
    __shared__ uint32_t tmem;
    __shared__ uint8_t active[NR];
    __shared__ uint8_t adapted[NR];
    __shared__ Item items[NR];
    __shared__ int nitems;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, rows = p.tile_rows, tiles = (p.S + rows - 1) / rows, step = gridDim.x;
    const bool issuer = warp == kFewThreads / 32;   // a whole warp; one lane copies and commits
    const uint32_t one = tc::elect_one();

    // Row `tid`'s adapter and length; the first tile's on their way during the set-up.
    int index = -1, len = 0;
    const auto look = [&](int tile) {
        const int t = tile * rows + tid;
        const bool is = tid < rows && t < p.S;
        index = is ? load_int(p.adapters + t) : -1;
        len = is ? load_int(p.lengths + t) : 0;
    };
    look(blockIdx.x);
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
            tc::tma_3d(sm + kXOff + s * T::kBBytes + kb * T::kBBlock, &ml, 64 * kb, h, tile * rows, &full[s]);
    };
    if (issuer && one) {
        // Nothing here but the low-rank products is written by the kernel
        // before this one: W_UV and the latent are fetched at once.
        fetch(blockIdx.x, 0, kXOff);
        for (int kb = 0; kb < kColBlocks; ++kb) tc::tma_2d(sm + kb * kABlock, &mw, 64 * kb, MLA_D_V * h, &full[0]);
        if (blockIdx.x + step < tiles) fetch(blockIdx.x + step, 1, 0);
    }
    bool ok = true;
    int issued = 0, it = 0;                         // issuing warp: tiles whose products are issued
    const auto multiply = [&](int n) {              // the n-th tile of this block
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[n & 1], (n >> 1) & 1));
        if (!ok) return;
        tc::fence_after();
        mma_latent(tm + (n & 1) * NR, base, kABlock, base + kXOff + (n & 1) * T::kBBytes, T::kBBlock, idesc_bf16(NR), one);
        if (one) tc::commit(&done[n & 1]);
        __syncwarp();
        ++issued;
    };
    for (int tile = blockIdx.x; tile < tiles; tile += step, ++it) {
        const int t0 = tile * rows, nrows = min(rows, p.S - t0);
        if (it > 0) look(tile);
        if (warp == 0) {        // NR <= 32
            const int a = valid_adapter(p, index), n = make_items(p, items, a, h);
            if (lane < NR) {
                active[lane] = len > 0;
                adapted[lane] = a >= 0;
            }
            if (lane == 0) nitems = n;
        }
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
        if (tid < kFewThreads) {
            if (p.rank <= 16) {
                if (it == 0) expand<2, kBatch, true>(p, delta, ts, items, nitems, nrows, t0, h);
                else expand<2, kBatch, false>(p, delta, ts, items, nitems, nrows, t0, h);
            } else {
                if (it == 0) expand<4, kBatch, true>(p, delta, ts, items, nitems, nrows, t0, h);
                else expand<4, kBatch, false>(p, delta, ts, items, nitems, nrows, t0, h);
            }
        }
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
        if (issuer && one && tile + 2 * step < tiles) fetch(tile + 2 * step, it & 1, 0);
        if (tid < kFewThreads) {
            float d[T::kRows];
            ld_rows<T::kRows>(tm + ((uint32_t)(32 * (warp & 3)) << 16) + (it & 1) * NR + first, d);
            tc::wait_ld();
            uint16_t x[T::kRows];
#pragma unroll
            for (int i = 0; i < T::kRows; ++i) {
                const int n = first + i;
                const float val = adapted[n] ? d[i] + delta[n * kDStride + v] : d[i];
                const float y = val * tc::sigmoid_f32(__uint_as_float((uint32_t)gate[i] << 16));
                // a select, so that nothing of an empty request is seen
                x[i] = active[n] ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : 0;
            }
            uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + at;
#pragma unroll
            for (int i = 0; i < T::kRows; ++i)
                if (first + i < nrows) out[(int64_t)i * row_step] = x[i];
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

// ------------------------------------------- project: B T through a ring of tcgen05 MMAs

constexpr int kEpiWarps = 8, kSlotWarp0 = 8, kMaxSlots = 6, kLatentWarp = 14, kItemWarp = 15;
constexpr int kThreads = 16 * 32;
constexpr int kWin = 16;                           // rows of a window

// NR rows a tile; RB ranks of a ring entry (its rows are 2 * RB bytes, the
// swizzle's span).
template <int NR, int RB>
struct Tile {
    static_assert(RB == 32 || RB == 64, "64- or 128-byte swizzle");
    static constexpr int kXBlock = NR * 128, kXBytes = kColBlocks * kXBlock;
    static constexpr int kSlotOff = kXOff + kXBytes;
    static constexpr int kBBytes = MLA_D_V * 2 * RB, kTBytes = kWin * 2 * RB;   // of a slot: B, then T hi, T lo
    static constexpr int kSlot = kBBytes + 2 * kTBytes;
    static constexpr int kSlots = RB == 32 ? kMaxSlots : 3;
    static constexpr int kSmem = kSlotOff + kSlots * kSlot + 1024;
    static constexpr int kRows = NR / 2;           // rows per thread in the epilogue
    // TMEM columns: two tiles' projections, then the entries of one tile or,
    // in halves of kAddBuf, of two.
    static constexpr int kAddCols = 2 * NR, kAddBuf = (512 - kAddCols) / 2 / kWin * kWin;
    static_assert((512 - kAddCols) / kWin >= NR / kWin * 9, "the entries of a tile, at two rows a request or more");
    static constexpr uint32_t kSwz = RB == 32 ? tc::kSw64 : tc::kSw128, kSbo = 16 * RB;
};

__device__ __forceinline__ float ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return __uint_as_float(r);
}

// A block's ring entries in order: tile, 16-row window, eight rows (or the
// request's rest) of a request there, chunk of RB ranks.
template <int NR, int RB>
struct Entries {
    int tile, win, item, chunk, items, r0, t0, nrows, chunks;

    __device__ void open(const LoraArgs &p) {       // the window's items
        t0 = tile * NR + win * kWin;
        nrows = min(kWin, p.S - t0);
        r0 = request_of(p, t0);
        items = nrows <= 0 ? 0 : (request_of(p, t0 + nrows - 1) - r0 + 1) << (p.qlen > 8);
    }
    __device__ void init(const LoraArgs &p) {
        tile = blockIdx.x;
        win = item = chunk = 0;
        chunks = (p.rank + RB - 1) / RB;
        open(p);
    }
    __device__ int in_window() const { return items * chunks; }
};

template <int NR, int RB>
struct Shared {
    uint64_t w_full, x_full, x_empty, d_full[2], d_free[2], add_free[2], s_full[kMaxSlots], s_empty[kMaxSlots], fin;
    uint32_t tmem;
    int abort_flag;
};

// Fills slot s with entries s, s + slots, ... of the block.
template <int NR, int RB>
__device__ void slot_filler(const LoraArgs &p, const CUtensorMap *mb, uint8_t *sm, Shared<NR, RB> &sh, int s, int h,
                            int tiles) {
    using T = Tile<NR, RB>;
    const int lane = threadIdx.x & 31;
    uint8_t *slot = sm + T::kSlotOff + s * T::kSlot;
    const int log_per = p.qlen > 8;     // a request's items, as a power of two
    Entries<NR, RB> e;
    e.init(p);
    int n = 0, skip = s;            // uses of the slot; entries to pass by first
    while (e.tile < tiles) {
        if (skip >= e.in_window()) {
            skip -= e.in_window();
            if (++e.win == NR / kWin) {
                e.win = 0;
                e.tile += gridDim.x;
            }
            if (e.tile < tiles) e.open(p);
            continue;
        }
        const int item = e.chunks == 2 ? skip >> 1 : skip / e.chunks, k0 = (skip - item * e.chunks) * RB;
        skip += T::kSlots;
        const int r = e.r0 + (item >> log_per), first = r * p.qlen + (item & log_per) * 8;
        const int lo = max(first, e.t0), hi = min(min(first + 8, (r + 1) * p.qlen), e.t0 + e.nrows);
        const int index = lo < hi ? __ldg(p.adapters + r) : -1;
        // T's rows of the window as the B operand, 16-byte chunks: hi, then
        // lo; other rows and ranks zero (without an adapter whatever is there,
        // unused).  On their way while the slot is waited for.
        constexpr int kChunks = RB / 8, kPer = kWin * 2 * kChunks / 32;
        uint4 v[kPer];
        const auto load = [&] {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int c = lane + 32 * j, row = c / (2 * kChunks), half = c / kChunks % 2, k = k0 + c % kChunks * 8;
                const int t = e.t0 + row;
                v[j] = make_uint4(0, 0, 0, 0);
                if (t >= lo && t < hi && k < p.rank)
                    v[j] = *reinterpret_cast<const uint4 *>(p.t + (((int64_t)t * p.H + h) * 2 + half) * p.rank + k);
            }
        };
        if (n > 0) load();
        if (!warp_wait(&sh.s_empty[s], (n & 1) ^ 1, &sh.abort_flag)) break;
        const int a = valid_adapter(p, index);
        if (lane == 0) {
            if (a >= 0) {
                mbar_arrive_expect_tx(&sh.s_full[s], T::kBBytes);
                tc::tma_2d(slot, mb, k0, (a * p.H + h) * MLA_D_V, &sh.s_full[s]);
            } else {
                mbar_arrive(&sh.s_full[s]);
            }
        }
        __syncwarp();
        if (n++ == 0) {     // T is written by the kernel before this one, B is not
            asm volatile("griddepcontrol.wait;" ::: "memory");
            load();
        }
        if (a >= 0) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int c = lane + 32 * j, row = c / (2 * kChunks), half = c / kChunks % 2, byte = c % kChunks * 16;
                uint8_t *d = slot + T::kBBytes + half * T::kTBytes + (row >> 3) * T::kSbo +
                             (RB == 32 ? tc::sw64(row, byte) : tc::sw128(row, byte));
                *reinterpret_cast<uint4 *>(d) = v[j];
            }
            tc::fence_async_smem();     // generic-proxy writes -> tensor-core reads
            __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sh.s_full[s]);
    }
    // Flagged elsewhere: let a copy of this slot's land before the block ends.
    if (*(volatile int *)&sh.abort_flag && n > 0) mbar_wait(&sh.s_full[s], (n - 1) & 1);
}

template <int NR, int RB>
__global__ void __launch_bounds__(kThreads, 1)
    project_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ml,
                   const __grid_constant__ CUtensorMap mb, const LoraArgs p) {
    using T = Tile<NR, RB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Shared<NR, RB> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, tiles = (p.S + NR - 1) / NR, step = gridDim.x;
    if (tid == 0) {
        mbar_init(&sh.w_full, 1);
        mbar_init(&sh.x_full, 1);
        mbar_init(&sh.x_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.d_full[i], 2);
            mbar_init(&sh.d_free[i], kEpiWarps);
            mbar_init(&sh.add_free[i], kEpiWarps);
        }
        for (int i = 0; i < T::kSlots; ++i) {
            mbar_init(&sh.s_full[i], 2);
            mbar_init(&sh.s_empty[i], 1);
        }
        mbar_init(&sh.fin, 2);
        sh.abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kLatentWarp) tc::tmem_alloc(&sh.tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t base = smem_u32(sm), tm = sh.tmem;
    const auto wait_warp = [&](uint64_t *bar, uint32_t par) { return warp_wait(bar, par, &sh.abort_flag); };
    if (warp == kLatentWarp) {
        // Neither W_UV nor the latent is written by the kernel before this
        // one.  Rows past S read as zeros (their outputs are not written).
        const uint32_t one = tc::elect_one();
        int fetched = 0;
        const auto fetch = [&](int tile) {
            if (one) {
                mbar_arrive_expect_tx(&sh.x_full, T::kXBytes);
                for (int kb = 0; kb < kColBlocks; ++kb)
                    tc::tma_3d(sm + kXOff + kb * T::kXBlock, &ml, 64 * kb, h, tile * NR, &sh.x_full);
            }
            __syncwarp();
            ++fetched;
        };
        if (one) {
            mbar_arrive_expect_tx(&sh.w_full, kXOff);
            for (int kb = 0; kb < kColBlocks; ++kb) tc::tma_2d(sm + kb * kABlock, &mw, 64 * kb, MLA_D_V * h, &sh.w_full);
        }
        fetch(blockIdx.x);
        bool ok = wait_warp(&sh.w_full, 0);
        int it = 0;
        for (int tile = blockIdx.x; ok && tile < tiles; tile += step, ++it) {
            if (!(ok = wait_warp(&sh.x_full, it & 1))) break;
            if (!(ok = wait_warp(&sh.d_free[it & 1], ((it >> 1) & 1) ^ 1))) break;
            tc::fence_after();
            mma_latent(tm + (it & 1) * NR, base, kABlock, base + kXOff, T::kXBlock, idesc_bf16(NR), one);
            if (one) {
                tc::commit(&sh.x_empty);
                tc::commit(&sh.d_full[it & 1]);
            }
            __syncwarp();
            if (tile + step < tiles) {
                if (!(ok = wait_warp(&sh.x_empty, it & 1))) break;
                fetch(tile + step);
            }
        }
        if (!ok) {          // flagged: the copies in flight land before the block ends
            mbar_wait(&sh.w_full, 0);
            mbar_wait(&sh.x_full, (fetched - 1) & 1);
        }
        // Every MMA issued must be complete before TMEM is released.
        if (one) tc::commit(&sh.fin);
        __syncwarp();
        mbar_wait(&sh.fin, 0);
    } else if (warp == kItemWarp) {
        const uint32_t one = tc::elect_one();
        bool ok = true, ready = false;      // the next slot is known to be full
        int it = 0, s = 0, s_phase = 0;
        const uint64_t b_desc = tc::sdesc(base + T::kSlotOff, 16, T::kSbo, T::kSwz);
        const uint64_t t_desc = tc::sdesc(base + T::kSlotOff + T::kBBytes, 16, T::kSbo, T::kSwz);
        Entries<NR, RB> e;
        e.init(p);
        for (int tile = blockIdx.x; ok && tile < tiles; tile += step, ++it) {
            int items = 0;
            e.tile = tile;
            for (e.win = 0; e.win < NR / kWin; ++e.win) {
                e.open(p);
                items += e.items;
            }
            const int buf = it & p.add_both, use = it >> p.add_both;
            if (!(ok = wait_warp(&sh.add_free[buf], (use & 1) ^ 1))) break;
            tc::fence_after();
            uint32_t add = tm + T::kAddCols + buf * T::kAddBuf;
            for (int i = 0; ok && i < items; ++i, add += kWin)
                for (int k0 = 0; k0 < p.rank; k0 += RB) {
                    if (!ready && !(ok = wait_warp(&sh.s_full[s], s_phase))) break;
                    tc::fence_after();
                    // 32 bytes of the ranks a step: 2 in a descriptor's address field
                    const uint64_t b = b_desc + s * (T::kSlot >> 4), x = t_desc + s * (T::kSlot >> 4);
                    uint64_t *empty = &sh.s_empty[s];
                    if (++s == T::kSlots) s = 0, s_phase ^= 1;
                    const uint32_t next = mbar_test(&sh.s_full[s], s_phase);    // the answer comes during the MMAs
                    // (An entry without an adapter multiplies what the slot
                    // holds into columns that nothing reads.)
#pragma unroll
                    for (int j = 0; j < RB / 16; ++j)
                        if (k0 + 16 * j < p.rank) {
                            mma_bf16_tc(add, b + 2 * j, x + 2 * j, idesc_bf16(kWin), k0 > 0 || j > 0, one);
                            mma_bf16_tc(add, b + 2 * j, x + (T::kTBytes >> 4) + 2 * j, idesc_bf16(kWin), true, one);
                        }
                    if (one) tc::commit(empty);
                    ready = __all_sync(0xffffffffu, next);
                }
            if (ok && one) tc::commit(&sh.d_full[it & 1]);
            __syncwarp();
        }
        if (one) tc::commit(&sh.fin);
        __syncwarp();
        mbar_wait(&sh.fin, 0);
    } else if (warp >= kSlotWarp0) {
        if (warp - kSlotWarp0 < T::kSlots) {
            slot_filler<NR, RB>(p, &mb, sm, sh, warp - kSlotWarp0, h, tiles);
        }
    } else {
        // Output v of rows first .. first + kRows - 1 of the tile.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int v = 32 * (warp & 3) + lane, first = (warp >> 2) * T::kRows;
        const int64_t row_step = (int64_t)p.H * MLA_D_V;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // Gates and, of row `lane`, length and adapter: the next tile's are
        // loaded before this one's results are stored.
        struct Inputs {
            uint16_t gate[T::kRows];
            int len, adapter;
        };
        const auto load = [&](Inputs &x, int tile) {
            const int t0 = tile * NR + first, nrows = min(T::kRows, p.S - t0);
            const uint16_t *gate = reinterpret_cast<const uint16_t *>(p.gate) + ((int64_t)t0 * p.H + h) * MLA_D_V + v;
#pragma unroll
            for (int i = 0; i < T::kRows; ++i) x.gate[i] = i < nrows ? __ldg(gate + i * row_step) : 0;
            x.len = 0;
            x.adapter = -1;
            if (lane < nrows) {
                const int r = request_of(p, t0 + lane);
                x.len = __ldg(p.lengths + r);
                x.adapter = __ldg(p.adapters + r);
            }
        };
        Inputs in, next;
        load(in, blockIdx.x);
        int it = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += step, ++it, in = next) {
            const int t0 = tile * NR + first, nrows = min(T::kRows, p.S - t0);
            const int64_t at = ((int64_t)t0 * p.H + h) * MLA_D_V + v;
            const uint32_t live = __ballot_sync(0xffffffffu, in.len > 0);
            const uint32_t adapted = __ballot_sync(0xffffffffu, in.adapter >= 0 && in.adapter < p.n);
            // Lane i: the column of row i's low-rank part.
            const int w0 = tile * NR, win = first / kWin * kWin, log_per = p.qlen > 8;
            int item = win ? (request_of(p, w0 + kWin - 1) - request_of(p, w0) + 1) << log_per : 0;
            const int r = request_of(p, t0 + lane);
            item += ((r - request_of(p, w0 + win)) << log_per) + ((t0 + lane - r * p.qlen) >> 3);
            const int col = T::kAddCols + (it & p.add_both) * T::kAddBuf + item * kWin + (first + lane) % kWin;
            if (!warp_wait(&sh.d_full[it & 1], (it >> 1) & 1, &sh.abort_flag)) break;
            tc::fence_after();
            float d[T::kRows];
#pragma unroll
            for (int c = 0; c < T::kRows; c += 8)
                tc::ld8(tm + lanes + (it & 1) * NR + first + c, d + c);
            float add[T::kRows];
#pragma unroll
            for (int i = 0; i < T::kRows; ++i) {
                const int c = __shfl_sync(0xffffffffu, col, i);
                add[i] = ld1(tm + lanes + (adapted >> i & 1 ? c : T::kAddCols));
            }
            tc::wait_ld();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.d_free[it & 1]);
                mbar_arrive(&sh.add_free[it & p.add_both]);
            }
            if (tile + step < tiles) load(next, tile + step);
            // (Without branches between the rows: one at a time they would
            // take 2,400 cycles.)
            uint16_t x[T::kRows];
#pragma unroll
            for (int i = 0; i < T::kRows; ++i) {
                const float val = adapted >> i & 1 ? d[i] + add[i] : d[i];
                const float y = val * tc::sigmoid_f32(__uint_as_float((uint32_t)in.gate[i] << 16));
                // a select, so that nothing of an empty request is seen
                x[i] = live >> i & 1 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : 0;
            }
            uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + at;
#pragma unroll
            for (int i = 0; i < T::kRows; ++i)
                if (i < nrows) out[i * row_step] = x[i];
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kLatentWarp) tc::tmem_free(tm, 512);
}

bool encode_bf16(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dim, const cuuint64_t *stride,
                 const cuuint32_t *box, CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    const cuuint32_t es[3] = {1, 1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dim, stride, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_NONE,
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
    // cost more than the taller tiles' start: at 768 of them (128 requests of
    // eight rows, 12 heads) the whole call takes 12.3 us at rank 16 and 23.6 at
    // rank 128 by tcgen05, 14.9 and 35.1 by warp MMAs; at 1,536 27.0 and 39.4 at
    // rank 64, 39.3 and 52.4 at rank 72 (one block an SM).  Below that number
    // warp MMAs are ahead for small ranks and few pairs only (192 blocks at rank
    // 16 7.2 us against 7.6; at 384 already 10.8 against 10.0, at rank 128 21.9
    // against 16.0): the limit is on the high side.
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

template <class... Args>
cudaError_t launch_project(void (*kernel)(Args...), int nr, int threads, int smem, const LoraArgs &p, int sms,
                           cudaStream_t st, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min((p.S + nr - 1) / nr, std::max(1, sms / p.H)), p.H, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The latent as [S][H][512], NR rows a box.
bool encode_latent(CUtensorMap *m, const LoraArgs &p, int nr) {
    const cuuint64_t dim[3] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)p.H, (cuuint64_t)p.S};
    const cuuint64_t stride[2] = {(cuuint64_t)MLA_D_LATENT * 2, (cuuint64_t)p.H * MLA_D_LATENT * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)nr};
    return encode_bf16(m, p.latent, 3, dim, stride, box);
}

template <int NR>
cudaError_t project_few(const CUtensorMap &mw, const LoraArgs &p, int sms, cudaStream_t st) {
    CUtensorMap ml;
    if (!encode_latent(&ml, p, NR)) return cudaErrorInvalidValue;
    cudaError_t e = smem_attr_once<project_few_kernel<NR>>(FewTile<NR>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_project(project_few_kernel<NR>, p.tile_rows, kFewThreads + 32, FewTile<NR>::kSmem, p, sms, st, mw, ml,
                          p);
}

template <int NR, int RB>
cudaError_t project(const CUtensorMap &mw, const LoraArgs &p, int sms, cudaStream_t st) {
    // lora_b as [n * H * 128, rank]; columns past the rank read as zeros.
    const cuuint64_t bdim[2] = {(cuuint64_t)p.rank, (cuuint64_t)p.n * p.H * MLA_D_V};
    const cuuint64_t bstride[1] = {(cuuint64_t)p.rank * 2};
    const cuuint32_t bbox[2] = {(cuuint32_t)RB, (cuuint32_t)MLA_D_V};
    CUtensorMap ml, mb;
    if (!encode_latent(&ml, p, NR) ||
        !encode_bf16(&mb, p.b, 2, bdim, bstride, bbox, RB == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    cudaError_t e = smem_attr_once<project_kernel<NR, RB>>(Tile<NR, RB>::kSmem);
    if (e != cudaSuccess) return e;
    LoraArgs q = p;
    const int items = ((kWin + p.qlen - 2) / p.qlen + 1) << (p.qlen > 8);      // of a window, at most
    q.add_both = items * (NR / kWin) * kWin <= Tile<NR, RB>::kAddBuf;
    return launch_project(project_kernel<NR, RB>, NR, kThreads, Tile<NR, RB>::kSmem, p, sms, st, mw, ml, mb, q);
}

}  // namespace

int64_t value_lora_workspace(int64_t rows, int heads, int rank) { return rows * heads * rank * 4; }

cudaError_t value_lora_launch(const void *latent, const void *w_uv, const void *gate, const int32_t *lengths,
                              const void *lora_a, const void *lora_b, const int32_t *adapters, const float *lora_scale,
                              int num_adapters, int rank, int R, int qlen, int H, void *out, void *workspace, int sms,
                              cudaStream_t st) {
    if (!tc::encode_fn()) return cudaErrorNotSupported;
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
    p.inv_qlen = ((1ull << 35) + qlen - 1) / qlen;
    p.H = H;
    p.rank = rank;
    p.n = num_adapters;
    CUtensorMap mw;
    if (!encode_rows(&mw, w_uv, (int64_t)H * MLA_D_V, MLA_D_V)) return cudaErrorInvalidValue;
    cudaError_t e = shrink(p, R, sms, st);
    if (e != cudaSuccess) return e;
    // 32-row tiles, unless 16-row ones leave no block of a head with two.
    const bool low = (p.S + 15) / 16 <= std::max(1, sms / H);
    // With one row a request every row has an entry of its own, whose way
    // through the ring costs more than its warp MMAs: 64 requests of 12 heads
    // 6.8 us by warp MMAs and 7.9 through the ring at rank 16, 9.4 and 11.7 at
    // rank 64 (and a 32-row tile's entries would not fit TMEM).  With eight
    // rows a request (256 of rank 64) 46 and 28 us, with four 29 and 20.
    if (qlen == 1) {
        p.tile_rows = low ? 16 : 32;
        // Down to four rows while every tile has a block of its own: a row's
        // expansion takes its block's time (64 requests of rank 64 11.3 us
        // with 16 rows, 9.4 with eight; 16 of them 11.0, and 7.4 with four).
        const auto tiles = [&](int rows) { return (p.S + rows - 1) / rows; };
        while (low && p.tile_rows > 4 && tiles(p.tile_rows / 2) <= std::max(1, sms / H)) p.tile_rows /= 2;
        return low ? project_few<16>(mw, p, sms, st) : project_few<32>(mw, p, sms, st);
    }
    if (rank <= 32) return low ? project<16, 32>(mw, p, sms, st) : project<32, 32>(mw, p, sms, st);
    return low ? project<16, 64>(mw, p, sms, st) : project<32, 64>(mw, p, sms, st);
}

cudaError_t value_lora_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
