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
//   shrink: one block per request and tile of its (row, head) pairs, which
//     share A: T = latent A^T * lora_scale by warp MMAs on fragments loaded
//     straight from global memory (a lane's 16 bytes are two k-steps' worth:
//     the products' order over k is free).  Eight warps take 64 latent
//     columns each and are joined in shared memory.  T goes to the workspace
//     as two bf16 terms, hi + lo (2^-17 of the product; one term would add
//     2^-9, as much as the output's own rounding).
//   project: one block per (rows, head).  W_UV[h] (M = 128 outputs) times the
//     rows' latents (N) by tcgen05 MMAs on TMA tiles into TMEM, as in the
//     plain projection; meanwhile the 16 warps form B T by warp MMAs into a
//     float32 tile, reading B[a, h] once per request of the tile (every
//     column of a warp MMA is a row of its own, so rows of other requests
//     need no mask).  The epilogue adds the two and gates.
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

// ------------------------------------------------------------------ shrink

constexpr int kShrinkWarps = 8;
constexpr int kNChunk = 8;              // n-tiles (of 8 ranks) whose sums a warp holds at once

// MT tiles of 16 (row, head) pairs per block.
template <int MT>
__global__ void __launch_bounds__(kShrinkWarps * 32) shrink_kernel(const LoraArgs p, int tiles) {
    extern __shared__ float part[];     // [warps][16 * MT][kNChunk * 8 + 1]
    constexpr int kCols = kNChunk * 8 + 1;
    asm volatile("griddepcontrol.launch_dependents;");
    const int r = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int a = adapter_of(p, r);
    if (a < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int pairs = p.qlen * p.H, m0 = tile * 16 * MT;
    const int64_t row0 = (int64_t)r * pairs;
    const float scale = __ldg(p.scale + a);
    const int c0 = warp * 64 + 8 * q;   // this lane's columns: c0 .. c0 + 7 and c0 + 32 ..
    uint4 x[MT][2][2];                  // [tile][32-column block][row g, g + 8]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = min(m0 + 16 * m + 8 * i + g, pairs - 1);
            const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + (row0 + row) * MLA_D_LATENT + c0);
#pragma unroll
            for (int b = 0; b < 2; ++b) x[m][b][i] = __ldg(src + 4 * b);
        }
    const int ntiles = p.rank / 8;
    for (int n0 = 0; n0 < ntiles; n0 += kNChunk) {
        const int nn = min(kNChunk, ntiles - n0);
        float acc[MT][kNChunk][4] = {};
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
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint4 u = x[m][b][0], v = x[m][b][1], k = w[n][b];
                        const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                        mma_bf16(acc[m][n], a0, k.x, k.y);
                        mma_bf16(acc[m][n], a1, k.z, k.w);
                    }
        if (n0 > 0) __syncthreads();
#pragma unroll
        for (int n = 0; n < kNChunk; ++n)
            if (n < nn)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part[(warp * 16 * MT + 16 * m + g + 8 * (i >> 1)) * kCols + 8 * n + 2 * q + (i & 1)] =
                            acc[m][n][i];
        __syncthreads();
        const int cols = 8 * nn;
        for (int e = threadIdx.x; e < 16 * MT * cols; e += kShrinkWarps * 32) {
            const int row = e / cols, k = e - row * cols;
            if (m0 + row >= pairs) break;
            float s = 0.f;
#pragma unroll
            for (int w8 = 0; w8 < kShrinkWarps; ++w8) s += part[(w8 * 16 * MT + row) * kCols + k];
            s *= scale;
            const __nv_bfloat16 hi = __float2bfloat16_rn(s);
            __nv_bfloat16 *dst = p.t + (row0 + m0 + row) * 2 * p.rank + 8 * n0 + k;
            dst[0] = hi;
            // no lo beside an infinite hi (inf - inf)
            dst[p.rank] = __float2bfloat16_rn(isinf(__bfloat162float(hi)) ? 0.f : s - __bfloat162float(hi));
        }
    }
}

// ------------------------------------------------------------------ project

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kColBlocks = MLA_D_LATENT / 64;      // 128-byte column blocks of the K axis
constexpr int kABlock = MLA_D_V * 128;             // one column block of W_UV[h]: 16 KB
constexpr int kBOff = kColBlocks * kABlock;
constexpr int kDStride = MLA_D_V + 4;              // float32 tile rows, a bank apart per row pair

template <int NR>
struct Tile {
    static constexpr int kBBlock = NR * 128;
    static constexpr int kDOff = kBOff + kColBlocks * kBBlock;
    static constexpr int kSmem = kDOff + NR * kDStride * 4 + 1024;
    static constexpr uint32_t kTmemCols = NR <= 32 ? 32 : 64;
    static constexpr int kPairs = NR * (MLA_D_V / 2) / kThreads;     // gate / output words per thread
    // kind::f16: bf16 A and B (K-major), f32 D, M = 128, N = NR.
    static constexpr uint32_t kIdesc =
        (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

__device__ __forceinline__ void mma_bf16_tc(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate));
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

// 1 / (1 + e^-x); e^-x = inf gives 0.
__device__ __forceinline__ float sigmoid_f32(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x)));
    return r;
}

// B[a, h] T of the tile's rows [t0, t0 + nrows) -> delta[row][v].  Warp w
// takes outputs 16 (w % 8) .. + 15 of every second request.
__device__ void expand(const LoraArgs &p, float *delta, int t0, int nrows, int h) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int v0 = 16 * (warp & 7);
    const int r_end = (t0 + nrows - 1) / p.qlen;
    for (int r = t0 / p.qlen + (warp >> 3); r <= r_end; r += 2) {
        const int a = adapter_of(p, r);
        if (a < 0) continue;
        const int s = max(r * p.qlen, t0), e = min((r + 1) * p.qlen, t0 + nrows);
        const __nv_bfloat16 *bsrc = p.b + (((int64_t)a * p.H + h) * MLA_D_V + v0 + g) * p.rank + 8 * q;
        for (int n0 = s; n0 < e; n0 += 8) {
            const int row = min(n0 + g, e - 1);        // columns past the request are not kept
            const __nv_bfloat16 *tsrc = p.t + ((int64_t)row * p.H + h) * 2 * p.rank + 8 * q;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int k = 0; k < p.rank; k += 32) {
                uint4 u = make_uint4(0, 0, 0, 0), v = u, hi = u, lo = u;
                if (k + 8 * q < p.rank) {
                    u = __ldg(reinterpret_cast<const uint4 *>(bsrc + k));
                    v = __ldg(reinterpret_cast<const uint4 *>(bsrc + 8 * p.rank + k));
                    hi = *reinterpret_cast<const uint4 *>(tsrc + k);
                    lo = *reinterpret_cast<const uint4 *>(tsrc + p.rank + k);
                }
                const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                mma_bf16(acc, a0, hi.x, hi.y);
                mma_bf16(acc, a1, hi.z, hi.w);
                mma_bf16(acc, a0, lo.x, lo.y);
                mma_bf16(acc, a1, lo.z, lo.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 2 * q + (i & 1);
                if (n < e) delta[(n - t0) * kDStride + v0 + g + 8 * (i >> 1)] = acc[i];
            }
        }
    }
}

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
    project_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ml, const LoraArgs p) {
    using T = Tile<NR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *delta = reinterpret_cast<float *>(sm + T::kDOff);
    __shared__ uint64_t full, done;
    __shared__ uint32_t tmem;
    __shared__ uint8_t active[NR], adapted[NR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.x * NR, h = blockIdx.y;
    const int nrows = min(NR, p.S - t0);

    if (tid == 0) {
        mbar_init(&full, 1);
        mbar_init(&done, 1);
        mbar_fence_init();
    }
    if (warp == 0) tc::tmem_alloc(&tmem, T::kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (tid == 0) {
        // Nothing here but the low-rank products is written by the kernel
        // before this one: W_UV and the latent are fetched first.  Rows past
        // S read as zeros (their outputs are not written).
        mbar_arrive_expect_tx(&full, kColBlocks * (kABlock + T::kBBlock));
        for (int kb = 0; kb < kColBlocks; ++kb) {
            tma_2d(sm + kb * kABlock, &mw, 64 * kb, MLA_D_V * h, &full);
            tma_3d(sm + kBOff + kb * T::kBBlock, &ml, 64 * kb, h, t0, &full);
        }
    }
    for (int i = tid; i < NR; i += kThreads) {
        const int r = (t0 + i) / p.qlen;
        active[i] = i < nrows && __ldg(p.lengths + r) > 0;
        adapted[i] = i < nrows && adapter_of(p, r) >= 0;
    }
    // This thread's gate words (bf16 pairs w = tid + 512 k: row w / 64, pair
    // w % 64), in flight during the copies and the products.
    uint32_t gw[T::kPairs];
#pragma unroll
    for (int k = 0; k < T::kPairs; ++k) {
        const int w = tid + kThreads * k, r = w / (MLA_D_V / 2), i = w - r * (MLA_D_V / 2);
        gw[k] = r < nrows ? __ldg(reinterpret_cast<const uint32_t *>(p.gate + ((int64_t)(t0 + r) * p.H + h) * MLA_D_V +
                                                                     2 * i))
                          : 0u;
    }
    const uint32_t base = smem_u32(sm), tm = tmem;
    bool ok = true, issued = false;
    if (tid == 0) {
        ok = mbar_wait(&full, 0);
        if (ok) {
            issued = true;
            tc::fence_after();
#pragma unroll
            for (int j = 0; j < MLA_D_LATENT / 16; ++j) {
                const int kb = j >> 2, off = (j & 3) * 32;
                mma_bf16_tc(tm, tc::sdesc(base + kb * kABlock + off, 16, 1024, tc::kSw128),
                            tc::sdesc(base + kBOff + kb * T::kBBlock + off, 16, 1024, tc::kSw128), T::kIdesc, j > 0);
            }
            tc::commit(&done);
        }
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    expand(p, delta, t0, nrows, h);
    ok = __syncthreads_and(ok);
    if (ok) ok = mbar_wait(&done, 0);
    ok = __syncthreads_and(ok);
    if (!ok) {
        // Flagged.  The copies and MMAs in flight finish (one more bounded
        // wait each) before TMEM is released and the CTA ends.
        if (tid == 0) {
            mbar_wait(&full, 0);
            if (issued) mbar_wait(&done, 0);
        }
        tc::fence_before();
        __syncthreads();
        if (warp == 0) tc::tmem_free(tm, T::kTmemCols);
        return;
    }
    tc::fence_after();
    if (warp < 4) {
        const int v = 32 * warp + lane;
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
            float d[16];
            tc::ld16(tm + ((uint32_t)(32 * warp) << 16) + c, d);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float *x = delta + (c + i) * kDStride + v;
                *x = adapted[c + i] ? d[i] + *x : d[i];
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tm, T::kTmemCols);
#pragma unroll
    for (int k = 0; k < T::kPairs; ++k) {
        const int w = tid + kThreads * k, r = w / (MLA_D_V / 2), i = w - r * (MLA_D_V / 2);
        if (r >= nrows) break;
        uint32_t res = 0u;      // a select, so that nothing of an empty request is seen
        if (active[r]) {
            const float2 val = *reinterpret_cast<const float2 *>(delta + r * kDStride + 2 * i);
            res = pack_bf16x2(val.x * sigmoid_f32(bf16_lo(gw[k])), val.y * sigmoid_f32(bf16_hi(gw[k])));
        }
        *reinterpret_cast<uint32_t *>(p.out + ((int64_t)(t0 + r) * p.H + h) * MLA_D_V + 2 * i) = res;
    }
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

template <int MT>
cudaError_t shrink(const LoraArgs &p, int R, cudaStream_t st) {
    constexpr int smem = kShrinkWarps * 16 * MT * (kNChunk * 8 + 1) * 4;
    cudaError_t e = smem_attr_once<shrink_kernel<MT>>(smem);
    if (e != cudaSuccess) return e;
    const int tiles = (p.qlen * p.H + 16 * MT - 1) / (16 * MT);
    shrink_kernel<MT><<<(unsigned)R * tiles, kShrinkWarps * 32, smem, st>>>(p, tiles);
    return cudaGetLastError();
}

template <int NR>
cudaError_t project(const CUtensorMap &mw, const void *latent, const LoraArgs &p, cudaStream_t st) {
    const cuuint64_t dim[3] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)p.H, (cuuint64_t)p.S};
    const cuuint64_t stride[2] = {(cuuint64_t)MLA_D_LATENT * 2, (cuuint64_t)p.H * MLA_D_LATENT * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)NR};
    CUtensorMap ml;
    if (!encode_bf16(&ml, latent, 3, dim, stride, box)) return cudaErrorInvalidValue;
    cudaError_t e = smem_attr_once<project_kernel<NR>>(Tile<NR>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.S + NR - 1) / NR, p.H, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
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
    const cuuint64_t dim[2] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)H * MLA_D_V};
    const cuuint64_t stride[1] = {(cuuint64_t)MLA_D_LATENT * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)MLA_D_V};
    CUtensorMap mw;
    if (!encode_bf16(&mw, w_uv, 2, dim, stride, box)) return cudaErrorInvalidValue;
    // A block's adapter is read once per tile: taller tiles where there are enough of them.
    cudaError_t e = (int64_t)R * ((qlen * H + 31) / 32) > 2 * (int64_t)sms ? shrink<3>(p, R, st) : shrink<1>(p, R, st);
    if (e != cudaSuccess) return e;
    // Rows per CTA (one CTA per SM): the fewest that still leave at most two waves.
    const auto ctas = [&](int nr) { return (int64_t)((p.S + nr - 1) / nr) * H; };
    if (ctas(16) <= 2 * (int64_t)sms) return project<16>(mw, latent, p, st);
    if (ctas(32) <= 2 * (int64_t)sms) return project<32>(mw, latent, p, st);
    return project<64>(mw, latent, p, st);
}

cudaError_t value_lora_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
