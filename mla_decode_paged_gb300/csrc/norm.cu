// Residual addition, root-mean-square norm and output in 16 or 8 bits.
//
// What it computes, for every row t of `width` columns, in float32:
//   s = x[t] + residual[t];  residual_out[t] = round(s)
//   y = s * rsqrt(mean(s^2) + eps) * weight
//   out[t] = round(y), or e4m3 codes of y / scale with scale = amax / 448
//   over the row, over each 128 columns, or one given number.
//
// Bound by DRAM: 7 bytes per element with a bf16 residual and an e4m3
// output, each read or written once; by launch and two trips to memory for a
// few rows.
//
// A row stays in registers between its loads and its stores: thread i of the
// row's T threads holds the 8-column vectors i, i + T, ... (16-byte loads,
// coalesced; VPT vectors a thread, all loads issued before the first use), the
// sum of squares (and a row's maximum) is joined by shuffles and, where more
// than one warp holds the row, through shared memory.  128 columns are 16
// consecutive vectors, so a group's maximum stays inside a half warp (T is a
// multiple of 16).
//
// Batches of many wide rows run a persistent form of the same: a block's next
// rows arrive by bulk copies in a ring in shared memory while it works on
// one, and its weights stay in registers.
//
// Measured (bf16, residual added in bf16): 64 rows of 7,168 in 2.9 us; 16,384
// rows of 7,168 with group scales in 145 us, 5.7 TB/s (one row after another
// without the ring: 219 us); 100,000 rows of 1,024 likewise in 111 us, 6.4 TB/s.
// Wide rows: 4,000 of 16,384 in 92 us, 5.7 TB/s (float32 residual: 128, 6.2).
// Above that a thread of a block of up to 1,024 holds four vectors at 64
// registers and spills 88 to 484 bytes: 4,000 of 32,768 without a residual 129
// us (4.1 TB/s), with one 217 (4.8), in float32 357 (4.4).
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // the smallest normal float: its reciprocal is finite

struct NormArgs {
    const void *x, *residual;
    const void *weight;
    void *out, *residual_out;
    float *scales;
    int64_t x_stride, residual_stride, residual_out_stride, out_stride, rows;
    float eps, inv_scale, inv_width;
    int vecs, groups, residual_type, quant;
};

// Maximum that keeps a NaN (a row or group that holds one gets a NaN scale).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack_f16x2(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return pack_bf16x2(a, b); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) { return pack_f16x2(a, b); }

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}

// Eight e4m3 codes of f * inv, saturating (NaN stays NaN).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE,
                                                    __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
        w[i] = a | b << 16;
    }
    return make_uint2(w[0], w[1]);
}

// amax -> the scale of an e4m3 block: 1 for a block of zeros, never below
// the smallest normal float; NaN stays NaN.
__device__ __forceinline__ float block_scale(float amax) {
    return amax == 0.f ? 1.f : max_nan(__fdiv_rn(amax, kE4m3Max), kMinScale);
}

// Sum (MAX: NaN-keeping maximum) over a row's threads; `warps` of them hold
// the row, starting at warp `warp0` of the block.  With one warp a row no
// barrier is passed, so rows of a block may end at different times.
template <bool MAX, bool ONE_WARP>
__device__ __forceinline__ float row_reduce(float v, float *red, int warps) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? max_nan(v, o) : v + o;
    }
    if (ONE_WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.f;   // maxima are of magnitudes: 0 is neutral for both
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? max_nan(v, o) : v + o;
    }
    return v;
}

// ONE_WARP: blockDim = (32, rows a block), a warp a row; else blockDim.x
// threads, at most MAX, hold one row.  RES: the residual's element size (0:
// none).  A row's loads are issued once the row before is in float32.
template <typename T, int VPT, bool ONE_WARP, int MAX, int RES>
__global__ void __launch_bounds__(MAX) norm_kernel(const NormArgs a) {
    __shared__ float red[3][32];
    const int threads = blockDim.x, tid = threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    constexpr int kParts = RES == 4 ? 2 : 1;        // 16-byte vectors of 8 columns of the residual
    uint4 xv[VPT], rv[VPT][kParts];
    const auto fetch = [&](int64_t row) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride);
        const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.residual) +
                                                         row * a.residual_stride * RES);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) {
                xv[k] = x[v];
                if (RES)
#pragma unroll
                    for (int p = 0; p < kParts; ++p) rv[k][p] = r[kParts * v + p];
            }
        }
    };
    const int64_t row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row0 < a.rows) fetch(row0);
    for (int64_t row = row0; row < a.rows; row += step) {
        float s[VPT][8], ssq = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) {
                unpack8<T>(xv[k], s[k]);
                if (RES == 4) {
                    const uint4 r0 = rv[k][0], r1 = rv[k][kParts - 1];
                    const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[k][i] += __uint_as_float(w[i]);
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.residual_out) +
                                                           row * a.residual_out_stride) + 2 * v;
                    o[0] = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
                    o[1] = make_float4(s[k][4], s[k][5], s[k][6], s[k][7]);
                } else if (RES == 2) {
                    float r[8];
                    unpack8<T>(rv[k][0], r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[k][i] += r[i];
                    reinterpret_cast<uint4 *>(static_cast<T *>(a.residual_out) + row * a.residual_out_stride)[v] =
                        pack8<T>(s[k]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) ssq = fmaf(s[k][i], s[k][i], ssq);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = 0.f;
            }
        }
        if (row + step < a.rows) fetch(row + step);
        ssq = row_reduce<false, ONE_WARP>(ssq, red[0], threads >> 5);
        float rstd = rsqrtf(fmaf(ssq, a.inv_width, a.eps));
        if (ssq == INFINITY) {
            // The squares overflow (or an element is infinite): the same row
            // scaled by 2^-80, beside whose mean square eps is nothing.
            ssq = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[k][i] *= 0x1p-80f;
                    ssq = fmaf(s[k][i], s[k][i], ssq);
                }
            rstd = rsqrtf(row_reduce<false, ONE_WARP>(ssq, red[2], threads >> 5) * a.inv_width);
        }
        const uint4 *w = static_cast<const uint4 *>(a.weight);
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) {
                float wt[8];
                unpack8<T>(__ldg(w + v), wt);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[k][i] = s[k][i] * rstd * wt[i];
                    amax = max_nan(amax, fabsf(s[k][i]));
                }
            }
            if (a.quant == MLA_QUANT_GROUP) {
                // this vector's group: the 16 vectors of a half warp
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                if (v < a.vecs) {
                    const float sc = block_scale(amax);
                    if ((v & 15) == 0) a.scales[row * a.groups + (v >> 4)] = sc;
                    reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.out_stride)[v] =
                        pack8_e4m3(s[k], __fdiv_rn(1.f, sc));
                }
                amax = 0.f;
            }
        }
        if (a.quant == MLA_QUANT_NONE) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * a.out_stride);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * threads;
                if (v < a.vecs) o[v] = pack8<T>(s[k]);
            }
        } else if (a.quant != MLA_QUANT_GROUP) {
            float inv = a.inv_scale;
            if (a.quant == MLA_QUANT_ROW) {
                const float sc = block_scale(row_reduce<true, ONE_WARP>(amax, red[1], threads >> 5));
                if (tid == 0) a.scales[row] = sc;
                inv = __fdiv_rn(1.f, sc);
            }
            uint2 *o = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.out_stride);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * threads;
                if (v < a.vecs) o[v] = pack8_e4m3(s[k], inv);
            }
        }
        if (!ONE_WARP) __syncthreads();   // red is reused by the next row
    }
}

// ------------------------------------------------- many rows: a ring of rows

constexpr int kMaxRing = 4, kMaxBlocks = 16;    // rows in a block's ring, blocks an SM
constexpr int kRingThreads = 512, kRingVpt = 4; // of a block, at most: a row of 16,384 columns
constexpr int kRingBytes = 110 * 1024;      // of shared memory, two blocks an SM

struct RingArgs {
    NormArgs n;
    int x_bytes, row_bytes;     // of a row of x; of x and the residual
    int depth;                  // rows in the ring
};

// blockDim.x threads hold a row, VPT vectors each, weights included; RES:
// the residual's element size (0: none).
template <typename T, int VPT, int RES>
__global__ void __launch_bounds__(kRingThreads, 2) norm_ring_kernel(const RingArgs ra) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][2][32];
    __shared__ __align__(8) uint64_t full[kMaxRing];
    const NormArgs &a = ra.n;
    const int threads = blockDim.x, tid = threadIdx.x, warps = threads >> 5, lane = tid & 31, warp = tid >> 5;
    const int64_t step = gridDim.x;
    const int depth = ra.depth;
    if (tid == 0) {
        for (int s = 0; s < depth; ++s) mbar_init(&full[s], 1);
        mbar_fence_init();
    }
    __syncthreads();
    const auto fetch = [&](int64_t row, int s) {
        uint8_t *dst = ring + s * ra.row_bytes;
        mbar_arrive_expect_tx(&full[s], ra.row_bytes);
        bulk_g2s(dst, static_cast<const T *>(a.x) + row * a.x_stride, ra.x_bytes, &full[s]);
        if (RES)
            bulk_g2s(dst + ra.x_bytes, static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * RES,
                     ra.row_bytes - ra.x_bytes, &full[s]);
    };
    if (tid == 0)
        for (int s = 0; s < depth; ++s)
            if (blockIdx.x + s * step < a.rows) fetch(blockIdx.x + s * step, s);
    uint4 w[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int v = tid + k * threads;
        w[k] = v < a.vecs ? __ldg(static_cast<const uint4 *>(a.weight) + v) : make_uint4(0, 0, 0, 0);
    }
    int it = 0, s = 0, phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += step, ++it) {
        const int buf = it & 1;
        const bool ok = mbar_wait(&full[s], phase);
        const uint4 *xs = reinterpret_cast<const uint4 *>(ring + s * ra.row_bytes);
        const uint4 *rs = reinterpret_cast<const uint4 *>(ring + s * ra.row_bytes + ra.x_bytes);
        float y[VPT][8], ssq = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[k][i] = 0.f;
            if (v < a.vecs) {
                unpack8<T>(xs[v], y[k]);
                if (RES == 4) {
                    const uint4 r0 = rs[2 * v], r1 = rs[2 * v + 1];
                    const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[k][i] += __uint_as_float(r[i]);
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.residual_out) +
                                                           row * a.residual_out_stride) + 2 * v;
                    o[0] = make_float4(y[k][0], y[k][1], y[k][2], y[k][3]);
                    o[1] = make_float4(y[k][4], y[k][5], y[k][6], y[k][7]);
                } else if (RES == 2) {
                    float r[8];
                    unpack8<T>(rs[v], r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[k][i] += r[i];
                    reinterpret_cast<uint4 *>(static_cast<T *>(a.residual_out) + row * a.residual_out_stride)[v] =
                        pack8<T>(y[k]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) ssq = fmaf(y[k][i], y[k][i], ssq);
            }
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
        if (lane == 0) red[buf][0][warp] = ssq;
        if (!__syncthreads_and(ok)) {
            // Flagged.  The rows in flight land before the block ends.
            if (tid == 0)
                for (int k = 0; k < depth; ++k) {
                    if (row + k * step < a.rows) mbar_wait(&full[s], phase);
                    if (++s == depth) s = 0, phase ^= 1;
                }
            return;
        }
        // The row has been read by all: its place takes the row `depth` further on.
        if (tid == 0 && row + depth * step < a.rows) fetch(row + depth * step, s);
        if (++s == depth) s = 0, phase ^= 1;
        ssq = lane < warps ? red[buf][0][lane] : 0.f;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
        float rstd = rsqrtf(fmaf(ssq, a.inv_width, a.eps));
        if (ssq == INFINITY) {      // as in norm_kernel
            ssq = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[k][i] *= 0x1p-80f;
                    ssq = fmaf(y[k][i], y[k][i], ssq);
                }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
            __syncthreads();
            if (lane == 0) red[buf][0][warp] = ssq;
            __syncthreads();
            ssq = lane < warps ? red[buf][0][lane] : 0.f;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
            rstd = rsqrtf(ssq * a.inv_width);
        }
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) {
                float wt[8];
                unpack8<T>(w[k], wt);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[k][i] = y[k][i] * rstd * wt[i];
                    amax = max_nan(amax, fabsf(y[k][i]));
                }
            }
            if (a.quant == MLA_QUANT_NONE) {
                if (v < a.vecs)
                    reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * a.out_stride)[v] = pack8<T>(y[k]);
            } else if (a.quant == MLA_QUANT_GROUP) {
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                if (v < a.vecs) {
                    const float sc = block_scale(amax);
                    if ((v & 15) == 0) a.scales[row * a.groups + (v >> 4)] = sc;
                    reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.out_stride)[v] =
                        pack8_e4m3(y[k], __fdiv_rn(1.f, sc));
                }
                amax = 0.f;
            }
        }
        if (a.quant == MLA_QUANT_ROW || a.quant == MLA_QUANT_STATIC) {
            float inv = a.inv_scale;
            if (a.quant == MLA_QUANT_ROW) {
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                if (lane == 0) red[buf][1][warp] = amax;
                __syncthreads();
                amax = lane < warps ? red[buf][1][lane] : 0.f;
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                const float sc = block_scale(amax);
                if (tid == 0) a.scales[row] = sc;
                inv = __fdiv_rn(1.f, sc);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * threads;
                if (v < a.vecs)
                    reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.out_stride)[v] =
                        pack8_e4m3(y[k], inv);
            }
        }
    }
}

template <typename T, int VPT, int RES>
cudaError_t launch_ring(const RingArgs &ra, int sms, cudaStream_t st) {
    static_assert(VPT <= kRingVpt, "launch's limit");
    const int smem = ra.depth * ra.row_bytes;
    cudaError_t e = smem_attr_once<norm_ring_kernel<T, VPT, RES>>(kRingBytes);
    if (e != cudaSuccess) return e;
    const int threads = ((ra.n.vecs + VPT - 1) / VPT + 31) / 32 * 32;
    // As many blocks as stay resident at 64 registers a thread: narrow rows
    // need many in flight.
    const int per_sm = std::min(std::min(1024 / threads, 2 * kRingBytes / (smem + 2048)), kMaxBlocks);
    const int64_t grid = std::min<int64_t>((int64_t)per_sm * sms, ra.n.rows);
    norm_ring_kernel<T, VPT, RES><<<(unsigned)grid, threads, smem, st>>>(ra);
    return cudaGetLastError();
}

template <typename T, int VPT>
cudaError_t launch_ring_res(const RingArgs &ra, int sms, cudaStream_t st) {
    switch (ra.n.residual_type) {
        case -1: return launch_ring<T, VPT, 0>(ra, sms, st);
        case MLA_TYPE_F32: return launch_ring<T, VPT, 4>(ra, sms, st);
        default: return launch_ring<T, VPT, 2>(ra, sms, st);
    }
}

template <typename T, int RES>
cudaError_t launch_rows(const NormArgs &a, int sms, cudaStream_t st) {
    // A warp holds a row of up to 1,024 columns, one to four vectors a lane;
    // wider rows take a block.
    const int64_t cap = (int64_t)sms * 64;
    if (a.vecs <= 128) {
        const dim3 block(32, 4);
        const unsigned grid = (unsigned)std::min((a.rows + 3) / 4, cap);
        switch ((a.vecs + 31) / 32) {
            case 1: norm_kernel<T, 1, true, 128, RES><<<grid, block, 0, st>>>(a); break;
            case 2: norm_kernel<T, 2, true, 128, RES><<<grid, block, 0, st>>>(a); break;
            case 3: norm_kernel<T, 3, true, 128, RES><<<grid, block, 0, st>>>(a); break;
            default: norm_kernel<T, 4, true, 128, RES><<<grid, block, 0, st>>>(a);
        }
        return cudaGetLastError();
    }
    const int vpt = a.vecs <= 1024 ? 1 : a.vecs <= 2048 ? 2 : 4;
    const int threads = ((a.vecs + vpt - 1) / vpt + 31) / 32 * 32;
    const unsigned grid = (unsigned)std::min(a.rows, cap);
    if (vpt == 1) norm_kernel<T, 1, false, 1024, RES><<<grid, threads, 0, st>>>(a);
    else if (vpt == 2) norm_kernel<T, 2, false, 1024, RES><<<grid, threads, 0, st>>>(a);
    else norm_kernel<T, 4, false, 1024, RES><<<grid, threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const NormArgs &a, int sms, cudaStream_t st) {
    RingArgs ra;
    ra.n = a;
    ra.x_bytes = a.vecs * 16;
    ra.row_bytes = ra.x_bytes * (a.residual_type < 0 ? 1 : a.residual_type == MLA_TYPE_F32 ? 3 : 2);
    ra.depth = std::min(kRingBytes / ra.row_bytes, kMaxRing);
    // The ring takes rows too wide for one warp once every SM has one: 256 rows
    // of 7,168 take 4.0 us with it and 5.7 without, 500 6.2 and 9.4, 16,384 72
    // and 151.  Up to 1,024 columns a warp takes a row, the next row's loads in
    // flight: well ahead of the ring where there are most rows (100,000 x 1,024
    // 70 us against 79, with a residual 119 against 148; 65,536 x 576 39 against
    // 61, 8,192 x 512 4.3 against 5.5), up to a tenth behind it at the widest of
    // these and fewer rows (8,192 x 1,024 8.4 against 8.2, with a residual 14.2
    // against 12.6; 20,000 20.6 against 18.8, and 28.0 against 29.5).  A row
    // that does not fit the ring twice takes the blocks, and so does one of more
    // than 16,384 columns, more than a ring's block holds (without a residual up
    // to 28,160 would fit the ring twice).
    if (a.vecs > 128 && a.vecs <= kRingThreads * kRingVpt && a.rows >= sms && ra.depth >= 2) {
        if (a.vecs <= 512) return launch_ring_res<T, 1>(ra, sms, st);
        if (a.vecs <= 1024) return launch_ring_res<T, 2>(ra, sms, st);
        return launch_ring_res<T, 4>(ra, sms, st);
    }
    switch (a.residual_type) {
        case -1: return launch_rows<T, 0>(a, sms, st);
        case MLA_TYPE_F32: return launch_rows<T, 4>(a, sms, st);
        default: return launch_rows<T, 2>(a, sms, st);
    }
}

}  // namespace

// Arguments checked by mla_add_rms_norm: width a multiple of 8 up to 32,768,
// 16-byte aligned rows.
cudaError_t add_rms_norm_launch(const void *x, int64_t x_stride, int x_type, const void *residual,
                                int64_t residual_stride, int residual_type, const void *weight, float eps,
                                int64_t rows, int width, int quant, float scale, void *out, int64_t out_stride,
                                float *out_scales, void *residual_out, int64_t residual_out_stride, int sms,
                                cudaStream_t st) {
    NormArgs a = {};
    a.x = x;
    a.x_stride = x_stride;
    a.residual = residual;
    a.residual_stride = residual_stride;
    a.residual_type = residual ? residual_type : -1;
    a.weight = weight;
    a.out = out;
    a.out_stride = out_stride;
    a.scales = out_scales;
    a.residual_out = residual_out;
    a.residual_out_stride = residual_out_stride;
    a.rows = rows;
    a.eps = eps;
    a.inv_scale = quant == MLA_QUANT_STATIC ? 1.f / scale : 1.f;
    a.inv_width = 1.f / (float)width;
    a.vecs = width / 8;
    a.groups = (width + 127) / 128;
    a.quant = quant;
    return x_type == MLA_TYPE_BF16 ? launch<__nv_bfloat16>(a, sms, st) : launch<__half>(a, sms, st);
}

cudaError_t norm_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
