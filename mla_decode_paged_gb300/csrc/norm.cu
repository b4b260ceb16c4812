// Residual addition, root-mean-square norm and output in 16 or 8 bits.
//
// What it computes, for every row t of `width` columns, in float32:
//   s = x[t] + residual[t];  residual_out[t] = round(s)
//   y = s * rsqrt(mean(s^2) + eps) * weight
//   out[t] = round(y), or e4m3 codes of y / scale with scale = amax / 448
//   over the row, over each 128 columns, or one given number.
//
// Bound by DRAM: 7 bytes per element with a bf16 residual and an e4m3
// output, each read or written once.  A row stays in registers between its
// loads and its stores: thread i of the row's T threads holds the 8-column
// vectors i, i + T, ... (16-byte loads, coalesced; VPT vectors a thread, all
// loads issued before the first use), the sum of squares (and a row's
// maximum) is joined by shuffles and, where more than one warp holds the
// row, through shared memory.  128 columns are 16 consecutive vectors, so a
// group's maximum stays inside a half warp (T is a multiple of 16).
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
// threads hold one row.
template <typename T, int VPT, bool ONE_WARP>
__global__ void __launch_bounds__(ONE_WARP ? 256 : 1024) norm_kernel(const NormArgs a) {
    __shared__ float red[3][32];
    const int threads = blockDim.x, tid = threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.rows; row += step) {
        float s[VPT][8];
        uint4 xv[VPT], rv[VPT], rw[VPT];
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) xv[k] = x[v];
        }
        if (a.residual_type == MLA_TYPE_F32) {
            const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.residual) + row * a.residual_stride);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * threads;
                if (v < a.vecs) {
                    rv[k] = r[2 * v];
                    rw[k] = r[2 * v + 1];
                }
            }
        } else if (a.residual) {
            const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.residual) + row * a.residual_stride);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * threads;
                if (v < a.vecs) rv[k] = r[v];
            }
        }
        float ssq = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = tid + k * threads;
            if (v < a.vecs) {
                unpack8<T>(xv[k], s[k]);
                if (a.residual_type == MLA_TYPE_F32) {
                    const uint32_t w[8] = {rv[k].x, rv[k].y, rv[k].z, rv[k].w, rw[k].x, rw[k].y, rw[k].z, rw[k].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[k][i] += __uint_as_float(w[i]);
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.residual_out) +
                                                           row * a.residual_out_stride) + 2 * v;
                    o[0] = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
                    o[1] = make_float4(s[k][4], s[k][5], s[k][6], s[k][7]);
                } else if (a.residual) {
                    float r[8];
                    unpack8<T>(rv[k], r);
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

template <typename T>
cudaError_t launch(const NormArgs &a, int sms, cudaStream_t st) {
    // Up to 256 columns a warp holds a row in one vector a lane, up to 1,024
    // in two or four; wider rows take a block of up to 1,024 threads.
    const int64_t cap = (int64_t)sms * 64;
    if (a.vecs <= 128) {
        const int vpt = a.vecs <= 32 ? 1 : a.vecs <= 64 ? 2 : 4;
        const dim3 block(32, 4);
        const int64_t need = (a.rows + 3) / 4;
        const unsigned grid = (unsigned)(need < cap ? need : cap);
        if (vpt == 1) norm_kernel<T, 1, true><<<grid, block, 0, st>>>(a);
        else if (vpt == 2) norm_kernel<T, 2, true><<<grid, block, 0, st>>>(a);
        else norm_kernel<T, 4, true><<<grid, block, 0, st>>>(a);
        return cudaGetLastError();
    }
    const int vpt = a.vecs <= 1024 && a.rows <= 2 * (int64_t)sms ? 1 : a.vecs <= 512 ? 2 : 4;
    const int threads = (((a.vecs + vpt - 1) / vpt) + 31) / 32 * 32;
    const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
    if (vpt == 1) norm_kernel<T, 1, false><<<grid, threads, 0, st>>>(a);
    else if (vpt == 2) norm_kernel<T, 2, false><<<grid, threads, 0, st>>>(a);
    else norm_kernel<T, 4, false><<<grid, threads, 0, st>>>(a);
    return cudaGetLastError();
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

}  // namespace mla
