// Attention weight received by each cached token in one decode step.
//
// What it computes, for token j of request r at entry i = indptr[r] + j of
// the page list:
//   out[i] = decay * weights[i] + sum_{t, h} exp(sc * <q[t, h], K_j> - lse[t, h])
// over r's query rows t that see token j and heads h with lse[t, h] > -inf,
// K_j the e4m3 cache row of pages[i] and sc = scale * q_scale * kv_scale.
//
// One warp per token: a lane holds 18 of the row's 576 values, the products
// are summed by shuffles, row by row.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPairs = MLA_D_QK / 64;   // 9 column pairs a lane

struct TokenArgs {
    const void *q;
    int64_t q_row_stride, pool_rows, num_pages;
    const uint8_t *kv;
    const int32_t *pages, *indptr;
    const float *lse, *weights;
    float *out;
    int R, qlen, heads, causal, q8;
    float sc, decay;
};

__device__ __forceinline__ float2 e4m3_pair(uint16_t v) { return unpack_f16x2(e4m3x2_to_f16x2(v)); }

__global__ void __launch_bounds__(kThreads) token_weights_kernel(const TokenArgs a) {
    const int r = blockIdx.x, lane = threadIdx.x & 31;
    int base;
    const int len = request_len(a.indptr, r, a.num_pages, &base);
    for (int j = blockIdx.y * kWarps + (threadIdx.x >> 5); j < len; j += gridDim.y * kWarps) {
        const int64_t i = (int64_t)base + j;
        const uint16_t *k = reinterpret_cast<const uint16_t *>(kv_row(a.kv, a.pages, i, a.pool_rows));
        float2 kf[kPairs];
#pragma unroll
        for (int c = 0; c < kPairs; ++c) kf[c] = e4m3_pair(__ldg(k + lane + 32 * c));
        float sum = 0.f;
        for (int t = 0; t < a.qlen; ++t) {
            if (a.causal && j >= len - a.qlen + t + 1) continue;
            const int64_t row = (int64_t)r * a.qlen + t;
            for (int h = 0; h < a.heads; ++h) {
                const float lse = __ldg(a.lse + row * a.heads + h);
                if (lse == -INFINITY) continue;
                float dot = 0.f;
                if (a.q8) {
                    const uint16_t *q = reinterpret_cast<const uint16_t *>(
                        static_cast<const uint8_t *>(a.q) + row * a.q_row_stride + h * MLA_D_QK);
#pragma unroll
                    for (int c = 0; c < kPairs; ++c) {
                        const float2 v = e4m3_pair(__ldg(q + lane + 32 * c));
                        dot = fmaf(v.x, kf[c].x, fmaf(v.y, kf[c].y, dot));
                    }
                } else {
                    const uint32_t *q = reinterpret_cast<const uint32_t *>(
                        static_cast<const __nv_bfloat16 *>(a.q) + row * a.q_row_stride + h * MLA_D_QK);
#pragma unroll
                    for (int c = 0; c < kPairs; ++c) {
                        const uint32_t v = __ldg(q + lane + 32 * c);
                        dot = fmaf(bf16_lo(v), kf[c].x, fmaf(bf16_hi(v), kf[c].y, dot));
                    }
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                sum += expf(fmaf(dot, a.sc, -lse));
            }
        }
        if (lane == 0) a.out[i] = a.decay == 0.f ? sum : fmaf(a.decay, a.weights[i], sum);
    }
}

}  // namespace

cudaError_t token_weights_launch(const void *q, int64_t q_row_stride, const void *kv, int64_t pool_rows,
                                 const int32_t *pages, int64_t num_pages, const int32_t *indptr, int R, int qlen,
                                 int heads, float sc, const float *lse, float decay, const float *weights, float *out,
                                 bool causal, bool q8, int sms, cudaStream_t st) {
    TokenArgs a = {};
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.kv = static_cast<const uint8_t *>(kv);
    a.pool_rows = pool_rows;
    a.pages = pages;
    a.num_pages = num_pages;
    a.indptr = indptr;
    a.R = R;
    a.qlen = qlen;
    a.heads = heads;
    a.sc = sc;
    a.lse = lse;
    a.decay = decay;
    a.weights = weights;
    a.out = out;
    a.causal = causal;
    a.q8 = q8;
    const int chunks = (sms * 8 + R - 1) / R;
    token_weights_kernel<<<dim3(R, chunks < 65535 ? chunks : 65535), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t token_weights_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
