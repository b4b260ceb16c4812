// W_UV projection and sigmoid gate with one low-rank adapter per request.
//
// What it computes, for row t (request r = t / qlen), head h, output v, with
// a = adapters[r] (-1: no adapter):
//   val = sum_c latent[t, h, c] w_uv[h, v, c]
//         + lora_scale[a] * sum_k (sum_c latent[t, h, c] A[a, k, c]) B[a, h, v, k]
//   out[t, h*128 + v] = lengths[r] > 0 ? bf16(val * sigmoid(gate)) : 0
//
// One block per (row, head), a thread an output column.
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {
namespace {

struct LoraArgs {
    const __nv_bfloat16 *latent, *w_uv, *gate, *a, *b;
    const int32_t *lengths, *adapters;
    const float *scale;
    __nv_bfloat16 *out;
    int S, qlen, H, rank, n;
};

__device__ __forceinline__ float sigmoid_f32(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x)));
    return r;
}

__global__ void __launch_bounds__(MLA_D_V) value_lora_kernel(const LoraArgs p) {
    __shared__ float x[MLA_D_LATENT], t[MLA_MAX_LORA_RANK];
    const int v = threadIdx.x, h = blockIdx.y, row = blockIdx.x;
    const int r = row / p.qlen;
    const int64_t rh = (int64_t)row * p.H + h;
    int a = __ldg(p.adapters + r);
    if (a < -1 || a >= p.n) {
        flag(MLA_DEV_BAD_ADAPTER);
        a = -1;
    }
    for (int c = v; c < MLA_D_LATENT; c += MLA_D_V) x[c] = __bfloat162float(p.latent[rh * MLA_D_LATENT + c]);
    __syncthreads();
    float val = 0.f;
    const __nv_bfloat16 *w = p.w_uv + ((int64_t)h * MLA_D_V + v) * MLA_D_LATENT;
    for (int c = 0; c < MLA_D_LATENT; ++c) val = fmaf(x[c], __bfloat162float(w[c]), val);
    if (a >= 0) {
        if (v < p.rank) {
            const __nv_bfloat16 *ak = p.a + ((int64_t)a * p.rank + v) * MLA_D_LATENT;
            float s = 0.f;
            for (int c = 0; c < MLA_D_LATENT; ++c) s = fmaf(x[c], __bfloat162float(ak[c]), s);
            t[v] = s * __ldg(p.scale + a);
        }
        __syncthreads();
        const __nv_bfloat16 *b = p.b + (((int64_t)a * p.H + h) * MLA_D_V + v) * p.rank;
        float s = 0.f;
        for (int k = 0; k < p.rank; ++k) s = fmaf(t[k], __bfloat162float(b[k]), s);
        val += s;
    }
    const bool live = __ldg(p.lengths + r) > 0;
    const float g = __bfloat162float(p.gate[rh * MLA_D_V + v]);
    p.out[rh * MLA_D_V + v] = __float2bfloat16_rn(live ? val * sigmoid_f32(g) : 0.f);
}

}  // namespace

int64_t value_lora_workspace(int64_t, int, int) { return 0; }

cudaError_t value_lora_launch(const void *latent, const void *w_uv, const void *gate, const int32_t *lengths,
                              const void *lora_a, const void *lora_b, const int32_t *adapters, const float *lora_scale,
                              int num_adapters, int rank, int R, int qlen, int H, void *out, void *, int,
                              cudaStream_t st) {
    LoraArgs p = {};
    p.latent = static_cast<const __nv_bfloat16 *>(latent);
    p.w_uv = static_cast<const __nv_bfloat16 *>(w_uv);
    p.gate = static_cast<const __nv_bfloat16 *>(gate);
    p.a = static_cast<const __nv_bfloat16 *>(lora_a);
    p.b = static_cast<const __nv_bfloat16 *>(lora_b);
    p.lengths = lengths;
    p.adapters = adapters;
    p.scale = lora_scale;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.S = R * qlen;
    p.qlen = qlen;
    p.H = H;
    p.rank = rank;
    p.n = num_adapters;
    value_lora_kernel<<<dim3(p.S, H), MLA_D_V, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t value_lora_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
