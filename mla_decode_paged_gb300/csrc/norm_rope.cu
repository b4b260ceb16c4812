// Norm and position rotation of every head in one pass, with an output in
// 16 or 8 bits, in order or scattered to the rows of a cache.
//
// What it computes, for every row (token t, head h) of `width` columns, in
// float32:
//   y = x[t, h];  y[:n] *= rsqrt(mean(y[:n]^2) + eps) * weight       (n > 0)
//   columns s .. s + d of y rotated by the angles of positions[t]: column
//   pairs (i, i + d / 2) or (2i, 2i + 1) with cosine cos_sin[p, i] and sine
//   cos_sin[p, d / 2 + i]
//   out[t or slots[t], h] = round(y), or e4m3 codes of y / scale with
//   scale = amax / 448 over the row, or given.
//
// Bound by DRAM (4 bytes an element, 3 with an e4m3 output, each moved once)
// for many rows, by launch and the chain position -> table -> store for few.
//
// A group of G lanes holds a row in registers between its loads and its
// stores: lane i has the 8-column vectors i, i + G, ... (16-byte loads).  The
// sum of squares and the maximum are joined by shuffles inside the group, so
// rows pass no barrier.  The other column of a pair is half a rotation away,
// in another lane: its vector is loaded a second time (it is in L1 by then)
// rather than shuffled, which would need a lane and a register picked by the
// span's place.  Pairs of neighbours are inside a vector.
#include <algorithm>

#include <cuda_runtime.h>

#include "common.cuh"
#include "vec8.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const void *x, *weight;
    const int64_t *positions, *slots;
    const float *cos_sin;
    void *out;
    float *scales;
    int64_t x_row, x_head, out_row, out_head, num_positions, out_rows;
    uint32_t rows, heads, magic, shift;     // row / heads = row * magic >> (31 + shift), rows below 2^31
    int vecs, norm_vecs, rope0, rope_vecs, half;    // half: half the rotation's columns
    float eps, inv_norm, inv_scale;
    int quant;
};

// One row a group of G lanes, VPT vectors a lane.  PAIRS: neighbours make a
// pair.
template <typename T, int G, int VPT, bool PAIRS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeArgs a) {
    const int lane = threadIdx.x & 31, in = lane % G;
    constexpr int kPerWarp = 32 / G;
    const uint32_t step = gridDim.x * (kThreads / G);
    // The warp's rows are neighbours and its lanes stay together: a group past the last row holds none.
    const uint32_t first = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kPerWarp;
    const auto token_of = [&](uint32_t row) { return (uint32_t)(((uint64_t)row * a.magic) >> (31 + a.shift)); };
    const auto row_of = [&](uint32_t row, uint32_t t) {
        return static_cast<const uint4 *>(static_cast<const void *>(
            static_cast<const T *>(a.x) + (int64_t)t * a.x_row + (int64_t)(row - t * a.heads) * a.x_head));
    };
    uint4 xv[VPT];
    int64_t pos = 0, slot = 0;
    const auto fetch = [&](uint32_t row) {
        if (row >= a.rows) return;
        const uint32_t t = token_of(row);
        const uint4 *x = row_of(row, t);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (in + k * G < a.vecs) xv[k] = x[in + k * G];
        if (a.positions) pos = __ldg(a.positions + t);
        slot = a.slots ? __ldg(a.slots + t) : (int64_t)t;
    };
    uint4 wv[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        wv[k] = in + k * G < a.norm_vecs ? __ldg(static_cast<const uint4 *>(a.weight) + in + k * G) : make_uint4(0, 0, 0, 0);
    fetch(first + lane / G);
    for (uint32_t row0 = first; row0 < a.rows; row0 += step) {
        const uint32_t row = row0 + lane / G;
        const bool real = row < a.rows;
        const uint32_t t = real ? token_of(row) : 0;
        const uint4 *x = row_of(real ? row : 0, t);
        const int64_t to = slot;
        int64_t p = pos;
        if (a.positions && (p < 0 || p >= a.num_positions)) {
            if (real && in == 0 && to >= 0) flag(MLA_DEV_BAD_POSITION);
            p = 0;
        }
        float y[VPT][8], ssq = 0.f, up = 1.f, rstd = 1.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = in + k * G;
            if (real && v < a.vecs) {
                unpack8<T>(xv[k], y[k]);
                if (v < a.norm_vecs)
#pragma unroll
                    for (int i = 0; i < 8; ++i) ssq = fmaf(y[k][i], y[k][i], ssq);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[k][i] = 0.f;
            }
        }
        fetch(row + step);      // of the next row, on their way meanwhile
        if (a.norm_vecs > 0) {
#pragma unroll
            for (int d = G / 2; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
            rstd = rsqrtf(fmaf(ssq, a.inv_norm, a.eps));
            const bool over = ssq == INFINITY;
            if (__any_sync(0xffffffffu, over)) {
                // The squares overflow (or an element is infinite): the same
                // row scaled by 2^-80, beside whose mean square eps is nothing.
                float small = 0.f;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (in + k * G < a.norm_vecs)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float z = y[k][i] * 0x1p-80f;
                            small = fmaf(z, z, small);
                        }
#pragma unroll
                for (int d = G / 2; d >= 1; d >>= 1) small += __shfl_xor_sync(0xffffffffu, small, d);
                if (over) {
                    up = 0x1p-80f;
                    rstd = rsqrtf(small * a.inv_norm);
                }
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (in + k * G >= a.norm_vecs) continue;
                float w[8];
                unpack8<T>(wv[k], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[k][i] = y[k][i] * up * rstd * w[i];
            }
        }
        if (a.positions) {
            const float *cs = a.cos_sin + p * (2 * a.half);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = in + k * G, j = v - a.rope0;
                if (!real || j < 0 || j >= a.rope_vecs) continue;
                if (PAIRS) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(cs) + j);
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + a.half) + j);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = y[k][2 * i], w = y[k][2 * i + 1];
                        y[k][2 * i] = u * cc[i] - w * ss[i];
                        y[k][2 * i + 1] = w * cc[i] + u * ss[i];
                    }
                } else {
                    const int hv = a.rope_vecs >> 1;        // vectors of half a rotation
                    const bool front = j < hv;
                    const int other = front ? v + hv : v - hv, at = front ? j : j - hv;
                    float o[8];
                    unpack8<T>(x[other], o);
                    if (other < a.norm_vecs) {
                        float w[8];
                        unpack8<T>(__ldg(static_cast<const uint4 *>(a.weight) + other), w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = o[i] * up * rstd * w[i];
                    }
#pragma unroll
                    for (int i4 = 0; i4 < 2; ++i4) {
                        const float4 c = __ldg(reinterpret_cast<const float4 *>(cs) + 2 * at + i4);
                        const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + a.half) + 2 * at + i4);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float turn = o[4 * i4 + i] * ss[i];
                            y[k][4 * i4 + i] = y[k][4 * i4 + i] * cc[i] + (front ? -turn : turn);
                        }
                    }
                }
            }
        }
        // Where the row goes; a negative slot is padding.
        bool write = real && to >= 0;
        if (write && to >= a.out_rows) {
            if (in == 0) flag(MLA_DEV_BAD_PAGE);
            write = false;
        }
        const uint32_t h = real ? row - t * a.heads : 0;
        float inv = a.inv_scale;
        if (a.quant == MLA_QUANT_ROW) {
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(y[k][i]));
#pragma unroll
            for (int d = G / 2; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            const float sc = block_scale(amax);
            if (write && in == 0) a.scales[to * a.heads + h] = sc;
            inv = __fdiv_rn(1.f, sc);
        }
        __syncwarp();       // in place: no lane stores before the others have read their pairs
        if (!write) continue;
        const int64_t at = to * a.out_row + (int64_t)h * a.out_head;
        if (a.quant == MLA_QUANT_NONE) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + at);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (in + k * G < a.vecs) o[in + k * G] = pack8<T>(y[k]);
        } else {
            uint2 *o = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + at);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (in + k * G < a.vecs) o[in + k * G] = pack8_e4m3(y[k], inv);
        }
    }
}

template <typename T, int G, int VPT>
cudaError_t launch(const RopeArgs &a, bool pairs, int sms, cudaStream_t st) {
    const uint32_t per_block = kThreads / G, blocks = (a.rows + per_block - 1) / per_block;
    const unsigned grid = std::min(blocks, (uint32_t)sms * 16);
    if (pairs) norm_rope_kernel<T, G, VPT, true><<<grid, kThreads, 0, st>>>(a);
    else norm_rope_kernel<T, G, VPT, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_width(const RopeArgs &a, bool pairs, int sms, cudaStream_t st) {
    if (a.vecs <= 8) return launch<T, 8, 1>(a, pairs, sms, st);
    if (a.vecs <= 16) return launch<T, 8, 2>(a, pairs, sms, st);
    if (a.vecs <= 24) return launch<T, 8, 3>(a, pairs, sms, st);
    if (a.vecs <= 32) return launch<T, 16, 2>(a, pairs, sms, st);
    if (a.vecs <= 48) return launch<T, 16, 3>(a, pairs, sms, st);
    if (a.vecs <= 64) return launch<T, 32, 2>(a, pairs, sms, st);
    if (a.vecs <= 96) return launch<T, 32, 3>(a, pairs, sms, st);
    return launch<T, 32, 4>(a, pairs, sms, st);
}

}  // namespace

// Arguments checked by mla_norm_rope: width, norm_dim and rope_start
// multiples of 8, rope_dim of 16, width up to 1,024, 16-byte aligned rows.
cudaError_t norm_rope_launch(const void *x, int64_t x_row, int64_t x_head, int x_type, const void *weight, int norm_dim,
                             float eps, const int64_t *positions, const float *cos_sin, int64_t num_positions,
                             int rope_start, int rope_dim, bool pairs, int64_t tokens, int heads, int width, int quant,
                             float scale, const int64_t *slots, int64_t out_rows, void *out, int64_t out_row,
                             int64_t out_head, float *out_scales, int sms, cudaStream_t st) {
    RopeArgs a = {};
    a.x = x;
    a.x_row = x_row;
    a.x_head = x_head;
    a.weight = weight;
    a.positions = positions;
    a.slots = slots;
    a.cos_sin = cos_sin;
    a.out = out;
    a.scales = out_scales;
    a.out_row = out_row;
    a.out_head = out_head;
    a.num_positions = num_positions;
    a.out_rows = out_rows;
    a.rows = (uint32_t)(tokens * heads);
    a.heads = (uint32_t)heads;
    while ((1u << a.shift) < a.heads) ++a.shift;        // magic: 2^(31 + shift) / heads, up to 2^32 - 1
    a.magic = (uint32_t)(((1ull << (31 + a.shift)) + a.heads - 1) / a.heads);
    a.vecs = width / 8;
    a.norm_vecs = weight ? norm_dim / 8 : 0;
    a.rope0 = rope_start / 8;
    a.rope_vecs = rope_dim / 8;
    a.half = rope_dim / 2;
    a.eps = eps;
    a.inv_norm = weight ? 1.f / (float)norm_dim : 0.f;
    a.inv_scale = quant == MLA_QUANT_STATIC ? 1.f / scale : 1.f;
    a.quant = quant;
    return x_type == MLA_TYPE_BF16 ? launch_width<__nv_bfloat16>(a, pairs, sms, st)
                                   : launch_width<__half>(a, pairs, sms, st);
}

cudaError_t norm_rope_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
