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
// for many rows, by launch and the chain position -> table -> store for few:
// 4,096 tokens x 96 heads of 192 columns 45.6 us (6.6 TB/s), 16,384 rows of
// 576 columns normed, rotated, quantized and scattered 8.3 to 9.4 (3.9 TB/s
// with three caches in turn, 3.5 with four, which L2 does not hold), 64 x 64
// heads of 128 to codes with a scale a row 1.8.
//
// A group of G lanes holds a row in registers between its loads and its
// stores: 8-column vectors (16-byte loads, for wide rows by way of shared
// memory, the next row's on their way meanwhile), dealt to the lanes so that the
// two halves of a rotated pair lie in one lane (with partners loaded a second
// time the 96 heads took 68 us).  The sum of squares and the maximum are
// joined by shuffles inside the group, so rows pass no barrier; the arithmetic
// takes two columns an instruction, without which the 96 heads are bound by
// issue.  Weights are in shared memory.  Codes are those of products with the
// scale's reciprocal, one rounding beside those of y itself; but where columns
// of x come through as they are and the scale is given, those of the quotient,
// as kv_append writes them to the same rows (two multiply-adds and a clamp more
// an element: 16,384 x 64 rotated heads of 128 83 us and not 71).
#include <algorithm>

#include <cuda_runtime.h>

#include "common.cuh"
#include "vec8.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
// Blocks an SM holds, by what their registers allow (40 to 128 a thread):
// where one more of them would spill, rows in flight are worth less (16,384
// rows of 576 columns, 5 vectors a lane: 9.4 us with three blocks, 11.2 with
// four, which spill).
constexpr int blocks_per_sm(int vpt, bool head, bool pairs) {
    return vpt <= 2 ? (head && pairs ? 6 : 4) : vpt == 3 ? 4 : vpt <= 5 ? (head ? 2 : 3) : 2;
}

// Rows (one a group) a warp has on their way or in work through shared memory;
// 0: through registers.  Where a row takes most of the registers the next
// one's loads would otherwise wait for its stores (65,536 rows of 576 columns
// 25.5 us and not 27.8, 16,384 of 1,024 12.1 and 13.4; three rows 26.6 and 12.7;
// with 5 vectors a lane no gain, and 4,096 rows 3.3 us and not 3.1).
constexpr int deep(int vpt) { return vpt >= 8 ? 2 : 0; }

// Whether these lanes may form quotients (16,384 rows of 576 columns, none its
// own, 8.2 us; where 9 vectors a lane had the code too, 9.3).
constexpr bool exact(int vpt) { return vpt <= 5; }

struct RopeArgs {
    const void *x, *weight;
    const int64_t *positions, *slots;
    const float *cos_sin;
    void *out;
    float *scales;
    int64_t num_positions, out_rows;
    uint32_t x_row, x_head, out_row, out_head;      // strides, at most 2^30
    uint32_t rows, heads, magic, shift;     // row / heads = row * magic >> (31 + shift), rows below 2^31
    int vecs, norm_vecs, rope0, rope_vecs, half;    // half: half the rotation's columns
    int turns;              // pairs of a lane's places that hold halves of the rotation
    float eps, inv_norm, scale, inv_scale;
    int quant;
    bool exact;             // a given scale divides, as some columns are x's own
};

// Eight columns as four pairs.
struct Vec {
    uint64_t p[4];
};
template <typename T>
__device__ __forceinline__ Vec unpack(const uint4 &raw) {
    float f[8];
    unpack8<T>(raw, f);
    return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
__device__ __forceinline__ Vec load8(const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}
__device__ __forceinline__ void spread(const Vec &v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = parts(v.p[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

// Four e4m3 codes of two pairs.
__device__ __forceinline__ uint32_t codes(uint64_t a, uint64_t b) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(parts(a), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(parts(b), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
template <typename T>
__device__ __forceinline__ uint32_t round2(uint64_t v) {
    const float2 f = parts(v);
    return pack2<T>(f.x, f.y);
}

// One row a group of G lanes, VPT vectors a lane.  NORM: with a weight.
// PAIRS: neighbours make a pair.  HEAD: a scale a row, so its values are held
// until all of them are known.
template <typename T, int G, int VPT, bool NORM, bool PAIRS, bool HEAD>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(VPT, HEAD, PAIRS)) norm_rope_kernel(const RopeArgs a) {
    __shared__ uint4 weight[NORM ? MLA_MAX_ROPE_WIDTH / 8 : 1];
    const int lane = threadIdx.x & 31, in = lane % G;
    constexpr int kPerWarp = 32 / G;
    // The next row's loads beside this one's work.  (With a scale a row only
    // where halves make the work long: 16,384 x 64 heads of 128 82 us and not
    // 87, in pairs 78 and not 76, with six blocks an SM in its place.)
    constexpr bool kAhead = deep(VPT) == 0 && G < 32 && VPT <= (PAIRS ? 4 : 2) && !(HEAD && PAIRS);
    const uint32_t step = gridDim.x * (kThreads / G);
    // The warp's rows are neighbours and its lanes stay together: a group past
    // the last row repeats it and stores nothing.
    const uint32_t first = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kPerWarp;
    // This lane's vectors, and a bit each: it has one, it is normed, it is
    // rotated.  Halves: the first 2 * a.turns places of a lane hold the two
    // vectors of its pairs, front and back, or in lanes past the pairs others.
    int vec[VPT];
    uint32_t mine = 0, normed = 0, turned = 0;
    const int half_vecs = a.rope_vecs >> 1, spare = a.turns * G - half_vecs;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        int v = in + k * G;
        if (PAIRS) {
            if (v >= a.rope0 && v < a.rope0 + a.rope_vecs) turned |= 1u << k;
        } else {
            const int u = in + (k >> 1) * G;        // of this place's pair
            if (k < 2 * a.turns && u < half_vecs) {
                v = a.rope0 + u + (k & 1) * half_vecs;
                turned |= 1u << k;
            } else {
                v = k < 2 * a.turns ? in - (G - spare) + (k & 1) * spare : 2 * spare + (k - 2 * a.turns) * G + in;
                if (v >= a.rope0) v += a.rope_vecs;
            }
        }
        if (v < a.vecs) mine |= 1u << k;
        if (NORM && v < a.norm_vecs) normed |= 1u << k;
        vec[k] = v;
    }
    constexpr int kDeep = deep(VPT);
    extern __shared__ uint4 ring[];
    uint4 *at_ring = ring + (threadIdx.x >> 5) * (kDeep * VPT * 32) + lane;
    uint4 next[kDeep ? 1 : VPT];
    int64_t pos = 0, slot = 0;
    uint32_t head;
    const auto fetch = [&](uint32_t row) {
        row = min(row, a.rows - 1);
        const uint32_t t = (uint32_t)(((uint64_t)row * a.magic) >> (31 + a.shift));
        head = row - t * a.heads;
        if (kDeep) {
            if (a.positions) pos = a.positions[t];
            slot = a.slots ? a.slots[t] : (int64_t)t;
            return;
        }
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) +
                                                         ((uint64_t)t * a.x_row + (uint64_t)head * a.x_head));
#pragma unroll
        for (int k = 0; k < VPT; ++k) next[kDeep ? 0 : k] = (mine >> k & 1) ? x[vec[k]] : make_uint4(0, 0, 0, 0);
        // (After x: 16,384 x 64 heads of 128 81 us, before it 83.)
        if (a.positions) pos = a.positions[t];
        slot = a.slots ? a.slots[t] : (int64_t)t;
    };
    // Into the ring: every lane its own vectors, which it alone reads.
    const auto copy = [&](uint32_t row0, int stage) {
        if (row0 < a.rows) {
            const uint32_t row = min(row0 + lane / G, a.rows - 1);
            const uint32_t t = (uint32_t)(((uint64_t)row * a.magic) >> (31 + a.shift));
            const uint4 *x = reinterpret_cast<const uint4 *>(
                static_cast<const T *>(a.x) + ((uint64_t)t * a.x_row + (uint64_t)(row - t * a.heads) * a.x_head));
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (mine >> k & 1) cp_async16(at_ring + (stage * VPT + k) * 32, x + vec[k]);
        }
        cp_async_commit();
    };
    grid_wait();
    if (kAhead) fetch(first + lane / G);
    if (kDeep) {
        fetch(first + lane / G);
#pragma unroll
        for (int i = 0; i + 1 < kDeep; ++i) copy(first + i * step, i);
    }
    int stage = 0;
    if (NORM) {
        for (int i = threadIdx.x; i < a.norm_vecs; i += kThreads) weight[i] = static_cast<const uint4 *>(a.weight)[i];
        __syncthreads();
    }
    for (uint32_t row0 = first; row0 < a.rows; row0 += step) {
        const uint32_t row = row0 + lane / G;
        if (!kAhead && !kDeep) fetch(row);
        const uint32_t h = head;
        // Where the row goes; a negative slot is padding.
        const int64_t to = slot;
        bool write = row < a.rows;
        if (a.slots) {
            if (write && to >= a.out_rows && in == 0) flag(MLA_DEV_BAD_PAGE);
            write = write && to >= 0 && to < a.out_rows;
        }
        const float *cs = a.cos_sin;
        if (a.positions) {
            const bool bad = (uint64_t)pos >= (uint64_t)a.num_positions;
            if (bad && to >= 0 && in == 0) flag(MLA_DEV_BAD_POSITION);
            cs += bad ? 0 : pos * (2 * a.half);
        }
        uint4 xv[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) xv[k] = next[kDeep ? 0 : k];
        if (kAhead) fetch(row + step);
        if (kDeep) {
            // The place of the row before, whose values have been used, takes the row kDeep - 1 ahead.
            copy(row0 + (kDeep - 1) * step, stage == 0 ? kDeep - 1 : stage - 1);
            fetch(row + step);
            cp_async_wait<kDeep ? kDeep - 1 : 0>();
#pragma unroll
            for (int k = 0; k < VPT; ++k) xv[k] = (mine >> k & 1) ? at_ring[(stage * VPT + k) * 32] : make_uint4(0, 0, 0, 0);
            stage = stage == kDeep - 1 ? 0 : stage + 1;
        }
        float rstd = 1.f;
        if (NORM) {
            uint64_t sums[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const Vec y = unpack<T>(xv[k]);
                if (normed >> k & 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sums[i & 1] = fma2(y.p[i], y.p[i], sums[i & 1]);
            }
            const float2 s0 = parts(sums[0]), s1 = parts(sums[1]);
            float ssq = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
            for (int d = G / 2; d >= 1; d >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, d);
            rstd = rsqrtf(fmaf(ssq, a.inv_norm, a.eps));
            if (__any_sync(0xffffffffu, ssq == INFINITY)) {
                // The squares overflow (or an element is infinite): the sum of
                // the row scaled by 2^-80, beside whose mean eps is nothing.
                // (The factor may be subnormal, down to 2^-128: 2^-22 off.)
                float small = 0.f;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (!(normed >> k & 1)) continue;
                    float y[8];
                    unpack8<T>(xv[k], y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) small = fmaf(y[i] * 0x1p-80f, y[i] * 0x1p-80f, small);
                }
#pragma unroll
                for (int d = G / 2; d >= 1; d >>= 1) small += __shfl_xor_sync(0xffffffffu, small, d);
                if (ssq == INFINITY) rstd = rsqrtf(small * a.inv_norm) * 0x1p-80f;
            }
        }
        const uint64_t rstd2 = pair(rstd, rstd);
        // Vector k of this lane, normed; with PAIRS rotated too.
        const auto value = [&](int k) {
            Vec y = unpack<T>(xv[k]);
            if (NORM && (normed >> k & 1)) {
                const Vec f = unpack<T>(weight[vec[k]]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y.p[i] = mul2(mul2(y.p[i], rstd2), f.p[i]);
            }
            if (PAIRS && (turned >> k & 1)) {
                const float *at = cs + 4 * (vec[k] - a.rope0);
                const float4 c = *reinterpret_cast<const float4 *>(at);
                const float4 s = *reinterpret_cast<const float4 *>(at + a.half);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = parts(y.p[i]);
                    y.p[i] = pair(u.x * cc[i] - u.y * ss[i], u.y * cc[i] + u.x * ss[i]);
                }
            }
            return y;
        };
        // The vectors of places k and k + 1, halves of the same pairs, rotated.
        const auto rotate = [&](Vec &u, Vec &v, int k) {
            const float *at = cs + 8 * (vec[k] - a.rope0);
            const Vec c = load8(at), s = load8(at + a.half);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t w = fma2(v.p[i] ^ 0x8000000080000000ull, s.p[i], mul2(u.p[i], c.p[i]));
                v.p[i] = fma2(u.p[i], s.p[i], mul2(v.p[i], c.p[i]));
                u.p[i] = w;
            }
        };
        // use(k, its value) for every place; pairs of neighbours from the last
        // one, so that a rotation at the heads' end has its cosines loaded before
        // the row's stores (4,096 x 96 heads 45.6 us, from the first 47.5).
        const auto each = [&](auto use) {
#pragma unroll
            for (int i = 0; i < VPT; i += PAIRS ? 1 : 2) {
                const int k = PAIRS ? VPT - 1 - i : i;
                Vec u = value(k);
                if (PAIRS || k + 1 == VPT) {
                    use(k, u);
                } else {
                    Vec v = value(k + 1 < VPT ? k + 1 : k);
                    if (turned >> k & 1) rotate(u, v, k);
                    use(k, u);
                    use(k + 1, v);
                }
            }
        };
        const uint64_t at = (uint64_t)to * a.out_row + (uint64_t)h * a.out_head;
        if (!HEAD && a.quant == MLA_QUANT_NONE) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + at);
            each([&](int k, const Vec &v) {
                const uint4 y = make_uint4(round2<T>(v.p[0]), round2<T>(v.p[1]), round2<T>(v.p[2]), round2<T>(v.p[3]));
                if (write && (mine >> k & 1)) o[vec[k]] = y;
            });
            continue;
        }
        uint2 *o = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + at);
        const auto store = [&](int k, uint64_t q0, uint64_t q1, uint64_t q2, uint64_t q3) {
            const uint2 q = make_uint2(codes(q0, q1), codes(q2, q3));
            if (write && (mine >> k & 1)) o[vec[k]] = q;
        };
        const auto store_product = [&](int k, const Vec &v, float inv) {
            const uint64_t f = pair(inv, inv);
            store(k, mul2(v.p[0], f), mul2(v.p[1], f), mul2(v.p[2], f), mul2(v.p[3], f));
        };
        if (HEAD) {
            Vec held[HEAD ? VPT : 1];
            float amax = 0.f;
            each([&](int k, const Vec &v) {
                held[HEAD ? k : 0] = v;
                float y[8];
                spread(v, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(y[i]));
            });
#pragma unroll
            for (int d = G / 2; d >= 1; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            const float sc = block_scale(amax), inv = __fdiv_rn(1.f, sc);
            if (write && in == 0) a.scales[(uint64_t)to * a.heads + h] = sc;
#pragma unroll
            for (int k = 0; k < VPT; ++k) store_product(k, held[HEAD ? k : 0], inv);
        } else if (exact(VPT) && a.exact) {
            const Divisor d = divisor_of(a.scale);
            each([&](int k, const Vec &v) { store(k, quotient2(v.p[0], d), quotient2(v.p[1], d), quotient2(v.p[2], d), quotient2(v.p[3], d)); });
        } else {
            each([&](int k, const Vec &v) { store_product(k, v, a.inv_scale); });
        }
    }
}

template <typename T, int G, int VPT, bool NORM, bool PAIRS, bool HEAD>
cudaError_t launch_kernel(RopeArgs a, int sms, cudaStream_t st) {
    a.turns = PAIRS ? 0 : (a.rope_vecs / 2 + G - 1) / G;
    const uint32_t per_block = kThreads / G, blocks = (a.rows + per_block - 1) / per_block;
    constexpr int smem = deep(VPT) * VPT * kThreads * 16;
    if (smem > 0) {
        cudaError_t e = smem_attr_once<norm_rope_kernel<T, G, VPT, NORM, PAIRS, HEAD>>(smem);
        if (e != cudaSuccess) return e;
    }
    return launch_early(norm_rope_kernel<T, G, VPT, NORM, PAIRS, HEAD>,
                        std::min(blocks, (uint32_t)sms * blocks_per_sm(VPT, HEAD, PAIRS)), kThreads, smem, st, a);
}

template <typename T, int G, int VPT>
cudaError_t launch(const RopeArgs &a, bool pairs, int sms, cudaStream_t st) {
    const bool head = a.quant == MLA_QUANT_ROW;
    if (a.weight) {
        if (pairs) return head ? launch_kernel<T, G, VPT, true, true, true>(a, sms, st) : launch_kernel<T, G, VPT, true, true, false>(a, sms, st);
        return head ? launch_kernel<T, G, VPT, true, false, true>(a, sms, st) : launch_kernel<T, G, VPT, true, false, false>(a, sms, st);
    }
    if (pairs) return head ? launch_kernel<T, G, VPT, false, true, true>(a, sms, st) : launch_kernel<T, G, VPT, false, true, false>(a, sms, st);
    return head ? launch_kernel<T, G, VPT, false, false, true>(a, sms, st) : launch_kernel<T, G, VPT, false, false, false>(a, sms, st);
}

template <typename T>
cudaError_t launch_width(const RopeArgs &a, bool pairs, int sms, cudaStream_t st) {
    // The fewest lanes that hold a row in few registers and, with halves, both
    // of a pair in one lane.  Rows of 384 columns and more that leave the SMs
    // idle take a warp each, very many of them 8 lanes (us, of 576 columns to
    // codes in a cache's rows, by a warp, 16 lanes and 8: 64 rows 2.3, 2.7, 3.4;
    // 1,024 2.4, 2.8, 3.4; 4,096 3.4, 3.3, 3.6; 8,192 5.3, 5.0, 4.5; 10,000
    // 5.9, 5.6, 6.2; 12,288 7.2, 6.4, 6.6; 16,384 10.2, 9.4, 8.3; 65,536 48, 34,
    // 25: whole turns of the grid make the steps).
    const auto fits = [&](int g, int vpt) { return a.vecs <= g * vpt && (pairs || 2 * ((a.rope_vecs / 2 + g - 1) / g) <= vpt); };
    if (fits(4, 2)) return launch<T, 4, 2>(a, pairs, sms, st);
    if (fits(8, 2)) return launch<T, 8, 2>(a, pairs, sms, st);
    if (fits(8, 3)) return launch<T, 8, 3>(a, pairs, sms, st);
    if (fits(8, 4)) return launch<T, 8, 4>(a, pairs, sms, st);
    if (fits(16, 3)) return launch<T, 16, 3>(a, pairs, sms, st);
    if (a.rows < 16 * (uint32_t)sms && fits(32, 3)) return launch<T, 32, 3>(a, pairs, sms, st);
    if (a.rows < 16 * (uint32_t)sms && fits(32, 4)) return launch<T, 32, 4>(a, pairs, sms, st);
    if (a.rows >= 64 * (uint32_t)sms && fits(8, 9) && !a.exact) return launch<T, 8, 9>(a, pairs, sms, st);
    if (fits(16, 5)) return launch<T, 16, 5>(a, pairs, sms, st);
    if (a.exact) return launch<T, 32, 4>(a, pairs, sms, st);
    return launch<T, 16, 8>(a, pairs, sms, st);
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
    a.x_row = (uint32_t)x_row;
    a.x_head = (uint32_t)x_head;
    a.weight = weight;
    a.positions = positions;
    a.slots = slots;
    a.cos_sin = cos_sin;
    a.out = out;
    a.scales = out_scales;
    a.out_row = (uint32_t)out_row;
    a.out_head = (uint32_t)out_head;
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
    a.scale = quant == MLA_QUANT_STATIC ? scale : 1.f;
    a.inv_scale = 1.f / a.scale;
    const int norm_end = 8 * a.norm_vecs, rope_end = rope_start + rope_dim;
    a.exact = quant == MLA_QUANT_STATIC && !(norm_end >= width || (rope_end >= width && norm_end >= rope_start));
    a.quant = quant;
    return x_type == MLA_TYPE_BF16 ? launch_width<__nv_bfloat16>(a, pairs, sms, st)
                                   : launch_width<__half>(a, pairs, sms, st);
}

cudaError_t norm_rope_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
