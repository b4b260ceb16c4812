// The query that attend takes: W_UK absorbed into its first 512 columns, its
// last 64 rotated -- tcgen05 kernel (sm_103a).
//
// What it computes, for token t and head h of q [T, H, 128 + 64]:
//   out[t, h, c]       = sum_n q[t, h, n] * w_uk[h, n, c]         (c < 512)
//   out[t, h, 512 + i] = column 128 + i of q[t, h], rotated by the angles of positions[t]
// in float32, rounded once to bf16, or to e4m3 codes of out / q_scale.
//
// Bound by DRAM: a row reads 384 bytes and writes 1,152 (bf16) or 576
// (e4m3), 85 or 137 FLOP a byte; a head's W_UK is 128 KB more, which counts
// up to some hundred tokens.  4,096 tokens x 96 heads to e4m3 75 us (5.2 TB/s),
// to bf16 113 (5.5); 2,048 x 12 8.4; 64 x 12 3.5, which is the chain of loads,
// MMAs and stores of one unit.
//
// Design: one persistent CTA per SM walks a contiguous range of units (head,
// chunk of NC columns, tile of 128 tokens; tokens fastest, so W_UK's chunk
// stays in shared memory until the head changes).  The queries are the MMA's
// M = 128 rows, K-major as they lie in memory; W_UK's columns are its N, and
// W_UK[h] [128][512], columns contiguous, is the MN-major operand as it lies:
// nothing is transposed.  128 columns at a time go to one of four accumulators
// in TMEM, whose two warpgroups round and store them in turn while the MMAs
// fill the others (two accumulators of 256: e4m3 78 us, bf16 112): a warp's 32 rows of 128 bytes pass through shared
// memory, so that eight lanes write a row (by TMA stores of 128 rows x 128
// bytes, 1,270 cycles each: 122 us for 4,096 x 96 heads in bf16, 107 in e4m3).
//   warps 0..7    two epilogue warpgroups
//   warp 8        TMA loads: W_UK 128 columns at a time, the tiles' queries
//   warp 9        MMA issuer
//   warps 10..13  the rotated columns, registers only
#include <cuda_runtime.h>

#include "common.cuh"
#include "tc.cuh"
#include "vec8.cuh"

namespace mla {
namespace {

constexpr int kProdWarp = 8, kMmaWarp = 9, kRopeWarp0 = 10, kRopeWarps = 4;
constexpr int kThreads = (kRopeWarp0 + kRopeWarps) * 32;
constexpr int kBufs = 4;       // accumulators
constexpr int kTile = 128, kNope = 128, kBlock = kTile * 128;     // 128 rows of 128 bytes
constexpr int kHeadCols = kNope + MLA_D_ROPE;

struct AbsorbArgs {
    const __nv_bfloat16 *q;
    int64_t q_row, q_head, out_row, num_positions;
    void *out;
    const int64_t *positions;
    const float *cos_sin;
    int T, H, tiles;
    float inv_scale;
    bool pairs;
};

template <int NC, bool FP8>
struct Cfg {
    static constexpr int Sub = NC < 128 ? NC : 128, Subs = NC / Sub, Chunks = MLA_D_LATENT / NC;
    static constexpr int Stages = NC == 512 ? 2 : 3;        // query tiles
    static constexpr int Cols = FP8 ? 128 : 64;             // of a row's 128 bytes
    static_assert(Sub % Cols == 0, "whole stores");
    static constexpr int OffQ = NC / 64 * kBlock, OffOut = OffQ + Stages * 2 * kBlock;
    static constexpr int OffMisc = OffOut + 2 * kBlock;
    static constexpr uint32_t TmemCols = kBufs * Sub;
    // kind::f16: bf16 operands, B MN-major, f32 sums, M = 128, N = Sub.
    static constexpr uint32_t Idesc =
        (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(Sub >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

template <class C>
struct Misc {
    uint64_t w_full[C::Subs], w_free[C::Subs], q_full[C::Stages], q_free[C::Stages], d_full[kBufs], d_free[kBufs], fin;
    uint32_t tmem;
    int abort_flag;
};

// The CTA's units in order; every role walks them on its own.
template <class C>
struct Walk {
    int64_t u, end;
    int tile, chunk, h, tiles;
    bool fresh;     // W_UK's chunk is not the unit before's

    __device__ explicit Walk(const AbsorbArgs &a) {
        const int64_t all = (int64_t)a.H * C::Chunks * a.tiles;
        u = all * blockIdx.x / gridDim.x;
        end = all * (blockIdx.x + 1) / gridDim.x;
        tiles = a.tiles;
        const int hc = (int)(u / a.tiles);
        tile = (int)(u - (int64_t)hc * a.tiles);
        h = hc / C::Chunks;
        chunk = hc - h * C::Chunks;
        fresh = true;
    }
    __device__ bool valid() const { return u < end; }
    __device__ bool last() const { return u + 1 == end || tile + 1 == tiles; }     // with this chunk
    __device__ void next() {
        ++u;
        fresh = ++tile == tiles;
        if (!fresh) return;
        tile = 0;
        if (++chunk == C::Chunks) chunk = 0, ++h;
    }
};

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                         uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(one));
}

template <class C>
__device__ void producer(const AbsorbArgs &a, const CUtensorMap *mq, const CUtensorMap *mw, uint8_t *sm, Misc<C> &ms) {
    const int lane = threadIdx.x & 31;
    int it = 0, loads = 0;      // tiles, W_UK chunks
    int subs = 0;               // of the last chunk whose copies are issued
    bool ok = true;
    for (Walk<C> w(a); ok && w.valid(); w.next(), ++it) {
        if (w.fresh) {
            for (int s = 0; s < C::Subs && ok; ++s) {
                if (!(ok = warp_wait(&ms.w_free[s], (loads & 1) ^ 1, &ms.abort_flag))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ms.w_full[s], C::Sub / 64 * kBlock);
                    for (int b = s * (C::Sub / 64); b < (s + 1) * (C::Sub / 64); ++b)
                        tc::tma_2d(sm + b * kBlock, mw, w.chunk * (C::Sub * C::Subs) + 64 * b, kNope * w.h, &ms.w_full[s]);
                }
                __syncwarp();
                subs = s + 1;
            }
            if (!ok) break;
            ++loads;
        }
        const int s = it % C::Stages;
        if (!(ok = warp_wait(&ms.q_free[s], ((it / C::Stages) & 1) ^ 1, &ms.abort_flag))) break;
        if (lane == 0) {
            mbar_arrive_expect_tx(&ms.q_full[s], 2 * kBlock);
            for (int b = 0; b < 2; ++b)
                tc::tma_3d(sm + C::OffQ + (2 * s + b) * kBlock, mq, 64 * b, w.h, w.tile * kTile, &ms.q_full[s]);
        }
        __syncwarp();
    }
    if (!ok) {      // flagged: the copies in flight land before the CTA ends
        for (int k = it < C::Stages ? 0 : it - C::Stages; k < it; ++k)
            mbar_wait(&ms.q_full[k % C::Stages], (k / C::Stages) & 1);
        for (int s = 0; s < C::Subs; ++s) {
            const int n = s < subs && subs < C::Subs ? loads + 1 : loads;
            if (n > 0) mbar_wait(&ms.w_full[s], (n - 1) & 1);
        }
    }
}

template <class C>
__device__ void mma_issuer(const AbsorbArgs &a, uint8_t *sm, Misc<C> &ms) {
    const uint32_t base = smem_u32(sm), tm = ms.tmem;
    const uint32_t one = tc::elect_one();
    int it = 0, g = 0, loads = 0;
    bool ok = true;
    for (Walk<C> w(a); ok && w.valid(); w.next(), ++it) {
        const int s = it % C::Stages;
        if (w.fresh) ++loads;
        if (!(ok = warp_wait(&ms.q_full[s], (it / C::Stages) & 1, &ms.abort_flag))) break;
        const uint64_t qd = tc::sdesc(base + C::OffQ + 2 * s * kBlock, 16, 1024, tc::kSw128);
        for (int sub = 0; sub < C::Subs; ++sub, ++g) {
            const int d = g % kBufs;
            if (w.fresh && !(ok = warp_wait(&ms.w_full[sub], (loads - 1) & 1, &ms.abort_flag))) break;
            if (!(ok = warp_wait(&ms.d_free[d], ((g / kBufs) & 1) ^ 1, &ms.abort_flag))) break;
            tc::fence_after();
            // 16 of n a step: 32 bytes of a query's row, 16 rows of 128 bytes of each of W_UK's 64-column blocks.
            const uint64_t wd = tc::sdesc(base + sub * (C::Sub / 64) * kBlock, kBlock, 1024, tc::kSw128);
#pragma unroll
            for (int j = 0; j < kNope / 16; ++j)
                mma_bf16(tm + d * C::Sub, qd + (j >> 2) * (kBlock >> 4) + (j & 3) * 2, wd + j * (2048 >> 4), C::Idesc,
                         j > 0, one);
            if (one) {
                tc::commit(&ms.d_full[d]);
                if (w.last()) tc::commit(&ms.w_free[sub]);
                if (sub == C::Subs - 1) tc::commit(&ms.q_free[s]);
            }
            __syncwarp();
        }
    }
    // Every MMA issued must be complete before TMEM is released.
    if (one) tc::commit(&ms.fin);
    __syncwarp();
    mbar_wait(&ms.fin, 0);
}

template <class C, bool FP8>
__device__ void epilogue(const AbsorbArgs &a, uint8_t *sm, Misc<C> &ms) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, row0 = 32 * (warp & 3);
    const uint32_t taddr = ms.tmem + ((uint32_t)row0 << 16);
    uint8_t *buf = sm + C::OffOut + warp * (32 * 128);      // of this warp's 32 rows of 128 bytes
    constexpr int kSize = FP8 ? 1 : 2;
    int g = 0;
    bool ok = true;
    for (Walk<C> w(a); ok && w.valid(); w.next()) {
        for (int sub = 0; sub < C::Subs; ++sub, ++g) {
            if ((g & 1) != wg) continue;
            const int d = g % kBufs;
            if (!(ok = warp_wait(&ms.d_full[d], (g / kBufs) & 1, &ms.abort_flag))) break;
            tc::fence_after();
            // Eight lanes write a row's 128 bytes, four rows at once.
            const int t0 = w.tile * kTile + row0 + (lane >> 3), rows = a.T - t0;
            uint8_t *to = static_cast<uint8_t *>(a.out) +
                          (t0 * a.out_row + (int64_t)w.h * MLA_D_QK + w.chunk * (C::Sub * C::Subs) + sub * C::Sub) * kSize +
                          16 * (lane & 7);
#pragma unroll 1
            for (int b = 0; b < C::Sub / C::Cols; ++b, to += 128) {
                uint32_t out[32];       // 128 bytes of this lane's row
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[C::Cols / 2];
#pragma unroll
                    for (int i = 0; i < C::Cols / 32; ++i)
                        tc::ld16(taddr + d * C::Sub + b * C::Cols + half * (C::Cols / 2) + 16 * i,
                                 *reinterpret_cast<float(*)[16]>(v + 16 * i));
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (FP8) {
                            const float *f = v + 4 * i;
                            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                                make_float2(f[0] * a.inv_scale, f[1] * a.inv_scale), __NV_SATFINITE, __NV_E4M3);
                            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                                make_float2(f[2] * a.inv_scale, f[3] * a.inv_scale), __NV_SATFINITE, __NV_E4M3);
                            out[16 * half + i] = lo | hi << 16;
                        } else {
                            out[16 * half + i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                        }
                    }
                }
                if (b == C::Sub / C::Cols - 1) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.d_free[d]);
                }
                // Through shared memory (chunks turned by the row: no conflicts) into whole rows.
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                        make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3);
                    const uint4 x = *reinterpret_cast<const uint4 *>(buf + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                    if (4 * i < rows) *reinterpret_cast<uint4 *>(to + 4 * i * a.out_row * kSize) = x;
                }
            }
        }
    }
}

// Columns 512 .. 575, apart from the units: the grid's warps of this role share
// the batch's (eight tokens, head) in order, heads fastest, so that a token's
// sines stay in registers over its heads (as part of the units every head
// fetched them again: 104 us for 4,096 x 96 heads to e4m3, without a rotation
// 78).  Four lanes a token, lane i the pairs 8i .. 8i + 7, four heads at once.
template <bool FP8>
__device__ void rotate(const AbsorbArgs &a) {
    constexpr int kHalf = MLA_D_ROPE / 2, kHeads = 4;
    const int lane = threadIdx.x & 31, i4 = lane & 3;
    const int v0 = a.pairs ? 2 * i4 : i4, v1 = a.pairs ? 2 * i4 + 1 : i4 + 4;       // this lane's vectors
    const int64_t n = (int64_t)((a.T + 7) / 8) * a.H;
    const int rw = blockIdx.x * kRopeWarps + (threadIdx.x >> 5) - kRopeWarp0, warps = gridDim.x * kRopeWarps;
    int64_t at = n * rw / warps;
    const int64_t end = n * (rw + 1) / warps;
    int group = (int)(at / a.H), h0 = (int)(at - (int64_t)group * a.H);
    for (; at < end; ++group, h0 = 0) {
        const int heads = (int)min(end - at, (int64_t)(a.H - h0));
        at += heads;
        const bool real = 8 * (int64_t)group + (lane >> 2) < a.T;
        const int t = real ? 8 * group + (lane >> 2) : a.T - 1;
        const __nv_bfloat16 *x = a.q + t * a.q_row + h0 * a.q_head + kNope;
        uint4 u[kHeads], v[kHeads];
        const auto fetch = [&](int h) {
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                const uint4 *from = reinterpret_cast<const uint4 *>(x + min(h + k, heads - 1) * a.q_head);
                u[k] = from[v0];
                v[k] = from[v1];
            }
        };
        fetch(0);
        float c[8], s[8];
        if (a.positions) {
            int64_t p = a.positions[t];
            if ((uint64_t)p >= (uint64_t)a.num_positions) {
                if (i4 == 0 && h0 == 0 && real) flag(MLA_DEV_BAD_POSITION);
                p = 0;
            }
            const float4 *cs = reinterpret_cast<const float4 *>(a.cos_sin + p * MLA_D_ROPE) + 2 * i4;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                *reinterpret_cast<float4 *>(&c[4 * j]) = cs[j];
                *reinterpret_cast<float4 *>(&s[4 * j]) = cs[kHalf / 4 + j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = s[j] = 0.f;
        }
        const int64_t o = t * a.out_row + (int64_t)h0 * MLA_D_QK + MLA_D_LATENT;
#pragma unroll 1
        for (int h = 0; h < heads; h += kHeads) {
            uint4 cu[kHeads], cv[kHeads];
#pragma unroll
            for (int k = 0; k < kHeads; ++k) cu[k] = u[k], cv[k] = v[k];
            if (h + kHeads < heads) fetch(h + kHeads);      // on their way meanwhile
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                float y[2][8], x0[8], x1[8];
                unpack8<__nv_bfloat16>(cu[k], x0);
                unpack8<__nv_bfloat16>(cv[k], x1);
                if (!a.positions) {         // as they are (0 * inf would not be)
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[0][j] = x0[j], y[1][j] = x1[j];
                } else if (a.pairs) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[0][2 * j] = x0[2 * j] * c[j] - x0[2 * j + 1] * s[j];
                        y[0][2 * j + 1] = x0[2 * j + 1] * c[j] + x0[2 * j] * s[j];
                        y[1][2 * j] = x1[2 * j] * c[4 + j] - x1[2 * j + 1] * s[4 + j];
                        y[1][2 * j + 1] = x1[2 * j + 1] * c[4 + j] + x1[2 * j] * s[4 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[0][j] = x0[j] * c[j] - x1[j] * s[j];
                        y[1][j] = x1[j] * c[j] + x0[j] * s[j];
                    }
                }
                if (!real || h + k >= heads) continue;
                const int64_t to = o + (h + k) * MLA_D_QK;
                if (FP8) {
                    uint2 *p = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + to);
                    p[v0] = pack8_e4m3(y[0], a.inv_scale);
                    p[v1] = pack8_e4m3(y[1], a.inv_scale);
                } else {
                    uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to);
                    p[v0] = pack8<__nv_bfloat16>(y[0]);
                    p[v1] = pack8<__nv_bfloat16>(y[1]);
                }
            }
        }
    }
}

template <int NC, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    absorb_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mw,
                  const AbsorbArgs a) {
    using C = Cfg<NC, FP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<C> &ms = *reinterpret_cast<Misc<C> *>(sm + C::OffMisc);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        tc::prefetch_map(&mq);
        tc::prefetch_map(&mw);
        for (int s = 0; s < C::Subs; ++s) {
            mbar_init(&ms.w_full[s], 1);
            mbar_init(&ms.w_free[s], 1);
        }
        for (int s = 0; s < C::Stages; ++s) {
            mbar_init(&ms.q_full[s], 1);
            mbar_init(&ms.q_free[s], 1);
        }
        for (int d = 0; d < kBufs; ++d) {
            mbar_init(&ms.d_full[d], 1);
            mbar_init(&ms.d_free[d], 4);
        }
        mbar_init(&ms.fin, 1);
        ms.abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&ms.tmem, C::TmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    grid_wait();
    if (warp < kProdWarp) epilogue<C, FP8>(a, sm, ms);
    else if (warp == kProdWarp) producer<C>(a, &mq, &mw, sm, ms);
    else if (warp == kMmaWarp) mma_issuer<C>(a, sm, ms);
    else rotate<FP8>(a);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kMmaWarp) tc::tmem_free(ms.tmem, C::TmemCols);
}

// The query [T][H][192], read in boxes of 64 columns x 128 tokens.
bool encode_q(CUtensorMap *m, const void *q, int H, int T, int64_t head, int64_t row) {
    const cuuint64_t dim[3] = {(cuuint64_t)kHeadCols, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t stride[2] = {(cuuint64_t)(head * 2), (cuuint64_t)(row * 2)};
    const cuuint32_t box[3] = {64, 1, kTile}, one[3] = {1, 1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dim, stride, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_w(CUtensorMap *m, const void *w_uk, int H) {
    const cuuint64_t dim[2] = {(cuuint64_t)MLA_D_LATENT, (cuuint64_t)H * kNope};
    const cuuint64_t stride[1] = {(cuuint64_t)MLA_D_LATENT * 2};
    const cuuint32_t box[2] = {64, kNope}, one[2] = {1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(w_uk), dim, stride, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NC, bool FP8>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mw, const AbsorbArgs &a, int sms, cudaStream_t st) {
    using C = Cfg<NC, FP8>;
    constexpr int smem = C::OffMisc + sizeof(Misc<C>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = smem_attr_once<absorb_kernel<NC, FP8>>(smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.H * C::Chunks * a.tiles;
    return launch_early(absorb_kernel<NC, FP8>, (unsigned)(units < sms ? units : sms), kThreads, smem, st, mq, mw, a);
}

}  // namespace

// Arguments checked by mla_query_absorb.
cudaError_t query_absorb_launch(const void *q, int64_t q_row, int64_t q_head, const void *w_uk, const int64_t *positions,
                                const float *cos_sin, int64_t num_positions, bool pairs, int T, int H, float q_scale,
                                bool fp8, void *out, int64_t out_row, int sms, cudaStream_t st) {
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    CUtensorMap mq, mw;
    if (!encode_q(&mq, q, H, T, q_head, q_row) || !encode_w(&mw, w_uk, H)) return cudaErrorInvalidValue;
    AbsorbArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_row = q_row;
    a.q_head = q_head;
    a.out = out;
    a.out_row = out_row;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.num_positions = num_positions;
    a.pairs = pairs;
    a.T = T;
    a.H = H;
    a.tiles = (T + kTile - 1) / kTile;
    a.inv_scale = fp8 ? 1.f / q_scale : 1.f;
    const int64_t heads_tiles = (int64_t)H * a.tiles;
    if (heads_tiles >= 4 * (int64_t)sms) return fp8 ? launch<512, true>(mq, mw, a, sms, st) : launch<512, false>(mq, mw, a, sms, st);
    if (fp8 || heads_tiles * 4 >= sms) return fp8 ? launch<128, true>(mq, mw, a, sms, st) : launch<128, false>(mq, mw, a, sms, st);
    return launch<64, false>(mq, mw, a, sms, st);
}

cudaError_t query_absorb_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
