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
// up to some hundred tokens.
//
// Design: one persistent CTA per SM walks a contiguous range of units (head,
// chunk of NC columns, tile of 128 tokens; tokens fastest, so W_UK's chunk
// stays in shared memory until the head changes).  The queries are the MMA's
// M = 128 rows, K-major as they lie in memory; W_UK's columns are its N, and
// W_UK[h] [128][512], columns contiguous, is the MN-major operand as it lies:
// nothing is transposed.  SUB columns at a time go to one of two accumulators
// in TMEM, each with a warpgroup of its own that rounds it and stores 128
// rows x 128 bytes by TMA (which drops the rows past T), while the MMAs fill
// the other.
//   warps 0..7    two epilogue warpgroups, one an accumulator
//   warp 8        TMA loads: W_UK a SUB at a time, the tiles' queries
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
    static constexpr int Sub = NC < 256 ? NC : 256, Subs = NC / Sub, Chunks = MLA_D_LATENT / NC;
    static constexpr int Stages = NC == 512 ? 2 : 3, Bufs = NC == 512 ? 1 : 2;     // query tiles; a warpgroup's stores
    static constexpr int Cols = FP8 ? 128 : 64;                                      // of a store
    static_assert(Sub % Cols == 0, "whole stores");
    static constexpr int OffQ = NC / 64 * kBlock, OffOut = OffQ + Stages * 2 * kBlock;
    static constexpr int OffMisc = OffOut + 2 * Bufs * kBlock;
    static constexpr uint32_t TmemCols = 2 * Sub;
    // kind::f16: bf16 operands, B MN-major, f32 sums, M = 128, N = Sub.
    static constexpr uint32_t Idesc =
        (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(Sub >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

template <class C>
struct Misc {
    uint64_t w_full[C::Subs], w_free[C::Subs], q_full[C::Stages], q_free[C::Stages], d_full[2], d_free[2], fin;
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

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}
// All but the newest N stores of this thread have read their shared memory.
template <int N>
__device__ __forceinline__ void tma_store_wait() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
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
            const int d = g & 1;
            if (w.fresh && !(ok = warp_wait(&ms.w_full[sub], (loads - 1) & 1, &ms.abort_flag))) break;
            if (!(ok = warp_wait(&ms.d_free[d], ((g >> 1) & 1) ^ 1, &ms.abort_flag))) break;
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
__device__ void epilogue(const AbsorbArgs &a, const CUtensorMap *mo, uint8_t *sm, Misc<C> &ms) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, row = threadIdx.x & 127;
    const uint32_t taddr = ms.tmem + wg * C::Sub + ((uint32_t)(32 * (warp & 3)) << 16);
    const bool lead = row == 0;
    int g = 0, stores = 0;
    bool ok = true;
    for (Walk<C> w(a); ok && w.valid(); w.next()) {
        for (int sub = 0; sub < C::Subs; ++sub, ++g) {
            if ((g & 1) != wg) continue;
            if (!(ok = warp_wait(&ms.d_full[wg], (g >> 1) & 1, &ms.abort_flag))) break;
            tc::fence_after();
#pragma unroll 1
            for (int b = 0; b < C::Sub / C::Cols; ++b, ++stores) {
                uint32_t out[32];       // 128 bytes of this row
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[C::Cols / 2];
#pragma unroll
                    for (int i = 0; i < C::Cols / 32; ++i)
                        tc::ld16(taddr + b * C::Cols + half * (C::Cols / 2) + 16 * i,
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
                    if (lane == 0) mbar_arrive(&ms.d_free[wg]);
                }
                // The buffer's store before has read it.
                uint8_t *buf = sm + C::OffOut + (wg * C::Bufs + stores % C::Bufs) * kBlock;
                if (lead) tma_store_wait<C::Bufs - 1>();
                named_sync(1 + wg, 128);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(buf + row * 128 + ((i ^ (row & 7)) << 4)) =
                        make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                tc::fence_async_smem();
                named_sync(1 + wg, 128);
                if (lead)
                    tma_store_3d(mo, buf, w.chunk * (C::Sub * C::Subs) + sub * C::Sub + b * C::Cols, w.h, w.tile * kTile);
            }
        }
    }
    if (lead) tma_store_wait<0>();
}

// Columns 512 .. 575: four lanes a token, lane i the pairs 8i .. 8i + 7.
template <class C, bool FP8>
__device__ void rotate(const AbsorbArgs &a) {
    constexpr int kBatch = 2, kHalf = MLA_D_ROPE / 2;
    const int rw = (threadIdx.x >> 5) - kRopeWarp0, i4 = threadIdx.x & 3, sub = (threadIdx.x & 31) >> 2;
    for (Walk<C> w(a); w.valid(); w.next()) {
        // A tile's chunks share its tokens.
        const int t0 = w.tile * kTile + w.chunk * (kTile / C::Chunks), t1 = min(t0 + kTile / C::Chunks, a.T);
#pragma unroll 1
        for (int at = t0 + rw * 8; at < t1; at += kRopeWarps * 8 * kBatch) {
            uint4 u[kBatch], v[kBatch];
            float c[kBatch][8], s[kBatch][8];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = at + kRopeWarps * 8 * k + sub;
                if (t >= t1) continue;
                const uint4 *x = reinterpret_cast<const uint4 *>(a.q + t * a.q_row + w.h * a.q_head + kNope);
                u[k] = __ldg(x + (a.pairs ? 2 * i4 : i4));
                v[k] = __ldg(x + (a.pairs ? 2 * i4 + 1 : i4 + 4));
                if (!a.positions) continue;
                int64_t p = __ldg(a.positions + t);
                if (p < 0 || p >= a.num_positions) {
                    if (i4 == 0 && w.h == 0) flag(MLA_DEV_BAD_POSITION);
                    p = 0;
                }
                const float4 *cs = reinterpret_cast<const float4 *>(a.cos_sin + p * MLA_D_ROPE) + 2 * i4;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    *reinterpret_cast<float4 *>(&c[k][4 * j]) = __ldg(cs + j);
                    *reinterpret_cast<float4 *>(&s[k][4 * j]) = __ldg(cs + kHalf / 4 + j);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = at + kRopeWarps * 8 * k + sub;
                if (t >= t1) continue;
                float y[16], x[16];
                unpack8<__nv_bfloat16>(u[k], *reinterpret_cast<float(*)[8]>(x));
                unpack8<__nv_bfloat16>(v[k], *reinterpret_cast<float(*)[8]>(x + 8));
                if (!a.positions) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = x[j];
                } else if (a.pairs) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[2 * j] = x[2 * j] * c[k][j] - x[2 * j + 1] * s[k][j];
                        y[2 * j + 1] = x[2 * j + 1] * c[k][j] + x[2 * j] * s[k][j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[j] = x[j] * c[k][j] - x[8 + j] * s[k][j];
                        y[8 + j] = x[8 + j] * c[k][j] + x[j] * s[k][j];
                    }
                }
                const int64_t o = t * a.out_row + (int64_t)w.h * MLA_D_QK + MLA_D_LATENT;
                const int v0 = a.pairs ? 2 * i4 : i4, v1 = a.pairs ? 2 * i4 + 1 : i4 + 4;
                const float(&y0)[8] = *reinterpret_cast<float(*)[8]>(y);
                const float(&y1)[8] = *reinterpret_cast<float(*)[8]>(y + 8);
                if (FP8) {
                    uint2 *to = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + o);
                    to[v0] = pack8_e4m3(y0, a.inv_scale);
                    to[v1] = pack8_e4m3(y1, a.inv_scale);
                } else {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + o);
                    to[v0] = pack8<__nv_bfloat16>(y0);
                    to[v1] = pack8<__nv_bfloat16>(y1);
                }
            }
        }
    }
}

template <int NC, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    absorb_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mw,
                  const __grid_constant__ CUtensorMap mo, const AbsorbArgs a) {
    using C = Cfg<NC, FP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<C> &ms = *reinterpret_cast<Misc<C> *>(sm + C::OffMisc);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        tc::prefetch_map(&mq);
        tc::prefetch_map(&mw);
        tc::prefetch_map(&mo);
        for (int s = 0; s < C::Subs; ++s) {
            mbar_init(&ms.w_full[s], 1);
            mbar_init(&ms.w_free[s], 1);
        }
        for (int s = 0; s < C::Stages; ++s) {
            mbar_init(&ms.q_full[s], 1);
            mbar_init(&ms.q_free[s], 1);
        }
        for (int d = 0; d < 2; ++d) {
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
    if (warp < kProdWarp) epilogue<C, FP8>(a, &mo, sm, ms);
    else if (warp == kProdWarp) producer<C>(a, &mq, &mw, sm, ms);
    else if (warp == kMmaWarp) mma_issuer<C>(a, sm, ms);
    else rotate<C, FP8>(a);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kMmaWarp) tc::tmem_free(ms.tmem, C::TmemCols);
}

// A [T][H][cols] tensor read or written in boxes of 128 bytes x 128 tokens.
bool encode(CUtensorMap *m, const void *p, bool bytes, int cols, int H, int T, int64_t head, int64_t row) {
    const int es = bytes ? 1 : 2;
    const cuuint64_t dim[3] = {(cuuint64_t)cols, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t stride[2] = {(cuuint64_t)(head * es), (cuuint64_t)(row * es)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), 1, kTile}, one[3] = {1, 1, 1};
    return tc::encode_fn()(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
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
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mw, const CUtensorMap &mo, const AbsorbArgs &a, int sms,
                   cudaStream_t st) {
    using C = Cfg<NC, FP8>;
    constexpr int smem = C::OffMisc + sizeof(Misc<C>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = smem_attr_once<absorb_kernel<NC, FP8>>(smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.H * C::Chunks * a.tiles;
    return launch_early(absorb_kernel<NC, FP8>, (unsigned)(units < sms ? units : sms), kThreads, smem, st, mq, mw, mo, a);
}

}  // namespace

// Arguments checked by mla_query_absorb.
cudaError_t query_absorb_launch(const void *q, int64_t q_row, int64_t q_head, const void *w_uk, const int64_t *positions,
                                const float *cos_sin, int64_t num_positions, bool pairs, int T, int H, float q_scale,
                                bool fp8, void *out, int64_t out_row, int sms, cudaStream_t st) {
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    CUtensorMap mq, mw, mo;
    if (!encode(&mq, q, false, kHeadCols, H, T, q_head, q_row) || !encode_w(&mw, w_uk, H) ||
        !encode(&mo, out, fp8, MLA_D_QK, H, T, MLA_D_QK, out_row))
        return cudaErrorInvalidValue;
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
    if (heads_tiles >= 4 * (int64_t)sms) return fp8 ? launch<512, true>(mq, mw, mo, a, sms, st) : launch<512, false>(mq, mw, mo, a, sms, st);
    if (fp8 || heads_tiles * 4 >= sms) return fp8 ? launch<128, true>(mq, mw, mo, a, sms, st) : launch<128, false>(mq, mw, mo, a, sms, st);
    return launch<64, false>(mq, mw, mo, a, sms, st);
}

cudaError_t query_absorb_status(unsigned int *flags, bool clear) { return read_status(flags, clear); }

}  // namespace mla
