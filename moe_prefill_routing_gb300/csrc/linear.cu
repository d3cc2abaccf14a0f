// Dense products on the 5th-generation tensor cores (tcgen05 + TMEM), operands
// staged by TMA: moe_linear (bias, activation and residual in the epilogue)
// and its gradients.
//
// All three products have one form: D[m][n] = sum_r A[m][r] B[n][r], stored at
// out[n * ldo + m], with the output's contiguous dimension as the MMA's M:
//
//   y  [t][n] : m = n (output feature), n = t, r = i.  A = W  (r contiguous), B = x  (r contiguous)
//   dx [t][i] : m = i, n = t, r = n.                   A = W  (m contiguous), B = dP (r contiguous)
//   dW [n][i] : m = i, n = n, r = t.                   A = x  (m contiguous), B = dP (n contiguous)
//
// A few tokens therefore fill only the MMA's N (16 columns at least) while
// its M = 128 rows are always weights, and neighbouring lanes of the
// accumulator are neighbouring output elements.
//
// A tile's reduction is split over the Z CTAs of a thread-block cluster when
// there are fewer tiles than SMs; each leaves its fp32 accumulator in its
// own shared memory and the cluster adds them in rank order through
// distributed shared memory (results are deterministic).
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

namespace moe {
namespace {

constexpr int LM = 128;                      // MMA M
constexpr int LK = 64;                       // reduction per stage: one 128-byte row
constexpr int kLinThreads = 192;             // producer, MMA, four accumulator warps
constexpr uint32_t kLinATile = LM * LK * 2;  // 16 KB
constexpr int kLinMaxStages = 8;
constexpr int kLinMaxSplit = 8;  // portable cluster size
constexpr uint64_t kLinDrainNs = 200000000ull;

struct LinArgs {
    const float *bias;
    const void *residual;
    void *pre;
    void *out;
    uint32_t *status;
    int64_t ldr, ldo, ldp;
    int M, N, R;
    int bn, stages, split, n_mt;
    int f16, out_f32, act;
    int vec_out, vec_res, vec_pre;  // four neighbouring elements are one aligned access
};

struct LinCtrl {
    uint64_t full[kLinMaxStages];
    uint64_t empty[kLinMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

__host__ __device__ __forceinline__ uint32_t lin_b_tile(int bn, bool b_mn)
{
    return uint32_t(b_mn && bn < 64 ? 64 : bn) * LK * 2;
}

__device__ __forceinline__ float4 dsmem_ld4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// sqrt(2/pi) (z + 0.044715 z^3); (1 + tanh u) / 2 is 1 / (1 + e^-2u)
__device__ __forceinline__ float gelu_u(float z)
{
    return 0.7978845608028654f * (z + 0.044715f * z * z * z);
}

template <int ACT>
__device__ __forceinline__ float act_t(float z)
{
    if constexpr (ACT == MOE_ACT_RELU)
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    else if constexpr (ACT == MOE_ACT_SILU)
        return __fdividef(z, 1.0f + __expf(-z));
    else if constexpr (ACT == MOE_ACT_GELU)
        return 0.5f * z * erfcf(z * -0.7071067811865476f);
    else if constexpr (ACT == MOE_ACT_GELU_TANH)
        return __fdividef(z, 1.0f + __expf(-2.0f * gelu_u(z)));
    else
        return z;
}

// f(integral_constant<int, act>)
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case MOE_ACT_RELU:
        return f(std::integral_constant<int, MOE_ACT_RELU>());
    case MOE_ACT_SILU:
        return f(std::integral_constant<int, MOE_ACT_SILU>());
    case MOE_ACT_GELU:
        return f(std::integral_constant<int, MOE_ACT_GELU>());
    case MOE_ACT_GELU_TANH:
        return f(std::integral_constant<int, MOE_ACT_GELU_TANH>());
    default:
        return f(std::integral_constant<int, MOE_ACT_NONE>());
    }
}

__device__ __forceinline__ float act_of(float z, int act)
{
    float y;
    with_act(act, [&](auto a) { y = act_t<decltype(a)::value>(z); });
    return y;
}

__device__ __forceinline__ float act_grad(float z, int act)
{
    switch (act) {
    case MOE_ACT_RELU:
        return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
        const float s = __fdividef(1.0f, 1.0f + __expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU:
        return 0.5f * erfcf(z * -0.7071067811865476f) +
               0.3989422804014327f * z * __expf(-0.5f * z * z);
    case MOE_ACT_GELU_TANH: {
        const float s = __fdividef(1.0f, 1.0f + __expf(-2.0f * gelu_u(z)));
        const float du = 0.7978845608028654f * (1.0f + 3.0f * 0.044715f * z * z);
        return s + z * 2.0f * s * (1.0f - s) * du;
    }
    default:
        return 1.0f;
    }
}

__device__ __forceinline__ uint16_t to16(float v, int f16)
{
    return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ float from16(uint16_t v, int f16)
{
    return f16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}

// Four neighbouring elements (the first `n` of them exist) of a 16-bit or
// fp32 tensor from element index `at`.
__device__ __forceinline__ void load4(float (&v)[4], const void *p, int64_t at, int n, int f32,
                                      int f16, bool vec)
{
    if (vec && n == 4) {
        if (f32) {
            const float4 q = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
            const ushort4 q =
                *reinterpret_cast<const ushort4 *>(static_cast<const uint16_t *>(p) + at);
            v[0] = from16(q.x, f16), v[1] = from16(q.y, f16);
            v[2] = from16(q.z, f16), v[3] = from16(q.w, f16);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = i >= n ? 0.0f
               : f32  ? static_cast<const float *>(p)[at + i]
                      : from16(static_cast<const uint16_t *>(p)[at + i], f16);
}

__device__ __forceinline__ void store4(const float (&v)[4], void *p, int64_t at, int n, int f32,
                                       int f16, bool vec)
{
    if (vec && n == 4) {
        if (f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) =
                make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<ushort4 *>(static_cast<uint16_t *>(p) + at) = make_ushort4(
                to16(v[0], f16), to16(v[1], f16), to16(v[2], f16), to16(v[3], f16));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) {
            if (f32)
                static_cast<float *>(p)[at + i] = v[i];
            else
                static_cast<uint16_t *>(p)[at + i] = to16(v[i], f16);
        }
}

// Bounded wait of the stop path.
__device__ __forceinline__ void lin_drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kLinDrainNs)
            return;
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kLinThreads)
    k_linear(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
             const LinArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ LinCtrl ctl;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int bn = p.bn, S = p.stages;
    const uint32_t b_bytes = lin_b_tile(bn, B_MN);
    const uint32_t stage_bytes = kLinATile + b_bytes;
    const uint32_t z = cluster_ctarank();
    const int tile = int(blockIdx.x) / p.split;
    const int m0 = (tile % p.n_mt) * LM, n0 = (tile / p.n_mt) * bn;
    const int nk = (p.R + LK - 1) / LK;
    const int kb0 = int(int64_t(nk) * z / p.split), kb1 = int(int64_t(nk) * (z + 1) / p.split);
    const uint32_t tmem_cols = bn < 32 ? 32u : uint32_t(bn);
    volatile int *abort_flag = &ctl.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        mbar_init(&ctl.done, 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        tmem_alloc(&ctl.tmem_base, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0 && lane == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag)) {
                ok = false;
                break;
            }
            uint64_t *fb = &ctl.full[stage];
            mbar_arrive_expect_tx(fb, stage_bytes);
            uint8_t *sa = smem + stage * stage_bytes, *sb = sa + kLinATile;
            const int k0 = kb * LK;
            if (A_MN) {  // 64 m x 64 r boxes, m contiguous
                tma_load_2d(sa, &map_a, fb, m0, k0);
                tma_load_2d(sa + 8192, &map_a, fb, m0 + 64, k0);
            } else {
                tma_load_2d(sa, &map_a, fb, k0, m0);
            }
            if (B_MN) {
                for (int c = 0; c < bn; c += 64)
                    tma_load_2d(sb + c * (LK * 2), &map_b, fb, n0 + c, k0);
            } else {
                tma_load_2d(sb, &map_b, fb, k0, n0);
            }
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok)  // stopped: let the copies already issued land
            for (int s = 0; s < S; ++s)
                if ((issued >> s) & 1u)
                    lin_drain(&ctl.full[s], (issued_par >> s) & 1u);
    } else if (warp == 1 && lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        uint32_t idesc = idesc_bf16_f32(LM, uint32_t(bn), A_MN, B_MN);
        if (p.f16)
            idesc &= ~((7u << 7) | (7u << 10));  // f16 operands: format 0
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&ctl.full[stage], phase, abort_flag))
                break;
            tc_fence_after_sync();
            const uint32_t sa = smem_u32(smem + stage * stage_bytes), sb = sa + kLinATile;
#pragma unroll
            for (int kk = 0; kk < LK / 16; ++kk) {
                // r contiguous: 16 of them are 32 bytes inside the 128-byte row;
                // m or n contiguous: 16 rows of 128 bytes, 64-element chunks 8 KB apart
                const uint64_t da = A_MN ? smem_desc_sw128(sa + kk * 2048, 8192, 1024)
                                         : smem_desc_sw128(sa + kk * 32, 16, 1024);
                const uint64_t db = B_MN ? smem_desc_sw128(sb + kk * 2048, 8192, 1024)
                                         : smem_desc_sw128(sb + kk * 32, 16, 1024);
                tc_mma_f16(tmem_base, da, db, idesc, kb != kb0 || kk != 0);
            }
            tc_commit(&ctl.empty[stage]);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        tc_commit(&ctl.done);  // arrives once every MMA issued here has completed
    }
    __syncwarp();

    // accumulator -> own shared memory, fp32 [n][m] (the ring is free: every
    // copy has been consumed by an MMA and every MMA has completed)
    float *acc = reinterpret_cast<float *>(smem);
    bool done = mbar_wait(&ctl.done, 0, abort_flag);
    if (!done)  // stopped: the MMAs in flight still read shared and write tensor memory
        lin_drain(&ctl.done, 0);
    done = __syncthreads_and(done);  // the producer's copies have landed, also when stopped
    if (warp >= 2) {
        const int m = (warp & 3) * 32 + int(lane);
        tc_fence_after_sync();
        const uint32_t t0 = tmem_base + (uint32_t(warp & 3) << 21);
        const int cols = min(bn, (p.N - n0 + 15) & ~15);
        for (int c = 0; c < cols; c += 16) {
            uint32_t r[16];
            if (kb1 > kb0 && done) {
                tmem_ld_32x32b_x16(t0 + uint32_t(c), r);
                tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                acc[(c + j) * LM + m] = kb1 > kb0 && done ? __uint_as_float(r[j]) : 0.0f;
        }
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, tmem_cols);
    }
    if (threadIdx.x == 0 && ctl.abort_flag && p.status)
        atomicOr(p.status, MOE_STATUS_TIMEOUT);
    __syncwarp();
    cluster_sync();

    // the cluster shares the tile's elements, four neighbouring m at a time
    const int cols = min(bn, p.N - n0);
    const uint32_t step = uint32_t(p.split) * kLinThreads;
    for (uint32_t q = z * kLinThreads + threadIdx.x; q < uint32_t(cols) * (LM / 4); q += step) {
        const int n = int(q / (LM / 4)), m = int(q % (LM / 4)) * 4;
        const int left = min(4, p.M - (m0 + m));
        if (left <= 0)
            continue;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r = 0; r < p.split; ++r) {
            const float4 o = dsmem_ld4(dsmem_addr(acc + n * LM + m, r));
            v[0] += o.x, v[1] += o.y, v[2] += o.z, v[3] += o.w;
        }
        const int64_t row = n0 + n;
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left)
                    v[i] += p.bias[m0 + m + i];
        }
        if (p.pre)
            store4(v, p.pre, row * p.ldp + m0 + m, left, 0, p.f16, p.vec_pre);
        if (p.act != MOE_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = act_of(v[i], p.act);
        }
        if (p.residual) {
            float a[4];
            load4(a, p.residual, row * p.ldr + m0 + m, left, p.out_f32, p.f16, p.vec_res);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] += a[i];
        }
        store4(v, p.out, row * p.ldo + m0 + m, left, p.out_f32, p.f16, p.vec_out);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its shared memory is read
}

// ---- large products: pairs of CTAs ---------------------------------------------
//
// Tiles of 256 (m) x bn (n): one tcgen05.mma of a CTA pair per 16 of r, each
// CTA loading its 128 rows of A and half the rows of B, so a stage of
// 64 r costs each SM 32 KB of loads (bn = 256) for 512 cycles of MMA; the
// same tile on one SM would load 64 KB.  Pairs walk the tiles
// (persistent); two accumulators in tensor memory let the eight epilogue
// warps work on one tile while the MMAs fill the other.  Neighbouring lanes
// are neighbouring outputs, so the epilogue stores straight from registers,
// 64 or 128 contiguous bytes per warp and column.
constexpr int kPairThreads = 320;  // producer, MMA, eight epilogue warps
constexpr int kPairEpiWarps = 8;
constexpr int kPairStages = 7;

struct PairCtrl {
    uint64_t full[kPairStages];
    uint64_t empty[kPairStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem_base;
    int abort_flag;
};

// 32 columns of a tile for one lane (output feature m): registers -> epilogue
// -> global.  `n` columns exist from the first one's row on.
template <int ACT>
__device__ __forceinline__ void pair_columns(const LinArgs &p, const uint32_t (&r)[32], int64_t row,
                                             int m, float bias, int n)
{
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j)
        v[j] = __uint_as_float(r[j]) + bias;
    if (p.pre) {
        uint16_t *o = static_cast<uint16_t *>(p.pre) + row * p.ldp + m;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n)
                o[int64_t(j) * p.ldp] = to16(v[j], p.f16);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
        v[j] = act_t<ACT>(v[j]);
    if (p.residual) {
        if (p.out_f32) {
            const float *a = static_cast<const float *>(p.residual) + row * p.ldr + m;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < n)
                    v[j] += a[int64_t(j) * p.ldr];
        } else {
            const uint16_t *a = static_cast<const uint16_t *>(p.residual) + row * p.ldr + m;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < n)
                    v[j] += from16(a[int64_t(j) * p.ldr], p.f16);
        }
    }
    if (p.out_f32) {
        float *o = static_cast<float *>(p.out) + row * p.ldo + m;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n)
                o[int64_t(j) * p.ldo] = v[j];
    } else {
        uint16_t *o = static_cast<uint16_t *>(p.out) + row * p.ldo + m;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n)
                o[int64_t(j) * p.ldo] = to16(v[j], p.f16);
    }
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b, const LinArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    // the same offset in both CTAs: dynamic shared memory starts at the same address
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ PairCtrl ctl;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int bn = p.bn, half = bn / 2, S = p.stages;
    const uint32_t stage_bytes = kLinATile + uint32_t(half) * (LK * 2);
    const uint32_t tmem_cols = 2u * uint32_t(bn);
    const int nk = (p.R + LK - 1) / LK;
    const int n_nt = (p.N + bn - 1) / bn;
    const int64_t tiles = int64_t(p.n_mt) * n_nt;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
    volatile int *abort_flag = &ctl.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 2 * kPairEpiWarps);  // both CTAs' warps
        }
        ctl.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&map_a);
        prefetch_tmap(&map_b);
    }
    if (warp == 1)
        tmem_alloc_pair(&ctl.tmem_base, tmem_cols);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    // Tiles in blocks of 16 n tiles, n fastest: the pairs running at one time
    // share few rows of both operands.
    auto tile_at = [&](int64_t t, int &m0, int &n0) {
        const int64_t block = int64_t(16) * p.n_mt;
        const int b = int(t / block);
        const int wide = min(16, n_nt - 16 * b);
        const int64_t u = t - b * block;
        m0 = int(u / wide) * (2 * LM);
        n0 = (16 * b + int(u % wide)) * bn;
    };

    if (warp == 0 && lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = first; ok && t < tiles; t += step) {
            int m0, n0;
            tile_at(t, m0, n0);
            m0 += int(rank) * LM;
            n0 += int(rank) * half;
            for (int kb = 0; kb < nk; ++kb) {
                if (!mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if (rank == 0)  // both CTAs' bytes complete on the even CTA's barrier
                    mbar_arrive_expect_tx(&ctl.full[stage], 2 * stage_bytes);
                const uint32_t fb = dsmem_addr(&ctl.full[stage], 0);
                uint8_t *sa = smem + stage * stage_bytes, *sb = sa + kLinATile;
                const int k0 = kb * LK;
                if (A_MN) {
                    tma_load_2d_pair(sa, &map_a, fb, m0, k0);
                    tma_load_2d_pair(sa + 8192, &map_a, fb, m0 + 64, k0);
                } else {
                    tma_load_2d_pair(sa, &map_a, fb, k0, m0);
                }
                if (B_MN) {
                    for (int c = 0; c < half; c += 64)
                        tma_load_2d_pair(sb + c * (LK * 2), &map_b, fb, n0 + c, k0);
                } else {
                    tma_load_2d_pair(sb, &map_b, fb, k0, n0);
                }
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every stage released: this CTA's copies have landed and been read
        for (int i = 0; ok && i < S; ++i) {
            ok = mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {  // stopped: copies in flight take microseconds; give them a millisecond
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000u) {
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, aphase = 0;
        uint32_t idesc = idesc_bf16_f32(2 * LM, uint32_t(bn), A_MN, B_MN);
        if (p.f16)
            idesc &= ~((7u << 7) | (7u << 10));
        bool ok = true;
        for (int64_t t = first; ok && t < tiles; t += step) {
            if (!mbar_wait(&ctl.acc_empty[buf], aphase ^ 1u, abort_flag))
                break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + uint32_t(buf * bn);
            for (int kb = 0; kb < nk; ++kb) {
                if (!mbar_wait(&ctl.full[stage], phase, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sa = smem_u32(smem + stage * stage_bytes), sb = sa + kLinATile;
#pragma unroll
                for (int kk = 0; kk < LK / 16; ++kk) {
                    const uint64_t da = A_MN ? smem_desc_sw128(sa + kk * 2048, 8192, 1024)
                                             : smem_desc_sw128(sa + kk * 32, 16, 1024);
                    const uint64_t db = B_MN ? smem_desc_sw128(sb + kk * 2048, 8192, 1024)
                                             : smem_desc_sw128(sb + kk * 32, 16, 1024);
                    tc_mma_f16_pair(d, da, db, idesc, (kb | kk) != 0);
                }
                tc_commit_pair(&ctl.empty[stage]);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            tc_commit_pair(&ctl.acc_full[buf]);
            if (++buf == 2) {
                buf = 0;
                aphase ^= 1u;
            }
        }
        // (the epilogue warps of both CTAs wait for every accumulator, so the
        // MMAs are done when the cluster meets below)
    } else if (warp >= 2) {
        const int q = warp & 3, part = (warp - 2) >> 2;  // TMEM lane quadrant, half of the columns
        int buf = 0;
        uint32_t aphase = 0;
        for (int64_t t = first; t < tiles; t += step) {
            int m0, n0;
            tile_at(t, m0, n0);
            const int m = m0 + int(rank) * LM + q * 32 + int(lane);
            const float bias = p.bias && m < p.M ? p.bias[m] : 0.0f;
            bool ok = mbar_wait(&ctl.acc_full[buf], aphase, abort_flag);
            if (!__all_sync(0xffffffffu, ok))
                break;
            tc_fence_after_sync();
            const uint32_t t0 = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(buf * bn);
            with_act(p.act, [&](auto act) {
                for (int c = part * half; c < (part + 1) * half; c += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t0 + uint32_t(c), r);
                    tmem_ld_wait();
                    const int n = min(32, p.N - (n0 + c));
                    if (m < p.M && n > 0)
                        pair_columns<decltype(act)::value>(p, r, int64_t(n0) + c, m, bias, n);
                    __syncwarp();
                }
            });
            tc_fence_before_sync();
            if (lane == 0)
                mbar_arrive_cluster(dsmem_addr(&ctl.acc_empty[buf], 0));
            if (++buf == 2) {
                buf = 0;
                aphase ^= 1u;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && ctl.abort_flag && p.status)
        atomicOr(p.status, MOE_STATUS_TIMEOUT);
    cluster_sync();  // both CTAs are done with each other's shared memory and barriers
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, tmem_cols);
    }
}

// ---- dP and db ---------------------------------------------------------------

constexpr int kGradThreads = 256;
constexpr int kGradCols = 128;      // columns of a CTA: 32 lanes x 4
constexpr int kGradMaxChunks = 128;  // rows of partial column sums

struct GradArgs {
    const void *dy, *pre;
    uint16_t *dp;     // null: not written
    float *part;      // [chunks][N] or null
    int64_t lddy, lddp;
    int T, N, rows;   // rows per chunk
    int dy_f32, f16, act;
    int vec_dy, vec_pre;
};

// dP = dy act'(pre), and the column sums of one chunk of rows: eight rows at
// a time, four columns a thread; the eight row groups are added in order.
__global__ void __launch_bounds__(kGradThreads) k_act_grad(const GradArgs p)
{
    __shared__ float red[8][kGradCols];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * kGradCols + lane * 4;
    const int left = min(4, p.N - c);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = int64_t(blockIdx.y) * p.rows;
    const int64_t t1 = min(int64_t(p.T), t0 + p.rows);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0)
        for (int64_t t = t0 + g; t < t1; t += 8) {
            float d[4];
            load4(d, p.dy, t * p.lddy + c, left, p.dy_f32, p.f16, p.vec_dy);
            if (p.act != MOE_ACT_NONE) {
                float z[4];
                load4(z, p.pre, t * p.N + c, left, 0, p.f16, p.vec_pre);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d[i] *= act_grad(z[i], p.act);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[i] += d[i];
            if (p.dp)  // lddp is a multiple of 8 and c of 4
                store4(d, p.dp, t * p.lddp + c, left, 0, p.f16, true);
        }
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        red[g][lane * 4 + i] = s[i];
    __syncthreads();
    const int col = blockIdx.x * kGradCols + threadIdx.x;
    if (threadIdx.x < kGradCols && col < p.N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += red[i][threadIdx.x];
        p.part[int64_t(blockIdx.y) * p.N + col] = v;
    }
}

__global__ void __launch_bounds__(kGradThreads)
    k_col_sum(const float *part, int chunks, int N, float *db)
{
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x * kGradThreads + threadIdx.x;
    if (c >= N)
        return;
    float v = 0.0f;
    for (int i = 0; i < chunks; ++i)
        v += part[int64_t(i) * N + c];
    db[c] = v;
}

// ---- host ---------------------------------------------------------------------

// 16-bit matrix [rows, cols], cols contiguous, rows ld elements apart, read in
// boxes of 64 columns x box_rows rows with the 128-byte swizzle.
cudaError_t lin_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
                    int box_rows, int f16)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
    const cuuint32_t box[2] = {LK, cuuint32_t(box_rows)}, estr[2] = {1, 1};
    const CUresult r =
        encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Operand {
    const void *p;
    int64_t rows, cols, ld;  // as stored: cols contiguous
};

cudaError_t launch_clustered(const void *kern, unsigned grid, unsigned cluster, unsigned threads,
                             size_t smem, cudaStream_t s, void **args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

// D[m][n] = sum_r A[m][r] B[n][r]; a.M, a.N, a.R and the epilogue fields are
// set, the tiling is chosen here.
template <bool A_MN, bool B_MN>
cudaError_t launch_linear(const Operand &A, const Operand &B, LinArgs a, cudaStream_t s)
{
    constexpr int which = B_MN ? 2 : A_MN ? 1 : 0;
    const int sms = device_sm_count();
    const int nk = (a.R + LK - 1) / LK;
    CUtensorMap ma, mb;
    const int64_t pair_tiles = int64_t((a.M + 2 * LM - 1) / (2 * LM)) * ((a.N + 255) / 256);
    if (pair_tiles >= sms / 2) {  // at least one tile for every pair of SMs
        a.bn = 256;
        a.n_mt = (a.M + 2 * LM - 1) / (2 * LM);
        a.split = 1;
        a.stages = kPairStages;
        const size_t smem = 1024 + size_t(a.stages) * (kLinATile + a.bn / 2 * LK * 2);
        cudaError_t e = lin_map(&ma, A.p, A.rows, A.cols, A.ld, A_MN ? LK : LM, a.f16);
        if (e == cudaSuccess)
            e = lin_map(&mb, B.p, B.rows, B.cols, B.ld, B_MN ? LK : a.bn / 2, a.f16);
        const void *kern = reinterpret_cast<const void *>(k_linear_pair<A_MN, B_MN>);
        if (e == cudaSuccess)
            e = ensure_smem_limit(kern, kSlotLinearPair0 + which, smem);
        if (e != cudaSuccess)
            return e;
        void *args[] = {&ma, &mb, &a};
        return launch_clustered(kern, unsigned(std::min<int64_t>(pair_tiles, sms / 2)) * 2, 2,
                                kPairThreads, smem, s, args);
    }
    a.bn = a.N <= 16 ? 16 : a.N <= 32 ? 32 : a.N <= 64 ? 64 : 128;
    a.n_mt = (a.M + LM - 1) / LM;
    const int64_t tiles = int64_t(a.n_mt) * ((a.N + a.bn - 1) / a.bn);
    // split the reduction while that still adds CTAs (two fit an SM) and
    // leaves each at least four stages
    a.split = 1;
    while (a.split < kLinMaxSplit && tiles * a.split * 2 <= 2 * sms && nk / (a.split * 2) >= 4)
        a.split *= 2;
    if (tiles * a.split > INT_MAX)
        return cudaErrorInvalidValue;
    const uint32_t stage = kLinATile + lin_b_tile(a.bn, B_MN);
    a.stages = std::min<int>(kLinMaxStages, 96 * 1024 / stage);
    const size_t ring = size_t(a.stages) * stage;
    const size_t smem = 1024 + std::max(ring, size_t(a.bn) * LM * 4);
    cudaError_t e = lin_map(&ma, A.p, A.rows, A.cols, A.ld, A_MN ? LK : LM, a.f16);
    if (e == cudaSuccess)
        e = lin_map(&mb, B.p, B.rows, B.cols, B.ld, B_MN ? LK : a.bn, a.f16);
    const void *kern = reinterpret_cast<const void *>(k_linear<A_MN, B_MN>);
    if (e == cudaSuccess)
        e = ensure_smem_limit(kern, kSlotLinear0 + which, 112 * 1024);
    if (e != cudaSuccess)
        return e;
    void *args[] = {&ma, &mb, &a};
    return launch_clustered(kern, unsigned(tiles * a.split), unsigned(a.split), kLinThreads, smem, s,
                            args);
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline size_t align256(size_t b)
{
    return (b + 255) & ~size_t(255);
}

// whether groups of four elements of rows `ld` apart are aligned accesses
inline int vec4(const void *p, int64_t ld, int size)
{
    return ld % 4 == 0 && aligned(p, 4 * size);
}

inline bool is16(int dtype)
{
    return dtype == MOE_DT_BF16 || dtype == MOE_DT_F16;
}

}  // namespace
}  // namespace moe

extern "C" int moe_linear(const void *x, int64_t ldx, const void *W, const float *bias,
                          const void *residual, int64_t ldr, int dtype, int act, int T, int K,
                          int N, void *pre, void *y, int64_t ldy, int y_dtype, uint32_t *status,
                          moe_stream_t stream)
{
    using namespace moe;
    if (!is16(dtype) || (y_dtype != dtype && y_dtype != MOE_DT_F32))
        return MOE_ERR_DTYPE;
    if (T < 0 || K < 1 || K % 8 != 0 || N < 1 || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH ||
        ldx < K || ldx % 8 != 0 || ldy < N || (residual && ldr < N))
        return MOE_ERR_SHAPE;
    if (!W || (T > 0 && (!x || !y)))
        return MOE_ERR_NULL;
    const int ysize = y_dtype == MOE_DT_F32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 4) || !aligned(residual, ysize) ||
        !aligned(y, ysize) || !aligned(pre, 2) || !aligned(status, 4))
        return MOE_ERR_ALIGN;
    if (T == 0)
        return MOE_OK;
    LinArgs a = {};
    a.bias = bias;
    a.residual = residual;
    a.pre = pre;
    a.out = y;
    a.status = status;
    a.ldr = ldr, a.ldo = ldy, a.ldp = N;
    a.M = N, a.N = T, a.R = K;
    a.f16 = dtype == MOE_DT_F16, a.out_f32 = y_dtype == MOE_DT_F32, a.act = act;
    a.vec_out = vec4(y, ldy, ysize), a.vec_res = vec4(residual, ldr, ysize);
    a.vec_pre = vec4(pre, N, 2);
    return launch_linear<false, false>({W, N, K, K}, {x, T, K, ldx}, a,
                                       reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

extern "C" size_t moe_linear_grad_workspace_bytes(int T, int N)
{
    if (T < 0 || N < 1)
        return 0;
    const size_t ldp = (size_t(N) + 7) & ~size_t(7);
    return moe::align256(size_t(T) * ldp * 2) +
           moe::align256(size_t(moe::kGradMaxChunks) * N * sizeof(float));
}

extern "C" int moe_linear_grad(const void *x, int64_t ldx, const void *W, const void *pre,
                               const void *dy, int64_t lddy, int dy_dtype, int dtype, int act,
                               int T, int K, int N, void *dx, void *dW, int dw_dtype, float *db,
                               void *ws, size_t ws_bytes, uint32_t *status, moe_stream_t stream)
{
    using namespace moe;
    if (!is16(dtype) || (dy_dtype != dtype && dy_dtype != MOE_DT_F32) ||
        (dw_dtype != dtype && dw_dtype != MOE_DT_F32))
        return MOE_ERR_DTYPE;
    if (T < 0 || K < 1 || K % 8 != 0 || N < 1 || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH ||
        lddy < N || (dW && (ldx < K || ldx % 8 != 0)))
        return MOE_ERR_SHAPE;
    if (!ws || (dx && !W) ||
        (T > 0 && (!dy || (dW && !x) || (act != MOE_ACT_NONE && !pre))))
        return MOE_ERR_NULL;
    if (ws_bytes < moe_linear_grad_workspace_bytes(T, N))
        return MOE_ERR_WORKSPACE;
    const int dysize = dy_dtype == MOE_DT_F32 ? 4 : 2, dwsize = dw_dtype == MOE_DT_F32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(pre, 2) || !aligned(dy, dysize) ||
        !aligned(dx, 2) || !aligned(dW, dwsize) || !aligned(db, 4) || !aligned(ws, 256) ||
        !aligned(status, 4))
        return MOE_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (dW && cudaMemsetAsync(dW, 0, size_t(N) * K * dwsize, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (db && cudaMemsetAsync(db, 0, size_t(N) * 4, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const int64_t ldp = (int64_t(N) + 7) & ~int64_t(7);
    uint16_t *dp = static_cast<uint16_t *>(ws);
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) +
                                            align256(size_t(T) * ldp * 2));
    const bool products = dx || dW;
    // dy is the products' operand as it is
    const bool direct =
        act == MOE_ACT_NONE && dy_dtype == dtype && lddy % 8 == 0 && aligned(dy, 16);
    if (db || (products && !direct)) {
        GradArgs g = {};
        g.dy = dy, g.pre = pre;
        g.dp = products && !direct ? dp : nullptr;
        g.part = db ? part : nullptr;
        g.lddy = lddy, g.lddp = ldp;
        g.T = T, g.N = N;
        g.dy_f32 = dy_dtype == MOE_DT_F32, g.f16 = dtype == MOE_DT_F16, g.act = act;
        g.vec_dy = vec4(dy, lddy, dysize), g.vec_pre = vec4(pre, N, 2);
        const int cb = (N + kGradCols - 1) / kGradCols;
        int chunks = std::max(1, std::min({(T + 31) / 32, 8 * device_sm_count() / cb,
                                           kGradMaxChunks}));
        g.rows = (T + chunks - 1) / chunks;
        chunks = (T + g.rows - 1) / g.rows;
        if (launch_pdl(k_act_grad, dim3(cb, chunks), dim3(kGradThreads), 0, s, g) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (db && launch_pdl(k_col_sum, dim3((N + kGradThreads - 1) / kGradThreads),
                             dim3(kGradThreads), 0, s, static_cast<const float *>(part), chunks,
                             N, db) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    const Operand P = direct ? Operand{dy, T, N, lddy} : Operand{dp, T, N, ldp};
    LinArgs a = {};
    a.status = status;
    a.f16 = dtype == MOE_DT_F16;
    a.act = MOE_ACT_NONE;
    a.ldo = K;
    if (dx) {
        a.out = dx;
        a.M = K, a.N = T, a.R = N;
        a.vec_out = vec4(dx, K, 2);
        if (launch_linear<true, false>({W, N, K, K}, P, a, s) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    if (dW) {
        a.out = dW;
        a.out_f32 = dw_dtype == MOE_DT_F32;
        a.M = K, a.N = N, a.R = T;
        a.vec_out = vec4(dW, K, dwsize);
        if (launch_linear<true, true>({x, T, K, ldx}, P, a, s) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}
