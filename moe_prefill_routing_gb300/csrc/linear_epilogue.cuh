// Epilogues of the dense products: bias, activation, residual and the writing
// of 16-bit or fp32 outputs from accumulators in tensor memory.
#pragma once

#include "../../include/moe_prefill.h"
#include "internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace moe {
namespace {

// y = act(sums + bias) + residual; pre = sums + bias.
struct EpiArgs {
    const float *bias;
    const void *residual;
    void *pre;
    void *out;
    int64_t ldr, ldo, ldp;
    int f16, out_f32, act;
    int vec_out, vec_res, vec_pre;  // rows and base are 16-byte aligned
    uint32_t flags;  // the epilogue's choices in one word, see EpiFlags
};

// What the epilogue of k_linear_pair asks for again and again, in a register:
// a field of one of two products is a constant load at a run-time offset, and
// a chain of branches on five of them took about 400 cycles.
enum EpiFlags : uint32_t {
    kEpiBias = 1,
    kEpiPre = 2,
    kEpiResidual = 4,
    kEpiF32 = 8,
    kEpiF16 = 16,
    kEpiVecOut = 32,
    kEpiVecRes = 64,
    kEpiVecPre = 128,
    kEpiMul = 256,
    kEpiAct = 512,  // times the activation
};

// 1 / (1 + 2^x): exponential and reciprocal by one special-function
// instruction each (2 units in the last place); 2^x past 2^126 gives 0, where
// the true value is below 2^-126.
__device__ __forceinline__ float sigmoid_2(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

__device__ __forceinline__ void dsmem_st4(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                          uint32_t w)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y),
                 "r"(z), "r"(w)
                 : "memory");
}

// Phi(z) and e^(-z^2/2), Phi the normal distribution function, from
// erfc(x) = t P(t) e^(-x^2), t = 1 / (1 + 0.43 x), x >= 0.  P, of degree 7, was
// fitted to e^(x^2) erfc(x) / t for the smallest relative error over
// x = 0 ... 9.6 (8.5e-8; e^(-x^2) is below 2^-126 from there on), by least
// squares whose weights grow where the error is largest.  A relative error,
// because GELU's values for negative z are z Phi(z) itself: in fp32 Phi is off
// by 1.5e-6 of itself down to z = -5 and 8e-6 at -13, most of it z^2's rounding
// in the exponent.  (The library's erfc takes registers that the epilogue
// lacks.)
__device__ __forceinline__ float cdf_t(float z)  // 1 / t
{
    return 1.0f + 0.43f * 0.7071067811865476f * fabsf(z);
}

__device__ __forceinline__ float cdf_e(float z)  // log2 of e^(-z^2/2)
{
    return z * z * -0.7213475204444817f;
}

__device__ __forceinline__ float cdf(float z, float t, float e)
{
    float q = 0.0736689789f;
    q = q * t - 0.310215612f;
    q = q * t + 0.383441133f;
    q = q * t - 0.0854884358f;
    q = q * t + 0.246721865f;
    q = q * t + 0.204987442f;
    q = q * t + 0.244369731f;
    q = q * t + 0.242514975f;
    q = 0.5f * q * t * e;
    return z > 0.0f ? 1.0f - q : q;
}

__device__ __forceinline__ float2 normal_cdf(float z)
{
    float t, e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(cdf_t(z)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(cdf_e(z)));
    return make_float2(cdf(z, t, e), e);
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kTanh1 = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float kTanh3 = 0.07135481627260025f;   // 2 sqrt(2/pi) 0.044715

// Of SiLU and GELU-tanh, act(z) = z / (1 + 2^x): x.  (1 + tanh u) / 2 is
// 1 / (1 + e^-2u), u = sqrt(2/pi) (z + 0.044715 z^3).
template <int ACT>
__device__ __forceinline__ float gate_x(float z)
{
    if constexpr (ACT == MOE_ACT_SILU)
        return z * -kLog2E;
    else
        return z * (-kLog2E * kTanh1 - kLog2E * kTanh3 * (z * z));
}

template <int ACT>
__device__ __forceinline__ float act_t(float z)
{
    if constexpr (ACT == MOE_ACT_RELU)
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    else if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU_TANH)
        return z * sigmoid_2(gate_x<ACT>(z));
    else if constexpr (ACT == MOE_ACT_GELU)
        return z * normal_cdf(z).x;
    else
        return z;
}

template <int R>
__device__ __forceinline__ void ex2_all(float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; ++i)
        asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x[i]));
}

template <int R>
__device__ __forceinline__ void rcp_all(float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; ++i)
        asm volatile("rcp.approx.ftz.f32 %0, %0;" : "+f"(x[i]));
}

// act_t of R values, each step for all of them in turn (volatile keeps that
// order): left to the compiler, one value's chain followed another's, and
// 4096 x 2816 x 11264 with GELU-tanh took 168 us instead of 158.
template <int ACT, int R>
__device__ __forceinline__ void act_all(float (&z)[R])
{
    if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU_TANH) {
        float s[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            s[i] = gate_x<ACT>(z[i]);
        ex2_all(s);
#pragma unroll
        for (int i = 0; i < R; ++i)
            s[i] += 1.0f;
        rcp_all(s);
#pragma unroll
        for (int i = 0; i < R; ++i)
            z[i] *= s[i];
    } else if constexpr (ACT == MOE_ACT_GELU) {
        float t[R], e[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            t[i] = cdf_t(z[i]);
            e[i] = cdf_e(z[i]);
        }
        rcp_all(t);
        ex2_all(e);
#pragma unroll
        for (int i = 0; i < R; ++i)
            z[i] *= cdf(z[i], t[i], e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            z[i] = act_t<ACT>(z[i]);
    }
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

template <int ACT>
__device__ __forceinline__ float act_grad(float z)
{
    if constexpr (ACT == MOE_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_2(gate_x<ACT>(z));
        return s * (1.0f + z * (1.0f - s));
    } else if constexpr (ACT == MOE_ACT_GELU) {
        const float2 c = normal_cdf(z);
        return c.x + 0.3989422804014327f * z * c.y;
    } else if constexpr (ACT == MOE_ACT_GELU_TANH) {
        const float s = sigmoid_2(gate_x<ACT>(z));
        // (z^2 cut where s is 0 or 1 long since, lest 0 times infinity come out)
        const float du2 = kTanh1 + 3.0f * kTanh3 * fminf(z * z, 1e8f);
        return s + z * s * (1.0f - s) * du2;
    } else {
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

// The epilogue, after the bias, of four neighbouring outputs (the first `left`
// exist) in each of R rows, `by` apart (those less than `rows` ahead exist).
template <int R>
__device__ __forceinline__ void finish_rows(const EpiArgs &p, float (&v)[R][4], int64_t row, int by,
                                            int rows, int col, int left)
{
    if (p.pre) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * by < rows)
                store4(v[i], p.pre, (row + i * by) * p.ldp + col, left, 0, p.f16, p.vec_pre);
    }
    float a[R][4];
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * by < rows)
                load4(a[i], p.residual, (row + i * by) * p.ldr + col, left, p.out_f32, p.f16,
                      p.vec_res);
    }
    if (p.act != MOE_ACT_NONE)
        with_act(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = act_t<decltype(act)::value>(v[i][j]);
        });
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[i][j] += i * by < rows ? a[i][j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i * by < rows)
            store4(v[i], p.out, (row + i * by) * p.ldo + col, left, p.out_f32, p.f16, p.vec_out);
}

constexpr uint64_t kLinDrainNs = 200000000ull;

// Bounded wait of the stop path.
__device__ __forceinline__ void lin_drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kLinDrainNs)
            return;
}

// Adds (or, first, copies) an accumulator of bn columns to the sum of the
// earlier chains; whole warp, its 32 lanes of tensor memory.  Not inlined: few
// calls come here, and the others' code stays short.
__device__ __noinline__ void add_small_chain(uint32_t acc, uint32_t sum, int bn, bool add)
{
#pragma unroll 1
    for (int c = 0; c < bn; c += 16) {
        uint32_t r[16], o[16];
        tmem_ld_32x32b_x16(acc + uint32_t(c), r);
        if (add)
            tmem_ld_32x32b_x16(sum + uint32_t(c), o);
        tmem_ld_wait();
        if (add) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(o[j]));
        }
        tmem_store_32x32b_x16(sum + uint32_t(c), r);
    }
    tmem_store_wait();
}

// ---- epilogue warps of CTA pairs ------------------------------------------------

constexpr int kPairEpiWarps = 8;
constexpr int kPairParts = kPairEpiWarps / 4;  // warps that share 32 rows
// Columns that an epilogue warp works on at once.  Fewer leave latencies bare,
// more make the loop's code too long for the instruction caches: 4096 x 2816
// x 11264 with GELU-tanh and pre takes 166 us with 8, 161 with 16, 164 with 32 (on one GPU).
constexpr int kCols = 16;
// A slot: 32 rows of 32 elements E, in 16-byte pieces laid out as the 64-byte
// (16-bit) or 128-byte (fp32) swizzle of a TMA copy has them, which also puts
// eight rows' same pieces into different banks.
template <typename E>
__device__ __forceinline__ uint4 *slot_at(uint8_t *slot, int r, int c)
{
    constexpr int kPieces = 2 * int(sizeof(E));  // 4 (16-bit) or 8 of a row
    const int x = sizeof(E) == 4 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
    return reinterpret_cast<uint4 *>(slot) + r * kPieces + x;
}

// Element by element, where 16-byte pieces are not aligned: rows [0, rows) x
// columns [0, cols) of a matrix with ld elements between rows.
template <bool STORE, typename E>
__device__ __noinline__ void move_by_element(uint8_t *slot, E *p, int64_t ld, int rows, int cols)
{
    constexpr int kPer = 16 / int(sizeof(E));
    const int lane = threadIdx.x & 31;
    if (lane < cols)
#pragma unroll 16
        for (int r = 0; r < rows; ++r) {
            E *at = reinterpret_cast<E *>(slot_at<E>(slot, r, lane / kPer)) + lane % kPer;
            if (STORE)
                p[int64_t(r) * ld + lane] = *at;
            else
                *at = p[int64_t(r) * ld + lane];
        }
}

// The residual's 32 rows x `cols` columns into a slot.
template <typename E>
__device__ __forceinline__ void load_slot(uint8_t *slot, const void *residual, int64_t at,
                                          int64_t ld, int rows, int cols, bool vec)
{
    constexpr int kPieces = 2 * int(sizeof(E)), kPer = 16 / int(sizeof(E));
    constexpr int kRows = 32 / kPieces;  // rows a warp moves at once
    const int lane = threadIdx.x & 31;
    E *p = static_cast<E *>(const_cast<void *>(residual)) + at;
    if (vec && cols == 32) {
        const int r0 = lane / kPieces, c = lane % kPieces;
        const E *q = p + int64_t(r0) * ld + c * kPer;
        uint4 v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (r0 + i * kRows < rows)
                v[i] = *reinterpret_cast<const uint4 *>(q + int64_t(i * kRows) * ld);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            *slot_at<E>(slot, r0 + i * kRows, c) = v[i];
    } else {
        move_by_element<false>(slot, p, ld, rows, cols);
    }
}

// A written slot to the output: one TMA store (which leaves out what is past
// the matrix), or element by element.
template <typename E>
__device__ __forceinline__ void store_slot(uint8_t *slot, const CUtensorMap *map, void *out,
                                           int64_t m0, int n0, int64_t ld, int rows, int cols,
                                           bool vec)
{
    if (vec) {
        fence_proxy_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            tma_store_2d(map, slot, n0, int(m0));
            bulk_commit();
        }
    } else {
        __syncwarp();
        move_by_element<true>(slot, static_cast<E *>(out) + m0 * ld + n0, ld, rows, cols);
        __syncwarp();
    }
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int f16)
{
    if (f16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack16(uint32_t v, int f16)
{
    if (f16)
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// One warp's memory for the epilogue: two slots, used in turn, and 32 floats
// of bias.
struct EpiMemory {
    uint8_t *slots;
    uint32_t bytes;  // of a slot
    float *bias;
    uint32_t turn;
    bool strict;  // the last store may have been from the next slot

    // The next slot, once the store that last read it is done with it: only
    // the last store may still be reading, its own slot being the other one.
    __device__ __forceinline__ uint8_t *take()
    {
        if ((threadIdx.x & 31) == 0) {
            if (strict)
                bulk_wait_read<0>();
            else
                bulk_wait_read<1>();
        }
        __syncwarp();
        uint8_t *s = slots + (turn & 1u) * bytes;
        ++turn;
        return s;
    }
};

// A row's kCols 16-bit values, from column h of a slot on.
__device__ __forceinline__ void put16(uint8_t *slot, int h, const float (&v)[kCols], int f16)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i)
        *slot_at<uint16_t>(slot, lane, h / 8 + i) = make_uint4(
            pack16(v[8 * i], v[8 * i + 1], f16), pack16(v[8 * i + 2], v[8 * i + 3], f16),
            pack16(v[8 * i + 4], v[8 * i + 5], f16), pack16(v[8 * i + 6], v[8 * i + 7], f16));
}

// The epilogue of 32 rows (lane = row) x kCols columns, from column h of the
// slots on: factor, bias (`bias`: theirs), pre, activation, residual (in
// `slot`), output.
template <bool EXTRA>
__device__ __forceinline__ void pair_cols(uint32_t flags, const float *mul, const float *bias,
                                          uint8_t *pre, uint8_t *slot, int h, float (&v)[kCols])
{
    const int lane = threadIdx.x & 31;
    const int f16 = flags & kEpiF16;
    if (EXTRA && (flags & kEpiMul)) {
        const float m = *mul;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            v[j] *= m;
    }
    if (flags & kEpiBias) {
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(bias + j);
            v[j] += q.x, v[j + 1] += q.y, v[j + 2] += q.z, v[j + 3] += q.w;
        }
    }
    if (flags & kEpiPre)
        put16(pre, h, v, f16);
    if (flags >= kEpiAct)
        with_act(int(flags / kEpiAct), [&](auto act) { act_all<decltype(act)::value>(v); });
    if (flags & kEpiF32) {
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
            float4 *at = reinterpret_cast<float4 *>(slot_at<float>(slot, lane, (h + i) / 4));
            if (flags & kEpiResidual) {
                const float4 q = *at;
                v[i] += q.x, v[i + 1] += q.y, v[i + 2] += q.z, v[i + 3] += q.w;
            }
            *at = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else {
        if (flags & kEpiResidual) {
#pragma unroll
            for (int i = 0; i < kCols; i += 8) {
                const uint4 q = *slot_at<uint16_t>(slot, lane, (h + i) / 8);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack16(w[j], f16);
                    v[i + 2 * j] += f.x;
                    v[i + 2 * j + 1] += f.y;
                }
            }
        }
        put16(slot, h, v, f16);
    }
}

// Adds (or, first, copies) columns c .. c + 31, c + 64 .. of an accumulator to
// the sum of the earlier chains; whole warp, its 32 lanes of tensor memory.  Not inlined: the
// epilogue's registers are its loop's.
__device__ __noinline__ void add_chain(uint32_t acc, uint32_t sum, int c, int width, bool add)
{
#pragma unroll 1
    for (; c < width; c += 32 * kPairParts) {
        uint32_t r[32], o[32];
        tmem_ld_32x32b_x32(acc + uint32_t(c), r);
        if (add)
            tmem_ld_32x32b_x32(sum + uint32_t(c), o);
        tmem_ld_wait();
        if (add) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(o[j]));
        }
        tmem_store_32x32b_x32(sum + uint32_t(c), r);
    }
    tmem_store_wait();
}

// ---- host ---------------------------------------------------------------------

// Outputs [rows, cols], rows ld elements apart, written 32 x 32 from a slot.
cudaError_t out_map(CUtensorMap *m, void *out, int64_t rows, int64_t cols, int64_t ld, int f32,
                    int f16)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
    const CUresult r =
        encode(m,
               f32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
               : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

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

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline size_t align256(size_t b)
{
    return (b + 255) & ~size_t(255);
}

// whether 16-byte pieces of rows `ld` apart are aligned accesses (so are groups of four)
inline int vec16(const void *p, int64_t ld, int size)
{
    return ld * size % 16 == 0 && aligned(p, 16);
}

}  // namespace
}  // namespace moe
