// What the router's forward and gradient kernels share: which logits a lane
// holds, reductions over the lanes that hold one token's row, and the scores.
//
// A token's open experts have logits l_e.  The softmax mode's probabilities
// are e^(l-m) / sum e^(l-m) with m the row's maximum; the sigmoid mode's are
// s / sum s with s = sigmoid(l).  The latter ratio is formed from
// s' = s e^(-c), c = min(m, 0), which cannot underflow for the largest entry:
//   l >= 0: s' = 1 / (1 + e^-l)  (c is 0 then),   l < 0: s' = e^(l-c) / (1 + e^l).
// Renormalised weights are the same ratio over the chosen experts alone, with
// the maximum of their own logits, so a selection bias that picks experts far
// below the row's maximum loses nothing.
#pragma once

#include "../../include/moe_prefill.h"
#include "internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

namespace moe {
namespace route {

constexpr uint32_t kFull = 0xffffffffu;

// L is float, or uint16_t for bf16 and fp16 values (f16 says which).
__device__ __forceinline__ float to_f(float v, int) { return v; }
__device__ __forceinline__ float to_f(uint16_t v, int f16)
{
    return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(uint32_t(v) << 16);
}
__device__ __forceinline__ void from_f(float v, float &o, int) { o = v; }
__device__ __forceinline__ void from_f(float v, uint16_t &o, int f16)
{
    o = f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// e^x and 1/x of normal numbers, results below 2^-126 as 0: one multiply and
// one special-function instruction (2 units in the last place, plus the
// rounding of x log2(e) for the exponential).
__device__ __forceinline__ float exp_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

__device__ __forceinline__ float rcp_ftz(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Floats as unsigned integers in the same order (-0 as +0, so that the two
// tie).  -inf marks a closed expert; its key is below that of every number.
constexpr uint32_t kClosed = 0x007fffffu;

__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// sigmoid(l) e^(-c) with c = min(row maximum, 0), see the top of this file;
// 0 for l = -inf.
__device__ __forceinline__ float sig_scaled(float l, float c)
{
    const float e = exp_ftz(-fabsf(l));
    const float num = l >= 0.0f ? 1.0f : exp_ftz(l - c);
    return num * rcp_ftz(1.0f + e);
}

// The same of a lane's logits.  Where the row's maximum is not negative (c is
// 0 in every lane) nothing is lost in the plain form, a third of the work.
template <int V>
__device__ __forceinline__ void sig_scaled(float (&s)[V], const float (&l)[V], float c)
{
    if (c == 0.0f) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i] = rcp_ftz(1.0f + exp_ftz(-l[i]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i] = sig_scaled(l[i], c);
    }
}

// The experts of a lane in a group of G lanes: C neighbouring ones at a time
// (one 8- or 16-byte access, or one element); expert_of grows with i.
template <int C, int G>
__device__ __forceinline__ int expert_of(int lane, int i)
{
    return (i / C) * (G * C) + lane * C + i % C;
}

template <int BYTES>
struct Vec;
template <>
struct Vec<2> {
    using type = uint16_t;
};
template <>
struct Vec<4> {
    using type = uint32_t;
};
template <>
struct Vec<8> {
    using type = uint2;
};
template <>
struct Vec<16> {
    using type = uint4;
};

// A lane's V logits of a row as they are stored.  C > 1: E, the distance of
// rows and the base are multiples of C elements.
template <typename L, int V, int C, int G>
struct RawRow {
    using Q = typename Vec<C * int(sizeof(L))>::type;
    static_assert(V % C == 0, "whole accesses");
    union {
        Q q;
        L v[C];
    } u[V / C];

    __device__ __forceinline__ void load(const L *row, int lane, int E)
    {
#pragma unroll
        for (int i = 0; i < V / C; ++i) {
            const int e = expert_of<C, G>(lane, i * C);
            u[i].q = Q{};
            if (e < E)
                u[i].q = *reinterpret_cast<const Q *>(row + e);
        }
    }

    // as floats, -inf past E
    __device__ __forceinline__ void to(float (&l)[V], int lane, int E, int f16) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            l[i] = expert_of<C, G>(lane, i / C * C) < E ? to_f(u[i / C].v[i % C], f16) : -INFINITY;
    }
};

template <typename L, int V, int C, int G>
__device__ __forceinline__ void store_row(const float (&d)[V], L *row, int lane, int E, int f16)
{
    if constexpr (C == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + G * i;
            if (e < E)
                from_f(d[i], row[e], f16);
        }
    } else {
        using Q = typename Vec<C * int(sizeof(L))>::type;
#pragma unroll
        for (int i = 0; i < V / C; ++i) {
            const int e = expert_of<C, G>(lane, i * C);
            union {
                Q q;
                L v[C];
            } u;
#pragma unroll
            for (int c = 0; c < C; ++c)
                from_f(d[i * C + c], u.v[c], f16);
            if (e < E)
                *reinterpret_cast<Q *>(row + e) = u.q;
        }
    }
}

// Reductions over the group of W warps that holds one token's row.  W > 1:
// the CTA's groups have a barrier each; `red` (the group's own) is
// double-buffered so that one barrier per reduction is enough.
template <int W>
struct Group {
    uint2 (*red)[W];
    int buf = 0;

    __device__ __forceinline__ int warp() const { return int(threadIdx.x >> 5) % W; }

    __device__ __forceinline__ void sync()
    {
        if constexpr (W == 1)
            __syncwarp();
        else  // (barrier 0 is the CTA's)
            asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x) / (32 * W)), "n"(32 * W)
                         : "memory");
    }

    // largest key of the group; e becomes the lowest e of those that have it
    __device__ __forceinline__ uint32_t best(uint32_t key, int &e)
    {
        uint32_t km = __reduce_max_sync(kFull, key);
        const uint32_t have = __ballot_sync(kFull, key == km);
        uint32_t em;
        if ((have & (have - 1)) == 0)
            em = uint32_t(__shfl_sync(kFull, e, __ffs(int(have)) - 1));
        else
            em = __reduce_min_sync(kFull, key == km ? uint32_t(e) : 0xffffffffu);
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf][warp()] = make_uint2(km, em);
            sync();
            uint2 b = red[buf][0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                const uint2 o = red[buf][i];
                if (o.x > b.x || (o.x == b.x && o.y < b.y))
                    b = o;
            }
            buf ^= 1;
            km = b.x;
            em = b.y;
        }
        e = int(em);
        return km;
    }

    __device__ __forceinline__ uint32_t largest(uint32_t key)
    {
        uint32_t km = __reduce_max_sync(kFull, key);
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf][warp()].x = km;
            sync();
#pragma unroll
            for (int i = 0; i < W; ++i)
                km = max(km, red[buf][i].x);
            buf ^= 1;
        }
        return km;
    }

    __device__ __forceinline__ float sum(float v)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(kFull, v, o);
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf][warp()].x = __float_as_uint(v);
            sync();
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i)
                v += __uint_as_float(red[buf][i].x);
            buf ^= 1;
        }
        return v;
    }
};

// ---- host ---------------------------------------------------------------------

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int size_of(int dtype)
{
    return dtype == MOE_DT_F32 ? 4 : 2;
}

inline int check_sizes(int l_dtype, int T, int E, int k, int64_t ld, int score)
{
    if (l_dtype != MOE_DT_F32 && l_dtype != MOE_DT_BF16 && l_dtype != MOE_DT_F16)
        return MOE_ERR_DTYPE;
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || k > E ||
        int64_t(T) * k > INT_MAX || ld < E ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

// Calls f<L, V, W, C>(): a warp per token up to 512 experts (V up to 16 a
// lane), four warps up to 2048, a CTA of `Warps` warps above; C elements per
// access where the rows' length, distance and base allow it (`vec(C)`).
template <int Warps, typename Vecs, typename F>
auto by_shape(int dtype, int E, Vecs vec, F f)
{
    using std::integral_constant;
#define MOE_ROUTE_CASE(L, V, W, C)                                                              \
    return f(L(), integral_constant<int, V>(), integral_constant<int, W>(),                     \
             integral_constant<int, C>())
    constexpr int kV = MOE_MAX_EXPERTS / (32 * Warps);
    if (dtype == MOE_DT_F32) {
        if (E <= 32)
            MOE_ROUTE_CASE(float, 1, 1, 1);
        if (E <= 64)
            MOE_ROUTE_CASE(float, 2, 1, 1);
        if (E <= 512 && vec(4)) {
            if (E <= 128)
                MOE_ROUTE_CASE(float, 4, 1, 4);
            if (E <= 256)
                MOE_ROUTE_CASE(float, 8, 1, 4);
            MOE_ROUTE_CASE(float, 16, 1, 4);
        }
        if (E <= 128)
            MOE_ROUTE_CASE(float, 4, 1, 1);
        if (E <= 256)
            MOE_ROUTE_CASE(float, 8, 1, 1);
        if (E <= 512)
            MOE_ROUTE_CASE(float, 16, 1, 1);
        if (E <= 1024)
            MOE_ROUTE_CASE(float, 8, 4, 1);
        if (E <= 2048)
            MOE_ROUTE_CASE(float, 16, 4, 1);
        MOE_ROUTE_CASE(float, kV, Warps, 1);
    }
    if (E <= 32)
        MOE_ROUTE_CASE(uint16_t, 1, 1, 1);
    if (E <= 64)
        MOE_ROUTE_CASE(uint16_t, 2, 1, 1);
    if (E <= 128 && vec(4))
        MOE_ROUTE_CASE(uint16_t, 4, 1, 4);
    if (E <= 128)
        MOE_ROUTE_CASE(uint16_t, 4, 1, 1);
    if (E <= 512 && vec(8)) {
        if (E <= 256)
            MOE_ROUTE_CASE(uint16_t, 8, 1, 8);
        MOE_ROUTE_CASE(uint16_t, 16, 1, 8);
    }
    if (E <= 256)
        MOE_ROUTE_CASE(uint16_t, 8, 1, 1);
    if (E <= 512)
        MOE_ROUTE_CASE(uint16_t, 16, 1, 1);
    if (E <= 1024)
        MOE_ROUTE_CASE(uint16_t, 8, 4, 1);
    if (E <= 2048)
        MOE_ROUTE_CASE(uint16_t, 16, 4, 1);
    MOE_ROUTE_CASE(uint16_t, kV, Warps, 1);
#undef MOE_ROUTE_CASE
}

}  // namespace route
}  // namespace moe
