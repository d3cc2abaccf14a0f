// The router: logits -> top-k experts, weights, counts and the balance and z
// losses (moe_route), and their gradient (moe_route_grad).
//
// Mathematics.  A token's open experts have logits l_e.  The softmax mode's
// probabilities are e^(l-m) / sum e^(l-m) with m the row's maximum; the sigmoid
// mode's are s / sum s with s = sigmoid(l).  The latter ratio is formed from
// s' = s * e^(-c), c = min(m, 0), which cannot underflow for the largest
// entry:  l >= 0: s' = 1 / (1 + e^-l) (c is 0 then),
//         l < 0:  s' = e^(l-c) / (1 + e^l).
// Renormalised weights are the same ratio over the chosen experts alone, with
// the maximum of their own logits, so a selection bias that picks experts far
// below the row's maximum loses nothing.
//
// Every token's row is read once into registers by one warp (E <= 512) or one
// CTA (larger E); statistics, choice and weights come from there.
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxCtas = 304;  // rows of partial sums in the workspace
constexpr int kFinalThreads = 1024;

struct RouteArgs {
    const void *logits;
    const float *bias;     // may be null
    const uint8_t *mask;   // may be null
    int32_t *ids;
    float *w;
    float *part_prob;    // [grid][E] sums of p over the CTA's tokens
    int32_t *part_count; // [grid][E]
    float4 *part_scal;   // [grid] {sum lse^2, live tokens, status bits, -}
    int64_t ld;
    int T, E, k;
    int sigmoid, norm, stats;
    float scale;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename L>
__device__ __forceinline__ L from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// Floats as unsigned integers in the same order (-0 as +0, so that the two
// tie); 0 is below every float and marks a closed expert.
__device__ __forceinline__ uint32_t key_of(float v)
{
    uint32_t b = __float_as_uint(v);
    if (b == 0x80000000u)
        b = 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// sigmoid(l) e^(-c) with c = min(row maximum, 0), see the top of this file.
__device__ __forceinline__ float sig_scaled(float l, float c)
{
    const float e = __expf(-fabsf(l));
    const float num = l >= 0.0f ? 1.0f : c == 0.0f ? e : __expf(l - c);
    return __fdividef(num, 1.0f + e);
}

// Reductions over the group of W warps that holds one token's row.  W > 1:
// the group is the CTA; `red` is double-buffered so that one barrier per
// reduction is enough.
template <int W>
struct Group {
    uint2 (*red)[W];
    int buf = 0;

    __device__ __forceinline__ void sync()
    {
        if (W == 1)
            __syncwarp();
        else
            __syncthreads();
    }

    // largest key of the group and the lowest e that has it
    __device__ __forceinline__ uint32_t best(uint32_t key, int &e)
    {
        const uint32_t km = __reduce_max_sync(kFull, key);
        uint32_t em = __reduce_min_sync(kFull, key == km ? uint32_t(e) : 0xffffffffu);
        uint32_t kk = km;
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf][threadIdx.x >> 5] = make_uint2(km, em);
            __syncthreads();
            uint2 b = red[buf][0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                const uint2 o = red[buf][i];
                if (o.x > b.x || (o.x == b.x && o.y < b.y))
                    b = o;
            }
            buf ^= 1;
            kk = b.x;
            em = b.y;
        }
        e = int(em);
        return kk;
    }

    __device__ __forceinline__ float sum(float v)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(kFull, v, o);
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf][threadIdx.x >> 5].x = __float_as_uint(v);
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i)
                v += __uint_as_float(red[buf][i].x);
            buf ^= 1;
        }
        return v;
    }
};

// Dynamic shared memory: per group the chosen experts (id, logit), then
// counts and probability sums of the CTA's tokens.
size_t route_smem(int E, int k, int W)
{
    return size_t(kRouteWarps / W) * k * 8 + size_t(E) * 8;
}

// One token per group of W warps at a time; lane i of the group holds experts
// i, i + 32W, ... (V of them).  Choosing: k rounds of the group's largest
// key; the holder then drops it.
template <typename L, int V, int W>
__global__ void __launch_bounds__(kRouteThreads) k_route(const RouteArgs p)
{
    constexpr int G = 32 * W;                 // threads of a group
    constexpr int kGroups = kRouteWarps / W;  // groups of the CTA
    extern __shared__ uint8_t smem[];
    __shared__ uint2 red[2][W];
    __shared__ uint32_t s_flags;
    __shared__ int s_live;
    __shared__ float s_z[kGroups];
    const int g = threadIdx.x / G, lane = threadIdx.x % G;
    int *sel_e = reinterpret_cast<int *>(smem) + g * p.k;
    float *sel_l = reinterpret_cast<float *>(smem) + kGroups * p.k + g * p.k;
    int *cnt = reinterpret_cast<int *>(smem) + 2 * kGroups * p.k;
    float *ps = reinterpret_cast<float *>(cnt + p.E);
    Group<W> gr{red};
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
        cnt[e] = 0;
        ps[e] = 0.0f;
    }
    if (threadIdx.x == 0) {
        s_flags = 0;
        s_live = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    const L *logits = static_cast<const L *>(p.logits);
    float bias[V], acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + G * i;
        bias[i] = p.bias && e < p.E ? p.bias[e] : 0.0f;
        acc[i] = 0.0f;
    }
    const bool need_p = p.stats || (!p.norm && !p.sigmoid) || (p.bias && !p.sigmoid);
    bool bad = false;
    int live = 0;
    float zsum = 0.0f;

    for (int64_t t = int64_t(blockIdx.x) * kGroups + g; t < p.T;
         t += int64_t(gridDim.x) * kGroups) {
        int32_t *ids = p.ids + t * p.k;
        float *w = p.w + t * p.k;
        float l[V];
        uint32_t key[V], kmax = 0;
        const bool masked = p.mask && !p.mask[t];
        if (!masked) {
            const L *row = logits + t * p.ld;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + G * i;
                l[i] = e < p.E ? to_f(row[e]) : -INFINITY;
            }
            uint32_t own = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(l[i] < INFINITY)) {  // NaN or +inf: closed, and reported
                    bad = true;
                    l[i] = -INFINITY;
                }
                key[i] = l[i] > -INFINITY ? key_of(l[i]) : 0u;
                own = max(own, key[i]);
            }
            int e = 0;
            kmax = gr.best(own, e);
        }
        if (kmax == 0) {  // takes no part
            for (int j = lane; j < p.k; j += G) {
                ids[j] = -1;
                w[j] = 0.0f;
            }
            continue;
        }
        const float m = of_key(kmax);
        const float c = p.sigmoid ? fminf(m, 0.0f) : 0.0f;
        float inv = 0.0f;
        if (need_p) {
            float s[V], sum = 0.0f, sume = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float ex = __expf(l[i] - m);  // 0 for closed experts
                s[i] = !p.sigmoid ? ex : key[i] ? sig_scaled(l[i], c) : 0.0f;
                sum += s[i];
                sume += ex;
            }
            sum = gr.sum(sum);
            inv = 1.0f / sum;
            if (p.stats) {
                if (p.sigmoid)
                    sume = gr.sum(sume);
                else
                    sume = sum;
                const float lse = m + logf(sume);
                zsum += lse * lse;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] += s[i] * inv;
            }
            if (p.bias && !p.sigmoid) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i])
                        key[i] = key_of(s[i] * inv + bias[i]);
            }
        }
        if (p.bias && p.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i])
                    key[i] = key_of(sig_scaled(l[i], 0.0f) + bias[i]);
        }
        ++live;

        uint32_t bk = 0;
        int be = 0;
        auto rescan = [&] {
            bk = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > bk) {
                    bk = key[i];
                    be = lane + G * i;
                }
        };
        rescan();
        int n = 0;
        for (; n < p.k; ++n) {
            int e = be;
            if (gr.best(bk, e) == 0)
                break;
            if (e % G == lane) {
                sel_e[n] = e;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e == lane + G * i) {
                        key[i] = 0;
                        sel_l[n] = l[i];
                    }
                rescan();
            }
        }
        gr.sync();
        uint32_t own = 0;
        for (int j = lane; j < n; j += G)
            own = max(own, key_of(sel_l[j]));
        int e = 0;
        const float ms = of_key(gr.best(own, e));
        const float cs = fminf(ms, 0.0f);
        float mul = p.scale;
        if (p.norm) {
            float sum = 0.0f;
            for (int j = lane; j < n; j += G)
                sum += p.sigmoid ? sig_scaled(sel_l[j], cs) : __expf(sel_l[j] - ms);
            mul = p.scale / gr.sum(sum);
        } else if (!p.sigmoid) {
            mul = p.scale * inv;
        }
        for (int j = lane; j < p.k; j += G) {
            float v = 0.0f;
            int id = -1;
            if (j < n) {
                id = sel_e[j];
                v = mul * (p.sigmoid ? sig_scaled(sel_l[j], p.norm ? cs : 0.0f)
                                     : __expf(sel_l[j] - (p.norm ? ms : m)));
                if (p.stats)
                    atomicAdd(&cnt[id], 1);
            }
            ids[j] = id;
            w[j] = v;
        }
        gr.sync();  // sel_* is written again for the next token
    }

    if (bad)
        atomicOr(&s_flags, MOE_STATUS_BAD_LOGIT);
    if (lane == 0) {
        atomicAdd(&s_live, live);
        s_z[g] = zsum;
    }
    // the groups' probability sums, added in the groups' order
    for (int q = 0; q < kGroups && p.stats; ++q) {
        if (g == q) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + G * i < p.E)
                    ps[lane + G * i] += acc[i];
        }
        __syncthreads();
    }
    __syncthreads();
    if (p.stats)
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            p.part_prob[int64_t(blockIdx.x) * p.E + e] = ps[e];
            p.part_count[int64_t(blockIdx.x) * p.E + e] = cnt[e];
        }
    if (threadIdx.x == 0) {
        float z = 0.0f;
        for (int q = 0; q < kGroups; ++q)
            z += s_z[q];
        p.part_scal[blockIdx.x] =
            make_float4(z, __int_as_float(s_live), __uint_as_float(s_flags), 0.0f);
    }
}

struct FinalArgs {
    const float *part_prob;
    const int32_t *part_count;
    const float4 *part_scal;
    uint32_t *status;
    int32_t *counts;  // each may be null
    float *prob;
    float *loss;
    int E, k, parts, stats;
};

__device__ __forceinline__ float block_sum(float v, float *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < int(blockDim.x >> 5); ++i)
        v += red[i];
    return v;
}

// The partial sums of k_route's CTAs, added in their order: counts, mean
// probabilities, losses and the status word.
__global__ void __launch_bounds__(kFinalThreads) k_route_final(const FinalArgs p)
{
    __shared__ float red[kFinalThreads / 32];
    __shared__ int s_live;
    __shared__ float s_z;
    pdl_wait();
    if (threadIdx.x == 0) {
        int live = 0;
        uint32_t flags = 0;
        float z = 0.0f;
        for (int i = 0; i < p.parts; ++i) {
            const float4 v = p.part_scal[i];
            z += v.x;
            live += __float_as_int(v.y);
            flags |= __float_as_uint(v.z);
        }
        s_live = live;
        s_z = z;
        *p.status = flags;
    }
    __syncthreads();
    if (!p.stats)
        return;
    const float n = float(max(s_live, 1));
    float dot = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kFinalThreads) {
        float s = 0.0f;
        int c = 0;
        for (int i = 0; i < p.parts; ++i) {
            s += p.part_prob[int64_t(i) * p.E + e];
            c += p.part_count[int64_t(i) * p.E + e];
        }
        const float pr = s / n;
        dot += float(c) / (n * float(p.k)) * pr;
        if (p.prob)
            p.prob[e] = pr;
        if (p.counts)
            p.counts[e] = c;
    }
    dot = block_sum(dot, red);
    if (threadIdx.x == 0) {
        if (p.counts)
            p.counts[p.E] = s_live;
        if (p.loss) {
            p.loss[0] = float(p.E) * dot;
            p.loss[1] = s_z / n;
        }
    }
}

struct RouteGradArgs {
    const void *logits;
    const uint8_t *mask;
    const int32_t *ids;
    const int32_t *counts;  // may be null
    const float *dw;        // may be null
    const float *dloss;     // may be null
    void *dlogits;
    int64_t ld, ldd;
    int T, E, k;
    int sigmoid, norm;
    float scale;
};

// G = sum dw w + g0 balance + g1 z.  With p the probabilities, q the chosen
// experts' scores over their sum, n tokens, f_e = counts[e] / (n k):
//   balance:  da_e = p_e (c_e - sum p c),   c_e = g0 E f_e / n
//   norm:     da_j += q_j scale (dw_j - sum q dw)            (chosen j)
//   no norm, softmax:  da_e += s_e (scale dw_e - sum s scale dw)
//   no norm, sigmoid:  da_j += s_j scale dw_j
//   sigmoid:  dl = da sigmoid(-l)           (a = log sigmoid(l))
//   z:        dl_e += 2 g1 lse softmax(l)_e / n
// One pass: the row is read once, its gradient written once.
template <typename L, int V, int W>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(const RouteGradArgs p)
{
    constexpr int G = 32 * W;
    constexpr int kGroups = kRouteWarps / W;
    extern __shared__ uint8_t smem[];
    __shared__ uint2 red[2][W];
    const int g = threadIdx.x / G, lane = threadIdx.x % G;
    float *dsel = reinterpret_cast<float *>(smem) + size_t(g) * p.E;  // by expert; zeros
    Group<W> gr{red};
    for (int e = lane; e < p.E; e += G)
        dsel[e] = 0.0f;
    gr.sync();
    pdl_wait();
    pdl_launch_dependents();

    const L *logits = static_cast<const L *>(p.logits);
    L *out = static_cast<L *>(p.dlogits);
    float cf[V], gz = 0.0f;
    const bool aux = p.counts && p.dloss;
    {
        float c0 = 0.0f;
        if (aux) {
            const float n = float(max(p.counts[p.E], 1));
            c0 = p.dloss[0] * float(p.E) / (n * n * float(p.k));
            gz = 2.0f * p.dloss[1] / n;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + G * i;
            cf[i] = aux && e < p.E ? c0 * float(p.counts[e]) : 0.0f;
        }
    }

    for (int64_t t = int64_t(blockIdx.x) * kGroups + g; t < p.T;
         t += int64_t(gridDim.x) * kGroups) {
        L *orow = out + t * p.ldd;
        const L *row = logits + t * p.ld;
        float l[V];
        uint32_t kmax = 0;
        const bool masked = p.mask && !p.mask[t];
        if (!masked) {
            uint32_t own = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + G * i;
                l[i] = e < p.E ? to_f(row[e]) : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(l[i] < INFINITY))
                    l[i] = -INFINITY;
                own = max(own, l[i] > -INFINITY ? key_of(l[i]) : 0u);
            }
            int e = 0;
            kmax = gr.best(own, e);
        }
        if (kmax == 0) {
            for (int e = lane; e < p.E; e += G)
                orow[e] = from_f<L>(0.0f);
            continue;
        }
        const float m = of_key(kmax);
        const float c = p.sigmoid ? fminf(m, 0.0f) : 0.0f;
        float s[V], sum = 0.0f, sume = 0.0f, pc = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float ex = __expf(l[i] - m);
            s[i] = !p.sigmoid ? ex : l[i] > -INFINITY ? sig_scaled(l[i], c) : 0.0f;
            sum += s[i];
            sume += ex;
            pc += s[i] * cf[i];
        }
        sum = gr.sum(sum);
        sume = p.sigmoid ? gr.sum(sume) : sum;
        const float inv = 1.0f / sum;
        pc = gr.sum(pc) * inv;

        // the chosen experts' share
        float dot = 0.0f;  // no norm, softmax: sum s scale dw
        if (p.dw) {
            const int32_t *ids = p.ids + t * p.k;
            const float *dw = p.dw + t * p.k;
            auto logit_of = [&](int j, int &id) {
                id = ids[j];
                const float v =
                    id >= 0 && id < p.E ? to_f(row[id]) : -INFINITY;
                return v < INFINITY ? v : -INFINITY;
            };
            int id;
            if (p.norm) {
                uint32_t own = 0;
                for (int j = lane; j < p.k; j += G) {
                    const float v = logit_of(j, id);
                    own = max(own, v > -INFINITY ? key_of(v) : 0u);
                }
                int e = 0;
                const uint32_t ks = gr.best(own, e);
                if (ks) {
                    const float ms = of_key(ks), cs = fminf(ms, 0.0f);
                    float sq = 0.0f, sd = 0.0f;
                    for (int j = lane; j < p.k; j += G) {
                        const float v = logit_of(j, id);
                        if (v > -INFINITY) {
                            const float q = p.sigmoid ? sig_scaled(v, cs) : __expf(v - ms);
                            sq += q;
                            sd += q * dw[j];
                        }
                    }
                    const float iq = 1.0f / gr.sum(sq);
                    const float mean = gr.sum(sd) * iq;
                    for (int j = lane; j < p.k; j += G) {
                        const float v = logit_of(j, id);
                        if (v > -INFINITY) {
                            const float q = p.sigmoid ? sig_scaled(v, cs) : __expf(v - ms);
                            dsel[id] = q * iq * p.scale * (dw[j] - mean);
                        }
                    }
                }
            } else {
                for (int j = lane; j < p.k; j += G) {
                    const float v = logit_of(j, id);
                    if (v > -INFINITY) {
                        const float q = p.sigmoid ? sig_scaled(v, 0.0f) : __expf(v - m) * inv;
                        const float d = q * p.scale * dw[j];
                        dsel[id] = d;
                        dot += d;
                    }
                }
                dot = p.sigmoid ? 0.0f : gr.sum(dot);
            }
        }
        gr.sync();
        const float zc = gz * (m + logf(sume)) / sume;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + G * i;
            if (e >= p.E)
                continue;
            float d = s[i] * inv * (cf[i] - pc - dot) + dsel[e];
            if (p.sigmoid)
                d *= __fdividef(1.0f, 1.0f + __expf(l[i]));
            d += zc * __expf(l[i] - m);
            orow[e] = from_f<L>(l[i] > -INFINITY ? d : 0.0f);
        }
        gr.sync();
        if (p.dw)
            for (int j = lane; j < p.k; j += G) {
                const int id = p.ids[t * p.k + j];
                if (id >= 0 && id < p.E)
                    dsel[id] = 0.0f;
            }
        gr.sync();
    }
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline size_t align256(size_t b)
{
    return (b + 255) & ~size_t(255);
}

inline int size_of(int dtype)
{
    return dtype == MOE_DT_F32 ? 4 : 2;
}

int route_sizes(int T, int E, int k, int64_t ld)
{
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || k > E ||
        int64_t(T) * k > INT_MAX || ld < E)
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

// A warp per token up to 512 experts (16 a lane), a CTA per token above.
template <template <typename, int, int> class F, typename... A>
cudaError_t by_shape(int dtype, int E, A &&...a)
{
    auto typed = [&](auto zero) {
        using L = decltype(zero);
        if (E <= 32)
            return F<L, 1, 1>::go(a...);
        if (E <= 64)
            return F<L, 2, 1>::go(a...);
        if (E <= 128)
            return F<L, 4, 1>::go(a...);
        if (E <= 256)
            return F<L, 8, 1>::go(a...);
        if (E <= 512)
            return F<L, 16, 1>::go(a...);
        if (E <= 1024)
            return F<L, 4, kRouteWarps>::go(a...);
        return F<L, 16, kRouteWarps>::go(a...);
    };
    if (dtype == MOE_DT_F32)
        return typed(0.0f);
    if (dtype == MOE_DT_BF16)
        return typed(__nv_bfloat16());
    return typed(__half());
}

int route_grid(int T, int W)
{
    const int per = kRouteWarps / W;
    const int need = int((int64_t(T) + per - 1) / per);
    return std::max(1, std::min({need, 2 * device_sm_count(), kRouteMaxCtas}));
}

template <typename L, int V, int W>
struct LaunchRoute {
    static cudaError_t go(const RouteArgs &a, int &grid, cudaStream_t s)
    {
        grid = route_grid(a.T, W);
        return launch_pdl(k_route<L, V, W>, dim3(grid), dim3(kRouteThreads),
                          route_smem(a.E, a.k, W), s, a);
    }
};

template <typename L, int V, int W>
struct LaunchRouteGrad {
    static cudaError_t go(const RouteGradArgs &a, cudaStream_t s)
    {
        return launch_pdl(k_route_grad<L, V, W>, dim3(route_grid(a.T, W)), dim3(kRouteThreads),
                          size_t(kRouteWarps / W) * a.E * 4, s, a);
    }
};

}  // namespace
}  // namespace moe

extern "C" size_t moe_route_workspace_bytes(int T, int E)
{
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS)
        return 0;
    const size_t rows = std::min(std::max(T, 1), moe::kRouteMaxCtas);
    return 256 + moe::align256(rows * sizeof(float4)) + moe::align256(rows * E * 8);
}

extern "C" int moe_route(const void *logits, int64_t ld, int l_dtype, const float *bias,
                         const uint8_t *mask, int T, int E, int k, int score, int norm,
                         float scale, int32_t *ids, float *w, int32_t *counts, float *prob,
                         float *loss, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    using namespace moe;
    if (l_dtype != MOE_DT_F32 && l_dtype != MOE_DT_BF16 && l_dtype != MOE_DT_F16)
        return MOE_ERR_DTYPE;
    const int rc = route_sizes(T, E, k, ld);
    if (rc != MOE_OK)
        return rc;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
        return MOE_ERR_SHAPE;
    if (!ws || (T > 0 && (!logits || !ids || !w)))
        return MOE_ERR_NULL;
    if (ws_bytes < moe_route_workspace_bytes(T, E))
        return MOE_ERR_WORKSPACE;
    if (!aligned(logits, size_of(l_dtype)) || !aligned(bias, 4) || !aligned(ids, 4) ||
        !aligned(w, 4) || !aligned(counts, 4) || !aligned(prob, 4) || !aligned(loss, 4) ||
        !aligned(ws, 256))
        return MOE_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t rows = std::min(std::max(T, 1), kRouteMaxCtas);
    uint8_t *b = static_cast<uint8_t *>(ws);
    float4 *scal = reinterpret_cast<float4 *>(b + 256);
    float *pp = reinterpret_cast<float *>(b + 256 + align256(rows * sizeof(float4)));
    int32_t *pc = reinterpret_cast<int32_t *>(pp + rows * E);
    const int stats = counts || prob || loss;
    const RouteArgs a{logits, bias, mask, ids, w, pp, pc, scal, ld, T, E, k,
                      score == MOE_SCORE_SIGMOID, norm != 0, stats, scale};
    int grid = 1;
    cudaError_t e = by_shape<LaunchRoute>(l_dtype, E, a, grid, s);
    if (e != cudaSuccess)
        return MOE_ERR_CUDA;
    const FinalArgs f{pp, pc, scal, reinterpret_cast<uint32_t *>(ws), counts, prob, loss,
                      E, k, grid, stats};
    e = launch_pdl(k_route_final, dim3(1), dim3(kFinalThreads), 0, s, f);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_route_grad(const void *logits, int64_t ld, int l_dtype, const uint8_t *mask,
                              const int32_t *ids, const int32_t *counts, const float *dw,
                              const float *dloss, int T, int E, int k, int score, int norm,
                              float scale, void *dlogits, int64_t ldd, moe_stream_t stream)
{
    using namespace moe;
    if (l_dtype != MOE_DT_F32 && l_dtype != MOE_DT_BF16 && l_dtype != MOE_DT_F16)
        return MOE_ERR_DTYPE;
    const int rc = route_sizes(T, E, k, ld);
    if (rc != MOE_OK)
        return rc;
    if ((score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || ldd < E)
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!logits || !ids || !dlogits)
        return MOE_ERR_NULL;
    if (!aligned(logits, size_of(l_dtype)) || !aligned(dlogits, size_of(l_dtype)) ||
        !aligned(ids, 4) || !aligned(counts, 4) || !aligned(dw, 4) || !aligned(dloss, 4))
        return MOE_ERR_ALIGN;
    const RouteGradArgs a{logits, mask, ids, counts, dw, dloss, dlogits, ld, ldd, T, E, k,
                          score == MOE_SCORE_SIGMOID, norm != 0, scale};
    return by_shape<LaunchRouteGrad>(l_dtype, E, a, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
