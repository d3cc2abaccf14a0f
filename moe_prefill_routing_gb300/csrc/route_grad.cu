// The gradient of the router's weights and losses (moe_route_grad).  The
// scores and their ratios: route.cuh.
//
// G = sum dw w + g0 balance + g1 z.  With p the probabilities, a the log
// scores, q the chosen experts' scores over their sum, n tokens and
// f_e = counts[e] / (n k):
//   balance:           da_e  = p_e (c_e - sum p c),   c_e = g0 E f_e / n
//   norm:              da_j += q_j scale (dw_j - sum q dw)            (chosen j)
//   no norm, softmax:  da_e += s_e (scale dw_e - sum s scale dw)
//   no norm, sigmoid:  da_j += s_j scale dw_j
//   sigmoid:           dl_e  = da_e sigmoid(-l_e)      (a = log sigmoid(l))
//   z:                 dl_e += 2 g1 lse softmax(l)_e / n
// One pass: a token's row is read once (a token ahead), its gradient written
// once; the weights' part is k values a token, set out by expert in shared
// memory.
//
// 32768 tokens x 256 experts, bf16: 14.7 us, 2.4 TB/s of the 35.7 MB it moves;
// bound by instructions (some 330 a token, six tenths of the issue slots; the
// rest waits for loads and reductions).  2048 x 512, fp32: 3.7 us, launch and
// one token's latency.
#include "route.cuh"

namespace moe {
namespace {

using namespace route;

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;

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
    int sigmoid, norm, f16;
    float scale;
};

// Sums of N values over a group; every lane gets them.
template <int N, int W>
__device__ __forceinline__ void sum_all(float (&v)[N], Group<W> &gr)
{
    if constexpr (W == 1) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += __shfl_xor_sync(kFull, v[i], o);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = gr.sum(v[i]);
    }
}

// CTAs that an SM holds at once, by registers; the grid is as many (eight an
// SM, 2.7 rounds of them, took 16.2 us instead of 13.9, four of 128 experts
// are 8 % faster than three)
template <int V, int J>
constexpr int kGradResident = V >= 16 || J > 1 ? 2 : V >= 8 ? 3 : 4;

// J: slots of a lane (k <= 32 W J).
template <typename L, int V, int W, int C, int J>
__global__ void __launch_bounds__(kGradThreads, kGradResident<V, J>)
    k_route_grad(const RouteGradArgs p)
{
    constexpr int G = 32 * W;
    constexpr int kGroups = kGradWarps / W;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint2 red[W > 1 ? kGroups : 1][2][W];
    const int g = threadIdx.x / G, lane = threadIdx.x % G;
    const int E4 = (p.E + 3) & ~3;
    float *dsel = reinterpret_cast<float *>(smem) + size_t(g) * E4;  // by expert; zeros
    Group<W> gr{red[W > 1 ? g : 0]};
    for (int e = lane; e < p.E; e += G)
        dsel[e] = 0.0f;
    gr.sync();
    pdl_wait();
    pdl_launch_dependents();

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
            const int e = expert_of<C, G>(lane, i);
            cf[i] = aux && e < p.E ? c0 * float(p.counts[e]) : 0.0f;
        }
    }

    // what a token's gradient is made from, loaded one token ahead
    RawRow<L, V, C, G> raw;
    int id[J];    // the lane's slots: expert (-1: none) and scale dw
    float d[J];
    bool on;
    int64_t t = int64_t(blockIdx.x) * kGroups + g;
    const int64_t step = int64_t(gridDim.x) * kGroups;
    const L *row = static_cast<const L *>(p.logits) + t * p.ld;
    L *orow = static_cast<L *>(p.dlogits) + t * p.ldd;
    auto fetch = [&](int64_t at, const L *from) {
        on = !p.mask || p.mask[at];
        raw.load(from, lane, p.E);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int slot = lane + G * j;
            id[j] = p.dw && slot < p.k ? p.ids[at * p.k + slot] : -1;
            d[j] = p.dw && slot < p.k ? p.scale * p.dw[at * p.k + slot] : 0.0f;
        }
    };
    if (t < p.T)
        fetch(t, row);
    for (; t < p.T; t += step, row += step * p.ld, orow += step * p.ldd) {
        float l[V], v[J], dj[J];
        int e[J];
        raw.to(l, lane, p.E, p.f16);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            e[j] = on ? id[j] : -1;
            // the slot's logit (read again: this lane need not hold it)
            v[j] = uint32_t(e[j]) < uint32_t(p.E) ? to_f(row[e[j]], p.f16) : -INFINITY;
            if (!(v[j] < INFINITY))
                v[j] = -INFINITY;
            // a slot without weight may hold anything, and 0 times a NaN is one
            dj[j] = v[j] > -INFINITY ? d[j] : 0.0f;
        }
        float own = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!(l[i] < INFINITY))
                l[i] = -INFINITY;
            own = fmaxf(own, l[i]);
        }
        const uint32_t kmax = on ? gr.largest(key_of(own)) : kClosed;
        if (t + step < p.T)
            fetch(t + step, row + step * p.ld);
        if (kmax == kClosed) {  // takes no part
#pragma unroll
            for (int i = 0; i < V; ++i)
                l[i] = 0.0f;
            store_row<L, V, C, G>(l, orow, lane, p.E, p.f16);
            continue;
        }
        const float m = of_key(kmax);
        const float c = p.sigmoid ? fminf(m, 0.0f) : 0.0f;
        float s[V];
        enum { kS, kP, kQ, kD, kE, kSums };  // sums: s, s c, q, q dw, e^(l-m)
        float sums[kSums] = {};
        if (p.sigmoid) {
            sig_scaled(s, l, c);
#pragma unroll
            for (int i = 0; i < V; ++i)
                sums[kE] += exp_ftz(l[i] - m);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] = exp_ftz(l[i] - m);  // 0 for closed experts
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sums[kS] += s[i];
            sums[kP] += s[i] * cf[i];
        }
        // the chosen experts' scores: over their own maximum, or as they are
        float q[J], ms = m, cs = 0.0f;
        if (p.dw && p.norm) {
            uint32_t o = kClosed;
#pragma unroll
            for (int j = 0; j < J; ++j)
                o = max(o, key_of(v[j]));
            ms = of_key(gr.largest(o));  // -inf where no slot has weight
            cs = fminf(ms, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            q[j] = v[j] == -INFINITY ? 0.0f
                   : p.sigmoid       ? sig_scaled(v[j], cs)
                                     : exp_ftz(v[j] - ms);
            sums[kQ] += q[j];
            sums[kD] += q[j] * dj[j];
        }
        if (p.sigmoid) {
            sum_all(sums, gr);
        } else if (aux && p.dw) {
            float four[4] = {sums[kS], sums[kP], sums[kQ], sums[kD]};
            sum_all(four, gr);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sums[i] = four[i];
        } else {  // without counts or without dw two of them are 0
            float three[3] = {sums[kS], aux ? sums[kP] : sums[kQ], sums[kD]};
            sum_all(three, gr);
            sums[kS] = three[0];
            (aux ? sums[kP] : sums[kQ]) = three[1];
            sums[kD] = three[2];
        }
        const float inv = rcp_ftz(sums[kS]);
        const float sume = p.sigmoid ? sums[kE] : sums[kS];
        float mul = p.sigmoid ? 1.0f : inv, mean = 0.0f, base = sums[kP] * inv;
        if (p.norm) {
            mul = sums[kQ] > 0.0f ? rcp_ftz(sums[kQ]) : 0.0f;
            mean = sums[kD] * mul;
        } else if (!p.sigmoid) {
            base += sums[kD] * inv;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (v[j] > -INFINITY) {
                // (a slot whose score is all of the sum has a constant weight:
                // exactly 0, not what the reciprocal's rounding leaves of dw)
                const bool alone = p.norm && q[j] == sums[kQ];
                dsel[e[j]] = alone ? 0.0f : q[j] * mul * (dj[j] - mean);
            }
        gr.sync();
        const float zc = gz * (m + __logf(sume)) * rcp_ftz(sume);
        float ds[V];
#pragma unroll
        for (int i = 0; i < V; i += C) {
            const int x = expert_of<C, G>(lane, i);
            if constexpr (C >= 4) {
#pragma unroll
                for (int h = 0; h < C; h += 4) {
                    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (x < p.E)
                        f = *reinterpret_cast<const float4 *>(dsel + x + h);
                    ds[i + h] = f.x, ds[i + h + 1] = f.y, ds[i + h + 2] = f.z, ds[i + h + 3] = f.w;
                }
            } else {
                ds[i] = x < p.E ? dsel[x] : 0.0f;
            }
        }
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float da = s[i] * inv * (cf[i] - base) + ds[i];
                const float o = da * rcp_ftz(1.0f + exp_ftz(l[i])) + zc * exp_ftz(l[i] - m);
                l[i] = l[i] > -INFINITY ? o : 0.0f;
            }
        } else {  // s, ds and with them the gradient are 0 for closed experts
            const float z0 = zc - inv * base;
            // (a second loop cost several warps a token more than the selection:
            // 4096 x 2048 31.5 us, 30.4 so; for one warp it is the other way round)
            if (W == 1 && fabsf(z0) < INFINITY) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    l[i] = s[i] * (inv * cf[i] + z0) + ds[i];
            } else {  // dloss or dw overflowed: no 0 times infinity for those
#pragma unroll
                for (int i = 0; i < V; ++i)
                    l[i] = s[i] > 0.0f ? s[i] * (inv * cf[i] + z0) + ds[i] : ds[i];
            }
        }
        store_row<L, V, C, G>(l, orow, lane, p.E, p.f16);
        gr.sync();
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (v[j] > -INFINITY)
                dsel[e[j]] = 0.0f;
        gr.sync();
    }
}

}  // namespace
}  // namespace moe

extern "C" int moe_route_grad(const void *logits, int64_t ld, int l_dtype, const uint8_t *mask,
                              const int32_t *ids, const int32_t *counts, const float *dw,
                              const float *dloss, int T, int E, int k, int score, int norm,
                              float scale, void *dlogits, int64_t ldd, moe_stream_t stream)
{
    using namespace moe;
    const int rc = check_sizes(l_dtype, T, E, k, ld, score);
    if (rc != MOE_OK)
        return rc;
    if (ldd < E)
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!logits || !ids || !dlogits)
        return MOE_ERR_NULL;
    const int size = size_of(l_dtype);
    if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(ids, 4) ||
        !aligned(counts, 4) || !aligned(dw, 4) || !aligned(dloss, 4))
        return MOE_ERR_ALIGN;
    RouteGradArgs a = {};
    a.logits = logits, a.mask = mask, a.ids = ids, a.counts = counts, a.dw = dw, a.dloss = dloss;
    a.dlogits = dlogits, a.ld = ld, a.ldd = ldd, a.T = T, a.E = E, a.k = k;
    a.sigmoid = score == MOE_SCORE_SIGMOID, a.norm = norm != 0, a.f16 = l_dtype == MOE_DT_F16;
    a.scale = scale;
    const cudaError_t e = by_shape<kGradWarps>(
        l_dtype, E,
        [&](int c) {
            return E % c == 0 && ld % c == 0 && ldd % c == 0 && aligned(logits, c * size) &&
                   aligned(dlogits, c * size);
        },
        [&](auto l, auto v, auto w, auto c) {
            constexpr int V = decltype(v)::value, W = decltype(w)::value, C = decltype(c)::value;
            using L = decltype(l);
            const int per = kGradWarps / W;
            constexpr int kMany = (MOE_MAX_TOPK + 32 * W - 1) / (32 * W);
            const bool one = k <= 32 * W;  // one slot a lane
            auto kern = one ? k_route_grad<L, V, W, C, 1> : k_route_grad<L, V, W, C, kMany>;
            const int resident = one ? kGradResident<V, 1> : kGradResident<V, kMany>;
            const int grid = std::min((T - 1) / per + 1, resident * device_sm_count());
            return launch_pdl(kern, dim3(grid), dim3(kGradThreads),
                              size_t(per) * ((E + 3) & ~3) * 4, reinterpret_cast<cudaStream_t>(stream), a);
        });
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
