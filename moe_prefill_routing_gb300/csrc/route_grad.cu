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
// One pass: a token's row is read once, its gradient written once; the
// weights' part is k values a token, set out by expert in shared memory.
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

// J: slots of a lane (k <= 32 W J).
template <typename L, int V, int W, int C, int J>
__global__ void __launch_bounds__(kGradThreads, V >= 16 || J > 1 ? 2 : 4) k_route_grad(const RouteGradArgs p)
{
    constexpr int G = 32 * W;
    constexpr int kGroups = kGradWarps / W;
    extern __shared__ __align__(16) uint8_t smem[];
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

    for (int64_t t = int64_t(blockIdx.x) * kGroups + g; t < p.T;
         t += int64_t(gridDim.x) * kGroups) {
        L *orow = static_cast<L *>(p.dlogits) + t * p.ldd;
        const L *row = logits + t * p.ld;
        float l[V];
        uint32_t kmax = kClosed;
        int id[J];         // the lane's slots: expert (-1: none), its logit, scale dw
        float v[J], d[J];
        if (!p.mask || p.mask[t]) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = lane + G * j;
                id[j] = p.dw && at < p.k ? p.ids[t * p.k + at] : -1;
                d[j] = p.dw && at < p.k ? p.scale * p.dw[t * p.k + at] : 0.0f;
            }
            load_row<L, V, C, G>(l, row, lane, p.E, p.f16);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                v[j] = uint32_t(id[j]) < uint32_t(p.E) ? to_f(row[id[j]], p.f16) : -INFINITY;
                if (!(v[j] < INFINITY))
                    v[j] = -INFINITY;
            }
            float own = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(l[i] < INFINITY))
                    l[i] = -INFINITY;
                own = fmaxf(own, l[i]);
            }
            kmax = gr.largest(key_of(own));
        }
        if (kmax == kClosed) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                l[i] = 0.0f;
            store_row<L, V, C, G>(l, orow, lane, p.E, p.f16);
            continue;
        }
        const float m = of_key(kmax);
        const float c = p.sigmoid ? fminf(m, 0.0f) : 0.0f;
        float s[V], sum = 0.0f, sume = 0.0f, pc = 0.0f;
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sume += exp_ftz(l[i] - m);
                s[i] = sig_scaled(l[i], c);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] = exp_ftz(l[i] - m);  // 0 for closed experts
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sum += s[i];
            pc += s[i] * cf[i];
        }

        // the chosen experts' scores
        float q[J], sq = 0.0f, sd = 0.0f;
        if (p.dw) {
            float ms = m, cs = 0.0f;  // no norm: the scores themselves
            if (p.norm) {
                uint32_t own = kClosed;
#pragma unroll
                for (int j = 0; j < J; ++j)
                    own = max(own, key_of(v[j]));
                ms = of_key(gr.largest(own));  // -inf where no slot has weight
                cs = fminf(ms, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                q[j] = v[j] == -INFINITY ? 0.0f
                       : p.sigmoid       ? sig_scaled(v[j], cs)
                                         : exp_ftz(v[j] - ms);
                sq += q[j];
                sd += q[j] * d[j];
            }
        }
        sum = gr.sum(sum);
        const float inv = rcp_ftz(sum);
        pc = aux ? gr.sum(pc) * inv : 0.0f;
        sume = !p.sigmoid ? sum : aux ? gr.sum(sume) : 1.0f;
        float dot = 0.0f;  // no norm, softmax: sum s scale dw
        if (p.dw) {
            float mul = 1.0f, mean = 0.0f;
            if (p.norm) {
                sq = gr.sum(sq);
                mul = sq > 0.0f ? rcp_ftz(sq) : 0.0f;
                mean = gr.sum(sd) * mul;
            } else if (!p.sigmoid) {
                mul = inv;
                dot = gr.sum(sd) * inv;
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (v[j] > -INFINITY)
                    dsel[id[j]] = q[j] * mul * (d[j] - mean);
        }
        gr.sync();
        const float zc = gz * (m + __logf(sume)) * rcp_ftz(sume);
        const float base = pc + dot;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_of<C, G>(lane, i);
            float o = s[i] * inv * (cf[i] - base) + (e < p.E ? dsel[e] : 0.0f);
            if (p.sigmoid)
                o = o * rcp_ftz(1.0f + exp_ftz(l[i])) + zc * exp_ftz(l[i] - m);
            else
                o += zc * s[i];
            l[i] = l[i] > -INFINITY ? o : 0.0f;
        }
        store_row<L, V, C, G>(l, orow, lane, p.E, p.f16);
        gr.sync();
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (v[j] > -INFINITY)
                    dsel[id[j]] = 0.0f;
        }
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
            const int grid = std::min((T - 1) / per + 1, 8 * device_sm_count());
            // one slot a lane serves k up to 32 (or the CTA's 256 lanes)
            auto kern = W > 1 || k <= 32 ? k_route_grad<L, V, W, C, 1>
                                         : k_route_grad<L, V, W, C, W == 1 ? 8 : 1>;
            return launch_pdl(kern, dim3(grid), dim3(kGradThreads),
                              size_t(per) * E * 4, reinterpret_cast<cudaStream_t>(stream), a);
        });
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
