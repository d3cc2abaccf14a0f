// The router: logits -> top-k experts, weights, counts and the balance and z
// losses (moe_route).  The scores and their ratios: route.cuh.
//
// Every token's row is read once into registers by one warp (E <= 512), four
// (E <= 2048) or one CTA; statistics, choice and weights come from there.
// (8192 tokens of 1024 experts: 55 us with four warps, 215 with a CTA, whose
// every reduction waits for 16 warps.)  Counts and probability sums are kept
// per CTA; k_route_final adds the CTAs' rows in their order, so the losses
// are deterministic.
#include "route.cuh"

namespace moe {
namespace {

using namespace route;

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxCtas = 304;  // rows of partial sums in the workspace
constexpr int kFinalCtas = 8;       // one cluster
constexpr int kFinalThreads = 512;
constexpr uint32_t kTaken = 0;  // key of an expert already chosen

// Status bits of calls without a workspace, see moe_take_status.
__device__ uint32_t g_status;

// CTAs that an SM holds at once, by registers; the grid is as many
template <int V>
constexpr int kRouteResident = V >= 16 ? 1 : 2;

struct RouteArgs {
    const void *logits;
    const float *bias;     // may be null
    const uint8_t *mask;   // may be null
    int32_t *ids;
    float *w;
    uint2 *part;        // [grid][E] {sum of p over the CTA's tokens, count}
    float4 *part_scal;  // [grid] {sum lse^2, tokens that take part, status bits, -}
    uint32_t *status;
    int32_t *counts;  // each may be null
    float *prob;
    float *loss;
    int64_t ld;
    int T, E, k;
    int sigmoid, norm, stats, f16;
    float scale;
};

// Dynamic shared memory: the CTA's counts, then per group the experts under
// choice (id and logit; for k <= 32 also key and id as one number, 32 of each
// and a spare) or, once its tokens are done, its probability sums.
__host__ __device__ inline int sel_slots(int k)
{
    return k > 32 ? (k + 3) & ~3 : 36;
}

__host__ __device__ inline int group_words(int k, int E)
{
    const int sel = (k > 32 ? 2 : 4) * sel_slots(k);
    return sel > E ? sel : (E + 3) & ~3;
}

size_t route_smem(int E, int k, int W)
{
    return size_t((E + 3) & ~3) * 4 + size_t(kRouteWarps / W) * group_words(k, E) * 4;
}

// Sum over the CTA in a fixed order; every thread gets it.
template <int WARPS, typename X>
__device__ __forceinline__ X cta_sum(X v, X *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i)
        v += red[i];
    return v;
}

// Threshold of a warp's choice: a key that at least k open experts reach, or
// kClosed + 1 (every open expert's is at least that).  The k-th largest of the
// lanes' own maxima will do, since each lane has one; maxima that tie count
// once, which only lowers it.
__device__ __forceinline__ uint32_t warp_threshold(uint32_t own, uint32_t kmax, int k)
{
    uint32_t t = kmax;
#pragma unroll 4
    for (int j = 1; j < k; ++j) {
        own = own == t ? kTaken : own;
        t = __reduce_max_sync(kFull, own);
    }
    return max(t, kClosed + 1);
}

// One token per group of W warps at a time; a lane holds V of its logits.
//
// Choosing (a warp, k <= 32): keys at or above warp_threshold are collected
// in shared memory, k of them at least and rarely more than a few extra (512
// experts: 12 for k = 10), each with its expert as one 64-bit number that
// orders them (key, then the lower expert); each lane takes one and counts
// how many are larger, which is its slot.  With more than 32 (ties, or one lane holding most),
// k > 32, or more warps per token: k rounds of the group's largest key, whose
// holder drops it and looks for its next best.
//
// Bound by instructions, not memory: some 500 a token at 128 experts (sigmoid,
// bias, losses, k = 8), 1100 at 512 (softmax, losses, k = 10), with 70 % of
// the issue slots taken.  With k_route_final 25.6 us for 32768 tokens x 128
// experts (18.9 MB, 2.8 us of memory traffic), 9.0 us for 2048 x 512, of which
// the launches, one token's chain of reductions and the final sums are most;
// 2.5 us for one token.  (Two tokens a warp would halve the shuffles but
// double the lane maxima's rounds, which one instruction each reduces.)
template <typename L, int V, int W, int C, bool BIAS>
__global__ void __launch_bounds__(kRouteThreads, kRouteResident<V>) k_route(const RouteArgs p)
{
    constexpr int G = 32 * W;                 // threads of a group
    constexpr int kGroups = kRouteWarps / W;  // groups of the CTA
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint2 red[W > 1 ? kGroups : 1][2][W];
    __shared__ float s_sum[kRouteWarps];
    __shared__ float s_z[kGroups];
    __shared__ int s_live[kGroups];
    __shared__ uint32_t s_flags;
    const int g = threadIdx.x / G, lane = threadIdx.x % G;
    int *cnt = reinterpret_cast<int *>(smem);
    float *ps = reinterpret_cast<float *>(cnt + ((p.E + 3) & ~3)) + g * group_words(p.k, p.E);
    uint64_t *sel_o = reinterpret_cast<uint64_t *>(ps);  // key, then ~expert
    int *sel_e = reinterpret_cast<int *>(sel_o + (p.k > 32 ? 0 : sel_slots(p.k)));
    float *sel_l = reinterpret_cast<float *>(sel_e + sel_slots(p.k));
    Group<W> gr{red[W > 1 ? g : 0]};
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads)
        cnt[e] = 0;
    if (threadIdx.x == 0)
        s_flags = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    const L *logits = static_cast<const L *>(p.logits);
    float acc[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = expert_of<C, G>(lane, i);
        acc[i] = 0.0f;
        bias[i] = BIAS && e < p.E ? p.bias[e] : 0.0f;
    }
    const bool need_p = p.stats || (!p.norm && !p.sigmoid) || BIAS;
    bool bad = false;
    int live = 0;
    float zsum = 0.0f;

    int64_t t = int64_t(blockIdx.x) * kGroups + g;
    const int64_t step = int64_t(gridDim.x) * kGroups;
    const L *row = logits + t * p.ld;
    int32_t *ids = p.ids + t * p.k;
    float *w = p.w + t * p.k;
    // the row, loaded a token ahead where registers allow it (128 experts,
    // 32768 tokens: 25.3 us, 26.0 without)
    constexpr bool kAhead = V <= 4;
    RawRow<L, V, C, G> raw;
    bool on = false;
    auto fetch = [&](int64_t at, const L *from) {
        on = !p.mask || p.mask[at];
        if (on || kAhead)
            raw.load(from, lane, p.E);
    };
    if (kAhead && t < p.T)
        fetch(t, row);
    for (; t < p.T; t += step, row += step * p.ld, ids += step * p.k, w += step * p.k) {
        float l[V];
        uint32_t key[V], own = kClosed, kmax = kClosed;
        if (!kAhead)
            fetch(t, row);
        if (on) {
            raw.to(l, lane, p.E, p.f16);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(l[i] < INFINITY)) {  // NaN or +inf: closed, and reported
                    bad = true;
                    l[i] = -INFINITY;
                }
                key[i] = key_of(l[i]);
                own = max(own, key[i]);
            }
            kmax = gr.largest(own);
        }
        if (kAhead && t + step < p.T)
            fetch(t + step, row + step * p.ld);
        if (kmax == kClosed) {  // takes no part
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
            if (p.sigmoid) {
                sig_scaled(s, l, c);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sume += exp_ftz(l[i] - m);  // 0 for closed experts
                    sum += s[i];
                }
                sum = gr.sum(sum);
                sume = gr.sum(sume);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = exp_ftz(l[i] - m);
                    sum += s[i];
                }
                sum = sume = gr.sum(sum);
            }
            inv = rcp_ftz(sum);
            if (p.stats) {
                const float lse = m + __logf(sume);
                zsum += lse * lse;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] += s[i] * inv;
            }
            if (BIAS) {
                const float mul = p.sigmoid ? exp_ftz(c) : inv;  // s to scores
                own = kClosed;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (l[i] > -INFINITY)
                        key[i] = key_of(s[i] * mul + bias[i]);
                    own = max(own, key[i]);
                }
                kmax = gr.largest(own);
            }
        }
        ++live;

        int slot = p.k, id = -1;  // this lane's slot (>= k: none), its expert and logit
        float lid = -INFINITY;
        int n = 0;          // slots filled
        bool held = false;  // the choice is in the lanes, else in sel_*
        if (W == 1 && p.k <= 32) {
            const uint32_t th = warp_threshold(own, kmax, p.k);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                mine += key[i] >= th;
            int at = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(kFull, at, o);
                at += lane >= o ? up : 0;
            }
            const int all = __shfl_sync(kFull, at, 31);
            at -= mine;
            held = all <= 32;
            if (held) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] >= th) {
                        const int e = expert_of<C, G>(lane, i);
                        sel_o[at] = uint64_t(key[i]) << 32 | uint32_t(~e);
                        if (BIAS)
                            sel_l[at] = l[i];
                        ++at;
                    }
                if (lane == 0)
                    sel_o[all] = 0;  // the loop below takes two at a time
                __syncwarp();
                const uint64_t o = lane < all ? sel_o[lane] : ~0ull;
                id = ~int(uint32_t(o));
                lid = BIAS ? sel_l[min(lane, 31)] : of_key(uint32_t(o >> 32));
                slot = 0;
                for (int j = 0; j < all; j += 2) {
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(sel_o + j);
                    slot += q.x > o;
                    slot += q.y > o;
                }
                slot = lane < all ? slot : p.k;
                n = min(all, p.k);
            }
        }
        if (!held) {
            uint32_t bk = kTaken;
            int bi = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > bk) {
                    bk = key[i];
                    bi = i;
                }
            while (true) {
                int e = expert_of<C, G>(lane, bi);
                kmax = gr.best(bk, e);
                if (kmax <= kClosed)
                    break;
                if (bk == kmax && expert_of<C, G>(lane, bi) == e) {
                    sel_e[n] = e;
                    const int drop = bi;
                    bk = kTaken;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (i == drop) {
                            key[i] = kTaken;
                            sel_l[n] = l[i];
                        }
                        if (key[i] > bk) {
                            bk = key[i];
                            bi = i;
                        }
                    }
                }
                if (++n == p.k)
                    break;
            }
            gr.sync();
        }
        // f(slot, expert, logit) for each slot of the lane
        auto each = [&](auto f) {
            if (held) {
                if (slot < p.k)
                    f(slot, id, lid);
            } else {
                for (int j = lane; j < n; j += G)
                    f(j, sel_e[j], sel_l[j]);
            }
        };
        float ms = 0.0f, cs = 0.0f, mul = p.scale;
        if (p.norm) {
            ms = m;  // without a bias the row's maximum is the first choice
            if (BIAS) {
                uint32_t o = kClosed;
                each([&](int, int, float v) { o = max(o, key_of(v)); });
                ms = of_key(gr.largest(o));
            }
            cs = fminf(ms, 0.0f);
            float sum = 0.0f;
            each([&](int, int, float v) {
                sum += p.sigmoid ? sig_scaled(v, cs) : exp_ftz(v - ms);
            });
            mul = p.scale * rcp_ftz(gr.sum(sum));
        } else if (!p.sigmoid) {
            ms = m;
            mul = p.scale * inv;
        }
        each([&](int j, int e, float v) {
            ids[j] = e;
            w[j] = mul * (p.sigmoid ? sig_scaled(v, cs) : exp_ftz(v - ms));
            if (p.stats)
                atomicAdd(&cnt[e], 1);
        });
        for (int j = n + lane; j < p.k; j += G) {
            ids[j] = -1;
            w[j] = 0.0f;
        }
        gr.sync();  // sel_* is written again for the next token
    }

    if (bad)
        atomicOr(p.status ? &s_flags : &g_status, MOE_STATUS_BAD_LOGIT);
    if (lane == 0) {
        s_live[g] = live;
        s_z[g] = zsum;
    }
    __syncthreads();
    if (p.stats) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_of<C, G>(lane, i);
            if (e < p.E)
                ps[e] = acc[i];
        }
        __syncthreads();
    }
    float z = 0.0f;
    int tokens = 0;
    for (int q = 0; q < kGroups; ++q) {
        z += s_z[q];
        tokens += s_live[q];
    }
    const bool alone = gridDim.x == 1;  // one CTA had every token
    const float nt = float(max(tokens, 1));
    float dot = 0.0f;
    for (int e = threadIdx.x; e < p.E && p.stats; e += kRouteThreads) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kGroups; ++q)
            s += ps[(q - g) * group_words(p.k, p.E) + e];
        if (alone) {
            const float pr = s / nt;
            dot += float(cnt[e]) / (nt * float(p.k)) * pr;
            if (p.prob)
                p.prob[e] = pr;
            if (p.counts)
                p.counts[e] = cnt[e];
        } else {
            p.part[int64_t(blockIdx.x) * p.E + e] = make_uint2(__float_as_uint(s), uint32_t(cnt[e]));
        }
    }
    if (!p.status)  // nobody asked for more than ids and weights
        return;
    if (!alone) {
        if (threadIdx.x == 0)
            p.part_scal[blockIdx.x] =
                make_float4(z, __int_as_float(tokens), __uint_as_float(s_flags), 0.0f);
        return;
    }
    if (threadIdx.x == 0)
        *p.status = s_flags;
    if (!p.stats)
        return;
    dot = cta_sum<kRouteWarps>(dot, s_sum);
    if (threadIdx.x == 0) {
        if (p.counts)
            p.counts[p.E] = tokens;
        if (p.loss) {
            p.loss[0] = float(p.E) * dot;
            p.loss[1] = z / nt;
        }
    }
}

// The partial sums of k_route's CTAs (`parts` rows), added in their order:
// counts, mean probabilities, losses and the status word.  One cluster of
// eight CTAs; a CTA takes `cols` experts at a time, its threads the rows of
// partial sums 512 / cols abreast (cols: 16 up to 128 experts, so that all
// eight CTAs have some, then 32 and 64).  All latency: about 3 us, of which
// a sum and its count in one access and losses sent to CTA 0 rather than
// fetched by it (one meeting of the cluster less) saved 1.2.
__global__ void __launch_bounds__(kFinalThreads) k_route_final(const RouteArgs p, int parts)
{
    __shared__ float red_f[kFinalThreads / 32];
    __shared__ int red_i[kFinalThreads / 32];
    __shared__ float s_prob[kFinalThreads];
    __shared__ int s_count[kFinalThreads];
    __shared__ int s_dots[kFinalCtas];  // of CTA 0: every CTA's share of the balance loss
    __shared__ uint32_t s_flags;
    const uint32_t rank = cluster_ctarank();
    const int cols = p.E <= 128 ? 16 : p.E <= 256 ? 32 : 64, rows = kFinalThreads / cols;
    const int col = threadIdx.x % cols, row = threadIdx.x / cols;
    if (threadIdx.x == 0)
        s_flags = 0;
    __syncwarp();  // the cluster's barriers are for whole warps
    cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    float z = 0.0f;
    int live = 0;
    uint32_t flags = 0;
    if (int(threadIdx.x) < parts) {
        const float4 v = p.part_scal[threadIdx.x];
        z = v.x;
        live = __float_as_int(v.y);
        flags = __float_as_uint(v.z);
    }
    float dot = 0.0f, n = 0.0f;
    for (int e0 = int(rank) * cols, first = 1; e0 < p.E || first;
         e0 += kFinalCtas * cols, first = 0) {
        const bool in = e0 + col < p.E && p.stats;
        float s = 0.0f;
        int c = 0;
        if (in) {
            const uint2 *at = p.part + e0 + col;
#pragma unroll 8
            for (int i = row; i < parts; i += rows) {
                const uint2 v = at[int64_t(i) * p.E];
                s += __uint_as_float(v.x);
                c += int(v.y);
            }
        }
        s_prob[threadIdx.x] = s;
        s_count[threadIdx.x] = c;
        if (first) {  // their loads are in flight with the first rows'
            live = cta_sum<kFinalThreads / 32>(live, red_i);
            z = cta_sum<kFinalThreads / 32>(z, red_f);
            if (flags)
                atomicOr(&s_flags, flags);
            n = float(max(live, 1));
        }
        __syncthreads();
        if (row == 0 && in) {
#pragma unroll 7
            for (int i = 1; i < rows; ++i) {
                s += s_prob[i * cols + col];
                c += s_count[i * cols + col];
            }
            const float pr = s / n;
            dot += float(c) / (n * float(p.k)) * pr;
            if (p.prob)
                p.prob[e0 + col] = pr;
            if (p.counts)
                p.counts[e0 + col] = c;
        }
        __syncthreads();
    }
    dot = cta_sum<kFinalThreads / 32>(dot, red_f);
    __syncwarp();
    cluster_wait();  // every CTA has started, so its shared memory is there
    if (threadIdx.x == 0)
        dsmem_st(dsmem_addr(&s_dots[rank], 0), __float_as_int(dot));
    __syncwarp();
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        *p.status = s_flags;
        if (p.counts)
            p.counts[p.E] = live;
        if (p.loss) {
            float d = 0.0f;
#pragma unroll
            for (int r = 0; r < kFinalCtas; ++r)
                d += __int_as_float(s_dots[r]);
            p.loss[0] = float(p.E) * d;
            p.loss[1] = z / n;
        }
    }
}

inline size_t align256(size_t b)
{
    return (b + 255) & ~size_t(255);
}

inline size_t part_rows(int T)
{
    return std::min(std::max(T, 1), kRouteMaxCtas);
}

}  // namespace

uint32_t *route_status_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_status) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

}  // namespace moe

extern "C" size_t moe_route_workspace_bytes(int T, int E)
{
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS)
        return 0;
    const size_t rows = moe::part_rows(T);
    return 256 + moe::align256(rows * sizeof(float4)) + moe::align256(rows * E * 8);
}

extern "C" int moe_route(const void *logits, int64_t ld, int l_dtype, const float *bias,
                         const uint8_t *mask, int T, int E, int k, int score, int norm,
                         float scale, int32_t *ids, float *w, int32_t *counts, float *prob,
                         float *loss, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    using namespace moe;
    const int rc = check_sizes(l_dtype, T, E, k, ld, score);
    if (rc != MOE_OK)
        return rc;
    const int stats = counts || prob || loss;
    if ((stats && !ws) || (T > 0 && (!logits || !ids || !w)))
        return MOE_ERR_NULL;
    if (ws && ws_bytes < moe_route_workspace_bytes(T, E))
        return MOE_ERR_WORKSPACE;
    if (!aligned(logits, size_of(l_dtype)) || !aligned(bias, 4) || !aligned(ids, 4) ||
        !aligned(w, 4) || !aligned(counts, 4) || !aligned(prob, 4) || !aligned(loss, 4) ||
        !aligned(ws, 256))
        return MOE_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t rows = part_rows(T);
    uint8_t *b = static_cast<uint8_t *>(ws);
    RouteArgs a = {};
    a.logits = logits, a.bias = bias, a.mask = mask, a.ids = ids, a.w = w;
    if (ws) {
        a.part_scal = reinterpret_cast<float4 *>(b + 256);
        a.part = reinterpret_cast<uint2 *>(b + 256 + align256(rows * sizeof(float4)));
    }
    a.status = reinterpret_cast<uint32_t *>(ws);
    a.counts = counts, a.prob = prob, a.loss = loss;
    a.ld = ld, a.T = T, a.E = E, a.k = k;
    a.sigmoid = score == MOE_SCORE_SIGMOID, a.norm = norm != 0;
    a.stats = stats, a.f16 = l_dtype == MOE_DT_F16;
    a.scale = scale;
    const int size = size_of(l_dtype);
    int grid = 1;
    cudaError_t e = by_shape<kRouteWarps>(
        l_dtype, E,
        [&](int c) { return E % c == 0 && ld % c == 0 && aligned(logits, c * size); },
        [&](auto l, auto v, auto w, auto c) {
            constexpr int V = decltype(v)::value, W = decltype(w)::value, C = decltype(c)::value;
            using L = decltype(l);
            const int per = kRouteWarps / W;
            grid = std::max(1, std::min({(T - 1) / per + 1, kRouteResident<V> * device_sm_count(),
                                         kRouteMaxCtas}));
            auto kern = bias ? k_route<L, V, W, C, true> : k_route<L, V, W, C, false>;
            return launch_pdl(kern, dim3(grid), dim3(kRouteThreads), route_smem(E, k, W), s, a);
        });
    if (e == cudaSuccess && grid > 1 && ws) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kFinalCtas);
        cfg.blockDim = dim3(kFinalThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kFinalCtas;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, k_route_final, a, grid);
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
