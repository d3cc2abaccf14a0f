// The norms before and after a block, its gate and the scaled residual add
// (moe_block_norm), and their gradients (moe_block_norm_grad).
//
// Per row, with r(v) = (mean(v^2) + eps)^-1/2:
//   xn = alpha x + g r(o) (o . post),   h = xn r(xn) . pre
// and from dxn and dh, with a = dh . pre, r1 = r(o), r2 = r(xn):
//   dS = dxn + r2 a - r2^3 mean(a . xn) xn
//   dx = alpha dS,   q = sum(dS . post . o),   dg = r1 q
//   do = g r1 dS . post - r1^2 (g r1 q / d) o
//   dpost = sum over rows of g r1 dS . o,   dpre = sum over rows of r2 dh . xn
//
// Each tensor crosses memory once: a CTA takes a row at a time, a thread eight
// neighbouring elements of it (1, 2 or 4 times), kept in registers between the
// sums.  All sums are fp32 in a fixed order; a thread's part of a mean is divided
// by d before the parts are added, so that it does not overflow sooner than a
// thread's 8 to 32 squares do.
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "mx_rows.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <climits>
#include <type_traits>

namespace moe {
namespace {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxD = kNormMaxThreads * 8 * 4;
constexpr int kNormGradCtas = 608;  // at most: rows of partial column sums
constexpr int kSumThreads = 256;

struct NormArgs {
    const void *x, *o;
    const float *pre, *post, *gate;
    const uint8_t *mask;
    void *xn, *h;
    uint8_t *codes, *scales;
    int64_t ldx, ldo, ldxn, ldh;
    int T, d;
    int post_norm, sigmoid, k_tiles;
    int vec_x, vec_o, vec_xn, vec_h;
    float alpha, eps;
};

struct NormGradArgs {
    const void *xn, *o, *dxn, *dh;
    const float *pre, *post, *gate;
    const uint8_t *mask;
    void *dx, *d_o;
    float *dgate, *part;  // part: [CTAs][2][d], dpre's and dpost's
    int64_t ldxn, ldo, lddxn, lddh, lddx, lddo;
    int T, d;
    int post_norm, sigmoid;
    int vec_xn, vec_o, vec_dxn, vec_dh, vec_dx, vec_do;
    float alpha, eps;
};

// Sums of N values over the CTA's threads, in every thread; one barrier, two
// sets of words in turn.
struct BlockSum {
    float (*red)[3][kNormMaxThreads / 32];
    int turn;

    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        const int warps = int(blockDim.x) >> 5;
        if (warps == 1)
            return;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                red[turn][i][threadIdx.x >> 5] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
            for (int w = 0; w < warps; ++w)
                s += red[turn][i][w];
            v[i] = s;
        }
        turn ^= 1;
    }
};

__device__ __forceinline__ float gate_of(const float *gate, int sigmoid, int64_t t)
{
    if (!gate)
        return 1.0f;
    const float g = gate[t];
    return sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// Eight weights of a row of d (1 where there are none), 0 past its end.
__device__ __forceinline__ void load_weights(float (&w)[8], const float *p, int c, int d)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = c + i >= d ? 0.0f : p ? p[c + i] : 1.0f;
}

template <typename S, typename B, int R>
__global__ void __launch_bounds__(kNormMaxThreads) k_block_norm(const NormArgs p)
{
    __shared__ float red[2][3][kNormMaxThreads / 32];
    BlockSum sum{red, 0};
    const int G = int(blockDim.x);
    const float inv_d = 1.0f / float(p.d);
    pdl_wait();
    pdl_launch_dependents();
    float pre[R][8], post[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (int(threadIdx.x) + r * G) * 8;
        load_weights(pre[r], p.pre, c, p.d);
        load_weights(post[r], p.post, c, p.d);
    }
    const int rows = p.codes ? (p.T + 127) / 128 * 128 : p.T;
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const bool live = t < p.T && (!p.mask || p.mask[t]);
        float v[R][8];
        if (live) {
            Oct<S> x[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (int(threadIdx.x) + r * G) * 8;
                x[r].load(static_cast<const S *>(p.x) + t * p.ldx + c, p.d - c, p.vec_x);
            }
            if (p.o) {
                Oct<B> o[R];
                float k = gate_of(p.gate, p.sigmoid, t);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int c = (int(threadIdx.x) + r * G) * 8;
                    o[r].load(static_cast<const B *>(p.o) + t * p.ldo + c, p.d - c, p.vec_o);
                }
                if (p.post_norm) {
                    float s[1] = {0.0f};
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float f[8];
                        o[r].to(f);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[0] += f[i] * f[i];
                    }
                    s[0] *= inv_d;
                    sum(s);
                    k *= rsqrtf(s[0] + p.eps);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int c = (int(threadIdx.x) + r * G) * 8;
                    float f[8];
                    o[r].to(f);
                    x[r].to(v[r]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[r][i] = p.alpha * v[r][i] + f[i] * (k * post[r][i]);
                    x[r].from(v[r]);
                    x[r].store(static_cast<S *>(p.xn) + t * p.ldxn + c, p.d - c, p.vec_xn);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[r].to(v[r]);  // the stream as it is stored
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[r][i] = 0.0f;
                const int c = (int(threadIdx.x) + r * G) * 8;
                if (p.o && t < p.T) {
                    Oct<S> zero;
                    zero.from(v[r]);
                    zero.store(static_cast<S *>(p.xn) + t * p.ldxn + c, p.d - c, p.vec_xn);
                }
            }
        }
        if (!p.pre)
            continue;
        float k = 0.0f;
        if (live) {
            float s[1] = {0.0f};
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[0] += v[r][i] * v[r][i];
            s[0] *= inv_d;
            sum(s);
            k = rsqrtf(s[0] + p.eps);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (int(threadIdx.x) + r * G) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[r][i] = live ? v[r][i] * k * pre[r][i] : 0.0f;
            Oct<B> h;
            h.from(v[r]);
            if (p.h && t < p.T)
                h.store(static_cast<B *>(p.h) + t * p.ldh + c, p.d - c, p.vec_h);
            if (p.codes) {
                h.to(v[r]);  // codes of h as it is stored
                const uint32_t byte = mx_scale_byte(max_of_block(max_bits8(v[r])));
                const uint32_t word = word_of_tile(byte);
                if (t < p.T && c < p.d)
                    *reinterpret_cast<uint32_t *>(p.codes + t * (p.d / 2) + c / 2) =
                        mx_encode8(v[r], byte);
                if ((threadIdx.x & 15) == 0 && c < p.k_tiles * 128)
                    *mx_scale_word(p.scales, t, c / 128, p.k_tiles) = word;
            }
        }
    }
}

template <typename S, typename B, int R>
__global__ void __launch_bounds__(kNormMaxThreads) k_block_norm_grad(const NormGradArgs p)
{
    __shared__ float red[2][3][kNormMaxThreads / 32];
    BlockSum sum{red, 0};
    const int G = int(blockDim.x);
    const float inv_d = 1.0f / float(p.d);
    pdl_wait();
    pdl_launch_dependents();
    float pre[R][8], post[R][8], dpre[R][8] = {}, dpost[R][8] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (int(threadIdx.x) + r * G) * 8;
        load_weights(pre[r], p.pre, c, p.d);
        load_weights(post[r], p.post, c, p.d);
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        if (p.mask && !p.mask[t]) {
            float zero[8] = {};
            Oct<S> zs;
            Oct<B> zb;
            zs.from(zero);
            zb.from(zero);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (int(threadIdx.x) + r * G) * 8;
                zs.store(static_cast<S *>(p.dx) + t * p.lddx + c, p.d - c, p.vec_dx);
                if (p.o)
                    zb.store(static_cast<B *>(p.d_o) + t * p.lddo + c, p.d - c, p.vec_do);
            }
            if (p.dgate && threadIdx.x == 0)
                p.dgate[t] = 0.0f;
            continue;
        }
        float ds[R][8];
        Oct<B> o[R], dh[R];
        Oct<S> xn[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (int(threadIdx.x) + r * G) * 8;
            Oct<S> in;
            in.load(static_cast<const S *>(p.dxn) + (p.dxn ? t * p.lddxn + c : 0),
                    p.dxn ? p.d - c : 0, p.vec_dxn);
            in.to(ds[r]);
            dh[r].load(static_cast<const B *>(p.dh) + (p.dh ? t * p.lddh + c : 0),
                       p.dh ? p.d - c : 0, p.vec_dh);
            xn[r].load(static_cast<const S *>(p.xn) + t * p.ldxn + c, p.dh ? p.d - c : 0, p.vec_xn);
            o[r].load(static_cast<const B *>(p.o) + (p.o ? t * p.ldo + c : 0), p.o ? p.d - c : 0,
                      p.vec_o);
        }
        const float g = p.o ? gate_of(p.gate, p.sigmoid, t) : 1.0f;
        float s[3] = {};  // xn^2, a xn, o^2
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x[8], h[8], f[8];
            xn[r].to(x);
            dh[r].to(h);
            o[r].to(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] += x[i] * x[i];
                s[1] += h[i] * pre[r][i] * x[i];
                s[2] += f[i] * f[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            s[i] *= inv_d;
        sum(s);
        const float r2 = p.dh ? rsqrtf(s[0] + p.eps) : 0.0f;
        const float r1 = p.post_norm ? rsqrtf(s[2] + p.eps) : 1.0f;
        const float c2 = r2 * r2 * r2 * s[1];
        float q[1] = {0.0f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (int(threadIdx.x) + r * G) * 8;
            float x[8], h[8], f[8];
            xn[r].to(x);
            dh[r].to(h);
            o[r].to(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dpre[r][i] += h[i] * (x[i] * r2);
                ds[r][i] += r2 * (h[i] * pre[r][i]) - c2 * x[i];
                q[0] += ds[r][i] * (post[r][i] * f[i]);
                x[i] = p.alpha * ds[r][i];
            }
            Oct<S> out;
            out.from(x);
            out.store(static_cast<S *>(p.dx) + t * p.lddx + c, p.d - c, p.vec_dx);
        }
        if (!p.o)
            continue;
        if (p.post_norm || p.dgate)
            sum(q);
        if (p.dgate && threadIdx.x == 0)
            p.dgate[t] = r1 * q[0] * (p.sigmoid ? g * (1.0f - g) : 1.0f);
        const float k = g * r1, c1 = p.post_norm ? r1 * r1 * (k * (q[0] * inv_d)) : 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (int(threadIdx.x) + r * G) * 8;
            float f[8];
            o[r].to(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float e = k * ds[r][i];
                dpost[r][i] += e * f[i];
                f[i] = e * post[r][i] - c1 * f[i];
            }
            o[r].from(f);
            o[r].store(static_cast<B *>(p.d_o) + t * p.lddo + c, p.d - c, p.vec_do);
        }
    }
    if (!p.part)
        return;
    float *part = p.part + int64_t(blockIdx.x) * 2 * p.d;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (int(threadIdx.x) + r * G) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < p.d) {
                part[c + i] = dpre[r][i];
                part[p.d + c + i] = dpost[r][i];
            }
    }
}

// The CTAs' column sums: a CTA takes 32 columns of the 2 d, its warps every
// eighth row, added in order.
__global__ void __launch_bounds__(kSumThreads)
    k_norm_col_sum(const float *part, int rows, int d, float *dpre, float *dpost)
{
    constexpr int kWarps = kSumThreads / 32;
    __shared__ float red[kWarps][32];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float v = 0.0f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int i = g; i < rows; i += kWarps)
            v += part[int64_t(i) * 2 * d + c];
    }
    red[g][lane] = v;
    __syncthreads();
    if (g == 0 && c < 2 * d) {
#pragma unroll
        for (int i = 1; i < kWarps; ++i)
            v += red[i][lane];
        if (c < d) {
            if (dpre)
                dpre[c] = v;
        } else if (dpost) {
            dpost[c - d] = v;
        }
    }
}

// ---- host ---------------------------------------------------------------------

struct Shape {
    int threads, r;
};

// Threads and rounds of a row of d elements (`whole`: up to a multiple of 128).
Shape norm_shape(int d, bool whole)
{
    const int chunks = whole ? mx_k_tiles(d) * 16 : (d + 7) / 8;
    const int r = chunks <= kNormMaxThreads ? 1 : chunks <= 2 * kNormMaxThreads ? 2 : 4;
    return {((chunks + r - 1) / r + 31) / 32 * 32, r};
}

template <typename F>
cudaError_t with_types(int s, int b, int r, F f)
{
    const auto with_r = [&](auto sv, auto bv) {
        using S = decltype(sv);
        using B = decltype(bv);
        return r == 1   ? f(S(), B(), std::integral_constant<int, 1>())
               : r == 2 ? f(S(), B(), std::integral_constant<int, 2>())
                        : f(S(), B(), std::integral_constant<int, 4>());
    };
    if (s == MOE_DT_BF16)
        return with_r(__nv_bfloat16(), __nv_bfloat16());
    if (s == MOE_DT_F16)
        return with_r(__half(), __half());
    return b == MOE_DT_BF16  ? with_r(float(), __nv_bfloat16())
           : b == MOE_DT_F16 ? with_r(float(), __half())
                             : with_r(float(), float());
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// the stream's type, or a 16-bit one beside an fp32 stream
inline bool types_ok(int s, int b)
{
    return s >= MOE_DT_BF16 && s <= MOE_DT_F32 && b >= MOE_DT_BF16 && b <= MOE_DT_F32 &&
           (s == b || s == MOE_DT_F32);
}

// CTAs of a launch over T rows: as many as the device holds at once.
template <typename K>
int norm_ctas(K kern, int threads, int64_t rows, int most)
{
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess)
        per_sm = 1;
    const int64_t ctas = int64_t(std::max(1, per_sm)) * device_sm_count();
    return int(std::min<int64_t>({ctas, rows, most}));
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm(const void *x, int64_t ldx, int x_dtype, const void *o, int64_t ldo,
                              int b_dtype, const float *pre, const float *post, const float *gate,
                              const uint8_t *mask, int T, int d, int post_norm, int gate_act,
                              float alpha, float eps, void *xn, int64_t ldxn, void *h, int64_t ldh,
                              uint8_t *codes, uint8_t *scales, moe_stream_t stream)
{
    using namespace moe;
    if (!types_ok(x_dtype, b_dtype))
        return MOE_ERR_DTYPE;
    if (T < 0 || T > INT_MAX - 511 || d < 1 || d > kNormMaxD || ldx < d || (o && ldo < d) ||
        (xn && ldxn < d) || (h && ldh < d) || (codes && d % 32 != 0) ||
        gate_act < MOE_GATE_PLAIN || gate_act > MOE_GATE_SIGMOID)
        return MOE_ERR_SHAPE;
    // (tensors without rows may have no address)
    if (T > 0 && (!x || (!o && !pre) || (o && !xn) || (!o && (post || gate || xn)) ||
                  (pre ? !h && !codes : h || codes) || !codes != !scales))
        return MOE_ERR_NULL;
    const int xs = dtype_size(x_dtype), bs = dtype_size(b_dtype);
    if (!aligned(x, xs) || !aligned(xn, xs) || !aligned(o, bs) || !aligned(h, bs) ||
        !aligned(pre, 4) || !aligned(post, 4) || !aligned(gate, 4) || !aligned(codes, 16) ||
        !aligned(scales, 16))
        return MOE_ERR_ALIGN;
    if (T == 0)
        return MOE_OK;
    NormArgs a = {};
    a.x = x, a.o = o, a.pre = pre, a.post = post, a.gate = gate, a.mask = mask;
    a.xn = xn, a.h = h, a.codes = codes, a.scales = scales;
    a.ldx = ldx, a.ldo = ldo, a.ldxn = ldxn, a.ldh = ldh;
    a.T = T, a.d = d, a.post_norm = post_norm != 0, a.sigmoid = gate_act == MOE_GATE_SIGMOID;
    a.k_tiles = mx_k_tiles(d);
    a.vec_x = rows_vec(x, ldx, xs), a.vec_o = rows_vec(o, ldo, bs);
    a.vec_xn = rows_vec(xn, ldxn, xs), a.vec_h = rows_vec(h, ldh, bs);
    a.alpha = alpha, a.eps = eps;
    const Shape sh = norm_shape(d, codes != nullptr);
    const int64_t rows = codes ? (int64_t(T) + 127) / 128 * 128 : T;
    const cudaError_t e = with_types(x_dtype, b_dtype, sh.r, [&](auto s, auto b, auto r) {
        const auto kern = k_block_norm<decltype(s), decltype(b), decltype(r)::value>;
        return launch_pdl(kern, dim3(norm_ctas(kern, sh.threads, rows, INT_MAX)),
                          dim3(sh.threads), 0, reinterpret_cast<cudaStream_t>(stream), a);
    });
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" size_t moe_block_norm_grad_workspace_bytes(int T, int d)
{
    if (T < 0 || d < 1 || d > moe::kNormMaxD)
        return 0;
    const size_t rows = std::min(T, moe::kNormGradCtas);
    return std::max<size_t>(256, (rows * 2 * d * sizeof(float) + 255) / 256 * 256);
}

extern "C" int moe_block_norm_grad(const void *xn, int64_t ldxn, int x_dtype, const void *o,
                                   int64_t ldo, int b_dtype, const float *pre, const float *post,
                                   const float *gate, const uint8_t *mask, const void *dxn,
                                   int64_t lddxn, const void *dh, int64_t lddh, int T, int d,
                                   int post_norm, int gate_act, float alpha, float eps, void *dx,
                                   int64_t lddx, void *d_o, int64_t lddo, float *dpre,
                                   float *dpost, float *dgate, void *ws, size_t ws_bytes,
                                   moe_stream_t stream)
{
    using namespace moe;
    if (!types_ok(x_dtype, b_dtype))
        return MOE_ERR_DTYPE;
    if (T < 0 || T > INT_MAX - 511 || d < 1 || d > kNormMaxD || (dh && ldxn < d) ||
        (o && (ldo < d || lddo < d)) || (dxn && lddxn < d) || (dh && lddh < d) || lddx < d ||
        gate_act < MOE_GATE_PLAIN || gate_act > MOE_GATE_SIGMOID)
        return MOE_ERR_SHAPE;
    const bool sums = dpre || dpost;
    if ((T > 0 && (!dx || (o && !d_o) || (dh && (!xn || !pre)) || (!dh && (!dxn || dpre)) ||
                   (!o && (post || gate || dpost || dgate || d_o)) || (dgate && !gate))) ||
        (sums && !ws))
        return MOE_ERR_NULL;
    if (sums && ws_bytes < moe_block_norm_grad_workspace_bytes(T, d))
        return MOE_ERR_WORKSPACE;
    const int xs = dtype_size(x_dtype), bs = dtype_size(b_dtype);
    if (!aligned(xn, xs) || !aligned(dxn, xs) || !aligned(dx, xs) || !aligned(o, bs) ||
        !aligned(dh, bs) || !aligned(d_o, bs) || !aligned(pre, 4) || !aligned(post, 4) ||
        !aligned(gate, 4) || !aligned(dpre, 4) || !aligned(dpost, 4) || !aligned(dgate, 4) ||
        (sums && !aligned(ws, 256)))
        return MOE_ERR_ALIGN;
    const cudaStream_t stm = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        for (float *p : {dpre, dpost})
            if (p && cudaMemsetAsync(p, 0, size_t(d) * sizeof(float), stm) != cudaSuccess)
                return MOE_ERR_CUDA;
        return MOE_OK;
    }
    NormGradArgs a = {};
    a.xn = xn, a.o = o, a.dxn = dxn, a.dh = dh;
    a.pre = pre, a.post = post, a.gate = gate, a.mask = mask;
    a.dx = dx, a.d_o = d_o, a.dgate = dgate, a.part = sums ? static_cast<float *>(ws) : nullptr;
    a.ldxn = ldxn, a.ldo = ldo, a.lddxn = lddxn, a.lddh = lddh, a.lddx = lddx, a.lddo = lddo;
    a.T = T, a.d = d, a.post_norm = o && post_norm, a.sigmoid = gate_act == MOE_GATE_SIGMOID;
    a.vec_xn = rows_vec(xn, ldxn, xs), a.vec_o = rows_vec(o, ldo, bs);
    a.vec_dxn = rows_vec(dxn, lddxn, xs), a.vec_dh = rows_vec(dh, lddh, bs);
    a.vec_dx = rows_vec(dx, lddx, xs), a.vec_do = rows_vec(d_o, lddo, bs);
    a.alpha = o ? alpha : 1.0f, a.eps = eps;
    const Shape sh = norm_shape(d, false);
    int ctas = 0;
    cudaError_t e = with_types(x_dtype, b_dtype, sh.r, [&](auto s, auto b, auto r) {
        const auto kern = k_block_norm_grad<decltype(s), decltype(b), decltype(r)::value>;
        ctas = norm_ctas(kern, sh.threads, T, kNormGradCtas);
        return launch_pdl(kern, dim3(ctas), dim3(sh.threads), 0, stm, a);
    });
    if (e == cudaSuccess && sums)
        e = launch_pdl(k_norm_col_sum, dim3((2 * d + 31) / 32), dim3(kSumThreads), 0, stm,
                       static_cast<const float *>(ws), ctas, d, dpre, dpost);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
