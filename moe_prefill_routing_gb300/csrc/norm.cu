// The norms before and after a block, its gate and the scaled residual add
// (moe_block_norm), and their gradients (moe_block_norm_grad).
//
// Per row, with r(v) = (mean(v^2) + eps)^-1/2:
//   xn = alpha x + g r(o) (o . post),   h = xn r(xn) . pre
// and from dxn and dh, with a = dh . pre, r1 = r(o), r2 = r(xn):
//   dS = dxn + r2 (a - c2 r2 xn),   c2 = r2 mean(a . xn)
//   dx = alpha dS,   q = mean(dS . post . o),   dg = d r1 q
//   do = g r1 dS . post - r1^2 q (g r1 o)
//   dpost = sum over rows of g r1 dS . o,   dpre = sum over rows of r2 dh . xn
// in which r1 and r2 multiply one value each time and never one another: r2^3 of a row
// around 2^45 is subnormal, of one around 2^-43 infinite.
//
// Each tensor crosses memory once: a group of warps takes a row at a time, a thread
// eight neighbouring elements of it (1, 2 or 4 times), kept in registers or its
// slots between the sums, while the next row is on its way.  All sums are fp32 in a
// fixed order; a thread's part of a mean is divided by d before the parts are
// added, so that it does not overflow sooner than a thread's 8 to 32 squares (or
// products) do.
//
// 32768 rows x 2816: bf16 123 us (738 MB, 6.0 TB/s), with MXFP4 rows 165, an fp32
// stream 168 (6.6 TB/s); gradients 217 (1.1 GB, 5.1 TB/s) and, of an fp32 stream,
// 255 (6.5 TB/s).  What bounds the 16-bit forms are instructions and their
// latencies: 60 % of the issue slots, in the gradients with 12 warps an SM.  2048 x
// 2560 from memory: 12.8 us, with MXFP4 rows 15.3, gradients 21.2.  Rows too wide for
// a ring are read where they are used: gradients of 16384 x 7168 with an fp32 stream
// 567 us (3.7 TB/s), of 4096 x 16384 bf16 353 (2.3 TB/s).
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "mx_rows.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

namespace moe {
namespace {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxD = kNormMaxThreads * 8 * 4;
constexpr int kNormStages = 2;      // rows of a ring: one in use, one on its way
constexpr int kNormGradCtas = 608;  // at most: rows of partial column sums
constexpr int kSumThreads = 1024;

struct NormArgs {
    const void *x, *o;
    const float *pre, *post, *gate;
    const uint8_t *mask;
    void *xn, *h;
    uint8_t *codes, *scales;
    int64_t ldx, ldo, ldxn, ldh;
    int T, d;
    int post_norm, sigmoid, k_tiles, warps, ring_bytes;  // of a group
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
    int post_norm, sigmoid, warps, ring_bytes;  // of a group
    int vec_xn, vec_o, vec_dxn, vec_dh, vec_dx, vec_do;
    float alpha, eps;
};

// The threads of a CTA that have one row: CTAs take several rows side by side
// where rows are short.
struct Group {
    int id, t, size, warps, count;  // t: the thread's place in it; count: groups of the CTA

    __device__ __forceinline__ Group(int warps_) : size(32 * warps_), warps(warps_)
    {
        id = int(threadIdx.x) / size;
        t = int(threadIdx.x) - id * size;
        count = int(blockDim.x) / size;
    }

    __device__ __forceinline__ void sync() const
    {
        if (count == 1)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
    }
};

// Sums over a group, in every thread; one barrier, two sets of words in turn.
struct GroupSum {
    const Group &gr;
    float *red;  // the group's [2][warps][8]
    int turn;

    __device__ __forceinline__ float *words()
    {
        turn ^= 1;
        return red + (turn ? 8 * gr.warps : 0);
    }

    __device__ __forceinline__ float one(float v)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if (gr.warps == 1)
            return v;
        const int lane = int(threadIdx.x) & 31;
        float *const w = words();
        if (lane == 0)
            w[gr.t >> 5] = v;
        gr.sync();
        // every warp adds the warps' sums (16 at most) across its lanes
        v = lane < gr.warps ? w[lane] : 0.0f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return __shfl_sync(0xffffffffu, v, 0);
    }

    // Eight values, of which the first N are wanted: lanes pass on the half of the
    // values that they do not keep, so that four lanes have one each in the end.
    template <int N>
    __device__ __forceinline__ void eight(float (&v)[8])
    {
        const int lane = int(threadIdx.x) & 31;
#pragma unroll
        for (int n = 4; n; n >>= 1) {
            const bool upper = lane & (4 * n);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = upper ? v[i + n] : v[i], pass = upper ? v[i] : v[i + n];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, pass, 4 * n);
            }
        }
        float s = v[0];  // of value lane / 4
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        if (gr.warps > 1) {
            float *const w = words();
            if ((lane & 3) == 0)
                w[(gr.t >> 5) * 8 + (lane >> 2)] = s;
            gr.sync();
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < kNormMaxThreads / 32; i += 4)
                if (i + (lane & 3) < gr.warps)
                    s += w[(i + (lane & 3)) * 8 + (lane >> 2)];
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s += __shfl_xor_sync(0xffffffffu, s, 1);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __shfl_sync(0xffffffffu, s, 4 * i);
    }
};

__device__ __forceinline__ float gate_of(float g, bool some, int sigmoid)
{
    return !some ? 1.0f : sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// Its slope: of a sigmoid s(g) s(-g), as 1 - s(g) has no digits left past g = 17.
__device__ __forceinline__ float gate_slope(float g, int sigmoid)
{
    return sigmoid ? 1.0f / ((1.0f + expf(-g)) * (1.0f + expf(g))) : 1.0f;
}

// How a kernel reads rows.
enum Mode {
    kDirect,   // where they are used
    kRing,     // ahead of their use; 16-byte pieces of rows are aligned, d a multiple of 8
    kShifted,  // ahead of their use, rows that start and end anywhere
};

// Rows of a tensor of [rows, d].  In a ring, cp.async brings them ahead of their use
// into slots of shared memory of the thread (fp32, kShifted: the warp) that reads
// them, so that what is in flight takes neither barriers nor registers.  A tensor
// that is not there reads as zeros.
//
// Eight fp32 are two 16-byte pieces; copied by the thread that uses them, every
// instruction would touch half of each 32-byte sector of memory.  A warp copies
// (and, through a slot that has been read, writes) neighbouring pieces with
// neighbouring lanes instead: 32768 rows x 2816 of an fp32 stream 210 -> 185 us (169
// with later changes).
//
// kShifted: what is brought are the aligned 16-byte pieces of memory that a row lies
// in, one more to a warp than its elements fill, which the warp then shifts into
// place; results leave through a slot, neighbouring words by neighbouring lanes.
// (Element by element from the thread that uses them, 32768 x 2815 bf16 took 490 us
// instead of 248, its gradients 1113 instead of 519; 2.0 and 2.4 times the aligned
// 2816's, from the instructions of the way through the slots.)
template <typename E, int R, int MODE>
struct Rows {
    static constexpr int kPieces = sizeof(E) == 4 ? 2 : 1;  // of 16 bytes: eight elements
    static constexpr int kWarp = 32 * kPieces + (MODE == kShifted);  // a warp's of a round
    const E *p;
    int64_t ld;
    int d, vec, G, t;  // G, t: the group's threads, and which this one is
    uint4 *slots;      // [stage][R][warps][kWarp], from the warp's first on

    __device__ __forceinline__ Rows(const void *tensor, int64_t ld_, int d_, int vec_,
                                    const Group &gr, uint8_t *&smem)
        : p(static_cast<const E *>(tensor)), ld(ld_), d(d_), vec(vec_), G(gr.size), t(gr.t),
          slots(reinterpret_cast<uint4 *>(smem) + (gr.t >> 5) * kWarp)
    {
        if (MODE == kDirect)
            return;
        smem += kNormStages * R * gr.warps * kWarp * 16;
#pragma unroll
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < kNormStages; ++i) {
                if (MODE == kShifted) {
                    for (int j = t & 31; !p && j < kWarp; j += 32)
                        at(i, r)[j] = make_uint4(0, 0, 0, 0);
                } else if (!p || (t + r * G) * 8 >= d) {  // never fetched
#pragma unroll
                    for (int q = 0; q < kPieces; ++q)
                        *mine(i, r, q) = make_uint4(0, 0, 0, 0);
                }
            }
        __syncwarp();
    }

    __device__ __forceinline__ uint4 *at(int stage, int r) const
    {
        return slots + (stage * R + r) * (G >> 5) * kWarp;
    }

    // The thread's q-th piece (fp32: lanes 4 - 7 of eight take theirs in the other
    // order, which keeps eight lanes' banks apart).
    __device__ __forceinline__ uint4 *mine(int stage, int r, int q) const
    {
        return at(stage, r) + (t & 31) * kPieces + (kPieces == 2 ? q ^ ((t >> 2) & 1) : 0);
    }

    // The words of the warp's 256 elements, from the lane's first on.
    __device__ __forceinline__ uint32_t *words(int stage, int r) const
    {
        return reinterpret_cast<uint32_t *>(at(stage, r)) + (t & 31);
    }

    // kShifted: a row's bytes before its first element in its first piece.
    __device__ __forceinline__ int shift(int64_t row) const
    {
        return int(reinterpret_cast<uintptr_t>(p + row * ld) & 15);
    }

    __device__ __forceinline__ void fetch(int64_t row, int stage) const
    {
        if (MODE == kDirect || !p)
            return;
        if (MODE == kShifted || kPieces == 2)
            __syncwarp();  // the slot's last row has been read by every lane
        const int lane = t & 31, w = (t & ~31) * kPieces + lane;
        if (MODE == kShifted) {
            const int before = shift(row), total = before + d * int(sizeof(E));
            const uint8_t *const from = reinterpret_cast<const uint8_t *>(p + row * ld) - before;
            // (nothing before the tensor is read)
            const int early = int(max(reinterpret_cast<const uint8_t *>(p) - from, ptrdiff_t(0)));
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q <= kPieces; ++q) {
                    const int c = (w + 32 * q + r * G * kPieces) * 16;  // of the row's bytes
                    const int n = min(max(total - c, 0), 16);           // those past it: zeros
                    uint4 *const to = at(stage, r) + 32 * q + lane;
                    if (q == kPieces && lane)
                        continue;
                    if (early && c == 0) {
                        *to = make_uint4(0, 0, 0, 0);
                        for (int b = early; b < n; b += int(sizeof(E)))
                            reinterpret_cast<E *>(to)[b / int(sizeof(E))] =
                                reinterpret_cast<const E *>(from)[b / int(sizeof(E))];
                    } else {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         smem_u32(to)),
                                     "l"(n ? from + c : from + 16), "r"(n)
                                     : "memory");
                    }
                }
            return;
        }
        const uint4 *from = reinterpret_cast<const uint4 *>(p + row * ld) + w;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                if ((w + 32 * q + r * G * kPieces) * (8 / kPieces) < d)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     smem_u32(at(stage, r) + 32 * q + lane)),
                                 "l"(from + r * G * kPieces + 32 * q)
                                 : "memory");
    }

    // kShifted, after async_wait and a barrier of the warp: the row's elements to
    // where `mine` finds them.
    __device__ __forceinline__ void settle(int64_t row, int stage) const
    {
        if (MODE != kShifted || !p)
            return;
        const int before = shift(row);
        if (!before)
            return;
        if (kPieces == 1) {
            uint32_t w[R][8];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 a = mine(stage, r, 0)[0], b = mine(stage, r, 0)[1];
                w[r][0] = a.x, w[r][1] = a.y, w[r][2] = a.z, w[r][3] = a.w;
                w[r][4] = b.x, w[r][5] = b.y, w[r][6] = b.z, w[r][7] = b.w;
            }
            __syncwarp();
            if (before & 8) {
#pragma unroll
                for (int i = 0; i < R * 6; ++i)
                    w[i / 6][i % 6] = w[i / 6][i % 6 + 2];
            }
            if (before & 4) {
#pragma unroll
                for (int i = 0; i < R * 5; ++i)
                    w[i / 5][i % 5] = w[i / 5][i % 5 + 1];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[r][i] = __funnelshift_r(w[r][i], w[r][i + 1], (before & 2) * 8);
                *mine(stage, r, 0) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
            }
        } else {
            uint32_t w[R][8];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[r][i] = words(stage, r)[32 * i + (before >> 2)];
            __syncwarp();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    words(stage, r)[32 * i] = w[r][i];
            __syncwarp();
        }
    }

    // After async_wait (and settle).
    __device__ __forceinline__ Oct<E> read(int64_t row, int stage, int r) const
    {
        const int c = (t + r * G) * 8;
        Oct<E> o;
        if (MODE != kDirect && kPieces == 2) {
            const uint4 a = *mine(stage, r, 0), b = *mine(stage, r, 1);
            const bool other = (t >> 2) & 1;
            o.set(0, other ? b : a);
            o.set(kPieces - 1, other ? a : b);
        } else if (MODE != kDirect) {
            o.set(0, *mine(stage, r, 0));
        } else {
            o.load(p + (p ? row * ld + c : 0), p ? d - c : 0, vec);
        }
        return o;
    }

    // The thread's eight elements of a row of another tensor of [rows, d]; fp32 and
    // kShifted through slots whose row has been read.
    __device__ __forceinline__ void put(void *to, int64_t to_ld, int64_t row, int stage, int r,
                                        int to_vec, const Oct<E> &o) const
    {
        const int lane = t & 31, c = (t + r * G) * 8;
        E *out = static_cast<E *>(to) + row * to_ld;
        if (MODE == kDirect || (MODE == kRing && kPieces == 1)) {
            if (MODE == kDirect || c < d)
                o.store(out + c, MODE == kRing ? 8 : d - c, MODE == kRing || to_vec);
            return;
        }
        __syncwarp();
        if (MODE == kShifted || c < d) {
            const bool other = kPieces == 2 && ((t >> 2) & 1);
            const uint4 a = o.get(0), b = o.get(kPieces - 1);
            *mine(stage, r, 0) = other ? b : a;
            if (kPieces == 2)
                *mine(stage, r, 1) = other ? a : b;
        }
        __syncwarp();
        if (MODE == kRing) {
            const int w = (t & ~31) * kPieces + lane + r * G * kPieces;
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                if ((w + 32 * q) * 4 < d)
                    reinterpret_cast<uint4 *>(out)[w + 32 * q] = at(stage, r)[32 * q + lane];
            return;
        }
        const int n = min(d - (c - lane * 8), 256);  // of the warp's elements
        if (kPieces == 2) {
            uint32_t *const first = reinterpret_cast<uint32_t *>(out) + (c - lane * 8);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (lane + 32 * i < n)
                    first[lane + 32 * i] = words(stage, r)[32 * i];
        } else {
            // words where they are aligned: from the second element on where the first
            // one lies in the upper half of a word
            uint16_t *const first = reinterpret_cast<uint16_t *>(out) + (c - lane * 8);
            const int odd = int(reinterpret_cast<uintptr_t>(first) >> 1 & 1);
            const uint32_t *const a = words(stage, r);
            if (odd && lane == 0 && n > 0)
                first[0] = uint16_t(a[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = 2 * (lane + 32 * i) + odd;
                const uint32_t v =
                    odd ? __funnelshift_r(a[32 * i], a[32 * i + 1], 16) : a[32 * i];
                if (e + 1 < n)
                    *reinterpret_cast<uint32_t *>(first + e) = v;
                else if (e < n)
                    first[e] = uint16_t(v);
            }
        }
    }
};

// A thread's part of a row that is looked at more than once: read from a ring's
// slot each time (registers are what limits the rows that an SM works on), kept
// in registers without one.
template <typename E, int R, int MODE>
struct Part {
    const Rows<E, R, MODE> &rows;
    Oct<E> kept[MODE == kDirect ? R : 1];

    __device__ __forceinline__ Part(const Rows<E, R, MODE> &rows_, int64_t row) : rows(rows_)
    {
        if (MODE == kDirect) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                kept[MODE == kDirect ? r : 0] = rows.read(row, 0, r);
        }
    }

    __device__ __forceinline__ void get(int stage, int r, Two (&v)[4]) const
    {
        if (MODE == kDirect)
            kept[MODE == kDirect ? r : 0].to(v);
        else
            rows.read(0, stage, r).to(v);
    }
};

// Weights of a row (1 where there are none, 0 past its end): in registers where
// a thread has eight, in shared memory (of the whole CTA) where it has more.
template <int R>
struct Weights {
    Two w[R == 1 ? 4 : 1];
    const ulonglong2 *slots;
    int G;

    // (to be used after a barrier of the CTA)
    __device__ __forceinline__ void load(const float *p, int d, const Group &gr, uint8_t *&smem)
    {
        G = gr.size;
        float4 *mine = reinterpret_cast<float4 *>(smem) + gr.t;
        slots = reinterpret_cast<const ulonglong2 *>(mine);
        if (R > 1)
            smem += R * 2 * G * 16;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (gr.t + r * G) * 8;
            float v[8];
            if (R == 1 || gr.id == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = c + i >= d ? 0.0f : p ? p[c + i] : 1.0f;
            }
            if (R == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[R == 1 ? i : 0] = two(v[2 * i], v[2 * i + 1]);
            } else if (gr.id == 0) {
                mine[(2 * r) * G] = make_float4(v[0], v[1], v[2], v[3]);
                mine[(2 * r + 1) * G] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }

    __device__ __forceinline__ void get(int r, Two (&v)[4]) const
    {
        if (R == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = w[R == 1 ? i : 0];
        } else {
            const ulonglong2 a = slots[(2 * r) * G], b = slots[(2 * r + 1) * G];
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        }
    }
};

__device__ __forceinline__ void async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Until only the latest group is on its way.
__device__ __forceinline__ void async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(1) : "memory");
}

template <typename S, typename B, int R, int MODE>
__global__ void __maxnreg__(R == 1 ? 64 : R == 2 ? (sizeof(S) == 4 ? 80 : 88) : 128)
    k_block_norm(const NormArgs p)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float red[2 * 8 * kNormMaxThreads / 32];
    const Group gr(p.warps);
    GroupSum sum{gr, red + 2 * 8 * gr.id * gr.warps, 0};
    const int G = gr.size;
    const float inv_d = 1.0f / float(p.d);
    uint8_t *smem = smem_raw + gr.id * p.ring_bytes;  // a ring for each group, then the weights
    const Rows<S, R, MODE> xs(p.x, p.ldx, p.d, p.vec_x, gr, smem);
    const Rows<B, R, MODE> os(p.o, p.ldo, p.d, p.vec_o, gr, smem);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t rows = p.codes ? (int64_t(p.T) + 127) / 128 * 128 : p.T;
    const int64_t step = int64_t(gridDim.x) * gr.count;
    const int64_t first = int64_t(blockIdx.x) * gr.count + gr.id;
    // nonzero for a row that takes part; as it is loaded, so that nothing waits for
    // it before it is used (a row later)
    auto is_live = [&](int64_t t) -> uint32_t { return t >= p.T ? 0u : !p.mask ? 1u : p.mask[t]; };
    // the next turn's row is on its way while one is worked on
    int64_t ahead = first;
    int in = 0;
    auto fetch = [&](uint32_t live) {
        if (live) {
            xs.fetch(ahead, in);
            os.fetch(ahead, in);
        }
        async_commit();
        ahead += step;
        in ^= 1;
    };
    uint32_t live = is_live(first);
    fetch(live);
    uint32_t next = is_live(ahead);
    float gate = p.gate && live ? p.gate[first] : 0.0f;
    Weights<R> pre, post;
    smem = smem_raw + gr.count * p.ring_bytes;
    pre.load(p.pre, p.d, gr, smem);
    post.load(p.post, p.d, gr, smem);
    if (R > 1)
        __syncthreads();
    int out = 0;
    for (int64_t t = first; t < rows; t += step) {
        fetch(next);
        const uint32_t coming = is_live(ahead);
        const float g = gate_of(gate, p.gate, p.sigmoid);
        gate = p.gate && t + step < p.T ? p.gate[t + step] : 0.0f;
        async_wait();
        if (MODE == kShifted || (MODE == kRing && (sizeof(S) == 4 || sizeof(B) == 4)))
            __syncwarp();  // other lanes' copies
        Two v[R][4];
        if (live) {
            xs.settle(t, out);
            os.settle(t, out);
            const Part<S, R, MODE> x(xs, t);
            if (p.o) {
                const Part<B, R, MODE> o(os, t);
                float k = g;
                if (p.post_norm) {
                    Two squares = 0;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        Two f[4];
                        o.get(out, r, f);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            squares = fma(f[i], f[i], squares);
                    }
                    k *= rsqrtf(sum.one(sum_of(squares) * inv_d) + p.eps);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Two f[4], w[4];
                    o.get(out, r, f);
                    x.get(out, r, v[r]);
                    post.get(r, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[r][i] = fma(both(p.alpha), v[r][i], mul(f[i], mul(both(k), w[i])));
                    Oct<S> xn;
                    xn.from(v[r]);
                    xs.put(p.xn, p.ldxn, t, out, r, p.vec_xn, xn);
                    xn.to(v[r]);  // the stream as it is stored
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    x.get(out, r, v[r]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[r][i] = 0;
                if (p.o && t < p.T) {
                    Oct<S> zero;
                    zero.from(v[r]);
                    xs.put(p.xn, p.ldxn, t, out, r, p.vec_xn, zero);
                }
            }
        }
        if (p.pre) {
            if (live) {
                Two squares = 0;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        squares = fma(v[r][i], v[r][i], squares);
                const float k = rsqrtf(sum.one(sum_of(squares) * inv_d) + p.eps);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Two w[4];
                    pre.get(r, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[r][i] = mul(mul(v[r][i], both(k)), w[i]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (gr.t + r * G) * 8;
                Oct<B> h;
                h.from(v[r]);
                if (p.h && t < p.T)
                    os.put(p.h, p.ldh, t, out, r, p.vec_h, h);
                if (p.codes) {
                    float f[8];
                    h.to(f);  // codes of h as it is stored
                    // (0 past the row's end, where a norm of NaN makes NaN of zeros too)
                    const uint32_t top = max_of_lanes<4>(h.max_bits());
                    const uint32_t byte = c < p.d ? mx_scale_byte(top) : 0u;
                    const uint32_t word = word_of_tile<4>(byte);
                    if (t < p.T && c < p.d)
                        *reinterpret_cast<uint32_t *>(p.codes + t * (p.d / 2) + c / 2) =
                            mx_encode8(f, byte);
                    if ((gr.t & 15) == 0 && c < p.k_tiles * 128)
                        *mx_scale_word(p.scales, t, c / 128, p.k_tiles) = word;
                }
            }
        }
        live = next;
        next = coming;
        out ^= 1;
    }
}

template <typename S, typename B, int R, int MODE>
__global__ void __maxnreg__(R == 1 ? 96 : 128) k_block_norm_grad(const NormGradArgs p)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float red[2 * 8 * kNormMaxThreads / 32];
    const Group gr(p.warps);
    GroupSum sum{gr, red + 2 * 8 * gr.id * gr.warps, 0};
    const int G = gr.size;
    const float inv_d = 1.0f / float(p.d);
    uint8_t *smem = smem_raw + gr.id * p.ring_bytes;  // a ring for each group, then the weights
    const Rows<S, R, MODE> xns(p.dh ? p.xn : nullptr, p.ldxn, p.d, p.vec_xn, gr, smem);
    const Rows<S, R, MODE> dxns(p.dxn, p.lddxn, p.d, p.vec_dxn, gr, smem);
    const Rows<B, R, MODE> os(p.o, p.ldo, p.d, p.vec_o, gr, smem);
    const Rows<B, R, MODE> dhs(p.dh, p.lddh, p.d, p.vec_dh, gr, smem);
    // (the slots of a tensor that is not there stay zeros)
    const Rows<S, R, MODE> &spare = p.dxn ? dxns : xns;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = int64_t(gridDim.x) * gr.count;
    const int64_t first = int64_t(blockIdx.x) * gr.count + gr.id;
    // nonzero for a row that takes part; as it is loaded, so that nothing waits for
    // it before it is used (a row later)
    auto is_live = [&](int64_t t) -> uint32_t { return t >= p.T ? 0u : !p.mask ? 1u : p.mask[t]; };
    int64_t ahead = first;
    int in = 0;
    auto fetch = [&](uint32_t live) {
        if (live) {
            xns.fetch(ahead, in);
            dxns.fetch(ahead, in);
            os.fetch(ahead, in);
            dhs.fetch(ahead, in);
        }
        async_commit();
        ahead += step;
        in ^= 1;
    };
    uint32_t live = is_live(first);
    fetch(live);
    uint32_t next = is_live(ahead);
    float gate = p.gate && live ? p.gate[first] : 0.0f;
    Weights<R> pre, post;
    smem = smem_raw + gr.count * p.ring_bytes;
    pre.load(p.pre, p.d, gr, smem);
    post.load(p.post, p.d, gr, smem);
    if (R > 1)
        __syncthreads();
    Two dpre[R][4] = {}, dpost[R][4] = {};
    int out = 0;
    for (int64_t t = first; t < p.T; t += step) {
        fetch(next);
        const uint32_t coming = is_live(ahead);
        const float raw = gate, g = gate_of(raw, p.gate, p.sigmoid);
        gate = p.gate && t + step < p.T ? p.gate[t + step] : 0.0f;
        async_wait();
        if (MODE == kShifted || (MODE == kRing && (sizeof(S) == 4 || sizeof(B) == 4)))
            __syncwarp();  // other lanes' copies
        if (live) {
            xns.settle(t, out);
            dxns.settle(t, out);
            os.settle(t, out);
            dhs.settle(t, out);
            const Part<S, R, MODE> xn(xns, t), dxn(dxns, t);
            const Part<B, R, MODE> dh(dhs, t), o(os, t);
            // the means (q's dS is made of three terms) all at once
            Two xx = 0, ax = 0, oo = 0, dq = 0, aq = 0, xq = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                Two x[4], h[4], f[4], d[4], w[4], v[4];
                xn.get(out, r, x);
                dh.get(out, r, h);
                o.get(out, r, f);
                dxn.get(out, r, d);
                pre.get(r, w);
                post.get(r, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Two a = mul(h[i], w[i]), u = mul(v[i], f[i]);
                    xx = fma(x[i], x[i], xx);
                    ax = fma(a, x[i], ax);
                    oo = fma(f[i], f[i], oo);
                    dq = fma(d[i], u, dq);
                    aq = fma(a, u, aq);
                    xq = fma(x[i], u, xq);
                }
            }
            float s[8] = {sum_of(xx) * inv_d, sum_of(ax) * inv_d, sum_of(oo) * inv_d,
                          sum_of(dq) * inv_d, sum_of(aq) * inv_d, sum_of(xq) * inv_d};
            sum.eight<6>(s);
            const float r2 = p.dh ? rsqrtf(s[0] + p.eps) : 0.0f;
            const float r1 = p.post_norm ? rsqrtf(s[2] + p.eps) : 1.0f;
            const float c2 = r2 * s[1];
            const float q = s[3] + r2 * (s[4] - c2 * (r2 * s[5]));
            const float dgate = r1 * q * float(p.d);
            const float k = g * r1, c1 = p.post_norm ? r1 * (r1 * q) : 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                Two x[4], h[4], f[4], d[4], w[4], v[4];
                xn.get(out, r, x);
                dh.get(out, r, h);
                o.get(out, r, f);
                dxn.get(out, r, d);
                pre.get(r, w);
                post.get(r, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = mul(x[i], both(r2));
                    f[i] = mul(f[i], both(k));
                    dpre[r][i] = fma(h[i], x[i], dpre[r][i]);
                    d[i] = fma(both(r2), fma(both(-c2), x[i], mul(h[i], w[i])), d[i]);
                    dpost[r][i] = fma(d[i], f[i], dpost[r][i]);
                    f[i] = fma(both(k), mul(d[i], v[i]), mul(both(-c1), f[i]));
                    d[i] = mul(both(p.alpha), d[i]);
                }
                Oct<S> dx;
                dx.from(d);
                spare.put(p.dx, p.lddx, t, out, r, p.vec_dx, dx);
                if (p.o) {
                    Oct<B> d_o;
                    d_o.from(f);
                    os.put(p.d_o, p.lddo, t, out, r, p.vec_do, d_o);
                }
            }
            // (here, as the row's stores need not wait for the slope: 16384 x 7168 with an
            // fp32 stream 567 us, ahead of them 640)
            if (p.dgate && gr.t == 0)
                p.dgate[t] = dgate * gate_slope(raw, p.sigmoid);
        } else {
            float zero[8] = {};
            Oct<S> zs;
            Oct<B> zb;
            zs.from(zero);
            zb.from(zero);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                spare.put(p.dx, p.lddx, t, out, r, p.vec_dx, zs);
                if (p.o)
                    os.put(p.d_o, p.lddo, t, out, r, p.vec_do, zb);
            }
            if (p.dgate && gr.t == 0)
                p.dgate[t] = 0.0f;
        }
        live = next;
        next = coming;
        out ^= 1;
    }
    if (!p.part)
        return;
    float *part = p.part + int64_t(blockIdx.x) * 2 * p.d;
    const auto each = [&](auto f) {  // f(which, r, i, value)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float a, b;
                apart(dpre[r][i / 2], a, b);
                f(0, r, i, a), f(0, r, i + 1, b);
                apart(dpost[r][i / 2], a, b);
                f(1, r, i, a), f(1, r, i + 1, b);
            }
    };
    if (gr.count == 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (gr.t + r * G) * 8;
            if (p.d % 8 == 0) {
                if (c < p.d) {
                    ulonglong2 *a = reinterpret_cast<ulonglong2 *>(part + c);
                    ulonglong2 *b = reinterpret_cast<ulonglong2 *>(part + p.d + c);
                    a[0] = make_ulonglong2(dpre[r][0], dpre[r][1]);
                    a[1] = make_ulonglong2(dpre[r][2], dpre[r][3]);
                    b[0] = make_ulonglong2(dpost[r][0], dpost[r][1]);
                    b[1] = make_ulonglong2(dpost[r][2], dpost[r][3]);
                }
            }
        }
        if (p.d % 8 != 0)
            each([&](int which, int r, int i, float v) {
                const int c = (gr.t + r * G) * 8 + i;
                if (c < p.d)
                    part[which * p.d + c] = v;
            });
        return;
    }
    // the groups' sums, in order, through the rings' memory (of 2 R 8 G floats a
    // group, see norm_shape)
    float *all = reinterpret_cast<float *>(smem_raw);
    const int words = 2 * R * 8 * G;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    each([&](int which, int r, int i, float v) {
        all[gr.id * words + ((which * R + r) * 8 + i) * G + gr.t] = v;
    });
    __syncthreads();
    for (int j = int(threadIdx.x); j < words; j += int(blockDim.x)) {
        float v = 0.0f;
        for (int k = 0; k < gr.count; ++k)
            v += all[k * words + j];
        const int which = j / (R * 8 * G), r = j / (8 * G) % R, i = j / G % 8;
        const int c = (j % G + r * G) * 8 + i;
        if (c < p.d)
            part[which * p.d + c] = v;
    }
}

// The CTAs' column sums: a CTA takes 32 columns of the 2 d, its 32 warps every
// 32nd row (all of a warp's 19 rows at most are on their way at once; with eight
// warps the rows' latencies added up: 2048 x 2560 25.6 us), added in order.
__global__ void __launch_bounds__(kSumThreads)
    k_norm_col_sum(const float *part, int rows, int d, float *dpre, float *dpost)
{
    constexpr int kWarps = kSumThreads / 32;
    __shared__ float red[kWarps][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float v = 0.0f;
    if (c < 2 * d) {
#pragma unroll
        for (int i = 0; i < (kNormGradCtas + kWarps - 1) / kWarps; ++i)
            if (g + i * kWarps < rows)
                v += part[int64_t(g + i * kWarps) * 2 * d + c];
    }
    red[g][lane] = v;
    __syncthreads();
    // warp g adds column g across its lanes
    v = red[lane][g];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    const int column = blockIdx.x * 32 + g;
    if (lane == 0 && column < 2 * d) {
        if (column < d) {
            if (dpre)
                dpre[column] = v;
        } else if (dpost) {
            dpost[column - d] = v;
        }
    }
}

// ---- host ---------------------------------------------------------------------

constexpr size_t kNormSmem = 200 * 1024;  // the most dynamic shared memory of a CTA

// How a launch lays rows out.
struct Shape {
    int warps, r, groups;  // of a row; rounds of eight elements a thread; rows side by side
    int mode;
    size_t ring_bytes, smem;  // of a group, of a CTA

    int threads() const { return 32 * warps * groups; }
};

// A thread has eight elements of rows that a warp can hold so, else 16 (its share
// of a row's sums and addresses costs about as much as eight elements do), or
// 32 past 8192; eight too where the rows do not go round the SMs, and only a
// row's time counts, and where rows that are not aligned would leave an SM one CTA
// (gradients of 32768 x 2815 fp32 864 -> 654 us, of 16384 x 4095 with an fp32 stream
// 484 -> 385; aligned ones, whose CTAs wait less, are faster with 16: 32768 x 2816
// with an fp32 stream 257 us, 460 with eight).  `whole`: rows up to a multiple of
// 128; `bytes`: of a row's element in all `tensors` that are read; `sums`: column
// sums are kept.
Shape norm_shape(int64_t rows, int d, bool whole, bool vec, int tensors, int bytes, bool sums)
{
    const int chunks = whole ? mx_k_tiles(d) * 16 : (d + 7) / 8;
    Shape s;
    size_t weights = 0;
    const auto lay = [&](int r) {
        s.r = r;
        s.warps = ((chunks + r - 1) / r + 31) / 32;
        s.groups = std::max(1, 8 / s.warps);
        weights = r > 1 ? size_t(4) * r * 32 * s.warps * 16 : 0;
        s.ring_bytes = size_t(kNormStages) * r * s.warps * (32 * 8 * bytes + (vec ? 0 : tensors) * 16);
        s.smem = s.groups * s.ring_bytes + weights;
    };
    lay(chunks <= (rows > device_sm_count() ? 32 : kNormMaxThreads) ? 1
        : chunks <= 2 * kNormMaxThreads                             ? 2
                                                                    : 4);
    if (!vec && chunks <= kNormMaxThreads && s.smem > kNormSmem / 2)
        lay(1);
    // (rows that are not aligned gain nothing from the way through the slots where
    // they fill half a warp, and two tensors' loads are few: norm of 100000 x 101 bf16
    // 56 us, kShifted 73; of 50000 x 191 50 and 38)
    s.mode = s.r > 2 || s.smem > kNormSmem || (!vec && tensors == 2 && chunks <= 16) ? kDirect
             : vec                                                                  ? kRing
                                                                                    : kShifted;
    if (s.mode == kDirect)
        s.ring_bytes = 0;
    if (sums && s.groups > 1)  // the groups' sums pass through the rings' memory
        s.ring_bytes = std::max(s.ring_bytes, size_t(2) * s.r * 8 * 32 * s.warps * 4);
    s.smem = s.groups * s.ring_bytes + weights;
    return s;
}

// f(S, B, R, MODE) of the types, the rounds and how rows are read.  Of the gradient's
// four tensors one round always goes through a ring, and two do unless they have
// more than 8 bytes an element; of the norm's two, two rounds always do.
template <bool GRAD, typename F>
cudaError_t with_types(int s, int b, int r, int mode, F f)
{
    const auto with_r = [&](auto sv, auto bv) {
        using S = decltype(sv);
        using B = decltype(bv);
        const auto with_mode = [&](auto rv) {
            if constexpr (GRAD ? sizeof(S) == 4 && decltype(rv)::value == 2
                               : decltype(rv)::value == 1)
                if (mode == kDirect)
                    return f(S(), B(), rv, std::integral_constant<int, kDirect>());
            return mode == kRing ? f(S(), B(), rv, std::integral_constant<int, kRing>())
                                 : f(S(), B(), rv, std::integral_constant<int, kShifted>());
        };
        return r == 1   ? with_mode(std::integral_constant<int, 1>())
               : r == 2 ? with_mode(std::integral_constant<int, 2>())
                        : f(S(), B(), std::integral_constant<int, 4>(),
                            std::integral_constant<int, kDirect>());
    };
    if (s == MOE_DT_BF16)
        return with_r(__nv_bfloat16(), __nv_bfloat16());
    if (s == MOE_DT_F16)
        return with_r(__half(), __half());
    return b == MOE_DT_BF16  ? with_r(float(), __nv_bfloat16())
           : b == MOE_DT_F16 ? with_r(float(), __half())
                             : with_r(float(), float());
}

// Launches a norm kernel on as many CTAs as the device holds at once (what it
// holds is asked once per kernel, number of warps and device).
template <auto KERN, typename Args>
cudaError_t launch_norm(Args &a, const Shape &sh, int64_t rows, int most, int &ctas, cudaStream_t s)
{
    constexpr int kDevices = 16;
    static std::atomic<int> per_sm[kDevices][kNormMaxThreads / 32 + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    int held = dev < kDevices ? per_sm[dev][sh.warps].load(std::memory_order_acquire) : 0;
    if (!held) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(KERN),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, KERN, sh.threads(), sh.smem);
        if (e != cudaSuccess)
            return e;
        held = std::max(held, 1);
        if (dev < kDevices)
            per_sm[dev][sh.warps].store(held, std::memory_order_release);
    }
    a.warps = sh.warps, a.ring_bytes = int(sh.ring_bytes);
    ctas = int(std::min<int64_t>(
        {int64_t(held) * device_sm_count(), (rows + sh.groups - 1) / sh.groups, most}));
    return launch_pdl(KERN, dim3(ctas), dim3(sh.threads()), sh.smem, s, a);
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
    const bool vec = d % 8 == 0 && a.vec_x && (!o || (a.vec_o && a.vec_xn)) && (!h || a.vec_h);
    const Shape sh = norm_shape(T, d, codes != nullptr, vec, 2, xs + bs, false);
    const int64_t rows = codes ? (int64_t(T) + 127) / 128 * 128 : T;
    int ctas = 0;
    const cudaError_t e =
        with_types<false>(x_dtype, b_dtype, sh.r, sh.mode, [&](auto s, auto b, auto r, auto g) {
            constexpr auto kern =
                k_block_norm<decltype(s), decltype(b), decltype(r)::value, decltype(g)::value>;
            return launch_norm<kern>(a, sh, rows, INT_MAX, ctas,
                                     reinterpret_cast<cudaStream_t>(stream));
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
    const bool vec = d % 8 == 0 && (!dh || (a.vec_xn && a.vec_dh)) && (!dxn || a.vec_dxn) &&
                     a.vec_dx && (!o || (a.vec_o && a.vec_do));
    const Shape sh = norm_shape(T, d, false, vec, 4, 2 * (xs + bs), sums);
    int ctas = 0;
    cudaError_t e =
        with_types<true>(x_dtype, b_dtype, sh.r, sh.mode, [&](auto s, auto b, auto r, auto g) {
            constexpr auto kern =
                k_block_norm_grad<decltype(s), decltype(b), decltype(r)::value, decltype(g)::value>;
            return launch_norm<kern>(a, sh, T, kNormGradCtas, ctas, stm);
        });
    if (e == cudaSuccess && sums)
        e = launch_pdl(k_norm_col_sum, dim3((2 * d + 31) / 32), dim3(kSumThreads), 0, stm,
                       static_cast<const float *>(ws), ctas, d, dpre, dpost);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
