// Dense products on the 5th-generation tensor cores (tcgen05 + TMEM), operands
// staged by TMA: moe_linear (bias, activation and residual in the epilogue)
// and its gradients.
//
// All three products have one form: out[i][j] = sum_r X[i][r] Y[j][r], j the
// output's contiguous dimension:
//
//   y  [t][n] : i = t, j = n (output feature), r = i.  X = x  (r contiguous), Y = W (r contiguous)
//   dx [t][i] : i = t, j = i, r = n.                   X = dP (r contiguous), Y = W (j contiguous)
//   dW [n][i] : i = n, j = i, r = t.                   X = dP (i contiguous), Y = x (j contiguous)
//
// k_linear, for few rows or few tiles: Y is the MMA's A operand (M = 128),
// so that a few tokens fill only the MMA's N (16 columns at least) and the
// weights stream through whole tiles.  k_linear_pair, for the rest: 256 x bn
// tiles on pairs of CTAs, rows as M.
//
// Either way a tile's reduction can be split over the CTAs of a thread-block
// cluster when there are fewer tiles than SMs: each CTA finishes a share of
// the tile, to which the others send their fp32 sums through distributed
// shared memory, and adds them in rank order (results are deterministic).
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

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

// The tensor core adds with truncation, so a sum of numbers of one sign drifts
// by up to 2^-23 of itself per MMA of 16 r (measured: 2.4e-8 with bf16
// operands, 7.7e-8 with fp16 ones, whose products have more bits).  Sums are cut
// into chains of steps of 64 r, four MMAs each, that are added outside the
// tensor core: of 8 steps for an fp32 output (8e-7 and 2.5e-6), and for 16-bit
// outputs of as many as drift by a quarter of half a unit at most, 256 for
// fp16 and 2048 for bf16.
__host__ __device__ constexpr int chain_steps(bool f32, bool f16)
{
    return f32 ? 8 : f16 ? 256 : 2048;
}

struct LinArgs : EpiArgs {
    const float *mul;  // EXTRA kernels: the sums are multiplied by *mul (no bias then), or null
    uint32_t *status;
    int M, N, R;     // k_linear: M = j, N = i; k_linear_pair: M = i, N = j
    int a_mn, b_mn;  // the operand's m (n) is contiguous, not its r
    int bn, stages, split, n_mt;
    int two;         // EXTRA kernels: X = X1 + X2, each summed over all r
    int stall;       // EXTRA kernels, self-test: CTA stall - 1's first stage waits for 16 bytes
    int chain;       // steps of 64 r that one accumulator sums, see chain_steps
};

// Status bits of calls without a status word, see moe_take_status.
__device__ uint32_t g_status;

__device__ __noinline__ void report_timeout(uint32_t *status)
{
    atomicOr(status ? status : &g_status, MOE_STATUS_TIMEOUT);
}

struct LinCtrl {
    uint64_t full[kLinMaxStages];
    uint64_t empty[kLinMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr int kSmallTmem = 256;  // columns of tensor memory of a CTA of k_linear

__host__ __device__ __forceinline__ uint32_t lin_b_tile(int bn, int b_mn)
{
    return uint32_t(b_mn && bn < 64 ? 64 : bn) * LK * 2;
}

// ---- few rows --------------------------------------------------------------------
//
// Tiles of 128 of Y's rows x bn of X's (16 ... 128), one CTA each, or `split`
// CTAs of a cluster that share the reduction: a few tokens against a weight
// matrix have as many tiles as 128 divides its rows (20 for 2560), and only
// all SMs together draw the memory's bandwidth.  Two CTAs fit an SM, 110 KB
// of loads in flight each.  Bound by memory, and by a fixed 4 us of launch,
// first loads, joining the parts and writing: 16 x 10240 x 2560 with a
// residual takes 14 us (52.9 MB, 3.8 TB/s, 5.3 without the fixed part);
// 1 x 2560 x 512, 4.6 us.
//
// Chains (chain_steps) have an accumulator each where those fit the CTA's
// tensor memory; more of them (fp32 outputs of 33 to 128 rows from R = 16384)
// take turns on two, which the accumulator warps add up in a third.
//
// EXTRA: with the two pieces of X and the factor that gradients from an fp32 dy
// may have (kernels of their own: both cost a call of 4.6 us 0.2).
template <bool EXTRA>
struct LinMaps {
    CUtensorMap a, b;
};
template <>
struct LinMaps<true> {
    CUtensorMap a, b, b2;  // b2: the second piece of X, if any
};

template <bool EXTRA>
__global__ void __launch_bounds__(kLinThreads)
    k_linear(const __grid_constant__ LinMaps<EXTRA> maps, const LinArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ LinCtrl ctl;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int bn = p.bn, S = p.stages;
    const uint32_t b_bytes = lin_b_tile(bn, p.b_mn);
    const uint32_t stage_bytes = kLinATile + b_bytes;
    const uint32_t z = cluster_ctarank();
    const int tile = int(blockIdx.x) / p.split;
    const int m0 = (tile % p.n_mt) * LM, n0 = (tile / p.n_mt) * bn;
    const int nk1 = (p.R + LK - 1) / LK, nk = nk1 << (EXTRA ? p.two : 0);  // of a piece, of all
    const int kb0 = int(int64_t(nk) * z / p.split), kb1 = int(int64_t(nk) * (z + 1) / p.split);
    // chains of p.chain steps
    const int chains = max(1, (kb1 - kb0 + p.chain - 1) / p.chain);
    const bool turns = chains * bn > kSmallTmem;  // on two accumulators; a third has the sum
    const int accs = turns ? 1 : chains;          // to add up at the end
    uint32_t tmem_cols = 32;
    while (tmem_cols < uint32_t((turns ? 3 : chains) * bn))
        tmem_cols *= 2;
    volatile int *abort_flag = &ctl.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 4);  // the accumulator warps
        }
        mbar_init(&ctl.done, 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.a);
        prefetch_tmap(&maps.b);
    }
    __syncwarp();
    cluster_arrive();
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

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        const bool one = elect_one();
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag));
            if (!ok)
                break;
            if (one) {
                uint64_t *fb = &ctl.full[stage];
                const bool stall = EXTRA && p.stall == int(blockIdx.x) + 1 && kb == kb0;
                mbar_arrive_expect_tx(fb, stage_bytes + (stall ? 16u : 0u));
                uint8_t *sa = smem + stage * stage_bytes, *sb = sa + kLinATile;
                const CUtensorMap *ma = &maps.a, *mb = &maps.b;
                int step = kb;
                if constexpr (EXTRA)
                    if (step >= nk1)
                        mb = &maps.b2, step -= nk1;
                const int k0 = step * LK;
                if (p.a_mn) {  // 64 m x 64 r boxes, m contiguous
                    tma_load_2d(sa, ma, fb, m0, k0);
                    tma_load_2d(sa + 8192, ma, fb, m0 + 64, k0);
                } else {
                    tma_load_2d(sa, ma, fb, k0, m0);
                }
                if (p.b_mn) {
                    for (int c = 0; c < bn; c += 64)
                        tma_load_2d(sb + c * (LK * 2), mb, fb, n0 + c, k0);
                } else {
                    tma_load_2d(sb, mb, fb, k0, n0);
                }
            }
            __syncwarp();
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) {  // stopped: let the copies already issued land
            report_timeout(p.status);
            for (int s = 0; s < S; ++s)
                if ((issued >> s) & 1u)
                    lin_drain(&ctl.full[s], (issued_par >> s) & 1u);
        }
    } else if (warp == 1) {
        // the whole warp walks the loop and one lane issues, so that
        // descriptors and addresses stay warp-uniform
        int stage = 0;
        uint32_t phase = 0;
        uint32_t idesc = idesc_bf16_f32(LM, uint32_t(bn), p.a_mn, p.b_mn);
        if (p.f16)
            idesc &= ~((7u << 7) | (7u << 10));  // f16 operands: format 0
        const uint32_t sa = smem_u32(smem), sb = sa + kLinATile;
        // r contiguous: 16 of them are 32 bytes inside the 128-byte row; m or n
        // contiguous: 16 rows of 128 bytes, 64-element chunks 8 KB apart
        const uint64_t da0 = p.a_mn ? smem_desc_sw128(sa, 8192, 1024) : smem_desc_sw128(sa, 16, 1024);
        const uint64_t db0 = p.b_mn ? smem_desc_sw128(sb, 8192, 1024) : smem_desc_sw128(sb, 16, 1024);
        const bool one = elect_one();
        uint32_t d = tmem_base, aphase = 0;
        int left = p.chain, buf = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (turns && left == p.chain) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&ctl.acc_empty[buf], aphase ^ 1u, abort_flag));
                if (!ok)
                    break;
                tc_fence_after_sync();
                d = tmem_base + uint32_t(buf * bn);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[stage], phase, abort_flag));
            if (!ok)
                break;
            tc_fence_after_sync();
            if (one) {
                const uint64_t off = uint64_t(uint32_t(stage) * (stage_bytes >> 4));
#pragma unroll
                for (int kk = 0; kk < LK / 16; ++kk)
                    tc_mma_f16(d, da0 + off + kk * (p.a_mn ? 128 : 2),
                               db0 + off + kk * (p.b_mn ? 128 : 2), idesc,
                               left != p.chain || kk != 0);
                tc_commit(&ctl.empty[stage]);
            }
            if (--left == 0 || kb + 1 == kb1) {
                left = p.chain;
                if (!turns) {
                    d += uint32_t(bn);
                } else {
                    if (one)
                        tc_commit(&ctl.acc_full[buf]);
                    if (++buf == 2) {
                        buf = 0;
                        aphase ^= 1u;
                    }
                }
            }
            __syncwarp();
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok)
            report_timeout(p.status);
        if (one)
            tc_commit(&ctl.done);  // arrives once every MMA issued here has completed
    }
    // CTA z of the cluster finishes 128 / Z of the tile's m: every CTA sends it
    // its sums of those, and it adds them in rank order.  They go beside the
    // ring, which may still be in use there, or (128 columns) into the ring
    // once every CTA is done with it.
    const bool beside = bn < LM;
    float *acc = reinterpret_cast<float *>(smem + (beside ? S * stage_bytes : 0u));
    const int slice = LM / p.split, pitch = bn + 4;  // acc: [Z][128 / Z][pitch]
    const int cols = min(bn, p.N - n0);
    // what a thread finishes: four neighbouring m, always the same, of every `by`-th n
    const int quads = slice / 4, by = kLinThreads / quads;
    const int mq = int(threadIdx.x) % quads * 4, at = m0 + int(z) * slice + mq;
    const int left = min(4, p.M - at);
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bias[i] = p.bias && i < left ? p.bias[at + i] : 0.0f;
    bool done = false;
    if (warp >= 2) {
        const uint32_t lanes = tmem_base + (uint32_t(warp & 3) << 21);
        for (int i = 0; turns && i < chains; ++i) {
            if (!__all_sync(0xffffffffu,
                            mbar_wait(&ctl.acc_full[i & 1], (i >> 1) & 1, abort_flag))) {
                report_timeout(p.status);
                break;
            }
            tc_fence_after_sync();
            add_small_chain(lanes + uint32_t((i & 1) * bn), lanes + uint32_t(2 * bn), bn, i > 0);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ctl.acc_empty[i & 1]);
        }
        __syncwarp();
        done = mbar_wait(&ctl.done, 0, abort_flag);
        if (!done) {  // stopped: the MMAs in flight still read shared and write tensor memory
            report_timeout(p.status);
            lin_drain(&ctl.done, 0);
        }
        done = __all_sync(0xffffffffu, done) && kb1 > kb0;
    }
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    if (!beside)
        cluster_sync();
    if (warp >= 2) {
        tc_fence_after_sync();
        const int m = (warp & 3) * 32 + int(lane);
        const uint32_t t0 =
            tmem_base + (uint32_t(warp & 3) << 21) + uint32_t(turns ? 2 * bn : 0);
        const uint32_t to = dsmem_addr(acc + (int(z) * slice + m % slice) * pitch, m / slice);
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
            uint32_t r[16] = {};
            if (done) {
                tmem_ld_32x32b_x16(t0 + uint32_t(c), r);
                tmem_ld_wait();
#pragma unroll 1
                for (int i = 1; i < accs; ++i) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(t0 + uint32_t(i * bn + c), o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(o[j]));
                }
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                dsmem_st4(to + uint32_t(c + j) * 4, r[j], r[j + 1], r[j + 2], r[j + 3]);
        }
        tc_fence_before_sync();
    }
    __syncwarp();
    cluster_sync();
    // R rows at a time; one where that is all there is (less code to fetch
    // counts in a call of a few microseconds: 4.3 against 4.9 us for one token)
    auto finish = [&](auto count) {
        constexpr int R = decltype(count)::value;
#pragma unroll 1
        for (int n = int(threadIdx.x) / quads; n < cols; n += R * by) {
            float v[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = bias[j];
                if (i == 0 || n + i * by < cols) {
                    const float *a = acc + mq * pitch + n + i * by;
                    for (int r = 0; r < p.split; ++r, a += slice * pitch) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[i][j] += a[j * pitch];
                    }
                }
            }
            if (EXTRA && p.mul) {
                const float mul = *p.mul;
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[i][j] *= mul;
            }
            finish_rows<R>(p, v, n0 + n, by, cols - n, at, left);
        }
    };
    if (left > 0) {
        if (cols <= by)
            finish(std::integral_constant<int, 1>());
        else
            finish(std::integral_constant<int, 4>());
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// ---- large products: pairs of CTAs ---------------------------------------------
//
// out[m * ldo + n] = sum_r A[m][r] B[n][r] in tiles of 256 (m) x bn (n): one
// tcgen05.mma of a CTA pair per 16 of r, each CTA loading its 128 rows of A
// and half the rows of B.  A piece of 64 r costs each SM 32 KB of loads
// (bn = 256) for 512 cycles of MMA; the same tile on one SM would load 48.
// Pairs walk the tiles (persistent); two accumulators in tensor memory let
// eight epilogue warps work on one tile while the MMAs fill the other.  An
// epilogue warp takes 32 rows x 32 columns at a time, half of the columns in
// one go: tensor memory (read one step ahead) -> registers -> one of its two
// slots of shared memory -> one TMA store.  (On 4096 x 2816 x 11264 with GELU-tanh,
// pre and bias: rows read back from shared memory and stored by the warp 220
// us, each lane storing its row from registers, 32 bytes at a time, 203 us,
// where TMA stores took 168: both put 8 to 32 lines into an instruction.)
//
// Bound by the tensor cores: that product with GELU-tanh takes 148 - 154 us
// (1.72 PFLOP/s), without pre and activation 140 (1.85 PFLOP/s), its MMAs
// alone 133.  The rest is 184 MB of outputs, the last round of tiles and its
// epilogue.
//
// split > 1: a cluster of `split` pairs shares one tile's reduction.
//
// A launch takes one product or two: dx and dW, whose own launches would each
// leave SMs idle in their last round and pay the start twice, or the wide and
// the narrow tiles of one (mixed_columns).
constexpr int kPairThreads = 320;  // producer, MMA, eight epilogue warps
constexpr int kPairRing = 6;    // pieces of 64 r of both operands in shared memory
// A stage, which is loaded, awaited and released as one, has one piece where
// tiles have kPairWide columns or more: the ring is refilled sooner (4096 x
// 11264 x 2816: 153 -> 148 us, 4096 x 2816 x 11264: 153.5 -> 151.5).  Two
// pieces halve the barriers for narrower tiles, whose MMAs take less time than
// a barrier's round (160 columns, 2000 x 1024 x 3000: 15.0 us, 16.3 with one;
// 64 columns, 300 x 2560 x 2560: 12.5, 15.2 with one).
constexpr int kPairWide = 224;
constexpr int kPairMaxSplit = 4;     // a cluster of eight CTAs

struct PairCtrl {
    uint64_t full[kPairRing];
    uint64_t empty[kPairRing];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem_base;
    int abort_flag;
};

struct PairArgs {
    CUtensorMap a[2], b[2], out[2], pre[2];
    LinArgs p[2];
    int tiles[2];       // 0 for an absent second product
    int bn;             // the larger of the two
    int cut;            // a sum is cut into chains, see chain_steps
    uint32_t sub_bytes; // of shared memory for 64 r of both operands
    uint32_t slot;      // bytes of one slot of an epilogue warp
    // Pair q of the grid's first takes tiles q, q + pairs, ... of product 0;
    // the `extra` pairs that get one more of them take at most `shared`
    // tiles of product 1, the others what is left.
    int shared;
    // sums of `chunks` rows of partial column sums, or null
    const float *part;
    float *db;
    int chunks, db_n;
};

struct PairArgsExtra : PairArgs {
    CUtensorMap a2[2];  // the second piece of X, if any
};

template <bool EXTRA>
using PairArgsOf = std::conditional_t<EXTRA, PairArgsExtra, PairArgs>;

// What one CTA loads of B per 64 r.
__host__ __device__ __forceinline__ uint32_t pair_b_bytes(int bn, int b_mn)
{
    const int half = bn / 2;
    return uint32_t(b_mn ? (half + 63) / 64 * 64 : half) * (LK * 2);
}

// SUB: pieces of a stage.  EXTRA: as k_linear's.
template <int SUB, bool EXTRA>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_linear_pair(const __grid_constant__ PairArgsOf<EXTRA> g)
{
    extern __shared__ uint8_t smem_raw[];
    // the same offset in every CTA: dynamic shared memory starts at the same address
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ PairCtrl ctl;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    const uint32_t rank = crank & 1u, lead = crank & ~1u;  // place in the pair, its even CTA
    const int z = int(crank >> 1), Z = g.p[0].split;
    constexpr int S = kPairRing / SUB;
    const uint32_t sub_bytes = g.sub_bytes;
    uint8_t *stg = smem + kPairRing * sub_bytes;
    // two accumulators and, where chains are cut, the sum of the earlier ones
    const uint32_t tmem_need = uint32_t(g.bn) * (g.cut ? 3 : 2);
    const uint32_t tmem_cols = tmem_need <= 128 ? 128u : tmem_need <= 256 ? 256u : 512u;
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
        for (int i = 0; i < (g.tiles[1] ? 2 : 1); ++i) {
            prefetch_tmap(&g.a[i]);
            prefetch_tmap(&g.b[i]);
        }
    }
    __syncwarp();
    cluster_arrive();
    if (warp == 1)
        tmem_alloc_pair(&ctl.tmem_base, tmem_cols);
    tc_fence_before_sync();
    __syncthreads();
    cluster_wait();  // the other CTAs' barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    // The pair's i-th tile: its product and its place there; false past the
    // last.  Tiles of a product are numbered in blocks of 16 m tiles, m
    // fastest: the pairs running at one time share few rows of both operands
    // (the product above takes 151.5 us so, 155 with blocks of 8 or 11).
    const int pairs = int(gridDim.x) / (2 * Z), pair = int(blockIdx.x) / (2 * Z);
    struct Tile {
        int which, m0, n0, nk0, nk1;
    };
    auto tile_at = [&](int i, Tile &o) {
        const int extra = g.tiles[0] % pairs;
        const int mine = g.tiles[0] / pairs + (pair < extra ? 1 : 0);
        int t;
        o.which = i < mine ? 0 : 1;
        if (i < mine) {
            t = pair + i * pairs;
        } else {
            const int j = i - mine;
            if (j >= g.shared && pair < extra)
                return false;
            t = j < g.shared ? j * pairs + pair
                             : g.shared * pairs + (j - g.shared) * (pairs - extra) + pair - extra;
            if (t >= g.tiles[1])
                return false;
        }
        const LinArgs &p = g.p[o.which];
        const int n_nt = (p.N + p.bn - 1) / p.bn, block = 16 * n_nt;
        const int b = t / block, tall = min(16, p.n_mt - 16 * b), u = t - b * block;
        o.n0 = u / tall * p.bn;
        o.m0 = (16 * b + u % tall) * (2 * LM);
        const int nk = (p.R + LK - 1) / LK << (EXTRA ? p.two : 0);
        o.nk0 = int(int64_t(nk) * z / Z);
        o.nk1 = int(int64_t(nk) * (z + 1) / Z);
        return true;
    };
    Tile w;

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        const bool one = elect_one();
        bool ok = true;
        for (int i = 0; ok && tile_at(i, w); ++i) {
            const LinArgs &p = g.p[w.which];
            const CUtensorMap *map_b = &g.b[w.which];
            const int a_mn = p.a_mn, b_mn = p.b_mn, half = p.bn / 2;
            const uint32_t tx = 2 * (kLinATile + pair_b_bytes(p.bn, b_mn));
            const int m0 = w.m0 + int(rank) * LM, n0 = w.n0 + int(rank) * half;
            for (int kb = w.nk0; kb < w.nk1; kb += SUB) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag));
                if (!ok)
                    break;
                if (one) {
                    const int subs = min(SUB, w.nk1 - kb);
                    if (rank == 0) {  // both CTAs' bytes complete on the even CTA's barrier
                        const bool stall = EXTRA && p.stall && p.stall - 1 == int(blockIdx.x) &&
                                           i == 0 && kb == w.nk0;
                        mbar_arrive_expect_tx(&ctl.full[stage],
                                              uint32_t(subs) * tx + (stall ? 16u : 0u));
                    }
                    const uint32_t fb = dsmem_addr(&ctl.full[stage], lead);
#pragma unroll
                    for (int h = 0; h < SUB; ++h) {
                        if (h >= subs)
                            break;
                        uint8_t *sa = smem + (stage * SUB + h) * sub_bytes;
                        uint8_t *sb = sa + kLinATile;
                        const CUtensorMap *map_a = &g.a[w.which];
                        int step = kb + h;
                        if constexpr (EXTRA) {
                            const int nk1 = (p.R + LK - 1) / LK;  // of a piece
                            if (step >= nk1)
                                map_a = &g.a2[w.which], step -= nk1;
                        }
                        const int k0 = step * LK;
                        if (a_mn) {  // 64 m x 64 r boxes, m contiguous
                            tma_load_2d_pair(sa, map_a, fb, m0, k0);
                            tma_load_2d_pair(sa + 8192, map_a, fb, m0 + 64, k0);
                        } else {
                            tma_load_2d_pair(sa, map_a, fb, k0, m0);
                        }
                        if (b_mn) {
                            for (int c = 0; c < half; c += 64)
                                tma_load_2d_pair(sb + c * (LK * 2), map_b, fb, n0 + c, k0);
                        } else {
                            tma_load_2d_pair(sb, map_b, fb, k0, n0);
                        }
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every stage released: this CTA's copies have landed and been read
        for (int i = 0; ok && i < S; ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag));
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
    } else if (warp == 1 && rank == 0) {
        // The whole warp walks the loop and one lane issues, so that
        // descriptors and addresses stay warp-uniform (issued from inside an
        // `if (lane == 0)` loop, a stage of four MMAs took about 690 cycles
        // where the tensor core needs 512).
        int stage = 0, buf = 0;
        uint32_t phase = 0, aphase = 0;
        const uint32_t sa = smem_u32(smem), sb = sa + kLinATile;
        const bool one = elect_one();
        bool ok = true;
        for (int i = 0; ok && tile_at(i, w); ++i) {
            const LinArgs &p = g.p[w.which];
            uint32_t idesc =
                idesc_bf16_f32(2 * LM, uint32_t(p.bn), uint32_t(p.a_mn), uint32_t(p.b_mn));
            if (p.f16)
                idesc &= ~((7u << 7) | (7u << 10));
            const uint64_t da0 = smem_desc_sw128(sa, p.a_mn ? 8192 : 16, 1024);
            const uint64_t db0 = smem_desc_sw128(sb, p.b_mn ? 8192 : 16, 1024);
            const uint32_t ia = p.a_mn ? 128 : 2, ib = p.b_mn ? 128 : 2;
            const int chain = p.chain;
            uint32_t d = 0;
            int left = 0;  // steps to go in this chain
            for (int kb = w.nk0; kb < w.nk1; kb += SUB) {
                const bool start = left == 0;
                if (start) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&ctl.acc_empty[buf], aphase ^ 1u, abort_flag));
                    if (!ok)
                        break;
                    d = tmem_base + uint32_t(buf * g.bn);
                    left = chain;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[stage], phase, abort_flag));
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (one) {
#pragma unroll
                    for (int h = 0; h < SUB; ++h) {
                        const uint32_t off = uint32_t(stage * SUB + h) * (sub_bytes >> 4);
                        if (kb + h < w.nk1) {
#pragma unroll
                            for (uint32_t kk = 0; kk < LK / 16; ++kk)
                                tc_mma_f16_pair(d, da0 + (off + kk * ia), db0 + (off + kk * ib),
                                                idesc, !start || h != 0 || kk != 0);
                        }
                    }
                    tc_commit_pair(&ctl.empty[stage], uint16_t(3u << lead));
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                left -= SUB;
                if (left <= 0 || kb + SUB >= w.nk1) {  // the chain is complete
                    left = 0;
                    if (one)
                        tc_commit_pair(&ctl.acc_full[buf], uint16_t(3u << lead));
                    __syncwarp();
                    if (++buf == 2) {
                        buf = 0;
                        aphase ^= 1u;
                    }
                }
            }
        }
        // (the epilogue warps of both CTAs wait for every accumulator, so the
        // MMAs are done when the cluster meets below)
    } else if (warp >= 2) {
        if (g.db) {  // while the first tile is on its way
            const int threads = 32 * kPairEpiWarps;
            for (int64_t c = int64_t(blockIdx.x) * threads + int(threadIdx.x) - 64; c < g.db_n;
                 c += int64_t(gridDim.x) * threads) {
                float v = 0.0f;
#pragma unroll 8
                for (int i = 0; i < g.chunks; ++i)
                    v += g.part[int64_t(i) * g.db_n + c];
                g.db[c] = v;
            }
            __syncwarp();
        }
        const int q = warp & 3, part = (warp - 2) >> 2;  // TMEM lane quadrant; even or odd 32 columns
        EpiMemory mem{stg + uint32_t(warp - 2) * 2 * g.slot, g.slot,
                      reinterpret_cast<float *>(stg + kPairEpiWarps * 2 * g.slot) + (warp - 2) * 32,
                      0, true};
        int buf = 0;
        uint32_t aphase = 0;
        for (int i = 0; Z == 1 && tile_at(i, w); ++i) {
            const LinArgs &p = g.p[w.which];
            const uint32_t flags = p.flags;
            const int n0 = w.n0, chain = p.chain;
            const int64_t row = int64_t(w.m0) + int(rank) * LM + q * 32;
            const int rows = int(min(int64_t(32), p.M - row)), width = min(p.bn, p.N - n0);
            const float *bias_at = flags & kEpiBias ? p.bias + n0 + lane : nullptr;
            auto bias_of = [&](int c) {
                return bias_at && c + int(lane) < width ? bias_at[c] : 0.0f;
            };
            float bias = bias_of(part * 32);
            const uint32_t lanes = tmem_base + (uint32_t(q * 32) << 16);
            auto release = [&] {  // this accumulator has been read
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(dsmem_addr(&ctl.acc_empty[buf], lead));
                if (++buf == 2) {
                    buf = 0;
                    aphase ^= 1u;
                }
            };
            bool ok = true;
            // a sum cut into chains is put together in tensor memory
            int chains = (w.nk1 - w.nk0 + chain - 1) / chain;
            const bool cut = chains > 1;
            const uint32_t t1 = lanes + uint32_t(2 * g.bn);
            for (bool sum = false; cut && chains > 0; --chains, sum = true) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.acc_full[buf], aphase, abort_flag));
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t t0 = lanes + uint32_t(buf * g.bn);
                add_chain(t0, t1, part * 32, width, sum);
                release();
            }
            const uint32_t t0 = cut ? t1 : lanes + uint32_t(buf * g.bn);
            uint32_t r[kCols];
            const bool some = rows > 0 && part * 32 < width;
#pragma unroll 1
            for (int c = part * 32; c == part * 32 || c < width; c += 32 * kPairParts) {
                const int cols = min(32, width - c);
                // (before a tile's first, another product's stores, perhaps)
                mem.strict = (flags & kEpiPre) || c == part * 32;
                uint8_t *slot = mem.take(), *pre = slot;
                if (flags & kEpiPre)
                    pre = mem.take();
                if ((flags & kEpiResidual) && some) {
                    const int64_t at = row * p.ldr + n0 + c;
                    if (flags & kEpiF32)
                        load_slot<float>(slot, p.residual, at, p.ldr, rows, cols,
                                         flags & kEpiVecRes);
                    else
                        load_slot<uint16_t>(slot, p.residual, at, p.ldr, rows, cols,
                                            flags & kEpiVecRes);
                }
                if (flags & kEpiBias)
                    mem.bias[lane] = bias;
                __syncwarp();
                if (c == part * 32) {
                    if (!cut)
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(&ctl.acc_full[buf], aphase, abort_flag));
                    if (!ok || !some)
                        break;
                    tc_fence_after_sync();
                    tmem_ld_32x32b_x16(t0 + uint32_t(c), r);
                }
                const int next = c + 32 * kPairParts;
                if (next < width)
                    bias = bias_of(next);
#pragma unroll 1
                for (int h = 0; h < 32; h += kCols) {
                    float v[kCols];
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        v[j] = __uint_as_float(r[j]);
                    const int ahead = h + kCols < 32 ? c + h + kCols : next;
                    if (ahead < width)
                        tmem_ld_32x32b_x16(t0 + uint32_t(ahead), r);
                    pair_cols<EXTRA>(flags, p.mul, mem.bias + h, pre, slot, h, v);
                }
                if (flags & kEpiPre)
                    store_slot<uint16_t>(pre, &g.pre[w.which], p.pre, row, n0 + c, p.ldp, rows, cols,
                                         flags & kEpiVecPre);
                if (flags & kEpiF32)
                    store_slot<float>(slot, &g.out[w.which], p.out, row, n0 + c, p.ldo, rows, cols,
                                      flags & kEpiVecOut);
                else
                    store_slot<uint16_t>(slot, &g.out[w.which], p.out, row, n0 + c, p.ldo, rows,
                                         cols, flags & kEpiVecOut);
            }
            if (!ok)
                break;
            if (!cut)
                release();
        }
        if (lane == 0)
            bulk_wait<0>();  // every store written before the CTA (and its memory) goes
    }
    __syncwarp();
    if (Z > 1) {
        // One tile per cluster; each pair has summed its share of r.  CTA z
        // of the Z that hold the same rows finishes 128 / Z of them: every
        // CTA sends it its sums of those rows (into memory beside the ring,
        // which may still be in use there), and it adds them in rank order.
        const LinArgs &p = g.p[0];
        tile_at(0, w);
        const int bn = p.bn, n0 = w.n0;
        float *acc = reinterpret_cast<float *>(stg);  // [Z][128 / Z][pitch]
        const int pitch = bn + 4, slice = LM / Z;     // float4 rows, conflict-free
        // what a thread finishes: four neighbouring columns, always the same, of
        // every `by`-th row
        const int quads = bn / 4, t = int(threadIdx.x), by = kPairThreads / quads;
        const int n = t % quads * 4, left = min(4, p.N - (n0 + n));
        float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bias[i] = i < left ? p.bias[n0 + n + i] : 0.0f;
        }
        if (warp >= 2) {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&ctl.acc_full[0], 0, abort_flag));
            const int q = warp & 3, part = (warp - 2) >> 2, m = q * 32 + int(lane);
            tc_fence_after_sync();
            const uint32_t t0 = tmem_base + (uint32_t(q * 32) << 16);
            const uint32_t to =
                dsmem_addr(acc + (z * slice + m % slice) * pitch, 2 * uint32_t(m / slice) + rank);
#pragma unroll 1
            for (int c = part * 64; c < bn; c += 64 * kPairParts) {
                uint32_t r[2][32] = {};
                if (ok) {
                    tmem_ld_32x32b_x32(t0 + uint32_t(c), r[0]);
                    tmem_ld_32x32b_x32(t0 + uint32_t(c) + 32, r[1]);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int j = 0; j < 64; j += 4)
                    dsmem_st4(to + (c + j) * 4, r[j >> 5][j & 31], r[j >> 5][(j & 31) + 1],
                              r[j >> 5][(j & 31) + 2], r[j >> 5][(j & 31) + 3]);
            }
            tc_fence_before_sync();
        }
        __syncwarp();
        cluster_sync();
        const int m0 = w.m0 + int(rank) * LM + z * slice;
        const int rows = min(slice, p.M - m0);
        if (left > 0) {
            constexpr int kBatch = 4;
#pragma unroll 1
            for (int m = t / quads; m < rows; m += kBatch * by) {
                float v[kBatch][4];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[i][j] = 0.0f;
                    const float *a = acc + min(m + i * by, slice - 1) * pitch + n;
#pragma unroll
                    for (int r = 0; r < kPairMaxSplit; ++r)
                        if (r < Z) {
                            const float4 o =
                                *reinterpret_cast<const float4 *>(a + r * slice * pitch);
                            v[i][0] += o.x, v[i][1] += o.y, v[i][2] += o.z, v[i][3] += o.w;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[i][j] += bias[j];
                }
                if (EXTRA && p.mul) {
                    const float mul = *p.mul;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[i][j] *= mul;
                }
                finish_rows<kBatch>(p, v, int64_t(m0) + m, by, rows - m, n0 + n, left);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x == 0 && ctl.abort_flag)
        report_timeout(g.p[0].status);
    __syncwarp();
    cluster_sync();  // the CTAs are done with each other's shared memory and barriers
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, tmem_cols);
    }
}

// ---- dP and db ---------------------------------------------------------------

constexpr int kGradThreads = 256;
constexpr int kGradGroups = 8;       // rows of a CTA side by side, one per warp
constexpr int kGradCols = 256;       // columns of a CTA: 32 lanes x 8
constexpr int kGradUnroll = 2;       // rows of a warp in flight
constexpr int kGradMaxChunks = 128;  // rows of partial column sums

struct GradArgs {
    const void *dy, *pre;
    uint16_t *dp;     // null: not written
    uint16_t *dp2;    // what dp's rounding leaves, rounded; null: not written
    float *part;      // [chunks][N] or null
    const uint32_t *maxima;  // [kMaxima] of |dy| by k_dy_max: dp and dp2 are scaled; or null
    float *unscale;          // receives 1 / scale
    int64_t lddy, lddp;
    int T, N, rows;   // rows per chunk
    int vec;          // 16-byte accesses of dy and pre are aligned
};

// Eight neighbouring elements, the first `n` of which exist.
template <bool F32>
struct Eight {
    uint4 q[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void *p, int64_t at, int n, bool vec)
    {
        if (vec && n == 8) {
            const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) +
                                                             at * (F32 ? 4 : 2));
            q[0] = __ldcs(v);  // read once: leave the cache to dP
            if (F32)
                q[F32 ? 1 : 0] = __ldcs(v + 1);
            return;
        }
        uint32_t w[F32 ? 8 : 4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                if (F32)
                    w[F32 ? i : 0] = static_cast<const uint32_t *>(p)[at + i];
                else
                    w[i >> 1] |= uint32_t(static_cast<const uint16_t *>(p)[at + i])
                                 << (16 * (i & 1));
            }
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (F32)
            q[F32 ? 1 : 0] = make_uint4(w[F32 ? 4 : 0], w[F32 ? 5 : 0], w[F32 ? 6 : 0], w[F32 ? 7 : 0]);
    }

    __device__ __forceinline__ void to(float (&v)[8], int f16) const
    {
        const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
        if constexpr (F32) {
            const uint32_t u[4] = {q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(w[i]);
                v[i + 4] = __uint_as_float(u[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack16(w[i], f16);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

// fp32 gradients reach below fp16's range (losses that are means over many
// tokens), so for fp16 operands dP is multiplied by a power of two that takes
// the largest finite |dy| to 2^13 ... 2^14 (|act'| <= 1.13): what is 2^-27 of
// the largest keeps all its bits, and products are multiplied by the
// reciprocal in fp32.  k_dy_max gives each CTA's maximum, as the bits of a float.
constexpr int kMaxima = 256;
constexpr int kMaxThreads = 256;

__global__ void __launch_bounds__(kMaxThreads)
    k_dy_max(const float *dy, int64_t ld, int T, int N, int vec, uint32_t *maxima)
{
    __shared__ uint32_t red[kMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    uint32_t m = 0;
    auto take = [&](uint32_t v) {
        v &= 0x7fffffffu;
        m = max(m, v < 0x7f800000u ? v : 0u);
    };
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const uint32_t *row = reinterpret_cast<const uint32_t *>(dy + t * ld);
        int n = 0;
        if (vec) {
            n = N / 4 * 4;
            for (int c = int(threadIdx.x) * 4; c < n; c += kMaxThreads * 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(row + c);
                take(v.x), take(v.y), take(v.z), take(v.w);
            }
        }
        for (int c = n + int(threadIdx.x); c < N; c += kMaxThreads)
            take(row[c]);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kMaxThreads / 32; ++i)
            m = max(m, red[i]);
        maxima[blockIdx.x] = m;
    }
}

__device__ __forceinline__ float pow2(int e)  // -126 <= e <= 127
{
    return __int_as_float((e + 127) << 23);
}

// dP = dy act'(pre), and the column sums of one chunk of rows.  A warp takes
// every eighth row of the chunk, eight columns a lane, two rows' loads in
// flight; the warps' sums are added in order.  Bound by memory: dy and pre
// are read and dP written once: 48 us for 4096 x 11264 (5.8 TB/s, 0.85 of a
// copy's), at 26 instructions an element with six tenths of the issue slots
// taken (58 with the 16-bit type chosen at run time, 32 instructions).  Four
// CTAs an SM with two rows in flight each; two CTAs with four rows took a
// seventh longer.
//
// From an fp32 dy, dP may be written in two pieces (its value in 16 bits, and
// what that leaves), for a product that is wanted in more than 16 bits.
template <int ACT, bool F32, bool F16>
__global__ void __launch_bounds__(kGradThreads, 4) k_act_grad(GradArgs p)
{
    __shared__ float red[kGradGroups][kGradCols];
    __shared__ uint32_t most;
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * kGradCols + lane * 8;
    const int left = min(8, p.N - c);
    pdl_wait();
    pdl_launch_dependents();
    float scale = 1.0f;
    if (F32 && F16 && p.maxima) {
        if (threadIdx.x == 0)
            most = 0;
        __syncthreads();
        static_assert(kMaxima == kGradThreads, "a maximum per thread");
        const uint32_t m = __reduce_max_sync(0xffffffffu, p.maxima[threadIdx.x]);
        if (lane == 0)
            atomicMax(&most, m);
        __syncthreads();
        // (subnormal maxima count as 2^-126)
        const int e = most ? min(13 - (max(int(most >> 23), 1) - 127), 126) : 0;
        scale = pow2(e);
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            *p.unscale = pow2(-e);
    }
    const int64_t t0 = int64_t(blockIdx.y) * p.rows;
    const int64_t t1 = min(int64_t(p.T), t0 + p.rows);
    float s[8] = {};
    if (left > 0)
        for (int64_t t = t0 + g; t < t1; t += kGradGroups * kGradUnroll) {
            Eight<F32> dy[kGradUnroll];
            Eight<false> pre[kGradUnroll];
#pragma unroll
            for (int u = 0; u < kGradUnroll; ++u) {
                const int64_t r = t + u * kGradGroups;
                if (r < t1) {
                    dy[u].load(p.dy, r * p.lddy + c, left, p.vec);
                    if (ACT != MOE_ACT_NONE)
                        pre[u].load(p.pre, r * p.N + c, left, p.vec);
                }
            }
#pragma unroll
            for (int u = 0; u < kGradUnroll; ++u) {
                const int64_t r = t + u * kGradGroups;
                if (r >= t1)
                    break;
                float d[8];
                dy[u].to(d, F16);
                if (ACT != MOE_ACT_NONE) {
                    float z[8];
                    pre[u].to(z, F16);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] *= act_grad<ACT>(z[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i] += d[i];  // 0 past N
                if (p.dp) {  // lddp is a multiple of 8: whole vectors, past N too
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (F32 && F16) {
                            d[2 * i] *= scale;
                            d[2 * i + 1] *= scale;
                        }
                        w[i] = pack16(d[2 * i], d[2 * i + 1], F16);
                    }
                    *reinterpret_cast<uint4 *>(p.dp + r * p.lddp + c) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                    if (F32 && p.dp2) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = unpack16(w[i], F16);
                            // (0 beside an infinity, which is itself enough)
                            const float a = d[2 * i] - f.x, b = d[2 * i + 1] - f.y;
                            w[i] = pack16(fabsf(a) < INFINITY ? a : 0.0f,
                                          fabsf(b) < INFINITY ? b : 0.0f, F16);
                        }
                        *reinterpret_cast<uint4 *>(p.dp2 + r * p.lddp + c) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[g][lane * 8 + i] = s[i];
    __syncthreads();
    const int col = blockIdx.x * kGradCols + threadIdx.x;
    if (col < p.N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kGradGroups; ++i)
            v += red[i][threadIdx.x];
        p.part[int64_t(blockIdx.y) * p.N + col] = v;
    }
}

// db: the chunks' column sums; a CTA takes 32 columns, its warps every eighth
// chunk, added in order.
__global__ void __launch_bounds__(kGradThreads)
    k_col_sum(const float *part, int chunks, int N, float *db)
{
    __shared__ float red[kGradGroups][32];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float v = 0.0f;
    if (c < N) {
#pragma unroll 8
        for (int i = g; i < chunks; i += kGradGroups)
            v += part[int64_t(i) * N + c];
    }
    red[g][lane] = v;
    __syncthreads();
    if (g == 0 && c < N) {
#pragma unroll
        for (int i = 1; i < kGradGroups; ++i)
            v += red[i][lane];
        db[c] = v;
    }
}

using GradKernel = void (*)(GradArgs);

template <int ACT>
GradKernel act_grad_kernel(bool f32, bool f16)
{
    if (f32)
        return f16 ? k_act_grad<ACT, true, true> : k_act_grad<ACT, true, false>;
    return f16 ? k_act_grad<ACT, false, true> : k_act_grad<ACT, false, false>;
}

GradKernel act_grad_kernel(int act, bool f32, bool f16)
{
    switch (act) {
    case MOE_ACT_RELU:
        return act_grad_kernel<MOE_ACT_RELU>(f32, f16);
    case MOE_ACT_SILU:
        return act_grad_kernel<MOE_ACT_SILU>(f32, f16);
    case MOE_ACT_GELU:
        return act_grad_kernel<MOE_ACT_GELU>(f32, f16);
    case MOE_ACT_GELU_TANH:
        return act_grad_kernel<MOE_ACT_GELU_TANH>(f32, f16);
    default:
        return act_grad_kernel<MOE_ACT_NONE>(f32, f16);
    }
}

// ---- host ---------------------------------------------------------------------

// A 16-bit matrix as stored: rows x cols, cols contiguous, rows ld elements apart.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;
};

// Its tensor map: boxes of 64 columns x box_rows rows with the 128-byte swizzle.
cudaError_t lin_map(CUtensorMap *m, const Operand &o, int box_rows, int f16)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(o.cols), cuuint64_t(o.rows)};
    const cuuint64_t strides[1] = {cuuint64_t(o.ld) * 2};
    const cuuint32_t box[2] = {LK, cuuint32_t(box_rows)}, estr[2] = {1, 1};
    const CUresult r =
        encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void *>(o.p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// out[i][j] = sum_r X[i][r] Y[j][r], with a's epilogue fields.  With a.two, X is
// the sum of X and a matrix of the same shape at X2.
struct Product {
    Operand X, Y;
    bool x_mn, y_mn;  // i (j) is contiguous, not r
    int rows, cols, R;
    LinArgs a;
    const void *X2;

    int steps() const { return (R + LK - 1) / LK << a.two; }  // of 64 r
    Operand second() const { return {a.two ? X2 : X.p, X.rows, X.cols, X.ld}; }
};

// Dynamic shared memory of a launch of k_linear_pair whose tiles take
// `sub_bytes` per 64 r: the ring, and the epilogue's slots (4 KB where an
// output is fp32) or the parts of a split tile.  A CTA has 227 KB at most, a
// few hundred bytes of them static: tilings that need more than kPairSmem are
// not chosen.
constexpr size_t kPairSmem = 226 * 1024;

uint32_t pair_sub_bytes(int bn, int b_mn)
{
    return kLinATile + pair_b_bytes(bn, b_mn);
}

uint32_t pair_slot(bool f32)
{
    return f32 ? 4096 : 2048;
}

size_t pair_smem(uint32_t sub_bytes, int bn, int split, bool f32)
{
    return 1024 + size_t(kPairRing) * sub_bytes +
           (split > 1 ? size_t(LM) * (bn + 4) * 4
                      : size_t(kPairEpiWarps) * (2 * pair_slot(f32) + 128));
}

// Tiling of a product, chosen by estimated SM cycles.
struct Tiling {
    bool pair;
    int bn, split;
    int64_t tiles;
    double tile_cycles, cycles;  // of a tile, of the product
};

// What a tile of k_linear_pair takes per 64 of r, from times at bn = 64 ...
// 256 (4096 x 2816 x 11264: 144 us at 256, 154 at 192, 183 at 128).
double pair_step(int bn, bool y_mn)
{
    return 200.0 + 1.65 * (2.0 * pair_b_bytes(bn, y_mn) / (LK * 2));
}

// A tile's epilogue hides behind the next tile's MMAs, except the last one's.
// It takes about 9700 cycles for 256 plain columns (17000 with GELU-tanh and
// pre), of which a part does not depend on the columns.  (Counted as 1500 per
// 64 columns, reductions of 128 and 256 took a third longer; as 2400, 4096 x
// 512 x 8192 took 69 us instead of 42.)  Starting takes about 5000 cycles, and
// joining the parts of a split tile about 8000.
constexpr double kStartCycles = 5000.0, kJoinCycles = 8000.0;
constexpr double kEpiStart = 2500.0, kEpiCycles = 1800.0;
// Three times as many columns fit tensor memory.  (Of a Y whose j is
// contiguous, half of 160 columns is loaded as 128: shared memory holds no
// more than 128 of those columns beside fp32 slots, see pair_smem.)
constexpr int kCutMaxBn = 160;

bool is_cut(const Product &q)
{
    return q.steps() > chain_steps(q.a.out_f32, q.a.f16);
}

double epi_cycles(int bn)
{
    return kEpiStart + kEpiCycles * ((bn + 63) / 64);
}

// A tile of one pair, unsplit, while others follow.
double tile_cycles(const Product &q, int bn)
{
    return std::max(pair_step(bn, q.y_mn) * q.steps(), epi_cycles(bn));
}

// f32: an output of the launch is; cut: a sum of the launch is, into chains.
Tiling choose_tiling(const Product &q, int sms, bool f32, bool cut)
{
    Tiling t{false, 0, 1, 0, 0.0, 0.0};
    if (q.rows <= 128)
        return t;
    const int nk = q.steps(), pairs = std::max(1, sms / 2);
    for (int bn = f32 || cut ? kCutMaxBn : 256; bn >= 64; bn -= 32) {
        if (pair_smem(pair_sub_bytes(bn, q.y_mn), bn, 1, f32) > kPairSmem)
            continue;
        const int64_t tiles =
            ((int64_t(q.rows) + 255) / 256) * ((int64_t(q.cols) + bn - 1) / bn);
        for (int z = 1; z <= kPairMaxSplit; z *= 2) {
            // a split tile needs room for the parts beside the ring
            if (z > 1 && (nk / z < 4 || tiles * z > pairs || (bn != 64 && bn != 128)))
                break;
            if (z > 1 && (nk + z - 1) / z > chain_steps(q.a.out_f32, q.a.f16))
                continue;  // its chains are not cut further
            const double main = pair_step(bn, q.y_mn) * ((nk + z - 1) / z);
            const int64_t waves = (tiles + pairs - 1) / pairs;
            const double c = kStartCycles + main + (z > 1 ? kJoinCycles : epi_cycles(bn)) +
                             double(waves - 1) * tile_cycles(q, bn);
            if (!t.pair || c < t.cycles)
                t = Tiling{true, bn, z, tiles, tile_cycles(q, bn), c};
        }
    }
    return t;
}

// Tiles t0 of c0 cycles and then t1 of c1 on `pairs` pairs, as k_linear_pair
// takes them: the cycles until the last is done, and the `shared` for it.
double two_parts(int64_t t0, double c0, int64_t t1, double c1, int64_t pairs, int &shared)
{
    const int64_t per = t0 / pairs, extra = t0 % pairs, others = pairs - extra;
    double best = 0.0;
    for (int64_t s = 0; s <= (t1 + pairs - 1) / pairs; ++s) {
        const int64_t rest = std::max<int64_t>(0, t1 - s * pairs);
        const double more = extra ? (per + 1) * c0 + std::min(s, t1) * c1 : 0.0;
        const double c = std::max(more, per * c0 + (s + (rest + others - 1) / others) * c1);
        if (s == 0 || c < best) {
            best = c;
            shared = int(s);
        }
    }
    return best;
}

// Columns of the product to leave to narrower tiles, so that its last round
// is fuller and its last epilogue shorter; 0 if that gains nothing.  (4096 x
// 2816 x 11264 with GELU-tanh and pre: 704 tiles of 256 columns are 9.3 rounds
// of 76 pairs, 161 us; 656 and 96 of half the width end after 9.7, 155 us.
// 4096 x 512 x 8192: 46.8 -> 41.5, 2048 x 10240 x 2560: 89.7 -> 85.4.)
int64_t mixed_columns(const Product &q, int sms, const Tiling &t, Tiling &narrow)
{
    const int64_t pairs = std::max(1, sms / 2), n_mt = (int64_t(q.rows) + 255) / 256;
    if (!t.pair || t.split != 1 || t.tiles <= pairs)
        return 0;
    const int64_t n_nt = (q.cols + t.bn - 1) / t.bn;
    double best = t.cycles;
    int64_t columns = 0;
    // at most two rounds' worth of wide tiles are replaced
    for (int64_t j = std::max<int64_t>(1, n_nt - 2 * pairs / n_mt - 1); j < n_nt; ++j)
        for (int bn : {64, 96, 128, 192}) {
            if (bn >= t.bn)
                break;
            const int64_t left = q.cols - j * t.bn;
            const int64_t tiles = n_mt * ((left + bn - 1) / bn);
            const double each = tile_cycles(q, bn);
            int shared;
            const double c = kStartCycles + epi_cycles(bn) +
                             two_parts(n_mt * j, t.tile_cycles, tiles, each, pairs, shared);
            if (c < best) {
                best = c;
                columns = left;
                narrow = Tiling{true, bn, 1, tiles, each, c};
            }
        }
    return columns;
}

// Columns [from, from + cols) of a product, `from` a multiple of 32.
Product columns_of(const Product &q, int64_t from, int64_t cols)
{
    Product o = q;
    const auto at = [&](const void *p, int64_t n) {
        return p ? static_cast<uint8_t *>(const_cast<void *>(p)) + n : nullptr;
    };
    const int64_t size = q.a.out_f32 ? 4 : 2;
    o.cols = int(cols);
    (q.y_mn ? o.Y.cols : o.Y.rows) = cols;
    o.Y.p = at(q.Y.p, from * 2 * (q.y_mn ? 1 : q.Y.ld));
    o.a.bias = reinterpret_cast<const float *>(at(q.a.bias, from * 4));
    o.a.residual = at(q.a.residual, from * size);
    o.a.pre = at(q.a.pre, from * 2);
    o.a.out = at(q.a.out, from * size);
    return o;
}

// k_linear's arguments and shared memory for a product, and its CTAs.
LinArgs small_args(const Product &q, int sms, int64_t &ctas, size_t &smem)
{
    const int nk = q.steps();
    LinArgs a = q.a;
    a.M = q.cols, a.N = q.rows, a.R = q.R;
    a.a_mn = q.y_mn, a.b_mn = q.x_mn;
    a.chain = chain_steps(a.out_f32, a.f16);
    // (128 columns leave no room for a second chain)
    a.bn = q.rows <= 16 ? 16 : q.rows <= 32 ? 32 : q.rows <= 64 || nk > a.chain || a.out_f32 ? 64
                                                                                            : 128;
    a.n_mt = (q.cols + LM - 1) / LM;
    const int64_t tiles = int64_t(a.n_mt) * ((int64_t(q.rows) + a.bn - 1) / a.bn);
    // split the reduction while the CTAs still fit at once and each has at
    // least four stages, or until an fp32 output's chains have an accumulator
    // each
    const int fit = kSmallTmem / a.bn * a.chain;
    a.split = 1;
    while (a.split < kLinMaxSplit &&
           ((tiles * a.split * 2 <= 2 * sms && nk / (a.split * 2) >= 4) ||
            (a.out_f32 && nk > fit * a.split)))
        a.split *= 2;
    ctas = tiles * a.split;
    const uint32_t stage = kLinATile + lin_b_tile(a.bn, a.b_mn);
    // two CTAs an SM; the parts beside the ring, or in it at 128 columns
    const uint32_t parts = a.bn < LM ? uint32_t(LM) * (a.bn + 4) * 4 : 0;
    a.stages = std::min<int>(kLinMaxStages, (110 * 1024 - parts) / stage);
    smem = 1024 + size_t(a.stages) * stage + parts;
    return a;
}

constexpr size_t kSmallSmem = 112 * 1024;

cudaError_t launch_small(const Product &q, cudaStream_t s)
{
    int64_t ctas;
    size_t smem;
    LinArgs a = small_args(q, device_sm_count(), ctas, smem);
    if (ctas > INT_MAX)
        return cudaErrorInvalidValue;
    LinMaps<false> maps;
    LinMaps<true> more;
    cudaError_t e = lin_map(&maps.a, q.Y, q.y_mn ? LK : LM, a.f16);
    if (e == cudaSuccess)
        e = lin_map(&maps.b, q.X, q.x_mn ? LK : a.bn, a.f16);
    const bool extra = a.two || a.mul || a.stall;
    const void *kern = extra ? reinterpret_cast<const void *>(k_linear<true>)
                             : reinterpret_cast<const void *>(k_linear<false>);
    if (extra) {
        more.a = maps.a, more.b = more.b2 = maps.b;
        if (e == cudaSuccess && a.two)
            e = lin_map(&more.b2, q.second(), q.x_mn ? LK : a.bn, a.f16);
    }
    if (e == cudaSuccess)
        e = ensure_smem_limit(kern, extra ? kSlotLinearExtra : kSlotLinear, kSmallSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {extra ? static_cast<void *>(&more) : &maps, &a};
    return launch_clustered(kern, unsigned(ctas), unsigned(a.split), kLinThreads, smem, s, args);
}

struct ColSums {
    const float *part;
    float *db;
    int chunks, n;
};

// One or two products in one launch; both unsplit if two.
cudaError_t launch_pairs(const Product *q, const Tiling *t, int count, const ColSums &sums,
                         cudaStream_t s)
{
    const int sms = device_sm_count(), pairs = std::max(1, sms / 2);
    PairArgsExtra g = {};  // (a launch without EXTRA takes its first part)
    bool f32 = false, extra = false;
    g.part = sums.part, g.db = sums.db, g.chunks = sums.chunks, g.db_n = sums.n;
    for (int i = 0; i < count; ++i) {
        if (t[i].tiles > INT_MAX / 2)
            return cudaErrorInvalidValue;
        LinArgs &a = g.p[i];
        a = q[i].a;
        a.M = q[i].rows, a.N = q[i].cols, a.R = q[i].R;
        a.a_mn = q[i].x_mn, a.b_mn = q[i].y_mn;
        a.bn = t[i].bn, a.split = t[i].split;
        a.n_mt = int((int64_t(a.M) + 2 * LM - 1) / (2 * LM));
        a.flags = (a.bias ? kEpiBias : 0) | (a.pre ? kEpiPre : 0) |
                  (a.residual ? kEpiResidual : 0) | (a.out_f32 ? kEpiF32 : 0) |
                  (a.f16 ? kEpiF16 : 0) | (a.vec_out ? kEpiVecOut : 0) |
                  (a.vec_res ? kEpiVecRes : 0) | (a.vec_pre ? kEpiVecPre : 0) |
                  (a.mul ? kEpiMul : 0) |
                  uint32_t(a.act) * kEpiAct;
        a.chain = chain_steps(a.out_f32, a.f16);
        g.cut |= a.split == 1 && is_cut(q[i]);
        g.tiles[i] = int(t[i].tiles);
        g.bn = std::max(g.bn, a.bn);
        g.sub_bytes = std::max(g.sub_bytes, pair_sub_bytes(a.bn, a.b_mn));
        f32 |= a.out_f32 != 0;
        extra |= a.two || a.mul || a.stall;
        cudaError_t e = lin_map(&g.a[i], q[i].X, q[i].x_mn ? LK : LM, a.f16);
        if (e == cudaSuccess && a.two)
            e = lin_map(&g.a2[i], q[i].second(), q[i].x_mn ? LK : LM, a.f16);
        if (e == cudaSuccess)
            e = lin_map(&g.b[i], q[i].Y, q[i].y_mn ? LK : a.bn / 2, a.f16);
        // outputs by TMA where their rows are aligned (a split tile's are not)
        if (e == cudaSuccess && a.vec_out && a.split == 1)
            e = out_map(&g.out[i], a.out, a.M, a.N, a.ldo, a.out_f32, a.f16);
        if (e == cudaSuccess && a.pre && a.vec_pre && a.split == 1)
            e = out_map(&g.pre[i], a.pre, a.M, a.N, a.ldp, 0, a.f16);
        if (e != cudaSuccess)
            return e;
    }
    g.slot = pair_slot(f32);
    const int split = t[0].split;
    int clusters = g.tiles[0];
    if (split == 1) {
        clusters = int(std::min<int64_t>(int64_t(g.tiles[0]) + g.tiles[1], pairs));
        two_parts(g.tiles[0], t[0].tile_cycles, g.tiles[1], count == 2 ? t[1].tile_cycles : 0.0,
                  clusters, g.shared);
    }
    const size_t smem = pair_smem(g.sub_bytes, g.bn, split, f32);
    const bool wide = g.bn >= kPairWide;
    const void *kern = extra ? wide ? reinterpret_cast<const void *>(k_linear_pair<1, true>)
                                    : reinterpret_cast<const void *>(k_linear_pair<2, true>)
                       : wide ? reinterpret_cast<const void *>(k_linear_pair<1, false>)
                              : reinterpret_cast<const void *>(k_linear_pair<2, false>);
    const cudaError_t e = ensure_smem_limit(kern, kSlotLinearPair + 2 * extra + wide, kPairSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {extra ? static_cast<void *>(&g) : static_cast<PairArgs *>(&g)};
    return launch_clustered(kern, unsigned(clusters * 2 * split), unsigned(2 * split), kPairThreads,
                            smem, s, args);
}

// One launch of k_linear_pair (`pair`) or k_linear.
struct Launch {
    bool pair;
    int count;  // of products
    Product q[2];
    Tiling t[2];
};

// The launches that compute the products (the one with the longer reduction
// first): their number, at most two.
int plan_launches(Product *q, int count, int sms, Launch (&out)[2])
{
    if (count == 2 && q[1].steps() > q[0].steps())
        std::swap(q[0], q[1]);
    Tiling t[2] = {};
    bool f32 = false, cut = false;
    for (int i = 0; i < count; ++i) {
        f32 |= q[i].a.out_f32 != 0;
        cut |= is_cut(q[i]);
    }
    for (int i = 0; i < count; ++i)
        t[i] = choose_tiling(q[i], sms, f32, cut);
    const int64_t narrow = count == 1 ? mixed_columns(q[0], sms, t[0], t[1]) : 0;
    if (narrow) {
        const int64_t wide = q[0].cols - narrow;
        t[0].tiles = (int64_t(q[0].rows) + 255) / 256 * (wide / t[0].bn);
        out[0] = Launch{
            true, 2, {columns_of(q[0], 0, wide), columns_of(q[0], wide, narrow)}, {t[0], t[1]}};
        return 1;
    }
    if (count == 2 && t[0].pair && t[1].pair && t[0].split == 1 && t[1].split == 1) {
        out[0] = Launch{true, 2, {q[0], q[1]}, {t[0], t[1]}};
        return 1;
    }
    for (int i = 0; i < count; ++i)
        out[i] = Launch{t[i].pair, 1, {q[i], {}}, {t[i], {}}};
    return count;
}

// The products and the column sums, if any.
cudaError_t launch_products(Product *q, int count, ColSums sums, cudaStream_t s)
{
    Launch l[2];
    const int n = plan_launches(q, count, device_sm_count(), l);
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n && e == cudaSuccess; ++i) {
        if (l[i].pair) {
            e = launch_pairs(l[i].q, l[i].t, l[i].count, sums, s);
            sums.db = nullptr;
        } else {
            e = launch_small(l[i].q[0], s);
        }
    }
    if (e == cudaSuccess && sums.db)
        e = launch_pdl(k_col_sum, dim3((sums.n + 31) / 32), dim3(kGradThreads), 0, s, sums.part,
                       sums.chunks, sums.n, sums.db);
    return e;
}

// (sizes rounded up to whole tiles stay below 2^31)
inline bool sizes_ok(int T, int K, int N, int act)
{
    constexpr int kMost = INT_MAX - 511;
    return T >= 0 && T <= kMost && K >= 1 && K <= kMost && K % 8 == 0 && N >= 1 && N <= kMost &&
           act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH;
}

inline bool is16(int dtype)
{
    return dtype == MOE_DT_BF16 || dtype == MOE_DT_F16;
}

}  // namespace
}  // namespace moe

namespace moe {

uint32_t *linear_status_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_status) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

namespace {

int linear(const void *x, int64_t ldx, const void *W, const float *bias, const void *residual,
           int64_t ldr, int dtype, int act, int T, int K, int N, void *pre, void *y, int64_t ldy,
           int y_dtype, uint32_t *status, int stall, moe_stream_t stream)
{
    if (!is16(dtype) || (y_dtype != dtype && y_dtype != MOE_DT_F32))
        return MOE_ERR_DTYPE;
    if (!sizes_ok(T, K, N, act) || ldx < K || ldx % 8 != 0 || ldy < N || (residual && ldr < N))
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
    a.stall = stall;
    a.ldr = ldr, a.ldo = ldy, a.ldp = N;
    a.f16 = dtype == MOE_DT_F16, a.out_f32 = y_dtype == MOE_DT_F32, a.act = act;
    a.vec_out = vec16(y, ldy, ysize), a.vec_res = vec16(residual, ldr, ysize);
    a.vec_pre = vec16(pre, N, 2);
    Product q{{x, T, K, ldx}, {W, N, K, K}, false, false, T, N, K, a};
    return launch_products(&q, 1, ColSums{}, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

extern "C" int moe_linear(const void *x, int64_t ldx, const void *W, const float *bias,
                          const void *residual, int64_t ldr, int dtype, int act, int T, int K,
                          int N, void *pre, void *y, int64_t ldy, int y_dtype, uint32_t *status,
                          moe_stream_t stream)
{
    return moe::linear(x, ldx, W, bias, residual, ldr, dtype, act, T, K, N, pre, y, ldy, y_dtype,
                       status, 0, stream);
}

extern "C" int moe_selftest_linear_wait_limit(const void *x, const void *W, int T, int K, int N,
                                              void *y, uint32_t *status, int cta,
                                              moe_stream_t stream)
{
    if (cta < 0 || cta == INT_MAX)
        return MOE_ERR_SHAPE;
    return moe::linear(x, K, W, nullptr, nullptr, 0, MOE_DT_BF16, MOE_ACT_NONE, T, K, N, nullptr, y,
                       N, MOE_DT_BF16, status, cta + 1, stream);
}

namespace moe {
namespace {

// What moe_linear_grad's workspace holds: dP in 16 bits, the partial column
// sums, the maxima and the factor of a scaled dP, and dP's second piece.
struct GradLayout {
    size_t part, maxima, unscale, dp2, total;

    GradLayout(int T, int N, bool two)
    {
        const size_t ldp = (size_t(N) + 7) & ~size_t(7), dp = align256(size_t(T) * ldp * 2);
        part = dp;
        maxima = part + align256(size_t(kGradMaxChunks) * N * sizeof(float));
        unscale = maxima + align256(kMaxima * sizeof(uint32_t));
        dp2 = unscale + 256;
        total = dp2 + (two ? dp : 0);
    }
};

}  // namespace
}  // namespace moe

extern "C" size_t moe_linear_grad_workspace_bytes(int T, int N)
{
    return moe::sizes_ok(T, 8, N, MOE_ACT_NONE) ? moe::GradLayout(T, N, true).total : 0;
}

extern "C" size_t moe_linear_grad_workspace_bytes_for(int T, int N, int dy_dtype, int dw_dtype)
{
    const bool two = dy_dtype == MOE_DT_F32 && dw_dtype == MOE_DT_F32;
    return moe::sizes_ok(T, 8, N, MOE_ACT_NONE) ? moe::GradLayout(T, N, two).total : 0;
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
    if (!sizes_ok(T, K, N, act) || lddy < N || (dW && (ldx < K || ldx % 8 != 0)))
        return MOE_ERR_SHAPE;
    if (!ws || (dx && !W) ||
        (T > 0 && (!dy || (dW && !x) || (act != MOE_ACT_NONE && !pre))))
        return MOE_ERR_NULL;
    const bool two = dW && dy_dtype == MOE_DT_F32 && dw_dtype == MOE_DT_F32;
    const GradLayout layout(T, N, two);
    if (ws_bytes < layout.total)
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
    uint8_t *const base = static_cast<uint8_t *>(ws);
    uint16_t *dp = static_cast<uint16_t *>(ws);
    uint16_t *dp2 = two ? reinterpret_cast<uint16_t *>(base + layout.dp2) : nullptr;
    float *part = reinterpret_cast<float *>(base + layout.part);
    const bool products = dx || dW;
    const bool scaled = products && dtype == MOE_DT_F16 && dy_dtype == MOE_DT_F32;
    float *unscale = scaled ? reinterpret_cast<float *>(base + layout.unscale) : nullptr;
    // dy is the products' operand as it is
    const bool direct =
        act == MOE_ACT_NONE && dy_dtype == dtype && lddy % 8 == 0 && aligned(dy, 16);
    int chunks = 0;
    if (db || (products && !direct)) {
        GradArgs g = {};
        g.dy = dy, g.pre = pre;
        g.dp = products && !direct ? dp : nullptr;
        g.dp2 = dp2;
        g.part = db ? part : nullptr;
        if (scaled) {
            uint32_t *maxima = reinterpret_cast<uint32_t *>(base + layout.maxima);
            if (launch_pdl(k_dy_max, dim3(kMaxima), dim3(kMaxThreads), 0, s,
                           static_cast<const float *>(dy), lddy, T, N, vec16(dy, lddy, 4),
                           maxima) != cudaSuccess)
                return MOE_ERR_CUDA;
            g.maxima = maxima, g.unscale = unscale;
        }
        g.lddy = lddy, g.lddp = ldp;
        g.T = T, g.N = N;
        g.vec = vec16(dy, lddy, dysize) && (act == MOE_ACT_NONE || vec16(pre, N, 2));
        const int cb = (N + kGradCols - 1) / kGradCols;
        // about eight CTAs an SM, each with at least one round of rows
        chunks = std::max(1, std::min({(T + 31) / 32, 8 * device_sm_count() / cb, kGradMaxChunks}));
        g.rows = (T + chunks - 1) / chunks;
        chunks = (T + g.rows - 1) / g.rows;
        const GradKernel kern =
            act_grad_kernel(act, dy_dtype == MOE_DT_F32, dtype == MOE_DT_F16);
        if (launch_pdl(kern, dim3(cb, chunks), dim3(kGradThreads), 0, s, g) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    const Operand P = direct ? Operand{dy, T, N, lddy} : Operand{dp, T, N, ldp};
    LinArgs a = {};
    a.status = status;
    a.f16 = dtype == MOE_DT_F16;
    a.act = MOE_ACT_NONE;
    a.mul = unscale;
    a.ldo = K;
    Product q[2];
    int count = 0;
    if (dx) {
        a.out = dx;
        a.vec_out = vec16(dx, K, 2);
        q[count++] = Product{P, {W, N, K, K}, false, true, T, K, N, a};
    }
    if (dW) {
        a.out = dW;
        a.out_f32 = dw_dtype == MOE_DT_F32;
        a.vec_out = vec16(dW, K, dwsize);
        a.two = two;
        q[count++] = Product{P, {x, T, K, ldx}, true, true, N, K, T, a, dp2};
    }
    return launch_products(q, count, ColSums{part, db, chunks, N}, s) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

extern "C" int moe_selftest_linear_plan(int T, int K, int N, int what, int f32, int sms,
                                        int64_t *plan)
{
    using namespace moe;
    if (!plan)
        return MOE_ERR_NULL;
    const bool two = what & 8;
    what &= ~8;
    if (!sizes_ok(T, K, N, MOE_ACT_NONE) || T == 0 || what < 1 || what > 6 || what == 3 ||
        what == 5 || sms < 2 || (two && (!f32 || !(what & 4))))
        return MOE_ERR_SHAPE;
    Product q[2];
    int count = 0;
    LinArgs a = {};
    a.out_f32 = f32 != 0;
    if (what & 1)
        q[count++] = Product{{nullptr, T, K, K}, {nullptr, N, K, K}, false, false, T, N, K, a};
    a.two = two;
    if (what & 4)
        q[count++] = Product{{nullptr, T, N, N}, {nullptr, T, K, K}, true, true, N, K, T, a};
    a.two = a.out_f32 = 0;
    if (what & 2)
        q[count++] = Product{{nullptr, T, N, N}, {nullptr, N, K, K}, false, true, T, K, N, a};
    Launch l[2];
    plan[0] = plan_launches(q, count, sms, l);
    plan[1] = plan[2] = 0;
    for (int i = 0; i < plan[0]; ++i) {
        size_t smem = 0;
        int64_t ctas = 0;
        if (l[i].pair) {
            uint32_t sub = 0;
            int bn = 0;
            bool wide = false;
            for (int j = 0; j < l[i].count; ++j) {
                sub = std::max(sub, pair_sub_bytes(l[i].t[j].bn, l[i].q[j].y_mn));
                bn = std::max(bn, l[i].t[j].bn);
                wide |= l[i].q[j].a.out_f32 != 0;
                ctas += 2 * l[i].t[j].split * l[i].t[j].tiles;
            }
            smem = pair_smem(sub, bn, l[i].t[0].split, wide);
            if (l[i].t[0].split == 1)
                ctas = std::min<int64_t>(ctas, sms / 2 * 2);
        } else {
            small_args(l[i].q[0], sms, ctas, smem);
        }
        plan[1] = std::max(plan[1], int64_t(smem));
        plan[2] = std::max(plan[2], ctas);
    }
    return MOE_OK;
}
