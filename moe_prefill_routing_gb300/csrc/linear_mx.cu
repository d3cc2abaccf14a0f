// The dense product with both operands in MXFP4 (moe_linear_mxfp4) on the
// tensor cores' 4-bit path: tcgen05.mma.kind::mxf4, which multiplies E2M1 codes
// and applies the blocks' power-of-two scales itself.  Codes come by TMA with
// the 128-byte swizzle (a row of 128 bytes is 256 of K), scale tiles as they
// are; tcgen05.cp puts the scales into tensor memory beside the accumulators.
//
//   y[t][n] = act(sum_i x[t][i] W[n][i] + bias[n]) + residual[t][n]
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "mx_rows.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <climits>
#include <type_traits>

namespace moe {
namespace {

constexpr int MM = 128;                     // rows of a CTA's operand A
constexpr int MK = 256;                     // of K per stage: one 128-byte row
constexpr int kMxThreads = 192;             // producer, MMA, four accumulator warps
constexpr uint32_t kMxATile = MM * MK / 2;  // 16 KB
constexpr uint32_t kMxScales = 2 * kMxTileBytes;  // of 128 rows per stage
constexpr int kMxMaxStages = 8;
constexpr int kMxMaxSplit = 8;  // portable cluster size
// Rows that the kernel quantises itself: at most so many, of so many stages a CTA.
constexpr int kMxQuantRows = 16, kMxQuantStages = 8;
constexpr int kMxScaleCols = 16;  // of tensor memory: two tiles of A's and two of B's scales

// Stages of 256 of K, four MMAs each, that one accumulator sums; sums of more
// are cut into chains that are added outside the tensor core, which adds with
// truncation: a sum of one sign loses up to 2^-23 of itself in an MMA (measured over
// blocks of very different scales: 2.4e-8, so 6.2e-6 after 64 stages and 1.5e-6 after
// 16; blocks of like scales lose nothing, as their products have few bits).  16-bit
// outputs may drift by a quarter of half a unit (see linear.cu).
__host__ __device__ constexpr int mx_chain(bool f32, bool f16)
{
    return f32 ? 16 : f16 ? 256 : 2048;
}

struct MxArgs : EpiArgs {
    uint32_t *status;
    const uint8_t *a_scales, *b_scales;
    int M, N, K, k_tiles;
    int bn, stages, split, n_mt;
    int chain;
    int stall;  // self-test: CTA stall - 1's first stage waits for 16 bytes
    // QUANT kernels: x as it is, its type (MOE_DT_*) and whether 16-byte accesses
    // are aligned
    const void *rows;
    int64_t ld;
    int type, vec;
};

// Status bits of calls without a status word, see moe_take_status.
__device__ uint32_t g_status;

__device__ __noinline__ void report_timeout(uint32_t *status)
{
    atomicOr(status ? status : &g_status, MOE_STATUS_TIMEOUT);
}

struct MxCtrl {
    uint64_t full[kMxMaxStages];
    uint64_t empty[kMxMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t done;
    uint64_t rows_full[kMxQuantStages];
    uint32_t tmem_base;
    int abort_flag;
};

struct MxMaps {
    CUtensorMap a, b;
};

__host__ __device__ __forceinline__ uint32_t mx_stage_bytes(int bn, bool quant)
{
    return kMxATile + kMxScales + (quant ? 0 : uint32_t(bn) * (MK / 2) + kMxScales);
}

// What a CTA of a QUANT kernel holds of x: codes and scales of its stages.
__host__ __device__ __forceinline__ uint32_t mx_rows_bytes(int stages)
{
    return uint32_t(stages) * (kMxQuantRows * (MK / 2) + kMxScales);
}

// A block of 32 elements of row t, from column c on, to a stage's B tile and scales.
template <typename E>
__device__ __forceinline__ void mx_quant_block(const MxArgs &p, int t, int c, uint8_t *tile,
                                               uint8_t *scales, int block)
{
    Oct<E> in[4];
    const E *x = static_cast<const E *>(p.rows) + int64_t(t) * p.ld + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        in[i].load(x + 8 * i, p.K - c, p.vec);  // a whole block or nothing
    uint32_t m = in[0].max_bits();
#pragma unroll
    for (int i = 1; i < 4; ++i)
        m = max(m, in[i].max_bits());
    const uint32_t byte = mx_scale_byte(m);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[8];
        in[i].to(v);
        w[i] = mx_encode8(v, byte);
    }
    // a block is one 16-byte piece of the row's 128 bytes, in their swizzle
    reinterpret_cast<uint4 *>(tile)[t * 8 + (block ^ (t & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
    scales[(block >> 2) * kMxTileBytes + t * 16 + (block & 3)] = uint8_t(byte);
}

// Columns of tensor memory: the accumulator, or two of them and the sum where
// a sum is cut into chains; then the scales.
__host__ __device__ __forceinline__ uint32_t mx_columns(int bn, bool cut)
{
    const uint32_t need = uint32_t(bn) * (cut ? 3 : 1) + kMxScaleCols;
    uint32_t cols = 32;
    while (cols < need)
        cols *= 2;
    return cols;
}

// Tiles of 128 of W's rows (A) x bn of x's (16 ... 128), one CTA each, or `split`
// CTAs of a cluster that share the reduction and join their parts through
// distributed shared memory, each finishing 128 / split of the tile's features.
//
// What bounds it is latency: a launch's start, the first weights, the join.  One
// row x 2560 x 10240 takes 5.5 us (13.9 MB, 2.5 TB/s), 16 x 10240 x 2560 8.5.
//
// QUANT: the accumulator warps, which have nothing to do yet, quantise the CTA's
// part of a few rows while the weights are on their way (one launch, and no memory
// for the codes): the first of these with GELU 8.3 -> 7.2 us.
template <bool QUANT>
__global__ void __launch_bounds__(kMxThreads)
    k_linear_mx(const __grid_constant__ MxMaps maps, const MxArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ MxCtrl ctl;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int bn = p.bn, S = p.stages;
    const uint32_t b_bytes = QUANT ? 0u : uint32_t(bn) * (MK / 2);
    const uint32_t stage_bytes = mx_stage_bytes(bn, QUANT);
    const uint32_t z = cluster_ctarank();
    const int tile = int(blockIdx.x) / p.split;
    const int m0 = (tile % p.n_mt) * MM, n0 = (tile / p.n_mt) * bn;
    const int nk = (p.K + MK - 1) / MK;
    const int kb0 = int(int64_t(nk) * z / p.split), kb1 = int(int64_t(nk) * (z + 1) / p.split);
    const int chains = (kb1 - kb0 + p.chain - 1) / p.chain;
    // the same in every CTA of the launch: the most stages of one
    const int most = (nk + p.split - 1) / p.split;
    const bool cut = most > p.chain;
    const uint32_t tmem_cols = mx_columns(bn, cut);
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
        if (QUANT)
            for (int s = 0; s < kMxQuantStages; ++s)
                mbar_init(&ctl.rows_full[s], 4);  // the accumulator warps
        if (p.stall == int(blockIdx.x) + 1)
            mbar_expect_tx(&ctl.full[0], 16);
        ctl.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.a);
        if (!QUANT)
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
    // QUANT: behind the ring, the tiles of x and then their scales
    uint8_t *x_tiles = smem + S * stage_bytes;
    uint8_t *x_scales = x_tiles + (kb1 - kb0) * (kMxQuantRows * (MK / 2));
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        const bool one = elect_one();
        bool ok = true;
        const int64_t a_at = int64_t(m0 / 128) * p.k_tiles, b_at = int64_t(n0 / 128) * p.k_tiles;
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag));
            if (!ok)
                break;
            if (one) {
                uint64_t *fb = &ctl.full[stage];
                const uint32_t tiles = uint32_t(min(2, p.k_tiles - 2 * kb)) * kMxTileBytes;
                mbar_arrive_expect_tx(fb, kMxATile + b_bytes + (QUANT ? 1 : 2) * tiles);
                uint8_t *sa = smem + stage * stage_bytes, *sb = sa + kMxATile, *ss = sb + b_bytes;
                tma_load_2d(sa, &maps.a, fb, kb * (MK / 2), m0);
                bulk_load(ss, p.a_scales + (a_at + 2 * kb) * kMxTileBytes, tiles, fb);
                if (!QUANT) {
                    tma_load_2d(sb, &maps.b, fb, kb * (MK / 2), n0);
                    bulk_load(ss + kMxScales, p.b_scales + (b_at + 2 * kb) * kMxTileBytes, tiles,
                              fb);
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
        // the whole warp walks the loop and one lane issues
        int stage = 0;
        uint32_t phase = 0;
        const uint32_t sa = smem_u32(smem), sb = sa + kMxATile, ss = sb + b_bytes;
        const uint64_t da0 = smem_desc_sw128(sa, 16, 1024);
        const uint64_t db0 = smem_desc_sw128(QUANT ? smem_u32(x_tiles) : sb, 16, 1024);
        const uint64_t ds0 = smem_desc_rows16(ss);
        const uint64_t dx0 = smem_desc_rows16(QUANT ? smem_u32(x_scales) : ss + kMxScales);
        const uint32_t scales = tmem_base + tmem_cols - kMxScaleCols;
        const bool one = elect_one();
        uint32_t d = tmem_base, aphase = 0;
        int left = p.chain, buf = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (cut && left == p.chain) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&ctl.acc_empty[buf], aphase ^ 1u, abort_flag));
                if (!ok)
                    break;
                tc_fence_after_sync();
                d = tmem_base + uint32_t(buf * bn);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[stage], phase, abort_flag));
            if (QUANT && ok)
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.rows_full[kb - kb0], 0, abort_flag));
            if (!ok)
                break;
            tc_fence_after_sync();
            if (one) {
                const uint32_t off = uint32_t(stage) * (stage_bytes >> 4);
                const uint32_t x_at = uint32_t(kb - kb0);  // QUANT: its tile of x
                const uint32_t b_off = QUANT ? x_at * (kMxQuantRows * (MK / 2) >> 4) : off;
                const uint32_t x_off = QUANT ? x_at * (kMxScales >> 4) : off;
                const int rest = p.K - kb * MK;
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i)
                    if (rest > int(i) * 128) {
                        tc_copy_32x128b(scales + 4 * i, ds0 + (off + i * (kMxTileBytes >> 4)));
                        tc_copy_32x128b(scales + 8 + 4 * i,
                                        dx0 + (x_off + i * (kMxTileBytes >> 4)));
                    }
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk)
                    if (rest > int(kk) * 64)
                        tc_mma_mxf4(d, da0 + (off + kk * 2), db0 + (b_off + kk * 2),
                                    idesc_mxf4(MM, uint32_t(bn), kk & 1), scales + 4 * (kk >> 1),
                                    scales + 8 + 4 * (kk >> 1), left != p.chain || kk != 0);
                tc_commit(&ctl.empty[stage]);
            }
            if (--left == 0 || kb + 1 == kb1) {
                left = p.chain;
                if (cut) {
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
            tc_commit(&ctl.done);  // arrives once everything issued here has completed
    }
    // CTA z of the cluster finishes 128 / Z of the tile's m: every CTA sends it
    // its sums of those, and it adds them in rank order.  They go beside the
    // ring, which may still be in use there, or (128 columns) into the ring
    // once every CTA is done with it.
    const bool beside = bn < MM;
    float *acc = reinterpret_cast<float *>(
        smem + (beside ? S * stage_bytes + (QUANT ? mx_rows_bytes(most) : 0u) : 0u));
    const int slice = MM / p.split, pitch = bn + 4;  // acc: [Z][128 / Z][pitch]
    const int cols = min(bn, p.N - n0);
    // what a thread finishes: four neighbouring m, always the same, of every `by`-th n
    const int quads = slice / 4, by = kMxThreads / quads;
    const int mq = int(threadIdx.x) % quads * 4, at = m0 + int(z) * slice + mq;
    const int left = min(4, p.M - at);
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bias[i] = p.bias && i < left ? p.bias[at + i] : 0.0f;
    bool done = false;
    if (QUANT && warp >= 2) {
        // a thread has a block of 32: eight to a row and stage
        for (int kb = kb0; kb < kb1; ++kb) {
            uint8_t *tile = x_tiles + (kb - kb0) * (kMxQuantRows * (MK / 2));
            uint8_t *tile_scales = x_scales + (kb - kb0) * kMxScales;
            for (int i = int(threadIdx.x) - 64; i < p.N * 8; i += 128) {
                const int t = i >> 3, block = i & 7, c = kb * MK + block * 32;
                if (p.type == MOE_DT_F32)
                    mx_quant_block<float>(p, t, c, tile, tile_scales, block);
                else if (p.type == MOE_DT_F16)
                    mx_quant_block<__half>(p, t, c, tile, tile_scales, block);
                else
                    mx_quant_block<__nv_bfloat16>(p, t, c, tile, tile_scales, block);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ctl.rows_full[kb - kb0]);
        }
    }
    if (warp >= 2) {
        const uint32_t lanes = tmem_base + (uint32_t(warp & 3) << 21);
        for (int i = 0; cut && i < chains; ++i) {
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
        const uint32_t t0 = tmem_base + (uint32_t(warp & 3) << 21) + uint32_t(cut ? 2 * bn : 0);
        const uint32_t to = dsmem_addr(acc + (int(z) * slice + m % slice) * pitch, m / slice);
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
            uint32_t r[16] = {};
            if (done) {
                tmem_ld_32x32b_x16(t0 + uint32_t(c), r);
                tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                dsmem_st4(to + uint32_t(c + j) * 4, r[j], r[j + 1], r[j + 2], r[j + 3]);
        }
        tc_fence_before_sync();
    }
    __syncwarp();
    cluster_sync();
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

// ---- many rows: pairs of CTAs ---------------------------------------------------
//
// Tiles of 256 of x's rows (A) x bn of W's (B), one tcgen05.mma of a CTA pair per
// 64 of K: each CTA loads its 128 rows of A and half the rows of B, the scales of
// its own rows of A and those of all rows of B.  Pairs walk the tiles
// (persistent); two accumulators let the epilogue warps work on one tile while
// the MMAs fill the other.  Sums that are cut (fp32 outputs) take them chain after
// chain, and the epilogue warps add the chains up in registers.
//
// A stage's round trip, from its release to its next data's arrival, takes 1.14 us
// however little is loaded, so it is spread over many stages (192 columns: six; 4096
// x 11264 x 11264 217, 175, 151 and 142 us with three to six).  What bounds a long
// reduction are that and the MMAs of 64 of K (137 us with 256 columns and five stages,
// 7.6 PFLOP/s; with 192 140, 126 without the epilogue, 116 without loads either), a
// short one the loads and stores: 4096 x 2816 x 11264 46.4 us (5.6 PFLOP/s); with 192
// columns 51, 45 without MMAs, 39 without stores.
constexpr int kMxPairStages = 8;  // at most
constexpr int kMxEpiCols = 64;    // of an epilogue warp (32 rows), all in registers at once
constexpr int kMxEpiWarps = 12;   // at most: 192 columns (256 go round)
constexpr int kMxPairThreads = 64 + 32 * kMxEpiWarps;
constexpr uint32_t kMxSlot = 2048;  // of an epilogue warp: 32 rows of 64 bytes

struct MxPairCtrl {
    uint64_t full[kMxPairStages];
    uint64_t empty[kMxPairStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t shared_read[2];  // the columns that the other accumulator shares
    uint32_t tmem_base;
    int abort_flag;
};

struct MxPairArgs {
    CUtensorMap a, b, a_scales, b_scales, out;
    MxArgs p;  // M: x's rows, N: W's
    int tiles, stages;
    uint32_t stage_bytes;
};

// Tiles of 128 rows' scales that bn of B's rows lie in (tiles of 192 start in the
// middle of one every other time).  Widths are multiples of 64: with 224, whose
// scales start at an odd column of tensor memory every other time, the MMA ended in
// a misaligned-address error.
__host__ __device__ constexpr int mx_b_tiles(int bn)
{
    return bn > 128 ? 2 : 1;
}

// Columns between the two accumulators.  Two of 256 and the scales do not fit the
// 512 columns: they share 48, the first one's last, which the epilogue takes out
// first.
constexpr int kMxAccStep = 208;

__host__ __device__ constexpr int mx_acc_step(int bn)
{
    return bn < kMxAccStep ? bn : kMxAccStep;
}

// What one CTA loads per stage.
__host__ __device__ __forceinline__ uint32_t mx_pair_stage(int bn)
{
    return kMxATile + uint32_t(bn / 2) * (MK / 2) + (1 + mx_b_tiles(bn)) * kMxScales;
}

// A slot's 16-byte piece c of row r, as the 64-byte swizzle of a TMA copy has it.
__device__ __forceinline__ uint4 *mx_slot_at(uint8_t *slot, int r, int c)
{
    return reinterpret_cast<uint4 *>(slot) + r * 4 + (c ^ ((r >> 1) & 3));
}

// A slot's columns to memory element by element, where 16-byte pieces are not
// aligned.
template <typename E>
__device__ __noinline__ void mx_store_by_element(uint8_t *slot, E *p, int64_t ld, int rows,
                                                 int cols)
{
    constexpr int kPer = 16 / int(sizeof(E));
    const int lane = threadIdx.x & 31;
    if (lane < cols)
#pragma unroll 16
        for (int r = 0; r < rows; ++r)
            p[int64_t(r) * ld + lane] =
                reinterpret_cast<E *>(mx_slot_at(slot, r, lane / kPer))[lane % kPer];
}

// The epilogue's blocks: 32 rows (lane = row) x 64 bytes of the output.
template <typename E>
struct MxBlock {
    static constexpr int kColumns = 64 / int(sizeof(E));
    static constexpr bool kF32 = sizeof(E) == 4;
    static constexpr int kF16 = std::is_same<E, __half>::value;

    // The residual's block on its way, and into the slot: 16-byte pieces of rows
    // lane / 4 + 8 i where they are aligned and exist whole (`vec`); else, just as
    // many words, 16-bit elements of column `lane` of rows 2 i and 2 i + 1, or fp32
    // ones of column lane % 16 of row 2 i + lane / 16.
    static __device__ __forceinline__ void ask(uint4 (&q)[4], const E *p, int64_t ld, int rows,
                                               int cols, bool vec)
    {
        const int lane = threadIdx.x & 31;
        if (vec && cols >= kColumns) {
            const E *at = p + (lane >> 2) * ld + (lane & 3) * (16 / int(sizeof(E)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((lane >> 2) + 8 * i < rows)
                    q[i] = *reinterpret_cast<const uint4 *>(at + 8 * i * ld);
            return;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (kF32) {
                const int r = 2 * i + (lane >> 4), c = lane & 15;
                w[i] = r < rows && c < cols
                           ? __float_as_uint(reinterpret_cast<const float *>(p)[r * ld + c])
                           : 0u;
            } else {
                const uint16_t *at = reinterpret_cast<const uint16_t *>(p) + 2 * i * ld + lane;
                const uint32_t a = lane < cols && 2 * i < rows ? at[0] : 0u;
                const uint32_t b = lane < cols && 2 * i + 1 < rows ? at[ld] : 0u;
                w[i] = a | b << 16;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }

    static __device__ __forceinline__ void place(uint8_t *slot, const uint4 (&q)[4], int cols,
                                                 bool vec)
    {
        const int lane = threadIdx.x & 31;
        if (vec && cols >= kColumns) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *mx_slot_at(slot, (lane >> 2) + 8 * i, lane & 3) = q[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint4 v = q[i / 4];
            const uint32_t w = i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
            if constexpr (kF32) {
                reinterpret_cast<uint32_t *>(
                    mx_slot_at(slot, 2 * i + (lane >> 4), (lane & 15) / 4))[lane & 3] = w;
            } else {
                reinterpret_cast<uint16_t *>(mx_slot_at(slot, 2 * i, lane / 8))[lane & 7] =
                    uint16_t(w);
                reinterpret_cast<uint16_t *>(mx_slot_at(slot, 2 * i + 1, lane / 8))[lane & 7] =
                    uint16_t(w >> 16);
            }
        }
    }

    static __device__ __forceinline__ void add(const uint8_t *slot, float *v)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 q = *mx_slot_at(const_cast<uint8_t *>(slot), lane, c);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (kF32) {
                    v[4 * c + j] += __uint_as_float(w[j]);
                } else {
                    const float2 f = unpack16(w[j], kF16);
                    v[8 * c + 2 * j] += f.x;
                    v[8 * c + 2 * j + 1] += f.y;
                }
            }
        }
    }

    static __device__ __forceinline__ void put(uint8_t *slot, const float *v)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = kF32 ? __float_as_uint(v[4 * c + j])
                            : pack16(v[8 * c + 2 * j], v[8 * c + 2 * j + 1], kF16);
            *mx_slot_at(slot, lane, c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// An epilogue warp's 64 columns of an accumulator, or (ADD) their sum with what it has,
// eight at a time (with sixteen more registers spill: 4096 x 11264 x 2816 fp32 with a
// residual 60.8 us instead of 57.4; uncut it would take 55.1).
template <bool ADD>
__device__ __forceinline__ void mx_take_columns(uint32_t from, uint32_t (&r0)[32],
                                                uint32_t (&r1)[32])
{
    if (!ADD) {
        tmem_ld_32x32b_x32(from, r0);
        tmem_ld_32x32b_x32(from + 32, r1);
        tmem_ld_wait();
        return;
    }
#pragma unroll
    for (int c = 0; c < kMxEpiCols; c += 8) {
        uint32_t r[8];
        tmem_ld_32x32b_x8(from + uint32_t(c), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t &sum = c < 32 ? r0[(c + j) & 31] : r1[(c + j) & 31];
            sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(r[j]));
        }
    }
}

enum MxTiles { kNarrow, kCut, kWide };  // kCut: sums are cut into chains; kWide: 256 columns

template <int ACT, typename E, MxTiles TILES>
__global__ void __launch_bounds__(kMxPairThreads, 1)
    k_linear_mx_pair(const __grid_constant__ MxPairArgs g)
{
    constexpr bool WIDE = TILES == kWide, CUT = TILES == kCut;
    extern __shared__ uint8_t smem_raw[];
    // the same offset in both CTAs: dynamic shared memory starts at the same address
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    __shared__ MxPairCtrl ctl;
    const MxArgs &p = g.p;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int bn = WIDE ? 256 : p.bn, half = bn / 2, S = g.stages;
    const uint32_t stage_bytes = g.stage_bytes;
    uint8_t *stg = smem + S * stage_bytes;
    volatile int *abort_flag = &ctl.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 2 * 4 * (bn / kMxEpiCols));  // both CTAs' warps
            mbar_init(&ctl.shared_read[b], 2 * 4);
        }
        if (p.stall == int(blockIdx.x) + 1)
            mbar_expect_tx(&ctl.full[0], 16);
        ctl.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&g.a);
        prefetch_tmap(&g.b);
        prefetch_tmap(&g.a_scales);
        prefetch_tmap(&g.b_scales);
    }
    __syncwarp();
    cluster_arrive();
    if (warp == 1)
        tmem_alloc_pair(&ctl.tmem_base, 512);
    tc_fence_before_sync();
    __syncthreads();
    cluster_wait();  // the other CTA's barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;
    pdl_wait();
    pdl_launch_dependents();

    const int pairs = int(gridDim.x) / 2, pair = int(blockIdx.x) / 2;
    const int nk = (p.K + MK - 1) / MK;
    // tile t: blocks of 16 m tiles, m fastest, so that the pairs running at one
    // time share few rows of both operands
    const int block = 16 * ((p.N + bn - 1) / bn);
    auto place = [&](int t, int &m0, int &n0) {
        const int b = t / block, tall = min(16, p.n_mt - 16 * b), u = t - b * block;
        n0 = u / tall * bn;
        m0 = (16 * b + u % tall) * (2 * MM) + int(rank) * MM;
    };
    int m0, n0;

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        const bool one = elect_one();
        bool ok = true;
        for (int t = pair; ok && t < g.tiles; t += pairs) {
            place(t, m0, n0);
            for (int kb = 0; kb < nk; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag));
                if (!ok)
                    break;
                if (one) {
                    if (rank == 0)  // both CTAs' bytes complete on the even CTA's barrier
                        mbar_arrive_expect_tx(&ctl.full[stage], 2 * stage_bytes);
                    const uint32_t fb = dsmem_addr(&ctl.full[stage], 0);
                    uint8_t *sa = smem + stage * stage_bytes;
                    uint8_t *sb = sa + kMxATile, *ss = sb + half * (MK / 2);
                    tma_load_2d_pair(sa, &g.a, fb, kb * (MK / 2), m0);
                    tma_load_2d_pair(sb, &g.b, fb, kb * (MK / 2), n0 + int(rank) * half);
                    tma_load_3d_pair(ss, &g.a_scales, fb, 0, 2 * kb, m0 / 128);
                    tma_load_3d_pair(ss + kMxScales, &g.b_scales, fb, 0, 2 * kb, n0 / 128);
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
        // One lane walks and issues, without a branch: what lies past the end of K in
        // the last stage is zeros, codes and scales.  Its turn takes 0.18 us, a stage's
        // MMAs of 192 columns 0.20 (9.5 PFLOP/s), so every step of it counts: a test
        // for each MMA made 4096 x 11264 x 11264 162 us instead of 133 without its
        // epilogue, a walk of the whole warp 142.8 instead of 140.4 with it.
        const uint32_t sa = smem_u32(smem), sb = sa + kMxATile, ss = sb + half * (MK / 2);
        const uint64_t da0 = smem_desc_sw128(sa, 16, 1024), db0 = smem_desc_sw128(sb, 16, 1024);
        const uint64_t ds0 = smem_desc_rows16(ss);
        const uint32_t idesc = idesc_mxf4(2 * MM, uint32_t(bn), 0);
        const auto walk = [&](auto count) {
            constexpr uint32_t kB = decltype(count)::value;  // scale tiles of B
            // of tensor memory, twice: A's two scale tiles, then B's two of kB
            constexpr uint32_t kSet = 8 + 8 * kB, kTile = kMxTileBytes >> 4;
            const uint32_t scales = tmem_base + 512 - 2 * kSet;
            int stage = 0, buf = 0;
            uint32_t phase = 0, aphase = 0, set = 0;
            for (int t = pair; t < g.tiles; t += pairs) {
                place(t, m0, n0);
                int kb = 0;
                do {  // a chain
                    const int last = CUT ? min(kb + p.chain, nk) : nk;
                    uint32_t some = 0;
                    if (!mbar_wait(&ctl.acc_empty[buf], aphase ^ 1u, abort_flag))
                        return;
                    // the other accumulator's shared columns: it was filled a tile ago
                    if (WIDE && t != pair &&
                        !mbar_wait(&ctl.shared_read[buf ^ 1], buf ? aphase : aphase ^ 1u,
                                   abort_flag))
                        return;
                    tc_fence_after_sync();
                    const uint32_t d = tmem_base + uint32_t(buf * mx_acc_step(bn));
                    const uint32_t b_scales = 8 + uint32_t(n0 % 128) / 32;
                    for (; kb < last; ++kb) {
                        if (!mbar_wait(&ctl.full[stage], phase, abort_flag))
                            return;
                        tc_fence_after_sync();
                        const uint32_t off = uint32_t(stage) * (stage_bytes >> 4);
                        uint64_t *const released = &ctl.empty[stage];
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        const uint32_t at = scales + set;
                        set ^= kSet;
                        tc_copy_32x128b_pair(at, smem_desc_at(ds0, off));
                        tc_copy_32x128b_pair(at + 4, smem_desc_at(ds0, off + kTile));
#pragma unroll
                        for (uint32_t i = 0; i < kB; ++i) {
                            tc_copy_32x128b_pair(at + 8 + 4 * i,
                                                 smem_desc_at(ds0, off + (2 + 2 * i) * kTile));
                            tc_copy_32x128b_pair(at + 8 + 4 * (kB + i),
                                                 smem_desc_at(ds0, off + (3 + 2 * i) * kTile));
                        }
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk)
                            tc_mma_mxf4_pair(d, smem_desc_at(da0, off + 2 * kk),
                                             smem_desc_at(db0, off + 2 * kk),
                                             idesc | (kk & 1) << 5 | (kk & 1) << 30,
                                             at + 4 * (kk >> 1), at + b_scales + 4 * kB * (kk >> 1),
                                             kk != 0 ? 1u : some);
                        tc_commit_pair(released, 3);
                        some = 1;
                    }
                    tc_commit_pair(&ctl.acc_full[buf], 3);
                    if (++buf == 2) {
                        buf = 0;
                        aphase ^= 1u;
                    }
                } while (CUT && kb < nk);
            }
        };
        if (elect_one()) {
            if (mx_b_tiles(bn) == 2)
                walk(std::integral_constant<uint32_t, 2>());
            else
                walk(std::integral_constant<uint32_t, 1>());
        }
        __syncwarp();
        // (the epilogue warps of both CTAs wait for every accumulator, so the
        // MMAs are done when the cluster meets below)
    } else if (warp >= 2 && (warp - 2) >> 2 < bn / kMxEpiCols) {  // (12 warps at most)
        // A warp takes its 64 columns into registers at once and gives the
        // accumulator back; then block after block: bias, activation, residual, one
        // slot of shared memory, one TMA store.  (With 16 columns at a time and the
        // accumulator kept till the end, 4096 x 256 x 11264 took 33 us.)
        using Block = MxBlock<E>;
        constexpr int C = Block::kColumns, kBlocks = kMxEpiCols / C;
        const int q = warp & 3, part = (warp - 2) >> 2;  // lane quadrant; which 64 columns
        uint8_t *slot = stg + uint32_t(warp - 2) * kMxSlot;
        float *bias = reinterpret_cast<float *>(stg + kMxEpiWarps * kMxSlot) +
                      (warp - 2) * kMxEpiCols;
        const uint32_t lanes = tmem_base + (uint32_t(q * 32) << 16);
        const bool any_res = p.residual, vec_res = p.vec_res;
        // WIDE: four parts for the three warps of a quadrant, whose roles go round: the
        // one that has had the longest rest takes the shared columns (0), the next but
        // one (2) two parts.
        int buf = 0, role = (part + 2) % 3;
        uint32_t aphase = 0;
        bool more = false;  // the second of two parts
        for (int t = pair; t < g.tiles;) {
            place(t, m0, n0);
            const int c0 = (WIDE ? (role + more + (buf ? 0 : 3)) & 3 : part) * kMxEpiCols;
            const int64_t row = int64_t(m0) + q * 32;
            const int rows = int(min(int64_t(32), p.M - row));
            const int col = n0 + c0, width = min(kMxEpiCols, p.N - col);
            uint32_t r0[32], r1[32];
            if constexpr (CUT) {  // all chains but the last
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    r0[i] = r1[i] = 0u;
                int chains = (nk - 1) / p.chain;
                for (; chains > 0; --chains) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&ctl.acc_full[buf], aphase, abort_flag)))
                        break;
                    tc_fence_after_sync();
                    mx_take_columns<true>(lanes + uint32_t(buf * mx_acc_step(bn) + c0), r0, r1);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster_relaxed(dsmem_addr(&ctl.acc_empty[buf], 0));
                    if (++buf == 2) {
                        buf = 0;
                        aphase ^= 1u;
                    }
                }
                if (chains > 0)
                    break;
            }
            const E *res = static_cast<const E *>(p.residual) + (any_res ? row * p.ldr + col : 0);
            E *out = static_cast<E *>(p.out) + row * p.ldo + col;
            uint4 ahead[4] = {};
            if (any_res)
                Block::ask(ahead, res, p.ldr, rows, width, vec_res);
            if (p.bias) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kMxEpiCols; i += 32)
                    bias[i + lane] = i + int(lane) < width ? p.bias[col + i + int(lane)] : 0.0f;
                __syncwarp();
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&ctl.acc_full[buf], aphase, abort_flag)))
                break;
            tc_fence_after_sync();
            mx_take_columns<CUT>(lanes + uint32_t(buf * mx_acc_step(bn) + c0), r0, r1);
            tc_fence_before_sync();  // these columns have been read
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_cluster_relaxed(dsmem_addr(&ctl.acc_empty[buf], 0));
                if (WIDE && role == 0)
                    mbar_arrive_cluster_relaxed(dsmem_addr(&ctl.shared_read[buf], 0));
            }
            more = WIDE && role == 2 && !more;
            if (!more) {
                t += pairs;
                role = role ? role - 1 : 2;
                if (++buf == 2) {
                    buf = 0;
                    aphase ^= 1u;
                }
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int cols = min(C, width - b * C);
                if (rows <= 0 || cols <= 0)
                    break;
                float v[C];
#pragma unroll
                for (int j = 0; j < C; ++j)
                    v[j] = __uint_as_float(b * C + j < 32 ? r0[(b * C + j) & 31]
                                                          : r1[(b * C + j) & 31]);
                if (p.bias) {
#pragma unroll
                    for (int j = 0; j < C; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(bias + b * C + j);
                        v[j] += f.x, v[j + 1] += f.y, v[j + 2] += f.z, v[j + 3] += f.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < C; j += 16) {
                    float w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = v[j + i];
                    act_all<ACT>(w);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[j + i] = w[i];
                }
                if (lane == 0)
                    bulk_wait_read<0>();  // the last store is done with the slot
                __syncwarp();
                if (any_res) {
                    Block::place(slot, ahead, cols, vec_res);
                    if (b + 1 < kBlocks)
                        Block::ask(ahead, res + (b + 1) * C, p.ldr, rows, width - (b + 1) * C,
                                   vec_res);
                    __syncwarp();
                    Block::add(slot, v);
                }
                Block::put(slot, v);
                if (p.vec_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&g.out, slot, col + b * C, int(row));
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    mx_store_by_element(slot, out + b * C, p.ldo, rows, cols);
                }
            }
        }
        if (lane == 0)
            bulk_wait<0>();  // every store written before the CTA (and its memory) goes
    }
    __syncthreads();
    if (threadIdx.x == 0 && ctl.abort_flag)
        report_timeout(p.status);
    __syncwarp();
    cluster_sync();  // the CTAs are done with each other's shared memory and barriers
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

using MxPairKernel = void (*)(MxPairArgs);

template <int ACT, MxTiles TILES>
MxPairKernel mx_pair_kernel(bool f32, bool f16)
{
    if constexpr (TILES == kCut)
        return k_linear_mx_pair<ACT, float, kCut>;
    else
        return f32   ? k_linear_mx_pair<ACT, float, TILES>
               : f16 ? k_linear_mx_pair<ACT, __half, TILES>
                     : k_linear_mx_pair<ACT, __nv_bfloat16, TILES>;
}

template <MxTiles TILES>
MxPairKernel mx_pair_kernel(int act, bool f32, bool f16)
{
    switch (act) {
    case MOE_ACT_RELU:
        return mx_pair_kernel<MOE_ACT_RELU, TILES>(f32, f16);
    case MOE_ACT_SILU:
        return mx_pair_kernel<MOE_ACT_SILU, TILES>(f32, f16);
    case MOE_ACT_GELU:
        return mx_pair_kernel<MOE_ACT_GELU, TILES>(f32, f16);
    case MOE_ACT_GELU_TANH:
        return mx_pair_kernel<MOE_ACT_GELU_TANH, TILES>(f32, f16);
    default:
        return mx_pair_kernel<MOE_ACT_NONE, TILES>(f32, f16);
    }
}

// ---- host ---------------------------------------------------------------------

// Codes [rows, K / 2]: boxes of 128 bytes x box_rows rows with the 128-byte swizzle.
cudaError_t mx_map(CUtensorMap *m, const uint8_t *codes, int64_t rows, int K, int box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(K) / 2, cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(K) / 2};
    const cuuint32_t box[2] = {MK / 2, cuuint32_t(box_rows)}, estr[2] = {1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes),
                              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Scale tiles [row_tiles, k_tiles, 512]: boxes of the two tiles of a stage of
// `box_rows` neighbouring tiles of 128 rows.
cudaError_t mx_scale_map(CUtensorMap *m, const uint8_t *scales, int64_t rows, int K, int box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t kt = cuuint64_t(mx_k_tiles(K));
    const cuuint64_t dims[3] = {kMxTileBytes / 4, kt, cuuint64_t((rows + 127) / 128)};
    const cuuint64_t strides[2] = {kMxTileBytes, kt * kMxTileBytes};
    const cuuint32_t box[3] = {kMxTileBytes / 4, 2, cuuint32_t(box_rows)}, estr[3] = {1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(scales),
                              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Outputs [M, N], written in blocks of 32 rows x 64 bytes from a slot.
cudaError_t mx_out_map(CUtensorMap *m, const MxArgs &a)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const int size = a.out_f32 ? 4 : 2;
    const cuuint64_t dims[2] = {cuuint64_t(a.N), cuuint64_t(a.M)};
    const cuuint64_t strides[1] = {cuuint64_t(a.ldo) * size};
    const cuuint32_t box[2] = {cuuint32_t(64 / size), 32}, estr[2] = {1, 1};
    const CUresult r =
        encode(m,
               a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
               : a.f16   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               2, a.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct MxProduct {
    const uint8_t *x, *x_scales, *W, *W_scales;
    int T, K, N;
    EpiArgs epi;
    uint32_t *status;
    // in place of x: rows to quantise (k_linear_mx alone)
    const void *rows;
    int64_t ld;
    int type;
    int stall;  // MxArgs::stall
};

constexpr size_t kMxLoneSmem = 226 * 1024;  // of a CTA that takes all of an SM's tensor memory

// Columns, tiles and split of k_linear_mx.
struct MxSmall {
    int bn, n_mt, split;
    int64_t tiles;

    MxSmall(int T, int K, int N, int sms)
    {
        const int nk = (K + MK - 1) / MK;
        bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
        n_mt = int((int64_t(N) + MM - 1) / MM);
        tiles = int64_t(n_mt) * ((int64_t(T) + bn - 1) / bn);
        // split the reduction while the CTAs still fit at once and each has two stages
        split = 1;
        while (split < kMxMaxSplit && tiles * split * 2 <= 2 * sms && nk / (split * 2) >= 2)
            split *= 2;
    }

    // Whether the kernel quantises x itself: its CTAs hold their part of x beside
    // the ring, and a few rows take them no longer than the weights' first stages.
    bool quantises(int T, int K) const
    {
        const int nk = (K + MK - 1) / MK;
        return T <= kMxQuantRows && (nk + split - 1) / split <= kMxQuantStages;
    }
};

cudaError_t launch_mx_small(const MxProduct &q, cudaStream_t s)
{
    const int nk = (q.K + MK - 1) / MK;
    const MxSmall l(q.T, q.K, q.N, device_sm_count());
    const bool quant = q.rows != nullptr;
    MxArgs a = {};
    static_cast<EpiArgs &>(a) = q.epi;
    a.status = q.status;
    a.a_scales = q.W_scales, a.b_scales = q.x_scales;
    a.rows = q.rows, a.ld = q.ld, a.type = q.type;
    a.vec = quant && rows_vec(q.rows, q.ld, dtype_size(q.type));
    a.M = q.N, a.N = q.T, a.K = q.K, a.k_tiles = mx_k_tiles(q.K);
    a.chain = mx_chain(a.out_f32, a.f16), a.stall = q.stall;
    a.bn = l.bn, a.n_mt = l.n_mt, a.split = l.split;
    if (l.tiles * a.split > INT_MAX)
        return cudaErrorInvalidValue;
    const uint32_t stage = mx_stage_bytes(a.bn, quant);
    const uint32_t parts = (a.bn < MM ? uint32_t(MM) * (a.bn + 4) * 4 : 0) +
                           (quant ? mx_rows_bytes((nk + a.split - 1) / a.split) : 0);
    a.stages = std::min<int>(kMxMaxStages, (110 * 1024 - parts) / stage);
    size_t smem = 1024 + std::max<size_t>(size_t(a.stages) * stage + parts,
                                          a.bn < MM ? 0 : size_t(MM) * (a.bn + 4) * 4);
    // Two CTAs share an SM's 512 columns of tensor memory.  One that takes them
    // all must be alone there, be the other of its own cluster or of another
    // kernel's: two clusters that each wait for tensor memory the other holds
    // would wait for ever.
    if (mx_columns(a.bn, (nk + a.split - 1) / a.split > a.chain) > 256)
        smem = kMxLoneSmem;
    MxMaps maps = {};
    cudaError_t e = mx_map(&maps.a, q.W, q.N, q.K, MM);
    if (e == cudaSuccess && !quant)
        e = mx_map(&maps.b, q.x, q.T, q.K, a.bn);
    const void *kern = quant ? reinterpret_cast<const void *>(k_linear_mx<true>)
                             : reinterpret_cast<const void *>(k_linear_mx<false>);
    if (e == cudaSuccess)
        e = ensure_smem_limit(kern, kSlotLinearMx + quant, kMxLoneSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {&maps, &a};
    return launch_clustered(kern, unsigned(l.tiles * a.split), unsigned(a.split), kMxThreads, smem,
                            s, args);
}

// Columns of a tile of k_linear_mx_pair: those with the least estimated time, in
// cycles, of a round of tiles and of the last tile's epilogue, by times at 64 ... 256.
// (4096 x 10240 x 2560 in 9, 5, 3 and 3 rounds 76, 46, 34 and 41 us, x 512 x 2560 12.5,
// 9.5, 8.4 and 9.1; with 192 and 256 columns 4096 x 2816 x 11264 50.9 and 46.4, x 11264
// x 11264 141 and 137, 8192 x 4096 x 4096 48.4 and 44.0.)
int mx_pair_columns(const MxProduct &q, int pairs)
{
    constexpr struct {
        int bn;
        double round, stage;
    } kTimes[] = {{256, 2260, 540}, {192, 1800, 435}, {128, 1320, 390}, {64, 1050, 376}};
    const int nk = (q.K + MK - 1) / MK;
    const bool cut = nk > mx_chain(q.epi.out_f32, q.epi.f16);
    const double part = (q.epi.residual ? 3500 : 1000) * (q.epi.out_f32 ? 2 : 1);
    int best = 0;
    double least = 0.0;
    for (const auto &w : kTimes) {
        if (cut && w.bn == 256)
            continue;
        const int64_t tiles = ((int64_t(q.T) + 255) / 256) * ((int64_t(q.N) + w.bn - 1) / w.bn);
        const double c = double((tiles + pairs - 1) / pairs) * (w.round + nk * w.stage) +
                         part * (w.bn > 192 ? 2 : 1);
        if (!best || c < least) {
            best = w.bn;
            least = c;
        }
    }
    return best;
}

cudaError_t launch_mx_pair(const MxProduct &q, cudaStream_t s)
{
    const int pairs = std::max(1, device_sm_count() / 2);
    MxPairArgs g = {};
    MxArgs &a = g.p;
    static_cast<EpiArgs &>(a) = q.epi;
    a.status = q.status, a.stall = q.stall;
    a.chain = mx_chain(a.out_f32, a.f16);
    a.M = q.T, a.N = q.N, a.K = q.K, a.k_tiles = mx_k_tiles(q.K);
    a.bn = mx_pair_columns(q, pairs);
    a.n_mt = int((int64_t(q.T) + 2 * MM - 1) / (2 * MM));
    const int64_t tiles = int64_t(a.n_mt) * ((int64_t(q.N) + a.bn - 1) / a.bn);
    if (tiles > INT_MAX / 2)
        return cudaErrorInvalidValue;
    g.tiles = int(tiles);
    g.stage_bytes = mx_pair_stage(a.bn);
    const size_t epi = size_t(kMxEpiWarps) * (kMxSlot + kMxEpiCols * 4);
    g.stages = std::min<int>(kMxPairStages, int((kMxLoneSmem - 1024 - epi) / g.stage_bytes));
    cudaError_t e = mx_map(&g.a, q.x, q.T, q.K, MM);
    if (e == cudaSuccess)
        e = mx_map(&g.b, q.W, q.N, q.K, a.bn / 2);
    if (e == cudaSuccess)
        e = mx_scale_map(&g.a_scales, q.x_scales, q.T, q.K, 1);
    if (e == cudaSuccess)
        e = mx_scale_map(&g.b_scales, q.W_scales, q.N, q.K, mx_b_tiles(a.bn));
    if (e == cudaSuccess && a.vec_out)
        e = mx_out_map(&g.out, a);
    const MxTiles how = a.bn == 256 ? kWide : (q.K + MK - 1) / MK > a.chain ? kCut : kNarrow;
    const auto kern = reinterpret_cast<const void *>(
        how == kWide  ? mx_pair_kernel<kWide>(a.act, a.out_f32, a.f16)
        : how == kCut ? mx_pair_kernel<kCut>(a.act, a.out_f32, a.f16)
                      : mx_pair_kernel<kNarrow>(a.act, a.out_f32, a.f16));
    if (e == cudaSuccess)
        e = ensure_smem_limit(kern,
                              kSlotLinearMxPair + 7 * a.act +
                                  (how == kCut ? 6 : 3 * (how == kWide) + (a.out_f32 ? 2 : a.f16)),
                              kMxLoneSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {&g};
    return launch_clustered(kern, unsigned(2 * std::min<int64_t>(tiles, pairs)), 2, kMxPairThreads,
                            kMxLoneSmem, s, args);
}

// Which kernel.  Pairs of CTAs waste most of their 256 rows on a few, but a tile
// takes them 2.3 us and 0.22 for each stage of its whole reduction however few
// its rows are, where k_linear_mx splits the reduction eight ways at best and
// joins the parts in 3 to 10 us that grow with the rows.  Measured (us, k_linear_mx
// and pairs): 64 rows x 2560 x 10240 10.0 and 7.5 - 8.3, x 10240 x 2560 9.4 and 11.2, x
// 11264 x 11264 (split by two) 23.0 and 17.3, x 512 x 2560 8.1 and 4.0; 128 x 10240
// x 2560 14.5 and 11.5; 32 x 2560 x 2560 5.1 and 6.6, x 512 x 2560 6.2 and 4.0.
bool mx_takes_pairs(const MxProduct &q)
{
    const int nk = (q.K + MK - 1) / MK;
    if (!q.epi.out_f32 && nk > mx_chain(false, q.epi.f16))  // the pairs cut fp32 sums alone
        return false;
    if (q.T > 64)
        return true;
    if (q.T > 32)
        return nk <= 20 || MxSmall(q.T, q.K, q.N, device_sm_count()).split < kMxMaxSplit;
    return q.T > kMxQuantRows && nk <= 4;
}

cudaError_t launch_mx(const MxProduct &q, cudaStream_t s)
{
    return mx_takes_pairs(q) ? launch_mx_pair(q, s) : launch_mx_small(q, s);
}

}  // namespace

uint32_t *linear_mx_status_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_status) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

}  // namespace moe

namespace moe {
namespace {

constexpr int kMost = INT_MAX - 511;

// What both entry points check of a product, x's operands apart.
int mx_check(const uint8_t *W, const uint8_t *W_scales, const float *bias, const void *residual,
             int64_t ldr, int act, int T, int K, int N, const void *y, int64_t ldy, int y_dtype,
             const uint32_t *status)
{
    if (y_dtype != MOE_DT_BF16 && y_dtype != MOE_DT_F16 && y_dtype != MOE_DT_F32)
        return MOE_ERR_DTYPE;
    if (T < 0 || T > kMost || K < 32 || K > kMost || K % 32 != 0 || N < 1 || N > kMost ||
        act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH || ldy < N || (residual && ldr < N))
        return MOE_ERR_SHAPE;
    if (!W || !W_scales || (T > 0 && !y))
        return MOE_ERR_NULL;
    const int size = dtype_size(y_dtype);
    return aligned(W, 16) && aligned(W_scales, 16) && aligned(bias, 4) && aligned(residual, size) &&
                   aligned(y, size) && aligned(status, 4)
               ? MOE_OK
               : MOE_ERR_ALIGN;
}

int mx_linear(const uint8_t *x, const uint8_t *x_scales, const void *rows, int64_t ld, int type,
              const uint8_t *W, const uint8_t *W_scales, const float *bias, const void *residual,
              int64_t ldr, int act, int T, int K, int N, void *y, int64_t ldy, int y_dtype,
              uint32_t *status, cudaStream_t s, int stall = 0)
{
    const int size = dtype_size(y_dtype);
    EpiArgs e = {};
    e.bias = bias, e.residual = residual, e.out = y;
    e.ldr = ldr, e.ldo = ldy;
    e.f16 = y_dtype == MOE_DT_F16, e.out_f32 = y_dtype == MOE_DT_F32, e.act = act;
    e.vec_out = vec16(y, ldy, size), e.vec_res = vec16(residual, ldr, size);
    const MxProduct q{x, x_scales, W, W_scales, T, K, N, e, status, rows, ld, type, stall};
    return launch_mx(q, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Where moe_linear_rows_mxfp4's workspace holds the scales.
inline size_t mx_codes_bytes(int T, int K)
{
    return align256(size_t(T) * (K / 2));
}

}  // namespace
}  // namespace moe

extern "C" int moe_linear_mxfp4(const uint8_t *x, const uint8_t *x_scales, const uint8_t *W,
                                const uint8_t *W_scales, const float *bias, const void *residual,
                                int64_t ldr, int act, int T, int K, int N, void *y, int64_t ldy,
                                int y_dtype, uint32_t *status, moe_stream_t stream)
{
    using namespace moe;
    const int rc =
        mx_check(W, W_scales, bias, residual, ldr, act, T, K, N, y, ldy, y_dtype, status);
    if (rc != MOE_OK)
        return rc;
    if (T > 0 && (!x || !x_scales))
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_scales, 16))
        return MOE_ERR_ALIGN;
    if (T == 0)
        return MOE_OK;
    return mx_linear(x, x_scales, nullptr, 0, 0, W, W_scales, bias, residual, ldr, act, T, K, N, y,
                     ldy, y_dtype, status, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_linear_rows_mxfp4_workspace_bytes(int T, int K, int N)
{
    using namespace moe;
    if (T <= 0 || T > kMost || K < 32 || K > kMost || K % 32 != 0 || N < 1 || N > kMost ||
        MxSmall(T, K, N, device_sm_count()).quantises(T, K))
        return 0;
    return mx_codes_bytes(T, K) + align256(size_t(mx_scale_bytes(T, K)));
}

extern "C" int moe_linear_rows_mxfp4(const void *x, int64_t ldx, int x_dtype, const uint8_t *W,
                                     const uint8_t *W_scales, const float *bias,
                                     const void *residual, int64_t ldr, int act, int T, int K,
                                     int N, void *y, int64_t ldy, int y_dtype, void *ws,
                                     size_t ws_bytes, uint32_t *status, moe_stream_t stream)
{
    using namespace moe;
    if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F16 && x_dtype != MOE_DT_F32)
        return MOE_ERR_DTYPE;
    const int rc = mx_check(W, W_scales, bias, residual, ldr, act, T, K, N, y, ldy, y_dtype, status);
    if (rc != MOE_OK)
        return rc;
    const size_t need = moe_linear_rows_mxfp4_workspace_bytes(T, K, N);
    if (ldx < K)
        return MOE_ERR_SHAPE;
    if ((T > 0 && !x) || (need && !ws))
        return MOE_ERR_NULL;
    if (ws_bytes < need)
        return MOE_ERR_WORKSPACE;
    if (!aligned(x, dtype_size(x_dtype)) || (need && !aligned(ws, 256)))
        return MOE_ERR_ALIGN;
    if (T == 0)
        return MOE_OK;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!need)
        return mx_linear(nullptr, nullptr, x, ldx, x_dtype, W, W_scales, bias, residual, ldr, act,
                         T, K, N, y, ldy, y_dtype, status, s);
    uint8_t *codes = static_cast<uint8_t *>(ws), *scales = codes + mx_codes_bytes(T, K);
    const int quantised = moe_quantize_rows_mxfp4(x, ldx, x_dtype, T, K, codes, scales, stream);
    return quantised != MOE_OK ? quantised
                               : mx_linear(codes, scales, nullptr, 0, 0, W, W_scales, bias, residual,
                                           ldr, act, T, K, N, y, ldy, y_dtype, status, s);
}

extern "C" int moe_selftest_linear_mxfp4_wait_limit(const void *x, const uint8_t *x_scales,
                                                    const uint8_t *W, const uint8_t *W_scales,
                                                    int T, int K, int N, void *y, int y_dtype,
                                                    uint32_t *status, int cta, moe_stream_t stream)
{
    using namespace moe;
    const int rc = mx_check(W, W_scales, nullptr, nullptr, 0, MOE_ACT_NONE, T, K, N, y, N, y_dtype,
                            status);
    if (rc != MOE_OK)
        return rc;
    if (T == 0 || cta < 0 || cta == INT_MAX ||
        (!x_scales && moe_linear_rows_mxfp4_workspace_bytes(T, K, N)))
        return MOE_ERR_SHAPE;
    if (!x)
        return MOE_ERR_NULL;
    if (!aligned(x, x_scales ? 16 : 2) || !aligned(x_scales, 16))
        return MOE_ERR_ALIGN;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return x_scales ? mx_linear(static_cast<const uint8_t *>(x), x_scales, nullptr, 0, 0, W,
                                W_scales, nullptr, nullptr, 0, MOE_ACT_NONE, T, K, N, y, N, y_dtype,
                                status, s, cta + 1)
                    : mx_linear(nullptr, nullptr, x, K, MOE_DT_BF16, W, W_scales, nullptr, nullptr,
                                0, MOE_ACT_NONE, T, K, N, y, N, y_dtype, status, s, cta + 1);
}
