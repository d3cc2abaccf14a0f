// Rows to MXFP4 and back (moe_quantize_rows_mxfp4, moe_dequantize_rows_mxfp4).
// The format: mx_rows.cuh.
//
// 4096 x 11264 bf16 takes 21.3 us (117 MB, 5.5 TB/s) and back 21.7, 8192 x 16384
// 58 and 59.  What bounds them is memory (to write zeros to the 92 MB takes 23.3
// us, to the 268 MB 66.7) and, quantising, instructions (67 % of the issue slots):
// there a thread has sixteen elements and eight lanes a scale tile's 128 of one row
// (with eight elements a thread, twice the lanes per block, 31 us).  Reading back, a
// thread has eight, whose 16 bytes of output then lie side by side.
#include "../../include/moe_prefill.h"
#include "internal.h"
#include "mx_rows.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <climits>

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kQuantLanes = 8, kReadLanes = 16;  // of 128 elements
constexpr int kQuantAhead = 2, kReadAhead = 4;   // pieces of 128 a thread has in flight
// CTAs that an SM holds; twice as many are launched where each of their threads has
// a full turn of pieces (quantising 4096 x 11264 21.3 us, with 8 an SM 22.5, with 16
// 22.0; 2048 x 2560 3.4 us, with 10 an SM 5.0).
constexpr int kRowCtas = 5;

struct MxRowsArgs {
    const void *x;  // rows to quantise, or null
    void *y;        // rows to write
    int64_t ld;
    uint8_t *codes, *scales;
    int64_t rows, all_rows;  // all_rows: of the scale tiles
    int K, k_tiles, vec;
};

// Walks pieces (row, tile along K) with one division at the start.
struct Piece {
    int64_t row;
    int kt;

    __device__ Piece(int64_t i, int k_tiles) : row(i / k_tiles), kt(int(i % k_tiles)) {}

    __device__ __forceinline__ void advance(int64_t rows, int tiles, int k_tiles)
    {
        row += rows;
        kt += tiles;
        if (kt >= k_tiles) {
            kt -= k_tiles;
            ++row;
        }
    }
};

template <typename E>
__global__ void __launch_bounds__(kRowThreads, 4) k_quant_rows(const MxRowsArgs p)
{
    constexpr int kPieces = kRowThreads / kQuantLanes;
    const int lane = threadIdx.x % kQuantLanes;
    const int64_t step = int64_t(gridDim.x) * kPieces;
    const int64_t step_rows = step / p.k_tiles;
    const int step_tiles = int(step % p.k_tiles);
    Piece at(int64_t(blockIdx.x) * kPieces + threadIdx.x / kQuantLanes, p.k_tiles);
    pdl_wait();
    pdl_launch_dependents();
    // (all of a warp's pieces walk on while one of them has rows left)
    while (__any_sync(0xffffffffu, at.row < p.all_rows)) {
        Oct<E> in[kQuantAhead][2];
        Piece of[kQuantAhead] = {at, at};
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            of[u] = at;
            const int c = at.kt * 128 + lane * 16, left = at.row < p.rows ? p.K - c : 0;
            const E *x = static_cast<const E *>(p.x) + (left > 0 ? at.row * p.ld + c : 0);
            in[u][0].load(x, left, p.vec);
            in[u][1].load(x + 8, left - 8, p.vec);
            at.advance(step_rows, step_tiles, p.k_tiles);
        }
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            const uint32_t byte = mx_scale_byte(
                max_of_lanes<2>(max(in[u][0].max_bits(), in[u][1].max_bits())));
            const uint32_t word = word_of_tile<2>(byte);
            const int c = of[u].kt * 128 + lane * 16;
            if (of[u].row < p.rows && c < p.K) {
                float v[8];
                uint2 codes;
                in[u][0].to(v);
                codes.x = mx_encode8(v, byte);
                in[u][1].to(v);
                codes.y = mx_encode8(v, byte);
                *reinterpret_cast<uint2 *>(p.codes + of[u].row * (p.K / 2) + c / 2) = codes;
            }
            if (lane == 0 && of[u].row < p.all_rows)
                *mx_scale_word(p.scales, of[u].row, of[u].kt, p.k_tiles) = word;
        }
    }
}

// 128 elements of a row, eight from each of 16 lanes (of `mask`), n of which exist:
// through `slot`, neighbouring words by neighbouring lanes.  For 16-bit rows that are
// not aligned (element by element, 4096 x 11264 took 131 us instead of 34) and fp32
// ones, whose 16-byte pieces would fill half a sector an instruction (48 instead of 39).
template <typename E>
__device__ __forceinline__ void put_piece(E *to, int n, const Oct<E> &o, uint32_t *slot,
                                          uint32_t mask)
{
    const int lane = threadIdx.x % kReadLanes;
    __syncwarp(mask);  // the slot has been read
#pragma unroll
    for (int i = 0; i < Oct<E>::kWords / 4; ++i)
        reinterpret_cast<uint4 *>(slot)[lane * (Oct<E>::kWords / 4) + i] = o.get(i);
    __syncwarp(mask);
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 16 * i < n)
                reinterpret_cast<uint32_t *>(to)[lane + 16 * i] = slot[lane + 16 * i];
    } else {
        // from the second element on where the first lies in the upper half of a word
        uint16_t *const first = reinterpret_cast<uint16_t *>(to);
        const int odd = int(reinterpret_cast<uintptr_t>(to) >> 1 & 1);
        if (odd && lane == 0)
            first[0] = uint16_t(slot[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = lane + 16 * i, e = 2 * w + odd;
            const uint32_t v = odd ? __funnelshift_r(slot[w], slot[w + 1], 16) : slot[w];
            if (e + 1 < n)
                *reinterpret_cast<uint32_t *>(first + e) = v;
            else if (e < n)
                first[e] = uint16_t(v);
        }
    }
}

template <typename E, bool VEC>
__global__ void __launch_bounds__(kRowThreads, 4) k_dequant_rows(const MxRowsArgs p)
{
    constexpr int kSlot = VEC ? 4 : kReadLanes * Oct<E>::kWords + 4;  // of a piece, and a word more
    __shared__ __align__(16) uint32_t slots[kRowThreads / kReadLanes * kSlot];
    uint32_t *const slot = slots + threadIdx.x / kReadLanes * kSlot;
    const uint32_t mask = 0xffffu << (threadIdx.x & 16);
    constexpr int kPieces = kRowThreads / kReadLanes;
    const int lane = threadIdx.x % kReadLanes;
    const int64_t step = int64_t(gridDim.x) * kPieces;
    const int64_t step_rows = step / p.k_tiles;
    const int step_tiles = int(step % p.k_tiles);
    Piece at(int64_t(blockIdx.x) * kPieces + threadIdx.x / kReadLanes, p.k_tiles);
    pdl_wait();
    pdl_launch_dependents();
    while (at.row < p.rows) {
        uint32_t code[kReadAhead], word[kReadAhead];
        Piece of[kReadAhead] = {at, at, at, at};
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            of[u] = at;
            const int c = at.kt * 128 + lane * 8;
            code[u] = word[u] = 0;
            if (at.row < p.rows && c < p.K) {
                code[u] = __ldcs(
                    reinterpret_cast<const uint32_t *>(p.codes + at.row * (p.K / 2) + c / 2));
                word[u] = *mx_scale_word(p.scales, at.row, at.kt, p.k_tiles);
            }
            at.advance(step_rows, step_tiles, p.k_tiles);
        }
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const int c = of[u].kt * 128 + lane * 8;
            if (of[u].row >= p.rows || (VEC && c >= p.K))
                continue;
            float v[8];
            mx_decode8(code[u], (word[u] >> (8 * (lane >> 2))) & 0xffu, v);
            Oct<E> out;
            out.from(v);
            E *const y = static_cast<E *>(p.y) + of[u].row * p.ld;
            if (VEC)
                out.store(y + c, 8, true);
            else
                put_piece(y + of[u].kt * 128, min(p.K - of[u].kt * 128, 128), out, slot, mask);
        }
    }
}

// `lanes` of a piece of 128 elements, `ahead` of which a thread has in flight.
cudaError_t launch(void (*kern)(MxRowsArgs), const MxRowsArgs &a, int64_t rows, int lanes, int ahead,
                   cudaStream_t s)
{
    const int64_t pieces = rows * a.k_tiles, of_cta = kRowThreads / lanes;
    const int64_t held = int64_t(device_sm_count()) * kRowCtas;
    const auto ctas_of = [&](int64_t n) { return (pieces + n - 1) / n; };
    const int64_t ctas =
        std::min(ctas_of(of_cta), std::clamp(ctas_of(of_cta * ahead), held, 2 * held));
    return launch_pdl(kern, dim3(unsigned(ctas)), dim3(kRowThreads), 0, s, a);
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int check(const void *x, int64_t ld, int dtype, int rows, int K, const uint8_t *codes,
          const uint8_t *scales)
{
    if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16 && dtype != MOE_DT_F32)
        return MOE_ERR_DTYPE;
    if (rows < 0 || rows > INT_MAX - 511 || K < 32 || K % 32 != 0 || K > INT_MAX - 511 || ld < K)
        return MOE_ERR_SHAPE;
    if (rows > 0 && (!x || !codes || !scales))
        return MOE_ERR_NULL;
    if (!aligned(x, dtype_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 16))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_mxfp4_scale_bytes(int rows, int K)
{
    return rows < 0 || K < 32 || K % 32 != 0 ? 0 : size_t(moe::mx_scale_bytes(rows, K));
}

extern "C" int moe_quantize_rows_mxfp4(const void *x, int64_t ldx, int dtype, int rows, int K,
                                       uint8_t *codes, uint8_t *scales, moe_stream_t stream)
{
    using namespace moe;
    const int rc = check(x, ldx, dtype, rows, K, codes, scales);
    if (rc != MOE_OK || rows == 0)
        return rc;
    MxRowsArgs a = {};
    a.x = x, a.ld = ldx, a.codes = codes, a.scales = scales;
    a.rows = rows, a.all_rows = (int64_t(rows) + 127) / 128 * 128;
    a.K = K, a.k_tiles = mx_k_tiles(K);
    a.vec = rows_vec(x, ldx, dtype_size(dtype));
    const auto kern = dtype == MOE_DT_F32   ? k_quant_rows<float>
                      : dtype == MOE_DT_F16 ? k_quant_rows<__half>
                                            : k_quant_rows<__nv_bfloat16>;
    return launch(kern, a, a.all_rows, kQuantLanes, kQuantAhead,
                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

extern "C" int moe_dequantize_rows_mxfp4(const uint8_t *codes, const uint8_t *scales, int rows,
                                         int K, void *y, int64_t ldy, int dtype,
                                         moe_stream_t stream)
{
    using namespace moe;
    if (dtype == MOE_DT_F16)  // does not hold every scale
        return MOE_ERR_DTYPE;
    const int rc = check(y, ldy, dtype, rows, K, codes, scales);
    if (rc != MOE_OK || rows == 0)
        return rc;
    MxRowsArgs a = {};
    a.y = y, a.ld = ldy;
    a.codes = const_cast<uint8_t *>(codes), a.scales = const_cast<uint8_t *>(scales);
    a.rows = a.all_rows = rows;
    a.K = K, a.k_tiles = mx_k_tiles(K);
    a.vec = rows_vec(y, ldy, dtype_size(dtype));
    const auto kern = dtype == MOE_DT_F32 ? k_dequant_rows<float, false>
                      : a.vec             ? k_dequant_rows<__nv_bfloat16, true>
                                          : k_dequant_rows<__nv_bfloat16, false>;
    return launch(kern, a, rows, kReadLanes, kReadAhead, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
