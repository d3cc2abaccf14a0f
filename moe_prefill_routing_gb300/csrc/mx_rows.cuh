// Rows in MXFP4 (OCP Microscaling: 4-bit E2M1 elements, one power-of-two scale
// for each 32 along the row) in the layout that tcgen05.mma.kind::mxf4 reads,
// and rows of 16-bit or fp32 elements eight at a time.
//
// Codes [rows, K / 2]: element 2i in the low half of byte i.  Scales: byte S of
// 2^(S - 127), in tiles of 128 rows x 4 blocks (128 of K) of 512 bytes,
// [ceil(rows / 128), ceil(K / 128), 512]: of a tile, row 32 q + l, block b at
// byte 16 l + 4 q + b, so that one tcgen05.cp (32 lanes x 16 bytes) brings a
// tile into the four columns of tensor memory where the MMA looks for it.
// What lies past the last row or block is 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace moe {

constexpr int kMxTileBytes = 512;

__host__ __device__ __forceinline__ int mx_k_tiles(int K)
{
    return (K + 127) / 128;
}

inline int64_t mx_scale_bytes(int64_t rows, int K)
{
    return (rows + 127) / 128 * mx_k_tiles(K) * kMxTileBytes;
}

// Where the four scale bytes of row t, tile kt along K, are (a 32-bit word).
__device__ __forceinline__ uint32_t *mx_scale_word(uint8_t *scales, int64_t t, int kt, int k_tiles)
{
    return reinterpret_cast<uint32_t *>(scales + ((t >> 7) * k_tiles + kt) * kMxTileBytes +
                                        (t & 31) * 16 + ((t >> 5) & 3) * 4);
}

// The scale byte of a block whose largest |v| has these bits:
// floor(log2 max) - 2 (2: the exponent of E2M1's largest value, 6 = 1.5 x 2^2),
// at least -127; 255 (NaN) where an element is a NaN or an infinity.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t max_bits)
{
    const int f = int(max_bits >> 23);
    return f == 255 ? 255u : uint32_t(max(f - 2, 0));
}

// Eight elements (v 2^-x, x = byte - 127) to codes: nearest, ties to the even
// code, past 6 saturated, the sign kept; 0 for a block without a finite scale.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], uint32_t byte)
{
    if (byte == 255u)
        return 0u;
    const float r = __uint_as_float((254u - byte) << 23);  // byte <= 252: 2^-125 at least
    uint32_t w;
    asm("{\n"
        ".reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n"
        "}\n"
        : "=r"(w)
        : "f"(v[0] * r), "f"(v[1] * r), "f"(v[2] * r), "f"(v[3] * r), "f"(v[4] * r),
          "f"(v[5] * r), "f"(v[6] * r), "f"(v[7] * r));
    return w;
}

// What eight codes and their scale byte stand for (exact in bf16 and fp32).
__device__ __forceinline__ void mx_decode8(uint32_t w, uint32_t byte, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n"
        ".reg .b8 a, b, c, d;\n"
        "mov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n"
        "}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
    // 2^-127 is subnormal; 255 stands for NaN
    const float s = byte == 0u     ? __uint_as_float(1u << 22)
                    : byte == 255u ? __uint_as_float(0x7fc00000u)
                                   : __uint_as_float(byte << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// The largest of L neighbouring lanes' values.
template <int L>
__device__ __forceinline__ uint32_t max_of_lanes(uint32_t m)
{
#pragma unroll
    for (int o = 1; o < L; o *= 2)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The scale bytes of a tile's four blocks, of L lanes each, as a word (in every
// lane).
template <int L>
__device__ __forceinline__ uint32_t word_of_tile(uint32_t byte)
{
    uint32_t w = byte << (8 * (threadIdx.x / L % 4));
    w |= __shfl_xor_sync(0xffffffffu, w, L);
    return w | __shfl_xor_sync(0xffffffffu, w, 2 * L);
}

// ---- two fp32 values that one instruction works on ---------------------------------

using Two = unsigned long long;

__device__ __forceinline__ Two two(float a, float b)
{
    Two v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}

__device__ __forceinline__ Two both(float a)
{
    return two(a, a);
}

__device__ __forceinline__ void apart(Two v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ float sum_of(Two v)
{
    float a, b;
    apart(v, a, b);
    return a + b;
}

__device__ __forceinline__ Two mul(Two a, Two b)
{
    Two v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

// ---- eight neighbouring elements of a row ----------------------------------------

// As they are stored, in 32-bit words (two 16-bit elements a word).
template <typename E>
struct alignas(16) Oct {
    static constexpr int kWords = 2 * int(sizeof(E));
    uint32_t w[kWords];

    // The first n exist (the others are 0); vec: 16-byte accesses are aligned.
    __device__ __forceinline__ void load(const E *p, int n, bool vec)
    {
        if (vec && n >= 8) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                set(i, __ldcs(reinterpret_cast<const uint4 *>(p) + i));
        } else {
            using Bits = std::conditional_t<sizeof(E) == 4, uint32_t, uint16_t>;
            const Bits *q = reinterpret_cast<const Bits *>(p);
            uint32_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = i < n ? uint32_t(q[i]) : 0u;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = sizeof(E) == 4 ? e[i % 8] : e[2 * i % 8] | e[(2 * i + 1) % 8] << 16;
        }
    }

    __device__ __forceinline__ void set(int i, uint4 q)
    {
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }

    __device__ __forceinline__ uint4 get(int i) const
    {
        return make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }

    __device__ __forceinline__ void store(E *p, int n, bool vec) const
    {
        if (vec && n >= 8) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] = get(i);
        } else {
            using Bits = std::conditional_t<sizeof(E) == 4, uint32_t, uint16_t>;
            Bits *q = reinterpret_cast<Bits *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    q[i] = Bits(sizeof(E) == 4 ? w[i % kWords]
                                               : w[i / 2 % kWords] >> (16 * (i & 1)));
        }
    }

    // The bits, as a float, of the largest |v|; of a NaN or an infinity if there
    // is one.
    __device__ __forceinline__ uint32_t max_bits() const
    {
        if constexpr (sizeof(E) == 4) {
            uint32_t m = w[0] & 0x7fffffffu;
#pragma unroll
            for (int i = 1; i < 8; ++i)
                m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int i = 1; i < 4; ++i)
                m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
            if constexpr (std::is_same<E, __nv_bfloat16>::value)
                return m << 16;
            else
                return __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
        }
    }

    __device__ __forceinline__ void to(float (&v)[8]) const
    {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        }
    }

    __device__ __forceinline__ void to(Two (&v)[4]) const
    {
        float f[8];
        to(f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = two(f[2 * i], f[2 * i + 1]);
    }

    __device__ __forceinline__ void from(const Two (&v)[4])
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            apart(v[i], f[2 * i], f[2 * i + 1]);
        from(f);
    }

    __device__ __forceinline__ void from(const float (&v)[8])
    {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<E, __nv_bfloat16>::value) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
        }
    }
};

// Whether 16-byte pieces of rows `ld` elements apart are aligned accesses.
inline bool rows_vec(const void *p, int64_t ld, int size)
{
    return ld * size % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

inline int dtype_size(int dtype)
{
    return dtype == 2 ? 4 : 2;  // MOE_DT_F32, or a 16-bit type
}

}  // namespace moe
