// byte_format.cuh -- the 8-bit KV cache: its layout in memory, how values become
// codes, and how codes become fp16 numbers again.
//
// SB = min(page_size, 16) neighbouring tokens of one KV head and side (K or V)
// share a scale 2^e, kept as the fp32 number it is; code c stands for c 2^e, c an
// int8 or an e4m3 float.  With a power of two, quantising is one rounding of an
// exact product, a value an fp16 number exactly, and an earlier code's change to
// a greater scale one rounding.
//
// A page of one head holds blocks of TB = min(page_size, 64) tokens; a block is
// one contiguous run in three parts:
//   K codes  [token][dim]; with d = 128 the two 64-byte halves of tokens 2 and 3
//            of every four are swapped
//   V codes  [token / SB][dim / 4][token % SB / 4][dim % 4][token % 4]
//   scales   [token / SB][K | V] fp32, padded to 16 bytes
// A 32-bit word holds four dims of a token of K, four tokens of a dim of V: what
// a lane of mma.m16n8k16 holds of one row of its A operand (K: tokens x dims, V^T:
// dims x tokens), whose k index may be permuted as one likes.  Sixteen bytes are
// four such words, and the swapped halves spread the rows that a warp reads at
// once over all banks of shared memory.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace pkv {

enum ByteFormat : int { kInt8 = 0, kE4m3 = 1 };

__host__ __device__ constexpr int byte_block_tokens(int page_size) { return page_size < 64 ? page_size : 64; }
__host__ __device__ constexpr int byte_scale_tokens(int page_size) { return page_size < 16 ? page_size : 16; }
// Bytes of a block of tb tokens and of its scales.
__host__ __device__ constexpr int byte_scale_bytes(int tb) { return tb >= 64 ? tb / 2 : 16; }
__host__ __device__ constexpr int byte_block_bytes(int tb, int d) { return 2 * tb * d + byte_scale_bytes(tb); }

// The exponent of a scale is in [least, most]; values beyond its greatest code
// times 2^most are stored as that.
template <int FMT>
struct Byte {
    static constexpr int kLeast = FMT == kInt8 ? -24 : -15;
    static constexpr int kMost = FMT == kInt8 ? 9 : 7;
    static constexpr int kTopExp = FMT == kInt8 ? 6 : 8;                        // the greatest code is 1.984375 2^6 = 127
    static constexpr uint32_t kTopMant = FMT == kInt8 ? 0x7e0000u : 0x600000u;  // or 1.75 2^8 = 448: exponent, fp32 mantissa
    static constexpr float kLimit = FMT == kInt8 ? 65024.f : 57344.f;           // the greatest code times 2^most
};

#ifdef __CUDACC__

// 2^e for e in [-126, 127].
__device__ __forceinline__ float byte_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The exponent of a stored scale, one outside the format's range as the nearest in it.
template <int FMT>
__device__ __forceinline__ int byte_exponent(float s)
{
    return min(max((int)(__float_as_uint(s) >> 23 & 255) - 127, Byte<FMT>::kLeast), Byte<FMT>::kMost);
}

// The least exponent whose greatest code reaches the greatest magnitude, given as fp16 bits (not a NaN's).
template <int FMT>
__device__ __forceinline__ int byte_least_exponent(uint32_t top)
{
    const uint32_t b = __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
    const int e = (int)(b >> 23) - 127 - Byte<FMT>::kTopExp + ((b & 0x7fffffu) > Byte<FMT>::kTopMant);
    return min(max(e, Byte<FMT>::kLeast), Byte<FMT>::kMost);
}

__device__ __forceinline__ __half2 byte_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t byte_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// How a block's values become codes: x 2^-e in one or two exact steps.
template <int FMT>
struct ByteQuantiser {
    __half2 mul, pre;
    bool two, clamp;
    __device__ __forceinline__ ByteQuantiser(int e, uint32_t top)
    {
        // 2^-e is an fp16 number from e = -15 on; below (int8) x is multiplied by 2^9 first, which keeps it under 1
        two = FMT == kInt8 && e < -15;
        pre = __float2half2_rn(512.f);
        mul = __float2half2_rn(byte_pow2(two ? -e - 9 : -e));
        clamp = FMT == kInt8 && __half2float(__ushort_as_half((unsigned short)top)) > Byte<FMT>::kLimit;
    }
    // The codes of four values, a byte each.
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const
    {
        __half2 x = byte_half2(a), y = byte_half2(b);
        if constexpr (FMT == kInt8) {
            if (clamp) {
                const __half2 top = __float2half2_rn(Byte<FMT>::kLimit), least = __hneg2(top);
                x = __hmin2(__hmax2(x, least), top);
                y = __hmin2(__hmax2(y, least), top);
            }
            if (two) {
                x = __hmul2(x, pre);
                y = __hmul2(y, pre);
            }
            // fp16 numbers from 1024 to 2048 are 1 apart: the sum's rounding is the code's, which its low byte holds
            const __half2 magic = __float2half2_rn(1536.f);
            return __byte_perm(byte_word(__hfma2(x, mul, magic)), byte_word(__hfma2(y, mul, magic)), 0x6420);
        } else {
            // products that are too small for fp16 are beneath half the least code; greater than the greatest: saturated
            const __half2_raw u = __hmul2(x, mul), v = __hmul2(y, mul);
            return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(u, __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << 16;
        }
    }
};

// The codes of a word as fp16 numbers: bytes 0 and 1, and bytes 2 and 3.
template <int FMT>
__device__ __forceinline__ void byte_numbers(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (FMT == kInt8) {
        // n + 128 as the low byte of 1024 + (n + 128)
        const __half2 bias = byte_half2(0x64806480u);  // 1152
        const uint32_t u = w ^ 0x80808080u;
        lo = byte_word(__hsub2(byte_half2(__byte_perm(u, 0x64646464u, 0x4140)), bias));
        hi = byte_word(__hsub2(byte_half2(__byte_perm(u, 0x64646464u, 0x4342)), bias));
    } else {
        // the conversion of the type: shifts and masks of exponent and mantissa under fp16's bias take seven
        // instructions a word instead of two (120k tokens of 8 heads decoded in 45.4 us, 43.7 with this)
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

// Four codes c 2^k (k <= 0) rounded to codes again, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t byte_shift(uint32_t w, int k)
{
    uint32_t lo, hi;
    byte_numbers<FMT>(w, lo, hi);
    const float f = byte_pow2(max(k, -100));
    auto scaled = [&](uint32_t x) {
        const float2 v = __half22float2(byte_half2(x));
        return make_float2(v.x * f, v.y * f);
    };
    const float2 a = scaled(lo), b = scaled(hi);
    auto code = [](float x) -> uint32_t {
        if constexpr (FMT == kInt8)
            return (uint32_t)__float2int_rn(x) & 255u;
        else
            return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    };
    return code(a.x) | code(a.y) << 8 | code(b.x) << 16 | code(b.y) << 24;
}

// A 4 x 4 transposition of bytes.
__device__ __forceinline__ uint4 byte_transpose(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);
    const uint32_t AB = __byte_perm(a, b, 0x7362), CD = __byte_perm(c, d, 0x7362);
    return make_uint4(__byte_perm(ab, cd, 0x5410), __byte_perm(ab, cd, 0x7632), __byte_perm(AB, CD, 0x5410),
                      __byte_perm(AB, CD, 0x7632));
}

// Byte offsets inside a block: of 16 bytes of K or less, which start at dim x of
// its token r; of the 16 bytes of V that hold dims 4 x4 .. and tokens 4 t .. of a
// scale block of 2^lg tokens, from that block's start; and where the parts are.
template <int D>
__device__ __forceinline__ int byte_k_at(int r, int x) { return r * D + (D == 128 ? x ^ ((r & 2) << 5) : x); }
__device__ __forceinline__ int byte_v_at(int x4, int t, int lg) { return ((x4 << (lg - 2)) + t) * 16; }
template <int D>
__device__ __forceinline__ int byte_v_part(int tb, int r, int lg) { return (tb + (r >> lg << lg)) * D; }
template <int D>
__device__ __forceinline__ int byte_scale_part(int tb, int r, int lg) { return 2 * tb * D + (r >> lg) * 8; }

#endif  // __CUDACC__

}  // namespace pkv
