// quant_format.cuh -- the 4-bit KV cache: its layout in memory, how 32 values
// become codes, and how codes become fp16 values again.
//
// 32 neighbouring dims of one token, KV head and side (K or V) share two fp16
// numbers s and b; code n in 0..15 stands for the fp16 number nearest to
// s (16 + n) + b.  16 + n is an fp16 number whose four low code bits sit at
// mantissa bits 6..9 of the constant 16, so a code is one AND/OR away from it
// and a value one packed fused multiply-add (one rounding) away from the code.
//
// A page of one head holds blocks of TB = min(page_size, 64) tokens (so that a
// 64-token tile is whole blocks); a block is one contiguous run of
// TB * d * 5 / 4 bytes in four parts, GR = d / 32:
//   K codes   [token][t 4][j GR][e 2] 16-bit halves; field f of a half is the
//             code of dim 32 j + 8 f + 2 t + e
//   K params  [token][s | b][j GR] fp16
//   V codes   [token / 8][g 8][t 4][j GR][e 2] halves; field f is the code of
//             dim 32 j + 8 f + g of token 2 t + e of the eight
//   V params  [token / 8][t 4][j GR][s | b][e 2] fp16
// Code fields of a 16-bit half: f = 0 bits 6..9, f = 1 bits 2..5, f = 2 bits
// 10..13, f = 3 the low two bits at 14..15 and the high two at 0..1: the halves
// of two codes (e = 0, 1) are one word, from which a mask takes f = 0 in place,
// a shift by 4 either way f = 1 and f = 2, and a byte swap f = 3.
// These are the register fragments of mma.m16n8k16: lane (g, t) finds in its
// word j the A operand's (row g, k pair t) of K (tokens x dims) and of V^T
// (dims x tokens).  Each token owns whole halves, so that a token is written
// without reading its neighbours.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pkv {

constexpr float kQuantLimit = 16384.f;  // values beyond it are stored as it: b = lo - 16 s stays finite

__host__ __device__ inline int quant_block_tokens(int page_size) { return page_size < 64 ? page_size : 64; }
__host__ __device__ inline int quant_block_bytes(int tb, int d) { return tb * d * 5 / 4; }

// Byte offsets inside a block of tb tokens.
template <int D>
struct QuantLayout {
    static constexpr int GR = D / 32;
    static constexpr int kRow = D / 2;            // K code bytes of a token
    static constexpr int kParamRow = GR * 4;      // K param bytes of a token
    static constexpr int kVGroup = 8 * D / 2;     // V code bytes of eight tokens
    static constexpr int kVParamGroup = 8 * GR * 4;
    __host__ __device__ static int k_params(int tb) { return tb * kRow; }
    __host__ __device__ static int v_codes(int tb) { return tb * (kRow + kParamRow); }
    __host__ __device__ static int v_params(int tb) { return tb * (2 * kRow + kParamRow); }
    __host__ __device__ static int bytes(int tb) { return tb * D * 5 / 4; }
};

#ifdef __CUDACC__

// The packed pair 16 + n of field f of a word's two halves.
template <int F>
__device__ __forceinline__ uint32_t quant_field(uint32_t w)
{
    const uint32_t x = F == 0 ? w : F == 1 ? w << 4 : F == 2 ? w >> 4 : __byte_perm(w, 0, 0x2301);
    uint32_t n;  // (x & mask) | 16: one instruction, which the compiler makes two of when both constants are immediates
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(n) : "r"(x), "r"(0x03c003c0u), "r"(0x4c004c00u));
    return n;
}

// s (16 + n) + b of a packed pair, rounded once.
__device__ __forceinline__ uint32_t quant_value(uint32_t n16, __half2 s, __half2 b)
{
    const __half2 v = __hfma2(*reinterpret_cast<const __half2 *>(&n16), s, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// s and b of a group with least value lo and greatest hi (both within
// +-kQuantLimit), exactly as the format defines them, although (hi - lo) / 15
// and lo - 16 s need more bits than fp32 has: every comparison of an exact sum
// x y + z against an fp16 number c is made on the sum rounded towards the side
// that keeps its order with c (c is itself an fp32 number, so rounding down
// keeps x y + z >= c, and rounding down keeps x y + z < c).
__device__ __forceinline__ void quant_params(float lo, float hi, __half &s, __half &b)
{
    // least fp16 s with 15 s >= hi - lo: rounding up all the way gives it or,
    // past a representable quotient, its successor
    const __half s1 = __float2half_ru(__fmul_ru(__fsub_ru(hi, lo), 0x1.111112p-4f));
    // (its bits less one are its predecessor's)
    const __half s0 = __ushort_as_half((unsigned short)(__half_as_ushort(s1) - 1));
    s = __fmaf_rd(15.f, __half2float(s0), lo) >= hi ? s0 : s1;
    s = hi > lo ? s : __ushort_as_half(0);
    // nearest to lo - 16 s, the lower one on a tie
    const float sf = __half2float(s);
    const __half b0 = __float2half_rd(__fmaf_rd(-16.f, sf, lo)), b1 = __float2half_ru(__fmaf_ru(-16.f, sf, lo));
    const float mid = 0.5f * (__half2float(b0) + __half2float(b1));
    b = __fmaf_rd(16.f, sf, mid) < lo ? b1 : b0;
}

#endif  // __CUDACC__

}  // namespace pkv
