// quant.cu -- writing the 4-bit KV cache and reading it back.
//
// append: K and V of new tokens, packed [T][Hkv][d] fp16 with a stride between
// tokens, become codes in the pages their rows' block tables name, at positions
// seq_lens[i] .. ; lengths advance once every CTA has read them.
// read: tokens of the cache become packed fp16 K and V again.
//
// Both are one pass over their data: append reads 2 bytes per value and writes
// 0.625, read the other way round.  42k tokens of 8 heads, d = 128, are 226 MB,
// 33 us at the copy rate: read takes 39 us, append 50, where its some fifteen
// instructions per value are the bound (issue 73%, ALU 62%, DRAM 49%).
//
// A warp takes eight tokens, four lanes each, and loops over KV heads and sides,
// so that rows, pages and offsets are looked up once for all of them; short
// calls split the heads over more warps.  Lane t of a token's four holds the
// words (t, j), the codes of dims 32 j + 8 f + 2 t and the next (f = 0..3).
// append brings a tile (eight tokens of one head and side) into shared memory
// while it works on the one before, and reads its words from there: read from
// global memory 16 bytes at a time they cost an exchange among the four lanes
// (two instructions per value, 65 against 62 us when this was tried), four bytes
// at a time many L1 lookups (d = 64: 39.2 against 37.7 us).  read does make that
// exchange, since four-byte stores would reach L2 one by one.
#include "append_rows.cuh"
#include "pkv_device.cuh"
#include "pkv_kernels.h"
#include "quant_format.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs per SM of the append: with 80 registers a thread 49.6 us (42k tokens of 8
// heads), with the 64 of four CTAs 55.3 us, with two CTAs 53.7 us.
constexpr int kAppendCtas = 3;

// Row of packed token x, offsets[0] <= x < offsets[B]: the last i in [0, B) with offsets[i] <= x.
__device__ __forceinline__ int row_of(const int32_t *offsets, int B, int x)
{
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// 4x4 transpose over a quad: lane t gives word f of v to lane f, which gets
// them in the order of t.
__device__ __forceinline__ uint4 quad_transpose(const uint32_t (&v)[4], int t)
{
    const bool up = (t & 2) != 0, odd = (t & 1) != 0;
    const uint32_t k0 = up ? v[2] : v[0], k1 = up ? v[3] : v[1];
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 2);
    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 2);
    const uint32_t own = odd ? k1 : k0, across = odd ? r1 : r0;
    const uint32_t near = __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
    const uint32_t far = __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 1);
    const uint32_t a0 = odd ? near : own, a1 = odd ? own : near;          // lanes of this half of the quad
    const uint32_t b0 = odd ? far : across, b1 = odd ? across : far;      // of the other half
    return up ? make_uint4(b0, b1, a0, a1) : make_uint4(a0, a1, b0, b1);
}

template <int GR>
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[GR])
{
    if constexpr (GR == 4) {
        const uint4 v = *static_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *static_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

template <int GR>
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[GR])
{
    if constexpr (GR == 4)
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// 16 bytes from global to shared memory, and waiting for all but the last N
// batches of such copies.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 1 / x for normal x, within 2^-23 of itself.
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half lo, __half hi) { return as_word(__halves2half2(lo, hi)); }

// The four code pairs of quantise_rows() below, decided exactly; out of line, so
// that the loop around it stays small.  y is near enough to tell the two codes
// in question, and the border between them decides.
__device__ __noinline__ uint4 quant_codes_exact(uint4 x, float s, float b)
{
    if (!(s > 0.f))  // 0 or NaN
        return make_uint4(0, 0, 0, 0);
    const float i = rcp_approx(s), c = -fmaf(16.f, s, b) * i;
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 v = __half22float2(as_half2(xs[u]));
        uint32_t n[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float z = fminf(fmaxf(e ? v.y : v.x, -kQuantLimit), kQuantLimit);
            const float below = floorf(fminf(fmaxf(fmaf(z, i, c), -1.f), 15.f));  // the lower of the two
            n[e] = (uint32_t)(z >= __fmaf_ru(below + 16.5f, s, b) ? fminf(below + 1.f, 15.f) : fmaxf(below, 0.f));
        }
        w[u] = n[0] | n[1] << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One head's K or V of the warp's eight tokens: x[j][f] are this lane's dims
// 32 j + 8 f + 2 t and the next of its token; w[j] becomes its word (t, j).
// Returns s | b << 16 of group t & (GR - 1) of the token.
//
// n = x i + c, one fused multiply-add with i = 1 / s and c = M + 1/2 - (16 s + b) i,
// M = 192, is the code in fixed point: floats in [128, 256) are 2^-16 apart, so
// that the code stands in the bits from 16 on and the distance to the border
// below it in the low 16.  i is within 2^-23 of itself, which scales the at most
// 16 steps from lo as a whole (2^-19); 16 s + b, c and n are rounded once each.
// With a = |16 + b / s| that makes 2^-24 a, 2^-17 + 2^-21.9 a and 2^-17, less
// than E = 3 + a / 16 units of 2^-16 together (a is at most 15 2^11, where lo is
// just below a power of two and hi a step of fp16 above: E is 1924 or less; the
// warp takes its groups' greatest).  A value whose low bits are E from a border
// or further has its code; elsewhere -- of normal values one in some 2600, 98 in
// a hundred of them ties, since x, s and b lie on coarse grids -- and where lo or
// hi come out beyond the codes, are beyond the limit or NaN, the border itself
// decides.
template <int GR>
__device__ __forceinline__ uint32_t quantise_rows(const uint32_t (&x)[GR][4], int t, uint32_t (&w)[GR])
{
    constexpr float kM = 192.f, kM5 = 192.5f;
    constexpr uint32_t kMCode = 0x43404340u;  // two upper halves of M
    uint32_t mm[4];  // least | -greatest of the lane's eight values of group j (twice over for GR = 2)
#pragma unroll
    for (int j = 0; j < GR; ++j) {
        const __half2 a = as_half2(x[j][0]), b = as_half2(x[j][1]), c = as_half2(x[j][2]), d = as_half2(x[j][3]);
        const uint32_t mn = as_word(__hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d)));
        const uint32_t mx = as_word(__hneg2(__hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d))));
        mm[j] = as_word(__hmin2_nan(as_half2(__byte_perm(mn, mx, 0x5410)), as_half2(__byte_perm(mn, mx, 0x7632))));
        if (GR == 2)
            mm[j + 2] = mm[j];
    }
    // lane t ends with group t & (GR - 1) of its token
    const bool up = (t & 2) != 0, odd = (t & 1) != 0;
    auto least = [](uint32_t a, uint32_t b) { return as_word(__hmin2_nan(as_half2(a), as_half2(b))); };
    const uint32_t k0 = least(up ? mm[2] : mm[0], __shfl_xor_sync(0xffffffffu, up ? mm[0] : mm[2], 2));
    const uint32_t k1 = least(up ? mm[3] : mm[1], __shfl_xor_sync(0xffffffffu, up ? mm[1] : mm[3], 2));
    const uint32_t m = least(odd ? k1 : k0, __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1));
    const float lo0 = __low2float(as_half2(m)), hi0 = -__high2float(as_half2(m));
    const float lo = fminf(fmaxf(lo0, -kQuantLimit), kQuantLimit), hi = fminf(fmaxf(hi0, -kQuantLimit), kQuantLimit);
    const bool nan = lo0 != lo0 || hi0 != hi0;
    __half s, b;
    quant_params(lo, hi, s, b);
    const uint32_t mine = nan ? 0x7fff7fffu : as_word(s, b);
    const float sf = __half2float(s);
    const float i_mine = sf > 0.f ? rcp_approx(sf) : 0.f;  // s = 0: every code is 0
    float c_mine = fmaf(-fmaf(16.f, sf, __half2float(b)), i_mine, kM5);
    const uint32_t E = __reduce_max_sync(0xffffffffu, min((uint32_t)fmaf(fabsf(c_mine - kM5), 0.0625f, 4.f), 0x3fffu));
    const uint32_t EE = E * 0x10001u;  // one for the warp
    // a NaN's low bits are ones: next to a border
    if (lo != lo0 || hi != hi0 || fmaf(lo, i_mine, c_mine) < kM || fmaf(hi, i_mine, c_mine) >= kM + 16.f)
        c_mine = __uint_as_float(0x7fffffffu);
    const int base = threadIdx.x & 28;
#pragma unroll
    for (int j = 0; j < GR; ++j) {
        const float i = __shfl_sync(0xffffffffu, i_mine, base + j), c = __shfl_sync(0xffffffffu, c_mine, base + j);
        uint32_t nearest = 0x7fff7fffu;  // the least low bits, E further on, of either half
        uint32_t code[4];                // pairs of codes, one per field, beside M
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 v = __half22float2(as_half2(x[j][u]));
            const uint32_t n0 = __float_as_uint(fmaf(v.x, i, c)), n1 = __float_as_uint(fmaf(v.y, i, c));
            code[u] = __byte_perm(n0, n1, 0x7632);
            nearest = __viaddmin_u16x2(__byte_perm(n0, n1, 0x5410), EE, nearest);
        }
        w[j] = (code[0] << 6) + (code[1] << 2) + (code[2] << 10) - ((kMCode << 6) + (kMCode << 2) + (kMCode << 10)) +
               __byte_perm((code[3] << 6) & 0x03c003c0u, 0, 0x2301);
        const bool near = (~((nearest | 0x80008000u) - 2 * EE) & 0x80008000u) != 0;  // one of them below 2 E
        if (__any_sync(0xffffffffu, near)) {
            const __half2 sb = as_half2(__shfl_sync(0xffffffffu, mine, base + j));
            if (near) {
                const uint4 e = quant_codes_exact(make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]), __low2float(sb), __high2float(sb));
                w[j] = (e.x << 6) + (e.y << 2) + (e.z << 10) + __byte_perm(e.w << 6, 0, 0x2301);
            }
        }
    }
    return mine;
}

// V of one token alone, by its quad: the halves it owns in words it shares with
// its neighbour (token 2 t2 + e of the eight from r & ~7 of block hb).
template <int D>
__device__ __forceinline__ void store_v_token(uint8_t *hb, int tb, int r, int t, int t2, int e,
                                              const uint32_t (&w)[QuantLayout<D>::GR], uint32_t si)
{
    using Q = QuantLayout<D>;
    constexpr int GR = Q::GR;
    uint16_t *c16 = reinterpret_cast<uint16_t *>(hb + Q::v_codes(tb) + (r >> 3) * Q::kVGroup);
    uint16_t *p16 = reinterpret_cast<uint16_t *>(hb + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup);
#pragma unroll
    for (int j = 0; j < GR; ++j) {
        c16[((2 * t * 4 + t2) * GR + j) * 2 + e] = (uint16_t)w[j];
        c16[(((2 * t + 1) * 4 + t2) * GR + j) * 2 + e] = (uint16_t)(w[j] >> 16);
    }
    if (t < GR) {
        p16[(t2 * GR + t) * 4 + e] = (uint16_t)si;
        p16[(t2 * GR + t) * 4 + 2 + e] = (uint16_t)(si >> 16);
    }
}

// One new token per row: a CTA per row, which alone reads and advances its
// length; warp 0 takes K and warp 1 V, eight heads at a time, a quad each.  The
// values do not depend on the length, so the three loads a token's place hangs
// on (length, table entry) run beside theirs.
template <int D>
__global__ void __launch_bounds__(64) quant_append_one_kernel(const QuantAppendParams p)
{
    using Q = QuantLayout<D>;
    constexpr int GR = Q::GR;
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, side = threadIdx.x >> 5;
    const __half *from = (side ? p.v_new : p.k_new) + (int64_t)i * p.new_stride + 2 * t;
    const int N = p.seq_lens[i];
    int page = -1;
    if (N < 0 || N >= p.len_cap) {
        if (threadIdx.x == 0)
            report_error(p.ws, N < 0 ? kErrNegLen : kErrTooLong, i, N < 0 ? N : N + 1, N < 0 ? 0 : p.len_cap);
    } else {
        page = p.bt[(int64_t)i * p.bt_stride + (N >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0)
                report_error(p.ws, kErrBadPage, i, N >> p.log2P, page);
            page = -1;
        }
    }
    const int tb = 1 << p.tb_log2, slot = N & ((1 << p.log2P) - 1), r = slot & (tb - 1), t2 = (r & 7) >> 1, e = r & 1;
    uint8_t *blk = p.cache + (int64_t)max(page, 0) * p.Hkv * p.page_head_bytes + (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
    for (int h0 = 0; h0 < p.Hkv; h0 += 8) {
        const int h = h0 + g;
        uint32_t x[GR][4];
#pragma unroll
        for (int j = 0; j < GR; ++j)
#pragma unroll
            for (int f = 0; f < 4; ++f)
                x[j][f] = h < p.Hkv ? *reinterpret_cast<const uint32_t *>(from + h * D + 32 * j + 8 * f) : 0u;
        uint32_t w[GR];
        const uint32_t si = quantise_rows<GR>(x, t, w);
        const int j = (lane & 28) + ((2 * t) & (GR - 1));
        const uint32_t a = __shfl_sync(0xffffffffu, si, j), c = __shfl_sync(0xffffffffu, si, j + 1);
        if (page < 0 || h >= p.Hkv)
            continue;
        uint8_t *hb = blk + h * p.page_head_bytes;
        if (side == 0) {
            store_words<GR>(hb + r * Q::kRow + t * GR * 4, w);
            if (t < GR)
                reinterpret_cast<uint32_t *>(hb + Q::k_params(tb) + r * Q::kParamRow)[t] = __byte_perm(a, c, 2 * t < GR ? 0x5410 : 0x7632);
        } else {
            store_v_token<D>(hb, tb, r, t, t2, e, w, si);
        }
    }
    __syncthreads();  // every thread has read N before it changes
    if (threadIdx.x == 0)
        p.seq_lens_out[i] = page >= 0 ? N + 1 : N;
}

// A warp takes a group (append_map.cuh: eight cache positions of one row) for
// some of the heads' sides (2 h: K, 2 h + 1: V), then the next such unit a grid
// further on.
template <int D>
__global__ void __launch_bounds__(kThreads, kAppendCtas) quant_append_kernel(const QuantAppendParams p)
{
    using Q = QuantLayout<D>;
    constexpr int GR = Q::GR;
    constexpr int kPitch = 2 * D + 16;  // bytes between tokens of a tile: the quads' words are in 32 banks
    __shared__ int s_seen;
    __shared__ __align__(16) uint8_t s_tile[kWarps][2][8 * kPitch];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int e = g & 1, t2 = g >> 1;
    uint8_t *tile = s_tile[threadIdx.x >> 5][0];
    const int tb = 1 << p.tb_log2;
    // what the last CTA needs of its first rows, on its way already
    int my_off = 0, my_n = 0, my_N = 0;
    if ((int)threadIdx.x < p.B) {
        my_off = p.offsets[threadIdx.x];
        my_n = p.offsets[threadIdx.x + 1] - my_off;
        my_N = p.seq_lens[threadIdx.x];
    }
    bool bad = false;
    // a warp keeps its part of the heads' sides (those left over when the parts do not divide the warps stay idle)
    const unsigned warp = blockIdx.x * kWarps + (threadIdx.x >> 5), lines = gridDim.x * kWarps / (unsigned)p.parts;
    const unsigned line = warp / (unsigned)p.parts;
    const int it0 = (int)(warp - line * p.parts) * p.its_per_part, it1 = min(it0 + p.its_per_part, 2 * p.Hkv);
    for (int64_t gs = line < lines ? (int64_t)line : p.groups; gs < p.groups; gs += lines) {
        const int i = min(last_not_above(p.B, gs, [&](int r) { return append_first_group(p.offsets[r], r); }), p.B - 1);
        const int off = p.offsets[i], n = p.offsets[i + 1] - off;
        const int N = p.seq_lens[i];
        int64_t pos0;
        if (!append_group(gs, i, off, n, N, pos0) || !append_fits(p, i, N, off, n, false))
            continue;
        const int page = p.bt[(int64_t)i * p.bt_stride + (pos0 >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0)
                report_error(p.ws, kErrBadPage, i, (int)(pos0 >> p.log2P), page);
            bad = true;
            continue;
        }
        const int slot = (int)pos0 & ((1 << p.log2P) - 1), r = slot & (tb - 1);
        uint8_t *blk = p.cache + (int64_t)page * p.Hkv * p.page_head_bytes + (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
        const int pos = (int)pos0 + g;
        const bool live = pos >= N && pos < N + n;
        const unsigned lives = __ballot_sync(0xffffffffu, live);
        const bool pair = live && (lives >> (lane ^ 4) & 1);  // its neighbour in the V words is new too
        // where there is no new token, the nearest one's values are read and nothing is stored
        constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // of a token, tokens at a time
        int tok[8 / kRows];
#pragma unroll
        for (int r0 = 0; r0 < 8; r0 += kRows)
            tok[r0 / kRows] = append_token((int)pos0 + r0 + lane / kLanes, off, n, N);
        auto fetch = [&](int it) {
            const __half *from = (it & 1 ? p.v_new : p.k_new) + (it >> 1) * D + 8 * (lane % kLanes);
            const uint32_t to = smem_u32(tile + (it & 1) * 8 * kPitch + 16 * (lane % kLanes));
#pragma unroll
            for (int r0 = 0; r0 < 8; r0 += kRows) {
                copy16_async(to + (r0 + lane / kLanes) * kPitch, from + tok[r0 / kRows] * p.new_stride);
            }
            copies_commit();
        };
        __syncwarp();
        fetch(it0);
        // K and V of a head in turn
#pragma unroll 1
        for (int it = it0; it < it1; ++it) {
            if (it + 1 < it1) {
                fetch(it + 1);
                copies_wait<1>();
            } else {
                copies_wait<0>();
            }
            __syncwarp();
            uint32_t x[GR][4];
            const uint8_t *from = tile + (it & 1) * 8 * kPitch + g * kPitch + 4 * t;
            uint8_t *hb = blk + (it >> 1) * p.page_head_bytes;
#pragma unroll
            for (int j = 0; j < GR; ++j)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    x[j][f] = *reinterpret_cast<const uint32_t *>(from + 64 * j + 16 * f);
            __syncwarp();  // the tile may be filled again
            uint32_t w[GR];
            const uint32_t si = quantise_rows<GR>(x, t, w);  // s | b of group t & (GR - 1)
            if (!(it & 1)) {
                // s of the groups, then b: lane t writes two of the 2 GR halves
                const int j = (lane & 28) + ((2 * t) & (GR - 1));
                const uint32_t a = __shfl_sync(0xffffffffu, si, j), c = __shfl_sync(0xffffffffu, si, j + 1);
                if (live) {
                    store_words<GR>(hb + (r + g) * Q::kRow + t * GR * 4, w);
                    if (t < GR)
                        reinterpret_cast<uint32_t *>(hb + Q::k_params(tb) + (r + g) * Q::kParamRow)[t] =
                            __byte_perm(a, c, 2 * t < GR ? 0x5410 : 0x7632);
                }
                continue;
            }
            // this lane holds the halves g' = 2 t (low) and 2 t + 1 of its token; with the neighbouring token's it
            // makes the words g' = 2 t + e whole
            const uint32_t pick = e ? 0x3276 : 0x5410;
            uint32_t o[GR];
#pragma unroll
            for (int j = 0; j < GR; ++j) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 4);
                o[j] = __byte_perm(w[j], other, pick);
            }
            const uint32_t so = __shfl_xor_sync(0xffffffffu, si, 4);
            uint8_t *vc = hb + Q::v_codes(tb) + (r >> 3) * Q::kVGroup, *vp = hb + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup;
            if (pair) {
                store_words<GR>(vc + ((2 * t + e) * 4 + t2) * GR * 4, o);
                if (t < GR)
                    reinterpret_cast<uint32_t *>(vp)[(t2 * GR + t) * 2 + e] = __byte_perm(si, so, pick);
            } else if (live) {
                store_v_token<D>(hb, tb, r, t, t2, e, w, si);
            }
        }
    }
    append_finish<kThreads>(p, bad, my_off, my_n, my_N, &s_seen);
}

// A warp takes eight packed tokens, one per quad, and heads [h0, h0 + nh).  A
// token's V halves are gathered to the words its K row has: the halves g' = 2 t
// and 2 t + 1 of its words become lane t's word (t, j).
template <int D>
__global__ void __launch_bounds__(kThreads, 4) quant_read_kernel(const QuantReadParams p)
{
    using Q = QuantLayout<D>;
    constexpr int GR = Q::GR;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t chunk = unit / p.parts;
    const int h0 = (int)(unit - chunk * p.parts) * p.heads_per_part, h1 = min(h0 + p.heads_per_part, p.Hkv);
    if (chunk * 8 >= p.T)
        return;
    const int x = (int)min(chunk * 8 + g, (int64_t)0x7fffffff);
    bool live = x < p.T && x >= p.offsets[0] && x < p.offsets[p.B];  // in some row's span
    int page = -1;
    int64_t pos = 0;
    if (live) {
        const int i = row_of(p.offsets, p.B, x);
        const int N = min(p.seq_lens[i], p.len_cap);
        pos = (int64_t)(p.first ? p.first[i] : 0) + (x - p.offsets[i]);
        if (x >= p.offsets[i + 1]) {
            live = false;  // offsets that do not ascend
        } else if (pos < 0 || pos >= N) {
            if (t == 0)
                report_error(p.ws, kErrTooLong, i, (int)min(max(pos + 1, (int64_t)-0x7fffffff), (int64_t)0x7fffffff), N);
        } else {
            page = p.bt[(int64_t)i * p.bt_stride + (pos >> p.log2P)];
            if (page < 0 || page >= p.num_pages) {
                if (t == 0)
                    report_error(p.ws, kErrBadPage, i, (int)(pos >> p.log2P), page);
                page = -1;
            }
        }
    }
    const int tb = 1 << p.tb_log2, slot = (int)pos & ((1 << p.log2P) - 1), r = slot & (tb - 1), t2 = (r & 7) >> 1, e = r & 1;
    const bool there = page >= 0;
    const uint8_t *blk = p.cache + (int64_t)(there ? page : 0) * p.Hkv * p.page_head_bytes +
                         (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
    const int64_t dst = (int64_t)x * p.out_stride + 8 * t;
    for (int h = h0; h < h1; ++h) {
        const uint8_t *hb = blk + h * p.page_head_bytes;
        uint32_t k[GR], kp[GR], v0[GR], v1[GR], vp[2 * GR];
#pragma unroll
        for (int j = 0; j < GR; ++j)
            k[j] = kp[j] = v0[j] = v1[j] = vp[j] = vp[GR + j] = 0;
        if (there) {
            load_words<GR>(hb + r * Q::kRow + t * GR * 4, k);
            load_words<GR>(hb + Q::k_params(tb) + r * Q::kParamRow, kp);
            const uint8_t *vc = hb + Q::v_codes(tb) + (r >> 3) * Q::kVGroup;
            load_words<GR>(vc + (2 * t * 4 + t2) * GR * 4, v0);
            load_words<GR>(vc + ((2 * t + 1) * 4 + t2) * GR * 4, v1);
            const uint8_t *q = hb + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup + t2 * GR * 8;
#pragma unroll
            for (int j = 0; j < GR; j += 2) {
                const uint4 a = *reinterpret_cast<const uint4 *>(q + j * 8);
                vp[2 * j] = a.x, vp[2 * j + 1] = a.y, vp[2 * j + 2] = a.z, vp[2 * j + 3] = a.w;
            }
        }
        auto give = [&](__half *out, uint32_t w, uint32_t s2, uint32_t b2, int j) {
            const __half2 s = as_half2(s2), b = as_half2(b2);
            const uint32_t v[4] = {quant_value(quant_field<0>(w), s, b), quant_value(quant_field<1>(w), s, b),
                                   quant_value(quant_field<2>(w), s, b), quant_value(quant_field<3>(w), s, b)};
            const uint4 y = quad_transpose(v, t);
            if (live)
                *reinterpret_cast<uint4 *>(out + dst + h * D + 32 * j) = y;
        };
#pragma unroll
        for (int j = 0; j < GR; ++j)
            give(p.k_out, k[j], __byte_perm(kp[j >> 1], 0, j & 1 ? 0x3232 : 0x1010),
                 __byte_perm(kp[(GR + j) >> 1], 0, j & 1 ? 0x3232 : 0x1010), j);
        const uint32_t pick = e ? 0x7632 : 0x5410, both = e ? 0x3232 : 0x1010;
#pragma unroll
        for (int j = 0; j < GR; ++j)
            give(p.v_out, __byte_perm(v0[j], v1[j], pick), __byte_perm(vp[2 * j], 0, both), __byte_perm(vp[2 * j + 1], 0, both), j);
    }
}

template <class K, class P>
cudaError_t launch(K kern, const P &p, int64_t grid, int threads, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid > 0 ? grid : 1));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_quant_append(int d, QuantAppendParams p, int sms, cudaStream_t s)
{
    if (!p.offsets)
        return d == 128 ? launch(quant_append_one_kernel<128>, p, p.B, 64, s) : launch(quant_append_one_kernel<64>, p, p.B, 64, s);
    const int64_t grid = append_grid(p.T, p.B, p.Hkv, kAppendCtas * sms, kWarps, p.groups, p.parts, p.its_per_part);
    return d == 128 ? launch(quant_append_kernel<128>, p, grid, kThreads, s) : launch(quant_append_kernel<64>, p, grid, kThreads, s);
}

cudaError_t launch_quant_read(int d, QuantReadParams p, int sms, cudaStream_t s)
{
    const int64_t chunks = ((int64_t)p.T + 7) / 8;
    // several waves of warps, each with two heads or more unless the launch is a
    // single wave: of eight heads, two per warp 39 us (42k tokens) and 99 us
    // (117k), one 42 and 111 us, four 41 and 101 us, all eight 49 and 106 us
    const int64_t wave = 32 * (int64_t)sms;
    p.parts = split_work(chunks, p.Hkv, 8 * wave, INT64_MAX, p.heads_per_part);
    if (p.heads_per_part == 1 && p.Hkv > 1 && chunks * p.parts > 2 * wave) {
        p.heads_per_part = 2;
        p.parts = (p.Hkv + 1) / 2;
    }
    const int64_t grid = (chunks * p.parts + kWarps - 1) / kWarps;
    return d == 128 ? launch(quant_read_kernel<128>, p, grid, kThreads, s) : launch(quant_read_kernel<64>, p, grid, kThreads, s);
}

}  // namespace pkv
