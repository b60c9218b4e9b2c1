// byte.cu -- writing the 8-bit KV cache and reading it back.
//
// append: K and V of new tokens, packed [T][Hkv][d] fp16 with a stride between
// tokens, become codes in the pages their rows' block tables name, at positions
// seq_lens[i] .. ; lengths advance once every CTA has read them.
// read: tokens of the cache become packed fp16 K and V again.
//
// Both are one pass over their data: append reads 2 bytes per value and writes
// one, read the other way round.  35k tokens of 8 heads, d = 128, appended (213 MB,
// 31 us at the copy rate) and read back at once take 73 us; 117k tokens read, 718
// MB, 109 us, 0.97 of the copy rate; a token of each of 64 rows and its block 7.6 us.
//
// A warp takes a scale block (16 tokens, 8 in pages of 8) of one head and side at
// a time: a lane holds 8 dims of 8 or 4 neighbouring tokens, so that the block's
// greatest magnitude is one reduction over the warp, a token's codes are 8 bytes
// of a K row, and four tokens' are two whole pieces of V after a transposition in
// registers.  Rows, pages and offsets are looked up once for all of a block's
// heads and sides; short calls split those over more warps.
#include "append_rows.cuh"
#include "byte_format.cuh"

#include <type_traits>

namespace pkv {
namespace {

constexpr int kWarps = kByteWarps, kThreads = 32 * kWarps;
constexpr int kOneThreads = 512;  // of the append of one token per row, at most
// CTAs per SM.  35k tokens of 8 heads appended and read back 73.4 us; with 2 CTAs of
// the append 78 us, 4 (spills) 81 us; the read of 117k tokens 108.6 us, with 3 CTAs
// 116 us, 5 (spills) 130 us.  Copies to shared memory ahead of use, or lines of
// neighbouring blocks with the next one's page looked up ahead, took longer: 84 and
// 82 us.
constexpr int kAppendCtas = 3, kReadCtas = 4;

// Which tokens and dims of a block of 2^LG tokens a lane holds: dims 8 piece ..,
// tokens first .. first + kTokens - 1 (none where `first` is beyond the block).
template <int D, int LG>
struct Lane {
    static constexpr int kPieces = D / 8, kGroups = 32 / kPieces;
    static constexpr int kTokens = (1 << LG) / kGroups < 4 ? 4 : (1 << LG) / kGroups;
    static constexpr int kAtOnce = 8 / kTokens;  // sides whose loads a lane may have on their way together
    const int piece, first;
    __device__ __forceinline__ Lane() : piece((threadIdx.x & 31) % kPieces), first((threadIdx.x & 31) / kPieces * kTokens) {}
    __device__ __forceinline__ bool any() const { return kTokens * kGroups == 1 << LG || first < 1 << LG; }
};

// The row that block gs is in: its first packed token, its tokens and what `a` and
// `b` (nullptr: zeros) hold of it.  Of up to kFewRows rows every lane brings two, so
// that all of it takes one round trip, and sees whether the offsets ascend within T;
// whole warps only.
constexpr int kFewRows = 64;
struct Row {
    int i, off, n, a, b;
    bool ascend;
};
template <int LG>
__device__ __forceinline__ Row find_row(int64_t gs, const int32_t *offsets, int B, int T, const int32_t *pa, const int32_t *pb)
{
    if (B > kFewRows) {
        const int i = min(last_not_above(B, gs, [&](int r) { return append_first_group(offsets[r], r, LG); }), B - 1);
        const int off = offsets[i];
        return {i, off, offsets[i + 1] - off, pa[i], pb ? pb[i] : 0, true};
    }
    const int lane = threadIdx.x & 31;
    int o[2], e[2], x[2], y[2];
    unsigned m[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = min(lane + 32 * u, B - 1);
        o[u] = offsets[r], e[u] = offsets[r + 1], x[u] = pa[r], y[u] = pb ? pb[r] : 0;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
        m[u] = __ballot_sync(0xffffffffu, lane + 32 * u < B && append_first_group(o[u], lane + 32 * u, LG) <= gs);
    const int i = max(__popc(m[0]) + __popc(m[1]) - 1, 0);
    auto of = [&](const int (&v)[2]) { return __shfl_sync(0xffffffffu, i >= 32 ? v[1] : v[0], i & 31); };
    const int off = of(o);
    return {i, off, of(e) - off, of(x), of(y), __all_sync(0xffffffffu, min(o[0], o[1]) >= 0 && o[0] <= e[0] && o[1] <= e[1] && max(e[0], e[1]) <= T) != 0};
}

__device__ __forceinline__ uint32_t greatest(uint4 x)
{
    const __half2 a = __hmax2_nan(__hmax2_nan(__habs2(byte_half2(x.x)), __habs2(byte_half2(x.y))),
                                  __hmax2_nan(__habs2(byte_half2(x.z)), __habs2(byte_half2(x.w))));
    return max((uint32_t)__half_as_ushort(__low2half(a)), (uint32_t)__half_as_ushort(__high2half(a)));
}

constexpr uint32_t kInf = 0x7c00u;
constexpr uint32_t kNanBits = 0x7fffffffu;

// A block's scale after tokens with the greatest magnitude `top` have joined
// those it holds under the scale `was` (any: whether it holds some).
template <int FMT>
struct NewScale {
    int e, grow;  // grow: how far the earlier codes have to be shifted, 0 for not at all
    float s;
    __device__ __forceinline__ NewScale(uint32_t top, bool any, float was)
    {
        e = byte_least_exponent<FMT>(top > kInf ? kInf : top);
        grow = 0;
        const bool nan = top > kInf || (any && was != was);
        if (any) {
            const int e0 = byte_exponent<FMT>(was);
            if (e > e0 && !nan)
                grow = e - e0;
            e = max(e, e0);
        }
        s = nan ? __uint_as_float(kNanBits) : byte_pow2(e);
    }
};

// One head's side of a scale block: positions `first` .. of this lane's tokens x of
// a row whose N cached tokens n new ones follow (zeros where there is no new one).
// hb: the head's block in its page; r0: the scale block's first token there.
// WHOLE: all of the block's tokens are new.
template <int D, int FMT, int LG, bool WHOLE>
__device__ __forceinline__ void store_side(const Lane<D, LG> &ln, uint8_t *hb, int tb, int r0, bool v,
                                           const uint4 (&x)[Lane<D, LG>::kTokens], int first, int N, int n)
{
    constexpr int TL = Lane<D, LG>::kTokens;
    const bool held = !WHOLE && first - ln.first < N;
    float *scale = reinterpret_cast<float *>(hb + byte_scale_part<D>(tb, r0, LG)) + v;
    const float was = held ? *scale : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < TL; ++u)
        top = max(top, greatest(x[u]));
    top = __reduce_max_sync(0xffffffffu, top);
    const NewScale<FMT> ns(top, held, was);
    const ByteQuantiser<FMT> code(ns.e, top);
    if (ln.any() && !v) {
#pragma unroll
        for (int u = 0; u < TL; ++u) {
            const int pos = first + u;
            uint2 *to = reinterpret_cast<uint2 *>(hb + byte_k_at<D>(r0 + ln.first + u, 8 * ln.piece));
            if (WHOLE || (pos >= N && pos < N + n)) {
                *to = make_uint2(code(x[u].x, x[u].y), code(x[u].z, x[u].w));
            } else if (pos < N && ns.grow) {
                const uint2 c = *to;
                *to = make_uint2(byte_shift<FMT>(c.x, -ns.grow), byte_shift<FMT>(c.y, -ns.grow));
            }
        }
    } else if (ln.any()) {
        uint8_t *part = hb + byte_v_part<D>(tb, r0, LG);
#pragma unroll
        for (int q = 0; q < TL; q += 4) {
            const int pos = first + q;
            if (!WHOLE && (pos >= N + n || (pos + 4 <= N && !ns.grow)))
                continue;
            uint4 lo = byte_transpose(code(x[q].x, x[q].y), code(x[q + 1].x, x[q + 1].y), code(x[q + 2].x, x[q + 2].y),
                                      code(x[q + 3].x, x[q + 3].y));
            uint4 hi = byte_transpose(code(x[q].z, x[q].w), code(x[q + 1].z, x[q + 1].w), code(x[q + 2].z, x[q + 2].w),
                                      code(x[q + 3].z, x[q + 3].w));
            uint4 *to = reinterpret_cast<uint4 *>(part + byte_v_at(2 * ln.piece, (ln.first + q) >> 2, LG));
            uint4 *to2 = reinterpret_cast<uint4 *>(part + byte_v_at(2 * ln.piece + 1, (ln.first + q) >> 2, LG));
            if (!WHOLE && pos < N) {  // earlier tokens' bytes stay
                const uint32_t keep = pos + 4 <= N ? 0xffffffffu : 0xffffffffu >> (8 * (pos + 4 - N));
                auto join = [&](uint32_t now, uint32_t old) {
                    if (ns.grow)
                        old = byte_shift<FMT>(old, -ns.grow);
                    return (old & keep) | (now & ~keep);
                };
                const uint4 a = *to, b = *to2;
                lo = make_uint4(join(lo.x, a.x), join(lo.y, a.y), join(lo.z, a.z), join(lo.w, a.w));
                hi = make_uint4(join(hi.x, b.x), join(hi.y, b.y), join(hi.z, b.z), join(hi.w, b.w));
            }
            *to = lo;
            *to2 = hi;
        }
    }
    __syncwarp();  // every lane has read the scale
    if ((threadIdx.x & 31) == 0)
        *scale = ns.s;
}

// A group's scale block: found, fitting, and its page; `bad` where its id is out of range.
struct Block {
    int64_t pos0;
    int off, n, N, page, r0;
    bool any, bad;
};
// A block that holds earlier tokens is touched only where its row and the call
// stand, since their codes change with its scale: those of a refused row stay.  So
// the warps that have one look at all of the row's pages, a lane each, in the round
// trip of the block's own.  `ascend`: the offsets of more than kFewRows rows are in
// order, else the whole call is refused.  (64 rows of one token 5.00 us without, 5.17
// with; 256 of four 10.8 and 11.3; 1000 of one 24.8 and 25.7; 37k in 8 prompts 31.2 and 31.6.)
template <int LG>
__device__ __forceinline__ Block find_block(const QuantAppendParams &p, int64_t gs, bool ascend)
{
    Block b = {};
    const Row row = find_row<LG>(gs, p.offsets, p.B, p.T, p.seq_lens, nullptr);
    b.off = row.off, b.n = row.n, b.N = row.a;
    if (!append_group(gs, row.i, b.off, b.n, b.N, b.pos0, LG) || !append_fits(p, row.i, b.N, b.off, b.n, false))
        return b;
    const int32_t *pages = p.bt + (int64_t)row.i * p.bt_stride;
    const int lane = threadIdx.x & 31, at = (int)(b.pos0 >> p.log2P), last = (int)(((int64_t)b.N + b.n - 1) >> p.log2P);
    const bool held = b.pos0 < b.N;
    auto there = [&p](int page) { return page >= 0 && page < p.num_pages; };
    const int mine = pages[held ? min(at + lane, last) : at];
    b.page = __shfl_sync(0xffffffffu, mine, 0);
    bool stands = there(mine);
    if (held) {
        for (int x = at + 32; x <= last; x += 32)
            stands &= there(pages[min(x + lane, last)]);
        stands = __all_sync(0xffffffffu, stands) && ascend && row.ascend;
    }
    b.any = stands;
    b.bad = !there(b.page);
    if (b.bad && lane == 0)
        report_error(p.ws, kErrBadPage, row.i, at, b.page);
    b.r0 = (int)b.pos0 & ((1 << p.log2P) - 1);  // within the page
    return b;
}
template <int D>
__device__ __forceinline__ uint8_t *block_of(const QuantAppendParams &p, int page, int slot)
{
    return p.cache + (int64_t)page * p.Hkv * p.page_head_bytes + (int64_t)(slot >> p.tb_log2) * byte_block_bytes(1 << p.tb_log2, D);
}

// A scale block for some of the heads' sides (2 h: K, 2 h + 1: V), AT of them at
// once, then the next such unit a grid further on.
template <int D, int FMT, int LG, int AT>
__global__ void __launch_bounds__(kThreads, kAppendCtas) byte_append_kernel(const QuantAppendParams p)
{
    using Ln = Lane<D, LG>;
    constexpr int TL = Ln::kTokens;
    __shared__ int s_seen;
    pdl_wait();
    pdl_trigger();
    const Ln ln;
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
    bool ascend = true;
    if (p.B > kFewRows) {  // else every find_row() sees them all
        ascend = p.offsets[0] >= 0 && p.offsets[p.B] <= p.T && my_n >= 0;
        for (int r = (int)threadIdx.x + kThreads; r < p.B; r += kThreads)
            ascend &= p.offsets[r] <= p.offsets[r + 1];
        ascend = __syncthreads_and(ascend) != 0;
    }
    for (int64_t gs = line < lines ? (int64_t)line : p.groups; gs < p.groups; gs += lines) {
        const Block b = find_block<LG>(p, gs, ascend);
        bad |= b.bad;
        if (!b.any)
            continue;
        uint8_t *blk = block_of<D>(p, b.page, b.r0);
        const int first = (int)b.pos0 + ln.first;  // of this lane's positions; the row's end is an int
        const int64_t from = (int64_t)b.off * p.new_stride + 8 * ln.piece;
        // Blocks of new tokens alone go without the tests of each token: 64 x 1000
        // tokens of 8 heads, d = 64, in 37.6 us against 42.0; of d = 128, whose lanes hold
        // twice the tokens, no gain (67.0 and 66.8 us), and registers spill.
        const bool whole = TL == 4 && b.pos0 >= b.N && b.pos0 + (1 << LG) <= (int64_t)b.N + b.n;
        auto sides = [&](auto all) {
            constexpr bool WHOLE = decltype(all)::value;
            for (int it2 = it0; it2 < it1; it2 += AT) {
                uint4 x[AT][TL];
#pragma unroll
                for (int e = 0; e < AT; ++e)
#pragma unroll
                    for (int u = 0; u < TL; ++u) {
                        const int it = it2 + e, pos = first + u;
                        x[e][u] = make_uint4(0, 0, 0, 0);
                        if (ln.any() && it < it1 && (WHOLE || (pos >= b.N && pos < b.N + b.n)))
                            x[e][u] = *reinterpret_cast<const uint4 *>((it & 1 ? p.v_new : p.k_new) + from +
                                                                       (int64_t)(pos - b.N) * p.new_stride + (it >> 1) * D);
                    }
#pragma unroll
                for (int e = 0; e < AT; ++e) {
                    const int it = it2 + e;
                    if (it < it1)
                        store_side<D, FMT, LG, WHOLE>(ln, blk + (it >> 1) * p.page_head_bytes, tb, b.r0 & (tb - 1), it & 1, x[e], first,
                                                      b.N, b.n);
                }
            }
        };
        if (whole)
            sides(std::bool_constant<TL == 4>());
        else
            sides(std::false_type());
    }
    append_finish<kThreads>(p, bad, my_off, my_n, my_N, &s_seen);
}

// One new token per row: a CTA per row, which alone reads and advances its
// length; a warp (d = 64: half a warp) takes a head's side, a lane four dims.
template <int D, int FMT, int LG>
__global__ void __launch_bounds__(kOneThreads) byte_append_one_kernel(const QuantAppendParams p)
{
    constexpr int kLanes = D / 4, kPer = 32 / kLanes;  // of a head's side, and sides per warp
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x, l = (threadIdx.x & 31) % kLanes;
    const int at = (int)threadIdx.x / kLanes, step = (int)blockDim.x / kLanes;
    // the first side's values do not depend on the three loads a token's place hangs on
    auto load = [&](int side) {
        return side < 2 * p.Hkv ? *reinterpret_cast<const uint2 *>((side & 1 ? p.v_new : p.k_new) + (int64_t)i * p.new_stride +
                                                                   (side >> 1) * D + 4 * l)
                                : make_uint2(0, 0);
    };
    uint2 x = load(at);
    const int N = p.seq_lens[i];
    int page = -1;
    if (N < 0 || N >= p.len_cap) {
        if (threadIdx.x == 0)
            report_error(p.ws, N < 0 ? kErrNegLen : kErrTooLong, i, N < 0 ? N : (int)min((int64_t)N + 1, (int64_t)0x7fffffff),
                         N < 0 ? 0 : p.len_cap);
    } else {
        page = p.bt[(int64_t)i * p.bt_stride + (N >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0)
                report_error(p.ws, kErrBadPage, i, N >> p.log2P, page);
            page = -1;
        }
    }
    const int tb = 1 << p.tb_log2, slot = N & ((1 << p.log2P) - 1), r = slot & (tb - 1), u = r & ((1 << LG) - 1);
    uint8_t *blk = p.cache + (int64_t)max(page, 0) * p.Hkv * p.page_head_bytes + (int64_t)(slot >> p.tb_log2) * byte_block_bytes(tb, D);
    for (int it = at - at % kPer; it < 2 * p.Hkv && page >= 0; it += step) {
        const int mine = it + at % kPer, h = mine >> 1;
        const bool there = mine < 2 * p.Hkv, v = mine & 1;
        uint8_t *hb = blk + (int64_t)(there ? h : 0) * p.page_head_bytes;
        float *scale = reinterpret_cast<float *>(hb + byte_scale_part<D>(tb, r, LG)) + v;
        if (it >= step)
            x = load(mine);
        const float was = there && u > 0 ? *scale : 0.f;
        uint32_t top = greatest(make_uint4(x.x, x.y, 0, 0));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const NewScale<FMT> ns(top, u > 0, was);
        const uint32_t c = ByteQuantiser<FMT>(ns.e, top)(x.x, x.y);
        __syncwarp();  // every lane has read the scale
        if (!there)
            continue;
        if (!v) {
            if (ns.grow)
                for (int o = r - u; o < r; ++o) {
                    uint32_t *to = reinterpret_cast<uint32_t *>(hb + byte_k_at<D>(o, 4 * l));
                    *to = byte_shift<FMT>(*to, -ns.grow);
                }
            *reinterpret_cast<uint32_t *>(hb + byte_k_at<D>(r, 4 * l)) = c;
        } else {
            uint8_t *part = hb + byte_v_part<D>(tb, r, LG);
            if (ns.grow)
                for (int t = 0; 4 * t < u; ++t) {
                    uint4 *to = reinterpret_cast<uint4 *>(part + byte_v_at(l, t, LG));
                    const uint4 w = *to;
                    *to = make_uint4(byte_shift<FMT>(w.x, -ns.grow), byte_shift<FMT>(w.y, -ns.grow), byte_shift<FMT>(w.z, -ns.grow),
                                     byte_shift<FMT>(w.w, -ns.grow));
                }
            uint8_t *to = part + byte_v_at(l, u >> 2, LG) + (u & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[4 * j] = (uint8_t)(c >> (8 * j));
        }
        if (l == 0)
            *scale = ns.s;
    }
    __syncthreads();  // every thread has read N before it changes
    if (threadIdx.x == 0)
        p.seq_lens_out[i] = page >= 0 ? N + 1 : N;
}

// A scale block of a row for some of the heads' sides, as the append takes them:
// its tokens among those that the row's span wants.
template <int D, int FMT, int LG>
__global__ void __launch_bounds__(kThreads, kReadCtas) byte_read_kernel(const QuantReadParams p)
{
    using Ln = Lane<D, LG>;
    constexpr int TL = Ln::kTokens;
    pdl_wait();
    pdl_trigger();
    const Ln ln;
    const int tb = 1 << p.tb_log2;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), gs = unit / p.parts;
    const int part_no = (int)(unit - gs * p.parts), it0 = part_no * p.heads_per_part, it1 = min(it0 + p.heads_per_part, 2 * p.Hkv);
    if (gs >= p.groups)
        return;
    const Row row = find_row<LG>(gs, p.offsets, p.B, p.T, p.seq_lens, p.first);
    const int i = row.i, off = row.off, n = row.n, begin = row.b;
    int64_t pos0;
    if (off < 0 || (int64_t)off + n > p.T || !append_group(gs, i, off, n, begin, pos0, LG))
        return;  // offsets that do not ascend within the buffer have no tokens here
    const int N = min(row.a, p.len_cap);
    const int64_t from = max(pos0, (int64_t)begin), to = min(pos0 + (1 << LG), (int64_t)begin + n);
    int page = -1;
    if (pos0 >= 0 && from < N) {
        page = p.bt[(int64_t)i * p.bt_stride + (pos0 >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            if (part_no == 0 && (threadIdx.x & 31) == 0)
                report_error(p.ws, kErrBadPage, i, (int)(pos0 >> p.log2P), page);
            page = -1;
        }
    }
    if ((from < 0 || to > N) && part_no == 0 && (threadIdx.x & 31) == 0)
        report_error(p.ws, kErrTooLong, i, (int)(from < 0 ? max(from + 1, (int64_t)-0x7fffffff) : min(to, (int64_t)0x7fffffff)), N);
    if (!ln.any())
        return;
    const int slot = (int)pos0 & ((1 << p.log2P) - 1), r0 = slot & (tb - 1);
    const uint8_t *blk = p.cache + (int64_t)max(page, 0) * p.Hkv * p.page_head_bytes + (int64_t)(slot >> p.tb_log2) * byte_block_bytes(tb, D);
    const int64_t mine = pos0 + ln.first;  // this lane's first position
    for (int it = it0; it < it1; ++it) {
        const int h = it >> 1;
        const bool v = it & 1;
        const uint8_t *hb = blk + h * p.page_head_bytes;
        __half *out = (v ? p.v_out : p.k_out) + h * D + 8 * ln.piece;
        uint2 c[TL];
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < TL; ++u)
            c[u] = make_uint2(0, 0);
        if (page >= 0) {
            s = reinterpret_cast<const float *>(hb + byte_scale_part<D>(tb, r0, LG))[v];
            if (!v) {
#pragma unroll
                for (int u = 0; u < TL; ++u)
                    c[u] = *reinterpret_cast<const uint2 *>(hb + byte_k_at<D>(r0 + ln.first + u, 8 * ln.piece));
            } else {
                const uint8_t *part = hb + byte_v_part<D>(tb, r0, LG);
#pragma unroll
                for (int q = 0; q < TL; q += 4) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(part + byte_v_at(2 * ln.piece, (ln.first + q) >> 2, LG));
                    const uint4 b = *reinterpret_cast<const uint4 *>(part + byte_v_at(2 * ln.piece + 1, (ln.first + q) >> 2, LG));
                    const uint4 lo = byte_transpose(a.x, a.y, a.z, a.w), hi = byte_transpose(b.x, b.y, b.z, b.w);
                    c[q] = make_uint2(lo.x, hi.x);
                    c[q + 1] = make_uint2(lo.y, hi.y);
                    c[q + 2] = make_uint2(lo.z, hi.z);
                    c[q + 3] = make_uint2(lo.w, hi.w);
                }
            }
        }
        // the scale is an fp16 number too, and so are the products
        const __half2 s2 = __float2half2_rn(s != s ? s : byte_pow2(byte_exponent<FMT>(s)));
        auto value = [&](uint32_t w, uint32_t &lo, uint32_t &hi) {
            byte_numbers<FMT>(w, lo, hi);
            lo = byte_word(__hmul2(byte_half2(lo), s2));
            hi = byte_word(__hmul2(byte_half2(hi), s2));
        };
#pragma unroll
        for (int u = 0; u < TL; ++u) {
            const int64_t pos = mine + u;
            if (pos < from || pos >= to)
                continue;
            uint4 y;
            value(c[u].x, y.x, y.y);
            value(c[u].y, y.z, y.w);
            if (pos >= N)
                y = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(out + (off + (pos - begin)) * p.out_stride) = y;
        }
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

template <int D, int FMT, int LG>
cudaError_t launch_append(QuantAppendParams p, int sms, cudaStream_t s)
{
    if (!p.offsets) {
        const int64_t threads = 32 * ((2 * (int64_t)p.Hkv * D + 127) / 128);
        return launch(byte_append_one_kernel<D, FMT, LG>, p, p.B, (int)(threads < kOneThreads ? threads : kOneThreads), s);
    }
    const int64_t grid = byte_append_grid(p.T, p.B, p.Hkv, LG, (int64_t)kAppendCtas * sms, kWarps, p.groups, p.parts, p.its_per_part);
    // 64k tokens of 32 heads of d = 64: two sides at once 132 us, one after the other 150 us
    constexpr int AT = Lane<D, LG>::kAtOnce;
    return p.its_per_part < AT ? launch(byte_append_kernel<D, FMT, LG, 1>, p, grid, kThreads, s)
                               : launch(byte_append_kernel<D, FMT, LG, AT>, p, grid, kThreads, s);
}

template <int D, int FMT, int LG>
cudaError_t launch_read(QuantReadParams p, int sms, cudaStream_t s)
{
    const int64_t grid = byte_read_grid(p.T, p.B, p.Hkv, LG, (int64_t)kReadCtas * sms, kWarps, p.groups, p.parts, p.heads_per_part);
    return launch(byte_read_kernel<D, FMT, LG>, p, grid, kThreads, s);
}

// f<D, FMT, LG>() for the call's d, format and page size.
template <class F>
cudaError_t pick(int d, int fmt, int log2P, F f)
{
    auto page = [&](auto D, auto FMT) { return log2P == 3 ? f(D, FMT, std::integral_constant<int, 3>()) : f(D, FMT, std::integral_constant<int, 4>()); };
    auto format = [&](auto D) { return fmt == kInt8 ? page(D, std::integral_constant<int, kInt8>()) : page(D, std::integral_constant<int, kE4m3>()); };
    return d == 128 ? format(std::integral_constant<int, 128>()) : format(std::integral_constant<int, 64>());
}

}  // namespace

cudaError_t launch_byte_append(int d, int fmt, const QuantAppendParams &p, int sms, cudaStream_t s)
{
    return pick(d, fmt, p.log2P, [&](auto D, auto FMT, auto LG) { return launch_append<D(), FMT(), LG()>(p, sms, s); });
}

cudaError_t launch_byte_read(int d, int fmt, const QuantReadParams &p, int sms, cudaStream_t s)
{
    return pick(d, fmt, p.log2P, [&](auto D, auto FMT, auto LG) { return launch_read<D(), FMT(), LG()>(p, sms, s); });
}

}  // namespace pkv
