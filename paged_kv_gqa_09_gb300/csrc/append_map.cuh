// append_map.cuh -- which packed tokens a warp of the 4-bit and 8-bit caches'
// appends takes.
//
// A warp takes 2^lg cache positions of one row, the first a multiple of that: a
// group.  Eight are whole words of V in the 4-bit cache, eight or sixteen a block
// of the 8-bit one.  The rows' groups lie on one line, row i's from
// (offsets[i] >> lg) + 2 i on, which leaves each room for a first and a last group
// that are not full and needs no sum over the rows before; what is left over is
// idle.  A row without new tokens has places on the line all the same, but no
// group there: its last page, partly filled as it may be, is not looked at.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// Row i's first group, its new tokens packed from `off` on.
__host__ __device__ inline int64_t append_first_group(int off, int i, int lg = 3) { return (int64_t)(off >> lg) + 2 * (int64_t)i; }

// Groups on the line of T packed tokens of B rows.
__host__ __device__ inline int64_t append_groups(int T, int B, int lg = 3) { return T > 0 ? ((int64_t)T >> lg) + 2 * (int64_t)B : 0; }

// Whether group gs holds any of row i's n new tokens, which follow its N cached
// ones; pos0: the group's first position.
__host__ __device__ inline bool append_group(int64_t gs, int i, int off, int n, int N, int64_t &pos0, int lg = 3)
{
    const int k = (int)(gs - append_first_group(off, i, lg));
    pos0 = ((int64_t)(N >> lg) + k) * (1 << lg);
    return n > 0 && k >= 0 && pos0 < (int64_t)N + n;
}

// The packed token of position pos, or the row's nearest new one where pos holds none (n > 0).
__host__ __device__ inline int append_token(int pos, int off, int n, int N)
{
    const int first = pos < N ? N : pos, last = N + n - 1;
    return off + ((first < last ? first : last) - N);
}

// `n` things to do per token group (heads, or sides of heads) are split over
// `parts` warps, `most` at most, until the launch has at least `want`; each warp
// then does `per`.
inline int split_work(int64_t warps, int n, int64_t want, int64_t most, int &per)
{
    int parts = 1;
    while (parts < n && warps * parts < want && 2 * (int64_t)parts <= most)
        parts *= 2;
    per = (n + parts - 1) / parts;
    return (n + per - 1) / per;
}

// CTAs of an append, of `ctas` resident ones of `cta_warps` warps each, and how
// the groups' sides are split over their warps: a warp keeps its part and walks
// the line, so the parts of a group are no more than the warps there are (very
// many KV heads would make them so).  Some two to four units per warp: 42k
// tokens of 8 heads 49.6 us; coarser ones, of which some warps get two and some
// one, 62 us; finer ones, whose first tile nothing hides, 52 us.
inline int64_t append_grid(int T, int B, int Hkv, int ctas, int cta_warps, int64_t &groups, int &parts, int &per)
{
    const int64_t resident = (int64_t)ctas * cta_warps;
    groups = append_groups(T, B);
    parts = split_work(groups, 2 * Hkv, 2 * resident, resident, per);
    const int64_t grid = (groups * parts + cta_warps - 1) / cta_warps;
    return grid < ctas ? grid : ctas;
}

// How a scale block's sides (heads' K and V) are split over warps by the 8-bit
// cache's append and read: one each where that is no more than the `wave` of warps
// that are resident, else kByteSides.  A unit's warps should be near one another in
// time, since a token's heads are neighbours in memory, but a warp has to look up its
// row and page first.  Of eight heads appended, one and two a warp: 500 tokens 4.3 and
// 5.7 us, 2k 6.0 and 6.2, 4k 10.8 and 9.7 us.  35k tokens of 8 heads appended and read
// back: 2 sides each 73.4 us; the append with 4 77 us, 1 75 us; the read of 117k
// tokens with 2 sides 108.6 us, 1 114.6 us, 4 111 us, 8 116 us.
constexpr int kByteSides = 2;
inline void byte_split(int T, int B, int Hkv, int lg, int64_t wave, int64_t &groups, int &parts, int &per)
{
    groups = append_groups(T, B, lg);
    per = 2 * groups * Hkv <= wave ? 1 : kByteSides;
    parts = (int)((2 * (int64_t)Hkv + per - 1) / per);
}

// CTAs of an 8-bit append, of `ctas` resident ones of `cta_warps` warps each: warp w
// keeps part w % parts of the sides and takes groups w / parts, and so on, w / parts
// below warps / parts.
inline int64_t byte_append_grid(int T, int B, int Hkv, int lg, int64_t ctas, int cta_warps, int64_t &groups, int &parts, int &per)
{
    const int64_t wave = ctas * cta_warps;
    byte_split(T, B, Hkv, lg, wave, groups, parts, per);
    if (parts > wave) {  // a warp keeps its part: no more of them than there are warps
        per = (int)((2 * (int64_t)Hkv + wave - 1) / wave);
        parts = (int)((2 * (int64_t)Hkv + per - 1) / per);
    }
    const int64_t all = (groups * parts + cta_warps - 1) / cta_warps;
    return all < ctas ? all : ctas;
}

// CTAs of an 8-bit read: warp w has part w % parts of group w / parts, and no
// other.  With ctas = 0 the most there may be for any number of resident ones.
inline int64_t byte_read_grid(int T, int B, int Hkv, int lg, int64_t ctas, int cta_warps, int64_t &groups, int &parts, int &per)
{
    byte_split(T, B, Hkv, lg, ctas * cta_warps, groups, parts, per);
    return (groups * parts + cta_warps - 1) / cta_warps;
}
constexpr int kByteWarps = 8;  // of a CTA of either
constexpr int64_t kMostCtas = 0x7fffffff;

#ifdef __CUDACC__

// The last i in [0, B] with key(i) <= x, for ascending key with key(0) <= x;
// whole warps only, with one x: 33 keys at a time, so that up to 32 rows take
// one round trip.
template <class F>
__device__ __forceinline__ int last_not_above(int B, int64_t x, F key)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, at = lo + (lane + 1) * step;  // lo + step, lo + 2 step, ..
        const unsigned m = __ballot_sync(0xffffffffu, at <= lo + n && key(at) <= x);
        const int up = __popc(m) * step;
        lo += up;
        n = min(n - up, step - 1);
    }
    return lo;
}

#endif  // __CUDACC__

}  // namespace pkv
