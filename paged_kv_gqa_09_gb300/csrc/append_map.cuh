// append_map.cuh -- which packed tokens a warp of the 4-bit cache's append takes.
//
// A warp takes eight cache positions 8 k .. 8 k + 7 of one row, a group: those
// are whole words of V.  The rows' groups lie on one line, row i's from
// offsets[i] / 8 + 2 i on, which leaves each room for a first and a last group
// that are not full and needs no sum over the rows before; what is left over is
// idle.  A row without new tokens has places on the line all the same, but no
// group there: its last page, partly filled as it may be, is not looked at.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// Row i's first group, its new tokens packed from `off` on.
__host__ __device__ inline int64_t append_first_group(int off, int i) { return (int64_t)(off >> 3) + 2 * (int64_t)i; }

// Groups on the line of T packed tokens of B rows.
__host__ __device__ inline int64_t append_groups(int T, int B) { return T > 0 ? (int64_t)T / 8 + 2 * (int64_t)B : 0; }

// Whether group gs holds any of row i's n new tokens, which follow its N cached
// ones; pos0: the group's first position.
__host__ __device__ inline bool append_group(int64_t gs, int i, int off, int n, int N, int64_t &pos0)
{
    const int k = (int)(gs - append_first_group(off, i));
    pos0 = ((int64_t)(N >> 3) + k) * 8;
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

}  // namespace pkv
