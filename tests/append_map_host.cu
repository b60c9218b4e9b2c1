// Host entry point over the 4-bit append's map of groups to tokens
// (append_map.cuh), so that a CPU test can follow every token that the kernel
// reads and stores.  Built by tests/test_append_map.py into a temporary
// directory.
#include "append_map.cuh"

// Counts what each packed token is read and stored as: reads[x], stores[x] for
// x in [0, T); the number of reads outside that, and of groups whose page is
// looked up, in out[0] and out[1].
extern "C" void append_map_all(int B, int T, const int *off, const int *lens, int *reads, int *stores, long long *place,
                               long long *out)
{
    out[0] = out[1] = 0;
    for (int64_t gs = 0; gs < pkv::append_groups(T, B); ++gs) {
        int i = 0;  // the last row whose first group is not beyond gs
        while (i + 1 < B && pkv::append_first_group(off[i + 1], i + 1) <= gs)
            ++i;
        const int n = off[i + 1] - off[i], N = lens[i];
        int64_t pos0;
        if (!pkv::append_group(gs, i, off[i], n, N, pos0))
            continue;
        ++out[1];
        for (int64_t pos = pos0; pos < pos0 + 8; ++pos) {
            const int tok = pkv::append_token((int)pos, off[i], n, N);
            if (tok < 0 || tok >= T || tok < off[i] || tok >= off[i + 1]) {
                ++out[0];
                continue;
            }
            ++reads[tok];
            if (pos >= N && pos < (int64_t)N + n) {
                ++stores[tok];
                place[tok] = ((long long)i << 32) + pos;
            }
        }
    }
}

// Counts in units[g * 2 * Hkv + side] how often the launch's warps take that
// side of group g; returns the number of groups.
extern "C" long long append_units_all(int T, int B, int Hkv, int ctas, int cta_warps, int *units)
{
    int64_t groups;
    int parts, per;
    const int64_t grid = pkv::append_grid(T, B, Hkv, ctas, cta_warps, groups, parts, per), warps = grid * cta_warps, lines = warps / parts;
    for (int64_t w = 0; w < warps; ++w) {
        const int64_t line = w / parts, first = (w - line * parts) * per;
        if (line >= lines)
            continue;
        for (int64_t g = line; g < groups; g += lines)
            for (int64_t it = first; it < first + per && it < 2 * Hkv; ++it)
                ++units[g * 2 * Hkv + it];
    }
    return groups;
}
