// Host entry points over the launches of the 8-bit append and read
// (append_map.cuh), so that a CPU test can follow every side of every scale block
// to its warp.  Built by tests/test_byte_grid.py into a temporary directory.
#include "append_map.cuh"

// Counts in units[g * 2 * Hkv + side] how often the append's warps take that side of group g; out: groups, parts,
// sides per part, CTAs.
extern "C" void byte_append_units(int T, int B, int Hkv, int lg, int ctas, int *units, long long *out)
{
    int64_t groups;
    int parts, per;
    const int64_t grid = pkv::byte_append_grid(T, B, Hkv, lg, ctas, pkv::kByteWarps, groups, parts, per);
    out[0] = groups, out[1] = parts, out[2] = per, out[3] = grid;
    const unsigned warps = (unsigned)(grid > 0 ? grid : 1) * pkv::kByteWarps, lines = warps / (unsigned)parts;
    for (unsigned w = 0; units && w < warps; ++w) {  // as byte_append_kernel() does
        const unsigned line = w / (unsigned)parts;
        const int it0 = (int)(w - line * parts) * per, it1 = it0 + per < 2 * Hkv ? it0 + per : 2 * Hkv;
        for (int64_t g = line < lines ? (int64_t)line : groups; g < groups; g += lines)
            for (int it = it0; it < it1; ++it)
                ++units[g * 2 * Hkv + it];
    }
}

// The same for the read.
extern "C" void byte_read_units(int T, int B, int Hkv, int lg, int ctas, int *units, long long *out)
{
    int64_t groups;
    int parts, per;
    const int64_t grid = pkv::byte_read_grid(T, B, Hkv, lg, ctas, pkv::kByteWarps, groups, parts, per);
    out[0] = groups, out[1] = parts, out[2] = per, out[3] = grid;
    for (int64_t unit = 0; units && unit < (grid > 0 ? grid : 1) * pkv::kByteWarps; ++unit) {  // as byte_read_kernel() does
        const int64_t g = unit / parts;
        const int no = (int)(unit - g * parts), it0 = no * per, it1 = it0 + per < 2 * Hkv ? it0 + per : 2 * Hkv;
        for (int it = it0; g < groups && it < it1; ++it)
            ++units[g * 2 * Hkv + it];
    }
}
