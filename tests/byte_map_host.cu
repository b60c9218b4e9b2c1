// Host entry point over the map of scale blocks to tokens (append_map.cuh with
// groups of 2^lg positions), so that a CPU test can follow every token that the
// 8-bit append and read take.  Built by tests/test_byte_map.py into a temporary
// directory.
#include "append_map.cuh"

// places[x]: the position that packed token x gets, seen[x]: how often; out[0]: groups that hold new tokens, out[1]:
// such a group's first position that is no multiple of 2^lg.
extern "C" void byte_map_all(int B, int T, int lg, const int *off, const int *lens, int *seen, long long *places, long long *out)
{
    out[0] = out[1] = 0;
    for (int64_t gs = 0; gs < pkv::append_groups(T, B, lg); ++gs) {
        int i = 0;  // the last row whose first group is not beyond gs
        while (i + 1 < B && pkv::append_first_group(off[i + 1], i + 1, lg) <= gs)
            ++i;
        const int n = off[i + 1] - off[i], N = lens[i];
        int64_t pos0;
        if (!pkv::append_group(gs, i, off[i], n, N, pos0, lg))
            continue;
        ++out[0];
        out[1] += pos0 % (1 << lg) != 0;
        for (int64_t pos = pos0; pos < pos0 + (1 << lg); ++pos)
            if (pos >= N && pos < (int64_t)N + n) {
                const int64_t x = off[i] + (pos - N);
                ++seen[x];
                places[x] = ((int64_t)i << 32) + pos;
            }
    }
}
