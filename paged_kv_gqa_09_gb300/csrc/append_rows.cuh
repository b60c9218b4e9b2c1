// append_rows.cuh -- the rows of a ragged append: which are refused, and their
// lengths when it is done.
#pragma once

#include "append_map.cuh"
#include "pkv_device.cuh"
#include "pkv_kernels.h"

namespace pkv {

// Whether row i's n new tokens, packed from `off` on, are inside the packed
// buffer and fit behind its N tokens; what is wrong with the length goes to the
// error word when `report` is set.
__device__ __forceinline__ bool append_fits(const QuantAppendParams &p, int i, int N, int off, int n, bool report)
{
    if (n < 0 || off < 0 || (int64_t)off + n > p.T)
        return false;
    if (N < 0) {
        if (report)
            report_error(p.ws, kErrNegLen, i, N, 0);
        return false;
    }
    if ((int64_t)N + n > p.len_cap) {
        if (report)
            report_error(p.ws, kErrTooLong, i, (int)min((int64_t)N + n, (int64_t)0x7fffffff), p.len_cap);
        return false;
    }
    return true;
}

// The end of every CTA of the launch, all its threads: the last one to get here
// advances the lengths, which every other one has read by then; CTAs that met a
// bad page (any thread's `bad`) are counted above kBad.  my_off, my_n and my_N:
// offset, tokens and length of row threadIdx.x, where there is one; s_seen: in
// shared memory.
template <int THREADS>
__device__ __forceinline__ void append_finish(const QuantAppendParams &p, bool bad, int my_off, int my_n, int my_N, int *s_seen)
{
    constexpr int kBad = 1 << 20;
    const int any_bad = __syncthreads_or(bad ? 1 : 0);
    if (threadIdx.x == 0) {
        const int add = any_bad ? 1 + kBad : 1;
        *s_seen = atomicAdd(&p.ws->append_done, add) + add;
    }
    __syncthreads();
    if ((*s_seen & (kBad - 1)) != (int)gridDim.x)
        return;
    const bool pages_bad = *s_seen >= kBad;  // then the rows that met them are looked for again
    // offsets that do not ascend within the buffer give tokens to no row or to two: the whole call is refused
    bool span = false;
    for (int r = threadIdx.x; r < p.B; r += THREADS) {
        const bool first = r < THREADS;
        const int off = first ? my_off : p.offsets[r], nr = first ? my_n : p.offsets[r + 1] - off;
        if (off < 0 || nr < 0 || (int64_t)off + nr > p.T) {
            report_error(p.ws, kErrBadSpan, r, off, nr);
            span = true;
        }
    }
    span = __syncthreads_or(span ? 1 : 0) != 0;
    for (int r = threadIdx.x; r < p.B; r += THREADS) {
        const bool first = r < THREADS;
        const int Nr = first ? my_N : p.seq_lens[r];
        const int off = first ? my_off : p.offsets[r], nr = first ? my_n : p.offsets[r + 1] - off;
        bool ok = !span && append_fits(p, r, Nr, off, nr, true);
        if (pages_bad && ok && nr > 0)
            for (int64_t b = Nr >> p.log2P; b <= ((int64_t)Nr + nr - 1) >> p.log2P; ++b) {
                const int page = p.bt[(int64_t)r * p.bt_stride + b];
                ok = ok && page >= 0 && page < p.num_pages;
            }
        p.seq_lens_out[r] = ok ? Nr + nr : Nr;
    }
    if (threadIdx.x == 0)
        p.ws->append_done = 0;
}

}  // namespace pkv
