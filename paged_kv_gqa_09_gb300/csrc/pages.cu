// pages.cu -- pages and slots for new tokens, and the fp16 append that goes by slots.
//
// map: row i holds N tokens in have = ceil(N / P) pages and gets n more, so that
// it lacks need = ceil((N + n) / P) - have pages.  With off_i and rank_i the sums
// of n and need over the rows before, its k-th new token is packed token off_i + k
// and its j-th new page free_pages[count - 1 - rank_i - j]: every place follows
// from two prefix sums over the rows, so every CTA takes those for itself (rows
// are two ints each, tokens twelve bytes) and one launch without a grid-wide wait
// does it all.  A page is entered in the block table by the thread of the token
// at its start.  The last CTA to finish, when every other one has read the lengths
// and the free count, advances them.  Latency bounds it: 1.1M tokens of 256 rows,
// 14 MB, take 8.7 us, of which 1.8 are lengths and sums, 4 the tokens and 2.5 the
// launch and the last CTA; a token for each of 64 rows 3.2 us, little more than an
// empty launch among others.  Rows are taken 512 at a time, one such pass after the
// other, and beyond 512 by the last of several CTAs once more: a token each of 512
// rows 3.7 us, of 1024 5.7, of 4096 24.  A thread places pairs of tokens, four at a time: what
// a warp stores is whole sectors (four tokens a thread left halves: 9.3 us), and the
// loads of four pages are on their way at once (two 9.6, eight 9.0 us); two CTAs of
// 256 threads per SM (one 10.8, two of 512 threads 12.3 us).
//
// slots: K and V of packed tokens go to their slots, 16 bytes a lane: a copy.  35k
// tokens of 8 heads, d = 128, 290 MB, take 44.4 us, 0.96 of the copy rate, with eight
// pieces a lane on their way (four 44.8, two 47.1 us) and a warp per token (a grid of
// 8 CTAs per SM 46.2 us).
#include "pkv_device.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kInvalid = -2;      // in place of a row's rank: no length that the table could hold
constexpr int kNotServed = -1;    // no pages left for it, or no room in the packed buffer
constexpr int kBadCta = 1 << 20;  // CTAs that met a bad page of the free list count this much more
constexpr int kPairs = 4;         // of tokens that a thread has on their way at a time
constexpr int kFewTokens = 4;     // new tokens of a row up to which its own thread places them (64 rows 3.2 us, searched for 3.5)

// Two rows per thread are held at a time, with what their tokens need in shared memory.
constexpr int kMapThreads = 256, kMapRows = 2 * kMapThreads, kMapWarps = kMapThreads / 32;
struct MapRows {
    int off[kMapRows + 1];  // first packed token, at most T
    int len[kMapRows];      // N
    int rank[kMapRows];     // pages that the rows before need, or one of the above
    int page[kMapRows];     // of the row's last tokens, where that has room for more
    long long sum[2][kMapWarps];
};

struct MapRow {
    int N, n, need, rank;  // as above
    int page;              // as above; -1 where there is none, -2 where its id is out of range
    int status;            // DevErr, kErrNone when the row is served
    int off;               // at most T
};

__device__ __forceinline__ int pages_of(const MapParams &p, int N) { return (N >> p.log2P) + ((N & ((1 << p.log2P) - 1)) != 0); }

// Rows c0 + 2 tid and the next of this thread; off0 and rank0 are the sums over
// the rows before c0 and become those over the rows before the next chunk's.
// Returns whether every row has few new tokens.
__device__ __forceinline__ bool map_rows(const MapParams &p, int c0, int count, MapRows &s, MapRow (&row)[2], long long &off0,
                                         long long &rank0)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, mask = (1 << p.log2P) - 1;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = c0 + 2 * (int)threadIdx.x + u;
        row[u].N = i < p.B ? p.seq_lens[i] : 0;
        row[u].n = i < p.B ? p.new_lens[i] : 0;
    }
    bool few = true;
    long long n2[2], need2[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = c0 + 2 * (int)threadIdx.x + u;
        MapRow &r = row[u];
        r.status = r.N < 0 || r.n < 0 ? kErrNegLen : (long long)r.N + r.n > p.len_cap ? kErrTooLong : kErrNone;
        r.n = max(r.n, 0);
        r.need = r.status == kErrNone ? pages_of(p, r.N + r.n) - pages_of(p, r.N) : 0;
        // on its way while the sums are taken
        r.page = r.status == kErrNone && r.n > 0 && (r.N & mask) ? p.bt[(int64_t)i * p.bt_stride + (r.N >> p.log2P)] : -1;
        n2[u] = r.n;
        need2[u] = r.need;
        few &= r.n <= kFewTokens;
    }
    long long a = n2[0] + n2[1], b = need2[0] + need2[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        s.sum[0][w] = a;
        s.sum[1][w] = b;
    }
    few = __syncthreads_and(few) != 0;
    long long off = off0 + a - n2[0] - n2[1], rank = rank0 + b - need2[0] - need2[1];
#pragma unroll
    for (int v = 0; v < kMapWarps; ++v) {
        const long long x = s.sum[0][v], y = s.sum[1][v];
        off += v < w ? x : 0;
        rank += v < w ? y : 0;
        off0 += x;
        rank0 += y;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        MapRow &r = row[u];
        const int x = 2 * (int)threadIdx.x + u;
        r.off = (int)min(off, (long long)p.T);
        if (r.status == kErrNone && off + r.n > p.T)
            r.status = kErrBadSpan;
        if (r.status == kErrNone && r.need > 0 && rank + r.need > count)
            r.status = kErrNoPage;
        r.rank = r.status == kErrNone ? (int)min(rank, 0x7fffffffll)
                                      : r.status == kErrNoPage || r.status == kErrBadSpan ? kNotServed : kInvalid;
        if (r.page != -1 || (r.status == kErrNone && r.n > 0 && (r.N & mask)))
            if (r.page < 0 || r.page >= p.num_pages)
                r.page = -2;
        s.off[x] = r.off;
        s.len[x] = r.N;
        s.rank[x] = r.rank;
        s.page[x] = r.page;
        if (x == kMapRows - 1)
            s.off[kMapRows] = (int)min(off + n2[u], (long long)p.T);
        off += n2[u];
        rank += need2[u];
    }
    __syncthreads();
    return few;
}

// The lengths and the free count after the call, of the rows map_rows() has
// just seen; `pages_bad`: some id of the free list was out of range, so those are
// looked for.
__device__ __forceinline__ void map_finish(const MapParams &p, int c0, int count, bool pages_bad, const MapRow (&row)[2], int *s_taken)
{
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = c0 + 2 * (int)threadIdx.x + u;
        if (i >= p.B)
            continue;
        const MapRow &r = row[u];
        bool ok = r.status == kErrNone;
        if (r.status == kErrNegLen)
            report_error(p.ws, kErrNegLen, i, r.N < 0 ? r.N : p.new_lens[i], 0);
        else if (r.status == kErrTooLong)
            report_error(p.ws, kErrTooLong, i, (int)min((long long)r.N + r.n, 0x7fffffffll), p.len_cap);
        else if (r.status == kErrBadSpan)
            report_error(p.ws, kErrBadSpan, i, r.off, r.n);
        else if (r.status == kErrNoPage)
            report_error(p.ws, kErrNoPage, i, r.N, count);
        if (ok && r.need > 0)
            atomicMax(s_taken, r.rank + r.need);
        if (ok && r.page == -2) {
            report_error(p.ws, kErrBadPage, i, r.N >> p.log2P, p.bt[(int64_t)i * p.bt_stride + (r.N >> p.log2P)]);
            ok = false;
        }
        if (ok && pages_bad)
            for (int j = 0; ok && j < r.need; ++j) {
                const int page = p.free_pages[count - 1 - r.rank - j];
                ok = page >= 0 && page < p.num_pages;
            }
        p.seq_lens_out[i] = ok ? r.N + r.n : r.N;
    }
}

// The rows' tokens pass T: the first that does and those behind it get no range,
// since an append would take what fits of one.  By one warp of the CTA that has
// written the offsets, cut off at T.  (Found beside the sums, in every CTA, it took
// the 1.1M tokens from 8.7 to 9.9 us.)
__device__ __forceinline__ void map_cut(const MapParams &p)
{
    const int lane = threadIdx.x & 31;
    unsigned m = 0;
    int first = 0;
    __syncwarp();
    for (int i = 0; !m && i < p.B; i += 32) {
        m = __ballot_sync(0xffffffffu, i + lane < p.B && (long long)p.offsets[i + lane] + max(p.new_lens[i + lane], 0) > p.T);
        first = i + __ffs(m) - 1;
    }
    const int at = p.offsets[first];
    for (int i = first + 1 + lane; m && i <= p.B; i += 32)
        p.offsets[i] = at;
}

__global__ void __launch_bounds__(kMapThreads) map_pages_kernel(const MapParams p)
{
    __shared__ MapRows s;
    __shared__ int s_taken, s_seen;
    pdl_wait();
    pdl_trigger();
    const bool alone = gridDim.x == 1;
    if (threadIdx.x == 0)
        s_taken = 0;
    const int count = min(max(*p.free_count, 0), p.free_cap), mask = (1 << p.log2P) - 1;
    // this CTA's tokens [t0, t1), whole groups of four
    const long long quads = ((long long)p.T + 3) / 4, per = (quads + gridDim.x - 1) / gridDim.x;
    const int t0 = (int)min(4 * per * blockIdx.x, (long long)p.T), t1 = (int)min(4 * per * (blockIdx.x + 1), (long long)p.T);
    long long off0 = 0, rank0 = 0;
    bool bad = false;
    auto store = [&](int x, long long slot, int pos) {
        p.slots[x] = slot;
        if (p.positions)
            p.positions[x] = pos;
    };
    // Token x at position `at` of row i, which is on this page (of a row that is served).
    auto place = [&](int x, int i, int at, int N, int rank, int page) {
        const int blk = at >> p.log2P, in = at & mask, j = blk - pages_of(p, N);
        if (rank < 0) {
            if (rank == kNotServed && j >= 0 && in == 0)
                p.bt[(int64_t)i * p.bt_stride + blk] = -1;
            store(x, -1, 0);
            return;
        }
        const bool there = page >= 0 && page < p.num_pages;
        if (!there && j >= 0) {  // the page that had room is seen to elsewhere
            report_error(p.ws, kErrBadPage, i, blk, page);
            bad = true;
        }
        if (j >= 0 && in == 0)
            p.bt[(int64_t)i * p.bt_stride + blk] = there ? page : -1;
        store(x, there ? ((long long)page << p.log2P) + in : -1, there ? at : 0);
    };
    // Two tokens from an even one on.
    auto store2 = [&](int x, long long slot0, long long slot1, int pos0, int pos1) {
        *reinterpret_cast<longlong2 *>(p.slots + x) = make_longlong2(slot0, slot1);
        if (p.positions)
            *reinterpret_cast<int2 *>(p.positions + x) = make_int2(pos0, pos1);
    };
    MapRow row[2];
    for (int c0 = 0; c0 < p.B && (alone || blockIdx.x == 0 || off0 < t1); c0 += kMapRows) {
        const bool few = map_rows(p, c0, count, s, row, off0, rank0);
        const int nr = min(p.B - c0, kMapRows);
        if (blockIdx.x == 0) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (2 * (int)threadIdx.x + u < nr)
                    p.offsets[c0 + 2 * threadIdx.x + u] = row[u].off;
        }
        if (few) {
            // a step of a token per row or a few: from the thread that has the row, without a search
#pragma unroll
            for (int u = 0; u < 2; ++u)
                for (int k = max(t0 - row[u].off, 0); k < min(row[u].n, t1 - row[u].off); ++k) {
                    const int at = row[u].N + k, j = (at >> p.log2P) - pages_of(p, row[u].N);
                    place(row[u].off + k, c0 + 2 * (int)threadIdx.x + u, at, row[u].N, row[u].rank,
                          row[u].rank < 0 || j < 0 ? row[u].page : p.free_pages[count - 1 - row[u].rank - j]);
                }
        } else {
            const int lo = max(t0, s.off[0]), hi = min(t1, s.off[nr]);
            int r = 0;
            for (long long x8 = lo & ~1; lo < hi && x8 < hi; x8 += 2 * kPairs * kMapThreads) {
                // pairs of tokens, neighbouring threads' next to one another; all pages' loads before the first store
                int row_of[kPairs], at[kPairs], page0[kPairs], page1[kPairs];
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const long long xl = x8 + 2 * (k * kMapThreads + (int)threadIdx.x);
                    row_of[k] = -1;
                    if (xl >= hi)
                        continue;
                    const int x = max((int)xl, lo);
                    if (x >= s.off[r + 1]) {  // the last row at or before the pair's first token
                        int up = nr - 1;
                        for (++r; r < up;) {
                            const int mid = (r + up + 1) >> 1;
                            if (s.off[mid] <= x)
                                r = mid;
                            else
                                up = mid - 1;
                        }
                    }
                    row_of[k] = r;
                    at[k] = s.len[r] + (x - s.off[r]);
                    const int j = (at[k] >> p.log2P) - pages_of(p, s.len[r]), top = count - 1 - s.rank[r] - j;
                    const bool whole = x == (int)xl && x + 2 <= min(hi, s.off[r + 1]);  // both tokens are this row's
                    page0[k] = s.rank[r] < 0 || j < 0 ? s.page[r] : p.free_pages[top];
                    page1[k] = !whole || s.rank[r] < 0 ? -1 : (at[k] & mask) == mask ? p.free_pages[top - 1] : page0[k];
                }
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    if (row_of[k] < 0)
                        continue;
                    int y = row_of[k];
                    const int in = at[k] & mask, blk = at[k] >> p.log2P, x = max((int)(x8 + 2 * (k * kMapThreads + (int)threadIdx.x)), lo);
                    if ((unsigned)page0[k] < (unsigned)p.num_pages && (unsigned)page1[k] < (unsigned)p.num_pages) {
                        const long long a = ((long long)page0[k] << p.log2P) + in;
                        store2(x, a, in == mask ? (long long)page1[k] << p.log2P : a + 1, at[k], at[k] + 1);
                        if (in == 0 || in == mask)  // a new page starts with a new token
                            p.bt[(int64_t)(c0 + y) * p.bt_stride + blk + (in != 0)] = page1[k];
                        continue;
                    }
                    // of two rows, of one that is not served, or on a page out of range
                    place(x, c0 + y, at[k], s.len[y], s.rank[y], page0[k]);
                    if ((x & 1) || x + 1 >= hi)
                        continue;
                    while (y + 1 < nr && x + 1 >= s.off[y + 1])
                        ++y;
                    const int next = s.len[y] + (x + 1 - s.off[y]), j = (next >> p.log2P) - pages_of(p, s.len[y]);
                    place(x + 1, c0 + y, next, s.len[y], s.rank[y],
                          s.rank[y] < 0 || j < 0 ? s.page[y] : p.free_pages[count - 1 - s.rank[y] - j]);
                }
            }
        }
        if (alone) {
            const bool any_bad = __syncthreads_or(bad) != 0;
            map_finish(p, c0, count, any_bad, row, &s_taken);
        } else if (p.B > kMapRows) {
            __syncthreads();  // the sums are read until here
        }
    }
    // behind the last token
    for (long long x = (max((long long)t0, off0) & ~1ll) + 2 * threadIdx.x; off0 < t1 && x < t1; x += 2 * kMapThreads) {
        if (x >= off0 && x + 2 <= t1)
            store2((int)x, -1, -1, 0, 0);
        else
            store((int)(x < off0 ? x + 1 : x), -1, 0);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        p.offsets[p.B] = (int)min(off0, (long long)p.T);
    const int any_bad = alone ? 0 : __syncthreads_or(bad ? 1 : 0);
    if (blockIdx.x == 0 && threadIdx.x < 32 && off0 > p.T)
        map_cut(p);
    if (!alone) {
        if (threadIdx.x == 0) {
            const int add = any_bad ? 1 + kBadCta : 1;
            s_seen = atomicAdd(&p.ws->append_done, add) + add;
        }
        __syncthreads();
        if ((s_seen & (kBadCta - 1)) != (int)gridDim.x)
            return;
        if (p.B <= kMapRows) {  // its rows are all there are
            map_finish(p, 0, count, s_seen >= kBadCta, row, &s_taken);
        } else {
            off0 = rank0 = 0;
            for (int c0 = 0; c0 < p.B; c0 += kMapRows) {
                map_rows(p, c0, count, s, row, off0, rank0);
                map_finish(p, c0, count, s_seen >= kBadCta, row, &s_taken);
                __syncthreads();
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *p.free_count_out = count - s_taken;
        if (!alone)
            p.ws->append_done = 0;
    }
}

constexpr int kSlotThreads = 256;
constexpr int kSlotBatch = 8;  // 16-byte pieces a lane has in flight

// A warp per packed token; pieces of K and V in one line.
__global__ void __launch_bounds__(kSlotThreads) append_slots_kernel(const SlotParams p)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t x = (int64_t)blockIdx.x * (kSlotThreads / 32) + (threadIdx.x >> 5);
    if (x >= p.T)
        return;
    const int64_t slot = p.slots[x];
    if (slot < 0)
        return;
    if (slot >= p.num_slots) {
        if (lane == 0)
            report_error(p.ws, kErrBadSlot, (int)x, (int)min(slot, (int64_t)0x7fffffff), (int)min(p.num_slots, (int64_t)0x7fffffff));
        return;
    }
    for (int c0 = lane; c0 < 2 * p.pieces; c0 += 32 * kSlotBatch) {
        int4 v[kSlotBatch];
#pragma unroll
        for (int u = 0; u < kSlotBatch; ++u) {
            const int c = c0 + 32 * u;
            if (c < 2 * p.pieces)
                v[u] = c < p.pieces ? reinterpret_cast<const int4 *>(p.k_new + x * p.new_stride)[c]
                                    : reinterpret_cast<const int4 *>(p.v_new + x * p.new_stride)[c - p.pieces];
        }
#pragma unroll
        for (int u = 0; u < kSlotBatch; ++u) {
            const int c = c0 + 32 * u;
            if (c < 2 * p.pieces) {
                if (c < p.pieces)
                    reinterpret_cast<int4 *>(p.k_cache)[slot * p.pieces + c] = v[u];
                else
                    reinterpret_cast<int4 *>(p.v_cache)[slot * p.pieces + c - p.pieces] = v[u];
            }
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

}  // namespace

cudaError_t launch_map_pages(const MapParams &p, int sms, cudaStream_t s)
{
    const int64_t want = ((int64_t)p.T + 8 * kMapThreads - 1) / (8 * kMapThreads), most = 2 * (int64_t)sms;
    return launch(map_pages_kernel, p, want < most ? want : most, kMapThreads, s);
}

cudaError_t launch_append_slots(const SlotParams &p, cudaStream_t s)
{
    return launch(append_slots_kernel, p, ((int64_t)p.T + kSlotThreads / 32 - 1) / (kSlotThreads / 32), kSlotThreads, s);
}

}  // namespace pkv
