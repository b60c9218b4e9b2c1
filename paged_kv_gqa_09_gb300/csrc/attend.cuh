// attend.cuh -- decode attention over the tokens a sliding window and the row's
// first tokens leave visible, from the fp16 pages, the 4-bit or the 8-bit cache.
// The kernel and its launch, which attend.cu, attend_int8.cu and attend_e4m3.cu
// compile for a kind of cache each.
//
// For query head h of row i with visible tokens t:
//   s_t = scale q_h . K_t,  o = sum_t exp(s_t - m) V_t / l,  lse = m + ln l,
//   m = max_t s_t,  l = sum_t exp(s_t - m).
// One pass over the cache: 4 d flops per visible token and query head against
// 1.25 d bytes (4-bit), 2 d (8-bit) or 4 d (fp16) per token and KV head.  HBM
// bounds long batches (d = 128: 64 rows, 1.9M tokens of the 4-bit cache, 2.44 GB in
// 383 us; 2.1M of the 8-bit cache, 4.32 GB in 624 us; 64 rows in a window of 8191
// over fp16 pages, 1.85 GB in 274 us at most); the 4-bit cache's unpacking and
// latency short ones (117k tokens, 150 MB, 33.6 us; 120k of the 8-bit cache, 247 MB,
// 41.1 us; one row of 32k, 42 MB, 18.2 us).
//
// Work split.  A row's visible tokens lie in T_i tiles of 128 tokens (64 of fp16
// pages with d = 128, 256 of the 4-bit cache with d = 64; those between the sinks
// and the window are never touched).
// All tiles of the batch in (row, KV head, tile) order form one line, with one
// place more at each (row, head)'s end, cut into equal runs, one per CTA: every
// CTA derives the line's length and the cuts from the row lengths, so one launch
// balances rows of any lengths without a plan.  SMs do not stream equally fast
// (equal runs ended between 0.85 and 1.1 of their mean time), so a long run's
// last three sixteenths are cut off in two parts, which the CTAs claim as they
// come free.  The tiles that a segment (a run, or a part of one) holds of one
// (row, head) are a piece; a piece that is the whole (row, head) writes o and
// lse, any other its state (m, l, acc in fp32), and the CTA that finishes a (row, head)'s last piece merges
// its states in piece order, those of a very long row by groups first: the cuts
// do not depend on who takes a segment or comes last, so neither does the
// result.  Calls of few tiles go to clusters instead, one per (row, head).
//
// CTA: warp 4 is the producer, warps 0..3 the consumers.  The producer walks
// the run, reads block-table entries a batch of tiles ahead and streams each
// tile into a ring of shared-memory stages: fp16 pages with tiled TMA copies
// (128-byte swizzle), the 4-bit and 8-bit caches -- whose pages hold K and V of a
// head in one contiguous run per 64 tokens or page -- with plain bulk copies; a
// piece's first tile brings its q rows.  Consumer warp w takes a quarter of every tile's
// tokens, 16 or 32 at a time, with its own online softmax: scores S^T = K q^T (16 tokens x
// 8 heads) and O^T += V^T P^T (d x 8 heads) on mma.sync m16n8k16, fp16 in, fp32
// accumulate.  N = 8 heads is all a KV head has, so a tcgen05 tile would be
// 1/16 full; the registers that mma.sync reads are what the codes are unpacked
// into.  Every wait is bounded (1 s).
#pragma once

#include "pkv_device.cuh"
#include "pkv_kernels.h"
#include "byte_format.cuh"
#include "quant_format.cuh"

#include <atomic>
#include <type_traits>

namespace pkv {
namespace {

constexpr int kCW = 4;                    // consumer warps
constexpr int kThreads = 32 * (kCW + 1);  // + producer warp
constexpr int kMaxG = 8;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.402823466e38f;  // m before the first score: the least finite value (-inf - it is -inf)
constexpr float kNoTiles = -1.f;            // in place of a sum of weights: a cluster's CTA that has none to give
constexpr float kHalfMax = 65504.f;

// What a tile is made of.  kFp16: the fp16 pages; else a cache of codes, the log2
// of its tokens per block added to what it is, so that its tiles' addresses are
// constants.
constexpr int kFp16 = 0, k4Bit = 0, k8Bit = 16;  // k8Bit + 16 FMT
constexpr int kMany = 64;                        // + kMany: the 8-bit cache with d = 128, for many (row, head)s
constexpr int kFew = 128;                        // + kFew: the 8-bit cache, four query heads per KV head or less

template <int KIND>
constexpr bool kIs8Bit = KIND >= k8Bit;
template <int KIND>
constexpr int kBlockLog2 = KIND & 15;
template <int KIND>
constexpr int kFormat = KIND % kMany / 16 - 1;  // of an 8-bit cache

// The softmax weights that enter the product with V: fp16, the tensor cores' operand
// type, holds 11 bits of each, and what that rounding leaves is one more fp16 number.
// It is left out, is the weight of another column of the operand's eight -- a KV
// head's query heads, up to four then -- or has a product of its own.
enum class Weights { kRounded, kBeside, kTwice };
template <int KIND>
constexpr Weights kWeights = !kIs8Bit<KIND> ? Weights::kRounded : KIND & kFew ? Weights::kBeside : Weights::kTwice;
template <Weights W>
constexpr int kProducts = W == Weights::kTwice ? 2 : 1;

// The m that scores are taken from is set this far below a warp's greatest score
// (in log2 units), and set again only when one exceeds it by more than kMaxOver:
// the greatest weights lie in 2^7 .. 2^15, at the upper end of fp16, and most
// tiles need neither a reduction over tokens nor a rescaling.  fp16 ends at
// 2^-24, 2^-31 of the greatest weight: what smaller ones lose in o, while they
// count in the sum, is 2^-32 each at most.  (With the greatest weight at 1 it was
// 2^-25: rows of 2^20 tokens, whose first one leads the others by 25.4 and whose
// warps take a fifth of a row each, lost a fifth of what those add to o.)
constexpr float kMaxUnder = 7.f, kMaxOver = 15.f;

// x sl2 - m is one fused multiply-add, and m comes of a rounded x sl2: the greatest
// score is up to half a step of m off, the same for all of a head's tokens, which
// scales their weights and sum alike.  Past 2^28 that is 16
// and more, beyond fp16; from kFar on, where it is 2^-4, the products are rounded
// before the subtraction.
constexpr float kFar = 1048576.f;

constexpr int kTableLines = 32;  // lines of the block table each CTA brings into L2 at its start

constexpr int kFirst = 1, kLast = 2, kMasked = 4, kEnd = 8;

// Small calls go to clusters of 1, 2, 4, 8 or 16 CTAs, one cluster per (row, KV
// head): each CTA streams its share of the tiles, and the states are merged
// through distributed shared memory instead of global memory and an arrival
// there, which takes 2 us less.
constexpr int kMaxClusterLog2 = 4, kMaxCluster = 1 << kMaxClusterLog2;

// Bytes of a block, and how one becomes zeros: by the numbers that scale its codes
// or, where a code's own bits may be a NaN's (whatever shared memory held), whole.
template <int D, int KIND>
struct Block {
    using Q = QuantLayout<D>;
    static constexpr int kTokens = 1 << kBlockLog2<KIND>;
    __device__ static uint32_t bytes() { return kIs8Bit<KIND> ? byte_block_bytes(kTokens, D) : Q::bytes(kTokens); }
    __device__ static void clear(uint8_t *blk)
    {
        if constexpr (kIs8Bit<KIND>) {
            for (int x = 0; x < byte_block_bytes(kTokens, D); x += 16)
                *reinterpret_cast<uint4 *>(blk + x) = make_uint4(0, 0, 0, 0);
        } else {
            for (int x = 0; x < kTokens * Q::kParamRow; x += 4) {
                *reinterpret_cast<uint32_t *>(blk + Q::k_params(kTokens) + x) = 0;
                *reinterpret_cast<uint32_t *>(blk + Q::v_params(kTokens) + x) = 0;
            }
        }
    }
};

template <int D, int KIND, bool CLUSTER>
struct Layout {
    static constexpr bool QUANT = KIND != kFp16, BYTE = kIs8Bit<KIND>;
    // 16-token blocks of a tile per consumer warp: with two, a tile's barriers,
    // flags and page lookups cost half as much per token, and one block's
    // unpacking overlaps the other's products; one where a tile is 32 KB already
    static constexpr int MT = QUANT || D == 64 ? 2 : 1;
    // and how often it takes as many: tiles of 20 KB over the 4-bit cache with d = 64
    // too (64 rows, 0.98 GB, 182 us in 2 stages; twice the stages of half that 203
    // us), but in clusters, whose shares are few tiles
    static constexpr int NT = QUANT && !BYTE && D == 64 && !CLUSTER ? 2 : 1;
    static constexpr int kTile = 16 * kCW * MT * NT;  // tokens per stage
    static constexpr int kTileLog2 = MT * NT == 4 ? 8 : MT * NT == 2 ? 7 : 6;
    static constexpr int kTileBytes = kTile * D * 2;  // fp16: one of K, V
    static constexpr int kKvBytes = BYTE ? (kTile >> kBlockLog2<KIND>) * byte_block_bytes(1 << kBlockLog2<KIND>, D) : QUANT ? kTile * D * 5 / 4 : 2 * kTileBytes;
    static constexpr int kQBytes = kMaxG * D * 2;
    static constexpr int kStageBytes = kKvBytes + kQBytes;
    // as many CTAs as registers or shared memory hold; where that is three of 128
    // registers or four of 96 the compiler keeps some of a thread's in local memory:
    // 8 to 24 bytes over the 4-bit cache (in clusters of d = 128 and blocks of 64
    // alone), over the 8-bit one 8 in runs of d = 64 and, in blocks of 16 to 64 of
    // kMany, 24 with kFew and e4m3 and 40 without kFew.  fp16 pages with d = 64 (a
    // head's token is one 128-byte line among the others' heads) want more loads
    // from more warps in flight: 64 rows in a window of 8191, three CTAs of two
    // stages 166 us, two of three 208 us; clusters the latter (12.8 and 14.9 us
    // for eight rows).  The 8-bit cache's tiles are 32 KB with d = 128: two CTAs of
    // three stages (eight rows of up to 32k tokens 42.4 us, one of 32k 19.8 us;
    // three of two 43.2 and 21.0 us), but see launch_one() for kMany; tiles of 64
    // tokens, in five stages, leave a warp one block at a time (eight rows 57 us).
    // With d = 64, 64 rows of up to 32k: four CTAs of three stages 177.5 us, three of
    // four 179.5 us, but in clusters 8.1 and 7.4 us (five rows in a window)
    static constexpr int kCtasPerSm = BYTE ? (D == 128 ? (KIND & kMany ? 3 : 2) : CLUSTER ? 3 : 4) : QUANT ? (D == 64 ? 4 : 3) : D == 64 && !CLUSTER ? 3 : 2;
    static constexpr int kStages = BYTE ? (KIND & kMany ? 2 : D == 64 && CLUSTER ? 4 : 3) : QUANT ? (D == 64 ? (CLUSTER ? 4 : 2) : 3) : D == 64 && !CLUSTER ? 2 : 3;
    static constexpr int kMetaOff = kStages * kStageBytes;          // two int4 per stage
    static constexpr int kRedOff = kMetaOff + kStages * 32;         // m, l of [piece parity][warp][head]
    static constexpr int kBarOff = kRedOff + 2 * kCW * kMaxG * 2 * 4;   // full[S], empty[S], consumers
    static constexpr int kStateOff = (kBarOff + (2 * kStages + 1) * 8 + 15) & ~15;  // cluster: what its CTAs send this one
    static constexpr int kBytes = kStateOff + (CLUSTER ? kMaxG * (D + 2 * kMaxCluster) * 4 : 0);
    static constexpr int kAlloc = kBytes + 1024;
    // at a piece's end the warps exchange their states through its last stage
    static_assert(kStageBytes >= (kCW - 1) * kMaxG * D * 4, "a stage holds three warps' states");
    static_assert(QUANT || kStageBytes % 1024 == 0, "swizzled tiles keep 1024-byte alignment");
    static_assert(kCtasPerSm * (kAlloc + 1024) <= 228 * 1024, "resident CTAs");
};

// An output's rounding to fp16.  The weights sum up to a little more or less
// rounded than unrounded (see softmax_step()), so that a mean of values at the
// type's end could pass it and become infinite: finite results stay finite.
__device__ __forceinline__ float within_half(float x) { return fabsf(x) < INFINITY ? fminf(fmaxf(x, -kHalfMax), kHalfMax) : x; }
// What an accumulator is multiplied by for o.  A head whose scores are all -inf
// has weights of 0 alone: o = 0 (NaN where a value is infinite or NaN) and lse = -inf, as
// for a row that sees nothing, whichever way the work was cut.
__device__ __forceinline__ float over_sum(float l) { return l == 0.f ? 1.f : 1.f / l; }

__device__ __forceinline__ __half out_half(float x) { return __float2half_rn(within_half(x)); }
__device__ __forceinline__ uint32_t out_half2(float x, float y) { return pack_half2(within_half(x), within_half(y)); }

// What of a row of N tokens is visible: tokens [0, ns) and [w0, N), in tiles
// [0, a) and [b, b + T - a).
struct RowSpan {
    int N, ns, w0, a, b, T;
    // on the line of tiles each (row, head) that sees any takes one more: its
    // end costs about what a tile does (1.5 us)
    __device__ __forceinline__ int line() const { return T > 0 ? T + 1 : 0; }
    __device__ __forceinline__ int tile(int k) const { return k < a ? k : b + (k - a); }
};

template <int kTile>
__device__ __forceinline__ RowSpan row_span(const AttendParams &p, int len)
{
    RowSpan r;
    r.N = min(max(len, 0), p.len_cap);
    r.ns = min(p.sinks, r.N);
    r.w0 = max(r.ns, r.N - p.window);
    r.a = (int)(((unsigned)r.ns + kTile - 1) / kTile);
    r.b = max(r.a, r.w0 / kTile);
    r.T = r.a;
    if (r.w0 < r.N)
        r.T += max(0, (int)(((unsigned)r.N + kTile - 1) / kTile) - r.b);
    return r;
}

__device__ __forceinline__ bool visible(int tok, int ns, int w0, int N) { return tok < ns || (tok >= w0 && tok < N); }

// Byte offset of token t inside a K/V tile that TMA filled with swizzled boxes
// of (1 << btl) tokens x D columns, laid out [box][64-column block][token][128 bytes].
template <int D>
__device__ __forceinline__ uint32_t row_base(int t, int btl)
{
    const int b = t >> btl, s = t & ((1 << btl) - 1);
    return (uint32_t)(((b << btl) * (D / 64) + s) * 128);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// Runs of fewer tiles stay whole: their parts would be single tiles, whose
// states cost as much as they balance (eight mixed rows, runs of 17 tiles: 35 us
// whole, 43 us in parts).
constexpr int kMinSplitRun = 48;
// A claimed part finds its row by a scan over the batch; beyond this many rows
// runs stay whole too.
constexpr int kMaxSplitRows = 1024;

// Longer runs differ by one tile at most, instead of leaving the last CTAs without
// any (16 tiles and a little, 34.3 against 35.8 us; 9 tiles, 22.4 against 23.7
// us).  Shorter ones make more pieces that way, which costs more (4 to 5 tiles,
// 18.7 against 18.2 us), and runs in parts even out anyway.
constexpr int kMinEvenRun = 7;

// The cuts of the line of W tiles into runs of q tiles each, one more in the
// first `rem`, which lie on different SMs.  Run r's segments are
// parts * r + 0 .. parts - 1 in line order: H tiles, then M, then the rest.
// (The host keeps W and W + grid within an int.)
struct Cuts {
    int W, q, rem, H, M, parts;
    __device__ __forceinline__ Cuts(int W_, int grid, int B) : W(W_)
    {
        const int up = max((int)((unsigned)(W + grid - 1) / (unsigned)grid), 1);
        parts = up >= kMinSplitRun && B <= kMaxSplitRows ? 3 : 1;
        const bool even = parts == 1 && up > kMinEvenRun;
        q = even ? (int)((unsigned)W / (unsigned)grid) : up;
        rem = even ? W - q * grid : 0;
        H = q - 3 * (q / 16);
        M = 2 * (q / 16);
    }
    __device__ __forceinline__ int start(int r) const { return min(r * q + min(r, rem), W); }
    __device__ __forceinline__ int segment(int x) const
    {
        const int longer = rem * (q + 1);
        const int r = x < longer ? (int)((unsigned)x / (unsigned)(q + 1)) : rem + (int)((unsigned)(x - longer) / (unsigned)q);
        if (parts == 1)
            return r;
        const int y = x - start(r);
        return 3 * r + (y >= H) + (y >= H + M);
    }
    __device__ __forceinline__ int begin(int r, int part) const { return min(r * q + min(r, rem) + (part == 0 ? 0 : part == 1 ? H : H + M), W); }
    __device__ __forceinline__ int end(int r, int part) const { return part == parts - 1 ? start(r + 1) : begin(r, part + 1); }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The same shared-memory place in CTA `rank` of the cluster, and a store to it.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_store(uint32_t a, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t a, float2 v)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t a, float4 v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// What a cluster's 2^cl CTAs send CTA r, which merges dims r D / 2^cl ..: of each
// one's accumulators those dims, [rank][head][dim], then m and l [rank][head].
template <int D>
struct Inbox {
    uint32_t base;
    int cl, rank;  // of the sender
    template <class V>  // one dim, or two or four from a multiple of that on
    __device__ __forceinline__ void acc(int head, int dim, V v) const
    {
        constexpr int kLog2 = D == 128 ? 7 : 6;
        const int per = kLog2 - cl;
        cluster_store(cluster_addr(base + (((((rank * kMaxG) + head) << per) + (dim & ((1 << per) - 1))) << 2), dim >> per), v);
    }
    // to all of them, by a warp whose lanes h0 / 2 + 4 r0 hold heads h0 and h0 + 1
    __device__ __forceinline__ void sums(int h0, int r0, float m0, float m1, float l0, float l1) const
    {
        for (int r = r0; r < 1 << cl; r += 8) {
            const uint32_t m = cluster_addr(base + (kMaxG * D + rank * kMaxG + h0) * 4, r);
            cluster_store(m, m0);
            cluster_store(m + 4, m1);
            cluster_store(m + (kMaxG << (cl + 2)), l0);
            cluster_store(m + (kMaxG << (cl + 2)) + 4, l1);
        }
    }
};

// The 8-bit cache's first tiles of this CTA on their way to L2, by one warp while
// the producer still waits for the kernel before: three DRAM latencies (lengths,
// table, pages) less after the wait.  What that kernel may still be writing is read
// past L1 and only as a hint, of batches of a few windows of 32 rows: whatever it
// says, the tiles are looked up again.  Eight rows of up to 32k tokens 45.4 us
// without, 43.4 with one tile, 42.4 with two, 41.9 with three, 42.1 with four; one row
// of 32k 20.2, 19.2, 19.9, 21.2 and 21.6 us; 16 rows of 1k 11.1, 10.2, 9.6, 9.8 and 10.0
// us.
constexpr int kHintRows = 128, kHintTiles = 2;

template <int D, int KIND, bool CLUSTER>
__device__ __forceinline__ void hint_first_tiles(const AttendParams &p)
{
    using L = Layout<D, KIND, CLUSTER>;
    constexpr int kTile = L::kTile, TBL = kBlockLog2<KIND>, NBL = L::kTileLog2 - TBL;
    const int lane = threadIdx.x & 31, cta = (int)blockIdx.x;
    RowSpan rs;
    int i = 0, h = 0, k0 = 0, k1 = 0;
    if constexpr (CLUSTER) {
        const int cl = p.cluster_log2, unit = cta >> cl, r = cta - (unit << cl);
        i = unit / p.Hkv;
        h = unit - i * p.Hkv;
        rs = row_span<kTile>(p, __ldcg(p.seq_lens + i));
        const int up = (1 << cl) - 1;
        k0 = (rs.T * r + up) >> cl;
        k1 = (rs.T * (r + 1) + up) >> cl;
    } else {
        if (p.B > kHintRows)
            return;
        int W = 0;
        for (int at = 0; at < p.B; at += 32)
            W += at + lane < p.B ? row_span<kTile>(p, __ldcg(p.seq_lens + at + lane)).line() : 0;
        const Cuts cuts(__reduce_add_sync(0xffffffffu, W) * p.Hkv, (int)gridDim.x, p.B);
        int f = cuts.begin(cta, 0);
        const int end = cuts.end(cta, 0);
        for (int at = 0; at < p.B; at += 32) {
            const RowSpan mine = row_span<kTile>(p, at + lane < p.B ? __ldcg(p.seq_lens + at + lane) : 0);
            int incl = mine.line();
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += y;
            }
            const int tot = __shfl_sync(0xffffffffu, incl, 31) * p.Hkv;
            if (f >= tot) {
                f -= tot;
                continue;
            }
            const unsigned m = __ballot_sync(0xffffffffu, f < incl * p.Hkv);
            const int src = __ffs(m) - 1;
            f -= __shfl_sync(0xffffffffu, incl - mine.line(), src) * p.Hkv;
            i = at + src;
            rs.N = __shfl_sync(0xffffffffu, mine.N, src);
            rs.ns = __shfl_sync(0xffffffffu, mine.ns, src);
            rs.w0 = __shfl_sync(0xffffffffu, mine.w0, src);
            rs.a = __shfl_sync(0xffffffffu, mine.a, src);
            rs.b = __shfl_sync(0xffffffffu, mine.b, src);
            rs.T = __shfl_sync(0xffffffffu, mine.T, src);
            h = (int)((unsigned)f / (unsigned)(rs.T + 1));
            k0 = f - h * (rs.T + 1);
            k1 = min(rs.T, k0 + end - cuts.begin(cta, 0));
            break;
        }
    }
    const int k = k0 + (lane >> NBL);
    if (k >= k1 || (lane >> NBL) >= kHintTiles)
        return;
    const int tok = rs.tile(k) * kTile + ((lane & ((1 << NBL) - 1)) << TBL);
    if (!(tok < rs.ns || (tok + (1 << TBL) > rs.w0 && tok < rs.N)))
        return;
    const int pg = __ldcg(p.bt + (int64_t)i * p.bt_stride + (tok >> p.log2P));
    if (pg < 0 || pg >= p.num_pages)
        return;
    const uint32_t bytes = Block<D, KIND>::bytes();
    const uint8_t *from = p.cache + ((int64_t)pg * p.Hkv + h) * p.page_head_bytes +
                          (int64_t)((tok & ((1 << p.log2P) - 1)) >> TBL) * bytes;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------- producer

template <int D, int KIND, bool CLUSTER>
__device__ __forceinline__ void run_producer(const CUtensorMap *tmK, const CUtensorMap *tmV, const AttendParams &p,
                                             uint32_t sbase, uint8_t *basep, int4 *meta, uint32_t full0, uint32_t empty0)
{
    using L = Layout<D, KIND, CLUSTER>;
    constexpr bool QUANT = L::QUANT;
    constexpr int kTile = L::kTile;
    const int lane = threadIdx.x & 31;
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;
    const int tbl = QUANT ? kBlockLog2<KIND> : p.tb_log2, tb = 1 << tbl;
    const int nbl = L::kTileLog2 - tbl;  // log2 of the blocks per tile
    const uint32_t blk_bytes = QUANT ? Block<D, KIND>::bytes() : (uint32_t)(tb * D * 2);
    const uint64_t pol = l2_evict_first_policy();

    // test hook: the first stage is left out, so the consumers' bounded wait for it runs out
    int stage = p.starve_first_stage && cta == 0 ? 1 : 0;
    uint32_t ph = 0, pend = 0, pend_par = 0;
    bool ok = true;

    // Streams tiles [k0, k1) of (row i, KV head h): a piece, for `slot` (see finish_piece()).
    auto stream = [&](int i, int h, const RowSpan &rs, int k0, int k1, int slot, int unit_pieces) {
        // Block-table entries: lane l holds block l & (2^nbl - 1) of the batch's tile
        // l >> nbl, a batch ahead of the copies; -1: nothing visible in it, num_pages: bad id.
        auto page_of = [&](int kb) {
            const int k = kb + (lane >> nbl);
            if (k >= k1)
                return -1;
            const int tok = rs.tile(k) * kTile + ((lane & ((1 << nbl) - 1)) << tbl);
            if (!(tok < rs.ns || (tok + tb > rs.w0 && tok < rs.N)))
                return -1;
            const int pg = p.bt[(int64_t)i * p.bt_stride + (tok >> p.log2P)];
            if (pg < 0 || pg >= p.num_pages) {
                report_error(p.ws, kErrBadPage, i, tok >> p.log2P, pg);
                return p.num_pages;
            }
            return pg;
        };
        int pid = page_of(k0), pnx = -1;
        for (int k = k0; k < k1; ++k) {
            const int in_batch = (k - k0) & ((32 >> nbl) - 1);
            if (in_batch == 0) {
                if (k != k0)
                    pid = pnx;
                pnx = page_of(k + (32 >> nbl));
            }
            const int tok0 = rs.tile(k) * kTile;
            const uint32_t full = full0 + stage * 8;
            if (!__all_sync(0xffffffffu, mbar_wait(empty0 + stage * 8, ph ^ 1, kWaitNs))) {
                report_error(p.ws, kErrTimeout, cta, stage, 0);
                ok = false;
                return;
            }
            pend &= ~(1u << stage);
            const uint32_t dst = sbase + stage * L::kStageBytes;
            const bool mine_now = (lane >> nbl) == in_batch && pid >= 0;
            const int b = lane & ((1 << nbl) - 1);
            const bool bad = QUANT && mine_now && pid == p.num_pages;
            if (bad) {  // a bad page reads as zeros
                Block<D, KIND>::clear(basep + (dst - sbase) + b * blk_bytes);
                fence_proxy_async_smem();
            }
            __syncwarp();  // lane 0's arrival publishes the zeros
            const int copies = __popc(__ballot_sync(0xffffffffu, mine_now && !bad));
            if (lane == 0) {
                const bool whole = rs.ns >= tok0 + kTile || (tok0 >= rs.w0 && tok0 + kTile <= rs.N);
                const int flags = (k == k0 ? kFirst : 0) | (k == k1 - 1 ? kLast : 0) | (whole ? 0 : kMasked);
                meta[2 * stage] = make_int4(i * p.Hkv + h, tok0, flags, slot);
                meta[2 * stage + 1] = make_int4(rs.ns, rs.w0, rs.N, unit_pieces);
                mbar_arrive_expect_tx(full, copies * blk_bytes * (QUANT ? 1 : 2) + (k == k0 ? (uint32_t)(p.G * D * 2) : 0u));
                if (k == k0)
                    bulk_load(dst + L::kKvBytes, p.q + ((int64_t)i * p.Hq + h * p.G) * D, p.G * D * 2, full, pol);
            }
            __syncwarp();
            if (mine_now && !bad) {
                const int slot_in = (tok0 + (b << tbl)) & ((1 << p.log2P) - 1);
                if constexpr (QUANT) {
                    bulk_load(dst + b * blk_bytes,
                              p.cache + ((int64_t)pid * p.Hkv + h) * p.page_head_bytes + (int64_t)(slot_in >> tbl) * blk_bytes,
                              blk_bytes, full, pol);
                } else {
                    tma_load_5d(dst + b * blk_bytes, tmK, full, 0, slot_in, 0, h, pid, pol);
                    tma_load_5d(dst + L::kTileBytes + b * blk_bytes, tmV, full, 0, slot_in, 0, h, pid, pol);
                }
            }
            pend |= 1u << stage;
            pend_par = (pend_par & ~(1u << stage)) | (ph << stage);
            if (++stage == L::kStages) {
                stage = 0;
                ph ^= 1;
            }
        }
    };
    auto check_len = [&](int i, int len) {
        if (len < 0 || len > p.len_cap)
            report_error(p.ws, len < 0 ? kErrNegLen : kErrTooLong, i, len, p.len_cap);
    };

    if constexpr (CLUSTER) {
        // the cluster's (row, head), of which this CTA streams its share
        const int cl = p.cluster_log2, unit = cta >> cl, r = cta - (unit << cl), i = unit / p.Hkv, h = unit - i * p.Hkv;
        const int len = p.seq_lens[i];
        if (h == 0 && r == 0 && lane == 0)
            check_len(i, len);
        const RowSpan rs = row_span<kTile>(p, len);
        const int up = (1 << cl) - 1, k0 = (rs.T * r + up) >> cl, k1 = (rs.T * (r + 1) + up) >> cl;
        if (k0 < k1)
            stream(i, h, rs, k0, k1, cl == 0 ? -1 : 0, 0);
    } else {
        // the line of tiles and this CTA's run of it; rows [wb, wb + 32) are held one per lane
        int wb = 0;
        RowSpan mine;
        auto window = [&](int at) {
            const int len = at + lane < p.B ? p.seq_lens[at + lane] : 0;
            if (cta == 0 && at + lane < p.B)
                check_len(at + lane, len);
            return row_span<kTile>(p, len);
        };
        mine = window(0);
        int W = mine.line();
        for (int at = 32; at < p.B; at += 32)
            W += window(at).line();
        const Cuts cuts(__reduce_add_sync(0xffffffffu, W) * p.Hkv, grid, p.B);

        int run = cta, part = 0;  // this CTA's own run first
        while (ok) {
            const int start = cuts.begin(run, part), end = cuts.end(run, part);
            const int seg = cuts.parts * run + part;
            if (start < end) {
                // row_start: line index of the current row
                int cur = 0, row_start = 0;
                if (wb != 0) {
                    wb = 0;
                    mine = window(0);
                }
                for (;;) {
                    int incl = mine.line();
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o)
                            incl += y;
                    }
                    const int tot = __shfl_sync(0xffffffffu, incl, 31);
                    if (start < row_start + tot * p.Hkv) {
                        cur = __ffs(__ballot_sync(0xffffffffu, start < row_start + incl * p.Hkv)) - 1;
                        row_start += __shfl_sync(0xffffffffu, incl - mine.line(), cur) * p.Hkv;
                        break;
                    }
                    row_start += tot * p.Hkv;
                    wb += 32;
                    if (wb >= p.B)
                        break;  // the lengths changed under the launch: the segment lies inside the line
                    mine = window(wb);
                }
                int f = start;
                RowSpan rs;
                auto take = [&](int src) {
                    rs.N = __shfl_sync(0xffffffffu, mine.N, src);
                    rs.ns = __shfl_sync(0xffffffffu, mine.ns, src);
                    rs.w0 = __shfl_sync(0xffffffffu, mine.w0, src);
                    rs.a = __shfl_sync(0xffffffffu, mine.a, src);
                    rs.b = __shfl_sync(0xffffffffu, mine.b, src);
                    rs.T = __shfl_sync(0xffffffffu, mine.T, src);
                };
                take(cur);
                int h = rs.T > 0 ? (int)((unsigned)(f - row_start) / (unsigned)(rs.T + 1)) : 0;
                while (f < end && ok && rs.T > 0 && wb < p.B) {
                    const int u0 = row_start + h * (rs.T + 1), u1 = u0 + rs.T;
                    if (f < u1) {
                        const int c0 = u0 >= start ? seg : cuts.segment(u0), c1 = u1 <= end ? seg : cuts.segment(u1 - 1);
                        stream(wb + cur, h, rs, f - u0, min(u1, end) - u0, c0 == c1 ? -1 : seg == c0 ? 2 * seg + 1 : 2 * seg,
                               c0 | ((c1 - c0) << 16));
                    }
                    f = u1 + 1;
                    if (++h == p.Hkv && f < end) {  // the next row with visible tokens
                        row_start += (rs.T + 1) * p.Hkv;
                        h = 0;
                        unsigned m = __ballot_sync(0xffffffffu, mine.T > 0 && lane > cur);
                        while (!m && wb < p.B) {
                            wb += 32;
                            mine = window(wb);
                            m = __ballot_sync(0xffffffffu, mine.T > 0);
                        }
                        if (!m)
                            break;  // the lengths changed under the launch
                        cur = __ffs(m) - 1;
                        take(cur);
                    }
                }
            }
            if (cuts.parts == 1)
                break;
            // the next part to be claimed: every run's second, then every run's last
            int q = 0;
            if (lane == 0)
                q = atomicAdd(&p.ws->next_task, 1);
            q = __shfl_sync(0xffffffffu, q, 0);
            if (q >= 2 * grid)
                break;
            part = q < grid ? 1 : 2;
            run = q < grid ? q : q - grid;
        }
        if (cuts.parts > 1 && lane == 0 && atomicAdd(&p.ws->done_ctas, 1) == grid - 1) {
            // every CTA has made its last claim: ready for the next launch
            p.ws->next_task = 0;
            p.ws->done_ctas = 0;
        }
    }
    if (ok) {
        if (__all_sync(0xffffffffu, mbar_wait(empty0 + stage * 8, ph ^ 1, kWaitNs))) {
            pend &= ~(1u << stage);
            if (lane == 0) {
                meta[2 * stage] = make_int4(0, 0, kEnd, 0);
                mbar_arrive(full0 + stage * 8);
            }
        } else {
            report_error(p.ws, kErrTimeout, cta, stage, 1);
            ok = false;
        }
    }
    if (!ok && lane == 0)  // let every copy this CTA issued land before its shared memory goes away
        for (int s = 0; s < L::kStages; ++s)
            if (pend & (1u << s))
                mbar_wait(full0 + s * 8, (pend_par >> s) & 1u, kDrainNs);
}

// ---------------------------------------------------------------- consumers

// All consumer warps meet (bounded); what each wrote before is visible after.
__device__ __forceinline__ bool meet(uint32_t bar, uint32_t &phase)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase, kWaitNs));
    phase ^= 1;
    return ok;
}

// The state of one warp for the 8 heads of a piece: lane (r0, h0 / 2) holds
// heads h0, h0 + 1 and dims dim_of(x, r0) and kDimStep further on.
template <int D>
struct State {
    static constexpr int KS = D / 16;
    float m0, m1, l0, l1, O[KS][4];
    __device__ __forceinline__ void clear()
    {
        m0 = m1 = kNoMax;
        l0 = l1 = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x)
            O[x][0] = O[x][1] = O[x][2] = O[x][3] = 0.f;
    }
};

// 16 x + r0 and 8 further on; over the 8-bit cache, whose lanes read four dims at
// a time, 32 (x / 2) + 4 r0 + 2 (x & 1) and the next.
template <int KIND>
__device__ __forceinline__ int dim_of(int x, int r0)
{
    return kIs8Bit<KIND> ? 32 * (x >> 1) + 4 * r0 + 2 * (x & 1) : 16 * x + r0;
}
template <int KIND>
constexpr int kDimStep = kIs8Bit<KIND> ? 1 : 8;

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }

// What turns a raw score of block u into units of log2: one factor for all, or K's
// scale with it, that of a lane's two tokens.
struct OneScale {
    float sl2;
    __device__ __forceinline__ float times(int) const { return sl2; }
};
template <int MT>
struct BlockScales {
    float k[MT];
    __device__ __forceinline__ float times(int u) const { return k[u]; }
};

// Raw scores x[b] of MT blocks of 16 tokens -- x[b][0], x[b][1]: token r0 with
// heads h0 and h0 + 1, x[b][2], x[b][3]: token r0 + 8; bit 16 b + token of
// `vis` set where visible -- enter the running softmax in units of log2;
// returns the weights as the B operands of the PV product, rounded to fp16 and, with
// kTwice, what that left; with kBeside that is in place of heads 4 and more, whose
// scores have to be those of heads 0 and more once again.  Rounded alone they cost o
// about as much as its own rounding (2^-11 of the mean |v| at most; o is off by
// 2.1e-4 to 2.9e-4 of its size, else by 2.0e-4 to 2.1e-4).  Their sum is kept in fp32
// before that rounding, so that lse is not rounded with them.  Over the 8-bit cache
// nothing is left out.  That takes, beside: 16 rows of 1k 9.05 -> 9.30 us, eight of 4k
// 13.96 -> 14.2, 100 of 100 13.2 -> 13.6, 64 in a window of 4096 78.0 -> 78.4; twice, with
// eight heads, the same: 9.2 -> 9.7, 14.1 -> 15.0, 13.7 -> 15.3, 79.1 -> 81.5; 64 rows of up
// to 60k 0.4% and 1.2%.  (One kernel for either, which picks by the head count, took a
// row of 1k from 4.9 to 5.4.)
template <int D, int MT, Weights W, class Scales>
__device__ __forceinline__ void softmax_step(State<D> &st, const float (&x)[MT][4], uint32_t vis, const Scales &sc,
                                             uint32_t (&P)[kProducts<W>][MT][2])
{
    constexpr uint32_t kAll = MT == 2 ? 0xffffffffu : 0xffffu;
    const int r0 = (threadIdx.x & 31) >> 2;
    float y[MT][4];
    auto hide = [&] {
        if (vis != kAll) {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(vis >> (16 * u + 8 * (e >> 1) + r0) & 1))
                        y[u][e] = -INFINITY;
        }
    };
    auto scaled = [&](float m0, float m1) {
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[u][e] = fmaf(x[u][e], sc.times(u), (e & 1) ? -m1 : -m0);
        hide();
    };
    auto most = [&](int odd) {
        float a = -INFINITY;
#pragma unroll
        for (int u = 0; u < MT; ++u)
            a = fmaxf(a, fmaxf(y[u][odd], y[u][2 + odd]));
        return a;
    };
    scaled(st.m0, st.m1);
    if (__any_sync(0xffffffffu, fmaxf(most(0), most(1)) > kMaxOver || fmaxf(fabsf(st.m0), fabsf(st.m1)) >= kFar)) {
        scaled(0.f, 0.f);
        float n0 = fmaxf(st.m0, most(0) - kMaxUnder), n1 = fmaxf(st.m1, most(1) - kMaxUnder);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
        }
        const float f0 = ex2(st.m0 - n0), f1 = ex2(st.m1 - n1);
        st.m0 = n0;
        st.m1 = n1;
        st.l0 *= f0;
        st.l1 *= f1;
#pragma unroll
        for (int z = 0; z < State<D>::KS; ++z) {
            st.O[z][0] *= f0;
            st.O[z][1] *= f1;
            st.O[z][2] *= f0;
            st.O[z][3] *= f1;
        }
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float n = (e & 1) ? n1 : n0;
                y[u][e] = fabsf(n) < kFar ? fmaf(x[u][e], sc.times(u), -n) : __fmul_rn(x[u][e], sc.times(u)) - n;
            }
        hide();
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const float p0 = ex2(y[u][0]), p1 = ex2(y[u][1]), p2 = ex2(y[u][2]), p3 = ex2(y[u][3]);
        st.l0 += p0 + p2;
        st.l1 += p1 + p3;
        uint32_t a = pack_half2(p0, p1), b = pack_half2(p2, p3);
        if constexpr (W != Weights::kRounded) {
            const float2 fa = __half22float2(as_half2(a)), fb = __half22float2(as_half2(b));
            const uint32_t ra = pack_half2(p0 - fa.x, p1 - fa.y), rb = pack_half2(p2 - fb.x, p3 - fb.y);
            if constexpr (W == Weights::kBeside) {
                if (threadIdx.x & 2)
                    a = ra, b = rb;
            } else {
                P[1][u][0] = movmatrix_t(ra);
                P[1][u][1] = movmatrix_t(rb);
            }
        }
        P[0][u][0] = movmatrix_t(a);
        P[0][u][1] = movmatrix_t(b);
    }
}

// One tile of the fp16 pages: this warp's 16 or 32 tokens, of which `vis` (a bit
// per token) are visible.
template <int D>
__device__ __forceinline__ void fp16_tile(State<D> &st, const uint32_t (&qf)[D / 16][2], uint32_t kt, uint8_t *ktp, uint32_t vis,
                                          int w, int btl, float sl2)
{
    using L = Layout<D, kFp16, false>;
    constexpr int KS = D / 16, MT = L::MT, TW = 16 * MT;
    const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
    const uint32_t blk = 128u << btl;
    const uint32_t vt = kt + L::kTileBytes;
    if (vis != 0xffffffffu >> (32 - TW)) {
        // masked rows hold anything: zero them in V so that p = 0 meets no NaN
        uint8_t *vtp = ktp + L::kTileBytes;
        for (int x = lane; x < TW * (D / 8); x += 32) {
            const int tok = TW * w + x / (D / 8), c = x % (D / 8);
            if (!(vis >> (tok & (TW - 1)) & 1))
                *reinterpret_cast<int4 *>(vtp + row_base<D>(tok, btl) + (c >> 3) * blk + (((c & 7) ^ (tok & 7)) << 4)) =
                    make_int4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
    float x[MT][4];
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const uint32_t rowK = row_base<D>(TW * w + 16 * u + (mi & 1) * 8 + r8, btl);
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int z = 0; z < KS; ++z) {
            const uint32_t cc = (uint32_t)((((2 * z) & 7) + (mi >> 1)) ^ r8) << 4;
            uint32_t a0, a1, a2, a3;
            ldsm_x4(kt + rowK + (z >> 2) * blk + cc, a0, a1, a2, a3);
            mma_16816(z & 1 ? sb : sa, a0, a1, a2, a3, qf[z][0], qf[z][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[u][e] = sa[e] + sb[e];
    }
    uint32_t P[1][MT][2];
    softmax_step<D, MT, Weights::kRounded>(st, x, vis, OneScale{sl2}, P);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const uint32_t rowV = row_base<D>(TW * w + 16 * u + (mi >> 1) * 8 + r8, btl);
#pragma unroll
        for (int z = 0; z < KS; ++z) {
            const uint32_t cc = (uint32_t)((((2 * z) & 7) + (mi & 1)) ^ r8) << 4;
            uint32_t a0, a1, a2, a3;
            ldsm_x4_t(vt + rowV + (z >> 2) * blk + cc, a0, a1, a2, a3);
            mma_16816(st.O[z], a0, a1, a2, a3, P[0][u][0], P[0][u][1]);
        }
    }
}

template <int GR>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[GR])
{
    if constexpr (GR == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    }
}

// One tile of the 4-bit cache, of which this warp takes 32 tokens, four groups
// of eight: codes go from shared memory to the fragments of the tensor cores' A
// operand in registers (see quant_format.cuh).
template <int D, int TBL>
__device__ __forceinline__ void quant_tile(State<D> &st, const uint32_t (&qf)[D / 16][2], const uint8_t *kv, uint32_t vis, int w,
                                           float sl2)
{
    using Q = QuantLayout<D>;
    constexpr int GR = Q::GR, TB = 1 << TBL, MT = 2;
    const int lane = threadIdx.x & 31, r0 = lane >> 2, t = lane & 3;
    auto group = [&](int u) { return kv + ((32 * w + 8 * u) >> TBL) * Q::bytes(TB); };  // its block
    auto in = [&](int u) { return (32 * w + 8 * u) & (TB - 1); };                       // its first token there
    float x[MT][4];
    uint32_t k0[MT][GR], k1[MT][GR], c0[MT][GR], c1[MT][GR];  // K words of tokens r0 and r0 + 8, and their s and b
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const uint8_t *g0 = group(2 * u), *g1 = group(2 * u + 1);
        lds_words<GR>(g0 + (in(2 * u) + r0) * Q::kRow + t * GR * 4, k0[u]);
        lds_words<GR>(g1 + (in(2 * u + 1) + r0) * Q::kRow + t * GR * 4, k1[u]);
        lds_words<GR>(g0 + Q::k_params(TB) + (in(2 * u) + r0) * Q::kParamRow, c0[u]);
        lds_words<GR>(g1 + Q::k_params(TB) + (in(2 * u + 1) + r0) * Q::kParamRow, c1[u]);
        x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < GR; ++j)
#pragma unroll
        for (int u = 0; u < MT; ++u) {  // the two blocks' accumulations in turn: neither waits for its last product
            const __half2 s0 = as_half2(c0[u][j >> 1]), b0 = as_half2(c0[u][(GR + j) >> 1]);
            const __half2 s1 = as_half2(c1[u][j >> 1]), b1 = as_half2(c1[u][(GR + j) >> 1]);
            const __half2 s0j = (j & 1) ? __high2half2(s0) : __low2half2(s0), b0j = (j & 1) ? __high2half2(b0) : __low2half2(b0);
            const __half2 s1j = (j & 1) ? __high2half2(s1) : __low2half2(s1), b1j = (j & 1) ? __high2half2(b1) : __low2half2(b1);
            mma_16816(x[u], quant_value(quant_field<0>(k0[u][j]), s0j, b0j), quant_value(quant_field<0>(k1[u][j]), s1j, b1j),
                      quant_value(quant_field<1>(k0[u][j]), s0j, b0j), quant_value(quant_field<1>(k1[u][j]), s1j, b1j),
                      qf[2 * j][0], qf[2 * j][1]);
            mma_16816(x[u], quant_value(quant_field<2>(k0[u][j]), s0j, b0j), quant_value(quant_field<2>(k1[u][j]), s1j, b1j),
                      quant_value(quant_field<3>(k0[u][j]), s0j, b0j), quant_value(quant_field<3>(k1[u][j]), s1j, b1j),
                      qf[2 * j + 1][0], qf[2 * j + 1][1]);
        }
    uint32_t P[1][MT][2];
    softmax_step<D, MT, Weights::kRounded>(st, x, vis, OneScale{sl2}, P);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        uint32_t v0[GR], v1[GR], c0[2 * GR], c1[2 * GR];
        const uint8_t *g0 = group(2 * u), *g1 = group(2 * u + 1);
        lds_words<GR>(g0 + Q::v_codes(TB) + (in(2 * u) >> 3) * Q::kVGroup + lane * GR * 4, v0);
        lds_words<GR>(g1 + Q::v_codes(TB) + (in(2 * u + 1) >> 3) * Q::kVGroup + lane * GR * 4, v1);
        g0 += Q::v_params(TB) + (in(2 * u) >> 3) * Q::kVParamGroup + t * GR * 8;
        g1 += Q::v_params(TB) + (in(2 * u + 1) >> 3) * Q::kVParamGroup + t * GR * 8;
#pragma unroll
        for (int j = 0; j < GR; j += 2) {
            const uint4 a = *reinterpret_cast<const uint4 *>(g0 + j * 8), b = *reinterpret_cast<const uint4 *>(g1 + j * 8);
            c0[2 * j] = a.x, c0[2 * j + 1] = a.y, c0[2 * j + 2] = a.z, c0[2 * j + 3] = a.w;
            c1[2 * j] = b.x, c1[2 * j + 1] = b.y, c1[2 * j + 2] = b.z, c1[2 * j + 3] = b.w;
        }
        if (vis != 0xffffffffu) {
            // masked tokens' params become 0, and with them their values, whatever the page holds
            const uint32_t a = vis >> (16 * u + 2 * t), b = a >> 8;
            const uint32_t keep0 = ((a & 1) ? 0xffffu : 0u) | ((a & 2) ? 0xffff0000u : 0u);
            const uint32_t keep1 = ((b & 1) ? 0xffffu : 0u) | ((b & 2) ? 0xffff0000u : 0u);
#pragma unroll
            for (int j = 0; j < 2 * GR; ++j) {
                c0[j] &= keep0;
                c1[j] &= keep1;
            }
        }
#pragma unroll
        for (int j = 0; j < GR; ++j) {
            const __half2 s0 = as_half2(c0[2 * j]), b0 = as_half2(c0[2 * j + 1]);
            const __half2 s1 = as_half2(c1[2 * j]), b1 = as_half2(c1[2 * j + 1]);
            mma_16816(st.O[2 * j], quant_value(quant_field<0>(v0[j]), s0, b0), quant_value(quant_field<1>(v0[j]), s0, b0),
                      quant_value(quant_field<0>(v1[j]), s1, b1), quant_value(quant_field<1>(v1[j]), s1, b1), P[0][u][0], P[0][u][1]);
            mma_16816(st.O[2 * j + 1], quant_value(quant_field<2>(v0[j]), s0, b0), quant_value(quant_field<3>(v0[j]), s0, b0),
                      quant_value(quant_field<2>(v1[j]), s1, b1), quant_value(quant_field<3>(v1[j]), s1, b1), P[0][u][0], P[0][u][1]);
        }
    }
}

// Bits of 32 tokens in the order of the rows that byte_tile() gives them: row
// r < 8 of 16 is token 2 r, row r + 8 the next.
__device__ __forceinline__ uint32_t byte_rows(uint32_t vis)
{
    if (vis == 0xffffffffu)
        return vis;
    // even tokens to the low byte, odd ones to the high one, of either half
    uint32_t x = vis, y = (x ^ (x >> 1)) & 0x22222222u;
    x ^= y ^ (y << 1);
    y = (x ^ (x >> 2)) & 0x0c0c0c0cu;
    x ^= y ^ (y << 2);
    y = (x ^ (x >> 4)) & 0x00f000f0u;
    return x ^ y ^ (y << 4);
}

// One tile of the 8-bit cache, of which this warp takes 32 tokens, two blocks of
// 16 for the tensor cores.  Of K, a lane reads 16 bytes, dims 64 c + 16 t .. of a
// token, whose words w are its share of A in step 4 c + w: dims 64 c + 16 t + 4 w
// and the next at k = 2 t, 2 t + 1, the other two at 2 t + 8, 2 t + 9 (q's fragments
// follow that).  Row r0 < 8 of K's A is token 2 r0, row r0 + 8 the next: the rows
// that lanes read at a time have different halves swapped.  Of V, a lane reads
// tokens 4 t .. 4 t + 3 of dims 4 (r0 + 8 c) ..; the weights, which come as those of
// tokens 4 t and 4 t + 2, and of the two others, change places to match.
// K's scale is a factor of the scores.  V's multiplies what a block's codes add to
// O, in fp32; in pages of 8, where a product is over two blocks, the codes, whose
// values are exact fp16 numbers.  (In the weights' exponents, and out of the sum
// again, it costs 1% less, 3% in pages of 8, but then the fp16 weights have to span
// the scales too: beside a block of a scale 2^31 times as great, values were lost.)
template <int D, int KIND>
__device__ __forceinline__ void byte_tile(State<D> &st, const uint32_t (&qf)[D / 16][2], const uint8_t *kv, uint32_t vis, int w, float sl2)
{
    constexpr int FMT = kFormat<KIND>, TBL = kBlockLog2<KIND>, TB = 1 << TBL, LG = TBL < 4 ? TBL : 4, MT = 2, NC = D / 64;
    constexpr int BYTES = byte_block_bytes(TB, D);
    const int lane = threadIdx.x & 31, r0 = lane >> 2, t = lane & 3;
    const int tok = 2 * r0;  // of row r0
    BlockScales<MT> sc;
    float x[MT][4], sv[MT];
    uint4 kc[MT][2][NC];
    // V's scale; one outside the format's range, which only masked tokens' blocks may have, as the nearest in it
    auto scale_of = [](uint32_t s) { return byte_pow2(byte_exponent<FMT>(__uint_as_float(s))); };
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int at = 32 * w + 16 * u + (LG == 3 ? tok & 8 : 0), r = at & (TB - 1);  // this lane's scale block
        const uint8_t *blk = kv + (at >> TBL) * BYTES;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            // both tokens of a lane have the same halves swapped
            const int in = byte_k_at<D>(r + (LG == 3 ? tok & 7 : tok), 64 * c + 16 * t);
            kc[u][0][c] = *reinterpret_cast<const uint4 *>(blk + in);
            kc[u][1][c] = *reinterpret_cast<const uint4 *>(blk + in + D);
        }
        const uint2 s = *reinterpret_cast<const uint2 *>(blk + byte_scale_part<D>(TB, r, LG));
        // a lane's tokens are both in its block; where V's scale is NaN their scores are too
        sc.k[u] = (s.y & 0x7fffffffu) > 0x7f800000u ? __uint_as_float(0x7fffffffu) : sl2 * __uint_as_float(s.x);
        sv[u] = scale_of(s.y);
        x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < MT; ++u) {  // the two blocks' accumulations in turn: neither waits for its last product
                auto word = [&](const uint4 &v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
                uint32_t a0, a1, a2, a3;
                byte_numbers<FMT>(word(kc[u][0][c]), a0, a2);
                byte_numbers<FMT>(word(kc[u][1][c]), a1, a3);
                mma_16816(x[u], a0, a1, a2, a3, qf[4 * c + j][0], qf[4 * c + j][1]);
            }
    constexpr Weights W = kWeights<KIND>;
    uint32_t P[kProducts<W>][MT][2];
    softmax_step<D, MT, W>(st, x, byte_rows(vis), sc, P);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int at = 32 * w + 16 * u + (LG == 3 ? 8 * (t >> 1) : 0), r = at & (TB - 1);
        const uint8_t *vp = kv + (at >> TBL) * BYTES + byte_v_part<D>(TB, r, LG);
        uint32_t p[kProducts<W>][2];
#pragma unroll
        for (int z = 0; z < kProducts<W>; ++z) {
            p[z][0] = __byte_perm(P[z][u][0], P[z][u][1], 0x5410);
            p[z][1] = __byte_perm(P[z][u][0], P[z][u][1], 0x7632);
        }
        // masked tokens' bytes may be any: a weight of 0 does not hide an e4m3 NaN, nor an infinity that a scale makes
        uint32_t keep = 0xffffffffu;
        if ((FMT == kE4m3 || LG == 3) && vis != 0xffffffffu)
            keep = ((vis >> (16 * u + 4 * t) & 15u) * 0x00204081u & 0x01010101u) * 255u;
        __half2 s2;
        if constexpr (LG == 3)
            s2 = __float2half2_rn(scale_of(*reinterpret_cast<const uint32_t *>(kv + (at >> TBL) * BYTES + byte_scale_part<D>(TB, r, LG) + 4)));
        auto values = [&](uint32_t w, uint32_t &lo, uint32_t &hi) {
            byte_numbers<FMT>(w & keep, lo, hi);
            if constexpr (LG == 3) {
                lo = byte_word(__hmul2(byte_half2(lo), s2));
                hi = byte_word(__hmul2(byte_half2(hi), s2));
            }
        };
        auto products = [&](float (&o)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int z = kProducts<W> - 1; z >= 0; --z)
                mma_16816(o, a0, a1, a2, a3, p[z][0], p[z][1]);
        };
        auto add = [&](float (&O)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            if constexpr (LG == 3) {
                products(O, a0, a1, a2, a3);
            } else {
                float o[4] = {0.f, 0.f, 0.f, 0.f};
                products(o, a0, a1, a2, a3);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    O[e] = fmaf(o[e], sv[u], O[e]);
            }
        };
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(vp + byte_v_at(r0 + 8 * c, LG == 3 ? t & 1 : t, LG));
            uint32_t a0, a1, a2, a3;
            values(v.x, a0, a2);
            values(v.y, a1, a3);
            add(st.O[2 * c], a0, a1, a2, a3);
            values(v.z, a0, a2);
            values(v.w, a1, a3);
            add(st.O[2 * c + 1], a0, a1, a2, a3);
        }
    }
}

// Loads that a lane of a merge has in flight, and the pieces of such a batch.
constexpr int kBatch = 8;
template <int D>
__device__ __forceinline__ int merge_batch(int G)
{
    return (G > kCW ? kBatch / 2 : kBatch) * (128 / D);
}

// The states of n pieces of a (row, head), merged in piece order: piece `at` and
// those `step`, 2 step, .. further on, whose slots follow from the (row, head)'s
// first segment c0.  The result goes to o and lse (unit >= 0) or to the slot of
// piece `at`.  A warp takes a head at a time, or two when there are more heads
// than warps, and with d = 64 two pieces side by side.  Up to 32 pieces: one lane
// each for the maxima and sums, and their accumulators kBatch loads deep, issued
// beside those: each batch is an L2 round trip.
template <int D>
__device__ __forceinline__ void merge_pieces(const AttendParams &p, int unit, int c0, int first, int step, int n)
{
    constexpr int LP = D / 4, NP = 32 / LP;  // lanes per piece, pieces side by side
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LP, at = lane % LP;
    const int64_t slots = 2 * kAttnMaxSegs;
    float *pm = p.partials + slots * p.G * D, *pl = pm + slots * p.G;
    auto state = [&](int j, int g) {
        const int x = first + j * step;
        return (x == 0 ? 2 * c0 + 1 : 2 * (c0 + x)) * p.G + g;
    };
    auto merge = [&](auto heads) {  // heads w, w + 4, .. heads of them
        constexpr int NH = decltype(heads)::value, kPer = kBatch / NH;
        float M[NH], L[NH];
        float4 acc[NH];
#pragma unroll
        for (int q = 0; q < NH; ++q) {
            M[q] = kNoMax;
            L[q] = 0.f;
            acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int nj = min(n - j0, 32);
            float mj[NH], lj[NH], wj[NH];
#pragma unroll
            for (int q = 0; q < NH; ++q) {
                const int g = w + kCW * q;
                mj[q] = kNoMax;
                lj[q] = wj[q] = 0.f;
                if (lane < nj && g < p.G) {
                    mj[q] = __ldcg(pm + state(j0 + lane, g));
                    lj[q] = __ldcg(pl + state(j0 + lane, g));
                }
            }
            for (int b = 0; b < nj; b += kPer * NP) {
                float4 x[kPer][NH];
#pragma unroll
                for (int u = 0; u < kPer; ++u)
#pragma unroll
                    for (int q = 0; q < NH; ++q) {
                        const int g = w + kCW * q, j = b + u * NP + sub;
                        x[u][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (j < nj && g < p.G)
                            x[u][q] = __ldcg(reinterpret_cast<const float4 *>(p.partials + (int64_t)state(j0 + j, g) * D) + at);
                    }
#pragma unroll
                for (int q = 0; q < NH; ++q) {
                    if (b == 0) {
                        float mn = fmaxf(mj[q], M[q]);
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                        const float f = ex2(M[q] - mn);
                        M[q] = mn;
                        wj[q] = ex2(mj[q] - mn);
                        L[q] = L[q] * f + lj[q] * wj[q];  // this lane's share
                        acc[q].x *= f, acc[q].y *= f, acc[q].z *= f, acc[q].w *= f;
                    }
#pragma unroll
                    for (int u = 0; u < kPer; ++u) {
                        const float a = __shfl_sync(0xffffffffu, wj[q], (b + u * NP + sub) & 31);
                        acc[q].x = fmaf(x[u][q].x, a, acc[q].x), acc[q].y = fmaf(x[u][q].y, a, acc[q].y);
                        acc[q].z = fmaf(x[u][q].z, a, acc[q].z), acc[q].w = fmaf(x[u][q].w, a, acc[q].w);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < NH; ++q) {
            const int g = w + kCW * q;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                L[q] += __shfl_xor_sync(0xffffffffu, L[q], o);
                if (o >= LP) {
                    acc[q].x += __shfl_xor_sync(0xffffffffu, acc[q].x, o);
                    acc[q].y += __shfl_xor_sync(0xffffffffu, acc[q].y, o);
                    acc[q].z += __shfl_xor_sync(0xffffffffu, acc[q].z, o);
                    acc[q].w += __shfl_xor_sync(0xffffffffu, acc[q].w, o);
                }
            }
            if (g >= p.G)
                continue;
            if (unit < 0) {
                if (sub == 0)
                    __stcg(reinterpret_cast<float4 *>(p.partials + (int64_t)state(0, g) * D) + at, acc[q]);
                if (lane == 0) {
                    __stcg(pm + state(0, g), M[q]);
                    __stcg(pl + state(0, g), L[q]);
                }
                continue;
            }
            const float inv = over_sum(L[q]);
            const int64_t oh = (int64_t)unit * p.G + g;  // unit = row * Hkv + head
            if (sub == 0)
                *reinterpret_cast<uint2 *>(p.o + oh * D + at * 4) =
                    make_uint2(out_half2(acc[q].x * inv, acc[q].y * inv), out_half2(acc[q].z * inv, acc[q].w * inv));
            if (p.lse && lane == 0)
                p.lse[oh] = (M[q] + log2f(L[q])) * kLn2;
        }
    };
    if (p.G > kCW)
        merge(std::integral_constant<int, 2>());
    else
        merge(std::integral_constant<int, 1>());
}

// Batches of a merge up to which one CTA does all of it; beyond, groups of pieces
// are merged first, by the CTAs that finish them.  One row of 32k tokens over the
// 4-bit cache, one merge against two levels: 57 pieces in 15 batches, 21.5 and
// 19.1 us; in 8, 18.2 and 17.3 us; one KV head alone (456 in 114) 37.4 and 14.2
// us; over fp16 pages 38 in 5, 17.7 and 19.0 us.
constexpr int kMaxBatches = 6;

// A piece's end: the four warps' states become one, each warp merging its
// quarter of the dims, and go to o and lse (slot < 0), to the piece's slot or, in
// a cluster, to the CTAs that merge its dims.
template <int D, int KIND, bool CLUSTER>
__device__ __forceinline__ bool finish_piece(const AttendParams &p, State<D> &st, uint8_t *stage, float *red, int *s_last,
                                             const Inbox<D> &inbox, uint32_t cbar, uint32_t &cph, uint32_t empty, int4 mt, int4 mt2)
{
    constexpr int KS = D / 16, KQ = KS / kCW;  // 16-dim blocks a warp merges
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = lane >> 2, h0 = 2 * (lane & 3);
    const int G = p.G;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
        st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    if (lane < 4) {
        red[w * 16 + h0] = st.m0;
        red[w * 16 + h0 + 1] = st.m1;
        red[w * 16 + 8 + h0] = st.l0;
        red[w * 16 + 8 + h0 + 1] = st.l1;
    }
    if (!meet(cbar, cph))  // every warp has read the stage's tile
        return false;
    // block x of warp w goes to its owner x / KQ: [owner][writer slot][block][lane] float4
    float4 *ex = reinterpret_cast<float4 *>(stage);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
        const int own = x / KQ;
        if (own != w)
            ex[((own * (kCW - 1) + (w - (w > own))) * KQ + x % KQ) * 32 + lane] =
                make_float4(st.O[x][0], st.O[x][1], st.O[x][2], st.O[x][3]);
    }
    if (!meet(cbar, cph))
        return false;
    float M0 = kNoMax, M1 = kNoMax, L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int v = 0; v < kCW; ++v) {
        M0 = fmaxf(M0, red[v * 16 + h0]);
        M1 = fmaxf(M1, red[v * 16 + h0 + 1]);
    }
    float f0[kCW], f1[kCW];
#pragma unroll
    for (int v = 0; v < kCW; ++v) {
        f0[v] = ex2(red[v * 16 + h0] - M0);
        f1[v] = ex2(red[v * 16 + h0 + 1] - M1);
        L0 += red[v * 16 + 8 + h0] * f0[v];
        L1 += red[v * 16 + 8 + h0 + 1] * f1[v];
    }
    float R[KQ][4];
#pragma unroll
    for (int y = 0; y < KQ; ++y) {
        R[y][0] = R[y][1] = R[y][2] = R[y][3] = 0.f;
#pragma unroll
        for (int v = 0; v < kCW; ++v) {
            float4 s;
            if (v == w) {
#pragma unroll
                for (int ww = 0; ww < kCW; ++ww)  // static indexing of the register state
                    if (ww == w)
                        s = make_float4(st.O[ww * KQ + y][0], st.O[ww * KQ + y][1], st.O[ww * KQ + y][2], st.O[ww * KQ + y][3]);
            } else {
                s = ex[((w * (kCW - 1) + (v - (v > w))) * KQ + y) * 32 + lane];
            }
            R[y][0] += s.x * f0[v];
            R[y][1] += s.y * f1[v];
            R[y][2] += s.z * f0[v];
            R[y][3] += s.w * f1[v];
        }
    }
    fence_proxy_async_smem();  // the stage is refilled by bulk copies
    __syncwarp();
    if (lane == 0)
        mbar_arrive(empty);
    if constexpr (kWeights<KIND> == Weights::kBeside)  // what the remainders in heads 4 .. 7 add to heads 0 .. 3
#pragma unroll
        for (int y = 0; y < KQ; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                R[y][e] += __shfl_xor_sync(0xffffffffu, R[y][e], 2);
    const int unit = mt.x, slot = mt.w;
    const bool ok0 = h0 < G, ok1 = h0 + 1 < G;
    // over the 8-bit cache a lane's dims are neighbours: the accumulators of heads h0 and h0 + 1 from dim dr on
    constexpr bool BYTE = kIs8Bit<KIND>;
    using Run = std::conditional_t<KQ == 2, float4, float2>;
    const int dr = dim_of<KIND>(w * KQ, r0);
    auto run = [&](int e) {
        if constexpr (KQ == 2)
            return make_float4(R[0][e], R[0][2 + e], R[1][e], R[1][2 + e]);
        else
            return make_float2(R[0][e], R[0][2 + e]);
    };
    if (CLUSTER && slot >= 0 && BYTE) {
        inbox.acc(h0, dr, run(0));
        inbox.acc(h0 + 1, dr, run(1));
        if (w == 0)
            inbox.sums(h0, r0, M0, M1, L0, L1);
        return true;
    }
    if (CLUSTER && slot >= 0) {
#pragma unroll
        for (int y = 0; y < KQ; ++y) {
            const int d0 = dim_of<KIND>(w * KQ + y, r0);
            inbox.acc(h0, d0, R[y][0]);
            inbox.acc(h0, d0 + kDimStep<KIND>, R[y][2]);
            inbox.acc(h0 + 1, d0, R[y][1]);
            inbox.acc(h0 + 1, d0 + kDimStep<KIND>, R[y][3]);
        }
        if (w == 0)
            inbox.sums(h0, r0, M0, M1, L0, L1);
        return true;
    }
    if (CLUSTER || slot < 0) {
        const float i0 = over_sum(L0), i1 = over_sum(L1);
        __half *out = p.o + (int64_t)unit * G * D;
        auto give = [&](int h, Run v, float inv) {
            if constexpr (KQ == 2)
                *reinterpret_cast<uint2 *>(out + h * D + dr) = make_uint2(out_half2(v.x * inv, v.y * inv), out_half2(v.z * inv, v.w * inv));
            else
                *reinterpret_cast<uint32_t *>(out + h * D + dr) = out_half2(v.x * inv, v.y * inv);
        };
        if (BYTE && ok0)
            give(h0, run(0), i0);
        if (BYTE && ok1)
            give(h0 + 1, run(1), i1);
#pragma unroll
        for (int y = 0; y < (BYTE ? 0 : KQ); ++y) {
            const int d0 = dim_of<KIND>(w * KQ + y, r0);
            if (ok0) {
                out[h0 * D + d0] = out_half(R[y][0] * i0);
                out[h0 * D + d0 + kDimStep<KIND>] = out_half(R[y][2] * i0);
            }
            if (ok1) {
                out[(h0 + 1) * D + d0] = out_half(R[y][1] * i1);
                out[(h0 + 1) * D + d0 + kDimStep<KIND>] = out_half(R[y][3] * i1);
            }
        }
        if (p.lse && w == 0 && lane < 4) {
            if (ok0)
                p.lse[(int64_t)unit * G + h0] = (M0 + log2f(L0)) * kLn2;
            if (ok1)
                p.lse[(int64_t)unit * G + h0 + 1] = (M1 + log2f(L1)) * kLn2;
        }
        return true;
    }
    {
        float *acc = p.partials + (int64_t)slot * G * D;
        if (BYTE && ok0)
            *reinterpret_cast<Run *>(acc + h0 * D + dr) = run(0);
        if (BYTE && ok1)
            *reinterpret_cast<Run *>(acc + (h0 + 1) * D + dr) = run(1);
#pragma unroll
        for (int y = 0; y < (BYTE ? 0 : KQ); ++y) {
            const int d0 = dim_of<KIND>(w * KQ + y, r0);
            if (ok0) {
                acc[h0 * D + d0] = R[y][0];
                acc[h0 * D + d0 + kDimStep<KIND>] = R[y][2];
            }
            if (ok1) {
                acc[(h0 + 1) * D + d0] = R[y][1];
                acc[(h0 + 1) * D + d0 + kDimStep<KIND>] = R[y][3];
            }
        }
        if (w == 0 && lane < 4) {
            const int64_t slots = 2 * kAttnMaxSegs;
            float *pm = p.partials + slots * G * D + (int64_t)slot * G, *pl = pm + slots * G;
            if (ok0) {
                pm[h0] = M0;
                pl[h0] = L0;
            }
            if (ok1) {
                pm[h0 + 1] = M1;
                pl[h0 + 1] = L1;
            }
        }
    }
    const int c0 = mt2.w & 0xffff, n = (mt2.w >> 16) + 1, at = (slot >> 1) - c0;
    // many pieces: groups of 2^k first, k such that there are as many groups at most
    int k = 0;
    if (n > kMaxBatches * merge_batch<D>(p.G))
        for (k = 3; n > 1 << (2 * k); ++k) {
        }
    for (int level = k == 0 ? 1 : 0; level < 2; ++level) {
        const int first = level == 0 ? at >> k << k : 0, step = level == 0 ? 1 : 1 << k;
        const int members = level == 0 ? min(1 << k, n - first) : (n + step - 1) >> k;
        // a group's counter is that of a later segment, in which no (row, head) begins
        int *counter = p.counters + c0 + (level == 0 ? 1 + (at >> k) : 0);
        // the barrier orders the warps' states before thread 0's arrival, whose
        // release and acquire carry that order to the other CTAs of the unit
        if (!meet(cbar, cph))
            return false;
        if (threadIdx.x == 0) {
            int before;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
            *s_last = before == members - 1;
            if (before == members - 1)
                *counter = 0;  // ready for the next launch
        }
        if (!meet(cbar, cph))
            return false;
        if (!*s_last)
            return true;
        merge_pieces<D>(p, level == 0 ? -1 : unit, c0, first, step, members);
    }
    return true;
}

template <int D, int KIND, bool CLUSTER>
__device__ __forceinline__ void run_consumer(const AttendParams &p, uint32_t sbase, uint8_t *basep, const int4 *meta,
                                             uint32_t full0, uint32_t empty0, uint32_t cbar, int *s_last)
{
    using L = Layout<D, KIND, CLUSTER>;
    constexpr int KS = D / 16;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = lane >> 2;
    // two buffers: a warp may reach the next piece's end while another still reads this one's
    float *red = reinterpret_cast<float *>(basep + L::kRedOff);
    int parity = 0;
    State<D> st;
    st.clear();
    uint32_t qf[KS][2];
    int stage = 0;
    uint32_t ph = 0, cph = 0;
    const Inbox<D> inbox = {sbase + L::kStateOff, p.cluster_log2, (int)blockIdx.x & ((1 << p.cluster_log2) - 1)};
    for (;;) {
        if (!__all_sync(0xffffffffu, mbar_wait(full0 + stage * 8, ph, kWaitNs))) {
            report_error(p.ws, kErrTimeout, (int)blockIdx.x, stage, 2);
            return;
        }
        const int4 mt = meta[2 * stage];
        if (mt.z & kEnd) {
            if (CLUSTER && p.cluster_log2 > 0 && w == 0)  // a CTA without a tile
                inbox.sums(2 * (lane & 3), r0, kNoMax, kNoMax, kNoTiles, kNoTiles);
            break;
        }
        uint8_t *sp = basep + stage * L::kStageBytes;
        if (mt.z & kFirst) {
            const uint8_t *qs = sp + L::kKvBytes;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                qf[x][0] = qf[x][1] = 0u;
                const int g = kWeights<KIND> == Weights::kBeside ? r0 & (kMaxG / 2 - 1) : r0;  // this column's head
                if (g < p.G) {
                    const uint32_t *row = reinterpret_cast<const uint32_t *>(qs + g * D * 2);
                    if constexpr (L::BYTE) {
                        // dims 4 w + 16 t + 64 c .. of step x = 4 c + w (see byte_tile())
                        const uint2 q4 = *reinterpret_cast<const uint2 *>(row + 32 * (x >> 2) + 8 * (lane & 3) + 2 * (x & 3));
                        qf[x][0] = q4.x;
                        qf[x][1] = q4.y;
                    } else {
                        qf[x][0] = row[8 * x + (lane & 3)];
                        qf[x][1] = row[8 * x + 4 + (lane & 3)];
                    }
                }
            }
        }
        constexpr int TW = 16 * L::MT;  // tokens of the tile a warp takes at a time
        int4 mt2 = make_int4(0, 0, 0, 0);
        if (mt.z & (kMasked | kLast))
            mt2 = meta[2 * stage + 1];
#pragma unroll 1
        for (int part = w * L::NT; part < (w + 1) * L::NT; ++part) {
            uint32_t vis = 0xffffffffu >> (32 - TW);
            if (mt.z & kMasked)
                vis = __ballot_sync(0xffffffffu, lane < TW && visible(mt.y + TW * part + lane, mt2.x, mt2.y, mt2.z));
            if (!vis)
                continue;
            if constexpr (L::BYTE)
                byte_tile<D, KIND>(st, qf, sp, vis, part, p.scale_log2);
            else if constexpr (L::QUANT)
                quant_tile<D, kBlockLog2<KIND>>(st, qf, sp, vis, part, p.scale_log2);
            else
                fp16_tile<D>(st, qf, sbase + stage * L::kStageBytes, sp, vis, part, p.tb_log2, p.scale_log2);
        }
        __syncwarp();
        if (mt.z & kLast) {
            if (!finish_piece<D, KIND, CLUSTER>(p, st, sp, red + parity * kCW * 2 * kMaxG, s_last, inbox, cbar, cph,
                                                empty0 + stage * 8, mt, mt2)) {
                report_error(p.ws, kErrTimeout, (int)blockIdx.x, stage, 3);
                return;
            }
            if (CLUSTER)
                break;  // the only piece
            st.clear();
            parity ^= 1;
        } else if (lane == 0) {
            mbar_arrive(empty0 + stage * 8);
        }
        if (++stage == L::kStages) {
            stage = 0;
            ph ^= 1;
        }
    }
    // rows that see no token (a cluster's merge knows its own)
    for (int i = CLUSTER && p.cluster_log2 > 0 ? p.B : (int)blockIdx.x; i < p.B; i += gridDim.x) {
        if (row_span<L::kTile>(p, p.seq_lens[i]).T > 0)
            continue;
        int4 *out = reinterpret_cast<int4 *>(p.o + (int64_t)i * p.Hq * D);
        for (int x = threadIdx.x; x < p.Hq * D / 8; x += 32 * kCW)
            out[x] = make_int4(0, 0, 0, 0);
        if (p.lse)
            for (int x = threadIdx.x; x < p.Hq; x += 32 * kCW)
                p.lse[(int64_t)i * p.Hq + x] = -INFINITY;
    }
}

// The states of a cluster's CTAs become the (row, head)'s o and lse, each CTA
// taking its share of the dims, a thread four of them, from what it was sent: no
// other CTA's memory is looked at, so none has to wait for the others' end, and
// the way there is over when the cluster has met.  (Reading the others' states took
// 0.3 to 0.7 us more: 16 rows of 1k of the 8-bit cache 9.7 us, now 9.0; one row of 1k
// of the 4-bit cache 5.4, now 5.0.  Sent one dim at a time, the 8-bit cache's, four
// neighbouring ones a lane, took 1.8 us more in clusters of 16.)
template <int D>
__device__ __forceinline__ void merge_cluster(const AttendParams &p, const float *inbox)
{
    const int cl = p.cluster_log2, n = 1 << cl, per = (D / 4) >> cl;  // float4s of a head in this CTA's share
    if (cl == 0)
        return;  // the one CTA has written o and lse
    const int unit = (int)blockIdx.x >> cl, r = (int)blockIdx.x - (unit << cl);
    const float *ms = inbox + kMaxG * D, *ls = ms + (kMaxG << cl);
    cluster_arrive();
    cluster_wait();  // everything is there
    for (int x = threadIdx.x; x < p.G * per; x += kThreads) {
        const int g = x / per, q = x - g * per, d = 4 * (r * per + q);
        float M = kNoMax, Ls = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
            if (c < n)
                M = fmaxf(M, ms[c * kMaxG + g]);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c >= n)
                continue;
            const float l = ls[c * kMaxG + g], f = ex2(ms[c * kMaxG + g] - M);
            if (l != kNoTiles) {  // else nothing else was sent
                const float4 a = reinterpret_cast<const float4 *>(inbox)[(c * kMaxG + g) * per + q];
                Ls += l * f;
                A.x += a.x * f, A.y += a.y * f, A.z += a.z * f, A.w += a.w * f;
            }
        }
        const int64_t oh = (int64_t)unit * p.G + g;
        const float inv = over_sum(Ls);
        *reinterpret_cast<uint2 *>(p.o + oh * D + d) = make_uint2(out_half2(A.x * inv, A.y * inv), out_half2(A.z * inv, A.w * inv));
        if (p.lse && d == 0)
            p.lse[oh] = (M + log2f(Ls)) * kLn2;
    }
}

template <int D, int KIND, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, Layout<D, KIND, CLUSTER>::kCtasPerSm)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttendParams p)
{
    using L = Layout<D, KIND, CLUSTER>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_last;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *basep = smem_raw + (sbase - raw);
    int4 *meta = reinterpret_cast<int4 *>(basep + L::kMetaOff);
    const uint32_t full0 = sbase + L::kBarOff, empty0 = full0 + L::kStages * 8, cbar = empty0 + L::kStages * 8;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full0 + s * 8, 1);
            mbar_init(empty0 + s * 8, kCW);
        }
        mbar_init(cbar, kCW);
        fence_mbar_init();
    }
    if (CLUSTER && p.cluster_log2 > 0)
        cluster_arrive();  // here: the others may send
    if (!L::QUANT && threadIdx.x == 32 * kCW) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    __syncthreads();
    // The lengths, the table entries they lead to and the pages behind those are
    // three DRAM latencies in a row: the CTAs bring the table into L2 together
    // while the lengths are on their way (a hint: nothing is read).
    if (threadIdx.x < kTableLines) {
        const int64_t line = (int64_t)blockIdx.x + (int64_t)threadIdx.x * gridDim.x;
        if (line * 128 < (int64_t)p.B * p.bt_stride * 4)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p.bt) + line * 128));
    }
    if constexpr (L::BYTE)
        if (threadIdx.x < 32)
            hint_first_tiles<D, KIND, CLUSTER>(p);
    pdl_wait();
    pdl_trigger();
    if (CLUSTER && p.cluster_log2 > 0)
        cluster_wait();
    if (threadIdx.x >= 32 * kCW)
        run_producer<D, KIND, CLUSTER>(&tmK, &tmV, p, sbase, basep, meta, full0, empty0);
    else
        run_consumer<D, KIND, CLUSTER>(p, sbase, basep, meta, full0, empty0, cbar, &s_last);
    if constexpr (CLUSTER)
        merge_cluster<D>(p, reinterpret_cast<const float *>(basep + L::kStateOff));
}

// What is asked of a device once per kernel: whether its shared memory limit is
// raised, and how many clusters of 2^k CTAs it holds at once (plus one).
struct KernelOnDevice {
    std::atomic<int> ready{0};
    std::atomic<int> clusters[5] = {};
};

template <int D, int KIND, bool CLUSTER>
cudaError_t prepare(KernelOnDevice *&k)
{
    static KernelOnDevice on[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    k = &on[dev & 63];
    if (k->ready.load(std::memory_order_acquire))
        return cudaSuccess;
    auto kern = attend_kernel<D, KIND, CLUSTER>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D, KIND, CLUSTER>::kAlloc);
    if (e == cudaSuccess && CLUSTER)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        k->ready.store(1, std::memory_order_release);
    return e;
}

struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(int64_t grid, int smem, int cluster, cudaStream_t s)
    {
        cfg.gridDim = dim3((unsigned)(grid > 0 ? grid : 1));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 0 ? 2 : 1;
    }
};

// Tiles of a (row, head) per CTA of its cluster up to which clusters are used:
// beyond, the line's equal runs gain more by their balance than the merge costs,
// sooner over the 4-bit cache, where an idle warp costs more.  d = 128, four
// query heads per KV head, clusters against runs.  fp16: 8 tiles, 8.2 and 10.7 us
// (eight rows of 512 .. 2048 tokens); 16 tiles, 12.2 and 13.0 us (eight), 11.3 and
// 13.0 us (32 rows); 17 tiles in windows, 19.4 and 21.5 us; 32 tiles, 29.6 and
// 31.2 us (32 rows), where a batch less even than these would lose.  4-bit, each
// CTA with an SM of its own: 4 tiles, 9.0 and 12.0 us (one row of 8k); 8 tiles,
// 13.3 and 14.4 us (one row of 16k), which two CTAs an SM of 4 tiles each better
// where there can be (two rows of 2k .. 8k, 7.9 and 8.5 us); 4 tiles, two an SM,
// 10.1 and 10.5 us (four rows), 8 tiles 15.0 and 13.4 us (eight).  8-bit, two an SM:
// 8 tiles, 16.0 and 18.6 us (eight rows of 4k); 10 tiles, 15.6 and 19.5 us (32 rows in a
// window of 1000); 16 tiles, 23.1 and 21.9 us (32 rows of 512 .. 2048).  With an SM of
// its own (e4m3, one KV head) a limit of 6, then 8, is right there too: with 3, then 4,
// 15 rows of 4k take 7.2 instead of 6.8 us (d = 64) and 16 of 8k 12.9 instead of 11.9 (d =
// 128); with 12, then 16, 37 rows of 4k 9.7 instead of 8.4 us (d = 64).
constexpr int kMaxTilesFp16 = 20;
constexpr int kMaxTilesOwn[2] = {6, 8};  // CTAs with an SM of their own: tried first, tried last
constexpr int kMaxTilesShared[2] = {4, 10};  // 4-bit, 8-bit
constexpr int kMaxTilesMany = 256;

// The line of tiles in runs, a CTA each.
template <int D, int KIND>
cudaError_t launch_runs(const CUtensorMap &tk, const CUtensorMap &tv, const AttendParams &p, int64_t tiles, int sms, cudaStream_t s)
{
    using L = Layout<D, KIND, false>;
    KernelOnDevice *k;
    cudaError_t e = prepare<D, KIND, false>(k);
    if (e != cudaSuccess)
        return e;
    int64_t grid = (int64_t)sms * L::kCtasPerSm;
    grid = grid < kAttnMaxCtas ? grid : kAttnMaxCtas;
    Launch l(grid < tiles ? grid : tiles, L::kAlloc, 0, s);
    return cudaLaunchKernelEx(&l.cfg, attend_kernel<D, KIND, false>, tk, tv, p);
}

template <int D, int KIND>
cudaError_t launch_one(const CUtensorMap &tk, const CUtensorMap &tv, AttendParams p, int sms, cudaStream_t s)
{
    using L = Layout<D, KIND, false>;
    using LC = Layout<D, KIND, true>;
    // the most tiles of a (row, head), by the table's width and by the window
    auto most_tiles = [&p](int64_t tile) {
        const int64_t by_len = (p.len_cap + tile - 1) / tile;
        const int64_t by_win = (p.window + tile - 1) / tile + 1 + (p.sinks + tile - 1) / tile;
        return by_len < by_win ? by_len : by_win;
    };
    const int64_t most = most_tiles(LC::kTile), units = (int64_t)p.B * p.Hkv, tiles = units * most_tiles(L::kTile);
    KernelOnDevice *k;
    // Up to 2^top CTAs a cluster, none without a tile in the longest rows and all
    // resident at once (a second wave costs more than the merge saves).  fp16: as
    // many as that.  4-bit: as many as leave each an SM of its own, more only
    // where their share is too long (two rows of 2057 tokens, 128 CTAs 5.3, 256
    // 6.6 us; four, d = 64, 128, 256 and 512 CTAs 6.0, 6.2 and 9.2 us).
    const int64_t room = (int64_t)sms * LC::kCtasPerSm;
    int top = 0, own = 0;
    while (top < kMaxClusterLog2 && (2ll << top) <= most && units << (top + 1) <= room)
        ++top;
    while (own < top && units << (own + 1) <= sms)
        ++own;
    const int n = top + 1, tries = most < 2 || units > room ? 0 : L::QUANT ? 2 * n : n;
    for (int t = 0; t < tries; ++t) {
        const int cl = L::QUANT ? own + t % n : top - t;
        const int limit = !L::QUANT ? kMaxTilesFp16 : units << cl <= sms ? kMaxTilesOwn[t / n] : kMaxTilesShared[L::BYTE];
        if (cl > top || most > (int64_t)limit << cl)
            continue;
        cudaError_t e = prepare<D, KIND, true>(k);
        if (e != cudaSuccess)
            return e;
        Launch l(units << cl, LC::kAlloc, 1 << cl, s);
        int fit = k->clusters[cl].load(std::memory_order_relaxed) - 1;
        if (fit < 0) {
            e = cudaOccupancyMaxActiveClusters(&fit, attend_kernel<D, KIND, true>, &l.cfg);
            if (e != cudaSuccess)
                return e;
            k->clusters[cl].store(fit + 1, std::memory_order_relaxed);
        }
        if (units > fit)
            continue;
        p.cluster_log2 = cl;
        return cudaLaunchKernelEx(&l.cfg, attend_kernel<D, KIND, true>, tk, tv, p);
    }
    // more (row, head)s than CTAs: their ends, which cost a CTA some microseconds without a load, are hidden by a third
    // CTA per SM better than by a third stage.  64 rows in a window of 4096 82.6 and 76.6 us, 300 rows of up to 8k 106.9
    // and 103.2 us, 100 of 100 15.0 and 13.2 us; but 64 rows of up to 60k 604 and 608 us, eight of up to 32k 42.4 and
    // 43.2 us
    if constexpr (L::BYTE && D == 128 && !(KIND & kMany))
        if (units > (int64_t)sms * L::kCtasPerSm && most <= kMaxTilesMany)
            return launch_runs<D, KIND + kMany>(tk, tv, p, tiles, sms, s);
    return launch_runs<D, KIND>(tk, tv, p, tiles, sms, s);
}

// The 8-bit cache's kernels, by the tokens of its blocks and the heads that share a KV head.
template <int D, int KIND>
cudaError_t launch_blocks(const AttendParams &p, int sms, cudaStream_t s)
{
    const CUtensorMap none = {};
    switch (p.tb_log2) {
    case 3:
        return launch_one<D, KIND + 3>(none, none, p, sms, s);
    case 4:
        return launch_one<D, KIND + 4>(none, none, p, sms, s);
    case 5:
        return launch_one<D, KIND + 5>(none, none, p, sms, s);
    default:
        return launch_one<D, KIND + 6>(none, none, p, sms, s);
    }
}
template <int D, int FMT>
cudaError_t launch_byte(const AttendParams &p, int sms, cudaStream_t s)
{
    constexpr int kKind = k8Bit + 16 * FMT;
    return p.G <= kMaxG / 2 ? launch_blocks<D, kKind + kFew>(p, sms, s) : launch_blocks<D, kKind>(p, sms, s);
}

}  // namespace
}  // namespace pkv
