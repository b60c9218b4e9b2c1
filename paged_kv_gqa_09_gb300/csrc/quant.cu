// quant.cu -- writing the 4-bit KV cache and reading it back.
//
// append: K and V of new tokens, packed [T][Hkv][d] fp16 with a stride between
// tokens, become codes in the pages their rows' block tables name, at positions
// seq_lens[i] .. ; lengths advance once every CTA has read them.
// read: tokens of the cache become packed fp16 K and V again.
#include "pkv_device.cuh"
#include "pkv_kernels.h"
#include "quant_format.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// Row of packed token x: the i with offsets[i] <= x < offsets[i + 1], or -1.
// (Without offsets a row has one token.)
__device__ __forceinline__ int row_of(const int32_t *offsets, int B, int x)
{
    if (!offsets)
        return x < B ? x : -1;
    int lo = 0, hi = B;  // the first i with offsets[i + 1] > x
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid + 1] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo < B && offsets[lo] <= x ? lo : -1;
}

// OR over the four lanes of a quad of four words each; lane f ends with word f.
__device__ __forceinline__ uint32_t quad_or_transpose(const uint32_t (&c)[4], int f)
{
    const bool up = (f & 2) != 0;
    uint32_t k0 = up ? c[2] : c[0], k1 = up ? c[3] : c[1];
    k0 |= __shfl_xor_sync(0xffffffffu, up ? c[0] : c[2], 2);
    k1 |= __shfl_xor_sync(0xffffffffu, up ? c[1] : c[3], 2);
    const uint32_t mine = (f & 1) ? k1 : k0;
    return mine | __shfl_xor_sync(0xffffffffu, (f & 1) ? k0 : k1, 1);
}

// Whether row i's n new tokens fit behind its N tokens; the reason goes to the
// error word when `report` is set.
__device__ __forceinline__ bool append_fits(const QuantAppendParams &p, int i, int N, int off, int n, bool report)
{
    if (n < 0 || off < 0 || (int64_t)off + n > p.T) {
        if (report)
            report_error(p.ws, kErrBadSpan, i, off, n);
        return false;
    }
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

template <int D>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const QuantAppendParams p)
{
    using Q = QuantLayout<D>;
    constexpr int CH = D / 8;  // threads of one (token, head, side), eight dims each
    __shared__ int s_last;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / CH;  // (token, head, side)
    const int c = threadIdx.x % CH, j = c >> 2, f = c & 3;
    const int side = (int)(unit & 1);
    const int64_t th = unit >> 1;
    const int x = (int)min(th / p.Hkv, (int64_t)0x7fffffff), h = (int)(th % p.Hkv);
    const int i = x < p.T ? row_of(p.offsets, p.B, x) : -1;
    bool live = i >= 0;
    int N = 0, pos = 0, page = 0;
    if (live) {
        N = p.seq_lens[i];
        const int off = p.offsets ? p.offsets[i] : i, n = p.offsets ? p.offsets[i + 1] - off : 1;
        live = append_fits(p, i, N, off, n, false);
        pos = N + (x - off);
    }
    if (live) {
        page = p.bt[(int64_t)i * p.bt_stride + (pos >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            report_error(p.ws, kErrBadPage, i, pos >> p.log2P, page);
            p.row_bad[i] = 1;
            live = false;
        }
    }
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live)
        raw = *reinterpret_cast<const uint4 *>((side ? p.v_new : p.k_new) + (int64_t)x * p.new_stride + h * D + c * 8);
    const __half2 *r2 = reinterpret_cast<const __half2 *>(&raw);
    __half2 mn = __hmin2_nan(__hmin2_nan(r2[0], r2[1]), __hmin2_nan(r2[2], r2[3]));
    __half2 mx = __hmax2_nan(__hmax2_nan(r2[0], r2[1]), __hmax2_nan(r2[2], r2[3]));
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const float lo0 = __half2float(__hmin_nan(mn.x, mn.y)), hi0 = __half2float(__hmax_nan(mx.x, mx.y));
    const bool nan = lo0 != lo0 || hi0 != hi0;
    const float lo = fminf(fmaxf(lo0, -kQuantLimit), kQuantLimit), hi = fminf(fmaxf(hi0, -kQuantLimit), kQuantLimit);
    __half s, b;
    quant_params(lo, hi, s, b);
    const float sf = __half2float(s), bf = __half2float(b), inv = sf > 0.f ? 1.f / sf : 0.f;
    int n[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const float v = __half2float(u & 1 ? r2[u >> 1].y : r2[u >> 1].x);
        n[u] = nan ? 0 : quant_code(fminf(fmaxf(v, -kQuantLimit), kQuantLimit), sf, bf, inv);
    }
    if (nan)
        s = b = __ushort_as_half(0x7fff);
    uint32_t w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)  // dims 2t and 2t+1 of the eight
        w[t] = quant_place(n[2 * t], f) | quant_place(n[2 * t + 1], f) << 16;
    const uint32_t word = quad_or_transpose(w, f);
    if (live) {
        const int tb = 1 << p.tb_log2, slot = pos & ((1 << p.log2P) - 1);
        const int r = slot & (tb - 1);
        uint8_t *blk = p.cache + ((int64_t)page * p.Hkv + h) * p.page_head_bytes +
                       (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
        if (side == 0) {
            reinterpret_cast<uint32_t *>(blk)[r * (D / 8) + f * Q::GR + j] = word;
            if (f < 2)
                reinterpret_cast<__half *>(blk + Q::k_params(tb))[r * 2 * Q::GR + f * Q::GR + j] = f ? b : s;
        } else {
            // this lane holds the halves g = 2 f, 2 f + 1 of its token
            const int t = (r & 7) >> 1, e = r & 1;
            uint16_t *vc = reinterpret_cast<uint16_t *>(blk + Q::v_codes(tb) + (r >> 3) * Q::kVGroup);
            vc[((2 * f * 4 + t) * Q::GR + j) * 2 + e] = (uint16_t)word;
            vc[(((2 * f + 1) * 4 + t) * Q::GR + j) * 2 + e] = (uint16_t)(word >> 16);
            if (f < 2)
                reinterpret_cast<__half *>(blk + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup)[((t * Q::GR + j) * 2 + f) * 2 + e] =
                    f ? b : s;
        }
    }
    // the last CTA to get here advances the lengths: every other one has read
    // them by then, and its rows' flags are set
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(&p.ws->append_done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    for (int r = threadIdx.x; r < p.B; r += kThreads) {
        const int Nr = p.seq_lens[r];
        const int off = p.offsets ? p.offsets[r] : r, nr = p.offsets ? p.offsets[r + 1] - off : 1;
        const bool ok = append_fits(p, r, Nr, off, nr, true) && !__ldcg(p.row_bad + r);
        p.seq_lens_out[r] = ok ? Nr + nr : Nr;
        p.row_bad[r] = 0;
    }
    if (threadIdx.x == 0)
        p.ws->append_done = 0;
}

// One thread reads eight dims of one (token, head, side).
template <int D>
__global__ void __launch_bounds__(kThreads) quant_read_kernel(const QuantReadParams p)
{
    using Q = QuantLayout<D>;
    constexpr int CH = D / 8;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / CH;
    const int c = threadIdx.x % CH, j = c >> 2, f = c & 3;
    const int side = (int)(unit & 1);
    const int64_t th = unit >> 1;
    const int x = (int)min(th / p.Hkv, (int64_t)0x7fffffff), h = (int)(th % p.Hkv);
    const int i = x < p.T ? row_of(p.offsets, p.B, x) : -1;
    if (i < 0)
        return;
    const int N = min(p.seq_lens[i], p.len_cap);
    const int64_t pos = (int64_t)(p.first ? p.first[i] : 0) + (x - p.offsets[i]);
    uint32_t out[4] = {0, 0, 0, 0};
    int page = -1;
    if (pos < 0 || pos >= N) {
        report_error(p.ws, kErrTooLong, i, (int)min(max(pos + 1, (int64_t)-0x7fffffff), (int64_t)0x7fffffff), N);
    } else {
        page = p.bt[(int64_t)i * p.bt_stride + (pos >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
            report_error(p.ws, kErrBadPage, i, (int)(pos >> p.log2P), page);
            page = -1;
        }
    }
    if (page >= 0) {
        const int tb = 1 << p.tb_log2, slot = (int)pos & ((1 << p.log2P) - 1);
        const int r = slot & (tb - 1), t2 = (r & 7) >> 1, e = r & 1;
        const uint8_t *blk = p.cache + ((int64_t)page * p.Hkv + h) * p.page_head_bytes +
                             (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
        const __half *par = side == 0 ? reinterpret_cast<const __half *>(blk + Q::k_params(tb)) + r * 2 * Q::GR + j
                                      : reinterpret_cast<const __half *>(blk + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup) +
                                            (t2 * Q::GR + j) * 4 + e;
        const __half2 s2 = __half2half2(par[0]), b2 = __half2half2(par[side == 0 ? Q::GR : 2]);
        const uint16_t *vc = reinterpret_cast<const uint16_t *>(blk + Q::v_codes(tb) + (r >> 3) * Q::kVGroup);
#pragma unroll
        for (int t = 0; t < 4; ++t) {  // dims 2t and 2t+1 of the eight
            uint32_t w;
            if (side == 0)
                w = reinterpret_cast<const uint32_t *>(blk)[r * (D / 8) + t * Q::GR + j];
            else
                w = (uint32_t)vc[((2 * t * 4 + t2) * Q::GR + j) * 2 + e] |
                    (uint32_t)vc[(((2 * t + 1) * 4 + t2) * Q::GR + j) * 2 + e] << 16;
            const uint32_t n16 = f == 0 ? quant_field<0>(w) : f == 1 ? quant_field<1>(w)
                                 : f == 2 ? quant_field<2>(w) : quant_field<3>(w);
            out[t] = quant_value(n16, s2, b2);
        }
    }
    *reinterpret_cast<uint4 *>((side ? p.v_out : p.k_out) + (int64_t)x * p.out_stride + h * D + c * 8) =
        make_uint4(out[0], out[1], out[2], out[3]);
}

template <class K, class P>
cudaError_t launch(K kern, const P &p, int64_t threads, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((threads + kThreads - 1) / kThreads > 0 ? (threads + kThreads - 1) / kThreads : 1));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_quant_append(int d, const QuantAppendParams &p, cudaStream_t s)
{
    const int64_t threads = (int64_t)p.T * p.Hkv * 2 * (d / 8);
    return d == 128 ? launch(quant_append_kernel<128>, p, threads, s) : launch(quant_append_kernel<64>, p, threads, s);
}

cudaError_t launch_quant_read(int d, const QuantReadParams &p, cudaStream_t s)
{
    const int64_t threads = (int64_t)p.T * p.Hkv * 2 * (d / 8);
    return d == 128 ? launch(quant_read_kernel<128>, p, threads, s) : launch(quant_read_kernel<64>, p, threads, s);
}

}  // namespace pkv
