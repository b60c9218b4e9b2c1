// attend.cu -- decode attention over the tokens a sliding window and the row's
// first tokens leave visible, from the fp16 pages or from the 4-bit cache.
//
// One CTA per (row, KV head): tiles of 32 visible tokens are brought to shared
// memory as fp16, scored for the G query heads, and folded into a running
// maximum, sum and fp32 accumulator (the online softmax).
#include "pkv_device.cuh"
#include "pkv_kernels.h"
#include "quant_format.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, bool QUANT>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendParams p)
{
    using Q = QuantLayout<D>;
    constexpr int CH = D / 8;
    __shared__ __align__(16) __half s_k[kTile][D + 8], s_v[kTile][D + 8];
    __shared__ __align__(16) __half s_q[8][D];
    __shared__ float s_p[8][kTile], s_m[8], s_l[8], s_a[8];
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv, tid = threadIdx.x;
    int N = p.seq_lens[i];
    if (N < 0 || N > p.len_cap) {
        if (h == 0 && tid == 0)
            report_error(p.ws, N < 0 ? kErrNegLen : kErrTooLong, i, N, p.len_cap);
        N = N < 0 ? 0 : p.len_cap;
    }
    const int ns = min(p.sinks, N), w0 = max(ns, N - p.window), nv = ns + (N - w0);
    for (int x = tid; x < p.G * CH; x += kThreads)
        reinterpret_cast<uint4 *>(s_q)[x] = reinterpret_cast<const uint4 *>(p.q + ((int64_t)i * p.Hq + h * p.G) * D)[x];
    if (tid < 8) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.f;
    }
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // dim tid of each head (tid < D)
    for (int v0 = 0; v0 < nv; v0 += kTile) {
        __syncthreads();
        const int n = min(kTile, nv - v0);
        for (int x = tid; x < kTile * CH * 2; x += kThreads) {
            const int side = x & 1, c = (x >> 1) % CH, t = (x >> 1) / CH;
            uint32_t out[4] = {0, 0, 0, 0};
            if (t < n) {
                const int vis = v0 + t, pos = vis < ns ? vis : vis - ns + w0;
                const int page = p.bt[(int64_t)i * p.bt_stride + (pos >> p.log2P)];
                const int slot = pos & ((1 << p.log2P) - 1);
                if (page < 0 || page >= p.num_pages) {
                    report_error(p.ws, kErrBadPage, i, pos >> p.log2P, page);
                } else if (!QUANT) {
                    const uint4 u = reinterpret_cast<const uint4 *>(
                        (side ? p.v : p.k) + ((((int64_t)page << p.log2P) + slot) * p.Hkv + h) * D)[c];
                    out[0] = u.x;
                    out[1] = u.y;
                    out[2] = u.z;
                    out[3] = u.w;
                } else {
                    const int tb = 1 << p.tb_log2, r = slot & (tb - 1), t2 = (r & 7) >> 1, e = r & 1, j = c >> 2, f = c & 3;
                    const uint8_t *blk = p.cache + ((int64_t)page * p.Hkv + h) * p.page_head_bytes +
                                         (int64_t)(slot >> p.tb_log2) * Q::bytes(tb);
                    const __half *par = side == 0
                        ? reinterpret_cast<const __half *>(blk + Q::k_params(tb)) + r * 2 * Q::GR + j
                        : reinterpret_cast<const __half *>(blk + Q::v_params(tb) + (r >> 3) * Q::kVParamGroup) +
                              (t2 * Q::GR + j) * 4 + e;
                    const __half2 s2 = __half2half2(par[0]), b2 = __half2half2(par[side == 0 ? Q::GR : 2]);
                    const uint16_t *vc = reinterpret_cast<const uint16_t *>(blk + Q::v_codes(tb) + (r >> 3) * Q::kVGroup);
                    for (int u = 0; u < 4; ++u) {
                        uint32_t w;
                        if (side == 0)
                            w = reinterpret_cast<const uint32_t *>(blk)[r * (D / 8) + u * Q::GR + j];
                        else
                            w = (uint32_t)vc[((2 * u * 4 + t2) * Q::GR + j) * 2 + e] |
                                (uint32_t)vc[(((2 * u + 1) * 4 + t2) * Q::GR + j) * 2 + e] << 16;
                        const uint32_t n16 = f == 0 ? quant_field<0>(w) : f == 1 ? quant_field<1>(w)
                                             : f == 2 ? quant_field<2>(w) : quant_field<3>(w);
                        out[u] = quant_value(n16, s2, b2);
                    }
                }
            }
            *reinterpret_cast<uint4 *>(side ? &s_v[t][c * 8] : &s_k[t][c * 8]) = make_uint4(out[0], out[1], out[2], out[3]);
        }
        __syncthreads();
        for (int x = tid; x < p.G * kTile; x += kThreads) {
            const int g = x / kTile, t = x % kTile;
            float s = 0.f;
            for (int e = 0; e < D; ++e)
                s += __half2float(s_q[g][e]) * __half2float(s_k[t][e]);
            s_p[g][t] = t < n ? s * p.scale_log2 : -INFINITY;
        }
        __syncthreads();
        if (tid < p.G) {
            float m = s_m[tid];
            for (int t = 0; t < n; ++t)
                m = fmaxf(m, s_p[tid][t]);
            const float a = m == -INFINITY ? 1.f : ex2(s_m[tid] - m);
            float l = s_l[tid] * a;
            for (int t = 0; t < kTile; ++t) {
                const float e = m == -INFINITY ? 0.f : ex2(s_p[tid][t] - m);
                s_p[tid][t] = e;
                l += e;
            }
            s_m[tid] = m;
            s_l[tid] = l;
            s_a[tid] = a;
        }
        __syncthreads();
        if (tid < D)
            for (int g = 0; g < p.G; ++g) {
                float y = acc[g] * s_a[g];
                for (int t = 0; t < n; ++t)
                    y += s_p[g][t] * __half2float(s_v[t][tid]);
                acc[g] = y;
            }
    }
    __syncthreads();
    if (tid < D)
        for (int g = 0; g < p.G; ++g)
            p.o[((int64_t)i * p.Hq + h * p.G + g) * D + tid] = __float2half_rn(nv > 0 ? acc[g] / s_l[g] : 0.f);
    if (p.lse && tid < p.G)
        p.lse[(int64_t)i * p.Hq + h * p.G + tid] = nv > 0 ? (s_m[tid] + log2f(s_l[tid])) * kLn2 : -INFINITY;
}

template <int D, bool QUANT>
cudaError_t launch_one(const AttendParams &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * p.Hkv);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_kernel<D, QUANT>, p);
}

}  // namespace

cudaError_t launch_attend(int d, bool quant, const AttendParams &p, cudaStream_t s)
{
    if (d == 128)
        return quant ? launch_one<128, true>(p, s) : launch_one<128, false>(p, s);
    return quant ? launch_one<64, true>(p, s) : launch_one<64, false>(p, s);
}

}  // namespace pkv
