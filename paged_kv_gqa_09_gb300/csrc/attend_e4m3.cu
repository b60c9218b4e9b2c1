// attend_e4m3.cu -- decode attention over the 8-bit cache of e4m3 codes (attend.cuh).
#include "attend.cuh"

namespace pkv {
namespace {

template <int D>
cudaError_t launch_d(const AttendParams &p, int sms, cudaStream_t s)
{
    constexpr int kKind = k8Bit + 16 * kE4m3;
    const CUtensorMap none = {};
    switch (p.tb_log2) {
    case 3:
        return launch_one<D, kKind + 3>(none, none, p, sms, s);
    case 4:
        return launch_one<D, kKind + 4>(none, none, p, sms, s);
    case 5:
        return launch_one<D, kKind + 5>(none, none, p, sms, s);
    default:
        return launch_one<D, kKind + 6>(none, none, p, sms, s);
    }
}

}  // namespace

cudaError_t launch_attend_e4m3(int d, const AttendParams &p, int sms, cudaStream_t s)
{
    return d == 128 ? launch_d<128>(p, sms, s) : launch_d<64>(p, sms, s);
}

}  // namespace pkv
