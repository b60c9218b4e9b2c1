// attend.cu -- decode attention over the fp16 pages and the 4-bit cache (attend.cuh).
#include "attend.cuh"

namespace pkv {
namespace {

template <int D>
cudaError_t launch_d(const CUtensorMap &tk, const CUtensorMap &tv, const AttendParams &p, int sms, cudaStream_t s)
{
    if (!p.cache)
        return launch_one<D, kFp16>(tk, tv, p, sms, s);
    switch (p.tb_log2) {
    case 3:
        return launch_one<D, k4Bit + 3>(tk, tv, p, sms, s);
    case 4:
        return launch_one<D, k4Bit + 4>(tk, tv, p, sms, s);
    case 5:
        return launch_one<D, k4Bit + 5>(tk, tv, p, sms, s);
    default:
        return launch_one<D, k4Bit + 6>(tk, tv, p, sms, s);
    }
}

}  // namespace

cudaError_t launch_attend(int d, const CUtensorMap &tk, const CUtensorMap &tv, const AttendParams &p, int sms, cudaStream_t s)
{
    return d == 128 ? launch_d<128>(tk, tv, p, sms, s) : launch_d<64>(tk, tv, p, sms, s);
}

}  // namespace pkv
