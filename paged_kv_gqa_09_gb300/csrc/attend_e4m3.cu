// attend_e4m3.cu -- decode attention over the 8-bit cache of e4m3 codes (attend.cuh).
#include "attend.cuh"

namespace pkv {

cudaError_t launch_attend_e4m3(int d, const AttendParams &p, int sms, cudaStream_t s)
{
    return d == 128 ? launch_byte<128, kE4m3>(p, sms, s) : launch_byte<64, kE4m3>(p, sms, s);
}

}  // namespace pkv
