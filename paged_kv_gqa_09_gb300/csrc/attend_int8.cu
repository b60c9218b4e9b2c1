// attend_int8.cu -- decode attention over the 8-bit cache of int8 codes (attend.cuh).
#include "attend.cuh"

namespace pkv {

cudaError_t launch_attend_int8(int d, const AttendParams &p, int sms, cudaStream_t s)
{
    return d == 128 ? launch_byte<128, kInt8>(p, sms, s) : launch_byte<64, kInt8>(p, sms, s);
}

}  // namespace pkv
