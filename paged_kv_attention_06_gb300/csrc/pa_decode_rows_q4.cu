// The few-row kernel over 4-bit pools (pa_decode_q4).
#include "pa_decode_rows.cuh"

namespace pa {
namespace rows {

Kernels q4_kernels(int NT)
{
    return NT == 1 ? kernels_of<128, kQ4Pool, 1, kFull>() : kernels_of<128, kQ4Pool, 2, kFull>();
}

}  // namespace rows
}  // namespace pa
