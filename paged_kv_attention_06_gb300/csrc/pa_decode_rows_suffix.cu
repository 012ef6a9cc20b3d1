// The few-row kernel behind a shared prefix: every request's own keys, the states
// left for the merge with the prefix's (pa_decode_prefix).
#include "pa_decode_rows.cuh"

namespace pa {
namespace rows {

Kernels suffix_kernels(int D, int kind, int NT)
{
    if (kind == kQ4Pool)
        return NT == 1 ? kernels_of<128, kQ4Pool, 1, kSuffix>() : kernels_of<128, kQ4Pool, 2, kSuffix>();
    if (kind == kE4m3Pool)
        return NT == 1 ? kernels_of<128, kE4m3Pool, 1, kSuffix>() : kernels_of<128, kE4m3Pool, 2, kSuffix>();
    if (D == 64)
        return NT == 1 ? kernels_of<64, kBf16Pool, 1, kSuffix>() : kernels_of<64, kBf16Pool, 2, kSuffix>();
    return NT == 1 ? kernels_of<128, kBf16Pool, 1, kSuffix>() : kernels_of<128, kBf16Pool, 2, kSuffix>();
}

}  // namespace rows
}  // namespace pa
