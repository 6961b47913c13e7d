// The decode kernels (gemv_launch.h) with the low-rank adapters that rows name.
#include "gemv_launch.h"

namespace wq {

hipError_t launch_gemv_adapters(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                                const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                                const int32_t* col, const uint16_t* val, void* y, int y_f32, const LowRank& lr,
                                hipStream_t stream) {
  return launch_gemv_mfma<true>(x, M, K, packed, scales, zeros, N, row_ptr, col, val, y, y_f32, lr, stream);
}

}  // namespace wq
