// The decode kernels' entry (gemv_launch.h has the choice among them for 4-bit layers with one
// (s, z) per 128 input channels; gemv_fmt.hip that of the other weight formats).
#include "gemv_launch.h"

namespace wq {

constexpr int64_t kDotMinK = 12288;  // the single-row kernel from this K on (see launch_gemv)

// The decode kernels stage a tile's scales and zero-points in LDS: those of 284 000 channels fit beside 16 rows' slots.
bool gemv_fits(int64_t M, int64_t K, bool g64, bool adapters) {
  return ring_fits(1, M <= 4 ? 1 : (M <= 8 ? 2 : 4), (g64 ? 2 : 1) * (K / kGroup), adapters);
}

hipError_t launch_gemv(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                       const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                       const int32_t* col, const uint16_t* val, void* y, int y_f32, const LowRank& lr,
                       hipStream_t stream, WFormat f, bool mfma_only) {
  if (!f.plain()) return launch_gemv_fmt(x, M, K, packed, scales, zeros, N, row_ptr, col, val, y, y_f32, f, stream);
  // one activation row of a long layer: whole rows per wave and VALU dot products
  // (gemv_dot.hip). Measured at M = 1 (single-row against MFMA kernel, us): K = 4096
  // 7.0 / 6.7, 8192 11.1 / 9.8, 14336 14.7 / 15.3, 28672 26.6 / 30.0.
  if (!mfma_only && lr.r == 0 && K >= kDotMinK && gemv_dot_supported(M, K, scales, zeros))
    return launch_gemv_dot(x, K, packed, scales, zeros, N, row_ptr, col, val, y, y_f32, stream);
  return lr.row ? launch_gemv_adapters(x, M, K, packed, scales, zeros, N, row_ptr, col, val, y, y_f32, lr, stream)
                : launch_gemv_mfma<false>(x, M, K, packed, scales, zeros, N, row_ptr, col, val, y, y_f32, lr, stream);
}

}  // namespace wq
