// Root-mean-square norm of x + residual, with fp16 output or with per-row INT8 output
// in the byte order of the W4A8 product, for gfx950.
//
//   h = x + residual (float32, never rounded inside),   y = h / sqrt(mean(h^2) + eps) * weight,
// and for the INT8 output, over the channels that are not outliers,
//   s = amax|y| / 127 (1 when amax is 0),   xq = rint(y * (1 / s)),   0 on outlier channels,
// the outlier channels' y going to xo in fp16. The maximum keeps a NaN, which so becomes the
// row's scale: codes have none, and without it a row that an infinity or a NaN came into
// (or one of zeros with eps = 0) would leave as a plain row of zeros. h is also written, rounded to fp16: it
// is the residual of the next block.
//
// One block per row. A thread holds its channels of the row in registers between the
// three steps (sum of squares, amax, output), so x and residual are read once and each
// output is written once: 2 + 2 bytes in and 2 + 1 (INT8) or 2 + 2 (fp16) out per
// channel. Rows longer than a block's threads hold (32768 channels) are read again.
// The INT8 values and the fp16 outliers and sums are the only roundings.
//
// Bound by memory for many rows, by latency for few. Measured: INT8, 2048 rows of 4096
// channels with 8 outliers 16.2 us (58.7 MB, 3.6 TB/s; all rows at once, so that reading
// and writing do not overlap much), one row 3.8 us; fp16, 33 rows of 8192 4.1 us. Loading
// weights and outliers only when they are used: 21.8 and 7.0 us.
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

constexpr int kNormThreads = 1024;  // at most; a multiple of 64 that covers K / 16 units
constexpr int kNormOutliers = 16;

// 16 consecutive channels in float32: two 16-byte loads a tensor
__device__ __forceinline__ void load16(const f16* p, float* f) {
  const f16x8 a = as_f16x8(*reinterpret_cast<const uint4*>(p));
  const f16x8 b = as_f16x8(*reinterpret_cast<const uint4*>(p + 8));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = (float)a[e];
    f[8 + e] = (float)b[e];
  }
}

__device__ __forceinline__ void store16(f16* p, const float* f) {
  f16x8 a, b;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = (f16)f[e];
    b[e] = (f16)f[8 + e];
  }
  *reinterpret_cast<uint4*>(p) = __builtin_bit_cast(uint4, a);
  *reinterpret_cast<uint4*>(p + 8) = __builtin_bit_cast(uint4, b);
}

__device__ __forceinline__ void load_h(const f16* x, const f16* residual, uint32_t at, float* h) {
  load16(x + at, h);
  if (residual != nullptr) {
    float r[16];
    load16(residual + at, r);
#pragma unroll
    for (int e = 0; e < 16; ++e) h[e] += r[e];
  }
}

// Sum (or maximum) over the block's threads, the same value in every thread, added in
// a fixed order; the maximum keeps a NaN. red holds one value a wave; the two reductions of a row use two arrays,
// so one barrier each is enough.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(v, off);
    v = kMax ? __builtin_elementwise_maximum(v, o) : v + o;
  }
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
  for (int w = 1; w < waves; ++w) r = kMax ? __builtin_elementwise_maximum(r, red[w]) : r + red[w];
  return r;
}

// bit e set: channel 16 unit + e is an outlier. o: the list, one a lane (lane j the j-th),
// -1 past its end; it stays in registers and every lane sees it through scalar reads.
__device__ __forceinline__ uint32_t unit_outliers(int unit, int o, int n_out) {
  uint32_t m = 0;
  for (int j = 0; j < n_out; ++j) {
    const int ch = __builtin_amdgcn_readlane(o, j);
    m |= (ch >> 4) == unit ? 1u << (ch & 15) : 0u;
  }
  return m;
}
// the lane's entry of the list; an index outside [0, K) is clamped
__device__ __forceinline__ int load_outlier(const int32_t* outliers, int n_out, int K) {
  const int j = threadIdx.x & 63;
  return j < n_out ? min(max(outliers[j], 0), K - 1) : -1;
}

// Eight INT8 values of channels e0, e1, .. as bytes: y * inv + 1.5 * 2^23 rounds half to
// even and leaves the integer's two's complement in the low byte (|y * inv| <= 127; in a row
// whose scale is NaN the bytes stand for nothing).
__device__ __forceinline__ uint32_t pack_int8(float a, float b, float c, float d, float inv) {
  const float magic = 12582912.0f;
  const uint32_t ia = __builtin_bit_cast(uint32_t, __builtin_fmaf(a, inv, magic));
  const uint32_t ib = __builtin_bit_cast(uint32_t, __builtin_fmaf(b, inv, magic));
  const uint32_t ic = __builtin_bit_cast(uint32_t, __builtin_fmaf(c, inv, magic));
  const uint32_t id = __builtin_bit_cast(uint32_t, __builtin_fmaf(d, inv, magic));
  const uint32_t ab = __builtin_amdgcn_perm(ib, ia, 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm(id, ic, 0x04000c0cu);
  return ab | cd;
}

// kUnits: units of 16 channels a thread holds; kLong: the row has more than those. (One
// unit takes 64 registers: eight blocks of 256 threads a CU, so 2048 rows of 4096 channels
// run at once.)
template <bool kInt8, int kUnits, bool kLong>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_kernel(const f16* x, const f16* residual, const f16* __restrict__ weight, int64_t M, int K, float eps,
                   const int32_t* __restrict__ outliers, int n_out, f16* hout, f16* __restrict__ y,
                   int8_t* __restrict__ xq, float* __restrict__ sx, f16* __restrict__ xo) {
  __shared__ float red_sum[kNormThreads / 64], red_max[kNormThreads / 64];
  const int units = K >> 4, nt = (int)blockDim.x, t = (int)threadIdx.x;
  const int o = kInt8 ? load_outlier(outliers, n_out, K) : -1;
  for (int m = blockIdx.x; m < (int)M; m += gridDim.x) {
    const uint32_t row = (uint32_t)m * K;  // M K < 2^31
    float h[kUnits][16];
    f16x8 w[kUnits][2];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = t + u * nt;
      if (unit < units) {
        load_h(x, residual, row + 16 * unit, h[u]);
        w[u][0] = as_f16x8(*reinterpret_cast<const uint4*>(weight + 16 * unit));
        w[u][1] = as_f16x8(*reinterpret_cast<const uint4*>(weight + 16 * unit + 8));
      }
    }
    // an outlier channel's y is found again from its own h by the j-th thread
    float oh = 0.0f, ow = 0.0f;
    if (kInt8 && t < n_out) {
      oh = (float)x[row + o];
      if (residual != nullptr) oh += (float)residual[row + o];
      ow = (float)weight[o];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (t + u * nt < units)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = __builtin_fmaf(h[u][e], h[u][e], sum);
    if constexpr (kLong)
      for (int unit = t + kUnits * nt; unit < units; unit += nt) {
        float g[16];
        load_h(x, residual, row + 16 * unit, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum = __builtin_fmaf(g[e], g[e], sum);
      }
    sum = block_reduce<false>(sum, red_sum);
    const float r = 1.0f / sqrtf(sum / (float)K + eps);

    const auto scale = [&](float* v, const f16x8* f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = v[e] * r * (float)f[e >> 3][e & 7];
    };
    // a unit past the ones held: h and its weights again
    const auto reload = [&](float* g, int unit, bool write_h) {
      load_h(x, residual, row + 16 * unit, g);
      const f16x8 f[2] = {as_f16x8(*reinterpret_cast<const uint4*>(weight + 16 * unit)),
                          as_f16x8(*reinterpret_cast<const uint4*>(weight + 16 * unit + 8))};
      if (write_h && hout != nullptr) store16(hout + row + 16 * unit, g);
      scale(g, f);
    };
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = t + u * nt;
      if (unit < units) {
        if (hout != nullptr) store16(hout + row + 16 * unit, h[u]);
        scale(h[u], w[u]);
      }
    }
    if constexpr (!kInt8) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (t + u * nt < units) store16(y + row + 16 * (t + u * nt), h[u]);
      if constexpr (kLong)
        for (int unit = t + kUnits * nt; unit < units; unit += nt) {
          float g[16];
          reload(g, unit, true);
          store16(y + row + 16 * unit, g);
        }
    } else {
      float amax = 0.0f;
      // outlier channels count as 0
      const auto clear = [&](float* v, int unit) {
        const uint32_t om = unit_outliers(unit, o, n_out);
        if (om != 0)
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = (om >> e) & 1u ? 0.0f : v[e];
      };
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (t + u * nt < units) {
          clear(h[u], t + u * nt);
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(h[u][e]));
        }
      // (a long row's further units: h stays unwritten until the last pass reads them again)
      if constexpr (kLong)
        for (int unit = t + kUnits * nt; unit < units; unit += nt) {
          float g[16];
          reload(g, unit, false);
          clear(g, unit);
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(g[e]));
        }
      amax = block_reduce<true>(amax, red_max);
      const float s = amax == 0.0f ? 1.0f : amax / 127.0f;
      const float inv = amax == 0.0f ? 1.0f : 127.0f / amax;
      if (t == 0) sx[m] = s;
      if (t < kNormOutliers) xo[m * kNormOutliers + t] = t < n_out ? (f16)(oh * r * ow) : (f16)0.0f;
      // byte order of the 16 channels: 0,2,4,6, 1,3,5,7, 8,10,12,14, 9,11,13,15
      const auto write = [&](const float* v, int unit) {
        *reinterpret_cast<uint4*>(xq + row + 16 * unit) =
            make_uint4(pack_int8(v[0], v[2], v[4], v[6], inv), pack_int8(v[1], v[3], v[5], v[7], inv),
                       pack_int8(v[8], v[10], v[12], v[14], inv), pack_int8(v[9], v[11], v[13], v[15], inv));
      };
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (t + u * nt < units) write(h[u], t + u * nt);
      if constexpr (kLong)
        for (int unit = t + kUnits * nt; unit < units; unit += nt) {
          float g[16];
          reload(g, unit, true);
          clear(g, unit);
          write(g, unit);
        }
    }
    __syncthreads();  // the reduction arrays are reused by the block's next row
  }
}

// xq (in the products' byte order) * sx, with the outlier channels from xo: fp16 [M, K].
// A thread takes 16 channels. 2048 rows of 4096: 8.2 us (25 MB, 3.1 TB/s), one row 2.7 us.
__global__ void __launch_bounds__(256)
dequantize_act_int8_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx, const f16* __restrict__ xo,
                           const int32_t* __restrict__ outliers, int n_out, int64_t M, int K, f16* __restrict__ out) {
  const int units = K >> 4;
  const int o = load_outlier(outliers, n_out, K);
  const uint32_t total = (uint32_t)M * units, step = gridDim.x * 256u;  // M K < 2^31
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < total; i += step) {
    const uint32_t m = i / (uint32_t)units;
    const int unit = (int)(i - m * units);
    const uint4 p = *reinterpret_cast<const uint4*>(xq + (size_t)16 * i);
    const uint32_t d[4] = {p.x, p.y, p.z, p.w};
    const float s = sx[m];
    float v[16];
    constexpr int ord[16] = {0, 2, 4, 6, 1, 3, 5, 7, 8, 10, 12, 14, 9, 11, 13, 15};
#pragma unroll
    for (int j = 0; j < 16; ++j) v[ord[j]] = (float)(int8_t)(d[j >> 2] >> (8 * (j & 3))) * s;
    const uint32_t om = unit_outliers(unit, o, n_out);
    if (om != 0)
      for (int j = 0; j < n_out; ++j) {
        const int ch = __builtin_amdgcn_readlane(o, j);
        if ((ch >> 4) == unit) {
          const float f = (float)xo[(size_t)m * kNormOutliers + j];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = (ch & 15) == e ? f : v[e];
        }
      }
    store16(out + (size_t)16 * i, v);
  }
}

hipError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t M,
                              int64_t K, float eps, const int32_t* outliers, int64_t n_out, uint16_t* h, uint16_t* y,
                              int8_t* xq, float* sx, uint16_t* xo, hipStream_t stream) {
  const int64_t units = K / 16;
  const int64_t threads = units >= kNormThreads ? kNormThreads : (units + 63) / 64 * 64;
  const dim3 grid((unsigned)(M < 65536 ? M : 65536)), block((unsigned)threads);
  const auto f = [](const uint16_t* p) { return reinterpret_cast<const f16*>(p); };
  const auto g = [](uint16_t* p) { return reinterpret_cast<f16*>(p); };
  const auto run = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, stream, f(x), f(residual), f(weight), M, (int)K, eps, outliers,
                       (int)n_out, g(h), g(y), xq, sx, g(xo));
  };
  if (units <= threads)
    xq != nullptr ? run(add_rmsnorm_kernel<true, 1, false>) : run(add_rmsnorm_kernel<false, 1, false>);
  else if (units <= 2 * threads)
    xq != nullptr ? run(add_rmsnorm_kernel<true, 2, false>) : run(add_rmsnorm_kernel<false, 2, false>);
  else
    xq != nullptr ? run(add_rmsnorm_kernel<true, 1, true>) : run(add_rmsnorm_kernel<false, 1, true>);
  return hipGetLastError();
}

hipError_t launch_dequantize_act_int8(const int8_t* xq, const float* sx, const uint16_t* xo, const int32_t* outliers,
                                      int64_t n_out, int64_t M, int64_t K, uint16_t* out, hipStream_t stream) {
  const int64_t blocks = (M * (K / 16) + 255) / 256;
  hipLaunchKernelGGL(dequantize_act_int8_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                     stream, xq, sx, reinterpret_cast<const f16*>(xo), outliers, (int)n_out, M, (int)K,
                     reinterpret_cast<f16*>(out));
  return hipGetLastError();
}

}  // namespace wq
