// Down-projections of low-rank adapters that each row of a batch names for itself, for gfx950:
//   t[m] = fp16(s_a x[m] . L1_a^T),  a = adapter[m],
// L1 [n, r, K] fp16, s [n] float32 (or 1). The product kernels then add t[m] . L2_a^T to each output tile's fp32
// accumulators (adapters_add16 and adapters_add32, beside what they add for a branch that all rows share).
// t [M, r rounded up to 32]: zeros beyond r; rows of no adapter are left as they are, and nothing reads them.
//
//  adapters_down_dot_kernel  (few rows) a block for each row and few components: dot products, the waves split K.
//  adapters_down_kernel      (more rows) a block for each 16 rows and 16 or 32 components: one pass of 16x16x32
//    products for each adapter that the rows name, of which each row keeps its own.
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

constexpr int kDotWaves = 8;

template <int NC>
__global__ void __launch_bounds__(64 * kDotWaves)
adapters_down_dot_kernel(const f16* __restrict__ x, int K, const f16* __restrict__ L1, const float* __restrict__ scale,
                         int n, int r, const int32_t* __restrict__ adapter, f16* __restrict__ t, int tr) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int W = blockDim.x >> 6;
  const int m = blockIdx.y, j0 = blockIdx.x * NC;
  const int a = __builtin_amdgcn_readfirstlane(adapter[m]);
  if ((uint32_t)a >= (uint32_t)n) return;
  const f16* xrow = x + (int64_t)m * K + 8 * lane;
  const f16* lrow[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) lrow[c] = L1 + ((int64_t)a * r + min(j0 + c, r - 1)) * K + 8 * lane;
  float acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = 0.f;
  const int nsteps = (K + 511) >> 9;
  constexpr int SB = 2;  // steps whose loads are in flight together
  for (int s0 = wave; s0 < nsteps; s0 += W * SB) {
    // lane's channels in step s: 512 s + 8 lane .. + 7 (K is a multiple of 128: all in range or all out)
    uint4 xv[SB], lv[SB][NC];
#pragma unroll
    for (int u = 0; u < SB; ++u) {
      const int c0 = 512 * (s0 + W * u);
      const bool ok = c0 + 8 * lane < K;
      xv[u] = ok ? *reinterpret_cast<const uint4*>(xrow + c0) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        lv[u][c] = ok ? *reinterpret_cast<const uint4*>(lrow[c] + c0) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < SB; ++u) {
      const uint32_t xw[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint32_t lw[4] = {lv[u][c].x, lv[u][c].y, lv[u][c].z, lv[u][c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c] = __builtin_amdgcn_fdot2(as_f16x2(xw[e]), as_f16x2(lw[e]), acc[c], false);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) acc[c] += __shfl_xor(acc[c], off);
  __shared__ float red[kDotWaves][NC];
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) red[wave][c] = acc[c];
  }
  __syncthreads();
  if (threadIdx.x < NC && j0 + (int)threadIdx.x < tr) {
    const int c = threadIdx.x;
    float v = red[0][c];
    for (int w = 1; w < W; ++w) v += red[w][c];
    t[(int64_t)m * tr + j0 + c] = j0 + c < r ? (f16)(scale ? v * scale[a] : v) : (f16)0.0f;
  }
}

constexpr int kRowWaves = 16;
constexpr int kRowSteps = 8;                           // of a wave in a chunk of K
constexpr int kRowChunk = 32 * kRowWaves * kRowSteps;  // input channels of a chunk

template <int CT>
__global__ void __launch_bounds__(64 * kRowWaves)
adapters_down_kernel(const f16* __restrict__ x, int M, int K, const f16* __restrict__ L1,
                     const float* __restrict__ scale, int n, int r, const int32_t* __restrict__ adapter,
                     f16* __restrict__ t, int tr) {
  constexpr int U = CT / 16;  // 16x16 tiles
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j0 = blockIdx.x * CT, m0 = blockIdx.y * 16;
  const int id = adapter[min(m0 + q, M - 1)];
  uint32_t left = (uint32_t)__ballot(m0 + q < M && (uint32_t)id < (uint32_t)n) & 0xFFFFu;
  const f16* xr = x + (int64_t)min(m0 + q, M - 1) * K + 8 * h;
  __shared__ f32x4 red[kRowWaves - 1][U][64];
  uint4 av[kRowSteps];
  for (bool first = true; left != 0; first = false) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t members = (uint32_t)__ballot(id == a) & left;
    left &= ~members;
    const f16* lr0 = L1 + ((int64_t)a * r + min(j0 + q, r - 1)) * K + 8 * h;
    const f16* lr1 = L1 + ((int64_t)a * r + min(j0 + 16 + q, r - 1)) * K + 8 * h;
    f32x4 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < K; c0 += kRowChunk) {
      // a wave's steps of 32 channels: every 16th of the chunk (K a multiple of 128: whole steps)
      uint4 bv[kRowSteps][U];
#pragma unroll
      for (int i = 0; i < kRowSteps; ++i) {
        const int c = c0 + 32 * (wave + kRowWaves * i);
        if (c < K) {  // wave-uniform
          if (first || K > kRowChunk) av[i] = *reinterpret_cast<const uint4*>(xr + c);
          bv[i][0] = *reinterpret_cast<const uint4*>(lr0 + c);
          if constexpr (U > 1) bv[i][U - 1] = *reinterpret_cast<const uint4*>(lr1 + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kRowSteps; ++i)
        if (c0 + 32 * (wave + kRowWaves * i) < K) {
#pragma unroll
          for (int u = 0; u < U; ++u) acc[u] = mfma_16x16x32(as_f16x8(av[i]), as_f16x8(bv[i][u]), acc[u]);
        }
    }
    if (wave > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) red[wave - 1][u][lane] = acc[u];
    }
    __syncthreads();
    if (wave == 0) {
      const float s = scale ? scale[a] : 1.0f;
#pragma unroll
      for (int w = 0; w < kRowWaves - 1; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) acc[u] += red[w][u][lane];
      // row 4 h + i, component j0 + 16 u + q
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = j0 + 16 * u + q;
          if ((members >> (4 * h + i)) & 1u) t[(int64_t)(m0 + 4 * h + i) * tr + c] = c < r ? (f16)(s * acc[u][i]) : (f16)0.0f;
        }
    }
    __syncthreads();  // red is refilled
  }
}

hipError_t launch_adapters_down(const uint16_t* x, int64_t M, int64_t K, const Adapters& ad, int64_t r, uint16_t* t,
                                hipStream_t stream) {
  const int tr = (int)((r + 31) / 32 * 32);
  const f16* L1 = reinterpret_cast<const f16*>(ad.L1);
  constexpr int64_t kFew = 64;
  if (M <= kFew) {
    int64_t w = (K / 128 + 7) / 8;  // about two steps of 512 channels a wave
    w = w < 1 ? 1 : (w > kDotWaves ? kDotWaves : w);
    if (M * tr <= 1024)
      hipLaunchKernelGGL(adapters_down_dot_kernel<1>, dim3((unsigned)tr, (unsigned)M), dim3((unsigned)(64 * w)), 0,
                         stream, reinterpret_cast<const f16*>(x), (int)K, L1, ad.scale, (int)ad.n, (int)r, ad.row,
                         reinterpret_cast<f16*>(t), tr);
    else
      hipLaunchKernelGGL(adapters_down_dot_kernel<4>, dim3((unsigned)(tr / 4), (unsigned)M), dim3((unsigned)(64 * w)),
                         0, stream, reinterpret_cast<const f16*>(x), (int)K, L1, ad.scale, (int)ad.n, (int)r, ad.row,
                         reinterpret_cast<f16*>(t), tr);
    return hipGetLastError();
  }
  constexpr int64_t kRowsPerLaunch = 65535 * 16;  // gridDim.y limit
  for (int64_t m = 0; m < M; m += kRowsPerLaunch) {
    const int64_t mc = M - m < kRowsPerLaunch ? M - m : kRowsPerLaunch;
    hipLaunchKernelGGL(adapters_down_kernel<16>, dim3((unsigned)(tr / 16), (unsigned)((mc + 15) / 16)),
                       dim3(64 * kRowWaves), 0, stream, reinterpret_cast<const f16*>(x) + m * K, (int)mc, (int)K, L1,
                       ad.scale, (int)ad.n, (int)r, ad.row + m, reinterpret_cast<f16*>(t) + m * tr, tr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace wq
