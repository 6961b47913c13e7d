// Down-projections of low-rank adapters that each row of a batch names for itself, for gfx950:
//   t[m] = fp16(s_a x[m] . L1_a^T),  a = adapter[m],
// L1 [n, r, K] fp16, s [n] float32 (or 1). The product kernels then add t[m] . L2_a^T to each output tile's fp32
// accumulators (adapters_up16 and adapters_add32, beside what they add for a branch that all rows share).
// t [M, r rounded up to 32]: zeros beyond r; rows of no adapter are left as they are, and nothing reads them.
//
//  adapters_down_dot_kernel  (few rows) a block for each row and few components: dot products, the waves split K.
//    Bound by latency: 3.3 us for one row of 16 x 4096 or 16 of 32 x 4096, 5.8 for 64 of 64 x 3584 (up to
//    29 MB of L1).
//  adapters_down_kernel      (more rows) a block for each 16 rows, 16 components and chunk of K: 16x16x32 products, its
//    waves dealt to the adapters that the rows name; several chunks' partials are summed by adapters_finish_kernel.
//    Bound by the loads of a block's rows, one batch after another: 2048 rows of 16 x 4096 16 us, where their 18 MB of
//    x and L1 are 4.
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
  if (j0 >= r) {
    if (threadIdx.x < NC) t[(int64_t)m * tr + j0 + threadIdx.x] = (f16)0.0f;
    return;
  }
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
constexpr int kRowParts = 16;  // of a chunk of K, whose sums meet in pairs
constexpr int kRowBatch = 4;   // pairs of 32-channel steps whose loads a wave issues together

// Sums of consecutive parts, added in the pairs of a binary tree (a part that is left out counts as zero): the same
// whether one wave adds all sixteen, or each of several its own and tree_sum those.
struct PairSum {
  f32x4 held[5] = {};  // of 1, 2, 4, 8, 16 parts
  int n = 0;           // (uniform)
  template <int L = 0>
  __device__ __forceinline__ void add(f32x4 v) {
    if constexpr (L < 4) {
      if ((n >> L) & 1)
        add<L + 1>(held[L] + v);
      else
        held[L] = v;
    } else {
      held[4] = v;
    }
    if constexpr (L == 0) ++n;
  }
  __device__ __forceinline__ f32x4 sum() const {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int l = 0; l < 5; ++l)
      if ((n >> l) & 1) v = held[l] + v;
    return v;
  }
};

// v[0] .. v[per - 1], a power of two of them up to N, of each the lane's
template <int N>
__device__ __forceinline__ f32x4 tree_sum(const f32x4 (*v)[64], int per, int lane) {
  if constexpr (N == 1) {
    return v[0][lane];
  } else {
    f32x4 low = tree_sum<N / 2>(v, per, lane);
    if (per >= N) low += tree_sum<N / 2>(v + N / 2, per, lane);
    return low;
  }
}

// The waves are dealt to the adapters that the block's 16 rows name: all sixteen split K for one adapter, each has an
// adapter of its own from nine on. (Adapter after adapter, 96 rows of as many adapters took 250 us at K = 8192.) A
// wave's steps come in pairs, whole 128-byte lines of its rows. How many waves an adapter has goes by the other rows, so
// a chunk's sum is made of the same sixteen parts in the same order for any number of them: a row's bits are its own.
__global__ void __launch_bounds__(64 * kRowWaves)
adapters_down_kernel(const f16* __restrict__ x, int M, int K, const f16* __restrict__ L1,
                     const float* __restrict__ scale, int n, int r, const int32_t* __restrict__ adapter,
                     f16* __restrict__ t, int tr, int chunk, float* __restrict__ part) {
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const int c_lo = blockIdx.z * chunk, steps = (min(K, c_lo + chunk) - c_lo) / 64;  // chunks are multiples of 64
  __shared__ f32x4 red[kRowWaves][64];
  const int id = adapter[min(m0 + q, M - 1)];
  const uint32_t all = (uint32_t)__ballot(m0 + q < M && (uint32_t)id < (uint32_t)n) & 0xFFFFu;
  int count = 0;  // of adapters
  for (uint32_t left = all; left != 0; ++count)
    left &= ~(uint32_t)__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctz(left)));
  int shift = 4;  // log2 of the waves of an adapter
  while ((kRowWaves >> shift) < count) --shift;
  const int which = wave >> shift, sub = wave & ((1 << shift) - 1), per = 1 << shift;
  uint32_t members = 0;
  int a = 0;
  if (which < count) {
    uint32_t left = all;
    for (int i = 0; i <= which; ++i) {
      a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      members = (uint32_t)__ballot(id == a) & left;
      left &= ~members;
    }
    // rows of other adapters: a row that is read anyway
    const int row = (members >> q) & 1u ? q : __builtin_ctz(members);
    const f16* xr = x + (int64_t)(m0 + row) * K + c_lo + 8 * h;
    const f16* lr = L1 + ((int64_t)a * r + min(j0 + q, r - 1)) * K + c_lo + 8 * h;
    const int len = (steps + kRowParts - 1) / kRowParts;  // steps of 64 channels of a part; the last parts may have none
    const int s_lo = sub * (kRowParts >> shift) * len, s_hi = min(steps, (sub + 1) * (kRowParts >> shift) * len);
    PairSum sums;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    int end = s_lo + len;  // of the part
    for (int s = s_lo; s < s_hi; s += kRowBatch) {
      uint4 av[kRowBatch][2], bv[kRowBatch][2];
#pragma unroll
      for (int i = 0; i < kRowBatch; ++i)
        if (s + i < s_hi) {  // wave-uniform
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            av[i][u] = *reinterpret_cast<const uint4*>(xr + 64 * (s + i) + 32 * u);
            bv[i][u] = *reinterpret_cast<const uint4*>(lr + 64 * (s + i) + 32 * u);
          }
        }
#pragma unroll
      for (int i = 0; i < kRowBatch; ++i)
        if (s + i < s_hi) {
#pragma unroll
          for (int u = 0; u < 2; ++u) acc = mfma_16x16x32(as_f16x8(av[i][u]), as_f16x8(bv[i][u]), acc);
          if (s + i + 1 == end) {
            sums.add(acc);
            acc = f32x4{0.f, 0.f, 0.f, 0.f};
            end += len;
          }
        }
    }
    if (s_hi > end - len) sums.add(acc);  // a last part that is shorter
    red[wave][lane] = sums.sum();
  }
  __syncthreads();
  if (which >= count || sub != 0) return;
  const f32x4 acc = tree_sum<kRowWaves>(red + wave, per, lane);
  // row 4 h + i, component j0 + q
  const bool last = blockIdx.x == gridDim.x - 1;
  const float s = scale ? scale[a] : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!((members >> (4 * h + i)) & 1u)) continue;
    const int64_t row = (int64_t)(m0 + 4 * h + i) * tr;
    if (part != nullptr) {
      part[(int64_t)blockIdx.z * M * tr + row + j0 + q] = acc[i];
    } else {
      t[row + j0 + q] = j0 + q < r ? (f16)(s * acc[i]) : (f16)0.0f;
      if (last && j0 + 16 + q < tr) t[row + j0 + 16 + q] = (f16)0.0f;
    }
  }
}

// t from the partials of the chunks of K, in order; a thread for each value.
__global__ void __launch_bounds__(256)
adapters_finish_kernel(const float* __restrict__ part, int chunks, int M, const float* __restrict__ scale, int n, int r,
                       const int32_t* __restrict__ adapter, f16* __restrict__ t, int tr) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)M * tr;
  if (i >= all) return;
  const int a = adapter[i / tr], c = (int)(i % tr);
  if ((uint32_t)a >= (uint32_t)n) return;
  float v = 0.0f;
  if (c < r) {
    for (int k = 0; k < chunks; k += 4) {
      float p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = part[min(k + u, chunks - 1) * all + i];
#pragma unroll
      for (int u = 0; u < 4; ++u) v += k + u < chunks ? p[u] : 0.0f;
    }
    v *= scale ? scale[a] : 1.0f;
  }
  t[i] = (f16)v;
}

// Whether each row reads its adapter for itself: up to 64 MB in all, at worst from HBM. The other kernel reads an adapter
// once for 16 rows that name it, but a wave alone reads it where they name many. In us, whole calls of 128 channels by
// this one / the other, rows of one adapter and each its own:
//   16 components, K = 1024,   512 rows (16 MB)    8.8 /  9.0     9.8 / 25.8
//                             2048      (64 MB)   18.1 / 12.3    19.8 / 30.1
//                             4096     (128 MB)   33.5 / 20.2    36.1 / 39.5
//                  K = 4096,   512      (64 MB)   15.2 / 13.7    18.7 / 31.4
//                             1024     (128 MB)   24.4 / 17.7    28.0 / 50.9
//                             2048     (256 MB)   43.3 / 24.3    47.6 / 89.6
//                  K = 8192,   256      (64 MB)   19.2 / 16.5    30.6 / 33.6
//                              512     (128 MB)   30.6 / 21.2    49.4 / 54.2
//   64 components, K = 4096,   128      (64 MB)   11.9 / 12.9    18.8 / 31.0
//                              512     (256 MB)   21.3 / 16.9    39.8 / 82.4
// (So beyond the bound rows that each name their own would still be faster by themselves; prompts' rows come in runs.)
static bool few_rows(int64_t M, int64_t K, int64_t r) { return M * r <= ((int64_t)1 << 25) / K; }
static int64_t t_stride(int64_t r) { return (r + 31) / 32 * 32; }

// Chunks of K (64 channels' multiples) that give half of the CUs a block, each at least 1024 channels.
struct DownPlan {
  int64_t chunk, chunks;
};
static DownPlan down_plan(int64_t M, int64_t K, int64_t r) {
  const int64_t tiles = (M + 15) / 16 * ((r + 15) / 16), want = (128 + tiles - 1) / tiles, most = K / 1024;
  int64_t chunks = want < most ? want : most;
  chunks = chunks < 1 ? 1 : chunks;
  const int64_t chunk = ((K + chunks - 1) / chunks + 63) / 64 * 64;
  return DownPlan{chunk, (K + chunk - 1) / chunk};
}

constexpr int64_t kRowsPerLaunch = 65535 * 16;  // gridDim.y limit

size_t adapters_partial_bytes(int64_t M, int64_t K, int64_t r) {
  if (few_rows(M, K, r)) return 0;
  size_t most = 0;
  for (const int64_t rows : {M < kRowsPerLaunch ? M : kRowsPerLaunch, M % kRowsPerLaunch}) {
    if (rows == 0) continue;
    const DownPlan p = down_plan(rows, K, r);
    const size_t b = p.chunks > 1 ? ((size_t)p.chunks * rows * t_stride(r) * 4 + 255) / 256 * 256 : 0;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_adapters_down(const uint16_t* x, int64_t M, int64_t K, const Adapters& ad, int64_t r, float* part,
                                uint16_t* t, hipStream_t stream) {
  const int tr = (int)t_stride(r);
  const f16* L1 = reinterpret_cast<const f16*>(ad.L1);
  if (few_rows(M, K, r)) {
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
  for (int64_t m = 0; m < M; m += kRowsPerLaunch) {
    const int64_t mc = M - m < kRowsPerLaunch ? M - m : kRowsPerLaunch;
    const DownPlan p = down_plan(mc, K, r);
    f16* tm = reinterpret_cast<f16*>(t) + m * tr;
    hipLaunchKernelGGL(adapters_down_kernel, dim3((unsigned)((r + 15) / 16), (unsigned)((mc + 15) / 16),
                                                  (unsigned)p.chunks),
                       dim3(64 * kRowWaves), 0, stream, reinterpret_cast<const f16*>(x) + m * K, (int)mc, (int)K, L1,
                       ad.scale, (int)ad.n, (int)r, ad.row + m, tm, tr, (int)p.chunk, p.chunks > 1 ? part : nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.chunks > 1) {
      hipLaunchKernelGGL(adapters_finish_kernel, dim3((unsigned)((mc * tr + 255) / 256)), dim3(256), 0, stream, part,
                         (int)p.chunks, (int)mc, ad.scale, (int)ad.n, (int)r, ad.row + m, tm, tr);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace wq
