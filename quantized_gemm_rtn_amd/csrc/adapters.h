#pragma once
#include "wq_device.h"

namespace wq {

// Up-projections of the low-rank adapters that rows name, for a wave's NT 16-channel tiles of a decode kernel:
// acc[j] += t . L2_a^T, a = row[m]. For each adapter that rows m0 .. m0 + 15 name, one product of all of
// them, which its own rows keep (the others' sums may be anything: an adapter's infinities stay its own). The
// adapters are dealt to the block's waves in turn; their accumulators are summed at the end anyway.
template <int KW, int NT>
__device__ __forceinline__ void adapters_add16(f32x4 (&acc)[NT], const f16* t, const f16* up, int r,
                                               const int32_t* row, int n, int M, int N, int m0, int n0, int lane,
                                               int wave) {
  const int q = lane & 15, h = lane >> 4, tr = (r + 31) & ~31;
  const int id = row[min(m0 + q, M - 1)];
  uint32_t left = (uint32_t)__ballot((uint32_t)id < (uint32_t)n) & 0xFFFFu;
  const f16* ta = t + (size_t)min(m0 + q, M - 1) * tr + 8 * h;
  for (int turn = 0; left != 0; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t members = (uint32_t)__ballot(id == a) & left;
    left &= ~members;
    if (turn % KW != wave) continue;
    const f16* ub[NT];
    f32x4 own[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      ub[j] = up + ((size_t)a * N + min(n0 + 16 * j + q, N - 1)) * r;
      own[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int s = 0; s < r; s += 32) {
      const f16x8 av = as_f16x8(*reinterpret_cast<const uint4*>(ta + s));
      const int c = min(s + 8 * h, r - 8);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 b = *reinterpret_cast<const uint4*>(ub[j] + c);
        if (s + 8 * h >= r) b = uint4{0, 0, 0, 0};
        own[j] = mfma_16x16x32(av, as_f16x8(b), own[j]);
      }
    }
    const uint32_t mine = members >> (4 * h);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] += (mine >> i) & 1u ? own[j][i] : 0.0f;
  }
}

}  // namespace wq
