#pragma once
#include "wq_device.h"

namespace wq {

// Up-projections of the low-rank adapters that rows name, for a wave's NT 16-channel tiles of a decode kernel:
// acc[j] += t . L2_a^T, a = row[m]. For each adapter that rows m0 .. m0 + 15 name, one product of all of them, which its
// own rows keep (the others' sums may be anything: an adapter's infinities stay its own). The adapters are dealt to the
// block's KW waves in turn, whose accumulators are summed at the end anyway; the loads of a wave's go out together, with
// no branch between them. In us, no row / all rows of one / each row its own adapter: 64 rows of 8192 x 3584, rank 64,
// 23 / 29 / 40 (1 MB and 67 MB of L2), rank 16 23 / 26 / 31; 16 rows of it, rank 64, 11 / 13 / 16.
template <int KW, int NT>
__device__ __forceinline__ void adapters_add16(f32x4 (&acc)[NT], const f16* t, const f16* up, int r, int id, int n, int M,
                                               int N, int m0, int n0, int lane, int wave) {
  constexpr int UN = 16 / KW;  // adapters of a wave, at most
  static_assert(UN * KW == 16, "waves");
  const int q = lane & 15, h = lane >> 4;
  uint32_t left = (uint32_t)__ballot((uint32_t)id < (uint32_t)n) & 0xFFFFu;
  uint32_t members[UN];
  int ads[UN];
  int ad = 0;
#pragma unroll
  for (int v = 0; v < UN; ++v) {  // (none left: no rows, and the last one's loads again)
    members[v] = 0;
    for (int w = 0; w < KW && left != 0; ++w) {
      const int next = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      const uint32_t same = (uint32_t)__ballot(id == next) & left;
      left &= ~same;
      if (w == wave) {
        members[v] = same;
        ad = next;
      }
    }
    ads[v] = ad;
  }
  if (members[0] == 0) return;
  const f16* ta = t + (size_t)min(m0 + q, M - 1) * ((r + 31) & ~31) + 8 * h;
  for (int s = 0; s < r; s += 32) {
    const uint4 av = *reinterpret_cast<const uint4*>(ta + s);
    uint4 bv[UN][NT];
#pragma unroll
    for (int v = 0; v < UN; ++v)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        bv[v][j] = *reinterpret_cast<const uint4*>(up + ((size_t)ads[v] * N + min(n0 + 16 * j + q, N - 1)) * r +
                                                   min(s + 8 * h, r - 8));
#pragma unroll
    for (int v = 0; v < UN; ++v) {
      const uint32_t mine = members[v] >> (4 * h);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (s + 8 * h >= r) bv[v][j] = uint4{0, 0, 0, 0};
        const f32x4 own = mfma_16x16x32(as_f16x8(av), as_f16x8(bv[v][j]), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += (mine >> i) & 1u ? own[i] : 0.0f;
      }
    }
  }
}

}  // namespace wq
