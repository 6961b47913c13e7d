#pragma once
#include "wq_device.h"

namespace wq {

// Up-projections of the low-rank adapters that rows name, for a wave's NT 16-channel tiles of a decode kernel:
// add[j] = t . L2_a^T, a = row[m]. For each adapter that rows m0 .. m0 + 15 name, one product of all of them, which its
// own rows keep (the others' sums may be anything: an adapter's infinities stay its own). The adapters are dealt to the
// block's KW waves in turn; the loads of a wave's go out together, with no branch between them. In us, no row / all rows
// of one / each row its own adapter: 64 rows of 8192 x 3584, rank 64, 23 / 29 / 40 (1 MB and 67 MB of L2), rank 16
// 23 / 26 / 31; 16 rows of it, rank 64, 11 / 13 / 17.
// Which wave has a row's adapter depends on what the other rows name. So the products are kept apart from the waves' own
// sums, and join them after those have met (reduce_store_tiles): a row's bits are its own.
template <int NT>
struct AdapterTiles {
  f32x4 add[NT];   // of this wave's rows
  uint32_t mine;   // rows of the tile whose adapter this wave has,
  uint32_t named;  // and those that have any
};

template <int KW, int NT>
__device__ __forceinline__ AdapterTiles<NT> adapters_up16(const f16* t, const f16* up, int r, int id, int n, int M, int N,
                                                          int m0, int n0, int lane, int wave) {
  constexpr int UN = 16 / KW;  // adapters of a wave, at most
  static_assert(UN * KW == 16, "waves");
  const int q = lane & 15, h = lane >> 4;
  uint32_t left = (uint32_t)__ballot((uint32_t)id < (uint32_t)n) & 0xFFFFu;
  AdapterTiles<NT> out;
#pragma unroll
  for (int j = 0; j < NT; ++j) out.add[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  out.mine = 0;
  out.named = left;
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
    out.mine |= members[v];
  }
  if (out.mine == 0) return out;
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
      const uint32_t rows = members[v] >> (4 * h);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (s + 8 * h >= r) bv[v][j] = uint4{0, 0, 0, 0};
        const f32x4 own = mfma_16x16x32(as_f16x8(av), as_f16x8(bv[v][j]), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) out.add[j][i] += (rows >> i) & 1u ? own[i] : 0.0f;
      }
    }
  }
  return out;
}

}  // namespace wq
