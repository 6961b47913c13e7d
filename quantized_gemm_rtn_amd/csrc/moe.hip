// Expert routing and a mixture-of-experts layer for a few tokens, for gfx950.
//
//   route:    p = softmax(logits of a row), its top_k largest and their weights
//   experts:  y = sum over the row's experts e of w_e ((silu(x G_e^T) * (x U_e^T)) D_e^T),
//             silu(a) = a / (1 + exp(-a)), every matrix in 4 bits with (s, z) per 128 channels
//
// moe_up_kernel    one block for each active expert and 16 channels of its inner dimension: the
//   16 rows of G_e and of U_e, four waves splitting K, for all rows of x that name the expert.
//   h = silu(gate) * up is rounded once to fp16, the operand of the second product, and written
//   in the order that product's lanes read it.
// moe_down_kernel  one block for each 16 channels of the output: the 16 rows of D_e of every
//   active expert, one after the other, dealt out in equal shares to the block's waves, so the
//   sum over experts never leaves the block.
#include "gemv_kernels.h"

namespace wq {

constexpr int kMoeTokens = 192;     // rows of x that a block's lists hold; more come as further blocks
constexpr int kMoeMaxPairs = 1024;  // of them, (row, expert) pairs
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeWaves = 8;        // of a block, one block a CU
constexpr int kMoeUnit = 8;         // groups of 128 channels: what waves' shares are multiples of
constexpr int kMoeRowHalves = 136;  // of a staged row: 128 and padding (16 rows of a fragment in distinct banks)

// What some rows of x have to do, from their experts: the active experts in ascending order, each with its (row,
// expert) pairs, row * k + slot, in order. A row that names an expert twice has it once, with the weights' sum.
struct MoeLists {
  int32_t active, pad[3];             // experts
  uint16_t expert[kMoeMaxPairs];      // of the i-th active one,
  uint16_t start[kMoeMaxPairs + 8];   // its first pair (start[active]: their number),
  uint16_t tile[kMoeMaxPairs + 8];    // and its first tile of 16 pairs (tile[active]: theirs)
  uint16_t pair[kMoeMaxPairs];
};

struct MoeArgs {
  const f16* x;            // [M][H]
  const int32_t* experts;  // [M][k]
  const float* weights;    // [M][k]
  const uint32_t* up;      // [E][2I][H / 8], the gate's rows first
  const f16* up_s;
  const f16* up_z;
  const uint32_t* down;    // [E][H][I / 8]
  const f16* down_s;
  const f16* down_z;
  f16* h;                  // [M * k][I], each eight channels in the order of perm_x8
  MoeLists* lists;         // of each `tokens` rows
  void* y;
  int M, H, I, E, k, y_f32;
  int tokens;
};

__device__ __forceinline__ int sum_upto_64(int v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(v, off);
    v += lane >= off ? u : 0;
  }
  return v;
}

// The lists of rows m0 .. m0 + rows - 1, by the block, in its LDS.
struct MoeScratch {
  int16_t ids[kMoeMaxPairs];
  int32_t count[kMoeMaxExperts];
  int32_t sums[kMoeWaves][2];
};
__device__ __forceinline__ void moe_lists(MoeLists& l, MoeScratch& w, const MoeArgs& a, int m0, int rows) {
  constexpr int T = 64 * kMoeWaves, PER = kMoeMaxPairs / T, EPER = kMoeMaxExperts / T;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, pairs = rows * a.k;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + T * i;
    const int e = p < pairs ? a.experts[(int64_t)m0 * a.k + p] : -1;
    w.ids[p] = (int16_t)((uint32_t)e < (uint32_t)a.E ? e : -1);
  }
#pragma unroll
  for (int i = 0; i < EPER; ++i) w.count[EPER * t + i] = 0;
  __syncthreads();
  int place[PER], made[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + T * i, e = w.ids[p];
    bool first = e >= 0;
    if (first)
      for (int q = p / a.k * a.k; q < p; ++q) first = first && w.ids[q] != e;
    place[i] = first ? atomicAdd(&w.count[e], 1) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) made[i] = place[i] >= 0 ? w.count[w.ids[t + T * i]] : 0;  // pairs of the pair's expert
  // experts EPER t .. + EPER - 1: active ones and pairs before them (in one sum), and tiles
  int own[EPER], both = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < EPER; ++i) {
    own[i] = w.count[EPER * t + i];
    both += own[i] + (own[i] > 0 ? 1 << 16 : 0);
    tiles += (own[i] + 15) >> 4;
  }
  const int both_upto = sum_upto_64(both, lane), tiles_upto = sum_upto_64(tiles, lane);
  if (lane == 63) {
    w.sums[wave][0] = both_upto;
    w.sums[wave][1] = tiles_upto;
  }
  __syncthreads();
  int before = both_upto - both, tile = tiles_upto - tiles, total = 0, all = 0;
#pragma unroll
  for (int v = 0; v < kMoeWaves; ++v) {
    before += v < wave ? w.sums[v][0] : 0;
    tile += v < wave ? w.sums[v][1] : 0;
    total += w.sums[v][0];
    all += w.sums[v][1];
  }
#pragma unroll
  for (int i = 0; i < EPER; ++i)
    if (own[i] > 0) {
      l.expert[before >> 16] = (uint16_t)(EPER * t + i);
      l.start[before >> 16] = (uint16_t)before;
      l.tile[before >> 16] = (uint16_t)tile;
      w.count[EPER * t + i] = before & 0xFFFF;  // where its pairs begin
      before += own[i] + (1 << 16);
      tile += (own[i] + 15) >> 4;
    }
  if (t == 0) {
    l.active = total >> 16;
    l.start[total >> 16] = (uint16_t)total;
    l.tile[total >> 16] = (uint16_t)all;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (place[i] >= 0) l.pair[w.count[w.ids[t + T * i]] + place[i]] = (uint16_t)(t + T * i);
  __syncthreads();
  // in order (the atomics' is any): a pair's tile decides where its sums are split
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + T * i;
    if (place[i] >= 0) {
      const int from = w.count[w.ids[p]];
      int rank = 0;
      for (int q = from; q < from + made[i]; ++q) rank += l.pair[q] < p ? 1 : 0;
      place[i] = from + rank;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (place[i] >= 0) l.pair[place[i]] = (uint16_t)(t + T * i);
  __syncthreads();
}

// The active expert whose tiles hold tile `at` (at < tile[active]), the same in all lanes.
__device__ __forceinline__ int moe_expert_of(const MoeLists& l, int active, int at, int lane) {
  int i = 0;
  for (int first = 0; first < active; first += 64) {
    const int n = __popcll(__ballot(first + lane < active && l.tile[min(first + lane, active - 1) + 1] <= at));
    i += n;
    if (n < 64) break;
  }
  return i;
}

// The weight of a pair: of its slot and of later ones with the same expert.
__device__ __forceinline__ float moe_weight(const MoeArgs& a, int m0, int pair, int e) {
  const int row = pair / a.k;
  const int64_t at = (int64_t)m0 * a.k;
  float w = 0.0f;
  for (int q = pair; q < (row + 1) * a.k; ++q) w += a.experts[at + q] == e ? a.weights[at + q] : 0.0f;
  return w;
}

// (s, z) of a unit's groups for a lane's row of weights: one load of each where rows begin at multiples of eight
// groups, else a load a group.
template <bool VEC>
struct MoeSz;
template <>
struct MoeSz<true> {
  uint4 s, z;
  __device__ __forceinline__ void load(const f16* sp, const f16* zp, int g, int) {
    s = *reinterpret_cast<const uint4*>(sp + g);
    z = *reinterpret_cast<const uint4*>(zp + g);
  }
  __device__ __forceinline__ f16 scale(int i) const { return half_of(s, i); }
  __device__ __forceinline__ f16 zero(int i) const { return half_of(z, i); }
};
template <>
struct MoeSz<false> {
  uint32_t s[kMoeUnit], z[kMoeUnit];
  __device__ __forceinline__ void load(const f16* sp, const f16* zp, int g, int last) {
#pragma unroll
    for (int i = 0; i < kMoeUnit; ++i) {
      s[i] = reinterpret_cast<const uint16_t*>(sp)[min(g + i, last)];
      z[i] = reinterpret_cast<const uint16_t*>(zp)[min(g + i, last)];
    }
  }
  __device__ __forceinline__ f16 scale(int i) const { return bits_to_f16((uint16_t)s[i]); }
  __device__ __forceinline__ f16 zero(int i) const { return bits_to_f16((uint16_t)z[i]); }
};

// acc[j] += x . w[j]^T over groups g0 .. g0 + ng - 1 (g0 a multiple of kMoeUnit), for 16 rows of x and NW tiles of 16
// rows of weights, by one wave: D groups are in flight, each group's rows of x pass through the wave's slot of LDS
// into the order of the product's operand (4 XL rows; PERM: reordered to the codes' on the way).
//  w[j], sp[j], zp[j]: of the lane's row of weights, group 0 (w: its four words of a group).
//  xp[j]: the lane's eight channels of group 0 of row h + 4 j.
template <int NW, int XL, int D, bool VEC, bool PERM>
__device__ __forceinline__ void moe_stream(f32x4 (&acc)[NW], const uint32_t* const (&w)[NW],
                                           const f16* const (&sp)[NW], const f16* const (&zp)[NW],
                                           const f16* const (&xp)[XL], f16* slot, int g0, int ng, int lane) {
  static_assert(kMoeUnit % D == 0, "slots of a unit");
  const int r = lane & 15, h = lane >> 4;
  const uint32_t magic = magic_1024x2();
  const f16* frag = slot + min(r, 4 * XL - 1) * kMoeRowHalves + 32 * h;
  const int last = g0 + ng - 1;
  uint4 wbuf[D][NW], xbuf[D][XL];
  MoeSz<VEC> sz[NW], next[NW];
  const auto fetch = [&](int i, int g) {
#pragma unroll
    for (int j = 0; j < NW; ++j) wbuf[i][j] = *reinterpret_cast<const uint4*>(w[j] + (int64_t)g * 16);
#pragma unroll
    for (int j = 0; j < XL; ++j) xbuf[i][j] = *reinterpret_cast<const uint4*>(xp[j] + (int64_t)g * 128);
  };
  const auto group = [&](int i, int u) {  // slot i, u-th of its unit
#pragma unroll
    for (int j = 0; j < XL; ++j)
      *reinterpret_cast<uint4*>(slot + (h + 4 * j) * kMoeRowHalves + 8 * r) = PERM ? perm_x8(xbuf[i][j]) : xbuf[i][j];
    uint4 xa[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) xa[s] = *reinterpret_cast<const uint4*>(frag + 8 * s);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const f16 b = (f16)1024.0f + sz[j].zero(u), nb = (f16)960.0f - b;
      f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s)
        part = mfma_16x16x32(as_f16x8(xa[s]),
                             as_f16x8(step_operand<false>(wbuf[i][j], s, magic, f16x2{b, b}, f16x2{nb, nb}, f16x2{})),
                             part);
      acc[j] += (float)sz[j].scale(u) * part;
    }
  };
#pragma unroll
  for (int j = 0; j < NW; ++j) next[j].load(sp[j], zp[j], g0, last);
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(i, min(g0 + i, last));
  int g = g0;
  for (; g + kMoeUnit <= last; g += kMoeUnit) {  // (a unit with another after it is whole)
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      sz[j] = next[j];
      next[j].load(sp[j], zp[j], g + kMoeUnit, last);
    }
#pragma unroll
    for (int u = 0; u < kMoeUnit; ++u) {
      group(u % D, u);
      fetch(u % D, min(g + u + D, last));
      __builtin_amdgcn_sched_barrier(kSchedKeepGroups);  // the refill stays next to its consumption
    }
  }
#pragma unroll
  for (int j = 0; j < NW; ++j) sz[j] = next[j];
#pragma unroll
  for (int u = 0; u < kMoeUnit; ++u) {
    if (g + u <= last) {
      group(u % D, u);
      if constexpr (D < kMoeUnit)
        if (u + D < kMoeUnit) fetch(u % D, min(g + u + D, last));
    }
  }
}

// h of 16 pairs and 16 inner channels from their sums: rows 4 (lane / 16) + i
__device__ __forceinline__ void moe_store_h(const MoeArgs& a, const MoeLists& l, const f32x4 (&acc)[2], int m0, int c0,
                                            int first, int count, int lane) {
  const int r = lane & 15, h = lane >> 4, at = c0 + (r & 8) + perm_slot(r & 7);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * h + i;
    if (row < count) {
      const float gate = acc[0][i], v = gate / (1.0f + expf(-gate)) * acc[1][i];
      a.h[((int64_t)m0 * a.k + l.pair[first + row]) * a.I + at] = (f16)v;
    }
  }
}

struct MoeUpLds {
  MoeLists l;
  MoeScratch scratch;
  f32x4 part[kMoeWaves][2][2][64];  // a wave's sums of an item that it shares: the one it goes on with, the one it begins
  f16 slot[kMoeWaves][16 * kMoeRowHalves];
};

template <bool VEC>
__global__ void __launch_bounds__(64 * kMoeWaves)
moe_up_kernel(MoeArgs a) {
  extern __shared__ __align__(16) char smem[];
  MoeUpLds& lds = *reinterpret_cast<MoeUpLds*>(smem);
  const MoeLists& l = lds.l;
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = blockIdx.y * a.tokens, rows = min(a.tokens, a.M - m0);
  moe_lists(lds.l, lds.scratch, a, m0, rows);
  if (blockIdx.x == 0) {  // for the second product
    int32_t* out = reinterpret_cast<int32_t*>(a.lists + blockIdx.y);
    const int32_t* in = reinterpret_cast<const int32_t*>(&l);
    for (int i = t; i < (int)(sizeof(MoeLists) / 4); i += 64 * kMoeWaves) out[i] = in[i];
  }
  const int active = __builtin_amdgcn_readfirstlane(l.active);
  const int G = a.H >> 7, U = (G + kMoeUnit - 1) / kMoeUnit, C = a.I >> 4;
  // items: (expert, 16 channels, 16 pairs), the pairs fastest; the block's, whole, and the wave's share of their units
  const int64_t items = (int64_t)l.tile[active] * C;
  const int64_t i_lo = items * blockIdx.x / gridDim.x, i_hi = items * (blockIdx.x + 1) / gridDim.x;
  const int64_t units = (i_hi - i_lo) * U;
  const int64_t u_lo = units * wave / kMoeWaves, u_hi = units * (wave + 1) / kMoeWaves;
  int which = 0;
  int open_c0 = 0, open_first = 0, open_count = 0;  // of the item that the wave begins and others finish
  int64_t open_end = 0;
  if (u_lo < u_hi) which = moe_expert_of(l, active, (int)((i_lo + u_lo / U) / C), lane);
  for (int64_t u = u_lo; u < u_hi;) {
    const int64_t item = i_lo + u / U;
    const int q = (int)(u % U), n_units = (int)(U - q < u_hi - u ? U - q : u_hi - u);
    while (item >= (int64_t)l.tile[which + 1] * C) ++which;
    const int e = __builtin_amdgcn_readfirstlane(l.expert[which]);
    const int tiles = __builtin_amdgcn_readfirstlane(l.tile[which + 1] - l.tile[which]);
    const int rem = (int)(item - (int64_t)l.tile[which] * C);
    const int c0 = 16 * (rem / tiles), r0 = 16 * (rem % tiles);
    const int first = l.start[which] + r0, count = min(16, (int)l.start[which + 1] - first);
    const uint32_t* w[2];
    const f16 *sp[2], *zp[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = ((int64_t)e * 2 + j) * a.I + c0 + r;
      w[j] = a.up + n * (16 * G) + 4 * h;
      sp[j] = a.up_s + n * G;
      zp[j] = a.up_z + n * G;
    }
    const int g0 = kMoeUnit * q, ng = min(kMoeUnit * n_units, G - g0);
    const auto row_of = [&](int row) {
      return a.x + (int64_t)(m0 + l.pair[first + min(row, count - 1)] / a.k) * a.H + 8 * r;
    };
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (count <= 4) {
      const f16* xp[1] = {row_of(h)};
      moe_stream<2, 1, 8, VEC, true>(acc, w, sp, zp, xp, lds.slot[wave], g0, ng, lane);
    } else {
      const f16* xp[4] = {row_of(h), row_of(h + 4), row_of(h + 8), row_of(h + 12)};
      moe_stream<2, 4, 4, VEC, true>(acc, w, sp, zp, xp, lds.slot[wave], g0, ng, lane);
    }
    u += n_units;
    if (n_units == U) {
      moe_store_h(a, l, acc, m0, c0, first, count, lane);
    } else {
      const int begun = q == 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) lds.part[wave][begun][j][lane] = acc[j];
      if (begun) {
        open_end = u - n_units + U;
        open_c0 = c0;
        open_first = first;
        open_count = count;
      }
    }
  }
  __syncthreads();
  if (open_count > 0) {
    f32x4 acc[2] = {lds.part[wave][1][0][lane], lds.part[wave][1][1][lane]};
    for (int v = wave + 1; v < kMoeWaves && units * v / kMoeWaves < open_end; ++v) {
      if (units * v / kMoeWaves == units * (v + 1) / kMoeWaves) continue;  // (a wave without units)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[j] += lds.part[v][0][j][lane];
    }
    moe_store_h(a, l, acc, m0, open_c0, open_first, open_count, lane);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(64 * kMoeWaves)
moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) char smem[];
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = blockIdx.y * a.tokens, rows = min(a.tokens, a.M - m0);
  MoeLists& l = *reinterpret_cast<MoeLists*>(smem);
  f16* slot = reinterpret_cast<f16*>(smem + sizeof(MoeLists)) + wave * 16 * kMoeRowHalves;
  float* sums = reinterpret_cast<float*>(smem + sizeof(MoeLists) + kMoeWaves * 16 * kMoeRowHalves * 2);  // [wave][rows][16]
  float* mine = sums + wave * rows * 16;
  {
    const uint4* in = reinterpret_cast<const uint4*>(a.lists + blockIdx.y);
    for (int i = t; i < (int)(sizeof(MoeLists) / 16); i += 64 * kMoeWaves) reinterpret_cast<uint4*>(&l)[i] = in[i];
  }
  for (int i = lane; i < rows * 16; i += 64) mine[i] = 0.0f;
  __syncthreads();
  const int active = __builtin_amdgcn_readfirstlane(l.active);
  const int n0 = blockIdx.x * 16, G = a.I >> 7, U = (G + kMoeUnit - 1) / kMoeUnit;
  // items: (expert, 16 pairs); the wave's share of their units
  const int units = l.tile[active] * U;
  const int u_lo = units * wave / kMoeWaves, u_hi = units * (wave + 1) / kMoeWaves;
  int which = u_lo < u_hi ? moe_expert_of(l, active, u_lo / U, lane) : 0;
  for (int u = u_lo; u < u_hi;) {
    const int item = u / U, q = u % U, n_units = min(U - q, u_hi - u);
    while (item >= l.tile[which + 1]) ++which;
    const int e = __builtin_amdgcn_readfirstlane(l.expert[which]);
    const int first = l.start[which] + 16 * (item - l.tile[which]);
    const int count = min(16, (int)l.start[which + 1] - first);
    const int64_t n = (int64_t)e * a.H + n0 + r;
    const uint32_t* w[1] = {a.down + n * (16 * G) + 4 * h};
    const f16 *sp[1] = {a.down_s + n * G}, *zp[1] = {a.down_z + n * G};
    const int g0 = kMoeUnit * q, ng = min(kMoeUnit * n_units, G - g0);
    const auto row_of = [&](int row) {
      return a.h + ((int64_t)m0 * a.k + l.pair[first + min(row, count - 1)]) * a.I + 8 * r;
    };
    f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    if (count <= 4) {
      const f16* xp[1] = {row_of(h)};
      moe_stream<1, 1, 8, VEC, false>(acc, w, sp, zp, xp, slot, g0, ng, lane);
    } else {
      const f16* xp[4] = {row_of(h), row_of(h + 4), row_of(h + 8), row_of(h + 12)};
      moe_stream<1, 4, 8, VEC, false>(acc, w, sp, zp, xp, slot, g0, ng, lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * h + i;
      if (row < count) {
        const int p = l.pair[first + row];
        mine[p / a.k * 16 + r] += moe_weight(a, m0, p, e) * acc[0][i];
      }
    }
    u += n_units;
  }
  __syncthreads();
  for (int i = t; i < rows * 16; i += 64 * kMoeWaves) {
    float v = sums[i];
    for (int k = 1; k < kMoeWaves; ++k) v += sums[k * rows * 16 + i];
    const int64_t o = (int64_t)(m0 + (i >> 4)) * a.H + n0 + (i & 15);
    if (a.y_f32)
      static_cast<float*>(a.y)[o] = v;
    else
      static_cast<f16*>(a.y)[o] = (f16)v;
  }
}

static int64_t moe_tokens(int64_t M, int64_t k) {
  const int64_t most = kMoeMaxPairs / k < kMoeTokens ? kMoeMaxPairs / k : kMoeTokens;
  return M < most ? M : most;
}
static int64_t moe_chunks(int64_t M, int64_t k) { return (M + moe_tokens(M, k) - 1) / moe_tokens(M, k); }
static size_t moe_h_bytes(int64_t M, int64_t I, int64_t k) { return ((size_t)(M * k) * I * 2 + 255) / 256 * 256; }

size_t moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t k) {
  return moe_h_bytes(M, I, k) + (size_t)moe_chunks(M, k) * sizeof(MoeLists);
}

hipError_t launch_moe_experts(const uint16_t* x, int64_t M, int64_t H, const int32_t* experts, const float* weights,
                              int64_t k, int64_t E, const uint32_t* up, const uint16_t* up_s, const uint16_t* up_z,
                              int64_t I, const uint32_t* down, const uint16_t* down_s, const uint16_t* down_z, void* y,
                              int y_f32, void* workspace, hipStream_t stream) {
  MoeArgs a;
  a.x = reinterpret_cast<const f16*>(x);
  a.experts = experts;
  a.weights = weights;
  a.up = up;
  a.up_s = reinterpret_cast<const f16*>(up_s);
  a.up_z = reinterpret_cast<const f16*>(up_z);
  a.down = down;
  a.down_s = reinterpret_cast<const f16*>(down_s);
  a.down_z = reinterpret_cast<const f16*>(down_z);
  a.h = static_cast<f16*>(workspace);
  a.lists = reinterpret_cast<MoeLists*>(static_cast<char*>(workspace) + moe_h_bytes(M, I, k));
  a.y = y;
  a.M = (int)M;
  a.H = (int)H;
  a.I = (int)I;
  a.E = (int)E;
  a.k = (int)k;
  a.y_f32 = y_f32;
  a.tokens = (int)moe_tokens(M, k);
  const unsigned chunks = (unsigned)moe_chunks(M, k);
  const auto vec = [](int64_t K, const void* s, const void* z) {  // rows of (s, z) begin at multiples of 16 bytes
    return K / 128 % 8 == 0 && ((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  };
  // a block a CU, or fewer where there are fewer items
  const int64_t pairs = a.tokens * k, tiles = pairs < E + pairs / 16 ? pairs : E + pairs / 16;
  const int64_t items = tiles * (I / 16);
  const auto up_kernel = vec(H, up_s, up_z) ? moe_up_kernel<true> : moe_up_kernel<false>;
  hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(up_kernel), sizeof(MoeUpLds));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(up_kernel, dim3((unsigned)(items < kNumCu ? items : kNumCu), chunks), dim3(64 * kMoeWaves),
                     sizeof(MoeUpLds), stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const auto down_kernel = vec(I, down_s, down_z) ? moe_down_kernel<true> : moe_down_kernel<false>;
  const size_t lds = sizeof(MoeLists) + kMoeWaves * (16 * kMoeRowHalves * 2 + (size_t)a.tokens * 64);
  e = set_dynamic_lds(reinterpret_cast<const void*>(down_kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(down_kernel, dim3((unsigned)(H / 16), chunks), dim3(64 * kMoeWaves), lds, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Largest value over the wave's 64 lanes, in all of them.
__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v = max(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// A logit as an integer of the same order, NaN the largest, and back; kMasked: -infinity, which
// is never chosen.
constexpr int kMasked = (int)0x80000000;
__device__ __forceinline__ int logit_key(float v) {
  if (v != v) return 0x7FFFFFFF;
  if (v == -INFINITY) return kMasked;
  const int b = __builtin_bit_cast(int, v + 0.0f);  // (-0 is 0)
  return b < 0 ? b ^ 0x7FFFFFFF : b;
}
__device__ __forceinline__ float key_logit(int key) {
  return __builtin_bit_cast(float, key < 0 ? key ^ 0x7FFFFFFF : key);
}

// One wave a row, V neighbouring logits a lane: equal ones are then in order of lane and place,
// and a round takes the first lane that holds the largest.
template <typename T, int V>
__global__ void __launch_bounds__(256)
moe_route_kernel(const T* __restrict__ logits, int M, int E, int k, int renormalize, int32_t* __restrict__ experts,
                 float* __restrict__ weights) {
  const int lane = threadIdx.x & 63, row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= M) return;
  const T* in = logits + (int64_t)row * E;
  float x[V];
  int key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    x[v] = e < E ? (float)in[e] : -INFINITY;
    key[v] = logit_key(x[v]);
  }
  float top = 0.0f, chosen = 0.0f, p = 0.0f;  // of lane j: the j-th choice's
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    int best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    const int most = wave_max(best);
    if (most == kMasked) break;
    const int at = __builtin_ctzll(__ballot(best == most));
    int place = V - 1;
#pragma unroll
    for (int v = V - 2; v >= 0; --v) place = key[v] == most ? v : place;
    const int e = __builtin_amdgcn_readlane(lane * V + place, at);
    if (lane == at) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = v == place ? kMasked : key[v];
    }
    const float value = key_logit(most);
    if (j == 0) top = value;
    const float w = expf(value - top);
    chosen += w;
    if (lane == j) {
      mine = e;
      p = w;
    }
  }
  float total = chosen;
  if (!renormalize) {
    total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) total += x[v] == -INFINITY ? 0.0f : expf(x[v] - top);
    total = wave_sum(total);
  }
  if (lane < k) {
    experts[(int64_t)row * k + lane] = mine;
    weights[(int64_t)row * k + lane] = mine < 0 ? 0.0f : p / total;
  }
}

template <typename T>
static hipError_t route(const T* logits, int64_t M, int64_t E, int64_t k, int renormalize, int32_t* experts,
                        float* weights, hipStream_t stream) {
  const dim3 grid((unsigned)((M + 3) / 4));
#define WQ_ROUTE(V)                                                                                              \
  hipLaunchKernelGGL((moe_route_kernel<T, V>), grid, dim3(256), 0, stream, logits, (int)M, (int)E, (int)k,       \
                     renormalize, experts, weights)
  if (E <= 64)
    WQ_ROUTE(1);
  else if (E <= 128)
    WQ_ROUTE(2);
  else if (E <= 256)
    WQ_ROUTE(4);
  else if (E <= 512)
    WQ_ROUTE(8);
  else
    WQ_ROUTE(16);
#undef WQ_ROUTE
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int f32, int64_t M, int64_t E, int64_t k, int renormalize,
                            int32_t* experts, float* weights, hipStream_t stream) {
  return f32 ? route(static_cast<const float*>(logits), M, E, k, renormalize, experts, weights, stream)
             : route(static_cast<const f16*>(logits), M, E, k, renormalize, experts, weights, stream);
}

}  // namespace wq
