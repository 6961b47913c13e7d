// Expert routing and a mixture-of-experts layer for a few tokens, for gfx950.
//
//   route:    p = softmax(logits of a row), its top_k largest and their weights
//   experts:  y = sum over the row's experts e of w_e ((silu(x G_e^T) * (x U_e^T)) D_e^T),
//             silu(a) = a / (1 + exp(-a)), every matrix in 4 bits with (s, z) per 128 channels
//
// The layer's bound is the bytes of the experts that rows name: 17/32 of a byte a weight, read once for each 32 rows of an
// expert (a copy of 2 + 2 GiB runs at 4.95 TB/s on this card; the floors below are at that rate).
//
// moe_rows_kernel     Both products, G_e and U_e together and then D_e. The work is items, (an expert, 64 rows of its
//   weights, up to 32 of its (row, expert) pairs), dealt in turn to one block of eight waves a CU; a block's groups of 128
//   channels are cut into equal shares for its waves, wherever an item begins or ends, and what waves share of an item is
//   summed through LDS in the order of the waves. So all CUs have the same bytes to read, for any experts and sizes: one
//   block for an expert and 16 channels took 403 us where 16 rows name eight experts of 4096 x 14336, this split 171
//   (floor 151). Rows of x pass through a slot of LDS of the wave's own, which orders them as the matrix operand; nothing
//   in the loop waits for another wave. The lists of who needs what are made by every block of the first product for itself
//   (a launch of their own would be another wait for the whole card), and left for the second.
//   h = silu(gate) * up is rounded once to fp16, the operand of the second product, and written in the order that
//   product's lanes read it. The second product leaves each pair's sums in fp32, which moe_join_kernel weights and adds
//   in the order of the row's slots.
// moe_down_few_kernel The second product and the join for up to 4 rows: one block for 16 channels of the output, all
//   experts' groups shared out among its waves, each with its sums in LDS: no third launch (one token of two experts of
//   4096 x 14336: 31 + 17 us, 5.1 TB/s besides some 5 us a launch to begin and end; floor 38).
//
// What holds the large batches back (150 rows of four of 32 experts of 4096 x 1536: 79 + 45 + 5 us, floor 65) is the path
// for 17 to 32 pairs: 3 TB/s of weights where up to 4 pairs run at 4.5. Neither its vector instructions (28 us of the 79 on
// each SIMD), its matrix instructions (8 us), the rows of x that it reads nor the order of its instructions is the bound:
// changing each made no difference. Cutting the shares by cost instead of by groups was slower (batch of 16: 193 us).
#include "gemv_kernels.h"

namespace wq {

// Rows of x that a block's lists hold; more come as further blocks, which read the weights again. As many as their
// pairs allow, but where all of 1024 rows name one expert, whose pairs a block puts in order alone. In us, at most 192 /
// 256 / 512 / 1024 rows: 256 rows, four of 32 experts of 4096 x 1536, 207 / 160 / 161 / 161; 512 rows, two of them, 251 /
// 193 / 162 / 161; 512 rows, two of eight of 4096 x 14336, 1003 / 910 / 805 / 809; 1024 rows, one of 64 of 2048 x 1024,
// 279 / 205 / 121 / 78; 1024 rows that all name the same of 16 of 1024 x 512, 87 / 77 / 76 / 91.
constexpr int kMoeTokens = 512;
constexpr int kMoeMaxPairs = 1024;  // of them, (row, expert) pairs
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeWaves = 8;        // of a block, one block a CU
constexpr int kMoeUnit = 8;         // groups of 128 channels whose (s, z) a wave has in its table
constexpr int kMoePairs = 32;       // (row, expert) pairs of an item
// Rows of a batch up to which the kernels for few rows run: as many as one load of a group brings (in us, these kernels /
// the general ones, one and four rows: two of eight experts of 4096 x 14336 48.6 / 66.9 and 110 / 131, eight of 64 of
// 2048 x 1024 19.6 / 30.4 and 46.5 / 43.9, six of 60 of 2176 x 1408 23.2 / 29.5 and 49.6 / 46.1).
constexpr int kMoeFew = 4;
constexpr int kMoeRowHalves = 136;  // of a staged row: 128 and padding (16 rows of a fragment in distinct banks)

// What some rows of x have to do, from their experts: the active experts, those of the most pairs first (so that items
// dealt out in turn make equal sums), each with its (row, expert) pairs, row * k + slot, in order. A row that names an
// expert twice has it once, with the weights' sum.
struct MoeLists {
  int32_t active, pad[3];             // experts
  uint16_t expert[kMoeMaxPairs];      // of the i-th active one,
  uint16_t start[kMoeMaxPairs + 8];   // its first pair (start[active]: their number),
  uint16_t tile[kMoeMaxPairs + 8];    // and its first tile of kMoePairs pairs (tile[active]: theirs)
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
  float* v;                // [M * k][H]: the pairs' sums, unless few rows
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
  int32_t sums[kMoeWaves][3];
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
    const int begin = p / a.k * a.k;
    for (int j = 0; j < a.k - 1; j += 4) {  // earlier slots of the row, four reads at a time
      int other[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) other[v] = w.ids[min(begin + j + v, p)];
#pragma unroll
      for (int v = 0; v < 4; ++v) first = first && !(begin + j + v < p && other[v] == e);
    }
    place[i] = first ? atomicAdd(&w.count[e], 1) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) made[i] = place[i] >= 0 ? w.count[w.ids[t + T * i]] : 0;  // pairs of the pair's expert
  // experts EPER t .. + EPER - 1: pairs, tiles beyond an expert's first, and active ones, in one sum (11, 6 and 11 bits)
  // for each class of experts: of more than 16 pairs, of more than 4, the others, whose items take moe_rows_kernel's three
  // ways of unequal length (16 rows through small experts 85.2 us, in the experts' own order 88.5, 150 drafted 134 and 138)
  const auto packed = [](int n) { return n == 0 ? 0 : n | ((n - 1) / kMoePairs) << 11 | 1 << 17; };
  const auto class_of = [](int n) { return n > 16 ? 0 : (n > 4 ? 1 : 2); };
  int own[EPER], sum[3] = {0, 0, 0}, before[3];
#pragma unroll
  for (int i = 0; i < EPER; ++i) {
    own[i] = w.count[EPER * t + i];
#pragma unroll
    for (int c = 0; c < 3; ++c) sum[c] += class_of(own[i]) == c ? packed(own[i]) : 0;
  }
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    const int upto = sum_upto_64(sum[c], lane);
    if (lane == 63) w.sums[wave][c] = upto;
    before[c] = upto - sum[c];
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    before[c] += total;
#pragma unroll
    for (int v = 0; v < kMoeWaves; ++v) {
      before[c] += v < wave ? w.sums[v][c] : 0;
      total += w.sums[v][c];
    }
  }
  const auto put = [&](int at, int v) {
    l.start[at] = (uint16_t)(v & 2047);
    l.tile[at] = (uint16_t)(at + ((v >> 11) & 63));
  };
#pragma unroll
  for (int i = 0; i < EPER; ++i)
    if (own[i] > 0) {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (class_of(own[i]) == c) {
          l.expert[before[c] >> 17] = (uint16_t)(EPER * t + i);
          put(before[c] >> 17, before[c]);
          w.count[EPER * t + i] = before[c] & 2047;  // where its pairs begin
          before[c] += packed(own[i]);
        }
    }
  if (t == 0) {
    l.active = total >> 17;
    put(total >> 17, total);
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
      for (int q = 0; q < made[i]; q += 8) {  // eight reads at a time
        int other[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) other[v] = l.pair[from + min(q + v, made[i] - 1)];
#pragma unroll
        for (int v = 0; v < 8; ++v) rank += q + v < made[i] && other[v] < p ? 1 : 0;
      }
      place[i] = from + rank;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (place[i] >= 0) l.pair[place[i]] = (uint16_t)(t + T * i);
  __syncthreads();
}

// The same for up to 64 pairs, by the block's first wave: a pair a lane, the experts in the order of their first pairs.
__device__ __forceinline__ void moe_few_lists(MoeLists& l, const MoeArgs& a, int rows) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, pairs = rows * a.k, row = lane / a.k;
    const int id = lane < pairs ? a.experts[lane] : -1;
    const uint64_t below = ((uint64_t)1 << lane) - 1, row_below = below & ~(((uint64_t)1 << row * a.k) - 1);
    uint64_t left = __ballot((uint32_t)id < (uint32_t)a.E);
    int n = 0, at = 0;
    for (; left != 0; ++n) {
      const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      const uint64_t same = __ballot(id == e);
      const bool first = id == e && (same & row_below) == 0;
      const uint64_t members = __ballot(first);
      if (first) l.pair[at + __popcll(members & below)] = (uint16_t)lane;
      if (lane == 0) {
        l.expert[n] = (uint16_t)e;
        l.start[n] = (uint16_t)at;
        l.tile[n] = (uint16_t)n;
      }
      at += __popcll(members);
      left &= ~same;
    }
    if (lane == 0) {
      l.active = n;
      l.start[n] = (uint16_t)at;
      l.tile[n] = (uint16_t)n;
    }
  }
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

// NW tiles of 16 rows of one expert's weights: bases that all lanes share, and offsets in 32 bits. The lane's row of a tile
// is lane % 16 (w: its four words of a group); its (s, z) row is that of tile lane / 16 % NW.
template <int NW>
struct MoeTiles {
  const uint8_t* w[NW];
  const uint8_t *s, *z;   // of the expert
  uint32_t w_off, s_off;  // bytes
  uint32_t s_end;         // from s to the array's end, at most 2^31
  // tile j begins at row n[j] of the expert's `rows`
  __device__ __forceinline__ void set(const uint32_t* w0, const f16* s0, const f16* z0, int e, int E, int rows,
                                      const int (&n)[NW], int G, int lane) {
    int mine = n[0];
    const int64_t row0 = (int64_t)e * rows;
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      w[j] = reinterpret_cast<const uint8_t*>(w0) + (row0 + n[j]) * (64 * G);
      mine = (lane >> 4) % NW == j ? n[j] : mine;
    }
    w_off = (uint32_t)(lane & 15) * (64 * G) + 16 * (lane >> 4);
    s = reinterpret_cast<const uint8_t*>(s0) + row0 * (2 * G);
    z = reinterpret_cast<const uint8_t*>(z0) + row0 * (2 * G);
    s_off = (uint32_t)(mine + (lane & 15)) * (2 * G);
    const int64_t left = (int64_t)(E - e) * rows * (2 * G);
    s_end = (uint32_t)(left < (int64_t)1 << 31 ? left : (int64_t)1 << 31);
  }
};
struct __attribute__((packed, aligned(2))) EightHalves {
  uint4 v;
};

// acc[i][j] += x . w[j]^T over groups g0 .. g0 + ng - 1, for 16 MT rows of x and NW tiles of
// weights, by one wave: D groups are in flight; each group's rows of x pass through the wave's slot of LDS into the
// order of the product's operand (4 XL rows; PERM: reordered to the codes' on the way), and a unit's (s, 1024 + z)
// through its table, loaded a tile for each 16 lanes, at any alignment, for two units at once (for one, the rest of the
// line has mostly left the L2 when the next unit asks for it: the batch of 16 561 instead of 543 MB, 4 us more). Two
// groups' weights, the halves of 128-byte lines, are asked for together (apart: 2 us more of 130).
//  xs + xo[j] bytes: the lane's eight channels of group 0 of row lane / 16 + 4 j.
template <int MT, int NW, int XL, int D, bool PERM>
__device__ __forceinline__ void moe_stream(f32x4 (&acc)[MT][NW], const MoeTiles<NW>& tiles, const uint8_t* xs,
                                           const uint32_t (&xo)[XL], f16* slot, uint32_t* table, int g0, int ng, int lane) {
  static_assert(kMoeUnit % D == 0 && XL <= 4 * MT && (MT == 1 || XL == 4 * MT), "slots of a unit, rows");
  const int r = lane & 15, h = lane >> 4;
  const uint32_t magic = magic_1024x2();
  const f16* frag = slot + min(r, 4 * XL - 1) * kMoeRowHalves + 32 * h;
  const int last = g0 + ng - 1;
  constexpr int P = D >= 4 ? 2 : 1;  // groups whose weights are asked for together
  uint4 wbuf[D][NW], xbuf[D][XL];
  uint4 s8[2], z8[2];
  const auto fetch_sz = [&](int g) {
    // eight from group g on and eight after them, those of the array's end instead where it has fewer left
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t at = min(tiles.s_off + 2 * g + 16 * i, tiles.s_end - 16);
      s8[i] = reinterpret_cast<const EightHalves*>(tiles.s + at)->v;
      z8[i] = reinterpret_cast<const EightHalves*>(tiles.z + at)->v;
    }
  };
  const auto put_sz = [&](bool second, int g) {
    const f16x8 s = as_f16x8(second ? s8[1] : s8[0]), z = as_f16x8(second ? z8[1] : z8[0]);
    const uint32_t want = tiles.s_off + 2 * g;
    const int off = (int)(want - min(want, tiles.s_end - 16)) >> 1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= off) table[(i - off) * 16 * NW + h % NW * 16 + r] = as_u32(f16x2{s[i], (f16)((f16)1024.0f + z[i])});
    __builtin_amdgcn_wave_barrier();
  };
  const auto fetch_w = [&](int i, int g) {
#pragma unroll
    for (int j = 0; j < NW; ++j) wbuf[i][j] = *reinterpret_cast<const uint4*>(tiles.w[j] + 64 * g + tiles.w_off);
  };
  const auto fetch_x = [&](int i, int g) {
#pragma unroll
    for (int j = 0; j < XL; ++j) xbuf[i][j] = *reinterpret_cast<const uint4*>(xs + 256 * g + xo[j]);
  };
  const auto group = [&](int u, int g) {  // the unit's u-th, group g
    const int i = u % D;
#pragma unroll
    for (int j = 0; j < XL; ++j)
      *reinterpret_cast<uint4*>(slot + (h + 4 * j) * kMoeRowHalves + 8 * r) = PERM ? perm_x8(xbuf[i][j]) : xbuf[i][j];
    if (MT == 1) fetch_x(i, min(g + D, last));  // (of two tiles all, they would spill)
    uint4 xa[MT][4];
    uint32_t sz[NW];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < 4; ++s) xa[m][s] = *reinterpret_cast<const uint4*>(frag + m * 16 * kMoeRowHalves + 8 * s);
#pragma unroll
    for (int j = 0; j < NW; ++j) sz[j] = table[(u * NW + j) * 16 + r];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      if (MT > 1) __builtin_amdgcn_sched_barrier(0);  // (else the tiles' unpacked codes are all held at once, and spill)
      const f16x2 v = as_f16x2(sz[j]);
      const f16 nb = (f16)960.0f - v[1];
      f32x4 part[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) part[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const f16x8 b =
            as_f16x8(step_operand<false>(wbuf[i][j], s, magic, f16x2{v[1], v[1]}, f16x2{nb, nb}, f16x2{}));
#pragma unroll
        for (int m = 0; m < MT; ++m) part[m] = mfma_16x16x32(as_f16x8(xa[m][s]), b, part[m]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][j] += (float)v[0] * part[m];
    }
  };
  fetch_sz(g0);
#pragma unroll
  for (int i = 0; i < D; ++i) {
    fetch_w(i, min(g0 + i, last));
    fetch_x(i, min(g0 + i, last));
  }
  int g = g0;
  bool second = false;
  for (; g + kMoeUnit <= last; g += kMoeUnit) {  // (a unit with another after it is whole)
    put_sz(second, g);
    if (second) fetch_sz(g + kMoeUnit);
    second = !second;
#pragma unroll
    for (int u = 0; u < kMoeUnit; u += P) {
#pragma unroll
      for (int v = 0; v < P; ++v) group(u + v, g + u + v);
#pragma unroll
      for (int v = 0; v < P; ++v) {
        fetch_w((u + v) % D, min(g + u + v + D, last));
        if (MT > 1) fetch_x((u + v) % D, min(g + u + v + D, last));
      }
      __builtin_amdgcn_sched_barrier(kSchedKeepGroups);  // the refill stays next to its consumption
    }
  }
  put_sz(second, g);
#pragma unroll
  for (int u = 0; u < kMoeUnit; ++u) {
    if (g + u <= last) {
      group(u, g + u);
      if constexpr (D < kMoeUnit)
        if (u + D < kMoeUnit) {
          fetch_w(u % D, min(g + u + D, last));
          if (MT > 1) fetch_x(u % D, min(g + u + D, last));
        }
    }
    __builtin_amdgcn_sched_barrier(kSchedKeepGroups);
  }
}

// An item of the first (UP) or second product: 16 NW rows of weights of one expert (UP: half of them the gate's, half
// the up projection's) and up to kMoePairs of its pairs.
struct MoeItem {
  int which, e;      // active expert
  int c0;            // first channel
  int first, count;  // pairs
};

// What a wave makes of an item's sums, acc[i][j]: rows 16 i + 4 (lane / 16) + 0..3, channel lane % 16 of tile j.
template <bool UP, int MT, int NW>
__device__ __forceinline__ void moe_store(const MoeArgs& a, const MoeLists& l, const f32x4 (&acc)[MT][NW],
                                          const MoeItem& t, int m0, int lane) {
  const int r = lane & 15, h = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * m + 4 * h + i;
      if (row < t.count) {
        const int64_t pair = (int64_t)m0 * a.k + l.pair[t.first + row];
        if constexpr (UP) {
#pragma unroll
          for (int j = 0; j < NW / 2; ++j) {
            const float gate = acc[m][j][i], v = gate / (1.0f + expf(-gate)) * acc[m][j + NW / 2][i];
            a.h[pair * a.I + t.c0 + 16 * j + (r & 8) + perm_slot(r & 7)] = (f16)v;
          }
        } else {
#pragma unroll
          for (int j = 0; j < NW; ++j) a.v[pair * a.H + t.c0 + 16 * j + r] = acc[m][j][i];
        }
      }
    }
}

template <int MT, int NW>
struct MoeRowsLds {
  MoeLists l;
  f32x4 part[kMoeWaves][MT * NW][64];  // a wave's sums of the item that it goes on with
  union {
    MoeScratch scratch;
    struct {
      f16 slot[kMoeWaves][16 * MT * kMoeRowHalves];
      uint32_t table[kMoeWaves][kMoeUnit * NW * 16];
    };
  };
};

// One of the layer's two products, for all pairs: items dealt in turn to one block a CU, a block's groups (G an item)
// in equal shares for its waves; what waves share of an item they join through LDS.
// FEW: batches of up to kMoeFew rows, none of whose items has more pairs: 32 rows of weights an item and eight groups in
// flight, since an item's rows of x are few.
template <bool UP, bool FEW>
__global__ void __launch_bounds__(64 * kMoeWaves)
moe_rows_kernel(MoeArgs a) {
  constexpr int MT = FEW ? 1 : 2, NW = FEW ? 2 : 4;
  extern __shared__ __align__(16) char smem[];
  MoeRowsLds<MT, NW>& lds = *reinterpret_cast<MoeRowsLds<MT, NW>*>(smem);
  MoeLists& l = lds.l;
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = (int)blockIdx.y * a.tokens, rows = min(a.tokens, a.M - m0);
  if constexpr (FEW) {
    moe_few_lists(l, a, rows);
  } else if constexpr (UP) {
    moe_lists(l, lds.scratch, a, m0, rows);
    if (blockIdx.x == 0) {  // for the second product
      uint4* out = reinterpret_cast<uint4*>(a.lists + blockIdx.y);
      for (int i = t; i < (int)(sizeof(MoeLists) / 16); i += 64 * kMoeWaves) out[i] = reinterpret_cast<uint4*>(&l)[i];
    }
  } else {
    const uint4* in = reinterpret_cast<const uint4*>(a.lists + blockIdx.y);
    for (int i = t; i < (int)(sizeof(MoeLists) / 16); i += 64 * kMoeWaves) reinterpret_cast<uint4*>(&l)[i] = in[i];
    __syncthreads();
  }
  const int active = __builtin_amdgcn_readfirstlane(l.active);
  const int K = UP ? a.H : a.I, N = UP ? a.I : a.H;
  constexpr int CH = UP ? 8 * NW : 16 * NW;  // channels of an item
  const int G = K >> 7, C = N / CH;
  // items: (expert, eight channel places, pairs, one of the eight places): those that read the same weights are eight
  // apart, blocks of one XCD, so that its L2 reads them once
  // (32 bits hold 1024 tiles of 2048 channels' items, and a block's groups: 64-bit divisions took 1 us here)
  const uint32_t items = (uint32_t)l.tile[active] * C, nb = gridDim.x;
  const uint32_t mine = items > blockIdx.x ? (items - blockIdx.x + nb - 1) / nb : 0;  // blockIdx.x, blockIdx.x + nb, ..
  const uint32_t groups = mine * G;
  const uint32_t u_lo = groups * wave / kMoeWaves, u_hi = groups * (wave + 1) / kMoeWaves;
  MoeItem it = {};
  bool open = false;  // the wave begins an item that others finish
  uint32_t open_end = 0;
  f32x4 acc[MT][NW];
  uint32_t item = blockIdx.x + u_lo / G * nb;
  int g0 = (int)(u_lo % G);
  if (u_lo < u_hi) it.which = moe_expert_of(l, active, (int)(item / C), lane);
  for (uint32_t u = u_lo; u < u_hi; item += nb, g0 = 0) {
    const int ng = min(G - g0, (int)(u_hi - u));
    while (item >= (uint32_t)l.tile[it.which + 1] * C) ++it.which;
    it.e = __builtin_amdgcn_readfirstlane(l.expert[it.which]);
    const int before = __builtin_amdgcn_readfirstlane(l.tile[it.which]);
    const int n_tiles = __builtin_amdgcn_readfirstlane(l.tile[it.which + 1]) - before;
    const int rem = (int)item - before * C;
    int c = rem, tile = 0;
    if (n_tiles > 1) {
      const int c8 = rem / (8 * n_tiles) * 8, n = min(8, C - c8), in = rem - c8 * n_tiles;
      tile = in / n;
      c = c8 + in - tile * n;
    }
    it.c0 = CH * c;
    it.first = __builtin_amdgcn_readfirstlane(l.start[it.which]) + kMoePairs * tile;
    it.count = min(kMoePairs, __builtin_amdgcn_readfirstlane(l.start[it.which + 1]) - it.first);
    MoeTiles<NW> tiles;
    int n[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j)
      n[j] = UP ? j / (NW / 2) * a.I + it.c0 + 16 * (j % (NW / 2)) : it.c0 + 16 * j;
    if constexpr (UP)
      tiles.set(a.up, a.up_s, a.up_z, it.e, a.E, 2 * a.I, n, G, lane);
    else
      tiles.set(a.down, a.down_s, a.down_z, it.e, a.E, a.H, n, G, lane);
    const uint8_t* xs = reinterpret_cast<const uint8_t*>(UP ? a.x + (int64_t)m0 * a.H : a.h + (int64_t)m0 * a.k * a.I);
    const auto row_of = [&](int row) {
      const uint32_t p = l.pair[it.first + min(row, it.count - 1)];
      return (UP ? p / (uint32_t)a.k : p) * (256u * G) + 16 * r;
    };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NW; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    f16* slot = lds.slot[wave];
    uint32_t* table = lds.table[wave];
    f32x4(&top)[1][NW] = reinterpret_cast<f32x4(&)[1][NW]>(acc[0]);
    if (it.count <= 4) {
      const uint32_t xo[1] = {row_of(h)};
      moe_stream<1, NW, 1, FEW ? 8 : 4, UP>(top, tiles, xs, xo, slot, table, g0, ng, lane);
    } else if constexpr (!FEW) {
      if (it.count <= 16) {
        uint32_t xo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) xo[j] = row_of(h + 4 * j);
        moe_stream<1, NW, 4, 4, UP>(top, tiles, xs, xo, slot, table, g0, ng, lane);
      } else {
        uint32_t xo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xo[j] = row_of(h + 4 * j);
        moe_stream<2, NW, 8, 2, UP>(acc, tiles, xs, xo, slot, table, g0, ng, lane);
      }
    }
    u += ng;
    if (ng == G) {
      moe_store<UP>(a, l, acc, it, m0, lane);
    } else if (g0 == 0) {
      open = true;
      open_end = u - ng + G;
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NW; ++j) lds.part[wave][m * NW + j][lane] = acc[m][j];
    }
  }
  __syncthreads();
  if (open) {
    for (int v = wave + 1; v < kMoeWaves && groups * v / kMoeWaves < open_end; ++v) {
      if (groups * v / kMoeWaves == groups * (v + 1) / kMoeWaves) continue;  // (a wave without any)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NW; ++j) acc[m][j] += lds.part[v][m * NW + j][lane];
    }
    moe_store<UP>(a, l, acc, it, m0, lane);
  }
}

// The second product of up to kMoeFew rows, and the sum over experts with it: a block for each 16 output channels, all
// active experts' groups in equal shares for its waves, each wave's sums in LDS.
__global__ void __launch_bounds__(64 * kMoeWaves)
moe_down_few_kernel(MoeArgs a) {
  __shared__ __align__(16) MoeLists l;
  __shared__ __align__(16) f16 slots[kMoeWaves][4 * kMoeRowHalves];
  __shared__ uint32_t tables[kMoeWaves][kMoeUnit * 16];
  __shared__ float sums[kMoeWaves][kMoeFew * 16];
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  float* mine = sums[wave];
  mine[lane] = 0.0f;
  moe_few_lists(l, a, a.M);
  const int active = __builtin_amdgcn_readfirstlane(l.active);
  const int n0 = blockIdx.x * 16, G = a.I >> 7;
  const int groups = active * G;  // (an expert has one tile; at most 64 experts)
  const int u_lo = groups * wave / kMoeWaves, u_hi = groups * (wave + 1) / kMoeWaves;
  int which = u_lo / G, g0 = u_lo % G;
  for (int u = u_lo; u < u_hi; ++which, g0 = 0) {
    const int ng = min(G - g0, u_hi - u);
    const int e = __builtin_amdgcn_readfirstlane(l.expert[which]);
    const int first = __builtin_amdgcn_readfirstlane(l.start[which]);
    const int count = __builtin_amdgcn_readfirstlane(l.start[which + 1]) - first;
    const int n[1] = {n0};
    MoeTiles<1> tiles;
    tiles.set(a.down, a.down_s, a.down_z, e, a.E, a.H, n, G, lane);
    const uint32_t xo[1] = {l.pair[first + min(h, count - 1)] * (256u * G) + 16 * r};
    f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
    moe_stream<1, 1, 1, 8, false>(acc, tiles, reinterpret_cast<const uint8_t*>(a.h), xo, slots[wave], tables[wave], g0, ng, lane);
    if (h == 0) {  // rows 0 .. 3
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count) {
          const int p = l.pair[first + i];
          mine[p / a.k * 16 + r] += moe_weight(a, 0, p, e) * acc[0][0][i];
        }
    }
    u += ng;
  }
  __syncthreads();
  if (t < a.M * 16) {
    float v = sums[0][t];
#pragma unroll
    for (int k = 1; k < kMoeWaves; ++k) v += sums[k][t];
    const int64_t o = (int64_t)(t >> 4) * a.H + n0 + (t & 15);
    if (a.y_f32)
      static_cast<float*>(a.y)[o] = v;
    else
      static_cast<f16*>(a.y)[o] = (f16)v;
  }
}

// y of a row from its pairs' sums, in the order of its slots, four channels a thread.
__global__ void __launch_bounds__(256)
moe_join_kernel(MoeArgs a) {
  __shared__ int slots[16], n_slots;
  __shared__ float weight[16];
  const int m = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (threadIdx.x < 64) {
    // slots that stand for an expert's pair, and their weights
    const int lane = threadIdx.x;
    const int id = lane < a.k ? a.experts[(int64_t)m * a.k + lane] : -1;
    const float w = lane < a.k ? a.weights[(int64_t)m * a.k + lane] : 0.0f;
    bool first = (uint32_t)id < (uint32_t)a.E;
    float sum = w;
    for (int j = 0; j < a.k; ++j) {
      const int other = __builtin_amdgcn_readlane(id, j);
      const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j));
      first = first && !(j < lane && other == id);
      sum += j > lane && other == id ? v : 0.0f;
    }
    const uint64_t mask = __ballot(first);
    if (first) {
      const int at = __popcll(mask & (((uint64_t)1 << lane) - 1));
      slots[at] = lane;
      weight[at] = sum;
    }
    if (lane == 0) n_slots = __popcll(mask);
  }
  __syncthreads();
  if (c >= a.H) return;
  const float* v = a.v + (int64_t)m * a.k * a.H + c;
  const int n = n_slots;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  constexpr int AHEAD = 4;  // slots whose loads are in flight together
  for (int j = 0; j < n; j += AHEAD) {
    f32x4 p[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) p[i] = *reinterpret_cast<const f32x4*>(v + (int64_t)slots[min(j + i, n - 1)] * a.H);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (j + i < n) y += weight[j + i] * p[i];
  }
  const int64_t o = (int64_t)m * a.H + c;
  if (a.y_f32)
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + o) = y;
  else
    *reinterpret_cast<f16x4*>(static_cast<f16*>(a.y) + o) = f16x4{(f16)y[0], (f16)y[1], (f16)y[2], (f16)y[3]};
}

static int64_t moe_tokens(int64_t M, int64_t k) {
  const int64_t most = kMoeMaxPairs / k < kMoeTokens ? kMoeMaxPairs / k : kMoeTokens;
  return M < most ? M : most;
}
static int64_t moe_chunks(int64_t M, int64_t k) { return (M + moe_tokens(M, k) - 1) / moe_tokens(M, k); }
static size_t moe_round(size_t n) { return (n + 255) / 256 * 256; }
static size_t moe_h_bytes(int64_t M, int64_t I, int64_t k) { return moe_round((size_t)(M * k) * I * 2); }
static size_t moe_v_bytes(int64_t M, int64_t H, int64_t k) { return M <= kMoeFew ? 0 : moe_round((size_t)(M * k) * H * 4); }

size_t moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t k) {
  return moe_h_bytes(M, I, k) + moe_v_bytes(M, H, k) + (size_t)moe_chunks(M, k) * sizeof(MoeLists);
}

template <bool UP, bool FEW>
static hipError_t launch_rows_product(const MoeArgs& a, int64_t items, unsigned chunks, hipStream_t stream) {
  constexpr size_t lds = sizeof(MoeRowsLds<FEW ? 1 : 2, FEW ? 2 : 4>);
  const hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(moe_rows_kernel<UP, FEW>), lds);
  if (e != hipSuccess) return e;
  // a block a CU, or fewer where there are fewer items
  hipLaunchKernelGGL((moe_rows_kernel<UP, FEW>), dim3((unsigned)(items < kNumCu ? items : kNumCu), chunks),
                     dim3(64 * kMoeWaves), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_moe_experts(const uint16_t* x, int64_t M, int64_t H, const int32_t* experts, const float* weights,
                              int64_t k, int64_t E, const uint32_t* up, const uint16_t* up_s, const uint16_t* up_z,
                              int64_t I, const uint32_t* down, const uint16_t* down_s, const uint16_t* down_z, void* y,
                              int y_f32, void* workspace, hipStream_t stream) {
  MoeArgs a;
  char* ws = static_cast<char*>(workspace);
  a.x = reinterpret_cast<const f16*>(x);
  a.experts = experts;
  a.weights = weights;
  a.up = up;
  a.up_s = reinterpret_cast<const f16*>(up_s);
  a.up_z = reinterpret_cast<const f16*>(up_z);
  a.down = down;
  a.down_s = reinterpret_cast<const f16*>(down_s);
  a.down_z = reinterpret_cast<const f16*>(down_z);
  a.h = reinterpret_cast<f16*>(ws);
  a.v = reinterpret_cast<float*>(ws + moe_h_bytes(M, I, k));
  a.lists = reinterpret_cast<MoeLists*>(ws + moe_h_bytes(M, I, k) + moe_v_bytes(M, H, k));
  a.y = y;
  a.M = (int)M;
  a.H = (int)H;
  a.I = (int)I;
  a.E = (int)E;
  a.k = (int)k;
  a.y_f32 = y_f32;
  a.tokens = (int)moe_tokens(M, k);
  const unsigned chunks = (unsigned)moe_chunks(M, k);
  // tiles of pairs, at most
  const int64_t pairs = a.tokens * k, tiles = pairs < E + pairs / kMoePairs ? pairs : E + pairs / kMoePairs;
  if (M <= kMoeFew) {
    const hipError_t e = launch_rows_product<true, true>(a, tiles * (I / 16), chunks, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_down_few_kernel, dim3((unsigned)(H / 16)), dim3(64 * kMoeWaves), 0, stream, a);
    return hipGetLastError();
  }
  hipError_t e = launch_rows_product<true, false>(a, tiles * (I / 32), chunks, stream);
  if (e == hipSuccess) e = launch_rows_product<false, false>(a, tiles * (H / 64), chunks, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)M, (unsigned)((H + 1023) / 1024)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Largest value over the wave's 64 lanes, as a scalar: inside rows of 16 lanes, then across them (lane exchanges that cost
// a vector instruction each; through LDS, with the exponentials in every round, a call of 8191 rows of 160 took 10.5 us, not 9.4).
__device__ __forceinline__ int wave_max(int v) {
  const auto step = [&](auto ctrl, auto rows) {
    v = max(v, __builtin_amdgcn_update_dpp(v, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr 1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast 15 into rows 1 and 3,
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // 31 into rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
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
  int mine = -1, value = kMasked, first = kMasked;  // of lane j: the j-th choice, its key; the first one's
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
    first = j == 0 ? most : first;
    if (lane == j) {
      mine = e;
      value = most;
    }
  }
  const float top = first == kMasked ? 0.0f : key_logit(first);
  const float p = mine < 0 ? 0.0f : expf(key_logit(value) - top);
  float total = p;
  if (!renormalize) {
    total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) total += x[v] == -INFINITY ? 0.0f : expf(x[v] - top);
  }
  total = wave_sum(total);
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
