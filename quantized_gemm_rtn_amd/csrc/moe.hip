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

constexpr int kMoeTokens = 64;      // rows of x that a block's lists hold; more come as further blocks
constexpr int kMoeMaxPairs = 1024;  // of them, (row, expert) pairs: top_k <= 16
constexpr int kMoeMaxExperts = 1024;
constexpr int kUpWaves = 4, kUpDepth = 4;
constexpr int kDownWaves = 16, kDownDepth = 4;

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
  f16* h;                  // [M * k][I], each 128 channels in the order of moe_h_index
  int32_t* lists;          // of each 64 rows: see MoeLists
  void* y;
  int M, H, I, E, k, y_f32;
};

// What 64 rows of x have to do, from their experts: the active experts in ascending order, each
// with its (row, expert) pairs, and those pairs, row * k + slot. A row that names an expert
// twice has it once, with the weights' sum.
struct MoeLists {
  int32_t active;                      // experts
  int32_t pad[15];
  int32_t expert[kMoeMaxPairs];        // of the i-th active one,
  int32_t start[kMoeMaxPairs + 16];    // its first pair (start[active]: their number)
  int32_t pair[kMoeMaxPairs];
};

// Position of inner channel c among the 128 of its group: chunks of eight in the order that the
// four lane groups of a product's step read them, each in the order of perm_x8.
__device__ __forceinline__ int moe_h_index(int c) {
  return (c & ~127) | ((c >> 3) & 3) << 5 | ((c >> 5) & 3) << 3 | perm_slot(c & 7);
}

__device__ __forceinline__ int sum_upto_64(int v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(v, off);
    v += lane >= off ? u : 0;
  }
  return v;
}

// The lists of rows m0 .. m0 + rows - 1, by a block of 256 threads, in its LDS.
__device__ __forceinline__ void moe_lists(MoeLists& l, int (&ids)[kMoeMaxPairs], int (&count)[kMoeMaxExperts],
                                          int (&sums)[4], const MoeArgs& a, int m0, int rows) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, pairs = rows * a.k;
  constexpr int PER = kMoeMaxPairs / 256, EPER = kMoeMaxExperts / 256;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + 256 * i;
    int e = p < pairs ? a.experts[(int64_t)m0 * a.k + p] : -1;
    ids[p] = e = (uint32_t)e < (uint32_t)a.E ? e : -1;
  }
#pragma unroll
  for (int i = 0; i < EPER; ++i) count[EPER * t + i] = 0;
  __syncthreads();
  int place[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + 256 * i, e = ids[p];
    bool first = e >= 0;
    if (first)
      for (int q = p / a.k * a.k; q < p; ++q) first = first && ids[q] != e;
    place[i] = first ? atomicAdd(&count[e], 1) : -1;
  }
  __syncthreads();
  int made[PER];  // pairs of the pair's expert
#pragma unroll
  for (int i = 0; i < PER; ++i) made[i] = place[i] >= 0 ? count[ids[t + 256 * i]] : 0;
  // experts EPER t .. + EPER - 1: pairs and active ones before them, in one sum
  int own[EPER], both = 0;
#pragma unroll
  for (int i = 0; i < EPER; ++i) {
    own[i] = count[EPER * t + i];
    both += own[i] + (own[i] > 0 ? 1 << 16 : 0);
  }
  const int upto = sum_upto_64(both, lane);
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int before = upto - both, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? sums[w] : 0;
    total += sums[w];
  }
#pragma unroll
  for (int i = 0; i < EPER; ++i)
    if (own[i] > 0) {
      l.expert[before >> 16] = EPER * t + i;
      l.start[before >> 16] = before & 0xFFFF;
      count[EPER * t + i] = before & 0xFFFF;  // where its pairs begin
      before += own[i] + (1 << 16);
    }
  if (t == 0) {
    l.active = total >> 16;
    l.start[total >> 16] = total & 0xFFFF;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (place[i] >= 0) l.pair[count[ids[t + 256 * i]] + place[i]] = t + 256 * i;
  __syncthreads();
  // in order (the atomics' is any): a pair's tile decides where its sums are split
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = t + 256 * i;
    if (place[i] >= 0) {
      const int e = ids[p], from = count[e];
      int rank = 0;
      for (int q = from; q < from + made[i]; ++q) rank += l.pair[q] < p ? 1 : 0;
      place[i] = from + rank;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (place[i] >= 0) l.pair[place[i]] = t + 256 * i;
  __syncthreads();
}

// The weight of a pair: of its slot and of later ones with the same expert.
__device__ __forceinline__ float moe_weight(const MoeArgs& a, int m0, int pair, int e) {
  const int row = pair / a.k;
  const int64_t at = (int64_t)m0 * a.k;
  float w = 0.0f;
  for (int q = pair; q < (row + 1) * a.k; ++q) w += a.experts[at + q] == e ? a.weights[at + q] : 0.0f;
  return w;
}

__global__ void __launch_bounds__(64 * kUpWaves)
moe_up_kernel(MoeArgs a) {
  constexpr int KW = kUpWaves, D = kUpDepth;
  __shared__ MoeLists l;
  __shared__ int ids[kMoeMaxPairs], count[kMoeMaxExperts], sums[4];
  __shared__ f32x4 red[KW - 1][2][64];
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = blockIdx.z * kMoeTokens, rows = min(kMoeTokens, a.M - m0);
  moe_lists(l, ids, count, sums, a, m0, rows);
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // for the second product
    int32_t* out = a.lists + (int64_t)blockIdx.z * (sizeof(MoeLists) / 4);
    const int32_t* in = reinterpret_cast<const int32_t*>(&l);
    for (int i = t; i < (int)(sizeof(MoeLists) / 4); i += 64 * KW) out[i] = in[i];
  }
  if ((int)blockIdx.y >= l.active) return;
  const int e = __builtin_amdgcn_readfirstlane(l.expert[blockIdx.y]);
  const int start = __builtin_amdgcn_readfirstlane(l.start[blockIdx.y]);
  const int n_pairs = __builtin_amdgcn_readfirstlane(l.start[blockIdx.y + 1]) - start;
  const int n0 = blockIdx.x * 16, G = a.H >> 7;
  const int g_lo = (G * wave) / KW, ng = (G * (wave + 1)) / KW - g_lo;
  const uint32_t magic = magic_1024x2();

  // rows n0 + r of the gate (j = 0) and of the up projection (j = 1)
  const uint32_t* wrow[2];
  const f16 *srow[2], *zrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = ((int64_t)e * 2 + j) * a.I + n0 + r;
    wrow[j] = a.up + n * (16 * G) + 4 * h;
    srow[j] = a.up_s + n * G;
    zrow[j] = a.up_z + n * G;
  }
  for (int r0 = 0; r0 < n_pairs; r0 += 16) {
    const int pair = l.pair[start + min(r0 + r, n_pairs - 1)];
    const f16* xrow = a.x + (int64_t)(m0 + pair / a.k) * a.H + 32 * h;
    uint4 wbuf[D][2], xbuf[D][4];
    f16 sbuf[D][2], zbuf[D][2];
    const auto fetch = [&](int i, int g) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        wbuf[i][j] = *reinterpret_cast<const uint4*>(wrow[j] + (int64_t)g * 16);
        sbuf[i][j] = srow[j][g];
        zbuf[i][j] = zrow[j][g];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) xbuf[i][s] = *reinterpret_cast<const uint4*>(xrow + (int64_t)g * 128 + 8 * s);
    };
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    const auto group = [&](int i) {
      uint4 xa[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) xa[s] = perm_x8(xbuf[i][s]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f16 b = (f16)1024.0f + zbuf[i][j], nb = (f16)960.0f - b;
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
          part = mfma_16x16x32(as_f16x8(xa[s]),
                               as_f16x8(step_operand<false>(wbuf[i][j], s, magic, f16x2{b, b}, f16x2{nb, nb}, f16x2{})),
                               part);
        acc[j] += (float)sbuf[i][j] * part;
      }
    };
    const int last = max(ng - 1, 0);
    const int gl = min(g_lo, G - 1);
#pragma unroll
    for (int i = 0; i < D; ++i) fetch(i, gl + min(i, last));
    for (int b = 0; b < ng; b += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (b + i < ng) group(i);
        fetch(i, gl + min(b + D + i, last));
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) red[wave - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < KW - 1; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] += red[w][j][lane];
      const int at = moe_h_index(n0 + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + 4 * h + i;
        if (row < n_pairs) {
          const float gate = acc[0][i], v = gate / (1.0f + expf(-gate)) * acc[1][i];
          a.h[((int64_t)m0 * a.k + l.pair[start + row]) * a.I + at] = (f16)v;
        }
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(64 * kDownWaves)
moe_down_kernel(MoeArgs a) {
  constexpr int KW = kDownWaves, D = kDownDepth;
  extern __shared__ __align__(16) float sums[];  // [KW][rows][16]
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int m0 = blockIdx.z * kMoeTokens, rows = min(kMoeTokens, a.M - m0);
  const MoeLists* l = reinterpret_cast<const MoeLists*>(a.lists + (int64_t)blockIdx.z * (sizeof(MoeLists) / 4));
  float* mine = sums + wave * rows * 16;
  for (int i = lane; i < rows * 16; i += 64) mine[i] = 0.0f;
  const int n0 = blockIdx.x * 16, G = a.I >> 7;
  const uint32_t magic = magic_1024x2();
  const int active = l->active;
  // steps: an expert's groups for each 16 of its pairs
  int items = 0;
  for (int i = 0; i < active; ++i) items += (l->start[i + 1] - l->start[i] + 15) >> 4;
  const int total = items * G;
  const int s_lo = (int)((int64_t)total * wave / KW), s_hi = (int)((int64_t)total * (wave + 1) / KW);
  // the item that step s_lo is of
  int i0 = 0, r0 = 0;
  for (int left = s_lo / G; i0 < active; ++i0) {
    const int tiles = (l->start[i0 + 1] - l->start[i0] + 15) >> 4;
    if (left < tiles) {
      r0 = 16 * left;
      break;
    }
    left -= tiles;
  }
  for (int s = s_lo; s < s_hi;) {
    const int e = l->expert[i0], start = l->start[i0], n_pairs = l->start[i0 + 1] - start;
    const int g_lo = s % G, ng = min(G - g_lo, s_hi - s);
    const int pair = l->pair[start + min(r0 + r, n_pairs - 1)];
    const f16* hrow = a.h + ((int64_t)m0 * a.k + pair) * a.I + 8 * h;
    const int64_t n = (int64_t)e * a.H + n0 + r;
    const uint32_t* wrow = a.down + n * (16 * G) + 4 * h;
    const f16 *srow = a.down_s + n * G, *zrow = a.down_z + n * G;
    uint4 wbuf[D], xbuf[D][4];
    f16 sbuf[D], zbuf[D];
    const auto fetch = [&](int i, int g) {
      wbuf[i] = *reinterpret_cast<const uint4*>(wrow + (int64_t)g * 16);
      sbuf[i] = srow[g];
      zbuf[i] = zrow[g];
#pragma unroll
      for (int q = 0; q < 4; ++q) xbuf[i][q] = *reinterpret_cast<const uint4*>(hrow + (int64_t)g * 128 + 32 * q);
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D; ++i) fetch(i, g_lo + min(i, ng - 1));
    for (int b = 0; b < ng; b += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (b + i < ng) {
          const f16 bi = (f16)1024.0f + zbuf[i], nb = (f16)960.0f - bi;
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            part = mfma_16x16x32(as_f16x8(xbuf[i][q]),
                                 as_f16x8(step_operand<false>(wbuf[i], q, magic, f16x2{bi, bi}, f16x2{nb, nb}, f16x2{})),
                                 part);
          acc += (float)sbuf[i] * part;
        }
        fetch(i, g_lo + min(b + D + i, ng - 1));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 4 * h + i;
      if (row < n_pairs) {
        const int p = l->pair[start + row];
        mine[p / a.k * 16 + r] += moe_weight(a, m0, p, e) * acc[i];
      }
    }
    s += ng;
    r0 += 16;
    if (r0 >= n_pairs) {
      r0 = 0;
      ++i0;
    }
  }
  __syncthreads();
  for (int i = t; i < rows * 16; i += 64 * KW) {
    float v = sums[i];
    for (int w = 1; w < KW; ++w) v += sums[w * rows * 16 + i];
    const int64_t o = (int64_t)(m0 + (i >> 4)) * a.H + n0 + (i & 15);
    if (a.y_f32)
      static_cast<float*>(a.y)[o] = v;
    else
      static_cast<f16*>(a.y)[o] = (f16)v;
  }
}

static int64_t moe_chunks(int64_t M) { return (M + kMoeTokens - 1) / kMoeTokens; }
static size_t moe_h_bytes(int64_t M, int64_t I, int64_t k) { return ((size_t)(M * k) * I * 2 + 255) / 256 * 256; }

size_t moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t k) {
  return moe_h_bytes(M, I, k) + (size_t)moe_chunks(M) * sizeof(MoeLists);
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
  a.lists = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + moe_h_bytes(M, I, k));
  a.y = y;
  a.M = (int)M;
  a.H = (int)H;
  a.I = (int)I;
  a.E = (int)E;
  a.k = (int)k;
  a.y_f32 = y_f32;
  const int64_t tokens = M < kMoeTokens ? M : kMoeTokens, most = tokens * k < E ? tokens * k : E;
  const unsigned chunks = (unsigned)moe_chunks(M);
  hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(I / 16), (unsigned)most, chunks), dim3(64 * kUpWaves), 0, stream,
                     a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)kDownWaves * tokens * 64;
  if (lds > 65536) {
    e = set_dynamic_lds(reinterpret_cast<const void*>(moe_down_kernel), lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(H / 16), 1, chunks), dim3(64 * kDownWaves), lds, stream, a);
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
