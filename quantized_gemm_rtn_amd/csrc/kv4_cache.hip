// Writing and reading the 4-bit key/value cache, for gfx950.
//
// Each token's D key (value) channels of a head are one quantization group, in the
// asymmetric 4-bit form of the weights with the range widened to hold 0:
//   hi = max(x, 0), lo = min(x, 0),   s = fp16(max(fl32(fl32(hi - lo) / 15), 2^-14)),
//   z = clamp(rint(-lo / s), 0, 15),  q = clamp(rint(x / s) + z, 0, 15),  x ~ (q - z) s.
// (Weights' groups hold values of both signs; a token's channels need not, and without 0
// in the range every code of an all-positive group would be clamped.) All float32 steps
// are IEEE and correctly rounded, half to even; the file is built with
// -ffp-contract=off.
//
// kv4_append_kernel: one block per (sequence, tile of 32 tokens, head), so a word of
//   values, which holds eight tokens' codes of one channel, has one writer. D / 8
//   threads take a token: 8 channels each, range by lane exchanges, the key word is
//   whole and goes straight out; the value codes pass through LDS, where a thread
//   collects the eight tokens of its words. Words that also hold tokens that were in
//   the cache before are read first.
//   Bound by latency for single tokens (one each for 64 sequences, 8 heads of 128: 4.8 us)
//   and by memory for prompts (5755 tokens: 14.2 us, 30 MB, 2.1 TB/s: each block loads its
//   tokens, works and writes, with eight blocks a CU to overlap that). Both tensors' loads
//   first, quotients by a reciprocal (round_quotient), and ranges by exchanges inside a row
//   of lanes: 18.7 us without them.
// kv4_read_kernel: the way back, the same split: fp16 values of the new tokens (3.6 and
//   8.9 us for the same).
#include <type_traits>

#include "kv4.h"
#include "wq_launch.h"

namespace wq {

// a sequence's new tokens in the tile `tile`: positions [lo, hi)
__device__ __forceinline__ void tile_tokens(const KvSeq& s, int tile, int* lo, int* hi) {
  *lo = max(max(s.ctx - s.rows, 0), tile * kKvTile);
  *hi = min(s.ctx, (tile + 1) * kKvTile);
}

// largest value over the 8 or 16 lanes of a token, by exchanges inside rows of 16 lanes
template <int N>
__device__ __forceinline__ float token_max(float v) {
  const auto step = [&](auto ctrl) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false);
    v = fmaxf(v, __builtin_bit_cast(float, o));
  };
  step(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  step(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  step(std::integral_constant<int, 0x141>{});  // lane 7 - i of each eight
  if constexpr (N == 16) step(std::integral_constant<int, 0x140>{});  // lane 15 - i
  return v;
}

// rint(x / s), half to even, for fp16 x and s with |x| <= 15 s, from the reciprocal of s.
// x / s is a half-integer k + 1/2 exactly, or at least 2^-13 away from it: x and
// (k + 1/2) s are multiples of 2^-12 of the power of two below s. So x times the rounded
// reciprocal, rounded to a multiple of 2^-13 (1536 added and taken off again), is the
// half-integer itself in the first case and on the right side of it in the second.
__device__ __forceinline__ float round_quotient(float x, float reciprocal) {
  return rintf((x * reciprocal + 1536.0f) - 1536.0f);
}

template <int D>
__global__ void __launch_bounds__(256)
kv4_append_kernel(const f16* __restrict__ k, int64_t k_stride, const f16* __restrict__ v, int64_t v_stride, KvCache a,
                  int tiles, uint8_t* __restrict__ cache) {
  constexpr int TPT = D / 8;            // threads of a token
  constexpr int TOK = 256 / TPT;        // tokens of a pass
  constexpr int PASSES = kKvTile / TOK;
  __shared__ __align__(16) uint8_t codes[kKvTile][D + 4];
  const int h = blockIdx.x % a.hkv, first_tile = blockIdx.x / a.hkv % tiles;
  const int b = blockIdx.x / a.hkv / tiles, t = threadIdx.x;
  const KvSeq s = kv_sequence(a, b);
  const int begin = max(s.ctx - s.rows, 0);
  const int last = (s.ctx - 1) / kKvTile;  // rows > 0 and ctx > 0 where the loop runs
  if (s.rows == 0 || s.ctx == 0) return;
  // `tiles` comes from the caller's bound on the new tokens; a sequence with more is
  // still covered, in further rounds
  for (int tile = begin / kKvTile + first_tile; tile <= last; tile += tiles) {
    int lo, hi;
    tile_tokens(s, tile, &lo, &hi);
    const int page = tile / a.page_tiles;
    uint8_t* base = cache + kv_page_offset(a, b, h, page) +
                    (int64_t)(tile - page * a.page_tiles) * kv_tile_bytes<D>();
    const int part = t % TPT;
    // both tensors' loads first, so that their latencies pass together
    uint4 raw[2][PASSES];
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      const int pos = tile * kKvTile + pass * TOK + t / TPT;
      const int64_t row = s.first_row + min(max(pos - (s.ctx - s.rows), 0), s.rows - 1);
      raw[0][pass] = *reinterpret_cast<const uint4*>(k + row * k_stride + h * D + 8 * part);
      raw[1][pass] = *reinterpret_cast<const uint4*>(v + row * v_stride + h * D + 8 * part);
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass) {
        const int in = pass * TOK + t / TPT, pos = tile * kKvTile + in;
        if (pos >= lo && pos < hi) {  // the same for all threads of a token
          const f16x8 x = as_f16x8(raw[which][pass]);
          float f[8], top = 0.0f, bottom = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] = (float)x[e];
            top = fmaxf(top, f[e]);
            bottom = fminf(bottom, f[e]);
          }
          top = token_max<TPT>(top);
          bottom = -token_max<TPT>(-bottom);
          const f16 s16 = (f16)fmaxf(__fdiv_rn(top - bottom, 15.0f), 6.103515625e-05f);
          const float reciprocal = __fdiv_rn(1.0f, (float)s16);
          const float z = fminf(round_quotient(-bottom, reciprocal), 15.0f);
          uint32_t q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            q[e] = (uint32_t)(int)fminf(fmaxf(round_quotient(f[e], reciprocal) + z, 0.0f), 15.0f);
          if (which == 0) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= q[e] << (4 * e);
            *reinterpret_cast<uint32_t*>(base + kv_key_word<D>(in, part)) = w;
          } else {
            uint32_t* c = reinterpret_cast<uint32_t*>(&codes[in][8 * part]);
            c[0] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
            c[1] = q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24);
          }
          if (part == 0) {
            const int i = kv_meta_index(in);
            reinterpret_cast<f16*>(base + kv_meta_offset<D>(2 * which))[i] = s16;
            uint16_t* zeros = reinterpret_cast<uint16_t*>(base + kv_meta_offset<D>(2 * which + 1));
            const uint32_t iz = (uint32_t)(int)z;
            if (which == 0)
              zeros[kv_key_zero_index(in)] = kv_key_zero_bits(iz);
            else
              zeros[kv_value_zero_index(in)] = kv_value_zero_bits(in, iz);
          }
        }
      }
    }
    __syncthreads();
    uint8_t* vbase = base + kv_value_offset<D>();
    for (int i = t; i < 4 * D; i += 256) {
      const int c = i % D, g = i / D;
      uint32_t w = 0, fresh = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int in = 4 * g + (n & 3) + 16 * (n >> 2), pos = tile * kKvTile + in;
        if (pos >= lo && pos < hi) {
          w |= (uint32_t)codes[in][c] << (4 * n);
          fresh |= 0xFu << (4 * n);
        }
      }
      if (fresh == 0) continue;
      uint32_t* at = reinterpret_cast<uint32_t*>(vbase + kv_value_word(c, g));
      if (fresh != 0xFFFFFFFFu) w |= *at & ~fresh;
      *at = w;
    }
    __syncthreads();  // codes is refilled by the next round
  }
}

template <int D>
__global__ void __launch_bounds__(256)
kv4_read_kernel(const uint8_t* __restrict__ cache, KvCache a, int tiles, f16* __restrict__ k, f16* __restrict__ v) {
  constexpr int TPT = D / 8, TOK = 256 / TPT;
  __shared__ __align__(16) uint8_t codes[kKvTile][D + 4];
  const int h = blockIdx.x % a.hkv, first_tile = blockIdx.x / a.hkv % tiles;
  const int b = blockIdx.x / a.hkv / tiles, t = threadIdx.x;
  const KvSeq s = kv_sequence(a, b);
  const int part = t % TPT;
  // a sequence with more new tokens than its cache holds: the first of them are in no
  // page, and read as 0
  const int absent = max(s.rows - s.ctx, 0);
  for (int i = first_tile * TOK + t / TPT; i < absent; i += tiles * TOK) {
    const int64_t at = ((int64_t)(s.first_row + i) * a.hkv + h) * D + 8 * part;
    *reinterpret_cast<uint4*>(k + at) = uint4{0, 0, 0, 0};
    *reinterpret_cast<uint4*>(v + at) = uint4{0, 0, 0, 0};
  }
  if (s.rows == 0 || s.ctx == 0) return;
  const int begin = max(s.ctx - s.rows, 0), last = (s.ctx - 1) / kKvTile;
  for (int tile = begin / kKvTile + first_tile; tile <= last; tile += tiles) {
    int lo, hi;
    tile_tokens(s, tile, &lo, &hi);
    const int page = tile / a.page_tiles;
    const uint8_t* base = cache + kv_page_offset(a, b, h, page) +
                          (int64_t)(tile - page * a.page_tiles) * kv_tile_bytes<D>();
    const uint8_t* vbase = base + kv_value_offset<D>();
    for (int i = t; i < 4 * D; i += 256) {
      const int c = i % D, g = i / D;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(vbase + kv_value_word(c, g));
#pragma unroll
      for (int n = 0; n < 8; ++n) codes[4 * g + (n & 3) + 16 * (n >> 2)][c] = (uint8_t)((w >> (4 * n)) & 0xFu);
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < kKvTile / TOK; ++pass) {
      const int in = pass * TOK + t / TPT, pos = tile * kKvTile + in;
      if (pos < lo || pos >= hi) continue;
      const int64_t row = s.first_row + (pos - (s.ctx - s.rows));
      const int64_t at = (row * a.hkv + h) * D + 8 * part;
      const auto scale = [&](int which) {
        return (float)reinterpret_cast<const f16*>(base + kv_meta_offset<D>(which))[kv_meta_index(in)];
      };
      const auto zero = [&](int which) { return reinterpret_cast<const uint16_t*>(base + kv_meta_offset<D>(which)); };
      const float ks = scale(0), vs = scale(2);
      const float kz = (float)kv_key_zero(zero(1)[kv_key_zero_index(in)]);
      const float vz = (float)kv_value_zero(in, zero(3)[kv_value_zero_index(in)]);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(base + kv_key_word<D>(in, part));
      const uint32_t* c = reinterpret_cast<const uint32_t*>(&codes[in][8 * part]);
      f16x8 ko, vo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ko[e] = (f16)(((float)((w >> (4 * e)) & 0xFu) - kz) * ks);
        vo[e] = (f16)(((float)((c[e >> 2] >> (8 * (e & 3))) & 0xFFu) - vz) * vs);
      }
      *reinterpret_cast<uint4*>(k + at) = __builtin_bit_cast(uint4, ko);
      *reinterpret_cast<uint4*>(v + at) = __builtin_bit_cast(uint4, vo);
    }
    __syncthreads();
  }
}

KvCache kv4_cache_args(const Kv4View& c, int64_t T, int64_t head_dim) {
  KvCache a;
  a.page_table = c.page_table;
  a.seq_start = c.seq_start;
  a.ctx_len = c.ctx_len;
  a.num_pages = (int)c.num_pages;
  a.page_bytes = c.page_tokens * (head_dim + 8);
  a.B = (int)c.B;
  a.hkv = (int)c.kv_heads;
  a.max_pages = (int)c.max_pages;
  a.page_tiles = (int)(c.page_tokens / kKvTile);
  a.T = (int)T;
  return a;
}

// tiles a sequence with up to max_new new tokens may touch, at most what the grid takes
static int append_tiles(const Kv4View& c, int64_t max_new) {
  const int64_t most = (((int64_t)1 << 24) - 1) / (c.B * c.kv_heads);  // B kv_heads < 2^24, blocks too
  const int64_t want = (max_new + kKvTile - 2) / kKvTile + 1;
  return (int)(want < most ? want : most);
}

hipError_t launch_kv4_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, int64_t T,
                             int64_t head_dim, int64_t max_new, const Kv4View& c, void* cache, hipStream_t stream) {
  const KvCache a = kv4_cache_args(c, T, head_dim);
  const int tiles = append_tiles(c, max_new);
  const dim3 grid((unsigned)(c.B * tiles * c.kv_heads));
  const f16* kp = reinterpret_cast<const f16*>(k);
  const f16* vp = reinterpret_cast<const f16*>(v);
  if (head_dim == 128)
    hipLaunchKernelGGL((kv4_append_kernel<128>), grid, dim3(256), 0, stream, kp, k_stride, vp, v_stride, a, tiles,
                       static_cast<uint8_t*>(cache));
  else
    hipLaunchKernelGGL((kv4_append_kernel<64>), grid, dim3(256), 0, stream, kp, k_stride, vp, v_stride, a, tiles,
                       static_cast<uint8_t*>(cache));
  return hipGetLastError();
}

hipError_t launch_kv4_read(const void* cache, int64_t T, int64_t head_dim, int64_t max_new, const Kv4View& c,
                           uint16_t* k, uint16_t* v, hipStream_t stream) {
  const KvCache a = kv4_cache_args(c, T, head_dim);
  const int tiles = append_tiles(c, max_new);
  const dim3 grid((unsigned)(c.B * tiles * c.kv_heads));
  if (head_dim == 128)
    hipLaunchKernelGGL((kv4_read_kernel<128>), grid, dim3(256), 0, stream, static_cast<const uint8_t*>(cache), a,
                       tiles, reinterpret_cast<f16*>(k), reinterpret_cast<f16*>(v));
  else
    hipLaunchKernelGGL((kv4_read_kernel<64>), grid, dim3(256), 0, stream, static_cast<const uint8_t*>(cache), a,
                       tiles, reinterpret_cast<f16*>(k), reinterpret_cast<f16*>(v));
  return hipGetLastError();
}

}  // namespace wq
