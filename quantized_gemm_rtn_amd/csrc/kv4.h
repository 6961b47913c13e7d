// Layout of the 4-bit key/value cache, shared by the kernels that write and read it.
//
// A page of one key/value head is a run of tiles of 32 tokens; a tile of head dimension
// D is 32 (D + 8) contiguous bytes:
//   key codes    16 D bytes   |   value codes  16 D bytes
//   key scales, key zero-points, value scales, value zero-points: 32 fp16 each
// and the codes are laid out as the operands of the attention's matrix products, so that
// a wave's 64 lanes load them as whole runs of 16 bytes a lane and use them with no
// exchange between lanes. With lane = 16 g + c (g = 0..3, c = 0..15):
//  - keys: the word of token 16 b + c (b = 0, 1) and channels (D/4) g + 8 w .. + 7
//    (w < D/32; channel + j in nibble j) is word w of lane 16 g + c of half b: A operand
//    of step w of the 16x16x32 product keys . queries^T. D = 128: a half is 64 lanes x 4
//    words; D = 64: both halves share one run, words 2 b + w of a lane.
//  - values: the word of channel 16 k + c holds tokens 4 g + r + 16 b in nibble r + 4 b
//    (r = 0..3), the tokens whose scores lane 16 g + c holds after the first product, and
//    is word k % 4 of lane 16 g + c of run k / 4: A operand of the product
//    values^T . weights^T.
//  - scales: token 4 g + r + 16 b at index 8 g + 4 b + r, so that a lane's eight tokens
//    are one run of 16 bytes, in the order of the values' nibbles.
//  - zero-points: as what unpacking adds (see codes_minus_zero_x16). Keys: 1024 + z at
//    index 2 c + b, one word a lane. Values: at index 8 g + 2 r + b, 1024 + z for even r
//    and -(64 + z) for odd r, the pairs the unpacked codes of a lane's tokens come in.
#pragma once

#include "wq_device.h"

namespace wq {

constexpr int kKvTile = 32;      // tokens of a tile
constexpr int kKvQmax = 15;

struct KvCache {
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* seq_start;   // [B + 1]
  const int32_t* ctx_len;     // [B]
  int64_t page_bytes;         // of one head
  int B, hkv, max_pages, num_pages;
  int page_tiles;             // tiles of a page
  int T;                      // rows of the token-wise arrays
};

template <int D>
constexpr int kv_tile_bytes() { return kKvTile * (D + 8); }
template <int D>
constexpr int kv_key_offset() { return 0; }
template <int D>
constexpr int kv_value_offset() { return 16 * D; }
// which: 0 key scales, 1 key zero-points, 2 value scales, 3 value zero-points
template <int D>
constexpr int kv_meta_offset(int which) { return 32 * D + 64 * which; }

// byte offset of a key word in a tile: token 0..31, channels 8 block .. + 7
template <int D>
__device__ __forceinline__ int kv_key_word(int token, int block) {
  constexpr int W = D / 32;  // words of a lane and half
  const int lane = 16 * (block / W) + (token & 15), w = block % W, b = token >> 4;
  return D == 128 ? 1024 * b + 16 * lane + 4 * w : 16 * lane + 8 * b + 4 * w;
}
// byte offset, from the values' start, of the word of channel c and token group g
__device__ __forceinline__ int kv_value_word(int c, int g) {
  const int k = c >> 4;
  return 1024 * (k >> 2) + 16 * (16 * g + (c & 15)) + 4 * (k & 3);
}
// position of a token 0..31 among a tile's scales or zero-points
__device__ __forceinline__ int kv_meta_index(int token) {
  return 8 * ((token & 15) >> 2) + 4 * (token >> 4) + (token & 3);
}

// where and as which fp16 bits a token's zero-points are kept
__device__ __forceinline__ int kv_key_zero_index(int token) { return 2 * (token & 15) + (token >> 4); }
__device__ __forceinline__ uint16_t kv_key_zero_bits(uint32_t z) { return (uint16_t)(0x6400u | z); }
__device__ __forceinline__ uint32_t kv_key_zero(uint16_t bits) { return bits & 0xFu; }
__device__ __forceinline__ int kv_value_zero_index(int token) {
  return 8 * ((token & 15) >> 2) + 2 * (token & 3) + (token >> 4);
}
__device__ __forceinline__ uint16_t kv_value_zero_bits(int token, uint32_t z) {
  return (uint16_t)(token & 1 ? 0xD400u | (z << 4) : 0x6400u | z);
}
__device__ __forceinline__ uint32_t kv_value_zero(int token, uint16_t bits) {
  return (token & 1 ? bits >> 4 : bits) & 0xFu;
}
// the same eight bits under a fresh exponent: finite whatever was there
__device__ __forceinline__ uint4 kv_value_zeros_finite(uint4 v) {
  return uint4{(v.x & 0x000F000Fu) | 0x64006400u, (v.y & 0x00F000F0u) | 0xD400D400u,
               (v.z & 0x000F000Fu) | 0x64006400u, (v.w & 0x00F000F0u) | 0xD400D400u};
}
// exact fp16 q - z of the eight codes of a word of values, zeros as they are kept
__device__ __forceinline__ f16x8 kv_value_operand(uint32_t w, uint32_t magic, const uint4& zeros) {
  const uint4 q = codes_biased_x16(w, magic);
  const f16x2 sixteenth = {(f16)0.0625f, (f16)0.0625f};
  return as_f16x8(uint4{as_u32(as_f16x2(q.x) - as_f16x2(zeros.x)),
                        as_u32(__builtin_elementwise_fma(as_f16x2(q.y), sixteenth, as_f16x2(zeros.y))),
                        as_u32(as_f16x2(q.z) - as_f16x2(zeros.z)),
                        as_u32(__builtin_elementwise_fma(as_f16x2(q.w), sixteenth, as_f16x2(zeros.w)))});
}
// both halves of a lane's word of key zero-points as the pairs that unpacking takes
struct KeyZeros {
  f16x2 bias[2], nbias16[2];
};
__device__ __forceinline__ KeyZeros kv_key_zeros(uint32_t word) {
  KeyZeros k;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint32_t v = __builtin_amdgcn_perm(word, word, b ? 0x03020302u : 0x01000100u);
    k.bias[b] = as_f16x2(v);
    k.nbias16[b] = as_f16x2(((v & 0x000F000Fu) << 4) | 0xD400D400u);
  }
  return k;
}

// A sequence as a kernel sees it: every value is clamped to what the arrays hold, so
// lengths or page numbers outside them give wrong values but no access outside.
struct KvSeq {
  int first_row;  // of its new tokens in the token-wise arrays
  int rows;       // new tokens
  int ctx;        // tokens in the cache, the new ones last
};
__device__ __forceinline__ KvSeq kv_sequence(const KvCache& a, int b) {
  KvSeq s;
  const int s0 = min(max(a.seq_start[b], 0), a.T), s1 = min(max(a.seq_start[b + 1], s0), a.T);
  s.first_row = s0;
  s.rows = s1 - s0;
  const int64_t most = (int64_t)a.max_pages * a.page_tiles * kKvTile;
  s.ctx = (int)min((int64_t)max(a.ctx_len[b], 0), most);
  return s;
}
// offset in the cache of head h of the page numbered id (64 bits: a cache may be larger
// than 4 GiB), and of page `page` of sequence b
__device__ __forceinline__ int64_t kv_page_offset(const KvCache& a, int h, int id) {
  const int in = min(max(id, 0), a.num_pages - 1);
  return ((int64_t)in * a.hkv + h) * a.page_bytes;
}
__device__ __forceinline__ int64_t kv_page_offset(const KvCache& a, int b, int h, int page) {
  return kv_page_offset(a, h, a.page_table[(int64_t)b * a.max_pages + page]);
}

}  // namespace wq
