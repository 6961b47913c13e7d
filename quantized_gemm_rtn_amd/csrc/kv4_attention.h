// What the attention kernels over the 4-bit cache share.
#pragma once

#include "kv4.h"

namespace wq {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr float kNoRef = -1e30f;      // reference of a row that has seen nothing
constexpr float kTop = 12.8f;         // log2 of the largest weight times value scale after a move of r,
constexpr float kSlack = 3.1f;        // how far it may grow before the next (fp16 ends at 2^16),
constexpr float kMixed = 3.0f;        // and how far below that top it may stay
constexpr float kFar = 262144.0f;     // references from which float32 no longer holds these fractions,
constexpr float kNone = 1e29f;        // up to those that no score reaches
constexpr uint32_t kAlike = 2 << 10;  // value scales whose bits differ by less are within 2^kMixed
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kTileRows = 128;        // query rows of a block of kv4_tile_kernel
constexpr int kDecodeRows = 16;       // query rows of one column tile

struct AttnArgs {
  const f16* q;
  int64_t q_stride;
  const uint8_t* cache;
  f16* out;
  float* lse;         // may be null
  float* part_o;      // partials of the decode kernel, two a block: [block][2][rows][D]
  float2* part_s;     // [block][2][rows]: r, sum
  float* tpart_o;     // the same of the tile kernel: [block][2][kTileRows][D]
  float2* tpart_s;    // [block][2][kTileRows]
  int hq, group;      // query heads, and those of one key/value head
  int window;         // 0: none, also where the pages hold no more tokens than it
  float c;            // scale * log2(e)
  int shares, least;  // decode kernel: blocks a head, and the fewest tiles of one
  int pad;            // items count as multiples of `least` steps: one item a block
  int decode_rows;    // rows of an item of the decode kernel (16 or 32)
  int tshares;        // tile kernel: blocks a head, each an equal share of the work; or 0,
  int row_tiles;      // and a block takes every row_tiles-th row tile of a sequence,
  int snake;          // long and short ones in turn (see kv4_tile_kernel)
  int row_limit;      // sequences with more rows of a head belong to the tile kernel
};

// The last token that the window of a row at this position has passed, -1 for none (compared
// before it is subtracted: rows before the first token have negative positions).
__device__ __forceinline__ int last_passed(const AttnArgs& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window : -1;
}

// Tiles [t0, t1) of a sequence that rows row0 .. row1 (of one head group) can see.
struct TileRange {
  int t0, t1;
};
__device__ __forceinline__ TileRange tile_range(const KvSeq& s, const AttnArgs& p, int row0, int row1) {
  const int p0 = s.ctx - s.rows + row0 / p.group, p1 = s.ctx - s.rows + row1 / p.group;
  const int lo = last_passed(p, p0) + 1;
  TileRange r;
  r.t0 = lo / kKvTile;
  r.t1 = p1 < lo ? r.t0 : p1 / kKvTile + 1;
  return r;
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// What a row's sum of weights makes of its outputs, and the row's log of the sum of
// exponentials: 0 and -infinity where no token is seen (the sum is 0), NaN where a score was.
__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
__device__ __forceinline__ float log_sum(float ref, float sum) {
  return sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

// a * b with the fp16 factor read as it is (one mixed-precision instruction; the sum with
// 0 keeps the compiler from splitting it into a conversion and a product)
__device__ __forceinline__ float mul_mix(float a, f16 b) { return __builtin_fmaf(a, (float)b, 0.0f); }

// largest and smallest of eight fp16 values of at least 0, as bits (these order like integers)
template <class F>
__device__ __forceinline__ uint32_t of_eight(const f16x8& v, F pick) {
  const uint4 d = __builtin_bit_cast(uint4, v);
  const u16x2 a = pick(__builtin_bit_cast(u16x2, d.x), __builtin_bit_cast(u16x2, d.y));
  const u16x2 b = pick(__builtin_bit_cast(u16x2, d.z), __builtin_bit_cast(u16x2, d.w));
  const u16x2 m = pick(a, b);
  return pick(u16x2{m.x, 0}, u16x2{m.y, 0}).x;
}
__device__ __forceinline__ uint32_t max_bits8(const f16x8& v) {
  return of_eight(v, [](u16x2 x, u16x2 y) { return __builtin_elementwise_max(x, y); });
}
__device__ __forceinline__ uint32_t min_bits8(const f16x8& v) {
  return of_eight(v, [](u16x2 x, u16x2 y) { return __builtin_elementwise_min(x, y); });
}

// log2 of an fp16 value from its bits as they stand (less by at most 0.09), and log2 of the fp16
// with these bits
__device__ __forceinline__ float about_log2(f16 v) {
  return __builtin_fmaf((float)__builtin_bit_cast(uint16_t, v), 0.0009765625f, -15.0f);
}
__device__ __forceinline__ float log2_bits(uint32_t bits) {
  return __builtin_amdgcn_logf((float)__builtin_bit_cast(f16, (uint16_t)bits));
}

// A row's reference after a tile, from the row's `sum` (of the lanes' top scores and bounds on
// their value scales) and `one` (the largest that one token has of both); a row that does not
// need to move stays, whatever the wave's other rows do.
__device__ __forceinline__ float moved_reference(float ref, float sum, float one) {
  return sum - kTop > ref + kSlack ? fmaxf(ref, fminf(sum, one + kMixed) - kTop) : ref;
}
// Scores (times log2 e) so large that differences from a rounded reference are off by whole
// powers of two, if the product by p.c is fused with the subtraction: then the products are
// rounded first, and the largest of them is the reference.
__device__ __forceinline__ bool is_far(float ref) { return fabsf(ref) >= kFar && fabsf(ref) < kNone; }
__device__ __forceinline__ float far_reference(float ref, float to, float top) {
  return fabsf(top) >= kFar ? fmaxf(ref, top) : to;
}

// value of a lane of the wave (64 bits)
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}
__device__ __forceinline__ int64_t wave_sums_upto(int64_t v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t u = __shfl_up(v, off);
    v += lane >= off ? u : 0;
  }
  return v;
}

// The tile kernel's work, dealt out in equal shares of its area: the area of a row is the
// number of tokens it sees (its row over the group instead of its token, times 2 group, so
// that sums over rows have a closed form in integers), and a share is an interval of the
// areas of all rows of all sequences, one after the other. Rows count in whole items (128
// rows, as many steps whether all are there or not), and each for kItemTokens tokens more,
// what an item costs before its first and after its last tile. An item of area W and n
// tiles that begins at area X gives a share that ends at area x inside it the tiles up to
// n (x - X) / W.
constexpr int kItemTokens = 96;
__device__ __forceinline__ int64_t area_of_rows(const KvSeq& s, const AttnArgs& p, int64_t rows) {
  const int64_t g2 = 2 * p.group, p0 = s.ctx - s.rows + 1;  // tokens that the first row sees
  const int64_t none = p0 < 0 ? -p0 * p.group : 0;          // rows that see nothing
  const int64_t sees = p0 < 0 ? 0 : p0, r = rows > none ? rows - none : 0;
  // rows up to `grow` see one token more every group rows, the others the whole window
  const int64_t grow = p.window <= 0 ? r : (p.window <= sees ? 0 : min(r, (p.window - sees) * p.group));
  return g2 * sees * grow + grow * (grow - 1) + (r - grow) * g2 * p.window + g2 * kItemTokens * rows;
}
__device__ __forceinline__ int64_t items_of(const KvSeq& s, const AttnArgs& p) {
  return ((int64_t)s.rows * p.group + kTileRows - 1) / kTileRows;
}
__device__ __forceinline__ int64_t area_of_sequence(const KvCache& a, const AttnArgs& p, const KvSeq& s, int b) {
  return b < a.B && (int64_t)s.rows * p.group > p.row_limit ? area_of_rows(s, p, items_of(s, p) * kTileRows) : 0;
}
constexpr int kLeastItemTiles = 16;  // of a share: so many tiles for a whole item, at least
__device__ __forceinline__ int64_t share_area(const AttnArgs& p, int64_t total) {
  const int64_t n = (total + p.tshares - 1) / p.tshares;
  const int64_t least = (int64_t)2 * p.group * kLeastItemTiles * kKvTile * kTileRows;
  return n < least ? least : n;
}
// tiles of an item of n tiles, area W, beginning at area X, that lie before area x (the
// quotient in double: the same one wherever it is asked for)
__device__ __forceinline__ int tiles_before(int64_t x, int64_t X, int64_t W, int n) {
  return x <= X ? 0 : (x >= X + W ? n : min(n, (int)((double)(x - X) * (double)n / (double)W)));
}
// A wave's walk over the sequences, 64 at a time, one a lane, with their areas.
struct AreaWalk {
  int first;
  int64_t before;  // area of the sequences before `first`
  KvSeq s;
  int64_t area, upto;  // of the lane's sequence, and of those from `first` to it
};
__device__ __forceinline__ void area_load(AreaWalk& w, const KvCache& a, const AttnArgs& p, int lane) {
  w.s = kv_sequence(a, min(w.first + lane, a.B - 1));
  w.area = area_of_sequence(a, p, w.s, w.first + lane);
  w.upto = wave_sums_upto(w.area, lane);
}
// the walk's start, and the area in all
__device__ __forceinline__ int64_t area_begin(AreaWalk& w, const KvCache& a, const AttnArgs& p, int lane) {
  int64_t total = 0;
  for (int f = (a.B - 1) & ~63; f >= 0; f -= 64) {  // (the first sequences last: they stay)
    w.first = f;
    area_load(w, a, p, lane);
    total += lane_value(w.upto, 63);
  }
  w.before = 0;
  return total;
}
// An item that area `at` is of: sequence b, row tile rt, its area [X, next).
struct AreaItem {
  int b, rt, have;  // have: row tiles of the sequence
  KvSeq s;
  int64_t begins, X, next;
};
__device__ __forceinline__ int64_t area_before(const AreaItem& t, const AttnArgs& p, int rt) {
  return t.begins + area_of_rows(t.s, p, (int64_t)rt * kTileRows);
}
// false only if the lengths changed meanwhile
__device__ __forceinline__ bool area_find(AreaItem& t, AreaWalk& w, const KvCache& a, const AttnArgs& p, int64_t at,
                                          int lane) {
  while (w.before + lane_value(w.upto, 63) <= at) {
    if (w.first + 64 >= a.B) return false;
    w.before += lane_value(w.upto, 63);
    w.first += 64;
    area_load(w, a, p, lane);
  }
  const int j = __popcll(__ballot(w.before + w.upto <= at));
  t.b = w.first + j;
  t.s.first_row = __builtin_amdgcn_readlane(w.s.first_row, j);
  t.s.rows = __builtin_amdgcn_readlane(w.s.rows, j);
  t.s.ctx = __builtin_amdgcn_readlane(w.s.ctx, j);
  t.begins = w.before + lane_value(w.upto - w.area, j);
  t.have = (int)items_of(t.s, p);
  t.rt = 0;  // the last row tile that begins at or before `at`
  if (t.begins < at)
    for (int over = t.have; over - t.rt > 1;) {
      const int mid = (t.rt + over) >> 1;
      if (area_before(t, p, mid) <= at)
        t.rt = mid;
      else
        over = mid;
    }
  t.X = area_before(t, p, t.rt);
  t.next = area_before(t, p, t.rt + 1);
  return true;
}

// The item of a block that takes row tiles whole, its turn-th: the longest first, and with
// `snake` the later half from the other end.
__device__ __forceinline__ int row_tile_of(int turn, int have, int snake) {
  return snake && turn >= (have + 1) / 2 ? turn - (have + 1) / 2 : have - 1 - turn;
}

// kv4_tile.hip: the tile kernel, and what joins its items that were split
hipError_t launch_kv4_tile(const KvCache& a, const AttnArgs& p, int64_t head_dim, hipStream_t stream);

}  // namespace wq
