// Causal attention over the 4-bit key/value cache, for gfx950.
//
// For a new token at position p of its sequence and a query head with query vector q,
// over the tokens t <= p (and t > p - window), with the cache's k_t ~ (a_t - y_t) s_t and
// v_t ~ (c_t - z_t) u_t (4-bit codes a, c, integer zero-points y, z, scales s, u):
//   x_t = scale q . k_t = scale s_t (q . a_t - y_t sum(q)),
//   out = sum_t w_t v_t / sum_t w_t,   w_t = exp(x_t - r),
// in one pass over the tokens, r a running reference of the row. A row that sees no
// token gives 0 (and -inf for log sum exp).
//
// Both products run on matrix cores in fp16 with fp32 sums, transposed: keys . queries^T
// gives a lane several tokens' scores of one query row, and those are, as they stand,
// the lane's operand of values^T . weights^T, so the weights never leave registers and a
// row's statistics are one lane's scalars. The codes enter the products exactly, less
// their zero-points (as fp16 subnormals, which matrix cores keep, the codes themselves
// need half the unpacking, but their sums then carry 2^-18 of the largest term instead of
// 2^-24, and the zero-points come off as differences of large sums: measured, 1e-4 in a
// score of 50); the one rounding is that of w_t u_t to fp16 (an operand of the second product). Scores,
// maxima, sums and outputs are fp32.
//
// The reference r keeps the fp16 operands in range and precise: weights times value
// scales, 2^(x - r) u, are held near 2^10 at the row's largest, at most 2^14. It only
// moves (and everything summed so far is only rescaled) when a tile's scores or value
// scales would pass that bound, which any lane can see without asking the others.
//
//  kv4_decode_kernel   few query rows (16 or 32 a block): all tiles of all sequences are
//    dealt out in equal shares, one a block, whose four waves take tiles of 32 tokens in
//    turn and join through LDS at each row tile's end.
//  kv4_tile_kernel     many query rows: 128 a block; a tile of codes is turned into exact
//    fp16 integers once, in LDS, for all of them.
//  kv4_combine_kernel  joins the parts of rows that more than one block worked on.
#include "kv4.h"
#include "wq_launch.h"

namespace wq {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr float kNoRef = -1e30f;      // reference of a row that has seen nothing
constexpr float kTop = 10.0f;         // log2 of the largest weight times value scale after a move of r,
constexpr float kSlack = 4.0f;        // and how far it may grow before the next
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kDecodeRows = 16;       // query rows of one column tile
constexpr int kTileRows = 128;        // query rows of a block of kv4_tile_kernel

struct AttnArgs {
  const f16* q;
  int64_t q_stride;
  const uint8_t* cache;
  f16* out;
  float* lse;         // may be null
  float* part_o;      // partials of the decode kernel, two a block: [block][2][rows][D]
  float2* part_s;     // [block][2][rows]: r, sum
  float* tpart_o;     // partials of the tile kernel: [T * hq][tnsplit][D]
  float2* tpart_s;    // [T * hq][tnsplit]
  int hq, group;      // query heads, and those of one key/value head
  int window;         // 0: none
  float c;            // scale * log2(e)
  int shares, least;  // decode kernel: blocks a head, and the fewest tiles of one
  int decode_rows;    // rows of an item of the decode kernel (16 or 32)
  int tnsplit, tchunk_tiles;  // tile kernel: most chunks of a row, and their tiles
  int row_limit;      // sequences with more rows of a head belong to the tile kernel
};

// Tiles [t0, t1) of a sequence that rows row0 .. row1 (of one head group) can see.
struct TileRange {
  int t0, t1;
};
__device__ __forceinline__ TileRange tile_range(const KvSeq& s, const AttnArgs& p, int row0, int row1) {
  const int p0 = s.ctx - s.rows + row0 / p.group, p1 = s.ctx - s.rows + row1 / p.group;
  const int lo = p.window > 0 ? max(p0 - p.window + 1, 0) : 0;
  TileRange r;
  r.t0 = lo / kKvTile;
  r.t1 = p1 < lo ? r.t0 : p1 / kKvTile + 1;
  return r;
}
// ... and the tile kernel's chunks of them
struct TileSplit {
  int chunk, splits;
};
__device__ __forceinline__ TileSplit tile_split(const TileRange& r, const AttnArgs& p) {
  const int n = r.t1 - r.t0;
  TileSplit t;
  t.chunk = max(p.tchunk_tiles, (n + p.tnsplit - 1) / p.tnsplit);
  t.splits = (n + t.chunk - 1) / t.chunk;
  return t;
}

// The decode kernel's work: its items are a sequence's row tiles, in order, each as many
// steps as the sequence has visible tiles (one where it has none: its rows are still to
// be written). All steps of a head are dealt out in equal shares, one a block, so that
// blocks end together however the sequences' lengths differ; an item that lies in one
// share is finished there, others leave a partial in each. A wave looks at 64 sequences
// at a time, one a lane.
struct Sequences {
  KvSeq s;
  int t0, n;      // first visible tile, steps of an item (0: nothing to do here)
  int64_t steps, upto;  // of the sequence, and of those up to it, from `first` on
};
__device__ __forceinline__ Sequences load_sequences(const KvCache& a, const AttnArgs& p, int first, int lane) {
  Sequences q;
  const int b = first + lane;
  q.s = kv_sequence(a, min(b, a.B - 1));
  const int rows = q.s.rows * p.group;
  const bool mine = b < a.B && rows > 0 && rows <= p.row_limit;
  const TileRange r = tile_range(q.s, p, 0, rows - 1);
  q.t0 = r.t0;
  q.n = mine ? max(r.t1 - r.t0, 1) : 0;
  q.steps = (int64_t)q.n * ((rows + p.decode_rows - 1) / p.decode_rows);
  q.upto = q.steps;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t v = __shfl_up(q.upto, off);
    q.upto += lane >= off ? v : 0;
  }
  return q;
}
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}
// steps of a head in all; `q` holds the first 64 sequences
__device__ __forceinline__ int64_t total_steps(const KvCache& a, const AttnArgs& p, const Sequences& q, int lane) {
  int64_t n = lane_value(q.upto, 63);
  for (int first = 64; first < a.B; first += 64) n += lane_value(load_sequences(a, p, first, lane).upto, 63);
  return n;
}
__device__ __forceinline__ int64_t share_steps(const AttnArgs& p, int64_t total) {
  const int64_t n = total < (int64_t)1 << 31 ? (int64_t)((uint32_t)(total + p.shares - 1) / (uint32_t)p.shares)
                                             : (total + p.shares - 1) / p.shares;
  return n < p.least ? p.least : n;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// a * b with the fp16 factor read as it is (one mixed-precision instruction; the sum with
// 0 keeps the compiler from splitting it into a conversion and a product)
__device__ __forceinline__ float mul_mix(float a, f16 b) { return __builtin_fmaf(a, (float)b, 0.0f); }

// largest of eight positive fp16 values, as bits (positive fp16 order like integers)
__device__ __forceinline__ uint32_t max_bits8(const f16x8& v) {
  const uint4 d = __builtin_bit_cast(uint4, v);
  const u16x2 a = __builtin_elementwise_max(__builtin_bit_cast(u16x2, d.x), __builtin_bit_cast(u16x2, d.y));
  const u16x2 b = __builtin_elementwise_max(__builtin_bit_cast(u16x2, d.z), __builtin_bit_cast(u16x2, d.w));
  const u16x2 m = __builtin_elementwise_max(a, b);
  return max((uint32_t)m.x, (uint32_t)m.y);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kDepth = 2;  // tiles of a wave's ring: one in use, one on its way

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A lane's share of a tile in LDS. Read in assembly, with the wait inside: the compiler
// would hold any read of its own back until every load into LDS has landed, the later
// tiles' too.
template <int D>
struct TileData {
  u32x4 k[D / 64], v[D / 64], ks, vs, vz;
  uint32_t kz;
};
template <int D>
__device__ __forceinline__ void lds_tile(TileData<D>& t, uint32_t at, int lane) {
  const uint32_t code = at + 16 * lane, group = at + 16 * (lane >> 4), one = at + 4 * (lane & 15);
  if constexpr (D == 128) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:1024\n\t"
        "ds_read_b32 %7, %10 offset:4160\n\tds_read_b128 %4, %9 offset:4096\n\t"
        "ds_read_b128 %5, %9 offset:4224\n\tds_read_b128 %6, %9 offset:4288\n\t"
        "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %8 offset:3072\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(t.k[0]), "=&v"(t.k[1]), "=&v"(t.v[0]), "=&v"(t.v[1]), "=&v"(t.ks), "=&v"(t.vs), "=&v"(t.vz),
          "=&v"(t.kz)
        : "v"(code), "v"(group), "v"(one)
        : "memory");
  } else {
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b32 %5, %8 offset:2112\n\tds_read_b128 %2, %7 offset:2048\n\t"
        "ds_read_b128 %3, %7 offset:2176\n\tds_read_b128 %4, %7 offset:2240\n\t"
        "ds_read_b128 %1, %6 offset:1024\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(t.k[0]), "=&v"(t.v[0]), "=&v"(t.ks), "=&v"(t.vs), "=&v"(t.vz), "=&v"(t.kz)
        : "v"(code), "v"(group), "v"(one)
        : "memory");
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(256)
kv4_decode_kernel(KvCache a, AttnArgs p) {
  constexpr int KW = D / 32;   // steps of the first product
  constexpr int CT = D / 16;   // channel tiles of the second
  constexpr int ROWS = kDecodeRows * NT;
  constexpr int TILE = kv_tile_bytes<D>();
  // each wave's ring of tiles, and at the end the waves' results
  constexpr int kMerge = 4 * kDecodeRows * (D + 4) * 4;
  __shared__ __align__(16) uint8_t lds[kDepth * 4 * TILE > kMerge ? kDepth * 4 * TILE : kMerge];
  __shared__ float ref_s[4][kDecodeRows], sum_s[4][kDecodeRows];
  float(*merged)[kDecodeRows][D + 4] = reinterpret_cast<float(*)[kDecodeRows][D + 4]>(lds);
  // heads next to each other, so that the XCDs, which take blocks in turn, share every
  // sequence alike
  const int h = blockIdx.x % a.hkv, share = blockIdx.x / a.hkv;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t magic = magic_1024x2();

  int first = 0;        // of the 64 sequences at hand
  int64_t before = 0;   // steps of the sequences before them
  Sequences seqs = load_sequences(a, p, 0, lane);
  const int64_t total = total_steps(a, p, seqs, lane), per = share_steps(p, total);
  int64_t at = share * per;
  const int64_t until = at + per < total ? at + per : total;
  bool opening = true;  // the share's first item: its partial goes to slot 0, another's to slot 1
  while (at < until) {
    while (before + lane_value(seqs.upto, 63) <= at) {
      if (first + 64 >= a.B) return;  // (only if the lengths changed meanwhile)
      before += lane_value(seqs.upto, 63);
      first += 64;
      seqs = load_sequences(a, p, first, lane);
    }
    const int j = __popcll(__ballot(before + seqs.upto <= at));  // the sequence that step `at` is of
    const int b = first + j;
    KvSeq s;
    s.first_row = __builtin_amdgcn_readlane(seqs.s.first_row, j);
    s.rows = __builtin_amdgcn_readlane(seqs.s.rows, j);
    s.ctx = __builtin_amdgcn_readlane(seqs.s.ctx, j);
    const int t0 = __builtin_amdgcn_readlane(seqs.t0, j), steps = __builtin_amdgcn_readlane(seqs.n, j);
    const int rows = s.rows * p.group;
    const int64_t into = at - (before + lane_value(seqs.upto - seqs.steps, j));
    const int rt = rows > ROWS ? (int)(into / steps) : 0;
    const int from = (int)(into - (int64_t)rt * steps);
    const int count = (int)(until - at < steps - from ? until - at : steps - from);
    const bool whole = count == steps;
    at += count;
    const int row0 = rt * ROWS, row1 = min(rows, row0 + ROWS) - 1;
    const int p0 = s.ctx - s.rows + row0 / p.group, p1 = s.ctx - s.rows + row1 / p.group;

    // the lane's query rows: operands of the first product, and position
    f16x8 qf[NT][KW];
    int pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + kDecodeRows * n + c;
      const bool valid = row < rows;
      const int tok = valid ? row / p.group : 0;
      const int head = h * p.group + (valid ? row - tok * p.group : 0);
      pos[n] = valid ? s.ctx - s.rows + tok : -1;
      const f16* qp = p.q + (int64_t)(s.first_row + tok) * p.q_stride + head * D + (D / 4) * g;
#pragma unroll
      for (int w = 0; w < KW; ++w) qf[n][w] = as_f16x8(*reinterpret_cast<const uint4*>(qp + 8 * w));
    }

    f32x4 acc[NT][CT];
    float ref[NT], sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      ref[n] = kNoRef;
      sum[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[n][t] = f32x4{};
    }
    float vexp = 0.0f;          // value scales seen are at most 2^vexp, the fp16 with bits vbits
    uint32_t vbits = 0;

    const int begin = t0 + from, end = s.ctx > 0 ? begin + count : begin;
    int tile = begin + wave;
    int page = tile / a.page_tiles, in_page = tile - page * a.page_tiles;
    uint8_t* ring = lds + wave * kDepth * TILE;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)ring;
    // one tile's bytes, contiguous in memory, straight into a stage of the ring: D / 32
    // runs of 16 bytes a lane and one of 4
    constexpr int LOADS = D / 32 + 1;
    // numbers of 64 pages, one a lane: a load each tile would have to wait for the tiles
    // on their way
    int ids = 0, ids_page = page;
    const auto load_ids = [&]() {
      ids = a.page_table[(int64_t)b * a.max_pages + min(ids_page + lane, a.max_pages - 1)];
      asm volatile("" : "+v"(ids));  // waited for here
    };
    if (tile < end) load_ids();
    const auto fetch = [&](int stage) {
      if (page - ids_page >= 64) {
        ids_page = page;
        load_ids();
      }
      const int id = __builtin_amdgcn_readlane(ids, page - ids_page);
      const auto rsrc = buffer_rsrc(p.cache + kv_page_offset(a, h, id) + (int64_t)in_page * TILE, (uint32_t)TILE);
      auto* dst = (__attribute__((address_space(3))) uint8_t*)(ring + stage * TILE);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst + 1024 * i, 16, 16 * lane, 1024 * i, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst + 32 * D, 4, 4 * lane, 32 * D, 0, 0);
      in_page += 4;
      while (in_page >= a.page_tiles) {
        in_page -= a.page_tiles;
        ++page;
      }
    };
    int fetched = tile, stage_in = 0, stage = 0;
    const auto fetch_next = [&]() {
      if (fetched < end) fetch(stage_in);
      fetched += 4;
      stage_in = stage_in + 1 == kDepth ? 0 : stage_in + 1;
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch_next();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint4 d = perm_x8(__builtin_bit_cast(uint4, qf[n][w]));
        const uint32_t m = pos[n] < 0 ? 0u : 0xFFFFFFFFu;  // (a row that sees nothing may be no row at all)
        qf[n][w] = as_f16x8(uint4{d.x & m, d.y & m, d.z & m, d.w & m});
      }
    for (; tile < end; tile += 4) {
      fetch_next();
      // this tile's loads are done when only the later tiles' are left
      const int later = (end - 1 - tile) >> 2;
      if (later >= kDepth - 1)
        wait_vm<(kDepth - 1) * LOADS>();
      else if (kDepth > 2 && later == 1)
        wait_vm<LOADS>();
      else if (kDepth > 3 && later == 2)
        wait_vm<2 * LOADS>();
      else
        wait_vm<0>();
      const uint32_t at = ring_at + stage * TILE;
      stage = stage + 1 == kDepth ? 0 : stage + 1;
      TileData<D> cur;
      lds_tile<D>(cur, at, lane);

      // scores: lane's tokens 4 g + i + 16 half of the tile at index i + 4 half
      const f16x8 ks = __builtin_bit_cast(f16x8, cur.ks);
      const KeyZeros kz = kv_key_zeros(cur.kz);
      f16x8 vs = __builtin_bit_cast(f16x8, cur.vs);
      uint4 vz = __builtin_bit_cast(uint4, cur.vz);
      float x[NT][8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 sc[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n] = f32x4{};
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const f16x8 k = as_f16x8(codes_minus_zero_x16(cur.k[(KW * half + w) >> 2][(KW * half + w) & 3], magic, kz.bias[half], kz.nbias16[half]));
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[n] = mfma_16x16x32(k, qf[n][w], sc[n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[n][i + 4 * half] = mul_mix(sc[n][i], ks[i + 4 * half]);
      }

      const int first = tile * kKvTile;
      const bool edge = first + kKvTile - 1 > p0 || (p.window > 0 && first <= p1 - p.window);
      uint32_t seen[NT];
      if (edge) {
        // tokens past a row's own, before its window or past the cache's end: whatever
        // stands there, codes, scales or zero-points, has no part in the row
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          seen[n] = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int t = first + 4 * g + (e & 3) + 16 * (e >> 2);
            const bool see = t <= pos[n] && (p.window == 0 || t > pos[n] - p.window);
            x[n][e] = see ? x[n][e] : -INFINITY;
            seen[n] |= see ? 1u << e : 0u;
          }
        }
        uint32_t any = seen[0];
#pragma unroll
        for (int n = 1; n < NT; ++n) any |= seen[n];
#pragma unroll
        for (int e = 0; e < 8; ++e) vs[e] = (any >> e) & 1u ? vs[e] : (f16)0.0f;
        vz = kv_value_zeros_finite(vz);
      }

      float mx[NT];
      const uint32_t vmax = max_bits8(vs);
      bool move = vmax > vbits;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mx[n] = x[n][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx[n] = fmaxf(mx[n], x[n][e]);
        mx[n] *= p.c;
        move |= mx[n] + vexp - kTop > ref[n] + kSlack;
      }
      if (__any(move)) {
        uint32_t top = vmax;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        float grown = 0.0f;
        if (top > vbits) {
          // the next power of two: exponent field + 1, mantissa 0 (scales are normal fp16)
          const float ve = (float)((int)(top >> 10) + 1 - 15);
          grown = vbits == 0 ? 0.0f : ve - vexp;
          vexp = ve;
          vbits = ((top >> 10) << 10) | 0x3FFu;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float m = mx[n];
          m = fmaxf(m, __shfl_xor(m, 16));
          m = fmaxf(m, __shfl_xor(m, 32));
          const float to = fmaxf(ref[n] + grown, m + vexp - kTop);
          const float f = exp2_hw(ref[n] - to);
          ref[n] = to;
          sum[n] *= f;
#pragma unroll
          for (int t = 0; t < CT; ++t) acc[n][t] *= f;
        }
      }

      // weights, and weights times value scales as the operand of the second product
      f16x8 wf[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = exp2_hw(__builtin_fmaf(x[n][e], p.c, -ref[n]));
          sum[n] += w;
          wf[n][2 * (e & 3) + (e >> 2)] = (f16)mul_mix(w, vs[e]);
        }
      }
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const f16x8 v = kv_value_operand(cur.v[t >> 2][t & 3], magic, vz);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][t] = mfma_16x16x32(v, wf[n], acc[n][t]);
      }
    }

    // join the four waves
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float su = sum[n];
      su += __shfl_xor(su, 16);
      su += __shfl_xor(su, 32);
      __syncthreads();  // every wave is done with its ring, and with the previous column tile
      if (g == 0) {
        ref_s[wave][c] = ref[n];
        sum_s[wave][c] = su;
      }
      __syncthreads();
      float top = ref_s[0][c];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, ref_s[w][c]);
      const float f = exp2_hw(ref[n] - top);
#pragma unroll
      for (int t = 0; t < CT; ++t) *reinterpret_cast<f32x4*>(&merged[wave][c][16 * t + 4 * g]) = acc[n][t] * f;
      __syncthreads();
      // 16 threads a row, D / 16 channels each
      const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
      const int row = row0 + kDecodeRows * n + r;
      if (row < rows) {
        float best = ref_s[0][r];
#pragma unroll
        for (int w = 1; w < 4; ++w) best = fmaxf(best, ref_s[w][r]);
        float total_sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) total_sum = __builtin_fmaf(sum_s[w][r], exp2_hw(ref_s[w][r] - best), total_sum);
        float o[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i)
          o[i] = (merged[0][r][CT * part + i] + merged[1][r][CT * part + i]) +
                 (merged[2][r][CT * part + i] + merged[3][r][CT * part + i]);
        if (!whole) {
          const int64_t slot = ((int64_t)blockIdx.x * 2 + (opening ? 0 : 1)) * ROWS + kDecodeRows * n + r;
          float* dst = p.part_o + slot * D + CT * part;
#pragma unroll
          for (int i = 0; i < CT; i += 4) *reinterpret_cast<f32x4*>(dst + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
          if (part == 0) p.part_s[slot] = make_float2(best, total_sum);
        } else {
          const int tok = row / p.group;
          const int64_t at_row = (int64_t)(s.first_row + tok) * p.hq + h * p.group + (row - tok * p.group);
          const float inv = total_sum > 0.0f ? 1.0f / total_sum : 0.0f;
          f16* dst = p.out + at_row * D + CT * part;
#pragma unroll
          for (int i = 0; i < CT; i += 4) {
            typedef f16 f16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<f16x4*>(dst + i) =
                f16x4{(f16)(o[i] * inv), (f16)(o[i + 1] * inv), (f16)(o[i + 2] * inv), (f16)(o[i + 3] * inv)};
          }
          if (part == 0 && p.lse != nullptr) p.lse[at_row] = total_sum > 0.0f ? (best + log2f(total_sum)) * kLn2 : -INFINITY;
        }
      }
    }
    __syncthreads();
    opening = false;
  }
}

template <int D>
__global__ void __launch_bounds__(256)
kv4_tile_kernel(KvCache a, AttnArgs p, int row_tiles) {
  constexpr int KS = D / 16;   // steps of the first product
  constexpr int CT = D / 32;   // channel tiles of the second
  constexpr int RUNS = D / 64;
  // two tiles of 32 tokens: keys [step][lane], values [step][channel tile][lane], 16
  // bytes each, and the tiles' scales
  __shared__ __align__(16) uint4 kl[2][KS][64], vl[2][2][CT][64];
  __shared__ __align__(16) uint4 ksl[2][4], vsl[2][4];
  const int lane = threadIdx.x & 63, c = lane & 31, hl = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // heads next to each other: with eight of them, each XCD's L2 serves one
  const int h = blockIdx.x % a.hkv, split = blockIdx.x / a.hkv % p.tnsplit;
  const int rest = blockIdx.x / a.hkv / p.tnsplit;
  const int b = rest / row_tiles;
  const KvSeq s = kv_sequence(a, b);
  const int rows = s.rows * p.group;
  if (rows <= p.row_limit) return;
  const int have = (rows + kTileRows - 1) / kTileRows;
  // the last rows see the most tokens: they start first
  for (int back = rest % row_tiles; back < have; back += row_tiles) {
    const int rt = have - 1 - back;
    const int row0 = rt * kTileRows, row1 = min(rows, row0 + kTileRows) - 1;
    const TileRange range = tile_range(s, p, row0, row1);
    const TileSplit parts = tile_split(range, p);
    if (split > 0 && split >= parts.splits) continue;
    const int p0 = s.ctx - s.rows + row0 / p.group, p1 = s.ctx - s.rows + row1 / p.group;
    const int row = row0 + 32 * wave + c;
    const bool valid = row < rows;
    const int tok = valid ? row / p.group : 0;
    const int head = h * p.group + (valid ? row - tok * p.group : 0);
    const int pos = valid ? s.ctx - s.rows + tok : -1;
    f16x8 qf[KS];
    const f16* qp = p.q + (int64_t)(s.first_row + tok) * p.q_stride + head * D + 8 * hl;
#pragma unroll
    for (int w = 0; w < KS; ++w) {
      uint4 d = *reinterpret_cast<const uint4*>(qp + 16 * w);
      if (!valid) d = uint4{0, 0, 0, 0};
      qf[w] = as_f16x8(perm_x8(d));
    }
    f32x16 acc[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) acc[t] = f32x16{};
    float ref = kNoRef, sum = 0.0f, vexp = 0.0f;
    uint32_t vbits = 0;

    const int begin = range.t0 + split * parts.chunk, end = min(range.t1, begin + parts.chunk);
    // each wave turns one tile's keys or values into LDS operands: waves 0, 1 the first
    // tile's, waves 2, 3 the second's
    const int sub = wave >> 1;
    const bool is_v = wave & 1;
    const int g = lane >> 4, c16 = lane & 15;
    uint4 data[RUNS], scales, zeros;
    const auto load = [&](int tile) {
      tile = min(tile, end - 1);  // past the range: loaded again, and masked by position
      const int page = tile / a.page_tiles;
      const uint8_t* base = p.cache + kv_page_offset(a, b, h, page) +
                            (int64_t)(tile - page * a.page_tiles) * kv_tile_bytes<D>();
      const int off = is_v ? kv_value_offset<D>() : kv_key_offset<D>();
#pragma unroll
      for (int i = 0; i < RUNS; ++i) data[i] = *reinterpret_cast<const uint4*>(base + off + 1024 * i + 16 * lane);
      const uint8_t* meta = base + kv_meta_offset<D>(is_v ? 2 : 0);
      scales = *reinterpret_cast<const uint4*>(meta + 16 * (lane & 3));
      if (is_v)
        zeros = *reinterpret_cast<const uint4*>(meta + 64 + 16 * g);
      else
        zeros.x = *reinterpret_cast<const uint32_t*>(meta + 64 + 4 * c16);
    };
    const uint32_t magic = magic_1024x2();
    const auto stash = [&]() {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&data[0]);
      if (!is_v) {
        const KeyZeros kz = kv_key_zeros(zeros.x);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int block = (D / 32) * g + i;  // eight channels
            kl[sub][block >> 1][32 * (block & 1) + 16 * half + c16] =
                codes_minus_zero_x16(w[(D / 32) * half + i], magic, kz.bias[half], kz.nbias16[half]);
          }
        if (lane < 4) ksl[sub][lane] = scales;
      } else {
        // what stands past the cache's end may be anything; its weight is 0
        zeros = kv_value_zeros_finite(zeros);
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
          vl[sub][g >> 1][t >> 1][32 * (g & 1) + 16 * (t & 1) + c16] =
              __builtin_bit_cast(uint4, kv_value_operand(w[t], magic, zeros));
        if (lane < 4) vsl[sub][lane] = scales;
      }
    };

    if (begin < end) load(begin + sub);
    for (int tile = begin; tile < end; tile += 2) {
      __syncthreads();  // the previous tiles have been read
      stash();
      __syncthreads();
      if (tile + 2 < end) load(tile + 2 + sub);

      f32x16 sc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sc[u] = f32x16{};
#pragma unroll
        for (int w = 0; w < KS; ++w)
          sc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_f16x8(kl[u][w][lane]), qf[w], sc[u], 0, 0, 0);
      }
      // the lane's tokens: 8 q + 4 hl + i of a tile in register 4 q + i; quads q and
      // q + 2 (q = 0, 1) are one run of scales
      f16x8 vs[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f16x8 ks = as_f16x8(ksl[u][2 * q + hl]);
          vs[u][q] = as_f16x8(vsl[u][2 * q + hl]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = 4 * (q + 2 * (e >> 2)) + (e & 3);
            sc[u][r] = mul_mix(sc[u][r], ks[e]);
          }
        }
      const int first = tile * kKvTile;
      const bool edge = first + 2 * kKvTile - 1 > p0 || (p.window > 0 && first <= p1 - p.window) || tile + 1 >= end;
      if (edge) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int t = first + 32 * u + 8 * (e >> 2) + 4 * hl + (e & 3);
            const bool see = t <= pos && (p.window == 0 || t > pos - p.window) && tile + u < end;
            sc[u][e] = see ? sc[u][e] : -INFINITY;
          }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              vs[u][q][e] = sc[u][4 * (q + 2 * (e >> 2)) + (e & 3)] == -INFINITY ? (f16)0.0f : vs[u][q][e];
      }
      float mx = -INFINITY;
      uint32_t vmax = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sc[u][e]);
        vmax = max(vmax, max(max_bits8(vs[u][0]), max_bits8(vs[u][1])));
      }
      mx *= p.c;
      if (__any(vmax > vbits || mx + vexp - kTop > ref + kSlack)) {
        uint32_t top = vmax;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
        float grown = 0.0f;
        if (top > vbits) {
          const float ve = (float)((int)(top >> 10) + 1 - 15);
          grown = vbits == 0 ? 0.0f : ve - vexp;
          vexp = ve;
          vbits = ((top >> 10) << 10) | 0x3FFu;
        }
        const float m = fmaxf(mx, __shfl_xor(mx, 32));
        const float to = fmaxf(ref + grown, m + vexp - kTop);
        const float f = exp2_hw(ref - to);
        ref = to;
        sum *= f;
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[t] *= f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          f16x8 wf;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w = exp2_hw(__builtin_fmaf(sc[u][4 * (q + 2 * (e >> 2)) + (e & 3)], p.c, -ref));
            sum += w;
            wf[2 * (e & 3) + (e >> 2)] = (f16)mul_mix(w, vs[u][q][e]);
          }
#pragma unroll
          for (int t = 0; t < CT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_f16x8(vl[u][q][t][lane]), wf, acc[t], 0, 0, 0);
        }
    }
    sum += __shfl_xor(sum, 32);
    if (valid) {
      const int64_t slot = (int64_t)(s.first_row + tok) * p.hq + head;
      if (parts.splits > 1) {
        const int64_t at = slot * p.tnsplit + split;
        float* dst = p.tpart_o + at * D + 4 * hl;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(dst + 32 * t + 8 * q) =
                f32x4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
        if (hl == 0) p.tpart_s[at] = make_float2(ref, sum);
      } else {
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        f16* dst = p.out + slot * D + 4 * hl;
        typedef f16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f16x4*>(dst + 32 * t + 8 * q) =
                f16x4{(f16)(acc[t][4 * q] * inv), (f16)(acc[t][4 * q + 1] * inv), (f16)(acc[t][4 * q + 2] * inv),
                      (f16)(acc[t][4 * q + 3] * inv)};
        if (hl == 0 && p.lse != nullptr) p.lse[slot] = sum > 0.0f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
      }
    }
  }
}

// Joins the partials of rows that were split: those of the decode kernel (kTiled false)
// or of the tile kernel. W waves per row (1, 4 or 16, so that a wave takes about eight);
// rows that are already written are left alone. by_sequence: the rows looked at are the
// first row_limit of each sequence and head, not all of the output.
template <int D, int W, bool kTiled>
__global__ void __launch_bounds__(W < 4 ? 256 : 64 * W)
kv4_combine_kernel(KvCache a, AttnArgs p, int by_sequence) {
  constexpr int ROWS = W < 4 ? 4 / W : 1;  // rows of a block
  constexpr int N = D / 64;                // channels of a lane
  __shared__ float joined[W][D + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t item = (int64_t)blockIdx.x * ROWS + (W == 1 ? wave : 0);
  int b, h, row;
  KvSeq s;
  if (by_sequence) {
    row = (int)(item % p.row_limit);
    item /= p.row_limit;
    h = (int)(item % a.hkv);
    b = (int)(item / a.hkv);
    if (b >= a.B) return;
    s = kv_sequence(a, b);
    if (row >= s.rows * p.group) return;
  } else {
    if (item >= (int64_t)a.T * p.hq) return;
    const int token = (int)(item / p.hq), head = (int)(item % p.hq);
    // the token's sequence: the last one that starts at or before it
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.seq_start[mid] <= token)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    s = kv_sequence(a, b);
    const int tok = token - s.first_row;
    if (tok < 0 || tok >= s.rows) return;
    h = head / p.group;
    row = tok * p.group + head % p.group;
  }
  const int rows = s.rows * p.group;
  if ((rows > p.row_limit) != kTiled) return;
  const int64_t out_row = (int64_t)(s.first_row + row / p.group) * p.hq + h * p.group + row % p.group;

  // the row's partials: number i is at base + i * stride, but the first at `start`
  int parts;
  int64_t start, base, stride;
  const float* po;
  const float2* ps;
  if constexpr (kTiled) {
    const int row0 = row / kTileRows * kTileRows, row1 = min(rows, row0 + kTileRows) - 1;
    parts = tile_split(tile_range(s, p, row0, row1), p).splits;
    start = base = out_row * p.tnsplit;
    stride = 1;
    po = p.tpart_o;
    ps = p.tpart_s;
  } else {
    Sequences q = load_sequences(a, p, 0, lane);
    const int64_t per = share_steps(p, total_steps(a, p, q, lane));
    int64_t before = 0;
    for (int first = 64; first <= b; first += 64) {
      before += lane_value(q.upto, 63);
      q = load_sequences(a, p, first, lane);
    }
    const int n = __builtin_amdgcn_readlane(q.n, b & 63);
    const int64_t from = before + lane_value(q.upto - q.steps, b & 63) + (int64_t)(row / p.decode_rows) * n;
    const int64_t i0 = from / per, i1 = (from + n - 1) / per;
    parts = (int)(i1 - i0) + 1;
    // share i of head h is block i * hkv + h, two partials each: the share that the item
    // begins inside has it second
    const auto slot = [&](int64_t i, int second) {
      return ((i * a.hkv + h) * 2 + second) * p.decode_rows + row % p.decode_rows;
    };
    base = slot(i0, 0);
    stride = (int64_t)a.hkv * 2 * p.decode_rows;
    start = slot(i0, from > i0 * per);
    po = p.part_o;
    ps = p.part_s;
  }
  if (parts <= 1) return;
  const auto place = [&](int i) { return i == 0 ? start : base + i * stride; };
  // every wave finds the row's reference and sum, a partial a lane
  float best = kNoRef, total = 0.0f;
  for (int i = lane; i < parts; i += 64) best = fmaxf(best, ps[place(i)].x);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) best = fmaxf(best, __shfl_xor(best, off));
  for (int i = lane; i < parts; i += 64) {
    const float2 v = ps[place(i)];
    total = __builtin_fmaf(v.y, exp2_hw(v.x - best), total);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
  float o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.0f;
#pragma unroll 8
  for (int i = W == 1 ? 0 : wave; i < parts; i += W) {
    const int64_t at = place(i);
    const float f = exp2_hw(ps[at].x - best);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = __builtin_fmaf(po[at * D + N * lane + e], f, o[e]);
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < N; ++e) joined[wave][N * lane + e] = o[e];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      o[e] = joined[0][N * lane + e];
#pragma unroll
      for (int w = 1; w < W; ++w) o[e] += joined[w][N * lane + e];
    }
  }
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
  f16* dst = p.out + out_row * D + N * lane;
#pragma unroll
  for (int e = 0; e < N; ++e) dst[e] = (f16)(o[e] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[out_row] = total > 0.0f ? (best + log2f(total)) * kLn2 : -INFINITY;
}

namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kDecodeBlocks = 2;  // blocks a CU (three fit; measured slower by 2 %: more, shorter shares)
constexpr int64_t kLeastTiles = 8;    // of a share: two a wave

struct Plan {
  bool decode, tile;  // which kernels run
  int decode_rows, row_limit;
  int64_t shares;     // decode kernel: blocks a head
  int trow_tiles;     // tile kernel: row tiles of a sequence that get blocks of their own
  int tnsplit, tchunk;
  int64_t tslots, tmost;  // rows of its partials (0: not split), and a bound of tnsplit
};

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

Plan make_plan(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t max_q, int64_t max_ctx, int64_t window) {
  Plan p = {};
  const int64_t group = hq / hkv;
  const int64_t q = max_q < 1 ? 1 : (max_q > T ? T : max_q);
  const int64_t rows = q * group;
  constexpr int64_t kLimit = 2 * kDecodeRows;
  // a sequence's rows decide its kernel; from the host only the largest is known, and
  // that all are alike where there is one sequence or B max_q new tokens
  p.tile = rows > kLimit;
  p.decode = !p.tile || (B > 1 && B * q > T);
  p.row_limit = p.tile ? (p.decode ? (int)kLimit : 0) : 0x7FFFFFFF;
  p.decode_rows = p.tile || rows > kDecodeRows ? 2 * kDecodeRows : kDecodeRows;
  int64_t tiles = ceil_div(max_ctx < 1 ? 1 : max_ctx, kKvTile);
  if (window > 0) {  // q rows see up to window + q - 1 tokens, which may begin inside a tile
    const int64_t in_window = ceil_div(window + q - 1, kKvTile) + 1;
    tiles = in_window < tiles ? in_window : tiles;
  }
  p.shares = 1;
  if (p.decode) {
    // as many blocks as run well at once, each with an equal share; one a head where the
    // heads alone are as many
    constexpr int64_t resident = kCus * kDecodeBlocks;
    const int64_t most = ceil_div(B * ceil_div(p.tile ? kLimit : rows, p.decode_rows) * tiles, kLeastTiles);
    p.shares = resident / hkv < most ? resident / hkv : most;
    if (p.shares < 1) p.shares = 1;
  }
  p.tnsplit = 1;
  p.tchunk = (int)tiles;
  if (p.tile) {
    const int64_t blocks = B * hkv * ceil_div(rows, kTileRows);
    int64_t n = ceil_div(2 * kCus, blocks);
    const int64_t most = ceil_div(tiles, 16);
    p.tmost = n > most ? most : n;  // (never falls as max_ctx grows: see the workspace)
    p.tchunk = (int)ceil_div(tiles, p.tmost);
    p.tnsplit = (int)ceil_div(tiles, p.tchunk);
    if (p.tmost > 1) p.tslots = T * hq;
    const int64_t most_blocks = 0x7FFFFFFF / (B * hkv);  // split only where blocks are few
    p.trow_tiles = (int)(ceil_div(rows, kTileRows) < most_blocks ? ceil_div(rows, kTileRows) : most_blocks);
  }
  return p;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
// rows of partials, each with D sums, its reference and its sum
int64_t decode_slots(const Plan& pl, int64_t hkv) { return pl.shares > 1 ? hkv * pl.shares * 2 * pl.decode_rows : 0; }
size_t part_bytes(int64_t slots, int64_t D) { return round256((size_t)slots * (D * 4 + 8)); }

// items: rows to look at; parts: those of a row, about
template <int D, bool kTiled>
hipError_t combine(const KvCache& a, const AttnArgs& p, int64_t parts, int64_t items, int by_sequence,
                   hipStream_t stream) {
  if (parts <= 8)
    hipLaunchKernelGGL((kv4_combine_kernel<D, 1, kTiled>), dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, a,
                       p, by_sequence);
  else if (parts <= 32)
    hipLaunchKernelGGL((kv4_combine_kernel<D, 4, kTiled>), dim3((unsigned)items), dim3(256), 0, stream, a, p,
                       by_sequence);
  else
    hipLaunchKernelGGL((kv4_combine_kernel<D, 16, kTiled>), dim3((unsigned)items), dim3(1024), 0, stream, a, p,
                       by_sequence);
  return hipGetLastError();
}

template <int D>
hipError_t run(const KvCache& a, const AttnArgs& p, const Plan& pl, int64_t B, int64_t hkv, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const int64_t out_rows = (int64_t)a.T * p.hq;
  if (pl.tile) {
    const dim3 grid((unsigned)(B * hkv * pl.trow_tiles * pl.tnsplit));
    hipLaunchKernelGGL((kv4_tile_kernel<D>), grid, dim3(256), 0, stream, a, p, pl.trow_tiles);
    e = hipGetLastError();
  }
  if (e == hipSuccess && pl.decode) {
    const dim3 grid((unsigned)(hkv * pl.shares));
    if (pl.decode_rows == kDecodeRows)
      hipLaunchKernelGGL((kv4_decode_kernel<D, 1>), grid, dim3(256), 0, stream, a, p);
    else
      hipLaunchKernelGGL((kv4_decode_kernel<D, 2>), grid, dim3(256), 0, stream, a, p);
    e = hipGetLastError();
  }
  if (e == hipSuccess && pl.decode && pl.shares > 1)
    e = combine<D, false>(a, p, pl.shares / B + 1, pl.tile ? B * hkv * p.row_limit : out_rows, pl.tile, stream);
  if (e == hipSuccess && pl.tile && pl.tnsplit > 1) e = combine<D, true>(a, p, pl.tnsplit, out_rows, 0, stream);
  return e;
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q,
                                     int64_t max_ctx) {
  const Plan pl = make_plan(T, B, hq, hkv, max_q, max_ctx, 0);
  return part_bytes(decode_slots(pl, hkv), head_dim) + part_bytes(pl.tslots * pl.tmost, head_dim);
}

hipError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t T, int64_t hq, int64_t head_dim,
                                int64_t max_q, int64_t max_ctx, int64_t window, float scale, const void* cache,
                                const Kv4View& c, uint16_t* out, float* lse, void* workspace, hipStream_t stream) {
  const Plan pl = make_plan(T, c.B, hq, c.kv_heads, max_q, max_ctx, window);
  const KvCache a = kv4_cache_args(c, T, head_dim);
  AttnArgs p = {};
  p.q = reinterpret_cast<const f16*>(q);
  p.q_stride = q_stride;
  p.cache = static_cast<const uint8_t*>(cache);
  p.out = reinterpret_cast<f16*>(out);
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  const int64_t slots = decode_slots(pl, c.kv_heads), tslots = pl.tslots * pl.tnsplit;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_s = reinterpret_cast<float2*>(ws + (size_t)slots * head_dim * 4);
  ws += part_bytes(slots, head_dim);
  p.tpart_o = reinterpret_cast<float*>(ws);
  p.tpart_s = reinterpret_cast<float2*>(ws + (size_t)tslots * head_dim * 4);
  p.hq = (int)hq;
  p.group = (int)(hq / c.kv_heads);
  p.window = (int)window;
  p.c = scale * 1.44269504088896341f;
  p.shares = (int)pl.shares;
  p.least = (int)kLeastTiles;
  p.decode_rows = pl.decode_rows;
  p.tnsplit = pl.tnsplit;
  p.tchunk_tiles = pl.tchunk;
  p.row_limit = pl.row_limit;
  return head_dim == 128 ? run<128>(a, p, pl, c.B, c.kv_heads, stream) : run<64>(a, p, pl, c.B, c.kv_heads, stream);
}

}  // namespace wq
