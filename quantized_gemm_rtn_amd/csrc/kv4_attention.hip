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
// scales, 2^(x - r) u, are near 2^12.8 at the row's largest and at most 2^15.9, so that a
// token of the smallest scale keeps its bits beside one of the largest (2^27 apart). It
// only moves (and everything summed so far is only rescaled) when a lane's top score and
// log2 of its largest value scale pass that bound together, which any lane can see without
// asking the others. These may be two tokens', and their sum up to 27 more than any one
// has; so where r moves to is found token by token, score plus log2 of its own scale, of
// which the lane's sum may take it no further than kMixed. (With the sums alone operands
// were subnormal where tokens of unlike scales stood side by side, and lost their last bits.)
// Where r itself is so large that float32 does not hold such fractions of it, it is the
// largest score (see far_reference; scores of 1e8 gave infinite weights).
//
//  kv4_decode_kernel   few query rows (16 or 32 a block): all tiles of all sequences are
//    dealt out in equal shares, one a block, whose four waves take tiles of 32 tokens in
//    turn and join through LDS at each row tile's end. Bound by the cache's bytes, which
//    it reads once, through an LDS ring (loads that bypass registers: 127 us without, for
//    the first of these): 64 sequences of 7100 tokens, 8 heads of 128 99 us (5.0 TB/s); 16
//    of 2000, 32 heads 30-35 us (4-4.5 TB/s); one of 131 071, 8 heads 31 us (4.6 TB/s). A
//    wave's loop runs at 6.7 TB/s; beginning (lengths, page numbers, first tiles, each
//    waiting for the one before) and joining take the rest, and a short call all of it:
//    one sequence of 1000 tokens, 32 heads, 7.4 us.
//  kv4_tile_kernel     many query rows: 128 a block; a tile of codes is turned into
//    exact fp16 integers once, in LDS, for all of them (see there).
//  kv4_combine_kernel  joins the parts of rows that more than one block worked on. Bound
//    by latency: 4.3 us for 32 rows of 4 parts, 7.7 us for 4096 rows, most of two.
#include "kv4_attention.h"
#include "wq_launch.h"

namespace wq {

// The decode kernel's work: its items are a sequence's row tiles, in order, each as many
// steps as the sequence has visible tiles (one where it has none: its rows are still to
// be written). All steps of a head are dealt out in equal shares, one a block, so that
// blocks end together however the sequences' lengths differ; an item that lies in one
// share is finished there, others leave a partial in each. Where there is less work than
// blocks for it (p.pad), items count as a multiple of the fewest steps of a share, the
// last of them empty, so that a share has one item: two are done one after the other, and
// the latency of a block is what such a call takes (8 sequences of 3 to 5 drafted tokens,
// window 1000, in 4 heads: 13.1 us without, 8.8 us with). A wave looks at 64 sequences at
// a time, one a lane.
struct Sequences {
  KvSeq s;
  int t0, tiles;  // first visible tile, tiles of an item
  int n;          // steps of an item (0: nothing to do here)
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
  q.tiles = max(r.t1 - r.t0, 1);
  q.n = mine ? (p.pad ? (q.tiles + p.least - 1) & -p.least : q.tiles) : 0;
  q.steps = (int64_t)q.n * ((rows + p.decode_rows - 1) / p.decode_rows);
  q.upto = wave_sums_upto(q.steps, lane);
  return q;
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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kDepth = 2;  // tiles of a wave's ring: one in use, one on its way (stages 0 and 1)

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
    const int last = t0 + __builtin_amdgcn_readlane(seqs.tiles, j);
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
    int pos[NT], passed[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + kDecodeRows * n + c;
      const bool valid = row < rows;
      const int tok = valid ? row / p.group : 0;
      const int head = h * p.group + (valid ? row - tok * p.group : 0);
      pos[n] = valid ? s.ctx - s.rows + tok : -1;
      passed[n] = last_passed(p, pos[n]);
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

    const int begin = t0 + from, end = s.ctx > 0 ? min(begin + count, last) : begin;
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
    bool far = false;  // a row's scores are (see far_reference), the same for the wave
    int fetched = tile, stage_in = 0, stage = 0;
    const auto fetch_next = [&]() {
      if (fetched < end) fetch(stage_in);
      fetched += 4;
      stage_in ^= 1;
    };
    fetch_next();
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
      // this tile's loads are done when only the next one's are left
      if (tile + 4 < end)
        wait_vm<LOADS>();
      else
        wait_vm<0>();
      const uint32_t at = ring_at + stage * TILE;
      stage ^= 1;
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
          const uint32_t word = cur.k[(KW * half + w) >> 2][(KW * half + w) & 3];
          const f16x8 k = as_f16x8(codes_minus_zero_x16(word, magic, kz.bias[half], kz.nbias16[half]));
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[n] = mfma_16x16x32(k, qf[n][w], sc[n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[n][i + 4 * half] = mul_mix(sc[n][i], ks[i + 4 * half]);
      }

      const int first = tile * kKvTile;
      const bool edge = first + kKvTile - 1 > p0 || (p.window > 0 && p1 - first >= p.window);
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
            const bool see = t <= pos[n] && t > passed[n];
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
      const float ve = log2_bits(vmax);
      bool move = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mx[n] = x[n][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx[n] = fmaxf(mx[n], x[n][e]);
        mx[n] = __builtin_fmaf(mx[n], p.c, ve);
        move |= mx[n] - kTop > ref[n] + kSlack;
      }
      float factor = p.c;
      if (__any(move) || far) {
        float to[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float m = mx[n];
          m = fmaxf(m, __shfl_xor(m, 16));
          m = fmaxf(m, __shfl_xor(m, 32));
          float one = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) one = fmaxf(one, __builtin_fmaf(x[n][e], p.c, about_log2(vs[e])));
          one = fmaxf(one, __shfl_xor(one, 16));
          one = fmaxf(one, __shfl_xor(one, 32));
          to[n] = moved_reference(ref[n], m, one);
          far |= is_far(to[n]);
        }
        if (__any(far)) {
          factor = 1.0f;
          far = false;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, x[n][e] *= p.c);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            to[n] = far_reference(ref[n], to[n], top);
            far |= is_far(to[n]);
          }
          far = __any(far);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f = exp2_hw(ref[n] - to[n]);
          ref[n] = to[n];
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
          const float w = exp2_hw(__builtin_fmaf(x[n][e], factor, -ref[n]));
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
          const float inv = inverse_sum(total_sum);
          f16* dst = p.out + at_row * D + CT * part;
#pragma unroll
          for (int i = 0; i < CT; i += 4) {
            typedef f16 f16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<f16x4*>(dst + i) =
                f16x4{(f16)(o[i] * inv), (f16)(o[i + 1] * inv), (f16)(o[i + 2] * inv), (f16)(o[i + 3] * inv)};
          }
          if (part == 0 && p.lse != nullptr)
            p.lse[at_row] = log_sum(best, total_sum);
        }
      }
    }
    __syncthreads();
    opening = false;
  }
}

// Joins the decode kernel's partials of rows that were split. W waves per row (1, 4 or
// 16, so that a wave takes about eight); rows that are already written are left alone.
// by_sequence: the rows looked at are the first row_limit of each sequence and head, not
// all of the output.
template <int D, int W>
__global__ void __launch_bounds__(W < 4 ? 256 : 64 * W)
kv4_combine_kernel(KvCache a, AttnArgs p, int by_sequence) {
  constexpr int ROWS = W < 4 ? 4 / W : 1;  // rows of a block
  constexpr int N = D / 64;                // channels of a lane
  __shared__ float joined[W][D + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t item = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + (W == 1 ? wave : 0);
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
  if (rows > p.row_limit) return;
  const int64_t out_row = (int64_t)(s.first_row + row / p.group) * p.hq + h * p.group + row % p.group;

  // the row's partials: those of shares i0 .. i1 of its head. Share i is block i * hkv + h,
  // with two partials: an item that begins inside the share comes second.
  Sequences q = load_sequences(a, p, 0, lane);
  const int64_t per = share_steps(p, total_steps(a, p, q, lane));
  int64_t before = 0;
  for (int first = 64; first <= b; first += 64) {
    before += lane_value(q.upto, 63);
    q = load_sequences(a, p, first, lane);
  }
  const int n = __builtin_amdgcn_readlane(q.n, b & 63);
  const int64_t X = before + lane_value(q.upto - q.steps, b & 63) + (int64_t)(row / p.decode_rows) * n;
  const int64_t i0 = X / per;
  const int parts = (int)((X + n - 1) / per - i0) + 1;
  if (parts <= 1) return;
  const auto place = [&](int i) {
    return (((i0 + i) * a.hkv + h) * 2 + (i == 0 && X > i0 * per ? 1 : 0)) * p.decode_rows + row % p.decode_rows;
  };
  // The wave's first partials are on their way while every wave finds the row's reference
  // and sum, a partial a lane.
  constexpr int AHEAD = 8;
  float ahead[AHEAD][N], ahead_r[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = (W == 1 ? 0 : wave) + W * k;
    if (i < parts) {
      const int64_t at = place(i);
      ahead_r[k] = p.part_s[at].x;
#pragma unroll
      for (int e = 0; e < N; ++e) ahead[k][e] = p.part_o[at * D + N * lane + e];
    }
  }
  float best = kNoRef, total = 0.0f;
  for (int i = lane; i < parts; i += 64) best = fmaxf(best, p.part_s[place(i)].x);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) best = fmaxf(best, __shfl_xor(best, off));
  for (int i = lane; i < parts; i += 64) {
    const float2 v = p.part_s[place(i)];
    total = __builtin_fmaf(v.y, exp2_hw(v.x - best), total);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
  float o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.0f;
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if ((W == 1 ? 0 : wave) + W * k < parts) {
      const float f = exp2_hw(ahead_r[k] - best);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = __builtin_fmaf(ahead[k][e], f, o[e]);
    }
#pragma unroll 8
  for (int i = (W == 1 ? 0 : wave) + W * AHEAD; i < parts; i += W) {
    const int64_t at = place(i);
    const float f = exp2_hw(p.part_s[at].x - best);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = __builtin_fmaf(p.part_o[at * D + N * lane + e], f, o[e]);
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
  const float inv = inverse_sum(total);
  f16* dst = p.out + out_row * D + N * lane;
#pragma unroll
  for (int e = 0; e < N; ++e) dst[e] = (f16)(o[e] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[out_row] = log_sum(best, total);
}

namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kDecodeBlocks = 2;  // blocks a CU (three fit; measured slower by 2 %: more, shorter shares)
constexpr int64_t kLeastTiles = 8;    // of a share: two a wave (a power of two)

struct Plan {
  bool decode, tile;  // which kernels run
  int decode_rows, row_limit;
  int64_t shares, most_shares;  // decode kernel: blocks a head, and their bound
  int pad;            // whether each has one item
  int64_t parts;      // shares of an item, about
  int64_t tshares, most_tshares;  // tile kernel: the same (0: whole row tiles), and its bound
  int row_tiles, snake;
};

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

Plan make_plan(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q, int64_t max_ctx,
               int64_t window) {
  Plan p = {};
  const int64_t group = hq / hkv;
  const int64_t q = max_q < 1 ? 1 : (max_q > T ? T : max_q);
  const int64_t rows = q * group;
  // Rows of a sequence and head up to which the decode kernel (32 rows an item, the cache
  // read once for each) beats the tile kernel (128 rows, whether there or not): with 64
  // rows 32 against 47 us (8 sequences of 4000 tokens, 4 heads), 25 against 51 us (one of
  // 20000); with 96 38 and 41, 34 and 69 us; with 128 rows it is 43 and 53 there, but 129
  // and 111 us for 32 sequences of 4000 tokens and 8 heads.
  constexpr int64_t kLimit = 96;
  // a sequence's rows decide its kernel; from the host only the largest is known, and
  // that all are alike where there is one sequence or B max_q new tokens
  const bool many = rows > kLimit, mixed = B > 1 && B * q > T;
  p.decode_rows = many || rows > kDecodeRows ? 2 * kDecodeRows : kDecodeRows;
  int64_t tiles = ceil_div(max_ctx < 1 ? 1 : max_ctx, kKvTile);
  if (window > 0) {  // q rows see up to window + q - 1 tokens, which may begin inside a tile
    const int64_t in_window = ceil_div(window + q - 1, kKvTile) + 1;
    tiles = in_window < tiles ? in_window : tiles;
  }
  // The decode kernel, for sequences of up to `most_rows` rows: as many blocks as run well
  // at once, each with an equal share; one a head where the heads alone are as many
  const auto deal = [&](int64_t most_rows, int& pad) {
    constexpr int64_t resident = kCus * kDecodeBlocks;
    const int64_t items = B * ceil_div(most_rows, p.decode_rows);
    const int64_t most = ceil_div(items * tiles, kLeastTiles), padded = items * ceil_div(tiles, kLeastTiles);
    pad = padded <= resident / hkv;
    const int64_t shares = pad ? padded : (resident / hkv < most ? resident / hkv : most);
    return shares < 1 ? (int64_t)1 : shares;
  };
  int pad_few = 0, pad_all = 0;
  const int64_t few = deal(many ? kLimit : rows, pad_few), all = deal(rows, pad_all);
  p.most_shares = few > all ? few : all;
  if (many) {
    // Whole row tiles, or equal shares of them: shares keep every CU busy to the end, but
    // cost partials (written, read and joined, some 50 000 cycles in all). In cycles, with
    // 5400 measured for two blocks' steps of 64 tokens on a CU and 4200 for one alone, from
    // bounds: all rows at most, each sequence as long as the longest.
    const int64_t per_seq = ceil_div(rows, kTileRows), by_rows = ceil_div(T * group, kTileRows) + B;
    const int64_t blocks = hkv * (B * per_seq < by_rows ? B * per_seq : by_rows);
    const double longest = (double)ceil_div(tiles, 2);
    const double mean = window > 0 ? longest : (longest > (double)q / 128 ? longest - (double)q / 128 : longest / 2);
    const double shared = blocks * mean / (2 * kCus) * 5400 + 50000;
    double whole = blocks * mean / (2 * kCus) * 5400 + longest * 2100;
    if (blocks <= 2 * kCus) whole = longest * 4200 > mean * 5400 ? longest * 4200 : mean * 5400;
    if (blocks <= kCus) whole = longest * 4200;
    const int64_t most = ceil_div(T * group * tiles, (int64_t)kLeastItemTiles * kTileRows) + 1;
    const int64_t most_blocks = 0xFFFFFF / (B * hkv);  // B hkv < 2^24, and so is the grid
    const int64_t fit = 2 * kCus / hkv < 1 ? 1 : 2 * kCus / hkv;
    p.tshares = fit < most ? fit : most;
    p.most_tshares = p.tshares;
    if (whole <= shared) {
      p.tshares = 0;
      p.row_tiles = (int)(per_seq < most_blocks ? per_seq : most_blocks);
      p.snake = B * hkv * per_seq <= 2 * kCus;
    }
    // Where few rows see long sequences, the decode kernel is faster all the same, and it
    // saves the pair of launches that a mixed batch takes. Whole calls of either, in us,
    // fitted to both kernels' times in 1400 batches of 97 to 2000 rows a sequence (1 to 64
    // sequences of up to 30 000 tokens, 1 to 32 heads, groups of 1 to 32, even and uneven,
    // with and without windows). In 700 others (to 256 sequences) the kernel it takes was
    // slower than the faster one by 1.1 % on average and 1.6 times at worst (21 and 13 us);
    // the tile kernel always by 15 % and 3.1 times, the decode kernel 67 % and 9 times. For
    // instance (decode, tile): 33 tokens after 4900, 4 heads on 1, 14 and 42; 52 after 6800,
    // 64 on 8, 43 and 58; 8 after 4000, 43 sequences, 16 heads of 64 on 1, 34 and 43; 17
    // after 1200, 16 sequences, 64 on 8, 60 and 48; up to 163, 4 sequences, 32 heads of 64
    // on 4, 31 and 22.
    const int64_t dec_seq = ceil_div(rows, p.decode_rows), dec_rows = ceil_div(T * group, p.decode_rows) + B;
    const double items = (double)hkv * (double)(B * dec_seq < dec_rows ? B * dec_seq : dec_rows);
    const double half = 0.5 + head_dim / 256.0;  // 64 channels take three quarters of 128's time
    const double by_decode = 11 + half * 0.18 * items * tiles / kCus + 4 * items / (2 * kCus) +
                             0.85e-3 * (head_dim / 128.0) * (double)(T * hq);
    const double by_tile = 7 + half * 0.38e-3 * (whole < shared ? whole : shared) + 5.0 * blocks / (2 * kCus) +
                           (whole <= shared ? 0 : 5) + (mixed ? 6.5 : 0);
    p.tile = by_tile <= by_decode;
  }
  p.decode = !p.tile || mixed;
  p.row_limit = p.tile ? (p.decode ? (int)kLimit : 0) : 0x7FFFFFFF;
  p.shares = !p.decode ? 1 : (p.tile ? few : all);
  p.pad = p.tile ? pad_few : pad_all;
  p.parts = p.shares / (B * ceil_div(p.tile ? kLimit : rows, p.decode_rows)) + 1;
  return p;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
// rows of partials, each with D sums, its reference and its sum
int64_t decode_slots(const Plan& pl, int64_t hkv, int64_t shares) {
  return shares > 1 ? hkv * shares * 2 * pl.decode_rows : 0;
}
int64_t tile_slots(const Plan& pl, int64_t hkv, int64_t shares) {
  return shares > 1 ? hkv * shares * 2 * kTileRows : 0;
}
size_t part_bytes(int64_t slots, int64_t D) { return round256((size_t)slots * (D * 4 + 8)); }

// waves that join a row of `parts` partials, about: eight each
int join_waves(int64_t parts) { return parts <= 8 ? 1 : (parts <= 32 ? 4 : 16); }

// items: rows to look at; parts: those of a row, about
template <int D>
hipError_t combine(const KvCache& a, const AttnArgs& p, int64_t parts, int64_t items, int by_sequence,
                   hipStream_t stream) {
  // blocks in two dimensions: one holds 2^32 threads
  const auto grid = [](int64_t blocks) {
    constexpr int64_t x = 1 << 20;
    return dim3((unsigned)(blocks < x ? blocks : x), (unsigned)ceil_div(blocks, x));
  };
  if (join_waves(parts) == 1)
    hipLaunchKernelGGL((kv4_combine_kernel<D, 1>), grid(ceil_div(items, 4)), dim3(256), 0, stream, a, p, by_sequence);
  else if (join_waves(parts) == 4)
    hipLaunchKernelGGL((kv4_combine_kernel<D, 4>), grid(items), dim3(256), 0, stream, a, p, by_sequence);
  else
    hipLaunchKernelGGL((kv4_combine_kernel<D, 16>), grid(items), dim3(1024), 0, stream, a, p, by_sequence);
  return hipGetLastError();
}

template <int D>
hipError_t run(const KvCache& a, const AttnArgs& p, const Plan& pl, int64_t B, int64_t hkv, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (pl.tile) e = launch_kv4_tile(a, p, D, stream);
  if (e == hipSuccess && pl.decode) {
    const dim3 grid((unsigned)(hkv * pl.shares));
    if (pl.decode_rows == kDecodeRows)
      hipLaunchKernelGGL((kv4_decode_kernel<D, 1>), grid, dim3(256), 0, stream, a, p);
    else
      hipLaunchKernelGGL((kv4_decode_kernel<D, 2>), grid, dim3(256), 0, stream, a, p);
    e = hipGetLastError();
  }
  if (e == hipSuccess && pl.decode && pl.shares > 1)
    e = combine<D>(a, p, pl.parts, pl.tile ? B * hkv * p.row_limit : (int64_t)a.T * p.hq, pl.tile, stream);
  return e;
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q,
                                     int64_t max_ctx) {
  const Plan pl = make_plan(T, B, hq, hkv, head_dim, max_q, max_ctx, 0);
  // whichever kernels run: a shorter batch may take others than the longest
  return part_bytes(decode_slots(pl, hkv, pl.most_shares), head_dim) + part_bytes(tile_slots(pl, hkv, pl.most_tshares), head_dim);
}

int kv4_attention_plan(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q, int64_t max_ctx,
                       int64_t window) {
  const Plan pl = make_plan(T, B, hq, hkv, head_dim, max_q, max_ctx, window);
  return (pl.decode ? 1 : 0) | (pl.tile ? 2 : 0) | (pl.tile && pl.tshares > 0 ? 4 : 0) |
         (pl.decode && pl.shares > 1 ? join_waves(pl.parts) << 8 : 0);
}

hipError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t T, int64_t hq, int64_t head_dim,
                                int64_t max_q, int64_t max_ctx, int64_t window, float scale, const void* cache,
                                const Kv4View& c, uint16_t* out, float* lse, void* workspace, hipStream_t stream) {
  // a window of all tokens that the pages hold hides none
  if (window >= c.max_pages * c.page_tokens) window = 0;
  const Plan pl = make_plan(T, c.B, hq, c.kv_heads, head_dim, max_q, max_ctx, window);
  const KvCache a = kv4_cache_args(c, T, head_dim);
  AttnArgs p = {};
  p.q = reinterpret_cast<const f16*>(q);
  p.q_stride = q_stride;
  p.cache = static_cast<const uint8_t*>(cache);
  p.out = reinterpret_cast<f16*>(out);
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  const int64_t slots = decode_slots(pl, c.kv_heads, pl.shares);
  const int64_t tslots = pl.tile ? tile_slots(pl, c.kv_heads, pl.tshares) : 0;
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
  p.pad = pl.pad;
  p.decode_rows = pl.decode_rows;
  p.tshares = (int)pl.tshares;
  p.row_tiles = pl.row_tiles;
  p.snake = pl.snake;
  p.row_limit = pl.row_limit;
  return head_dim == 128 ? run<128>(a, p, pl, c.B, c.kv_heads, stream) : run<64>(a, p, pl, c.B, c.kv_heads, stream);
}

}  // namespace wq
