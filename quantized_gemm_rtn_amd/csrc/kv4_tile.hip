// Causal attention over the 4-bit cache for many query rows, for gfx950: the tile kernel
// (kv4_attention.hip has the mathematics, the kernel for few rows, and the choice).
//
// A block has 128 rows of one key/value head, four waves 32 each, and takes 64 tokens a
// step: two barriers, between which the waves unpack a quarter of the step's codes each
// into LDS as the products' operands, and after which every wave reads all of them, once
// for each of its two products (keys . queries^T, values^T . weights^T, 32x32x16). Queries,
// scores, weights and sums stay in registers: 252 of the 256 that two blocks a CU have, which
// the build checks (with 258 a prompt of 2048 took 96 us instead of 63; the same bound given
// to the compiler changes its schedule, 75 us). The codes of the next step are on their way
// meanwhile.
//
// Measured: 1357 tokens in chunks of 700, 535 and 122 after up to 6000, 32 heads on 8: 126
// GFLOP in 185-195 us (0.66 PFLOP/s); a prompt of 2048 67 us, nearly all of it its last rows'
// 32 steps, alone on their CUs. Two blocks' steps take 5400 cycles a CU: matrix units are
// busy for 2048 of them, vector units for 2800, and LDS for 2500 (32 rows a wave need 1 KB
// of operands a matrix instruction, its full rate at the matrix units' own). None fills the
// step because each block's phases follow on one another and only two blocks overlap. Tried
// and slower: 64 rows a wave (spills); three blocks a CU with 32 tokens at a time; eight
// waves that halve the tokens; the next step's scores made while this one's weights are;
// one barrier a step.
#include "kv4_attention.h"

namespace wq {

template <int D>
__global__ void __launch_bounds__(256)
kv4_tile_kernel(KvCache a, AttnArgs p) {
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
  const int h = blockIdx.x % a.hkv, share = blockIdx.x / a.hkv;
  const int sub = wave >> 1;   // of the two tiles of a step, the one that the wave unpacks,
  const bool is_v = wave & 1;  // and which half of it
  const int g = lane >> 4, c16 = lane & 15;
  const uint32_t magic = magic_1024x2();

  // Either an equal share of the work of all rows, or (no shares) whole row tiles of one
  // sequence. Their last rows see the most tokens and start first; where all blocks fit
  // the card at once, two a CU (the second 256 next to the first), the later half goes
  // the other way, and a CU's two blocks make the same sum of work.
  AreaWalk walk;
  AreaItem item;
  int64_t per = 0, from = 0, until = 1, total = 0;
  int turn = 0;
  if (p.tshares > 0) {
    total = area_begin(walk, a, p, lane);
    per = share_area(p, total);
    from = share * per;
    until = from + per < total ? from + per : total;
    if (from >= until) return;
    if (!area_find(item, walk, a, p, from, lane)) return;
  } else {
    item.b = share / p.row_tiles;
    item.s = kv_sequence(a, item.b);
    item.have = (int)items_of(item.s, p);
    turn = share % p.row_tiles;
    if (item.s.rows * p.group <= p.row_limit || turn >= item.have) return;
    item.rt = row_tile_of(turn, item.have, p.snake);
    item.X = 0;
    item.next = 1;
  }
  for (int64_t at = from; at < until;) {
    const KvSeq s = item.s;
    const int b = item.b, rows = s.rows * p.group;
    const int row0 = item.rt * kTileRows, row1 = min(rows, row0 + kTileRows) - 1;
    const int64_t X = item.X, next = item.next;
    const TileRange range = tile_range(s, p, row0, row1);
    const int tiles = range.t1 - range.t0;
    const int begin = range.t0 + tiles_before(from, X, next - X, tiles);
    const int end = range.t0 + tiles_before(until, X, next - X, tiles);
    // an item that lies in the share is finished here (one with no tiles where it begins)
    const bool whole = tiles > 0 ? end - begin == tiles : X >= from;
    const bool opening = X <= from;  // its partial goes to slot 0, a later item's to slot 1
    at = next;
    // the next item: the sequence's next row tile, or another sequence's first
    if (p.tshares == 0) {
      turn += p.row_tiles;
      at = turn < item.have ? 0 : 1;
      item.rt = row_tile_of(min(turn, item.have - 1), item.have, p.snake);
    } else if (at < until) {
      if (item.rt + 1 < item.have) {
        ++item.rt;
        item.X = next;
        item.next = area_before(item, p, item.rt + 1);
      } else if (!area_find(item, walk, a, p, at, lane)) {
        return;
      }
    }
    if (begin == end && !whole) continue;
    const int p0 = s.ctx - s.rows + row0 / p.group, p1 = s.ctx - s.rows + row1 / p.group;
    const int row = row0 + 32 * wave + c;
    const bool valid = row < rows;
    const int tok = valid ? row / p.group : 0;
    const int head = h * p.group + (valid ? row - tok * p.group : 0);
    const int pos = valid ? s.ctx - s.rows + tok : -1, passed = last_passed(p, pos);
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
    float ref = kNoRef, sum = 0.0f;
    bool far = false;  // a row's scores are (see far_reference), the same for the wave

    // each wave turns one tile's keys or values into LDS operands: waves 0, 1 the first
    // tile's of a step, waves 2, 3 the second's. Page numbers come through the scalar
    // cache, a step ahead.
    const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.page_table + (int64_t)b * a.max_pages);
    uint4 data[RUNS], scales, zeros;
    int loading = max(min(begin + sub, end - 1), 0);
    int page = loading / a.page_tiles, in_page = loading - page * a.page_tiles;
    int id = begin < end ? table[page] : 0;
    const auto load = [&]() {
      const uint8_t* base = p.cache + kv_page_offset(a, h, id) + (int64_t)in_page * kv_tile_bytes<D>();
      const int off = is_v ? kv_value_offset<D>() : kv_key_offset<D>();
#pragma unroll
      for (int i = 0; i < RUNS; ++i) data[i] = *reinterpret_cast<const uint4*>(base + off + 1024 * i + 16 * lane);
      const uint8_t* meta = base + kv_meta_offset<D>(is_v ? 2 : 0);
      scales = *reinterpret_cast<const uint4*>(meta + 16 * (lane & 3));
      if (is_v)
        zeros = *reinterpret_cast<const uint4*>(meta + 64 + 16 * g);
      else
        zeros.x = *reinterpret_cast<const uint32_t*>(meta + 64 + 4 * c16);
      // the next step's (past the range the last tile again, masked by position)
      const bool more = loading + 2 < end;
      loading += more ? 2 : 0;
      in_page += more ? 2 : 0;
      while (in_page >= a.page_tiles) {
        in_page -= a.page_tiles;
        ++page;
      }
      id = table[page];
    };
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

    if (begin < end) load();
    for (int tile = begin; tile < end; tile += 2) {
      __syncthreads();  // the previous tiles have been read
      stash();
      __syncthreads();
      if (tile + 2 < end) load();

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
      const bool edge = first + 2 * kKvTile - 1 > p0 || (p.window > 0 && p1 - first >= p.window) || tile + 1 >= end;
      if (edge) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int t = first + 32 * u + 8 * (e >> 2) + 4 * hl + (e & 3);
            const bool see = t <= pos && t > passed && tile + u < end;
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
      mx = __builtin_fmaf(mx, p.c, log2_bits(vmax));
      float factor = p.c;
      if (__any(mx - kTop > ref + kSlack) || far) {
        float one = mx;
        const uint32_t vmin = min(min(min_bits8(vs[0][0]), min_bits8(vs[0][1])),
                                  min(min_bits8(vs[1][0]), min_bits8(vs[1][1])));
        if (__any(vmax - vmin > kAlike)) {
          one = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                one = fmaxf(one, __builtin_fmaf(sc[u][4 * (q + 2 * (e >> 2)) + (e & 3)], p.c, about_log2(vs[u][q][e])));
        }
        one = fmaxf(one, __shfl_xor(one, 32));
        float to = moved_reference(ref, fmaxf(mx, __shfl_xor(mx, 32)), one);
        if (__any(is_far(to)) || far) {
          factor = 1.0f;
          float top = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[u][e] *= p.c);
          to = far_reference(ref, to, fmaxf(top, __shfl_xor(top, 32)));
          far = __any(is_far(to));
        }
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
            const float w = exp2_hw(__builtin_fmaf(sc[u][4 * (q + 2 * (e >> 2)) + (e & 3)], factor, -ref));
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
      if (!whole) {
        const int64_t place = ((int64_t)blockIdx.x * 2 + (opening ? 0 : 1)) * kTileRows + 32 * wave + c;
        float* dst = p.tpart_o + place * D + 4 * hl;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(dst + 32 * t + 8 * q) =
                f32x4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
        if (hl == 0) p.tpart_s[place] = make_float2(ref, sum);
      } else {
        const float inv = inverse_sum(sum);
        f16* dst = p.out + slot * D + 4 * hl;
        typedef f16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f16x4*>(dst + 32 * t + 8 * q) =
                f16x4{(f16)(acc[t][4 * q] * inv), (f16)(acc[t][4 * q + 1] * inv), (f16)(acc[t][4 * q + 2] * inv),
                      (f16)(acc[t][4 * q + 3] * inv)};
        if (hl == 0 && p.lse != nullptr) p.lse[slot] = log_sum(ref, sum);
      }
    }
  }
}

// Joins the partials of the items that more than one share worked on: block (head, share
// i, slice of the rows) those of the item that share i begins but does not end. 16 lanes
// take a row, D / 16 channels each, a wave 4 PASSES rows, AHEAD partials at a time. With
// few partials of a row (PW = 1) a wave takes all of them, with many (PW = 4) the block's
// four waves take them in turn and join theirs through LDS. Which shares have tiles of the
// item the lanes find out for 64 of them at once (a quotient in double each). Bound by the
// partials' bytes where there are many rows (67 MB written and read for 1357 tokens of 32
// heads: 16 us), else by latency: one row tile of 59 000 tokens in 85 shares takes 24 us,
// and took 110 us with a wave for all of a row's partials.
template <int D, int PW, int PASSES, int AHEAD>
__global__ void __launch_bounds__(256)
kv4_tile_combine_kernel(KvCache a, AttnArgs p) {
  constexpr int N = D / 64;  // runs of four channels of a lane
  constexpr int ROWS = 4 * PASSES * (4 / PW);  // rows of the block
  __shared__ f32x4 o_s[PW][PW > 1 ? ROWS : 1][D / 4];
  __shared__ float2 s_s[PW][ROWS];
  const int lane = threadIdx.x & 63, part = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.hkv, share = blockIdx.x / a.hkv;
  // one wave looks for the share's last item (every block does: with four it took 6 us of
  // the kernel for each 2048 blocks); it must begin in this share and go on in the next
  __shared__ AreaItem item_s;
  __shared__ int64_t per_s;
  __shared__ int split_s;
  if (wave == 0) {
    AreaWalk walk;
    AreaItem t;
    const int64_t total = area_begin(walk, a, p, lane), per = share_area(p, total);
    const int64_t from = share * per, until = from + per;
    const bool split = until < total && area_find(t, walk, a, p, until - 1, lane) && t.X >= from && t.next > until;
    if (lane == 0) {
      if (split) item_s = t;
      per_s = per;
      split_s = split;
    }
  }
  __syncthreads();
  if (!split_s) return;
  const AreaItem t = item_s;
  const int64_t per = per_s, from = share * per;
  const int rows = t.s.rows * p.group, row0 = t.rt * kTileRows, row1 = min(rows, row0 + kTileRows) - 1;
  const int slice = ROWS * blockIdx.y, in = (PW == 1 ? 4 * PASSES * wave : 0) + (lane >> 4);
  if (row0 + slice > row1) return;
  const TileRange range = tile_range(t.s, p, row0, row1);
  const int n = range.t1 - range.t0;
  const int64_t W = t.next - t.X;
  const int parts = (int)((t.next - from + per - 1) / per);  // shares of the item
  float best[PASSES], sum[PASSES];
  f32x4 o[PASSES][N];
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    best[k] = kNoRef;
    sum[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) o[k][j] = f32x4{};
  }
  for (int i0 = 0; i0 < parts; i0 += 64) {
    const int64_t x = from + min(i0 + lane, parts - 1) * per;
    const int had = tiles_before(x + per, t.X, W, n) - tiles_before(x, t.X, W, n);
    if (__any(had == n)) return;  // a share that had all wrote the rows
    uint64_t mine = __ballot(i0 + lane < parts && had > 0) & (PW == 1 ? ~0ull : 0x1111111111111111ull << wave);
    while (mine != 0) {
      bool has[AHEAD];
      float2 v[AHEAD][PASSES];
      f32x4 d[AHEAD][PASSES][N];
#pragma unroll
      for (int g = 0; g < AHEAD; ++g) {
        has[g] = mine != 0;
        if (!has[g]) continue;
        const int i = i0 + __builtin_ctzll(mine);
        mine &= mine - 1;
        const int64_t first = (((int64_t)(share + i) * a.hkv + h) * 2 + (i == 0 && t.X > from ? 1 : 0)) * kTileRows;
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
          const int64_t at = first + min(slice + in + 4 * k, row1 - row0);
          v[g][k] = p.tpart_s[at];
#pragma unroll
          for (int j = 0; j < N; ++j)
            d[g][k][j] = *reinterpret_cast<const f32x4*>(p.tpart_o + at * D + 64 * j + 4 * part);
        }
      }
#pragma unroll
      for (int g = 0; g < AHEAD; ++g) {
        if (!has[g]) continue;
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
          const float to = fmaxf(best[k], v[g][k].x), keep = exp2_hw(best[k] - to), f = exp2_hw(v[g][k].x - to);
          best[k] = to;
          sum[k] = sum[k] * keep + v[g][k].y * f;
#pragma unroll
          for (int j = 0; j < N; ++j) o[k][j] = o[k][j] * keep + d[g][k][j] * f;
        }
      }
    }
  }
  const auto store = [&](int row, float top, float all, const f32x4(&v)[N]) {
    if (row > row1) return;
    const int tok = row / p.group;
    const int64_t out_row = (int64_t)(t.s.first_row + tok) * p.hq + h * p.group + (row - tok * p.group);
    const float inv = inverse_sum(all);
    typedef f16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int j = 0; j < N; ++j)
      *reinterpret_cast<f16x4*>(p.out + out_row * D + 64 * j + 4 * part) =
          f16x4{(f16)(v[j][0] * inv), (f16)(v[j][1] * inv), (f16)(v[j][2] * inv), (f16)(v[j][3] * inv)};
    if (part == 0 && p.lse != nullptr) p.lse[out_row] = log_sum(top, all);
  };
  if constexpr (PW == 1) {
#pragma unroll
    for (int k = 0; k < PASSES; ++k) store(row0 + slice + in + 4 * k, best[k], sum[k], o[k]);
  } else {
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      if (part == 0) s_s[wave][in + 4 * k] = make_float2(best[k], sum[k]);
#pragma unroll
      for (int j = 0; j < N; ++j) o_s[wave][in + 4 * k][16 * j + part] = o[k][j];
    }
    __syncthreads();
    const int r = threadIdx.x >> 4;
    if (r >= ROWS) return;
    float top = s_s[0][r].x, all = 0.0f;
#pragma unroll
    for (int w = 1; w < PW; ++w) top = fmaxf(top, s_s[w][r].x);
    f32x4 v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = f32x4{};
#pragma unroll
    for (int w = 0; w < PW; ++w) {
      const float f = exp2_hw(s_s[w][r].x - top);
      all += s_s[w][r].y * f;
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += o_s[w][r][16 * j + part] * f;
    }
    store(row0 + slice + r, top, all, v);
  }
}

template <int D>
hipError_t join(const KvCache& a, const AttnArgs& p, unsigned blocks, bool many, hipStream_t stream) {
  if (many)
    hipLaunchKernelGGL((kv4_tile_combine_kernel<D, 4, 2, 2>), dim3(blocks, kTileRows / 8), dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((kv4_tile_combine_kernel<D, 1, 2, 2>), dim3(blocks, kTileRows / 32), dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

hipError_t launch_kv4_tile(const KvCache& a, const AttnArgs& p, int64_t head_dim, hipStream_t stream) {
  const dim3 grid((unsigned)(p.tshares > 0 ? (int64_t)a.hkv * p.tshares : (int64_t)a.hkv * a.B * p.row_tiles));
  if (head_dim == 128)
    hipLaunchKernelGGL((kv4_tile_kernel<128>), grid, dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((kv4_tile_kernel<64>), grid, dim3(256), 0, stream, a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.tshares <= 1) return e;
  // shares of a row tile, about: with many, few blocks have work, and each should have little
  const bool many = p.tshares > 6 * ((int64_t)a.T * p.group / kTileRows + 1);
  return head_dim == 128 ? join<128>(a, p, grid.x, many, stream) : join<64>(a, p, grid.x, many, stream);
}

}  // namespace wq
