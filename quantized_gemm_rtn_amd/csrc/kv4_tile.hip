// Causal attention over the 4-bit cache for many query rows, for gfx950: the tile kernel
// (kv4_attention.hip has the mathematics, the kernel for few rows, and the choice).
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

// Joins the partials of the items that more than one share worked on: block (head, share
// i, quarter of the rows) those of the item that share i begins but does not end. Sixteen
// lanes take a row, D / 16 channels each, so that a wave has four rows on their way.
template <int D>
__global__ void __launch_bounds__(256)
kv4_tile_combine_kernel(KvCache a, AttnArgs p) {
  constexpr int N = D / 16;  // channels of a lane
  const int lane = threadIdx.x & 63;
  const int h = blockIdx.x % a.hkv, share = blockIdx.x / a.hkv;
  AreaWalk walk;
  const int64_t total = area_begin(walk, a, p, lane), per = share_area(p, total);
  const int64_t from = share * per, until = from + per;
  if (until >= total) return;  // (the last share ends its items)
  AreaItem t;
  if (!area_find(t, walk, a, p, until - 1, lane)) return;
  // the share's last item: it must begin in this share and go on in the next
  if (t.X < from || t.next <= until) return;
  const int rows = t.s.rows * p.group, row0 = t.rt * kTileRows, row1 = min(rows, row0 + kTileRows) - 1;
  const TileRange range = tile_range(t.s, p, row0, row1);
  const int n = range.t1 - range.t0;
  const int64_t W = t.next - t.X;
  // shares of the item, with the tiles that each had; one that had all wrote the rows
  int parts = 0;
  for (int64_t x = from; x < t.next; x += per, ++parts)
    if (tiles_before(x + per, t.X, W, n) - tiles_before(x, t.X, W, n) == n) return;
  const int part = threadIdx.x & 15;
#pragma unroll
  for (int pass = 0; pass < kTileRows / 64; ++pass) {
    const int in = 64 * pass + 16 * blockIdx.y + (threadIdx.x >> 4), row = row0 + in;
    if (row > row1) continue;
    float best = kNoRef, total_sum = 0.0f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.0f;
    for (int i = 0; i < parts; ++i) {
      const int64_t x = from + i * per;
      if (tiles_before(x + per, t.X, W, n) == tiles_before(x, t.X, W, n)) continue;
      const int64_t at = (((int64_t)(share + i) * a.hkv + h) * 2 + (i == 0 && t.X > from ? 1 : 0)) * kTileRows + in;
      const float2 v = p.tpart_s[at];
      const float to = fmaxf(best, v.x), keep = exp2_hw(best - to), f = exp2_hw(v.x - to);
      best = to;
      total_sum = total_sum * keep + v.y * f;
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const f32x4 d = *reinterpret_cast<const f32x4*>(p.tpart_o + at * D + 64 * (e >> 2) + 4 * part);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[e + k] = o[e + k] * keep + d[k] * f;
      }
    }
    const int tok = row / p.group;
    const int64_t out_row = (int64_t)(t.s.first_row + tok) * p.hq + h * p.group + (row - tok * p.group);
    const float inv = total_sum > 0.0f ? 1.0f / total_sum : 0.0f;
    typedef f16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<f16x4*>(p.out + out_row * D + 64 * (e >> 2) + 4 * part) =
          f16x4{(f16)(o[e] * inv), (f16)(o[e + 1] * inv), (f16)(o[e + 2] * inv), (f16)(o[e + 3] * inv)};
    if (part == 0 && p.lse != nullptr)
      p.lse[out_row] = total_sum > 0.0f ? (best + log2f(total_sum)) * kLn2 : -INFINITY;
  }
}

hipError_t launch_kv4_tile(const KvCache& a, const AttnArgs& p, int64_t head_dim, hipStream_t stream) {
  const dim3 grid((unsigned)(p.tshares > 0 ? (int64_t)a.hkv * p.tshares : (int64_t)a.hkv * a.B * p.row_tiles));
  if (head_dim == 128)
    hipLaunchKernelGGL((kv4_tile_kernel<128>), grid, dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((kv4_tile_kernel<64>), grid, dim3(256), 0, stream, a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.tshares <= 1) return e;
  const dim3 quarters(grid.x, 4);
  if (head_dim == 128)
    hipLaunchKernelGGL((kv4_tile_combine_kernel<128>), quarters, dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((kv4_tile_combine_kernel<64>), quarters, dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace wq
