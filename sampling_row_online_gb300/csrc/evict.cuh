// A cache within a budget: how much attention each cached slot has received,
// and the eviction of the slots that received least.
#pragma once

#include <cstdint>

#include "attention_tile.cuh"

namespace spec {

// ------------------------------------------- attention weight of each slot
// For every kv head the weights of all new tokens' rows that see a slot s,
//   sum_r exp(scale q_r . k_s - lse_r),
// are added to weights[b, h, s]; a new token's own slot starts anew.  With the
// rows' lse given there is no maximum to look for and nothing to join: every
// slot's sum is finished by the warp that reads its key.
struct WeightsParams : AttnParams {  // lse is read
  float *weights;                    // [B, Hk, per * page]
  int most;                          // rows of a kv head, rounded up to a multiple of 8
};

// The list of all (sequence, kv head, tile of 128 tokens) is cut into equal
// stretches, one per CTA; a warp takes 16 tokens of every tile.  Tokens are the
// 16 rows of the m16n8k16 products, query rows their 8 columns, in the fragment
// order of attn_stream_kernel: the key codes are converted once for all rows,
// and the queries lie in shared memory as finished fragments.  A
// lane's sums are those of its two tokens, over its two rows of each tile of 8;
// four lanes join them at the end.  The next tile's keys are on their way
// meanwhile.
constexpr int WT = 256, WTOK = 128;  // threads, tokens of a tile

template <int D, int KIND, int DT>
__global__ void __launch_bounds__(WT, 2) cache_weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int CH = D / 64;
  const float NINF = __uint_as_float(0xff800000u);
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ unsigned s_scan[WT / 32];
  __shared__ int s_seq;
  __shared__ unsigned s_base;
  uint4 *const s_q = reinterpret_cast<uint4 *>(dyn);                      // [row tile][CH][2][lane]
  float2 *const s_f = reinterpret_cast<float2 *>(dyn + p.most * D * 2);  // [row]: factor, -lse log2e
  const CacheView &c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();

  const auto work_of = [&](int b) -> unsigned {
    if (b >= p.B) return 0;
    const Seq s = sequence(p, b);
    if (s.cnt < 0 && blockIdx.x == 0) atomicOr(p.status, ST_SLOTS);
    return s.cnt > 0 ? static_cast<unsigned>(c.Hk) * ((s.ctx + s.cnt + WTOK - 1) / WTOK) : 0;
  };
  unsigned total = 0, w = 0, upto = 0;
  for (int b0 = 0; b0 < p.B; b0 += WT) {
    unsigned sum;
    w = work_of(b0 + threadIdx.x);
    upto = total + block_scan<WT / 32>(w, s_scan, sum);
    total += sum;
  }
  const unsigned nc = min(gridDim.x, total);
  if (blockIdx.x >= nc) return;
  const Share share(total, nc);
  const unsigned my0 = share.start(blockIdx.x);
  int left = static_cast<int>(share.start(blockIdx.x + 1) - my0);
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += WT) {
    if (p.B > WT) {
      unsigned sum;
      w = work_of(b0 + threadIdx.x);
      upto = before + block_scan<WT / 32>(w, s_scan, sum);
      before += sum;
    }
    if (my0 < upto && my0 >= upto - w) s_seq = b0 + threadIdx.x, s_base = upto - w;
  }
  __syncthreads();

  int b = s_seq, h, j;  // of the stretch's next tile
  Seq s = sequence(p, b);
  {
    const unsigned tiles = (s.ctx + s.cnt + WTOK - 1) / WTOK, r = my0 - s_base;
    h = static_cast<int>(r / tiles);
    j = static_cast<int>(r - h * tiles);
  }
  const long long S = static_cast<long long>(c.per) * c.page;
  for (;;) {
    const int len = s.ctx + s.cnt, tiles = (len + WTOK - 1) / WTOK, end = min(tiles, j + left), rows = s.cnt * p.G;
    float *const out = p.weights + (static_cast<long long>(b) * c.Hk + h) * S;
    const int32_t *const table = c.table + static_cast<long long>(b) * c.per;
    {
      const int here = (rows + 7) & ~7;
      __syncthreads();  // the queries before have been used
      for (int rt = warp; rt < here / 8; rt += WT / 32) {
        const int r = 8 * rt + g;
        bool live = r < rows;
        const long long lse_at = (static_cast<long long>(b) * p.N + r / p.G) * (c.Hk * p.G) + h * p.G + r % p.G;
        const float lse = live ? p.lse[lse_at] : NINF;
        live = lse != NINF;
        const long long base = live ? b * p.q_sb + (r / p.G) * p.q_sn + (h * p.G + r % p.G) * p.q_sh + 16 * t : 0;
        float y[CH][16], amax = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            Raw8<DT> raw;
            raw.v[0] = make_uint4(0, 0, 0, 0);
            if (live) raw = p.q_vec ? load8<DT, true>(p.q, base + 64 * i + 8 * e) : load8<DT, false>(p.q, base + 64 * i + 8 * e);
            float x[8];
            unpack8<DT>(raw, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[i][8 * e + k] = x[k], amax = fmaxf(amax, fabsf(x[k]));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);  // amax * 2^-e lies in [1, 2)
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
        if (t == 0) s_f[8 * rt + g] = live ? make_float2(f, lse * -1.4426950408889634f) : make_float2(0.f, NINF);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float *z = y[i] + 8 * hf;
            s_q[((rt * CH + i) * 2 + hf) * 32 + lane] =
                make_uint4(f32_to_f16x2(z[0] * down, z[1] * down), f32_to_f16x2(z[2] * down, z[3] * down),
                           f32_to_f16x2(z[4] * down, z[5] * down), f32_to_f16x2(z[6] * down, z[7] * down));
          }
      }
      __syncthreads();

      // this warp's 16 tokens of tile i: page, codes and scale
      const auto page_id = [&](int i) {
        const int tok = i * WTOK + 16 * warp;
        return i < end && tok < len ? table[tok >> c.log_page] : -1;
      };
      uint4 kw[2][CH];
      float scale = -1.f;
      const auto load = [&](int i, int page) {
        const bool there = i < end && i * WTOK + 16 * warp < len;
        const int in = (i * WTOK + 16 * warp) & (c.page - 1);
        const bool ok = there && static_cast<unsigned>(page) < static_cast<unsigned>(c.pages);
        if (there && !ok && lane == 0) atomicOr(p.status, ST_PAGE);
        const long long id = static_cast<long long>(ok ? page : 0) * c.Hk + h;
        const unsigned char *at = c.k + (id * c.page + in + g) * D + 16 * t;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < CH; ++q) kw[e][q] = ok ? ldg_na(reinterpret_cast<const uint4 *>(at + 8 * e * D + 64 * q)) : make_uint4(0, 0, 0, 0);
        scale = ok ? c.k_scale[id] : -1.f;
      };
      load(j, page_id(j));
      int page = page_id(j + 1);
      for (int i = j; i < end; ++i) {
        const int tok = i * WTOK + 16 * warp;
        uint32_t a[CH][4][4];
#pragma unroll
        for (int q = 0; q < CH; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t u[4] = {kw[e][q].x, kw[e][q].y, kw[e][q].z, kw[e][q].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) pairs_of<KIND>(KIND == KIND_I8 ? u[x] ^ 0x80808080u : u[x], a[q][x][e], a[q][x][2 + e]);
          }
        const float ks = scale;
        load(i + 1, page);
        page = page_id(i + 2);
        if (!(ks >= 0.f)) continue;  // nothing there, or a bad page, whose slots stay as they are
        // lanes 0 and 1 of a group of four write tokens g and g + 8
        const int mine = tok + g + 8 * t;
        float old = 0.f;
        if (t < 2 && mine < s.ctx) old = out[mine];
        const bool edge = tok + 16 > s.ctx;
        float sum[2] = {0.f, 0.f};
#pragma unroll 2
        for (int rt = 0; rt < here / 8; ++rt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < CH; ++q)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint4 bq = s_q[((rt * CH + q) * 2 + hf) * 32 + lane];
              mma16816(d, a[q][2 * hf], bq.x, bq.y);
              mma16816(d, a[q][2 * hf + 1], bq.z, bq.w);
            }
          const float4 f = reinterpret_cast<const float4 *>(s_f)[4 * rt + t];
          float x[4] = {fmaf(d[0], f.x * ks, f.y), fmaf(d[1], f.z * ks, f.w), fmaf(d[2], f.x * ks, f.y), fmaf(d[3], f.z * ks, f.w)};
          if (edge) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int node = min((8 * rt + 2 * t + (k & 1)) / p.G, p.N - 1), n = tok + g + 8 * (k >> 1) - s.ctx;
              bool seen = n < 0;
              if (n >= 0 && n < s.cnt)
                seen = p.mask ? (p.mask[(static_cast<long long>(b) * p.N + node) * p.W + (n >> 5)] >> (n & 31)) & 1 : n <= node;
              if (!seen) x[k] = NINF;
            }
          }
          sum[0] += ex2(x[0]) + ex2(x[1]);
          sum[1] += ex2(x[2]) + ex2(x[3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        }
        if (t < 2 && mine < len) out[mine] = old + (t ? sum[1] : sum[0]);
      }
    }
    left -= end - j;
    if (left <= 0) return;
    j = 0;
    if (++h == c.Hk) {
      h = 0;
      do s = sequence(p, ++b);
      while (s.cnt <= 0);
    }
  }
}

// Many rows per kv head: the same sums with the products on the tensor cores,
// keys as the 128 rows of A and queries as the columns of B, so that a thread
// has a token and adds up what it reads of tensor memory.  While a tile is
// weighed, the next one's codes become fp16 operands and its products run; two
// CTAs per SM fill one another's waits.  Two threads per token take half of the
// rows each and join a tile later.  What bounds it is shared memory, which the
// products' operands, their conversion and the rows' lse (read by every warp)
// share: 8 x 32 tokens over up to 32768 slots, 128 rows: 93 us.  So rows whose
// magnitudes are alike have one factor, in a register (with a factor for each row
// 103).  Measured and dropped: conversion and weights in warps of their own 91, but
// 1024 rows 217 (203 here); with codes by bulk copies 102.
constexpr int WR = 128;  // most rows of a chunk
template <int D>
struct WeightsLayout {
  static constexpr int OP = 128 * D * 2;                 // an operand
  static constexpr int K = 0, Q = 2 * OP;                // two tiles of keys, the queries
  static constexpr int F = Q + OP;                       // [WR] each: factors, -lse log2e, nodes
  static constexpr int PART = F + 3 * WR * 4;            // [2][128] sums of the second threads
  static constexpr int SCALE = PART + 2 * 128 * 4;       // [4][8] of sixteen tokens: a thread may still read those of two tiles before
  static constexpr int BARS = SCALE + 128;
  static constexpr int SMEM = BARS + 32;
};

template <int D, int KIND, int DT>
__global__ void __launch_bounds__(WT, 2) cache_weights_tile_kernel(const __grid_constant__ WeightsParams p) {
  using L = WeightsLayout<D>;
  constexpr int PER = D / 16, STEP = WT / PER, LOADS = 128 / STEP;  // 16-code pieces of a row; rows at a time
  const float NINF = __uint_as_float(0xff800000u);
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ unsigned s_scan[WT / 32];
  __shared__ int s_seq;
  __shared__ unsigned s_base;
  __shared__ int s_most[WT / 32], s_least[WT / 32];
  float *const s_fac = reinterpret_cast<float *>(smem + L::F), *const s_nl = s_fac + WR;
  int *const s_node = reinterpret_cast<int *>(s_nl + WR);
  float *const s_part = reinterpret_cast<float *>(smem + L::PART), *const s_scale = reinterpret_cast<float *>(smem + L::SCALE);
  uint64_t *const bar = reinterpret_cast<uint64_t *>(smem + L::BARS);
  uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(smem + L::BARS + 16);
  const CacheView &c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();

  const auto work_of = [&](int b) -> unsigned {
    if (b >= p.B) return 0;
    const Seq s = sequence(p, b);
    if (s.cnt < 0 && blockIdx.x == 0) atomicOr(p.status, ST_SLOTS);
    return s.cnt > 0 ? static_cast<unsigned>(c.Hk) * ((s.ctx + s.cnt + WTOK - 1) / WTOK) : 0;
  };
  unsigned total = 0, w = 0, upto = 0;
  for (int b0 = 0; b0 < p.B; b0 += WT) {
    unsigned sum;
    w = work_of(b0 + tid);
    upto = total + block_scan<WT / 32>(w, s_scan, sum);
    total += sum;
  }
  const unsigned nc = min(gridDim.x, total);
  if (blockIdx.x >= nc) return;
  const Share share(total, nc);
  const unsigned my0 = share.start(blockIdx.x);
  int left = static_cast<int>(share.start(blockIdx.x + 1) - my0);
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += WT) {
    if (p.B > WT) {
      unsigned sum;
      w = work_of(b0 + tid);
      upto = before + block_scan<WT / 32>(w, s_scan, sum);
      before += sum;
    }
    if (my0 < upto && my0 >= upto - w) s_seq = b0 + tid, s_base = upto - w;
  }
  if (tid == 0) {
    mbar_init(bar, 1), mbar_init(bar + 1, 1);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(s_tmem, 256);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);
  const uint32_t base = smem_u32(smem);

  int b = s_seq, h, j;  // of the stretch's next tile
  Seq s = sequence(p, b);
  {
    const unsigned tiles = (s.ctx + s.cnt + WTOK - 1) / WTOK, r = my0 - s_base;
    h = static_cast<int>(r / tiles);
    j = static_cast<int>(r - h * tiles);
  }
  const long long S = static_cast<long long>(c.per) * c.page;
  bool lost = false;
  uint32_t uses = 0;  // tiles so far, all chunks: buffer uses & 1, phase (uses >> 1) & 1
  for (;;) {
    const int len = s.ctx + s.cnt, tiles = (len + WTOK - 1) / WTOK, end = min(tiles, j + left), rows = s.cnt * p.G;
    float *const out = p.weights + (static_cast<long long>(b) * c.Hk + h) * S;
    const int32_t *const table = c.table + static_cast<long long>(b) * c.per;
    for (int r0 = 0; r0 < rows; r0 += WR) {
      const int here = min(WR, rows - r0), columns = (here + 31) & ~31;
      __syncthreads();  // the chunk before has been used
      // queries: half a row to a thread, as fp16 under a power of two: one for all
      // rows of the chunk, unless their magnitudes lie too far apart
      bool alike;
      float common;
      {
        const int r = tid >> 1, half = tid & 1, row = r0 + r;
        bool live = r < here;
        const int node = row / p.G, head = h * p.G + row % p.G;
        const float lse = live ? p.lse[(static_cast<long long>(b) * p.N + node) * (c.Hk * p.G) + head] : NINF;
        live = lse != NINF;
        const long long at = live ? b * p.q_sb + node * p.q_sn + head * p.q_sh + half * (D / 2) : 0;
        Raw8<DT> raw[D / 16];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          raw[k].v[0] = make_uint4(0, 0, 0, 0);
          if (live) raw[k] = p.q_vec ? load8<DT, true>(p.q, at + 8 * k) : load8<DT, false>(p.q, at + 8 * k);
          float x[8];
          unpack8<DT>(raw[k], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);  // amax * 2^-e lies in [1, 2)
        int most = __reduce_max_sync(0xffffffffu, amax > 0.f ? e : -127), least = __reduce_min_sync(0xffffffffu, amax > 0.f ? e : 127);
        if (lane == 0) s_most[warp] = most, s_least[warp] = least;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WT / 32; ++k) most = max(most, s_most[k]), least = min(least, s_least[k]);
        // The largest in [2^14, 2^15): a row whose largest is 2^14 below it is rounded
        // as under its own power.
        alike = most - least <= 14;
        if (alike) e = max(most - 14, -126);
        common = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
        if (half == 0) {
          s_fac[r] = live ? f : 0.f;
          s_nl[r] = live ? lse * -1.4426950408889634f : NINF;
          s_node[r] = min(node, p.N - 1);
        }
        if (r < columns)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            float x[8];
            unpack8<DT>(raw[k], x);
            const int chunk = half * (D / 16) + k;  // of 8 elements
            *reinterpret_cast<uint4 *>(smem + L::Q + (chunk >> 3) * 16384 + r * 128 + ((chunk & 7) ^ (r & 7)) * 16) =
                make_uint4(f32_to_f16x2(x[0] * down, x[1] * down), f32_to_f16x2(x[2] * down, x[3] * down),
                           f32_to_f16x2(x[4] * down, x[5] * down), f32_to_f16x2(x[6] * down, x[7] * down));
          }
      }
      // codes of a tile: LOADS pieces of 16 to a thread, STEP rows apart
      const int piece = tid % PER, row0 = tid / PER;
      int page[LOADS], scale_page = -1;
      uint4 raw[LOADS];
      float scale = -1.f;  // of this thread's sixteen tokens (the first 8 threads)
      const auto find = [&](int i) {
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          const int tok = i * WTOK + row0 + k * STEP;
          page[k] = i < end && tok < len ? table[tok >> c.log_page] : -1;
        }
        if (tid < 8) scale_page = i < end && i * WTOK + 16 * tid < len ? table[(i * WTOK + 16 * tid) >> c.log_page] : -1;
      };
      const auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          const int tok = i * WTOK + row0 + k * STEP;
          const bool ok = static_cast<unsigned>(page[k]) < static_cast<unsigned>(c.pages);
          raw[k] = make_uint4(0, 0, 0, 0);
          if (ok) raw[k] = ldg_na(reinterpret_cast<const uint4 *>(c.k + ((static_cast<long long>(page[k]) * c.Hk + h) * c.page + (tok & (c.page - 1))) * D + 16 * piece));
        }
        if (tid < 8) {
          const bool ok = static_cast<unsigned>(scale_page) < static_cast<unsigned>(c.pages);
          if (!ok && i < end && i * WTOK + 16 * tid < len) atomicOr(p.status, ST_PAGE);
          scale = ok ? c.k_scale[static_cast<long long>(scale_page) * c.Hk + h] : -1.f;
        }
      };
      const auto convert = [&](uint32_t use) {
        const int buf = use & 1;
        const int panel = piece >> 2;
        unsigned char *to = smem + L::K + buf * L::OP + panel * 16384;
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          const int row = row0 + k * STEP;
          uint4 lo, hi;
          codes_to_f16<KIND, false>(raw[k], lo, hi);
          *reinterpret_cast<uint4 *>(to + row * 128 + (((2 * piece) & 7) ^ (row & 7)) * 16) = lo;
          *reinterpret_cast<uint4 *>(to + row * 128 + (((2 * piece + 1) & 7) ^ (row & 7)) * 16) = hi;
        }
        if (tid < 8) s_scale[8 * (use & 3) + tid] = scale;
        fence_async_smem();
      };
      const auto issue = [&](int buf) {
        if (warp != 0) return;
        tc_after_sync();
        const uint64_t dK = tc_desc(base + L::K + buf * L::OP, 0), dQ = tc_desc(base + L::Q, 0);
        const uint32_t id = 1u << 4 | static_cast<uint32_t>(columns / 8) << 17 | (128 / 16) << 24;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          tc_mma_ss_warp(tmem + buf * WR, dK + off, dQ + off, id, k > 0);
        }
        tc_commit_warp(bar + buf);
      };
      find(j);
      load(j);
      convert(uses);
      find(j + 1);
      load(j + 1);
      find(j + 2);
      tc_before_sync();
      __syncthreads();
      issue(uses & 1);
      const int token = 32 * (warp & 3) + lane, second = warp >> 2;
      float mine = 0.f, old = 0.f;  // the first thread's sum of the tile before, and the weight so far
      bool done = false;
      const auto finish = [&](int i, int buf) {  // both threads' sums of tile i
        const int tok = i * WTOK + token;
        if (second || !done) return;
        out[tok] = old + (mine + s_part[128 * buf + token]);
      };
      for (int i = j; i < end; ++i, ++uses) {
        const int buf = uses & 1;
        if (i + 1 < end) {
          convert(uses + 1);
          load(i + 2);
          find(i + 3);
        }
        tc_before_sync();
        __syncthreads();  // the next tile's operand; the second threads' sums of the tile before
        if (i + 1 < end) issue(buf ^ 1);
        if (i > j) finish(i - 1, buf ^ 1);
        old = !second && i * WTOK + token < len && (i * WTOK + token < s.ctx || r0 > 0) ? out[i * WTOK + token] : 0.f;
        if (!lost && !__all_sync(0xffffffffu, tile_wait<0>(bar + buf, (uses >> 1) & 1))) lost = true;
        tc_after_sync();
        const int tok = i * WTOK + token, n = tok - s.ctx;
        const float ks = s_scale[8 * (uses & 3) + (token >> 4)];
        const bool edge = (i + 1) * WTOK > s.ctx;
        float2 sum = make_float2(0.f, 0.f), other = sum;
        const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21) + buf * WR;
        // 32 rows at a time, in turn with the other thread
        const float kf = ks * common;
        const bool easy = alike && !__any_sync(0xffffffffu, !(fabsf(kf) < INFINITY));
        if (__builtin_expect(edge, 0)) {
#pragma unroll 1
          for (int q = second * 32; q < columns; q += 64) {
            uint32_t bits = n < 0 ? ~0u : 0u;  // the rows that see the slot
            if (n >= 0 && n < s.cnt) {
              if (!p.mask) {  // those of its own node and later ones
                const int before = n * p.G - r0 - q;
                bits = before <= 0 ? ~0u : before < 32 ? ~0u << before : 0u;
              } else {
#pragma unroll 8
                for (int e = 0; e < 32; ++e)
                  bits |= ((p.mask[(static_cast<long long>(b) * p.N + s_node[q + e]) * p.W + (n >> 5)] >> (n & 31)) & 1) << e;
              }
            }
            __syncwarp();
            uint32_t x[32];
            tmem_ld32(at + q, x);
            tc_wait_ld32(x);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (bits >> e & 1) sum.x += ex2(fmaf(__uint_as_float(x[e]) * ks, s_fac[q + e], s_nl[q + e]));
          }
        } else if (easy) {
#pragma unroll 1
          for (int q = second * 32; q < columns; q += 64) {
            uint32_t x[32];
            tmem_ld32(at + q, x);
            tc_wait_ld32(x);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 l = *reinterpret_cast<const float4 *>(s_nl + q + e);
              float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(kf, kf), make_float2(l.x, l.y));
              sum = add2(sum, make_float2(ex2(y.x), ex2(y.y)));
              y = fma2(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), make_float2(kf, kf), make_float2(l.z, l.w));
              other = add2(other, make_float2(ex2(y.x), ex2(y.y)));
            }
          }
          sum = add2(sum, other);
        } else {
#pragma unroll 1
          for (int q = second * 32; q < columns; q += 64) {
            uint32_t x[32];
            tmem_ld32(at + q, x);
            tc_wait_ld32(x);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(s_fac + q + e), l = *reinterpret_cast<const float4 *>(s_nl + q + e);
              float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(ks, ks), make_float2(0.f, 0.f));
              y = fma2(y, make_float2(f.x, f.y), make_float2(l.x, l.y));
              sum = add2(sum, make_float2(ex2(y.x), ex2(y.y)));
              y = fma2(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), make_float2(ks, ks), make_float2(0.f, 0.f));
              y = fma2(y, make_float2(f.z, f.w), make_float2(l.z, l.w));
              other = add2(other, make_float2(ex2(y.x), ex2(y.y)));
            }
          }
          sum = add2(sum, other);
        }
        mine = sum.x + sum.y;
        done = ks >= 0.f && tok < len;  // a bad page's slots stay as they are
        if (second) s_part[128 * buf + token] = mine;
      }
      tc_before_sync();
      __syncthreads();
      finish(end - 1, (uses - 1) & 1);
    }
    left -= end - j;
    if (left <= 0) break;
    j = 0;
    if (++h == c.Hk) {
      h = 0;
      do s = sequence(p, ++b);
      while (s.cnt <= 0);
    }
  }
  if (lost) atomicOr(p.status, ST_TIMEOUT);
  tc_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_after_sync();
    tmem_free(tmem, 256);
  }
}

// ---------------------------------------------------------------- eviction
struct EvictParams {
  CacheView c;
  const int32_t *ctx;
  float *weights;  // [B, Hk, per * page]
  int keep, first, last;
  int32_t *out_index, *out_ctx;
  int32_t *status;
};
constexpr int EV_NT = 1024, EV_BINS = 2048;      // threads, bins
constexpr int EV_SLICE = 40960;                  // slots of a CTA at a time
static_assert(EV_NT == 1024, "full_scan");
constexpr int EV_SMEM = (EV_SLICE + 2 * EV_BINS) * 4;

// Weights as whole numbers of the same order: NaN below everything, both zeros
// equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_weight(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// As block_scan, for a full CTA: every warp adds the warps' sums up by itself (a
// loop over 32 of them takes a thousand clocks).
__device__ __forceinline__ unsigned full_scan(unsigned x, unsigned *s, unsigned &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto scan = [&](unsigned y) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    return y;
  };
  x = scan(x);
  __syncthreads();  // the previous use of s is over
  if (lane == 31) s[warp] = x;
  __syncthreads();
  const unsigned y = scan(s[lane]), below = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  sum = __shfl_sync(0xffffffffu, y, 31);
  return warp ? x + below : x;
}

// A cluster per kv head and sequence finds the k-th largest weight by its
// digits, 11, 11 and 10 bits from the top (a histogram each, added up through
// distributed shared memory), and then goes over the slots in order: what is
// above it, and of its equals the first ones, is listed, and its weight moves
// along.  Every CTA has a slice of the slots in shared memory, so the weights
// are read once and may be overwritten.  Slots that do not fit are left to one
// CTA, which reads them once for each digit and once more: a slot never moves
// up, so it too overwrites only what it has read.  What bounds it is the chain
// of counts, barriers and scans, and the fetch of code that runs a few times:
// all loops are short.  64 heads of up to 32768 slots: 19 us (a slot to a lane, with
// ballots, and the first digit counted after loading: 27).
__global__ void __launch_bounds__(EV_NT) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ unsigned s_scan[EV_NT / 32], s_digit, s_rem, s_total;
  uint32_t *const s_key = reinterpret_cast<uint32_t *>(dyn);
  unsigned *const s_hist = reinterpret_cast<unsigned *>(dyn) + EV_SLICE;  // two of them
  const CacheView &c = p.c;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int b = blockIdx.y, h = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31;
#pragma unroll 1
  for (int i = tid; i < 2 * EV_BINS; i += EV_NT) s_hist[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = p.ctx[b];
  const long long S = static_cast<long long>(c.per) * c.page;
  int32_t *const index = p.out_index + (static_cast<long long>(b) * c.Hk + h) * p.keep;
  const bool fits = ctx >= 0 && ctx <= S, moves = fits && ctx > p.keep;
  // this CTA's slots: [s0, s1), EV_SLICE of them at a time
  int slice = ((ctx + C - 1) / C + 3) & ~3;
  const bool joint = C > 1 && slice <= EV_SLICE;
  if (!joint) slice = ctx;
  const int s0 = joint ? min(rank * slice, ctx) : 0, s1 = joint ? min(s0 + slice, ctx) : ctx;
  float *const wts = p.weights + (static_cast<long long>(b) * c.Hk + h) * S;
  const int lo = p.first, hi = ctx - p.last;  // of the slots between these the largest are kept
  const auto load = [&](int from, bool count) {  // keys; counts of their first digit
    const int n = min(EV_SLICE, s1 - from), first = max(lo - from, 0), end = min(hi - from, n);
#pragma unroll 2
    for (int i = 4 * tid; i < n; i += 4 * EV_NT) {
      const float4 x = *reinterpret_cast<const float4 *>(wts + from + i);
      const uint32_t u[4] = {weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w)};
      *reinterpret_cast<uint4 *>(s_key + i) = make_uint4(u[0], u[1], u[2], u[3]);
      if (!count) continue;
      const bool all = i >= first && i + 4 <= end;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (all || (i + k >= first && i + k < end)) atomicAdd(&s_hist[u[k] >> 21], 1u);
    }
  };
  const bool one = s1 - s0 <= EV_SLICE;
  int bad = 0;
  __syncthreads();  // counts are zero
  if (moves) {
    if (one) load(s0, true);
    const int blocks = (ctx + c.page - 1) >> c.log_page;
#pragma unroll 1
    for (int i = tid; i < blocks; i += EV_NT)
      bad |= static_cast<unsigned>(c.table[static_cast<long long>(b) * c.per + i]) >= static_cast<unsigned>(c.pages);
  }
  bad = __syncthreads_or(bad);
  const bool ok = fits && !bad;
  if (rank == 0 && tid == 0) {
    if (!fits) atomicOr(p.status, ST_SLOTS);
    if (bad) atomicOr(p.status, ST_PAGE);
    if (h == 0) p.out_ctx[b] = ok ? min(ctx, p.keep) : ctx;
  }
  if (!ok || !moves) {
#pragma unroll 1
    for (int i = rank * EV_NT + tid; i < p.keep; i += C * EV_NT) index[i] = ok && i < ctx ? i : -1;
    return;
  }
  if (!joint && rank > 0) return;

  unsigned rem = p.keep - p.first - p.last;  // of hi - lo, which are more
  uint32_t key = 0;                          // the digits found so far, at their place
  const bool some = rem > 0;
  if (some) {
    int up = 32;  // bits below the digits found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11, down = up - bits;
      unsigned *const hist = s_hist + (pass & 1) * EV_BINS;
      if (pass == 2) {  // the other CTAs have read the first digit's counts before the second digit's barrier
#pragma unroll 1
        for (int i = tid; i < EV_BINS; i += EV_NT) hist[i] = 0;
        __syncthreads();
      }
#pragma unroll 1
      for (int from = s0; from < s1 && !(one && pass == 0); from += EV_SLICE) {
        if (!one) {
          __syncthreads();
          load(from, pass == 0);
          if (pass == 0) continue;
          __syncthreads();
        }
        const int first = max(lo - from, 0), end = min(min(hi, s1) - from, EV_SLICE);
        const auto count = [&](uint32_t u) {
          if (u >> up == key >> up) atomicAdd(&hist[u >> down & ((1u << bits) - 1)], 1u);
        };
#pragma unroll 2
        for (int i = (first & ~3) + 4 * tid; i < end; i += 4 * EV_NT) {
          const uint4 u = *reinterpret_cast<const uint4 *>(s_key + i);
          if (i >= first && i + 4 <= end) {
            count(u.x), count(u.y), count(u.z), count(u.w);
          } else {
#pragma unroll 1
            for (int k = max(i, first); k < min(i + 4, end); ++k) count(s_key[k]);
          }
        }
      }
      if (joint) cluster_sync();
      else __syncthreads();
      // four bins to a thread, from the top
      const bool has = tid < EV_BINS / 4;
      const unsigned *mine = &hist[has ? EV_BINS - 4 - 4 * tid : 0];
      uint4 n = make_uint4(0, 0, 0, 0);
      if (has) n = *reinterpret_cast<const uint4 *>(mine);
      if (joint && has) {
#pragma unroll 2
        for (int i = 1; i < C; ++i) {
          const uint4 x = dsmem_ld_v4(dsmem_addr(mine, (rank + i) & (C - 1)));
          n.x += x.x, n.y += x.y, n.z += x.z, n.w += x.w;
        }
      }
      const unsigned four = n.x + n.y + n.z + n.w, each[4] = {n.w, n.z, n.y, n.x};
      unsigned sum;
      unsigned above = full_scan(four, s_scan, sum) - four;
      if (has && above < rem && above + four >= rem) {
        int e = 0;
        while (above + each[e] < rem) above += each[e++];
        s_digit = EV_BINS - 1 - 4 * tid - e, s_rem = rem - above;
      }
      __syncthreads();
      key |= s_digit << down;
      rem = s_rem;
      up = down;
    }
  }
  // Slots between the given ones in order: all above the key, and the first `rem`
  // of those that equal it.  Four to a lane; a warp's are neighbours.
  unsigned n_more = 0, n_same = 0;  // before this stretch of slots
#pragma unroll 1
  for (int from = s0; from < max(s1, s0 + 1); from += EV_SLICE) {
    if (!one) {
      __syncthreads();
      load(from, false);
      __syncthreads();
    }
    const int n = min(EV_SLICE, s1 - from), first = max(lo - from, 0), end = some ? min(hi - from, n) : 0;
    const int part = (max(end - (first & ~3), 0) + 4 * EV_NT - 1) / (4 * EV_NT) * 128;
    const int w0 = (first & ~3) + (tid >> 5) * part, w1 = min(w0 + part, end);
    const auto look = [&](int i, uint32_t (&u)[4], unsigned &more, unsigned &same) {  // a bit for each of slots i to i + 3
      more = same = 0;
      if (i >= w1) return;
      const uint4 x = *reinterpret_cast<const uint4 *>(s_key + i);
      u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
#pragma unroll
      for (int k = 0; k < 4; ++k) more |= (u[k] > key) << k, same |= (u[k] == key) << k;
      if (i < first || i + 4 > end) {
        const unsigned in = (i < first ? 15u << (first - i) : 15u) & (i + 4 > end ? (1u << (end - i)) - 1 : 15u);
        more &= in, same &= in;
      }
    };
    uint32_t u[4];
    unsigned more, same, both = 0;  // of the warp
#pragma unroll 1
    for (int i = w0 + 4 * lane; i < w1; i += 128) {
      look(i, u, more, same);
      both += __popc(more) | __popc(same) << 16;
    }
    both = __reduce_add_sync(0xffffffffu, both);
    unsigned sum;
    const unsigned upto = full_scan(lane == 0 ? both : 0, s_scan, sum);  // the stretch's weights have been read
    if (joint) {
      if (tid == 0) s_total = sum;
      cluster_sync();
#pragma unroll 1
      for (int i = 0; i < rank; ++i) {
        const unsigned x = static_cast<unsigned>(dsmem_ld_s32(dsmem_addr(&s_total, i)));
        n_more += x & 0xffffu, n_same += x >> 16;
      }
    }
    // the first slots stay where they are, the last ones follow all others
#pragma unroll 1
    for (int i = from + tid; i < min(lo, from + n); i += EV_NT) index[i] = i;
#pragma unroll 1
    for (int i = max(hi, from) + tid; i < from + n; i += EV_NT) {
      const int pos = p.keep - p.last + i - hi;
      index[pos] = i;
      wts[pos] = key_weight(s_key[i - from]);
    }
    const unsigned start = __shfl_sync(0xffffffffu, upto, 0) - both;
    unsigned m = n_more + (start & 0xffffu), e = n_same + (start >> 16);
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += 128) {
      const int i = i0 + 4 * lane;
      look(i, u, more, same);
      const unsigned mine = __popc(more) | __popc(same) << 16;
      unsigned before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
      }
      const unsigned all = __shfl_sync(0xffffffffu, before, 31);
      before -= mine;
      unsigned mm = m + (before & 0xffffu), ee = e + (before >> 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool above = more >> k & 1, equal = same >> k & 1;
        if (above || (equal && ee < rem)) {
          const unsigned pos = lo + mm + min(ee, rem);
          index[pos] = from + i + k;
          wts[pos] = key_weight(u[k]);
        }
        mm += above, ee += equal;
      }
      m += all & 0xffffu, e += all >> 16;
    }
    n_more += sum & 0xffffu, n_same += sum >> 16;
  }
  if (joint) cluster_sync();  // no CTA leaves while others read its counts
}

// A code's magnitude in the upper byte of each half of the result: e4m3 as its
// seven bits, which are in order; int8 as the absolute value (128 for -128).
__device__ __forceinline__ uint32_t magnitudes(int kind, uint32_t w, uint32_t sofar) {
  const uint32_t a = w & 0xff00ff00u, b = w << 8 & 0xff00ff00u;
  if (kind == KIND_E4M3) {
    asm("max.u16x2 %0, %0, %1;" : "+r"(sofar) : "r"(a & 0x7f007f00u));
    asm("max.u16x2 %0, %0, %1;" : "+r"(sofar) : "r"(b & 0x7f007f00u));
  } else {
    const uint32_t x = __vabsdiffs2(a, 0), y = __vabsdiffs2(b, 0);
    asm("max.u16x2 %0, %0, %1;" : "+r"(sofar) : "r"(x));
    asm("max.u16x2 %0, %0, %1;" : "+r"(sofar) : "r"(y));
  }
  return sofar;
}

// A cluster per kv head, tensor and sequence moves the kept rows together, some
// blocks to a CTA at a time: their rows are gathered in shared memory, the
// largest magnitude of each block gives its scale, and the codes are written
// once the whole cluster has read.  A row never moves to a later block, so
// whatever later rounds take is still there.  What bounds it are its instructions
// and the barriers of a round, which four CTAs on an SM hide: 64 heads to 4096
// slots, the whole call 50 us (three CTAs 57, two 64; 1024 threads 71; rows in
// registers 52 to 60).
constexpr int EM_NT = 512, EM_BYTES = 32768, EM_ROWS = EM_BYTES / 64, EM_BLOCKS = EM_ROWS / 16;
constexpr int EM_SMEM = EM_BYTES + EM_ROWS * 12;
constexpr int EM_V = EM_BYTES / 16 / EM_NT;      // vectors of a thread
constexpr float EM_SAME = 0.f, EM_ANY = -1.f;    // instead of a power of two that codes are multiplied by
__global__ void __launch_bounds__(EM_NT, 4) evict_move_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];  // rows; where they come from; their scales
  __shared__ unsigned s_amax[EM_BLOCKS];
  __shared__ unsigned char *s_to[EM_BLOCKS];
  const CacheView &c = p.c;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int b = blockIdx.y, h = blockIdx.x / C >> 1, tensor = blockIdx.x / C & 1, tid = threadIdx.x, lane = tid & 31;
  uint4 *const s_row = reinterpret_cast<uint4 *>(dyn);
  const uint4 **const s_at = reinterpret_cast<const uint4 **>(dyn + EM_BYTES);
  float *const s_from = reinterpret_cast<float *>(dyn + EM_BYTES + EM_ROWS * 8), *const s_ratio = reinterpret_cast<float *>(s_at);
  pdl_wait();
  pdl_launch_dependents();
  if (p.ctx[b] <= p.keep || p.out_ctx[b] != p.keep) return;  // nothing to move, or an error
  unsigned char *const codes = tensor ? c.v : c.k;
  float *const scales = tensor ? c.v_scale : c.k_scale;
  const int32_t *const index = p.out_index + (static_cast<long long>(b) * c.Hk + h) * p.keep;
  const int32_t *const table = c.table + static_cast<long long>(b) * c.per;
  const int log_row = c.D == 128 ? 3 : 2, last = (1 << log_row) - 1, most = EM_BYTES / c.D;  // vectors of a row; rows at a time
#pragma unroll 1
  for (int round = 0; round < p.keep; round += most * C) {
    const int r0 = round + rank * most, rows = max(0, min(most, p.keep - r0));
    const int vectors = rows << log_row, blocks = (rows + c.page - 1) >> c.log_page;
#pragma unroll 1
    for (int row = tid; row < rows; row += EM_NT) {
      const int slot = index[r0 + row];
      const long long id = static_cast<long long>(table[slot >> c.log_page]) * c.Hk + h;
      s_from[row] = scales[id];
      s_at[row] = reinterpret_cast<const uint4 *>(codes + (id * c.page + (slot & (c.page - 1))) * c.D);
    }
    if (tid < blocks) {
      s_amax[tid] = 0;
      s_to[tid] = codes + ((static_cast<long long>(table[(r0 >> c.log_page) + tid]) * c.Hk + h) << (c.log_page + log_row + 4));
    }
    __syncthreads();
#pragma unroll 8
    for (int k = tid; k < vectors; k += EM_NT) cp_async16(s_row + k, s_at[k >> log_row] + (k & last));
    cp_async_wait_all();
    __syncthreads();
    // a warp's vectors are neighbours, some sixteens of rows
    const int k0 = (tid - lane) * EM_V + lane;
    float most_here = 0.f;
#pragma unroll
    for (int v = 0; v < EM_V; ++v) {
      const int k = k0 + 32 * v, blk = (k - lane) >> log_row >> c.log_page;
      if (k - lane >= vectors) break;
      if (k < vectors) {
        const uint4 w = s_row[k];
        uint32_t x = magnitudes(c.kind, w.w, magnitudes(c.kind, w.z, magnitudes(c.kind, w.y, magnitudes(c.kind, w.x, 0))));
        x = max(x & 0xffffu, x >> 16) >> 8;
        float m;
        if (c.kind == KIND_E4M3) {
          float y[4];
          decode4(KIND_E4M3, x, y);
          m = x < 0x7f ? y[0] : 448.f;  // a NaN code, which the cache does not have, is as large as any
        } else {
          m = static_cast<float>(x);
        }
        most_here = fmaxf(most_here, m * s_from[k >> log_row]);
      }
      if (v + 1 == EM_V || k - lane + 32 >= vectors || (k - lane + 32) >> log_row >> c.log_page != blk) {  // the block's last
        const uint32_t largest = __reduce_max_sync(0xffffffffu, __float_as_uint(most_here));
        if (lane == 0) atomicMax(&s_amax[blk], largest);
        most_here = 0.f;
      }
    }
    __syncthreads();
    // What a row's codes are multiplied by.  The same scale, the same codes (-128 is
    // not among them: its block's scale is larger).  A power of two: e4m3 in fp16,
    // where codes times 2^-14 to 2^15 are exact as far as their rounding to e4m3 can
    // tell; conversions between 8 and 32 bits would bound the kernel.
    const auto inverse = [&](int blk) { return 1.f / scale_for(c.kind, s_amax[blk]); };
#pragma unroll 1
    for (int row = tid; row < rows; row += EM_NT) {
      const float from = s_from[row], ratio = from * inverse(row >> c.log_page);
      const bool two = ((__float_as_uint(from) | __float_as_uint(ratio)) & 0x7fffffu) == 0 && from >= 0x1p-126f && ratio >= 0x1p-14f && ratio <= 0x1p15f;
      s_ratio[row] = !two ? EM_ANY : ratio == 1.f ? EM_SAME : ratio;
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    if (tid < blocks) scales[(s_to[tid] - codes) >> (c.log_page + log_row + 4)] = scale_for(c.kind, s_amax[tid]);
#pragma unroll
    for (int v = 0; v < EM_V; ++v) {
      const int k = k0 + 32 * v;
      if (k >= vectors) break;
      const int row = k >> log_row, blk = row >> c.log_page;
      const float ratio = s_ratio[row];
      const uint4 w = s_row[k];
      uint32_t u[4] = {w.x, w.y, w.z, w.w};
      if (ratio == EM_SAME) {
      } else if (ratio > 0.f && c.kind == KIND_E4M3) {
        const uint32_t r2 = f32_to_f16x2(ratio, ratio);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 x, y;\n\tmov.b32 {a, b}, %0;\n\tcvt.rn.f16x2.e4m3x2 x, a;\n\tcvt.rn.f16x2.e4m3x2 y, b;\n\t"
              "mul.rn.f16x2 x, x, %1;\n\tmul.rn.f16x2 y, y, %1;\n\t"
              "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, y;\n\tmov.b32 %0, {a, b};\n\t}"
              : "+r"(u[j])
              : "r"(r2));
        }
      } else {
        const float from = s_from[row], inv = inverse(blk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[4];
          decode4(c.kind, u[j], x);
          if (ratio > 0.f) u[j] = encode4_finite(c.kind, x[0], x[1], x[2], x[3], ratio);
          else u[j] = encode4(c.kind, x[0] * from * inv, x[1] * from * inv, x[2] * from * inv, x[3] * from * inv);
        }
      }
      *reinterpret_cast<uint4 *>(s_to[blk] + ((row & (c.page - 1)) << (log_row + 4)) + ((k & last) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __syncthreads();
  }
}

}  // namespace spec
