// A cache within a budget: how much attention each cached slot has received,
// and the eviction of the slots that received least.
#pragma once

#include <cstdint>

#include "attention.cuh"

namespace spec {

// ------------------------------------------- attention weight of each slot
// For every kv head the weights of all new tokens' rows that see a slot s,
//   sum_r exp(scale q_r . k_s - lse_r),
// are added to weights[b, h, s]; a new token's own slot starts anew.  With the
// rows' lse given there is no maximum to look for and nothing to join: every
// slot's sum is finished by the warp that reads its key.
struct WeightsParams : AttnParams {  // lse is read
  float *weights;                    // [B, Hk, per * page]
  int chunk;                         // rows that are in shared memory together, a multiple of 8
};

// The list of all (sequence, kv head, tile of 128 tokens) is cut into equal
// stretches, one per CTA; a warp takes 16 tokens of every tile.  Tokens are the
// 16 rows of the m16n8k16 products, query rows their 8 columns, in the fragment
// order of attn_stream_kernel: the key codes are converted once for all rows of
// a chunk, and the queries lie in shared memory as finished fragments.  A
// lane's sums are those of its two tokens, over its two rows of each tile of 8;
// four lanes join them at the end.  The next tile's keys are on their way
// meanwhile.
constexpr int WT = 256, WTOK = 128;  // threads, tokens of a tile
constexpr int WMAX = 256;            // most rows of a chunk

template <int D, int KIND, int DT>
__global__ void __launch_bounds__(WT, 2) cache_weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int CH = D / 64;
  const float NINF = __uint_as_float(0xff800000u);
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ unsigned s_scan[WT / 32];
  __shared__ int s_seq;
  __shared__ unsigned s_base;
  uint4 *const s_q = reinterpret_cast<uint4 *>(dyn);                      // [row tile][CH][2][lane]
  float2 *const s_f = reinterpret_cast<float2 *>(dyn + p.chunk * D * 2);  // [row]: factor, -lse log2e
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
    for (int r0 = 0; r0 < rows; r0 += p.chunk) {
      const int here = min(p.chunk, (rows - r0 + 7) & ~7);
      __syncthreads();  // the chunk before has been used
      for (int rt = warp; rt < here / 8; rt += WT / 32) {
        const int r = r0 + 8 * rt + g;
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
        if (t < 2 && mine < len && (mine < s.ctx || r0 > 0)) old = out[mine];
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
              const int node = min((r0 + 8 * rt + 2 * t + (k & 1)) / p.G, p.N - 1), n = tok + g + 8 * (k >> 1) - s.ctx;
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

// ---------------------------------------------------------------- eviction
struct EvictParams {
  CacheView c;
  const int32_t *ctx;
  float *weights;  // [B, Hk, per * page]
  int keep, first, last;
  int32_t *out_index, *out_ctx;
  int32_t *status;
};
constexpr int EV_NT = 512, EV_BINS = 2048;

// Weights as whole numbers of the same order: NaN below everything, both zeros
// equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A CTA per kv head and sequence finds the k-th largest weight by its digits,
// 11, 11 and 10 bits from the top (a histogram each), and then goes over the
// slots in order: what is above it, and of its equals the first ones, is
// listed, and its weight moves along.  A slot never moves up, so a stretch of
// slots that has been read may be overwritten.
__global__ void __launch_bounds__(EV_NT) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ unsigned s_hist[EV_BINS], s_scan[EV_NT / 32];
  __shared__ unsigned s_digit, s_rem;
  __shared__ int s_bad;
  const CacheView &c = p.c;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int ctx = p.ctx[b];
  const long long S = static_cast<long long>(c.per) * c.page;
  int32_t *const index = p.out_index + (static_cast<long long>(b) * c.Hk + h) * p.keep;
  bool ok = ctx >= 0 && ctx <= S;
  if (!ok && tid == 0) atomicOr(p.status, ST_SLOTS);
  if (tid == 0) s_bad = 0;
  __syncthreads();
  if (ok && ctx > p.keep) {
    const int blocks = (ctx + c.page - 1) >> c.log_page;
    for (int i = tid; i < blocks; i += EV_NT)
      if (static_cast<unsigned>(c.table[static_cast<long long>(b) * c.per + i]) >= static_cast<unsigned>(c.pages)) s_bad = 1;
    __syncthreads();
    if (s_bad) {
      ok = false;
      if (tid == 0) atomicOr(p.status, ST_PAGE);
    }
  }
  if (h == 0 && tid == 0) p.out_ctx[b] = ok ? min(ctx, p.keep) : ctx;
  if (!ok || ctx <= p.keep) {
    for (int i = tid; i < p.keep; i += EV_NT) index[i] = ok && i < ctx ? i : -1;
    return;
  }
  float *const wts = p.weights + (static_cast<long long>(b) * c.Hk + h) * S;
  const int lo = p.first, hi = ctx - p.last;
  unsigned rem = p.keep - p.first - p.last;  // of hi - lo, which are more
  uint32_t key = 0;                          // the digits found so far, at their place
  const bool some = rem > 0;
  if (some) {
    int up = 32;  // bits below the digits found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11, down = up - bits;
      for (int i = tid; i < EV_BINS; i += EV_NT) s_hist[i] = 0;
      __syncthreads();
      for (int i0 = lo + tid; i0 < hi; i0 += 4 * EV_NT) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = i0 + e * EV_NT < hi ? wts[i0 + e * EV_NT] : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = weight_key(w[e]);
          if (i0 + e * EV_NT < hi && (pass == 0 || u >> up == key >> up)) atomicAdd(&s_hist[u >> down & ((1u << bits) - 1)], 1u);
        }
      }
      __syncthreads();
      // four bins to a thread, from the top
      unsigned n[4], four = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = s_hist[EV_BINS - 1 - 4 * tid - e], four += n[e];
      unsigned sum;
      unsigned above = block_scan<EV_NT / 32>(four, s_scan, sum) - four;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (above < rem && above + n[e] >= rem) s_digit = EV_BINS - 1 - 4 * tid - e, s_rem = rem - above;
        above += n[e];
      }
      __syncthreads();
      key |= s_digit << down;
      rem = s_rem;
      up = down;
    }
  }
  // in order: `rem` of those that equal the key, and all above it
  unsigned placed = 0, equal = 0;  // so far
#pragma unroll 1
  for (int s0 = 0; s0 < ctx; s0 += 4 * EV_NT) {
    const int at = s0 + 4 * tid;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (at < ctx) {
      const float4 x = *reinterpret_cast<const float4 *>(wts + at);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    unsigned more = 0, same = 0;  // bits of the four slots
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s = at + e;
      if (s >= ctx) continue;
      const uint32_t u = weight_key(w[e]);
      if (s < lo || s >= hi || (some && u > key)) more |= 1u << e;
      else if (some && u == key) same |= 1u << e;
    }
    const unsigned both = __popc(more) | __popc(same) << 16;
    unsigned sum;
    const unsigned upto = block_scan<EV_NT / 32>(both, s_scan, sum) - both;  // every weight of the stretch has been read
    unsigned n_more = upto & 0xffffu, n_same = upto >> 16;
    // of the first n equals of this stretch, those that are kept
    const auto kept_equals = [&](unsigned n) { return min(equal + n, rem) - min(equal, rem); };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is_same = same >> e & 1;
      if ((more >> e & 1) || (is_same && equal + n_same < rem)) {
        const unsigned pos = placed + n_more + kept_equals(n_same);
        index[pos] = at + e;
        wts[pos] = w[e];
      }
      n_more += more >> e & 1, n_same += is_same;
    }
    placed += (sum & 0xffffu) + kept_equals(sum >> 16);
    equal += sum >> 16;
  }
}

// A CTA per kv head, tensor and sequence moves the kept rows together, some
// blocks at a time: their rows are gathered in shared memory, the largest
// magnitude of each block gives its scale, and the codes are written.  A row
// never moves to a later block, so whatever later blocks take is still there.
constexpr int EM_NT = 256, EM_BYTES = 65536, EM_ROWS = EM_BYTES / 64, EM_BLOCKS = EM_ROWS / 16;
__global__ void __launch_bounds__(EM_NT) evict_move_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];  // rows, then their scales
  __shared__ unsigned s_amax[EM_BLOCKS];
  const CacheView &c = p.c;
  const int b = blockIdx.y, h = blockIdx.x >> 1, tensor = blockIdx.x & 1, tid = threadIdx.x, lane = tid & 31;
  float *const s_from = reinterpret_cast<float *>(dyn + EM_BYTES);
  pdl_wait();
  pdl_launch_dependents();
  if (p.ctx[b] <= p.keep || p.out_ctx[b] != p.keep) return;  // nothing to move, or an error
  unsigned char *const codes = tensor ? c.v : c.k;
  float *const scales = tensor ? c.v_scale : c.k_scale;
  const int32_t *const index = p.out_index + (static_cast<long long>(b) * c.Hk + h) * p.keep;
  const int32_t *const table = c.table + static_cast<long long>(b) * c.per;
  const int log_row = c.D == 128 ? 3 : 2, most = EM_BYTES / c.D;  // vectors of a row, rows at a time
  uint4 *const s_row = reinterpret_cast<uint4 *>(dyn);
#pragma unroll 1
  for (int r0 = 0; r0 < p.keep; r0 += most) {
    const int rows = min(most, p.keep - r0), vectors = rows << log_row, blocks = (rows + c.page - 1) >> c.log_page;
    for (int i = tid; i < blocks; i += EM_NT) s_amax[i] = 0;
    for (int k = tid; k < vectors; k += EM_NT) {
      const int row = k >> log_row, slot = index[r0 + row];
      const long long id = static_cast<long long>(table[slot >> c.log_page]) * c.Hk + h;
      cp_async16(s_row + k, codes + (id * c.page + (slot & (c.page - 1))) * c.D + ((k & ((1 << log_row) - 1)) << 4));
      if ((k & ((1 << log_row) - 1)) == 0) s_from[row] = scales[id];
    }
    cp_async_wait_all();
    __syncthreads();
    for (int k0 = tid - lane; k0 < vectors; k0 += EM_NT) {  // a warp's vectors belong to one block
      const int k = k0 + lane;
      float m = 0.f;
      if (k < vectors) {
        const uint4 w = s_row[k];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[4];
          decode4(c.kind, u[j], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[e]));
        }
        m *= s_from[k >> log_row];
      }
      const uint32_t largest = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if (lane == 0) atomicMax(&s_amax[k0 >> log_row >> c.log_page], largest);
    }
    __syncthreads();
    for (int k = tid; k < vectors; k += EM_NT) {
      const int row = k >> log_row, blk = row >> c.log_page;
      const float scale = scale_for(c.kind, s_amax[blk]), inv = 1.f / scale, from = s_from[row];
      const uint4 w = s_row[k];
      uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[4];
        decode4(c.kind, u[j], x);
        u[j] = encode4(c.kind, x[0] * from * inv, x[1] * from * inv, x[2] * from * inv, x[3] * from * inv);
      }
      const int slot = r0 + row;
      const long long id = static_cast<long long>(table[slot >> c.log_page]) * c.Hk + h;
      reinterpret_cast<uint4 *>(codes + (id * c.page + (slot & (c.page - 1))) * c.D)[k & ((1 << log_row) - 1)] = make_uint4(u[0], u[1], u[2], u[3]);
      if (k == (blk << c.log_page) << log_row) scales[id] = scale;
    }
    __syncthreads();
  }
}

}  // namespace spec
