// Attention of new tokens (one token, a chain or a tree of drafts, a part of
// a prompt) over a paged 8-bit key/value cache.
//
//   s(r, j) = scale * q_r . (ck_j * sk) over the slots j that row r sees,
//   out_r   = sum_j softmax(s(r, .))_j * (cv_j * sv),
//
// with codes ck, cv and one scale sk, sv per (page, kv head).  In base 2 and
// with x = s log2e + log2(sv) the weights are w = 2^(x - m), m 13 below a
// running maximum of x that is at most 2.9 behind, and
//
//   out = sum_j w_j cv_j / sum_j w_j / sv_j:
//
// the value's scale rides in the exponent, so the largest weight that meets
// the codes lies in [2^13, 2^15.9] whatever the scales are (fp16 keeps its full
// precision down to 2^-27 of it), and both scales cost nothing more than the
// multiply-add that every score needs anyway.  Codes of both kinds
// are exact in fp16 (e4m3 as code * 2^-8, by moving bits; int8 by an offset),
// queries are fp16 with a power of two per row, and the products accumulate in
// fp32; the one rounding inside is that of the weights to fp16 (half a step
// 2^-12 relative).  Sums, maxima and the output stay in fp32 until the output
// is rounded once.
//
// Rows: row r of kv head h is node r / G, query head h G + r % G, with G the
// query heads per kv head.
#pragma once

#include <cstdint>

#include "cache.cuh"

namespace spec {

struct AttnParams {
  CacheView c;
  const void *q;              // [B, N, Hq, D], strides in elements
  long long q_sb, q_sn, q_sh;
  int q_vec;                  // rows of q are 16-byte aligned
  void *out;                  // [B, N, Hq, D]
  float *lse;                 // [B, N, Hq] or NULL
  const int32_t *ctx, *counts;
  const uint32_t *mask;       // [B, N, W] or NULL (chain)
  int B, N, W, G;
  float scale_log2;           // scale * log2(e)
  float *pieces;              // two unfinished pieces per CTA
  int *done;                  // arrivals per segment, by its first CTA; zero between calls
  int32_t *status;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float WEIGHT_UP = 13.f, WEIGHT_SLACK = 2.9f;  // the largest weight is 2^13 to 2^15.9
constexpr float LEAST_V_SCALE = 7.888609052210118e-31f;  // 2^-100: below it a block counts as zero

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Two codes, each in the upper byte of a half, as fp16: e4m3 as value * 2^-8
// (sign to the sign, the seven other bits to the top of exponent and mantissa;
// subnormals stay exact), the lower bytes do not matter.
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t x) { return ((x >> 1) & 0x3f803f80u) | (x & 0x80008000u); }
// int8 codes plus 128, each in the lower byte of a half, as fp16:
// 0x6400 | u is 1024 + u.
__device__ __forceinline__ uint32_t i8_halves(uint32_t x) {
  const uint32_t u = (x & 0x00ff00ffu) | 0x64006400u;
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));  // 1152
  return r;
}
// Codes j and j + 1 of the word w (j = 0 or 2).
template <int KIND, int J>
__device__ __forceinline__ uint32_t pair_of(uint32_t w) {
  if (KIND == KIND_E4M3) return e4m3_halves(prmt(w, 0, J == 0 ? 0x1404 : 0x3424));
  return i8_halves(prmt(w, 0, J == 0 ? 0x4140 : 0x4342));  // w: codes + 128 already
}
// Code j of words a and b.
template <int KIND>
__device__ __forceinline__ uint32_t pair_across(uint32_t a, uint32_t b, int j) {
  if (KIND == KIND_E4M3) return e4m3_halves(prmt(a, b, 0x4400 + 0x1111 * j));
  return i8_halves(prmt(a, b, 0x0400 + 0x1111 * j));
}

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- sequences
struct Seq {
  int ctx, cnt;  // cnt < 0: the sequence does not fit its pages
};
__device__ __forceinline__ Seq sequence(const AttnParams &p, int b) {
  Seq s;
  s.ctx = p.ctx[b];
  s.cnt = p.counts ? p.counts[b] : p.N;
  if (s.ctx < 0 || s.cnt < 0 || s.cnt > p.N || static_cast<long long>(s.ctx) + s.cnt > static_cast<long long>(p.c.per) * p.c.page)
    s.cnt = -1;
  return s;
}

// Fills the rows that no work item writes: those past a sequence's count
// (zero, lse -inf) and those of a sequence that does not fit (NaN).
template <int DT, int NTH>
__device__ __forceinline__ void fill_rest(const AttnParams &p, int D) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Seq s = sequence(p, b);
    if (s.cnt == p.N) continue;
    if (s.cnt < 0 && threadIdx.x == 0) atomicOr(p.status, ST_SLOTS);
    const float v = s.cnt < 0 ? __uint_as_float(0x7fc00000u) : 0.f;
    const int Hq = p.c.Hk * p.G;
    const float x[8] = {v, v, v, v, v, v, v, v};
    const Raw8<DT> r = pack8<DT>(x);
    const long long from = static_cast<long long>(b) * p.N + max(s.cnt, 0), to = static_cast<long long>(b + 1) * p.N;
    for (long long i = from * Hq * D / 8 + threadIdx.x; i < to * Hq * D / 8; i += NTH) store8<DT, true>(p.out, i * 8, r);
    if (p.lse)
      for (long long i = from * Hq + threadIdx.x; i < to * Hq; i += NTH) p.lse[i] = s.cnt < 0 ? v : __uint_as_float(0xff800000u);
  }
}

// ======================================================================
// Few rows per kv head: each warp streams its own tokens.
// ======================================================================
// The work is the list of all (sequence, kv head, tile of 16 rows, step of 16
// tokens), in that order, and every warp of the grid takes an equal stretch of
// it, so ragged lengths need no schedule.  A warp copies the steps ahead into
// a ring with cp.async; every lane reads back only what it copied itself, so
// the loop has no barrier at all.  The m16n8k16 fragments allow any order of
// the contracted index: a lane's 16 bytes of a key row serve four k-steps, and
// its 16 bytes of each of four value rows serve 16 column tiles, so nothing is
// exchanged and nothing is transposed; the weights go from the accumulators of
// the first product to the operand of the second in registers.
//
// A stretch that ends inside a segment (a row tile of a kv head) leaves a
// piece (m, l, out); the CTA merges the pieces of its warps, and the last CTA
// to arrive at a segment merges those of its CTAs in index order.
constexpr int AW = 12;           // warps
constexpr int ANT = 32 * AW;
constexpr int ASTAGES = 2;       // steps in flight per warp
constexpr int ASTEP = 16;        // tokens per step

template <int D>
struct StreamLayout {
  static constexpr int KB = ASTEP * D, STAGE = 2 * KB + 256;     // codes of keys and values, scales
  static constexpr int PIECE = (16 * D + 32) * 4;                // out, m, l
  static constexpr int RING = AW * ASTAGES * STAGE;
  static constexpr int SMEM = RING + AW * PIECE + 64;
  static_assert(PIECE <= ASTAGES * STAGE, "a warp's last piece lies in its own ring");
};

struct Segment {  // a row tile of a kv head, and the part of it that a piece covers
  long long at;   // first step in the list of all work
  int b, h, tile, steps, s0, s1, ctx, cnt;
};

// Writes one quarter row: 4 columns from `d` of row r.
template <int DT>
__device__ __forceinline__ void put4(const AttnParams &p, const Segment &g, int D, int r, int d, float4 x) {
  const long long row = (static_cast<long long>(g.b) * p.N + r / p.G) * (p.c.Hk * p.G) + g.h * p.G + r % p.G;
  uint2 w;
  if (DT == DT_BF16) w = make_uint2(f32_to_bf16x2(x.x, x.y), f32_to_bf16x2(x.z, x.w));
  else w = make_uint2(f32_to_f16x2(x.x, x.y), f32_to_f16x2(x.z, x.w));
  *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * D + d) = w;
}
__device__ __forceinline__ void put_lse(const AttnParams &p, const Segment &g, int r, float m, float l) {
  if (!p.lse) return;
  const long long row = (static_cast<long long>(g.b) * p.N + r / p.G) * (p.c.Hk * p.G) + g.h * p.G + r % p.G;
  p.lse[row] = l == 0.f ? __uint_as_float(0xff800000u) : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int KIND, int DT>
__global__ void __launch_bounds__(ANT, 1) attn_stream_kernel(const __grid_constant__ AttnParams p) {
  using L = StreamLayout<D>;
  constexpr int CH = D / 64, NT8 = D / 8;                // 16-byte chunks of a key row per lane; column tiles
  constexpr float VFIX = KIND == KIND_E4M3 ? 256.f : 1.f;  // fp16 codes are value / VFIX
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Segment s_seg[2 * AW];
  __shared__ int s_has[2 * AW];
  __shared__ long long s_start[AW + 1];  // first step of each warp's stretch
  __shared__ long long s_base[AW];       // first step of the sequence that holds it
  __shared__ int s_seq[AW];
  __shared__ long long s_scan[AW];
  __shared__ int s_last[2];
  const CacheView &c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the list of all work: total, and where this CTA's warps start
  const auto work_of = [&](int b) -> long long {
    const Seq s = sequence(p, b);
    if (s.cnt <= 0) return 0;
    return static_cast<long long>(c.Hk) * ((s.cnt * p.G + 15) / 16) * ((s.ctx + s.cnt + ASTEP - 1) / ASTEP);
  };
  long long total = 0, nc = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += ANT) {
      const int b = b0 + threadIdx.x;
      const long long w = b < p.B ? work_of(b) : 0;
      long long x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = x;
      __syncthreads();
      long long before = run;
      for (int i = 0; i < AW; ++i) {
        if (i < warp) before += s_scan[i];
        run += s_scan[i];
      }
      if (pass == 1) {
        const long long first = before + x - w;
        for (int i = 0; i < AW; ++i)
          if (w > 0 && s_start[i] >= first && s_start[i] < first + w) s_seq[i] = b, s_base[i] = first;
      }
    }
    if (pass == 0) {
      total = run;
      nc = min(static_cast<long long>(gridDim.x), total);
      if (static_cast<long long>(blockIdx.x) < nc && threadIdx.x <= AW)
        s_start[threadIdx.x] = total * (static_cast<long long>(blockIdx.x) * AW + threadIdx.x) / (nc * AW);
      __syncthreads();
      if (static_cast<long long>(blockIdx.x) >= nc) break;
    }
  }
  fill_rest<DT, ANT>(p, D);
  if (static_cast<long long>(blockIdx.x) >= nc) return;
  __syncthreads();

  const uint32_t ring = smem_u32(smem) + warp * ASTAGES * L::STAGE;
  unsigned char *ring_ptr = smem + warp * ASTAGES * L::STAGE;
  const long long my0 = s_start[warp], my1 = s_start[warp + 1];
  if (lane < 2) s_has[2 * warp + lane] = 0;

  // a place in the list of all work
  struct Cursor {
    int b, h, tile, step, steps, tiles, ctx, cnt;
  };
  const auto enter = [&](Cursor &u) {  // the sequence u.b, or the next one that has work
    for (;; ++u.b) {
      const Seq s = sequence(p, u.b);
      if (s.cnt <= 0) continue;
      u.ctx = s.ctx, u.cnt = s.cnt;
      u.steps = (s.ctx + s.cnt + ASTEP - 1) / ASTEP;
      u.tiles = (s.cnt * p.G + 15) / 16;
      return;
    }
  };
  const auto next_segment = [&](Cursor &u) {
    u.step = 0;
    if (++u.tile < u.tiles) return;
    u.tile = 0;
    if (++u.h < c.Hk) return;
    u.h = 0;
    ++u.b;
    enter(u);
  };
  if (my1 > my0) {
    Cursor at;  // what is consumed
    at.b = s_seq[warp];
    enter(at);
    {
      long long r = my0 - s_base[warp];
      at.step = static_cast<int>(r % at.steps);
      r /= at.steps;
      at.tile = static_cast<int>(r % at.tiles);
      at.h = static_cast<int>(r / at.tiles);
    }
    Cursor is = at;  // what is copied ahead
    long long copied = my0;
    int held_b = -1, held_p = 0, held = 0;  // page ids held_p + lane of sequence held_b

    const auto copy_step = [&]() {
      const int slot = static_cast<int>(copied - my0) % ASTAGES;
      if (copied < my1) {
        if (is.step == is.steps) next_segment(is);
        const int tok = is.step * ASTEP, blk = tok >> c.log_page, in = tok & (c.page - 1);
        if (is.b != held_b || blk < held_p || blk >= held_p + 32) {
          held_b = is.b, held_p = blk;
          const int blocks = (is.ctx + is.cnt + c.page - 1) >> c.log_page;
          held = blk + lane < blocks ? c.table[static_cast<long long>(is.b) * c.per + blk + lane] : 0;
        }
        int page = __shfl_sync(0xffffffffu, held, blk - held_p);
        const bool bad = static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages);
        if (bad) page = 0;
        const long long id = static_cast<long long>(page) * c.Hk + is.h;
        const long long off = (id * c.page + in) * D;
        const uint32_t dst = ring + slot * L::STAGE;
        const unsigned char *k = c.k + off + (4 * (g >> 1) + (g & 1)) * D + 16 * t;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < CH; ++j) cp_async<16>(dst + ((i * CH + j) * 32 + lane) * 16, k + 2 * i * D + 64 * j);
        const unsigned char *v = c.v + off + 4 * t * D + g * NT8;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async<NT8>(dst + L::KB + (i * 32 + lane) * NT8, v + i * D);
        const uint32_t sc = dst + 2 * L::KB + lane * 8;
        if (!bad) {
          cp_async<4>(sc, c.k_scale + id);
          cp_async<4>(sc + 4, c.v_scale + id);
        } else {  // a NaN scale makes the rows NaN
          if (lane == 0) atomicOr(p.status, ST_PAGE);
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(sc), "r"(0x7fc00000u), "r"(0x3f800000u) : "memory");
        }
        ++is.step;
      }
      ++copied;
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ASTAGES; ++i) copy_step();

    long long now = my0;
    bool first_piece = true;
    while (now < my1) {
      if (at.step == at.steps) next_segment(at);
      Segment seg;
      seg.b = at.b, seg.h = at.h, seg.tile = at.tile, seg.steps = at.steps, seg.ctx = at.ctx, seg.cnt = at.cnt;
      seg.at = now - at.step, seg.s0 = at.step;
      seg.s1 = static_cast<int>(min(static_cast<long long>(at.steps), at.step + (my1 - now)));
      const int rows = min(16, at.cnt * p.G - at.tile * 16);

      // queries as fp16 fragments with a power of two per row
      uint32_t qf[CH * 4][4];
      float fac[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int rr = g + 8 * half, r = at.tile * 16 + rr;
        const bool live = rr < rows;
        const long long base = live ? at.b * p.q_sb + (r / p.G) * p.q_sn + (at.h * p.G + r % p.G) * p.q_sh : 0;
        float x[CH][16];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            x[i][j] = live ? one_element<DT>(p.q, base + 64 * i + 16 * t + j) : 0.f;
            amax = fmaxf(amax, fabsf(x[i][j]));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // amax * 2^-e lies in [1, 2)
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        fac[half] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2 * VFIX;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            qf[i * 4 + w][half] = f32_to_f16x2(x[i][4 * w] * down, x[i][4 * w + 1] * down);
            qf[i * 4 + w][2 + half] = f32_to_f16x2(x[i][4 * w + 2] * down, x[i][4 * w + 3] * down);
          }
      }
      float o[NT8][4];
#pragma unroll
      for (int j = 0; j < NT8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      float m[2], base_m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // exponents' offset (as subtracted: 0 for -inf), sum
      float m0[2], l0[2] = {0.f, 0.f};  // maximum and sum over blocks without values
      m[0] = m[1] = m0[0] = m0[1] = __uint_as_float(0xff800000u);

      for (int step = seg.s0; step < seg.s1; ++step, ++now) {
        const int slot = static_cast<int>(now - my0) % ASTAGES;
        cp_async_wait<ASTAGES - 1>();
        const unsigned char *st = ring_ptr + slot * L::STAGE;
        const float2 sc = *reinterpret_cast<const float2 *>(st + 2 * L::KB + lane * 8);
        // scores: two tiles of 8 tokens; column n of tile i is token
        // 4 (n / 2) + n % 2 + 2 i, so a lane holds tokens 4 t .. 4 t + 3
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          uint4 a = lds128(st + (j * 32 + lane) * 16), b = lds128(st + ((CH + j) * 32 + lane) * 16);
          uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (KIND == KIND_I8) aw[w] ^= 0x80808080u, bw[w] ^= 0x80808080u;
            mma16816(s[0], qf[4 * j + w], pair_of<KIND, 0>(aw[w]), pair_of<KIND, 2>(aw[w]));
            mma16816(s[1], qf[4 * j + w], pair_of<KIND, 0>(bw[w]), pair_of<KIND, 2>(bw[w]));
          }
        }
        const bool zero = sc.y <= LEAST_V_SCALE;  // no values in this block: it counts in the sum only
        const float lv = zero ? 0.f : lg2(sc.y), rv = 1.f / sc.y;
        const float f0 = fac[0] * sc.x, f1 = fac[1] * sc.x;
        float x[2][4];  // row (g, g + 8), token 4 t + j
        x[0][0] = fmaf(s[0][0], f0, lv), x[0][1] = fmaf(s[0][1], f0, lv), x[0][2] = fmaf(s[1][0], f0, lv), x[0][3] = fmaf(s[1][1], f0, lv);
        x[1][0] = fmaf(s[0][2], f1, lv), x[1][1] = fmaf(s[0][3], f1, lv), x[1][2] = fmaf(s[1][2], f1, lv), x[1][3] = fmaf(s[1][3], f1, lv);
        if ((step + 1) * ASTEP > at.ctx) {  // new tokens, or slots past the last one
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int node = min((at.tile * 16 + g + 8 * half) / p.G, p.N - 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = step * ASTEP + 4 * t + j - at.ctx;
              bool seen = n < 0;
              if (n >= 0 && n < at.cnt)
                seen = p.mask ? (p.mask[(static_cast<long long>(at.b) * p.N + node) * p.W + (n >> 5)] >> (n & 31)) & 1 : n <= node;
              if (!seen) x[half][j] = __uint_as_float(0xff800000u);
            }
          }
        }
        if (zero) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float top = fmaxf(fmaxf(x[half][0], x[half][1]), fmaxf(x[half][2], x[half][3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float nm = fmaxf(m0[half], top), nb = nm == __uint_as_float(0xff800000u) ? 0.f : nm;
            l0[half] *= ex2(m0[half] - nb);
            m0[half] = nm;
#pragma unroll
            for (int j = 0; j < 4; ++j) l0[half] += ex2(x[half][j] - nb);
          }
          copy_step();
          ++at.step;
          continue;
        }
        // the offset moves only when a weight would pass 2^15.9
        bool up = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float top = fmaxf(fmaxf(x[half][0], x[half][1]), fmaxf(x[half][2], x[half][3]));
          up |= top > m[half] + (WEIGHT_UP + WEIGHT_SLACK);
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float top = fmaxf(fmaxf(x[half][0], x[half][1]), fmaxf(x[half][2], x[half][3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float nm = fmaxf(m[half], top - WEIGHT_UP);
            const float nb = nm == __uint_as_float(0xff800000u) ? 0.f : nm;
            const float a = ex2(m[half] - nb);  // 0 from -inf
            m[half] = nm, base_m[half] = nb, l[half] *= a;
#pragma unroll
            for (int j = 0; j < NT8; ++j) o[j][2 * half] *= a, o[j][2 * half + 1] *= a;
          }
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[half][j] = ex2(x[half][j] - base_m[half]);
            sum[half] += x[half][j];
          }
        l[0] = fmaf(sum[0], rv, l[0]);
        l[1] = fmaf(sum[1], rv, l[1]);
        const uint32_t pf[4] = {f32_to_f16x2(x[0][0], x[0][1]), f32_to_f16x2(x[1][0], x[1][1]),
                                f32_to_f16x2(x[0][2], x[0][3]), f32_to_f16x2(x[1][2], x[1][3])};
        uint32_t v[4][NT8 / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 a = lds128(st + L::KB + (i * 32 + lane) * 16);
            v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(st + L::KB + (i * 32 + lane) * 8);
            v[i][0] = a.x, v[i][1] = a.y;
          }
          if (KIND == KIND_I8)
#pragma unroll
            for (int w = 0; w < NT8 / 4; ++w) v[i][w] ^= 0x80808080u;
        }
#pragma unroll
        for (int w = 0; w < NT8 / 4; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816(o[4 * w + j], pf, pair_across<KIND>(v[0][w], v[1][w], j), pair_across<KIND>(v[2][w], v[3][w], j));
        copy_step();
        ++at.step;
      }
      // a lane holds columns [t D / 4, (t + 1) D / 4) of rows g and g + 8
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (__any_sync(0xffffffffu, l0[half] > 0.f)) {  // joined so that neither sum overflows
          const float nm = fmaxf(m[half], m0[half] - 60.f), nb = nm == __uint_as_float(0xff800000u) ? 0.f : nm;
          const float a = ex2(m[half] - nb);
          l[half] = l[half] * a + l0[half] * ex2(m0[half] - nb);
          m[half] = nm;
#pragma unroll
          for (int j = 0; j < NT8; ++j) o[j][2 * half] *= a, o[j][2 * half + 1] *= a;
        }
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      }
      if (seg.s0 == 0 && seg.s1 == seg.steps) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int rr = g + 8 * half;
          if (rr < rows) {
            const float inv = l[half] == 0.f ? 0.f : VFIX / l[half];
#pragma unroll
            for (int q = 0; q < NT8 / 2; ++q) {
              const int j = (4 * q) % NT8, e = 2 * half + (4 * q) / NT8;
              put4<DT>(p, seg, D, at.tile * 16 + rr, t * (D / 4) + 4 * q,
                       make_float4(o[j][e] * inv, o[j + 1][e] * inv, o[j + 2][e] * inv, o[j + 3][e] * inv));
            }
            if (t == 0) put_lse(p, seg, at.tile * 16 + rr, m[half], l[half]);
          }
        }
      } else {
        // the first piece has its own place, the last one takes the ring's
        const int which = first_piece ? 0 : 1;
        float4 *to = reinterpret_cast<float4 *>(which ? ring_ptr : smem + L::RING + warp * L::PIECE);
        if (which) {  // every lane's copies have landed and been read
          cp_async_wait<0>();
          __syncwarp();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int q = 0; q < NT8 / 2; ++q) {
            const int j = (4 * q) % NT8, e = 2 * half + (4 * q) / NT8;
            to[(half * (NT8 / 2) + q) * 32 + lane] = make_float4(o[j][e], o[j + 1][e], o[j + 2][e], o[j + 3][e]);
          }
        if (t == 0) {
          float *ml = reinterpret_cast<float *>(to) + 16 * D;
          ml[g] = m[0], ml[g + 8] = m[1], ml[16 + g] = l[0], ml[24 + g] = l[1];
        }
        if (lane == 0) s_seg[2 * warp + which] = seg, s_has[2 * warp + which] = 1;
      }
      first_piece = false;
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // ---- the CTA's pieces: neighbours of one segment are merged
  const auto piece_at = [&](int i) -> const float * {
    return reinterpret_cast<const float *>((i & 1) ? smem + (i >> 1) * ASTAGES * L::STAGE : smem + L::RING + (i >> 1) * L::PIECE);
  };
  constexpr int QUADS = 16 * D / 4;  // float4 of a piece
  constexpr int PF = 16 * D + 32;    // floats of a piece
  const auto cta_start = [&](long long i) { return total * i / nc; };
  float *const mine = p.pieces + static_cast<long long>(blockIdx.x) * 2 * PF;
  Segment open[2];
  bool is_open[2] = {false, false};
  for (int i = 0; i < 2 * AW;) {
    if (!s_has[i]) {
      ++i;
      continue;
    }
    const Segment seg = s_seg[i];
    int n = i, s1 = seg.s1, idx[AW + 1], cnt = 0;  // a segment has at most one piece per warp
    for (; n < 2 * AW; ++n) {
      if (!s_has[n]) continue;
      if (s_seg[n].at != seg.at) break;
      idx[cnt++] = n;
      s1 = s_seg[n].s1;
    }
    const bool whole = seg.s0 == 0 && s1 == seg.steps;
    const int rows = min(16, seg.cnt * p.G - seg.tile * 16);
    const int which = seg.s0 > 0 ? 0 : 1;
    if (!whole) open[which] = seg, is_open[which] = true;
    for (int k = threadIdx.x; k < QUADS; k += ANT) {
      const int ln = k & 31, q = (k >> 5) % (NT8 / 2), row = (k >> 5) / (NT8 / 2) * 8 + (ln >> 2);
      if (row >= rows) continue;
      float M = __uint_as_float(0xff800000u);
      for (int e = 0; e < cnt; ++e) M = fmaxf(M, piece_at(idx[e])[16 * D + row]);
      const float bm = M == __uint_as_float(0xff800000u) ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int e = 0; e < cnt; ++e) {
        const float *pc = piece_at(idx[e]);
        const float a = ex2(pc[16 * D + row] - bm);
        const float4 x = reinterpret_cast<const float4 *>(pc)[k];
        acc.x = fmaf(a, x.x, acc.x), acc.y = fmaf(a, x.y, acc.y), acc.z = fmaf(a, x.z, acc.z), acc.w = fmaf(a, x.w, acc.w);
        sum = fmaf(a, pc[16 * D + 16 + row], sum);
      }
      const bool head = q == 0 && (ln & 3) == 0;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : VFIX / sum;
        put4<DT>(p, seg, D, seg.tile * 16 + row, (ln & 3) * (D / 4) + 4 * q, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (head) put_lse(p, seg, seg.tile * 16 + row, M, sum);
      } else {
        float *to = mine + which * PF;
        reinterpret_cast<float4 *>(to)[k] = acc;
        if (head) to[16 * D + row] = M, to[16 * D + 16 + row] = sum;
      }
    }
    i = n;
  }
  if (!is_open[0] && !is_open[1]) return;

  // ---- segments that several CTAs share: the last to arrive merges
  __threadfence();
  __syncthreads();
  for (int which = 0; which < 2; ++which) {
    if (!is_open[which]) continue;
    const Segment seg = open[which];
    const auto holder = [&](long long f) {  // the CTA whose stretch holds step f
      long long i = f * nc / total;
      while (cta_start(i) > f) --i;
      while (cta_start(i + 1) <= f) ++i;
      return static_cast<int>(i);
    };
    const int c0 = holder(seg.at), c1 = holder(seg.at + seg.steps - 1), n = c1 - c0 + 1;
    if (threadIdx.x == 0) s_last[which] = atomicAdd(p.done + c0, 1) == n - 1;
    __syncthreads();
    if (!s_last[which]) continue;
    __threadfence();
    const int rows = min(16, seg.cnt * p.G - seg.tile * 16);
    const auto shared_piece = [&](int e) { return p.pieces + (static_cast<long long>(c0 + e) * 2 + (e == 0 ? 1 : 0)) * PF; };
    for (int k = threadIdx.x; k < QUADS; k += ANT) {
      const int ln = k & 31, q = (k >> 5) % (NT8 / 2), row = (k >> 5) / (NT8 / 2) * 8 + (ln >> 2);
      if (row >= rows) continue;
      float M = __uint_as_float(0xff800000u);
#pragma unroll 4
      for (int e = 0; e < n; ++e) M = fmaxf(M, __ldcg(shared_piece(e) + 16 * D + row));
      const float bm = M == __uint_as_float(0xff800000u) ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll 4
      for (int e = 0; e < n; ++e) {
        const float *pc = shared_piece(e);
        const float a = ex2(__ldcg(pc + 16 * D + row) - bm);
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(pc) + k);
        acc.x = fmaf(a, x.x, acc.x), acc.y = fmaf(a, x.y, acc.y), acc.z = fmaf(a, x.z, acc.z), acc.w = fmaf(a, x.w, acc.w);
        sum = fmaf(a, __ldcg(pc + 16 * D + 16 + row), sum);
      }
      const float inv = sum == 0.f ? 0.f : VFIX / sum;
      put4<DT>(p, seg, D, seg.tile * 16 + row, (ln & 3) * (D / 4) + 4 * q, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      if (q == 0 && (ln & 3) == 0) put_lse(p, seg, seg.tile * 16 + row, M, sum);
    }
    if (threadIdx.x == 0) p.done[c0] = 0;  // zero again for the next call
  }
}

}  // namespace spec
