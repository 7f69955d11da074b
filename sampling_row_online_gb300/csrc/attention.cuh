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
// the codes lies in [2^13, 2^15.9] whatever the scales are, and both scales cost
// nothing more than the multiply-add that every score needs anyway.  (The tile
// kernel starts at 2^8 over eight or more tiles of tokens.)  What is rounded:
// * weights to fp16 before they meet the codes, by half a step, 2^-11 relative,
//   or by fp16's least half step 2^-25 below 2^-14: 2^-38 of the largest weight
//   (2^-33 where that is 2^8).  The sum takes them in fp32, before that.
// * queries to fp16 under a power of two per row that puts the largest element
//   in [1, 2): bf16 and fp16 elements stay exact down to 2^-14 of it, below that
//   they are off by 2^-25 of it at most.
// * the output, once.
// Codes are exact in fp16 (e4m3 by the conversion instruction, int8 by an
// offset); products accumulate, and maxima, sums and the output are held, in
// fp32.  exp2 flushes weights below 2^-126, which is why value scales of one row
// should lie within 2^80 of one another: a slot's part of the sum is w / sv.
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
constexpr float LEAST_V_SCALE = 7.888609052210118e-31f;  // 2^-100: up to it a block counts as zero
// A slot adds up to 2^15.9 / sv, below 2^115.9, to the sum: held as 2^-18 of
// it, under an offset that is 18 higher, 2^30 slots stay below 2^128.
constexpr float SUM_UP = 18.f, SUM_DOWN = 3.814697265625e-06f;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Two e4m3 codes, each in the upper byte of a half, as fp16 of value * 2^-8
// (sign to the sign, the seven other bits to the top of exponent and mantissa;
// subnormals stay exact, and any bits give a finite number); the lower bytes do
// not matter.
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t x) { return ((x >> 1) & 0x3f803f80u) | (x & 0x80008000u); }
// int8 codes plus 128 in halves 0x6400 | u, which are 1024 + u, as fp16.
__device__ __forceinline__ uint32_t i8_halves(uint32_t u) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));  // 1152
  return r;
}
// The two codes in the lower and in the upper half of a word as fp16 (int8:
// plus 128 already, each in the lower byte of its half; e4m3: in the halves'
// bytes).
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Codes 0, 1 and 2, 3 of a word (int8: plus 128).
template <int KIND>
__device__ __forceinline__ void pairs_of(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (KIND == KIND_E4M3) {
    e4m3_pairs(w, lo, hi);
  } else {
    lo = i8_halves(prmt(w, 0x64646464u, 0x4140));
    hi = i8_halves(prmt(w, 0x64646464u, 0x4342));
  }
}
// Codes j and j + 1 (j = 0 or 2) of the words a and b: (a_j, b_j) and
// (a_j+1, b_j+1).
template <int KIND, int J>
__device__ __forceinline__ void pairs_across(uint32_t a, uint32_t b, uint32_t &lo, uint32_t &hi) {
  if (KIND == KIND_E4M3) {
    e4m3_pairs(prmt(a, b, J == 0 ? 0x5140 : 0x7362), lo, hi);
  } else {
    lo = i8_halves((prmt(a, b, J == 0 ? 0x0400 : 0x0602) & 0x00ff00ffu) | 0x64006400u);
    hi = i8_halves((prmt(a, b, J == 0 ? 0x0501 : 0x0703) & 0x00ff00ffu) | 0x64006400u);
  }
}

// An 8 x 8 tile of 16-bit elements, transposed: lane 4 g + t gives row g,
// columns 2 t and 2 t + 1, and gets those of the transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Asynchronous copy to shared memory under the L2 policy `pol`.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, uint64_t pol) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(pol) : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "l"(pol) : "memory");
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

// Equal stretches of `total` work items for `n` workers: the first `rem` have
// one more.  (32-bit arithmetic, one division: at a call's start and end every
// instruction is fetched for the first time, and 64-bit divisions took
// microseconds.)
struct Share {
  unsigned total, n, each, rem;
  __device__ __forceinline__ Share(unsigned total_, unsigned n_) : total(total_), n(n_), each(total_ / n_), rem(total_ - total_ / n_ * n_) {}
  __device__ __forceinline__ unsigned start(unsigned i) const { return i * each + min(i, rem); }
  __device__ __forceinline__ unsigned holder(unsigned item) const {  // each > 0
    const unsigned big = rem * (each + 1);
    return item < big ? item / (each + 1) : rem + (item - big) / each;
  }
};
// Inclusive sum over the CTA's threads; `sum` is the CTA's.
template <int WARPS>
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned *s, unsigned &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous use of s is over
  if (lane == 31) s[warp] = x;
  __syncthreads();
  sum = 0;
#pragma unroll 1
  for (int i = 0; i < WARPS; ++i) {
    if (i == warp) x += sum;
    sum += s[i];
  }
  return x;
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
// The work is the list of all (sequence, kv head, step of 16 tokens), in that
// order, and every warp of the grid takes an equal stretch of it, so ragged
// lengths need no schedule.  A warp copies the steps ahead into a ring with
// cp.async; every lane reads back only what it copied itself, so the loop has
// no barrier at all.
//
// Tokens are the 16 rows of the m16n8k16 products and query rows their 8
// columns (RT tiles of them): S^T = K Q^T, O^T += V^T P^T.  So the codes are
// operand A, converted once for all rows, and one token's 8 or fewer rows
// waste nothing.  The fragments allow any order of the contracted index and of
// the rows: a lane's 16 bytes of a key row serve four k-steps, its 16 bytes of
// each of four value rows serve 8 tiles of 16 columns, and only the weights are
// exchanged between the lanes, by a transpose of 8 x 8 tiles.
//
// One token, 8 rows per head, 64 sequences of up to 32768 tokens: 594 to 628 us,
// 5.2 TB/s, bound by how evenly the SMs are served; 24 rows at up to 8192
// tokens: 227 to 232 us (e4m3), 244 to 251 us (int8), bound by a step's
// instructions.  At head size 128 the forms for 8 and for 24 rows spill 20 to
// 32 bytes a thread; what that costs has not been measured.
//
// A stretch that ends inside a segment (the rows of a kv head) leaves a piece
// (out, offset, sum); the CTA merges the pieces of its warps, and the last CTA
// to arrive at a segment merges those of its CTAs in index order.
//
// SMs are not served alike (of equal stretches the slowest ends 12 % after the
// median), but shorter stretches on more CTAs lost more at their ends than
// they levelled: 615 us with one stretch per resident CTA, 616 with two, 634
// with eight (one token, 64 sequences of up to 32768 tokens, 8 rows per head).
constexpr int ASTEP = 16;        // tokens per step
constexpr int ALEAST = 2;        // steps per warp at least, before more CTAs take part

template <int D, int RT>
struct StreamLayout {
  // 128 registers a thread and two CTAs per SM, or 255 and one (12 warps of
  // 168 spilled: 16 rows at 8192 tokens 211 us, 8 warps 185 us)
  static constexpr int WARPS = 8, THREADS = 32 * WARPS, RESIDENT = RT == 1 ? 2 : 1;
  static constexpr int STAGES = RT <= 2 ? 2 : 3;                 // steps in flight per warp
  static constexpr int KB = ASTEP * D, STAGE = 2 * KB + 256;     // codes of keys and values, scales
  static constexpr int ROWS = 8 * RT;
  static constexpr int PIECE = ROWS * D + 2 * ROWS;              // floats: out, offset, sum
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int SMEM = RING + WARPS * PIECE * 4;          // and the warps' first pieces
  static constexpr int WORK = 2 * PIECE;                         // floats per CTA that other CTAs read
  static_assert(PIECE * 4 <= STAGES * STAGE, "a warp's last piece lies in its own ring");
};

struct Segment {  // the rows of a kv head, and the part of their steps that a piece covers
  unsigned at;    // first step in the list of all work
  int b, h, steps, s0, s1, ctx, cnt;
};

// Writes 4 columns from `d` of row r.
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

// What a row's products take: `down`, then `inv`, 2^-18 / sum together (0 where
// nothing is seen); neither leaves fp32's range where the sum does not.
struct Inverse {
  float down, inv;
  __device__ __forceinline__ explicit Inverse(float sum) {
    const bool big = sum > 1.f;
    down = big ? SUM_DOWN : 1.f;
    inv = sum == 0.f ? 0.f : 1.f / (big ? sum : sum * (1.f / SUM_DOWN));
  }
  __device__ __forceinline__ float operator()(float x) const { return x * down * inv; }
  __device__ __forceinline__ float4 operator()(float4 x) const {
    return make_float4((*this)(x.x), (*this)(x.y), (*this)(x.z), (*this)(x.w));
  }
};

template <int D, int KIND, int DT, int RT>
__global__ void __launch_bounds__(StreamLayout<D, RT>::THREADS, StreamLayout<D, RT>::RESIDENT) attn_stream_kernel(const __grid_constant__ AttnParams p) {
  using L = StreamLayout<D, RT>;
  constexpr int AW = L::WARPS, ANT = L::THREADS, ASTAGES = L::STAGES;
  constexpr int CH = D / 64, VB = D / 8, MT = D / 16;  // 16-byte chunks of a key row, bytes of a value row per lane; column tiles
  const float NINF = __uint_as_float(0xff800000u);
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Segment s_seg[2 * AW];
  __shared__ int s_has[2 * AW];
  __shared__ unsigned s_base[AW];  // first step of the sequence that holds each warp's first
  __shared__ int s_seq[AW];
  __shared__ unsigned s_scan[AW];
  __shared__ int s_last[2];
  __shared__ int2 s_range[2];  // the CTAs of a segment: first, number
  const CacheView &c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the list of all work: total, and where this CTA's warps start
  int rest = 0;  // some sequence has rows that no step writes
  const auto work_of = [&](int b) -> unsigned {
    if (b >= p.B) return 0;
    const Seq s = sequence(p, b);
    rest |= s.cnt != p.N;
    return s.cnt > 0 ? static_cast<unsigned>(c.Hk) * ((s.ctx + s.cnt + ASTEP - 1) / ASTEP) : 0;
  };
  unsigned total = 0, w = 0, upto = 0;  // upto: of all sequences up to this thread's (of the last block of them)
  for (int b0 = 0; b0 < p.B; b0 += ANT) {
    unsigned sum;
    w = work_of(b0 + threadIdx.x);
    upto = total + block_scan<AW>(w, s_scan, sum);
    total += sum;
  }
  // fewer CTAs where a warp's stretch would be a step, but a warp for each
  // segment; and about sqrt(steps) CTAs to a segment at most: a step costs a
  // warp what a piece costs the last CTA
  const unsigned segments = static_cast<unsigned>(p.B) * c.Hk;
  const unsigned most = static_cast<unsigned>(sqrtf(static_cast<float>(total) * static_cast<float>(segments))) + 1;
  const unsigned nc = min(min(gridDim.x, total), max(min(most, (total + AW * ALEAST - 1) / (AW * ALEAST)), (segments + AW - 1) / AW));
  if (__syncthreads_or(rest)) fill_rest<DT, ANT>(p, D);
  if (blockIdx.x >= nc) return;
  const Share share(total, nc * AW);
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += ANT) {
    if (p.B > ANT) {
      unsigned sum;
      w = work_of(b0 + threadIdx.x);
      upto = before + block_scan<AW>(w, s_scan, sum);
      before += sum;
    }
#pragma unroll 1
    for (int i = 0; i < AW; ++i) {
      const unsigned first = share.start(blockIdx.x * AW + i);
      if (first < upto && first >= upto - w) s_seq[i] = b0 + threadIdx.x, s_base[i] = upto - w;
    }
  }
  __syncthreads();

  unsigned char *const ring_ptr = smem + warp * ASTAGES * L::STAGE;
  const uint32_t ring = smem_u32(ring_ptr);
  float *const work = p.pieces + static_cast<long long>(blockIdx.x) * L::WORK;
  float *const first_slot = reinterpret_cast<float *>(smem + L::RING) + warp * L::PIECE;
  const unsigned my0 = share.start(blockIdx.x * AW + warp);
  const int mine = static_cast<int>(share.start(blockIdx.x * AW + warp + 1) - my0);
  if (lane < 2) s_has[2 * warp + lane] = 0;

  // a place in the list of all work
  struct Cursor {
    int b, h, step, steps, ctx, cnt;
  };
  const auto enter = [&](Cursor &u) {  // the sequence u.b, or the next one that has work
    for (;; ++u.b) {
      const Seq s = sequence(p, u.b);
      if (s.cnt <= 0) continue;
      u.ctx = s.ctx, u.cnt = s.cnt;
      u.steps = (s.ctx + s.cnt + ASTEP - 1) / ASTEP;
      return;
    }
  };
  const auto next_segment = [&](Cursor &u) {
    u.step = 0;
    if (++u.h < c.Hk) return;
    u.h = 0;
    ++u.b;
    enter(u);
  };
  if (mine > 0) {
    Cursor at;  // what is consumed
    at.b = s_seq[warp];
    enter(at);
    {
      const unsigned r = my0 - s_base[warp];
      at.h = static_cast<int>(r / at.steps);
      at.step = static_cast<int>(r) - at.h * at.steps;
    }
    // the first segment's queries come closer while the copies are set up
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = 8 * rt + g;
      if (r < at.cnt * p.G)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const uint16_t *>(p.q) + at.b * p.q_sb + (r / p.G) * p.q_sn +
                                                      (at.h * p.G + r % p.G) * p.q_sh + t * (D / 4)));
    }
    Cursor is = at;  // what is copied ahead
    int copied = 0;
    int held_b = -1, held_p = 0, held = 0;  // page ids held_p + lane of sequence held_b
    const unsigned char *kp = nullptr, *vp = nullptr;
    const float *scales = nullptr;
    const long long vs_off = c.v_scale - c.k_scale;
    const uint64_t pol = policy_evict_first();  // what is read once does not push the kernel's code out of L2
    bool bad = false, fresh = true;  // fresh: another page, or its first step

    const auto copy_step = [&]() {
      if (copied < mine) {
        if (is.step == is.steps) next_segment(is), fresh = true;
        const int tok = is.step * ASTEP, in = tok & (c.page - 1);
        if (fresh || in == 0) {
          const int blk = tok >> c.log_page;
          if (is.b != held_b || blk < held_p || blk >= held_p + 32) {
            held_b = is.b, held_p = blk;
            const int blocks = (is.ctx + is.cnt + c.page - 1) >> c.log_page;
            held = blk + lane < blocks ? c.table[static_cast<long long>(is.b) * c.per + blk + lane] : 0;
          }
          int page = __shfl_sync(0xffffffffu, held, blk - held_p);
          bad = static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages);
          if (bad) page = 0;
          const long long id = static_cast<long long>(page) * c.Hk + is.h;
          const long long off = (id * c.page + in) * D;
          kp = c.k + off + g * D + 16 * t;
          vp = c.v + off + 2 * t * D + g * VB;
          scales = c.k_scale + id;
          fresh = false;
        }
        const uint32_t dst = ring + copied % ASTAGES * L::STAGE;
#pragma unroll
        for (int i = 0; i < 2; ++i)  // tokens g and g + 8
#pragma unroll
          for (int j = 0; j < CH; ++j) cp_async<16>(dst + ((i * CH + j) * 32 + lane) * 16, kp + 8 * i * D + 64 * j, pol);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
          cp_async<VB>(dst + L::KB + (i * 32 + lane) * VB, vp + ((i & 1) + 8 * (i >> 1)) * D, pol);
        const uint32_t sc = dst + 2 * L::KB + lane * 8;
        if (!bad) {
          cp_async<4>(sc, scales, pol);
          cp_async<4>(sc + 4, scales + vs_off, pol);
        } else {  // a NaN scale makes the rows NaN that see the page
          if (lane == 0) atomicOr(p.status, ST_PAGE);
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(sc), "r"(0x7fc00000u), "r"(0x3f800000u) : "memory");
        }
        kp += ASTEP * D, vp += ASTEP * D;
        ++is.step;
      }
      ++copied;
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < ASTAGES; ++i) copy_step();

    int now = 0;
    bool first_piece = true;
    while (now < mine) {
      if (at.step == at.steps) next_segment(at);
      Segment seg;
      seg.b = at.b, seg.h = at.h, seg.steps = at.steps, seg.ctx = at.ctx, seg.cnt = at.cnt;
      seg.at = my0 + now - at.step, seg.s0 = at.step;
      seg.s1 = min(at.steps, at.step + mine - now);
      const int rows = at.cnt * p.G;

      // queries as fp16 fragments with a power of two per row: a lane loads of
      // row g, and looks after the scores of rows 2 t and 2 t + 1
      uint32_t qf[RT][CH * 4][2];
      float fac[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = 8 * rt + g;
        const bool live = r < rows;
        const long long base = live ? at.b * p.q_sb + (r / p.G) * p.q_sn + (at.h * p.G + r % p.G) * p.q_sh + 16 * t : 0;
        Raw8<DT> raw[CH][2];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            raw[i][e].v[0] = make_uint4(0, 0, 0, 0);
            if (live) raw[i][e] = p.q_vec ? load8<DT, true>(p.q, base + 64 * i + 8 * e) : load8<DT, false>(p.q, base + 64 * i + 8 * e);
          }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y[8];
            unpack8<DT>(raw[i][e], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // amax * 2^-e lies in [1, 2)
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
        fac[rt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        fac[rt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float y[8];
            unpack8<DT>(raw[i][w >> 1], y);
            const float *z = y + 4 * (w & 1);
            qf[rt][4 * i + w][0] = f32_to_f16x2(z[0] * down, z[1] * down);
            qf[rt][4 * i + w][1] = f32_to_f16x2(z[2] * down, z[3] * down);
          }
      }
      float o[RT][MT][4];
      // exponents' offset (as subtracted: 0 for -inf), sum; the same over blocks without values
      float m[RT][2], base_m[RT][2], l[RT][2], m0[RT][2], l0[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int j = 0; j < MT; ++j) o[rt][j][0] = o[rt][j][1] = o[rt][j][2] = o[rt][j][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) m[rt][e] = m0[rt][e] = NINF, base_m[rt][e] = l[rt][e] = l0[rt][e] = 0.f;
      }

      for (int step = seg.s0; step < seg.s1; ++step, ++now, ++at.step) {
        cp_async_wait<ASTAGES - 1>();
        const unsigned char *st = ring_ptr + now % ASTAGES * L::STAGE;
        const float2 sc = *reinterpret_cast<const float2 *>(st + 2 * L::KB + lane * 8);
        // scores of tokens g (0, 1) and g + 8 (2, 3) and rows 2 t, 2 t + 1; two chains of products
        float s[RT][CH][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int j = 0; j < CH; ++j) s[rt][j][0] = s[rt][j][1] = s[rt][j][2] = s[rt][j][3] = 0.f;
        uint32_t kw[CH][2][4];
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 a = lds128(st + ((i * CH + j) * 32 + lane) * 16);
            kw[j][i][0] = a.x, kw[j][i][1] = a.y, kw[j][i][2] = a.z, kw[j][i][3] = a.w;
          }
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int j = 0; j < CH; ++j) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) pairs_of<KIND>(KIND == KIND_I8 ? kw[j][i][w] ^ 0x80808080u : kw[j][i][w], a[i], a[2 + i]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) mma16816(s[rt][j], a, qf[rt][4 * j + w][0], qf[rt][4 * j + w][1]);
          }
        const bool edge = (step + 1) * ASTEP > at.ctx;  // new tokens, or slots past the last one
        const bool zero = sc.y <= LEAST_V_SCALE;        // no values in this block: it counts in a sum of its own
        const float lv = zero ? 0.f : lg2(sc.y), rv = 1.f / sc.y * SUM_DOWN;
        float x[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = fac[rt][j & 1] * sc.x;
            x[rt][j] = fmaf(CH == 2 ? s[rt][0][j] + s[rt][CH - 1][j] : s[rt][0][j], f, lv);
          }
        if (edge) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int node = min((8 * rt + 2 * t + (j & 1)) / p.G, p.N - 1), n = step * ASTEP + g + 8 * (j >> 1) - at.ctx;
              bool seen = n < 0;
              if (n >= 0 && n < at.cnt)
                seen = p.mask ? (p.mask[(static_cast<long long>(at.b) * p.N + node) * p.W + (n >> 5)] >> (n & 31)) & 1 : n <= node;
              if (!seen) x[rt][j] = NINF;
            }
        }
        const auto over_tokens = [](float v) {  // maximum over a row's tokens
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        };
        if (zero) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float nm = fmaxf(m0[rt][e], over_tokens(fmaxf(x[rt][e], x[rt][2 + e]))), nb = nm == NINF ? 0.f : nm;
              l0[rt][e] = l0[rt][e] * ex2(m0[rt][e] - nb) + ex2(x[rt][e] - nb) + ex2(x[rt][2 + e] - nb);
              m0[rt][e] = nm;
            }
          copy_step();
          continue;
        }
        // the offset moves only when a weight would pass 2^15.9
        bool up = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int e = 0; e < 2; ++e) up |= fmaxf(x[rt][e], x[rt][2 + e]) > m[rt][e] + (WEIGHT_UP + WEIGHT_SLACK);
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float nm = fmaxf(m[rt][e], over_tokens(fmaxf(x[rt][e], x[rt][2 + e])) - WEIGHT_UP);
              const float nb = nm == NINF ? 0.f : nm;
              const float a = ex2(m[rt][e] - nb);  // 0 from -inf
              m[rt][e] = nm, base_m[rt][e] = nb, l[rt][e] *= a;
#pragma unroll
              for (int j = 0; j < MT; ++j) o[rt][j][e] *= a, o[rt][j][2 + e] *= a;
            }
        }
        uint32_t pf[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[rt][j] = ex2(x[rt][j] - base_m[rt][j & 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) l[rt][e] = fmaf(x[rt][e] + x[rt][2 + e], rv, l[rt][e]);
          pf[rt][0] = transpose8(f32_to_f16x2(x[rt][0], x[rt][1]));
          pf[rt][1] = transpose8(f32_to_f16x2(x[rt][2], x[rt][3]));
        }
        uint32_t v[4][VB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 a = lds128(st + L::KB + (i * 32 + lane) * 16);
            v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(st + L::KB + (i * 32 + lane) * 8);
            v[i][0] = a.x, v[i][1] = a.y;
          }
        }
        if (edge) {  // rows that are not there, or another page's for a bad one, may hold anything, NaN codes too
          const int end = sc.x == sc.x ? at.ctx + at.cnt - step * ASTEP - 2 * t : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < VB / 4; ++w)
              if ((i & 1) + 8 * (i >> 1) >= end) v[i][w] = 0;
        }
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
          if (KIND == KIND_I8)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i][w] ^= 0x80808080u;
          // rows g and g + 8 of a column tile are bytes j and j + 1
          uint32_t a[2][4];
          pairs_across<KIND, 0>(v[0][w], v[1][w], a[0][0], a[0][1]);
          pairs_across<KIND, 0>(v[2][w], v[3][w], a[0][2], a[0][3]);
          pairs_across<KIND, 2>(v[0][w], v[1][w], a[1][0], a[1][1]);
          pairs_across<KIND, 2>(v[2][w], v[3][w], a[1][2], a[1][3]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) mma16816(o[rt][2 * w + j], a[j], pf[rt][0], pf[rt][1]);
        }
        copy_step();
      }
      // a lane holds columns [g D / 8, (g + 1) D / 8) of rows 2 t and 2 t + 1 of each tile
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float &lr = l[rt][e], &mr = m[rt][e];
          mr += SUM_UP;
          if (__any_sync(0xffffffffu, l0[rt][e] > 0.f)) {  // joined so that neither sum overflows
            const float nm = fmaxf(mr, m0[rt][e] - 60.f), nb = nm == NINF ? 0.f : nm;
            const float a = ex2(mr - nb);
            lr = lr * a + l0[rt][e] * ex2(m0[rt][e] - nb);
            mr = nm;
#pragma unroll
            for (int j = 0; j < MT; ++j) o[rt][j][e] *= a, o[rt][j][2 + e] *= a;
          }
          lr += __shfl_xor_sync(0xffffffffu, lr, 4);
          lr += __shfl_xor_sync(0xffffffffu, lr, 8);
          lr += __shfl_xor_sync(0xffffffffu, lr, 16);
        }
      const bool whole = seg.s0 == 0 && seg.s1 == seg.steps;
      // the first piece has its own place, the last one takes the ring's
      const int which = first_piece ? 0 : 1;
      float *const to = which ? reinterpret_cast<float *>(ring_ptr) : first_slot;
      if (!whole && which) {  // every lane's copies have landed and been read
        cp_async_wait<0>();
        __syncwarp();
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * rt + 2 * t + e;
          const Inverse over(l[rt][e]);
#pragma unroll
          for (int q = 0; q < MT / 2; ++q) {
            const float4 z = make_float4(o[rt][2 * q][e], o[rt][2 * q][2 + e], o[rt][2 * q + 1][e], o[rt][2 * q + 1][2 + e]);
            if (!whole) reinterpret_cast<float4 *>(to)[((rt * 2 + e) * (MT / 2) + q) * 32 + lane] = z;
            else if (r < rows) put4<DT>(p, seg, D, r, g * VB + 4 * q, over(z));
          }
          if (g == 0) {
            if (!whole) to[L::ROWS * D + r] = m[rt][e], to[L::ROWS * D + L::ROWS + r] = l[rt][e];
            else if (r < rows) put_lse(p, seg, r, m[rt][e], l[rt][e]);
          }
        }
      if (!whole && lane == 0) s_seg[2 * warp + which] = seg, s_has[2 * warp + which] = 1;
      first_piece = false;
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // ---- the CTA's pieces: neighbours of one segment are merged
  const auto piece_at = [&](int i) -> const float * {
    return reinterpret_cast<const float *>(i & 1 ? smem + (i >> 1) * ASTAGES * L::STAGE : smem + L::RING + (i >> 1) * L::PIECE * 4);
  };
  constexpr int QUADS = L::ROWS * D / 4;  // float4 of a piece
  // row and first column of float4 k of a piece
  const auto row_of = [](int k) { return (k >> 5) / MT * 8 + 2 * (k & 3) + (k >> 5) / (MT / 2) % 2; };
  const auto col_of = [](int k) { return ((k & 31) >> 2) * VB + (k >> 5) % (MT / 2) * 4; };
  Segment open[2];
  bool is_open[2] = {false, false};
#pragma unroll 1
  for (int i = 0; i < 2 * AW;) {
    if (!s_has[i]) {
      ++i;
      continue;
    }
    const Segment seg = s_seg[i];
    int n = i, last = i;  // the segment's pieces are among slots i .. last
#pragma unroll 1
    for (; n < 2 * AW; ++n) {
      if (!s_has[n]) continue;
      if (s_seg[n].at != seg.at) break;
      last = n;
    }
    const bool whole = seg.s0 == 0 && s_seg[last].s1 == seg.steps;
    const int rows = seg.cnt * p.G, which = seg.s0 > 0 ? 0 : 1;
    if (!whole) open[which] = seg, is_open[which] = true;
#pragma unroll 1
    for (int k = threadIdx.x; k < QUADS; k += ANT) {
      const int row = row_of(k);
      if (row >= rows) continue;
      float M = NINF;
      for (int e = i; e <= last; ++e)
        if (s_has[e]) M = fmaxf(M, piece_at(e)[L::ROWS * D + row]);
      const float bm = M == NINF ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      for (int e = i; e <= last; ++e) {
        if (!s_has[e]) continue;
        const float *pc = piece_at(e);
        const float a = ex2(pc[L::ROWS * D + row] - bm);
        const float4 x = reinterpret_cast<const float4 *>(pc)[k];
        acc.x = fmaf(a, x.x, acc.x), acc.y = fmaf(a, x.y, acc.y), acc.z = fmaf(a, x.z, acc.z), acc.w = fmaf(a, x.w, acc.w);
        sum = fmaf(a, pc[L::ROWS * D + L::ROWS + row], sum);
      }
      const bool head = col_of(k) == 0;
      if (whole) {
        put4<DT>(p, seg, D, row, col_of(k), Inverse(sum)(acc));
        if (head) put_lse(p, seg, row, M, sum);
      } else {
        float *to = work + which * L::PIECE;
        reinterpret_cast<float4 *>(to)[k] = acc;
        if (head) to[L::ROWS * D + row] = M, to[L::ROWS * D + L::ROWS + row] = sum;
      }
    }
    i = n;
  }
  if (!is_open[0] && !is_open[1]) return;

  // ---- segments that several CTAs share: the last to arrive merges
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2 && is_open[threadIdx.x]) {  // a thread for each
    const Segment &seg = open[threadIdx.x];
    const int c0 = share.holder(seg.at) / AW, c1 = share.holder(seg.at + seg.steps - 1) / AW;
    s_range[threadIdx.x] = make_int2(c0, c1 - c0 + 1);
    s_last[threadIdx.x] = atomicAdd(p.done + c0, 1) == c1 - c0;
    __threadfence();
  }
  __syncthreads();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!is_open[which] || !s_last[which]) continue;
    const Segment seg = open[which];
    const int c0 = s_range[which].x, n = s_range[which].y;
    const int rows = seg.cnt * p.G;
    const auto shared_piece = [&](int e) { return p.pieces + static_cast<long long>(c0 + e) * L::WORK + (e == 0 ? L::PIECE : 0); };
#pragma unroll 1
    for (int k = threadIdx.x; k < QUADS; k += ANT) {
      const int row = row_of(k);
      if (row >= rows) continue;
      float M = NINF, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int e0 = 0; e0 < n; e0 += 8) {  // eight pieces a round trip
        float mm[8], ll[8], top = M;
        float4 x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float *pc = shared_piece(min(e0 + e, n - 1));
          mm[e] = e0 + e < n ? __ldcg(pc + L::ROWS * D + row) : NINF;
          ll[e] = __ldcg(pc + L::ROWS * D + L::ROWS + row);
          x[e] = __ldcg(reinterpret_cast<const float4 *>(pc) + k);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, mm[e]);
        const float base = top == NINF ? 0.f : top;
        float a = ex2(M - base);
        M = top;
        acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a, sum *= a;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e0 + e >= n) continue;
          a = ex2(mm[e] - base);
          acc.x = fmaf(a, x[e].x, acc.x), acc.y = fmaf(a, x[e].y, acc.y), acc.z = fmaf(a, x[e].z, acc.z), acc.w = fmaf(a, x[e].w, acc.w);
          sum = fmaf(a, ll[e], sum);
        }
      }
      put4<DT>(p, seg, D, row, col_of(k), Inverse(sum)(acc));
      if (col_of(k) == 0) put_lse(p, seg, row, M, sum);
    }
    if (threadIdx.x == 0) p.done[c0] = 0;  // zero again for the next call
  }
}

}  // namespace spec
