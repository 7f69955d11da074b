// Causal attention among the tokens of whole prompts, packed one behind the
// other: tensor cores with the accumulators in tensor memory.
//
//   out_i = sum_{j <= i} softmax(scale q_i . k_j) v_j   in i's own sequence.
//
// In base 2 and with x = s * scale * log2e the weights are w = 2^(x - m).  For fp16
// m is 8 below the maximum of x over the first tile where that is above -inf, and
// moves to 8 below the maximum again where the weights of a later tile come to
// more than 60000 together.  So the largest weight of a row lies in [2^7.9, 60000],
// fp16 keeps full precision down to 2^-22 of it, and a tile's maximum is looked for
// only where m moves: its sum tells.  bf16 has the range of 32 bits, and so may its
// values: all its weights are 2^-33 of that, which keeps the sums of 2^17 tiles of
// them below 1, and the output's below the largest value.
// One number of 32 bits holds the offset to a sixteenth up to 2^20, but from 2^27
// on it is off by more than the 8, and weights would pass the limit under any of
// them.  So beyond 2^20 it is two numbers, the maximum as rounded and the rest,
// every tile's maximum is looked for, and exponents are taken from both before they
// are weighed: the largest weight is the same whatever the scores (1 beyond 2^40,
// where weights are 1 or 0).
// What is rounded: weights to the inputs' type before they meet the values (one
// instruction takes one type; half a step, 2^-8 relative for bf16 and 2^-11 for
// fp16), and the output, once.  Sums (of the unrounded weights), maxima,
// products and lse are fp32.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "device.cuh"
#include "elements.cuh"
#include "share.cuh"
#include "tcgen05.cuh"

namespace spec {

// The rows of a tile are G query heads (that share a kv head) of `tile` tokens,
// token by token; two tiles, A and B, go through the token tiles together.
constexpr int PT = 128;              // rows of a tile, tokens of a token tile
constexpr int P_SOFT = 256;          // softmax threads: a thread per row of A and of B
constexpr int P_NT = P_SOFT + 128;   // and a warp each for copies, A's products, B's products, a look at the values
// Registers: 168 a thread at launch, then 256 * 208 + 128 * 88 = 384 * 168.
constexpr int P_REG = 168, P_REG_SOFT = 208, P_REG_REST = 88;
static_assert(P_SOFT * P_REG_SOFT + 128 * P_REG_REST <= P_NT * P_REG, "register split");
template <int DT>
constexpr float P_UP = DT == DT_BF16 ? 8.f - 33.f : 8.f;  // the largest weight where the offset has moved
template <int DT>
constexpr float P_MOST = DT == DT_BF16 ? 60000.f / (1ll << 33) : 60000.f;
constexpr float P_FAR = 1 << 20;     // offsets beyond are two numbers
constexpr int P_SHORT = 16;          // token tiles of segments that are not shared between CTAs
constexpr int P_EXTRA = 2;           // token tiles that take as long as a segment's begin and end
constexpr int P_STEPS = 64;          // most row pairs after which their ends fall on token tiles alike again

struct PromptParams {
  CUtensorMap q, k, v;    // [T, Hq / G, G, D] and [T, Hk, D]
  void *out;              // [T, Hq, D]
  float *lse;             // [T, Hq] or NULL
  const int32_t *starts;  // [B + 1]
  int B, T, Hq;
  int G, heads, per_kv;   // query heads of a tile, groups of them, groups of a kv head
  int tile;               // tokens of a row tile: 128 / G
  int period, gain;       // after `period` pairs of row tiles their ends are `gain` token tiles further
  int ends[P_STEPS + 1];  // token tiles of the first i pairs together
  float scale_log2;       // scale * log2(e)
  float *pieces;          // [CTA][2][2 groups] unfinished pieces
  int *done;              // [CTA][2 groups] arrivals per segment, by its first CTA; zero between calls
  int32_t *status;
};

struct PromptLast {  // of the segment whose output is still to be read
  long long row;
  int tok, any, live, whole, seg, first, n, which;  // not whole: first CTA of the segment, number of CTAs, the piece's place
  float m, lo, l;
};

template <int D>
struct PromptLayout {
  static constexpr int OP = PT * D * 2;  // an operand tile
  static constexpr int Q = 0, K = 2 * OP, V = 4 * OP, MARKS = 6 * OP;  // two tiles each
  static constexpr int LAST = MARKS + 3 * D * 4;  // [P_SOFT] PromptLast
  static constexpr int BARS = LAST + P_SOFT * sizeof(PromptLast);  // MARKS: first tokens with NaN, +inf, -inf in each column
  static constexpr int SMEM = BARS + 256;
  static constexpr int PIECE = PT * D + 3 * PT;  // floats: out, offset, sum, the offset's second number
};

struct PromptBars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_seen[2], q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2];
  uint64_t turn[2];
  uint32_t tmem;
  int marked;                  // 1 + the segment that the marks are of
  int ended[P_SOFT / 32];      // segments that each softmax warp is done with
};
static_assert(sizeof(PromptBars) <= 256, "barriers");

// A segment: a pair of row tiles of one group of heads of a sequence.
struct PromptPlace {
  int b, h, r, j, n;  // r: pair, j: token tile, n: token tiles of the pair
  int start, len;
};
__device__ __forceinline__ int prompt_pair_tiles(const PromptParams &p, int len, int r) {
  return (min((r + 1) * 2 * p.tile, len) + PT - 1) / PT;
}
// Token tiles of the first k pairs, none of them cut short.
__device__ __forceinline__ unsigned prompt_tiles_before(const PromptParams &p, unsigned k) {
  const unsigned m = k / p.period, e = k - m * p.period;
  return m * p.ends[p.period] + p.gain * p.period * (m * (m - 1) / 2) + p.ends[e] + e * m * p.gain;
}
__device__ __forceinline__ unsigned prompt_head_tiles(const PromptParams &p, int len) {
  if (len <= 0) return 0;
  const unsigned pairs = (len + 2 * p.tile - 1) / (2 * p.tile);
  return prompt_tiles_before(p, pairs - 1) + (len + PT - 1) / PT;
}
__device__ __forceinline__ void prompt_enter(const PromptParams &p, PromptPlace &u) {  // sequence u.b, or the next with tokens
  for (;; ++u.b) {
    u.start = p.starts[u.b];
    u.len = p.starts[u.b + 1] - u.start;
    if (u.len > 0) return;
  }
}
__device__ __forceinline__ void prompt_next(const PromptParams &p, PromptPlace &u) {  // the next segment
  u.j = 0;
  if (++u.r * 2 * p.tile >= u.len) {
    u.r = 0;
    if (++u.h == p.heads) {
      u.h = 0;
      ++u.b;
      prompt_enter(p, u);
    }
  }
  u.n = prompt_pair_tiles(p, u.len, u.r);
}
// The first token of row tile g of the pair (from len on where it has none).  A
// row tile that is alone in its pair goes to A and to B in turn, so that short
// sequences keep both busy.
__device__ __forceinline__ int prompt_from(const PromptParams &p, const PromptPlace &u, int g) {
  const int from = 2 * u.r * p.tile;
  if (from + p.tile < u.len) return from + g * p.tile;
  return ((u.h ^ u.b) & 1) == g ? from : u.len;
}
// Token tiles that it sees.
__device__ __forceinline__ int prompt_group_tiles(const PromptParams &p, const PromptPlace &u, int g) {
  const int from = prompt_from(p, u, g);
  return from >= u.len ? 0 : (min(from + p.tile, u.len) + PT - 1) / PT;
}
// Tokens of tile j in sixteens: the products stop there.
__device__ __forceinline__ int prompt_sixteens(const PromptPlace &u, int j) { return (min(PT, u.len - j * PT) + 15) / 16; }
// The first token tile that some row of the pair does not see all of.
__device__ __forceinline__ int prompt_first_edge(const PromptParams &p, const PromptPlace &u) { return (2 * u.r * p.tile + 1) / PT; }

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return DT == DT_BF16 ? f32_to_bf16x2(lo, hi) : f32_to_f16x2(lo, hi);
}

// 64 bytes of a row.  A store instruction takes a clock for each of its 32 rows,
// so there are two of 32 bytes where the address allows it, not four.
__device__ __forceinline__ void store64(void *to, const uint32_t *y, bool wide) {
#pragma unroll
  for (int i = 0; i < 16; i += 8) {
    uint32_t *at = static_cast<uint32_t *>(to) + i;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(y[i]), "r"(y[i + 1]), "r"(y[i + 2]), "r"(y[i + 3]),
                   "r"(y[i + 4]), "r"(y[i + 5]), "r"(y[i + 6]), "r"(y[i + 7])
                   : "memory");
    } else {
      reinterpret_cast<uint4 *>(at)[0] = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
      reinterpret_cast<uint4 *>(at)[1] = make_uint4(y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
    }
  }
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
               "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
               "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
               : "memory");
}

// A persistent CTA per SM takes an equal stretch of the list of all (sequence,
// group of heads, pair of row tiles, token tile).  Segments that several CTAs
// share leave pieces (out, offset, sum), which the last CTA to arrive joins in
// index order, so results do not depend on timing.
//
//   copies    Q of both row tiles, K and V tiles, as swizzled operands (TMA)
//   products  S = Q K^T, O += P V (P in tensor memory; head size 128: over S), A and B in turn
//   softmax   a thread per row: S -> P under the running offset; the output
//   values    looks for values that are not finite where some row does not see
//             all of the tile: 0 * inf is not 0.  They are taken out, and marked
//             with their token, and rows that see them get them at the end.
//
// What bounds it is a row tile's chain: scores to weights 1130 clocks (512 of
// exponentials), 130 to 250 to the products' warp, 900 for the issue of 16
// products, 400 until the scores are there; two row tiles share it, a pair of
// tiles every 2600 clocks, of which the products need 2048.  One prompt of 16384
// tokens, 32 heads on 8: 1535 to 1640 us with the power limit of the card, 1340 to
// 1433 TFLOP/s; 8 of 2048: 254 to 278 us, 990 to 1083 TFLOP/s.  Head size 64 has half
// of the products, but the same softmax; its weights have columns of their own, and
// the next scores are multiplied before them: 1254 to 1282 us, 858 to 877 TFLOP/s.
// (1217 to 1225 with offsets of one number, which do not do for large scores; 1350
// beside that with weights over the scores as for 128.)  12 bytes a thread are
// stored to local memory and 104 loaded.  A segment's begin and end cost about two
// token tiles.
// Measured and dropped (the prompt of 16384, us): output threads of their own,
// 512 threads of 128 registers, 1656; half of the weights stored and multiplied
// at a time 1806; all of a tile's scores in registers 1932 (spills).  For head size
// 64, beside 1225: two score buffers of 64 tokens a row tile 1627 (twice the steps),
// the next scores already under the last quarter of the weights 1279 to 1336
// (spills), no turns 1449.
template <int D, int DT>
__global__ void __launch_bounds__(P_NT, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using L = PromptLayout<D>;
  // Head size 64 leaves tensor memory for weights of their own (64 columns a row
  // tile), so the next scores come before the weights' product, not after it.
  constexpr bool APART = D == 64;
  extern __shared__ __align__(1024) unsigned char psm[];
  __shared__ unsigned s_scan[P_NT / 32];
  __shared__ int s_seq[2], s_last[2];
  __shared__ unsigned s_base[2], s_segs[2];
  PromptBars &bar = *reinterpret_cast<PromptBars *>(psm + L::BARS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float NINF = __uint_as_float(0xff800000u), QNAN = __uint_as_float(0x7fc00000u);
  pdl_wait();
  pdl_launch_dependents();

  // ---- the list of all work, and this CTA's stretch of it
  int wrong = 0, longer = 0;
#pragma unroll 1
  for (int b = tid; b <= p.B; b += P_NT) {
    const int s = p.starts[b], e = b < p.B ? p.starts[b + 1] : s;
    wrong |= s < 0 || e < s || e > p.T;
    longer |= e - s > P_SHORT * PT;
  }
  wrong = __syncthreads_or(wrong);
  const bool shared = __syncthreads_or(longer);
  // Work is counted in token tiles.  Where all segments are short they stay
  // whole, each with the CTA that has most of it, and count their begin and end
  // too: pieces and their joining cost about ten token tiles.  (One prompt of
  // 512 tokens 16 us, 32 shared; of 2048 tokens 54 and 67.)
  const int extra = shared ? 0 : P_EXTRA;
  const auto pairs_of = [&](int len) -> unsigned { return (len + 2 * p.tile - 1) / (2 * p.tile); };
  const auto length_of = [&](int b) { return b < p.B && !wrong ? p.starts[b + 1] - p.starts[b] : 0; };
  const auto work_of = [&](int b) -> unsigned {
    const int len = length_of(b);
    return (prompt_head_tiles(p, len) + extra * pairs_of(len)) * p.heads;
  };
  unsigned total = 0, w = 0, upto = 0;  // upto: of all sequences up to this thread's (of the last block of them)
  for (int b0 = 0; b0 < p.B; b0 += P_NT) {
    unsigned sum;
    w = work_of(b0 + tid);
    upto = total + block_scan<P_NT / 32>(w, s_scan, sum);
    total += sum;
  }
  {  // rows of no sequence
    const long long row = static_cast<long long>(p.Hq) * D / 8, lo = wrong ? 0 : p.starts[0], hi = wrong ? 0 : p.starts[p.B];
    const float v = wrong ? QNAN : 0.f, x[8] = {v, v, v, v, v, v, v, v};
    const Raw8<DT> raw = pack8<DT>(x);
    const long long step = static_cast<long long>(gridDim.x) * P_NT, me = static_cast<long long>(blockIdx.x) * P_NT + tid;
    for (long long i = me; i < lo * row; i += step) store8<DT, true>(p.out, i * 8, raw);
    for (long long i = hi * row + me; i < p.T * row; i += step) store8<DT, true>(p.out, i * 8, raw);
    if (p.lse) {
      for (long long i = me; i < lo * p.Hq; i += step) p.lse[i] = wrong ? v : NINF;
      for (long long i = hi * p.Hq + me; i < static_cast<long long>(p.T) * p.Hq; i += step) p.lse[i] = wrong ? v : NINF;
    }
  }
  if (wrong && blockIdx.x == 0 && tid == 0) atomicOr(p.status, ST_LENGTH);
  const unsigned nc = wrong ? 0 : min(gridDim.x, total);
  if (blockIdx.x >= nc) return;
  const Share share(total, nc);
  const unsigned cut[2] = {share.start(blockIdx.x), share.start(blockIdx.x + 1)};
  unsigned before = 0, segs_before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += P_NT) {
    unsigned sum, segs = 0;
    if (p.B > P_NT) {
      w = work_of(b0 + tid);
      upto = before + block_scan<P_NT / 32>(w, s_scan, sum);
      before += sum;
    }
    if (!shared) {
      const unsigned mine = pairs_of(length_of(b0 + tid)) * p.heads;
      segs = segs_before + block_scan<P_NT / 32>(mine, s_scan, sum) - mine;
      segs_before += sum;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (cut[e] < upto && cut[e] >= upto - w) s_seq[e] = b0 + tid, s_base[e] = upto - w, s_segs[e] = segs;
  }
  __syncthreads();
  // The place of cut e, and how many token tiles of all sequences come before.
  const auto place_of = [&](int e, unsigned &tiles) {
    PromptPlace u;
    u.b = s_seq[e];
    prompt_enter(p, u);
    unsigned r = cut[e] - s_base[e];
    const unsigned pairs = pairs_of(u.len), head = prompt_head_tiles(p, u.len) + extra * pairs;
    u.h = static_cast<int>(r / head);
    r -= u.h * head;
    unsigned lo = 0, hi = pairs;  // the last pair that starts at or before r
    while (hi - lo > 1) {
      const unsigned mid = (lo + hi) >> 1;
      if (prompt_tiles_before(p, mid) + extra * mid <= r) lo = mid;
      else hi = mid;
    }
    u.r = static_cast<int>(lo);
    u.n = prompt_pair_tiles(p, u.len, u.r);
    u.j = static_cast<int>(r - prompt_tiles_before(p, lo) - extra * lo);
    tiles = cut[e];
    if (!shared) {
      tiles -= u.j + extra * (s_segs[e] + u.h * pairs + lo);
      if (u.j && 2 * u.j >= u.n + extra) {  // from the next segment on
        tiles += u.n;
        u.j = u.n;
      } else {
        u.j = 0;
      }
    }
    return u;
  };
  unsigned my0, my1;
  PromptPlace at = place_of(0, my0);
  if (shared) my1 = cut[1];
  else if (cut[1] < total) place_of(1, my1);
  else my1 = total - extra * segs_before;
  if (my0 >= my1) return;
  if (at.j == at.n) prompt_next(p, at);
  const int count = static_cast<int>(my1 - my0);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], 1), mbar_init(&bar.k_empty[i], 2);
      mbar_init(&bar.v_full[i], 1), mbar_init(&bar.v_empty[i], 3), mbar_init(&bar.v_seen[i], 1);
      mbar_init(&bar.q_full[i], 1), mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1), mbar_init(&bar.p_full[i], 4), mbar_init(&bar.o_done[i], 1), mbar_init(&bar.turn[i], 1);
    }
    mbar_arrive(&bar.turn[0]);  // A begins
    fence_mbar_init();
    bar.marked = 0;
    for (int i = 0; i < P_SOFT / 32; ++i) bar.ended[i] = 0;
  }
  if (warp == P_SOFT / 32) tmem_alloc(&bar.tmem, 512);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&bar.tmem);

  // a wait that ran out: the role goes on without waiting, its loops end, and
  // the call reports a timeout
  bool lost = false;
  const auto wait = [&](uint64_t *b, uint32_t parity) {  // warp-wide
    if (!lost && !__all_sync(0xffffffffu, tile_wait<0>(b, parity))) lost = true;
  };
  const auto wait2 = [&](uint64_t *b, uint32_t parity, uint64_t *c, uint32_t parity_c) {  // both: the polls overlap
    if (lost) return;
    bool done = false;
#pragma unroll 1
    for (int polls = 0; polls < 1 << 20 && !done; ++polls) {
      const bool x = mbar_try_wait(b, parity), y = mbar_try_wait(c, parity_c);
      done = __all_sync(0xffffffffu, x && y);
    }
    lost = !done;
  };
  const auto lazy_wait = [&](uint64_t *b, uint32_t parity) {  // where latency hides
    if (!lost && !__all_sync(0xffffffffu, tile_wait<100>(b, parity))) lost = true;
  };
  const auto one = [&](uint64_t *b, uint32_t parity) {  // a single thread
    if (!lost && !tile_wait<0>(b, parity)) lost = true;
  };

  if (warp < P_SOFT / 32) {
    // ------------------------------------------------------------ softmax
    more_registers<P_REG_SOFT>();
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane field of the addresses
    const uint32_t tS = tmem + lanes + g * PT, tO = tmem + lanes + 256 + g * D, tP = APART ? tmem + lanes + 384 + g * 64 : tS;
    const int tok_in = r / p.G, head_in = r - tok_in * p.G, first_in = 32 * (warp & 3) / p.G;  // first_in: of the warp's first row
    // scores times f; a scale of zero as the least number, so that a hidden
    // column's infinite score stays infinite
    const float f = p.scale_log2 == 0.f ? __uint_as_float(1u) : p.scale_log2;
    const uint32_t flip = f < 0.f ? 0x80000000u : 0u, hidden = 0xff800000u ^ flip;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t uses = 0, outs = 0;  // tiles of this group, its segments whose output has been awaited
    // The output of a segment waits for its last products, so it is read only
    // after the next segment's first weights have been made, and written while
    // the products with them run.
    // What it takes then lies in shared memory.
    PromptLast &last = reinterpret_cast<PromptLast *>(psm + L::LAST)[tid];
    bool there = false;
    // `between` runs as soon as O has been read.
    const auto output = [&](auto between) {
      const bool any = last.any;  // it had tiles
      const int *mark = reinterpret_cast<const int *>(psm + L::MARKS);
      if (any) {
        wait(&bar.o_done[g], (APART ? uses - 1 : outs) & 1);
        ++outs;
        tc_after_sync();
      }
      const bool marked = *reinterpret_cast<const volatile int *>(&bar.marked) == last.seg + 1;
      const float inv = last.whole ? 1.f / last.l : 1.f;
      if (any && last.whole && !marked) {
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          uint32_t ob[32];  // the output's row in its type
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + c + 32 * q, o);
            tc_wait_ld32(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) ob[16 * q + e] = pack2<DT>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          }
          tc_before_sync();
          if (c + 64 == D) between();
          if (last.live)
#pragma unroll
            for (int q = 0; q < 2; ++q) store64(static_cast<uint16_t *>(p.out) + last.row * D + c + 32 * q, ob + 16 * q, wide);
          __syncwarp();
        }
      } else if (any) {
        float *const piece = p.pieces + ((static_cast<long long>(blockIdx.x) * 2 + last.which) * 2 + g) * L::PIECE;
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t o[16];
          __syncwarp();
          tmem_ld16(tO + 16 * q, o);
          tc_wait_ld(o);
          float z[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            z[e] = __uint_as_float(o[e]) * inv;
            if (marked) {  // values that are not finite, for the rows that see them
              const int d = 16 * q + e;
              if (last.tok >= mark[D + d]) z[e] += INFINITY;
              if (last.tok >= mark[2 * D + d]) z[e] -= INFINITY;
              if (last.tok >= mark[d]) z[e] = QNAN;
            }
          }
          if (!last.live) continue;
          if (last.whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              const float x[8] = {z[e], z[e + 1], z[e + 2], z[e + 3], z[e + 4], z[e + 5], z[e + 6], z[e + 7]};
              store8<DT, true>(p.out, last.row * D + 16 * q + e, pack8<DT>(x));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              reinterpret_cast<float4 *>(piece)[(4 * q + e / 4) * PT + r] = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
          }
        }
        tc_before_sync();
        between();
      } else {
        between();
      }
      float *const piece = p.pieces + ((static_cast<long long>(blockIdx.x) * 2 + last.which) * 2 + g) * L::PIECE;
      if (last.live) {
        if (last.whole) {
          if (p.lse) p.lse[last.row] = (last.m + (last.lo + log2f(last.l))) * 0.6931471805599453f;
        } else {
          if (!any)  // nothing that this row tile sees
            for (int k = 0; k < D / 4; ++k) reinterpret_cast<float4 *>(piece)[k * PT + r] = make_float4(0.f, 0.f, 0.f, 0.f);
          piece[PT * D + r] = last.m, piece[PT * D + PT + r] = last.l, piece[PT * D + 2 * PT + r] = last.lo;
        }
      }
      if (!last.whole) {
        // a segment that several CTAs share: the last to arrive joins, in order
        const int c0 = last.first, n = last.n;
        __threadfence();
        named_sync(1 + g, 128);
        if (r == 0) {
          s_last[g] = atomicAdd(p.done + 2 * c0 + g, 1) == n - 1;
          __threadfence();
        }
        named_sync(1 + g, 128);
        if (*reinterpret_cast<volatile int *>(&s_last[g])) {
          __threadfence();
          if (last.live) {
            const auto part = [&](int e) { return p.pieces + ((static_cast<long long>(c0 + e) * 2 + (e == 0 ? 1 : 0)) * 2 + g) * L::PIECE; };
            float M = NINF, low = 0.f, sum = 0.f;
#pragma unroll 4
            for (int e = 0; e < n; ++e) M = fmaxf(M, __ldcg(part(e) + PT * D + r));
            const bool far = fabsf(M) > P_FAR / 2;  // otherwise a piece whose offset is two numbers counts nothing
            if (__builtin_expect(far, 0)) {  // the largest second number beside the first one
              low = NINF;
              for (int e = 0; e < n; ++e)
                if (__ldcg(part(e) + PT * D + r) == M) low = fmaxf(low, __ldcg(part(e) + PT * D + 2 * PT + r));
            }
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {  // 32 columns at a time: eight loads a piece, of two pieces, on their way together
              float4 z[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) z[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              sum = 0.f;
#pragma unroll 2
              for (int e = 0; e < n; ++e) {
                const float *from = part(e);
                float x0 = __ldcg(from + PT * D + r) - M;  // every row sees a token
                if (__builtin_expect(far, 0)) x0 += __ldcg(from + PT * D + 2 * PT + r) - low;
                const float a = ex2(x0), le = __ldcg(from + PT * D + PT + r);
                float4 x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = __ldcg(reinterpret_cast<const float4 *>(from) + (8 * q + k) * PT + r);
                sum = fmaf(a, le, sum);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  z[k].x = fmaf(a, x[k].x, z[k].x), z[k].y = fmaf(a, x[k].y, z[k].y);
                  z[k].z = fmaf(a, x[k].z, z[k].z), z[k].w = fmaf(a, x[k].w, z[k].w);
                }
              }
              const float over = 1.f / sum;
              uint32_t y[16];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[2 * k] = pack2<DT>(z[k].x * over, z[k].y * over), y[2 * k + 1] = pack2<DT>(z[k].z * over, z[k].w * over);
              store64(static_cast<uint16_t *>(p.out) + last.row * D + 32 * q, y, wide);
            }
            if (p.lse) p.lse[last.row] = (M + (low + log2f(sum))) * 0.6931471805599453f;
          }
          if (r == 0) p.done[2 * c0 + g] = 0;  // zero again for the next call
        }
        named_sync(1 + g, 128);  // s_last may be written again
      }
      there = false;
    };
    const auto ended = [&](int seg) {  // segments that are done with
      __syncwarp();
      if (lane == 0) *reinterpret_cast<volatile int *>(&bar.ended[warp]) = seg;
    };
    for (int i = 0, seg = 0;; ++seg) {
      // tiles s0 .. mine - 1; after the last segment none, to write the last output
      const bool over = i >= count;
      const int s0 = over ? 0 : at.j, end = over ? 0 : min(at.n, s0 + count - i), mine = over ? 0 : min(end, prompt_group_tiles(p, at, g));
      const int from = prompt_from(p, at, g), tok = from + tok_in;
      const bool live = tok_in < p.tile && tok < at.len;
      float m = NINF, lo = 0.f, l = 0.f;  // offset (two numbers beyond P_FAR), sum
      float less = 0.f;                   // exponents are score * f - less
      bool look = true;                   // while some row has no offset yet, or one beyond P_FAR
      const uint32_t uses0 = uses;
      for (int j = s0; j < mine || there; ++j) {
        const auto weighed = [&]() {
          __syncwarp();
          if (j < mine && lane == 0) mbar_arrive(&bar.p_full[g]);
        };
        if (j < mine) {
        wait(&bar.s_full[g], uses & 1);
        tc_after_sync();
        const int lim = tok - j * PT;  // the last column that the row sees
        const bool edge = from + first_in < j * PT + PT - 1;
        const auto hide = [&](uint32_t (&s)[32], int q) {
          if (__builtin_expect(edge, 0)) {
            const int n = lim + 1 - 32 * q;
            const uint32_t bits = n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;  // the columns that the row sees
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1)) s[e] = hidden;
          }
        };
        const auto largest = [&]() {  // of the scores, turned around for a negative scale
          float top = NINF;
#pragma unroll 1
          for (int q = 0; 32 * q < at.len - j * PT && q < 4; ++q) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * q, s);
            tc_wait_ld32(s);
            hide(s, q);
#pragma unroll
            for (int e = 0; e < 32; e += 2) top = fmaxf(fmaxf(top, __uint_as_float(s[e] ^ flip)), __uint_as_float(s[e + 1] ^ flip));
          }
          return top;
        };
        float sum = 0.f;
        const auto exponent = [&](float top) { return __fmul_rn(top, fabsf(f)); };
        // The offset to P_UP below the tile's largest exponent, if that is above it and
        // the row's own sum or offset asks for it: no row changes another's bits.
        const auto rise = [&]() {
          const float top = largest();
          float nm = exponent(top), nl = 0.f, a = 1.f;
          if (fabsf(nm) > P_FAR && nm != NINF) {  // the product, and what it was rounded by
            nl = fmaf(top, fabsf(f), -nm);
            if (fabsf(nl) < P_FAR / 16) nl -= P_UP<DT>;  // beyond, all weights are 1 or 0
          } else {
            nm = __fsub_rn(nm, P_UP<DT>);
          }
          const float up = (nm - m) + (nl - lo);
          const bool own = !(sum <= P_MOST<DT>) || fabsf(m) > P_FAR;
          if (own && nm > NINF && !(up <= 0.f)) a = ex2(-up), m = nm, lo = nl;  // NaN for an infinite score
          l *= a;
          if (uses != uses0) {  // O holds the products of this segment's earlier tiles
            if (APART) {  // elsewhere they are done before the scores
              wait(&bar.o_done[g], (uses - 1) & 1);
              tc_after_sync();
            }
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * q, o);
              tc_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st16(tO + 16 * q, o);
            }
          }
          look = __any_sync(0xffffffffu, live && !(fabsf(m) <= P_FAR));
          less = m == NINF ? 0.f : m;
          if (__builtin_expect(!look, 1)) return;
          // where offsets are two numbers, exponents, over f, take the scores' place
          const float over = 1.f / f;
          const bool two = fabsf(m) > P_FAR;
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t s[16];
            tmem_ld16(tS + 16 * q, s);
            tc_wait_ld(s);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (two) s[e] = __float_as_uint((fmaf(__uint_as_float(s[e]), f, -less) - lo) * over);
            tmem_st16(tS + 16 * q, s);
          }
          tc_wait_st();
          if (two) less = 0.f;
        };
        uint32_t pk[64];  // in the inputs' type
        const auto weights = [&]() {
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t s[2][32];
          tmem_ld32(tS, s[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tc_wait_ld32(s[q & 1]);
            if (q < 3) tmem_ld32(tS + 32 * (q + 1), s[(q + 1) & 1]);
            hide(s[q & 1], q);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 x = fma2(make_float2(__uint_as_float(s[q & 1][e]), __uint_as_float(s[q & 1][e + 1])), make_float2(f, f), make_float2(-less, -less));
              x.x = ex2(x.x), x.y = ex2(x.y);
              part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], x);
              pk[16 * q + e / 2] = pack2<DT>(x.x, x.y);
            }
          }
          const float2 both = add2(part[0], part[1]);
          sum = both.x + both.y;
        };
        // The offset is found in the first tile where a row has a score above -inf, and
        // moves where a sum tells that some weight is above 2^8.8 (2^-24.2 for bf16), or
        // in every tile where offsets are two numbers.  After that no sum is looked at:
        // there is no third pass.
        float limit = P_MOST<DT>;
        if (look) {
          const float here = __fsub_rn(exponent(largest()), P_UP<DT>), top = m == NINF ? here : m;
          look = __any_sync(0xffffffffu, live && fabsf(top) > P_FAR / 2 && top != NINF);
          if (__builtin_expect(look, 0)) {
            limit = -1.f;
          } else {
            m = top;
            less = m == NINF ? 0.f : m;
            look = __any_sync(0xffffffffu, live && m == NINF);
          }
        }
#pragma unroll 1
        for (;;) {
          weights();
          if (__builtin_expect(!__any_sync(0xffffffffu, live && sum > limit), 1)) break;
          rise();
          limit = INFINITY;
        }
        l += sum;
        if (APART && uses) {  // the weights before these have been multiplied
          wait(&bar.o_done[g], (uses - 1) & 1);
          tc_after_sync();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st16(tP + 16 * q, pk + 16 * q);  // weights, if not apart over scores that have been read
        tc_wait_st();
        tc_before_sync();
        }
        if (__builtin_expect(!there, 1)) {
          weighed();
        } else {
          output(weighed);
          ended(seg);
        }
        if (j < mine) ++uses;
      }
      if (over) break;
      // ---- the end of the segment
      last.any = mine > s0, last.live = live, last.whole = s0 == 0 && end == at.n;
      last.seg = seg, last.tok = tok, last.which = s0 > 0 ? 0 : 1;
      last.m = m, last.lo = lo, last.l = l;
      last.row = static_cast<long long>(at.start + tok) * p.Hq + at.h * p.G + head_in;
      if (!last.whole) {
        const unsigned f0 = my0 + i - s0;
        last.first = share.holder(f0);
        last.n = static_cast<int>(share.holder(f0 + at.n - 1)) - last.first + 1;
      }
      there = last.any || (from < at.len && !last.whole);
      if (!there) ended(seg + 1);
      i += end - s0;
      if (i < count) prompt_next(p, at);
    }
  } else {
    fewer_registers<P_REG_REST>();
    const int role = warp - P_SOFT / 32;
    if (role == 0) {
      // ------------------------------------------------------------ copies
      if (lane == 0) {
        const uint32_t sm = smem_u32(psm);
        const int kv_bytes = L::OP, q_bytes = p.tile * p.G * D * 2;
        uint32_t q_uses[2] = {0, 0};
        PromptPlace u = at;
        int s0 = u.j, issued = 0;
        for (int i = 0; i < count; ++i) {
          const uint32_t s = i & 1, ph = (i >> 1) & 1;
          const int row = u.start + u.j * PT, kv = u.h / p.per_kv;
          one(&bar.k_empty[s], ph ^ 1);
          if (lost) break;
          mbar_arrive_expect_tx(&bar.k_full[s], kv_bytes);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) tma_load(sm + L::K + s * L::OP + x * 16384, &p.k, 64 * x, kv, row, &bar.k_full[s]);
          if (u.j == s0)
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              if (s0 >= prompt_group_tiles(p, u, g)) continue;
              one(&bar.q_empty[g], (q_uses[g] & 1) ^ 1);
              if (lost) break;
              ++q_uses[g];
              mbar_arrive_expect_tx(&bar.q_full[g], q_bytes);
#pragma unroll
              for (int x = 0; x < D / 64; ++x)
                tma_load(sm + L::Q + g * L::OP + x * 16384, &p.q, 64 * x, 0, u.h, u.start + prompt_from(p, u, g), &bar.q_full[g]);
            }
          if (!lost) one(&bar.v_empty[s], ph ^ 1);
          if (lost) {
            issued = 2 * i + 1;
            break;
          }
          mbar_arrive_expect_tx(&bar.v_full[s], kv_bytes);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) tma_load(sm + L::V + s * L::OP + x * 16384, &p.v, 64 * x, kv, row, &bar.v_full[s]);
          issued = 2 * i + 2;
          if (++u.j == u.n && i + 1 < count) prompt_next(p, u), s0 = 0;
        }
        // no copy outlives the CTA, even after a wait that ran out
        const bool was = lost;
        lost = false;
        for (int k = max(0, issued - 4); k < issued; ++k) one(k & 1 ? &bar.v_full[(k >> 1) & 1] : &bar.k_full[(k >> 1) & 1], (k >> 2) & 1);
        for (int g = 0; g < 2; ++g)
          if (q_uses[g]) one(&bar.q_full[g], (q_uses[g] - 1) & 1);
        lost |= was;
      }
    } else if (role <= 2) {
      // ---------------------------------------------------------- products
      // A warp for each row tile.  They take turns: PV of a tile and S of the
      // next tile (with P apart the other way round) for A, then for B, so that one row tile's softmax runs under
      // the other's products; without turns the products mix, both row tiles
      // wait for both, and their softmaxes run at the same time.  What a warp
      // waits for, and its arrivals, pass under the other's products.
      constexpr uint32_t TYPE = DT == DT_BF16 ? 1u << 7 | 1u << 10 : 0u;
      constexpr uint32_t ID_S = TYPE | 1u << 4 | (PT / 16) << 24;  // without the columns
      constexpr uint32_t ID_O = TYPE | 1u << 4 | 1u << 16 | (D / 8) << 17 | (PT / 16) << 24;  // values run along the tokens
      const int g = role - 1;
      const uint32_t sm = smem_u32(psm), tS = tmem + g * PT, tO = tmem + 256 + g * D, tP = APART ? tmem + 384 + g * 64 : tS;
      const uint64_t dQ = tc_desc(sm + L::Q + g * L::OP, 0), dK0 = tc_desc(sm + L::K, 0), dV0 = tc_desc(sm + L::V, 16384);
      uint32_t uses = 0, q_uses = 0, seen[2] = {0, 0};
      PromptPlace next = at;
      int j = 0, sixteens = 0, tiles = 0, coming = prompt_group_tiles(p, next, g);  // of tile i's pair, of the next one's
      int edge = 0, coming_edge = prompt_first_edge(p, next);
      for (int i = -1; i < count; ++i) {
        const uint32_t s = i & 1, t = (i + 1) & 1;
        const uint64_t dV = dV0 + (s * L::OP >> 4), dK = dK0 + (t * L::OP >> 4);
        const bool more = i + 1 < count, has_v = i >= 0 && j < tiles, has_k = more && next.j < coming;
        if (more) wait(&bar.k_full[t], ((i + 1) >> 1) & 1);
        if (has_k && (i < 0 || next.j == 0)) wait(&bar.q_full[g], q_uses & 1), ++q_uses;
        if (i >= 0) {
          wait(&bar.v_full[s], (i >> 1) & 1);
          if (j >= edge) wait(&bar.v_seen[s], seen[s] & 1), ++seen[s];
        }
        if (has_v) wait2(&bar.turn[g], (i + 1) & 1, &bar.p_full[g], uses & 1), ++uses;
        else wait(&bar.turn[g], (i + 1) & 1);
        tc_after_sync();
        const int six_v = sixteens;
        sixteens = prompt_sixteens(next, next.j);
        const auto weighted = [&]() {
          if (six_v == PT / 16) {
#pragma unroll
            for (int k = 0; k < PT / 16; ++k)  // 16 tokens at a time
              tc_mma_ts_warp(tO, tP + 8 * k, dV + (k * 2048 >> 4), ID_O, k > 0 || (i > 0 && j > 0));
          } else {
#pragma unroll 1
            for (int k = 0; k < six_v; ++k) tc_mma_ts_warp(tO, tP + 8 * k, dV + (k * 2048 >> 4), ID_O, k > 0 || (i > 0 && j > 0));
          }
        };
        const auto scores = [&]() {
          const auto off = [](int k) -> uint64_t { return ((k >> 2) * 16384 + (k & 3) * 32) >> 4; };  // 32 bytes of the rows at a time, 16384 between panels
          if (sixteens == PT / 16) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) tc_mma_ss_warp(tS, dQ + off(k), dK + off(k), ID_S | (PT / 8) << 17, k > 0);
          } else {
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) tc_mma_ss_warp(tS, dQ + off(k), dK + off(k), ID_S | static_cast<uint32_t>(2 * sixteens) << 17, k > 0);
          }
        };
        const auto scores_end = [&]() {
          if (has_k) {
            tc_commit_warp(&bar.s_full[g]);
            tc_commit_warp(&bar.k_empty[t]);
            if (next.j + 1 == coming) tc_commit_warp(&bar.q_empty[g]);
          } else if (more) {
            mbar_arrive_warp(&bar.k_empty[t]);
          }
        };
        if (APART) {
          if (has_k) scores();
          scores_end();
          if (has_v) {
            weighted();
            tc_commit_warp(&bar.o_done[g]);
          }
          mbar_arrive_warp(&bar.turn[g ^ 1]);
        } else {
          // o_done: once a segment, for its output.  A phase for every tile could be
          // taken for the one after it, since the softmax does not wait for the tiles
          // before: those products are done when the scores issued after them are.
          if (has_v) {
            weighted();
            if (j + 1 == tiles || !has_k) tc_commit_warp(&bar.o_done[g]);
          }
          if (has_k) scores();
          mbar_arrive_warp(&bar.turn[g ^ 1]);
          scores_end();
        }
        if (has_v) tc_commit_warp(&bar.v_empty[s]);
        else if (i >= 0) mbar_arrive_warp(&bar.v_empty[s]);
        j = next.j, tiles = coming, edge = coming_edge;
        if (++next.j == next.n && i + 2 < count) {
          prompt_next(p, next);
          coming = prompt_group_tiles(p, next, g);
          coming_edge = prompt_first_edge(p, next);
        }
      }
    } else {
      // ------------------------------------------------------------ values
      constexpr uint32_t EXP = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
      PromptPlace u = at;
      int *const mark = reinterpret_cast<int *>(psm + L::MARKS);
      int seg = 0;
      for (int i = 0; i < count; ++i) {
        const uint32_t s = i & 1, ph = (i >> 1) & 1;
        lazy_wait(&bar.v_full[s], ph);
        if (u.j >= prompt_first_edge(p, u)) {
          unsigned char *const tile = psm + L::V + s * L::OP;
          // rows that are not seen by all, up to where the products stop
          const int r0 = max(0, 2 * u.r * p.tile + 1 - u.j * PT), r1 = 16 * prompt_sixteens(u, u.j);
          uint32_t most = 0;
          const unsigned char *from = tile + lane / 8 % (D / 64) * 16384 + lane % 8 * 16;
          constexpr int STEP = 256 / D;  // rows at a time
#pragma unroll 4
          for (int row = r0 + lane / (D / 8); row < r1; row += STEP) {
            const uint4 x = lds128(from + row * 128);
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(x.x & 0x7fff7fffu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(x.y & 0x7fff7fffu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(x.z & 0x7fff7fffu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(x.w & 0x7fff7fffu));
          }
          if (__any_sync(0xffffffffu, (most & 0xffffu) >= EXP || (most >> 16) >= EXP)) {
            volatile int *const marked = &bar.marked, *const ended = bar.ended;
            if (*marked != seg + 1) {  // the marks of an earlier segment may still be read
              for (int polls = 0; !lost && !__all_sync(0xffffffffu, ended[lane % (P_SOFT / 32)] >= seg); ++polls) {
                __nanosleep(100);
                lost = polls > 1 << 18;
              }
              for (int d = lane; d < 3 * D; d += 32) mark[d] = INT32_MAX;
              __syncwarp();
              if (lane == 0) *marked = seg + 1;
            }
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < L::OP / 64; ++k) {  // two elements at a time: panel, row, swizzled chunk of eight
              uint32_t *const word = reinterpret_cast<uint32_t *>(tile) + k * 16 + (lane & 15);
              const int byte = (k * 16 + (lane & 15)) * 4, panel = byte >> 14, row = (byte >> 7) & 127;
              const int d0 = panel * 64 + ((((byte >> 4) & 7) ^ (row & 7)) << 3) + ((byte & 15) >> 1);
              const uint32_t x = *word;
              uint32_t y = x;
              if (lane < 16) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t half = (x >> (16 * e)) & 0xffffu, size = half & 0x7fffu;
                  if (size < EXP) continue;
                  y &= e ? 0x0000ffffu : 0xffff0000u;
                  const int kind = size > EXP ? 0 : half & 0x8000u ? 2 : 1;
                  atomicMin(&mark[kind * D + d0 + e], u.j * PT + row);
                }
                if (y != x) *word = y;
              }
            }
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.v_seen[s]);
        }
        // also where there was nothing to look at: a warp that let phases pass
        // could take one for another
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_empty[s]);
        if (++u.j == u.n && i + 1 < count) prompt_next(p, u), ++seg;
      }
    }
  }
  if (lost) atomicOr(p.status, ST_TIMEOUT);
  tc_before_sync();
  __syncthreads();
  if (warp == P_SOFT / 32) {
    tc_after_sync();
    tmem_free(tmem, 512);
  }
}

// Rows that the copies cannot take as they lie (not 16-byte aligned, or their
// strides are not), to [T, H, D].
struct PackParams {
  const uint16_t *src;
  long long sn, sh;  // strides in elements
  uint16_t *dst;
  int T, H, D;
};
__global__ void __launch_bounds__(256) prompt_pack_kernel(const __grid_constant__ PackParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const long long n = static_cast<long long>(p.T) * p.H * p.D;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const long long row = i / p.D;
    p.dst[i] = p.src[row / p.H * p.sn + row % p.H * p.sh + i % p.D];
  }
}

}  // namespace spec
