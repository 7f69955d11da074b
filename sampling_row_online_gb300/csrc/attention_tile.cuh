// Attention over the 8-bit cache where a kv head has many query rows (chains
// times grouped heads, trees, parts of a prompt): tensor cores with the
// accumulators in tensor memory.  The mathematics is attention.cuh's.
#pragma once

#include "attention.cuh"

namespace spec {

// ------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t *at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Arrives on the barrier once all products issued so far by this thread are done.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// D (tensor memory, fp32) = A B^T (+ D): A in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// Columns of this warp's 32 lanes: thread = lane, register = column.  What a
// load names may be used after the wait that names it.
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Shared-memory operand of 128-byte swizzled rows (8 rows of 128 bytes to an
// atom of 1024); `lead` is the distance of neighbouring 64-element blocks where
// the rows run along the contracted axis (0 otherwise).
__device__ __forceinline__ uint64_t tc_desc(uint32_t at, uint32_t lead) {
  return static_cast<uint64_t>((at & 0x3ffffu) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// Generic writes to shared memory become visible to the tensor cores.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// ======================================================================
// A persistent CTA per SM.  The list of all work is (sequence, kv head, tile of
// 128 rows, tile of 128 tokens); every CTA takes an equal stretch of it.  Its
// tiles alternate between two groups of 256 softmax threads, A and B, each
// with its own scores, weights, accumulator, maximum and sum: they meet only at
// the end of a segment (a row tile of a kv head), so one group's softmax runs
// under the other's products.
//
//   copy warp    pages -> raw ring (bulk copies of 8-bit codes), scales -> ring
//   conversion   raw codes -> fp16 tiles in the swizzled operand layout
//   products     S = Q K^T, O += P V (P in tensor memory, over S)
//   softmax      two threads per row, half of the tokens each: S -> P, lazy
//                rescaling of O, the output
//
// Codes cannot be an operand next to fp16 (one instruction takes one type), and
// e4m3 queries and weights would cost the precision that the cache has.
//
// What bounds it is the dependent chain of a group's tile: scores, weights,
// products and the signals between them take about 5000 clocks for two tiles
// (1024 each of products, 1792 of shared-memory traffic), and the two groups run
// in phase, so that their weights slow each other down.  Every token tile is
// copied and converted once for each 128 rows of its kv head.  At these
// register counts it spills (382 bytes of stores and 520 of loads a thread at head
// size 128, 362 and 496 at 64).  32 trees of 63 nodes over up to 16384 tokens, 32
// heads on 8: 528 to 559 us over several GPUs, 730 to 772 TFLOP/s; 48 rows per
// head at up to 8192 tokens: 294 us, 2.8 TB/s; 1024 new tokens of 4 sequences
// behind 8192: 747 us, 782 TFLOP/s of what a chain sees.
constexpr int TQ = 128, TK = 128;    // rows, tokens of a tile
constexpr int T_SOFT = 512;          // softmax threads: two groups, two threads per row
constexpr int T_CONV = 256;          // conversion threads: half for keys, half for values, so that neither waits for the other's buffer
constexpr int T_NT = T_SOFT + T_CONV + 128;  // and a warp for each group's products, one for copies, an idle one
// Registers: 72 a thread at launch, then 88 for the softmax, 56 for the
// conversion and 40 for the rest: 512 * 88 + 256 * 56 + 128 * 40 = 896 * 72.
constexpr int T_REG = 72, T_REG_SOFT = 88, T_REG_CONV = 56, T_REG_REST = 40;
static_assert(T_SOFT * T_REG_SOFT + T_CONV * T_REG_CONV + 128 * T_REG_REST <= T_NT * T_REG, "register split");
constexpr int T_RAW = 4;             // raw slots: keys and values of two tiles
constexpr int T_SCALES = 8;          // tiles of scales: more than the copy warp can be ahead

// A bounded wait in a few instructions (the roles share the instruction cache
// and the issue slots, of which polls without a pause took half).  REST: the
// pause between polls, in nanoseconds.  The limit is in polls: tens of
// milliseconds at least.
template <int REST>
__device__ __forceinline__ bool tile_wait(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
  for (int polls = 0; polls < 1 << 20; ++polls) {
    if (mbar_try_wait(bar, parity)) return true;
    if (REST) __nanosleep(REST);
  }
  return false;
}
// A barrier of n threads of the CTA.  It has no limit: whoever gives up a wait
// goes on to every barrier all the same, without waiting again.
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void mbar_arrive_many(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

template <int D>
struct TileLayout {
  static constexpr int OP = 128 * D * 2;            // an fp16 operand tile
  static constexpr int RAWB = 128 * D;              // a raw tile
  static constexpr int Q = 0, K = OP, V = 3 * OP, RAW = 5 * OP;
  static constexpr int SCALES = RAW + T_RAW * RAWB;  // [T_SCALES][8] (key scale, log2 of the value scale)
  static constexpr int ML = SCALES + T_SCALES * 64;  // [4][128] floats: maxima that a row's threads exchange
  static constexpr int BARS = ML + 2048;
  static constexpr int MISC = BARS + 40 * 8;
  static constexpr int SMEM = MISC + 64;
  static constexpr int PIECE = 128 * D + 256;       // floats: out, offset, sum
};

struct TileBars {
  uint64_t raw_full[T_RAW], raw_empty[T_RAW], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2];
  uint64_t sc_full[T_SCALES], q_full[2];  // q_full: for each group's product warp, segments with a tile of the group
};
static_assert(sizeof(TileBars) <= 40 * 8, "barriers");

template <int V>
struct Number {
  static constexpr int value = V;
};
template <bool V>
struct Flag {
  static constexpr bool value = V;
};

struct TileCursor {
  int b, h, rt, j, n, tiles, ctx, cnt;  // n: token tiles of this row tile
};
__device__ __forceinline__ int token_tiles(const AttnParams &p, int ctx, int cnt, int rt) {
  // without a mask a row tile sees no further than its last node
  const int last = p.mask ? cnt : min(((rt + 1) * TQ - 1) / p.G + 1, cnt);
  return (ctx + last + TK - 1) / TK;
}
__device__ __forceinline__ void tile_enter(const AttnParams &p, TileCursor &u) {
  for (;; ++u.b) {
    const Seq s = sequence(p, u.b);
    if (s.cnt <= 0) continue;
    u.ctx = s.ctx, u.cnt = s.cnt;
    u.tiles = (s.cnt * p.G + TQ - 1) / TQ;
    return;
  }
}
__device__ __forceinline__ void tile_next(const AttnParams &p, TileCursor &u) {  // the next segment
  u.j = 0;
  if (++u.rt == u.tiles) {
    u.rt = 0;
    if (++u.h == p.c.Hk) {
      u.h = 0;
      ++u.b;
      tile_enter(p, u);
    }
  }
  u.n = token_tiles(p, u.ctx, u.cnt, u.rt);
}

// Sixteen codes as fp16, in order.
template <int KIND, bool SAFE>
__device__ __forceinline__ void codes_to_f16(uint4 w, uint4 &lo, uint4 &hi) {
  uint32_t u[4] = {w.x, w.y, w.z, w.w}, r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (KIND == KIND_E4M3) {
      if (SAFE) {  // any bits give finite numbers: rows past the last slot may hold anything
        r[2 * i] = e4m3_halves(prmt(u[i], 0, 0x1404));
        r[2 * i + 1] = e4m3_halves(prmt(u[i], 0, 0x3424));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r[2 * i]) : "r"(0x5c005c00u));  // 256
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r[2 * i + 1]) : "r"(0x5c005c00u));
      } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(r[2 * i]), "=r"(r[2 * i + 1])
            : "r"(u[i]));
      }
    } else {
      const uint32_t x = u[i] ^ 0x80808080u;
      r[2 * i] = prmt(x, 0x64646464u, 0x4140);
      r[2 * i + 1] = prmt(x, 0x64646464u, 0x4342);
      asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(r[2 * i]) : "r"(0x64806480u));
      asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(r[2 * i + 1]) : "r"(0x64806480u));
    }
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}
// A raw tile [128][D] into panels of 64 columns of 128-byte swizzled rows.
template <int D, int KIND, bool SAFE>
__device__ __forceinline__ void convert_tile(const unsigned char *raw, unsigned char *to, int tid) {
  constexpr int PER = D / 16, STEP = T_CONV / 2 / PER, BATCH = 4;  // rows per turn, turns loaded at once
  static_assert(STEP % 8 == 0 && 128 % (STEP * BATCH) == 0, "a thread's rows are equal modulo 8");
  // eight neighbouring lanes take four 16-byte pieces of an even row and four
  // of the odd row after it, in the other half where a row has two: their
  // loads and their stores touch every bank once
  const int odd = (tid >> 2) & 1, panel = D == 128 ? odd ^ ((tid >> 3) & 1) : 0, c = tid & 3;
  const int row = (D == 128 ? (tid >> 4) : (tid >> 3)) * 2 + odd;
  const unsigned char *from = raw + row * D + panel * 64 + c * 16;
  unsigned char *base = to + panel * 16384 + row * 128;
  unsigned char *first = base + ((2 * c) ^ (row & 7)) * 16, *second = base + ((2 * c + 1) ^ (row & 7)) * 16;
#pragma unroll 1
  for (int k0 = 0; k0 < 128; k0 += STEP * BATCH) {
    uint4 w[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) w[k] = lds128(from + (k0 + k * STEP) * D);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      uint4 x[2];
      codes_to_f16<KIND, SAFE>(w[k], x[0], x[1]);
      *reinterpret_cast<uint4 *>(first + (k0 + k * STEP) * 128) = x[0];
      *reinterpret_cast<uint4 *>(second + (k0 + k * STEP) * 128) = x[1];
    }
  }
}

template <int D, int KIND, int DT>
__global__ void __launch_bounds__(T_NT, 1) attn_tile_kernel(const __grid_constant__ AttnParams p) {
  using L = TileLayout<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  TileBars &bar = *reinterpret_cast<TileBars *>(smem + L::BARS);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::MISC);
  volatile int *s_last = reinterpret_cast<volatile int *>(smem + L::MISC + 4);
  int *s_seq = reinterpret_cast<int *>(smem + L::MISC + 8);
  volatile int *s_bad = reinterpret_cast<volatile int *>(smem + L::MISC + 32);  // [T_RAW]: a slot holds another page's rows
  unsigned *s_base = reinterpret_cast<unsigned *>(smem + L::MISC + 16);
  unsigned *s_scan = reinterpret_cast<unsigned *>(smem + L::ML);
  const CacheView &c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = T_NT / 32;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the list of all work, and this CTA's stretch of it
  int rest = 0;  // some sequence has rows that no tile writes
  const auto head_work = [&](int ctx, int cnt) -> unsigned {  // tiles of one kv head
    const int tiles = (cnt * p.G + TQ - 1) / TQ;
    if (p.mask) return static_cast<unsigned>(tiles) * token_tiles(p, ctx, cnt, 0);
    unsigned w = 0;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) w += token_tiles(p, ctx, cnt, t);
    return w;
  };
  const auto work_of = [&](int b) -> unsigned {
    if (b >= p.B) return 0;
    const Seq s = sequence(p, b);
    rest |= s.cnt != p.N;
    return s.cnt > 0 ? head_work(s.ctx, s.cnt) * c.Hk : 0;
  };
  unsigned total = 0, w = 0, upto = 0;  // upto: of all sequences up to this thread's (of the last block of them)
  for (int b0 = 0; b0 < p.B; b0 += T_NT) {
    unsigned sum;
    w = work_of(b0 + tid);
    upto = total + block_scan<NW>(w, s_scan, sum);
    total += sum;
  }
  const unsigned nc = min(gridDim.x, total);
  if (__syncthreads_or(rest)) fill_rest<DT, T_NT>(p, D);
  if (blockIdx.x >= nc) return;
  const Share share(total, nc);
  const unsigned my0 = share.start(blockIdx.x);
  const int count = static_cast<int>(share.start(blockIdx.x + 1) - my0);
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += T_NT) {
    if (p.B > T_NT) {
      unsigned sum;
      w = work_of(b0 + tid);
      upto = before + block_scan<NW>(w, s_scan, sum);
      before += sum;
    }
    if (my0 < upto && my0 >= upto - w) *s_seq = b0 + tid, *s_base = upto - w;
  }
  if (tid == 0) {
    for (int i = 0; i < T_RAW; ++i) mbar_init(&bar.raw_full[i], 1), mbar_init(&bar.raw_empty[i], T_CONV / 64);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], T_CONV / 64), mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], T_CONV / 64), mbar_init(&bar.v_empty[i], 1);
      mbar_init(&bar.s_full[i], 1), mbar_init(&bar.p_full[i], 8), mbar_init(&bar.o_done[i], 1);
    }
    for (int i = 0; i < T_SCALES; ++i) mbar_init(&bar.sc_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.q_full[i], T_SOFT / 32);
    fence_mbar_init();
  }
  if (warp == (T_SOFT + T_CONV) / 32) tmem_alloc(s_tmem, 512);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);

  TileCursor at;
  at.b = *s_seq;
  tile_enter(p, at);
  {
    unsigned r = my0 - *s_base;
    const unsigned head = head_work(at.ctx, at.cnt);
    at.rt = 0;
    at.h = static_cast<int>(r / head);
    r -= at.h * head;
    for (;;) {
      at.n = token_tiles(p, at.ctx, at.cnt, at.rt);
      if (r < static_cast<unsigned>(at.n)) break;
      r -= at.n;
      ++at.rt;
    }
    at.j = static_cast<int>(r);
  }
  // a wait that ran out: the role goes on without waiting, its loops end, and
  // the call reports a timeout
  bool lost = false;
  const auto rest_wait = [&](auto rest, uint64_t *b, uint32_t parity) {  // warp-wide
    constexpr int REST = decltype(rest)::value;
    if (!lost && !__all_sync(0xffffffffu, tile_wait<REST>(b, parity))) lost = true;
  };
  const auto wait = [&](uint64_t *b, uint32_t parity) { rest_wait(Number<0>{}, b, parity); };
  const auto lazy_wait = [&](uint64_t *b, uint32_t parity) { rest_wait(Number<40>{}, b, parity); };  // where latency hides
  const auto arrive = [&](uint64_t *b) {  // once for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };

  if (warp < T_SOFT / 32) {
    // ------------------------------------------------------------ softmax
    more_registers<T_REG_SOFT>();
    const int grp = (warp >> 2) & 1, half = warp >> 3, quarter = 2 * half + grp, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane field of the addresses
    const uint32_t tS = tmem + lanes + grp * 128 + 64 * half, tO = tmem + lanes + 256;
    float *xch = reinterpret_cast<float *>(smem + L::ML);
    const float2 *scales = reinterpret_cast<const float2 *>(smem + L::SCALES);
    const float NINF = __uint_as_float(0xff800000u);
    uint32_t uses = 0;                                       // tiles of this group
    const auto meet = [&]() { named_sync(1, T_SOFT); };      // all softmax threads
    const auto pair = [&]() { named_sync(2 + (warp & 7), 64); };  // this warp and the other half's of the same rows
    float *const mine = p.pieces + static_cast<long long>(blockIdx.x) * 2 * L::PIECE;
    int i = 0;
    while (i < count) {
      // ---- a segment: its queries
      const int rows = min(TQ, at.cnt * p.G - at.rt * TQ), row = at.rt * TQ + r, node = row / p.G;
      float fac;
      {
        const bool mine_live = r < rows;
        const long long base = mine_live ? at.b * p.q_sb + node * p.q_sn + (at.h * p.G + row % p.G) * p.q_sh + quarter * (D / 4) : 0;
        Raw8<DT> raw[D / 32];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          if (mine_live) raw[k] = p.q_vec ? load8<DT, true>(p.q, base + 8 * k) : load8<DT, false>(p.q, base + 8 * k);
          else raw[k].v[0] = make_uint4(0, 0, 0, 0);
          float x[8];
          unpack8<DT>(raw[k], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
        xch[quarter * 128 + r] = amax;
        meet();
        amax = fmaxf(fmaxf(xch[r], xch[128 + r]), fmaxf(xch[256 + r], xch[384 + r]));
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
        // a negative scale turns the query around, so that scores only grow with the products
        const float down = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), p.scale_log2);
        fac = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * fabsf(p.scale_log2);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          float x[8];
          unpack8<DT>(raw[k], x);
          const uint4 w = make_uint4(f32_to_f16x2(x[0] * down, x[1] * down), f32_to_f16x2(x[2] * down, x[3] * down),
                                     f32_to_f16x2(x[4] * down, x[5] * down), f32_to_f16x2(x[6] * down, x[7] * down));
          const int chunk = quarter * (D / 32) + k;  // of 8 elements
          *reinterpret_cast<uint4 *>(smem + L::Q + (chunk >> 3) * 16384 + r * 128 + ((chunk & 7) ^ (r & 7)) * 16) = w;
        }
        fence_async_smem();
      }
      const int s0 = at.j, end = min(at.n - at.j, count - i) + i;
      const bool has[2] = {end - i >= 2 || !(i & 1), end - i >= 2 || (i & 1)};  // the group has a tile
      // A product warp waits for the segments of its group's tiles alone.  The
      // softmax ends such a segment after that group's last product, so the
      // barrier is never a phase ahead of the warp; a warp that also waited for
      // the other group's segments could fall two phases behind, where parities
      // are equal again.
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (has[e]) arrive(&bar.q_full[e]);
      // A tile is weighed again, and the accumulator scaled, when the offset
      // moves.  Over a long axis the largest weight starts at 2^8: fp16 then
      // keeps its full precision down to 2^-22 of it, and the offset moves once
      // or twice; at 2^13 some row of the tile's 128 moved it in half of the tiles.
      const float up = at.n >= 8 ? 8.f : WEIGHT_UP;
      float m = NINF, base = 0.f, l = 0.f, m0 = NINF, l0 = 0.f;
      const uint32_t uses0 = uses;
      const bool live = 32 * (warp & 3) < rows;  // this warp has rows to look after
      const int k0 = i + ((i ^ grp) & 1);  // the group's first tile
      if (!live && k0 < end) uses += (end - k0 + 1) / 2;
      for (int k = k0; live && k < end; k += 2, ++uses) {
        const int tok0 = (s0 + k - i) * TK + 64 * half;
        wait(&bar.sc_full[k % T_SCALES], (k / T_SCALES) & 1);
        wait(&bar.s_full[grp], uses & 1);
        tc_after_sync();
        {
          const float2 *sc_at = scales + (k % T_SCALES) * 8 + 4 * half;
          const bool edge = tok0 + 64 > at.ctx;  // new tokens, or slots past the last one
          // the slots that the row sees, of 32 columns
          const auto seen32 = [&](int q) -> uint32_t {
            const int n0 = tok0 + 32 * q - at.ctx;  // node of the first column
            const auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
            uint32_t bits = low(node + 1 - n0);
            if (p.mask) {
              const uint32_t *words = p.mask + (static_cast<long long>(at.b) * p.N + min(node, p.N - 1)) * p.W;
              const int w = n0 >> 5;  // rounds down; words before the first are context
              const uint32_t x = w < 0 ? ~0u : w < p.W ? words[w] : 0u, y = w + 1 < 0 ? ~0u : w + 1 < p.W ? words[w + 1] : 0u;
              bits = __funnelshift_r(x, y, n0 & 31);
            }
            return bits & low(at.cnt - n0);
          };
          // weights under the offset so far, and their largest exponent
          uint32_t pk[32];
          float sum = 0.f, hi = NINF;
          bool any_zero = false;
          const auto weights = [&](auto at_edge) {
            sum = 0.f, hi = NINF;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t s[2][16];
              tmem_ld16(tS + 32 * q, s[0]);
              tmem_ld16(tS + 32 * q + 16, s[1]);
              tc_wait_ld(s[0]);
              tc_wait_ld(s[1]);
              uint32_t bits = ~0u;
              if constexpr (decltype(at_edge)::value) bits = seen32(q);
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {  // 16 tokens that share their scales
                const float2 sc = sc_at[2 * q + hf];
                const bool zero = sc.y == NINF;  // a block without values: every exponent becomes -inf
                any_zero |= zero;
                const float f = fac * sc.x, off = sc.y - base;  // NaN for a bad page
                float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  float2 x = fma2(make_float2(__uint_as_float(s[hf][e]), __uint_as_float(s[hf][e + 1])), make_float2(f, f), make_float2(off, off));
                  if constexpr (decltype(at_edge)::value) {  // after the scale: a bad page is NaN only where it is seen
                    if (!((bits >> (16 * hf + e)) & 1)) x.x = NINF;
                    if (!((bits >> (16 * hf + e + 1)) & 1)) x.y = NINF;
                  }
                  hi = fmaxf(fmaxf(hi, x.x), x.y);
                  x.x = ex2(x.x), x.y = ex2(x.y);
                  part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], x);
                  pk[16 * q + 8 * hf + e / 2] = f32_to_f16x2(x.x, x.y);
                }
                const float2 both = add2(part[0], part[1]);
                if (!zero) sum = fmaf((both.x + both.y) * SUM_DOWN, ex2(-sc.y), sum);
              }
            }
          };
          if (edge) weights(Flag<true>{});
          else weights(Flag<false>{});
          // both halves go by the whole tile's maximum
          float *xmine = xch + 256 * grp + 128 * half + r, *xother = xch + 256 * grp + 128 * (half ^ 1) + r;
          *xmine = hi + base;
          pair();
          const float top = fmaxf(hi + base, *xother);
          if (__any_sync(0xffffffffu, top > m + (WEIGHT_UP + WEIGHT_SLACK))) {
            // the offset moves, and the tile is weighed again
            const float nm = fmaxf(m, top - up), nb = nm == NINF ? 0.f : nm, a = ex2(m - nb);
            l *= a;
            m = nm, base = nb;
            if (uses != uses0) {  // O holds the products of this segment's earlier tiles
              wait(&bar.o_done[grp], (uses - 1) & 1);
              tc_after_sync();
#pragma unroll 1
              for (int q = 0; q < D / 64; ++q) {  // each half takes half of the columns
                const uint32_t col = tO + grp * 128 + half * (D / 2) + 32 * q;
                uint32_t o[2][16];
                tmem_ld16(col, o[0]);
                tmem_ld16(col + 16, o[1]);
                tc_wait_ld(o[0]);
                tc_wait_ld(o[1]);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e >> 4][e & 15] = __float_as_uint(__uint_as_float(o[e >> 4][e & 15]) * a);
                tmem_st16(col, o[0]);
                tmem_st16(col + 16, o[1]);
              }
            }
            if (edge) weights(Flag<true>{});
            else weights(Flag<false>{});
          }
          if (any_zero) {  // blocks without values count in a sum of their own
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              if (sc_at[q].y != NINF) continue;
              const float f = fmaxf(fac * sc_at[q].x, 1e-37f);
              const uint32_t bits = edge ? seen32(q >> 1) >> (16 * (q & 1)) : ~0u;
              uint32_t s[16];
              tmem_ld16(tS + 16 * q, s);
              tc_wait_ld(s);
              float t = m0;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (!((bits >> e) & 1)) s[e] = 0xff800000u;
                t = fmaxf(t, __uint_as_float(s[e]) * f);
              }
              const float nb = t == NINF ? 0.f : t;
              l0 *= ex2(m0 - nb);
              m0 = t;
#pragma unroll
              for (int e = 0; e < 16; ++e) l0 += ex2(__uint_as_float(s[e]) * f - nb);
            }
          }
          l += sum;
          tmem_st16(tS, pk);  // weights over scores that have been read
          tmem_st16(tS + 16, pk + 16);
        }
        tc_wait_st();
        tc_before_sync();
        __syncwarp();  // the first rows' warps arrive for those without rows, too
        if (lane == 0) mbar_arrive_many(&bar.p_full[grp], (warp & 3) == 0 ? 4 - (rows - 1) / 32 : 1);
      }
      // ---- the end of the segment: both groups' parts meet
      if (live && has[grp]) {
        wait(&bar.o_done[grp], (uses - 1) & 1);
        tc_after_sync();
      }
      tc_before_sync();
      meet();
      tc_after_sync();
      // all products with the queries are done: their place takes the sums
      float4 *sums = reinterpret_cast<float4 *>(smem + L::Q);
      sums[quarter * 128 + r] = make_float4(m + SUM_UP, l, m0, l0);
      meet();
      float M = NINF, mg[2];
      float4 each[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        each[e] = sums[e * 128 + r];
        M = fmaxf(M, fmaxf(each[e].x, each[e].z - 60.f));  // blocks without values: neither sum overflows
      }
      mg[0] = each[0].x, mg[1] = each[1].x;
      const float bm = M == NINF ? 0.f : M;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += each[e].y * ex2(each[e].x - bm) + each[e].w * ex2(each[e].z - bm);
      const bool whole = s0 == 0 && s0 + end - i == at.n;
      const int which = s0 > 0 ? 0 : 1;
      const Inverse over(sum);
      const float aw = ex2(mg[0] - bm) * (whole ? over.inv : 1.f), bw = ex2(mg[1] - bm) * (whole ? over.inv : 1.f);
      float *piece = mine + which * L::PIECE;
      const long long orow = (static_cast<long long>(at.b) * p.N + node) * (c.Hk * p.G) + at.h * p.G + row % p.G;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {  // a quarter of the columns each
        if (!live) break;
        const int col = quarter * (D / 4) + 16 * q;
        uint32_t x[16], y[16];
        float z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = y[e] = 0;
        if (has[0]) tmem_ld16(tO + col, x);
        if (has[1]) tmem_ld16(tO + 128 + col, y);
        tc_wait_ld(x);
        tc_wait_ld(y);
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = __uint_as_float(x[e]) * aw + __uint_as_float(y[e]) * bw;
        if (r < rows) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              float w[8];
#pragma unroll
              for (int g = 0; g < 8; ++g) w[g] = z[e + g] * over.down;
              store8<DT, true>(p.out, orow * D + col + e, pack8<DT>(w));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              reinterpret_cast<float4 *>(piece)[((col + e) / 4) * 128 + r] = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
          }
        }
      }
      tc_before_sync();
      if (r < rows && quarter == 0) {
        if (whole) {
          if (p.lse) p.lse[orow] = sum == 0.f ? NINF : (M + log2f(sum)) * 0.6931471805599453f;
        } else {
          piece[128 * D + r] = M, piece[128 * D + 128 + r] = sum;
        }
      }
      if (!whole) __threadfence();
      meet();  // the accumulators are free
      if (!whole) {
        // a segment that several CTAs share: the last to arrive merges, in order
        const unsigned f0 = my0 + i - s0;
        const int c0 = share.holder(f0), n = static_cast<int>(share.holder(f0 + at.n - 1)) - c0 + 1;
        if (tid == 0) {
          *s_last = atomicAdd(p.done + c0, 1) == n - 1;
          __threadfence();
        }
        meet();
        if (*s_last) {
          __threadfence();
          if (r < rows) {
            const auto part = [&](int e) { return p.pieces + (static_cast<long long>(c0 + e) * 2 + (e == 0 ? 1 : 0)) * L::PIECE; };
            float M2 = NINF;
            for (int e = 0; e < n; ++e) M2 = fmaxf(M2, __ldcg(part(e) + 128 * D + r));
            const float b2 = M2 == NINF ? 0.f : M2;
            float sum2 = 0.f;
            for (int e = 0; e < n; ++e) sum2 = fmaf(ex2(__ldcg(part(e) + 128 * D + r) - b2), __ldcg(part(e) + 128 * D + 128 + r), sum2);
            const Inverse over2(sum2);
#pragma unroll 1
            for (int q = 0; q < D / 64; ++q) {
              const int col = quarter * (D / 4) + 16 * q;
              float z[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = 0.f;
              for (int e = 0; e < n; ++e) {
                const float a = ex2(__ldcg(part(e) + 128 * D + r) - b2);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const float4 x = __ldcg(reinterpret_cast<const float4 *>(part(e)) + (col / 4 + g) * 128 + r);
                  z[4 * g] = fmaf(a, x.x, z[4 * g]), z[4 * g + 1] = fmaf(a, x.y, z[4 * g + 1]);
                  z[4 * g + 2] = fmaf(a, x.z, z[4 * g + 2]), z[4 * g + 3] = fmaf(a, x.w, z[4 * g + 3]);
                }
              }
#pragma unroll
              for (int e = 0; e < 16; e += 8) {
                float w[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) w[g] = over2(z[e + g]);
                store8<DT, true>(p.out, orow * D + col + e, pack8<DT>(w));
              }
            }
            if (quarter == 0 && p.lse) p.lse[orow] = sum2 == 0.f ? NINF : (M2 + log2f(sum2)) * 0.6931471805599453f;
          }
          if (tid == 0) p.done[c0] = 0;  // zero again for the next call
        }
        meet();  // s_last may be written again
      }
      i = end;
      if (i < count) tile_next(p, at);
    }
  } else if (warp < (T_SOFT + T_CONV) / 32) {
    // --------------------------------------------------------- conversion
    fewer_registers<T_REG_CONV>();
    const int ct = (tid - T_SOFT) % (T_CONV / 2), t = (tid - T_SOFT) / (T_CONV / 2);  // keys or values
    int left = at.n - at.j;  // tiles of the segment from here on
    TileCursor u = at;
    for (int i = 0; i < count; ++i) {
      if (left == 0) tile_next(p, u), left = u.n;
      const int j = u.n - left;
      --left;
      const bool written = (j + 1) * TK <= u.ctx + u.cnt;  // every row of the tile
      const uint32_t buf = i & 1, ph = (i >> 1) & 1;
      const int slot = (2 * i + t) % T_RAW;
      lazy_wait(&bar.raw_full[slot], ((2 * i + t) / T_RAW) & 1);
      lazy_wait(t ? &bar.v_empty[buf] : &bar.k_empty[buf], ph ^ 1);
      const unsigned char *raw = smem + L::RAW + slot * L::RAWB;
      unsigned char *to = smem + (t ? L::V : L::K) + buf * L::OP;
      if (written && !s_bad[slot]) convert_tile<D, KIND, false>(raw, to, ct);
      else convert_tile<D, KIND, true>(raw, to, ct);
      fence_async_smem();
      arrive(t ? &bar.v_full[buf] : &bar.k_full[buf]);
      if (lane == 0) mbar_arrive(&bar.raw_empty[slot]);
    }
  } else {
    fewer_registers<T_REG_REST>();
    const int extra = warp - (T_SOFT + T_CONV) / 32;
    if (extra == 0 || extra == 2) {
    // ----------------------------------------------------------- products
    // A warp for each group: the issue of one group's products and the waits
    // around it hide behind the other group's.
    if (lane == 0) {
      constexpr uint32_t ID_S = 1u << 4 | (TK / 8) << 17 | (TQ / 16) << 24;           // fp16 x fp16 -> fp32
      constexpr uint32_t ID_O = 1u << 4 | 1u << 16 | (D / 8) << 17 | (TQ / 16) << 24;  // values run along the tokens
      const int g = extra >> 1;
      const uint32_t base = smem_u32(smem), tS = tmem + g * 128, tO = tmem + 256 + g * 128;
      const uint64_t dQ = tc_desc(base + L::Q, 0), dK = tc_desc(base + L::K + g * L::OP, 0), dV = tc_desc(base + L::V + g * L::OP, 16384);
      const auto one = [&](uint64_t *b, uint32_t parity) {
        if (!lost && !tile_wait<0>(b, parity)) lost = true;
      };
      TileCursor u = at;
      int i = g;  // this group's next tile
      uint32_t ph = 0, ph_q = 0;
      for (int seg1 = at.n - at.j;; tile_next(p, u), seg1 += u.n) {
        if (i < min(seg1, count)) one(&bar.q_full[g], ph_q), ph_q ^= 1;
        for (const int end = min(seg1, count), first = i; i < end; i += 2, ph ^= 1) {
          one(&bar.k_full[g], ph);
          tc_after_sync();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {  // 32 bytes of the rows at a time, 16384 between panels
            const uint64_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
            tc_mma_ss(tS, dQ + off, dK + off, ID_S, k > 0);
          }
          tc_commit(&bar.s_full[g]);
          tc_commit(&bar.k_empty[g]);
          one(&bar.v_full[g], ph);
          one(&bar.p_full[g], ph);
          tc_after_sync();
#pragma unroll
          for (int k = 0; k < TK / 16; ++k)  // 16 tokens at a time
            tc_mma_ts(tO, tS + 64 * (k >> 2) + 8 * (k & 3), dV + (k * 2048 >> 4), ID_O, k > 0 || i != first);
          tc_commit(&bar.o_done[g]);
          tc_commit(&bar.v_empty[g]);
        }
        if (seg1 >= count) break;
      }
    }
    } else if (extra == 1) {
    // -------------------------------------------------------------- copies
    TileCursor u = at;
    int left = at.n - at.j, issued = 0;
    // lane g < 8 looks after the tokens 16 g of a tile
    const auto page_id = [&](const TileCursor &v, int j) {
      const int tok = j * TK + 16 * (lane & 7);
      return tok < v.ctx + v.cnt ? c.table[static_cast<long long>(v.b) * c.per + (tok >> c.log_page)] : 0;
    };
    int page = page_id(u, u.j);
    for (int i = 0; i < count; ++i) {
      const int j = u.n - left, tok = j * TK + 16 * (lane & 7), len = u.ctx + u.cnt;
      const bool there = lane < 8 && tok < len, bad = there && static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages);
      const long long id = static_cast<long long>(bad ? 0 : page) * c.Hk + u.h;
      const bool any_bad = __any_sync(0xffffffffu, bad);
      if (bad) atomicOr(p.status, ST_PAGE);
      float ks = 0.f, vs = 1.f;
      if (there) ks = c.k_scale[id], vs = c.v_scale[id];
      // the next tile's pages, while this one's copies wait for their slots
      TileCursor v = u;
      if (--left == 0 && i + 1 < count) tile_next(p, v), left = v.n;
      const int next = i + 1 < count ? page_id(v, v.n - left) : 0;
      // one copy for each page: its first 16 tokens in the tile stand for it
      const int in = tok & (c.page - 1);
      const bool lead = there && (in == 0 || (lane & 7) == 0);
      const uint32_t bytes = static_cast<uint32_t>(min(c.page, TK) * D);
      const uint32_t pages = __popc(__ballot_sync(0xffffffffu, lead));
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int slot = (2 * i + t) % T_RAW;
        lazy_wait(&bar.raw_empty[slot], (((2 * i + t) / T_RAW) & 1) ^ 1);
        if (lost) break;  // no copy into a slot that may be in use
        if (lane == 0) {
          s_bad[slot] = any_bad;
          mbar_arrive_expect_tx(&bar.raw_full[slot], bytes * pages);
        }
        __syncwarp();
        if (lead)
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(smem + L::RAW + slot * L::RAWB + 16 * (lane & 7) * D)),
                       "l"((t ? c.v : c.k) + (id * c.page + in) * D), "r"(bytes), "r"(smem_u32(&bar.raw_full[slot]))
                       : "memory");
        issued = 2 * i + t + 1;
      }
      if (lane < 8) {
        const float lv = bad ? 0.f : vs <= LEAST_V_SCALE ? __uint_as_float(0xff800000u) : lg2(vs);
        reinterpret_cast<float2 *>(smem + L::SCALES)[(i % T_SCALES) * 8 + lane] = make_float2(bad ? __uint_as_float(0x7fc00000u) : ks, lv);
      }
      arrive(&bar.sc_full[i % T_SCALES]);
      u = v;
      page = next;
    }
    // no copy outlives the CTA, even after a wait that ran out
    lost = false;
    for (int k = max(0, issued - T_RAW); k < issued; ++k) wait(&bar.raw_full[k % T_RAW], (k / T_RAW) & 1);
    }
  }
  if (lost) atomicOr(p.status, ST_TIMEOUT);
  tc_before_sync();
  __syncthreads();
  if (warp == (T_SOFT + T_CONV) / 32) {
    tc_after_sync();
    tmem_free(tmem, 512);
  }
}

}  // namespace spec
