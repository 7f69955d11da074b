// Host side of the operators around the paged 8-bit key/value cache: argument
// validation, launch geometry and the C ABI declared in include/spec_verify.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "attention.cuh"
#include "attention_tile.cuh"
#include "cache.cuh"
#include "evict.cuh"
#include "host.h"
#include "spec_verify.h"

namespace spec {

// Launches as a programmatic dependent of what precedes it on the stream.
int launch_dependent(const void *fn, dim3 grid, int threads, int smem, cudaStream_t stream, void *params, const char *what, unsigned cluster) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void *args[] = {params};
  const cudaError_t e = launch_kernel(&cfg, fn, args);
  return e == cudaSuccess ? static_cast<int>(SPEC_OK) : cuda_fail(e, what);
}

namespace {

bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
int size_of(int dtype) { return dtype == SPEC_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype == SPEC_F32 || dtype == SPEC_BF16 || dtype == SPEC_F16; }

// 16-byte vectors may be used at every row of h.
bool vectors(const spec_heads_t &h, int esz) {
  return aligned16(h.data) && h.stride_b * esz % 16 == 0 && h.stride_n * esz % 16 == 0 && h.stride_h * esz % 16 == 0;
}

int check_cache(const spec_cache_t *c, const int32_t *table, int per, int B, CacheView *view) {
  if (!c) return fail(SPEC_ERR_ARG, "cache is NULL");
  if (c->kind != SPEC_E4M3 && c->kind != SPEC_I8) return fail(SPEC_ERR_DTYPE, "cache kind must be SPEC_E4M3 or SPEC_I8");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(SPEC_ERR_ARG, "head_dim must be 64 or 128");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(SPEC_ERR_ARG, "page_size must be 16, 32, 64 or 128");
  if (c->kv_heads < 1 || c->kv_heads > 32767) return fail(SPEC_ERR_ARG, "kv_heads out of range [1, 32767]");
  if (c->pages < 1) return fail(SPEC_ERR_ARG, "pages must be >= 1");
  if (per < 1 || static_cast<long long>(per) * c->page_size > (1 << 30))
    return fail(SPEC_ERR_ARG, "pages_per_seq out of range (1 to 2^30 tokens)");
  if (B < 0 || B > 65535) return fail(SPEC_ERR_ARG, "B out of range [0, 65535]");
  if (B > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return fail(SPEC_ERR_ARG, "a cache pointer is NULL");
  if (B > 0 && !table) return fail(SPEC_ERR_ARG, "page_table is NULL");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(SPEC_ERR_ALIGN, "the cache's codes must be 16-byte aligned");
  view->k = static_cast<unsigned char *>(c->k);
  view->v = static_cast<unsigned char *>(c->v);
  view->k_scale = c->k_scale;
  view->v_scale = c->v_scale;
  view->table = table;
  view->pages = c->pages;
  view->Hk = c->kv_heads;
  view->page = c->page_size;
  view->log_page = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  view->D = c->head_dim;
  view->kind = c->kind;
  view->per = per;
  return SPEC_OK;
}

// Blocks that n rows from any slot on can touch.
unsigned blocks_of(int n, int page) { return static_cast<unsigned>((static_cast<long long>(n) + page - 2) / page + 1); }

// rows * D elements of a block: one warp up to 2048, a CTA up to 8192 or 16384.
template <int DT>
const void *pick_write(int elements, bool vec) {
  if (elements <= 2048) return vec ? reinterpret_cast<const void *>(&cache_write_kernel<DT, 32, 8, true>)
                                   : reinterpret_cast<const void *>(&cache_write_kernel<DT, 32, 8, false>);
  if (elements <= 8192) return vec ? reinterpret_cast<const void *>(&cache_write_kernel<DT, 256, 4, true>)
                                   : reinterpret_cast<const void *>(&cache_write_kernel<DT, 256, 4, false>);
  return vec ? reinterpret_cast<const void *>(&cache_write_kernel<DT, 256, 8, true>)
             : reinterpret_cast<const void *>(&cache_write_kernel<DT, 256, 8, false>);
}

// vec: units of eight elements, at most two to a thread; `one`: one to a
// thread.  Otherwise single elements, or two for neighbouring pairs.
template <int DT, class P>
const void *pick_norm_rope(bool vec, bool one, bool pairs) {
  if (vec && one)
    return pairs ? reinterpret_cast<const void *>(&norm_rope_rows_kernel<DT, true, P>)
                 : reinterpret_cast<const void *>(&norm_rope_rows_kernel<DT, false, P>);
  if (vec) return reinterpret_cast<const void *>(&norm_rope_kernel<DT, 8, 2, P>);
  return pairs ? reinterpret_cast<const void *>(&norm_rope_kernel<DT, 2, 8, P>)
               : reinterpret_cast<const void *>(&norm_rope_kernel<DT, 1, 16, P>);
}
// A call's tensors and sizes into p, and its launch: spec_qk_norm_rope, and with
// P = NormRopeAxesParams (p.axes set) spec_qk_norm_rope_axes.
template <class P>
int norm_rope(P &p, const spec_heads_t *q, const spec_heads_t *k, const spec_heads_t *out_q, const spec_heads_t *out_k,
              const void *q_weight, const void *k_weight, const int32_t *base, const int32_t *offset, int B, int N, int Hq, int Hk,
              int D, int dtype, int norm, float eps, const double *inv_freq, const int32_t *axis, int rot, int pairs, void *stream_ptr) {
  constexpr bool AXES = std::is_same_v<P, NormRopeAxesParams>;
  if (!known_dtype(dtype)) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_F32, SPEC_BF16 or SPEC_F16");
  if (B < 0 || N < 0 || static_cast<long long>(B) * N > INT_MAX / 2) return fail(SPEC_ERR_ARG, "B and N must be >= 0 and B * N < 2^30");
  if (Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535) return fail(SPEC_ERR_ARG, "head counts out of range [0, 65535]");
  if (D < 2 || D > 512 || D % 2) return fail(SPEC_ERR_ARG, "head_dim must be even and in [2, 512]");
  if (rot < 0 || rot > D || rot % 2) return fail(SPEC_ERR_ARG, "rot must be even and in [0, head_dim]");
  if (norm != 0 && norm != 1) return fail(SPEC_ERR_ARG, "norm must be 0 or 1");
  if (pairs != 0 && pairs != 1) return fail(SPEC_ERR_ARG, "pairs must be 0 or 1");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SPEC_ERR_ARG, "eps must be finite and >= 0");
  if (rot > 0 && !inv_freq) return fail(SPEC_ERR_ARG, "inv_freq is NULL");
  if (AXES && rot > 0 && !axis) return fail(SPEC_ERR_ARG, "axis is NULL");
  if (!norm && (q_weight || k_weight)) return fail(SPEC_ERR_ARG, "weights are given without the norm");
  if (B == 0 || N == 0 || Hq + Hk == 0) return SPEC_OK;
  if ((Hq > 0 && (!q || !out_q || !q->data || !out_q->data)) || (Hk > 0 && (!k || !out_k || !k->data || !out_k->data)))
    return fail(SPEC_ERR_ARG, "a tensor is NULL");
  if (AXES && rot > 0 && !offset) return fail(SPEC_ERR_ARG, "positions is NULL");
  const int esz = size_of(dtype);
  const spec_heads_t *src[2] = {q, k}, *dst[2] = {out_q, out_k};
  const void *weight[2] = {q_weight, k_weight};
  const int heads[2] = {Hq, Hk};
  bool vec = D % 8 == 0 && (pairs ? rot % 8 == 0 : rot % 16 == 0);
  for (int i = 0; i < 2; ++i) {
    p.heads[i] = heads[i];
    if (heads[i] == 0) continue;
    p.src[i] = src[i]->data;
    p.dst[i] = dst[i]->data;
    p.weight[i] = weight[i];
    p.ssb[i] = src[i]->stride_b, p.ssn[i] = src[i]->stride_n, p.ssh[i] = src[i]->stride_h;
    p.dsb[i] = dst[i]->stride_b, p.dsn[i] = dst[i]->stride_n, p.dsh[i] = dst[i]->stride_h;
    vec = vec && vectors(*src[i], esz) && vectors(*dst[i], esz) && aligned16(weight[i]);
  }
  p.base = base;
  p.offset = offset;
  p.B = B, p.N = N, p.D = D, p.rot = rot;
  p.norm = norm, p.pairs = pairs, p.eps = eps;
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return fail(SPEC_ERR_ARG, "inv_freq must be finite");
    if constexpr (AXES) {
      if (axis[i] < 0 || axis[i] >= p.axes) return fail(SPEC_ERR_ARG, "axis out of range [0, axes)");
      p.axis[i] = static_cast<uint8_t>(axis[i]);
    }
    // turns per position; whole turns drop out, since positions are whole
    const double turns = inv_freq[i] * 0.15915494309189533577, frac = turns - std::floor(turns);
    p.freq[i] = frac >= 1.0 ? 0ull : static_cast<unsigned long long>(std::ldexp(frac, 64));
  }
  const int ve = vec ? 8 : pairs ? 2 : 1;
  const int npair = pairs ? 0 : rot / 2 / ve, units = npair + (D - 2 * npair * ve) / ve;
  p.lanes = 1;
  while (p.lanes < units && p.lanes < 32) p.lanes *= 2;
  // norm_rope_rows_kernel has a CTA each for a token's queries and keys
  const unsigned tensors = vec && units <= p.lanes && Hq > 0 && Hk > 0 ? 2 : 1;
  // one wave of four CTAs per SM where that is at most ROPE_TOKENS tokens to a
  // CTA: its set-up is a small part then
  const long long tokens = static_cast<long long>(B) * N, wave = 4LL * num_sms();
  p.per_cta = static_cast<int>(std::min<long long>(ROPE_TOKENS, (tokens * tensors + wave - 1) / wave));
  const void *fn = dtype == SPEC_F32    ? pick_norm_rope<DT_F32, P>(vec, units <= p.lanes, pairs)
                   : dtype == SPEC_BF16 ? pick_norm_rope<DT_BF16, P>(vec, units <= p.lanes, pairs)
                                        : pick_norm_rope<DT_F16, P>(vec, units <= p.lanes, pairs);
  return launch_dependent(fn, dim3(static_cast<unsigned>((tokens + p.per_cta - 1) / p.per_cta), tensors), 256,
                p.per_cta * (rot / 2) * static_cast<int>(sizeof(float2)), static_cast<cudaStream_t>(stream_ptr), &p,
                "norm_rope_kernel launch");
}

// The attention's kernel, its block and shared memory, and the floats of its
// workspace per CTA.
struct AttnChoice {
  const void *fn;
  int threads, smem, ctas;  // ctas: per SM
  size_t work;
  int rows, tokens;         // of a work item
};
// By the rows per kv head.  Up to 24 a warp's own matrix instructions, 8 rows at
// a time, are faster; beyond, the tensor cores with accumulators in tensor
// memory, 128 rows at a time.  (64 sequences of up to 8192 tokens, 8 kv heads,
// e4m3 / int8: 4 rows 171 / 172 us, 16 rows 185 / 203, 24 rows 227 / 245; the
// tile kernel takes 274 / 279 for 24 and 32 rows and 294 / 307 for 48.)
template <int D, int KIND, int DT>
AttnChoice choose_attn(long long rows) {
  if (rows <= 8) {
    using L = StreamLayout<D, 1>;
    return {reinterpret_cast<const void *>(&attn_stream_kernel<D, KIND, DT, 1>), L::THREADS, L::SMEM, L::RESIDENT, L::WORK, L::ROWS, ASTEP};
  }
  if (rows <= 16) {
    using L = StreamLayout<D, 2>;
    return {reinterpret_cast<const void *>(&attn_stream_kernel<D, KIND, DT, 2>), L::THREADS, L::SMEM, L::RESIDENT, L::WORK, L::ROWS, ASTEP};
  }
  if (rows <= 24) {
    using L = StreamLayout<D, 3>;
    return {reinterpret_cast<const void *>(&attn_stream_kernel<D, KIND, DT, 3>), L::THREADS, L::SMEM, L::RESIDENT, L::WORK, L::ROWS, ASTEP};
  }
  using L = TileLayout<D>;
  return {reinterpret_cast<const void *>(&attn_tile_kernel<D, KIND, DT>), T_NT, L::SMEM, 1, 2 * L::PIECE, TQ, TK};
}
AttnChoice choose_attn(int D, int kind, int dtype, long long rows) {
  const bool bf = dtype == SPEC_BF16;
  if (D == 128 && kind == SPEC_E4M3) return bf ? choose_attn<128, KIND_E4M3, DT_BF16>(rows) : choose_attn<128, KIND_E4M3, DT_F16>(rows);
  if (D == 128) return bf ? choose_attn<128, KIND_I8, DT_BF16>(rows) : choose_attn<128, KIND_I8, DT_F16>(rows);
  if (kind == SPEC_E4M3) return bf ? choose_attn<64, KIND_E4M3, DT_BF16>(rows) : choose_attn<64, KIND_E4M3, DT_F16>(rows);
  return bf ? choose_attn<64, KIND_I8, DT_BF16>(rows) : choose_attn<64, KIND_I8, DT_F16>(rows);
}

// Up to 48 rows a warp's own matrix instructions; beyond, the tensor cores with
// accumulators in tensor memory, 128 rows at a time.  (64 sequences of up to 8192
// tokens, 8 kv heads, e4m3, head size 128: 16, 32, 48, 56 and 64 rows 88, 114, 148,
// 167 and 180 us, the tile kernel 147, 148, 162, 162 and 163; head size 64: 48 and 56
// rows 102 and 115, the tile kernel 106 and 107.  8 of up to 32768: 72 and 81, the
// tile kernel 80 and 80.)
struct WeightsChoice {
  const void *fn;
  int most, smem;
};
template <int D, int KIND, int DT>
WeightsChoice choose_weights(long long rows) {
  if (rows > 48) return {reinterpret_cast<const void *>(&cache_weights_tile_kernel<D, KIND, DT>), WR, WeightsLayout<D>::SMEM};
  const int most = static_cast<int>((rows + 7) / 8 * 8);
  return {reinterpret_cast<const void *>(&cache_weights_kernel<D, KIND, DT>), most, most * (D * 2 + 8)};
}
template <int D>
WeightsChoice choose_weights(int kind, int dtype, long long rows) {
  const bool bf = dtype == SPEC_BF16;
  if (kind == SPEC_E4M3) return bf ? choose_weights<D, KIND_E4M3, DT_BF16>(rows) : choose_weights<D, KIND_E4M3, DT_F16>(rows);
  return bf ? choose_weights<D, KIND_I8, DT_BF16>(rows) : choose_weights<D, KIND_I8, DT_F16>(rows);
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" {

int spec_qk_norm_rope(const spec_heads_t *q, const spec_heads_t *k, const spec_heads_t *out_q, const spec_heads_t *out_k,
                      const void *q_weight, const void *k_weight, const int32_t *base, const int32_t *offset, int B, int N,
                      int Hq, int Hk, int D, int dtype, int norm, float eps, const double *inv_freq, int rot, int pairs,
                      void *stream_ptr) {
  NvtxRange nvtx_range("spec_qk_norm_rope");
  NormRopeParams p;
  std::memset(&p, 0, sizeof p);
  return norm_rope(p, q, k, out_q, out_k, q_weight, k_weight, base, offset, B, N, Hq, Hk, D, dtype, norm, eps, inv_freq, nullptr, rot, pairs,
                   stream_ptr);
}

int spec_qk_norm_rope_axes(const spec_heads_t *q, const spec_heads_t *k, const spec_heads_t *out_q, const spec_heads_t *out_k,
                           const void *q_weight, const void *k_weight, const int32_t *base, const int32_t *positions, int axes,
                           int B, int N, int Hq, int Hk, int D, int dtype, int norm, float eps, const double *inv_freq,
                           const int32_t *axis, int rot, int pairs, void *stream_ptr) {
  NvtxRange nvtx_range("spec_qk_norm_rope_axes");
  if (axes < 1 || axes > SPEC_MAX_AXES) return fail(SPEC_ERR_ARG, "axes out of range [1, SPEC_MAX_AXES]");
  NormRopeAxesParams p;
  std::memset(&p, 0, sizeof p);
  p.axes = axes;
  return norm_rope(p, q, k, out_q, out_k, q_weight, k_weight, base, positions, B, N, Hq, Hk, D, dtype, norm, eps, inv_freq, axis, rot, pairs,
                   stream_ptr);
}

int spec_cache_write(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *ctx_len,
                     const int32_t *counts, const spec_heads_t *k, const spec_heads_t *v, int B, int N, int dtype,
                     void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_write");
  CacheWriteParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (!known_dtype(dtype)) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_F32, SPEC_BF16 or SPEC_F16");
  if (N < 0 || N > (1 << 30)) return fail(SPEC_ERR_ARG, "N out of range [0, 2^30]");
  if (B == 0 || N == 0) return SPEC_OK;
  if (!ctx_len || !k || !v || !k->data || !v->data) return fail(SPEC_ERR_ARG, "NULL pointer");
  const int esz = size_of(dtype);
  const spec_heads_t *src[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = src[i]->data;
    p.sb[i] = src[i]->stride_b, p.sn[i] = src[i]->stride_n, p.sh[i] = src[i]->stride_h;
  }
  p.ctx = ctx_len;
  p.counts = counts;
  p.N = N;
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, 1, &w))) return st;
  p.status = w->status;
  const bool vec = vectors(*k, esz) && vectors(*v, esz);
  const int elements = std::min(N, p.c.page) * p.c.D;  // of a block at most
  const void *fn = dtype == SPEC_F32    ? pick_write<DT_F32>(elements, vec)
                   : dtype == SPEC_BF16 ? pick_write<DT_BF16>(elements, vec)
                                        : pick_write<DT_F16>(elements, vec);
  return launch_dependent(fn, dim3(blocks_of(N, p.c.page), static_cast<unsigned>(2 * p.c.Hk), static_cast<unsigned>(B)), elements <= 2048 ? 32 : 256, 0,
                stream, &p, "cache_write_kernel launch");
}

int spec_cache_read(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *start,
                    const int32_t *counts, void *out_k, void *out_v, int B, int N, int dtype, void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_read");
  CacheReadParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (!known_dtype(dtype)) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_F32, SPEC_BF16 or SPEC_F16");
  if (N < 0 || N > (1 << 30)) return fail(SPEC_ERR_ARG, "N out of range [0, 2^30]");
  if (B == 0 || N == 0) return SPEC_OK;
  if (!out_k || !out_v) return fail(SPEC_ERR_ARG, "output pointer is NULL");
  if (!aligned16(out_k) || !aligned16(out_v)) return fail(SPEC_ERR_ALIGN, "the outputs must be 16-byte aligned");
  p.out[0] = out_k, p.out[1] = out_v;
  p.start = start;
  p.counts = counts;
  p.N = N;
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, 1, &w))) return st;
  p.status = w->status;
  const void *fn = dtype == SPEC_F32    ? reinterpret_cast<const void *>(&cache_read_kernel<DT_F32>)
                   : dtype == SPEC_BF16 ? reinterpret_cast<const void *>(&cache_read_kernel<DT_BF16>)
                                        : reinterpret_cast<const void *>(&cache_read_kernel<DT_F16>);
  return launch_dependent(fn, dim3(blocks_of(N, p.c.page), static_cast<unsigned>(p.c.Hk), static_cast<unsigned>(B)), 256, 0, stream, &p,
                "cache_read_kernel launch");
}

int spec_cache_attention(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *ctx_len,
                         const int32_t *counts, const spec_heads_t *q, const uint32_t *mask, int B, int N, int Hq, int dtype,
                         float scale, void *out, float *lse, void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_attention");
  AttnParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_BF16 or SPEC_F16");
  if (N < 0 || N > SPEC_MAX_NEW_TOKENS) return fail(SPEC_ERR_ARG, "N out of range [0, 65536]");
  if (Hq < 1 || Hq > 65535 || Hq % p.c.Hk) return fail(SPEC_ERR_ARG, "Hq must be a multiple of kv_heads, at most 65535");
  if (!std::isfinite(scale)) return fail(SPEC_ERR_ARG, "scale must be finite");
  if (B == 0 || N == 0) return SPEC_OK;
  if (!ctx_len || !q || !q->data || !out) return fail(SPEC_ERR_ARG, "NULL pointer");
  if (!aligned16(out)) return fail(SPEC_ERR_ALIGN, "out must be 16-byte aligned");
  p.q = q->data;
  p.q_sb = q->stride_b, p.q_sn = q->stride_n, p.q_sh = q->stride_h;
  p.out = out;
  p.lse = lse;
  p.ctx = ctx_len;
  p.counts = counts;
  p.mask = mask;
  p.B = B, p.N = N, p.W = (N + 31) / 32, p.G = Hq / p.c.Hk;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.q_vec = vectors(*q, 2);
  const AttnChoice k = choose_attn(p.c.D, p.c.kind, dtype, static_cast<long long>(N) * p.G);
  // the kernels count their work items in 31 bits; a kv head's rows fit 31 bits
  // with them (fewer than 2^16 per token, no more tokens than slots)
  const double row_tiles = std::ceil(static_cast<double>(N) * p.G / k.rows);
  const double steps = std::ceil(static_cast<double>(pages_per_seq) * p.c.page / k.tokens);
  if (static_cast<double>(B) * p.c.Hk * row_tiles * steps >= 2147483648.0)
    return fail(SPEC_ERR_ARG, "B * Hq * N * pages_per_seq is too large");
  const cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic smem)");
  const int grid = num_sms() * k.ctas;
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, (grid * k.work + 3) / 4, &w, static_cast<size_t>(grid)))) return st;
  p.pieces = reinterpret_cast<float *>(w->partials);
  p.done = w->attn_done;
  p.status = w->status;
  return launch_dependent(k.fn, dim3(static_cast<unsigned>(grid)), k.threads, k.smem, stream, &p, "attention kernel launch");
}

int spec_cache_commit(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *ctx_len,
                      const int32_t *parent, int per_sequence, const int32_t *node_tokens, const int32_t *path,
                      const int32_t *length, int B, int N, int path_len, int32_t *out_index, int32_t *out_ctx_len,
                      void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_commit");
  CacheCommitParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (N < 1 || N > SPEC_MAX_TREE_NODES) return fail(SPEC_ERR_ARG, "N out of range [1, 1024]");
  if (path_len < 1 || path_len > N) return fail(SPEC_ERR_ARG, "need 1 <= path_len <= N");
  if (per_sequence != 0 && per_sequence != 1) return fail(SPEC_ERR_ARG, "per_sequence must be 0 or 1");
  if (B == 0) return SPEC_OK;
  if (!ctx_len || !parent || !node_tokens || !path || !length || !out_index || !out_ctx_len)
    return fail(SPEC_ERR_ARG, "NULL pointer");
  p.ctx = ctx_len;
  p.parent = parent;
  p.parent_stride = per_sequence ? N : 0;
  p.tokens = node_tokens;
  p.path = path;
  p.length = length;
  p.N = N, p.P = path_len;
  p.out_index = out_index;
  p.out_ctx = out_ctx_len;
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, 1, &w))) return st;
  p.status = w->status;
  const int share = (2 * p.c.Hk + 7) / 8;  // a warp for each kv head and tensor
  return launch_dependent(reinterpret_cast<const void *>(&cache_commit_kernel), dim3(static_cast<unsigned>(share), static_cast<unsigned>(B)), 256, 0,
                stream, &p, "cache_commit_kernel launch");
}

int spec_cache_weights(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *ctx_len,
                       const int32_t *counts, const spec_heads_t *q, const uint32_t *mask, const float *lse, int B, int N, int Hq,
                       int dtype, float scale, float *weights, void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_weights");
  WeightsParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_BF16 or SPEC_F16");
  if (N < 0 || N > SPEC_MAX_NEW_TOKENS) return fail(SPEC_ERR_ARG, "N out of range [0, 65536]");
  if (Hq < 1 || Hq > 65535 || Hq % p.c.Hk) return fail(SPEC_ERR_ARG, "Hq must be a multiple of kv_heads, at most 65535");
  if (!std::isfinite(scale)) return fail(SPEC_ERR_ARG, "scale must be finite");
  if (B == 0 || N == 0) return SPEC_OK;
  if (!ctx_len || !q || !q->data || !lse || !weights) return fail(SPEC_ERR_ARG, "NULL pointer");
  if (!aligned16(weights)) return fail(SPEC_ERR_ALIGN, "weights must be 16-byte aligned");
  p.q = q->data;
  p.q_sb = q->stride_b, p.q_sn = q->stride_n, p.q_sh = q->stride_h;
  p.lse = const_cast<float *>(lse);
  p.weights = weights;
  p.ctx = ctx_len;
  p.counts = counts;
  p.mask = mask;
  p.B = B, p.N = N, p.W = (N + 31) / 32, p.G = Hq / p.c.Hk;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.q_vec = vectors(*q, 2);
  const long long rows = static_cast<long long>(N) * p.G;
  if (rows > INT_MAX / 2) return fail(SPEC_ERR_ARG, "N * Hq / kv_heads is too large");
  const WeightsChoice k = p.c.D == 128 ? choose_weights<128>(p.c.kind, dtype, rows) : choose_weights<64>(p.c.kind, dtype, rows);
  p.most = k.most;
  const double tiles = std::ceil(static_cast<double>(pages_per_seq) * p.c.page / WTOK);
  if (static_cast<double>(B) * p.c.Hk * tiles >= 2147483648.0) return fail(SPEC_ERR_ARG, "B * kv_heads * pages_per_seq is too large");
  const cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic smem)");
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, 1, &w))) return st;
  p.status = w->status;
  return launch_dependent(k.fn, dim3(static_cast<unsigned>(2 * num_sms())), WT, k.smem, stream, &p, "cache_weights_kernel launch");
}

int spec_cache_evict(const spec_cache_t *cache, const int32_t *page_table, int pages_per_seq, const int32_t *ctx_len, float *weights,
                     int B, int keep, int first, int last, int32_t *out_index, int32_t *out_ctx_len, void *stream_ptr) {
  NvtxRange nvtx_range("spec_cache_evict");
  EvictParams p = {};
  int st = check_cache(cache, page_table, pages_per_seq, B, &p.c);
  if (st) return st;
  if (keep < 1 || keep > (1 << 30)) return fail(SPEC_ERR_ARG, "keep out of range [1, 2^30]");
  if (first < 0 || last < 0 || first > keep || last > keep - first) return fail(SPEC_ERR_ARG, "first and last must be >= 0 and at most keep together");
  if (B == 0) return SPEC_OK;
  if (!ctx_len || !weights || !out_index || !out_ctx_len) return fail(SPEC_ERR_ARG, "NULL pointer");
  if (out_ctx_len == ctx_len) return fail(SPEC_ERR_ARG, "out_ctx_len must not be ctx_len");
  if (!aligned16(weights)) return fail(SPEC_ERR_ALIGN, "weights must be 16-byte aligned");
  p.ctx = ctx_len;
  p.weights = weights;
  p.keep = keep, p.first = first, p.last = last;
  p.out_index = out_index;
  p.out_ctx = out_ctx_len;
  const void *select = reinterpret_cast<const void *>(&evict_select_kernel), *move = reinterpret_cast<const void *>(&evict_move_kernel);
  cudaError_t e = cudaFuncSetAttribute(move, cudaFuncAttributeMaxDynamicSharedMemorySize, EM_SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_SMEM);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic smem)");
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if ((st = get_ws(stream, 1, &w))) return st;
  p.status = w->status;
  // CTAs of a cluster: up to 8, as far as there is work for them and all of them
  // run together
  const auto cluster = [](long long work, long long groups, int per_sm) {
    unsigned n = 1;
    while (n < 8 && n < work && 2 * n * groups <= static_cast<long long>(per_sm) * num_sms()) n *= 2;
    return n;
  };
  const unsigned Hk = static_cast<unsigned>(p.c.Hk), batch = static_cast<unsigned>(B);
  const long long heads = static_cast<long long>(Hk) * batch, slots = static_cast<long long>(p.c.per) * p.c.page;
  // One CTA as far as its shared memory holds the slots, and more where few heads
  // leave SMs idle.  (64 heads of up to 32768 slots, the whole call: one CTA 54 us,
  // two 52; 8 heads of 32768: one 34 us, four 25.)
  unsigned n = 1;
  while (n < 8 && (static_cast<long long>(n) * EV_SLICE < slots || (n * 8192ll < slots && 2 * n * heads <= num_sms()))) n *= 2;
  if ((st = launch_dependent(select, dim3(Hk * n, batch), EV_NT, EV_SMEM, stream, &p, "evict_select_kernel launch", n))) return st;
  const int rows = EM_BYTES / p.c.D;
  n = cluster((keep + rows - 1) / rows, 2 * heads, 4);
  return launch_dependent(move, dim3(2 * Hk * n, batch), EM_NT, EM_SMEM, stream, &p, "evict_move_kernel launch", n);
}

}  // extern "C"
