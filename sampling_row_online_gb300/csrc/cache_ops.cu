// Host side of the operators around the paged 8-bit key/value cache: argument
// validation, launch geometry and the C ABI declared in include/spec_verify.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "attention.cuh"
#include "attention_tile.cuh"
#include "cache.cuh"
#include "host.h"
#include "spec_verify.h"

namespace spec {
namespace {

bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
int size_of(int dtype) { return dtype == SPEC_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype == SPEC_F32 || dtype == SPEC_BF16 || dtype == SPEC_F16; }

// 16-byte vectors may be used at every row of h.
bool vectors(const spec_heads_t &h, int esz) {
  return aligned16(h.data) && h.stride_b * esz % 16 == 0 && h.stride_n * esz % 16 == 0 && h.stride_h * esz % 16 == 0;
}

// Launches as a programmatic dependent of what precedes it on the stream.
int launch(const void *fn, dim3 grid, int threads, int smem, cudaStream_t stream, void *params, const char *what) {
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  void *args[] = {params};
  const cudaError_t e = launch_kernel(&cfg, fn, args);
  return e == cudaSuccess ? static_cast<int>(SPEC_OK) : cuda_fail(e, what);
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
template <int DT>
const void *pick_norm_rope(bool vec, bool one, bool pairs) {
  if (vec && one)
    return pairs ? reinterpret_cast<const void *>(&norm_rope_rows_kernel<DT, true>)
                 : reinterpret_cast<const void *>(&norm_rope_rows_kernel<DT, false>);
  if (vec) return reinterpret_cast<const void *>(&norm_rope_kernel<DT, 8, 2>);
  return pairs ? reinterpret_cast<const void *>(&norm_rope_kernel<DT, 2, 8>)
               : reinterpret_cast<const void *>(&norm_rope_kernel<DT, 1, 16>);
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

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" {

int spec_qk_norm_rope(const spec_heads_t *q, const spec_heads_t *k, const spec_heads_t *out_q, const spec_heads_t *out_k,
                      const void *q_weight, const void *k_weight, const int32_t *base, const int32_t *offset, int B, int N,
                      int Hq, int Hk, int D, int dtype, int norm, float eps, const double *inv_freq, int rot, int pairs,
                      void *stream_ptr) {
  NvtxRange nvtx_range("spec_qk_norm_rope");
  if (!known_dtype(dtype)) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_F32, SPEC_BF16 or SPEC_F16");
  if (B < 0 || N < 0 || static_cast<long long>(B) * N > INT_MAX / 2) return fail(SPEC_ERR_ARG, "B and N must be >= 0 and B * N < 2^30");
  if (Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535) return fail(SPEC_ERR_ARG, "head counts out of range [0, 65535]");
  if (D < 2 || D > 512 || D % 2) return fail(SPEC_ERR_ARG, "head_dim must be even and in [2, 512]");
  if (rot < 0 || rot > D || rot % 2) return fail(SPEC_ERR_ARG, "rot must be even and in [0, head_dim]");
  if (norm != 0 && norm != 1) return fail(SPEC_ERR_ARG, "norm must be 0 or 1");
  if (pairs != 0 && pairs != 1) return fail(SPEC_ERR_ARG, "pairs must be 0 or 1");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SPEC_ERR_ARG, "eps must be finite and >= 0");
  if (rot > 0 && !inv_freq) return fail(SPEC_ERR_ARG, "inv_freq is NULL");
  if (!norm && (q_weight || k_weight)) return fail(SPEC_ERR_ARG, "weights are given without the norm");
  if (B == 0 || N == 0 || Hq + Hk == 0) return SPEC_OK;
  if ((Hq > 0 && (!q || !out_q || !q->data || !out_q->data)) || (Hk > 0 && (!k || !out_k || !k->data || !out_k->data)))
    return fail(SPEC_ERR_ARG, "a tensor is NULL");
  const int esz = size_of(dtype);
  NormRopeParams p;
  std::memset(&p, 0, sizeof p);
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
  const void *fn = dtype == SPEC_F32    ? pick_norm_rope<DT_F32>(vec, units <= p.lanes, pairs)
                   : dtype == SPEC_BF16 ? pick_norm_rope<DT_BF16>(vec, units <= p.lanes, pairs)
                                        : pick_norm_rope<DT_F16>(vec, units <= p.lanes, pairs);
  return launch(fn, dim3(static_cast<unsigned>((tokens + p.per_cta - 1) / p.per_cta), tensors), 256,
                p.per_cta * (rot / 2) * static_cast<int>(sizeof(float2)), static_cast<cudaStream_t>(stream_ptr), &p,
                "norm_rope_kernel launch");
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
  return launch(fn, dim3(blocks_of(N, p.c.page), static_cast<unsigned>(2 * p.c.Hk), static_cast<unsigned>(B)), elements <= 2048 ? 32 : 256, 0,
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
  return launch(fn, dim3(blocks_of(N, p.c.page), static_cast<unsigned>(p.c.Hk), static_cast<unsigned>(B)), 256, 0, stream, &p,
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
  return launch(k.fn, dim3(static_cast<unsigned>(grid)), k.threads, k.smem, stream, &p, "attention kernel launch");
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
  return launch(reinterpret_cast<const void *>(&cache_commit_kernel), dim3(static_cast<unsigned>(share), static_cast<unsigned>(B)), 256, 0,
                stream, &p, "cache_commit_kernel launch");
}

}  // extern "C"
