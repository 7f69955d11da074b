// Kernels around the paged 8-bit key/value cache: the norms and the rotation
// of queries and keys, the quantised write, the read-back, and the commit of
// an accepted path.  All of them are bound by memory traffic or, at the sizes
// of a decoding step, by the latency of a few dependent loads; none holds a
// contraction.
//
// A block is one page of one kv head: page_size rows of D codes, contiguous,
// with one fp32 scale; a value is code * scale.  The scales that these
// kernels give are powers of two (the least with amax <= qmax * scale, at
// least 2^-100).  So the division of a value by its scale is exact, an e4m3
// code that moves to a larger scale changes its exponent only (no second
// rounding unless it becomes subnormal), and the stored bits are a function
// of the inputs that any fp32 arithmetic reproduces.
#pragma once

#include <cstdint>
#include <type_traits>

#include "device.cuh"
#include "elements.cuh"
#include "ptx.cuh"

namespace spec {

constexpr int KIND_E4M3 = 0, KIND_I8 = 1;           // SPEC_E4M3, SPEC_I8
constexpr int MAX_ROPE = 256;                       // rotated pairs per head

struct CacheView {  // spec_cache_t and the call's page table
  unsigned char *k, *v;       // codes [pages, Hk, page, D]
  float *k_scale, *v_scale;   // [pages, Hk]
  const int32_t *table;       // [B, per]
  int pages, Hk, page, log_page, D, kind, per;
};

// ---------------------------------------------------------------- codes
// Four codes of a word as fp32.
__device__ __forceinline__ void decode4(int kind, uint32_t w, float (&x)[4]) {
  if (kind == KIND_E4M3) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 f = f16x2_to_f32(lo), g = f16x2_to_f32(hi);
    x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
  } else {  // the code + 128 as the low bits of 2^23 + code + 128; conversion instructions run at a quarter of the rate
    w ^= 0x80808080u;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | j)) - 8388736.f;
  }
}
// Four fp32 values (already divided by the scale) as codes: nearest, ties to
// even; infinities become +-qmax, NaN 0.
__device__ __forceinline__ uint32_t encode4(int kind, float a, float b, float c, float d) {
  if (kind == KIND_E4M3) {
    a = a == a ? a : 0.f, b = b == b ? b : 0.f, c = c == c ? c : 0.f, d = d == d ? d : 0.f;
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | static_cast<uint32_t>(hi) << 16;
  }
  const float x[4] = {a, b, c, d};
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)  // adding 1.5 * 2^23 rounds to a whole number in the sum's low bits
    u[j] = __float_as_uint(__fadd_rn(fminf(fmaxf(x[j] == x[j] ? x[j] : 0.f, -127.f), 127.f), 12582912.f));
  return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}
// As encode4 for finite values: a_j * inv with inv a power of two.  int8:
// adding 1.5 * 2^23 rounds to a whole number in the sum's low bits.
__device__ __forceinline__ uint32_t encode4_finite(int kind, float a, float b, float c, float d, float inv) {
  if (kind == KIND_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
    return lo | static_cast<uint32_t>(hi) << 16;
  }
  const uint32_t x = __float_as_uint(fmaf(a, inv, 12582912.f)), y = __float_as_uint(fmaf(b, inv, 12582912.f));
  const uint32_t z = __float_as_uint(fmaf(c, inv, 12582912.f)), w = __float_as_uint(fmaf(d, inv, 12582912.f));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}
// Largest magnitude of eight elements, as fp32 bits (inf and NaN: 0x7f800000
// and above); 16-bit types are compared as bits, two at a time.
template <int DT>
__device__ __forceinline__ uint32_t magnitude8(const Raw8<DT> &r, uint32_t sofar) {
  if constexpr (DT == DT_F32) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) sofar = max(sofar, w[j] & 0x7fffffffu);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("max.u16x2 %0, %0, %1;" : "+r"(sofar) : "r"(w[j] & 0x7fff7fffu));
  }
  return sofar;
}
template <int DT>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t x) {  // of what magnitude8 gathered
  if constexpr (DT == DT_F32) return x;
  const uint32_t h = max(x & 0xffffu, x >> 16);
  return DT == DT_BF16 ? h << 16 : __float_as_uint(f16x2_to_f32(h).x);
}

// The least power of two with amax <= qmax * scale, at least 2^-100, from the
// bits of amax: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6.
__device__ __forceinline__ float scale_for(int kind, uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  const uint32_t m = amax_bits & 0x7fffffu;
  const int s = kind == KIND_E4M3 ? e - 8 + (m > 0x600000u) : e - 6 + (m > 0x7e0000u);
  return __uint_as_float(static_cast<uint32_t>(max(s, -100) + 127) << 23);
}

// The page of block `blk` of sequence b, or -1 (and a status bit).
__device__ __forceinline__ int page_of(const CacheView &c, int b, int blk, int32_t *status) {
  const int id = c.table[static_cast<long long>(b) * c.per + blk];
  if (static_cast<unsigned>(id) < static_cast<unsigned>(c.pages)) return id;
  atomicOr(status, ST_PAGE);
  return -1;
}

// Rounds the rows of a block outside [lo, hi) to a larger scale (ratio =
// old / new < 1), 16 codes at a time; thread `tid` of NTH.  A single warp reads
// four times before it writes.
template <int NTH>
__device__ __forceinline__ void rescale_block(unsigned char *blk, int kind, int page, int D, int lo, int hi, float ratio, int tid) {
  constexpr int FLY = NTH == 32 ? 4 : 1;
  const int log_row = D == 128 ? 3 : 2, chunks = page << log_row;
  uint4 *at = reinterpret_cast<uint4 *>(blk);
  for (int c0 = tid; c0 < chunks; c0 += NTH * FLY) {
    uint4 w[FLY];
    bool mine[FLY];
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int c = c0 + i * NTH, row = c >> log_row;
      mine[i] = c < chunks && (row < lo || row >= hi);
      if (mine[i]) w[i] = at[c];
    }
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      if (!mine[i]) continue;
      uint32_t *u = &w[i].x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[4];
        decode4(kind, u[j], x);
        u[j] = encode4(kind, x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
      }
      at[c0 + i * NTH] = w[i];
    }
  }
}

// Maximum over a block of NTH threads of non-negative fp32 bits.
template <int NTH>
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t *s) {
  x = __reduce_max_sync(0xffffffffu, x);
  if (NTH == 32) return x;
  __syncthreads();  // the previous use of s is over
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = s[0];
#pragma unroll
  for (int i = 1; i < NTH / 32; ++i) x = max(x, s[i]);
  return x;
}

// ------------------------------------------------- quantised cache write
struct CacheWriteParams {
  CacheView c;
  const void *src[2];          // keys, values: [B, N, Hk, D] with strides in elements
  long long sb[2], sn[2], sh[2];
  const int32_t *ctx, *counts;
  int N;
  int32_t *status;
};

// One CTA per (block that the new rows may touch, kv head and tensor,
// sequence).  The new rows of the block are read once and kept in registers
// (MOST chunks of eight a thread), their maximum gives the scale, and the
// codes follow: 3 bytes of traffic per 16-bit element, the floor.  The block
// is re-read only where its scale grows under rows that it already holds.
// 8 sequences of up to 8000 rows, bf16 to int8: 49 us, 6.0 TB/s (the floor is
// 43.5); one row each of 64 sequences: 2.7 us, the latency of length, page and
// row.
template <int DT, int NTH, int MOST, bool VEC>
__global__ void __launch_bounds__(NTH, NTH == 256 && DT != DT_F32 ? (MOST == 4 ? 5 : 4) : 1) cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
  __shared__ uint32_t s_max[NTH / 32];
  const CacheView &c = p.c;
  const int b = blockIdx.z, h = blockIdx.y >> 1, t = blockIdx.y & 1;
  pdl_wait();
  pdl_launch_dependents();
  const int start = p.ctx[b], count = p.counts ? p.counts[b] : p.N;
  if (start < 0 || count < 0 || count > p.N || static_cast<long long>(start) + count > static_cast<long long>(c.per) * c.page) {
    if (threadIdx.x == 0) atomicOr(p.status, ST_SLOTS);
    return;
  }
  const int blk = (start >> c.log_page) + blockIdx.x;
  const int first = blk << c.log_page;  // of the block; may pass the last slot, then nothing is left below
  const int lo = max(start, first), hi = min(start + count, first + c.page);
  if (hi <= lo) return;
  const int page = page_of(c, b, blk, p.status);
  if (page < 0) return;
  const long long id = static_cast<long long>(page) * c.Hk + h;
  float *scale_at = (t ? c.v_scale : c.k_scale) + id;
  unsigned char *codes = (t ? c.v : c.k) + id * c.page * c.D;
  const bool empty = first >= start;  // the block holds nothing before the new rows
  const float old = empty ? 0.f : *scale_at;

  const int log_row = c.D == 128 ? 4 : 3, chunks = (hi - lo) << log_row;  // 16 or 8 chunks to a row
  const int row0 = threadIdx.x >> log_row, col = (threadIdx.x & ((1 << log_row) - 1)) * 8;
  // a thread's chunks are NTH / 16 or NTH / 8 rows apart
  const long long base = b * p.sb[t] + h * p.sh[t] + (lo - start + row0) * p.sn[t] + col, apart = (NTH >> log_row) * p.sn[t];
  Raw8<DT> raw[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    if (threadIdx.x + i * NTH < chunks) raw[i] = load8<DT, VEC>(p.src[t], base + i * apart);
  }
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    if (threadIdx.x + i * NTH < chunks) amax = magnitude8<DT>(raw[i], amax);
  amax = block_max<NTH>(magnitude_bits<DT>(amax), s_max);
  const bool finite = amax < 0x7f800000u;
  if (!finite) {  // the largest finite magnitude, and a report
    amax = 0;
#pragma unroll 1
    for (int i = 0; i < MOST; ++i) {
      const int k = threadIdx.x + i * NTH;
      if (k >= chunks) break;
      float x[8];
      unpack8<DT>(load8<DT, VEC>(p.src[t], base + i * apart), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t y = __float_as_uint(x[j]) & 0x7fffffffu;
        if (y < 0x7f800000u) amax = max(amax, y);
      }
    }
    amax = block_max<NTH>(amax, s_max);
    if (threadIdx.x == 0) atomicOr(p.status, ST_NONFINITE);
  }
  const float scale = fmaxf(scale_for(c.kind, amax), old);
  if (threadIdx.x == 0) *scale_at = scale;  // every thread has read the old one before the maximum's barrier
  const float inv = 1.f / scale;            // exact for powers of two
  const bool simple = finite && (__float_as_uint(scale) & 0x7fffffu) == 0;
  unsigned char *to = codes + static_cast<long long>(lo - first) * c.D;
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int k = threadIdx.x + i * NTH;
    if (k < chunks) {
      float x[8];
      unpack8<DT>(raw[i], x);
      uint2 w;
      if (simple) {
        w.x = encode4_finite(c.kind, x[0], x[1], x[2], x[3], inv);
        w.y = encode4_finite(c.kind, x[4], x[5], x[6], x[7], inv);
      } else {
        w.x = encode4(c.kind, x[0] / scale, x[1] / scale, x[2] / scale, x[3] / scale);
        w.y = encode4(c.kind, x[4] / scale, x[5] / scale, x[6] / scale, x[7] / scale);
      }
      *reinterpret_cast<uint2 *>(to + k * 8) = w;  // the block's rows are contiguous
    }
  }
  if (!empty && scale > old) rescale_block<NTH>(codes, c.kind, c.page, c.D, lo - first, hi - first, old / scale, threadIdx.x);
}

// ------------------------------------------------------------- read-back
struct CacheReadParams {
  CacheView c;
  void *out[2];  // [B, N, Hk, D]
  const int32_t *start, *counts;
  int N;
  int32_t *status;
};

// One CTA per (block, kv head, sequence): the block's rows of both tensors,
// 16 codes to a thread; rows past the count are zero, a sequence that does
// not fit its pages and the rows of a bad page are NaN.  Bound by HBM: 8
// sequences of up to 32768 rows, e4m3 to bf16, 234 us, 6.3 TB/s with the zeros.
template <int DT>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheReadParams p) {
  const CacheView &c = p.c;
  const int b = blockIdx.z, h = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  int start = p.start ? p.start[b] : 0, count = p.counts ? p.counts[b] : p.N;
  float fill = 0.f;
  if (start < 0 || count < 0 || count > p.N || static_cast<long long>(start) + count > static_cast<long long>(c.per) * c.page) {
    if (threadIdx.x == 0) atomicOr(p.status, ST_SLOTS);
    start = count = 0;
    fill = __uint_as_float(0x7fc00000u);
  }
  const int blk = (start >> c.log_page) + blockIdx.x;
  const long long first = static_cast<long long>(blk) << c.log_page;
  const int lo = static_cast<int>(max(static_cast<long long>(start), first) - start);  // rows of the output
  const int hi = static_cast<int>(min(static_cast<long long>(p.N), first + c.page - start));
  const int held = min(hi, count);
  int page = -1;
  if (held > lo && (page = page_of(c, b, blk, p.status)) < 0) fill = __uint_as_float(0x7fc00000u);
  const long long id = static_cast<long long>(max(page, 0)) * c.Hk + h;
  const int per_row = c.D / 16;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float scale = (t ? c.v_scale : c.k_scale)[id];
    const unsigned char *codes = (t ? c.v : c.k) + id * c.page * c.D;
    for (int k = threadIdx.x; k < (hi - lo) * per_row; k += 256) {
      const int row = lo + k / per_row, d = (k % per_row) * 16;
      float x[16];
      if (row < held && page >= 0) {
        const uint4 w = ldg_na(reinterpret_cast<const uint4 *>(codes + (start + row - first) * c.D + d));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float y[4];
          decode4(c.kind, u[j], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * j + e] = y[e] * scale;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = row < held || count == 0 ? fill : 0.f;
      }
      const long long o = ((static_cast<long long>(b) * p.N + row) * c.Hk + h) * c.D + d;
      float lo8[8], hi8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) lo8[j] = x[j], hi8[j] = x[8 + j];
      store8<DT, true>(p.out[t], o, pack8<DT>(lo8));
      store8<DT, true>(p.out[t], o + 8, pack8<DT>(hi8));
    }
  }
}

// --------------------------------------------- commit of an accepted path
struct CacheCommitParams {
  CacheView c;
  const int32_t *ctx, *parent, *tokens, *path, *length;
  int N, P, parent_stride;  // parent_stride: 0 (one tree) or N
  int32_t *out_index, *out_ctx;
  int32_t *status;
};
constexpr int COMMIT_MAX_NODES = 1024;

// A few CTAs per sequence share its kv heads and tensors, so that the path is
// found a few times only.  The nodes of the accepted path:
// every thread walks from its nodes towards the root comparing tokens (the
// token of depth d is path[d - 1]) and the lowest index that arrives wins;
// equal token paths hold equal rows, so which of several is taken does not
// matter.  Node i of the path moves from slot ctx + index[i] to ctx + i.
// index[i] >= i, so with the rows taken in ascending order none is overwritten
// before it has been read.  A warp takes a kv head and tensor by itself: it
// reads a block's new rows once for their maximum and once more (from L2) to
// write them, unless they fit its registers.  The bytes are few; the latency of
// walk and reads counts, and with four CTAs per SM the issue slots: 32 trees of
// 63 nodes 4.3 us, 256 of 255 nodes 10.3 us (four vectors in flight 11.0, with
// spills; a division and conversion instructions for each element 18; a CTA per
// head and tensor 32; one with a barrier per block 46).
__global__ void __launch_bounds__(256, 4) cache_commit_kernel(const __grid_constant__ CacheCommitParams p) {
  __shared__ int s_par[COMMIT_MAX_NODES], s_tok[COMMIT_MAX_NODES], s_path[COMMIT_MAX_NODES], s_index[COMMIT_MAX_NODES];
  __shared__ int s_node, s_bad, s_first;
  const CacheView &c = p.c;
  const int b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.length[b], ctx = p.ctx[b];
  if (threadIdx.x == 0) s_node = INT32_MAX, s_bad = 0, s_first = INT32_MAX;
  const bool fits = len >= 1 && len <= min(p.P, p.N);
  for (int i = threadIdx.x; i < p.N; i += 256) {
    s_par[i] = p.parent[static_cast<long long>(b) * p.parent_stride + i];
    s_tok[i] = p.tokens[static_cast<long long>(b) * p.N + i];
  }
  if (fits)
    for (int i = threadIdx.x; i < len - 1; i += 256) s_path[i] = p.path[static_cast<long long>(b) * p.P + i];
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += 256)
    if (i == 0 ? s_par[i] != -1 : s_par[i] < 0 || s_par[i] >= i) s_bad = 1;
  __syncthreads();
  if (fits && !s_bad)
    for (int i = threadIdx.x; i < p.N; i += 256) {
      int at = i, d = len - 1;
      while (d > 0 && at > 0 && s_tok[at] == s_path[d - 1]) at = s_par[at], --d;
      if (d == 0 && at == 0) atomicMin(&s_node, i);
    }
  __syncthreads();
  // length -1 marks an error that the verification has reported already
  const bool tree_ok = fits && !s_bad && s_node != INT32_MAX;
  const bool slots_ok = ctx >= 0 && (!tree_ok || static_cast<long long>(ctx) + s_node < static_cast<long long>(c.per) * c.page);
  const bool ok = tree_ok && slots_ok;
  if (threadIdx.x == 0) {
    if (!tree_ok && len != -1) atomicOr(p.status, ST_PARENT);
    if (!slots_ok) atomicOr(p.status, ST_SLOTS);
    if (ok)
      for (int at = s_node, d = len - 1; d >= 0; at = s_par[at], --d) {
        s_index[d] = at;
        if (at != d) s_first = d;
      }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.P; i += 256)
      p.out_index[static_cast<long long>(b) * p.P + i] = ok && i < len ? s_index[i] : -1;
    if (threadIdx.x == 0) p.out_ctx[b] = ok ? ctx + len : ctx;
  }
  if (!ok || s_first >= len) return;

  // the pages of the path's rows, over the tokens of the path (done with)
  int *s_page = s_path;
  for (int i = s_first + threadIdx.x; i < len; i += 256) s_page[i] = page_of(c, b, (ctx + s_index[i]) >> c.log_page, p.status);
  __syncthreads();

  constexpr int BATCH = 2;  // vectors of 16 codes per lane in flight
  const int lane = threadIdx.x & 31, log_row = c.D == 128 ? 3 : 2;  // vectors of a row: 8 or 4
  for (int ht = blockIdx.x * 8 + (threadIdx.x >> 5); ht < 2 * c.Hk; ht += gridDim.x * 8) {
    const int h = ht >> 1;
    unsigned char *base = ht & 1 ? c.v : c.k;
    float *scales = ht & 1 ? c.v_scale : c.k_scale;
    for (int row = s_first; row < len;) {
      const int in = (ctx + row) & (c.page - 1), n = min(len - row, c.page - in), vectors = n << log_row;
      const int page = page_of(c, b, (ctx + row) >> c.log_page, p.status);
      const long long id = static_cast<long long>(max(page, 0)) * c.Hk + h;
      const float old = scales[id];
      uint4 raw[BATCH];
      float from[BATCH];  // scales of the vectors; -1: a bad page, or past the last row
      const auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int k = k0 + 32 * i, r = row + (k >> log_row);
          raw[i] = make_uint4(0, 0, 0, 0);
          from[i] = -1.f;
          if (k >= vectors || s_page[r] < 0) continue;
          const long long at = static_cast<long long>(s_page[r]) * c.Hk + h;
          const int slot = (ctx + s_index[r]) & (c.page - 1);
          from[i] = scales[at];
          raw[i] = reinterpret_cast<const uint4 *>(base + (at * c.page + slot) * c.D)[k & ((1 << log_row) - 1)];
        }
      };
      uint32_t amax = 0;
      for (int k0 = lane; k0 - lane < vectors; k0 += 32 * BATCH) {
        load(k0);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          float x[4], most = 0.f;  // fmaxf passes over NaN
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            decode4(c.kind, u[j], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(x[e]));
          }
          if (!(from[i] >= 0.f)) continue;
          most *= from[i];
          if (most < INFINITY) {  // false for NaN
            amax = max(amax, __float_as_uint(fabsf(most)));  // not a negative zero
          } else {  // a huge scale: the largest of the finite products
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              decode4(c.kind, j < 2 ? (j ? raw[i].y : raw[i].x) : (j == 2 ? raw[i].z : raw[i].w), x);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = fabsf(x[e] * from[i]);
                if (a < INFINITY) amax = max(amax, __float_as_uint(a));
              }
            }
          }
        }
      }
      amax = __reduce_max_sync(0xffffffffu, amax);
      // a block's scale never shrinks here: the rows of other nodes still stand in it
      const float scale = fmaxf(scale_for(c.kind, amax), old);
      unsigned char *codes = base + id * c.page * c.D;
      // powers of two (every scale of this library's own): the product with
      // the inverse is the quotient
      const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
      const float inv = 1.f / scale;
      for (int k0 = lane; page >= 0 && k0 - lane < vectors; k0 += 32 * BATCH) {
        if (vectors > 32 * BATCH) load(k0);  // else they are in registers
        __syncwarp();
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          if (from[i] < 0.f) continue;
          uint32_t *u = &raw[i].x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[4];
            decode4(c.kind, u[j], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= from[i];
            if (exact) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] *= inv;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] /= scale;
            }
            u[j] = encode4(c.kind, x[0], x[1], x[2], x[3]);
          }
          reinterpret_cast<uint4 *>(codes + static_cast<long long>(in) * c.D)[k0 + 32 * i] = raw[i];
        }
        __syncwarp();
      }
      if (page >= 0 && scale > old) {
        if (lane == 0) scales[id] = scale;
        rescale_block<32>(codes, c.kind, c.page, c.D, in, in + n, old / scale, lane);
      }
      __syncwarp();
      row += n;
    }
  }
}

// ------------------------------- norms of queries and keys with the rotation
struct NormRopeParams {
  const void *src[2];  // queries, keys
  void *dst[2];
  const void *weight[2];
  long long ssb[2], ssn[2], ssh[2], dsb[2], dsn[2], dsh[2];  // strides in elements
  int heads[2];
  const int32_t *base, *offset;
  int B, N, D, rot, per_cta;  // per_cta: tokens per CTA
  int norm, pairs, lanes;     // lanes: threads per row (a power of two, <= 32)
  float eps;
  unsigned long long freq[MAX_ROPE];  // 2^64 turns per position, modulo 2^64
};
// The same for positions with several axes: offset is [B, N, axes], and pair i
// turns by the position on axis[i].
struct NormRopeAxesParams : NormRopeParams {
  int axes;
  uint8_t axis[MAX_ROPE];
};
// The position of token `tok` (token n of sequence b) that pair i turns by;
// `axis`: what axis_of gave for it.
template <class P>
__device__ __forceinline__ int axis_of(const P &p, int i) {
  if constexpr (std::is_same_v<P, NormRopeAxesParams>) return p.axis[i];
  return 0;
}
template <class P>
__device__ __forceinline__ long long position_of(const P &p, int tok, int b, int axis) {
  const long long base = p.base ? p.base[b] : 0;
  if constexpr (std::is_same_v<P, NormRopeAxesParams>) return base + p.offset[static_cast<long long>(tok) * p.axes + axis];
  return base + (p.offset ? p.offset[tok] : tok - b * p.N);
}

// Several tokens to a CTA, `lanes` threads to a row (one head of one token).
// A thread takes units of the row: eight elements of the first half with the
// eight that they are rotated with (halves), or eight elements by themselves
// (neighbouring pairs, and what is not rotated).  The rotation's angle is
// exact: pos * freq modulo 2^64 is the fraction of a turn in 64 bits, from
// which 24 go into sincospi; a table of the CTA's tokens holds cos and sin, so
// that all heads share them.  This form takes any even head size, stride and
// alignment: single elements, or two for neighbouring pairs, where vectors do
// not fit.
constexpr int ROPE_TOKENS = 16;  // most tokens of a CTA
template <int DT, int VE, int MAXU, class P = NormRopeParams>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ P p) {
  extern __shared__ float2 s_trig[];  // [per_cta][rot / 2]
  __shared__ long long s_from[ROPE_TOKENS][2], s_to[ROPE_TOKENS][2];
  const int half = p.rot / 2;
  const int tokens = p.B * p.N, first = blockIdx.x * p.per_cta, here = min(p.per_cta, tokens - first);
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 2 * here) {
    const int tk = threadIdx.x >> 1, w = threadIdx.x & 1, b = (first + tk) / p.N, n = (first + tk) - b * p.N;
    s_from[tk][w] = b * p.ssb[w] + n * p.ssn[w];
    s_to[tk][w] = b * p.dsb[w] + n * p.dsn[w];
  }
  for (int i = threadIdx.x; i < here * half; i += 256) {
    const int tk = i / half, tok = first + tk, b = tok / p.N;
    const long long pos = position_of(p, tok, b, axis_of(p, i - tk * half));
    const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freq[i - tk * half];
    // signed fraction of a turn times two, in units of pi
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    s_trig[i] = make_float2(c, s);
  }
  __syncthreads();
  const int heads = p.heads[0] + p.heads[1];
  const int lane = threadIdx.x & (p.lanes - 1);
  const int npair = p.pairs ? 0 : half / VE;         // units of two vectors
  const int units = npair + (p.D - 2 * npair * VE) / VE;
  const int nrot = p.pairs ? p.rot / VE : npair;     // units that are rotated
  const int rows = here * heads, step = 256 / p.lanes;
  const float over_d = 1.f / static_cast<float>(p.D);
  const auto place = [&](int u) { return u < npair ? u * VE : (npair + u) * VE; };  // a unit's first element
  // every thread runs the same number of turns: the row sums are shuffles
  for (int row0 = threadIdx.x / p.lanes; row0 - static_cast<int>(threadIdx.x) / p.lanes < rows; row0 += step) {
    Raw8<DT> raw[VE == 8 ? MAXU : 1][2];
    float single[VE == 8 ? 1 : MAXU][2][VE];
    const bool live = row0 < rows;
    const int tk = live ? row0 / heads : 0, hh = row0 - tk * heads;
    const int w = hh >= p.heads[0], h = hh - (w ? p.heads[0] : 0);
    if (live) {
      const long long from = s_from[tk][w] + h * p.ssh[w];
#pragma unroll
      for (int i = 0; i < MAXU; ++i) {
        const int u = lane + i * p.lanes;
        if (u >= units) continue;
        if constexpr (VE == 8) {
          raw[i][0] = load8<DT, true>(p.src[w], from + place(u));
          if (u < npair) raw[i][1] = load8<DT, true>(p.src[w], from + place(u) + half);
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            single[i][0][j] = one_element<DT>(p.src[w], from + place(u) + j);
            if (u < npair) single[i][1][j] = one_element<DT>(p.src[w], from + place(u) + half + j);
          }
        }
      }
    }
    {
      float r = 1.f;
      if (p.norm) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < MAXU; ++i) {
          const int u = lane + i * p.lanes;
          if (!live || u >= units) continue;
          float x[VE];
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            if (side == 1 && u >= npair) continue;
            if constexpr (VE == 8) unpack8<DT>(raw[i][side], x);
            else
#pragma unroll
              for (int j = 0; j < VE; ++j) x[j] = single[i][side][j];
#pragma unroll
            for (int j = 0; j < VE; ++j) sum = fmaf(x[j], x[j], sum);
          }
        }
        for (int o = p.lanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        r = rsqrtf(fmaf(sum, over_d, p.eps));
      }
      if (!live) continue;
      const void *weight = p.weight[w];
      const float2 *trig = s_trig + tk * half;
      const long long to = s_to[tk][w] + h * p.dsh[w];
#pragma unroll
      for (int i = 0; i < MAXU; ++i) {
        const int u = lane + i * p.lanes;
        if (u >= units) continue;
        const int at = place(u);
        const bool two = u < npair;
        float x[2][VE];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          if (side == 1 && !two) continue;
          if constexpr (VE == 8) unpack8<DT>(raw[i][side], x[side]);
          else
#pragma unroll
            for (int j = 0; j < VE; ++j) x[side][j] = single[i][side][j];
          if (weight) {
            float g[VE];
            if constexpr (VE == 8) unpack8<DT>(load8<DT, true>(weight, at + side * half), g);
            else
#pragma unroll
              for (int j = 0; j < VE; ++j) g[j] = one_element<DT>(weight, at + side * half + j);
#pragma unroll
            for (int j = 0; j < VE; ++j) x[side][j] *= r * g[j];
          } else {
#pragma unroll
            for (int j = 0; j < VE; ++j) x[side][j] *= r;
          }
        }
        if (two) {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float2 cs = trig[at + j];
            const float a = x[0][j], c = x[1][j];
            x[0][j] = a * cs.x - c * cs.y;
            x[1][j] = c * cs.x + a * cs.y;
          }
        } else if (u < nrot) {
          if constexpr (VE > 1) {
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
              const float2 cs = trig[(at + j) / 2];
              const float a = x[0][j], c = x[0][j + 1];
              x[0][j] = a * cs.x - c * cs.y;
              x[0][j + 1] = c * cs.x + a * cs.y;
            }
          }
        }
        if constexpr (VE == 8) {
          store8<DT, true>(p.dst[w], to + at, pack8<DT>(x[0]));
          if (two) store8<DT, true>(p.dst[w], to + at + half, pack8<DT>(x[1]));
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            put_element<DT>(p.dst[w], to + at + j, x[0][j]);
            if (two) put_element<DT>(p.dst[w], to + at + half + j, x[1][j]);
          }
        }
      }
    }
  }
}

// The same for rows of whole vectors with one unit to a thread, which is every
// usual head: two rows in flight, the weights in registers, a CTA for the
// queries or the keys of its tokens (blockIdx.y).  What a row costs is
// instructions (about 85 a vector), so nothing is divided or looked up per
// row.  16380 tokens, 40 heads of 128, bf16: half of the head rotated in
// neighbouring pairs 66.5 us, 5.0 TB/s, bound by issue (the kernel above took
// 112); the whole head in two halves 71.9 us, 4.7 TB/s, with two units of a row to a
// thread and 36 bytes of spills each way (fp32: 104.9 us, 12 bytes).  With three axes
// 68.6 and 75.5 us (52 bytes; fp32 106.6).
template <int DT, bool PAIRS, class P = NormRopeParams>
__global__ void __launch_bounds__(256, 4) norm_rope_rows_kernel(const __grid_constant__ P p) {
  extern __shared__ float2 s_trig[];  // [per_cta][rot / 2]
  __shared__ long long s_from[ROPE_TOKENS], s_to[ROPE_TOKENS];
  const int w = p.heads[0] == 0 || blockIdx.y == 1;  // queries or keys
  const int half = p.rot / 2;
  const int tokens = p.B * p.N, first = blockIdx.x * p.per_cta, here = min(p.per_cta, tokens - first);
  if (threadIdx.x < here) {
    const int tk = threadIdx.x, b = (first + tk) / p.N, n = (first + tk) - b * p.N;
    s_from[tk] = b * p.ssb[w] + n * p.ssn[w];
    s_to[tk] = b * p.dsb[w] + n * p.dsn[w];
  }
  // the thread's frequency (one for all its angles if half divides 256), while
  // the launch before still runs: constant memory serves lanes that differ one
  // after the other (384 tokens of 40 heads: 6.0 us, read after the wait 6.4;
  // 16380 tokens 66.5 and 68.3)
  const bool same = half == 0 || 256 % half == 0;
  unsigned long long freq = half ? p.freq[threadIdx.x % half] : 0;
  int axis = half ? axis_of(p, threadIdx.x % half) : 0;
  asm volatile("" : "+l"(freq), "+r"(axis));  // read here
  pdl_wait();
  pdl_launch_dependents();
  const int u = threadIdx.x & (p.lanes - 1), npair = PAIRS ? 0 : half / 8;
  const bool live = u < npair + (p.D - 16 * npair) / 8, two = u < npair;
  const int at = two || PAIRS ? u * 8 : (npair + u) * 8;  // the unit's first element
  const bool turned = PAIRS ? at < p.rot : two;
  float g[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) g[0][j] = g[1][j] = 1.f;
  if (p.weight[w] && live) {
    unpack8<DT>(load8<DT, true>(p.weight[w], at), g[0]);
    if (two) unpack8<DT>(load8<DT, true>(p.weight[w], at + half), g[1]);
  }
  // with several axes every angle has a position to load: four at a time; otherwise
  // one (two halves 71.9 us, 384 tokens 5.6; by the compiler's choice 72.5 and 5.8)
#pragma unroll(std::is_same_v<P, NormRopeAxesParams> ? 4 : 1)
  for (int i = threadIdx.x; i < here * half; i += 256) {
    const int tk = i / half, tok = first + tk, b = tok / p.N;
    if (!same) freq = p.freq[i - tk * half], axis = axis_of(p, i - tk * half);
    const long long pos = position_of(p, tok, b, axis);
    const unsigned long long turn = static_cast<unsigned long long>(pos) * freq;
    // signed fraction of a turn times two, in units of pi
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    s_trig[i] = make_float2(c, s);
  }
  __syncthreads();
  const float over_d = 1.f / static_cast<float>(p.D);
  const int step = 256 / p.lanes, row0 = threadIdx.x / p.lanes;
  const int heads = p.heads[w];
  {
    const void *const src = p.src[w];
    void *const dst = p.dst[w];
    const long long ssh = p.ssh[w], dsh = p.dsh[w];
    const int step_tk = step / heads, step_h = step - step_tk * heads;
    int tk = row0 / heads, h = row0 - tk * heads;
    // every thread runs the same number of turns: the row sums are shuffles
    for (int left = here * heads; left > 0; left -= 2 * step) {
      float x[2][2][8];
      int tks[2], hs[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        tks[e] = tk, hs[e] = h;
        tk += step_tk, h += step_h;
        if (h >= heads) h -= heads, ++tk;
        Raw8<DT> r[2];
#pragma unroll
        for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) r[0].v[i] = r[1].v[i] = make_uint4(0, 0, 0, 0);
        if (live && tks[e] < here) {
          const long long from = s_from[tks[e]] + hs[e] * ssh + at;
          r[0] = load8<DT, true>(src, from);
          if (two) r[1] = load8<DT, true>(src, from + half);
        }
        unpack8<DT>(r[0], x[e][0]);
        if (!PAIRS) unpack8<DT>(r[1], x[e][1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (p.norm) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum = fmaf(x[e][0][j], x[e][0][j], sum);
            if (!PAIRS) sum = fmaf(x[e][1][j], x[e][1][j], sum);
          }
          for (int o = p.lanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float r = rsqrtf(fmaf(sum, over_d, p.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[e][0][j] *= r * g[0][j];
            if (!PAIRS) x[e][1][j] *= r * g[1][j];
          }
        }
        if (!live || tks[e] >= here) continue;
        const float4 *trig = reinterpret_cast<const float4 *>(s_trig + tks[e] * half + (PAIRS ? at / 2 : at));
        if (turned) {
#pragma unroll
          for (int j = 0; j < (PAIRS ? 2 : 4); ++j) {  // two angles at a time
            const float4 cs = trig[j];
            if (PAIRS) {
              float *y = x[e][0] + 4 * j;
              const float a = y[0], b = y[1], c = y[2], d = y[3];
              y[0] = a * cs.x - b * cs.y, y[1] = b * cs.x + a * cs.y;
              y[2] = c * cs.z - d * cs.w, y[3] = d * cs.z + c * cs.w;
            } else {
              float *y = x[e][0] + 2 * j, *z = x[e][1] + 2 * j;
              const float a = y[0], b = z[0], c = y[1], d = z[1];
              y[0] = a * cs.x - b * cs.y, z[0] = b * cs.x + a * cs.y;
              y[1] = c * cs.z - d * cs.w, z[1] = d * cs.z + c * cs.w;
            }
          }
        }
        const long long to = s_to[tks[e]] + hs[e] * dsh + at;
        store8<DT, true>(dst, to, pack8<DT>(x[e][0]));
        if (two) store8<DT, true>(dst, to + half, pack8<DT>(x[e][1]));
      }
    }
  }
}

}  // namespace spec
