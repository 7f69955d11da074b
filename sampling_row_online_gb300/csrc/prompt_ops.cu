// Host side of the attention over whole prompts.
#include <algorithm>
#include <climits>
#include <cmath>
#include <numeric>

#include "host.h"
#include "prompt.cuh"
#include "spec_verify.h"

namespace spec {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(f) : nullptr;
  }();
  return fn;
}

// A tensor [T, H, D] of 16-bit elements as the copies see it.
struct Rows {
  const void *data;
  int64_t sn, sh;  // strides in elements
  int H;
};
// The copies need 16-byte aligned rows with positive strides, in any order.
bool fits(const Rows &x, int T) {
  const auto stride = [](int64_t s) { return s > 0 && s % 8 == 0 && s < (1ll << 38); };
  return (reinterpret_cast<uintptr_t>(x.data) & 15u) == 0 && (T == 1 || stride(x.sn)) && (x.H == 1 || (stride(x.sh) && stride(x.sh * x.H)));
}
int encode(CUtensorMap *map, const Rows &x, int T, int D, int dtype, int group, int rows) {  // group: 0, or heads of a box
  const cuuint64_t sh = x.H == 1 ? D * 2 : x.sh * 2, sn = T == 1 ? D * 2 : x.sn * 2;
  const cuuint64_t dims3[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(x.H), static_cast<cuuint64_t>(T)}, strides3[2] = {sh, sn};
  const cuuint32_t box3[3] = {64, 1, static_cast<cuuint32_t>(rows)}, ones[4] = {1, 1, 1, 1};
  const cuuint64_t dims4[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(std::max(group, 1)), static_cast<cuuint64_t>(x.H / std::max(group, 1)),
                               static_cast<cuuint64_t>(T)};
  const cuuint64_t strides4[3] = {sh, sh * std::max(group, 1), sn};
  const cuuint32_t box4[4] = {64, static_cast<cuuint32_t>(std::max(group, 1)), 1, static_cast<cuuint32_t>(rows)};
  const CUresult e = encode_tiled()(map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, group ? 4 : 3,
                                    const_cast<void *>(x.data), group ? dims4 : dims3, group ? strides4 : strides3, group ? box4 : box3, ones,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? static_cast<int>(SPEC_OK) : fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

struct PromptChoice {
  const void *fn;
  int smem;
  size_t piece;  // floats of a group's piece
};
template <int D>
PromptChoice choose_prompt(int dtype) {
  using L = PromptLayout<D>;
  return {dtype == SPEC_BF16 ? reinterpret_cast<const void *>(&prompt_kernel<D, DT_BF16>) : reinterpret_cast<const void *>(&prompt_kernel<D, DT_F16>),
          L::SMEM, L::PIECE};
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int spec_prompt_attention(const spec_heads_t *q, const spec_heads_t *k, const spec_heads_t *v, const int32_t *starts, int B,
                                     int T, int Hq, int Hk, int D, int dtype, float scale, void *out, float *lse, void *stream_ptr) {
  NvtxRange nvtx_range("spec_prompt_attention");
  if (dtype != SPEC_BF16 && dtype != SPEC_F16) return fail(SPEC_ERR_DTYPE, "dtype must be SPEC_BF16 or SPEC_F16");
  if (D != 64 && D != 128) return fail(SPEC_ERR_ARG, "head_dim must be 64 or 128");
  if (B < 0 || B > 65535) return fail(SPEC_ERR_ARG, "B out of range [0, 65535]");
  if (T < 0 || T > (1 << 30)) return fail(SPEC_ERR_ARG, "T out of range [0, 2^30]");
  if (Hk < 1 || Hk > 32767) return fail(SPEC_ERR_ARG, "kv_heads out of range [1, 32767]");
  if (Hq < 1 || Hq > 65535 || Hq % Hk) return fail(SPEC_ERR_ARG, "Hq must be a multiple of kv_heads, at most 65535");
  if (!std::isfinite(scale)) return fail(SPEC_ERR_ARG, "scale must be finite");
  if (T == 0) return SPEC_OK;
  if (!q || !k || !v || !q->data || !k->data || !v->data || !starts || !out) return fail(SPEC_ERR_ARG, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(out) & 15u) return fail(SPEC_ERR_ALIGN, "out must be 16-byte aligned");
  PromptParams p = {};
  p.out = out;
  p.lse = lse;
  p.starts = starts;
  p.B = B, p.T = T, p.Hq = Hq;
  // the most query heads of a kv head, not above 128, that divide them
  const int group = Hq / Hk;
  p.G = std::min(group, PT);
  while (group % p.G) --p.G;
  p.heads = Hq / p.G, p.per_kv = group / p.G, p.tile = PT / p.G;
  const int pair = 2 * p.tile, same = std::gcd(pair, PT);
  p.period = PT / same, p.gain = pair / same;
  for (int i = 1; i <= p.period; ++i) p.ends[i] = p.ends[i - 1] + (i * pair + PT - 1) / PT;
  // the kernel counts its work items in 31 bits
  const double pairs = std::ceil(static_cast<double>(T) / pair), tiles = std::ceil(static_cast<double>(T) / PT);
  if ((pairs * (tiles + 2) / 2 + pairs + B) * p.heads >= 2147483648.0) return fail(SPEC_ERR_ARG, "T * T * Hq is too large");
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!encode_tiled()) return fail(SPEC_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available");

  const PromptChoice c = D == 128 ? choose_prompt<128>(dtype) : choose_prompt<64>(dtype);
  const cudaError_t e = cudaFuncSetAttribute(c.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, c.smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic smem)");
  Rows rows[3] = {{q->data, q->stride_n, q->stride_h, Hq}, {k->data, k->stride_n, k->stride_h, Hk}, {v->data, v->stride_n, v->stride_h, Hk}};
  const int grid = num_sms();
  const size_t pieces = c.piece * 4 * grid;  // floats: two segments of a CTA, two groups
  size_t parts = (pieces + 3) / 4;
  for (const Rows &x : rows)
    if (!fits(x, T)) parts += static_cast<size_t>(T) * x.H * D / 8;
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int st = get_ws(stream, parts, &w, 2 * static_cast<size_t>(grid));
  if (st) return st;
  p.pieces = reinterpret_cast<float *>(w->partials);
  p.done = w->attn_done;
  p.status = w->status;
  float4 *at = w->partials + (pieces + 3) / 4;
  for (Rows &x : rows) {
    if (fits(x, T)) continue;
    PackParams pack = {static_cast<const uint16_t *>(x.data), x.sn, x.sh, reinterpret_cast<uint16_t *>(at), T, x.H, D};
    if ((st = launch_dependent(reinterpret_cast<const void *>(&prompt_pack_kernel), dim3(static_cast<unsigned>(8 * grid)), 256, 0, stream, &pack,
                               "prompt_pack_kernel launch")))
      return st;
    x.data = at, x.sn = static_cast<int64_t>(x.H) * D, x.sh = D;
    at += static_cast<size_t>(T) * x.H * D / 8;
  }
  if ((st = encode(&p.q, rows[0], T, D, dtype, p.G, p.tile))) return st;
  if ((st = encode(&p.k, rows[1], T, D, dtype, 0, PT))) return st;
  if ((st = encode(&p.v, rows[2], T, D, dtype, 0, PT))) return st;
  return launch_dependent(c.fn, dim3(static_cast<unsigned>(grid)), P_NT, c.smem, stream, &p, "prompt_kernel launch");
}
