// Host side of the attention over whole prompts.
#include <algorithm>
#include <climits>
#include <cmath>

#include "host.h"
#include "prompt.cuh"
#include "spec_verify.h"

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
  p.q = q->data, p.q_sn = q->stride_n, p.q_sh = q->stride_h;
  p.k = k->data, p.k_sn = k->stride_n, p.k_sh = k->stride_h;
  p.v = v->data, p.v_sn = v->stride_n, p.v_sh = v->stride_h;
  p.out = out;
  p.lse = lse;
  p.starts = starts;
  p.B = B, p.T = T, p.Hq = Hq, p.G = Hq / Hk, p.D = D;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  Workspace *w = nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int st = get_ws(stream, 1, &w);
  if (st) return st;
  p.status = w->status;
  const long long ctas = (static_cast<long long>(T) * Hq + 7) / 8;
  if (ctas > INT_MAX) return fail(SPEC_ERR_ARG, "T * Hq is too large");
  const void *fn = dtype == SPEC_BF16 ? reinterpret_cast<const void *>(&prompt_plain_kernel<DT_BF16>)
                                      : reinterpret_cast<const void *>(&prompt_plain_kernel<DT_F16>);
  return launch_dependent(fn, dim3(static_cast<unsigned>(ctas)), 256, 0, stream, &p, "prompt attention launch");
}
