// Causal attention among the tokens of whole prompts, packed one behind the
// other.
#pragma once

#include <cstdint>

#include "device.cuh"
#include "elements.cuh"

namespace spec {

struct PromptParams {
  const void *q, *k, *v;  // [T, Hq, D], [T, Hk, D], strides in elements
  long long q_sn, q_sh, k_sn, k_sh, v_sn, v_sh;
  void *out;              // [T, Hq, D]
  float *lse;             // [T, Hq] or NULL
  const int32_t *starts;  // [B + 1]
  int B, T, Hq, G, D;
  float scale_log2;
  int32_t *status;
};

// One warp per token and query head.
template <int DT>
__global__ void __launch_bounds__(256) prompt_plain_kernel(const __grid_constant__ PromptParams p) {
  __shared__ int s_bad;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i <= p.B; i += 256) {
    const int s = p.starts[i];
    if (s < 0 || s > p.T || (i > 0 && s < p.starts[i - 1])) s_bad = 1;
  }
  __syncthreads();
  const bool bad = s_bad;
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, ST_LENGTH);
  const long long item = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.T) * p.Hq) return;
  const int lane = threadIdx.x & 31, tok = static_cast<int>(item / p.Hq), h = static_cast<int>(item % p.Hq), per = p.D / 32;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
  float out_lse = -INFINITY;
  if (bad) {
    out_lse = o[0] = o[1] = o[2] = o[3] = __uint_as_float(0x7fc00000u);
  } else if (tok >= p.starts[0] && tok < p.starts[p.B]) {
    int lo = 0, hi = p.B;  // the last sequence that starts at or before the token
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.starts[mid] <= tok) lo = mid;
      else hi = mid;
    }
    for (int e = 0; e < per; ++e) q[e] = one_element<DT>(p.q, tok * p.q_sn + h * p.q_sh + lane * per + e);
    for (int j = p.starts[lo]; j <= tok; ++j) {
      float s = 0.f;
      for (int e = 0; e < per; ++e) s = fmaf(q[e], one_element<DT>(p.k, j * p.k_sn + h / p.G * p.k_sh + lane * per + e), s);
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float nm = fmaxf(m, s), a = exp2f(m - nm), w = exp2f(s - nm);
      m = nm, l = l * a + w;
      for (int e = 0; e < per; ++e) o[e] = fmaf(w, one_element<DT>(p.v, j * p.v_sn + h / p.G * p.v_sh + lane * per + e), o[e] * a);
    }
    for (int e = 0; e < per; ++e) o[e] /= l;
    out_lse = (m + log2f(l)) * 0.6931471805599453f;
  }
  for (int e = 0; e < per; ++e) put_element<DT>(p.out, item * p.D + lane * per + e, o[e]);
  if (p.lse && lane == 0) p.lse[item] = out_lse;
}

}  // namespace spec
