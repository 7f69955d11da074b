// Host helpers that the translation units share: error reporting, launches,
// per-stream workspaces.  Defined in spec_verify.cu.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>
#include <string>

namespace spec {

// An NVTX range around each entry point (free when no tool is attached), so
// that profilers can attribute kernels to calls.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Record the calling thread's error message; return the status code.
int fail(int code, const std::string &msg);
int cuda_fail(cudaError_t e, const char *what);

// cudaLaunchKernelExC, or the injected failure of spec_debug_fail_launch.
cudaError_t launch_kernel(const cudaLaunchConfig_t *cfg, const void *fn, void **args);

// Per (device, stream): the status word (never reallocated), the partials of
// the current call (rows of the verification: float4 per job and slice; pieces
// of the attention; grow-only), counters, and a staging area for the
// host-buffer entry point.
struct Workspace {
  int device = -1;
  cudaStream_t stream = nullptr;
  int32_t *status = nullptr;  // status word, then the item tickets (zeroed once)
  float4 *partials = nullptr;
  size_t cap_parts = 0;
  unsigned char *stage = nullptr;
  size_t stage_cap = 0;
  int *ngram_done = nullptr;  // n-gram drafter: finished-CTA counters, zero between calls
  size_t ngram_cap = 0;
  int *attn_done = nullptr;   // cache attention: arrived-CTA counters, zero between calls
  size_t attn_cap = 0;
  // What partials and counters have outgrown, until spec_shutdown: a CUDA graph
  // captured before still points there.  A buffer grows to twice its size at
  // least, so all that it has outgrown is smaller than it, and in 2^40 bytes.
  void *outgrown[128] = {};
  int n_outgrown = 0;
};

// The stream's workspace with room for nparts partials and, where asked for,
// nattn counters of the cache attention.
int get_ws(cudaStream_t stream, size_t nparts, Workspace **out, size_t nattn = 0);

int num_sms();

// Launches one kernel, whose parameters are *params, as a programmatic
// dependent of what precedes it on the stream, in clusters of `cluster` CTAs
// along x (cache_ops.cu).
int launch_dependent(const void *fn, dim3 grid, int threads, int smem, cudaStream_t stream, void *params, const char *what, unsigned cluster = 1);

}  // namespace spec
