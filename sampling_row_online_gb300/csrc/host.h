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

// Per (device, stream): the status word (never reallocated), the row
// partials of the current call (float4 per job and slice, grow-only), and a
// staging area for the host-buffer entry point.
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
};

// The stream's workspace with room for nparts partials and, where asked for,
// nattn counters of the cache attention.
int get_ws(cudaStream_t stream, size_t nparts, Workspace **out, size_t nattn = 0);

int num_sms();

}  // namespace spec
