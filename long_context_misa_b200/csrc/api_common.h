// What the C entry points share: the status text, injected failures, profiler
// ranges.  Defined in api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "misa.h"

namespace misa {
namespace api {

// One NVTX range per library call that launches work, named after the entry
// point, so that a profiler's timeline shows each call around its kernels.
// Without a profiler attached the calls are no-ops.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

// Record the thread's error text and return `st`.
misa_status fail(misa_status st, const char *fmt, ...);
misa_status cuda_fail(cudaError_t e, const char *where);
bool aligned16(const void *p);
// Consume one injected failure, if any (after validation, before any launch).
bool injected_failure(const char *where, misa_status *st);

}  // namespace api
}  // namespace misa
