// nvtx_range.h -- MHA_NVTX_RANGE(name) for the entry points and their steps.
#pragma once

#include <nvtx3/nvToolsExt.h>

// An NVTX range over the rest of the scope: every public entry point that launches work and
// every step inside it (projection, attention, ...) shows up by name in a profiler's timeline;
// without a profiler attached the calls return at once.
namespace {
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};
}  // namespace
#define MHA_NVTX_CAT2(a, b) a##b
#define MHA_NVTX_CAT(a, b) MHA_NVTX_CAT2(a, b)
#define MHA_NVTX_RANGE(name) NvtxRange MHA_NVTX_CAT(nvtx_range_, __LINE__)(name)
