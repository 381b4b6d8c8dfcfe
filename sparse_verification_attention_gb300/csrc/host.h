// Host-side helpers shared by the translation units that hold C entries:
// error reporting, argument checks, and the driver's tensor-map encoder.
#pragma once

#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include "internal.h"

namespace sva {

// Record the calling thread's last error and return its status.
__attribute__((format(printf, 2, 3))) sv_status fail(sv_status st, const char* fmt, ...);
sv_status cuda_fail(cudaError_t e, const char* what);
bool aligned(const void* p, size_t a);

sv_status check_shape(const sv_shape* s);
// most: sequences that may have contexts of their own.
sv_status check_kv(const sv_shape* s, const sv_kv* kv, bool need_v, int most = kMaxVarB);
sv_status check_parents(const int32_t* parent, int T);
// anc[t]: bit u set when draft t sees draft u.
void fill_ancestors(const int32_t* parent, int T, unsigned long long* anc);
// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 get_encode();

// An NVTX range named after the C-ABI call, around its whole host side
// (validation, planning, launches), for timeline tools; a no-op without one.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

}  // namespace sva
