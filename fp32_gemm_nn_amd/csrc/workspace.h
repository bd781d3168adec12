// The per-stream workspace of split products (kept in misgemm.hip), for the
// other translation units: 64 MiB of partial sums and 65,536 counters, which
// every user leaves at zero. Internal to libmisgemm.
#ifndef MISGEMM_WORKSPACE_H
#define MISGEMM_WORKSPACE_H

#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace misgemm_workspace {

constexpr size_t kFloats = size_t(16) << 20;
constexpr int kCounters = 1 << 16;

// The workspace of `stream`, allocated on first use. False if there is none
// and none can be had (out of memory, or the stream is being captured into a
// graph): the caller then runs unsplit.
bool get(hipStream_t stream, float **partials, int **counters);

}  // namespace misgemm_workspace

#endif  // MISGEMM_WORKSPACE_H
