// Host helpers shared by the translation units that hold C entry points: the thread-local error line, the SM
// count, the per-launch profiler scope and the tensor-map encoder.  Defined in api.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

// records a one-line reason for gdn_last_error_string() and returns `code`
int fail(int code, const char *fmt, ...);
int num_sms();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// while profiling is on, brackets the launches in its scope with two events (gdn_profile_enable)
struct ProfScope {
  int idx = -1;
  cudaStream_t st;
  const char *name;
  ProfScope(const char *n, cudaStream_t s);
  ~ProfScope();
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

}  // namespace gdn

#define PROF(name) gdn::ProfScope _prof_scope(name, st)

#define CK(expr)                                                                                  \
  do {                                                                                            \
    int _e = (expr);                                                                              \
    if (_e != 0) return gdn::fail(GDN_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString((cudaError_t)_e)); \
  } while (0)
