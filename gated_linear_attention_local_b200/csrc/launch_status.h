// Status reporting for entry points defined outside api.cu, so that every entry
// point fills sgla_last_cuda_error() and sgla_kernel_launch_count() the same way.
#pragma once

#include <cuda_runtime.h>

#include "simple_gla.h"

namespace sgla {

// Result of one kernel launch: on success it is counted in
// sgla_kernel_launch_count() and SGLA_OK is returned; on failure the CUDA error,
// prefixed by `where`, becomes the calling thread's sgla_last_cuda_error() and
// SGLA_ERR_CUDA is returned.
sgla_status launch_status(cudaError_t e, const char *where);

// One kernel launch of an entry point defined outside api.cu, counted and (while
// sgla_profile_begin recording is on) timed as those inside it are:
//   LaunchRecord rec(stream);  status = rec.done(launch(...), "kernel name");
class LaunchRecord {
  public:
    explicit LaunchRecord(cudaStream_t st);
    sgla_status done(cudaError_t e, const char *name);

  private:
    cudaStream_t st_;
    cudaEvent_t begin_;
};

// A failed CUDA runtime call other than a launch: recorded as above.
sgla_status cuda_failure(cudaError_t e, const char *where);

}  // namespace sgla
