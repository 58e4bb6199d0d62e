// Host interfaces between the selective scan's files.
#pragma once

#include <cuda_runtime.h>

#include "gtr.h"

namespace gtr {

struct SsmParams;

// The checks of the sizes alone: GTR_ERR_INVALID_ARG before GTR_ERR_UNSUPPORTED.
gtr_status_t validate_ssm_shape(int B, int grid_H, int grid_W, int D, int N, int G, int dtype);
// Argument checks of the selective scan's calls, on the host before anything is enqueued.
gtr_status_t validate_ssm(const SsmParams& p, int grid_H, int grid_W, int direction, int dtype);
// A scan of a few tokens for many channels (gtr_ssm_step.cu).
gtr_status_t launch_ssm_walk(const SsmParams& p, int dtype, cudaStream_t stream);

}  // namespace gtr
