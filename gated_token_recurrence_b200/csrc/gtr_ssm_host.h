// Host interfaces between the selective scan's files.
#pragma once

#include "gtr.h"

namespace gtr {

struct SsmParams;

// Argument checks of the selective scan's calls, on the host before anything is enqueued.
gtr_status_t validate_ssm(const SsmParams& p, int grid_H, int grid_W, int direction, int dtype);

}  // namespace gtr
