// Host-side launcher of the rotating cache append (internal; the public call is
// mla_rope_append in include/mla.h). Arguments are validated by the caller.
#pragma once

#include <cuda_runtime.h>

#include "../../include/mla.h"

namespace mla {

cudaError_t launch_rope_append(const mla_rope_append_args* a, cudaStream_t st);

}  // namespace mla
