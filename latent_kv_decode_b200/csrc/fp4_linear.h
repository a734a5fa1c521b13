// Host-side launchers of the FP4-weight products (internal; the public call is
// mla_fp4_linear in include/mla.h). Arguments are validated by the caller.
#pragma once

#include <cuda_runtime.h>

#include "../../include/mla.h"

namespace mla {

size_t fp4_linear_workspace_bytes(const mla_fp4_linear_args* a);
bool fp4_few_tokens(const mla_fp4_linear_args* a);          // the calls launch_fp4_few takes
cudaError_t launch_fp4_few(const mla_fp4_linear_args* a, int sms, cudaStream_t st);
cudaError_t launch_fp4_linear(const mla_fp4_linear_args* a, void* ws, int sms, cudaStream_t st);

}  // namespace mla
