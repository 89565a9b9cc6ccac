// etp_grad_norm.hpp -- launchers of the norm of many tensors.
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/etp_dense.h"

namespace etp {

struct GradList {
    int n;
    const etp_tensor *tensors;
    void *const *out;  // or null: in place
};
size_t grad_norm_workspace_bytes(const GradList &g);
hipError_t launch_grad_norm(const GradList &g, float *norm, void *ws, hipStream_t stream);
hipError_t launch_clip_grads(const GradList &g, float max_norm, float *norm, void *ws, hipStream_t stream);

}  // namespace etp
