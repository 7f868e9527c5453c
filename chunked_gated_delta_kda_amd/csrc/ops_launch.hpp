// ops_launch.hpp -- host-side launchers of the operators beside the delta rule (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace ops {

inline size_t dtype_bytes(int dt) { return dt == KDA_DTYPE_F32 ? 4 : 2; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// short convolution (ops_conv.hip)
hipError_t launch_conv_fwd(const kda_conv_args &a, int32_t *err, hipStream_t st);
hipError_t launch_conv_decode(const kda_conv_args &a, hipStream_t st);
size_t conv_bwd_workspace(int64_t T, int64_t C, int W);
hipError_t launch_conv_bwd(const kda_conv_args &a, const kda_conv_grads &g, float *ws, int32_t *err, hipStream_t st);

// selective state space scan (ops_ssm.hip)
size_t ssm_workspace(int64_t T, int64_t D, int64_t N, int64_t G, int64_t S);
hipError_t launch_ssm_fwd(const kda_ssm_args &a, float *ws, int32_t *err, hipStream_t st);
hipError_t launch_ssm_decode(const kda_ssm_args &a, hipStream_t st);
// its gradients (ops_ssm_bwd.hip)
size_t ssm_bwd_workspace(int64_t T, int64_t D, int64_t N, int64_t G);
hipError_t launch_ssm_bwd(const kda_ssm_args &a, const kda_ssm_grads &g, float *ws, int32_t *err, hipStream_t st);

// paged token attention (ops_attn.hip)
size_t attn_workspace(int64_t B, int64_t hq, int64_t hkv, int64_t dh, int64_t width, int64_t page);
hipError_t launch_attn_decode(const kda_attn_args &a, float *ws, int32_t *err, hipStream_t st);

}  // namespace ops
}  // namespace kda
