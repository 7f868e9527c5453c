// ops_lin_bwd_f16.hip -- ops_lin_bwd.hip's kernels for fp16, compiled beside those for bf16.
#define KDA_LIN_BWD_F16
#include "ops_lin_bwd.hip"
