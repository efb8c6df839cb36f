// AllReduce + residual + RMSNorm with e4m3 outputs, f32 inputs (norm_e4m3.cuh).
#include "norm_e4m3.cuh"

namespace ccl {

cudaError_t launch_allreduce_rmsnorm_e4m3_f32(const Launch &L, const NormE4m3Launch &N, LaunchInfo *info) { return quant_dtype<F32>(L, N, info); }

}  // namespace ccl
