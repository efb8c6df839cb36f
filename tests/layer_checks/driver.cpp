// The host front ends of the operators around layers (csrc/layers.cpp, and the
// norm with an 8-bit output in csrc/ccl.cpp) against fakes of the CUDA runtime
// and of the kernel launchers, so that their refusals are tested without a
// GPU: a call that passes every check counts a launch.
#include "../../reducescatter_reduction_gb300/csrc/ccl.cpp"
#include "../../reducescatter_reduction_gb300/csrc/layers.cpp"

static int g_launches;
static cudaError_t launched(LaunchInfo *info)
{
    ++g_launches;
    info->kernels = 1;
    return cudaSuccess;
}

namespace ccl {
#define FAKE(name) cudaError_t name(const Launch &, LaunchInfo *info) { return launched(info); }
FAKE(launch_reduce_f32) FAKE(launch_reduce_f16) FAKE(launch_reduce_bf16) FAKE(launch_reduce_i32)
FAKE(launch_tma_f32) FAKE(launch_tma_f16) FAKE(launch_tma_bf16) FAKE(launch_tma_i32)
FAKE(launch_bulkred_f32) FAKE(launch_bulkred_f16) FAKE(launch_bulkred_bf16) FAKE(launch_bulkred_i32)
FAKE(launch_gather)
cudaError_t launch_compare(const Launch &, LaunchInfo *info, bool) { return launched(info); }
cudaError_t launch_allreduce_rmsnorm(const Launch &, const NormLaunch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_allreduce_rmsnorm_e4m3_f32(const Launch &, const NormE4m3Launch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_allreduce_rmsnorm_e4m3_f16(const Launch &, const NormE4m3Launch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_allreduce_rmsnorm_e4m3_bf16(const Launch &, const NormE4m3Launch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_expert_sort(const Launch &, const SortLaunch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_expert_rows(const Launch &, const RowsLaunch &, LaunchInfo *info) { return launched(info); }
cudaError_t launch_grads(const Launch &, const GradLaunch &, LaunchInfo *info) { return launched(info); }
bool launch_table_estimate(int, int, int, int, double, int, double *) { return false; }
bool launch_table_prefers_tma(int, int, int, int, double) { return false; }
}  // namespace ccl

extern "C" {
cudaError_t cudaGetDevice(int *d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int)
{
    *v = 152;
    return cudaSuccess;
}
static char g_block[kCommDeviceBytes];
cudaError_t cudaMalloc(void **p, size_t)
{
    *p = g_block;
    return cudaSuccess;
}
cudaError_t cudaFree(void *) { return cudaSuccess; }
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { return cudaSuccess; }
const char *cudaGetErrorName(cudaError_t) { return "error"; }
const char *cudaGetErrorString(cudaError_t) { return "error"; }
CCL_API int fake_launches(void) { return g_launches; }
}
