// The host side of the balance loss's launches (csrc/balance.cu's object)
// against fakes of the CUDA runtime: which calls it makes, and what it does
// when one of them fails.
#include <cstdio>
#include <string>

#include "../../reducescatter_reduction_gb300/csrc/internal.h"

#define EXPORT __attribute__((visibility("default")))

static std::string g_log;
static int g_fail_launch, g_fail_attribute;   // the n-th from here on fails (0: none)

extern "C" {

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *, void **)
{
    const bool fails = g_fail_launch && --g_fail_launch == 0;
    g_log += std::string(fails ? "failed launch " : "launch ") + std::to_string(cfg->blockDim.x) + "\n";
    return fails ? cudaErrorLaunchOutOfResources : cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int)
{
    const bool fails = g_fail_attribute && --g_fail_attribute == 0;
    g_log += fails ? "failed attribute\n" : "attribute\n";
    return fails ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *at, int value, size_t bytes, cudaStream_t stream)
{
    char line[128];
    snprintf(line, sizeof line, "memset %zu %d %zu %zu\n", size_t(at), value, bytes, size_t(stream));
    g_log += line;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }

// what the object's kernels register with; nothing is launched through these
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
unsigned __cudaPopCallConfiguration(void *, void *, size_t *, void *) { return 0; }
cudaError_t __cudaGetKernel(void *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }

EXPORT const char *fake_log(void) { return g_log.c_str(); }
EXPORT size_t fake_scratch_head(void) { return ccl::kScratchHead + size_t(ccl::kMaxPartials) * 16; }
EXPORT size_t fake_scratch_counters(void) { return size_t(ccl::kScratchCells + ccl::kMaxRanks) * 4; }

EXPORT int fake_balance(int p, size_t rows, unsigned experts, unsigned k, int pass, size_t scratch, size_t stream, int fail_launch,
                        int fail_attribute)
{
    g_log.clear();
    g_fail_launch = fail_launch;
    g_fail_attribute = fail_attribute;
    ccl::Launch L;
    L.p = p;
    L.dtype = ccl::DT_F32;
    for (int r = 0; r < p; ++r) L.src[r] = L.dst[r] = reinterpret_cast<void *>(size_t(1 + r) << 30);
    L.device = 64;      // beyond what is remembered: its attributes are set by every call
    L.num_sms = 152;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    const int32_t *ids[ccl::kMaxRanks];
    for (int r = 0; r < p; ++r) ids[r] = reinterpret_cast<const int32_t *>(size_t(100 + r) << 30);
    ccl::BalanceLaunch N;
    N.pass = pass;
    N.rows = rows;
    N.experts = experts;
    N.k = k;
    N.ids = ids;
    N.coef = 1.0f;
    N.counts = reinterpret_cast<int32_t *>(size_t(1) << 44);
    N.tokens = reinterpret_cast<int32_t *>(size_t(2) << 44);
    N.loss = reinterpret_cast<float *>(size_t(3) << 44);
    N.scratch = reinterpret_cast<void *>(scratch);
    ccl::LaunchInfo info;
    return int(ccl::launch_balance(L, N, &info));
}

}  // extern "C"
