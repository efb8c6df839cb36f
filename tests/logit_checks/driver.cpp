// The host front end of the logit operators (csrc/logits.cpp) against fakes
// of the CUDA runtime and of the kernel launchers, so that its refusals are
// tested without a GPU: a call that passes every check counts a launch.
#include <cstdarg>
#include <cstdio>

#include "../../reducescatter_reduction_gb300/csrc/logits.cpp"

static char g_message[512];
static int g_launches;
static bool g_alias;

namespace ccl {
ccl_status_t fail(ccl_status_t st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_message, sizeof g_message, fmt, ap);
    va_end(ap);
    return st;
}
ccl_status_t cuda_fail(cudaError_t, const char *what) { return fail(CCL_ERR_CUDA, "%s", what); }
bool debug_on() { return false; }
static cudaError_t launched(const Launch &L, LaunchInfo *info)
{
    ++g_launches;
    g_alias = L.alias;
    info->kernels = 1;
    return cudaSuccess;
}
cudaError_t launch_logit_rules(const Launch &L, const RulesLaunch &, LaunchInfo *info) { return launched(L, info); }
cudaError_t launch_distill(const Launch &L, const DistillLaunch &, LaunchInfo *info) { return launched(L, info); }
cudaError_t launch_balance(const Launch &L, const BalanceLaunch &, LaunchInfo *info) { return launched(L, info); }
}  // namespace ccl

extern "C" cudaError_t cudaGetDevice(int *d)
{
    *d = 0;
    return cudaSuccess;
}
extern "C" cudaError_t cudaSetDevice(int) { return cudaSuccess; }

extern "C" __attribute__((visibility("default"))) ccl_comm *fake_comm(int p, void *const *in, void *const *out)
{
    ccl_comm *c = new ccl_comm;
    c->p = p;
    for (int r = 0; r < p; ++r) {
        c->in[r] = in[r];
        c->out[r] = out[r];
    }
    return c;
}
extern "C" __attribute__((visibility("default"))) void fake_comm_free(ccl_comm *c) { delete c; }
extern "C" __attribute__((visibility("default"))) const char *fake_message(void) { return g_message; }
extern "C" __attribute__((visibility("default"))) int fake_launches(void) { return g_launches; }
extern "C" __attribute__((visibility("default"))) int fake_alias(void) { return g_alias; }
