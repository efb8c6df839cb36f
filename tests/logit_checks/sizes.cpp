// The host front end of the logit operators together with the host side of
// their launches (the objects of csrc/*.cu), against fakes of the CUDA
// runtime, so that what a size makes of a call is seen without a GPU.
#include <cstdarg>
#include <cstdio>

#include "../../reducescatter_reduction_gb300/csrc/logits.cpp"

#define EXPORT __attribute__((visibility("default")))

static char g_message[512];
static int g_launches;

namespace ccl {
ccl_status_t fail(ccl_status_t st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_message, sizeof g_message, fmt, ap);
    va_end(ap);
    return st;
}
ccl_status_t cuda_fail(cudaError_t err, const char *what) { return fail(CCL_ERR_CUDA, "%s: %d", what, int(err)); }
bool debug_on() { return false; }
}  // namespace ccl

extern "C" {

cudaError_t cudaGetDevice(int *d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **)
{
    ++g_launches;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *)
{
    *n = 16;
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }

// what the objects' kernels register with; nothing is launched through these
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
unsigned __cudaPopCallConfiguration(void *, void *, size_t *, void *) { return 0; }
cudaError_t __cudaGetKernel(void *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }

EXPORT ccl_comm *fake_comm(int p)
{
    ccl_comm *c = new ccl_comm;
    c->p = p;
    c->num_sms = 152;
    for (int r = 0; r < p; ++r) c->in[r] = c->out[r] = reinterpret_cast<void *>(size_t(1 + r) << 52);
    return c;
}
EXPORT void fake_comm_free(ccl_comm *c) { delete c; }
EXPORT const char *fake_message(void) { return g_message; }
EXPORT int fake_launches(void) { return g_launches; }

}  // extern "C"
