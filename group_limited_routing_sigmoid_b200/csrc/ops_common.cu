// Host-side state of the handle-free operators: the thread's last error text
// and the SM count of each device.
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "ops_common.cuh"

namespace beam {
namespace ops {

namespace {
thread_local char g_error[512];
std::atomic<int> g_sms[64];
}  // namespace

int fail(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return code;
}

int check_cuda(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return BEAM_OK;
    (void)cudaGetLastError();   // a launch error stays out of the caller's next check
    return fail(BEAM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int sm_count()
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = g_sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        g_sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace ops
}  // namespace beam

extern "C" const char *beam_ops_error(void) { return beam::ops::g_error; }
