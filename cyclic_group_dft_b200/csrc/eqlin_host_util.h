// eqlin_host_util.h -- host helpers of the handle-free operators (norm, rotary positions,
// attention): argument checks shared by their entry points, the current device, and launches
// with programmatic stream serialization.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include <cuda_runtime.h>

#include "eqlin.h"
#include "eqlin_report.h"

namespace eqlin {
namespace host {

inline bool known_dtype(int t) { return t == EQLIN_F32 || t == EQLIN_BF16 || t == EQLIN_F16; }
inline int elem_bytes(int t) { return t == EQLIN_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
// log2 of a supported group size (1 is a layer without a group axis), or -1
inline int log2_group(int64_t G) {
    for (int k = 0; k <= 4; ++k)
        if (G == (int64_t(1) << k)) return k;
    return -1;
}

// The current device: its number and SM count.  Only the answer to "is it an sm_100 device,
// with how many SMs" is kept between calls, by device number.
inline int current_device(int* device, int* sms) {
    static std::atomic<int> known[64];   // SM count, 0 unknown, -1 not an sm_100 device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda(e, "cudaGetDevice");
    int v = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (v == 0) {
        int major = 0, minor = 0;
        if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return report_cuda(e, "device query");
        if (major != 10 || minor != 0) v = -1;
        if (dev < 64) known[dev].store(v, std::memory_order_relaxed);
    }
    if (v < 0) return report(EQLIN_ERR_UNSUPPORTED, "needs a compute capability 10.0 (sm_100a) device");
    if (device) *device = dev;
    *sms = v;
    return EQLIN_OK;
}

inline bool use_pdl() {
    static const bool on = [] {
        const char* e = std::getenv("EQLIN_PDL");
        return !(e && e[0] == '0');
    }();
    return on;
}

// Launch with programmatic stream serialization: the kernel's prologue may run while the
// previous kernel of the stream drains; it waits in griddepcontrol.wait before it touches
// global memory.
template <class... KArgs, class... Args>
int launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const char* what,
           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = use_pdl() ? 1 : 0;
    cudaError_t e;
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(smem))) != cudaSuccess)
        return report_cuda(e, what);
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? EQLIN_OK : report_cuda(e, what);
}

}  // namespace host
}  // namespace eqlin
