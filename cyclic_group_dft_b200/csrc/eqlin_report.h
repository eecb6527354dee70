// eqlin_report.h -- the calling thread's error message (eqlin_last_error), shared by the
// translation units of the library.  Defined in eqlin_api.cu.
#pragma once

#include <cuda_runtime.h>

namespace eqlin {

// Records `msg` as the thread's latest error and returns `code`.  Never throws.
int report(int code, const char* msg) noexcept;
// The same for a CUDA runtime error: "<what>: <error string>", EQLIN_ERR_CUDA.
int report_cuda(cudaError_t e, const char* what) noexcept;

}  // namespace eqlin
