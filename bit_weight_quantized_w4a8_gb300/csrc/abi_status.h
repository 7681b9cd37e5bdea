// abi_status.h -- status codes and messages of the C entry points, shared by
// the files that define them (abi.cu holds the message).
#pragma once

#include <cuda_runtime.h>

namespace w4a8 {

// Records `message` for w4a8_last_error and returns `code`.
int status_fail(int code, const char* message);
// W4A8_OK with the message cleared, or W4A8_ERR_CUDA with the reason.
int status_done(cudaError_t e, const char* what);
// SMs of the current device, or a status code with its message.
int status_sm_count(int* out);

}  // namespace w4a8
