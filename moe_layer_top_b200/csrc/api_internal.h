// What the translation units of the C ABI share (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Records the message that moe_last_error_string() returns on this thread; returns `code`.
int api_fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// MOE_OK on an sm_100 device (then *sms, unless NULL, is its SM count), else an error code.
int api_device_check(int* sms);

// The current device's status word for operators whose caller brings none.
cudaError_t operator_status_word(int** word);

}  // namespace moe
