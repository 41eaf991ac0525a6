// What the entry points of the C ABI share across source files: the error
// message and the device check. Neither lets a C++ exception out.
#pragma once

#include <hip/hip_runtime.h>

// Sets this thread's ttt_last_error() message and returns `code`.
int ttt_fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// TTT_OK when the current device is a gfx950 (asked once per device), else an error code.
int ttt_check_device();

// A launcher's status as a return code of the ABI.
int ttt_launched(hipError_t e, const char *what);
