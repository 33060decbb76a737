// What the C-ABI files share: the error message of the calling thread, the
// per-device state and the checks of pointers.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "kernels.h"

namespace w4api {

// Sets this thread's message and returns `code`.
int fail(int code, const char *fmt, ...);
// Clears the message and returns W4A16_OK.
int ok();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device's properties and the address of its status word.
int device_state(w4::DeviceInfo &info, unsigned int *&status);
// Every non-null pointer must be memory of `device` or managed memory.
int check_device_ptrs(const char *who, int device, std::initializer_list<const void *> ptrs);
// The status of a launch, as a status code with its message.
int launched(cudaError_t e, const char *what);

}  // namespace w4api
