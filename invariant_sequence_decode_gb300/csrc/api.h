// api.h - what the files of the C ABI share: statuses, messages, checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace luce {

// Sets the calling thread's message and returns code.
int fail(int code, const char* fmt, ...);

// Clears the message and returns LUCE_OK.
int ok();

// LUCE_OK, or LUCE_ECUDA with the error's message.
int cuda_status(cudaError_t e, const char* what);

static inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace luce

#define REQUIRE(cond, code, ...) \
    do {                         \
        if (!(cond)) return luce::fail(code, __VA_ARGS__); \
    } while (0)
