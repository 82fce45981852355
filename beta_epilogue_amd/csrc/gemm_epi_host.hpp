// gemm_epi_host.hpp -- what the host-side translation units of the library
// share: the thread's error text, type sizes, and the checks every run makes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_epi.h"

namespace gemm_epi {

// Sets the calling thread's gemm_epi_last_error() text and returns code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();

int elem_bytes(int type);
bool is_float_out(int type);

// a * b in *out; false if it does not fit or either is negative.
bool mul_ok(int64_t a, int64_t b, int64_t* out);

// The current device and its compute units; GEMM_EPI_ERR_DEVICE unless gfx950.
int device_query(int* device, int* cus);

// Whether t is one of the public element type codes (NONE excluded).
inline bool is_type(int t) { return t > GEMM_EPI_NONE && t <= GEMM_EPI_U8; }

// GEMM_EPI_ERR_DEVICE unless the current device is `device`.
int check_device(int device);

// The caller's workspace: at least `need` bytes at a 256-byte boundary (none: NULL).
int check_workspace(const void* ws, int64_t have, int64_t need);

// The status of the launch just made (hipGetLastError).
int launched();

inline int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace gemm_epi
