// Host helpers of gdn_api.cpp that the other sources of the C ABI share.
#pragma once

#include <hip/hip_runtime_api.h>

#include "gdn.h"

namespace gdn {

// Sets the calling thread's gdn_last_error() message and returns `status`.
int api_fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

void api_clear_error();

// GDN_DEBUG_CHECK=1: checks a device cu_seqlens table of n_seq + 1 entries
// and waits for the result (skipped while the stream is being captured).
int api_debug_check_cu(const gdn_tensor* cu, int64_t n_seq, int64_t t_total, hipStream_t s);

}  // namespace gdn
