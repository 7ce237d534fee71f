// mx_api.h - what the translation units that implement the C ABI share:
// status text, argument helpers and the device check (defined in api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mxfp8.h"

namespace mx {

// Record the text mxfp8_last_error() returns on this thread; returns st.
mxfp8_status fail(mxfp8_status st, const char* fmt, ...);
mxfp8_status cuda_fail(cudaError_t e, const char* what);

// Current device, checked to be sm_103.  Returns MXFP8_OK and fills *sms.
mxfp8_status current_device(int* sms);

// The quantise and repack kernels index 32-element blocks and 4-byte packed
// scale words with 32-bit integers: B*R*(K/32) blocks and the packed scale
// words of (B, R, K) must each fit in 31 bits.
mxfp8_status check_block_count(int64_t B, int64_t R, int64_t K, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

}  // namespace mx
