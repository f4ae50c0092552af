// mnb_api_common.hpp -- status, error text and argument checks shared by the
// files that implement the C ABI (defined in mnb_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mnb.h"

namespace mnb {
namespace api {

// Records the reason ("mnb: ...") for this thread and returns s.
mnb_status fail(mnb_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the thread's error and records the variant it enqueued; NULL, for a
// query that enqueues nothing, keeps the last one.
mnb_status ok(const char* variant);
mnb_status check_ptr(const void* p, uintptr_t align, const char* name);
// A gfx950 device must be current.
mnb_status check_device();
mnb_status launched(hipError_t e, const char* variant);

}  // namespace api
}  // namespace mnb

#define MNB_TRY(x)                           \
    do {                                     \
        const mnb_status s_ = (x);           \
        if (s_ != MNB_OK) return s_;         \
    } while (0)
