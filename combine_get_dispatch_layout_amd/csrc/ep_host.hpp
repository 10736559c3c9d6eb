// What the host runtime's files share (api.cpp, moe_api.cpp): the error text
// of the calling thread and a handle's insides.
#pragma once

#include <stdint.h>

#include "ep.h"

namespace epk {

// Stores "file:line reason" as the calling thread's error text; returns st.
ep_status host_fail(ep_status st, const char* file, int line, const char* fmt, ...)
    __attribute__((format(printf, 4, 5), visibility("hidden")));

struct HandleInfo {
    const ep_config* cfg;
    int64_t num_tokens;         // -1 before the first layout
    bool pending;               // waits for ep_combine_overlap
    const int32_t* psum_expert;
    const int32_t* num_unaligned;
    uint32_t* flags;
};

HandleInfo handle_info(const ep_handle* h) __attribute__((visibility("hidden")));

}  // namespace epk
