// Where a workspace's parts start.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// A caller's workspace starts at any multiple of 16 bytes.  Where a part needs
// more (a tensor map in global memory: 128 bytes), the parts start at the next
// multiple of kWsAlign, and kWsSlack bytes of the workspace's size are for that.
constexpr size_t kWsAlign = 256;
constexpr size_t kWsSlack = kWsAlign - 16;
inline uint8_t *ws_start(void *ws) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + kWsAlign - 1) & ~(static_cast<uintptr_t>(kWsAlign) - 1));
}

}  // namespace moe
