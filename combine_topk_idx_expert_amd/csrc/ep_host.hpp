// ep_host.hpp -- what the host sides of the library share: the message of the
// last error, status helpers and checks of pointers and element types.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "ep_mi355x.h"
#include "ep_route.hpp"  // F32 / Bf16 / F16 element access

namespace ep {

extern thread_local std::string g_last_error __attribute__((visibility("hidden")));

// Keeps the message for ep_last_error and returns st.
__attribute__((visibility("hidden"), format(printf, 2, 3))) ep_status fail(ep_status st, const char* fmt, ...);

#define EP_HIP(call)                                                                      \
  do {                                                                                    \
    hipError_t e_ = (call);                                                               \
    if (e_ != hipSuccess) return fail(EP_ERR_HIP, "%s: %s", #call, hipGetErrorString(e_)); \
  } while (0)

#define EP_LAUNCHED(name)                                                                     \
  do {                                                                                        \
    hipError_t e_ = hipGetLastError();                                                        \
    if (e_ != hipSuccess) return fail(EP_ERR_HIP, "launch of %s: %s", name, hipGetErrorString(e_)); \
  } while (0)

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

constexpr int kCUs = 256;  // MI355X

inline bool known_type(int32_t type) { return type == EP_TYPE_F32 || type == EP_TYPE_BF16 || type == EP_TYPE_F16; }

inline uintptr_t type_bytes(int32_t type) { return type == EP_TYPE_F32 ? 4 : 2; }

// Calls f with the element-access type of an EP_TYPE_* value.
template <typename F>
ep_status with_type(int32_t type, F f) {
  switch (type) {
    case EP_TYPE_F32: return f(F32{});
    case EP_TYPE_BF16: return f(Bf16{});
    case EP_TYPE_F16: return f(F16{});
    default: return fail(EP_ERR_SHAPE, "unknown element type %d", type);
  }
}

}  // namespace ep
