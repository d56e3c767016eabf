// What the host sides of include/moe.h and include/moe_block.h share: errors,
// checks of pointers, and sizes of the machine.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "ep_static.h"
#include "moe.h"

namespace moe {
namespace host {

constexpr size_t kPtrAlign = 16;
// Bytes a call may move before its rows stream past the caches: the 256 MB
// last-level cache of an MI355X.
constexpr int64_t kKeepBytes = 256ll << 20;

// Blocks of a grouped product: one a compute unit of an MI355X.
constexpr int kGemmBlocks = 256;

inline int fail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return ep::set_error(code, buf);
}

inline int ok() { return ep::set_error(EP_OK, ""); }

struct Pointer {
    const void* ptr;
    const char* name;
    size_t align;
    bool required;
};

inline int check_pointers(const Pointer* p, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!p[i].ptr) {
            if (p[i].required)
                return fail(EP_ERR_NULL, "%s is NULL", p[i].name);
            continue;
        }
        if (reinterpret_cast<uintptr_t>(p[i].ptr) % p[i].align)
            return fail(EP_ERR_ALIGN, "%s = %p is not %zu-byte aligned", p[i].name, p[i].ptr,
                        p[i].align);
    }
    return EP_OK;
}

template <int N>
int check_pointers(const Pointer (&p)[N])
{
    return check_pointers(p, N);
}

}  // namespace host
}  // namespace moe
