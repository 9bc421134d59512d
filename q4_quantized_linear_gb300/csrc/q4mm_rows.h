// q4mm_rows.h -- host side of the kernels over rows of activations: element
// types, the vector width that a call's addresses allow, and the threads that
// hold a row.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/q4mm.h"
#include "q4mm_internal.h"

namespace q4 {

inline int type_size(int type)
{
    return type == Q4_TYPE_F32 ? 4 : type == Q4_TYPE_F16 || type == Q4_TYPE_BF16 ? 2 : type == Q4_TYPE_I8 ? 1 : 0;
}
inline bool is_float_type(int type) { return type == Q4_TYPE_F32 || type == Q4_TYPE_F16 || type == Q4_TYPE_BF16; }
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Widest access (in bytes, a power of two, at most 16) at which every row of
// every matrix added so far starts.
struct RowAlign {
    uintptr_t bits = 16;
    // of the first matrix; whether a row's start within 16 bytes is the same in all
    uintptr_t start = 0, stride = 0;
    bool none = true, alike = true;
    void add(const void *p, int64_t ld_bytes)
    {
        if (!p) return;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), ld = static_cast<uintptr_t>(ld_bytes);
        bits |= at | ld;
        if (none) start = at, stride = ld;
        alike = alike && ((at ^ start) & 15) == 0 && ((ld ^ stride) & 15) == 0;
        none = false;
    }
    int bytes() const { return static_cast<int>(bits & (~bits + 1)); }
};

// How rows are read and written: vectors of `vec` elements, 16 bytes or a single
// element. any: a row starts anywhere, its vectors are the aligned 16-byte words
// that hold some of it, and the codes and channels' parameters beside it are
// aligned to their elements alone.
struct RowAccess {
    int vec;
    bool any;
};

// The library's own bookkeeping (maps of plans and kernel limits) may run out of
// host memory: no exception leaves a C entry point.
template <typename F> int guarded(F body) noexcept
{
    try {
        return body();
    } catch (...) {
        return Q4_ERR_NO_MEMORY;
    }
}

} // namespace q4
