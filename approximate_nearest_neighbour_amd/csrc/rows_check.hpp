// Argument checks that the row operators' entry points share.
#pragma once

#include "status.hpp"

#include <hip/hip_runtime.h>

#include <string>

namespace ivfpq {

constexpr int kMaxRowDim = 1 << 20;

inline bool type_ok(int type) { return type == IVFPQ_F32 || type == IVFPQ_BF16 || type == IVFPQ_F16; }

inline size_t type_size(int type) { return type == IVFPQ_F32 ? 4 : 2; }

inline bool aligned(const void *p, size_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

inline ivfpq_status launched(hipError_t e, const char *what)
{
    if (e != hipSuccess)
        return fail(IVFPQ_E_DEVICE, std::string(what) + ": " + hipGetErrorString(e));
    return ok();
}

} // namespace ivfpq
