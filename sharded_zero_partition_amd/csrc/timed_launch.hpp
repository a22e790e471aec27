// timed_launch.hpp -- kernel launches of the tensor sets (device translation
// units only).
#pragma once

#include <hip/hip_ext.h>

#include "zp_internal.hpp"

namespace zp {

// A launch whose kernel's start and end are recorded where events are given (an
// ordinary one, which a stream being captured takes, where not).
template <typename K, typename... Args>
void launch(K kernel, dim3 grid, int threads, hipStream_t s, const KernelEvents& ev, Args... args) {
    if (ev.start || ev.stop) hipExtLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, ev.start, ev.stop, 0, args...);
    else hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, args...);
}

}  // namespace zp
