// threads.hpp -- included before a kernel source, with the HIP launch macro replaced: a launch only
// records how many threads it would start.  Host code alone; nothing reaches a GPU.
#pragma once

#include <hip/hip_runtime.h>

#include <vector>

namespace threads {
std::vector<unsigned long long>& launched();
inline void record(dim3 grid, dim3 block) {
    launched().push_back((unsigned long long)grid.x * grid.y * grid.z * block.x * block.y * block.z);
}
}  // namespace threads

#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, ...) threads::record(grid, block)
