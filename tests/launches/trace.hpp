// trace.hpp -- included before a kernel source, with the HIP launch macro replaced: a launch only
// records which kernel (with its template arguments) it would start.  Host code alone; nothing
// reaches a GPU.
#pragma once

#include <hip/hip_runtime.h>

#include <cxxabi.h>
#include <cstdlib>
#include <set>
#include <string>
#include <typeinfo>
#include <vector>

namespace trace {

std::set<std::string>& all();            // every kernel that a launch in the sources names
std::vector<std::string>& launched();    // those of the launches so far, in order

template <auto KERNEL>
struct Tag {};

// "norm_apply_kernel<8, true, 4, false>" out of the mangled name of its tag
template <auto KERNEL>
std::string name() {
    char* p = abi::__cxa_demangle(typeid(Tag<KERNEL>).name(), nullptr, nullptr, nullptr);
    std::string s(p);
    free(p);
    for (const std::string space : {"(anonymous namespace)::", "svdq::", "__device_stub__", "void "})
        for (size_t at; (at = s.find(space)) != std::string::npos;) s.erase(at, space.size());
    s.erase(0, s.find('&') + 1);
    const size_t args = s.find(">(");                 // the kernel's parameters
    if (args != std::string::npos) s.erase(args + 1);
    return s[0] == '(' ? s.substr(1) : s;
}

template <auto KERNEL>
inline bool known = all().insert(name<KERNEL>()).second;

template <auto KERNEL>
void record() {
    (void)&known<KERNEL>;
    launched().push_back(name<KERNEL>());
}

}  // namespace trace

#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, ...) trace::record<kernel>()
