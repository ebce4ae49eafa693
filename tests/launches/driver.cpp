// driver.cpp -- prints every kernel that the adapters' and the group norm's launchers can start,
// then, for each call read from stdin, the kernels that it starts, in order.
//   lora  M K N R segments adapters bf16
//   norm  B rows C groups x_bf16 out_bf16 vec in_place
#include "trace.hpp"

#include <cstdio>
#include <cstring>

#include "launch.hpp"

namespace trace {
std::set<std::string>& all() {
    static std::set<std::string> s;
    return s;
}
std::vector<std::string>& launched() {
    static std::vector<std::string> v;
    return v;
}
}  // namespace trace

// what the kernels' registration refers to, and nothing here calls
extern "C" {
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipErrorUnknown; }
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) { return hipErrorUnknown; }
}

int main() {
    for (const std::string& s : trace::all()) printf("all|%s\n", s.c_str());
    char line[256];
    while (fgets(line, sizeof line, stdin) != nullptr) {
        long long v[8] = {};
        trace::launched().clear();
        if (sscanf(line, "lora %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6) == 7) {
            svdq::LoraBatchArgs a{};
            a.M = v[0]; a.K = (int)v[1]; a.N = (int)v[2]; a.R = (int)v[3];
            a.n_segments = (int)v[4]; a.n_adapters = (int)v[5]; a.bf16 = (int)v[6];
            svdq::launch_lora_batch(a, nullptr);
        } else if (sscanf(line, "norm %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7) == 8) {
            static char x, out;
            svdq::GroupNormArgs a{};
            a.B = v[0]; a.rows = v[1]; a.C = (int)v[2]; a.groups = (int)v[3];
            a.x_bf16 = (int)v[4]; a.out_bf16 = (int)v[5]; a.vec = (int)v[6];
            a.x = &x; a.out = v[7] ? &x : &out;
            svdq::launch_group_norm(a, nullptr);
        } else {
            return 2;
        }
        printf("call");
        for (const std::string& s : trace::launched()) printf("|%s", s.c_str());
        printf("\n");
    }
    return 0;
}
