// packed_driver.cpp -- as driver.cpp for svdq_layer_norm, svdq_rotary and svdq_attention: every kernel
// that their launchers can start, then, for each call read from stdin, those that it starts.
//   layer  M C vec x_bf16 y_bf16 out_bf16
//   rotary M q_heads k_heads D halves vec word x_bf16 out_bf16
//   attn   Mq Mk H G D n cap bias
#include "trace.hpp"

#include <cstdio>

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
        long long v[9] = {};
        trace::launched().clear();
        if (sscanf(line, "layer %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5) == 6) {
            svdq::LayerNormArgs a{};
            a.M = v[0]; a.C = (int)v[1]; a.vec = (int)v[2];
            a.x_bf16 = (int)v[3]; a.y_bf16 = (int)v[4]; a.out_bf16 = (int)v[5];
            svdq::launch_layer_norm(a, nullptr);
        } else if (sscanf(line, "rotary %lld %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7, v + 8) == 9) {
            svdq::RotaryArgs a{};
            a.M = v[0]; a.q_heads = (int)v[1]; a.k_heads = (int)v[2]; a.D = (int)v[3];
            a.halves = (int)v[4]; a.vec = (int)v[5]; a.word = (int)v[6];
            a.x_bf16 = (int)v[7]; a.out_bf16 = (int)v[8];
            svdq::launch_rotary(a, nullptr);
        } else if (sscanf(line, "attn %lld %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7) == 8) {
            static float slopes;
            svdq::AttentionArgs a{};
            a.Mq = v[0]; a.Mk = v[1]; a.H = (int)v[2]; a.G = (int)v[3]; a.D = (int)v[4]; a.n = (int)v[5];
            a.cap = v[6] ? 30.f : 0.f;
            a.slopes = v[7] ? &slopes : nullptr;
            const bool fits = svdq::attention_fits(a.Mq, a.H, a.G, a.n);
            const long long bytes = svdq::attention_workspace_bytes(a.Mq, a.Mk, a.H, a.G, a.D, a.n);
            if (fits) svdq::launch_attention(a, nullptr);
            printf("bytes|%d|%lld\n", (int)fits, bytes);
        } else {
            return 2;
        }
        printf("call");
        for (const std::string& s : trace::launched()) printf("|%s", s.c_str());
        printf("\n");
    }
    return 0;
}
