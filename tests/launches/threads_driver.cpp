// threads_driver.cpp -- for each call read from stdin the threads of the launches that it makes:
//   layer  M C vec x_bf16
//   rotary M q_heads k_heads D halves vec word
//   attn   Mq Mk H G D n
#include "threads.hpp"

#include <cstdio>

#include "launch.hpp"

std::vector<unsigned long long>& threads::launched() {
    static std::vector<unsigned long long> v;
    return v;
}

int main() {
    char line[256];
    while (fgets(line, sizeof line, stdin) != nullptr) {
        long long v[7] = {};
        threads::launched().clear();
        if (sscanf(line, "layer %lld %lld %lld %lld", v, v + 1, v + 2, v + 3) == 4) {
            svdq::LayerNormArgs a{};
            a.M = v[0]; a.C = (int)v[1]; a.vec = (int)v[2]; a.x_bf16 = (int)v[3];
            svdq::launch_layer_norm(a, nullptr);
        } else if (sscanf(line, "rotary %lld %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6) == 7) {
            svdq::RotaryArgs a{};
            a.M = v[0]; a.q_heads = (int)v[1]; a.k_heads = (int)v[2]; a.D = (int)v[3];
            a.halves = (int)v[4]; a.vec = (int)v[5]; a.word = (int)v[6];
            svdq::launch_rotary(a, nullptr);
        } else if (sscanf(line, "attn %lld %lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4, v + 5) == 6) {
            svdq::AttentionArgs a{};
            a.Mq = v[0]; a.Mk = v[1]; a.H = (int)v[2]; a.G = (int)v[3]; a.D = (int)v[4]; a.n = (int)v[5];
            if (svdq::attention_fits(a.Mq, a.H, a.G, a.n)) svdq::launch_attention(a, nullptr);
        } else {
            return 2;
        }
        printf("call");
        for (const unsigned long long n : threads::launched()) printf(" %llu", n);
        printf("\n");
    }
    return 0;
}
