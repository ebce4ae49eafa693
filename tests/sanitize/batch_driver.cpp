// batch_driver.cpp -- as host_driver.cpp for svdq_lora_batch and svdq_group_norm: argument sets that
// must be refused and the size queries up to their limits, for host code built with sanitizers.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/svdq.h"

static int failures = 0;
static void check(bool ok, const char* what) {
    if (!ok) {
        std::printf("wrong: %s\n", what);
        ++failures;
    }
}
#define MUST_FAIL(expr) check((expr) != SVDQ_OK && std::strlen(svdq_last_error()) > 0, #expr)
#define MUST_PASS(expr) check((expr) == SVDQ_OK, #expr)

struct Lora {
    int64_t M = 5;
    int32_t K = 128, N = 100, R = 16, S = 2, n = 3;
    const void* x = (void*)(uintptr_t(1) << 20);
    int64_t xs = 128;
    const void *down = x, *up = x;
    const float* al = (const float*)x;
    const int32_t *rk = nullptr, *st = (const int32_t*)x, *id = st;
    const void* base = x;
    int64_t bs = 100;
    int32_t act = 0, dt = 0;
    void* out = (void*)x;
    int64_t os = 100;
    void* ws = (void*)x;
    int64_t wb = int64_t(1) << 40;
    svdq_status call() const {
        return svdq_lora_batch(M, K, N, R, S, n, x, xs, down, up, al, rk, st, id, base, bs, act, dt, out, os, ws, wb, nullptr);
    }
};

struct Norm {
    int64_t B = 2, rows = 9;
    int32_t C = 64, G = 8;
    float eps = 1e-5f;
    int32_t xd = 1;
    const void* x = (void*)(uintptr_t(1) << 20);
    int64_t xs = 64;
    const void *w = nullptr, *b = nullptr;
    int32_t md = 0;
    const void *ms = x, *mt = x;
    int64_t mst = 64;
    int32_t act = 2, od = 1;
    void* out = (void*)(uintptr_t(1) << 21);
    int64_t os = 64;
    void* ws = (void*)x;
    int64_t wb = int64_t(1) << 60;
    svdq_status call() const {
        return svdq_group_norm(B, rows, C, G, eps, xd, x, xs, w, b, md, ms, mt, mst, act, od, out, os, ws, wb, nullptr);
    }
};

#define REFUSED(type, change)     \
    {                             \
        type a;                   \
        change;                   \
        MUST_FAIL(a.call());      \
    }

int main() {
    const auto at = [](uintptr_t p) { return (void*)p; };
    REFUSED(Lora, a.M = -1) REFUSED(Lora, a.M = INT64_MAX) REFUSED(Lora, a.M = INT64_MIN) REFUSED(Lora, a.K = 0)
    REFUSED(Lora, a.K = -64) REFUSED(Lora, a.K = INT32_MAX) REFUSED(Lora, a.N = 0) REFUSED(Lora, a.N = INT32_MIN)
    REFUSED(Lora, a.N = INT32_MAX; a.bs = a.os = INT64_MAX) REFUSED(Lora, a.R = 24) REFUSED(Lora, a.R = INT32_MAX - 15)
    REFUSED(Lora, a.S = -1) REFUSED(Lora, a.S = 0) REFUSED(Lora, a.n = -1) REFUSED(Lora, a.n = INT32_MAX)
    REFUSED(Lora, a.xs = INT64_MIN) REFUSED(Lora, a.xs = 129) REFUSED(Lora, a.x = nullptr) REFUSED(Lora, a.x = at(8))
    REFUSED(Lora, a.down = nullptr) REFUSED(Lora, a.up = at(2)) REFUSED(Lora, a.al = nullptr) REFUSED(Lora, a.st = nullptr)
    REFUSED(Lora, a.id = nullptr) REFUSED(Lora, a.rk = (const int32_t*)at(2)) REFUSED(Lora, a.bs = 99) REFUSED(Lora, a.act = -1)
    REFUSED(Lora, a.dt = 7) REFUSED(Lora, a.os = -100) REFUSED(Lora, a.out = nullptr) REFUSED(Lora, a.ws = at(8))
    REFUSED(Lora, a.wb = INT64_MIN)
    REFUSED(Norm, a.B = INT64_MAX) REFUSED(Norm, a.B = -1) REFUSED(Norm, a.rows = INT64_MIN) REFUSED(Norm, a.rows = INT64_MAX)
    REFUSED(Norm, a.C = INT32_MIN; a.G = -1) REFUSED(Norm, a.C = 65537; a.G = 1) REFUSED(Norm, a.G = 0) REFUSED(Norm, a.G = INT32_MIN)
    REFUSED(Norm, a.eps = -INFINITY) REFUSED(Norm, a.eps = NAN) REFUSED(Norm, a.eps = 0) REFUSED(Norm, a.xd = -1) REFUSED(Norm, a.md = 9)
    REFUSED(Norm, a.od = 2) REFUSED(Norm, a.act = 3) REFUSED(Norm, a.x = nullptr) REFUSED(Norm, a.x = at(1)) REFUSED(Norm, a.xs = 63)
    REFUSED(Norm, a.w = at(1)) REFUSED(Norm, a.ms = at(2)) REFUSED(Norm, a.mst = INT64_MIN) REFUSED(Norm, a.os = 0)
    REFUSED(Norm, a.out = (void*)a.x; a.od = 0) REFUSED(Norm, a.ws = nullptr) REFUSED(Norm, a.wb = -1)

    int64_t bytes = -1;
    for (int64_t M : {int64_t(0), int64_t(1), int64_t(4097), int64_t(1) << 22})
        for (int32_t n : {0, 1, 1000, 1 << 16})
            for (int32_t R : {16, 48, 128}) {
                bytes = -1;
                MUST_PASS(svdq_lora_batch_workspace_bytes(M, 1 << 24, 8, R, n, &bytes));
                check(bytes >= 0 && (M == 0 || n == 0 ? bytes == 0 : bytes >= M * R * 4 && bytes % 1024 == 0), "adapters' workspace");
            }
    for (int64_t B : {0, 1, 65535})
        for (int64_t rows : {int64_t(0), int64_t(1), int64_t(4097), int64_t(1) << 30})
            for (int32_t C : {1, 64, 330, 65535, 65536})
                for (int32_t G : {1, C % 5 == 0 ? 5 : 1, C}) {
                    bytes = -1;
                    MUST_PASS(svdq_group_norm_workspace_bytes(B, rows, C, G, &bytes));
                    check(B * rows == 0 ? bytes == 0 : bytes >= B * G * 8, "norm's workspace");
                }
    std::printf("%d failures\n", failures);
    return failures != 0;
}
