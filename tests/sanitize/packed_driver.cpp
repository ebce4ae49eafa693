// packed_driver.cpp -- as batch_driver.cpp for svdq_layer_norm, svdq_rotary and svdq_attention: argument
// sets that must be refused, at the types' limits too, and the size query, for host code built with
// sanitizers.
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
#define REFUSED(type, change)     \
    {                             \
        type a;                   \
        change;                   \
        MUST_FAIL(a.call());      \
    }

static const void* at(uintptr_t p) { return (const void*)p; }
static const uintptr_t kAt = uintptr_t(1) << 20;

struct Layer {
    int64_t M = 5;
    int32_t C = 64, n = 2;
    float eps = 1e-6f;
    int32_t xd = 1, yd = 1, md = 0, od = 1;
    const void *x = at(kAt), *y = at(2 * kAt), *w = x, *b = x, *g = x, *s = x, *t = x;
    int64_t xs = 64, ys = 64, ms = 64, xos = 64, os = 64;
    const int32_t* st = (const int32_t*)x;
    void *xo = (void*)at(3 * kAt), *out = (void*)at(4 * kAt);
    svdq_status call() const {
        return svdq_layer_norm(M, C, n, eps, xd, x, xs, yd, y, ys, w, b, st, md, g, s, t, ms, xo, xos, od, out, os, nullptr);
    }
};

struct Rotary {
    int64_t M = 5;
    int32_t H = 4, G = 2, D = 64, n = 3;
    int32_t axes[4] = {8, 12, 12, 0};
    const int32_t* ax = axes;
    int32_t pr = 0, xd = 1, od = 1;
    const float* pos = (const float*)at(kAt);
    int64_t ps = 3;
    const double* f = (const double*)at(kAt);
    float eps = 1e-6f;
    const void *qw = at(kAt), *kw = qw, *q = qw, *k = at(2 * kAt);
    int64_t qs = 512, ks = 512, qos = 256, kos = 128;
    void *qo = (void*)at(3 * kAt), *ko = (void*)at(4 * kAt);
    svdq_status call() const {
        return svdq_rotary(M, H, G, D, n, ax, pr, pos, ps, f, eps, qw, kw, xd, q, qs, k, ks, od, qo, qos, ko, kos, nullptr);
    }
};

struct Attn {
    int64_t Mq = 5, Mk = 7;
    int32_t H = 4, G = 2, D = 64, n = 2;
    float scale = 0.125f, cap = 0.f;
    int32_t mask = 0;
    const int32_t *qs = (const int32_t*)at(kAt), *ks = qs, *pf = nullptr;
    const float* sl = nullptr;
    const void *q = at(kAt), *k = q, *v = q;
    int64_t qst = 256, kst = 128, vst = 128, ost = 256;
    void *out = (void*)at(2 * kAt), *ws = nullptr;
    int64_t wb = 0;
    svdq_status call() const {
        return svdq_attention(Mq, Mk, H, G, D, n, scale, cap, mask, qs, ks, pf, sl, q, qst, k, kst, v, vst, out, ost, ws, wb, nullptr);
    }
};

int main() {
    REFUSED(Layer, a.M = INT64_MIN) REFUSED(Layer, a.M = INT64_MAX) REFUSED(Layer, a.C = INT32_MIN) REFUSED(Layer, a.C = INT32_MAX)
    REFUSED(Layer, a.n = INT32_MIN) REFUSED(Layer, a.n = INT32_MAX) REFUSED(Layer, a.eps = NAN) REFUSED(Layer, a.eps = -1.f)
    REFUSED(Layer, a.xd = INT32_MAX) REFUSED(Layer, a.yd = 2) REFUSED(Layer, a.md = -1) REFUSED(Layer, a.od = 7)
    REFUSED(Layer, a.xs = INT64_MIN) REFUSED(Layer, a.ys = -1) REFUSED(Layer, a.ms = 0) REFUSED(Layer, a.xos = INT64_MIN) REFUSED(Layer, a.os = 63)
    REFUSED(Layer, a.x = nullptr) REFUSED(Layer, a.x = at(1)) REFUSED(Layer, a.y = nullptr) REFUSED(Layer, a.y = at(3)) REFUSED(Layer, a.w = at(1))
    REFUSED(Layer, a.g = at(2)) REFUSED(Layer, a.st = nullptr) REFUSED(Layer, a.out = nullptr) REFUSED(Layer, a.xo = a.out)
    REFUSED(Layer, a.C = 8193; a.xs = a.ys = a.ms = a.xos = a.os = INT64_MAX)

    REFUSED(Rotary, a.M = INT64_MIN) REFUSED(Rotary, a.M = INT64_MAX) REFUSED(Rotary, a.H = INT32_MIN) REFUSED(Rotary, a.G = INT32_MAX)
    REFUSED(Rotary, a.D = INT32_MIN) REFUSED(Rotary, a.D = INT32_MAX - 1) REFUSED(Rotary, a.n = INT32_MIN) REFUSED(Rotary, a.n = INT32_MAX)
    REFUSED(Rotary, a.ax = nullptr) REFUSED(Rotary, a.axes[0] = INT32_MIN) REFUSED(Rotary, a.axes[0] = a.axes[1] = a.axes[2] = INT32_MAX)
    REFUSED(Rotary, a.pr = -1) REFUSED(Rotary, a.pos = nullptr) REFUSED(Rotary, a.ps = INT64_MIN) REFUSED(Rotary, a.f = nullptr)
    REFUSED(Rotary, a.eps = INFINITY) REFUSED(Rotary, a.xd = 3) REFUSED(Rotary, a.od = 3) REFUSED(Rotary, a.qs = INT64_MIN) REFUSED(Rotary, a.kos = 0)
    REFUSED(Rotary, a.q = nullptr) REFUSED(Rotary, a.ko = nullptr) REFUSED(Rotary, a.qo = (void*)a.q)

    REFUSED(Attn, a.Mq = INT64_MIN) REFUSED(Attn, a.Mq = INT64_MAX) REFUSED(Attn, a.Mk = INT64_MAX) REFUSED(Attn, a.Mk = -1)
    REFUSED(Attn, a.H = INT32_MIN) REFUSED(Attn, a.H = INT32_MAX; a.G = 1) REFUSED(Attn, a.G = INT32_MIN) REFUSED(Attn, a.D = INT32_MIN)
    REFUSED(Attn, a.D = INT32_MAX - 7) REFUSED(Attn, a.n = INT32_MAX) REFUSED(Attn, a.n = INT32_MIN) REFUSED(Attn, a.scale = NAN)
    REFUSED(Attn, a.scale = 0.f) REFUSED(Attn, a.cap = NAN) REFUSED(Attn, a.cap = -0.5f) REFUSED(Attn, a.mask = INT32_MAX) REFUSED(Attn, a.qs = nullptr)
    REFUSED(Attn, a.pf = a.qs) REFUSED(Attn, a.qst = INT64_MIN) REFUSED(Attn, a.kst = INT64_MAX) REFUSED(Attn, a.vst = 127) REFUSED(Attn, a.ost = INT64_MAX - 7)
    REFUSED(Attn, a.k = nullptr) REFUSED(Attn, a.out = nullptr) REFUSED(Attn, a.ws = (void*)at(8)) REFUSED(Attn, a.Mk = 1 << 20)
    REFUSED(Attn, a.Mk = 1 << 20; a.ws = (void*)a.q; a.wb = INT64_MIN)

    for (int64_t Mq : {int64_t(0), int64_t(1), int64_t(4097), int64_t(1) << 24})
        for (int64_t Mk : {int64_t(0), int64_t(1), int64_t(1) << 30})
            for (int32_t H : {1, 24, 1 << 16})
                for (int32_t G : {1, H})
                    for (int32_t n : {0, 1, 1 << 16}) {
                        int64_t bytes = -1;
                        const svdq_status s = svdq_attention_workspace_bytes(Mq, Mk, H, G, 128, n, &bytes);
                        check(s == SVDQ_OK ? bytes >= 0 && bytes < int64_t(1) << 34 && (Mq > 0 || bytes == 0) : s == SVDQ_ERR_UNSUPPORTED_CONFIG,
                              "attention's workspace");
                    }
    std::printf("%d failures\n", failures);
    return failures != 0;
}
