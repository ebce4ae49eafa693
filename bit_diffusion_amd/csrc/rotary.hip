// rotary.hip -- the q and k heads of a fused q, k, v linear made ready for attention: an optional
// RMS norm over each head's D channels, then every channel pair (a, b) turned by its angle,
//   (a cos t - b sin t, a sin t + b cos t),  t = positions[row, axis of the pair] freqs[pair],
// the pairs dealt over up to four axes (time, height, width, ...) in order.
//
// Angles.  t reaches 1e6 and more where frames lie far from the first, and a float holds it to
// 2^-24 of that only.  So the product is formed in binary64, in turns, its whole turns are taken
// off there, and the rest, at most half a turn, goes to sincospif.  One angle serves all heads of
// its row: a workgroup fills a table of kRows rows x D / 2 pairs in LDS once and takes all heads
// through it.
//
// Bound: memory, q and k once in and once out.  Aligned heads: a lane holds 8 channels (16 bytes
// of bf16) in adjacent pairs, or 8 from either half, and a head is a group of 8, 16 or 32 lanes of
// one wave, so the norm's sum needs no LDS; the next head is loaded before this one is turned, the
// first before the table is made.  Other head widths and alignments: a lane holds single pairs.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>
#include <type_traits>

namespace svdq {
namespace {

constexpr int kThreads = 256;
constexpr int kCus = 256;    // of the GPU
constexpr int kMaxPairs = 128;
constexpr int kRows = 16;    // rows of a workgroup, at most
// Heads that a group of lanes takes: so many pay for the angle table and its start (4608 rows of 48
// heads of 128: 30.5 us, with 4 heads 36, with one 39; 6001 rows of 20 heads of 96, fp32: 16.6, 16.5 and
// 24.3).
constexpr int kPerGroup = 16;

// cos and sin of `rows` rows' angles: table[row][pair].
__device__ __forceinline__ void fill_table(const RotaryArgs& a, int64_t row0, int rows, float2* table) {
    const int P = a.D >> 1;
    for (int i = threadIdx.x; i < rows * P; i += kThreads) {
        const int r = i / P, p = i - r * P;
        const int axis = (p >= a.ends[0]) + (p >= a.ends[1]) + (p >= a.ends[2]);
        const double turns = (double)a.pos[(row0 + r) * a.pos_stride + axis] * a.freqs[p] * 0.15915494309189533577;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        table[i] = make_float2(c, s);
    }
}
// A barrier that waits for this wave's LDS accesses only: loads stay in flight.
__device__ __forceinline__ void sync() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The sum over each LANES (8, 16, 32) neighbouring lanes, in all of them.
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
    v += dpp<0xB1>(0.f, v);     // the neighbour
    v += dpp<0x4E>(0.f, v);     // the other two of four
    v += dpp<0x141>(0.f, v);    // the other half of eight, mirrored
    if constexpr (LANES > 8) v += dpp<0x140>(0.f, v);
    if constexpr (LANES > 16) v += __shfl_xor(v, 16, kWave);
    return v;
}

// A group of lanes' head: its row in the workgroup and its number there; `by` heads further each time.
struct Item {
    int r, h;
};
struct Step {
    int heads, r, h;
    __device__ __forceinline__ Step(int by, int heads_) : heads(heads_), r(by / heads_), h(by - by / heads_ * heads_) {}
    __device__ __forceinline__ void next(Item& t) const {
        t.r += r;
        t.h += h;
        if (t.h >= heads) {
            t.h -= heads;
            ++t.r;
        }
    }
};

// 8 channels as loaded.
template <bool BF16>
struct Vec {
    uint4 u[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        const uint4* s = (const uint4*)((const char*)p + at * (BF16 ? 2 : 4));
        u[0] = s[0];
        if constexpr (!BF16) u[1] = s[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[BF16 ? 0 : 1].x, u[BF16 ? 0 : 1].y, u[BF16 ? 0 : 1].z, u[BF16 ? 0 : 1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = __uint_as_float(!BF16 ? w[j] : (j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    }
};

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
    if constexpr (BF16) {
        *(uint4*)((uint16_t*)p + at) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        float4* d = (float4*)((float*)p + at);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// LANES: lanes of a head, a power of two; those past its vectors idle.
template <int LANES, bool HALVES, bool XBF, bool OBF>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int per) {
    __shared__ float2 table[kRows * kMaxPairs];
    const int64_t row0 = (int64_t)blockIdx.x * per;
    const int rows = (int)min((int64_t)per, a.M - row0), P = a.D >> 1;
    constexpr int NV = HALVES ? 2 : 1, kHeads = kThreads / LANES;   // heads at a time
    const int l = threadIdx.x % LANES, first = threadIdx.x / LANES;
    const bool on = l * 8 < (HALVES ? P : a.D);
    const int ch[2] = {l * 8, P + l * 8};
    const int heads = a.q_heads + a.k_heads;
    const float inv_d = 1.f / (float)a.D;
    float wq[NV][8], wk[NV][8];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) wq[n][j] = wk[n][j] = 1.f;
    if (on) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (a.q_weight != nullptr) wq[n][j] = bf16_to_f32(((const uint16_t*)a.q_weight)[ch[n] + j]);
                if (a.k_weight != nullptr) wk[n][j] = bf16_to_f32(((const uint16_t*)a.k_weight)[ch[n] + j]);
            }
    }
    Vec<XBF> v[NV];
    auto fetch = [&](const Item& t) {
        if (t.r >= rows || !on) return;
        const bool q = t.h < a.q_heads;
        const int64_t at = (row0 + t.r) * (q ? a.q_stride : a.k_stride) + (int64_t)(q ? t.h : t.h - a.q_heads) * a.D;
#pragma unroll
        for (int n = 0; n < NV; ++n) v[n].load(q ? a.q : a.k, at + ch[n]);
    };
    const Step step(kHeads, heads);
    Item t{first / heads, first % heads}, ahead = t;
    fetch(t);                   // on its way while the table is made
    fill_table(a, row0, rows, table);
    sync();
    for (; __any(t.r < rows); t = ahead) {
        const bool q = t.h < a.q_heads, mine = t.r < rows && on;
        float x[NV][8];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[n][j] = 0.f;
            if (mine) v[n].get(x[n]);
        }
        step.next(ahead);
        fetch(ahead);
        if (a.q_weight != nullptr || a.k_weight != nullptr) {
            float s = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(x[n][j], x[n][j], s);
            s = rsqrt_hw(fmaf(group_sum<LANES>(s), inv_d, a.eps));
            if ((q ? a.q_weight : a.k_weight) != nullptr) {
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[n][j] *= s * (q ? wq[n][j] : wk[n][j]);
            }
        }
        if (!mine) continue;
        const float2* cs = table + t.r * P + (HALVES ? l * 8 : l * 4);
        float y[NV][8];
#pragma unroll
        for (int p = 0; p < (HALVES ? 8 : 4); ++p) {
            float& ya = y[0][HALVES ? p : 2 * p];
            float& yb = y[NV - 1][HALVES ? p : 2 * p + 1];
            const float xa = x[0][HALVES ? p : 2 * p], xb = x[NV - 1][HALVES ? p : 2 * p + 1];
            ya = fmaf(xa, cs[p].x, -xb * cs[p].y);
            yb = fmaf(xa, cs[p].y, xb * cs[p].x);
        }
        const int64_t at = (row0 + t.r) * (q ? a.q_out_stride : a.k_out_stride) + (int64_t)(q ? t.h : t.h - a.q_heads) * a.D;
#pragma unroll
        for (int n = 0; n < NV; ++n) store8<OBF>(q ? a.q_out : a.k_out, at + ch[n], y[n]);
    }
}

// The two channels of a pair: side by side and aligned as one (WORD), or anyhow.
template <bool WORD, bool BF16>
__device__ __forceinline__ float2 load_pair(const void* p, int64_t at, int a, int b) {
    if constexpr (WORD && BF16) {
        const uint32_t w = *(const uint32_t*)((const uint16_t*)p + at + a);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else if constexpr (WORD) {
        return *(const float2*)((const float*)p + at + a);
    } else if constexpr (BF16) {
        return make_float2(bf16_to_f32(((const uint16_t*)p)[at + a]), bf16_to_f32(((const uint16_t*)p)[at + b]));
    } else {
        return make_float2(((const float*)p)[at + a], ((const float*)p)[at + b]);
    }
}
template <bool WORD, bool BF16>
__device__ __forceinline__ void store_pair(void* p, int64_t at, int a, int b, float2 v) {
    if constexpr (WORD && BF16) {
        *(uint32_t*)((uint16_t*)p + at + a) = pack_bf16(v.x, v.y);
    } else if constexpr (WORD) {
        *(float2*)((float*)p + at + a) = v;
    } else if constexpr (BF16) {
        const uint32_t w = pack_bf16(v.x, v.y);
        ((uint16_t*)p)[at + a] = (uint16_t)w;
        ((uint16_t*)p)[at + b] = (uint16_t)(w >> 16);
    } else {
        ((float*)p)[at + a] = v.x;
        ((float*)p)[at + b] = v.y;
    }
}

// Any even D and any alignment: as above, a lane holding the pairs lane, lane + LANES, ...
template <int LANES, int NP, bool WORD, bool XBF, bool OBF>
__global__ __launch_bounds__(kThreads) void rotary_pairs_kernel(RotaryArgs a, int per) {
    __shared__ float2 table[kRows * kMaxPairs];
    const int64_t row0 = (int64_t)blockIdx.x * per;
    const int rows = (int)min((int64_t)per, a.M - row0), P = a.D >> 1, heads = a.q_heads + a.k_heads;
    constexpr int kHeads = kThreads / LANES;
    const int l = threadIdx.x % LANES, first = threadIdx.x / LANES;
    const float inv_d = 1.f / (float)a.D;
    int ca[NP], cb[NP];
    float2 wq[NP], wk[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int p = l + n * LANES;
        ca[n] = WORD || !a.halves ? 2 * p : p;
        cb[n] = WORD || !a.halves ? 2 * p + 1 : p + P;
        wq[n] = wk[n] = make_float2(1.f, 1.f);
        if (p < P && a.q_weight != nullptr) wq[n] = load_pair<false, true>(a.q_weight, 0, ca[n], cb[n]);
        if (p < P && a.k_weight != nullptr) wk[n] = load_pair<false, true>(a.k_weight, 0, ca[n], cb[n]);
    }
    float2 v[NP];
    auto fetch = [&](const Item& t) {
        if (t.r >= rows) return;
        const bool q = t.h < a.q_heads;
        const int64_t at = (row0 + t.r) * (q ? a.q_stride : a.k_stride) + (int64_t)(q ? t.h : t.h - a.q_heads) * a.D;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (l + n * LANES < P) v[n] = load_pair<WORD, XBF>(q ? a.q : a.k, at, ca[n], cb[n]);
    };
    const Step step(kHeads, heads);
    Item t{first / heads, first % heads}, ahead = t;
    fetch(t);
    fill_table(a, row0, rows, table);
    sync();
    for (; __any(t.r < rows); t = ahead) {
        const bool q = t.h < a.q_heads, mine = t.r < rows;
        float2 x[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) x[n] = mine && l + n * LANES < P ? v[n] : make_float2(0.f, 0.f);
        step.next(ahead);
        fetch(ahead);
        if (a.q_weight != nullptr || a.k_weight != nullptr) {
            float s = 0.f;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                s = fmaf(x[n].x, x[n].x, s);
                s = fmaf(x[n].y, x[n].y, s);
            }
            s = rsqrt_hw(fmaf(group_sum<LANES>(s), inv_d, a.eps));
            if ((q ? a.q_weight : a.k_weight) != nullptr) {
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    x[n].x *= s * (q ? wq[n].x : wk[n].x);
                    x[n].y *= s * (q ? wq[n].y : wk[n].y);
                }
            }
        }
        if (!mine) continue;
        const int64_t at = (row0 + t.r) * (q ? a.q_out_stride : a.k_out_stride) + (int64_t)(q ? t.h : t.h - a.q_heads) * a.D;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int p = l + n * LANES;
            if (p >= P) continue;
            const float2 cs = table[t.r * P + p];
            store_pair<WORD, OBF>(q ? a.q_out : a.k_out, at, ca[n], cb[n],
                                  make_float2(fmaf(x[n].x, cs.x, -x[n].y * cs.y), fmaf(x[n].x, cs.y, x[n].y * cs.x)));
        }
    }
}

template <bool XBF, bool OBF>
void launch(const RotaryArgs& a, hipStream_t st) {
    const int heads = a.q_heads + a.k_heads, vecs = (a.halves ? a.D / 2 : a.D) / 8;
    const int lanes = a.vec ? (vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32) : a.D <= 128 ? 16 : 32, at_once = kThreads / lanes;
    const int64_t rows = std::min<int64_t>(a.M / kCus, (kPerGroup * at_once + heads - 1) / heads);
    // two at least where one each would be 2^24 workgroups: a launch has fewer than 2^32 threads
    const int per = (int)std::min<int64_t>(kRows, std::max<int64_t>(a.M > (int64_t)1 << 23 ? 2 : 1, rows));
    const dim3 grid((unsigned)((a.M + per - 1) / per)), block(kThreads);
    if (!a.vec) {
        auto pairs = [&](auto n, auto np) {
            if (a.word) hipLaunchKernelGGL((rotary_pairs_kernel<n.value, np.value, true, XBF, OBF>), grid, block, 0, st, a, per);
            else hipLaunchKernelGGL((rotary_pairs_kernel<n.value, np.value, false, XBF, OBF>), grid, block, 0, st, a, per);
        };
        if (a.D <= 64) pairs(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
        else if (a.D <= 128) pairs(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
        else pairs(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
        return;
    }
    auto go = [&](auto n) {
        if constexpr (n.value < 32) {
            if (a.halves) {
                hipLaunchKernelGGL((rotary_kernel<n.value, true, XBF, OBF>), grid, block, 0, st, a, per);
                return;
            }
        }
        hipLaunchKernelGGL((rotary_kernel<n.value, false, XBF, OBF>), grid, block, 0, st, a, per);
    };
    if (lanes == 8) go(std::integral_constant<int, 8>{});
    else if (lanes == 16) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 32>{});   // never pairs of halves, which have 16 vectors at most
}

}  // namespace

void launch_rotary(const RotaryArgs& a, hipStream_t st) {
    if (a.x_bf16) a.out_bf16 ? launch<true, true>(a, st) : launch<true, false>(a, st);
    else a.out_bf16 ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace svdq
