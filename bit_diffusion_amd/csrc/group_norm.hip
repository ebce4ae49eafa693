// group_norm.hip -- group normalisation of channels-last images, affine, optionally modulated
// by per-image scale and shift rows, with an activation.
//
// x is B images of `rows` positions x C channels, channels contiguous.  Per image and group of
// cg = C / groups channels, over n = rows cg values:
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  r = 1 / sqrt(var + eps)
//   out  = act(((x - mean) r w_c + b_c) (1 + scale_bc) + shift_bc)
// with the channel's terms folded to (x - mean) A_c + D_c, A = r w (1 + scale),
// D = b (1 + scale) + shift.  All of it in fp32; squares are summed about a mean, never about
// zero, so a large common offset costs no more than the rounding of the mean, 2^-24 of it.
//
// Bound: memory, x once and out once.  A workgroup works on a slab: a range of channels that
// is whole groups (or, for a group too wide, a part of one), so neighbouring lanes read
// neighbouring channels and no group is shared where it fits.
//   one launch (few rows): every workgroup of a slab takes the statistics of all its rows and
//             normalises its own share of them, which it keeps in registers meanwhile.  The
//             others' rows are read again from the caches; nothing is exchanged.  In place only
//             where a slab has one workgroup.
//   two launches (many rows): statistics of row tiles, then every workgroup joins those of its
//             groups, in a fixed order, and normalises a tile.
// Statistics of a thread go chunk by chunk, two passes over each in registers, joined as
// (count, mean, sum of squares about the mean): for two sets the joined M2 is
// M2a + M2b + d^2 na nb / (na + nb), d the difference of the means.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>
#include <numeric>
#include <type_traits>

namespace svdq {
namespace {

constexpr int kThreads = 256;      // of every workgroup
constexpr int kChunk = 8;         // rows of a thread's chunk in the statistics,
constexpr int kApply = 4;         // and in the launch that only normalises
// The one launch: vectors of a slab, at most (1 x 2048 x 256 channels, 8192 vectors: 6.8 us, in
// two launches 8.6; 2 x 2048 x 320 fp32, 10240: 14.8 us, 9.3), and vectors that all its
// workgroups read (2 x 1024 x 640, 0.8 million: 9.1 us, in two launches 10.9; 8 images, 3.3
// million: 18.5 us, 14.7).
constexpr int kOneVectors = 8192;
constexpr int64_t kOneReads = 1 << 20;
constexpr int64_t kStreamBytes = (int64_t)32 << 20;   // x that the L2s do not hold
constexpr int kMaxTiles = 256;    // row tiles of an image
constexpr int kWide = 512;        // channels of the widest slab (64 vectors of 8)

struct Shape {
    GroupNormArgs a;
    int cg;        // channels of a group
    int width;     // channels of a slab (the last part of a wide group may be narrower)
    int gs;        // groups of a slab (1 where a group is cut into parts)
    int parts;     // slabs of one group (1: a slab is whole groups)
    int slabs;     // slabs of an image
    int vpt;       // vectors of a slab
    float inv_vpt;
    int ty;        // row lanes of a workgroup
    int tiles;     // row tiles of an image
    int tile_rows;
};

// Channels [c0, c0 + w) of slab `s`, its first group and its part of that group.
__device__ __forceinline__ void slab_range(const Shape& p, int s, int& c0, int& w, int& g0, int& part) {
    if (p.parts == 1) {
        c0 = s * p.width; w = p.width; g0 = s * p.gs; part = 0;
    } else {
        g0 = s / p.parts; part = s - g0 * p.parts;
        c0 = g0 * p.cg + part * p.width;
        w = min(p.width, p.cg - part * p.width);
    }
}

// VEC consecutive channels of one position, as loaded: 16 bytes (8 of bf16, 4 of fp32) or one.
template <int VEC, bool BF16>
struct Vec {
    uint32_t w[VEC == 1 ? 1 : 4];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        if constexpr (VEC == 1) {
            w[0] = BF16 ? ((const uint16_t*)base)[at] : ((const uint32_t*)base)[at];
        } else {
            static_assert(VEC == (BF16 ? 8 : 4), "16 bytes");
            const uint4 u = *(const uint4*)((const char*)base + at * (BF16 ? 2 : 4));
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (BF16) return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        else return __uint_as_float(w[j]);
    }
};

// To memory, past the caches where STREAM.
template <bool STREAM, class T>
__device__ __forceinline__ void put(T v, void* p) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, (T*)p);
    else *(T*)p = v;
}

template <int VEC, bool BF16, bool STREAM>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&y)[VEC]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    char* p = (char*)base + at * (BF16 ? 2 : 4);
    if constexpr (BF16 && VEC == 8)
        put<STREAM>(u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])}, p);
    else if constexpr (BF16 && VEC == 4) put<STREAM>(u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])}, p);
    else if constexpr (BF16) put<STREAM>((uint16_t)pack_bf16(y[0], 0.f), p);
    else if constexpr (VEC == 1) put<STREAM>(y[0], p);
    else
#pragma unroll
        for (int h = 0; h < VEC; h += 4) put<STREAM>(f32x4{y[h], y[h + 1], y[h + 2], y[h + 3]}, p + h * 4);
}

// Statistics of a set of n values: their mean and the sum of their squares about it.
struct Moments {
    float n, mean, m2;
    // The union with another set, in this order; an empty set changes nothing.
    __device__ __forceinline__ void join(float bn, float bmean, float bm2) {
        const float tot = n + bn, inv = __builtin_amdgcn_rcpf(tot);
        // 1 and not nearly 1 for the first set: equal values keep their mean exactly
        const float share = bn > 0.f ? (n > 0.f ? bn * inv : 1.f) : 0.f, d = bmean - mean;
        mean += d * share;
        // weighted before it is squared: next to an empty set d is a whole mean, whose square
        // may overflow
        m2 += bm2 + d * (n * share) * d;
        n = tot;
    }
    template <int CTRL, int ROWS = 0xf>
    __device__ __forceinline__ void join_dpp() {
        join(dpp<CTRL, ROWS>(0.f, n), dpp<CTRL, ROWS>(0.f, mean), dpp<CTRL, ROWS>(0.f, m2));
    }
    // The union over each `lanes` (a power of two) lanes, in the last of them.
    __device__ __forceinline__ void join_lanes(int lanes) {
        if (lanes > 1) join_dpp<kShr + 1>();
        if (lanes > 2) join_dpp<kShr + 2>();
        if (lanes > 4) join_dpp<kShr + 4>();
        if (lanes > 8) join_dpp<kShr + 8>();
        if (lanes > 16) join_dpp<kBcast15, 0xa>();
        if (lanes > 32) join_dpp<kBcast31, 0xc>();
    }
};

// n / d for 0 <= n < 2^15, 0 < d < 2^15 and inv = 1 / d to an ulp: n + 1/2 keeps the quotient half a
// 2^15th away from the whole numbers.
__device__ __forceinline__ int quotient(int n, float inv) { return (int)(((float)n + 0.5f) * inv); }

// f(activation, whether out is bf16), both as types: the branch stands outside the loop over rows.
template <class F>
__device__ __forceinline__ void by_kind(int act, int bf16, F f) {
    auto kind = [&](auto b) {
        if (act == 1) f(std::integral_constant<int, 1>{}, b);
        else if (act == 2) f(std::integral_constant<int, 2>{}, b);
        else f(std::integral_constant<int, 0>{}, b);
    };
    if (bf16) kind(std::true_type{});
    else kind(std::false_type{});
}

// A slab's channels in LDS: first weight, bias, modulation scale and shift, loaded by different
// waves at a time (one after the other each would cost a memory latency); then what
// out = act((x - mean) A + D) takes, formed once for the workgroup.
struct Terms {
    float v[4][kWide];
    struct Source {
        const void* p;
        int64_t at;
        int kind;
        bool half;
        uint32_t first;   // the thread's first value as loaded
        __device__ __forceinline__ uint32_t get(int ch) const {
            return half ? ((const uint16_t*)p)[at + ch] : ((const uint32_t*)p)[at + ch];
        }
        __device__ __forceinline__ float value(uint32_t u) const {
            return p == nullptr ? (kind == 0 ? 1.f : 0.f) : __uint_as_float(half ? u << 16 : u);
        }
    };
    static __device__ __forceinline__ int channel() { return threadIdx.x & 63; }
    // starts the loads; what comes between this and put() need not wait for them
    static __device__ __forceinline__ Source load(const GroupNormArgs& a, int image, int c0, int width) {
        // & 3 takes nothing away, but without it the compiler selects the pointer's place among the
        // kernel's arguments and loads it from there, a memory latency more (1 x 4096 x 320: 11.8
        // us, 10.7 with it)
        const int kind = (threadIdx.x >> 6) & 3;
        Source s{kind == 0 ? a.weight : kind == 1 ? a.bias : kind == 2 ? a.mod_scale : a.mod_shift,
                 (kind < 2 ? 0 : (int64_t)image * a.mod_stride) + c0, kind, kind < 2 || a.mod_bf16 != 0, 0};
        if (s.p != nullptr && channel() < width) s.first = s.get(channel());
        return s;
    }
    __device__ __forceinline__ void put(const Source& s, int width) {
        if (channel() < width) v[s.kind][channel()] = s.value(s.first);
        for (int ch = channel() + kThreads / 4; ch < width; ch += kThreads / 4)
            v[s.kind][ch] = s.value(s.p == nullptr ? 0u : s.get(ch));
    }
    // v[0], v[1], v[2] become mean, A, D; cg: channels of a group in this slab
    __device__ __forceinline__ void fold(const float* mean, const float* rstd, int width, int cg) {
        const float inv = __builtin_amdgcn_rcpf((float)cg);
        for (int ch = threadIdx.x; ch < width; ch += kThreads) {
            const int g = quotient(ch, inv);
            const float m = 1.f + v[2][ch], A = rstd[g] * v[0][ch] * m, D = v[1][ch] * m + v[3][ch];
            v[0][ch] = mean[g];
            v[1][ch] = A;
            v[2][ch] = D;
        }
        __syncthreads();
    }
    template <int VEC>
    __device__ __forceinline__ void take(int ch, float (&mean)[VEC], float (&A)[VEC], float (&D)[VEC]) const {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            mean[j] = v[0][ch + j];
            A[j] = v[1][ch + j];
            D[j] = v[2][ch + j];
        }
    }
};

// A thread's running statistics, channel by channel.
template <int VEC>
struct Stats {
    float n, mean[VEC], m2[VEC];
    __device__ __forceinline__ void clear() {
        n = 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) mean[j] = m2[j] = 0.f;
    }
    // R rows, the first `live` (1 to R) of them counted; WHOLE: all of them.  Their mean is exact
    // for equal values, and finite where the values' sum is not: eighths of a whole chunk, four at
    // a time (no partial sum of equal values is rounded away); of a part of one, the first value
    // and the mean of the differences from it (for whole chunks too: 2 x 1024 x 640 9.7 us for 9.2).
    template <bool WHOLE, int R, bool XBF>
    __device__ __forceinline__ void add(const Vec<VEC, XBF> (&v)[R], int live) {
        static_assert(R == 8, "two halves of four");
        const float nc = WHOLE ? (float)R : (float)live, tot = n + nc;
        const float share = n > 0.f ? nc * __builtin_amdgcn_rcpf(tot) : 1.f, wgt = n * share;
        float s[VEC], q[VEC];
        if constexpr (WHOLE) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float t[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    t[h] = v[4 * h].get(j) * (1.f / R);
#pragma unroll
                    for (int i = 1; i < 4; ++i) t[h] = fmaf(v[4 * h + i].get(j), 1.f / R, t[h]);
                }
                s[j] = t[0] + t[1];
            }
        } else {
            const float inv_nc = __builtin_amdgcn_rcpf(nc);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[j] = 0.f;
#pragma unroll
            for (int i = 1; i < R; ++i)
                if (i < live) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s[j] += v[i].get(j) - v[0].get(j);
                }
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[j] = v[0].get(j) + s[j] * inv_nc;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = v[0].get(j) - s[j];
            q[j] = d * d;
        }
#pragma unroll
        for (int i = 1; i < R; ++i)
            if (WHOLE || i < live) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = v[i].get(j) - s[j];
                    q[j] += d * d;
                }
            }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = s[j] - mean[j];
            mean[j] += d * share;
            m2[j] += q[j] + d * wgt * d;
        }
        n = tot;
    }
    // `count` rows from x, `step` values apart
    template <int R, bool XBF>
    __device__ __forceinline__ void take(const void* x, int64_t at, int64_t step, int64_t count) {
        Vec<VEC, XBF> v[R];
        for (; count >= R; count -= R, at += R * step) {
#pragma unroll
            for (int i = 0; i < R; ++i) v[i].load(x, at + i * step);
            add<true>(v, R);
        }
        if (count > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (i < count) v[i].load(x, at + i * step);
            add<false>(v, (int)count);
        }
    }
};

// How a thread's vector lies in the groups: all of it in one, parts of it in two (a group has at
// least as many channels), or anyhow.
enum Span { kWhole, kTwo, kAny };

// Joins a workgroup's statistics by group.  A thread first joins its channels of one group; the
// entries (one, two or VEC a vector) stand in LDS as [row lane][vector][entry].  Waves take the
// groups in turn; where there are fewer groups than waves, several share a group's row lanes.
// In the end stat[0][g] is group g's mean and stat[1][g] what `finish` makes of its M2, for every
// thread.
template <int VEC, Span SPAN>
struct GroupJoin {
    static constexpr int EPV = SPAN == kWhole ? 1 : SPAN == kTwo ? 2 : VEC;
    static constexpr int kWaves = kThreads / 64;
    float n[kThreads * EPV], mean[kThreads * EPV], m2[kThreads * EPV];
    float part[3][kWaves];
    float stat[2][kWide];

    // cg: channels of a group in this slab
    template <class F>
    __device__ __forceinline__ void join(const Shape& p, int cg, const Stats<VEC>& st, int ty, int tx, F finish) {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        if (ty < p.ty) {
            const int at = (ty * p.vpt + tx) * EPV;
            if constexpr (SPAN == kAny) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    n[at + j] = st.n;
                    mean[at + j] = st.mean[j];
                    m2[at + j] = st.m2[j];
                }
            } else {
                // the first k channels lie in one group, the others in the next
                const int k = SPAN == kWhole ? VEC : min(VEC, (quotient(tx * VEC, __builtin_amdgcn_rcpf((float)cg)) + 1) * cg - tx * VEC);
                // their means about one of them, as in Stats::add
                const float m0 = st.mean[0], m1 = st.mean[VEC - 1];
                float mv[2] = {0.f, 0.f}, qv[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const bool in = SPAN == kWhole || j < k;
                    mv[0] += in ? st.mean[j] - m0 : 0.f;
                    mv[1] += in ? 0.f : st.mean[j] - m1;
                }
                mv[0] = m0 + mv[0] / (float)k;
                mv[1] = k < VEC ? m1 + mv[1] / (float)(VEC - k) : 0.f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const bool in = SPAN == kWhole || j < k;
                    const float d = st.mean[j] - (in ? mv[0] : mv[1]), t = st.m2[j] + st.n * d * d;
                    qv[0] += in ? t : 0.f;
                    qv[1] += in ? 0.f : t;
                }
#pragma unroll
                for (int h = 0; h < EPV; ++h) {
                    n[at + h] = st.n * (float)(h == 0 ? k : VEC - k);
                    mean[at + h] = mv[h];
                    m2[at + h] = qv[h];
                }
            }
        }
        __syncthreads();
        int log_per = 0;
        while ((2 << log_per) * p.gs <= kWaves) ++log_per;
        const int per = 1 << log_per;                             // waves of a group
        const int lanes = (p.ty + per - 1) >> log_per;            // row lanes of a wave
        for (int u = w; u < p.gs * per; u += kWaves) {
            const int g = u >> log_per, y0 = (u - (g << log_per)) * lanes, y1 = min(y0 + lanes, p.ty);
            // the group's entries of a row lane: of vectors v0 to v0 + wd - 1 (kAny: of channels)
            const int lo = g * cg, v0 = SPAN == kAny ? lo : lo / VEC;
            const int wd = SPAN == kAny ? cg : (lo + cg - 1) / VEC - v0 + 1;
            const float inv = __builtin_amdgcn_rcpf((float)wd);
            const int dy = quotient(64, inv), dc = 64 - dy * wd, ly = quotient(lane, inv);
            int y = y0 + ly, c = lane - ly * wd;
            Moments m{0.f, 0.f, 0.f};
            while (y < y1) {
                const int v = v0 + c;
                const int at = SPAN == kAny ? y * p.vpt * VEC + v
                                            : (y * p.vpt + v) * EPV + (SPAN == kTwo && v * VEC < lo ? 1 : 0);
                m.join(n[at], mean[at], m2[at]);
                y += dy;
                c += dc;
                if (c >= wd) { c -= wd; ++y; }
            }
            m.join_lanes(64);
            if (lane == 63) {
                if (per == 1) {
                    stat[0][g] = m.mean;
                    stat[1][g] = finish(m.m2);
                } else {
                    part[0][u] = m.n;
                    part[1][u] = m.mean;
                    part[2][u] = m.m2;
                }
            }
        }
        __syncthreads();
        if (per > 1) {
            if (w < p.gs) {
                const bool on = lane < per;
                Moments m{on ? part[0][w * per + lane] : 0.f, on ? part[1][w * per + lane] : 0.f,
                          on ? part[2][w * per + lane] : 0.f};
                m.join_lanes(per);
                if (lane == per - 1) {
                    stat[0][w] = m.mean;
                    stat[1][w] = finish(m.m2);
                }
            }
            __syncthreads();
        }
    }
};

// Bound by the launch, the latency of its loads and the joins: 2 x 64 x 1280 channels 4.6 us in a
// graph, 2 x 1024 x 640 9.1 us.
//
// One launch: workgroup (tile, slab, image) normalises R rows a thread, which it keeps, and takes
// the statistics of the whole slab, kChunk rows a thread at a time, in the same order as every
// other workgroup of the slab, so that all get the same ones.
template <int VEC, bool XBF, Span SPAN, int R>
__global__ __launch_bounds__(kThreads) void norm_one_kernel(Shape p) {
    __shared__ GroupJoin<VEC, SPAN> lds;
    __shared__ Terms terms;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, tile = blockIdx.y, b = blockIdx.z, rows = (int)a.rows;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = quotient(tid, p.inv_vpt), tx = tid - ty * p.vpt, c = c0 + tx * VEC;
    const bool on = ty < p.ty;
    const int64_t x0 = ((int64_t)b * rows) * a.x_stride + c;
    const Terms::Source src = Terms::load(a, b, c0, width);
    const int64_t step = (int64_t)p.ty * a.x_stride;
    Vec<VEC, XBF> own[R];
    Stats<VEC> st;
    st.clear();
    if (on && ty < rows) {
        const int64_t own0 = x0 + (int64_t)(tile * p.tile_rows + ty) * a.x_stride;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (tile * p.tile_rows + ty + i * p.ty < rows) own[i].load(a.x, own0 + i * step);
        st.template take<kChunk, XBF>(a.x, x0 + (int64_t)ty * a.x_stride, step, (rows - ty + p.ty - 1) / p.ty);
    }
    terms.put(src, width);
    const float inv = 1.f / ((float)rows * (float)p.cg);
    lds.join(p, p.cg, st, ty, tx, [&](float m2) { return 1.f / sqrtf(m2 * inv + a.eps); });
    terms.fold(lds.stat[0], lds.stat[1], width, p.cg);
    if (!on) return;
    float mean[VEC], A[VEC], D[VEC];
    terms.take(tx * VEC, mean, A, D);
    const int64_t o0 = ((int64_t)b * rows) * a.out_stride + c;
    by_kind(a.act, a.out_bf16, [&](auto act, auto obf) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = tile * p.tile_rows + ty + i * p.ty;
            if (r < rows) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = activate((own[i].get(j) - mean[j]) * A[j] + D[j], act);
                store_vec<VEC, decltype(obf)::value, false>(a.out, o0 + (int64_t)r * a.out_stride, y);
            }
        }
    });
}

// Bound by memory: 65536 x 512 channels 13 us (5.2 TB/s), 262144 x 256 channels of fp32 52 us
// (5.2 TB/s).
//
// Two launches, the first: (mean, M2) of each group (or part of one) of a row tile to
// work[b][group][part * tiles + tile].
template <int VEC, bool XBF, Span SPAN, int R>
__global__ __launch_bounds__(kThreads) void norm_stats_kernel(Shape p) {
    __shared__ GroupJoin<VEC, SPAN> lds;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, tile = blockIdx.y, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = quotient(tid, p.inv_vpt), tx = tid - ty * p.vpt;
    const int64_t first = (int64_t)tile * p.tile_rows, end = min(first + p.tile_rows, a.rows);
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c0 + tx * VEC;
    const int64_t step = (int64_t)p.ty * a.x_stride;
    Stats<VEC> st;
    st.clear();
    if (ty < p.ty && tx * VEC < width && first + ty < end)
        st.template take<R, XBF>(a.x, x0 + (first + ty) * a.x_stride, step, (end - first - ty + p.ty - 1) / p.ty);
    lds.join(p, p.parts == 1 ? p.cg : width, st, ty, tx, [](float m2) { return m2; });
    for (int g = tid; g < p.gs; g += kThreads)
        ((float2*)a.work)[((int64_t)b * a.groups + g0 + g) * p.parts * p.tiles + part * p.tiles + tile] =
            make_float2(lds.stat[0][g], lds.stat[1][g]);
}

// The second: the tiles are taken in the other order, the last ones read being the likeliest
// in the caches, and out goes past them where x is large (STREAM), to leave them to x.  Bound by
// memory: 65536 x 512 channels 22 us (6.1 TB/s, part of x from the caches), 262144 x 256 channels
// of fp32 to bf16 65 us (6.2 TB/s).
template <int VEC, bool XBF, int R, bool STREAM>
__global__ __launch_bounds__(kThreads) void norm_apply_kernel(Shape p) {
    __shared__ float stat[2][kWide];
    __shared__ Terms terms;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int tile = p.tiles - 1 - blockIdx.y, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = quotient(tid, p.inv_vpt), tx = tid - ty * p.vpt, c = c0 + tx * VEC;
    const bool on = ty < p.ty && tx * VEC < width;
    const int64_t first = (int64_t)tile * p.tile_rows, end = min(first + p.tile_rows, a.rows);
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c;
    const Terms::Source src = Terms::load(a, b, c0, width);
    const int64_t step = (int64_t)p.ty * a.x_stride, out_step = (int64_t)p.ty * a.out_stride;
    Vec<VEC, XBF> v[R];
    int64_t r = first + ty;
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (r + (int64_t)i * p.ty < end) v[i].load(a.x, x0 + r * a.x_stride + i * step);
    };
    if (on) load();                             // ahead of the statistics
    const int q_all = p.parts * p.tiles;
    const float inv = 1.f / ((float)a.rows * (float)p.cg);
    const float last_rows = (float)(a.rows - (int64_t)(p.tiles - 1) * p.tile_rows);
    // `lanes` lanes to a group, so that a wave's loads for several groups are in flight together
    int lanes = 64;
    while (lanes > 1 && lanes >= 2 * q_all) lanes /= 2;
    for (int g = (w * 64 + lane) / lanes; g < p.gs; g += kThreads / lanes) {
        const float2* src = (const float2*)a.work + ((int64_t)b * a.groups + g0 + g) * q_all;
        Moments m{0.f, 0.f, 0.f};
        for (int q = lane & (lanes - 1); q < q_all; q += lanes) {
            const int pt = p.parts == 1 ? 0 : q / p.tiles, ti = q - pt * p.tiles;
            const int wq = p.parts == 1 ? p.cg : min(p.width, p.cg - pt * p.width);
            const float2 v = src[q];
            m.join((ti == p.tiles - 1 ? last_rows : (float)p.tile_rows) * (float)wq, v.x, v.y);
        }
        m.join_lanes(lanes);
        if ((lane & (lanes - 1)) == lanes - 1) {
            stat[0][g] = m.mean;
            stat[1][g] = 1.f / sqrtf(m.m2 * inv + a.eps);
        }
    }
    terms.put(src, width);
    __syncthreads();
    terms.fold(stat[0], stat[1], width, p.parts == 1 ? p.cg : width);
    if (!on) return;
    float mean[VEC], A[VEC], D[VEC];
    terms.take(tx * VEC, mean, A, D);
    const int64_t o0 = ((int64_t)b * a.rows) * a.out_stride + c;
    by_kind(a.act, a.out_bf16, [&](auto act, auto obf) {
        while (r < end) {
            const int64_t o = o0 + r * a.out_stride;
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (r + (int64_t)i * p.ty < end) {
                    float y[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) y[j] = activate((v[i].get(j) - mean[j]) * A[j] + D[j], act);
                    store_vec<VEC, decltype(obf)::value, STREAM>(a.out, o + i * out_step, y);
                }
            r += (int64_t)p.ty * R;
            load();
        }
    });
}

// Whether vectors of v channels fit the groups: a slab of whole groups and whole vectors is not
// too wide, or a wide group is itself whole vectors.
bool vectors_fit(int C, int cg, int v) {
    return C % v == 0 && (std::lcm((int64_t)cg, (int64_t)v) <= 64 * v || cg % v == 0);
}

// Cuts the channels into slabs of `v`-channel vectors: the narrowest even cut into whole groups
// of `least` channels or more, else the widest.
Shape plan(const GroupNormArgs& a, int v, int least) {
    Shape p{};
    p.a = a;
    p.cg = a.C / a.groups;
    const int most = 64 * v;   // at most 64 vectors
    const int64_t unit = std::lcm((int64_t)p.cg, (int64_t)v);
    if (unit <= most) {
        const int units = (int)(a.C / unit);
        int m = 1;
        for (int k = 1; k <= units && k * unit <= most; ++k)
            if (units % k == 0 && m * unit < least) m = k;
        p.parts = 1;
        p.width = (int)unit * m;
        p.gs = p.width / p.cg;
        p.slabs = units / m;
    } else {
        p.width = most;
        p.parts = (p.cg + most - 1) / most;
        p.gs = 1;
        p.slabs = a.groups * p.parts;
    }
    p.vpt = p.width / v;
    p.inv_vpt = 1.f / (float)p.vpt;
    return p;
}

// The cut of the two launches: about 1024 workgroups (kMaxTiles at most for a slab of one image),
// each at least one chunk (2 x 65536 x 256 channels: 38.8 us; with 512 38.9, with 2048 43.6).
Shape split_plan(const GroupNormArgs& a, int v) {
    // slabs of 64 channels make whole cache lines (33.5 million values: 47 us, with 32 61 us), of 32
    // more workgroups (1.3 million: 12.1 us, with 64 12.5 us)
    Shape p = plan(a, v, a.B * a.rows * a.C < (1 << 22) ? 32 : 64);
    p.ty = kThreads / p.vpt;
    const int64_t step = (int64_t)p.ty * kChunk;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kMaxTiles, 1024 / std::max<int64_t>(1, a.B * p.slabs)));
    const int64_t per = std::max<int64_t>(1, (a.rows + want * step - 1) / (want * step)) * step;
    p.tile_rows = (int)per;
    p.tiles = (int)((a.rows + per - 1) / per);
    return p;
}

template <int VEC, bool XBF, Span SPAN>
void split(const GroupNormArgs& a, hipStream_t st) {
    const Shape p = split_plan(a, VEC);
    const dim3 grid((unsigned)p.slabs, (unsigned)p.tiles, (unsigned)a.B);
    hipLaunchKernelGGL((norm_stats_kernel<VEC, XBF, SPAN, kChunk>), grid, dim3(kThreads), 0, st, p);
    // 33.5 million values of bf16 (64 MB): 37.5 us with streaming stores, 47.6 without, and no less
    // with a reader of out behind them; 1.3 million: 12.5 us both ways, but the reader 1.2 us slower
    if (a.B * a.rows * a.C >= kStreamBytes / (XBF ? 2 : 4))
        hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF, kApply, true>), grid, dim3(kThreads), 0, st, p);
    else hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF, kApply, false>), grid, dim3(kThreads), 0, st, p);
}

template <int VEC, bool XBF, Span SPAN, int R>
void one(Shape p, hipStream_t st) {
    p.ty = kThreads / p.vpt;
    p.tile_rows = p.ty * R;
    p.tiles = (int)((p.a.rows + p.tile_rows - 1) / p.tile_rows);
    const dim3 grid((unsigned)p.slabs, (unsigned)p.tiles, (unsigned)p.a.B);
    hipLaunchKernelGGL((norm_one_kernel<VEC, XBF, SPAN, R>), grid, dim3(kThreads), 0, st, p);
}

template <int VEC, bool XBF, Span SPAN>
void run(const GroupNormArgs& a, hipStream_t st) {
    // slabs of 4 vectors or more (2 x 256 x 1280 channels: 6.1 us, of 8 6.9 us)
    const Shape p = plan(a, VEC, 4 * VEC);
    const int64_t vectors = p.vpt * a.rows, all = vectors * p.slabs * a.B;   // of a slab, of x
    // one row a thread while that takes 256 workgroups at most, else four (2 x 64 x 1280 channels:
    // 4.6 us, with four 4.85; 8 x 64 x 1280: 5.1 us, with one 5.4)
    const bool few = vectors <= kThreads || all <= 256 * kThreads;
    const int own = kThreads / p.vpt * (few ? 1 : 4);             // rows of a workgroup
    const int64_t tiles = (a.rows + own - 1) / own;          // each reads the whole slab
    // in place, a slab's second workgroup would overwrite rows that the first still reads
    if (p.parts > 1 || vectors > kOneVectors || all * tiles > kOneReads || (a.x == a.out && tiles > 1))
        split<VEC, XBF, SPAN>(a, st);
    else if (few) one<VEC, XBF, SPAN, 1>(p, st);
    else one<VEC, XBF, SPAN, 4>(p, st);
}

template <int VEC, bool XBF>
void run_vec(const GroupNormArgs& a, hipStream_t st) {
    const int cg = a.C / a.groups;
    if constexpr (VEC == 1) run<1, XBF, kWhole>(a, st);
    else if (cg % VEC == 0) run<VEC, XBF, kWhole>(a, st);
    else if (cg > VEC) run<VEC, XBF, kTwo>(a, st);
    else run<VEC, XBF, kAny>(a, st);
}

}  // namespace

int64_t group_norm_workspace_bytes(int64_t B, int64_t rows, int C, int groups) {
    // any of the vectors may be taken, by the types and the buffers' alignment
    int64_t most = 0;
    for (int v : {1, 4, 8}) {
        GroupNormArgs a{};
        a.B = B; a.rows = rows; a.C = C; a.groups = groups;
        if (B == 0 || rows == 0 || !vectors_fit(C, C / groups, v)) continue;
        const Shape p = split_plan(a, v);
        most = std::max(most, B * groups * (int64_t)p.parts * p.tiles * (int64_t)sizeof(float2));
    }
    return most;
}

void launch_group_norm(const GroupNormArgs& a, hipStream_t st) {
    const bool vec = a.vec && vectors_fit(a.C, a.C / a.groups, a.x_bf16 ? 8 : 4);
    if (a.x_bf16) vec ? run_vec<8, true>(a, st) : run_vec<1, true>(a, st);
    else vec ? run_vec<4, false>(a, st) : run_vec<1, false>(a, st);
}

}  // namespace svdq
