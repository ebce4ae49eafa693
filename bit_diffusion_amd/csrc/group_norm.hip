// group_norm.hip -- group normalisation of channels-last images, affine, optionally modulated
// by per-image scale and shift rows, with an activation.
//
// x is B images of `rows` positions x C channels, channels contiguous.  Per image and group of
// cg = C / groups channels, over n = rows cg values:
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  r = 1 / sqrt(var + eps)
//   out  = act(((x - mean) r w_c + b_c) (1 + scale_bc) + shift_bc)
// with the channel's terms folded to (x - mean) A_c + D_c, A = r w (1 + scale),
// D = b (1 + scale) + shift.  All of it in fp32; squares are summed about a mean, never about
// zero, so a large common offset costs nothing.
//
// Bound: memory, x once and out once.  A workgroup works on a slab: a range of channels that
// is whole groups (or, for a group too wide, a part of one), so neighbouring lanes read
// neighbouring channels and no group is shared where it fits.
//   one launch (few rows): every workgroup of a slab takes the statistics of all its rows and
//             normalises its own share of them, which it keeps in registers meanwhile.  The
//             others' rows are read again from the caches; nothing is exchanged.
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

constexpr int kSplitThreads = 256;
constexpr int kChunk = 8;         // rows of a thread's chunk in the statistics,
constexpr int kApply = 4;         // and in the launch that only normalises
constexpr int kOneVectors = 8192; // vectors of a slab in the one launch, at most
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
        if (bn > 0.f) {
            // 1 and not nearly 1 for the first set: equal values keep their mean exactly
            const float share = n > 0.f ? bn * __builtin_amdgcn_rcpf(n + bn) : 1.f, d = bmean - mean;
            mean += d * share;
            m2 += bm2 + d * d * (n * share);
            n += bn;
        }
    }
    // The union over each `lanes` (a power of two) lanes, in the first of them.
    __device__ __forceinline__ void join_lanes(int lanes) {
        for (int d = 1; d < lanes; d <<= 1) join(__shfl_down(n, d, 64), __shfl_down(mean, d, 64), __shfl_down(m2, d, 64));
    }
};

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
    __device__ __forceinline__ void load(const GroupNormArgs& a, int image, int c0, int width, int threads) {
        const int w = threadIdx.x >> 6, kind = w & 3;
        const void* p = kind == 0 ? a.weight : kind == 1 ? a.bias : kind == 2 ? a.mod_scale : a.mod_shift;
        const int64_t at = (kind < 2 ? 0 : (int64_t)image * a.mod_stride) + c0;
        const bool half = kind < 2 || a.mod_bf16;
        for (int ch = (w >> 2) * 64 + (threadIdx.x & 63); ch < width; ch += threads / 4) {
            float f = kind == 0 ? 1.f : 0.f;
            if (p != nullptr) f = half ? bf16_to_f32(((const uint16_t*)p)[at + ch]) : ((const float*)p)[at + ch];
            v[kind][ch] = f;
        }
    }
    // v[0], v[1], v[2] become mean, A, D; cg: channels of a group in this slab
    __device__ __forceinline__ void fold(const float* mean, const float* rstd, int width, int cg, int threads) {
        for (int ch = threadIdx.x; ch < width; ch += threads) {
            const int g = ch / cg;
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
    // R rows, the first `live` (1 to R) of them counted
    template <int R, bool XBF>
    __device__ __forceinline__ void add(const Vec<VEC, XBF> (&v)[R], int live) {
        const float nc = (float)live, tot = n + nc;
        const float share = n > 0.f ? nc * __builtin_amdgcn_rcpf(tot) : 1.f, wgt = n * share;
        float s[VEC], q[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[j] = v[0].get(j);
        rows(v, live, [&](const Vec<VEC, XBF>& r) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[j] += r.get(j);
        });
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            s[j] = live == R ? s[j] * (1.f / R) : s[j] / nc;   // exact for equal values
            const float d = v[0].get(j) - s[j];
            q[j] = d * d;
        }
        rows(v, live, [&](const Vec<VEC, XBF>& r) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = r.get(j) - s[j];
                q[j] += d * d;
            }
        });
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = s[j] - mean[j];
            mean[j] += d * share;
            m2[j] += q[j] + d * d * wgt;
        }
        n = tot;
    }

private:
    // f for rows 1 to live - 1; a whole chunk has no branch
    template <int R, bool XBF, class F>
    static __device__ __forceinline__ void rows(const Vec<VEC, XBF> (&v)[R], int live, F f) {
        if (live == R) {
#pragma unroll
            for (int i = 1; i < R; ++i) f(v[i]);
        } else {
#pragma unroll
            for (int i = 1; i < R; ++i)
                if (i < live) f(v[i]);
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
template <int VEC, Span SPAN, int BD>
struct GroupJoin {
    static constexpr int EPV = SPAN == kWhole ? 1 : SPAN == kTwo ? 2 : VEC;
    static constexpr int kWaves = BD / 64;
    float n[BD * EPV], mean[BD * EPV], m2[BD * EPV];
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
                const int k = SPAN == kWhole ? VEC : min(VEC, (tx * VEC / cg + 1) * cg - tx * VEC);
                float mv[2] = {0.f, 0.f}, qv[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const bool in = SPAN == kWhole || j < k;
                    mv[0] += in ? st.mean[j] : 0.f;
                    mv[1] += in ? 0.f : st.mean[j];
                }
                mv[0] /= (float)k;
                mv[1] = k < VEC ? mv[1] / (float)(VEC - k) : 0.f;
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
        int per = 1;                                              // waves of a group
        while (per * 2 * p.gs <= kWaves) per *= 2;
        const int lanes = (p.ty + per - 1) / per;                 // row lanes of a wave
        for (int u = w; u < p.gs * per; u += kWaves) {
            const int g = u / per, y0 = (u - g * per) * lanes, y1 = min(y0 + lanes, p.ty);
            // the group's entries of a row lane: of vectors v0 to v0 + wd - 1 (kAny: of channels)
            const int lo = g * cg, v0 = SPAN == kAny ? lo : lo / VEC;
            const int wd = SPAN == kAny ? cg : (lo + cg - 1) / VEC - v0 + 1;
            const int dy = 64 / wd, dc = 64 - dy * wd;
            int y = y0 + lane / wd, c = lane - lane / wd * wd;
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
            if (lane == 0) {
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
                if (lane == 0) {
                    stat[0][w] = m.mean;
                    stat[1][w] = finish(m.m2);
                }
            }
            __syncthreads();
        }
    }
};

// One launch: workgroup (tile, slab, image) normalises R rows a thread, which it keeps, and takes
// the statistics of the whole slab, kChunk rows a thread at a time, in the same order as every
// other workgroup of the slab, so that all get the same ones.
template <int VEC, bool XBF, Span SPAN, int R, int BD>
__global__ __launch_bounds__(BD) void norm_one_kernel(Shape p) {
    __shared__ GroupJoin<VEC, SPAN, BD> lds;
    __shared__ Terms terms;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, tile = blockIdx.y, b = blockIdx.z, rows = (int)a.rows;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = tid / p.vpt, tx = tid - ty * p.vpt, c = c0 + tx * VEC;
    const bool on = ty < p.ty;
    const int64_t x0 = ((int64_t)b * rows) * a.x_stride + c;
    Vec<VEC, XBF> own[R], v[kChunk];
    auto load = [&](int r, int live) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i].load(a.x, x0 + (int64_t)(r + min(i, live - 1) * p.ty) * a.x_stride);
    };
    auto live_at = [&](int r) { return min(kChunk, (rows - r + p.ty - 1) / p.ty); };
    int r = ty;
    if (on && r < rows) {
        load(r, live_at(r));
#pragma unroll
        for (int i = 0; i < R; ++i)
            own[i].load(a.x, x0 + (int64_t)min(tile * p.tile_rows + ty + i * p.ty, rows - 1) * a.x_stride);
    }
    terms.load(a, b, c0, width, BD);
    Stats<VEC> st;
    st.clear();
    while (on && r < rows) {
        st.add(v, live_at(r));
        r += p.ty * kChunk;
        if (r < rows) load(r, live_at(r));
    }
    const float inv = 1.f / ((float)rows * (float)p.cg);
    lds.join(p, p.cg, st, ty, tx, [&](float m2) { return 1.f / sqrtf(m2 * inv + a.eps); });
    terms.fold(lds.stat[0], lds.stat[1], width, p.cg, BD);
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

// Two launches, the first: (mean, M2) of each group (or part of one) of a row tile to
// work[b][group][part * tiles + tile].
template <int VEC, bool XBF, Span SPAN, int R>
__global__ __launch_bounds__(kSplitThreads) void norm_stats_kernel(Shape p) {
    __shared__ GroupJoin<VEC, SPAN, kSplitThreads> lds;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, tile = blockIdx.y, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = tid / p.vpt, tx = tid - ty * p.vpt;
    const int64_t first = (int64_t)tile * p.tile_rows, end = min(first + p.tile_rows, a.rows);
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c0 + tx * VEC;
    Stats<VEC> st;
    st.clear();
    if (ty < p.ty && tx * VEC < width)
        for (int64_t r = first + ty; r < end; r += (int64_t)p.ty * R) {
            Vec<VEC, XBF> v[R];
            const int live = (int)min((int64_t)R, (end - r + p.ty - 1) / p.ty);
#pragma unroll
            for (int i = 0; i < R; ++i) v[i].load(a.x, x0 + (r + (int64_t)min(i, live - 1) * p.ty) * a.x_stride);
            st.add(v, live);
        }
    lds.join(p, p.parts == 1 ? p.cg : width, st, ty, tx, [](float m2) { return m2; });
    for (int g = tid; g < p.gs; g += kSplitThreads)
        ((float2*)a.work)[((int64_t)b * a.groups + g0 + g) * p.parts * p.tiles + part * p.tiles + tile] =
            make_float2(lds.stat[0][g], lds.stat[1][g]);
}

// The second: the tiles are taken in the other order, the last ones read being the likeliest
// in the caches, and out goes past them where x is large (STREAM), to leave them to x.
template <int VEC, bool XBF, int R, bool STREAM>
__global__ __launch_bounds__(kSplitThreads) void norm_apply_kernel(Shape p) {
    __shared__ float stat[2][kWide];
    __shared__ Terms terms;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int tile = p.tiles - 1 - blockIdx.y, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = tid / p.vpt, tx = tid - ty * p.vpt, c = c0 + tx * VEC;
    const bool on = ty < p.ty && tx * VEC < width;
    const int64_t first = (int64_t)tile * p.tile_rows, end = min(first + p.tile_rows, a.rows);
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c;
    Vec<VEC, XBF> v[R];
    int64_t r = first + ty;
    auto load = [&](int live) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i].load(a.x, x0 + (r + (int64_t)min(i, live - 1) * p.ty) * a.x_stride);
    };
    auto live_at = [&]() { return (int)min((int64_t)R, (end - r + p.ty - 1) / p.ty); };
    if (on && r < end) load(live_at());         // ahead of the statistics
    terms.load(a, b, c0, width, kSplitThreads);
    const int q_all = p.parts * p.tiles;
    const float inv = 1.f / ((float)a.rows * (float)p.cg);
    const float last_rows = (float)(a.rows - (int64_t)(p.tiles - 1) * p.tile_rows);
    // `lanes` lanes to a group, so that a wave's loads for several groups are in flight together
    int lanes = 64;
    while (lanes > 1 && lanes >= 2 * q_all) lanes /= 2;
    for (int g = (w * 64 + lane) / lanes; g < p.gs; g += kSplitThreads / lanes) {
        const float2* src = (const float2*)a.work + ((int64_t)b * a.groups + g0 + g) * q_all;
        Moments m{0.f, 0.f, 0.f};
        for (int q = lane & (lanes - 1); q < q_all; q += lanes) {
            const int pt = p.parts == 1 ? 0 : q / p.tiles, ti = q - pt * p.tiles;
            const int wq = p.parts == 1 ? p.cg : min(p.width, p.cg - pt * p.width);
            const float2 v = src[q];
            m.join((ti == p.tiles - 1 ? last_rows : (float)p.tile_rows) * (float)wq, v.x, v.y);
        }
        m.join_lanes(lanes);
        if ((lane & (lanes - 1)) == 0) {
            stat[0][g] = m.mean;
            stat[1][g] = 1.f / sqrtf(m.m2 * inv + a.eps);
        }
    }
    __syncthreads();
    terms.fold(stat[0], stat[1], width, p.parts == 1 ? p.cg : width, kSplitThreads);
    if (!on) return;
    float mean[VEC], A[VEC], D[VEC];
    terms.take(tx * VEC, mean, A, D);
    const int64_t o0 = ((int64_t)b * a.rows) * a.out_stride + c;
    by_kind(a.act, a.out_bf16, [&](auto act, auto obf) {
        while (r < end) {
            const int live = live_at();
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (i < live) {
                    float y[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) y[j] = activate((v[i].get(j) - mean[j]) * A[j] + D[j], act);
                    store_vec<VEC, decltype(obf)::value, STREAM>(a.out, o0 + (r + (int64_t)i * p.ty) * a.out_stride, y);
                }
            r += (int64_t)p.ty * R;
            if (r < end) load(live_at());
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
    return p;
}


// The cut of the two launches: about 1024 workgroups, each at least one chunk.
Shape split_plan(const GroupNormArgs& a, int v) {
    // slabs of 64 channels make whole cache lines (33.5 million values: 47 us, with 32 61 us), of 32
    // more workgroups (1.3 million: 12.1 us, with 64 12.5 us)
    Shape p = plan(a, v, a.B * a.rows * a.C < (1 << 22) ? 32 : 64);
    p.ty = kSplitThreads / p.vpt;
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
    hipLaunchKernelGGL((norm_stats_kernel<VEC, XBF, SPAN, kChunk>), grid, dim3(kSplitThreads), 0, st, p);
    // 33.5 million values of bf16 (64 MB): 37.5 us with streaming stores, 47.6 without, and no less
    // with a reader of out behind them; 1.3 million: 12.5 us both ways, but the reader 1.2 us slower
    if (a.B * a.rows * a.C * (XBF ? 2 : 4) >= kStreamBytes)
        hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF, kApply, true>), grid, dim3(kSplitThreads), 0, st, p);
    else hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF, kApply, false>), grid, dim3(kSplitThreads), 0, st, p);
}

template <int VEC, bool XBF, Span SPAN, int R, int BD>
void one(Shape p, hipStream_t st) {
    p.ty = BD / p.vpt;
    p.tile_rows = p.ty * R;
    p.tiles = (int)((p.a.rows + p.tile_rows - 1) / p.tile_rows);
    const dim3 grid((unsigned)p.slabs, (unsigned)p.tiles, (unsigned)p.a.B);
    hipLaunchKernelGGL((norm_one_kernel<VEC, XBF, SPAN, R, BD>), grid, dim3(BD), 0, st, p);
}

template <int VEC, bool XBF, Span SPAN>
void run(const GroupNormArgs& a, hipStream_t st) {
    const Shape p = plan(a, VEC, 4 * VEC);
    const int64_t vectors = p.vpt * a.rows;                  // of a slab
    if (p.parts > 1 || vectors > kOneVectors) split<VEC, XBF, SPAN>(a, st);
    else if (vectors <= 256 || vectors * p.slabs * a.B <= 256 * 256) one<VEC, XBF, SPAN, 1, 256>(p, st);
    else one<VEC, XBF, SPAN, 4, 256>(p, st);
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
