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
constexpr int kOneThreads = 512;
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

template <int VEC, bool BF16>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&y)[VEC]) {
    if constexpr (BF16) {
        uint16_t* p = (uint16_t*)base + at;
        if constexpr (VEC == 8) *(uint4*)p = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                        pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        else if constexpr (VEC == 4) *(uint2*)p = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        else p[0] = (uint16_t)pack_bf16(y[0], 0.f);
    } else {
        float* p = (float*)base + at;
        if constexpr (VEC == 1) p[0] = y[0];
        else
#pragma unroll
            for (int h = 0; h < VEC; h += 4) *(f32x4*)(p + h) = f32x4{y[h], y[h + 1], y[h + 2], y[h + 3]};
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

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

// A slab's weight, bias, modulation scale and shift in LDS.  The four kinds are loaded by
// different threads at a time: one after the other each would cost a memory latency.
struct Terms {
    float v[4][kWide];
    __device__ __forceinline__ void load(const GroupNormArgs& a, int image, int c0, int width, int threads) {
        for (int i = threadIdx.x; i < 4 * width; i += threads) {
            const int kind = i / width, ch = i - kind * width;
            const void* p = kind == 0 ? a.weight : kind == 1 ? a.bias : kind == 2 ? a.mod_scale : a.mod_shift;
            const int64_t at = (kind < 2 ? 0 : (int64_t)image * a.mod_stride) + c0 + ch;
            float f = kind == 0 ? 1.f : 0.f;
            if (p != nullptr) f = kind < 2 || a.mod_bf16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
            v[kind][ch] = f;
        }
    }
    // out = act((x - mean) A + D) for channel ch of the slab and r = 1 / sqrt(var + eps)
    __device__ __forceinline__ void fold(int ch, float r, float& A, float& D) const {
        const float m = 1.f + v[2][ch];
        A = r * v[0][ch] * m;
        D = v[1][ch] * m + v[3][ch];
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
        const float nc = (float)live, tot = n + nc, inv = 1.f / nc, share = nc / tot, wgt = n * share;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float s = 0.f, q = 0.f;
            if (live == R) {
#pragma unroll
                for (int i = 0; i < R; ++i) s += v[i].get(j);
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i) s += i < live ? v[i].get(j) : 0.f;
            }
            const float cm = s * inv;
            if (live == R) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float d = v[i].get(j) - cm;
                    q += d * d;
                }
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float d = i < live ? v[i].get(j) - cm : 0.f;
                    q += d * d;
                }
            }
            const float d = cm - mean[j];
            mean[j] += d * share;
            m2[j] += q + d * d * wgt;
        }
        n = tot;
    }
};

// Joins a workgroup's statistics by group.  Entries (a vector where it lies in one group, WHOLE,
// else a channel) stand in LDS as [row lane][entry]; a group's are its columns [g wd, (g + 1) wd).
// Waves take the groups in turn; where there are fewer groups than waves, several waves share a
// group's row lanes.  g's mean and M2 end in stat[0][g], stat[1][g] (both for every thread).
template <int VEC, bool WHOLE, int BD>
struct GroupJoin {
    static constexpr int EPV = WHOLE ? 1 : VEC;
    static constexpr int kWaves = BD / 64;
    float mean[BD * EPV], m2[BD * EPV], cnt[BD];
    float part[kWaves];
    float stat[2][kWide];

    template <class F>
    __device__ __forceinline__ void sums(const Shape& p, int wd, F f, float* to) {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, row_len = p.vpt * EPV;
        const int per = p.gs >= kWaves ? 1 : kWaves / p.gs;       // waves of a group
        const int lanes = (p.ty + per - 1) / per;                 // row lanes of a wave
        const int dy = 64 / wd, dc = 64 - dy * wd;
        for (int u = w; u < p.gs * per; u += kWaves) {
            const int g = u % p.gs, y0 = u / p.gs * lanes, y1 = min(y0 + lanes, p.ty);
            int y = y0 + lane / wd, c = lane - lane / wd * wd;
            float s = 0.f;
            while (y < y1) {
                s += f(y, y * row_len + g * wd + c, g);
                y += dy;
                c += dc;
                if (c >= wd) { c -= wd; ++y; }
            }
            s = wave_sum(s);
            if (lane == 0) (per == 1 ? to[g] : part[u]) = s;
        }
        if (per > 1) {
            __syncthreads();
            for (int g = threadIdx.x; g < p.gs; g += BD) {
                float s = 0.f;
                for (int k = 0; k < per; ++k) s += part[k * p.gs + g];
                to[g] = s;
            }
        }
        __syncthreads();
    }

    // width: channels of a group in this slab; total: values of a group behind the entries
    __device__ __forceinline__ void join(const Shape& p, int width, float total, const Stats<VEC>& st, int ty, int tx) {
        const int row_len = p.vpt * EPV, wd = WHOLE ? width / VEC : width;
        if (ty < p.ty) {
            const int at = ty * row_len + tx * EPV;
            if constexpr (WHOLE) {
                float mv = 0.f, qv = 0.f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) mv += st.mean[j];
                mv *= 1.f / VEC;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = st.mean[j] - mv;
                    qv += st.m2[j] + st.n * d * d;
                }
                mean[at] = mv;
                m2[at] = qv;
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    mean[at + j] = st.mean[j];
                    m2[at + j] = st.m2[j];
                }
            }
            if (tx == 0) cnt[ty] = WHOLE ? st.n * VEC : st.n;
        }
        __syncthreads();
        const float inv = 1.f / total;
        sums(p, wd, [&](int y, int at, int) { return cnt[y] * mean[at]; }, stat[0]);
        for (int g = threadIdx.x; g < p.gs; g += BD) stat[0][g] *= inv;
        __syncthreads();
        sums(p, wd, [&](int y, int at, int g) {
            const float d = mean[at] - stat[0][g];
            return m2[at] + cnt[y] * d * d;
        }, stat[1]);
    }
};

// One launch: workgroup (tile, slab, image) keeps its R rows a thread and takes the statistics
// of all tiles in order, so that every workgroup of the slab gets the same ones.
template <int VEC, bool XBF, bool WHOLE, int R, int BD>
__global__ __launch_bounds__(BD) void norm_one_kernel(Shape p) {
    __shared__ GroupJoin<VEC, WHOLE, BD> lds;
    __shared__ Terms terms;
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, tile = blockIdx.y, b = blockIdx.z, rows = (int)a.rows;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int ty = tid / p.vpt, tx = tid - ty * p.vpt, c = c0 + tx * VEC;
    const bool on = ty < p.ty;
    const int64_t x0 = ((int64_t)b * rows) * a.x_stride + c;
    auto live_at = [&](int k) { return min(R, (rows - (k * p.tile_rows + ty) + p.ty - 1) / p.ty); };
    auto load = [&](Vec<VEC, XBF> (&v)[R], int k, int live) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            v[i].load(a.x, x0 + (int64_t)(k * p.tile_rows + ty + min(i, live - 1) * p.ty) * a.x_stride);
    };
    Vec<VEC, XBF> own[R], v[R], next[R];
    int live = on ? live_at(0) : 0;
    if (live > 0) load(v, 0, live);
    terms.load(a, b, c0, width, BD);
    Stats<VEC> st;
    st.clear();
    for (int k = 0; live > 0; ++k) {
        const int live_next = k + 1 < p.tiles ? live_at(k + 1) : 0;
        if (live_next > 0) load(next, k + 1, live_next);
        st.add(v, live);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (k == tile) own[i] = v[i];
            v[i] = next[i];
        }
        live = live_next;
    }
    lds.join(p, p.cg, (float)rows * (float)p.cg, st, ty, tx);
    if (!on) return;
    const float inv = 1.f / ((float)rows * (float)p.cg);
    float mean[VEC], A[VEC], D[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int g = (tx * VEC + j) / p.cg;
        mean[j] = lds.stat[0][g];
        terms.fold(tx * VEC + j, 1.f / sqrtf(lds.stat[1][g] * inv + a.eps), A[j], D[j]);
    }
    const int64_t o0 = ((int64_t)b * rows) * a.out_stride + c;
    by_kind(a.act, a.out_bf16, [&](auto act, auto obf) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = tile * p.tile_rows + ty + i * p.ty;
            if (r < rows) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = activate((own[i].get(j) - mean[j]) * A[j] + D[j], act);
                store_vec<VEC, decltype(obf)::value>(a.out, o0 + (int64_t)r * a.out_stride, y);
            }
        }
    });
}

// Two launches, the first: (mean, M2) of each group (or part of one) of a row tile to
// work[b][group][part * tiles + tile].
template <int VEC, bool XBF, bool WHOLE, int R>
__global__ __launch_bounds__(kSplitThreads) void norm_stats_kernel(Shape p) {
    __shared__ GroupJoin<VEC, WHOLE, kSplitThreads> lds;
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
    const int gw = p.parts == 1 ? p.cg : width;
    lds.join(p, gw, (float)(end - first) * (float)gw, st, ty, tx);
    for (int g = tid; g < p.gs; g += kSplitThreads)
        ((float2*)a.work)[((int64_t)b * a.groups + g0 + g) * p.parts * p.tiles + part * p.tiles + tile] =
            make_float2(lds.stat[0][g], lds.stat[1][g]);
}

// The second: the tiles are taken in the other order, the last ones read being the likeliest
// in the caches.
template <int VEC, bool XBF, int R>
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
    const float total = (float)a.rows * (float)p.cg;
    const float last_rows = (float)(a.rows - (int64_t)(p.tiles - 1) * p.tile_rows);
    for (int g = w; g < p.gs; g += kSplitThreads / 64) {
        const float2* src = (const float2*)a.work + ((int64_t)b * a.groups + g0 + g) * q_all;
        // values behind partial sum q
        auto count = [&](int q) {
            const int pt = p.parts == 1 ? 0 : q / p.tiles, ti = q - pt * p.tiles;
            const int wq = p.parts == 1 ? p.cg : min(p.width, p.cg - pt * p.width);
            return (ti == p.tiles - 1 ? last_rows : (float)p.tile_rows) * (float)wq;
        };
        float s = 0.f;
        for (int q = lane; q < q_all; q += 64) s += count(q) * src[q].x;
        const float mean = wave_sum(s) / total;
        float m2 = 0.f;
        for (int q = lane; q < q_all; q += 64) {
            const float2 u = src[q];
            const float d = u.x - mean;
            m2 += u.y + count(q) * d * d;
        }
        m2 = wave_sum(m2);
        if (lane == 0) {
            stat[0][g] = mean;
            stat[1][g] = 1.f / sqrtf(m2 / total + a.eps);
        }
    }
    __syncthreads();
    if (!on) return;
    float mean[VEC], A[VEC], D[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int g = p.parts == 1 ? (tx * VEC + j) / p.cg : 0;
        mean[j] = stat[0][g];
        terms.fold(tx * VEC + j, stat[1][g], A[j], D[j]);
    }
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
                    store_vec<VEC, decltype(obf)::value>(a.out, o0 + (r + (int64_t)i * p.ty) * a.out_stride, y);
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

constexpr int kOneRows = 32; // rows a thread takes the statistics of in the one launch, at most
constexpr int kChunk = 8;    // rows of a thread's chunk in the statistics,
constexpr int kApply = 4;    // and in the other launch

// The cut of the two launches: about 1024 workgroups, each at least one chunk.
Shape split_plan(const GroupNormArgs& a, int v) {
    Shape p = plan(a, v, 64);
    p.ty = kSplitThreads / p.vpt;
    const int64_t step = (int64_t)p.ty * kChunk;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kMaxTiles, 1024 / std::max<int64_t>(1, a.B * p.slabs)));
    const int64_t per = std::max<int64_t>(1, (a.rows + want * step - 1) / (want * step)) * step;
    p.tile_rows = (int)per;
    p.tiles = (int)((a.rows + per - 1) / per);
    return p;
}

template <int VEC, bool XBF, bool WHOLE>
void split(const GroupNormArgs& a, hipStream_t st) {
    const Shape p = split_plan(a, VEC);
    const dim3 grid((unsigned)p.slabs, (unsigned)p.tiles, (unsigned)a.B);
    hipLaunchKernelGGL((norm_stats_kernel<VEC, XBF, WHOLE, kChunk>), grid, dim3(kSplitThreads), 0, st, p);
    hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF, kApply>), grid, dim3(kSplitThreads), 0, st, p);
}

template <int VEC, bool XBF, bool WHOLE, int R, int BD>
void one(Shape p, hipStream_t st) {
    p.ty = BD / p.vpt;
    p.tile_rows = p.ty * R;
    p.tiles = (int)((p.a.rows + p.tile_rows - 1) / p.tile_rows);
    const dim3 grid((unsigned)p.slabs, (unsigned)p.tiles, (unsigned)p.a.B);
    hipLaunchKernelGGL((norm_one_kernel<VEC, XBF, WHOLE, R, BD>), grid, dim3(BD), 0, st, p);
}

template <int VEC, bool XBF, bool WHOLE>
void run(const GroupNormArgs& a, hipStream_t st) {
    const Shape p = plan(a, VEC, 4 * VEC);
    const int64_t ty = kOneThreads / p.vpt;                  // row lanes of a workgroup
    const int64_t each = (a.rows + ty - 1) / ty;             // rows a thread of one workgroup would take
    if (p.parts > 1 || each > kOneRows) split<VEC, XBF, WHOLE>(a, st);
    else if (p.vpt * a.rows <= 256) one<VEC, XBF, WHOLE, 1, 256>(p, st);
    else if (each <= 1) one<VEC, XBF, WHOLE, 1, kOneThreads>(p, st);
    else one<VEC, XBF, WHOLE, 4, kOneThreads>(p, st);
}

template <int VEC, bool XBF>
void run_vec(const GroupNormArgs& a, hipStream_t st) {
    if (VEC == 1 || (a.C / a.groups) % VEC == 0) run<VEC, XBF, true>(a, st);
    else run<VEC, XBF, VEC == 1>(a, st);
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
