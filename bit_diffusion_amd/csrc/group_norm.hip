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
//   resident: an image's slab fits the registers of one workgroup: one launch, x read once,
//             mean, then squares about it, from the registers.
//   split:    otherwise two launches.  The first takes chunks of 8 rows per thread, two passes
//             over each in registers, and joins them as (count, mean, sum of squares about the
//             mean): for two sets the joined M2 is M2a + M2b + d^2 na nb / (na + nb), d the
//             difference of the means.  The second joins the row tiles' partial sums (every
//             workgroup for its own groups, in a fixed order) and normalises.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>
#include <numeric>

namespace svdq {
namespace {

constexpr int kRows = 8;          // rows of a chunk
constexpr int kSplitThreads = 256;
constexpr int kResidentThreads = 1024;
constexpr int kMaxTiles = 256;    // row tiles of an image
constexpr int kWide8 = 512;       // widest slab in 8-channel vectors, and in single channels
constexpr int kWide1 = 64;

struct Shape {
    GroupNormArgs a;
    int cg;        // channels of a group
    int width;     // channels of a slab (the last part of a wide group may be narrower)
    int gs;        // groups of a slab (1 where a group is cut into parts)
    int parts;     // slabs of one group (1: a slab is whole groups)
    int slabs;     // slabs of an image
    int vpt;       // vectors of a slab
    int ty;        // row lanes of a workgroup
    int tiles;     // row tiles of an image (split)
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

// VEC consecutive channels of one position, as loaded.
template <int VEC, bool BF16>
struct Vec {
    static constexpr int kWords = BF16 ? (VEC + 1) / 2 : VEC;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        if constexpr (BF16) {
            const uint16_t* p = (const uint16_t*)base + at;
            if constexpr (VEC == 8) put4(0, *(const uint4*)p);
            else w[0] = p[0];
        } else {
            const uint32_t* p = (const uint32_t*)base + at;
            if constexpr (VEC == 8) {
                put4(0, *(const uint4*)p);
                put4(4, *(const uint4*)(p + 4));
            } else {
                w[0] = p[0];
            }
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (BF16) return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        else return __uint_as_float(w[j]);
    }

private:
    __device__ __forceinline__ void put4(int at, uint4 u) {
        w[at] = u.x; w[at + 1] = u.y; w[at + 2] = u.z; w[at + 3] = u.w;
    }
};

template <int VEC>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&y)[VEC], int bf16) {
    if (bf16) {
        uint16_t* p = (uint16_t*)base + at;
        if constexpr (VEC == 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(y[2 * i]) | (f32_to_bf16(y[2 * i + 1]) << 16);
            *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            p[0] = (uint16_t)f32_to_bf16(y[0]);
        }
    } else {
        float* p = (float*)base + at;
        if constexpr (VEC == 8) {
            *(f32x4*)p = f32x4{y[0], y[1], y[2], y[3]};
            *(f32x4*)(p + 4) = f32x4{y[4], y[5], y[6], y[7]};
        } else {
            p[0] = y[0];
        }
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The channel's factor and offset.
__device__ __forceinline__ float load_mod(const void* p, int64_t at, int bf16) {
    return bf16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}

template <int VEC>
__device__ __forceinline__ void channel_terms(const GroupNormArgs& a, int b, int c, float r, float& A, float& D) {
    const float w = a.weight != nullptr ? bf16_to_f32(((const uint16_t*)a.weight)[c]) : 1.f;
    const float bias = a.bias != nullptr ? bf16_to_f32(((const uint16_t*)a.bias)[c]) : 0.f;
    const float ms = a.mod_scale != nullptr ? 1.f + load_mod(a.mod_scale, (int64_t)b * a.mod_stride + c, a.mod_bf16) : 1.f;
    const float mt = a.mod_shift != nullptr ? load_mod(a.mod_shift, (int64_t)b * a.mod_stride + c, a.mod_bf16) : 0.f;
    A = r * w * ms;
    D = bias * ms + mt;
}

// Sums over the entries of group g of an LDS array [ty][vpt * EPV], its columns [g wd, (g + 1) wd).
template <class F>
__device__ __forceinline__ float group_sum(int ty, int row_len, int wd, int g, F f) {
    const int lane = threadIdx.x & 63, n = ty * wd;
    float s = 0.f;
    for (int i = lane; i < n; i += 64) {
        const int y = i / wd, c = g * wd + (i - y * wd);
        s += f(y, y * row_len + c);
    }
    return wave_sum(s);
}

// One workgroup: one image's slab, kept in registers, R rows a thread.
// WHOLE: every 8-channel vector lies in one group (then a vector is one LDS entry, otherwise
// each channel is).
template <int VEC, bool XBF, bool WHOLE, int R, int BD>
__global__ __launch_bounds__(BD) void norm_resident_kernel(Shape p) {
    constexpr int EPV = WHOLE ? 1 : VEC;
    __shared__ float e[BD * EPV];
    __shared__ float stat[2][kWide8];   // mean and 1 / sqrt(var + eps) of each group
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, w = tid >> 6, waves = BD >> 6;
    const int b = blockIdx.y;
    int c0, width, g0, part;
    slab_range(p, blockIdx.x, c0, width, g0, part);
    const int vpt = p.vpt, ty = tid / vpt, tx = tid - ty * vpt;
    const bool on = ty < p.ty;
    const int rows = (int)a.rows;
    const int64_t x0 = ((int64_t)b * rows) * a.x_stride + c0 + tx * VEC;

    Vec<VEC, XBF> v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = ty + i * p.ty;
        if (on && r < rows) v[i].load(a.x, x0 + (int64_t)r * a.x_stride);
    }
    const int row_len = vpt * EPV, wd = WHOLE ? p.cg / VEC : p.cg;
    const float inv = 1.f / ((float)rows * (float)p.cg);
    float s[EPV];
#pragma unroll
    for (int j = 0; j < EPV; ++j) s[j] = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (on && ty + i * p.ty < rows) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[WHOLE ? 0 : j] += v[i].get(j);
        }
    if (on) {
#pragma unroll
        for (int j = 0; j < EPV; ++j) e[ty * row_len + tx * EPV + j] = s[j];
    }
    __syncthreads();
    for (int g = w; g < p.gs; g += waves) {
        const float sum = group_sum(p.ty, row_len, wd, g, [&](int, int at) { return e[at]; });
        if ((tid & 63) == 0) stat[0][g] = sum * inv;
    }
    __syncthreads();
    float mean[EPV];
#pragma unroll
    for (int j = 0; j < EPV; ++j) {
        mean[j] = on ? stat[0][(tx * VEC + j) / p.cg] : 0.f;
        s[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (on && ty + i * p.ty < rows) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = v[i].get(j) - mean[WHOLE ? 0 : j];
                s[WHOLE ? 0 : j] += d * d;
            }
        }
    if (on) {
#pragma unroll
        for (int j = 0; j < EPV; ++j) e[ty * row_len + tx * EPV + j] = s[j];
    }
    __syncthreads();
    for (int g = w; g < p.gs; g += waves) {
        const float sum = group_sum(p.ty, row_len, wd, g, [&](int, int at) { return e[at]; });
        if ((tid & 63) == 0) stat[1][g] = 1.f / sqrtf(sum * inv + a.eps);
    }
    __syncthreads();
    if (!on) return;
    float A[VEC], D[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int c = tx * VEC + j;
        channel_terms<VEC>(a, b, c0 + c, stat[1][c / p.cg], A[j], D[j]);
    }
    const int64_t o0 = ((int64_t)b * rows) * a.out_stride + c0 + tx * VEC;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = ty + i * p.ty;
        if (r < rows) {
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = activate((v[i].get(j) - mean[WHOLE ? 0 : j]) * A[j] + D[j], a.act);
            store_vec<VEC>(a.out, o0 + (int64_t)r * a.out_stride, y, a.out_bf16);
        }
    }
}

// Partial statistics of one row tile of a slab: (mean, M2) of each of its groups (or of its
// part of one) to work[b][group][part * tiles + tile].
template <int VEC, bool XBF, bool WHOLE>
__global__ __launch_bounds__(kSplitThreads) void norm_stats_kernel(Shape p) {
    constexpr int EPV = WHOLE ? 1 : VEC;
    __shared__ float e[2][kSplitThreads * EPV];   // mean, M2
    __shared__ float cnt[kSplitThreads];          // values behind an entry, by row lane
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, w = tid >> 6;
    const int tile = blockIdx.x, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.y, c0, width, g0, part);
    const int vpt = p.vpt, ty = tid / vpt, tx = tid - ty * vpt;
    const bool on = ty < p.ty && tx * VEC < width;
    const int64_t r_end = min((int64_t)(tile + 1) * p.tile_rows, a.rows);
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c0 + tx * VEC;

    float n = 0.f, mean[VEC], m2[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) mean[j] = m2[j] = 0.f;
    if (on) {
        for (int64_t r = (int64_t)tile * p.tile_rows + ty; r < r_end; r += (int64_t)p.ty * kRows) {
            Vec<VEC, XBF> v[kRows];
            const int live = (int)min((int64_t)kRows, (r_end - r + p.ty - 1) / p.ty);
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                v[i].load(a.x, x0 + (r + (int64_t)min(i, live - 1) * p.ty) * a.x_stride);
            const float nc = (float)live, tot = n + nc, wgt = n * nc / tot, share = nc / tot;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float s = 0.f, q = 0.f;
#pragma unroll
                for (int i = 0; i < kRows; ++i) s += i < live ? v[i].get(j) : 0.f;
                const float cm = s / nc;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const float d = i < live ? v[i].get(j) - cm : 0.f;
                    q += d * d;
                }
                const float d = cm - mean[j];
                mean[j] += d * share;
                m2[j] += q + d * d * wgt;
            }
            n = tot;
        }
    }
    const int row_len = vpt * EPV;
    if (ty < p.ty) {
        if constexpr (WHOLE) {
            float mv = 0.f, qv = 0.f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) mv += mean[j];
            mv *= 1.f / VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = mean[j] - mv;
                qv += m2[j] + n * d * d;
            }
            e[0][ty * row_len + tx] = mv;
            e[1][ty * row_len + tx] = qv;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                e[0][ty * row_len + tx * EPV + j] = mean[j];
                e[1][ty * row_len + tx * EPV + j] = m2[j];
            }
        }
        if (tx == 0) cnt[ty] = WHOLE ? n * VEC : n;
    }
    __syncthreads();
    const int wd = (p.parts == 1 ? p.cg : width) / (WHOLE ? VEC : 1);
    const float total = (float)(r_end - (int64_t)tile * p.tile_rows) * (float)(p.parts == 1 ? p.cg : width);
    const int q_all = p.parts * p.tiles;
    for (int g = w; g < p.gs; g += kSplitThreads / 64) {
        const float gm = group_sum(p.ty, row_len, wd, g, [&](int y, int at) { return cnt[y] * e[0][at]; }) / total;
        const float gq = group_sum(p.ty, row_len, wd, g, [&](int y, int at) {
            const float d = e[0][at] - gm;
            return e[1][at] + cnt[y] * d * d;
        });
        if ((tid & 63) == 0)
            ((float2*)a.work)[((int64_t)b * a.groups + g0 + g) * q_all + part * p.tiles + tile] = make_float2(gm, gq);
    }
}

template <int VEC, bool XBF>
__global__ __launch_bounds__(kSplitThreads) void norm_apply_kernel(Shape p) {
    __shared__ float stat[2][kWide8];   // a slab has at most that many groups
    const GroupNormArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int tile = blockIdx.x, b = blockIdx.z;
    int c0, width, g0, part;
    slab_range(p, blockIdx.y, c0, width, g0, part);
    const int vpt = p.vpt, ty = tid / vpt, tx = tid - ty * vpt;
    const int64_t r_end = min((int64_t)(tile + 1) * p.tile_rows, a.rows);
    const int q_all = p.parts * p.tiles;
    const float total = (float)a.rows * (float)p.cg;
    const float last_rows = (float)(a.rows - (int64_t)(p.tiles - 1) * p.tile_rows);
    for (int g = w; g < p.gs; g += kSplitThreads / 64) {
        const float2* src = (const float2*)a.work + ((int64_t)b * a.groups + g0 + g) * q_all;
        // values behind partial sum q
        auto count = [&](int q) {
            const int pt = q / p.tiles, ti = q - pt * p.tiles;
            const int wq = p.parts == 1 ? p.cg : min(p.width, p.cg - pt * p.width);
            return (ti == p.tiles - 1 ? last_rows : (float)p.tile_rows) * (float)wq;
        };
        float s = 0.f;
        for (int q = lane; q < q_all; q += 64) s += count(q) * src[q].x;
        const float mean = wave_sum(s) / total;
        float m2 = 0.f;
        for (int q = lane; q < q_all; q += 64) {
            const float2 v = src[q];
            const float d = v.x - mean;
            m2 += v.y + count(q) * d * d;
        }
        m2 = wave_sum(m2);
        if (lane == 0) {
            stat[0][g] = mean;
            stat[1][g] = 1.f / sqrtf(m2 / total + a.eps);
        }
    }
    __syncthreads();
    if (ty >= p.ty || tx * VEC >= width) return;
    float A[VEC], D[VEC], mean[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int c = tx * VEC + j, g = p.parts == 1 ? c / p.cg : 0;
        mean[j] = stat[0][g];
        channel_terms<VEC>(a, b, c0 + c, stat[1][g], A[j], D[j]);
    }
    const int64_t x0 = ((int64_t)b * a.rows) * a.x_stride + c0 + tx * VEC;
    const int64_t o0 = ((int64_t)b * a.rows) * a.out_stride + c0 + tx * VEC;
    for (int64_t r = (int64_t)tile * p.tile_rows + ty; r < r_end; r += (int64_t)p.ty * kRows) {
        Vec<VEC, XBF> v[kRows];
        const int live = (int)min((int64_t)kRows, (r_end - r + p.ty - 1) / p.ty);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            v[i].load(a.x, x0 + (r + (int64_t)min(i, live - 1) * p.ty) * a.x_stride);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (i < live) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = activate((v[i].get(j) - mean[j]) * A[j] + D[j], a.act);
                store_vec<VEC>(a.out, o0 + (r + (int64_t)i * p.ty) * a.out_stride, y, a.out_bf16);
            }
    }
}

// Whether 8-channel vectors fit the groups: a slab of whole groups and whole vectors is not
// too wide, or a wide group is itself whole vectors.
bool vectors_fit(int C, int cg) { return C % 8 == 0 && (std::lcm((int64_t)cg, (int64_t)8) <= kWide8 || cg % 8 == 0); }

// Cuts the channels into slabs of `v`-channel vectors.
Shape plan(const GroupNormArgs& a, int v) {
    Shape p{};
    p.a = a;
    p.cg = a.C / a.groups;
    const int most = v == 8 ? kWide8 : kWide1;
    const int64_t unit = v == 8 ? std::lcm((int64_t)p.cg, (int64_t)8) : p.cg;
    if (unit <= most) {
        // whole groups: the narrowest even cut of 64 channels or more, else the widest
        const int units = (int)(a.C / unit);
        int m = 1;
        for (int k = 1; k <= units && k * unit <= most; ++k)
            if (units % k == 0 && m * unit < 64) m = k;
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

// Row tiles of the split form: about 1024 workgroups, each at least one chunk.
void plan_tiles(Shape& p) {
    p.ty = kSplitThreads / p.vpt;
    const int64_t step = (int64_t)p.ty * kRows;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kMaxTiles, 1024 / std::max<int64_t>(1, p.a.B * p.slabs)));
    const int64_t per = std::max<int64_t>(1, (p.a.rows + want * step - 1) / (want * step)) * step;
    p.tile_rows = (int)per;
    p.tiles = (int)((p.a.rows + per - 1) / per);
}

template <int VEC, bool XBF, bool WHOLE>
void split(Shape p, hipStream_t st) {
    plan_tiles(p);
    const dim3 grid((unsigned)p.tiles, (unsigned)p.slabs, (unsigned)p.a.B);
    hipLaunchKernelGGL((norm_stats_kernel<VEC, XBF, WHOLE>), grid, dim3(kSplitThreads), 0, st, p);
    hipLaunchKernelGGL((norm_apply_kernel<VEC, XBF>), grid, dim3(kSplitThreads), 0, st, p);
}

template <int VEC, bool XBF, bool WHOLE, int R>
void resident(Shape p, hipStream_t st) {
    p.ty = kResidentThreads / p.vpt;
    const dim3 grid((unsigned)p.slabs, (unsigned)p.a.B);
    hipLaunchKernelGGL((norm_resident_kernel<VEC, XBF, WHOLE, R, kResidentThreads>), grid, dim3(kResidentThreads), 0, st, p);
}

template <int VEC, bool XBF, bool WHOLE>
void run(const Shape& p, hipStream_t st) {
    // rows a thread would hold; 16 of bf16 or 8 of fp32 take 64 of its 128 registers
    const int64_t ty = kResidentThreads / p.vpt, each = (p.a.rows + ty - 1) / ty;
    if (p.parts > 1 || each > (XBF ? 16 : 8)) split<VEC, XBF, WHOLE>(p, st);
    else if (each <= 1) resident<VEC, XBF, WHOLE, 1>(p, st);
    else if (each <= 4) resident<VEC, XBF, WHOLE, 4>(p, st);
    else if (each <= 8) resident<VEC, XBF, WHOLE, 8>(p, st);
    else if constexpr (XBF) resident<VEC, XBF, WHOLE, 16>(p, st);
}

template <int VEC, bool XBF>
void run_vec(const Shape& p, hipStream_t st) {
    if (VEC == 1 || p.cg % VEC == 0) run<VEC, XBF, true>(p, st);
    else run<VEC, XBF, VEC == 1>(p, st);
}

}  // namespace

int64_t group_norm_workspace_bytes(int64_t B, int64_t rows, int C, int groups) {
    // either cut may be taken, by the buffers' alignment
    int64_t most = 0;
    for (int v = 1; v <= 8; v += 7) {
        GroupNormArgs a{};
        a.B = B; a.rows = rows; a.C = C; a.groups = groups;
        if (B == 0 || rows == 0 || (v == 8 && !vectors_fit(C, C / groups))) continue;
        Shape p = plan(a, v);
        plan_tiles(p);
        most = std::max(most, B * groups * (int64_t)p.parts * p.tiles * (int64_t)sizeof(float2));
    }
    return most;
}

void launch_group_norm(const GroupNormArgs& a, hipStream_t st) {
    const int v = a.vec && vectors_fit(a.C, a.C / a.groups) ? 8 : 1;
    const Shape p = plan(a, v);
    if (v == 8) a.x_bf16 ? run_vec<8, true>(p, st) : run_vec<8, false>(p, st);
    else a.x_bf16 ? run_vec<1, true>(p, st) : run_vec<1, false>(p, st);
}

}  // namespace svdq
