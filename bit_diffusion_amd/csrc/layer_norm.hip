// layer_norm.hip -- what a transformer block does between two linears, in one pass: the branch's
// output through its gate onto the residual stream, and the stream's layer norm with each
// request's scale and shift.
//
// Rows are packed, segment i being request i's.  For a row of segment i, over its C values
//   h    = x + gate_i y                       (to x_out, rounded once)
//   mean = sum h / C,  var = sum (h - mean)^2 / C,  r = 1 / sqrt(var + eps)
//   out  = ((h - mean) r w + b) (1 + scale_i) + shift_i
// with the column's terms folded to (h - mean) r A + D, A = w (1 + scale), D = b (1 + scale) +
// shift.  All of it in fp32 from the unrounded h.
//
// Bound: memory, every row once.  A workgroup owns all columns of its rows, a thread the same
// columns of each, so A, D and gate stay in registers from row to row while the segment does not
// change (as fp32 rows they are three times a bf16 row's bytes, which the caches would else have to
// deliver with every row).  kRows rows go at a time: their loads are in flight together and two
// barriers serve all of them.
#include "common.hpp"
#include "launch.hpp"
#include "segments.hpp"

#include <algorithm>
#include <type_traits>

namespace svdq {
namespace {

constexpr int kCus = 256;    // of the GPU
constexpr int kVec = 4;      // columns of a thread's access where rows are aligned
constexpr int kWaves = 16;   // of the widest workgroup

// The sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kShr + 1>(0.f, v);
    v += dpp<kShr + 2>(0.f, v);
    v += dpp<kShr + 4>(0.f, v);
    v += dpp<kShr + 8>(0.f, v);
    v += dpp<kBcast15, 0xa>(0.f, v);
    v += dpp<kBcast31, 0xc>(0.f, v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// VEC columns at element `at`, as fp32 and back.
template <int VEC>
__device__ __forceinline__ void load(const void* p, int64_t at, bool bf16, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = bf16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
    } else if (bf16) {
        const uint2 u = *(const uint2*)((const uint16_t*)p + at);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xFFFF0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
        const float4 f = *(const float4*)((const float*)p + at);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    }
}

template <int VEC>
__device__ __forceinline__ void store(void* p, int64_t at, bool bf16, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        if (bf16) ((uint16_t*)p)[at] = (uint16_t)f32_to_bf16(v[0]);
        else ((float*)p)[at] = v[0];
    } else if (bf16) {
        *(uint2*)((uint16_t*)p + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
        *(float4*)((float*)p + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// V vectors of VEC columns a thread, kRows rows at a time; `per` rows a workgroup.  The last column
// vector may reach past C only where VEC is 1 (C is a multiple of VEC).
template <int VEC, int V, int kRows, int kThreads, bool XBF, bool YBF, bool OBF>
__global__ __launch_bounds__(kThreads) void layer_norm_kernel(LayerNormArgs a, int per) {
    __shared__ float part[3][kWaves][kRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int C = a.C, T = blockDim.x;
    const float inv = 1.f / (float)C;
    int row = (int)blockIdx.x * per;
    const int stop = min(row + per, (int)a.M);
    while (row < stop) {
        int seg = 0, end = stop;
        if (a.starts != nullptr) {
            seg = find_segment(a.starts, a.n_segments, row);
            const int next = a.starts[seg + 1];     // the row's segment's end, or the first segment's start
            if (seg < 0 || next <= row) {           // rows of no segment
                if (seg + 1 >= a.n_segments) return;
                row = max(next, row + 1);
                continue;
            }
            end = min(next, stop);
        }
        float A[V][VEC], D[V][VEC], gate[V][VEC];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + tid) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) { A[v][j] = 1.f; D[v][j] = 0.f; gate[v][j] = 1.f; }
            if (c < C) {
                const int64_t at = (int64_t)seg * a.mod_stride + c;
                float s[VEC], t[VEC];
                if (a.weight != nullptr) load<VEC>(a.weight, c, true, A[v]);
                if (a.bias != nullptr) load<VEC>(a.bias, c, true, D[v]);
                if (a.mod_gate != nullptr) load<VEC>(a.mod_gate, at, a.mod_bf16, gate[v]);
                if (a.mod_scale != nullptr) {
                    load<VEC>(a.mod_scale, at, a.mod_bf16, s);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) { A[v][j] *= 1.f + s[j]; D[v][j] *= 1.f + s[j]; }
                }
                if (a.mod_shift != nullptr) {
                    load<VEC>(a.mod_shift, at, a.mod_bf16, t);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) D[v][j] += t[j];
                }
            }
        }
        for (; row < end; row += kRows) {
            const int live = min(kRows, end - row);
            float h[kRows][V][VEC];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = (v * T + tid) * VEC;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) h[r][v][j] = 0.f;
                    if (c < C && r < live) load<VEC>(a.x, (row + r) * a.x_stride + c, XBF, h[r][v]);
                }
            if (a.y != nullptr) {
                float y[kRows][V][VEC];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int c = (v * T + tid) * VEC;
#pragma unroll
                        for (int j = 0; j < VEC; ++j) y[r][v][j] = 0.f;
                        if (c < C && r < live) load<VEC>(a.y, (row + r) * a.y_stride + c, YBF, y[r][v]);
                    }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) h[r][v][j] = fmaf(gate[v][j], y[r][v][j], h[r][v][j]);
            }
            if (a.x_out != nullptr) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int c = (v * T + tid) * VEC;
                        if (c < C && r < live) store<VEC>(a.x_out, (row + r) * a.x_out_stride + c, XBF, h[r][v]);
                    }
            }
            // the sum over the workgroup of each row's f, through part[at]
            auto sum = [&](int at, const float (&s)[kRows]) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float w = wave_sum(s[r]);
                    if (lane == 0) part[at][wave][r] = w;
                }
            };
            auto total = [&](int at, float (&s)[kRows]) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) s[r] = part[at][0][r];
                for (int w = 1; w < waves; ++w)
#pragma unroll
                    for (int r = 0; r < kRows; ++r) s[r] += part[at][w][r];
            };
            float m[kRows], q[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                m[r] = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) m[r] += h[r][v][j];
            }
            sum(0, m);
            __syncthreads();
            total(0, m);
            // about that mean, the squares and what its rounding left.  Equal values differ from it by
            // a few ulp, all the same: their sum is exact, its C-th part (divided, not multiplied) too
            float e[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                m[r] /= (float)C;   // a product would be contracted into h - m and never be rounded
                q[r] = e[r] = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool in = (v * T + tid) * VEC < C;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        h[r][v][j] = in ? h[r][v][j] - m[r] : 0.f;
                        e[r] += h[r][v][j];
                        q[r] = fmaf(h[r][v][j], h[r][v][j], q[r]);
                    }
                }
            }
            sum(1, e);
            sum(2, q);
            __syncthreads();
            total(1, e);
            total(2, q);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float off = e[r] / (float)C;
                const float var = fmaxf(fmaf(-off, off, q[r] * inv), 0.f);
                const float rstd = __builtin_amdgcn_rsqf(var + a.eps);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = (v * T + tid) * VEC;
                    float z[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) z[j] = fmaf((h[r][v][j] - off) * rstd, A[v][j], D[v][j]);
                    if (c < C && r < live) store<VEC>(a.out, (row + r) * a.out_stride + c, OBF, z);
                }
            }
        }
        row = end;
    }
}

template <int VEC, int V, int kRows, int kThreads>
void launch(const LayerNormArgs& a, int threads, hipStream_t st) {
    // a few workgroups a CU, each with whole sets of kRows rows
    const int64_t want = (a.M + 4 * kCus - 1) / (4 * kCus);
    const int per = (int)(want <= 1 ? 1 : (want + kRows - 1) / kRows * kRows);
    const dim3 grid((unsigned)((a.M + per - 1) / per)), block(threads);
    auto go = [&](auto xb, auto yb, auto ob) {
        hipLaunchKernelGGL((layer_norm_kernel<VEC, V, kRows, kThreads, xb.value, yb.value, ob.value>), grid, block, 0, st, a, per);
    };
    auto with_out = [&](auto xb, auto yb) { a.out_bf16 ? go(xb, yb, std::true_type{}) : go(xb, yb, std::false_type{}); };
    auto with_y = [&](auto xb) { a.y_bf16 ? with_out(xb, std::true_type{}) : with_out(xb, std::false_type{}); };
    a.x_bf16 ? with_y(std::true_type{}) : with_y(std::false_type{});
}

}  // namespace

void launch_layer_norm(const LayerNormArgs& a, hipStream_t st) {
    const int n = a.vec ? (a.C + kVec - 1) / kVec : a.C;   // column vectors of a row
    // vectors a thread so that a row's threads fit a workgroup: 256 of them, and for wide rows the
    // most that leave each its registers
    const int V = n <= 64 ? 1 : n <= 512 ? 2 : n <= 1024 ? 4 : 8;
    const int threads = ((n + V - 1) / V + 63) / 64 * 64;
    if (a.vec) {
        if (V == 1) launch<kVec, 1, 4, 64>(a, threads, st);
        else if (V == 2) launch<kVec, 2, 4, 256>(a, threads, st);
        else if (V == 4) launch<kVec, 4, 4, 256>(a, threads, st);
        else launch<kVec, 8, 1, 512>(a, threads, st);
    } else {
        if (V == 1) launch<1, 1, 4, 64>(a, threads, st);
        else if (V == 2) launch<1, 2, 4, 256>(a, threads, st);
        else if (V == 4) launch<1, 4, 4, 256>(a, threads, st);
        else launch<1, 8, 2, 1024>(a, threads, st);
    }
}

}  // namespace svdq
