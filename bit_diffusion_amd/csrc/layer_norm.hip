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
// deliver with every row).  A row at a time, the next one's loads in flight, and several workgroups a
// CU that wait at different barriers: four rows at a time, with one pair of barriers for all, held
// four times the registers and took 85 us where this takes 27 (4608 x 3072 bf16 with residual).
#include "common.hpp"
#include "launch.hpp"
#include "segments.hpp"

#include <algorithm>
#include <type_traits>

namespace svdq {
namespace {

constexpr int kCus = 256;    // of the GPU
constexpr int kWaves = 16;   // of the widest workgroup
// A CU's share of the rows goes over as many workgroups as read kFlight bytes at a time, up to kWavesCu waves
// of them, three quarters of that where x is fp32 (us, waves 18, 24 and 30; bf16: 4096 x 1152 12.1, 11.5, 11.4;
// 4608 x 3072 27.1, 27.5, 26.4; 9216 x 3072 52.7, 51.5, 53.5, without y 36.2, 32.6, 41.3; fp32 4608 x 3072 without
// y 20.9, 25.0, 25.4).
constexpr int kFlight = 57344, kWavesCu = 24;

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

// A barrier that waits for this wave's LDS accesses only: loads of the next row and stores of this
// one stay in flight (__syncthreads would wait for them).
__device__ __forceinline__ void sync() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// VEC columns at element `at`: as loaded, and as fp32.
template <int VEC, bool BF16>
struct Raw {
    uint32_t u[BF16 ? (VEC + 1) / 2 : VEC];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& w : u) w = 0;
    }
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (VEC == 1) {
            u[0] = BF16 ? ((const uint16_t*)p)[at] : ((const uint32_t*)p)[at];
        } else if constexpr (BF16 && VEC == 2) {
            u[0] = *(const uint32_t*)((const uint16_t*)p + at);
        } else if constexpr (BF16 || VEC == 2) {
            const uint2 w = *(const uint2*)((const char*)p + at * (BF16 ? 2 : 4));
            u[0] = w.x; u[1] = w.y;
        } else {
            const uint4 w = *(const uint4*)((const uint32_t*)p + at);
            u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (!BF16) return __uint_as_float(u[j]);
        else return __uint_as_float((j & 1) ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16);
    }
};

template <int VEC>
__device__ __forceinline__ void load(const void* p, int64_t at, bool bf16, float (&v)[VEC]) {
    Raw<VEC, true> b;
    Raw<VEC, false> f;
    if (bf16) b.load(p, at);
    else f.load(p, at);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = bf16 ? b.get(j) : f.get(j);
}

// To memory, past the caches where STREAM.
template <bool STREAM, class T>
__device__ __forceinline__ void put(T v, void* p) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, (T*)p);
    else *(T*)p = v;
}

template <bool STREAM, int VEC>
__device__ __forceinline__ void store(void* p, int64_t at, bool bf16, const float (&v)[VEC]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    char* to = (char*)p + at * (bf16 ? 2 : 4);
    if constexpr (VEC == 1) {
        if (bf16) put<STREAM>((uint16_t)pack_bf16(v[0], 0.f), to);
        else put<STREAM>(v[0], to);
    } else if constexpr (VEC == 2) {
        if (bf16) put<STREAM>(pack_bf16(v[0], v[1]), to);
        else put<STREAM>(f32x2{v[0], v[1]}, to);
    } else {
        if (bf16) put<STREAM>(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, to);
        else put<STREAM>(f32x4{v[0], v[1], v[2], v[3]}, to);
    }
}

// V vectors of VEC columns a thread; `per` rows a workgroup.  C is a multiple of VEC.  The next row is
// loaded while this one is normalised, but in the widest rows, which have no registers left for it.
template <int VEC, int V, int kThreads, bool XBF, bool YBF, bool OBF>
__global__ __launch_bounds__(kThreads) void layer_norm_kernel(LayerNormArgs a, int per) {
    __shared__ float part[3][kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int C = a.C, T = blockDim.x;
    const float c_count = (float)C;
    constexpr bool kAhead = V < 8;
    int row = (int)blockIdx.x * per;
    const int stop = min(row + per, (int)a.M);
    Raw<VEC, XBF> x[V];
    Raw<VEC, YBF> y[V];
    auto fetch = [&](int r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + tid) * VEC;
            x[v].clear();
            y[v].clear();
            if (c < C) {
                x[v].load(a.x, r * a.x_stride + c);
                if (a.y != nullptr) y[v].load(a.y, r * a.y_stride + c);
            }
        }
    };
    while (row < stop) {
        if (kAhead) fetch(row);  // what comes up to its use need not wait for it
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
        for (; row < end; ++row) {
            if (!kAhead) fetch(row);
            float h[V][VEC], m = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    h[v][j] = a.y != nullptr ? fmaf(gate[v][j], y[v].get(j), x[v].get(j)) : x[v].get(j);
                    m += h[v][j];
                }
            if (kAhead && row + 1 < end) fetch(row + 1);
            // the stream is read again only behind the next linears: kept out of the caches, it leaves them
            // to what the next one reads (bf16 rows of 3072, through the caches and so, us; alone: 4608 rows 27.4
            // and 26.6, 9216 rows 50.0 and 49.9; with svdq_quantize_act_packed behind: 1024 rows 21.9 and 20.4, 4608
            // rows 51.1 and 51.4, 9216 rows 79.6 and 77.7)
            if (a.x_out != nullptr) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = (v * T + tid) * VEC;
                    if (c < C) store<true>(a.x_out, row * a.x_out_stride + c, XBF, h[v]);
                }
            }
            // the workgroup's sum of every wave's f, through part[at]
            auto put = [&](int at, float f) {
                f = wave_sum(f);
                if (lane == 0) part[at][wave] = f;
            };
            auto total = [&](int at) {
                float f = part[at][0];
                for (int w = 1; w < waves; ++w) f += part[at][w];
                return f;
            };
            put(0, m);
            sync();
            m = total(0) / c_count;   // a product would be contracted into h - m and never be rounded
            // about that mean, the squares and what its rounding left.  Equal values differ from it by
            // a few ulp, all the same: their sum is exact, its C-th part (divided, not multiplied) too
            float e = 0.f, q = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = (v * T + tid) * VEC < C;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    h[v][j] = in ? h[v][j] - m : 0.f;
                    e += h[v][j];
                    q = fmaf(h[v][j], h[v][j], q);
                }
            }
            put(1, e);
            put(2, q);
            sync();
            const float off = total(1) / c_count;
            const float var = fmaxf(fmaf(-off, off, total(2) / c_count), 0.f);
            const float rstd = rsqrt_hw(var + a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (v * T + tid) * VEC;
                float z[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) z[j] = fmaf((h[v][j] - off) * rstd, A[v][j], D[v][j]);
                if (c < C) store<false>(a.out, row * a.out_stride + c, OBF, z);
            }
        }
    }
}

template <int VEC, int V, int kThreads>
void launch(const LayerNormArgs& a, int threads, hipStream_t st) {
    const int waves = threads / 64, row = a.C * ((a.x_bf16 ? 2 : 4) + (a.y == nullptr ? 0 : a.y_bf16 ? 2 : 4));
    const int64_t most = kCus * std::max(1, std::min((kFlight + row / 2) / row, (a.x_bf16 ? kWavesCu : kWavesCu * 3 / 4) / waves));
    // narrow rows have a workgroup each where the GPU holds them all (1238 x 1170, fp32 x: 9.7 -> 8.6 us; of 9 KB
    // and more not: 1300 x 3072 11.4 -> 12.7; nor element by element: 1238 x 1171 10.0 -> 11.2)
    const bool at_once = VEC > 1 && row <= 8192 && a.M * waves <= kCus * 32;
    const int per = at_once ? 1 : (int)((a.M + most - 1) / most);
    const dim3 grid((unsigned)((a.M + per - 1) / per)), block(threads);
    auto go = [&](auto xb, auto yb, auto ob) {
        hipLaunchKernelGGL((layer_norm_kernel<VEC, V, kThreads, xb.value, yb.value, ob.value>), grid, block, 0, st, a, per);
    };
    auto with_out = [&](auto xb, auto yb) { a.out_bf16 ? go(xb, yb, std::true_type{}) : go(xb, yb, std::false_type{}); };
    auto with_y = [&](auto xb) { a.y_bf16 ? with_out(xb, std::true_type{}) : with_out(xb, std::false_type{}); };
    a.x_bf16 ? with_y(std::true_type{}) : with_y(std::false_type{});
}

}  // namespace

void launch_layer_norm(const LayerNormArgs& a, hipStream_t st) {
    const int n = a.C / a.vec;   // column vectors of a row
    // two vectors a thread up to 1024 (4608 rows of 768 vectors: 26.9 us, with one 40, with four 30),
    // then as many as leave a row's threads in a workgroup their registers
    const int V = n <= 64 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : 8;
    const int threads = ((n + V - 1) / V + 63) / 64 * 64;
    auto go = [&](auto vec) {
        if (V == 1) launch<vec.value, 1, 64>(a, threads, st);
        else if (V == 2) launch<vec.value, 2, 512>(a, threads, st);
        else if (V == 4) launch<vec.value, 4, 512>(a, threads, st);
        else launch<vec.value, 8, vec.value == 1 ? 1024 : 512>(a, threads, st);
    };
    if (a.vec == 4) go(std::integral_constant<int, 4>{});
    else if (a.vec == 2) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1>{});
}

}  // namespace svdq
