// lora_batch.hip -- low-rank adapters of many requests beside one shared projection.
//
// The rows of a batch are cut into segments (one per request); segment i uses adapter
// s = seg_adapter[i] of a pool, or none:
//   out[m, n] = act(base[m, n] + sum_{j < rank_s} t[m, j] B_s[n, j]),
//   t[m, j]   = alpha_s sum_k x[m, k] A_s[j, k].
// Two launches: the down-projection writes t in fp32 to the workspace, the up-projection
// adds to base.  Both are bound by memory (x once; base and out once): 2 R flops per byte
// of x, R / 2 per byte of bf16 base and out.
//
// Tiles.  A workgroup owns rows of one segment only, so its adapter is uniform.  The
// offsets live in device memory (a captured graph replays with other offsets), so the grid
// is the most tiles any cut of M rows into n segments can need, and each workgroup finds its
// tile by a prefix sum of the segments' tile counts, 64 segments per step in one wave.
//
// t keeps fp32 accuracy through the bf16 MFMA: it is split into bf16 terms h = bf16(t),
// m = bf16(t - h), l = bf16(t - h - m) which multiply the same operand.  Two terms
// (off by 2^-16 of t at most) stand far below the half step 2^-8 of a bf16 output; a fp32
// output takes three (2^-24, fp32's own half step).
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace svdq {
namespace {

constexpr int kColTile = 256;    // output columns of a workgroup of the up-projection

struct Tile {
    int seg;    // segment index
    int row0;   // first row
    int rows;   // rows of the tile, 1 to the tile height; 0: no tile
};

// Tile `want` of the segments' tiles of `tm` rows, in order.  Offsets are clamped to [0, M]
// and a segment whose end lies before its start is empty, so that no offset reaches memory
// outside the rows.  Every lane of the wave calls it and gets the same answer.
__device__ __forceinline__ Tile find_tile(const int* __restrict__ starts, int n, int M, int tm,
                                          int want) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int c = 0; c < n; c += 64) {
        const int i = c + lane;
        int a = 0, len = 0;
        if (i < n) {
            a = min(max(starts[i], 0), M);
            len = max(min(max(starts[i + 1], 0), M) - a, 0);
        }
        const int nt = (len + tm - 1) / tm;
        int sum = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d, 64);
            if (lane >= d) sum += o;
        }
        const unsigned long long past = __ballot(before + sum > want);
        if (past != 0) {
            const int src = __ffsll(past) - 1;
            const int first = before + __shfl(sum - nt, src, 64);
            const int off = (want - first) * tm;
            return Tile{c + src, __shfl(a, src, 64) + off, min(tm, __shfl(len, src, 64) - off)};
        }
        before += __shfl(sum, 63, 64);
    }
    return Tile{0, 0, 0};
}

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// Adapter of a segment and its rank; -1 for none (and for an index outside the pool).
__device__ __forceinline__ int adapter_of(const LoraBatchArgs& a, int seg, int& rank) {
    const int s = a.ids[seg];
    if (s < 0 || s >= a.n_adapters) { rank = 0; return -1; }
    rank = a.ranks == nullptr ? a.R : min(max(a.ranks[s], 0), a.R);
    return rank == 0 ? -1 : s;
}

// Down-projection of one tile of 16 RBM rows: the W waves take the 64-channel steps of K in
// turn, each with the whole tile's accumulators, and their sums are added in wave order.
// With gridDim.y > 1 the steps are dealt over that many workgroups too and each writes its
// own partial t (the up-projection adds them in order).  A lane's 32 bytes of a step are
// contiguous (channels 16 q to 16 q + 15 of the step; both operands take the same order, and
// the sum does not mind), so four lanes cover a row's 128 bytes.
// RB: rank blocks of 16 in registers.  Blocks past the adapter's rank repeat its last one
// and are not stored.
template <int RBM, int RB, int W>
__global__ __launch_bounds__(W * 64) void lora_down_kernel(LoraBatchArgs a) {
    __shared__ f32x4 red[W][RBM * RB][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, r16 = lane & 15;
    const Tile t = find_tile(a.starts, a.n_segments, (int)a.M, RBM * 16, (int)blockIdx.x);
    if (t.rows == 0) return;
    int rank;
    const int s = adapter_of(a, t.seg, rank);
    if (s < 0) return;
    const int nrb = (rank + 15) >> 4;
    const int K = a.K, steps = K >> 6;

    const uint16_t* xp[RBM];
#pragma unroll
    for (int i = 0; i < RBM; ++i)
        xp[i] = (const uint16_t*)a.x + (int64_t)(t.row0 + min(i * 16 + r16, t.rows - 1)) * a.x_stride + q * 16;
    const uint16_t* dp[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j)
        dp[j] = (const uint16_t*)a.down + ((int64_t)s * a.R + min(j, nrb - 1) * 16 + r16) * K + q * 16;

    f32x4 acc[RBM][RB];
#pragma unroll
    for (int i = 0; i < RBM; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int workers = W * gridDim.y;
    for (int st = blockIdx.y * W + w; st < steps; st += workers) {
        const int k = st * 64;
        uint4 xv[RBM][2], dv[RB][2];
#pragma unroll
        for (int i = 0; i < RBM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[i][h] = *(const uint4*)(xp[i] + k + h * 8);
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) dv[j][h] = *(const uint4*)(dp[j] + k + h * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < RBM; ++i)
#pragma unroll
                for (int j = 0; j < RB; ++j) acc[i][j] = mfma16(dv[j][h], xv[i][h], acc[i][j]);
    }
    // D: lane (q, r16) holds ranks 4 q to 4 q + 3 of row r16
#pragma unroll
    for (int i = 0; i < RBM; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j) red[w][i * RB + j][lane] = acc[i][j];
    __syncthreads();
    float* out = a.work + (int64_t)blockIdx.y * a.M * a.R;
    for (int b = w; b < RBM * RB; b += W) {
        f32x4 v = red[0][b][lane];
#pragma unroll
        for (int o = 1; o < W; ++o) v += red[o][b][lane];
        const int row = b / RB * 16 + r16, rb = b % RB;
        if (row < t.rows && rb < nrb)
            *(f32x4*)(out + (int64_t)(t.row0 + row) * a.R + rb * 16 + q * 4) = v;
    }
}

// The words of 8 consecutive bf16 with elements at and past `live` cleared.
__device__ __forceinline__ uint4 keep_first(uint4 v, int live) {
    if (live >= 8) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = live >= 2 * i + 2 ? w[i] : live == 2 * i + 1 ? (w[i] & 0xFFFFu) : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// bf16 terms of v: the first is v rounded (to the largest finite value where rounding would
// overflow), the next ones the rests; an infinity or NaN stands in the first term alone.
template <int NT>
__device__ __forceinline__ void split_terms(float v, uint32_t (&t)[NT]) {
    uint32_t h = f32_to_bf16(v);
    const bool finite = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
    if (finite && (h & 0x7FFFu) == 0x7F80u) h -= 1;
    t[0] = h;
    float rest = v - bf16_to_f32(h);
#pragma unroll
    for (int i = 1; i < NT; ++i) {
        t[i] = finite ? f32_to_bf16(rest) : 0u;
        rest -= bf16_to_f32(t[i]);
    }
}

// Up-projection of a tile of 16 RBE rows x 256 columns, 64 columns to a wave, with the
// adapter's B as the MFMA's row operand, so that a lane ends with consecutive columns of one
// row: B's rows are dealt so that 16-byte pieces of base and out are loaded and stored, four
// lanes covering 64 contiguous bytes of a row.
template <int RBE, bool BF16>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraBatchArgs a) {
    constexpr int NT = BF16 ? 2 : 3;
    extern __shared__ uint4 terms[];   // [NT][kb][RBE][64] operands
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, r16 = lane & 15;
    const Tile t = find_tile(a.starts, a.n_segments, (int)a.M, RBE * 16, (int)blockIdx.x);
    if (t.rows == 0) return;
    int rank;
    const int s = adapter_of(a, t.seg, rank);
    if (s < 0 && a.act == 0 && a.base == a.out && a.base_stride == a.out_stride) return;
    const int nkb = (rank + 31) >> 5;

    if (s >= 0) {
        const float alpha = a.alphas[s];
        const int octets = nkb * 4;
        for (int idx = threadIdx.x; idx < RBE * 16 * octets; idx += 256) {
            const int r = idx / octets, o = idx - r * octets;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (r < t.rows && o * 8 < rank) {
                const float* p = a.work + (int64_t)(t.row0 + r) * a.R + o * 8;
                for (int ks = 0; ks < a.splits; ++ks, p += a.M * a.R) {
                    const f32x4 lo = *(const f32x4*)p, hi = *(const f32x4*)(p + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { v[e] += lo[e]; v[4 + e] += hi[e]; }
                }
            }
            uint32_t wd[NT][4];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t tv[NT];
                split_terms<NT>(o * 8 + e < rank ? alpha * v[e] : 0.f, tv);
#pragma unroll
                for (int i = 0; i < NT; ++i) wd[i][e >> 1] = (e & 1) ? wd[i][e >> 1] | (tv[i] << 16) : tv[i];
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
                terms[((i * nkb + (o >> 2)) * RBE + (r >> 4)) * 64 + (o & 3) * 16 + (r & 15)] =
                    make_uint4(wd[i][0], wd[i][1], wd[i][2], wd[i][3]);
        }
    }
    __syncthreads();

    const int c0 = blockIdx.y * kColTile + w * 64;
    if (c0 >= a.N) return;
    f32x4 acc[RBE][4];
#pragma unroll
    for (int i = 0; i < RBE; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (s >= 0) {
        const uint16_t* up[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int col = c0 + (BF16 ? (c >> 1) * 32 + (r16 >> 2) * 8 + (c & 1) * 4 + (r16 & 3) : c * 16 + r16);
            up[c] = (const uint16_t*)a.up + ((int64_t)s * a.N + min(col, a.N - 1)) * a.R;
        }
        for (int kb = 0; kb < nkb; ++kb) {
            const int k = kb * 32 + q * 8;
            uint4 bv[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                bv[c] = k < rank ? keep_first(*(const uint4*)(up[c] + k), rank - k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RBE; ++i)
                if (i * 16 < t.rows) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 tv = terms[((n * nkb + kb) * RBE + i) * 64 + lane];
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[i][c] = mfma16(bv[c], tv, acc[i][c]);
                    }
                }
        }
    }

#pragma unroll
    for (int i = 0; i < RBE; ++i) {
        const int row = i * 16 + r16;
        if (row >= t.rows) continue;
        const int64_t m = t.row0 + row;
        if constexpr (BF16) {
            const uint16_t* bp = a.base == nullptr ? nullptr : (const uint16_t*)a.base + m * a.base_stride;
            uint16_t* op = (uint16_t*)a.out + m * a.out_stride;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = c0 + h * 32 + q * 8;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = acc[i][2 * h + (e >> 2)][e & 3];
                if (a.vec && c + 8 <= a.N) {
                    if (bp != nullptr) {
                        const uint4 b = *(const uint4*)(bp + c);
                        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] += bf16_to_f32((bw[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
                    }
                    uint32_t ow[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ow[e] = f32_to_bf16(activate(y[2 * e], a.act)) | (f32_to_bf16(activate(y[2 * e + 1], a.act)) << 16);
                    *(uint4*)(op + c) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < a.N) {
                            const float b = bp != nullptr ? bf16_to_f32(bp[c + e]) : 0.f;
                            op[c + e] = (uint16_t)f32_to_bf16(activate(y[e] + b, a.act));
                        }
                }
            }
        } else {
            const float* bp = a.base == nullptr ? nullptr : (const float*)a.base + m * a.base_stride;
            float* op = (float*)a.out + m * a.out_stride;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int c = c0 + h * 16 + q * 4;
                f32x4 y = acc[i][h];
                if (a.vec && c + 4 <= a.N) {
                    if (bp != nullptr) y += *(const f32x4*)(bp + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = activate(y[e], a.act);
                    *(f32x4*)(op + c) = y;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.N) op[c + e] = activate(y[e] + (bp != nullptr ? bp[c + e] : 0.f), a.act);
                }
            }
        }
    }
}

// Most tiles of `tm` rows that n segments of M rows can need.
int64_t most_tiles(int64_t M, int n, int tm) { return std::min<int64_t>((M + (int64_t)n * (tm - 1)) / tm, M); }

int down_row_blocks(int64_t M) { return M >= 8192 ? 2 : 1; }

template <int RBM, int RB>
void down(const LoraBatchArgs& a, hipStream_t st) {
    constexpr int W = RBM * RB * 8 <= 64 ? 8 : 4;   // partial sums of W waves: 64 KB of LDS at most
    const dim3 grid((unsigned)most_tiles(a.M, a.n_segments, RBM * 16), (unsigned)a.splits);
    hipLaunchKernelGGL((lora_down_kernel<RBM, RB, W>), grid, dim3(W * 64), 0, st, a);
}

template <int RBM>
void down_rank(const LoraBatchArgs& a, hipStream_t st) {
    if (a.R <= 16) down<RBM, 1>(a, st);
    else if (a.R <= 32) down<RBM, 2>(a, st);
    else if (a.R <= 64) down<RBM, 4>(a, st);
    else down<RBM, 8>(a, st);
}

template <int RBE, bool BF16>
void up(const LoraBatchArgs& a, hipStream_t st) {
    const size_t lds = (size_t)(BF16 ? 2 : 3) * ((a.R + 31) / 32) * RBE * 64 * 16;
    const dim3 grid((unsigned)most_tiles(a.M, a.n_segments, RBE * 16), (unsigned)((a.N + kColTile - 1) / kColTile));
    hipLaunchKernelGGL((lora_up_kernel<RBE, BF16>), grid, dim3(256), lds, st, a);
}

}  // namespace

int lora_batch_splits(int64_t M, int K, int n_segments) {
    const int64_t tiles = most_tiles(M, n_segments, down_row_blocks(M) * 16);
    const int64_t want = (512 + tiles - 1) / tiles;
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, 8, K / 64 / 8}));
}

int64_t lora_batch_workspace_bytes(int64_t M, int K, int R, int n_segments) {
    if (M == 0 || n_segments == 0) return 0;
    return (int64_t)lora_batch_splits(M, K, n_segments) * M * R * 4;
}

void launch_lora_batch(const LoraBatchArgs& args, hipStream_t st) {
    LoraBatchArgs a = args;
    a.splits = lora_batch_splits(a.M, a.K, a.n_segments);
    if (down_row_blocks(a.M) == 2) down_rank<2>(a, st);
    else down_rank<1>(a, st);
    const bool tall = (a.M / 64) * ((a.N + kColTile - 1) / kColTile) >= 512;
    if (a.bf16) tall ? up<4, true>(a, st) : up<1, true>(a, st);
    else tall ? up<4, false>(a, st) : up<1, false>(a, st);
}

}  // namespace svdq
