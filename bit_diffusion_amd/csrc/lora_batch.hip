// lora_batch.hip -- low-rank adapters of many requests beside one shared projection.
//
// The rows of a batch are cut into segments (one per request); segment i uses adapter
// s = seg_adapter[i] of a pool, or none:
//   out[m, n] = act(base[m, n] + sum_{j < rank_s} t[m, j] B_s[n, j]),
//   t[m, j]   = alpha_s sum_k x[m, k] A_s[j, k].
// Both products are bound by memory (x once; base and out once): R flops per byte of x, R / 2 per
// byte of bf16 base and out; past rank 32 LDS, barriers and registers bind first.  Many rows take
// two launches, the down-projection (t to the workspace) and the up-projection (t, base -> out);
// few rows take one, in which every workgroup forms its rows' t itself.
//
// Tiles.  A workgroup owns rows of one segment only, so its adapter is uniform.  The
// offsets live in device memory (a captured graph replays with other offsets), so the grid
// is the most tiles any cut of M rows into n segments can need, and each workgroup finds its
// tile by a prefix sum of the segments' tile counts, 64 segments per step in one wave.
//
// Operands.  In the MFMA's operands neighbouring lanes hold different rows of a row-major
// matrix.  Loaded like that, each 16 bytes of a wave's load are a cache line of their own, and
// the line look-ups, not the bytes, set the time (8 bytes per cycle and CU measured).  So
// every matrix is loaded and stored with neighbouring lanes on neighbouring 16 bytes of a
// row, and turned into operand order, or back, through LDS private to the wave, its 16-byte
// slots exclusive-ored with the row so that neither side meets a bank twice.  t itself is
// kept in operand order in the workspace.
//
// t passes the bf16 MFMA as it is: its 24 significant bits are cut into three bf16 terms of 8
// which multiply the same operand, for a bf16 output too (base and the delta may cancel).
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace svdq {
namespace {

constexpr int kColTile = 256;    // output columns of a workgroup

struct Tile {
    int row0;   // first row
    int rows;   // rows of the tile, 1 to the tile height; 0: no tile
    int id;     // the segment's seg_adapter
    int block;  // the first of its blocks of 16 rows, counted over the segments in order
};

__device__ __forceinline__ int wave_scan(int v) {
    v += dpp<kShr + 1>(0, v);
    v += dpp<kShr + 2>(0, v);
    v += dpp<kShr + 4>(0, v);
    v += dpp<kShr + 8>(0, v);
    v += dpp<kBcast15, 0xa>(0, v);
    v += dpp<kBcast31, 0xc>(0, v);
    return v;
}

// Tile `want` of the segments' tiles of 16 TB rows, in order.  Offsets are clamped to [0, M]
// and a segment whose end lies before its start is empty, so that no offset reaches memory
// outside the rows.  Every lane of the wave calls it and gets the same answer.
template <int TB>
__device__ __forceinline__ Tile find_tile(const LoraBatchArgs& a, int want) {
    const int lane = threadIdx.x & 63, n = a.n_segments, M = (int)a.M;
    int before = 0, blocks = 0;
    for (int c = 0; c < n; c += 64) {
        const int i = c + lane;
        int r0 = 0, len = 0, id = -1;
        if (i < n) {
            id = a.ids[i];
            r0 = min(max(a.starts[i], 0), M);
            len = max(min(max(a.starts[i + 1], 0), M) - r0, 0);
        }
        const int nt = (len + 16 * TB - 1) / (16 * TB), nb = (len + 15) >> 4;
        const int sum = wave_scan(nt), bsum = TB == 1 ? sum : wave_scan(nb);
        const unsigned long long past = __ballot(before + sum > want);
        if (past != 0) {
            const int src = __ffsll(past) - 1;
            const int off = want - before - __builtin_amdgcn_readlane(sum - nt, src);
            return Tile{__builtin_amdgcn_readlane(r0, src) + off * 16 * TB,
                        min(16 * TB, __builtin_amdgcn_readlane(len, src) - off * 16 * TB),
                        __builtin_amdgcn_readlane(id, src),
                        blocks + __builtin_amdgcn_readlane(bsum - nb, src) + off * TB};
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        blocks += __builtin_amdgcn_readlane(bsum, 63);
    }
    return Tile{0, 0, -1, 0};
}

// A tile's adapter, its rank (0: none, as for an index outside the pool) and its scale.
struct Adapter {
    int s, rank;
    float alpha;
};

__device__ __forceinline__ Adapter adapter_of(const LoraBatchArgs& a, int id) {
    if (id < 0 || id >= a.n_adapters) return Adapter{0, 0, 0.f};
    return Adapter{id, a.ranks == nullptr ? a.R : min(max(a.ranks[id], 0), a.R), a.alphas[id]};
}

// Whether rows without adapter stay as they are: no activation, in place.
__device__ __forceinline__ bool unchanged(const LoraBatchArgs& a) { return a.act == 0 && a.base == a.out; }

__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

__device__ __forceinline__ uint4 only_if(bool on, uint4 v) {
    return make_uint4(on ? v.x : 0u, on ? v.y : 0u, on ? v.z : 0u, on ? v.w : 0u);
}

// Between a wave's writes to its LDS and its lanes' reads of one another's: the LDS serves a
// wave in order, so only the compiler has to keep them so.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 16 rows x 128 channels as loaded (v[g]: rows 4 g to 4 g + 3, 16 lanes to a row; zeros for a
// lane that is off) to the operands of 4 steps of 32 channels, through 4 KB of LDS.
__device__ __forceinline__ void to_operands(uint4* buf, const uint4 (&v)[4], bool on, uint4 (&op)[4]) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15;
    wave_sync();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int row = g * 4 + q;
        buf[row * 16 + (r16 ^ row)] = only_if(on, v[g]);
    }
    wave_sync();
#pragma unroll
    for (int k = 0; k < 4; ++k) op[k] = buf[r16 * 16 + ((k * 4 + q) ^ r16)];
}

// One wave's share of the down-projection: every stride-th step of 128 channels from `first`, 16
// rows x rank blocks rb0 to rb0 + RB - 1 (those past the adapter's last repeat it; the caller
// drops them).  U steps are loaded at a time; channels past K count as zeros.
// acc[j]: lane (q, r16) holds ranks 4 q to 4 q + 3 of block j for row r16.
template <int RB, int U>
__device__ __forceinline__ void down_steps(const LoraBatchArgs& a, const Tile& t, const Adapter& ad, int rb0,
                                           int first, int stride, uint4* buf, f32x4 (&acc)[RB]) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15, K = a.K;
    const uint16_t* xp[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
        xp[g] = (const uint16_t*)a.x + (int64_t)(t.row0 + min(g * 4 + q, t.rows - 1)) * a.x_stride;
    const uint16_t* dp = (const uint16_t*)a.down + ((int64_t)ad.s * a.R + q) * K;
    const int last = ((ad.rank + 15) >> 4) - 1;
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int steps = (K + 127) >> 7;
    for (int st = first; st < steps; st += U * stride) {
        uint4 xv[U][4], dv[U][RB][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min((st + u * stride) * 128 + r16 * 8, K - 8);
#pragma unroll
            for (int g = 0; g < 4; ++g) xv[u][g] = *(const uint4*)(xp[g] + k);
#pragma unroll
            for (int j = 0; j < RB; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    dv[u][j][g] = *(const uint4*)(dp + (int64_t)(min(rb0 + j, last) * 16 + g * 4) * K + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // zeroed here and not at the load, which nothing should have to wait for
            const bool on = (st + u * stride) * 128 + r16 * 8 < K;
            uint4 x[4];
            to_operands(buf, xv[u], on, x);
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                uint4 d[4];
                to_operands(buf, dv[u][j], on, d);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[j] = mfma16(d[k], x[k], acc[j]);
            }
        }
    }
}

constexpr uint32_t kHalf = 0x80;   // a step of a bf16's exponent

// bf16 terms of v: its first 8 significant bits, the next 8 and the last, cut and not rounded, so
// that they have v's sign and their sum is v (bits below 2^-133 apart).  In the place of a term
// whose bits are all zero stand halves of the one before it: an infinite operand then meets no
// zero, and gives the infinity that v itself gives (from |v| = 2^-100 on, where halves are exact).
__device__ __forceinline__ void split_terms(float v, uint32_t (&t)[3]) {
    const uint32_t u = __float_as_uint(v), h = (u >> 16) | (v != v ? 0x40u : 0u);   // a NaN keeps a bit
    const float rest = v - __uint_as_float(u & 0xFFFF0000u);
    const uint32_t m = __float_as_uint(rest) >> 16;
    const uint32_t l = __float_as_uint(rest - __uint_as_float(m << 16)) >> 16;
    const bool no_m = (m & 0x7FFFu) == 0, no_l = (l & 0x7FFFu) == 0;
    const bool cut_h = no_m && (h & 0x7FFFu) >= 3 * kHalf, cut_m = !no_m && no_l && (m & 0x7FFFu) >= 2 * kHalf;
    const uint32_t half = h - kHalf, quarter = half - kHalf, half_m = m - kHalf;
    t[0] = cut_h ? half : h;
    t[1] = cut_h ? (no_l ? quarter : half) : cut_m ? half_m : m;
    t[2] = cut_h && no_l ? quarter : cut_m ? half_m : l;
    if ((u & 0x7F800000u) == 0x7F800000u) t[0] = t[1] = t[2] = h;   // an infinity or a NaN: all three
}

// Ranks of the up-projection go in NB blocks of 32 (16 ranks in all: NB = 0, one half block).
// Every block of the instantiation is multiplied, with zeros at and past the adapter's rank.
constexpr int blocks_of(int NB) { return NB == 0 ? 1 : NB; }
// Operands of a block of 16 rows' t: one for each term; in the half block the first holds the
// first term in lanes q = 0, 1 and the second in q = 2, 3, the other a half of the third in both.
constexpr int ops_of(int NB) { return NB == 0 ? 2 : 3; }

// alpha times ranks j0 to j0 + 3 of row r16, `live` of them below the rank, to their places in
// the operands `to` [ops][blocks][64 lanes] (blocks = 0: the half block).
__device__ __forceinline__ void put_terms(uint2* to, int blocks, int j0, int r16, f32x4 v, float alpha, int live) {
    uint32_t t[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_terms(e < live ? alpha * v[e] : 0.f, t[e]);
    const int at = (((j0 >> 3) & 3) * 16 + r16) * 2 + ((j0 >> 2) & 1);   // lane's half operand
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const uint2 w = make_uint2(t[0][n] | (t[1][n] << 16), t[2][n] | (t[3][n] << 16));
        if (blocks > 0) {
            to[(n * blocks + (j0 >> 5)) * 128 + at] = w;
        } else if (n < 2) {
            to[n * 64 + at] = w;
        }
    }
    if (blocks == 0) {
        uint32_t half[4], rest[4];   // halves but for the least values, which stand whole in one place
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool cut = (t[e][2] & 0x7FFFu) >= 2 * kHalf;
            half[e] = cut ? t[e][2] - kHalf : t[e][2];
            rest[e] = cut ? half[e] : 0u;
        }
        to[128 + at] = make_uint2(half[0] | (half[1] << 16), half[2] | (half[3] << 16));
        to[192 + at] = make_uint2(rest[0] | (rest[1] << 16), rest[2] | (rest[3] << 16));
    }
}

// The words of 8 consecutive bf16 with elements at and past `live` cleared.
__device__ __forceinline__ uint4 keep_first(uint4 v, int live) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = live >= 2 * i + 2 ? w[i] : live == 2 * i + 1 ? (w[i] & 0xFFFFu) : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Workgroup `id` of a grid of tiles x inner.  Consecutive workgroups go to the 8 XCDs in turn.
// DEAL: the tiles go to the XCDs in turn, each with all its inner parts, which read the same rows
// of x, so these come to one L2 (2048 x 3072, rank 128: 28.9 us in all, 30.0 without).  The
// up-projection goes in order, neighbours on neighbouring columns of out: 600 x 4096, rank 128:
// 17.9 us in all, dealt 19.8; ranges of neighbouring tiles to an XCD cost most, 16384 x 4096 at
// rank 32 105 us for 95.
template <bool DEAL>
__device__ __forceinline__ void tile_of(int id, int inner, int& tile, int& part) {
    const int l = DEAL ? id >> 3 : id;
    tile = l / inner;
    part = l - tile * inner;
    if (DEAL) tile = tile * 8 + (id & 7);
}

// Down-projection of a tile of 16 rows, RB rank blocks: the W waves take the steps of K in turn
// and their sums are added in wave order through LDS.  16 waves of one step at a time (64
// registers) leave room for a second workgroup on the CU, which the few tiles past 256 need:
// 4096 x 3072, rank 16: 9.3 us (2.7 TB/s of x); 12.9 with two steps at a time and one workgroup
// a CU.  Bound by the latency of its few steps; 16384 x 4096 takes 37 us (3.6 TB/s).
template <int RB, int W, int U>
__global__ __launch_bounds__(W * 64) void lora_down_kernel(LoraBatchArgs a, int inner) {
    constexpr int kSums = W * RB * 64, kStage = W * 256;
    static_assert(kSums * 16 <= 65536 && kStage * 16 <= 65536, "64 KB of LDS");
    __shared__ uint4 lds[kSums > kStage ? kSums : kStage];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, r16 = lane & 15;
    int tile, part;
    tile_of<true>(blockIdx.x, inner, tile, part);
    const Tile t = find_tile<1>(a, tile);
    // offsets that break the rules may make more blocks than there is room for
    if (t.rows == 0 || t.block >= a.max_blocks) return;
    const Adapter ad = adapter_of(a, t.id);
    if (ad.rank == 0) return;
    const int rb0 = part * RB;
    const bool some = rb0 * 16 < ad.rank;   // uniform over the workgroup
    f32x4* red = (f32x4*)lds;
    if (some) {
        f32x4 acc[RB];
        down_steps<RB, U>(a, t, ad, rb0, w, W, lds + w * 256, acc);
        __syncthreads();                    // the sums take the operands' place
#pragma unroll
        for (int j = 0; j < RB; ++j) red[(w * RB + j) * 64 + lane] = acc[j];
        __syncthreads();
    }
    const int ranks = a.nb == 0 ? 16 : a.nb * 32;
    for (int b = w; b < RB; b += W) {
        const int j0 = (rb0 + b) * 16 + q * 4;
        if (j0 >= ranks) continue;
        f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
        if (some) {
#pragma unroll
            for (int o = 0; o < W; ++o) v += red[(o * RB + b) * 64 + lane];
        }
        put_terms((uint2*)a.work + (int64_t)t.block * ops_of(a.nb) * blocks_of(a.nb) * 128, a.nb, j0, r16, v, ad.alpha,
                  ad.rank - j0);
    }
}

// Down-projection of a tile of 16 TB rows, 16 NRB ranks, for ranks past 32: the rows and the
// adapter's A are staged once for the workgroup, 128 channels at a time, and each wave has RW
// row blocks x KW rank blocks over all of K.  D steps are in flight in registers (OCC: waves a
// SIMD that the registers must leave room for).  Bound by the CU's LDS and its barriers: 1.5 us
// a step of 96 rows x 128 ranks, of which LDS moves 216 KB; 16384 x 4096 at rank 128 takes 63 us
// (2.1 TB/s of x).  At rank 32 the narrow kernel is faster: 8192 x 12288 86 us in all, so 104.
// Steps are counted from another one in each tile, round the end of K: rows of x and A lie K
// elements apart, a distance that falls on few memory channels, and workgroups that walk K in
// step would all ask the same ones.
template <int TB, int NRB, int RW, int KW, int D, int OCC>
__global__ __launch_bounds__((TB / RW) * (NRB / KW) * 64, OCC) void lora_down_wide_kernel(LoraBatchArgs a, int inner) {
    constexpr int kWaves = (TB / RW) * (NRB / KW), kRows = 16 * (TB + NRB), kSet = kWaves * 4, kLoads = kRows / kSet;
    static_assert(kRows % kSet == 0 && kSet % 16 == 0, "whole loads");
    __shared__ uint4 lds[kRows * 16];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, q = lane >> 4, r16 = lane & 15, K = a.K;
    int tile, part;
    tile_of<true>(blockIdx.x, inner, tile, part);
    const Tile t = find_tile<TB>(a, tile);
    if (t.rows == 0) return;
    const Adapter ad = adapter_of(a, t.id);
    if (ad.rank == 0) return;
    const int rb0 = part * NRB;
    // thread's rows of the staged tile: tid / 16 + kSet i; rows first, then ranks (those past the
    // adapter's last block repeat its last row)
    const uint16_t* src[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (tid >> 4) + kSet * i, j = rb0 * 16 + r - 16 * TB;
        src[i] = r < 16 * TB
                     ? (const uint16_t*)a.x + (int64_t)(t.row0 + min(r, t.rows - 1)) * a.x_stride
                     : (const uint16_t*)a.down + ((int64_t)ad.s * a.R + min(j, (ad.rank + 15) / 16 * 16 - 1)) * K;
    }
    const int steps = (K + 127) >> 7, turn = (int)((unsigned)tile * 5u % (unsigned)steps);
    auto channel = [&](int st) {
        st = min(st, steps - 1) + turn;
        return (st >= steps ? st - steps : st) * 128 + r16 * 8;
    };
    auto load = [&](uint4 (&v)[kLoads], int st) {
        const int k = min(channel(st), K - 8);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) v[i] = *(const uint4*)(src[i] + k);
    };
    auto put = [&](const uint4 (&v)[kLoads], int st) {
        const int row = tid >> 4;
        const bool on = channel(st) < K;   // zeroed here and not at the load, which nothing should wait for
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) lds[(row + kSet * i) * 16 + (r16 ^ (row & 15))] = only_if(on, v[i]);
        __syncthreads();
    };
    f32x4 acc[RW][KW];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int j0 = w % (NRB / KW) * KW, i0 = w / (NRB / KW) * RW;
    auto work = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = (k * 4 + q) ^ r16;
            uint4 x[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) x[i] = lds[((i0 + i) * 16 + r16) * 16 + c];
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const uint4 d = lds[((TB + j0 + j) * 16 + r16) * 16 + c];
#pragma unroll
                for (int i = 0; i < RW; ++i) acc[i][j] = mfma16(d, x[i], acc[i][j]);
            }
        }
    };
    uint4 v[D][kLoads];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(v[d], d);
        __builtin_amdgcn_sched_barrier(0);   // in this order, so that the oldest can be waited for alone
    }
    for (int st = 0; st < steps; st += D) {
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d == 0 || st + d < steps) {
                put(v[d], st + d);
                load(v[d], st + d + D);
                __builtin_amdgcn_sched_barrier(0);
                work();
            }
    }
    const int ranks = a.nb * 32;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            const int at = (rb0 + j0 + j) * 16 + q * 4;
            if ((i0 + i) * 16 < t.rows && at < ranks && t.block + i0 + i < a.max_blocks)
                put_terms((uint2*)a.work + (int64_t)(t.block + i0 + i) * 3 * a.nb * 128, a.nb, at, r16, acc[i][j], ad.alpha,
                          ad.rank - at);
        }
}

// A wave's 16 RBE rows x 16 CB columns of out.
template <int RBE, int CB, int NB, bool BF16>
struct UpTile {
    static constexpr int kOps = ops_of(NB), kBlocks = blocks_of(NB);
    // operands of t in registers; the last one's in LDS where that makes room for another wave a
    // SIMD (16384 x 4096 at rank 32 96 us in all, 100 with it in registers; 8192 x 1024 at rank
    // 128, fp32, 37 and 39; rank 16 no less, 8192 x 3072 at rank 64 61 and 60)
    static constexpr int kHeld = (NB == 1 && CB == 4) || (NB == 4 && !BF16) ? kOps - 1 : kOps;
    static constexpr int kPer = BF16 ? 8 : 4;                 // columns of a 16-byte piece
    static constexpr int kLanes = 16 * CB / kPer;             // pieces, and lanes, of a row
    static constexpr int kPieces = RBE * 16 * kLanes / 64;    // a lane's pieces
    static constexpr int kChunks = NB == 0 ? 2 : NB * 4;      // 16-byte chunks of a row of B
    static constexpr int kUp = CB * 16 * kChunks / 64;        // a lane's chunks
    static constexpr int kLds = (CB * 16 * kChunks > RBE * 64 * CB ? CB * 16 * kChunks : RBE * 64 * CB);   // uint4 a wave
    using Base = uint4[kPieces];
    uint4 up[kUp];

    static __device__ __forceinline__ int piece_row(int p) { return (p * 64 + (threadIdx.x & 63)) / kLanes; }
    static __device__ __forceinline__ int piece_col() { return (threadIdx.x & 63) % kLanes * kPer; }

    static __device__ __forceinline__ void load_base(const LoraBatchArgs& a, const Tile& t, int c0, Base& base) {
        const int c = c0 + piece_col();
        const bool on = a.vec && a.base != nullptr && c + kPer <= a.N;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            base[p] = make_uint4(0, 0, 0, 0);
            if (on && piece_row(p) < t.rows)
                base[p] = *(const uint4*)((const char*)a.base +
                                          ((int64_t)(t.row0 + piece_row(p)) * a.base_stride + c) * (BF16 ? 2 : 4));
        }
    }

    // B's rows c0 to c0 + 16 CB - 1 (those past N repeat the last one), zeros at and past the rank
    __device__ __forceinline__ void load_up(const LoraBatchArgs& a, const Adapter& ad, int c0) {
        const int lane = threadIdx.x & 63, j = lane % kChunks * 8;
        const uint16_t* p = (const uint16_t*)a.up + (int64_t)ad.s * a.N * a.R + min(j, a.R - 8);
#pragma unroll
        for (int i = 0; i < kUp; ++i)
            up[i] = *(const uint4*)(p + (int64_t)min(c0 + (i * 64 + lane) / kChunks, a.N - 1) * a.R);
        if (ad.rank < kChunks * 8) {
#pragma unroll
            for (int i = 0; i < kUp; ++i) up[i] = keep_first(up[i], ad.rank - j);
        }
    }

    static constexpr int kSpread = 16 / kChunks;   // rows of B to 256 bytes of LDS

    // B to LDS; its registers are free then
    __device__ __forceinline__ void stage_up(uint4* lds) {
        const int lane = threadIdx.x & 63;
        wave_sync();
#pragma unroll
        for (int i = 0; i < kUp; ++i) {
            const int n = (i * 64 + lane) / kChunks, j = lane % kChunks;
            lds[n * kChunks + (j ^ (n / kSpread % kChunks))] = up[i];
        }
        wave_sync();
    }

    // acc = t B^T, lane (q, r16) with columns 16 c + 4 q to 16 c + 4 q + 3 of row 16 i + r16
    // (B is the MFMA's row operand; low: t's last operand, [RBE][kBlocks][64], where it is in LDS)
    static __device__ __forceinline__ void products(const uint4* lds, const uint4 (&tm)[RBE][kHeld][kBlocks],
                                                    const uint4* low, f32x4 (&acc)[RBE][CB]) {
        const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15;
#pragma unroll
        for (int i = 0; i < RBE; ++i)
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            uint4 last[RBE];
#pragma unroll
            for (int i = 0; i < RBE; ++i) last[i] = kHeld < kOps ? low[(i * kBlocks + b) * 64 + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                const int n = c * 16 + r16, j = NB == 0 ? q & 1 : b * 4 + q;
                const uint4 m = lds[n * kChunks + (j ^ (n / kSpread % kChunks))];
#pragma unroll
                for (int o = 0; o < kOps; ++o) {
#pragma unroll
                    for (int i = 0; i < RBE; ++i) acc[i][c] = mfma16(m, o < kHeld ? tm[i][o % kHeld][b] : last[i], acc[i][c]);
                }
            }
        }
    }

    static __device__ __forceinline__ int slot(int row, int chunk) {
        return row * CB * 4 + (chunk ^ (CB == 4 ? row & 15 : (row >> 1) & 7));
    }

    // acc from lanes that hold 4 columns to pieces of kPer columns
    static __device__ __forceinline__ void turn(uint4* lds, const f32x4 (&acc)[RBE][CB], float (&y)[kPieces][kPer]) {
        const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15;
        static_assert(CB == 4 || CB == 2, "slots of a row");
        f32x4* buf = (f32x4*)lds;
        wave_sync();
#pragma unroll
        for (int i = 0; i < RBE; ++i)
#pragma unroll
            for (int c = 0; c < CB; ++c) buf[slot(i * 16 + r16, c * 4 + q)] = acc[i][c];
        wave_sync();
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int h = 0; h < kPer / 4; ++h) {
                const f32x4 v = buf[slot(piece_row(p), piece_col() / 4 + h)];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[p][h * 4 + e] = v[e];
            }
    }

    template <int ACT>
    static __device__ __forceinline__ void store_as(const LoraBatchArgs& a, const Tile& t, int c0, const Base& base,
                                                    const float (&y)[kPieces][kPer]) {
        const int c = c0 + piece_col();
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (piece_row(p) >= t.rows) continue;
            const int64_t m = t.row0 + piece_row(p);
            if (a.vec && c + kPer <= a.N) {
                const uint32_t bw[4] = {base[p].x, base[p].y, base[p].z, base[p].w};
                float v[kPer];
                uint32_t ow[4];
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    v[e] = activate(y[p][e] + (!BF16 ? __uint_as_float(bw[e & 3])
                                                     : __uint_as_float((e & 1) ? bw[e >> 1] & 0xFFFF0000u : bw[(e >> 1) & 3] << 16)),
                                    ACT);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ow[e] = BF16 ? pack_bf16(v[(2 * e) % kPer], v[(2 * e + 1) % kPer]) : __float_as_uint(v[e]);
                *(uint4*)((char*)a.out + (m * a.out_stride + c) * (BF16 ? 2 : 4)) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (c + e < a.N) {
                        float v = y[p][e];
                        if constexpr (BF16) {
                            if (a.base != nullptr) v += bf16_to_f32(((const uint16_t*)a.base)[m * a.base_stride + c + e]);
                            ((uint16_t*)a.out)[m * a.out_stride + c + e] = (uint16_t)f32_to_bf16(activate(v, ACT));
                        } else {
                            if (a.base != nullptr) v += ((const float*)a.base)[m * a.base_stride + c + e];
                            ((float*)a.out)[m * a.out_stride + c + e] = activate(v, ACT);
                        }
                    }
            }
        }
    }

    static __device__ __forceinline__ void store(const LoraBatchArgs& a, const Tile& t, int c0, const Base& base,
                                                 const float (&y)[kPieces][kPer]) {
        if (a.act == 1) store_as<1>(a, t, c0, base, y);
        else if (a.act == 2) store_as<2>(a, t, c0, base, y);
        else store_as<0>(a, t, c0, base, y);
    }

    // rows without adapter: out = act(base)
    static __device__ __forceinline__ void store_base(const LoraBatchArgs& a, const Tile& t, int c0, const Base& base) {
        float y[kPieces][kPer];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int e = 0; e < kPer; ++e) y[p][e] = 0.f;
        store(a, t, c0, base, y);
    }
};

// Up-projection, bound by memory (base and out once) and, at rank 128, by the registers that t
// takes: 16384 x 4096 at rank 16 takes 52 us (5.2 TB/s), at rank 128 95 us (2.9 TB/s).
//
// A workgroup's rows x `blocks` blocks of 64 CB columns, 16 CB columns to each of 4 waves: t
// stays in registers; base is loaded two blocks ahead, B as soon as the block before has its own
// in LDS.
template <int RBE, int CB, int NB, bool BF16>
__device__ __forceinline__ void up_blocks(const LoraBatchArgs& a, const Tile& t, const Adapter& ad, int first,
                                          int blocks, uint4* lds, uint4* low) {
    using Up = UpTile<RBE, CB, NB, BF16>;
    constexpr int D = 2;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    auto col = [&](int b) { return ((first + b) * 4 + w) * 16 * CB; };
    Up u;
    typename Up::Base base[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < blocks) Up::load_base(a, t, col(d), base[d]);
    u.load_up(a, ad, col(0));
    uint4 tm[RBE][Up::kHeld][Up::kBlocks];
    const int wb = blocks_of(a.nb), ops = ops_of(a.nb);
#pragma unroll
    for (int i = 0; i < RBE; ++i) {
        const uint4* src = (const uint4*)a.work +
                           (int64_t)min(t.block + (i * 16 < t.rows ? i : 0), a.max_blocks - 1) * ops * wb * 64 + lane;
#pragma unroll
        for (int o = 0; o < Up::kHeld; ++o)
#pragma unroll
            for (int b = 0; b < Up::kBlocks; ++b) tm[i][o][b] = src[(o * wb + b) * 64];
        if constexpr (Up::kHeld < Up::kOps) {
#pragma unroll
            for (int b = 0; b < Up::kBlocks; ++b)
                if (((i * Up::kBlocks + b) & 3) == w) low[(i * Up::kBlocks + b) * 64 + lane] = src[(Up::kHeld * wb + b) * 64];
        }
    }
    if constexpr (Up::kHeld < Up::kOps) __syncthreads();
    for (int b = 0; b < blocks; b += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (b + d >= blocks) break;
            u.stage_up(lds);
            u.load_up(a, ad, col(min(b + d + 1, blocks - 1)));
            f32x4 acc[RBE][CB];
            float y[Up::kPieces][Up::kPer];
            Up::products(lds, tm, low, acc);
            Up::turn(lds, acc, y);
            Up::store(a, t, col(b + d), base[d], y);
            if (b + d + D < blocks) Up::load_base(a, t, col(b + d + D), base[d]);
        }
    }
}

// Waves a SIMD that the up-projection's registers must leave room for: at 32 rows, 32 columns a wave
// and rank 16 the compiler takes 97 unasked, one more than leaves room for 5 (4096 x 3072 21.6 us
// in all, 22.3 with 4 waves); tighter bounds elsewhere spill and cost time.
constexpr int up_waves(int RBE, int CB, int NB) { return RBE == 2 && CB == 2 && NB == 0 ? 5 : 1; }

// Up-projection of a tile of 16 RBE rows, `span` blocks of columns.
template <int RBE, int CB, int NB, bool BF16>
__global__ __launch_bounds__(256, up_waves(RBE, CB, NB)) void lora_up_kernel(LoraBatchArgs a, int inner, int span) {
    using Up = UpTile<RBE, CB, NB, BF16>;
    __shared__ uint4 lds[4][Up::kLds], low[Up::kHeld < Up::kOps ? RBE * Up::kBlocks * 64 : 1];
    int tile, part;
    tile_of<false>(blockIdx.x, inner, tile, part);
    const Tile t = find_tile<RBE>(a, tile);
    if (t.rows == 0) return;
    const int first = part * span, w = threadIdx.x >> 6;
    const int blocks = min(span, (a.N + 64 * CB - 1) / (64 * CB) - first);
    const Adapter ad = adapter_of(a, t.id);
    if (ad.rank == 0) {
        if (unchanged(a)) return;
        for (int b = 0; b < blocks; ++b) {
            const int c0 = ((first + b) * 4 + w) * 16 * CB;
            typename Up::Base base;
            Up::load_base(a, t, c0, base);
            Up::store_base(a, t, c0, base);
        }
        return;
    }
    if constexpr (NB > 2) {
        if (ad.rank <= 64) {
            up_blocks<RBE, CB, 2, BF16>(a, t, ad, first, blocks, lds[w], low);
            return;
        }
    }
    up_blocks<RBE, CB, NB, BF16>(a, t, ad, first, blocks, lds[w], low);
}

// Both products for a tile of 16 rows x 256 columns, 32 columns to each of 8 waves: the waves
// share the steps of K, and the rows' t goes through LDS.  Every workgroup of a tile reads its
// rows and A again (from the L2s), which costs less than a second launch while they are few
// and fit one round of CUs: 2 rows, 3072 -> 18432, rank 16: 6.8 us, two launches 8.1; 1237 rows,
// rank 64, in 332 workgroups: 14.3 us, in two launches 11.3.  Bound by a chain of dependent
// latencies: the launch, the segment, its adapter, K / 1024 steps, the join of the waves' sums.
template <int RB, bool BF16, int U>
__global__ __launch_bounds__(512) void lora_few_rows_kernel(LoraBatchArgs a, int inner) {
    constexpr int W = 8, NB = RB / 2;
    using Up = UpTile<1, 2, NB, BF16>;
    constexpr int kStage = Up::kLds > 256 ? Up::kLds : 256;
    static_assert(kStage >= RB * 64, "the sums take the operands' place");
    __shared__ uint4 lds[W][kStage];
    f32x4* red = (f32x4*)lds;
    __shared__ uint4 terms[Up::kOps][Up::kBlocks][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, r16 = lane & 15;
    int tile, part;
    tile_of<false>(blockIdx.x, inner, tile, part);
    const Tile t = find_tile<1>(a, tile);
    if (t.rows == 0) return;
    const int c0 = part * kColTile + w * 32;
    Up u;
    typename Up::Base base;
    Up::load_base(a, t, c0, base);
    const Adapter ad = adapter_of(a, t.id);
    if (ad.rank == 0) {
        if (!unchanged(a)) Up::store_base(a, t, c0, base);
        return;
    }
    u.load_up(a, ad, c0);
    f32x4 acc[RB];
    down_steps<RB, U>(a, t, ad, 0, w, W, lds[w], acc);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RB; ++j) red[(w * RB + j) * 64 + lane] = acc[j];
    __syncthreads();
    if (w < RB) {
        const int j0 = w * 16 + q * 4;
        f32x4 v = red[w * 64 + lane];
#pragma unroll
        for (int o = 1; o < W; ++o) v += red[(o * RB + w) * 64 + lane];
        put_terms((uint2*)&terms[0][0][0], NB, j0, r16, v, ad.alpha, ad.rank - j0);
    }
    __syncthreads();
    uint4 tm[1][Up::kHeld][Up::kBlocks];
#pragma unroll
    for (int o = 0; o < Up::kHeld; ++o)
#pragma unroll
        for (int b = 0; b < Up::kBlocks; ++b) tm[0][o][b] = terms[o][b][lane];
    f32x4 out[1][2];
    float y[Up::kPieces][Up::kPer];
    u.stage_up(lds[w]);
    Up::products(lds[w], tm, nullptr, out);
    Up::turn(lds[w], out, y);
    Up::store(a, t, c0, base, y);
}

// Most tiles of `tm` rows that n segments of M rows can need.
int64_t most_tiles(int64_t M, int n, int tm) { return std::min<int64_t>((M + (int64_t)n * (tm - 1)) / tm, M); }

// Blocks of 32 ranks of the pool (0: 16 ranks).
int rank_blocks(int R) { return R <= 16 ? 0 : R <= 32 ? 1 : R <= 64 ? 2 : 4; }

unsigned grid_of(int64_t tiles, int inner, bool deal) { return (unsigned)((deal ? (tiles + 7) / 8 * 8 : tiles) * inner); }

template <int RB, int W, int U>
void down(const LoraBatchArgs& a, hipStream_t st) {
    const int64_t tiles = most_tiles(a.M, a.n_segments, 16);
    const int inner = ((a.nb == 0 ? 1 : a.nb * 2) + RB - 1) / RB;
    hipLaunchKernelGGL((lora_down_kernel<RB, W, U>), dim3(grid_of(tiles, inner, true)), dim3(W * 64), 0, st, a, inner);
}

// Rows from which A is staged once a workgroup, for ranks past 32.  Such a workgroup walks all of K
// alone, where the narrow kernel's waves share it, so a longer K takes more workgroups to hide (us
// in all, wide and narrow.  Rank 64, K = 1024: 3500 rows 23.7 and 21.6, 4500 25.8 and 26.4; 2048:
// 4096 25.6 and 24.1, 7000 31.6 and 32.6; 3072: 6000 41.3 and 37.9, 9000 61.9 and 62.4, 16384 92.6
// and 101.9; 12288: 6000 103 and 85, 12000 140 and 154.  Rank 128, K = 1024: 2000 23.7 and 21.2,
// 3000 28.8 and 29.7; 2048: 3000 28.2 and 28.1, 5000 36.4 and 37.8; 3072: 5000 50.5 and 49.0, 7000
// 63.1 and 67.8; 12288: 5000 133 and 111, 8192 171 and 180).
int64_t wide_rows(const LoraBatchArgs& a) {
    return a.nb == 4 ? std::clamp<int64_t>(2 * (int64_t)a.K, 2304, 6144) : std::clamp<int64_t>(3 * (int64_t)a.K, 4096, 8192);
}

template <int TB, int NRB, int RW, int KW, int D, int OCC>
void down_wide(const LoraBatchArgs& a, hipStream_t st) {
    const int64_t tiles = most_tiles(a.M, a.n_segments, TB * 16);
    const int inner = (a.nb * 2 + NRB - 1) / NRB;
    hipLaunchKernelGGL((lora_down_wide_kernel<TB, NRB, RW, KW, D, OCC>), dim3(grid_of(tiles, inner, true)),
                       dim3((TB / RW) * (NRB / KW) * 64), 0, st, a, inner);
}

void launch_down(const LoraBatchArgs& a, hipStream_t st) {
    if (a.nb >= 2 && a.M >= wide_rows(a)) {
        // the lowest tiles that need one round of 256 CUs at most: a workgroup has a CU's LDS and
        // registers nearly to itself, and a few tiles too many cost another round (16384 x 4096,
        // rank 128, 16 segments: 152 us in all, with 64 rows to a tile 184; 12000 x 3072, rank 64:
        // 71.5 us, with 32 rows 74.4)
        const int tall = most_tiles(a.M, a.n_segments, 32) <= 256 ? 2
                         : most_tiles(a.M, a.n_segments, 64) <= 256 || most_tiles(a.M, a.n_segments, 96) > 256 ? 4 : 6;
        // low tiles leave CUs for a second workgroup on the other half of 128 ranks (4096 rows,
        // K = 4096: 46 us in all, 50 with one workgroup for all ranks)
        if (tall == 2) down_wide<2, 4, 1, 1, 2, 4>(a, st);
        else if (a.nb == 4) tall == 4 ? down_wide<4, 8, 2, 2, 3, 2>(a, st) : down_wide<6, 8, 3, 2, 3, 2>(a, st);
        else tall == 4 ? down_wide<4, 4, 2, 1, 3, 2>(a, st) : down_wide<6, 4, 3, 1, 3, 2>(a, st);
        return;
    }
    const int64_t tiles = most_tiles(a.M, a.n_segments, 16);
    // two rank blocks to a workgroup halve the reads of x where there are workgroups enough (two
    // and one, us in all: rank 32: 2000 rows of 3072 16.1 and 15.5, 16000 75 and 82; rank 64: 300
    // rows of 4096 12.9 and 12.3, 1000 of 3072 15.1 and 16.3; rank 128: 64 rows 11.4 and 10.2,
    // 600 17.5 and 21; four at 3500 47.7, two 45.0)
    const int rb = a.R / 16;
    if (rb >= 2 && tiles * ((rb + 1) / 2) >= (rb == 2 ? 256 : 128)) down<2, 8, 1>(a, st);
    else down<1, 16, 1>(a, st);
}

template <int RBE, int CB, int NB, bool BF16>
void up(const LoraBatchArgs& a, hipStream_t st) {
    const int64_t tiles = most_tiles(a.M, a.n_segments, RBE * 16);
    const int blocks = (a.N + 64 * CB - 1) / (64 * CB);
    // up to 2 blocks a workgroup, so that neighbours work on the rest of the same rows at a time;
    // 8 where t is large (16384 x 4096: rank 32 96 us in all, 108 with 8; rank 128 155, 168 with 2)
    constexpr int kMost = NB == 4 ? 8 : 2;
    int span = 1;
    while (span < kMost && span < blocks && tiles * ((blocks + 2 * span - 1) / (2 * span)) >= 1024) span *= 2;
    const int inner = (blocks + span - 1) / span;
    hipLaunchKernelGGL((lora_up_kernel<RBE, CB, NB, BF16>), dim3(grid_of(tiles, inner, false)), dim3(256), 0, st, a,
                       inner, span);
}

template <int RBE, bool BF16>
void up_rank(const LoraBatchArgs& a, hipStream_t st) {
    // columns of a wave: 64 cover whole cache lines of out, 32 make more and smaller workgroups
    // (16384 x 4096: rank 16 88.5 us in all with 64, 93.0 with 32; rank 32 96.4 and 101.7;
    // 4096 x 3072, rank 16 22.5 and 21.4)
    const bool wide = most_tiles(a.M, a.n_segments, RBE * 16) * ((a.N + 255) / 256) >= 2048;
    switch (a.nb) {
        case 0: wide ? up<RBE, 4, 0, BF16>(a, st) : up<RBE, 2, 0, BF16>(a, st); break;
        case 1: wide ? up<RBE, 4, 1, BF16>(a, st) : up<RBE, 2, 1, BF16>(a, st); break;
        case 2: wide ? up<RBE, 4, 2, BF16>(a, st) : up<RBE, 2, 2, BF16>(a, st); break;
        default: up<RBE, 2, 4, BF16>(a, st);
    }
}

template <bool BF16>
void few_rows(const LoraBatchArgs& a, hipStream_t st) {
    const int inner = (a.N + kColTile - 1) / kColTile;
    const dim3 grid((unsigned)(most_tiles(a.M, a.n_segments, 16) * inner)), block(512);
    if (a.R <= 16) hipLaunchKernelGGL((lora_few_rows_kernel<1, BF16, 2>), grid, block, 0, st, a, inner);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_few_rows_kernel<2, BF16, 1>), grid, block, 0, st, a, inner);
    else hipLaunchKernelGGL((lora_few_rows_kernel<4, BF16, 1>), grid, block, 0, st, a, inner);
}

}  // namespace

// Grids stay below 2^32 threads: at most 8 workgroups of 1024 a tile in the down-projection, one
// of 256 for each 128 columns in the other, tiles rounded up to whole XCDs.
bool lora_batch_fits(int64_t M, int N, int n_segments) {
    const int64_t tiles = most_tiles(M, n_segments, 16) + 8;
    return tiles < (int64_t)1 << 19 && tiles * (((int64_t)N + 127) / 128) < (int64_t)1 << 24;
}

int64_t lora_batch_workspace_bytes(int64_t M, int R, int n_segments) {
    if (n_segments == 0) return 0;
    // the operands of t, every block of 16 rows
    const int nb = rank_blocks(R);
    return most_tiles(M, n_segments, 16) * ops_of(nb) * blocks_of(nb) * 1024;
}

void launch_lora_batch(const LoraBatchArgs& args, hipStream_t st) {
    LoraBatchArgs a = args;
    a.nb = rank_blocks(a.R);
    a.max_blocks = (int)most_tiles(a.M, a.n_segments, 16);
    const int64_t inner = (a.N + kColTile - 1) / kColTile;
    // one launch while A is small (one and two launches, us: rank 16, K = 16384, 4 rows 14.2 and
    // 16.4; rank 32, K = 4096, 100 rows 8.5 and 9.0, K = 6144 11.0 and 10.4; rank 64, K = 1536, one
    // row 7.4 and 7.6, K = 2048 8.3 and 7.7)
    if (a.R <= 64 && a.max_blocks * inner <= 256 &&
        (int64_t)a.R * a.K <= (a.R <= 16 ? 1 << 18 : a.R <= 32 ? 1 << 17 : 3 << 15)) {
        a.bf16 ? few_rows<true>(a, st) : few_rows<false>(a, st);
        return;
    }
    if (a.n_adapters > 0) launch_down(a, st);
    // 32 rows to a workgroup where that leaves 1024 of them (16384 x 4096: rank 128 156 us in all,
    // with 16 173, rank 32 96 and 100; 300 x 3072, rank 32: 9.1, with 16 8.7); an fp32 output's
    // base takes the registers of the second 16 rows (30000 x 1024, rank 64: 90 us in all, 99 with
    // 32 rows)
    if (!a.bf16) up_rank<1, false>(a, st);
    else if ((a.M / 32) * inner >= 1024) up_rank<2, true>(a, st);
    else up_rank<1, true>(a, st);
}

}  // namespace svdq
