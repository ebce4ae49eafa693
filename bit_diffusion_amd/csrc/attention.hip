// attention.hip -- softmax attention of packed requests: rows of segment i see the keys of segment
// i, in grouped heads (H heads share G kv heads, H / G = rep to one).
//
//   s_ij = scale q_i . k_j,  capped:  s = cap tanh(s / cap),  biased:  s -= slope_h |i + off - j|,
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(s_ij - max_j s_ij) over the keys j that i sees:
//   all of the segment, or j < max(prefix, i + off + 1), off = keys - rows of the segment.
//
// One pass over the keys with the running maximum and sum of each row (fp32), tiles of 64 keys.
//
// Rows.  A workgroup owns up to 128 rows of one segment and one kv head: position major, the rep
// heads that share the kv head within (so single tokens fill rep rows of a tile, and its keys are
// read once for all of them).  Each of its 4 waves takes 32 rows and all keys.  The grid is the
// most tiles any cut of the rows can need; every workgroup finds its own by a prefix sum over the
// offsets in device memory.
//
// Products.  Both are 32x32x16 bf16 MFMAs, transposed: S^T = K Q^T and O^T = V^T P^T, so that a lane
// holds scores of one row only: row maximum and sum stay in the lane but for its other half (the
// lane 32 further), and what the first product leaves in registers is already the second one's
// operand, keys in the order 4 h to 4 h + 3, 8 + 4 h to 8 + 4 h + 3 of every 16 (h the lane's
// half).  V^T comes out of LDS in that order by the transposing read ds_read_b64_tr_b16.  P is
// rounded to bf16 (2^-8 of each weight at most, as V's own values were), and summed as rounded, which
// takes their common error out again; O, maxima and sums are fp32.
//
// Maximum.  What the weights are taken against need not be the largest score so far: bf16 and fp32
// hold a weight of 2^16 as well as 1.  So a row keeps the maximum of its first tile, and only
// where the weights' sum of a tile passes 2^16 are maximum, O and sum brought up to date and the tile's
// weights formed again (finding the largest score of every tile: 251 -> 260 us at 4608 rows and 24
// heads of 128).  With a bias by distance scores grow from tile to tile as a rule, and the largest is
// sought in each; O is rescaled only where it grew by more than 2^8.
//
// Few rows and keys: a wave's time is a tile's latency, so two waves share rows, each takes every other
// tile of keys (SHARE), and their maxima, sums and O meet in LDS.
//
// LDS.  K and V tiles, rows of 64 or 128 channels, twice each: the next tile's copies (LDS DMA,
// 16 bytes a lane) fly while this one is multiplied, one barrier a tile.  The 16-byte slots of a
// row are exclusive-ored with the row (K: for 16 rows of one channel slot; V: for 4 rows of 32
// channels), which the copies do by their source addresses.
//
// Masks.  A row sees the keys below its limit, so only a wave's tiles between its least and its
// largest limit are masked.  There, and in a segment's last tile, values of V that are not finite
// must not meet a weight 0: they are multiplied as 0, and counted in a second product over who sees
// them (poison below).
//
// Few row tiles: the keys of each are split over several workgroups, whose maxima, sums and O go to the
// workspace and are joined by a second launch.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>
#include <type_traits>

namespace svdq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;   // rows of a workgroup, or half as many where two waves share them
constexpr int kKeys = 64;            // keys of a tile
constexpr int kCus = 256;            // of the GPU
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;         // growth of a maximum, in powers of two, that O is rescaled for
constexpr float kMost = 65536.f;     // sum of 32 weights past which a row gets a new maximum
constexpr float kFine = 64.f;        // cap up to which, and |z| up to which above it, a capped score takes the
constexpr float kBend = 1.5f;        // first form and the second (Rows::capped)
constexpr float kLargest = 3.402823466e38f;

enum Mod { kPlain = 0, kCap = 1, kBias = 2, kBoth = 3 };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;

struct Tile {
    int seg;           // < 0: no such tile
    int q0, len;       // the segment's first row of q and its positions,
    int k0, keys;      // its first key and its keys
    int row0;          // the tile's first packed row
    int share;         // tiles of keys of a part that give every CU two, or 0 if not known
};
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int max_dpp(int v) { return max(v, dpp<CTRL, ROWS>(v, v)); }
// The largest over the wave, in every lane.
__device__ __forceinline__ int wave_max(int v) {
    v = max_dpp<kShr + 1>(v);
    v = max_dpp<kShr + 2>(v);
    v = max_dpp<kShr + 4>(v);
    v = max_dpp<kShr + 8>(v);
    v = max_dpp<kBcast15, 0xa>(v);
    v = max_dpp<kBcast31, 0xc>(v);
    return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp<kShr + 1>(0, v);
    v += dpp<kShr + 2>(0, v);
    v += dpp<kShr + 4>(0, v);
    v += dpp<kShr + 8>(0, v);
    v += dpp<kBcast15, 0xa>(0, v);
    v += dpp<kBcast31, 0xc>(0, v);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kShr + 1>(0.f, v);
    v += dpp<kShr + 2>(0.f, v);
    v += dpp<kShr + 4>(0.f, v);
    v += dpp<kShr + 8>(0.f, v);
    v += dpp<kBcast15, 0xa>(0.f, v);
    v += dpp<kBcast31, 0xc>(0.f, v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Tile `want` of the segments' tiles of ROWS rows (rep to a position).  Up to 64 segments: those
// with the most keys first (by powers of two), so that no long tile starts when the others are done;
// more: in order, and each workgroup goes through the offsets in front of its own, 64 a step (single rows over one
// key, one head, us: 64 of them 7.4, 1024 18, 4096 137, 16384 1800).  With a causal mask a segment's last rows first,
// which see the most.
template <int ROWS>
__device__ __forceinline__ Tile find_tile(const AttentionArgs& a, int rep, int want) {
    const int lane = threadIdx.x & 63, M = (int)a.Mq, Mk = (int)a.Mk;
    int next[4];
    auto fetch = [&](int i) {
        const int at = min(i, a.n - 1);
        next[0] = a.q_start[at];
        next[1] = a.q_start[at + 1];
        next[2] = a.kv_start[at];
        next[3] = a.kv_start[at + 1];
    };
    fetch(lane);
    for (int c = 0; c < a.n; c += 64) {
        const int q0 = min(max(next[0], 0), M), k0 = min(max(next[2], 0), Mk);
        const int len = c + lane < a.n ? max(min(max(next[1], 0), M) - q0, 0) : 0;
        const int keys = max(min(max(next[3], 0), Mk) - k0, 0);
        if (c + 64 < a.n) fetch(c + 64 + lane);
        const int nt = (len * rep + ROWS - 1) / ROWS;
        // products of row and key tiles, dealt to two workgroups a CU
        int share = 0;
        if (a.splits > 1 && a.n <= 64)
            share = (int)(wave_sum((float)nt * (float)((keys + kKeys - 1) / kKeys)) * ((float)a.G / (2 * kCus))) + 1;
        // a lane's turn: the number of its keys' bits, one turn for all of many segments; -1: no tile
        int turn = nt == 0 ? -1 : a.n > 64 ? 0 : 32 - __clz(keys);
        for (int now = a.n > 64 ? 0 : wave_max(turn); now >= 0; now = a.n > 64 ? -1 : wave_max(turn)) {
            const int mine = turn == now ? nt : 0, sum = wave_scan(mine);
            const unsigned long long past = __ballot(sum > want);
            if (past != 0) {
                const int src = __ffsll(past) - 1;
                const int off = want - __builtin_amdgcn_readlane(sum - mine, src);
                const int tile = a.causal ? __builtin_amdgcn_readlane(nt, src) - 1 - off : off;
                return Tile{c + src, __builtin_amdgcn_readlane(q0, src), __builtin_amdgcn_readlane(len, src),
                            __builtin_amdgcn_readlane(k0, src), __builtin_amdgcn_readlane(keys, src), tile * ROWS, share};
            }
            want -= __builtin_amdgcn_readlane(sum, 63);
            if (turn == now) turn = -1;
        }
    }
    return Tile{-1, 0, 0, 0, 0, 0, 0};
}

// The keys that packed row `row` of a segment sees: those below.
struct Limit {
    int causal, rep, keys, prefix, off;
    __device__ __forceinline__ Limit(const AttentionArgs& a, int seg, int len, int keys_)
        : causal(a.causal), rep(a.H / a.G), keys(keys_),
          prefix(a.prefix == nullptr ? 0 : min(max(a.prefix[seg], 0), keys_)), off(keys_ - len) {}
    __device__ __forceinline__ int of(int row) const {
        return causal ? min(max(max(prefix, row / rep + off + 1), 0), keys) : keys;
    }
};

__device__ __forceinline__ f32x16 mfma32(bf16x8 x, bf16x8 y, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
}

// The larger of the two halves' values, in both; NaN where either is.
__device__ __forceinline__ float both_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_elementwise_maximum(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float both_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

__device__ __forceinline__ uint64_t uniform_ptr(const void* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}
// Global -> LDS copy: each lane whose bit is set in `on` moves the 16 bytes at base + off to LDS
// address lds + 16 lane.  In asm so that the compiler does not wait for every copy in flight before
// each LDS read; wait_copies does.  An LDS copy that reads M0 right after its write needs one wait
// state.
__device__ __forceinline__ void copy16(uint64_t base, uint32_t off, uint32_t lds, uint64_t on) {
    uint64_t saved;
    asm volatile("s_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %3\n\ts_mov_b64 exec, %0"
                 : "=&s"(saved) : "v"(off), "s"(lds), "s"(base), "s"(on) : "memory", "scc");
}
// Every copy of this wave has landed, and every LDS access before is done.
__device__ __forceinline__ void wait_copies() { __builtin_amdgcn_s_waitcnt(0x0070); }
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// NB: blocks of 32 channels (D <= 32 NB, the rest counts as zero).
template <int NB>
struct Lds {
    static constexpr int kRow = NB <= 2 ? 128 : 256;             // bytes of a row
    static constexpr int kSlots = kRow / 16;
    static constexpr int kTile = kKeys * kRow;
    // 16-byte slot of channel slot `s` in row `r`
    static __device__ __forceinline__ int k_slot(int r, int s) { return s ^ (kSlots == 16 ? r & 15 : (r >> 1) & 7); }
    static __device__ __forceinline__ int v_slot(int r, int s) { return s ^ (kSlots == 16 ? (r & 3) << 2 : ((r >> 1) & 1) << 2); }
};

// One wave's rows.  NC: steps of 16 channels that Q K^T has (D <= 16 NC, NC <= 8).
template <int NC, int MOD>
struct Rows {
    static constexpr int NB = (NC + 1) / 2;
    f32x16 O[NB];      // O^T: lane (h, row) has channels 32 b + 8 (i / 4) + 4 h + i % 4
    bf16x8 Q[NC];      // channels 16 c + 8 h to + 7 of the lane's row
    float m, l;        // maximum of the row's scores (MOD = kPlain: unscaled; else times log2 e), this half's sum
    int limit;         // keys that the row sees
    int at;            // the key at distance 0
    float slope;       // times log2 e
    float c0, c1, cz;  // scale log2 e; with cap: cap log2 e, 2 scale log2 e / cap
    bool fine;         // cap <= kFine

    // cap log2 e tanh(y) of 16 products x, y = x scale / cap, z = 2 y log2 e.
    // Caps up to kFine: cap - 2 cap / (2^z + 1), whose error, 2^-23 of the cap, is 2^-17 of a weight at most where
    // weights are rounded by 2^-9.  Larger caps, whose error would grow past that: up to |z| = kBend as c0 x
    // (tanh(y) / y), a polynomial in z^2 (off by 2^-25.4 of it at most), so that what is far below the cap keeps its
    // relative precision; above as 1 - 2 / (2^|z| + 1), which cancels no more than half.  Which form a score takes
    // depends on it and the cap alone; where no lane needs the last, it is passed over.  (2 x 2048 rows of 8 heads of
    // 128, cap 50: 55.1 us, with the choice of a form 57.0; cap 65: the first form 55.3, the second 62.5; scores of
    // up to twice the cap 66.6 and, where most waves need the last, 89.6.)
    __device__ __forceinline__ void capped(f32x16& s) const {
        const auto each = [&](auto form) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = form(s[i], s[i] * cz);
        };
        if (fine) {
            const float c2 = 2.f * c1;
            each([&](float, float z) { return c1 - c2 * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(z) + 1.f); });
            return;
        }
        const auto small = [&](float x, float z) {
            const float w = z * z;
            const float p = fmaf(fmaf(fmaf(fmaf(3.5228786e-06f, w, -9.168231e-05f), w, 0.0019222912f), w, -0.040037446f), w, 1.f);
            return x * c0 * p;
        };
        const auto any = [&](float x, float z) {
            const float t = c1 * fmaf(-2.f, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(fabsf(z)) + 1.f), 1.f);
            const float below = small(x, z), above = copysignf(t, z);
            return fabsf(z) > kBend ? above : below;
        };
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(s[i]));
        if (__any(most * cz > kBend)) each(any);
        else each(small);
    }

    // scores of 32 keys from key0 on to the exponent's domain
    template <bool MASK>
    __device__ __forceinline__ void score(f32x16& s, int key0, int h) const {
        const float far = (float)(key0 + 4 * h - at);
        const int seen = limit - key0 - 4 * h;
        if constexpr ((MOD & kCap) != 0) capped(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int key = 8 * (i >> 2) + (i & 3);   // from the lane's first one on
            float x = s[i];
            if constexpr (MOD == kBias) x *= c0;
            if constexpr ((MOD & kBias) != 0) x = fmaf(-slope, fabsf(far + (float)key), x);
            if constexpr (MASK) x = key < seen ? x : -INFINITY;
            s[i] = x;
        }
    }
};

// All ones in the halves of a word of two bf16 that are not finite (their exponent bits plus one
// reach the sign's place).
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const s16x2 t = __builtin_bit_cast(s16x2, (w & 0x7F807F80u) + 0x00800080u);
    return __builtin_bit_cast(uint32_t, t >> 15);
}
__device__ __forceinline__ uint4 finite_only(uint4 v) {
    return make_uint4(v.x & ~not_finite(v.x), v.y & ~not_finite(v.y), v.z & ~not_finite(v.z), v.w & ~not_finite(v.w));
}
// Of a bf16: 1 for infinity, 2^8 for minus infinity, 2^16 for a NaN, else 0, as bf16.
__device__ __forceinline__ uint32_t kind16(uint32_t v) {
    const uint32_t bad = (v & 0x7F80u) == 0x7F80u;
    const uint32_t k = (v & 0x7Fu) != 0 ? 0x4780u : (v & 0x8000u) != 0 ? 0x4380u : 0x3F80u;
    return bad ? k : 0u;
}

template <int NB>
__device__ __forceinline__ uint4 v_operand(uint32_t vbase, int b, int kc) {
    // keys 16 kc + 4 h to + 3 and 8 further of the lane's channel in block b
    using L = Lds<NB>;
    const uint32_t at = (vbase ^ (uint32_t)(b * 64)) + kc * 16 * L::kRow;
    const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_u8*)(uintptr_t)at));
    const uint2 y = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_u8*)(uintptr_t)(at + 8 * L::kRow)));
    return make_uint4(x.x, x.y, y.x, y.y);
}

// A tile of 64 keys from key0 on: kb, vb the lane's read addresses in this tile's buffers.
template <int NC, int MOD, bool MASK>
__device__ __forceinline__ void step(Rows<NC, MOD>& w, int key0, uint32_t kb, uint32_t vb) {
    constexpr int NB = Rows<NC, MOD>::NB;
    using L = Lds<NB>;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    f32x16 s[2];
    __builtin_amdgcn_s_setprio(1);   // the other wave's weights wait for these products, not these for them
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        bf16x8 k[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            k[c] = *(lds_bf16x8*)(lds_u8*)(uintptr_t)((kb ^ (uint32_t)(c * 32)) + u * 32 * L::kRow);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) s[u] = mfma32(k[c], w.Q[c], s[u]);
    }
    // the first half of V is on its way while the weights are formed
    uint4 v[2][NB];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int b = 0; b < NB; ++b) v[c][b] = v_operand<NB>(vb, b, c);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (MASK || MOD != kPlain) w.template score<MASK>(s[u], key0 + 32 * u, h);
    // the weights against the maximum so far, and this half's sum of them
    const float unit = MOD == kPlain ? w.c0 : 1.f;
    uint4 P[4];
    auto weigh = [&]() {
        const float base = w.m == -INFINITY ? 0.f : -w.m * unit;   // no key yet: all weights are 0
        const bf16x2 ones{(__bf16)1.f, (__bf16)1.f};
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 8 * (c & 1) + 2 * j;
                e[j] = pack_bf16(__builtin_amdgcn_exp2f(fmaf(s[c >> 1][i], unit, base)),
                                 __builtin_amdgcn_exp2f(fmaf(s[c >> 1][i + 1], unit, base)));
                sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, e[j]), ones, sum, false);
            }
            P[c] = make_uint4(e[0], e[1], e[2], e[3]);
        }
        return sum;
    };
    // brings rows that need it, or whose maximum grew by more than `by`, to the maximum with this tile's
    // (the others stay as they are: a row's result does not depend on the rows beside it)
    auto grow = [&](bool need, float by) {
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(top, s[u][i]);
        top = __builtin_elementwise_maximum(w.m, both_max(top));
        need = need || (top - w.m) * unit > by;
        if (!__any(need)) return;
        const float keep = !need || top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((w.m - top) * unit);
        w.m = need ? top : w.m;
        w.l *= keep;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) w.O[b][i] *= keep;
    };
    float sum;
    if constexpr ((MOD & kBias) != 0) {
        grow(false, kGrow);
        sum = weigh();
    } else {
        sum = weigh();
        const bool need = !(sum < kMost) || w.m == -INFINITY;
        if (__any(need)) {
            const int other = __shfl_xor((int)need, 32, kWave);   // the row's other half
            grow(need || other != 0, INFINITY);
            sum = weigh();
        }
    }
    w.l += sum;
    // values that are not finite, found as what is not 0 after a product with 0: in a masked tile they
    // are multiplied as 0, and who sees them is looked after below
    bool bad = false;
    if constexpr (MASK) {
        const bf16x2 zeros{(__bf16)0.f, (__bf16)0.f};
        float z = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 x = c < 2 ? v[c][b] : v_operand<NB>(vb, b, c);
                z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x.x), zeros, z, false);
                z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x.y), zeros, z, false);
                z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x.z), zeros, z, false);
                z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x.w), zeros, z, false);
            }
        bad = __any(z != z);
        if (bad) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b) v[c][b] = finite_only(v[c][b]);
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint4 next[2][NB];
        if (half == 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b) next[c][b] = v_operand<NB>(vb, b, c + 2);
            if (MASK && bad) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int b = 0; b < NB; ++b) next[c][b] = finite_only(next[c][b]);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b) w.O[b] = mfma32(as_bf16x8(v[c][b]), as_bf16x8(P[2 * half + c]), w.O[b]);
        if (half == 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b) v[c][b] = next[c][b];
        }
    }
    if constexpr (MASK) {
        // who sees how many infinities, minus infinities and NaN (at most 64 of each: exact in fp32)
        if (bad) {
            uint4 one[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + 16 * c + 8 * (j >> 1) + 4 * h + 2 * (j & 1);
                    e[j] = (key < w.limit ? 0x3F80u : 0u) | (key + 1 < w.limit ? 0x3F800000u : 0u);
                }
                one[c] = make_uint4(e[0], e[1], e[2], e[3]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x16 n;
#pragma unroll
                for (int i = 0; i < 16; ++i) n[i] = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 x = v_operand<NB>(vb, b, c);
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                    uint32_t e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = kind16(xw[j] & 0xFFFFu) | kind16(xw[j] >> 16) << 16;
                    n = mfma32(as_bf16x8(make_uint4(e[0], e[1], e[2], e[3])), as_bf16x8(one[c]), n);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int k = (int)n[i];
                    const bool up = (k & 0xFF) != 0, down = (k & 0xFF00) != 0;
                    w.O[b][i] += k >= 1 << 16 || (up && down) ? NAN : up ? INFINITY : down ? -INFINITY : 0.f;
                }
            }
        }
    }
}

// in the place of a row's sum: of the first part, its result is written; this part has no keys and no O
constexpr float kDone = -1.f, kNone = -2.f;

// 1 / l for a row's sum l and maximum m.  A row that sees no key, or only scores of minus infinity, gives zeros; one
// whose maximum left the range when multiplied by scale log2 e has lost its weights, and is no number.
__device__ __forceinline__ float inverse(float l, float m) { return l == 0.f && m == -INFINITY ? 0.f : 1.f / l; }

// Where a split's O, maximum and sum of row (position m, head h) stand in the workspace.
__device__ __forceinline__ int64_t part_row(const AttentionArgs& a, int split, int64_t m, int h) {
    return ((int64_t)split * a.Mq + m) * a.H + h;
}

// SHARE: waves that share rows, each taking every SHARE-th tile of keys.
template <int NC, int MOD, int SHARE>
__global__ __launch_bounds__(kThreads, 2 / SHARE) void attention_kernel(AttentionArgs a) {
    constexpr int NB = Rows<NC, MOD>::NB, ROWS = kRows / SHARE;
    using L = Lds<NB>;
    constexpr int kBuf = SHARE * 2 * L::kTile;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kBuf];   // K, V of a tile, and of the next
    const int lane = threadIdx.x & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rep = a.H / a.G, D = a.D;

    // Consecutive workgroups go to the 8 XCDs in turn, which each get runs of a kv head's tiles.  With
    // several segments, and kv heads in eights, an XCD goes through its heads' tiles in step, so that
    // the longest of all heads start first (1024 rows each over 77, 300, 0 and 128 keys, 16 heads: 16.0
    // -> 13.0 us).  One segment's heads follow one another: without a mask its tiles are alike (4608 rows, 24 heads:
    // 252 us, in step 254); with a causal one they are not, and in step would serve many heads better (4608 rows, 24
    // heads 153 us, in step 128; 4096 rows, 16 heads 101 and 95; 2048 rows, 8 heads 28.1 and 28.2).
    // Parts of a tile are neighbours where there are few rows, else all first parts come before all second
    // ones: those that a tile has no keys for end at once, and among the others every second place of a
    // CU stayed empty (4 x 1024 rows of 4 heads with none cut in two: 55 us, so 28; 5 requests of 50 to 1400
    // rows, 4 heads: 25.1 -> 22.1).
    const int items = a.tiles * a.G;
    int split = a.parts_last ? (int)blockIdx.x / items : 0, j = (int)blockIdx.x - split * items, g, tile;
    const int xcd = j & 7;
    j >>= 3;
    const int runs = a.parts_last ? 1 : a.splits;
    const bool in_step = a.n > 1 && a.G % 8 == 0;
    if (!in_step) {
        const int total = items * runs, lo = total >> 3, more = total & 7;
        j += xcd * lo + min(xcd, more);
    }
    if (runs > 1) {
        split = j % runs;
        j /= runs;
    }
    if (in_step) {
        tile = j / (a.G / 8);
        g = (xcd - tile) * (a.G / 8) + j;
    } else {
        g = j / a.tiles;
        tile = j - g * a.tiles;
    }
    const Tile t = find_tile<ROWS>(a, rep, tile);
    if (t.seg < 0) return;
    const int klen = t.keys, rows = min(ROWS, t.len * rep - t.row0);
    const Limit limit(a, t.seg, t.len, klen);
    // the workgroup's tiles: its part of those that its last row sees
    const int tiles = (limit.of(t.row0 + rows - 1) + kKeys - 1) / kKeys;
    int per = tiles;
    bool joined = false;         // else the first part has all keys and writes the result
    if (a.splits > 1) {
        const int least = max(max(a.part, t.share), (tiles + a.splits - 1) / a.splits);
        const int parts = max((tiles + least - 1) / least, 1), alike = (tiles + parts - 1) / parts;
        // where they save more than writing and reading them costs
        joined = (float)(tiles - alike) > parts * a.part_tiles;
        if (joined) per = alike;
    }
    const int first = split * per, last = min(first + per, tiles);
    if (split > 0 && !joined) return;

    // the lane's row, or the last one's again
    const int mine = wave / SHARE * 32, turn = wave % SHARE;   // the wave's first row in the tile, its first tile of keys
    const bool active = mine < rows;
    const int row = t.row0 + min(mine + (lane & 31), rows - 1);
    const int pos = row / rep, head = g * rep + row - pos * rep;
    Rows<NC, MOD> w;
    w.m = -INFINITY;
    w.l = 0.f;
    w.limit = limit.of(row);
    w.at = pos + limit.off;
    w.slope = (MOD & kBias) != 0 ? a.slopes[head] * kLog2e : 0.f;
    w.c0 = a.scale * kLog2e;
    w.c1 = w.cz = 0.f;
    w.fine = __float_as_int(a.cap) <= __float_as_int(kFine);   // of positive floats, on the scalar unit
    if ((MOD & kCap) != 0) {
        w.c1 = fminf(a.cap * kLog2e, kLargest);
        // a tiny cap: 0 stays 0, what is not gives the cap
        w.cz = fminf(w.fine ? w.c0 * (2.f / a.cap) : 2.f * (w.c0 / a.cap), kLargest);
    }
    const uint16_t* qp = (const uint16_t*)a.q + (t.q0 + pos) * a.q_stride + (int64_t)head * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ch = 16 * c + 8 * h;
        w.Q[c] = as_bf16x8(ch < D ? *(const uint4*)(qp + ch) : make_uint4(0u, 0u, 0u, 0u));
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) w.O[b][i] = 0.f;

    // of them those that all its rows see whole; and the keys that the wave's last row sees
    const int whole = min(max(limit.of(t.row0) / kKeys, first), last);
    const int most = active ? limit.of(t.row0 + min(mine + 31, rows - 1)) : 0;

    // copies: an instruction fills 1 KB, kLanes lanes a row, kStep rows
    constexpr int kLanes = L::kSlots, kStep = 64 / kLanes;
    constexpr int kCopies = kKeys / kStep / kWaves;          // of a wave, for each of K and V
    const int crow = wave * kCopies * kStep + lane / kLanes, cslot = lane % kLanes;
    const uint32_t smem0 = (uint32_t)(uintptr_t)(lds_u8*)smem;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(smem0 + wave * kCopies * 1024);
    const uint32_t kbytes = (uint32_t)(a.k_stride * 2), vbytes = (uint32_t)(a.v_stride * 2);
    const char* kp = (const char*)a.k + ((int64_t)t.k0 * a.k_stride + (int64_t)g * D) * 2;
    const char* vp = (const char*)a.v + ((int64_t)t.k0 * a.v_stride + (int64_t)g * D) * 2;
    // where each copy reads, from the tile's first key on, and its lanes with a channel
    uint32_t koff[kCopies], voff[kCopies];
    uint64_t kon[kCopies], von;
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
        const int r = crow + j * kStep, ks = L::k_slot(r, cslot), vs = L::v_slot(r, cslot);
        koff[j] = r * kbytes + ks * 16;
        voff[j] = r * vbytes + vs * 16;
        kon[j] = __ballot(ks * 8 < D);
        von = __ballot(vs * 8 < D);      // the same for all: kStep is a multiple of the rows it goes by
    }
    static_assert(kStep % 4 == 0, "v_slot goes by the row modulo 4");
    auto copy_tile = [&](int tile, int buf) {
        const uint64_t kt = uniform_ptr(kp + (int64_t)tile * kKeys * kbytes), vt = uniform_ptr(vp + (int64_t)tile * kKeys * vbytes);
        const uint32_t to = lds0 + buf;
        const int past = tile * kKeys + kKeys - klen;        // keys past the segment's: its last again
        if (past <= 0) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                copy16(kt, koff[j], to + j * 1024, kon[j]);
                copy16(vt, voff[j], to + j * 1024 + L::kTile, von);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int r = crow + j * kStep, back = max(r - (kKeys - 1 - past), 0);
                copy16(kt, koff[j] - back * kbytes, to + j * 1024, kon[j]);
                copy16(vt, voff[j] - back * vbytes, to + j * 1024 + L::kTile, von);
            }
        }
    };
    // channels past D: zeros, which no copy overwrites
    if (D < L::kRow / 2) {
        for (int i = threadIdx.x; i < 2 * kBuf / 16; i += kThreads) *(uint4*)(smem + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    // the lane's reads of K (row lane % 32, slot h of every 2) and of V (4 lanes to a row of 16 channels)
    const uint32_t kr = (lane & 31) * L::kRow + L::k_slot(lane & 31, h) * 16;
    const int vrow = 4 * h + ((lane >> 2) & 3);
    const uint32_t vr = vrow * L::kRow + L::v_slot(vrow, ((lane >> 4) & 1) * 2 + ((lane >> 1) & 1)) * 16 + (lane & 1) * 8 + L::kTile;

    // tiles tile to tile + SHARE - 1 to buffer `buf`
    auto copy_tiles = [&](int tile, int buf) {
#pragma unroll
        for (int i = 0; i < SHARE; ++i)
            if (tile + i < last) copy_tile(tile + i, (buf * SHARE + i) * 2 * L::kTile);
    };
    copy_tiles(first, 0);
    const uint32_t own = turn * 2 * L::kTile;
    uint32_t at = smem0 + own;
    int now = first, buf = 1;
    for (; now + SHARE <= whole; now += SHARE, buf ^= 1) {
        wait_copies();
        barrier();   // these tiles are there, and the other buffer has been read
        copy_tiles(now + SHARE, buf);
        if (active) step<NC, MOD, false>(w, (now + turn) * kKeys, at + kr, at + vr);
        at = smem0 + own + buf * kBuf;
    }
    for (; now < last; now += SHARE, buf ^= 1) {
        wait_copies();
        barrier();
        copy_tiles(now + SHARE, buf);
        if (now + turn < last && (now + turn) * kKeys < most) step<NC, MOD, true>(w, (now + turn) * kKeys, at + kr, at + vr);
        at = smem0 + own + buf * kBuf;
    }
    if constexpr (SHARE > 1) {
        // the second wave's maximum, sum and O through LDS, as it holds them
        float* there = (float*)smem + wave / SHARE * (NB * 16 + 2) * kWave + lane;
        __syncthreads();
        if (turn == 1) {
            there[0] = w.m;
            there[kWave] = w.l;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) there[(2 + b * 16 + i) * kWave] = w.O[b][i];
        }
        __syncthreads();
        if (turn == 1) return;
        const float unit = MOD == kPlain ? w.c0 : 1.f, other = there[0], top = __builtin_elementwise_maximum(w.m, other);
        const float f0 = w.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((w.m - top) * unit);
        const float f1 = other == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((other - top) * unit);
        w.m = top;
        w.l = fmaf(there[kWave], f1, w.l * f0);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) w.O[b][i] = fmaf(there[(2 + b * 16 + i) * kWave], f1, w.O[b][i] * f0);
    }
    if (!active || mine + (lane & 31) >= rows) return;
    w.l = both_sum(w.l);
    if (a.splits > 1) {
        const int64_t at = part_row(a, split, t.q0 + pos, head), all = (int64_t)a.splits * a.Mq * a.H;
        float* ml = (float*)a.work + all * D + at * 2;
        if (h == 0) {
            ml[0] = MOD == kPlain ? w.m * w.c0 : w.m;
            ml[1] = !joined ? kDone : first < last ? w.l : kNone;
        }
        if (joined && first < last) {
            float* o = (float*)a.work + at * D;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int ch = 32 * b + 2 * i + 4 * h;
                    if (ch < D) *(float4*)(o + ch) = make_float4(w.O[b][i], w.O[b][i + 1], w.O[b][i + 2], w.O[b][i + 3]);
                }
        }
        if (joined) return;
    }
    const float inv = inverse(w.l, w.m);
    uint16_t* op = (uint16_t*)a.out + (t.q0 + pos) * a.out_stride + (int64_t)head * D;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int ch = 32 * b + 2 * i + 4 * h;
            if (ch < D)
                *(uint2*)(op + ch) = make_uint2(pack_bf16(w.O[b][i] * inv, w.O[b][i + 1] * inv),
                                                pack_bf16(w.O[b][i + 2] * inv, w.O[b][i + 3] * inv));
        }
}

// Joins the parts of rows (position, head), PER waves a row: each takes every PER-th part in their
// order, then the waves' sums are added in theirs.  Lane: part `lane`'s maximum and sum, and channels
// 2 lane, 2 lane + 1.  Rows between the first offset and the last are the segments'.
template <int PER>   // 1 or kWaves
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionArgs a) {
    __shared__ float2 sums[kWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t all = a.Mq * a.H, r = std::min((int64_t)blockIdx.x * (kWaves / PER) + wave / PER, all - 1);
    const int64_t m = r / a.H, head = r - m * a.H;
    const float* o = (const float*)a.work + r * a.D;
    const float2* ml = (const float2*)((const float*)a.work + all * a.splits * a.D) + r;
    const float2 mine = lane < a.splits ? ml[all * lane] : make_float2(-INFINITY, kNone);
    const bool live = m >= a.q_start[0] && m < a.q_start[a.n] &&
                      __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(mine.y))) != kDone;
    if (!live) return;                     // all of a row's waves
    float top = mine.x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = __builtin_elementwise_maximum(top, __shfl_xor(top, d, kWave));
    const float f = mine.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mine.x - top);
    float l = mine.y * f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d, kWave);
    // those with keys, the first ones; also where a part's weights are 0 against the others', for its O may
    // be no number
    const int parts = __popcll(__ballot(mine.y != kNone));
    float2 sum = make_float2(0.f, 0.f);
    if (2 * lane < a.D) {
        for (int s = wave % PER; s < parts; s += 4 * PER) {   // four loads in flight
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = *(const float2*)(o + all * min(s + u * PER, parts - 1) * a.D + 2 * lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = s + u * PER < parts;
                const float g = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), min(s + u * PER, parts - 1)));
                sum.x = fmaf(in ? v[u].x : 0.f, in ? g : 0.f, sum.x);
                sum.y = fmaf(in ? v[u].y : 0.f, in ? g : 0.f, sum.y);
            }
        }
    }
    if constexpr (PER > 1) {
        sums[wave][lane] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 1; w < PER; ++w) {
            sum.x += sums[wave / PER * PER + w][lane].x;
            sum.y += sums[wave / PER * PER + w][lane].y;
        }
    }
    if (wave % PER > 0 || 2 * lane >= a.D) return;
    const float inv = inverse(l, top);
    *(uint32_t*)((uint16_t*)a.out + m * a.out_stride + head * a.D + 2 * lane) = pack_bf16(sum.x * inv, sum.y * inv);
}

// The most tiles that any cut of Mq positions into n segments can need.
int64_t max_tiles(int64_t Mq, int rep, int n, int rows = kRows) {
    return std::min(Mq * ((rep + rows - 1) / rows), (Mq * rep + (int64_t)n * (rows - 1)) / rows);
}

// How a row tile's keys are cut: into `most` parts, of `part` key tiles or more.
struct Split {
    int most, part;
    float cost;   // of a part's O, in the time of a tile of keys
    int last;     // parts_last
};
// Where row tiles leave CUs idle, as many parts as make the longest segment that there may be shortest: a
// tile of keys takes a workgroup about as long as below, parts another launch and their rows' fp32 O
// written and read once more.  Which are cut, and how, is settled on the GPU, where the lengths are known.
// Us, one part and several: 8 single rows over up to 8000 keys, 8 kv heads 167 and 29; one row over 8192
// keys, 8 kv heads 133 and 13; 256 rows over 8192, 8 heads 143 and 26; 5 requests of 50 to 1400 rows, 4 heads
// 30.2 and 22.0; lost where all are as long, which only the GPU knows: 4 x 1024 rows of 4 heads 23.7 and 27.8.
Split split_of(int64_t Mq, int64_t Mk, int H, int G, int D, int n) {
    const Split whole{1, 1, 0.f, 0};
    const int64_t tiles = max_tiles(Mq, H / G, n), items = tiles * G, keys = (Mk + kKeys - 1) / kKeys;
    if (items == 0 || items >= 2 * kCus || n == 0) return whole;
    const bool few = Mq * (H / G) <= tiles * 32;      // rows of a tile, on average
    // of many rows a segment's share of the keys is known better than that
    const int64_t longest = few ? keys : std::min(keys, (4 * keys + n - 1) / n);
    const double tile_us = few ? 1.1 : 0.2 + 0.225 * ((D + 31) / 32), join_us = few ? 5 : 6;
    const double part_us = (double)Mq * H * (D + 2) * 8 / 3e6;
    const bool shared = max_tiles(Mq, H / G, n, kRows / 2) * G <= kCus;    // two waves to a row (launch_attention)
    double best = (shared ? (longest + 1) / 2 : longest) * tile_us;
    int64_t parts = 1;
    const int64_t places = few && n > 1 ? 3 * kCus : 2 * kCus;   // short segments leave theirs to the longest
    for (int64_t p = 2; p <= std::min({places / items, (longest + 3) / 4, (int64_t)kWave}); ++p) {
        const double us = (longest + p - 1) / p * tile_us + join_us + p * part_us;
        if (us < best) {
            best = us;
            parts = p;
        }
    }
    if (parts == 1) return whole;
    const int64_t part = n > 1 && few ? 4 : std::max<int64_t>(4, (longest + parts - 1) / parts);
    const int64_t most = std::min({(keys + part - 1) / part, std::max(parts, 3 * kCus / items), (int64_t)kWave});
    return most <= 1 ? whole : Split{(int)most, (int)part, (float)(part_us / tile_us), n > 1 && !few};
}

template <int NC, int SHARE>
void launch(const AttentionArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)(a.tiles * (int64_t)a.G * a.splits)), block(kThreads);
    if (a.cap != 0.f && a.slopes != nullptr) hipLaunchKernelGGL((attention_kernel<NC, kBoth, SHARE>), grid, block, 0, st, a);
    else if (a.cap != 0.f) hipLaunchKernelGGL((attention_kernel<NC, kCap, SHARE>), grid, block, 0, st, a);
    else if (a.slopes != nullptr) hipLaunchKernelGGL((attention_kernel<NC, kBias, SHARE>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((attention_kernel<NC, kPlain, SHARE>), grid, block, 0, st, a);
}

}  // namespace

bool attention_fits(int64_t Mq, int H, int G, int n) {
    return max_tiles(Mq, H / G, n) * G < (int64_t)1 << 23 && Mq * H < (int64_t)1 << 25;
}

int64_t attention_workspace_bytes(int64_t Mq, int64_t Mk, int H, int G, int D, int n) {
    const int splits = split_of(Mq, Mk, H, G, D, n).most;
    return splits <= 1 ? 0 : splits * Mq * H * (D + 2) * 4;
}

void launch_attention(const AttentionArgs& in, hipStream_t st) {
    AttentionArgs a = in;
    a.tiles = (int)max_tiles(a.Mq, a.H / a.G, a.n);
    const Split split = split_of(a.Mq, a.Mk, a.H, a.G, a.D, a.n);
    a.splits = split.most;
    a.part = split.part;
    a.part_tiles = split.cost;
    a.parts_last = split.last;
    // two waves to 32 rows, each with every other tile of keys, where every CU has a workgroup at most also
    // then (us, before and so: 662 rows of 8 heads of 128 18.6 and 14.4; 1024 rows of 4 heads of 64 15.4 and 10.9;
    // 500 and 200 causal rows of 4 heads over 2 14.8 and 11.7; 1500 rows of 4 heads of 128, in parts 20.8, 23.1)
    const int64_t halves = max_tiles(a.Mq, a.H / a.G, a.n, kRows / 2);
    if (a.splits == 1 && halves * a.G <= kCus) {
        a.tiles = (int)halves;
        if (a.D <= 32) launch<2, 2>(a, st);
        else if (a.D <= 64) launch<4, 2>(a, st);
        else if (a.D <= 96) launch<6, 2>(a, st);
        else launch<8, 2>(a, st);
        return;
    }
    // no step of Q K^T without channels (16 heads of 72, 6 requests, 4916 rows: 66 us with six steps, with five 63)
    switch (std::max(2, (a.D + 15) / 16)) {
        case 2: launch<2, 1>(a, st); break;
        case 3: launch<3, 1>(a, st); break;
        case 4: launch<4, 1>(a, st); break;
        case 5: launch<5, 1>(a, st); break;
        case 6: launch<6, 1>(a, st); break;
        case 7: launch<7, 1>(a, st); break;
        default: launch<8, 1>(a, st); break;
    }
    if (a.splits > 1) {
        // a row's waves read their parts side by side; with many rows there are waves enough (2048 rows of
        // 8 heads, 2 parts: the call 33.6 us, with four waves a row 42)
        const int64_t rows = a.Mq * a.H;
        if (rows >= 4096)
            hipLaunchKernelGGL(attention_join_kernel<1>, dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kThreads), 0, st, a);
        else
            hipLaunchKernelGGL(attention_join_kernel<kWaves>, dim3((unsigned)rows), dim3(kThreads), 0, st, a);
    }
}

}  // namespace svdq
