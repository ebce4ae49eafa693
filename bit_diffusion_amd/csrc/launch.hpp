// launch.hpp -- host-side launchers of the gfx950 kernels (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq {

struct QuantArgs {
    int64_t M;
    int K, r;
    int mode;       // 0 INT4 nibbles, 1 INT4 packed (packed_layout.hpp), 2 NVFP4 nibbles
    const void* x;
    const float* smooth_inv;
    const void* l1;   // [r, K] row-major; prepacked (launch_prepack_l1) in mode 1
    float S;
    void* codes;    // nibbles, or the packed activation buffer in mode 1
    void* scales;   // may be NULL in mode 1
    void* lora;
};

struct GemmArgs {
    int64_t M;
    int N, K, r;
    bool nvfp4;
    const void* acodes;
    const void* ascales;
    float Sa;
    const void* wcodes;
    const void* wscales;
    float Sw;
    const void* lora;
    const void* l2;
    const void* bias;
    int act;        // 0 none, 1 gelu-tanh
    int out_bf16;   // 0 fp32, 1 bf16
    void* out;
};

struct AwqArgs {
    int64_t M;
    int K, N;
    const void* x;
    const void* qweight;
    const void* scales;
    const void* zeros;
    const void* bias;
    int out_bf16;
    void* out;
};

struct PackedGemmArgs {
    int64_t M;
    int N, K, r;
    const void* act;   // packed activations
    const void* wgt;   // packed weights
    const void* lora;
    const void* l2;
    const void* bias;
    int act_fn;
    int out_bf16;
    void* out;
    int vec_store;     // set by the launcher
    int nfull, nsplit, gsplit;   // K split of the last round's tiles (set by the launcher)
    // the next layer's activation quantization in the epilogue (quantize_next); the tile's
    // bf16 outputs are not stored
    int quantize_next;
    int next_r;              // next layer's rank
    const float* next_si;    // [N] smoothing factors of the next layer
    const void* next_l1;     // bf16 [next_r, N] row-major, or NULL
    void* next_packed;       // the next layer's packed activation buffer (its K = N)
    float* next_scales;      // fp32 [M, N / 64] or NULL
    float* lora_work;        // fp32 [ceil(N / 192)][ceil(M / 256) * 256][next_r]: per-tile
                             // partial sums of the next layer's low-rank down-projection
    // K split (fp32 output, no activation): workspace for the splits' partial tiles, or NULL
    // (then no split)
    float* split_ws;
    int64_t split_ws_bytes;
};

struct LoraBatchArgs {
    int64_t M;
    int K, N, R;             // R: the pool's ranks, a multiple of 16 up to 128
    int n_adapters, n_segments;
    const void* x;           // bf16 [M, K]
    int64_t x_stride;
    const void* down;        // bf16 [n_adapters, R, K]
    const void* up;          // bf16 [n_adapters, N, R]
    const float* alphas;     // [n_adapters]
    const int* ranks;        // [n_adapters] or NULL (all R)
    const int* starts;       // [n_segments + 1]
    const int* ids;          // [n_segments]
    const void* base;        // [M, N] or NULL
    int64_t base_stride;
    int act;
    int bf16;                // type of base and out: 0 fp32, 1 bf16
    void* out;
    int64_t out_stride;
    void* work;              // t as MFMA operands, a set for every block of 16 rows
    int vec;                 // base and out take 16-byte accesses
    int nb, max_blocks;      // blocks of 32 ranks, and of 16 rows, in work (set by the launcher)
};

struct GroupNormArgs {
    int64_t B, rows;
    int C, groups;
    float eps;
    int x_bf16;              // 0 fp32, 1 bf16
    const void* x;           // [B rows, C]
    int64_t x_stride;
    const void* weight;      // bf16 [C] or NULL
    const void* bias;
    int mod_bf16;
    const void* mod_scale;   // [B, C] or NULL
    const void* mod_shift;
    int64_t mod_stride;
    int act;
    int out_bf16;
    void* out;
    int64_t out_stride;
    void* work;
    int vec;                 // x and out take 16-byte accesses
};

struct LayerNormArgs {
    int64_t M;
    int C, n_segments;
    float eps;
    int x_bf16;              // type of x and x_out: 0 fp32, 1 bf16
    const void* x;           // [M, C]
    int64_t x_stride;
    int y_bf16;
    const void* y;           // [M, C] or NULL
    int64_t y_stride;
    const void* weight;      // bf16 [C] or NULL
    const void* bias;
    const int* starts;       // [n_segments + 1], or NULL: all rows are segment 0
    int mod_bf16;
    const void* mod_gate;    // [n_segments, C] each, or NULL
    const void* mod_scale;
    const void* mod_shift;
    int64_t mod_stride;
    void* x_out;             // [M, C] or NULL
    int64_t x_out_stride;
    int out_bf16;
    void* out;
    int64_t out_stride;
    int vec;                 // elements of an access that every row takes: 4, 2 or 1
};

struct RotaryArgs {
    int64_t M;
    int q_heads, k_heads, D;
    int n_axes;
    int ends[4];             // pairs up to and with axis a (n_axes to 3: D / 2)
    int halves;              // pairs (i, i + D / 2) and not (2 i, 2 i + 1)
    const float* pos;        // [M, n_axes]
    int64_t pos_stride;
    const double* freqs;     // [D / 2]
    float eps;
    const void* q_weight;    // bf16 [D] or NULL: no norm
    const void* k_weight;
    int x_bf16;
    const void* q;           // [M, q_heads D]
    int64_t q_stride;
    const void* k;
    int64_t k_stride;
    int out_bf16;
    void* q_out;
    int64_t q_out_stride;
    void* k_out;
    int64_t k_out_stride;
    int vec;                 // rows take accesses of 8 channels (halves: 8 pairs), 16-byte aligned
    int word;                // pairs are side by side, rows aligned to a pair
};

struct AttentionArgs {
    int64_t Mq, Mk;
    int H, G, D, n;          // heads, kv heads, head dimension, segments
    float scale, cap;        // cap 0: none
    int causal;
    const int* q_start;      // [n + 1]
    const int* kv_start;
    const int* prefix;       // [n] or NULL
    const float* slopes;     // [H] or NULL
    const void* q;           // bf16 [Mq, H D]
    int64_t q_stride;
    const void* k;           // bf16 [Mk, G D]
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    void* out;               // bf16 [Mq, H D]
    int64_t out_stride;
    void* work;
    int tiles;               // the most row tiles (set by the launcher, as what follows)
    int splits, part;        // the most parts of a row tile's keys, and the least key tiles of one
    int parts_last;          // all first parts in front of all second ones
    float part_tiles;        // cost of writing and reading a part, in key tiles
};

// Largest workspace the K split of svdq_gemm_w4a4_packed uses (its split count is capped so
// that the partial tiles fit).
constexpr int64_t kSplitWorkspaceMax = (int64_t)64 << 20;

void launch_quantize_act(const QuantArgs& a, hipStream_t st);
void launch_gemm_int4(const GemmArgs& a, hipStream_t st);
void launch_gemm_nvfp4(const GemmArgs& a, hipStream_t st);
void launch_awq_gemv(const AwqArgs& a, hipStream_t st);

void launch_prepack_wgt(int N, int K, const void* wcodes, const void* wscales, void* out,
                        hipStream_t st);
void launch_merge_lora(int K, int N, int r, int rl, int ro, const void* l1, const void* l2,
                       const void* down, const void* up, float alpha, void* l1o, void* l2o,
                       hipStream_t st);
int64_t prepacked_l1_bytes(int r, int K);
void launch_prepack_l1(int r, int K, const void* l1, void* out, hipStream_t st);
void launch_pack_act(int64_t M, int K, const void* acodes, const void* ascales, void* out,
                     hipStream_t st);
bool gemm_w4a4_fp6_init();
void launch_gemm_w4a4_fp6(const PackedGemmArgs& a, hipStream_t st);
int64_t split_workspace_bytes(int64_t M, int N, int K, int act_fn, int out_bf16);
int cu_count();   // compute units of the current device (cached per device)
// device address and size of the K-split scratch array of the current device (noalloc.hip)
hipError_t noalloc_scratch(void** ptr, int64_t* bytes);

// measurement kernels (peaks.hip)
int64_t launch_mfma_peak(int kind, int iters, float* out, hipStream_t st);
void launch_copy(const void* src, void* dst, int64_t bytes, hipStream_t st);
void launch_read(const void* src, int64_t bytes, void* out, hipStream_t st);
int64_t quantize_next_workspace_bytes(int64_t M, int N, int next_r);

// adapters of many requests (lora_batch.hip)
bool lora_batch_fits(int64_t M, int N, int n_segments);   // one launch's grid
int64_t lora_batch_workspace_bytes(int64_t M, int R, int n_segments);
void launch_lora_batch(const LoraBatchArgs& a, hipStream_t st);

// group normalisation of channels-last images (group_norm.hip)
int64_t group_norm_workspace_bytes(int64_t B, int64_t rows, int C, int groups);
void launch_group_norm(const GroupNormArgs& a, hipStream_t st);

// residual, layer norm and modulation of packed rows (layer_norm.hip)
void launch_layer_norm(const LayerNormArgs& a, hipStream_t st);

// rotary positions with several axes (rotary.hip)
void launch_rotary(const RotaryArgs& a, hipStream_t st);

// attention of packed requests (attention.hip)
bool attention_fits(int64_t Mq, int H, int G, int n);   // one launch's grid
int64_t attention_workspace_bytes(int64_t Mq, int64_t Mk, int H, int G, int D, int n);
void launch_attention(const AttentionArgs& a, hipStream_t st);

// offline weight quantization (weights.hip)
void launch_calib_absmax(int64_t M, int K, const void* x, float* absmax, hipStream_t st);
void launch_smoothing_factors(int N, int K, const float* w, const float* x_absmax, float* w_absmax,
                              float* smooth_inv, hipStream_t st);
void launch_quantize_residual(int N, int K, int r, bool nvfp4, const float* w,
                              const float* smooth_inv, const void* l1, const void* l2, void* codes,
                              void* scales, float* global_scale, hipStream_t st);

// top-r factorization of the smoothed weight (lowrank.hip)
int64_t lowrank_workspace_bytes(int N, int K);
void launch_lowrank_factors(int N, int K, int r, int b, int iters, const float* w,
                            const float* smooth_inv, const float* omega, void* l1, void* l2,
                            float* sigma_out, void* workspace, hipStream_t st);

}  // namespace svdq
