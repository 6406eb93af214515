// model_ops.cuh -- descriptors and launchers of the operators between a layer's
// forward pass and its Muon step: packed causal attention and its gradients, 8-bit
// activation checkpoints, and the weight gradient taken from them.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace muon {

// element d of head h of row r: p[r * rs + h * hs + d]
struct HeadView {
    __nv_bfloat16* p;
    long long rs, hs;
};

struct AttnParams {
    HeadView q, k, v, out;        // forward operands (out: written by the forward, read by the backward)
    HeadView go, dq, dk, dv;      // backward only
    float* lse;                   // [hq][total_q]
    float* max_logits;            // forward only, may be nullptr
    float* delta;                 // backward scratch [hq][total_q]: D_i = grad_out_i . O_i
    const int* cu_q;
    const int* cu_k;
    int n_seqs, hq, hk, group, d;
    int total_q, total_k;
    float scale;
    int* err;
};

// device error word: a sequence whose cu_seqlens are out of range
constexpr int ERR_SEQLENS = 0x301;

// Tensor maps over [rows][heads][head_dim] arrays, boxes of AT_FWD_BOX or AT_BWD_BOX rows x
// 64 columns of one head, 128-byte swizzle, zeros outside (go: backward only).
constexpr int AT_FWD_BOX = 128, AT_BWD_BOX = 64;
struct HeadMaps {
    CUtensorMap q, k, v, go;
};

cudaError_t launch_attention(const AttnParams& p, const HeadMaps& m, cudaStream_t s);
cudaError_t launch_attention_backward(const AttnParams& p, const HeadMaps& m, cudaStream_t s);

// Outputs whose rows of no sequence are to be filled: vectors of heads, or (lse set) one float
// a row and head.
struct FillParams {
    struct Rows {
        HeadView x;
        float* lse;
        const int* cu;
        int heads, total;
    } array[3];
    int n, n_seqs, d;
};
cudaError_t launch_attention_fill(const FillParams& p, cudaStream_t s);

constexpr int CKPT_BLOCK = 32;    // values that share a scale byte

cudaError_t launch_checkpoint_store(const void* x, int x_bf16, int rows, int cols, long long xs, int8_t* codes,
                                    uint8_t* scales, int num_sms, cudaStream_t s);
cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* scales, int rows, int cols, void* x, int x_bf16,
                                   long long xs, int num_sms, cudaStream_t s);

// Split of a weight gradient over the SM pairs, and the workspace that it needs.
struct WgradPlan {
    int kblocks;              // blocks of 64 tokens
    int tiles_n;              // 256-column tiles of G
    int whole;                // first tiles, computed by one cluster each
    int rest, splits;         // the others, split along the tokens
    size_t partial_bytes;     // fp32 partial sums of the split tiles
    int dy_ld;                // row length of the copy of a dy that TMA cannot read
    size_t dy_bytes;          // its size, 0: dy is read where it is
};
WgradPlan weight_grad_plan(int tokens, int rows, int cols, bool dy_aligned);

struct WgradParams {
    const __nv_bfloat16* dy;
    long long dys;
    const int8_t* codes;
    const uint8_t* scales;
    void* g;
    int g_bf16, accumulate, vec;
    int tokens, rows, cols, ld;
    int kblocks, tiles_n, whole, rest, splits;
    float* partial;
    int* err;
};
cudaError_t launch_weight_grad_repack(const WgradParams& p, const WgradPlan& w, __nv_bfloat16* out, cudaStream_t s);
// dy (tokens x rows, bf16): boxes of 64 tokens x 64 columns, 128-byte swizzle; the codes
// (tokens x ld bytes): boxes of 64 tokens x 128 columns.
struct WgradMaps {
    CUtensorMap dy, codes;
};
cudaError_t launch_weight_grad(const WgradParams& p, const WgradMaps& maps, cudaStream_t s);

cudaError_t launch_qk_clip_grouped(float* wq, float* wk, const float* max_logits, int n_heads, int n_kv_heads,
                                   int head_dim, int cols, float tau, cudaStream_t s);

}  // namespace muon
