// attention.cu -- gradients of packed causal attention with grouped heads: one
// warp per row.  Lanes hold 32 keys (or queries) while logits are formed and head_dim
// elements while rows are summed.
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int WARPS = 4;
constexpr int DMAX = 128;

struct Seq { int q0, q1, k0, k1; };

// The sequence whose rows [cu[s], cu[s+1]) hold `row`, or -1.
__device__ __forceinline__ int find_seq(const int* cu, int n, int row) {
    for (int s = 0; s < n; ++s)
        if (row >= cu[s] && row < cu[s + 1]) return s;
    return -1;
}

__device__ __forceinline__ bool load_seq(const AttnParams& p, int s, Seq& q) {
    q = Seq{p.cu_q[s], p.cu_q[s + 1], p.cu_k[s], p.cu_k[s + 1]};
    const bool ok = q.q0 >= 0 && q.q0 <= q.q1 && q.q1 <= p.total_q && q.k0 >= 0 && q.k0 <= q.k1 && q.k1 <= p.total_k;
    if (!ok) atomicCAS(p.err, 0, ERR_SEQLENS);
    return ok;
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ float dot(const float* a, const __nv_bfloat16* b, int d) {
    float s = 0.f;
    for (int i = 0; i < d; ++i) s = fmaf(a[i], __bfloat162float(b[i]), s);
    return s;
}

__device__ __forceinline__ const __nv_bfloat16* at(const HeadView& v, int row, int head) {
    return v.p + row * v.rs + head * v.hs;
}

__global__ void __launch_bounds__(32 * WARPS) attention_dq_rows(const AttnParams p) {
    __shared__ float qs[WARPS][DMAX], gs[WARPS][DMAX];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = blockIdx.x * WARPS + w, h = blockIdx.y, hk = h / p.group;
    if (row >= p.total_q) return;
    const int s = find_seq(p.cu_q, p.n_seqs, row);
    Seq sq;
    if (s < 0 || !load_seq(p, s, sq)) return;
    float delta = 0.f;
    for (int i = lane; i < p.d; i += 32) {
        qs[w][i] = __bfloat162float(at(p.q, row, h)[i]);
        gs[w][i] = __bfloat162float(at(p.go, row, h)[i]);
        delta = fmaf(gs[w][i], __bfloat162float(at(p.out, row, h)[i]), delta);
    }
    delta = warp_sum(delta);
    __syncwarp();
    const float lse = p.lse[(size_t)h * p.total_q + row];
    if (lane == 0) p.delta[(size_t)h * p.total_q + row] = delta;
    const int last = min(row - sq.q0 + (sq.k1 - sq.k0) - (sq.q1 - sq.q0), sq.k1 - sq.k0 - 1);
    float o[DMAX / 32] = {};
    for (int j0 = 0; j0 <= last; j0 += 32) {
        const int j = j0 + lane;
        float ds = 0.f;
        if (j <= last) {
            const float pr = expf(p.scale * dot(qs[w], at(p.k, sq.k0 + j, hk), p.d) - lse);
            ds = pr * (dot(gs[w], at(p.v, sq.k0 + j, hk), p.d) - delta);
        }
        for (int jj = 0; jj < 32 && j0 + jj <= last; ++jj) {
            const float x = __shfl_sync(~0u, ds, jj);
            for (int c = 0; c < DMAX / 32; ++c)
                if (lane + 32 * c < p.d) o[c] = fmaf(x, __bfloat162float(at(p.k, sq.k0 + j0 + jj, hk)[lane + 32 * c]), o[c]);
        }
    }
    for (int c = 0; c < DMAX / 32; ++c)
        if (lane + 32 * c < p.d) p.dq.p[row * p.dq.rs + h * p.dq.hs + lane + 32 * c] = __float2bfloat16_rn(p.scale * o[c]);
}

__global__ void __launch_bounds__(32 * WARPS) attention_dkv_rows(const AttnParams p) {
    __shared__ float ks[WARPS][DMAX], vs[WARPS][DMAX];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = blockIdx.x * WARPS + w, hk = blockIdx.y;
    if (row >= p.total_k) return;
    const int s = find_seq(p.cu_k, p.n_seqs, row);
    Seq sq;
    if (s < 0 || !load_seq(p, s, sq)) return;
    for (int i = lane; i < p.d; i += 32) {
        ks[w][i] = __bfloat162float(at(p.k, row, hk)[i]);
        vs[w][i] = __bfloat162float(at(p.v, row, hk)[i]);
    }
    __syncwarp();
    const int lq = sq.q1 - sq.q0, first = max(0, row - sq.k0 - (sq.k1 - sq.k0) + lq);
    float dk[DMAX / 32] = {}, dv[DMAX / 32] = {};
    for (int h = hk * p.group; h < (hk + 1) * p.group; ++h)
        for (int i0 = first; i0 < lq; i0 += 32) {
            const int i = i0 + lane, r = sq.q0 + i;
            float pr = 0.f, ds = 0.f;
            if (i < lq) {
                pr = expf(p.scale * dot(ks[w], at(p.q, r, h), p.d) - p.lse[(size_t)h * p.total_q + r]);
                ds = pr * (dot(vs[w], at(p.go, r, h), p.d) - p.delta[(size_t)h * p.total_q + r]);
            }
            for (int ii = 0; ii < 32 && i0 + ii < lq; ++ii) {
                const float a = __shfl_sync(~0u, pr, ii), b = __shfl_sync(~0u, ds, ii);
                for (int c = 0; c < DMAX / 32; ++c)
                    if (lane + 32 * c < p.d) {
                        dv[c] = fmaf(a, __bfloat162float(at(p.go, sq.q0 + i0 + ii, h)[lane + 32 * c]), dv[c]);
                        dk[c] = fmaf(b, __bfloat162float(at(p.q, sq.q0 + i0 + ii, h)[lane + 32 * c]), dk[c]);
                    }
            }
        }
    for (int c = 0; c < DMAX / 32; ++c)
        if (lane + 32 * c < p.d) {
            p.dk.p[row * p.dk.rs + hk * p.dk.hs + lane + 32 * c] = __float2bfloat16_rn(p.scale * dk[c]);
            p.dv.p[row * p.dv.rs + hk * p.dv.hs + lane + 32 * c] = __float2bfloat16_rn(dv[c]);
        }
}

}  // namespace

cudaError_t launch_attention_backward(const AttnParams& p, cudaStream_t s) {
    if (p.n_seqs == 0) return cudaSuccess;
    if (p.total_q > 0) attention_dq_rows<<<dim3((p.total_q + WARPS - 1) / WARPS, p.hq), 32 * WARPS, 0, s>>>(p);
    if (p.total_k > 0) attention_dkv_rows<<<dim3((p.total_k + WARPS - 1) / WARPS, p.hk), 32 * WARPS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace muon
