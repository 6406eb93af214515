// weight_grad.cu -- G (+)= dy^T x^ with x^ read from an 8-bit checkpoint: one output
// element per thread, 16 tokens at a time through shared memory.
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int T = 16;

__device__ __forceinline__ float ckpt_unit(uint32_t e) {
    // 2^(E - 133): normal from E = 7, a power of two among the subnormals below, NaN at 255
    return __uint_as_float(e == 255u ? 0x7FC00000u : e >= 7u ? (e - 6u) << 23 : 0x10000u << e);
}

__global__ void __launch_bounds__(T * T) weight_grad_simple(const WgradParams p) {
    __shared__ float a[T][T + 1], b[T][T + 1];
    const int tx = threadIdx.x % T, ty = threadIdx.x / T;
    const int r = blockIdx.y * T + ty, c = blockIdx.x * T + tx;
    float acc = 0.f;
    for (int t0 = 0; t0 < p.tokens; t0 += T) {
        const int t = t0 + ty, rr = blockIdx.y * T + tx;
        a[ty][tx] = t < p.tokens && rr < p.rows ? __bfloat162float(p.dy[(size_t)t * p.dys + rr]) : 0.f;
        b[ty][tx] = t < p.tokens && c < p.cols
                        ? p.codes[(size_t)t * p.ld + c] * ckpt_unit(p.scales[((size_t)t * p.ld + c) / CKPT_BLOCK]) : 0.f;
        __syncthreads();
        for (int k = 0; k < T; ++k) acc = fmaf(a[k][ty], b[k][tx], acc);
        __syncthreads();
    }
    if (r >= p.rows || c >= p.cols) return;
    const size_t o = (size_t)r * p.cols + c;
    if (p.g_bf16) {
        __nv_bfloat16* g = static_cast<__nv_bfloat16*>(p.g) + o;
        *g = __float2bfloat16_rn(acc + (p.accumulate ? __bfloat162float(*g) : 0.f));
    } else {
        float* g = static_cast<float*>(p.g) + o;
        *g = acc + (p.accumulate ? *g : 0.f);
    }
}

}  // namespace

cudaError_t launch_weight_grad(const WgradParams& p, cudaStream_t s) {
    weight_grad_simple<<<dim3((p.cols + T - 1) / T, (p.rows + T - 1) / T), T * T, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace muon
