// checkpoint.cu -- activations kept in 8 bits: blocks of 32 values share a power-of-two
// unit 2^(E - 133), codes are int8.
//
// E is the smallest E >= 0 with rint(max|x| / unit) <= 127, i.e. max|x| < 127.5 * unit.
// With max|x| = m * 2^k, 1 <= m < 2, 127.5 = 1.9921875 * 2^6 gives unit 2^(k-6) when
// m < 1.9921875 and 2^(k-5) otherwise: E comes from the bits of max|x| by one addition
// (0x10000 carries into the exponent exactly from the mantissa of 1.9921875 on), and
// x / unit is exact, so a code has one rounding.
//
// Bound by memory: store reads 2 or 4 bytes and writes 33/32 a value, load the reverse.
// Four lanes share a block (8 values each), so a warp covers 256 consecutive values of a
// row with 16-byte accesses.
#include <algorithm>

#include "kernels.cuh"
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int CK_THREADS = 256;
constexpr int CK_VALS = 8;          // values of one thread

// 2^n for -149 <= n <= 127
__device__ __forceinline__ float pow2f(int n) {
    return __uint_as_float(n >= -126 ? (uint32_t)(n + 127) << 23 : 1u << (n + 149));
}

template <typename T>
__device__ __forceinline__ void load8(const T* x, int n, bool vec, float (&v)[CK_VALS]) {
    if (vec && n >= CK_VALS) {
        if (sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(x);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        } else {
            const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < CK_VALS; ++i) v[i] = i < n ? (float)x[i] : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(CK_THREADS) ckpt_store_kernel(const T* __restrict__ x, int cols, long long xs, int ld,
                                                                size_t total, int vec, int8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
    pdl_trigger();
    pdl_wait();
    // total = rows * ld / 8 eighths of blocks, a multiple of 4: the lanes of a block stay together
    const size_t stride = (size_t)gridDim.x * CK_THREADS;
    for (size_t u = (size_t)blockIdx.x * CK_THREADS + threadIdx.x; u < total; u += stride) {
        const int per_row = ld / CK_VALS;
        const size_t row = u / per_row;
        const int c = (int)(u - row * per_row) * CK_VALS;
        float v[CK_VALS];
        load8(x + row * xs + c, cols - c, vec != 0, v);
        uint32_t top = 0;               // bits of |x| order like |x|, with infinities and NaN above
#pragma unroll
        for (int i = 0; i < CK_VALS; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const unsigned quad = 0xFu << (threadIdx.x & 28);
        top = max(top, __shfl_xor_sync(quad, top, 1));
        top = max(top, __shfl_xor_sync(quad, top, 2));
        uint32_t E;
        if (top >= 0x7F800000u) E = 255;
        else if (top >= 0x00800000u) E = min((top + 0x10000u) >> 23, 254u);
        else E = (top + 0x8000u) >> 23;     // subnormal: unit 2^-133 holds all but the last binary 1/256
        uint32_t w[2] = {0, 0};
        if (E != 255u) {
            // 1 / unit = 2^(133 - E) in two exact factors
            const int n = 133 - (int)E;
            const float f0 = pow2f(n / 2), f1 = pow2f(n - n / 2);
#pragma unroll
            for (int i = 0; i < CK_VALS; ++i) {
                const int q = max(-127, min(127, __float2int_rn(v[i] * f0 * f1)));
                w[i / 4] |= (uint32_t)(q & 0xFF) << (8 * (i % 4));
            }
        }
        *reinterpret_cast<uint2*>(codes + row * ld + c) = make_uint2(w[0], w[1]);
        if ((threadIdx.x & 3) == 0) scales[row * (ld / CKPT_BLOCK) + c / CKPT_BLOCK] = (uint8_t)E;
    }
}

template <typename T>
__global__ void __launch_bounds__(CK_THREADS) ckpt_load_kernel(const int8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int cols, int ld,
                                                               size_t total, T* __restrict__ x, long long xs, int vec) {
    pdl_trigger();
    pdl_wait();
    const size_t stride = (size_t)gridDim.x * CK_THREADS;
    for (size_t u = (size_t)blockIdx.x * CK_THREADS + threadIdx.x; u < total; u += stride) {
        const int per_row = ld / CK_VALS;
        const size_t row = u / per_row;
        const int c = (int)(u - row * per_row) * CK_VALS;
        if (c >= cols) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(codes + row * ld + c);
        const uint32_t E = scales[row * (ld / CKPT_BLOCK) + c / CKPT_BLOCK];
        const float unit = E == 255u ? __uint_as_float(0x7FC00000u) : pow2f((int)E - 133);
        float v[CK_VALS];
#pragma unroll
        for (int i = 0; i < CK_VALS; ++i)
            v[i] = (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i % 4))) * unit;
        T* o = x + row * xs + c;
        if (vec && c + CK_VALS <= cols) {
            if (sizeof(T) == 2) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    b[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(o) = make_uint4(b[0], b[1], b[2], b[3]);
            } else {
                reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        } else {
            for (int i = 0; i < CK_VALS && c + i < cols; ++i) o[i] = (T)v[i];
        }
    }
}

int ckpt_grid(size_t total, int num_sms) {
    return (int)std::min<size_t>((total + CK_THREADS - 1) / CK_THREADS, (size_t)num_sms * 16);
}

}  // namespace

cudaError_t launch_checkpoint_store(const void* x, int x_bf16, int rows, int cols, long long xs, int8_t* codes,
                                    uint8_t* scales, int num_sms, cudaStream_t s) {
    const int ld = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    const size_t total = (size_t)rows * (ld / CK_VALS);
    const int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && xs % (x_bf16 ? 8 : 4) == 0;
    const dim3 g(ckpt_grid(total, num_sms)), b(CK_THREADS);
    return x_bf16 ? launch_pdl(ckpt_store_kernel<__nv_bfloat16>, g, b, 0, s, static_cast<const __nv_bfloat16*>(x), cols,
                               xs, ld, total, vec, codes, scales)
                  : launch_pdl(ckpt_store_kernel<float>, g, b, 0, s, static_cast<const float*>(x), cols, xs, ld, total,
                               vec, codes, scales);
}

cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* scales, int rows, int cols, void* x, int x_bf16,
                                   long long xs, int num_sms, cudaStream_t s) {
    const int ld = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    const size_t total = (size_t)rows * (ld / CK_VALS);
    const int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && xs % (x_bf16 ? 8 : 4) == 0;
    const dim3 g(ckpt_grid(total, num_sms)), b(CK_THREADS);
    return x_bf16 ? launch_pdl(ckpt_load_kernel<__nv_bfloat16>, g, b, 0, s, codes, scales, cols, ld, total,
                               static_cast<__nv_bfloat16*>(x), xs, vec)
                  : launch_pdl(ckpt_load_kernel<float>, g, b, 0, s, codes, scales, cols, ld, total,
                               static_cast<float*>(x), xs, vec);
}

}  // namespace muon
