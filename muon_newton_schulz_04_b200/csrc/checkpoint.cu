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
// Two lanes share a block (16 values each), so codes move 16 bytes a lane.  16384 x 4096 bf16
// on one B200: written in 33 us, read back in 34 (201 MB each, 6.1 and 5.9 TB/s of the 6.56
// TB/s of a copy).  What it took: no integer conversion (a quarter of the rate), no 64-bit
// division, maxima two bf16 at a time.
#include <algorithm>

#include "ckpt_format.cuh"
#include "kernels.cuh"
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int CK_THREADS = 256;
constexpr int CK_VALS = 16;         // values of a piece: half a block

// 2^n for -149 <= n <= 127
__device__ __forceinline__ float pow2f(int n) {
    return __uint_as_float(n >= -126 ? (uint32_t)(n + 127) << 23 : 1u << (n + 149));
}

// 16 values as they lie in memory: two bf16 or one fp32 a word.
template <typename T>
struct Values {
    uint32_t w[CK_VALS * sizeof(T) / 4];

    __device__ __forceinline__ void load(const T* x, int n, bool vec) {
        constexpr int WORDS = CK_VALS * sizeof(T) / 4;
        if (vec && n >= CK_VALS) {
            uint4 q[WORDS / 4];
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) q[i] = reinterpret_cast<const uint4*>(x)[i];
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                w[4 * i] = q[i].x;
                w[4 * i + 1] = q[i].y;
                w[4 * i + 2] = q[i].z;
                w[4 * i + 3] = q[i].w;
            }
        } else if (sizeof(T) == 2) {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)h[2 * i + 1] << 16 : 0u);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(x)[i] : 0u;
        }
    }
    // fp32 bits of the largest magnitude (bits of |x| order like |x|, infinities and NaN above)
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
        if (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < CK_VALS / 2; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
            m = max(m << 16, m & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int i = 0; i < CK_VALS; ++i) m = max(m, w[i % (sizeof(w) / 4)] & 0x7FFFFFFFu);
        }
        return m;
    }
    __device__ __forceinline__ float value(int i) const {
        if (sizeof(T) == 2) return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        return __uint_as_float(w[i % (sizeof(w) / 4)]);
    }
};

// Piece u of rows of per_row pieces: its row and first column.  I: an index type that holds
// the number of pieces (a 64-bit division costs as much as the rest).
template <typename I>
__device__ __forceinline__ void piece_at(I u, int per_row, size_t& row, int& col) {
    const I r = u / (I)per_row;
    row = (size_t)r;
    col = (int)(u - r * (I)per_row) * CK_VALS;
}

template <typename T, typename I>
__global__ void __launch_bounds__(CK_THREADS) ckpt_store_kernel(const T* __restrict__ x, int cols, long long xs, int ld,
                                                                I total, int vec, int8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
    pdl_trigger();
    pdl_wait();
    // total = rows * ld / 16 is even and pieces of a thread are a multiple of 32 apart: the lanes
    // of a block stay together
    const I stride = (I)gridDim.x * CK_THREADS;
    for (I u = (I)blockIdx.x * CK_THREADS + threadIdx.x; u < total; u += stride) {
        size_t row;
        int col;
        piece_at<I>(u, ld / CK_VALS, row, col);
        Values<T> v;
        v.load(x + row * xs + col, cols - col, vec != 0);
        uint32_t top = v.top();
        top = max(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
        uint32_t E;
        if (top >= 0x7F800000u) E = 255;
        // k = exponent field - 127: unit 2^(k-6) is E = k + 127
        else if (top >= 0x00800000u) E = min((top + 0x10000u) >> 23, 254u);
        else E = (top + 0x8000u) >> 23;     // subnormal: unit 2^-133 holds all but the last binary 1/256
        uint32_t w[CK_VALS / 4] = {};
        if (E != 255u) {
            // x / unit = x * 2^(133 - E) is exact; adding 1.5 * 2^23 rounds it to the nearest even integer
            // and leaves that in the low byte (a conversion runs at a quarter of the rate)
            uint32_t q[CK_VALS];
            if (E >= 6u && E < 254u) {
                const float f = pow2f(133 - (int)E);
#pragma unroll
                for (int i = 0; i < CK_VALS; ++i) q[i] = __float_as_uint(fmaf(v.value(i), f, 12582912.f));
            } else {
                // the smallest units, whose reciprocal takes two factors, and the largest one, where codes saturate
                const float f = E >= 6u ? pow2f(133 - (int)E) : pow2f(64), g = E >= 6u ? 1.f : pow2f(69 - (int)E);
#pragma unroll
                for (int i = 0; i < CK_VALS; ++i)
                    q[i] = __float_as_uint(fminf(fmaxf(v.value(i) * f * g, -127.f), 127.f) + 12582912.f);
            }
#pragma unroll
            for (int i = 0; i < CK_VALS; i += 4)
                w[i / 4] = __byte_perm(__byte_perm(q[i], q[i + 1], 0x0040), __byte_perm(q[i + 2], q[i + 3], 0x0040), 0x5410);
        }
        *reinterpret_cast<uint4*>(codes + row * ld + col) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((threadIdx.x & 1) == 0) scales[row * (ld / CKPT_BLOCK) + col / CKPT_BLOCK] = (uint8_t)E;
    }
}

template <typename T, typename I>
__global__ void __launch_bounds__(CK_THREADS) ckpt_load_kernel(const int8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int cols, int ld,
                                                               I total, T* __restrict__ x, long long xs, int vec) {
    pdl_trigger();
    pdl_wait();
    const I stride = (I)gridDim.x * CK_THREADS;
    for (I u = (I)blockIdx.x * CK_THREADS + threadIdx.x; u < total; u += stride) {
        size_t row;
        int col;
        piece_at<I>(u, ld / CK_VALS, row, col);
        const uint4 w4 = *reinterpret_cast<const uint4*>(codes + row * ld + col);
        const uint32_t E = scales[row * (ld / CKPT_BLOCK) + col / CKPT_BLOCK];
        if (col >= cols) continue;
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        T* o = x + row * xs + col;
        // (no integer conversions: they run at a quarter of the rate)
        if (sizeof(T) == 2) {
            const uint32_t pair = unit_bf16(E) * 0x10001u;
            const __nv_bfloat162 unit = *reinterpret_cast<const __nv_bfloat162*>(&pair);
            uint32_t b[CK_VALS / 2];
#pragma unroll
            for (int i = 0; i < CK_VALS / 2; ++i)
                b[i] = codes_to_bf16(__byte_perm(w[i / 2], 0, i % 2 ? 0x4342 : 0x4140), unit);
            if (vec && col + CK_VALS <= cols) {
                reinterpret_cast<uint4*>(o)[0] = make_uint4(b[0], b[1], b[2], b[3]);
                reinterpret_cast<uint4*>(o)[1] = make_uint4(b[4], b[5], b[6], b[7]);
            } else {
#pragma unroll
                for (int i = 0; i < CK_VALS; ++i)
                    if (col + i < cols) reinterpret_cast<uint16_t*>(o)[i] = (uint16_t)(b[i / 2] >> (16 * (i % 2)));
            }
        } else {
            // 2^23 + (code + 128) is a float's bit pattern
            const float unit = E == 255u ? __uint_as_float(0x7FC00000u) : pow2f((int)E - 133);
            uint32_t b[CK_VALS];
#pragma unroll
            for (int i = 0; i < CK_VALS; ++i)
                b[i] = __float_as_uint((__uint_as_float(__byte_perm(w[i / 4] ^ 0x80808080u, 0x4B000000u, 0x7540 + i % 4)) -
                                        8388736.f) * unit);
            if (vec && col + CK_VALS <= cols) {
#pragma unroll
                for (int i = 0; i < CK_VALS; i += 4)
                    reinterpret_cast<uint4*>(o)[i / 4] = make_uint4(b[i], b[i + 1], b[i + 2], b[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < CK_VALS; ++i)
                    if (col + i < cols) reinterpret_cast<uint32_t*>(o)[i] = b[i];
            }
        }
    }
}

template <typename T, typename I>
cudaError_t store(const T* x, int cols, long long xs, int ld, size_t total, int vec, int8_t* codes, uint8_t* scales, int grid,
                  cudaStream_t s) {
    return launch_pdl(ckpt_store_kernel<T, I>, dim3(grid), dim3(CK_THREADS), 0, s, x, cols, xs, ld, (I)total, vec, codes, scales);
}

template <typename T, typename I>
cudaError_t load(const int8_t* codes, const uint8_t* scales, int cols, int ld, size_t total, T* x, long long xs, int vec,
                 int grid, cudaStream_t s) {
    return launch_pdl(ckpt_load_kernel<T, I>, dim3(grid), dim3(CK_THREADS), 0, s, codes, scales, cols, ld, (I)total, x, xs, vec);
}

int ckpt_grid(size_t total, int num_sms) {
    return (int)std::min<size_t>((total + CK_THREADS - 1) / CK_THREADS, (size_t)num_sms * 64);
}

// 32-bit indexes while a thread's index, one stride past the end, stays below 2^32
bool small_index(size_t total, int grid) { return total + (size_t)grid * CK_THREADS < (1ull << 32); }

}  // namespace

cudaError_t launch_checkpoint_store(const void* x, int x_bf16, int rows, int cols, long long xs, int8_t* codes,
                                    uint8_t* scales, int num_sms, cudaStream_t s) {
    const int ld = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    const size_t total = (size_t)rows * (ld / CK_VALS);
    const int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && xs % (x_bf16 ? 8 : 4) == 0, grid = ckpt_grid(total, num_sms);
    const auto* h = static_cast<const __nv_bfloat16*>(x);
    const auto* f = static_cast<const float*>(x);
    if (small_index(total, grid))
        return x_bf16 ? store<__nv_bfloat16, uint32_t>(h, cols, xs, ld, total, vec, codes, scales, grid, s)
                      : store<float, uint32_t>(f, cols, xs, ld, total, vec, codes, scales, grid, s);
    return x_bf16 ? store<__nv_bfloat16, size_t>(h, cols, xs, ld, total, vec, codes, scales, grid, s)
                  : store<float, size_t>(f, cols, xs, ld, total, vec, codes, scales, grid, s);
}

cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* scales, int rows, int cols, void* x, int x_bf16,
                                   long long xs, int num_sms, cudaStream_t s) {
    const int ld = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    const size_t total = (size_t)rows * (ld / CK_VALS);
    const int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && xs % (x_bf16 ? 8 : 4) == 0, grid = ckpt_grid(total, num_sms);
    auto* h = static_cast<__nv_bfloat16*>(x);
    auto* f = static_cast<float*>(x);
    if (small_index(total, grid))
        return x_bf16 ? load<__nv_bfloat16, uint32_t>(codes, scales, cols, ld, total, h, xs, vec, grid, s)
                      : load<float, uint32_t>(codes, scales, cols, ld, total, f, xs, vec, grid, s);
    return x_bf16 ? load<__nv_bfloat16, size_t>(codes, scales, cols, ld, total, h, xs, vec, grid, s)
                  : load<float, size_t>(codes, scales, cols, ld, total, f, xs, vec, grid, s);
}

}  // namespace muon
