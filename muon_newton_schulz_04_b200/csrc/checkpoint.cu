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
// Two lanes share a block (16 values each), so codes move 16 bytes a lane; where the rows of x
// do not start on 16-byte addresses, a warp takes blocks, one value of each a lane.  16384 x
// 4096 bf16 on one B200: written in 33 us, read back in 34 (201 MB each, 6.1 and 5.9 TB/s of
// the 6.56 TB/s of a copy); fp32 49 and 72 us (floor 51 each).  16384 x 3999, a value or a code
// an access: bf16 76 and 54 us (floor 30 each), fp32 73 and 69 (50).  What it took: no integer
// conversion (a quarter of the rate), no 64-bit division, maxima two bf16 at a time.
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

    __device__ __forceinline__ void load(const T* x, int n) {
        constexpr int WORDS = CK_VALS * sizeof(T) / 4;
        if (n >= CK_VALS) {
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

// E of a block whose largest magnitude has the fp32 bits `top`.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    // k = exponent field - 127: unit 2^(k-6) is E = k + 127
    if (top >= 0x00800000u) return min((top + 0x10000u) >> 23, 254u);
    return (top + 0x8000u) >> 23;           // subnormal: unit 2^-133 holds all but the last binary 1/256
}

template <typename T, typename I>
__global__ void __launch_bounds__(CK_THREADS) ckpt_store_kernel(const T* __restrict__ x, int cols, long long xs, int ld,
                                                                I total, int8_t* __restrict__ codes,
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
        v.load(x + row * xs + col, cols - col);
        uint32_t top = v.top();
        top = max(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
        const uint32_t E = scale_of(top);
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
                                                               I total, T* __restrict__ x, long long xs) {
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
            if (col + CK_VALS <= cols) {
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
            if (col + CK_VALS <= cols) {
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

// Rows at any address: a warp takes a run of CK_RUN blocks of a row, a value of each a lane,
// all of them in flight.
constexpr int CK_RUN = 8;

__device__ __forceinline__ float read_value(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ float read_value(const float* x) { return *x; }

template <typename T, typename I>
__global__ void __launch_bounds__(CK_THREADS) ckpt_store_ragged_kernel(const T* __restrict__ x, int cols, long long xs, int ld,
                                                                       I total, int8_t* __restrict__ codes,
                                                                       uint8_t* __restrict__ scales) {
    pdl_trigger();
    pdl_wait();
    const int lane = (int)(threadIdx.x & 31u), blocks = ld / CKPT_BLOCK, per_row = (blocks + CK_RUN - 1) / CK_RUN;
    const I stride = (I)gridDim.x * (CK_THREADS / 32);
    for (I u = (I)blockIdx.x * (CK_THREADS / 32) + threadIdx.x / 32; u < total; u += stride) {
        const I row = u / (I)per_row;
        const int block0 = (int)(u - row * (I)per_row) * CK_RUN, n = min(CK_RUN, blocks - block0);
        const int col = block0 * CKPT_BLOCK + lane;
        const T* src = x + (size_t)row * xs + col;
        float v[CK_RUN];
#pragma unroll
        for (int p = 0; p < CK_RUN; ++p) v[p] = col + 32 * p < cols ? read_value(src + 32 * p) : 0.f;
        int8_t* out = codes + (size_t)row * ld + col;
        uint32_t mine = 0;                      // lane p keeps the scale of block p
#pragma unroll
        for (int p = 0; p < CK_RUN; ++p) {
            if (p >= n) break;
            const uint32_t E = scale_of(__reduce_max_sync(0xffffffffu, __float_as_uint(v[p]) & 0x7FFFFFFFu));
            float q;                            // as in ckpt_store_kernel
            if (E >= 6u && E < 254u) {
                q = fmaf(v[p], pow2f(133 - (int)E), 12582912.f);
            } else {
                const int e = 133 - (int)E;
                q = fminf(fmaxf(v[p] * pow2f(e / 2) * pow2f(e - e / 2), -127.f), 127.f) + 12582912.f;
            }
            out[32 * p] = E == 255u ? (int8_t)0 : (int8_t)(__float_as_uint(q) & 0xFFu);
            if (lane == p) mine = E;
        }
        if (lane < n) scales[(size_t)row * blocks + block0 + lane] = (uint8_t)mine;
    }
}

__device__ __forceinline__ void write_value(__nv_bfloat16* x, float v) { *x = __float2bfloat16_rn(v); }
__device__ __forceinline__ void write_value(float* x, float v) { *x = v; }

template <typename T, typename I>
__global__ void __launch_bounds__(CK_THREADS) ckpt_load_ragged_kernel(const int8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales, int cols, int ld,
                                                                      I total, T* __restrict__ x, long long xs) {
    pdl_trigger();
    pdl_wait();
    const int lane = (int)(threadIdx.x & 31u), blocks = ld / CKPT_BLOCK, per_row = (blocks + CK_RUN - 1) / CK_RUN;
    const I stride = (I)gridDim.x * (CK_THREADS / 32);
    for (I u = (I)blockIdx.x * (CK_THREADS / 32) + threadIdx.x / 32; u < total; u += stride) {
        const I row = u / (I)per_row;
        const int block0 = (int)(u - row * (I)per_row) * CK_RUN, n = min(CK_RUN, blocks - block0);
        const int col = block0 * CKPT_BLOCK + lane;
        const int8_t* src = codes + (size_t)row * ld + col;
        const uint32_t mine = lane < n ? scales[(size_t)row * blocks + block0 + lane] : 0u;     // of block `lane`
        int c[CK_RUN];
#pragma unroll
        for (int p = 0; p < CK_RUN; ++p) c[p] = p < n ? src[32 * p] : 0;
        const float unit = mine == 255u ? __uint_as_float(0x7FC00000u) : pow2f((int)mine - 133);
        T* out = x + (size_t)row * xs + col;
#pragma unroll
        for (int p = 0; p < CK_RUN; ++p) {
            const float v = (float)c[p] * __shfl_sync(0xffffffffu, unit, p);
            if (col + 32 * p < cols) write_value(out + 32 * p, v);
        }
    }
}

struct Launch {
    bool vec, small;        // rows on 16-byte addresses; 32-bit indexes hold every index of the loop, one stride past the end included
    size_t total;           // pieces (vec) or runs
    int ld;
    dim3 grid;
};

template <typename T>
Launch plan(const T* x, int rows, int cols, long long xs, int num_sms) {
    Launch l;
    l.ld = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    l.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && xs % (int)(16 / sizeof(T)) == 0;
    const size_t per_block = l.vec ? CK_THREADS : CK_THREADS / 32;
    l.total = (size_t)rows * (l.vec ? l.ld / CK_VALS : (l.ld / CKPT_BLOCK + CK_RUN - 1) / CK_RUN);
    l.grid = dim3((unsigned)std::min<size_t>((l.total + per_block - 1) / per_block, (size_t)num_sms * 64));
    l.small = l.total + l.grid.x * per_block < (1ull << 32);
    return l;
}

template <typename T>
cudaError_t store(const T* x, int rows, int cols, long long xs, int8_t* codes, uint8_t* scales, int num_sms, cudaStream_t s) {
    const Launch l = plan(x, rows, cols, xs, num_sms);
    const dim3 b(CK_THREADS);
    if (l.vec)
        return l.small ? launch_pdl(ckpt_store_kernel<T, uint32_t>, l.grid, b, 0, s, x, cols, xs, l.ld, (uint32_t)l.total, codes, scales)
                       : launch_pdl(ckpt_store_kernel<T, size_t>, l.grid, b, 0, s, x, cols, xs, l.ld, l.total, codes, scales);
    return l.small ? launch_pdl(ckpt_store_ragged_kernel<T, uint32_t>, l.grid, b, 0, s, x, cols, xs, l.ld, (uint32_t)l.total, codes, scales)
                   : launch_pdl(ckpt_store_ragged_kernel<T, size_t>, l.grid, b, 0, s, x, cols, xs, l.ld, l.total, codes, scales);
}

template <typename T>
cudaError_t load(const int8_t* codes, const uint8_t* scales, int rows, int cols, T* x, long long xs, int num_sms, cudaStream_t s) {
    const Launch l = plan(x, rows, cols, xs, num_sms);
    const dim3 b(CK_THREADS);
    if (l.vec)
        return l.small ? launch_pdl(ckpt_load_kernel<T, uint32_t>, l.grid, b, 0, s, codes, scales, cols, l.ld, (uint32_t)l.total, x, xs)
                       : launch_pdl(ckpt_load_kernel<T, size_t>, l.grid, b, 0, s, codes, scales, cols, l.ld, l.total, x, xs);
    return l.small ? launch_pdl(ckpt_load_ragged_kernel<T, uint32_t>, l.grid, b, 0, s, codes, scales, cols, l.ld, (uint32_t)l.total, x, xs)
                   : launch_pdl(ckpt_load_ragged_kernel<T, size_t>, l.grid, b, 0, s, codes, scales, cols, l.ld, l.total, x, xs);
}

}  // namespace

cudaError_t launch_checkpoint_store(const void* x, int x_bf16, int rows, int cols, long long xs, int8_t* codes,
                                    uint8_t* scales, int num_sms, cudaStream_t s) {
    return x_bf16 ? store(static_cast<const __nv_bfloat16*>(x), rows, cols, xs, codes, scales, num_sms, s)
                  : store(static_cast<const float*>(x), rows, cols, xs, codes, scales, num_sms, s);
}

cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* scales, int rows, int cols, void* x, int x_bf16,
                                   long long xs, int num_sms, cudaStream_t s) {
    return x_bf16 ? load(codes, scales, rows, cols, static_cast<__nv_bfloat16*>(x), xs, num_sms, s)
                  : load(codes, scales, rows, cols, static_cast<float*>(x), xs, num_sms, s);
}

}  // namespace muon
