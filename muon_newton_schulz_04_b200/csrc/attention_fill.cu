// attention_fill.cu -- rows of no sequence of the attention's outputs: 0, in lse -inf.
//
// A sequence begins where the one before ends, so these are the rows in front of the first
// sequence and behind the last.  A launch of its own in front of the attention, for outputs
// that hold nothing yet: written by a spare warp of the attention kernels instead, the rows
// cost calls that ask for none of this 1.6 % (8 sequences of 1024, 25 heads of 64: 68.3 us for
// 67.1, by the larger code), and filling whole outputs takes 12 and 32 us there.  Bound by the
// launch where there is little padding.
#include <algorithm>

#include "kernels.cuh"
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int AF_THREADS = 256;
constexpr int AF_BLOCKS = 148;
constexpr int AF_LANES = 16;            // threads of a vector: 16 bytes each, head_dim <= 128

__global__ void __launch_bounds__(AF_THREADS) attention_fill_kernel(const __grid_constant__ FillParams p) {
    pdl_trigger();
    pdl_wait();
    const FillParams::Rows& a = p.array[blockIdx.y];
    int before = 0, from = 0;           // rows 0 .. before - 1, and from `from` on
    if (p.n_seqs > 0) {
        before = min(max(a.cu[0], 0), a.total);
        from = min(max(a.cu[p.n_seqs], before), a.total);
    }
    const size_t rows = (size_t)before + (size_t)(a.total - from);
    const size_t n = rows * (size_t)a.heads;
    auto row = [&](size_t i) { return (long long)(i < (size_t)before ? i : i - before + from); };
    if (a.lse != nullptr) {             // [heads][total]
        for (size_t i = (size_t)blockIdx.x * AF_THREADS + threadIdx.x; i < n; i += (size_t)gridDim.x * AF_THREADS)
            a.lse[(i / rows) * (size_t)a.total + row(i % rows)] = -INFINITY;
        return;
    }
    const int col = (int)threadIdx.x % AF_LANES * 8;
    for (size_t i = ((size_t)blockIdx.x * AF_THREADS + threadIdx.x) / AF_LANES; i < n; i += (size_t)gridDim.x * (AF_THREADS / AF_LANES))
        if (col < p.d)
            *reinterpret_cast<uint4*>(a.x.p + row(i / a.heads) * a.x.rs + (long long)(i % a.heads) * a.x.hs + col) = make_uint4(0, 0, 0, 0);
}

}  // namespace

cudaError_t launch_attention_fill(const FillParams& p, cudaStream_t s) {
    if (p.n == 0) return cudaSuccess;
    return launch_pdl(attention_fill_kernel, dim3(AF_BLOCKS, (unsigned)p.n), dim3(AF_THREADS), 0, s, p);
}

}  // namespace muon
