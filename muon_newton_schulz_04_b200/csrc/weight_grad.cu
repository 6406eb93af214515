// weight_grad.cu -- G (+)= dy^T x^: the gradient of a linear layer's weight, with x^ read
// from its 8-bit checkpoint.
//
// A two-CTA tensor-core GEMM over the tokens: M = rows of G (columns of dy), N = columns of
// G (of x^), 256 x 256 a tile, 64 tokens a stage.  Both operands have the contraction along
// their rows in memory, so both are MN-major.  dy and the codes arrive by TMA; eight warps
// turn the codes into the bf16 operand in shared memory, a thread 32 codes of one scale:
// exact, as a code has 7 bits and the unit is a power of two.  So x^ exists in no memory
// outside the SM, and its traffic is a byte a value.
//
// Tiles beyond the last full round over the clusters are split along the tokens so that
// every cluster has work; their fp32 partial sums go through the caller's workspace and a
// second kernel adds them in order (no atomics: the same inputs give the same bits).
//
// One B200: 8191 tokens into 4096 x 4096 234 us at full clocks (1.17 PFLOP/s) to 292 under the
// power cap; bound by shared memory, where a stage's codes, its converted operand and both
// operands of the products take 640 cycles and the products 512 (192 us with the conversion
// left out).  16384 tokens into 768 x 768: 31 us, of which 6 join the partial sums of its 9
// tiles, split in 8.
#include <algorithm>

#include "kernels.cuh"
#include "ckpt_format.cuh"
#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int WG_TILE = 256;                    // rows and columns of G a tile
constexpr int WG_BK = 64;                       // tokens a stage
constexpr int WG_OPERAND = 128 * WG_BK * 2;     // bytes of this CTA's half of an operand
constexpr int WG_CHUNK = 64 * WG_BK * 2;        // 64 columns of it: 128-byte lines, one per token
constexpr int WG_CODES = 128 * WG_BK;           // bytes of the codes of this CTA's 128 columns
constexpr int WG_STAGES = 4;                    // (5 are no faster)
constexpr int WG_CLUSTERS = 74;                 // CTA pairs of a B200
constexpr int WG_EPI_WARPS = 8, WG_CVT_WARPS = 8;    // (epilogue: two warps for 32 rows, half of the columns each)
constexpr int WG_THREADS = 32 * (WG_EPI_WARPS + WG_CVT_WARPS + 2);
constexpr int WG_TMA_WARP = WG_EPI_WARPS + WG_CVT_WARPS, WG_MMA_WARP = WG_TMA_WARP + 1;
constexpr int WG_GROUP = 8;                     // stages whose scales a thread fetches at once
constexpr int WG_SMEM = 1024 + WG_STAGES * (2 * WG_OPERAND + WG_CODES) + 8 * (3 * WG_STAGES + 5) + 32 + WG_EPI_WARPS * 32 * 33 * 4;
constexpr int WG_MIN_BLOCKS = 4;                // fewest 64-token blocks of a split

constexpr int ERR_WG_LOAD = 0x221, ERR_WG_CVT = 0x222, ERR_WG_MMA = 0x223, ERR_WG_EPI = 0x224;

// bf16 A and B, both MN-major, fp32 accumulation, a 256 x 256 pair tile
constexpr uint32_t WG_IDESC = idesc_bf16_f32(WG_TILE, WG_TILE, 1) | (1u << 15);

// Work of cluster c: tiles c, c + clusters, ... of the `whole` first ones, then part
// (c % splits) of tile whole + c / splits.
struct WgUnit {
    int tile, k0, k1, slot;     // slot of the partial sum, -1: a whole tile
};

__device__ __forceinline__ bool unit_of(const WgradParams& p, int c, int i, WgUnit& u) {
    const int rounds = p.whole / WG_CLUSTERS;
    if (i < rounds) {
        u = WgUnit{c + i * WG_CLUSTERS, 0, p.kblocks, -1};
        return true;
    }
    if (i > rounds || c >= p.rest * p.splits) return false;
    const int part = c % p.splits;
    u.tile = p.whole + c / p.splits;
    u.k0 = (int)((long long)p.kblocks * part / p.splits);
    u.k1 = (int)((long long)p.kblocks * (part + 1) / p.splits);
    u.slot = p.splits > 1 ? c : -1;
    return true;
}

// Scale bytes of this thread's (token of the stage, block) for the WG_GROUP stages from kb.
__device__ __forceinline__ void load_scales(const WgradParams& p, int kb, int k1, int token, int block,
                                            uint32_t (&e)[WG_GROUP]) {
#pragma unroll
    for (int a = 0; a < WG_GROUP; ++a) {
        const int t = (kb + a) * WG_BK + token;
        e[a] = kb + a < k1 && t < p.tokens && block * CKPT_BLOCK < p.ld
                   ? __ldg(p.scales + (size_t)t * (p.ld / CKPT_BLOCK) + block) : 0u;
    }
}

// Turns a token's 32 codes at `src` into 64 bytes of its 128-byte line (128-byte swizzle:
// 16-byte column q of line t lies at q ^ (t & 7)); first: 16-byte column of the first value.
// Half h ^ swap of the codes is taken in turn h.
__device__ __forceinline__ void convert_block(uint32_t src, uint32_t line, uint32_t e, int token, int first, int swap) {
    const uint32_t u = unit_bf16(e) * 0x10001u;
    const __nv_bfloat162 unit = *reinterpret_cast<const __nv_bfloat162*>(&u);
    const uint4 c[2] = {lds128(src + 16u * swap), lds128(src + 16u * (swap ^ 1))};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint4 v;
            v.x = codes_to_bf16(__byte_perm(w[2 * q], 0, 0x4140), unit);
            v.y = codes_to_bf16(__byte_perm(w[2 * q], 0, 0x4342), unit);
            v.z = codes_to_bf16(__byte_perm(w[2 * q + 1], 0, 0x4140), unit);
            v.w = codes_to_bf16(__byte_perm(w[2 * q + 1], 0, 0x4342), unit);
            sts128(line + (uint32_t)(((first + 2 * (h ^ swap) + q) ^ (token & 7)) * 16), v);
        }
    }
}

// Arrives on a barrier of either CTA of the pair.  What the barrier orders lies in this CTA's
// own shared memory and is read there by this SM's tensor core, so release at CTA scope is
// enough, after the proxy fence; at cluster scope every stage would wait for a fence of all
// memory (8191 tokens into 4096 x 4096: 418 us instead of 245).
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}

// A warp's 32 x 32 block of G, a row a lane, goes through its buffer so that every store of the
// warp is 32 neighbours of one row: 32 lines a store otherwise, and G's rows may start at any
// address.
constexpr int WG_BUF = 32 * 33 * 4;

template <typename T>
__device__ __forceinline__ void store_block(const WgradParams& p, int row0, int col, const uint32_t (&v)[32], float* buf) {
    const int lane = (int)(threadIdx.x & 31u);
#pragma unroll
    for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = __uint_as_float(v[i]);
    __syncwarp();
    T* g = static_cast<T*>(p.g) + (size_t)row0 * p.cols + col + lane;
    const int rows = min(32, p.rows - row0);
    if (col + lane < p.cols) {
        float old[32];          // all rows of G in flight at once
#pragma unroll
        for (int r = 0; r < 32; ++r) old[r] = p.accumulate && r < rows ? (float)g[(size_t)r * p.cols] : 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r)
            if (r < rows) g[(size_t)r * p.cols] = (T)(buf[r * 33 + lane] + old[r]);
    }
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WG_THREADS, 1)
weight_grad_kernel(const __grid_constant__ WgradParams p, const __grid_constant__ WgradMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + WG_STAGES * WG_OPERAND;
    uint8_t* sC = sB + WG_STAGES * WG_OPERAND;
    uint64_t* full = reinterpret_cast<uint64_t*>(sC + WG_STAGES * WG_CODES);
    uint64_t* empty = full + WG_STAGES;
    uint64_t* raw = empty + WG_STAGES;
    uint64_t* tfull = raw + WG_STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const uint32_t warp = warp_id();
    const uint32_t rank = cluster_ctarank();
    const int cid = (int)cluster_id_x();
    if (threadIdx.x == 0) {
        for (int s = 0; s < WG_STAGES; ++s) {
            mbar_init(&full[s], 1 + 2 * WG_CVT_WARPS);  // used in CTA 0: its TMA warp and both CTAs' converting warps
            mbar_init(&raw[s], 1);                      // this CTA's codes have arrived
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * WG_EPI_WARPS);    // used in CTA 0
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WG_MMA_WARP) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_trigger();
    pdl_wait();

    if (warp == WG_TMA_WARP) {
        if (elect_one()) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            WgUnit u;
            for (int i = 0; ok && unit_of(p, cid, i, u); ++i) {
                const int row0 = u.tile / p.tiles_n * WG_TILE + (int)rank * 128;
                const int col0 = u.tile % p.tiles_n * WG_TILE + (int)rank * 128;
                for (int kb = u.k0; kb < u.k1; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err, ERR_WG_LOAD)) { ok = false; break; }
                    const uint32_t full0 = mapa_shared(smem_u32(&full[stage]), 0);
                    mbar_arrive_expect_tx(&raw[stage], WG_CODES);
                    tma_load_3d(sC + stage * WG_CODES, &maps.codes, &raw[stage], col0, kb * WG_BK, 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * WG_OPERAND);
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d_pair(sA + stage * WG_OPERAND + c * WG_CHUNK, &maps.dy, full0, row0 + 64 * c, kb * WG_BK, 0);
                    if (++stage == WG_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            for (int i = 0; i < WG_STAGES && ok; ++i) {
                if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err, ERR_WG_LOAD)) ok = false;
                if (++stage == WG_STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok || *abort_flag) {           // let loads in flight land
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) { }
            }
        }
    } else if (warp == WG_MMA_WARP) {
        if (rank == 0 && elect_one()) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            WgUnit u;
            for (int i = 0; ok && unit_of(p, cid, i, u); ++i) {
                const uint32_t acc = i & 1;
                if (!mbar_wait(&tempty[acc], ((uint32_t)(i >> 1) & 1u) ^ 1u, abort_flag, p.err, ERR_WG_MMA)) { ok = false; break; }
                tc_fence_after();
                for (int kb = u.k0; kb < u.k1; ++kb) {
                    if (!mbar_wait(&full[stage], phase, abort_flag, p.err, ERR_WG_MMA)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a = smem_u32(sA + stage * WG_OPERAND), b = smem_u32(sB + stage * WG_OPERAND);
#pragma unroll
                    for (int kk = 0; kk < WG_BK / 16; ++kk)
                        tc_mma_f16_pair(tmem + acc * 256u, smem_desc_sw128(a + kk * 2048, WG_CHUNK, 1024),
                                        smem_desc_sw128(b + kk * 2048, WG_CHUNK, 1024), WG_IDESC, kb != u.k0 || kk != 0);
                    tc_commit_pair(mapa_shared(smem_u32(&empty[stage]), 0));
                    tc_commit_pair(mapa_shared(smem_u32(&empty[stage]), 1));
                    if (++stage == WG_STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit_pair(mapa_shared(smem_u32(&tfull[acc]), 0));
                tc_commit_pair(mapa_shared(smem_u32(&tfull[acc]), 1));
            }
            if (!ok || *abort_flag) {
                tc_commit_pair(mapa_shared(smem_u32(drain), 0));
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 100000000ull) { }
            }
        }
    } else if (warp >= WG_EPI_WARPS) {
        // converting thread: one token of the stage and one block of 32 of this CTA's 128 columns.
        // The order of the block's halves is such that eight lanes read, and write, all banks.
        const int ct = (int)threadIdx.x - 32 * WG_EPI_WARPS, token = ct >> 2, blk = ct & 3;
        const int swap = (blk >> 1) ^ (token & 1);
        const uint32_t line = smem_u32(sB) + (uint32_t)((blk >> 1) * WG_CHUNK + token * 128);
        const uint32_t src = smem_u32(sC) + (uint32_t)(token * 128 + blk * 32);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        WgUnit u;
        for (int i = 0; ok && unit_of(p, cid, i, u); ++i) {
            const int block = (u.tile % p.tiles_n * WG_TILE + (int)rank * 128) / CKPT_BLOCK + blk;
            uint32_t next[WG_GROUP];
            load_scales(p, u.k0, u.k1, token, block, next);
            for (int kb = u.k0; kb < u.k1 && ok; kb += WG_GROUP) {
                uint32_t e[WG_GROUP];
#pragma unroll
                for (int a = 0; a < WG_GROUP; ++a) e[a] = next[a];
                load_scales(p, kb + WG_GROUP, u.k1, token, block, next);
#pragma unroll
                for (int a = 0; a < WG_GROUP; ++a) {
                    if (kb + a >= u.k1) break;
                    // the stage's operand is free, too: its codes were asked for after that
                    ok = mbar_wait(&raw[stage], phase, abort_flag, p.err, ERR_WG_CVT);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    convert_block(src + stage * WG_CODES, line + stage * WG_OPERAND, e[a], token, (blk & 1) * 4, swap);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if ((threadIdx.x & 31u) == 0) arrive_pair(mapa_shared(smem_u32(&full[stage]), 0));
                    if (++stage == WG_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else {
        const int lane = (int)(threadIdx.x & 31u);
        float* buf = reinterpret_cast<float*>(tmem_slot + 2) + warp * (WG_BUF / 4);
        bool ok = true;
        WgUnit u;
        for (int i = 0; ok && unit_of(p, cid, i, u); ++i) {
            const uint32_t acc = i & 1;
            ok = mbar_wait(&tfull[acc], (uint32_t)(i >> 1) & 1u, abort_flag, p.err, ERR_WG_EPI);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            const int in_tile = (int)rank * 128 + (int)(warp & 3u) * 32, c0 = (int)(warp >> 2) * 4;
            const int row0 = u.tile / p.tiles_n * WG_TILE + in_tile, col0 = u.tile % p.tiles_n * WG_TILE;
            const uint32_t t_acc = tmem + acc * 256u + ((warp & 3u) * 32u << 16);
            // partial sums lie as 32 x 32 blocks, each as eight groups of four columns: a store of the warp
            // covers 512 bytes (a row per lane: 32 lines a store)
            float4* part = u.slot >= 0 ? reinterpret_cast<float4*>(p.partial) +
                                             ((size_t)u.slot * 8 + in_tile / 32) * (WG_TILE * 8) + lane : nullptr;
#pragma unroll 1
            for (int c = c0; c < c0 + 4 && col0 + 32 * c < p.cols; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(t_acc + 32u * c, v);
                tmem_ld_wait();
                if (part != nullptr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        part[c * 256 + e * 32] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                                             __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                } else if (row0 >= p.rows) {
                    break;
                } else if (p.g_bf16) {
                    store_block<__nv_bfloat16>(p, row0, col0 + 32 * c, v, buf);
                } else {
                    store_block<float>(p, row0, col0 + 32 * c, v, buf);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
        }
    }
    tc_fence_before();
    cluster_sync_all();
    if (warp == WG_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Four values of one row of G.
__device__ __forceinline__ void store_four(const WgradParams& p, int row, int col, float4 s) {
    const float v[4] = {s.x, s.y, s.z, s.w};
    const size_t at = (size_t)row * p.cols + col;
    if (p.vec && !p.g_bf16) {
        float4* g = reinterpret_cast<float4*>(static_cast<float*>(p.g) + at);
        const float4 old = p.accumulate ? *g : make_float4(0.f, 0.f, 0.f, 0.f);
        *g = make_float4(s.x + old.x, s.y + old.y, s.z + old.z, s.w + old.w);
        return;
    }
    for (int e = 0; e < 4 && col + e < p.cols; ++e) {
        if (p.g_bf16) {
            __nv_bfloat16* g = static_cast<__nv_bfloat16*>(p.g) + at + e;
            *g = __float2bfloat16_rn(v[e] + (p.accumulate ? __bfloat162float(*g) : 0.f));
        } else {
            float* g = static_cast<float*>(p.g) + at + e;
            *g = v[e] + (p.accumulate ? *g : 0.f);
        }
    }
}

// Adds the partial sums of a split tile's 32 x 32 block in order and writes its rows.
__global__ void __launch_bounds__(256) weight_grad_join_kernel(const WgradParams p) {
    __shared__ float block[32][33];
    pdl_trigger();
    pdl_wait();
    const int tile = p.whole + (int)blockIdx.y, rb = (int)blockIdx.x / 8, cb = (int)blockIdx.x % 8;
    const int row0 = tile / p.tiles_n * WG_TILE + 32 * rb, col0 = tile % p.tiles_n * WG_TILE + 32 * cb;
    if (row0 >= p.rows || col0 >= p.cols) return;
    const int e = (int)threadIdx.x / 32, lane = (int)threadIdx.x % 32;
    const float4* src = reinterpret_cast<const float4*>(p.partial) +
                        ((size_t)blockIdx.y * p.splits * 8 + rb) * (WG_TILE * 8) + cb * 256 + e * 32 + lane;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < p.splits; ++k) {
        const float4 x = __ldcg(src + (size_t)k * (WG_TILE * WG_TILE / 4));
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    block[lane][4 * e] = s.x;
    block[lane][4 * e + 1] = s.y;
    block[lane][4 * e + 2] = s.z;
    block[lane][4 * e + 3] = s.w;
    __syncthreads();
    const int r = (int)threadIdx.x / 8, c = (int)threadIdx.x % 8 * 4;
    if (row0 + r < p.rows && col0 + c < p.cols)
        store_four(p, row0 + r, col0 + c, make_float4(block[r][c], block[r][c + 1], block[r][c + 2], block[r][c + 3]));
}

// dy with rows that TMA cannot read (an odd address or stride), copied to rows of a multiple
// of 8 elements.
__global__ void __launch_bounds__(256) weight_grad_repack_kernel(const __nv_bfloat16* __restrict__ dy, long long dys,
                                                                 int tokens, int rows, int ld,
                                                                 __nv_bfloat16* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    for (int t = blockIdx.x; t < tokens; t += gridDim.x)
        for (int r = threadIdx.x; r < rows; r += 256) out[(size_t)t * ld + r] = dy[(size_t)t * dys + r];
}

// dy is not read: G = 0, or stays.
__global__ void __launch_bounds__(256) weight_grad_zero_kernel(const WgradParams p) {
    pdl_trigger();
    pdl_wait();
    const size_t n = (size_t)p.rows * p.cols;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        if (p.g_bf16) static_cast<__nv_bfloat16*>(p.g)[i] = __float2bfloat16_rn(0.f);
        else static_cast<float*>(p.g)[i] = 0.f;
    }
}

}  // namespace

WgradPlan weight_grad_plan(int tokens, int rows, int cols, bool dy_aligned) {
    WgradPlan w{};
    w.kblocks = (tokens + WG_BK - 1) / WG_BK;
    w.tiles_n = (cols + WG_TILE - 1) / WG_TILE;
    const int tiles = (rows + WG_TILE - 1) / WG_TILE * w.tiles_n;
    w.whole = tiles / WG_CLUSTERS * WG_CLUSTERS;
    w.rest = tiles - w.whole;
    w.splits = w.rest == 0 ? 1 : std::max(1, std::min(WG_CLUSTERS / w.rest, w.kblocks / WG_MIN_BLOCKS));
    w.partial_bytes = w.splits > 1 ? (size_t)w.rest * w.splits * WG_TILE * WG_TILE * sizeof(float) : 0;
    w.dy_ld = (rows + 7) / 8 * 8;
    w.dy_bytes = dy_aligned || tokens == 0 ? 0 : ((size_t)tokens * w.dy_ld * 2 + 255) / 256 * 256;
    return w;
}

cudaError_t launch_weight_grad_repack(const WgradParams& p, const WgradPlan& w, __nv_bfloat16* out, cudaStream_t s) {
    return launch_pdl(weight_grad_repack_kernel, dim3(std::min(p.tokens, 16 * 148)), dim3(256), 0, s, p.dy, p.dys, p.tokens,
                      p.rows, w.dy_ld, out);
}

cudaError_t launch_weight_grad(const WgradParams& p, const WgradMaps& maps, cudaStream_t s) {
    if (p.tokens == 0) {
        if (p.accumulate) return cudaSuccess;
        const size_t n = (size_t)p.rows * p.cols;
        return launch_pdl(weight_grad_zero_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 16 * 148)), dim3(256), 0, s, p);
    }
    cudaError_t e = cudaFuncSetAttribute(weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WG_SMEM);
    if (e != cudaSuccess) return e;
    const int clusters = p.whole > 0 ? WG_CLUSTERS : p.rest * p.splits;
    e = launch_pdl(weight_grad_kernel, dim3(2 * clusters), dim3(WG_THREADS), WG_SMEM, s, p, maps);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_pdl(weight_grad_join_kernel, dim3(64, p.rest), dim3(256), 0, s, p);
}

}  // namespace muon
