// attention_fwd.cu -- packed causal attention with grouped heads: O = softmax(S) V, the
// log-sums of the rows and each head's largest logit.
//
// One CTA computes 256 query rows of one head of one sequence, as two tiles of 128 rows
// that take turns: while the tensor cores form one tile's products, the other tile's
// softmax runs.  K and V tiles of 128 rows stream through a ring in shared memory.
//
//   S = Q K^T      both operands from shared memory, 128 x 128 fp32 in tensor memory
//   P = exp(S - m) by one warpgroup per tile: a thread owns a row, so the row's maximum
//                  and sum need no exchange
//   O += P V       P is written back to tensor memory as bf16 and is the A operand there
//
// m is the running maximum that O is scaled by; it follows the true maximum only when that
// has grown by 2^8, so that O is rescaled rarely (P then stays below 2^8; sums and O are
// fp32, and P's rounding to bf16 is relative).
#include <algorithm>

#include "attention.cuh"
#include "kernels.cuh"

namespace muon {
namespace {

constexpr int FW_TILES = 2;                     // query tiles of a CTA
constexpr int FW_SOFTMAX = FW_TILES * 128;      // softmax threads
constexpr int FW_THREADS = FW_SOFTMAX + 64;     // + the TMA warp and the MMA warp

template <int DP>
struct FwLayout {
    static constexpr int TILE = DP / 64 * AT_CHUNK;                 // bytes of a q, k or v tile
    static constexpr int SLOTS = DP == 64 ? 8 : 5;                  // ring of k and v tiles
    static constexpr int BARRIERS = 1 + 2 * SLOTS + 5 * FW_TILES;
    static constexpr int SMEM = 1024 + (FW_TILES + SLOTS) * TILE + 8 * BARRIERS + 64;
    // 64-wide heads leave room for P beside S, so the next S need not wait for P V
    static constexpr bool P_APART = DP == 64;
    static constexpr uint32_t S_COL = 0;                            // + 128 per tile
    static constexpr uint32_t P_COL = P_APART ? 256 : 0;            // + P_STEP per tile
    static constexpr uint32_t P_STEP = P_APART ? 64 : 128;
    static constexpr uint32_t O_COL = P_APART ? 384 : 256;          // + DP per tile
    static_assert(SMEM <= 232448, "shared memory above the 227 KiB limit");
};

struct FwMaps {
    CUtensorMap q, k, v;
};

constexpr int ERR_FW_LOAD = 0x201, ERR_FW_MMA = 0x202, ERR_FW_SOFTMAX = 0x203;

// Raises *addr to v.  Signed order of the bits is the order of non-negative floats, the
// reverse unsigned order that of negative ones.
__device__ __forceinline__ void atomic_max_float(float* addr, float v) {
    v += 0.f;                                   // -0 counts as +0
    if (v >= 0.f) atomicMax(reinterpret_cast<int*>(addr), __float_as_int(v));
    else if (v < 0.f) atomicMin(reinterpret_cast<unsigned*>(addr), __float_as_uint(v));
}

template <int DP>
__global__ void __launch_bounds__(FW_THREADS, 1)
attention_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FwMaps maps) {
    using L = FwLayout<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = smem;
    uint8_t* ring = smem + FW_TILES * L::TILE;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + L::SLOTS * L::TILE);
    uint64_t* full = q_full + 1;
    uint64_t* empty = full + L::SLOTS;
    uint64_t* s_full = empty + L::SLOTS;        // per tile, as the following ones
    uint64_t* s_read = s_full + FW_TILES;       // the softmax has S in registers (P_APART)
    uint64_t* p_ready = s_read + FW_TILES;
    uint64_t* pv_done = p_ready + FW_TILES;     // P has been read (P_APART)
    uint64_t* o_full = pv_done + FW_TILES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + FW_TILES);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* found = reinterpret_cast<int*>(tmem_slot + 2);
    int4* info = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 3) + 15) & ~uintptr_t(15));

    const uint32_t warp = warp_id();
    const int head = (int)(blockIdx.x % (unsigned)p.hq);
    pdl_trigger();
    pdl_wait();             // cu_seqlens, too, may be the previous kernel's
    if (warp == 0) {
        SeqTile t;
        const bool ok = find_tile(p, false, FW_TILES * AT_ROWS, (int)(blockIdx.x / (unsigned)p.hq), blockIdx.x == 0, t);
        if (elect_one()) {
            *found = ok;
            info[0] = make_int4(t.q0, t.lq, t.k0, t.lk);
            // long rows first: the last blocks of a sequence see the most keys
            info[1] = make_int4(ok ? t.blocks - 1 - t.block : 0, 0, 0, 0);
        }
    } else if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(q_full, 1);
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < FW_TILES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_read[i], 128);
            mbar_init(&p_ready[i], 128);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_full[i], 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (*found) {
        const int4 sl = info[0];
        const int q0 = sl.x, lq = sl.y, k0 = sl.z, lk = sl.w;
        const int row0 = info[1].x * (FW_TILES * AT_ROWS);          // of the CTA, in the sequence
        const int shift = lk - lq;                                  // row i sees keys up to i + shift
        const int kv_head = head / p.group;
        // key tiles that a tile's rows see
        int n[FW_TILES];
#pragma unroll
        for (int w = 0; w < FW_TILES; ++w) {
            const int first = row0 + w * AT_ROWS, last = min(first + AT_ROWS, lq) - 1 + shift;
            n[w] = first >= lq || last < 0 ? 0 : last / AT_ROWS + 1;
        }
        const int nmax = max(n[0], n[1]);

        if (warp == 8) {
            if (elect_one() && nmax > 0) {
                mbar_arrive_expect_tx(q_full, FW_TILES * L::TILE);
                for (int w = 0; w < FW_TILES; ++w)
                    for (int c = 0; c < DP / 64; ++c)
                        tma_load_3d(sq + w * L::TILE + c * AT_CHUNK, &maps.q, q_full, 64 * c, head,
                                    q0 + row0 + w * AT_ROWS);
                // ring order: K0, K1, V0, K2, V1, ...: the order of use
                int slot = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int i = 0; i < 2 * nmax && ok; ++i) {
                    const bool is_v = i > 0 && (i % 2 == 0 || i == 2 * nmax - 1);
                    const int j = i == 0 ? 0 : is_v ? (i == 2 * nmax - 1 ? nmax - 1 : i / 2 - 1) : (i + 1) / 2;
                    if (!mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.err, ERR_FW_LOAD)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full[slot], L::TILE);
                    for (int c = 0; c < DP / 64; ++c)
                        tma_load_3d(ring + slot * L::TILE + c * AT_CHUNK, is_v ? &maps.v : &maps.k, &full[slot], 64 * c,
                                    kv_head, k0 + j * AT_ROWS);
                    if (++slot == L::SLOTS) { slot = 0; phase ^= 1u; }
                }
                // every load has landed before the CTA may end
                for (int i = 0; i < L::SLOTS && ok; ++i) {
                    if (!mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.err, ERR_FW_LOAD)) ok = false;
                    if (++slot == L::SLOTS) { slot = 0; phase ^= 1u; }
                }
                if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
            }
        } else if (warp == 9) {
            if (elect_one() && nmax > 0) {
                bool ok = mbar_wait(q_full, 0, abort_flag, p.err, ERR_FW_MMA);
                const uint32_t q_s = smem_u32(sq), ring_s = smem_u32(ring);
                // ring position of K_j and V_j
                auto k_at = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
                auto v_at = [&](int j) { return j == nmax - 1 ? 2 * nmax - 1 : 2 * j + 2; };
                auto wait_full = [&](int at) {
                    return mbar_wait(&full[at % L::SLOTS], (uint32_t)(at / L::SLOTS) & 1u, abort_flag, p.err, ERR_FW_MMA);
                };
                auto tile_s = [&](int at) { return ring_s + (uint32_t)(at % L::SLOTS) * L::TILE; };
                auto do_s = [&](int w, int j) {
                    tc_fence_after();
                    mma_abt<DP>(tmem + L::S_COL + 128u * w, q_s + w * L::TILE, tile_s(k_at(j)));
                    tc_commit(&s_full[w]);
                };
                ok = ok && wait_full(0);
                if (ok) {
                    for (int w = 0; w < FW_TILES; ++w)
                        if (n[w] > 0) do_s(w, 0);
                    tc_commit(&empty[0]);
                }
                for (int j = 0; j < nmax && ok; ++j) {
                    const bool more = j + 1 < nmax;
                    for (int w = 0; w < FW_TILES && ok; ++w) {
                        if (L::P_APART && j + 1 < n[w]) {
                            ok = wait_full(k_at(j + 1)) &&
                                 mbar_wait(&s_read[w], (uint32_t)j & 1u, abort_flag, p.err, ERR_FW_MMA);
                            if (!ok) break;
                            do_s(w, j + 1);
                        }
                        if (j < n[w]) {
                            ok = wait_full(v_at(j)) &&
                                 mbar_wait(&p_ready[w], (uint32_t)j & 1u, abort_flag, p.err, ERR_FW_MMA);
                            if (!ok) break;
                            tc_fence_after();
                            mma_tb<DP>(tmem + L::O_COL + (uint32_t)(DP * w), tmem + L::P_COL + L::P_STEP * w,
                                       tile_s(v_at(j)), j > 0);
                            if (L::P_APART) tc_commit(&pv_done[w]);
                            if (j + 1 == n[w]) tc_commit(&o_full[w]);
                        }
                        if (!L::P_APART && j + 1 < n[w]) {
                            // S takes P's place: products run in order, so P V has read it
                            ok = wait_full(k_at(j + 1));
                            if (!ok) break;
                            do_s(w, j + 1);
                        }
                    }
                    if (!ok) break;
                    tc_commit(&empty[v_at(j) % L::SLOTS]);
                    if (more) tc_commit(&empty[k_at(j + 1) % L::SLOTS]);
                }
                if (!ok || *abort_flag) spin_ns_at_most(2000000ull);    // products in flight end
            }
        } else {
            const int w = (int)(warp >> 2), t = (int)(threadIdx.x & 127u);
            const uint32_t lane_base = (warp & 3u) * 32u << 16;
            const int row = row0 + w * AT_ROWS + t;                 // in the sequence
            const uint32_t s_t = tmem + lane_base + L::S_COL + 128u * w, p_t = tmem + lane_base + L::P_COL + L::P_STEP * w,
                           o_t = tmem + lane_base + L::O_COL + (uint32_t)(DP * w);
            const float c = p.scale * AT_LOG2E;
            const int see = row + shift;                            // last key that this row sees
            const int full_tiles = row0 + w * AT_ROWS + shift + 1;  // keys that all rows see
            float m = -INFINITY, top = -INFINITY;                   // scaled by; true maximum
            float l = 0.f;
            bool ok = true;
            const int nw = n[w];
            for (int j = 0; j < nw; ++j) {
                ok = mbar_wait(&s_full[w], (uint32_t)j & 1u, abort_flag, p.err, ERR_FW_SOFTMAX);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(s_t + 32u * i, s[i]);
                tmem_ld_wait();
                if (L::P_APART) {
                    tc_fence_before();
                    mbar_arrive(&s_read[w]);
                }
                if ((j + 1) * AT_ROWS > full_tiles) {
                    const int seen = see - j * AT_ROWS;             // column of the last seen key
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i > seen) s[i / 32][i % 32] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][e]));
                }
                top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                if (L::P_APART && j > 0) {
                    ok = mbar_wait(&pv_done[w], (uint32_t)(j - 1) & 1u, abort_flag, p.err, ERR_FW_SOFTMAX);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                }
                const bool grow = m == -INFINITY ? top > -INFINITY : (top - m) * c > 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? (m == -INFINITY ? 0.f : ex2((m - top) * c)) : 1.f;
                    if (grow) m = top;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int i = 0; i < DP / 32; ++i) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(o_t + 32u * i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_32x32b_x32(o_t + 32u * i, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m * c;
                const uint64_t c2 = pack2(c, c), b2 = pack2(-base, -base);
                uint64_t sum2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pr[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int at = 64 * h + 2 * i;
                        float x, y;
                        unpack2(fma2(pack2(__uint_as_float(s[at / 32][at % 32]), __uint_as_float(s[at / 32][at % 32 + 1])),
                                     c2, b2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum2[i & 1] = add2(sum2[i & 1], pack2(x, y));
                        pr[i] = bf16x2(x, y);
                    }
                    tmem_st_32x32b_x32(p_t + 32u * h, pr);
                }
                float a, b;
                unpack2(add2(sum2[0], sum2[1]), a, b);
                l += a + b;
                if (lk - j * AT_ROWS < AT_ROWS) {
                    // rows behind the sequence's keys: P is 0 there, but 0 times what lies behind need not be
                    const int at = j == nmax - 1 ? 2 * nmax - 1 : 2 * j + 2;
                    ok = mbar_wait(&full[at % L::SLOTS], (uint32_t)(at / L::SLOTS) & 1u, abort_flag, p.err, ERR_FW_SOFTMAX);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    zero_rows<DP>(smem_u32(ring + (at % L::SLOTS) * L::TILE), lk - j * AT_ROWS, t, 128);
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_ready[w]);
            }
            if (ok && nw > 0) {
                ok = mbar_wait(&o_full[w], 0, abort_flag, p.err, ERR_FW_SOFTMAX);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            if (ok && row0 + w * AT_ROWS < lq) {
                const bool live = row < lq;
                const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
                __nv_bfloat16* o_g = p.out.p + (long long)(q0 + row) * p.out.rs + (long long)head * p.out.hs;
#pragma unroll 1
                for (int i = 0; i < DP / 32; ++i) {
                    uint32_t o[32];
                    if (nw > 0) {
                        tmem_ld_32x32b_x32(o_t + 32u * i, o);
                        tmem_ld_wait();
                    }
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (32 * i + 8 * e < p.d) {
                                uint32_t v[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    v[u] = inv == 0.f ? 0u : bf16x2(__uint_as_float(o[8 * e + 2 * u]) * inv,
                                                                    __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
                                *reinterpret_cast<uint4*>(o_g + 32 * i + 8 * e) = make_uint4(v[0], v[1], v[2], v[3]);
                            }
                        }
                    }
                }
                if (live) p.lse[(size_t)head * p.total_q + q0 + row] = (m == -INFINITY ? 0.f : m * p.scale) + logf(l);
                if (p.max_logits != nullptr) {
                    float best = live ? top : -INFINITY;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
                    if ((t & 31) == 0 && best > -INFINITY) atomic_max_float(p.max_logits + head, best * p.scale);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP>
cudaError_t launch_fwd(const AttnParams& p, const FwMaps& maps, cudaStream_t s) {
    using L = FwLayout<DP>;
    const cudaError_t e = cudaFuncSetAttribute(attention_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    // at most one partial block per sequence
    const unsigned tiles = (unsigned)(p.total_q / (FW_TILES * AT_ROWS) + std::min(p.n_seqs, p.total_q));
    return launch_pdl(attention_fwd_kernel<DP>, dim3(tiles * (unsigned)p.hq), dim3(FW_THREADS), L::SMEM, s, p, maps);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, const HeadMaps& m, cudaStream_t s) {
    if (p.total_q == 0 || p.n_seqs == 0) return cudaSuccess;
    const FwMaps maps{m.q, m.k, m.v};
    return p.d <= 64 ? launch_fwd<64>(p, maps, s) : launch_fwd<128>(p, maps, s);
}

}  // namespace muon
