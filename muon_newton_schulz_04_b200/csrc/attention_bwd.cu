// attention_bwd.cu -- gradients of packed causal attention with grouped heads.
//
//   P = exp(S - lse),  dP = dO V^T,  dS = P (dP - D),  D_i = dO_i . O_i
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two kernels, each owning what it sums, so that nothing is added with atomics and the
// same inputs give the same bits: the first takes 128 query rows of a head through the
// keys they see (S, dP, dQ: three products a tile pair), the second 128 key rows of a key
// head through the queries that see them, for every query head of the group (S^T, dP^T,
// dV, dK: four).  Forming S and dP twice costs seven products instead of five; in exchange
// there is no fp32 dQ in memory to add to (for 128-wide heads 64 KiB a tile pair).
//
// In the second kernel a row of the accumulators is a key, and lse and D belong to its columns.
// They enter through the products themselves: Q gets three more columns with -lse / scale
// split into three bf16 (24 bits), dO three with -D, K and V three of ones, one more MMA step
// each.  Read from shared memory instead, beside the tiles that the products read there, they
// took as long as the exponentials (3720 cycles a tile pair of 128-wide heads against 3000).
//
// In both, P and dS go back to tensor memory as bf16 in the place of the fp32 tile that they
// were formed from, and are the A operand there: only Q, K, V and dO tiles lie in shared
// memory.
//
// A CTA owns 128 rows and goes through the others in steps of as many as a head is wide.
// 128-wide heads: one CTA an SM, eight warps form P and dS (warp w has rows 32 (w % 4) ..,
// warps 0-3 the first 64 columns of a step, warps 4-7 the last).  64-wide heads: half the
// tensor memory, so two CTAs an SM, four such warps each, which also hide each other's start
// and end (eight sequences of 1024, 25 heads: 225 us with one CTA an SM, 188 with two).
//
// D comes from O as the forward pass rounded it, off by up to 2^-8 sum_d |dO_id O_id|.  The first
// kernel finds the exact one as it goes, D + sum_j dS_ij, since sum_j P_ij = 1, and leaves that
// for the second.  For its own dS that comes too late (to mend dQ afterwards would take
// sum_j P_ij k_j, a product more), but where a row block sees one step of keys, when D's
// rounding counts most, P and dP of all its keys are at hand and D is formed from them.
//
// Two spare warps take infinities and NaN out of K, Q and dO in the tiles that not every row
// sees all of (there 0 times them would reach rows that do not see them): 199-211 us instead of
// 188.  8192 rows in 5 sequences, 32 heads over 8 of 128: 1030 us at full clocks (443 and 587;
// 0.87 PFLOP/s by the formula's five products, 1.2 by the seven formed, where the sustained
// rate of plain products is 1.38) to 1230 under the power cap.
#include <algorithm>

#include "attention.cuh"
#include "kernels.cuh"

namespace muon {
namespace {

constexpr int ERR_DQ_LOAD = 0x211, ERR_DQ_MMA = 0x212, ERR_DQ_MATH = 0x213, ERR_DQ_CLEAN = 0x214;
constexpr int ERR_DKV_LOAD = 0x231, ERR_DKV_MMA = 0x232, ERR_DKV_MATH = 0x233, ERR_DKV_CLEAN = 0x234;

// What both kernels share.
template <int DP>
struct BwLayout {
    static constexpr int HALVES = DP / 64;                      // of a step's columns
    static constexpr int STEP = DP;                             // rows of a streamed tile
    static constexpr int MATH = 128 * HALVES, THREADS = MATH + 128;     // + a warpgroup: TMA, MMA, tensor memory
    static constexpr int W_TMA = MATH / 32, W_MMA = W_TMA + 1, W_TMEM = W_TMA + 2;     // W_TMEM and the last warp clean tiles
    static constexpr int CTAS = 2 / HALVES;                     // of an SM
    static constexpr int REGS = HALVES == 1 ? 128 : 168;        // a thread: at launch, then of the math warps and the others
    static constexpr int REGS_MATH = HALVES == 1 ? 168 : 200, REGS_OTHER = HALVES == 1 ? 88 : 104;
    static_assert(MATH * REGS_MATH + 128 * REGS_OTHER <= THREADS * REGS, "more registers than launched with");
    static constexpr int OWN = 128 * DP * 2, MOVING = STEP * DP * 2;    // bytes of the tiles
    static constexpr int MOST_SMEM = 232448 / CTAS - (CTAS - 1) * 1024;
    static constexpr uint32_t TMEM_COLS = 4 * DP;
    static constexpr int ON_FMA = 2;                            // of 8 pairs of exponentials
};

template <int DP>
__device__ __forceinline__ void math_sync() { named_sync(1, BwLayout<DP>::MATH); }

// One more K step of 16: D += A B^T of tiles of 128 and N rows of 16 columns without
// swizzle (core matrices of 8 rows x 16 bytes; groups of 8 rows 128 bytes apart, the two of a
// row 16 bytes times the rows).
template <int N>
__device__ __forceinline__ void mma_extra(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t idesc = idesc_bf16_f32(AT_ROWS, N, 0);
    tc_mma_f16(d_tmem, smem_desc_plain(a, 2048, 128), smem_desc_plain(b, N * 16, 128), idesc, 1u);
}

// Byte of the first column of row r of such a tile.
__device__ __forceinline__ uint32_t extra_at(int r) { return (uint32_t)((r >> 3) * 128 + (r & 7) * 16); }

// ============================================================================ dQ

template <int DP>
struct DqLayout : BwLayout<DP> {
    using Base = BwLayout<DP>;
    static constexpr int KS = DP == 64 ? 4 : 3, VS = DP == 64 ? 3 : 2;      // ring slots: K is used twice
    static constexpr int BARRIERS = 2 + 2 * KS + 2 * VS + 9;
    static constexpr int SMEM = 1024 + 2 * Base::OWN + (KS + VS) * Base::MOVING + 8 * BARRIERS + 2 * 128 * 4 + 64;
    static constexpr uint32_t S_COL = 0, DP_COL = 2 * DP, DQ_COL = 3 * DP;  // S: two buffers
    static_assert(SMEM <= Base::MOST_SMEM, "shared memory above the SM's 228 KiB");
};

struct BwMaps {
    CUtensorMap q, k, v, go;
};

template <int DP>
__global__ void __launch_bounds__(BwLayout<DP>::THREADS, BwLayout<DP>::CTAS)
attention_dq_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ BwMaps maps) {
    using L = DqLayout<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_q = smem, *s_do = s_q + L::OWN, *s_k = s_do + L::OWN, *s_v = s_k + L::KS * L::MOVING;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(s_v + L::VS * L::MOVING);
    uint64_t* do_full = q_full + 1;
    uint64_t *k_full = do_full + 1, *k_empty = k_full + L::KS, *v_full = k_empty + L::KS, *v_empty = v_full + L::VS;
    uint64_t *s_full = v_empty + L::VS, *dp_full = s_full + 2, *dp_read = dp_full + 1, *ds_ready = dp_read + 1,
             *dq_full = ds_ready + 2, *near = dq_full + 1, *clean = near + 1;
    float* exch = reinterpret_cast<float*>(clean + 1);            // [2][128]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(exch + 256);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* found = reinterpret_cast<int*>(tmem_slot + 2);
    volatile int* poisoned = reinterpret_cast<volatile int*>(tmem_slot + 3);      // infinities or NaN of K were set to zero
    int4* info = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 15) & ~uintptr_t(15));

    const uint32_t warp = warp_id();
    const int head = (int)(blockIdx.x % (unsigned)p.hq);
    pdl_wait();
    pdl_trigger();          // after the wait: the second kernel starts on what came before this one
    if (warp == 0) {
        SeqTile t;
        const bool ok = find_tile(p, false, AT_ROWS, (int)(blockIdx.x / (unsigned)p.hq), blockIdx.x, t);
        if (elect_one()) {
            *found = ok;
            info[0] = make_int4(t.q0, t.lq, t.k0, t.lk);
            info[1] = make_int4(ok ? t.blocks - 1 - t.block : 0, 0, 0, 0);      // long rows first
        }
    } else if (warp == L::W_TMEM) {
        tmem_alloc(tmem_slot, L::TMEM_COLS);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(q_full, 1);
        mbar_init(do_full, 1);
        for (int i = 0; i < L::KS; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < L::VS; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); }
        mbar_init(&s_full[0], 1);                       // one per buffer: S runs a tile ahead
        mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1);
        mbar_init(dp_read, L::MATH);
        mbar_init(&ds_ready[0], L::MATH);               // one per buffer: dS may run a tile ahead of its wait
        mbar_init(&ds_ready[1], L::MATH);
        mbar_init(dq_full, 1);
        mbar_init(near, 1);                             // the next edge tile may be cleaned
        mbar_init(clean, 2);                            // its K is fit for dS K
        *abort_flag = 0;
        *poisoned = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (*found) {
        const int4 sl = info[0];
        const int q0 = sl.x, lq = sl.y, k0 = sl.z, lk = sl.w;
        const int row0 = info[1].x * AT_ROWS, shift = lk - lq, kv_head = head / p.group;
        const int last = min(row0 + AT_ROWS, lq) - 1 + shift;       // last key that any row sees
        const int n = last < 0 ? 0 : last / L::STEP + 1;
        const int edge0 = max(0, row0 + shift + 1) / L::STEP;      // key tiles from this one on: some row does not see all of them

        if (warp >= L::W_TMA) {
            regs_less<L::REGS_OTHER>();     // one instruction for all warps of the group
            if (warp == L::W_TMA) {
                if (elect_one() && n > 0) {
                    mbar_arrive_expect_tx(q_full, L::OWN);
                    load_tile<DP, 128, AT_BWD_BOX>(s_q, &maps.q, q_full, head, q0 + row0);
                    bool ok = true;
                    for (int j = 0; j < n + L::KS; ++j) {       // the last turns only wait for the loads to be used
                        const int ks = j % L::KS, vs = j % L::VS;
                        if (!mbar_wait(&k_empty[ks], ((uint32_t)(j / L::KS) & 1u) ^ 1u, abort_flag, p.err, ERR_DQ_LOAD)) { ok = false; break; }
                        if (j < n) {
                            mbar_arrive_expect_tx(&k_full[ks], L::MOVING);
                            load_tile<DP, L::STEP, AT_BWD_BOX>(s_k + ks * L::MOVING, &maps.k, &k_full[ks], kv_head, k0 + j * L::STEP);
                        }
                        if (j == 0) {
                            mbar_arrive_expect_tx(do_full, L::OWN);
                            load_tile<DP, 128, AT_BWD_BOX>(s_do, &maps.go, do_full, head, q0 + row0);
                        }
                        if (j < n + L::VS &&
                            !mbar_wait(&v_empty[vs], ((uint32_t)(j / L::VS) & 1u) ^ 1u, abort_flag, p.err, ERR_DQ_LOAD)) { ok = false; break; }
                        if (j < n) {
                            mbar_arrive_expect_tx(&v_full[vs], L::MOVING);
                            load_tile<DP, L::STEP, AT_BWD_BOX>(s_v + vs * L::MOVING, &maps.v, &v_full[vs], kv_head, k0 + j * L::STEP);
                        }
                    }
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
                }
            } else if (warp == L::W_MMA) {
                if (elect_one() && n > 0) {
                    const uint32_t q_s = smem_u32(s_q), do_s = smem_u32(s_do), k_s = smem_u32(s_k), v_s = smem_u32(s_v);
                    auto wait = [&](uint64_t* b, int use) {
                        const bool ok = mbar_wait(b, (uint32_t)use & 1u, abort_flag, p.err, ERR_DQ_MMA);
                        tc_fence_after();
                        return ok;
                    };
                    auto do_s_product = [&](int j) {
                        mma_abt<DP, L::STEP>(tmem + L::S_COL + (uint32_t)(DP * (j & 1)), q_s, k_s + (uint32_t)(j % L::KS) * L::MOVING);
                        tc_commit(&s_full[j & 1]);
                    };
                    auto do_dp_product = [&](int j) {
                        mma_abt<DP, L::STEP>(tmem + L::DP_COL, do_s, v_s + (uint32_t)(j % L::VS) * L::MOVING);
                        tc_commit(dp_full);
                        tc_commit(&v_empty[j % L::VS]);
                    };
                    bool ok = wait(q_full, 0) && wait(&k_full[0], 0);
                    if (ok) do_s_product(0);
                    ok = ok && wait(do_full, 0) && wait(&v_full[0], 0);
                    if (ok) do_dp_product(0);
                    if (edge0 == 0) mbar_arrive(near);
                    for (int j = 0; j < n && ok; ++j) {
                        if (j + 1 < n) {
                            // its buffer held dS of tile j - 1, whose product runs before
                            if (!(ok = wait(&k_full[(j + 1) % L::KS], (j + 1) / L::KS))) break;
                            do_s_product(j + 1);
                            if (!(ok = wait(dp_read, j) && wait(&v_full[(j + 1) % L::VS], (j + 1) / L::VS))) break;
                            do_dp_product(j + 1);
                        }
                        if (!(ok = wait(&ds_ready[j & 1], j >> 1) && (j < edge0 || wait(clean, j - edge0)))) break;
                        if (j + 1 >= edge0 && j + 1 < n) mbar_arrive(near);
                        for (int h = 0; h < L::HALVES; ++h)
                            mma_tb_half<DP>(tmem + L::DQ_COL, tmem + L::S_COL + (uint32_t)(DP * (j & 1) + 64 * h),
                                            k_s + (uint32_t)(j % L::KS) * L::MOVING, h, j > 0 || h > 0);
                        tc_commit(&k_empty[j % L::KS]);
                    }
                    if (ok) tc_commit(dq_full);
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
                }
            } else if (warp >= L::W_TMEM && warp < L::W_TMEM + 2) {
                // dS is 0 for keys that a row does not see, but 0 times K need not be: rows behind the sequence's keys
                // become zero, as do infinities and NaN of keys that some row does not see (add_nonfinite gives them
                // back to the rows that do).  Done here, when S has read the tile, while dS is formed.
                const int lane = (int)threadIdx.x - 32 * L::W_TMEM;
                bool ok = true;
                for (int j = edge0; j < n && ok; ++j) {
                    ok = mbar_wait(near, (uint32_t)(j - edge0) & 1u, abort_flag, p.err, ERR_DQ_CLEAN) &&
                         mbar_wait(&s_full[j & 1], (uint32_t)(j >> 1) & 1u, abort_flag, p.err, ERR_DQ_CLEAN);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t tile = smem_u32(s_k + (j % L::KS) * L::MOVING);
                    const int behind = lk - j * L::STEP;
                    if (behind < L::STEP) zero_rows<DP>(tile, behind, L::STEP, lane, 64);
                    if (clean_rows<DP>(tile, max(0, row0 + shift + 1 - j * L::STEP), L::STEP, min(L::STEP, behind), lane, 64)) *poisoned = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) mbar_arrive(clean);
                }
            }
        } else {
            regs_more<L::REGS_MATH>();
            const int t = (int)(threadIdx.x & 127u), half = (int)(warp >> 2);
            const uint32_t lane_base = (warp & 3u) * 32u << 16;
            const int row = row0 + t;
            const bool live = row < lq;
            const size_t stat = (size_t)head * p.total_q + q0 + (live ? row : 0);
            const float c = p.scale * AT_LOG2E;
            // D of the rows: 16 bytes a lane, whole rows a warp, all loads in flight at once (a row per thread
            // reads 32 lines a load: 12000 cycles)
            {
                constexpr int LANES = DP / 8, ROWS = 32 / LANES, PER_WARP = 32 / L::HALVES, TURNS = PER_WARP / ROWS;
                const int lane = t & 31, r0 = (int)warp * PER_WARP + lane / LANES, col = lane % LANES * 8;
                uint4 x[TURNS], y[TURNS];
#pragma unroll
                for (int i = 0; i < TURNS; ++i) {
                    const long long r = row0 + r0 + i * ROWS;
                    x[i] = y[i] = make_uint4(0, 0, 0, 0);
                    if (r < lq && col < p.d) {
                        x[i] = *reinterpret_cast<const uint4*>(p.go.p + (q0 + r) * p.go.rs + (long long)head * p.go.hs + col);
                        y[i] = *reinterpret_cast<const uint4*>(p.out.p + (q0 + r) * p.out.rs + (long long)head * p.out.hs + col);
                    }
                }
#pragma unroll
                for (int i = 0; i < TURNS; ++i) {
                    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, v[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), sum);
                        sum = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), __uint_as_float(v[e] & 0xFFFF0000u), sum);
                    }
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane % LANES == 0) exch[r0 + i * ROWS] = sum;
                }
            }
            const float lse2 = live ? p.lse[stat] * AT_LOG2E : 0.f;
            math_sync<DP>();
            float D = exch[t];
            const uint64_t c2 = pack2(c, c), l2 = pack2(-lse2, -lse2);
            float rest = 0.f;                   // sum of dS: 0 but for the rounding of O in D
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                // (with one step the warps meet in barriers: one whose wait gave up goes on without waiting)
                ok = mbar_wait(&s_full[j & 1], (uint32_t)(j >> 1) & 1u, abort_flag, p.err, ERR_DQ_MATH);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok && n > 1) break;
                tc_fence_after();
                const uint32_t s_t = tmem + lane_base + L::S_COL + (uint32_t)(DP * (j & 1) + 64 * half);
                uint32_t s[2][32];
                load64(s_t, s);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const uint64_t x2 =
                        fma2(pack2(__uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1])), c2, l2);
                    float x, y;
                    if (i / 2 % 8 < L::ON_FMA) {
                        exp2_pair(x2, x, y);
                    } else {
                        unpack2(x2, x, y);
                        x = ex2(x);
                        y = ex2(y);
                    }
                    s[i / 32][i % 32] = __float_as_uint(x);
                    s[i / 32][i % 32 + 1] = __float_as_uint(y);
                }
                ok = ok && mbar_wait(dp_full, (uint32_t)j & 1u, abort_flag, p.err, ERR_DQ_MATH);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok && n > 1) break;
                tc_fence_after();
                uint32_t dp[2][32];
                load64(tmem + lane_base + L::DP_COL + 64u * half, dp);
                tc_fence_before();
                mbar_arrive(dp_read);
                int seen = row + shift - j * L::STEP - 64 * half;           // column of the last seen key
                const bool edge = (j + 1) * L::STEP > row0 + shift + 1;
                if (n == 1) {
                    // few keys: O's rounding in D is not small beside dP, and D = sum_j P_ij dP_ij is at hand
                    uint64_t d4[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
                    float x, y;
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        unpack2(mul2(pack2(__uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1])),
                                     pack2(__uint_as_float(dp[i / 32][i % 32]), __uint_as_float(dp[i / 32][i % 32 + 1]))), x, y);
                        d4[i / 2 & 1] = add2(d4[i / 2 & 1], pack2(i > seen ? 0.f : x, i + 1 > seen ? 0.f : y));
                    }
                    unpack2(add2(d4[0], d4[1]), x, y);
                    D = x + y;
                    if (L::HALVES == 2) {
                        math_sync<DP>();
                        exch[half * 128 + t] = D;
                        math_sync<DP>();
                        D += exch[(half ^ 1) * 128 + t];
                    }
                }
                if (row + shift == 0 && isfinite(D)) seen = -1;             // one key: P = 1 and dS = 0, exactly
                const uint64_t d2 = pack2(-D, -D);
                uint32_t ds[32];
                uint64_t sum2 = pack2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    uint64_t v = mul2(pack2(__uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1])),
                                      add2(pack2(__uint_as_float(dp[i / 32][i % 32]), __uint_as_float(dp[i / 32][i % 32 + 1])), d2));
                    if (edge) {
                        float x, y;
                        unpack2(v, x, y);
                        v = pack2(i > seen ? 0.f : x, i + 1 > seen ? 0.f : y);
                    }
                    sum2 = add2(sum2, v);
                    float x, y;
                    unpack2(v, x, y);
                    ds[i / 2] = bf16x2(x, y);
                }
                float a, b;
                unpack2(sum2, a, b);
                rest += a + b;
                tmem_st_32x32b_x32(s_t, ds);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&ds_ready[j & 1]);
            }
            if (ok && n > 0) {
                ok = mbar_wait(dq_full, 0, abort_flag, p.err, ERR_DQ_MATH);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            // sum_j P_ij = 1, so D + sum_j dS_ij is sum_j P_ij dP_ij without O's rounding: the
            // second kernel takes that
            if (L::HALVES == 2) {
                math_sync<DP>();
                exch[half * 128 + t] = rest;
                math_sync<DP>();
                rest += exch[(half ^ 1) * 128 + t];
            }
            if (ok) {
                if (half == 0 && live) p.delta[stat] = D + rest;
                // a key with an infinity or NaN has a logit of -inf, which leaves dS = 0 and the product 0 * x, or one that
                // makes lse NaN, and with it the whole row
                if (n > 0 && __any_sync(0xffffffffu, *poisoned != 0))
                    add_nonfinite<2 / L::HALVES>(p.k, p.d, tmem + lane_base + L::DQ_COL + 64u * half, 64 * half, 0.f,
                                                 k0 + max(0, row0 + shift + 1), k0 + row + shift, live, kv_head);
                for (int h = half; h < 2; h += L::HALVES)
                    store_rows<DP>(tmem + lane_base + L::DQ_COL + (uint32_t)(h * (DP / 2)), n > 0, n == 0, p.scale,
                                   smem_u32(s_q), h, (int)(warp & 3u) * 32, lq - row0,
                                   p.dq.p + (long long)(q0 + row0) * p.dq.rs + (long long)head * p.dq.hs, p.dq.rs, p.d);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::W_TMEM) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// ============================================================================ dK, dV

template <int DP>
struct DkvLayout : BwLayout<DP> {
    using Base = BwLayout<DP>;
    static constexpr int SLOTS = DP == 64 ? 3 : 2;              // of q and of dO
    static constexpr int BARRIERS = 2 + 4 * SLOTS + 9;
    static constexpr int ONES = 128 * 16 * 2, EXTRA = Base::STEP * 16 * 2;      // 16 more columns of the tiles
    static constexpr int SMEM = 1024 + ONES + 4 * EXTRA + 2 * Base::OWN + 2 * SLOTS * Base::MOVING + 8 * BARRIERS + 64;
    static constexpr uint32_t S_COL = 0, DP_COL = DP, DK_COL = 2 * DP, DV_COL = 3 * DP;
    static_assert(SMEM <= Base::MOST_SMEM, "shared memory above the SM's 228 KiB");
    static_assert((ONES + 4 * EXTRA) % 1024 == 0, "the tiles behind the extra columns start a swizzle atom");
};

template <int DP>
__global__ void __launch_bounds__(BwLayout<DP>::THREADS, BwLayout<DP>::CTAS)
attention_dkv_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ BwMaps maps) {
    using L = DkvLayout<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // the extra columns: ones beside K and V, two turns of those beside Q and beside dO
    uint8_t *s_ones = smem, *s_lse = s_ones + L::ONES, *s_d = s_lse + 2 * L::EXTRA;
    uint8_t *s_k = s_d + 2 * L::EXTRA, *s_v = s_k + L::OWN, *s_q = s_v + L::OWN, *s_do = s_q + L::SLOTS * L::MOVING;
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(s_do + L::SLOTS * L::MOVING);
    uint64_t* extra_ready = kv_full + 1;        // the ones, and the first item's columns
    uint64_t *q_full = extra_ready + 1, *q_empty = q_full + L::SLOTS, *do_full = q_empty + L::SLOTS, *do_empty = do_full + L::SLOTS;
    uint64_t *s_full = do_empty + L::SLOTS, *dp_full = s_full + 1, *p_ready = dp_full + 1, *ds_ready = p_ready + 2,
             *dkv_full = ds_ready + 1, *near = dkv_full + 1, *clean_do = near + 1, *clean_q = clean_do + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clean_q + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* found = reinterpret_cast<int*>(tmem_slot + 2);
    int4* info = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 3) + 15) & ~uintptr_t(15));

    const uint32_t warp = warp_id();
    const int kv_head = (int)(blockIdx.x % (unsigned)p.hk);
    pdl_trigger();
    // No wait here: of the first kernel's work only D is read, below, and that kernel let this one
    // start when all work before it was done.
    if (warp == 0) {
        SeqTile t;
        // first blocks of a sequence first: most queries see them
        const bool ok = find_tile(p, true, AT_ROWS, (int)(blockIdx.x / (unsigned)p.hk), blockIdx.x, t);
        if (elect_one()) {
            *found = ok;
            info[0] = make_int4(t.q0, t.lq, t.k0, t.lk);
            info[1] = make_int4(t.block, 0, 0, 0);
        }
    } else if (warp == L::W_TMEM) {
        tmem_alloc(tmem_slot, L::TMEM_COLS);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(kv_full, 1);
        mbar_init(extra_ready, L::MATH);
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&do_full[i], 1);
            mbar_init(&do_empty[i], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(&p_ready[0], L::MATH);        // the first, then the last 32 columns of both halves
        mbar_init(&p_ready[1], L::MATH);
        mbar_init(ds_ready, L::MATH);
        mbar_init(dkv_full, 1);
        mbar_init(near, 1);                     // the next edge item may be cleaned
        mbar_init(clean_do, 2);                 // its dO is fit for P^T dO
        mbar_init(clean_q, 2);                  // its Q is fit for dS^T Q
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
        const int key0 = info[1].x * AT_ROWS, shift = lk - lq;
        const int tiles = (lq + L::STEP - 1) / L::STEP, first = max(0, key0 - shift) / L::STEP;   // query tiles that see any of the keys
        const int per_head = max(0, tiles - first), n = per_head * p.group;
        // item `it`: query tile first + it % per_head of head kv_head * group + it / per_head; an edge item holds
        // queries that do not see every key of the CTA, or rows behind the sequence's queries
        const int diagonal = max(0, key0 + AT_ROWS - 1 - shift + L::STEP - 1) / L::STEP, partial = lq / L::STEP;
        auto is_edge = [&](int tile) { return tile < diagonal || tile >= partial; };

        if (warp >= L::W_TMA) {
            regs_less<L::REGS_OTHER>();     // one instruction for all warps of the group
            if (warp == L::W_TMA) {
                if (elect_one() && n > 0) {
                    mbar_arrive_expect_tx(kv_full, 2 * L::OWN);
                    load_tile<DP, 128, AT_BWD_BOX>(s_k, &maps.k, kv_full, kv_head, k0 + key0);
                    load_tile<DP, 128, AT_BWD_BOX>(s_v, &maps.v, kv_full, kv_head, k0 + key0);
                    bool ok = true;
                    int tile = first, head = kv_head * p.group;
                    for (int it = 0; it < n + L::SLOTS; ++it) {     // the last turns only wait for the loads to be used
                        const int slot = it % L::SLOTS;
                        const uint32_t par = ((uint32_t)(it / L::SLOTS) & 1u) ^ 1u;
                        if (!mbar_wait(&q_empty[slot], par, abort_flag, p.err, ERR_DKV_LOAD)) { ok = false; break; }
                        if (it < n) {
                            mbar_arrive_expect_tx(&q_full[slot], L::MOVING);
                            load_tile<DP, L::STEP, AT_BWD_BOX>(s_q + slot * L::MOVING, &maps.q, &q_full[slot], head, q0 + tile * L::STEP);
                        }
                        if (!mbar_wait(&do_empty[slot], par, abort_flag, p.err, ERR_DKV_LOAD)) { ok = false; break; }
                        if (it < n) {
                            mbar_arrive_expect_tx(&do_full[slot], L::MOVING);
                            load_tile<DP, L::STEP, AT_BWD_BOX>(s_do + slot * L::MOVING, &maps.go, &do_full[slot], head, q0 + tile * L::STEP);
                        }
                        if (++tile == tiles) { tile = first; ++head; }
                    }
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
                }
            } else if (warp == L::W_MMA) {
                if (elect_one() && n > 0) {
                    const uint32_t k_s = smem_u32(s_k), v_s = smem_u32(s_v), q_s = smem_u32(s_q), do_s = smem_u32(s_do);
                    auto wait = [&](uint64_t* b, int use) {
                        const bool ok = mbar_wait(b, (uint32_t)use & 1u, abort_flag, p.err, ERR_DKV_MMA);
                        tc_fence_after();
                        return ok;
                    };
                    // S^T - lse / scale and dP^T - D
                    const uint32_t ones_s = smem_u32(s_ones), lse_s = smem_u32(s_lse), d_s = smem_u32(s_d);
                    auto do_s_product = [&](int it, uint32_t q) {
                        mma_abt<DP, L::STEP>(tmem + L::S_COL, k_s, q);
                        mma_extra<L::STEP>(tmem + L::S_COL, ones_s, lse_s + (uint32_t)(it & 1) * L::EXTRA);
                        tc_commit(s_full);
                    };
                    auto do_dp_product = [&](int it, uint32_t dout) {
                        mma_abt<DP, L::STEP>(tmem + L::DP_COL, v_s, dout);
                        mma_extra<L::STEP>(tmem + L::DP_COL, ones_s, d_s + (uint32_t)(it & 1) * L::EXTRA);
                        tc_commit(dp_full);
                    };
                    auto q_at = [&](int it) { return q_s + (uint32_t)(it % L::SLOTS) * L::MOVING; };
                    auto do_at = [&](int it) { return do_s + (uint32_t)(it % L::SLOTS) * L::MOVING; };
                    bool ok = wait(kv_full, 0) && wait(&q_full[0], 0) && wait(extra_ready, 0);
                    if (ok) do_s_product(0, q_at(0));
                    ok = ok && wait(&do_full[0], 0);
                    if (ok) do_dp_product(0, do_at(0));
                    int tile = first, edges = 0;
                    for (int it = 0; it < n && ok; ++it) {
                        const bool more = it + 1 < n, edge = is_edge(tile);
                        if (++tile == tiles) tile = first;
                        if (it == 0 && edge) mbar_arrive(near);
                        for (int c = 0; c < 2 && ok; ++c) {
                            if (!(ok = wait(&p_ready[c], it))) break;
                            if (c == 0 && edge && !(ok = wait(clean_do, edges))) break;
                            for (int h = 0; h < L::HALVES; ++h)
                                mma_tb_quarter<DP>(tmem + L::DV_COL, tmem + L::S_COL + 64u * h + 16u * c, do_at(it), 2 * h + c,
                                                   it > 0 || c > 0 || h > 0);
                        }
                        if (!ok) break;
                        tc_commit(&do_empty[it % L::SLOTS]);
                        if (more && is_edge(tile)) mbar_arrive(near);
                        // (here already: the next item's Q may be cleaned as soon as its S^T is there)
                        if (edge && !(ok = wait(clean_q, edges++))) break;
                        if (more) {
                            // the next S^T takes the place of P^T: products run in order
                            if (!(ok = wait(&q_full[(it + 1) % L::SLOTS], (it + 1) / L::SLOTS))) break;
                            do_s_product(it + 1, q_at(it + 1));
                        }
                        if (!(ok = wait(ds_ready, it))) break;
                        for (int h = 0; h < L::HALVES; ++h)
                            mma_tb_half<DP>(tmem + L::DK_COL, tmem + L::DP_COL + 64u * h, q_at(it), h, it > 0 || h > 0);
                        tc_commit(&q_empty[it % L::SLOTS]);
                        if (more) {
                            if (!(ok = wait(&do_full[(it + 1) % L::SLOTS], (it + 1) / L::SLOTS))) break;
                            do_dp_product(it + 1, do_at(it + 1));
                        }
                    }
                    if (ok) tc_commit(dkv_full);
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
                }
            } else if (warp >= L::W_TMEM && warp < L::W_TMEM + 2) {
                // P and dS are 0 for queries that do not see a key, but 0 times dO or Q need not be: rows behind the
                // sequence's queries become zero, as do infinities and NaN of queries that do not see every key (keys
                // that they see get NaN all the same: by lse, or by D, which is not finite then).  Done here while S and
                // P are formed: dO when it has arrived (what dP^T makes of the rows that change does not matter, as P
                // is NaN or 0 there), Q when S^T has read it.
                const int lane = (int)threadIdx.x - 32 * L::W_TMEM;
                bool ok = true;
                int tile = first, edges = 0;
                for (int it = 0; it < n && ok; ++it) {
                    const int row0 = tile * L::STEP, slot = it % L::SLOTS;
                    const bool edge = is_edge(tile);
                    if (++tile == tiles) tile = first;
                    if (!edge) continue;
                    const int behind = lq - row0, blind = min(min(L::STEP, behind), key0 + AT_ROWS - 1 - shift - row0);
                    // (one loop and one copy of its code: few CTAs find it in the instruction cache)
#pragma unroll 1
                    for (int i = 0; i < 3 && ok; ++i) {
                        uint64_t* bar = i == 0 ? near : i == 1 ? &do_full[slot] : s_full;
                        const uint32_t use = (uint32_t)(i == 0 ? edges++ : i == 1 ? it / L::SLOTS : it);
                        ok = mbar_wait(bar, use & 1u, abort_flag, p.err, ERR_DKV_CLEAN);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok || i == 0) continue;
                        const uint32_t tile_s = smem_u32((i == 1 ? s_do : s_q) + slot * L::MOVING);
                        zero_rows<DP>(tile_s, behind, L::STEP, lane, 64);
                        clean_rows<DP>(tile_s, 0, L::STEP, blind, lane, 64);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (elect_one()) mbar_arrive(i == 1 ? clean_do : clean_q);
                    }
                }
            }
        } else {
            regs_more<L::REGS_MATH>();
            const int t = (int)(threadIdx.x & 127u), half = (int)(warp >> 2);
            const uint32_t lane_base = (warp & 3u) * 32u << 16;
            const int key = key0 + t;
            const float c = p.scale * AT_LOG2E;
            const uint64_t c2 = pack2(c, c);
            const uint32_t s_t = tmem + lane_base + L::S_COL + 64u * half, dp_t = tmem + lane_base + L::DP_COL + 64u * half;
            bool ok = true;
            int tile = first, head = kv_head * p.group;
            // the first half of the threads brings lse, the other one D, of a row of an item each: fetched two
            // items ahead, written one ahead (the item before has left the turn's columns by then)
            const bool brings_d = (int)threadIdx.x >= L::STEP;
            const int brings = (int)threadIdx.x % L::STEP;
            int f_tile = first, f_head = head;
            auto fetch = [&](int item) {
                const int row = f_tile * L::STEP + brings;
                float v = 0.f;
                if (item < n && row < lq) v = (brings_d ? p.delta : p.lse)[(size_t)f_head * p.total_q + q0 + row];
                if (++f_tile == tiles) { f_tile = first; ++f_head; }
                return v;
            };
            const float inv_scale = 1.f / p.scale;
            const uint32_t extra_s = smem_u32(brings_d ? s_d : s_lse) + extra_at(brings);
            auto put = [&](int item, float v) {
                v = brings_d ? -v : -v * inv_scale;
                const float hi = __bfloat162float(__float2bfloat16_rn(v));
                const float mid = __bfloat162float(__float2bfloat16_rn(v - hi));
                const uint32_t at = extra_s + (uint32_t)(item & 1) * L::EXTRA;
                asm volatile("st.shared.b32 [%0], %1;" :: "r"(at), "r"(bf16x2(hi, mid)) : "memory");
                asm volatile("st.shared.b16 [%0], %1;" :: "r"(at + 4u), "h"((uint16_t)bf16x2(v - hi - mid, 0.f)) : "memory");
                // 0 * D in the fourth column beside Q: a row whose D is not finite gets P = NaN where it sees a key
                if (brings_d)
                    asm volatile("st.shared.b16 [%0], %1;" :: "r"(at - 2u * L::EXTRA + 6u), "h"((uint16_t)bf16x2(0.f * v, 0.f)) : "memory");
            };
            float next = 0.f;
            pdl_wait();                             // D is there
            if (n > 0) {
                // columns 0-3 of the ones are 1, what is not written below of the extra columns 0
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int i = (int)threadIdx.x; i < (L::ONES + 4 * L::EXTRA) / 16; i += L::MATH) sts128(smem_u32(smem) + 16u * i, zero);
                math_sync<DP>();
                if (half == 0) sts128(smem_u32(s_ones) + extra_at(t), make_uint4(0x3F803F80u, 0x3F803F80u, 0u, 0u));
                put(0, fetch(0));
                next = fetch(1);
                fence_proxy_async_smem();
                mbar_arrive(extra_ready);
            }
            for (int it = 0; it < n; ++it) {
                if (it + 1 < n) {
                    put(it + 1, next);
                    fence_proxy_async_smem();       // p_ready below orders it before the products
                    next = fetch(it + 2);
                }
                const int row0 = tile * L::STEP;
                const bool edge = is_edge(tile);
                if (++tile == tiles) { tile = first; ++head; }
                // query i of the tile sees this thread's key when i >= unseen; rows from lq on are none
                const int unseen = key - shift - row0 - 64 * half, live = lq - row0 - 64 * half;

                ok = mbar_wait(s_full, (uint32_t)it & 1u, abort_flag, p.err, ERR_DKV_MATH);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[2][32];
                load64(s_t, s);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const uint64_t x2 = mul2(pack2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2);
                        float a, b;
                        if (i / 2 % 8 < L::ON_FMA) {
                            exp2_pair(x2, a, b);
                        } else {
                            unpack2(x2, a, b);
                            a = ex2(a);
                            b = ex2(b);
                        }
                        s[q][i] = __float_as_uint(a);
                        s[q][i + 1] = __float_as_uint(b);
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * q + i < unseen || 32 * q + i >= live) s[q][i] = 0u;
                    }
                    uint32_t pr[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) pr[i] = bf16x2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1]));
                    tmem_st_32x32b_x16(s_t + 16u * q, pr);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&p_ready[q]);
                }

                ok = mbar_wait(dp_full, (uint32_t)it & 1u, abort_flag, p.err, ERR_DKV_MATH);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t dp[2][32], pr[32];
                load64(dp_t, dp);
                if (edge) {         // P is 0 there, but dP - D need not be finite
                    // (the first query that sees key 0 sees no other: its P is 1 and dS 0, exactly)
                    const int first_ds = key == 0 ? unseen + 1 : unseen;
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (i < first_ds || i >= live) dp[i / 32][i % 32] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const uint32_t *x = &s[i / 32][i % 32], *y = &dp[i / 32][i % 32];
                    float a, b;
                    unpack2(mul2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                 pack2(__uint_as_float(y[0]), __uint_as_float(y[1]))), a, b);
                    pr[i / 2] = bf16x2(a, b);
                }
                tmem_st_32x32b_x32(dp_t, pr);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(ds_ready);
            }
            if (ok && n > 0) {
                ok = mbar_wait(dkv_full, 0, abort_flag, p.err, ERR_DKV_MATH);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            if (ok) {
                for (int h = half; h < 2; h += L::HALVES) {
                    const uint32_t col = (uint32_t)(h * (DP / 2));
                    store_rows<DP>(tmem + lane_base + L::DK_COL + col, n > 0, n == 0, p.scale, smem_u32(s_k), h,
                                   (int)(warp & 3u) * 32, lk - key0,
                                   p.dk.p + (long long)(k0 + key0) * p.dk.rs + (long long)kv_head * p.dk.hs, p.dk.rs, p.d);
                    store_rows<DP>(tmem + lane_base + L::DV_COL + col, n > 0, n == 0, 1.f, smem_u32(s_v), h,
                                   (int)(warp & 3u) * 32, lk - key0,
                                   p.dv.p + (long long)(k0 + key0) * p.dv.rs + (long long)kv_head * p.dv.hs, p.dv.rs, p.d);
                }
            }
        }
    }
    pdl_wait();             // whatever this CTA had to do: the grid ends after the first kernel's
    tc_fence_before();
    __syncthreads();
    if (warp == L::W_TMEM) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

template <int DP>
cudaError_t launch_bwd(const AttnParams& p, const BwMaps& maps, cudaStream_t s) {
    using L = BwLayout<DP>;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(attention_dq_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, DqLayout<DP>::SMEM)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(attention_dkv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvLayout<DP>::SMEM)) != cudaSuccess) return e;
    // a warpgroup that asks for more registers than the launch left would wait for good
    static const int regs = [] {
        cudaFuncAttributes a, b;
        return cudaFuncGetAttributes(&a, attention_dq_kernel<DP>) == cudaSuccess &&
               cudaFuncGetAttributes(&b, attention_dkv_kernel<DP>) == cudaSuccess ? std::min(a.numRegs, b.numRegs) : 0;
    }();
    if (regs < L::REGS) return cudaErrorInvalidConfiguration;
    if (p.total_q > 0) {
        e = launch_pdl(attention_dq_kernel<DP>, dim3(seq_blocks(p.total_q, AT_ROWS, p.n_seqs) * (unsigned)p.hq), dim3(L::THREADS),
                       DqLayout<DP>::SMEM, s, p, maps);
        if (e != cudaSuccess) return e;
    }
    if (p.total_k == 0) return cudaSuccess;
    // (without queries the kernel before is another one's, and its CTAs wait for nothing they read: cu_seqlens
    // and the zeros they write come after a plain launch)
    if (p.total_q == 0) {
        attention_dkv_kernel<DP><<<seq_blocks(p.total_k, AT_ROWS, p.n_seqs) * (unsigned)p.hk, L::THREADS, DkvLayout<DP>::SMEM, s>>>(p, maps);
        return cudaGetLastError();
    }
    return launch_pdl(attention_dkv_kernel<DP>, dim3(seq_blocks(p.total_k, AT_ROWS, p.n_seqs) * (unsigned)p.hk), dim3(L::THREADS),
                      DkvLayout<DP>::SMEM, s, p, maps);
}

}  // namespace

cudaError_t launch_attention_backward(const AttnParams& p, const HeadMaps& m, cudaStream_t s) {
    if (p.n_seqs == 0) return cudaSuccess;
    const BwMaps maps{m.q, m.k, m.v, m.go};
    return p.d <= 64 ? launch_bwd<64>(p, maps, s) : launch_bwd<128>(p, maps, s);
}

}  // namespace muon
