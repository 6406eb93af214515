// attention_fwd.cu -- packed causal attention with grouped heads: O = softmax(S) V, the
// log-sums of the rows and each head's largest logit.
//
// A query tile has 128 rows, an MMA warp and a softmax warpgroup; K and V tiles of 128 rows
// stream through a ring in shared memory.  For each key tile
//
//   S = Q K^T      both operands from shared memory, 128 x 128 fp32 in tensor memory
//   P = exp(S - m) a thread owns a row, so its maximum and sum need no exchange
//   O += P V       P is written back to tensor memory as bf16 and is the A operand there; it
//                  starts when the first 64 keys of P are there
//
// m is the maximum that P and O are scaled by; it follows the true maximum only when that has
// grown by 2^8, so that O is rescaled rarely (P stays below 2^8; sums and O are fp32, and P's
// rounding to bf16 is relative).
//
// The special function unit takes 8 cycles for a warp's exponentials, 1024 for 128 x 128: as
// long as the two products of a 128-wide head take, twice as long as those of a 64-wide one.
// So a quarter of a 64-wide head's and an eighth of a 128-wide one's are computed on the FMA
// pipe (exp2_pair), at 12 cycles a warp; the best mix of the two gets to 7.5 where the unit
// alone gets to 8.6.
//
// One B200: 8192 rows in 5 sequences (the longest 6500), 32 heads over 8 of 128: 338 us at full
// clocks (1.05 PFLOP/s, tensor pipe 52 % and special function unit 45 % of the cycles) to 396
// under the power cap.  8 sequences of 1024, 25 heads of 64: 66-74 us; a CTA has 4.5 key tiles
// there, and its start and end take as long as they do.
//
// O is divided by the sum of P at the end, so values beyond fp32's range / (2^8 keys) overflow
// where their mean would not.
//
// P is 0 where a row does not see a key (exp2_pair and ex2 both give 0 for -inf), but 0 times
// an infinity or a NaN is not: a spare warp takes those out of V in the tiles that not every
// row sees all of, beside the softmax, and what it took out is added again at the end to the
// rows that see it (66 us against 65 without).
#include <algorithm>

#include "attention.cuh"
#include "kernels.cuh"

namespace muon {
namespace {

// 128-wide heads: two query tiles a CTA, one CTA an SM, and P in the place of S.  64-wide
// heads: one tile, two CTAs an SM, which also hide each other's start and end, and P apart
// from S, so that the next S need not wait for P V.
template <int DP>
struct FwLayout {
    static constexpr int TILES = DP == 64 ? 1 : 2;
    static constexpr int SOFTMAX = TILES * 128;                     // softmax threads
    static constexpr int THREADS = SOFTMAX + 128;                   // + a warpgroup: TMA, an MMA warp per tile, tensor memory
    static constexpr int CTAS = 2 / TILES;                          // of an SM
    static constexpr int W_TMA = SOFTMAX / 32, W_MMA = W_TMA + 1, W_TMEM = W_TMA + 3;
    static constexpr int W_CLEAN = W_MMA + TILES, CLEANERS = 3 - TILES;     // W_TMEM and, with one tile, the warp before it
    // registers a thread: at launch, then of the softmax warpgroups and the other one
    static constexpr int REGS = TILES == 1 ? 128 : 168;
    static constexpr int REGS_SOFTMAX = TILES == 1 ? 200 : 216, REGS_OTHER = TILES == 1 ? 56 : 72;
    static_assert(SOFTMAX * REGS_SOFTMAX + 128 * REGS_OTHER <= THREADS * REGS, "more registers than launched with");
    static constexpr int TILE = DP / 64 * AT_CHUNK;                 // bytes of a q, k or v tile
    static constexpr int SLOTS = 5;                                 // ring of k and v tiles
    static constexpr int EDGES = TILES + 1;                         // most key tiles that not every row sees all of
    static constexpr int BARRIERS = 1 + 2 * SLOTS + 6 * TILES + 1 + EDGES;
    static constexpr int SMEM = (TILES + SLOTS) * TILE + 8 * BARRIERS + 64;
    static constexpr bool P_APART = DP == 64;
    static constexpr uint32_t TMEM_COLS = 512 / CTAS;
    static constexpr uint32_t S_COL = 0;                            // + 128 per tile
    static constexpr uint32_t P_COL = P_APART ? 128 : 0;            // + 128 per tile, P_HALF per 64 keys
    static constexpr uint32_t P_HALF = P_APART ? 32 : 64;
    static constexpr uint32_t O_COL = P_APART ? 192 : 256;          // + DP per tile
    static constexpr int ON_FMA = DP == 64 ? 2 : 1;                 // of 8 pairs of exponentials
    static_assert(SMEM <= 232448 / CTAS - (CTAS - 1) * 1024, "shared memory above the SM's 228 KiB");
};

struct FwMaps {
    CUtensorMap q, k, v;
};

constexpr int ERR_FW_LOAD = 0x201, ERR_FW_MMA = 0x202, ERR_FW_SOFTMAX = 0x203, ERR_FW_ALIGN = 0x204,
              ERR_FW_CLEAN = 0x205;

// Raises *addr to v.  Signed order of the bits is the order of non-negative floats, the
// reverse unsigned order that of negative ones.
__device__ __forceinline__ void atomic_max_float(float* addr, float v) {
    v += 0.f;                                   // -0 counts as +0
    if (v >= 0.f) atomicMax(reinterpret_cast<int*>(addr), __float_as_int(v));
    else if (v < 0.f) atomicMin(reinterpret_cast<unsigned*>(addr), __float_as_uint(v));
}

template <int DP>
__global__ void __launch_bounds__(FwLayout<DP>::THREADS, FwLayout<DP>::CTAS)
attention_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FwMaps maps) {
    using L = FwLayout<DP>;
    constexpr int TILES = L::TILES;
    extern __shared__ __align__(1024) uint8_t smem[];       // no room to align it here: 128-byte swizzled tiles
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, ERR_FW_ALIGN);
        return;
    }
    uint8_t* sq = smem;
    uint8_t* ring = smem + TILES * L::TILE;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + L::SLOTS * L::TILE);
    uint64_t* full = q_full + 1;
    uint64_t* empty = full + L::SLOTS;
    uint64_t* s_full = empty + L::SLOTS;        // per tile, as the following ones
    uint64_t* s_read = s_full + TILES;          // the softmax has S in registers (P_APART)
    uint64_t* p_ready = s_read + TILES;         // two: for each half of the keys
    uint64_t* pv_done = p_ready + 2 * TILES;    // P has been read, O holds it
    uint64_t* o_full = pv_done + TILES;
    uint64_t* near = o_full + TILES;            // the next edge tile may be cleaned
    uint64_t* clean = near + 1;                 // per edge tile: its V is fit for the product
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clean + L::EDGES);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* found = reinterpret_cast<int*>(tmem_slot + 2);
    volatile int* poisoned = reinterpret_cast<volatile int*>(tmem_slot + 3);      // infinities or NaN of V were set to zero
    int4* info = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 15) & ~uintptr_t(15));

    const uint32_t warp = warp_id();
    const int head = (int)(blockIdx.x % (unsigned)p.hq);
    pdl_trigger();
    pdl_wait();             // cu_seqlens, too, may be the previous kernel's
    if (warp == 0) {
        SeqTile t;
        const bool ok = find_tile(p, false, TILES * AT_ROWS, (int)(blockIdx.x / (unsigned)p.hq), blockIdx.x, t);
        if (elect_one()) {
            *found = ok;
            info[0] = make_int4(t.q0, t.lq, t.k0, t.lk);
            // long rows first: the last blocks of a sequence see the most keys
            info[1] = make_int4(ok ? t.blocks - 1 - t.block : 0, 0, 0, 0);
        }
    } else if (warp == L::W_TMEM) {
        tmem_alloc(tmem_slot, L::TMEM_COLS);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        mbar_init(q_full, 1);
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], TILES);
        }
        for (int i = 0; i < TILES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_read[i], 128);
            mbar_init(&p_ready[2 * i], 128);
            mbar_init(&p_ready[2 * i + 1], 128);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_full[i], 1);
        }
        *abort_flag = 0;
        *poisoned = 0;
        mbar_init(near, 1);
        for (int i = 0; i < L::EDGES; ++i) mbar_init(&clean[i], L::CLEANERS);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (*found) {
        const int4 sl = info[0];
        const int q0 = sl.x, lq = sl.y, k0 = sl.z, lk = sl.w;
        const int row0 = info[1].x * (TILES * AT_ROWS);          // of the CTA, in the sequence
        const int shift = lk - lq;                                  // row i sees keys up to i + shift
        const int kv_head = head / p.group;
        // key tiles that a tile's rows see, and keys
        int n[TILES], keys[TILES];
#pragma unroll
        for (int w = 0; w < TILES; ++w) {
            const int first = row0 + w * AT_ROWS, last = min(first + AT_ROWS, lq) - 1 + shift;
            n[w] = first >= lq || last < 0 ? 0 : last / AT_ROWS + 1;
            keys[w] = last + 1;
        }
        const int nmax = max(n[0], n[TILES - 1]), nmin = min(n[0], n[TILES - 1]);

        // Key tiles from this one on hold keys that some row does not see.
        const int edge0 = max(0, row0 + shift + 1) / AT_ROWS;

        if (warp >= L::W_TMA) {
            regs_less<L::REGS_OTHER>();     // one instruction for all warps of the group
            if (warp == L::W_TMA) {
                if (elect_one() && nmax > 0) {
                    mbar_arrive_expect_tx(q_full, TILES * L::TILE);
                    for (int w = 0; w < TILES; ++w)
                        load_tile<DP, AT_ROWS, AT_ROWS>(sq + w * L::TILE, &maps.q, q_full, head, q0 + row0 + w * AT_ROWS);
                    // ring order: K0, K1, V0, K2, V1, ...: the order of use
                    int slot = 0;
                    uint32_t phase = 0;
                    bool ok = true;
                    for (int i = 0; i < 2 * nmax && ok; ++i) {
                        const bool is_v = i > 0 && (i % 2 == 0 || i == 2 * nmax - 1);
                        const int j = i == 0 ? 0 : is_v ? (i == 2 * nmax - 1 ? nmax - 1 : i / 2 - 1) : (i + 1) / 2;
                        if (!mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.err, ERR_FW_LOAD)) { ok = false; break; }
                        mbar_arrive_expect_tx(&full[slot], L::TILE);
                        load_tile<DP, AT_ROWS, AT_ROWS>(ring + slot * L::TILE, is_v ? &maps.v : &maps.k, &full[slot], kv_head,
                                                        k0 + j * AT_ROWS);
                        if (++slot == L::SLOTS) { slot = 0; phase ^= 1u; }
                    }
                    // every load has landed before the CTA may end
                    for (int i = 0; i < L::SLOTS && ok; ++i) {
                        if (!mbar_wait(&empty[slot], phase ^ 1u, abort_flag, p.err, ERR_FW_LOAD)) ok = false;
                        if (++slot == L::SLOTS) { slot = 0; phase ^= 1u; }
                    }
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);
                }
            } else if (warp == L::W_MMA || warp == L::W_MMA + TILES - 1) {
                if (elect_one() && nmax > 0) {
                    const int w = (int)warp - L::W_MMA, nw = n[w], kw = keys[w];
                    bool ok = mbar_wait(q_full, 0, abort_flag, p.err, ERR_FW_MMA);
                    const uint32_t q_s = smem_u32(sq) + w * L::TILE, ring_s = smem_u32(ring);
                    const uint32_t s_t = tmem + L::S_COL + 128u * w, p_t = tmem + L::P_COL + 128u * w,
                                   o_t = tmem + L::O_COL + (uint32_t)(DP * w);
                    // ring position of K_j and V_j
                    auto k_at = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
                    auto v_at = [&](int j) { return j == nmax - 1 ? 2 * nmax - 1 : 2 * j + 2; };
                    auto wait_full = [&](int at) {
                        return mbar_wait(&full[at % L::SLOTS], (uint32_t)(at / L::SLOTS) & 1u, abort_flag, p.err, ERR_FW_MMA);
                    };
                    auto tile_s = [&](int at) { return ring_s + (uint32_t)(at % L::SLOTS) * L::TILE; };
                    auto do_s = [&](int j) {
                        if (!wait_full(k_at(j))) return false;
                        tc_fence_after();
                        mma_abt<DP, AT_ROWS>(s_t, q_s, tile_s(k_at(j)));
                        tc_commit(&s_full[w]);
                        tc_commit(&empty[k_at(j) % L::SLOTS]);
                        return true;
                    };
                    // A V tile may be cleaned from the tile before on: what its slot held then has been waited for.
                    const bool leads = w == (n[0] == nmax ? 0 : TILES - 1);
                    if (leads && edge0 == 0) mbar_arrive(near);
                    if (nw > 0) ok = ok && do_s(0);
                    for (int j = 0; j < nw && ok; ++j) {
                        if (L::P_APART && j + 1 < nw)
                            ok = mbar_wait(&s_read[w], (uint32_t)j & 1u, abort_flag, p.err, ERR_FW_MMA) && do_s(j + 1);
                        ok = ok && wait_full(v_at(j));
                        if (j >= edge0) ok = ok && mbar_wait(&clean[j - edge0], 0, abort_flag, p.err, ERR_FW_MMA);
                        if (leads && j + 1 >= edge0 && j + 1 < nw) mbar_arrive(near);
                        // a last tile of 64 keys at most leaves its upper half out
                        const int halves = kw - j * AT_ROWS > 64 ? 2 : 1;
                        for (int h = 0; h < halves && ok; ++h) {
                            if (!(ok = mbar_wait(&p_ready[2 * w + h], (uint32_t)j & 1u, abort_flag, p.err, ERR_FW_MMA))) break;
                            tc_fence_after();
                            mma_tb_half<DP>(o_t, p_t + L::P_HALF * h, tile_s(v_at(j)), h, j > 0 || h > 0);
                        }
                        if (!ok) break;
                        tc_commit(&pv_done[w]);
                        tc_commit(&empty[v_at(j) % L::SLOTS]);
                        if (j + 1 == nw) tc_commit(&o_full[w]);
                        // S takes P's place: products run in order, so P V has read it
                        if (!L::P_APART && j + 1 < nw) ok = do_s(j + 1);
                    }
                    // a tile that is done still passes the other one's K and V on, once they have arrived
                    for (int at = nw == 0 ? 0 : 2 * nw - 1; at < 2 * nmax && ok; ++at) {
                        if (nw > 0 && nw < nmax && at == 2 * nw) continue;      // V of its last tile
                        if (nw > 0 && nw == nmax) break;
                        ok = wait_full(at);
                        if (ok) mbar_arrive(&empty[at % L::SLOTS]);
                    }
                    if (!ok || *abort_flag) spin_ns_at_most(2000000ull);    // products in flight end
                }
            } else if (warp >= L::W_CLEAN && warp <= L::W_TMEM) {
                // P is 0 for keys that a row does not see, but 0 times V need not be: rows behind the sequence's keys
                // become zero, as do infinities and NaN of keys that some row does not see (add_nonfinite gives them
                // back to the rows that do).  Done here while the tile's softmax runs.
                const int lane = (int)threadIdx.x - 32 * L::W_CLEAN;
                bool ok = true;
                for (int j = edge0; j < nmax && ok; ++j) {
                    const int at = j == nmax - 1 ? 2 * nmax - 1 : 2 * j + 2, key0 = j * AT_ROWS;
                    ok = mbar_wait(near, (uint32_t)(j - edge0) & 1u, abort_flag, p.err, ERR_FW_CLEAN) &&
                         mbar_wait(&full[at % L::SLOTS], (uint32_t)(at / L::SLOTS) & 1u, abort_flag, p.err, ERR_FW_CLEAN);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t v_s = smem_u32(ring + (at % L::SLOTS) * L::TILE);
                    if (lk - key0 < AT_ROWS) zero_rows<DP>(v_s, lk - key0, AT_ROWS, lane, 32 * L::CLEANERS);
                    if (clean_rows<DP>(v_s, max(0, row0 + shift + 1 - key0), AT_ROWS, min(AT_ROWS, lk - key0), lane, 32 * L::CLEANERS)) *poisoned = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) mbar_arrive(&clean[j - edge0]);
                }
            }
        } else {
            regs_more<L::REGS_SOFTMAX>();
            const int w = (int)(warp >> 2), t = (int)(threadIdx.x & 127u);
            const uint32_t lane_base = (warp & 3u) * 32u << 16;
            const int row = row0 + w * AT_ROWS + t;                 // in the sequence
            const uint32_t s_t = tmem + lane_base + L::S_COL + 128u * w, p_t = tmem + lane_base + L::P_COL + 128u * w,
                           o_t = tmem + lane_base + L::O_COL + (uint32_t)(DP * w);
            const float c = p.scale * AT_LOG2E;
            const int see = row + shift;                            // last key that this row sees
            const int all_see = row0 + w * AT_ROWS + shift + 1;     // keys that all rows see
            float m = -INFINITY, top = -INFINITY;                   // scaled by; true maximum
            float l = 0.f;
            bool ok = true;
            const int nw = n[w];
            auto wait = [&](uint64_t* bar, int use) {
                ok = ok && mbar_wait(bar, (uint32_t)use & 1u, abort_flag, p.err, ERR_FW_SOFTMAX);
                ok = __all_sync(0xffffffffu, ok);
            };
            // The tiles' exponentials take turns (barriers 1 and 2): left alone, both would form them at
            // the same time and then wait for their products at the same time.
            if (TILES == 2 && w == 1 && nmin > 0) named_arrive(1, 256);
            // A warp whose wait gave up goes on without waiting: the others meet it in the barriers.
            for (int j = 0; j < nw; ++j) {
                wait(&s_full[w], j);
                tc_fence_after();
                const int key0 = j * AT_ROWS;
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(s_t + 32u * i, s[i]);
                tmem_ld_wait();
                if (L::P_APART) {
                    tc_fence_before();
                    mbar_arrive(&s_read[w]);
                }
                if (key0 + AT_ROWS > all_see) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (key0 + i > see) s[i / 32][i % 32] = 0xFF800000u;
                }
                float x8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x8[e] = fmaxf(__uint_as_float(s[0][2 * e]), __uint_as_float(s[0][2 * e + 1]));
#pragma unroll
                for (int i = 16; i < 128; i += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x8[e] = max3(x8[e], __uint_as_float(s[i / 32][i % 32 + 2 * e]),
                                     __uint_as_float(s[i / 32][i % 32 + 2 * e + 1]));
                // (a NaN among the logits is passed over here, and makes the sum NaN, as +inf does)
                top = max3(max3(top, x8[0], x8[1]), max3(x8[2], x8[3], x8[4]), max3(x8[5], x8[6], x8[7]));
                const bool grow = m == -INFINITY ? top > -INFINITY : (top - m) * c > 8.f;
                if (L::P_APART && j > 0) {                          // the P before has been read
                    wait(&pv_done[w], j - 1);
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? (m == -INFINITY ? 0.f : ex2((m - top) * c)) : 1.f;
                    if (grow) m = top;
                    l *= f;
                    if (j > 0) {                                    // (S of this tile came after P V of the last one)
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
                if (TILES == 2 && j < nmin) named_sync(1 + w, 256);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pr[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x2 = fma2(pack2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, b2);
                        float x, y;
                        if (i % 8 < L::ON_FMA) {
                            exp2_pair(x2, x, y);
                        } else {
                            unpack2(x2, x, y);
                            x = ex2(x);
                            y = ex2(y);
                        }
                        sum2[i & 1] = add2(sum2[i & 1], pack2(x, y));
                        pr[i] = bf16x2(x, y);
                    }
                    tmem_st_32x32b_x16(p_t + L::P_HALF * (q / 2) + 16u * (q % 2), pr);
                    if (q == 3 && TILES == 2 && j + w < nmin) named_arrive(2 - w, 256);
                    if (q % 2 == 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&p_ready[2 * w + q / 2]);
                    }
                }
                float a, b;
                unpack2(add2(sum2[0], sum2[1]), a, b);
                l += a + b;
            }
            if (ok && nmax > 0) {
                // q's tile is written over: its products, or without any its load, are done
                ok = mbar_wait(nw > 0 ? &o_full[w] : q_full, 0, abort_flag, p.err, ERR_FW_SOFTMAX);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            if (ok && row0 + w * AT_ROWS < lq) {
                const bool live = row < lq;
                // no key seen, or none with any weight: the sum is 0
                const bool none = m == -INFINITY && l == l;
                if (nw > 0 && __any_sync(0xffffffffu, *poisoned != 0))
                    add_nonfinite<DP / 32>(p.v, p.d, o_t, 0, 1.f, k0 + max(0, row0 + shift + 1), k0 + see, live, kv_head);
                const float inv = none ? 0.f : 1.f / l;
                for (int h = 0; h < 2; ++h)
                    store_rows<DP>(o_t + (uint32_t)(DP / 2 * h), nw > 0, none, inv, smem_u32(sq) + w * L::TILE, h,
                                   (int)(warp & 3u) * 32, lq - row0 - w * AT_ROWS,
                                   p.out.p + (long long)(q0 + row0 + w * AT_ROWS) * p.out.rs + (long long)head * p.out.hs,
                                   p.out.rs, p.d);
                if (live)
                    p.lse[(size_t)head * p.total_q + q0 + row] =
                        none ? -INFINITY : (m == -INFINITY ? 0.f : m * p.scale) + logf(l);
                if (p.max_logits != nullptr) {
                    // a row with a NaN logit is passed over; +inf counts, although its row's sum is NaN, too (inf - inf)
                    float best = live && (l == l || top == INFINITY) ? top : -INFINITY;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
                    if ((t & 31) == 0 && best > -INFINITY) atomic_max_float(p.max_logits + head, best * p.scale);
                }
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

template <int DP>
cudaError_t launch_fwd(const AttnParams& p, const FwMaps& maps, cudaStream_t s) {
    using L = FwLayout<DP>;
    cudaError_t e = cudaFuncSetAttribute(attention_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    // a warpgroup that asks for more registers than the launch left would wait for good
    static const int regs = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, attention_fwd_kernel<DP>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs < L::REGS) return cudaErrorInvalidConfiguration;
    const unsigned tiles = seq_blocks(p.total_q, L::TILES * AT_ROWS, p.n_seqs);
    return launch_pdl(attention_fwd_kernel<DP>, dim3(tiles * (unsigned)p.hq), dim3(L::THREADS), L::SMEM, s, p, maps);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, const HeadMaps& m, cudaStream_t s) {
    if (p.total_q == 0 || p.n_seqs == 0) return cudaSuccess;
    const FwMaps maps{m.q, m.k, m.v};
    return p.d <= 64 ? launch_fwd<64>(p, maps, s) : launch_fwd<128>(p, maps, s);
}

}  // namespace muon
