// attention.cuh -- device code shared by the attention kernels: sequence lookup, tensor
// memory operands and packed arithmetic.
#pragma once

#include "model_ops.cuh"
#include "ptx.cuh"

namespace muon {

constexpr int AT_ROWS = 128;                    // rows of a query or key tile = lanes of tensor memory
constexpr int AT_CHUNK = AT_ROWS * 128;         // bytes of 64 bf16 columns of a tile, one 128-byte swizzle span wide
constexpr float AT_LOG2E = 1.4426950408889634f;

// One tile of a sequence: rows [q0, q0 + lq) of q, [k0, k0 + lk) of k; `block` counts from
// 0 over the sequence's `blocks` blocks of rows.
struct SeqTile {
    int q0, lq, k0, lk, block, blocks;
};

// Bounds of sequence s, all 0 when they are out of range.
__device__ __forceinline__ bool seq_bounds(const AttnParams& p, int s, int& q0, int& q1, int& k0, int& k1) {
    q0 = p.cu_q[s];
    q1 = p.cu_q[s + 1];
    k0 = p.cu_k[s];
    k1 = p.cu_k[s + 1];
    if (q0 >= 0 && q0 <= q1 && q1 <= p.total_q && k0 >= 0 && k0 <= k1 && k1 <= p.total_k) return true;
    q0 = q1 = k0 = k1 = 0;
    return false;
}

// Numbers that find_tile gives blocks are below this.
__host__ __device__ __forceinline__ unsigned seq_blocks(int total, int rows, int n_seqs) { return (unsigned)(total / rows + n_seqs); }

// The block of `rows` query (or key) rows with number `t`; called by a whole warp, false when
// there is none.  Sequences whose bounds are out of range count as empty, and are reported:
// CTA 0 looks at all of up to 64 sequences, else CTA c at those from 32 c on.
//
// Up to 64 sequences: blocks are numbered in order, two looks of the warp at most.  More:
// those of sequence s from cu[s] / rows + s on, which is at or behind the end of the sequence
// before; a search finds them without a sum over all sequences, but CTAs without a block lie
// between the others (and bounds out of order may lead it past good sequences).  Forward pass
// of 12 heads of 64: 64 sequences of 128 tokens 21.4 us in order, 23.8 by the search; 256 of
// 128 109 and 89; 4096 of 16 3950 and 1010.
constexpr int AT_IN_ORDER = 64;

__device__ __forceinline__ bool find_tile(const AttnParams& p, bool by_key, int rows, int t, unsigned cta, SeqTile& r) {
    const int lane = (int)(threadIdx.x & 31u);
    const bool in_order = p.n_seqs <= AT_IN_ORDER;
    int lo = 0, hi = p.n_seqs, before = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    if (!in_order) {
        const long long s = 32ll * cta + lane;
        if (s < p.n_seqs && !seq_bounds(p, (int)s, q0, q1, k0, k1)) atomicCAS(p.err, 0, ERR_SEQLENS);
        const int* cu = by_key ? p.cu_k : p.cu_q;
        while (hi - lo > 32) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const unsigned from = __ballot_sync(0xffffffffu, at < hi && max(cu[min(at, hi - 1)], 0) / rows + at <= t);
            if (from == 0) return false;
            lo += (__popc(from) - 1) * step;
            hi = min(hi, lo + step);
        }
    }
    bool found = false;
    for (; lo < hi && (!found || (in_order && cta == 0)); lo += 32) {
        const int s = lo + lane;
        q0 = q1 = k0 = k1 = 0;
        if (s < hi && !seq_bounds(p, s, q0, q1, k0, k1) && in_order && cta == 0) atomicCAS(p.err, 0, ERR_SEQLENS);
        const int n = ((by_key ? k1 - k0 : q1 - q0) + rows - 1) / rows;
        int first = (by_key ? k0 : q0) / rows + s;
        if (in_order) {
            int end = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += v;
            }
            first = before + end - n;
            before += __shfl_sync(0xffffffffu, end, 31);
        }
        const unsigned in = __ballot_sync(0xffffffffu, t >= first && t - first < n);
        if (!found && in != 0) {
            const int l = __ffs((int)in) - 1;
            r.q0 = __shfl_sync(0xffffffffu, q0, l);
            r.lq = __shfl_sync(0xffffffffu, q1, l) - r.q0;
            r.k0 = __shfl_sync(0xffffffffu, k0, l);
            r.lk = __shfl_sync(0xffffffffu, k1, l) - r.k0;
            r.blocks = __shfl_sync(0xffffffffu, n, l);
            r.block = t - __shfl_sync(0xffffffffu, first, l);
            found = true;
        }
    }
    return found;
}

__device__ __forceinline__ void spin_ns_at_most(uint64_t ns) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < ns) { }
}

// ---------------------------------------------------------------- tensor memory

// D[tmem] (+)= A[tmem] * B[smem desc]: A holds one row per lane, two bf16 per column.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 lanes x 32 columns: thread i writes r[] to lane (base_lane + i), columns [col, col + 32).
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
           "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
           "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Moves registers between the warpgroups of a block: every warp of a warpgroup takes N from
// here on.  The sum over the block stays within what it was launched with.
template <int N>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }

// Barrier `id` of the block for `threads` threads.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
        " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void named_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Loads ROWS rows from `row` on of one head, DP columns, as chunks of 64 columns.
template <int DP, int ROWS, int BOX>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
        for (int r = 0; r < ROWS; r += BOX) tma_load_3d(dst + (c * ROWS + r) * 128, map, bar, 64 * c, head, row + r);
}

// ---------------------------------------------------------------- products of tiles
// Tiles lie in shared memory as 64-column chunks of AT_CHUNK bytes, 128-byte swizzled, one
// 128-byte line per row.

// Shared-memory descriptor of a tile without swizzle (see smem_desc_sw128).
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    return smem_desc_sw128(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61);
}

// D = A * B^T over DP columns: A a tile of 128 rows, B one of N, contraction along the rows.
template <int DP, int N>
__device__ __forceinline__ void mma_abt(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t idesc = idesc_bf16_f32(AT_ROWS, N, 0);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        const uint32_t c = (uint32_t)(kk / 4), off = (uint32_t)(kk % 4) * 32u;
        tc_mma_f16(d_tmem, smem_desc_sw128(a + c * AT_CHUNK + off, 16, 1024),
                   smem_desc_sw128(b + c * (N * 128u) + off, 16, 1024), idesc, kk != 0);
    }
}

// D (+)= A_h * B_h: rows 64 h .. 64 h + 63 of B are the contraction, A_h is 128 x 64 bf16 in
// tensor memory, B a tile of DP columns (128 rows when it has two chunks of columns).
template <int DP>
__device__ __forceinline__ void mma_tb_half(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, int h, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(AT_ROWS, DP, 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        tc_mma_f16_ts(d_tmem, a_tmem + 8u * kk, smem_desc_sw128(b + (uint32_t)(4 * h + kk) * 2048u, AT_CHUNK, 1024), idesc,
                      accumulate || kk != 0);
}

// The same for quarter q, 32 rows of B.
template <int DP>
__device__ __forceinline__ void mma_tb_quarter(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, int q, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(AT_ROWS, DP, 1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
        tc_mma_f16_ts(d_tmem, a_tmem + 8u * kk, smem_desc_sw128(b + (uint32_t)(2 * q + kk) * 2048u, AT_CHUNK, 1024), idesc,
                      accumulate || kk != 0);
}

// 64 fp32 columns of this thread's row.
__device__ __forceinline__ void load64(uint32_t taddr, uint32_t (&v)[2][32]) {
    tmem_ld_32x32b_x32(taddr, v[0]);
    tmem_ld_32x32b_x32(taddr + 32u, v[1]);
    tmem_ld_wait();
}

// Zeroes rows [first, rows) of a tile of DP columns; called by `threads` threads, `t` this one's
// index.  The caller orders the writes before the products that read the tile.
template <int DP>
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int rows, int t, int threads) {
#pragma unroll 1
    for (int i = first * 8 + t; i < rows * 8; i += threads)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
            sts128(tile + (uint32_t)(c * rows) * 128u + (uint32_t)i * 16u, make_uint4(0, 0, 0, 0));
}

__device__ __forceinline__ __nv_bfloat162 bits_bf162(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

__device__ __forceinline__ uint32_t lds32(uint32_t saddr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(saddr));
    return v;
}

__device__ __forceinline__ void sts32(uint32_t saddr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

// Sets infinities and NaN in rows [first, rows) of such a tile (0 <= first; none when rows <=
// first) to zero; true when this thread
// met one.  It looks for one first: a sum of the values times zero is NaN then (four products
// for eight values, and loads that wait for no store).
template <int DP>
__device__ __forceinline__ bool clean_rows(uint32_t tile, int first, int rows_in_tile, int rows, int t, int threads) {
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
    __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
    const uint32_t end = (uint32_t)max(0, rows) * 128u;
#pragma unroll 1
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll 2
        for (uint32_t at = (uint32_t)(first * 8 + t) * 16u; at < end; at += (uint32_t)threads * 16u) {
            const uint4 v = lds128(tile + (uint32_t)(c * rows_in_tile) * 128u + at);
            sum[0] = __hfma2(bits_bf162(v.x), zero, sum[0]);
            sum[1] = __hfma2(bits_bf162(v.y), zero, sum[1]);
            sum[2] = __hfma2(bits_bf162(v.z), zero, sum[2]);
            sum[3] = __hfma2(bits_bf162(v.w), zero, sum[3]);
        }
    const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
    const bool met = !(__low2float(all) == 0.f && __high2float(all) == 0.f);
    if (met) {
#pragma unroll 1
        for (int i = 0; i < DP / 64; ++i)
#pragma unroll 1
            for (uint32_t at = (uint32_t)(first * 8 + t) * 16u; at < end; at += (uint32_t)threads * 16u)
#pragma unroll 1
                for (uint32_t e = 0; e < 16; e += 4) {
                    const uint32_t word = tile + (uint32_t)(i * rows_in_tile) * 128u + at + e;
                    uint32_t v = lds32(word);
                    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
                    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
                    sts32(word, v);
                }
    }
    return met;
}

// Gives a row's accumulator the infinities and NaN, times f, that the products did without:
// those of the key rows of x from `first`, the first that a row of the CTA does not see, up to
// the last one that this row sees.  A key whose values the products had as well gives the same
// again.  Columns col .. col + 32 N - 1, at o_t in tensor memory; d: the head's width.
template <int N>
__device__ __noinline__ void add_nonfinite(const HeadView& x, int d, uint32_t o_t, int col, float f, int first, int last,
                                           bool live, int kv_head) {
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_t + 32u * i, o);
        tmem_ld_wait();
#pragma unroll 1
        for (int j = first; live && j <= last; ++j) {
            const __nv_bfloat16* v = x.p + (long long)j * x.rs + (long long)kv_head * x.hs + col + 32 * i;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (col + 32 * i + e < d) {
                    const float y = __bfloat162float(v[e]);
                    if (!isfinite(y)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y * f);
                }
        }
        __syncwarp();
        tmem_st_32x32b_x32(o_t + 32u * i, o);
    }
    tmem_st_wait();
}

// ---------------------------------------------------------------- arithmetic

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// NaN when one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// 2^x of two values on the FMA pipe, which has time to spare beside the special function unit:
// x = n + f with n the nearest integer (Cody-Waite), 2^f by its minimax polynomial of degree 4
// on [-1/2, 1/2] (Remez exchange; relative error 2.6e-6), times 2^n.  Below -126.5, -inf
// included, n is -127 and its factor's bit pattern that of 0, so that a masked logit has
// weight 0 exactly, as from ex2; NaN stays NaN, +inf gives NaN.
__device__ __forceinline__ void exp2_pair(uint64_t x2, float& a, float& b) {
    float x, y;
    unpack2(x2, x, y);
    x2 = pack2(max_nan(x, -127.f), max_nan(y, -127.f));
    constexpr float MAGIC = 12582912.f;         // 1.5 * 2^23: the sum's low bits are the nearest integer
    const uint64_t t2 = add2(x2, pack2(MAGIC, MAGIC));
    const uint64_t f2 = fma2(add2(t2, pack2(-MAGIC, -MAGIC)), pack2(-1.f, -1.f), x2);
    uint64_t p2 = fma2(f2, pack2(0x1.3997d6p-7f, 0x1.3997d6p-7f), pack2(0x1.ca1440p-5f, 0x1.ca1440p-5f));
    p2 = fma2(p2, f2, pack2(0x1.ec06dap-3f, 0x1.ec06dap-3f));
    p2 = fma2(p2, f2, pack2(0x1.62e0dcp-1f, 0x1.62e0dcp-1f));
    p2 = fma2(p2, f2, pack2(0x1.ffffe8p-1f, 0x1.ffffe8p-1f));
    float tx, ty;
    unpack2(t2, tx, ty);
    unpack2(mul2(p2, pack2(__uint_as_float((__float_as_uint(tx) << 23) + 0x3F800000u),
                           __uint_as_float((__float_as_uint(ty) << 23) + 0x3F800000u))), a, b);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Writes 32 rows of one half (DP / 2 columns) of an fp32 accumulator as bf16: the warp's
// lanes hold a row each, `taddr` the half's first column in tensor memory, f the row's factor
// (`zero`: the row is 0 whatever the accumulator holds).  Rows first .. first + 31 of the tile
// go through its 128-byte lines at `stage` (a q, k or v tile that no product reads any more;
// 16-byte unit u of row r at u ^ (r & 7)), so that each store of the warp covers whole rows:
// storing from a row per lane takes 32 lines a store (for a tile of two 128-wide query tiles,
// 4500 cycles against 700).  Rows from `live` on and columns from d on are not written.
template <int DP>
__device__ __forceinline__ void store_rows(uint32_t taddr, bool any, bool zero, float f, uint32_t stage, int half, int first,
                                           int live, __nv_bfloat16* g, long long rs, int d) {
    constexpr int UNITS = DP / 16;                              // 16-byte units of a row's half
    const int lane = (int)(threadIdx.x & 31u);
    const uint32_t line = stage + (DP == 128 ? (uint32_t)half * AT_CHUNK : 0u);
    const int unit0 = DP == 128 ? 0 : 4 * half;
#pragma unroll
    for (int i = 0; i < DP / 64; ++i) {
        uint32_t o[32];
        if (any) {
            tmem_ld_32x32b_x32(taddr + 32u * i, o);
            tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = zero ? 0u : bf16x2(__uint_as_float(o[8 * e + 2 * u]) * f, __uint_as_float(o[8 * e + 2 * u + 1]) * f);
            sts128(line + (uint32_t)((first + lane) * 128 + ((unit0 + 4 * i + e) ^ (lane & 7)) * 16),
                   make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int r = (32 * k + lane) / UNITS, u = (32 * k + lane) % UNITS, col = half * (DP / 2) + 8 * u;
        if (first + r < live && col < d)
            *reinterpret_cast<uint4*>(g + (first + r) * rs + col) =
                lds128(line + (uint32_t)((first + r) * 128 + ((unit0 + u) ^ (r & 7)) * 16));
    }
    __syncwarp();
}

}  // namespace muon
