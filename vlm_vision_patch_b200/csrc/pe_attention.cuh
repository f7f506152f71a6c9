// Attention over packed sequences, forward and backward (include/pe.h has the
// formulas).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "../../include/pe.h"
#include "pe_device.cuh"
#include "pe_packed.cuh"

namespace pe {

// ------------------------------------------------------------- one-CTA tcgen05

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Clock ticks after which a wait gives up: 2 s at the highest clock.
constexpr long long kWaitClocks = 4000000000ll;

__device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// What the roles of a block share about waiting.
struct Waits {
    int abort;                    // a wait has given up
#ifdef PE_DEBUG_BOUNDS
    long long limit;              // clock ticks after which one does
#endif
};

// A converged warp waits for a phase of a barrier that only this block arrives on;
// bounded like mbar_wait.  Every branch is the whole warp's, so a wait that is
// already over costs one look and one vote (a loop that lanes could leave one by
// one cost the issuing warps about 200 clocks per wait more).
#ifndef PE_DEBUG_BOUNDS
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile Waits *waits) {
    if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, try_wait(bar, parity))) {
        if (__any_sync(0xffffffffu, waits->abort != 0 || clock64() - t0 > kWaitClocks)) {
            waits->abort = 1;
            return false;
        }
    }
    return true;
}
#else
// The bounds-checking build lets tests set the limit, and looks at it before the
// hardware's own wait, which outlasts any load (in the product library this order took
// the kernels up to 6% longer).
__device__ __forceinline__ bool phase_over(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile Waits *waits) {
    if (__all_sync(0xffffffffu, phase_over(bar, parity))) return true;
    const long long t0 = clock64();
    do {
        if (__any_sync(0xffffffffu, waits->abort != 0 || clock64() - t0 > waits->limit)) {
            waits->abort = 1;
            return false;
        }
    } while (!__all_sync(0xffffffffu, try_wait(bar, parity)));
    return true;
}
#endif
// A role that has begun loads or products waits for them before it ends, by the clock
// alone and whether a wait of its own has given up or not: another role's may do so
// later, and the block then ends without a look at what is in flight.
__device__ __forceinline__ void warp_drain(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, try_wait(bar, parity)))
        if (__any_sync(0xffffffffu, clock64() - t0 > kWaitClocks)) return;
}
// The loads outside the ring, and the last of those begun in it.
__device__ __forceinline__ void drain_loads(uint64_t *first, uint64_t *full, int stages, int begun) {
    warp_drain(first, 0);
    for (int s = max(begun - stages, 0); s < begun; ++s) warp_drain(&full[s % stages], (s / stages) & 1);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Registers per thread from here on, for the four warps of a warpgroup.
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}

// Descriptors are passed as (low word, high word): a tile's k-step only changes the
// low word, and the issuing thread has little time per MMA.
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi_a, uint32_t hi_b, uint32_t idesc,
                                       bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %3};\n\t"
        "mov.b64 y, {%2, %4};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi_a), "r"(hi_b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A holds two bf16 per 32-bit column, K along the columns
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi_b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi_b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// Arrive on `bar` once every MMA issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Waits for this thread's tensor-memory loads; `v` are their results, which nothing
// may use (or copy) before.
template <int C>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[C][16]) {
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(v[c][e]));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Three-way maximum that keeps a NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x of two values on the FMA pipes, for x <= 2^7: x = n + f with n the nearest
// integer, 2^f by the polynomial of degree 4 with the least relative error on
// [-1/2, 1/2] (2.6e-6, found by exchange; probabilities keep 8 bits), and n added
// to the exponent.  x is held at -126, whose power no sum in fp32 notices.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
    const float kRound = 12582912.0f;                   // 1.5 * 2^23: the sum's last bits are n
    x = make_float2(fmaxf(x.x, -126.0f), fmaxf(x.y, -126.0f));
    const float2 t = add2(x, both(kRound));
    const float2 f = fma2(add2(t, both(-kRound)), both(-1.0f), x);
    float2 p = fma2(both(0.009570102207362652f), f, both(0.05591785907745361f));
    p = fma2(p, f, both(0.240247443318367f));
    p = fma2(p, f, both(0.6931217908859253f));
    p = fma2(p, f, both(0.9999992847442627f));
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// ------------------------------------------------------------- arguments

struct HeadsPtr {
    __nv_bfloat16 *p;
    int64_t row, head;            // strides in elements
    __device__ __forceinline__ __nv_bfloat16 *at(int64_t r, int h) const { return p + r * row + h * head; }
};

struct AttnParams {
    const int32_t *cu_q, *cu_k;
    int n_seq, Nq, Nk, Hq, Hkv, D, causal;
    float scale;
    HeadsPtr q, k, v, out, dout, dq, dk, dv;
    float *lse;                   // [Hq, Nq]
    unsigned n_tiles;             // tiles of the grid
    int tiles;                    // query tiles of a block, 1 or 2 (forward)
    int pack;                     // query heads of a key head side by side in a tile's rows (forward; 1: none)
    int splits;                   // parts, a block each: of the key axis (forward), of the heads that share a key head (keys)
    float *part_out, *part_lse2;  // when splits > 1: forward [splits, Hq, Nq, D] and [splits, Hq, Nq] (base 2);
                                  // keys [splits, 2, Nk, Hkv, D], dv then dk
    uint4 *stat;                  // [Hq, Nq]: -lse / scale and -dout . out, three bf16 and a 0 each (backward)
    int *err;
#ifdef PE_DEBUG_BOUNDS
    long long wait_clocks;        // after which a wait gives up
#endif
};

// Boundary s of a cumulative-length array, held inside [0, n] whatever it says.
__device__ __forceinline__ int boundary(const int32_t *cu, int s, int n) {
    const int v = cu[s];
    return v < 0 ? 0 : (v > n ? n : v);
}

// ------------------------------------------------------------- tiles and work

constexpr int kTile = 128;                  // rows of a tile: queries or keys
constexpr int kChunkBytes = kTile * 128;    // 128 rows of 64 bf16, 128-byte swizzle
constexpr float kLog2e = 1.4426950408889634f;

// The tile of sequence rows that a block works on.
struct Work {
    int q0, lq, k0, lk;    // the sequence's rows; lq, lk >= 0
    int row;               // first row of the tile within the sequence, or -1: nothing to do
    int h, z;              // head, and part (see AttnParams::splits)
};

// Tile, head and part of this block.  Blocks of one head follow one another, so that
// its keys and values are in L2 for all of them; under a causal mask the blocks with
// the most to do come first instead, over all heads and parts: the last query rows
// (REVERSE), the first key rows.
struct Place {
    int tile, h, z;
};
template <bool REVERSE>
__device__ __forceinline__ Place place_of(const AttnParams &P, int heads) {
    const unsigned b = blockIdx.x, tiles = P.n_tiles;
    Place p;
    if (P.causal) {
        const unsigned of_tile = heads * P.splits, t = b / of_tile, r = b - t * of_tile;
        p.tile = REVERSE ? tiles - 1 - t : t;
        p.z = r / heads;
        p.h = r - p.z * heads;
    } else {
        const unsigned r = b / tiles;
        p.tile = b - r * tiles;
        p.z = r / heads;
        p.h = r - p.z * heads;
    }
    return p;
}

// Tile `t` of the tiles of `rows` rows that cut the sequences of one side; called by
// one whole warp.  Sequence s has the tiles from F(s) = floor((cu[s] - cu[0]) / rows)
// + s on: enough for its rows (F(s + 1) - F(s) >= ceil(length / rows)), at most one
// too many, n / rows + n_seq in all, and F needs one boundary only, so that a tile
// finds its sequence by search, 32 places at a time, however many there are.
__device__ __forceinline__ Work find_work(const AttnParams &P, bool by_key, int t, int rows) {
    const int lane = threadIdx.x & 31;
    const int32_t *cu = by_key ? P.cu_k : P.cu_q;
    const int n = by_key ? P.Nk : P.Nq;
    int lo = 0, hi = P.n_seq;                              // the sequence is in [lo, hi)
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0, first = 0;
    while (true) {
        const int step = (hi - lo + 31) / 32, s = lo + lane * step;
        const bool there = s < hi;
        const int c0 = boundary(cu, 0, n);
        if (there && step == 1) {                          // the last look: all that the block needs
            q0 = boundary(P.cu_q, s, P.Nq), q1 = boundary(P.cu_q, s + 1, P.Nq);
            k0 = boundary(P.cu_k, s, P.Nk), k1 = boundary(P.cu_k, s + 1, P.Nk);
        }
        const int c = !there ? 0 : (step > 1 ? boundary(cu, s, n) : (by_key ? k0 : q0));
        first = (c - c0) / rows + s;
        const unsigned hit = __ballot_sync(0xffffffffu, there && first <= t);
        const int at = hit ? 31 - __clz(hit) : 0;
        if (step == 1) {
            Work w = {0, 0, 0, 0, -1, 0, 0};
            w.q0 = __shfl_sync(0xffffffffu, q0, at);
            w.lq = __shfl_sync(0xffffffffu, max(q1 - q0, 0), at);
            w.k0 = __shfl_sync(0xffffffffu, k0, at);
            w.lk = __shfl_sync(0xffffffffu, max(k1 - k0, 0), at);
            const int64_t row = (int64_t)(t - __shfl_sync(0xffffffffu, first, at)) * rows;
            if (row >= 0 && row < (by_key ? w.lk : w.lq)) w.row = (int)row;
            return w;
        }
        lo += at * step;
        hi = min(lo + step, hi);
    }
}

// A place in a ring of N stages, and the parity of its barriers' phase there.
template <int N>
struct Slot {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int by = 1) {
        at += by;
        if (at >= N) at -= N, phase ^= 1;
    }
};

// Keys that query row i of a sequence sees.
__device__ __forceinline__ int keys_seen(const AttnParams &P, const Work &w, int i) {
    return P.causal ? min(w.lk, max(0, i + 1 + w.lk - w.lq)) : w.lk;
}

// Rows [valid, end) of a tile in shared memory become zero (one warp): a tile's
// rows behind its sequence's end meet probabilities of 0, but they belong to
// whatever lies there, and 0 * NaN is not 0.  The swizzle permutes 16-byte
// groups within a row, so whole rows need no index arithmetic.
template <int CHUNKS, int CHUNK>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int valid, int end) {
    const int groups = (end - valid) * 8;
    for (int c = 0; c < CHUNKS; ++c)
        for (int i = threadIdx.x & 31; i < groups; i += 32)
            *reinterpret_cast<uint4 *>(tile + c * CHUNK + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// Descriptors of a tile (chunks of 64 columns, CHUNK bytes each): the low word of
// its first k-step, what the k-th step adds to it, and the high word.  K-major,
// steps of 16 columns ...
__device__ __forceinline__ uint32_t desc_k(uint32_t tile) { return (uint32_t)smem_desc(tile, 16, 1024, kLayoutSw128); }
template <int CHUNK>
__host__ __device__ constexpr uint32_t step_k(int k) { return (uint32_t)((k >> 2) * CHUNK + (k & 3) * 32) >> 4; }
// ... or read along its rows (MN-major): steps of 16 rows, N = the columns.
template <int CHUNK>
__device__ __forceinline__ uint32_t desc_mn(uint32_t tile) { return (uint32_t)smem_desc(tile, CHUNK, 1024, kLayoutSw128); }
__host__ __device__ constexpr uint32_t step_mn(int k) { return (uint32_t)(k * 2048) >> 4; }
// An operand of 16 columns without swizzle, 8 columns (16 bytes a row, rows one
// behind the other) at `tile` and 8 at tile + next.
__device__ __forceinline__ uint32_t desc_flat(uint32_t tile, uint32_t next) {
    return (uint32_t)smem_desc(tile, next, 128, kLayoutInterleave);
}
constexpr uint32_t kDescHiFlat = (128u >> 4) | (1u << 14);
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | ((uint32_t)kLayoutSw128 << 29);
__host__ __device__ constexpr uint32_t idesc_b_mn(int M, int N) { return idesc_bf16_f32(M, N) | (1u << 16); }

// ------------------------------------------------------------- hidden rows
//
// Under a causal mask a tile holds rows that some rows of the other side do not see.
// In the products over the tile they meet probabilities of 0, and 0 times a NaN or an
// infinity is not 0.  A result that is not finite is therefore looked at again, a warp
// a row: if a hidden row holds such a value in one of its columns, the column is summed
// anew over the rows seen, in fp32 without the tensor cores.  Only warps with rows that
// the mask cuts look, in kernels of their own: with this code behind it the unmasked
// forward loop took 7% longer (registers).  Summing anew is slow and meant to be rare: a
// NaN in one query's row in the middle of 8192 (12 heads on 2, head size 128) takes the
// backward pass from 0.7 to 86 ms, for the 127 keys of its tile that do not see it.

// Whether an element of this thread's row in N times 16 columns of tensor memory, `step`
// apart, is NaN or infinite; of the last only while `left` goes.
template <int N>
__device__ __forceinline__ bool tmem_odd(uint32_t taddr, int step, int left = 2 * N) {
    float odd = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (2 * c >= left) break;
        uint32_t o[1][16];
        tmem_ld_x16(taddr + c * step, o[0]);
        tmem_ld_wait_for(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) odd = fmaf(__uint_as_float(o[0][e]), 0.f, odd);
    }
    return !(odd == 0.f);
}
// Elements 4 lane .. 4 lane + 3 of a row of D, 0 behind it.
__device__ __forceinline__ float4 quad(const __nv_bfloat16 *row, int D) {
    const int e = 4 * (threadIdx.x & 31);
    if (e >= D) return make_float4(0.f, 0.f, 0.f, 0.f);
    const uint2 u = *reinterpret_cast<const uint2 *>(row + e);
    return make_float4(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x), bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
}
// The product of two rows, the same in every lane.
__device__ __forceinline__ float quad_dot(float4 a, float4 b) {
    float s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ void quad_add(float4 &acc, float f, float4 v) {
    acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
}
// Whether an element is NaN or infinite.
__device__ __forceinline__ bool quad_odd(float4 v) {
    return !(fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, v.w * 0.f))) == 0.f);
}
// Every 64th step: whether all columns to be summed anew are NaN already, as those are
// that belong to rows seen.
__device__ __forceinline__ bool quad_lost(int step, bool hit, float4 acc) {
    if ((step & 63) != 63) return false;
    const bool nan = acc.x != acc.x && acc.y != acc.y && acc.z != acc.z && acc.w != acc.w;
    return __all_sync(0xffffffffu, !hit || nan);
}
// f * acc to this lane's columns of a row, as bf16, or as fp32 in a part.
__device__ __forceinline__ void quad_store(__nv_bfloat16 *row, float *part, float f, float4 v) {
    const int e = 4 * (threadIdx.x & 31);
    if (part) *reinterpret_cast<float4 *>(part + e) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    else *reinterpret_cast<uint2 *>(row + e) = make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}

// ------------------------------------------------------------- forward
//
// A block takes 256 query rows of one sequence and head as two tiles of 128 (one
// tile when there are blocks for half of the SMs at most), and streams the sequence's keys and values past them.  Roles: warps 0-3 and
// 4-7 do the softmax of tile 0 and 1 (one thread per row: row maximum and sum
// need no shuffles), warp 8 loads, warp 9 issues the MMAs.  Scores (fp32) and
// probabilities (bf16) have columns of their own in tensor memory, so the scores
// of tile j + 1 are made while j's exponentials are, and the softmax never waits
// for a product.  The output accumulates in tensor memory too and is rescaled
// only when a row's maximum has grown by more than 2^8, which keeps P in bf16's
// range and is rare.
//
// Where sequences are short a block's start and end (its sequence's search, tensor
// memory, first loads, last stores: about 8 us) cost more than its products: the
// form with one tile (G = 1) is half as large in everything, so that two blocks
// share an SM.  FwdPlan says when.
//
// With few query rows a sequence (a new token each, say) the heads that share a
// key head stand side by side in one tile, so its keys are read once for all of
// them, and several blocks divide the key axis; a second kernel joins their parts.

constexpr int kAttnThreads = 384;
// Registers: 384 threads are launched with 168 each, which the softmax warpgroups
// and the others divide anew (256 * 208 + 128 * 88 = 384 * 168).  With 224 and 56
// the backward kernels' loading and issuing warps spilled (head size 128: 1808 us
// against 1660).  The forward kernels of two tiles spill 8 to 20 bytes a thread even so,
// the backward ones nothing.
constexpr int kLaunchRegs = 168, kRegsUp = 208, kRegsDown = 88;
constexpr int kPolyOf4 = 1;                     // of four pairs of exponentials, how many the FMA pipes take

template <int DP>
constexpr int kChunks = DP > 64 ? 2 : 1;

// Keys per tile: two tiles' scores, probabilities (half as wide) and outputs
// share the 512 columns of tensor memory, 3 KT + 2 DP <= 512.
template <int DP>
constexpr int kKeys = DP <= 64 ? 128 : (DP <= 80 ? 112 : (DP <= 96 ? 96 : 80));

// G query tiles a block.  With one (short sequences, below) two blocks share an SM:
// half of tensor memory and of shared memory, 192 threads (which may have 168
// registers each and take 120), and key tiles of 64.
template <int DP, int G>
struct FwdShape {
    static constexpr int kC = kChunks<DP>, KT = G == 1 ? 64 : kKeys<DP>;
    static constexpr int kThreads = G == 1 ? 192 : kAttnThreads, kWarps = 4 * G;   // softmax warps
    static constexpr uint32_t kCols = 256 * G;
    static constexpr int kChunk = KT * 128;                    // bytes of KT rows of 64 bf16
    static constexpr uint32_t kQ = kC * kChunkBytes, kKv = kC * kChunk;
    static constexpr int kStages = DP <= 64 ? 8 : (G == 1 ? 4 : 5);
    static constexpr size_t kSmem = G * kQ + (size_t)kStages * kKv + 1024;
    static constexpr uint32_t kColS = 0, kColP = G * KT, kColO = G * KT * 3 / 2;
    static_assert(G * (KT * 3 / 2 + DP) <= kCols && kSmem + 1024 <= 232448 * G / 2 && KT % 16 == 0, "on-chip memory");
};

struct FwdBars {
    uint64_t full[8], empty[8], tail, qfull, s_full[2], s_free[2], p_full[2], pv_done[2], drain[2], turn[2][4];
    uint32_t tmem;
    Waits waits;
    Work w;
    volatile int keys[4 * 2][2];                 // per softmax warp: this block's first key and keys behind it, for the end
};

// This warp's MMAs finish before their tensor memory is freed.
__device__ __forceinline__ void drain_mmas(uint32_t one, uint64_t *bar) {
    if (one) mma_commit(bar);
    __syncwarp();
    warp_drain(bar, 0);
}

// p = 2^(s sl2 - base) of one row of 16 C scores, as bf16 pairs; returns the row's
// sum.  Of four pairs POLY go to the FMA pipes: the special-function unit gives
// 16 results a clock and would bound the kernel alone.
template <int POLY, int C>
__device__ __forceinline__ float exp_row(const uint32_t (&s)[C][16], float sl2, float base, uint32_t (&pk)[C][8]) {
    float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = fma2(make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), both(sl2),
                                  both(-base));
            const float2 r = (e & 3) < POLY ? ex2_poly(x) : make_float2(ex2(x.x), ex2(x.y));
            sum[e & 1] = add2(sum[e & 1], r);
            pk[c][e] = pack_bf16x2(r.x, r.y);
        }
    const float2 t = add2(sum[0], sum[1]);
    return t.x + t.y;
}

// In place of the lse of a part whose keys a row sees, all with scores of -inf (a part
// of which it sees no key has -inf itself).
constexpr float kNoFiniteScore = -3.402823466e38f;

// Online softmax of one 128-row tile; all 128 threads of its warps.
template <int DP, int G, bool CAUSAL>
__device__ __forceinline__ void fwd_softmax(const AttnParams &P, FwdBars &B, const Work &w, int tile, int n_kv, int n_other, int kb, int h) {
    using S = FwdShape<DP, G>;
    constexpr int C = S::KT / 16;
    volatile Waits *abort = &B.waits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = B.tmem + ((uint32_t)(warp & 3) << 21);  // 32 lanes a warp, in bits 16..
    const uint32_t ts = lanes + S::kColS + tile * S::KT, tp = lanes + S::kColP + tile * (S::KT / 2);
    const uint32_t to = lanes + S::kColO + tile * DP;
    const int r = (warp & 3) * 32 + lane, rows = kTile / P.pack;   // place in the tile, query rows of a tile
    const int i = w.row + tile * rows + r / P.pack;                // row within the sequence
    const int head = P.pack > 1 ? h * P.pack + r % P.pack : h;
    // Rows of no use (behind the sequence, or of no head) hold what lies there: they
    // take no part in the warp's votes, or a result's last bits would depend on them.
    const bool mine = i < w.lq && r < rows * P.pack;
    const int limit = mine ? keys_seen(P, w, i) - kb : INT32_MAX;  // of this block's keys
    const float sl2 = P.scale * kLog2e;
    if (CAUSAL && lane == 0) B.keys[warp][0] = w.k0 + kb, B.keys[warp][1] = w.lk - kb;   // not in registers meanwhile
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n_kv; ++j) {
        if (!warp_wait(&B.s_full[tile], j & 1, abort)) return;
        tc_fence_after();
        uint32_t s[C][16];
#pragma unroll
        for (int c = 0; c < C; ++c) tmem_ld_x16(ts + 16 * c, s[c]);
        tmem_ld_wait_for(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.s_free[tile]));
        const bool cut = __any_sync(0xffffffffu, (j + 1) * S::KT > limit);
        if (cut) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (j * S::KT + 16 * c + e >= limit) s[c][e] = __float_as_uint(-INFINITY);
        }
        float mx4[4] = {m, m, m, m};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 16; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx4[k] = max3_nan(mx4[k], __uint_as_float(s[c][e + 2 * k]), __uint_as_float(s[c][e + 2 * k + 1]));
        const float mx = max3_nan(max3_nan(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]);
        if (__any_sync(0xffffffffu, mine && (mx - m) * sl2 > 8.0f)) {
            const float f = m == -INFINITY ? 0.f : ex2((m - mx) * sl2);
            l *= f;
            m = mx;
            if (j > 0) {
                if (!warp_wait(&B.pv_done[tile], (j - 1) & 1, abort)) return;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t o[16];
                    tmem_ld_x16(to + 16 * c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st_x16(to + 16 * c, o);
                }
                tmem_st_wait();                                    // (the next wait may give up)
            }
        }
        // a NaN or +inf score makes the row NaN, as the formula does; a row that has seen no key stays at 0
        const float base = mx == -INFINITY ? 0.f : fmaf(m, sl2, mx - mx);
        // the two warps of an SM quarter take turns at the exponentials (tile 0 first):
        // while one fills the special-function unit, the other waits, loads and stores
        const int turn = tile ? j : j - 1;
        if (turn >= 0 && turn < n_other && !warp_wait(&B.turn[tile][warp & 3], turn & 1, abort)) return;
        uint32_t pk[C][8];
        l += cut ? exp_row<0, C>(s, sl2, base, pk) : exp_row<kPolyOf4, C>(s, sl2, base, pk);
        if (lane == 0) mbar_arrive(smem_addr(&B.turn[1 - tile][warp & 3]));
        if (j > 0) {                                               // P V of j - 1 has read its P
            if (!warp_wait(&B.pv_done[tile], (j - 1) & 1, abort)) return;
            tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < C; ++c) tmem_st_x8(tp + 8 * c, pk[c]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.p_full[tile]));
    }
    if (n_kv > 0) {
        if (!warp_wait(&B.pv_done[tile], (n_kv - 1) & 1, abort)) return;
        tc_fence_after();
    }
    // A row that sees keys, all with scores of -inf, is NaN as in the formula (exp(-inf - -inf)); its l is
    // not used, as the polynomial's least power of 2 is not 0.
    const float inv = m == -INFINITY ? NAN : 1.0f / l;
    const int64_t at = (int64_t)head * P.Nq + w.q0 + i, part = (int64_t)w.z * P.Hq * P.Nq + at;
    __nv_bfloat16 *out = P.out.at(w.q0 + i, head);
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) {
        uint32_t o[1][16] = {{0}};
        if (n_kv > 0) {
            tmem_ld_x16(to + 16 * c, o[0]);
            tmem_ld_wait_for(o);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (!mine || 16 * c + 8 * g >= P.D) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = limit > 0 ? __uint_as_float(o[0][8 * g + e]) * inv : 0.f;
            if (P.splits > 1) {
                float4 *dst = reinterpret_cast<float4 *>(P.part_out + part * P.D + 16 * c + 8 * g);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                st_global_v4(out + 16 * c + 8 * g, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
    }
    if constexpr (CAUSAL) {
        // keys of this block's tiles from `limit` on are hidden from the row: fewer for every later one
        __syncwarp();
        const int k0 = B.keys[warp][0], end = min(B.keys[warp][1], n_kv * S::KT);
        const bool some = mine && limit > 0 && limit < end && l < INFINITY && m > -INFINITY;
        uint32_t again = 0;
        if (__any_sync(0xffffffffu, some)) {
            const bool lost = tmem_odd<DP / 16>(to, 16);               // (the whole warp)
            again = __ballot_sync(0xffffffffu, some && lost);
        }
        int looked = end;
        bool hit = false;
        __syncwarp();
        while (again) {
            const int src = 31 - __clz(again), seen = __shfl_sync(0xffffffffu, limit, src);
            again ^= 1u << src;
            const int row = w.q0 + __shfl_sync(0xffffffffu, i, src), a_head = __shfl_sync(0xffffffffu, head, src);
            const int kv = a_head / (P.Hq / P.Hkv);
            const float base = __shfl_sync(0xffffffffu, m * sl2, src), f = __shfl_sync(0xffffffffu, inv, src);
            while (looked > seen) hit |= quad_odd(quad(P.v.at(k0 + --looked, kv), P.D));
            if (!__any_sync(0xffffffffu, hit)) continue;
            const float4 q = quad(P.q.at(row, a_head), P.D);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < seen && !quad_lost(j, hit, acc); ++j)
                quad_add(acc, ex2(fmaf(quad_dot(q, quad(P.k.at(k0 + j, kv), P.D)), sl2, -base)), quad(P.v.at(k0 + j, kv), P.D));
            const int64_t to_part = (((int64_t)w.z * P.Hq + a_head) * P.Nq + row) * P.D;
            if (hit) quad_store(P.out.at(row, a_head), P.splits > 1 ? P.part_out + to_part : nullptr, f, acc);
        }
    }
    if (!mine) return;
    if (P.splits > 1) {
        const float v = m * sl2 + log2f(l);
        P.part_lse2[part] = limit <= 0 ? -INFINITY : (v == -INFINITY ? kNoFiniteScore : v);
    } else if (P.lse) P.lse[at] = limit > 0 ? m * P.scale + logf(l) : -INFINITY;
}

// Whether row r belongs to a sequence of `cu`.
__device__ __forceinline__ bool in_sequence(const int32_t *cu, int n_seq, int n, int r) {
    int lo = -1, hi = n_seq - 1;                          // the last sequence that begins at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (boundary(cu, mid, n) <= r) lo = mid; else hi = mid - 1;
    }
    return lo >= 0 && r < boundary(cu, lo + 1, n);
}

// Joins the parts of a row and head (one warp each): out = sum_z w_z out_z / sum_z
// w_z with w_z = 2^(lse2_z - max).  Parts without a finite score weigh nothing beside
// others; a row of such parts only takes their NaN.
__global__ void __launch_bounds__(256) pe_attn_join_kernel(const __grid_constant__ AttnParams P) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);          // [Hq, Nq]
    if (at >= (int64_t)P.Hq * P.Nq) return;
    const int h = (int)(at / P.Nq), r = (int)(at - (int64_t)h * P.Nq);
    if (!in_sequence(P.cu_q, P.n_seq, P.Nq, r)) return;
    const int64_t step = (int64_t)P.Hq * P.Nq;
    // at most 64 parts: a lane holds two of their statistics
    const float l0 = lane < P.splits ? P.part_lse2[lane * step + at] : -INFINITY;
    const float l1 = lane + 32 < P.splits ? P.part_lse2[(lane + 32) * step + at] : -INFINITY;
    float top = fmaxf(l0, l1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // a part that saw no key weighs nothing, and what its place holds is not read
    const float w0 = l0 == -INFINITY ? 0.f : ex2(l0 - top), w1 = l1 == -INFINITY ? 0.f : ex2(l1 - top);
    float sum = w0 + w1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int z = 0; z < P.splits; ++z) {
        const float w = __shfl_sync(0xffffffffu, z < 32 ? w0 : w1, z & 31);
        if (w != 0.f && 4 * lane < P.D) {
            const float4 v = *reinterpret_cast<const float4 *>(P.part_out + (z * step + at) * P.D + 4 * lane);
            o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    if (4 * lane < P.D)
        *reinterpret_cast<uint2 *>(P.out.at(r, h) + 4 * lane) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    const float lse2 = top + log2f(sum);
    if (lane == 0 && P.lse) P.lse[at] = sum == 0.f || lse2 <= 0.5f * kNoFiniteScore ? -INFINITY : lse2 / kLog2e;
}

// Loads (one warp): Q, then K0 K1 V0 K2 V1 ... (the order of use) through one ring.
template <int DP, int G>
__device__ __forceinline__ void fwd_load(const AttnParams &P, FwdBars &B, const Work &w, const CUtensorMap &mq,
                                         const CUtensorMap &mk, const CUtensorMap &mv, uint8_t *sq, uint8_t *ring, bool two,
                                         int n_max, int kb, int h, int hk) {
    using S = FwdShape<DP, G>;
    constexpr int KT = S::KT;
    volatile Waits *abort = &B.waits;
    const int lane = threadIdx.x & 31;
    if (n_max > 0 && lane == 0) {
        const int rows = kTile / P.pack;                    // the box of mq: rows x pack heads
        mbar_arrive_expect_tx(smem_addr(&B.qfull), (two ? 2 : 1) * S::kC * rows * P.pack * 128);
        for (int t = 0; t < (two ? 2 : 1); ++t)
            for (int c = 0; c < S::kC; ++c)
                tma_load_3d(smem_addr(sq + t * S::kQ + c * kChunkBytes), &mq, smem_addr(&B.qfull), 64 * c, h * P.pack,
                            w.q0 + w.row + t * rows);
    }
    int f = 0;
    bool ok = true;
    Slot<S::kStages> r;
    for (; f < 2 * n_max; ++f, r.next()) {
        const int slot = r.at;
        const bool is_v = f == 2 * n_max - 1 || (f > 0 && !(f & 1));
        const int j = f == 2 * n_max - 1 ? n_max - 1 : (is_v ? (f >> 1) - 1 : (f + 1) >> 1);
        ok = warp_wait(&B.empty[slot], r.phase ^ 1, abort);
        if (!ok) break;
        uint8_t *dst = ring + slot * S::kKv;
        const int valid = min(w.lk - kb - j * KT, KT);
        const bool clean = is_v && valid < KT;          // the last tile of V: zeros behind the sequence
        uint64_t *bar = clean ? &B.tail : &B.full[slot];
        if (lane == 0) {
            mbar_arrive_expect_tx(smem_addr(bar), S::kKv);
            for (int c = 0; c < S::kC; ++c)
                tma_load_3d(smem_addr(dst + c * S::kChunk), is_v ? &mv : &mk, smem_addr(bar), 64 * c, hk,
                            w.k0 + kb + j * KT);
        }
        __syncwarp();
        if (clean) {
            ok = warp_wait(&B.tail, 0, abort);
            if (!ok) {
                warp_drain(&B.tail, 0);
                break;
            }
            zero_rows<S::kC, S::kChunk>(dst, valid, (valid + 15) & ~15);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.full[slot]));
        }
    }
    if (n_max > 0) drain_loads(&B.qfull, B.full, S::kStages, f);
}

// MMAs of one query tile (one warp): S of the next keys as soon as the softmax has
// read the last, P V when P is there.  Each tile has a warp of its own: the issuing
// warp shares its instruction queue with the exponentials, and one warp for both
// tiles spent longer queueing than the tensor cores working.
template <int DP, int G>
__device__ __forceinline__ void fwd_mma(FwdBars &B, const Work &w, uint8_t *sq, uint8_t *ring, int t, int n, int n_max,
                                        int kb) {
    using S = FwdShape<DP, G>;
    constexpr int KT = S::KT;
    constexpr uint32_t kIdS = idesc_bf16_f32(kTile, KT), kIdO = idesc_b_mn(kTile, DP);
    volatile Waits *abort = &B.waits;
    const uint32_t one = elect_one(), tm = B.tmem;
    const uint32_t d_q = desc_k(smem_addr(sq)) + t * (S::kQ >> 4), d_k = desc_k(smem_addr(ring));
    const uint32_t d_v = desc_mn<S::kChunk>(smem_addr(ring));
    const uint32_t ts = tm + S::kColS + t * KT, tp = tm + S::kColP + t * (KT / 2), to = tm + S::kColO + t * DP;
    Slot<S::kStages> r;                                     // K0 K1 V0 K2 V1 ... in the order of the loads
    auto wait_full = [&] { return warp_wait(&B.full[r.at], r.phase, abort); };
    auto issue_s = [&] {
        const uint32_t b = d_k + r.at * (S::kKv >> 4);
        if (one) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                mma_ss(ts, d_q + step_k<kChunkBytes>(k), b + step_k<S::kChunk>(k), kDescHi, kDescHi, kIdS, k > 0);
            mma_commit(&B.s_full[t]);
            mma_commit(&B.empty[r.at]);
        }
        __syncwarp();
    };
    // a tile that needs none of these keys gives the slot back at once
    auto skip = [&] {
        if (one) mbar_arrive(smem_addr(&B.empty[r.at]));
        __syncwarp();
    };
    const int left = w.lk - kb;
    bool ok = n_max == 0 || (warp_wait(&B.qfull, 0, abort) && wait_full());
    if (ok && n_max > 0) {
        tc_fence_after();
        if (n > 0) issue_s();
        else skip();
        r.next();
    }
    for (int j = 0; j < n_max && ok; ++j) {
        if (j + 1 < n_max) {                                // the next scores, once the last have been read
            ok = wait_full() && (j + 1 >= n || warp_wait(&B.s_free[t], j & 1, abort));
            if (!ok) break;
            tc_fence_after();
            if (j + 1 < n) issue_s();
            else skip();
            r.next();
        }
        ok = wait_full() && (j >= n || warp_wait(&B.p_full[t], j & 1, abort));
        if (!ok) break;
        tc_fence_after();
        if (j < n) {
            const int steps = (min(left - j * KT, KT) + 15) / 16;
            const uint32_t b = d_v + r.at * (S::kKv >> 4);
            if (one) {
                mma_ts(to, tp, b, kDescHi, kIdO, j > 0);
                if (steps == KT / 16) {
#pragma unroll
                    for (int k = 1; k < KT / 16; ++k) mma_ts(to, tp + 8 * k, b + step_mn(k), kDescHi, kIdO, true);
                } else {
                    for (int k = 1; k < steps; ++k) mma_ts(to, tp + 8 * k, b + step_mn(k), kDescHi, kIdO, true);
                }
                mma_commit(&B.pv_done[t]);
                mma_commit(&B.empty[r.at]);
            }
            __syncwarp();
        } else {
            skip();
        }
        r.next();
    }
    drain_mmas(one, &B.drain[t]);
}

// mk, mv: boxes of FwdShape::KT rows; mq: of 128 / pack rows and pack heads.
template <int DP, int G, bool CAUSAL>
__global__ void __launch_bounds__(G == 1 ? 192 : kAttnThreads, G == 1 ? 2 : 1)
pe_attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnParams P) {
    using S = FwdShape<DP, G>;
    constexpr int KT = S::KT;
    extern __shared__ uint8_t raw[];
    __shared__ FwdBars B;
    uint8_t *sq = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023), *ring = sq + G * S::kQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = kTile / P.pack;
    constexpr int kLoad = S::kWarps, kMma = kLoad + 1;      // the warps that load and (from kMma on) issue MMAs
    if (warp == kMma) {
        const Place at = place_of<true>(P, P.pack > 1 ? P.Hkv : P.Hq);
        Work w = find_work(P, false, at.tile, P.tiles * rows);
        w.h = at.h;
        w.z = at.z;
        if (lane == 0) {
            B.w = w;
            B.waits.abort = 0;
#ifdef PE_DEBUG_BOUNDS
            B.waits.limit = P.wait_clocks;
#endif
            const int tiles = G > 1 && P.tiles > 1 && w.lq - w.row > rows ? 2 : 1;  // each gives a slot back
            for (int i = 0; i < S::kStages; ++i) mbar_init(smem_addr(&B.full[i]), 1), mbar_init(smem_addr(&B.empty[i]), tiles);
            mbar_init(smem_addr(&B.tail), 1);
            mbar_init(smem_addr(&B.qfull), 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(smem_addr(&B.drain[t]), 1);
                for (int u = 0; u < 4; ++u) mbar_init(smem_addr(&B.turn[t][u]), 1);
                mbar_init(smem_addr(&B.s_full[t]), 1);
                mbar_init(smem_addr(&B.s_free[t]), 4);
                mbar_init(smem_addr(&B.p_full[t]), 4);
                mbar_init(smem_addr(&B.pv_done[t]), 1);
            }
            fence_mbar_init();
            prefetch_tmap(&mq);
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
        }
    }
    if (warp == kLoad) {
        tmem_alloc(smem_addr(&B.tmem), S::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Work w = B.w;
    const int h = w.h, hk = P.pack > 1 ? h : h / (P.Hq / P.Hkv);
    if (P.splits > 1) griddep_launch_dependents();          // the joining kernel
    if (w.row < 0) {                                        // more blocks than tiles
        if (warp == kLoad) tmem_dealloc(B.tmem, S::kCols);
        return;
    }
    // key tiles that each query tile meets (the second tile may be missing) ...
    auto tiles_of = [&](int t) {
        const int last = min(w.row + (t + 1) * rows, w.lq) - 1;
        return t < P.tiles && w.lq - w.row > t * rows ? (keys_seen(P, w, last) + KT - 1) / KT : 0;
    };
    const bool two = G > 1 && P.tiles > 1 && w.lq - w.row > rows;
    const int all0 = tiles_of(0), all1 = tiles_of(1), all = max(all0, all1);
    // ... and this block's part of them, from key kb on
    const int from = (int)((int64_t)all * w.z / P.splits), to = (int)((int64_t)all * (w.z + 1) / P.splits);
    const int kb = from * KT, n_max = to - from;
    const int n0 = min(max(all0 - from, 0), n_max), n1 = min(max(all1 - from, 0), n_max);
    if (warp < S::kWarps) {
        if constexpr (G > 1) regs_up<kRegsUp>();
        if (warp < 4 || two) fwd_softmax<DP, G, CAUSAL>(P, B, w, warp >> 2, warp < 4 ? n0 : n1, warp < 4 ? n1 : n0, kb, h);
    } else {
        if constexpr (G > 1) regs_down<kRegsDown>();
        if (warp == kLoad) fwd_load<DP, G>(P, B, w, mq, mk, mv, sq, ring, two, n_max, kb, h, hk);
        else if (warp < kMma + (two ? 2 : 1)) fwd_mma<DP, G>(B, w, sq, ring, warp - kMma, warp == kMma ? n0 : n1, n_max, kb);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && B.waits.abort) atomicExch(P.err, (int)PE_ERR_DEVICE_TIMEOUT);
    if (warp == kLoad) {
        tc_fence_after();
        tmem_dealloc(B.tmem, S::kCols);
    }
}

// ------------------------------------------------------------- backward
//
// Two kernels of one shape, so that no sum needs atomics and two runs give the
// same bits: one block keeps 128 query rows and streams the keys past them (dq),
// then one block keeps 128 key rows and streams the queries past them (dk, dv).
// Both recompute the scores; that is 7 products of a tile pair instead of 5, and
// in exchange dq is summed in tensor memory rather than in fp32 in HBM.
//
// With x0, x1 the kept rows and y0, y1 the streamed ones (q, dout and k, v, or
// k, v and q, dout):   s = x0 y0^T,  dp = x1 y1^T,  p = exp(s - lse),
// ds = p (dp - delta);  kept rows += ds y0, and for keys also p y1.
// The streamed tiles hold 64 rows, so that two pairs (s, dp) fit in tensor
// memory beside the sums: warps 0-3 work on one while the tensor cores fill the
// other for warps 4-7.  p and ds go back to tensor memory as bf16 and are the A
// operands of the sums.
//
// For keys, lse and delta belong to columns: each thread would need all 64 pairs
// of every tile from shared memory (that took as long as the products).  Instead
// each goes into the product itself, as one more k-step: every kept row times
// (1, 1, 1, 0 ...), every query times its statistic as a sum of three bf16, which
// is 24 bits.  So s arrives as s - lse / scale and dp as dp - delta.

constexpr int kStream = 64;                       // streamed rows per tile
constexpr int kStreamChunk = kStream * 128;       // bytes of 64 rows of 64 bf16
constexpr uint32_t kSelect = kTile * 32, kStats = kStream * 16;

// Shared memory: the kept tiles, the ring, and for keys the two selectors of the
// statistics (128 rows of 16 bf16), the statistics of each stage's 64 queries
// (8 bf16) and 64 rows of zeros.  A stage lives from its load until the sums have
// read it, some three tiles' time, so the ring is as deep as fits in 212 KB (head
// size 64: 8 stages, 1186 us for 4 x 4096 rows against 1271 with 4).  The rest is
// left to L1: a fifth stage at head size 80 took the dq kernel from 669 to 743 us.
template <int DP, bool KEYS>
struct BwdShape {
    static constexpr uint32_t kKept = kChunks<DP> * kChunkBytes, kOne = kChunks<DP> * kStreamChunk;
    static constexpr uint32_t kFixed = 1024 + 2 * kKept + (KEYS ? 2 * kSelect + kStats : 0);
    static constexpr uint32_t kStage = 2 * kOne + (KEYS ? kStats : 0);
    static constexpr int kFit = (212 * 1024 - kFixed) / kStage, kStages = kFit < 8 ? kFit : 8;
    static constexpr uint32_t kTiles = 2 * kKept + kStages * 2 * kOne;
    // a warp that issues every second tile's scores meets every phase of its slots only then
    static_assert(kStages >= 2 && kStages % 2 == 0, "ring depth");
    static constexpr size_t kSmem = kFixed + (size_t)kStages * kStage;
};
constexpr int kBwdMaxStages = 8;


// `bytes` contiguous bytes to shared memory (both 16-byte aligned, a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// v as a sum of three bf16 (24 bits), the second word's high half 0.
__device__ __forceinline__ uint2 split3(float v) {
    const float h = __bfloat162float(__float2bfloat16_rn(v)), m = __bfloat162float(__float2bfloat16_rn(v - h));
    return make_uint2(pack_bf16x2(h, m), pack_bf16x2(v - h - m, 0.f));
}

// The streamed tiles of one block: for keys, the query tiles of every head that
// shares the key head, from the first that sees the tile's first key.
struct Stream {
    int first, per_head, n;                       // first tile, tiles per head, tiles in all
    int head;                                     // first query head (keys)
    int total;                                    // tiles streamed: n, or twice that (short query rows)
};

// delta comes from the stored output, whose rounding is as large as ds itself where
// a row sees few keys.  Rows of at most this many key tiles are swept twice: the
// first time only sums ds, which is what delta is off by.  (Beyond 256 keys it
// moves dq's error by 1 part in 100 and would cost a third of the kernel.  On 925 x 64
// rows, 16 heads of 80, it costs 3% of a training step: 2034 us against 1976; on 4 x 196
// 42.9 against 42.5.)
constexpr int kSweepTwice = 4;

struct BwdBars {
    uint64_t full[kBwdMaxStages], empty[kBwdMaxStages], tail, xfull, s_full[2], s_free[2], d_full[2], acc_done[2], acc_full, off_full, drain[3];
    float off[2][kTile];                          // what delta is off by, each group's part
    uint32_t tmem;
    Waits waits;
    Work w;
    Stream st;
};

template <bool KEYS>
__device__ __forceinline__ Stream stream_of(const AttnParams &P, const Work &w, int h) {
    Stream st = {0, 0, 0, 0, 0};
    if (KEYS) {
        const int share = P.Hq / P.Hkv, from = share * w.z / P.splits, to = share * (w.z + 1) / P.splits;
        st.head = h * share + from;
        const int i0 = P.causal ? max(0, w.row - (w.lk - w.lq)) : 0;
        st.first = i0 / kStream;
        st.per_head = max((w.lq + kStream - 1) / kStream - st.first, 0);
        st.n = st.per_head * (to - from);
    } else {
        const int last = min(w.row + kTile, w.lq) - 1;
        st.per_head = st.n = (keys_seen(P, w, last) + kStream - 1) / kStream;
    }
    st.total = !KEYS && st.n <= kSweepTwice ? 2 * st.n : st.n;
    return st;
}

// Columns of tensor memory.  Buffer b: s at b * 128, dp 64 behind it.  For queries
// each buffer's ds has columns of its own.  For keys p and ds of both buffers
// share one place, so a group stores them once the sums have read the last; with
// head sizes above 96 the two sums leave no room for that, and p and ds take the
// place of s and dp (the next scores of that buffer then wait for the sums).
template <int DP, bool KEYS>
struct BwdCols {
    static constexpr bool kAlias = KEYS && DP > 96, kShared = KEYS && !kAlias;
    static constexpr uint32_t kBuf = 128;
    static constexpr uint32_t kP = 256, kDs = KEYS ? 288 : 256;         // of the shared place, or of ds of buffer 0
    static constexpr uint32_t kAcc0 = kAlias ? 256 : 320, kAcc1 = KEYS ? kAcc0 + DP : 320;
    static_assert(kAcc1 + DP <= 512, "tensor memory");
    __device__ static uint32_t p(int b) { return kAlias ? b * kBuf : kP; }
    __device__ static uint32_t ds(int b) { return kAlias ? b * kBuf + 64 : (kShared ? kDs : kDs + 32 * b); }
};

// p and ds of 16 columns, the first of them `col`, as bf16 pairs.  CUT: some are masked.
template <bool KEYS, bool CUT>
__device__ __forceinline__ void bwd_chunk(const uint32_t (&s)[16], const uint32_t (&d)[16], float2 sl2, float nlse2,
                                          float ndelta, int col, int from, int upto, uint32_t (&pp)[8], uint32_t (&pd)[8]) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float2 sc = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float2 dp = make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]));
        const float2 x = KEYS ? mul2(sc, sl2) : fma2(sc, sl2, both(nlse2));
        float2 p = make_float2(ex2(x.x), ex2(x.y));
        float2 q = mul2(p, KEYS ? dp : add2(dp, both(ndelta)));
        if (CUT) {
            if (KEYS ? col + e < from : col + e >= upto) p.x = q.x = 0.f;
            if (KEYS ? col + e + 1 < from : col + e + 1 >= upto) p.y = q.y = 0.f;
        }
        if (KEYS) pp[e / 2] = pack_bf16x2(p.x, p.y);
        pd[e / 2] = pack_bf16x2(q.x, q.y);
    }
}

// p and ds of every second streamed tile, then half of the results; the 128
// threads of group g, one kept row each.
template <int DP, bool KEYS, bool CAUSAL>
__device__ __forceinline__ void bwd_group(const AttnParams &P, BwdBars &B, const Work &w, Stream st, int g, int h) {
    using T = BwdCols<DP, KEYS>;
    volatile Waits *abort = &B.waits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = B.tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t ts = lanes + g * T::kBuf, tp = lanes + T::p(g), td = lanes + T::ds(g);
    const int i = w.row + (warp & 3) * 32 + lane;           // kept row within the sequence
    const bool mine = i < (KEYS ? w.lk : w.lq);
    const float2 sl2 = both(P.scale * kLog2e);
    float nlse2 = 0.f, ndelta = 0.f;                        // of a kept query: -lse log2(e), -delta
    int limit = 0;
    if (!KEYS) {
        limit = mine ? keys_seen(P, w, i) : 0;
        if (mine) {
            const int64_t row = w.q0 + i, at = (int64_t)h * P.Nq + row;
            const __nv_bfloat16 *a = P.dout.at(row, h), *b = P.out.at(row, h);
            for (int e = 0; e < P.D; e += 8) {
                const uint4 u = *reinterpret_cast<const uint4 *>(a + e), v = *reinterpret_cast<const uint4 *>(b + e);
                const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ndelta -= bf16lo_to_f32(x[k]) * bf16lo_to_f32(y[k]) + bf16hi_to_f32(x[k]) * bf16hi_to_f32(y[k]);
            }
            nlse2 = -P.lse[at] * kLog2e;
        }
    }
    // the row's statistics for the key kernel
    auto put_stat = [&] {
        if (KEYS || !mine || g != 0) return;
        // a row that sees no key has lse = -inf; with a large finite value its p is 0 and no product inf * 0
        const int64_t at = (int64_t)h * P.Nq + w.q0 + i;
        const uint2 u = split3(limit > 0 ? -P.lse[at] / P.scale : -1e30f);
        // a delta that is not finite would reach s, and so dv, through the zeros it meets there: three times
        // bf16's largest value is 0 there and overflows in dp
        const uint2 v = ndelta - ndelta == 0.f ? split3(ndelta) : make_uint2(0x7F7F7F7Fu, 0x00007F7Fu);
        P.stat[at] = make_uint4(u.x, u.y, v.x, v.y);
    };
    // scores and dp of tile j, the n-th of this buffer, into registers
    auto take = [&](int n, uint32_t (&s)[4][16], uint32_t (&d)[4][16]) {
        if (!warp_wait(&B.s_full[g], n & 1, abort)) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            tmem_ld_x16(ts + 16 * c, s[c]);
            tmem_ld_x16(ts + 64 + 16 * c, d[c]);
        }
        tmem_ld_wait_for(s);
        tmem_ld_wait_for(d);
        if (!T::kAlias) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.s_free[g]));
        }
        return true;
    };
    int tile = g, j = g;                                    // of the current head's streamed tiles; of all
    if (!KEYS && st.total > st.n) {                         // the first of two sweeps
        float off = 0.f;
        for (; j < st.n; j += 2, tile += 2) {
            uint32_t s[4][16], d[4][16];
            if (!take(j >> 1, s, d)) return;
            const int upto = limit - tile * kStream;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p = ex2(fmaf(__uint_as_float(s[c][e]), sl2.x, nlse2));
                    if (16 * c + e < upto) off = fmaf(p, __uint_as_float(d[c][e]) + ndelta, off);
                }
            if (j > g && !warp_wait(&B.acc_done[g], ((j >> 1) - 1) & 1, abort)) return;   // every phase is met
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.d_full[g]));
        }
        B.off[g][(warp & 3) * 32 + lane] = off;             // both groups meet
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.off_full));
        if (!warp_wait(&B.off_full, 0, abort)) return;
        ndelta -= B.off[0][(warp & 3) * 32 + lane] + B.off[1][(warp & 3) * 32 + lane];
    }
    put_stat();
    const int shift = w.lk - w.lq;
    for (; j < st.total; j += 2, tile += 2) {
        const int n = j >> 1;
        while (tile >= st.per_head) tile -= st.per_head;
        uint32_t s[4][16], d[4][16];
        if (!take(n, s, d)) return;
        const int y = (st.first + tile) * kStream;          // first streamed row
        // queries a key row sees start at i - shift; keys a query row sees end at limit
        const bool cut = __any_sync(0xffffffffu, KEYS ? P.causal && y < i - shift : y + kStream > limit);
        // the columns that count: from `from` on (keys), before `limit` (queries)
        const int from = i - shift - y, upto = limit - y;
        uint32_t pp[4][8], pd[4][8];
        if (cut) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                bwd_chunk<KEYS, true>(s[c], d[c], sl2, nlse2, ndelta, 16 * c, from, upto, pp[c], pd[c]);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                bwd_chunk<KEYS, false>(s[c], d[c], sl2, nlse2, ndelta, 16 * c, from, upto, pp[c], pd[c]);
        }
        // The sums have read what was in its place: the tile before (of the other group)
        // when the place is shared, this group's last tile otherwise.  A barrier per
        // group, since a wait by parity may only look for the phase after the last one
        // known to be over; that is so here, as tile j - 3 was waited for at j - 2.
        if (T::kShared ? j > 0 : !T::kAlias && n > 0) {
            if (!warp_wait(&B.acc_done[T::kShared ? 1 - g : g], (T::kShared ? (j - 1) >> 1 : n - 1) & 1, abort)) return;
            tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (KEYS) tmem_st_x8(tp + 8 * c, pp[c]);
            tmem_st_x8(td + 8 * c, pd[c]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.d_full[g]));
    }
    if (st.n > 0) {
        if (!warp_wait(&B.acc_full, 0, abort)) return;
        tc_fence_after();
    }
    // keys: group 0 writes dv, group 1 dk; queries: every second 16 columns of dq
    const bool is_dv = KEYS && g == 0;
    const uint32_t acc = lanes + (is_dv ? T::kAcc0 : T::kAcc1);
    const float f = is_dv ? 1.0f : P.scale;
    __nv_bfloat16 *out = KEYS ? (is_dv ? P.dv : P.dk).at(w.k0 + i, h) : P.dq.at(w.q0 + i, h);
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) {
        if (!KEYS && (c & 1) != g) continue;
        uint32_t o[1][16] = {{0}};
        if (st.n > 0) {
            tmem_ld_x16(acc + 16 * c, o[0]);
            tmem_ld_wait_for(o);
        }
        if (!mine) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (16 * c + 8 * q >= P.D) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[0][8 * q + e]) * f;
            if (KEYS && P.splits > 1) {
                float4 *dst = reinterpret_cast<float4 *>(
                    P.part_out + ((((int64_t)w.z * 2 + g) * P.Nk + w.k0 + i) * P.Hkv + h) * P.D + 16 * c + 8 * q);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                st_global_v4(out + 16 * c + 8 * q, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
    }
    if (!CAUSAL || st.n == 0) return;
    // Streamed rows that the mask hides from a kept one: keys from `limit` on (fewer for every
    // later query), queries before i - shift (more for every later key).
    const int hidden = KEYS ? i - shift : limit, edge = KEYS ? st.first * kStream : min(st.n * kStream, w.lk);
    const bool whole = KEYS || limit == 0 || (nlse2 - nlse2 == 0.f && ndelta - ndelta == 0.f);   // (no key seen: 0)
    const bool some = mine && whole && (KEYS ? edge < hidden : hidden < edge);
    if (!__any_sync(0xffffffffu, some)) return;
    const bool lost = KEYS ? tmem_odd<DP / 16>(acc, 16) : tmem_odd<(DP / 16 + 1) / 2>(acc + 16 * g, 32, DP / 16 - g);
    uint32_t again = __ballot_sync(0xffffffffu, some && lost);
    int looked = edge;
    bool hit = false;
    __syncwarp();
    while (again) {
        const int src = KEYS ? __ffs(again) - 1 : 31 - __clz(again);
        again ^= 1u << src;
        const int row = (KEYS ? w.k0 : w.q0) + w.row + (warp & 3) * 32 + src, to = __shfl_sync(0xffffffffu, hidden, src);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (KEYS) {
            const int heads = st.n / st.per_head;
            for (; looked < to; ++looked)
                for (int y = st.head; y < st.head + heads; ++y)
                    hit |= quad_odd(quad((is_dv ? P.dout : P.q).at(w.q0 + looked, y), P.D));
            if (!__any_sync(0xffffffffu, hit)) continue;
            const float4 k = quad(P.k.at(row, h), P.D), v = quad(P.v.at(row, h), P.D);
            for (int y = st.head; y < st.head + heads; ++y)
                for (int r = to; r < w.lq && !quad_lost(r, hit, sum); ++r) {
                    const uint4 t = P.stat[(int64_t)y * P.Nq + w.q0 + r];
                    const float4 q = quad(P.q.at(w.q0 + r, y), P.D), dy = quad(P.dout.at(w.q0 + r, y), P.D);
                    const float nl = bf16lo_to_f32(t.x) + bf16hi_to_f32(t.x) + bf16lo_to_f32(t.y);
                    const float nd = bf16lo_to_f32(t.z) + bf16hi_to_f32(t.z) + bf16lo_to_f32(t.w);
                    const float p = ex2((quad_dot(q, k) + nl) * sl2.x);
                    if (is_dv) quad_add(sum, p, dy);
                    else quad_add(sum, p * (quad_dot(dy, v) + nd), q);
                }
            float *part = P.part_out + ((((int64_t)w.z * 2 + g) * P.Nk + row) * P.Hkv + h) * P.D;
            if (hit) quad_store((is_dv ? P.dv : P.dk).at(row, h), P.splits > 1 ? part : nullptr, f, sum);
        } else {
            const int kv = h / (P.Hq / P.Hkv);
            const float nl = __shfl_sync(0xffffffffu, nlse2, src), nd = __shfl_sync(0xffffffffu, ndelta, src);
            // (the other group has the other columns)
            while (looked > to) hit |= quad_odd(quad(P.k.at(w.k0 + --looked, kv), P.D)) && ((lane >> 2) & 1) == g;
            if (!__any_sync(0xffffffffu, hit)) continue;
            const float4 q = quad(P.q.at(row, h), P.D), dy = quad(P.dout.at(row, h), P.D);
            for (int j = 0; j < to && !quad_lost(j, hit, sum); ++j) {
                const float4 k = quad(P.k.at(w.k0 + j, kv), P.D), v = quad(P.v.at(w.k0 + j, kv), P.D);
                const float p = ex2(fmaf(quad_dot(q, k), sl2.x, nl));
                quad_add(sum, p * (quad_dot(dy, v) + nd), k);
            }
            if (hit) quad_store(P.dq.at(row, h), nullptr, f, sum);
        }
    }
}

// Loads (one warp): the kept tiles, then the streamed ones through the ring.
template <int DP, bool KEYS>
__device__ __forceinline__ void bwd_load(const AttnParams &P, BwdBars &B, const Work &w, Stream st,
                                         const CUtensorMap &mx0, const CUtensorMap &mx1, const CUtensorMap &my0,
                                         const CUtensorMap &my1, uint8_t *kept, uint8_t *ring, uint8_t *stats, int h) {
    using S = BwdShape<DP, KEYS>;
    constexpr int kC = kChunks<DP>;
    constexpr uint32_t kKept = S::kKept, kOne = S::kOne;                       // bytes of one kept / streamed tile
    volatile Waits *abort = &B.waits;
    const int lane = threadIdx.x & 31;
    const int y_len = KEYS ? w.lq : w.lk;                   // streamed rows of the sequence
    const int x_row = (KEYS ? w.k0 : w.q0) + w.row;
    if (lane == 0) {
        mbar_arrive_expect_tx(smem_addr(&B.xfull), 2 * kKept);
        for (int t = 0; t < 2; ++t)
            for (int c = 0; c < kC; ++c)
                for (int half = 0; half < 2; ++half)
                    tma_load_3d(smem_addr(kept + t * kKept + c * kChunkBytes + half * kStreamChunk), t ? &mx1 : &mx0,
                                smem_addr(&B.xfull), 64 * c, h, x_row + half * kStream);
    }
    int f = 0, tails = 0, tile = 0, y_head = KEYS ? st.head : h / (P.Hq / P.Hkv);
    bool ok = true;
    Slot<S::kStages> r;
    for (; f < st.total; ++f, ++tile, r.next()) {
        const int slot = r.at;
        ok = warp_wait(&B.empty[slot], r.phase ^ 1, abort);
        if (!ok) break;
        if (tile == st.per_head) {                          // the next head, or the second sweep
            tile = 0;
            if (KEYS) ++y_head;
        }
        const int row = (st.first + tile) * kStream;
        const int y_row = (KEYS ? w.q0 : w.k0) + row;
        const int valid = min(y_len - row, kStream);
        uint8_t *dst = ring + slot * 2 * kOne;
        const bool clean = valid < kStream;                 // the sequence's last tile: zeros behind it
        uint64_t *bar = clean ? &B.tail : &B.full[slot];
        if (lane == 0) {
            mbar_arrive_expect_tx(smem_addr(bar), 2 * kOne + (KEYS ? valid * 16 : 0));
            if (KEYS)
                bulk_load(smem_addr(stats + slot * kStats), P.stat + (int64_t)y_head * P.Nq + y_row, valid * 16,
                          smem_addr(bar));
            for (int t = 0; t < 2; ++t)
                for (int c = 0; c < kC; ++c)
                    tma_load_3d(smem_addr(dst + t * kOne + c * kStreamChunk), t ? &my1 : &my0, smem_addr(bar), 64 * c,
                                y_head, y_row);
        }
        __syncwarp();
        if (clean) {
            ok = warp_wait(&B.tail, tails & 1, abort);
            if (!ok) {
                warp_drain(&B.tail, tails & 1);
                break;
            }
            ++tails;
            const int end = (valid + 15) & ~15;
            for (int t = 0; t < 2; ++t) zero_rows<kC, kStreamChunk>(dst + t * kOne, valid, end);
            if (KEYS && lane < end - valid)
                *reinterpret_cast<uint4 *>(stats + slot * kStats + (valid + lane) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.full[slot]));
        }
    }
    drain_loads(&B.xfull, B.full, S::kStages, f);
}

// s and dp of every second streamed tile, buffer b (one warp each: while one waits
// for room, the other keeps the tensor cores busy).
template <int DP, bool KEYS>
__device__ __forceinline__ void bwd_scores(BwdBars &B, Stream st, uint8_t *kept, uint8_t *ring, uint8_t *select,
                                           uint8_t *stats, int b) {
    using T = BwdCols<DP, KEYS>;
    using S = BwdShape<DP, KEYS>;
    constexpr uint32_t kKept = S::kKept, kOne = S::kOne, kIdS = idesc_bf16_f32(kTile, kStream);
    volatile Waits *abort = &B.waits;
    const uint32_t one = elect_one(), tm = B.tmem;
    const uint32_t x0 = desc_k(smem_addr(kept)), x1 = desc_k(smem_addr(kept + kKept));
    bool ok = warp_wait(&B.xfull, 0, abort);
    Slot<S::kStages> r;
    r.at = b;
    for (int j = b; j < st.total && ok; j += 2, r.next(2)) {
        const int n = j >> 1, slot = r.at;
        ok = warp_wait(&B.full[slot], r.phase, abort) && (n == 0 || warp_wait(&B.s_free[b], (n - 1) & 1, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + b * T::kBuf, y0 = desc_k(smem_addr(ring + slot * 2 * kOne)), y1 = y0 + (kOne >> 4);
        if (one) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                mma_ss(d, x0 + step_k<kChunkBytes>(k), y0 + step_k<kStreamChunk>(k), kDescHi, kDescHi, kIdS, k > 0);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                mma_ss(d + 64, x1 + step_k<kChunkBytes>(k), y1 + step_k<kStreamChunk>(k), kDescHi, kDescHi, kIdS, k > 0);
            if (KEYS) {
                const uint32_t at = smem_addr(stats + slot * kStats), zeros = smem_addr(stats + S::kStages * kStats);
                const uint32_t z = desc_flat(at, zeros - at), sel = desc_flat(smem_addr(select), kTile * 16);
                mma_ss(d, sel, z, kDescHiFlat, kDescHiFlat, kIdS, true);
                mma_ss(d + 64, sel + (kSelect >> 4), z, kDescHiFlat, kDescHiFlat, kIdS, true);
            }
            mma_commit(&B.s_full[b]);
        }
        __syncwarp();
    }
    drain_mmas(one, &B.drain[b]);
}

// The sums over the streamed tiles (one warp).
template <int DP, bool KEYS>
__device__ __forceinline__ void bwd_sums(BwdBars &B, Stream st, uint8_t *ring, int y_len) {
    using T = BwdCols<DP, KEYS>;
    using S = BwdShape<DP, KEYS>;
    constexpr uint32_t kOne = S::kOne, kIdA = idesc_b_mn(kTile, DP);
    volatile Waits *abort = &B.waits;
    const uint32_t one = elect_one(), tm = B.tmem;
    // kept rows += A (tensor memory) times the streamed tile at z
    auto add = [&](uint32_t acc, uint32_t a, uint32_t z, int steps, bool more) {
        mma_ts(acc, a, z, kDescHi, kIdA, more);
        if (steps == kStream / 16) {
#pragma unroll
            for (int k = 1; k < kStream / 16; ++k) mma_ts(acc, a + 8 * k, z + step_mn(k), kDescHi, kIdA, true);
        } else {
            for (int k = 1; k < steps; ++k) mma_ts(acc, a + 8 * k, z + step_mn(k), kDescHi, kIdA, true);
        }
    };
    bool ok = true;
    Slot<S::kStages> r;
    int tile = 0;
    const int second = st.total - st.n;
    for (int j = 0; j < st.total && ok; ++j, ++tile, r.next()) {
        if (tile == st.per_head) tile = 0;
        const int b = j & 1, slot = r.at, row = (st.first + tile) * kStream;
        const int steps = (min(y_len - row, kStream) + 15) / 16;
        ok = warp_wait(&B.full[slot], r.phase, abort) && warp_wait(&B.d_full[b], (j >> 1) & 1, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t z0 = desc_mn<kStreamChunk>(smem_addr(ring + slot * 2 * kOne)), z1 = z0 + (kOne >> 4);
        if (one && j < second) {                            // the first of two sweeps adds nothing
            mbar_arrive(smem_addr(&B.acc_done[b]));
            mbar_arrive(smem_addr(&B.empty[slot]));
        } else if (one) {
            if (KEYS) add(tm + T::kAcc0, tm + T::p(b), z1, steps, j > second);
            add(tm + T::kAcc1, tm + T::ds(b), z0, steps, j > second);
            mma_commit(T::kAlias ? &B.s_free[b] : &B.acc_done[b]);
            mma_commit(&B.empty[slot]);
            if (j + 1 == st.total) mma_commit(&B.acc_full);
        }
        __syncwarp();
    }
    drain_mmas(one, &B.drain[2]);
}

// mx0, mx1: maps of the kept tensors, my0, my1 of the streamed ones (boxes of 64 rows).
template <int DP, bool KEYS, bool CAUSAL>
__global__ void __launch_bounds__(kAttnThreads, 1)
pe_attn_bwd_kernel(const __grid_constant__ CUtensorMap mx0, const __grid_constant__ CUtensorMap mx1,
                   const __grid_constant__ CUtensorMap my0, const __grid_constant__ CUtensorMap my1,
                   const __grid_constant__ AttnParams P) {
    using S = BwdShape<DP, KEYS>;
    extern __shared__ uint8_t raw[];
    __shared__ BwdBars B;
    uint8_t *kept = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023), *ring = kept + 2 * S::kKept;
    uint8_t *select = kept + S::kTiles, *stats = select + 2 * kSelect;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 9) {
        const Place at = place_of<!KEYS>(P, KEYS ? P.Hkv : P.Hq);
        Work w = find_work(P, KEYS, at.tile, kTile);
        w.h = at.h;
        w.z = at.z;
        if (lane == 0) {
            B.w = w;
            if (w.row >= 0) B.st = stream_of<KEYS>(P, w, w.h);
            B.waits.abort = 0;
#ifdef PE_DEBUG_BOUNDS
            B.waits.limit = P.wait_clocks;
#endif
            for (int i = 0; i < S::kStages; ++i) {
                mbar_init(smem_addr(&B.full[i]), 1);
                mbar_init(smem_addr(&B.empty[i]), 1);
            }
            mbar_init(smem_addr(&B.tail), 1);
            mbar_init(smem_addr(&B.xfull), 1);
            mbar_init(smem_addr(&B.acc_full), 1);
            mbar_init(smem_addr(&B.off_full), 8);
            for (int t = 0; t < 2; ++t) {
                mbar_init(smem_addr(&B.s_full[t]), 1);
                mbar_init(smem_addr(&B.s_free[t]), BwdCols<DP, KEYS>::kAlias ? 1 : 4);
                mbar_init(smem_addr(&B.d_full[t]), 4);
                mbar_init(smem_addr(&B.acc_done[t]), 1);
            }
            for (int t = 0; t < 3; ++t) mbar_init(smem_addr(&B.drain[t]), 1);
            fence_mbar_init();
            prefetch_tmap(&mx0);
            prefetch_tmap(&mx1);
            prefetch_tmap(&my0);
            prefetch_tmap(&my1);
        }
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(&B.tmem), 512);
        tmem_relinquish();
    }
    if (KEYS) {
        // 1 in columns 0, 1, 2 selects the first statistic, in 4, 5, 6 the second; the rest is 0
        for (int i = threadIdx.x; i < (int)((2 * kSelect + (S::kStages + 1) * kStats) / 16); i += blockDim.x) {
            const uint32_t one2 = 0x3F803F80u, one1 = 0x00003F80u;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i < kTile) v = make_uint4(one2, one1, 0, 0);
            if (i >= (int)(kSelect / 16) && i < (int)(kSelect / 16) + kTile) v = make_uint4(0, 0, one2, one1);
            *reinterpret_cast<uint4 *>(select + i * 16) = v;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Work &w = B.w;                                    // in shared memory: registers are short
    const int h = w.h;
    // the key kernel starts as the query kernel, whose statistics it reads, ends
    if (!KEYS) griddep_launch_dependents();
    if (KEYS && P.splits > 1) griddep_launch_dependents();  // the joining kernel
    if (KEYS) griddep_wait();                               // (before any bounded wait)
    if (w.row < 0) {                                        // more blocks than tiles
        if (warp == 8) tmem_dealloc(B.tmem, 512);
        return;
    }
    const Stream &st = B.st;                                // (each role copies what its loop needs)
    if (warp < 8) {
        regs_up<kRegsUp>();
        bwd_group<DP, KEYS, CAUSAL>(P, B, w, st, warp >> 2, h);
    } else {
        regs_down<kRegsDown>();
        if (st.n > 0) {
            if (warp == 8) bwd_load<DP, KEYS>(P, B, w, st, mx0, mx1, my0, my1, kept, ring, stats, h);
            else if (warp < 11) bwd_scores<DP, KEYS>(B, st, kept, ring, select, stats, warp - 9);
            else bwd_sums<DP, KEYS>(B, st, ring, KEYS ? w.lq : w.lk);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && B.waits.abort) atomicExch(P.err, (int)PE_ERR_DEVICE_TIMEOUT);
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(B.tmem, 512);
    }
}

// Adds the parts of dk and dv in order (one warp per key row and key head).
__global__ void __launch_bounds__(256) pe_attn_join_grads_kernel(const __grid_constant__ AttnParams P) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);          // [Nk, Hkv]
    if (at >= (int64_t)P.Nk * P.Hkv || 4 * lane >= P.D) return;
    const int r = (int)(at / P.Hkv), h = (int)(at - (int64_t)r * P.Hkv);
    if (!in_sequence(P.cu_k, P.n_seq, P.Nk, r)) return;
    const int64_t step = (int64_t)P.Nk * P.Hkv * P.D;
    const float *src = P.part_out + at * P.D + 4 * lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), k = v;
#pragma unroll 4
    for (int z = 0; z < P.splits; ++z) {
        const float4 a = *reinterpret_cast<const float4 *>(src + 2 * z * step);
        const float4 b = *reinterpret_cast<const float4 *>(src + (2 * z + 1) * step);
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
        k.x += b.x, k.y += b.y, k.z += b.z, k.w += b.w;
    }
    *reinterpret_cast<uint2 *>(P.dv.at(r, h) + 4 * lane) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    *reinterpret_cast<uint2 *>(P.dk.at(r, h) + 4 * lane) = make_uint2(pack_bf16x2(k.x, k.y), pack_bf16x2(k.z, k.w));
}

}  // namespace pe
