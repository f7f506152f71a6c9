// Attention over packed sequences, forward and backward (include/pe.h has the
// formulas).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "../../include/pe.h"
#include "pe_device.cuh"

namespace pe {

// ------------------------------------------------------------- one-CTA tcgen05

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A whole warp waits; all lanes go on, or none (a wait gave up).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(smem_addr(bar), parity, abort));
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

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A holds two bf16 per 32-bit column, K along the columns
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive on `bar` once every MMA this thread has issued is done.
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
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
    float *lse2, *delta;          // [Hq, Nq]: lse * log2(e), and dout . out (backward)
    int *err;
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
};

// Tile `t` of the tiles of `rows` rows that cut the sequences of `cu`, one
// sequence after the other; called by one whole warp.  There are at most
// n / rows + n_seq tiles.
__device__ __forceinline__ Work find_work(const AttnParams &P, bool by_key, int t, int rows) {
    const int lane = threadIdx.x & 31;
    const int32_t *cu = by_key ? P.cu_k : P.cu_q;
    const int n = by_key ? P.Nk : P.Nq;
    Work w = {0, 0, 0, 0, -1};
    for (int base = 0; base < P.n_seq; base += 32) {
        const int s = base + lane;
        int tiles = 0;
        if (s < P.n_seq) {
            const int len = boundary(cu, s + 1, n) - boundary(cu, s, n);
            tiles = len > 0 ? (len + rows - 1) / rows : 0;
        }
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, t < sum);
        if (hit) {
            const int src = __ffs(hit) - 1, seq = base + src;
            const int before = __shfl_sync(0xffffffffu, sum - tiles, src);
            w.q0 = boundary(P.cu_q, seq, P.Nq);
            w.lq = max(boundary(P.cu_q, seq + 1, P.Nq) - w.q0, 0);
            w.k0 = boundary(P.cu_k, seq, P.Nk);
            w.lk = max(boundary(P.cu_k, seq + 1, P.Nk) - w.k0, 0);
            w.row = (t - before) * rows;
            return w;
        }
        t -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return w;
}

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

// K-major operand (chunks of 64 columns, CHUNK bytes each), k-step of 16 columns.
template <int CHUNK>
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kstep) {
    return smem_desc(tile + (kstep >> 2) * CHUNK + (kstep & 3) * 32, 16, 1024, kLayoutSw128);
}
// The same tile read along its rows (MN-major): k-step of 16 rows, N = the columns.
template <int CHUNK>
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kstep) {
    return smem_desc(tile + kstep * 2048, CHUNK, 1024, kLayoutSw128);
}
__host__ __device__ constexpr uint32_t idesc_b_mn(int M, int N) { return idesc_bf16_f32(M, N) | (1u << 16); }

// ------------------------------------------------------------- forward
//
// A block takes 256 query rows of one sequence and head as two tiles of 128,
// and streams the sequence's keys and values past them in tiles of 128.  Roles:
// warps 0-3 and 4-7 do the softmax of tile 0 and 1 (one thread per row: row
// maximum and sum need no shuffles), warp 8 loads, warp 9 issues the MMAs.
// While one tile's softmax runs, the tensor cores work for the other.  Scores
// (fp32) and probabilities (bf16, in the same columns) stay in tensor memory;
// the output accumulates there too and is rescaled only when a row's maximum
// has grown by more than 2^8, which keeps P in bf16's range and is rare.

constexpr int kFwdThreads = 320;
constexpr int kFwdStages = 4;

template <int DP>
constexpr int kChunks = DP > 64 ? 2 : 1;

template <int DP>
constexpr size_t kFwdSmem = (size_t)(2 + kFwdStages) * kChunks<DP> * kChunkBytes + 1024 + 256;

struct FwdBars {
    uint64_t full[kFwdStages], empty[kFwdStages], tail, qfull, s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int abort;
    Work w;
};

// Online softmax of one 128-row tile; all 128 threads of its warps.
template <int DP>
__device__ __forceinline__ void fwd_softmax(const AttnParams &P, FwdBars &B, const Work &w, int tile, int n_kv, int h) {
    volatile int *abort = &B.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // 32 lanes a warp, in bits 16..
    const uint32_t ts = B.tmem + lanes + tile * 128, to = B.tmem + lanes + 256 + tile * 128;
    const int i = w.row + tile * kTile + (warp & 3) * 32 + lane;  // row within the sequence
    const int limit = keys_seen(P, w, i);
    const float sl2 = P.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n_kv; ++j) {
        if (!warp_wait(&B.s_full[tile], j & 1, abort)) return;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, s[c]);
        tmem_ld_wait();
        if (__any_sync(0xffffffffu, (j + 1) * kTile > limit)) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (j * kTile + 32 * c + e >= limit) s[c][e] = __float_as_uint(-INFINITY);
        }
        float mx = m;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(s[c][e]));
        if (__any_sync(0xffffffffu, (mx - m) * sl2 > 8.0f)) {
            // MMAs complete in order: S(j) is there, so P V of j - 1 is done
            const float f = m == -INFINITY ? 0.f : ex2((m - mx) * sl2);
            l *= f;
            m = mx;
            if (j > 0) {
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t o[16];
                    tmem_ld_x16(to + 16 * c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st_x16(to + 16 * c, o);
                }
            }
        }
        const float base = m == -INFINITY ? 0.f : m * sl2;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float a = ex2(fmaf(__uint_as_float(s[c][2 * e]), sl2, -base));
                const float b = ex2(fmaf(__uint_as_float(s[c][2 * e + 1]), sl2, -base));
                sum[e & 1] += a;
                sum[2 + (e & 1)] += b;
                pk[e] = pack_bf16x2(a, b);
            }
            tmem_st_x16(ts + 16 * c, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.p_full[tile]));
    }
    if (n_kv > 0) {
        if (!warp_wait(&B.o_full[tile], 0, abort)) return;
        tc_fence_after();
    }
    const bool mine = i < w.lq;
    const float inv = 1.0f / l;
    __nv_bfloat16 *out = P.out.at(w.q0 + i, h);
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) {
        uint32_t o[16] = {0};
        if (n_kv > 0) {
            tmem_ld_x16(to + 16 * c, o);
            tmem_ld_wait();
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(o[8 * g + 2 * e]) * inv, b = __uint_as_float(o[8 * g + 2 * e + 1]) * inv;
                pk[e] = limit > 0 ? pack_bf16x2(a, b) : 0u;
            }
            if (mine && 16 * c + 8 * g < P.D) st_global_v4(out + 16 * c + 8 * g, pk[0], pk[1], pk[2], pk[3]);
        }
    }
    if (mine && P.lse)
        P.lse[(int64_t)h * P.Nq + w.q0 + i] = limit > 0 ? m * P.scale + logf(l) : -INFINITY;
}

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
pe_attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnParams P) {
    constexpr int kC = kChunks<DP>;
    constexpr uint32_t kTileBytes = kC * kChunkBytes;
    extern __shared__ uint8_t raw[];
    __shared__ FwdBars B;
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    uint8_t *sq = smem, *ring = smem + 2 * kTileBytes;
    volatile int *abort = &B.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, hk = h / (P.Hq / P.Hkv);
    if (warp == 9) {
        const Work w = find_work(P, false, blockIdx.x, 2 * kTile);
        if (lane == 0) {
            B.w = w;
            B.abort = 0;
            for (int i = 0; i < kFwdStages; ++i) mbar_init(smem_addr(&B.full[i]), 1), mbar_init(smem_addr(&B.empty[i]), 1);
            mbar_init(smem_addr(&B.tail), 1);
            mbar_init(smem_addr(&B.qfull), 1);
            mbar_init(smem_addr(&B.drain), 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(smem_addr(&B.s_full[t]), 1);
                mbar_init(smem_addr(&B.p_full[t]), 4);
                mbar_init(smem_addr(&B.o_full[t]), 1);
            }
            fence_mbar_init();
            prefetch_tmap(&mq);
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
        }
    }
    __syncthreads();
    const Work w = B.w;
    if (w.row < 0) return;
    if (warp == 8) {
        tmem_alloc(smem_addr(&B.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int n_tiles = w.lq - w.row > kTile ? 2 : 1;
    int n_kv[2];                                            // key tiles that each query tile meets
    for (int t = 0; t < 2; ++t) {
        const int last = min(w.row + (t + 1) * kTile, w.lq) - 1;
        n_kv[t] = t < n_tiles ? (keys_seen(P, w, last) + kTile - 1) / kTile : 0;
    }
    const int n_max = max(n_kv[0], n_kv[1]);
    if (warp < 4) {
        fwd_softmax<DP>(P, B, w, 0, n_kv[0], h);
    } else if (warp < 8) {
        if (n_tiles > 1) fwd_softmax<DP>(P, B, w, 1, n_kv[1], h);
    } else if (warp == 8) {
        // ---- loads: Q, then K0 V0 K1 V1 ... through one ring
        if (n_max > 0 && lane == 0) {
            mbar_arrive_expect_tx(smem_addr(&B.qfull), n_tiles * kTileBytes);
            for (int t = 0; t < n_tiles; ++t)
                for (int c = 0; c < kC; ++c)
                    tma_load_3d(smem_addr(sq + t * kTileBytes + c * kChunkBytes), &mq, smem_addr(&B.qfull), 64 * c, h,
                                w.q0 + w.row + t * kTile);
        }
        int f = 0;
        bool ok = true;
        for (; f < 2 * n_max && ok; ++f) {
            const int slot = f % kFwdStages, j = f >> 1;
            const bool is_v = f & 1;
            ok = warp_wait(&B.empty[slot], ((f / kFwdStages) & 1) ^ 1, abort);
            if (!ok) break;
            uint8_t *dst = ring + slot * kTileBytes;
            const int valid = min(w.lk - j * kTile, kTile);
            const bool clean = is_v && valid < kTile;       // the last tile of V: zeros behind the sequence
            uint64_t *bar = clean ? &B.tail : &B.full[slot];
            if (lane == 0) {
                mbar_arrive_expect_tx(smem_addr(bar), kTileBytes);
                for (int c = 0; c < kC; ++c)
                    tma_load_3d(smem_addr(dst + c * kChunkBytes), is_v ? &mv : &mk, smem_addr(bar), 64 * c, hk,
                                w.k0 + j * kTile);
            }
            __syncwarp();
            if (clean) {
                ok = warp_wait(&B.tail, 0, abort);
                if (!ok) {
                    int never = 0;
                    mbar_wait(smem_addr(&B.tail), 0, &never);
                    break;
                }
                zero_rows<kC, kChunkBytes>(dst, valid, (valid + 15) & ~15);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&B.full[slot]));
            }
        }
        if (!ok) {   // a wait gave up: the copies in flight still land before the block ends
            int never = 0;
            mbar_wait(smem_addr(&B.qfull), 0, &never);
            for (int s = max(f - kFwdStages, 0); s < f; ++s) {
                mbar_wait(smem_addr(&B.full[s % kFwdStages]), (s / kFwdStages) & 1, &never);
            }
        }
    } else if (lane == 0 && n_max > 0) {
        // ---- MMAs
        constexpr uint32_t kIdS = idesc_bf16_f32(kTile, kTile), kIdO = idesc_b_mn(kTile, DP);
        const int ksteps = (P.D + 15) / 16;
        const uint32_t a_q = smem_addr(sq), a_r = smem_addr(ring);
        auto wait_full = [&](int f) {
            return mbar_wait(smem_addr(&B.full[f % kFwdStages]), (f / kFwdStages) & 1, abort);
        };
        auto issue_s = [&](int t, int f) {
            for (int k = 0; k < ksteps; ++k)
                mma_ss(B.tmem + t * 128, desc_k<kChunkBytes>(a_q + t * kTileBytes, k),
                       desc_k<kChunkBytes>(a_r + f % kFwdStages * kTileBytes, k), kIdS, k > 0);
            mma_commit(&B.s_full[t]);
        };
        bool ok = mbar_wait(smem_addr(&B.qfull), 0, abort) && wait_full(0);
        if (ok) {
            tc_fence_after();
            for (int t = 0; t < n_tiles; ++t)
                if (n_kv[t] > 0) issue_s(t, 0);
            mma_commit(&B.empty[0]);
        }
        for (int j = 0; j < n_max && ok; ++j) {
            const int fv = 2 * j + 1, fk = 2 * j + 2;
            const bool more = j + 1 < n_max;
            ok = wait_full(fv) && (!more || wait_full(fk));
            const int rows = min(w.lk - j * kTile, kTile);
            for (int t = 0; t < n_tiles && ok; ++t) {
                if (j < n_kv[t]) {
                    ok = mbar_wait(smem_addr(&B.p_full[t]), j & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const int psteps = (rows + 15) / 16;
                    for (int k = 0; k < psteps; ++k)
                        mma_ts(B.tmem + 256 + t * 128, B.tmem + t * 128 + 8 * k,
                               desc_mn<kChunkBytes>(a_r + fv % kFwdStages * kTileBytes, k), kIdO, j > 0 || k > 0);
                    if (j + 1 == n_kv[t]) mma_commit(&B.o_full[t]);
                }
                if (j + 1 < n_kv[t]) issue_s(t, fk);
            }
            if (!ok) break;
            mma_commit(&B.empty[fv % kFwdStages]);
            if (more) mma_commit(&B.empty[fk % kFwdStages]);
        }
        if (!ok) {   // MMAs in flight finish before their tensor memory is freed
            int never = 0;
            mma_commit(&B.drain);
            mbar_wait(smem_addr(&B.drain), 0, &never);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && B.abort) atomicExch(P.err, (int)PE_ERR_DEVICE_TIMEOUT);
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(B.tmem, 512);
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

constexpr int kStream = 64;                       // streamed rows per tile
constexpr int kStreamChunk = kStream * 128;       // bytes of 64 rows of 64 bf16
constexpr int kBwdThreads = 320;
constexpr int kBwdStages = 4;

template <int DP>
constexpr size_t kBwdSmem = (size_t)kChunks<DP> * (2 * kChunkBytes + kBwdStages * 2 * kStreamChunk) + 1024;

struct BwdBars {
    uint64_t full[kBwdStages], empty[kBwdStages], tail, xfull, s_full[2], d_full[2], acc_full, drain;
    uint32_t tmem;
    int abort;
    Work w;
    alignas(16) float stat[kBwdStages][2][kStream];   // lse2 and delta of the streamed queries
};

// 4 bytes to shared memory without waiting; zero when !take.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}
// This thread's copies so far, once they have landed, count as one arrival.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// The streamed tiles of one block: for keys, the query tiles of every head that
// shares the key head, from the first that sees the tile's first key.
struct Stream {
    int first, per_head, n;                       // first tile, tiles per head, tiles in all
};

template <bool KEYS>
__device__ __forceinline__ Stream stream_of(const AttnParams &P, const Work &w) {
    Stream st = {0, 0, 0};
    if (KEYS) {
        const int i0 = P.causal ? max(0, w.row - (w.lk - w.lq)) : 0;
        st.first = i0 / kStream;
        st.per_head = max((w.lq + kStream - 1) / kStream - st.first, 0);
        st.n = st.per_head * (P.Hq / P.Hkv);
    } else {
        const int last = min(w.row + kTile, w.lq) - 1;
        st.per_head = st.n = (keys_seen(P, w, last) + kStream - 1) / kStream;
    }
    return st;
}

// p and ds of every second streamed tile, then half of the results; the 128
// threads of group g, one kept row each.
template <int DP, bool KEYS>
__device__ __forceinline__ void bwd_group(const AttnParams &P, BwdBars &B, const Work &w, const Stream &st, int g, int h) {
    volatile int *abort = &B.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = B.tmem + lanes + g * 128, td = ts + 64;
    const int i = w.row + (warp & 3) * 32 + lane;           // kept row within the sequence
    const bool mine = i < (KEYS ? w.lk : w.lq);
    const float sl2 = P.scale * kLog2e;
    float lse2 = 0.f, delta = 0.f;
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
                    delta += bf16lo_to_f32(x[k]) * bf16lo_to_f32(y[k]) + bf16hi_to_f32(x[k]) * bf16hi_to_f32(y[k]);
            }
            // a row that sees no key has lse = -inf; +inf gives it p = 0 for every key
            lse2 = limit > 0 ? P.lse[at] * kLog2e : INFINITY;
            if (g == 0) {
                P.lse2[at] = lse2;
                P.delta[at] = delta;
            }
        }
    }
    const int shift = w.lk - w.lq;
    for (int j = g; j < st.n; j += 2) {
        const int n = j >> 1, stage = j % kBwdStages;
        if (KEYS && !warp_wait(&B.full[stage], (j / kBwdStages) & 1, abort)) return;
        if (!warp_wait(&B.s_full[g], n & 1, abort)) return;
        tc_fence_after();
        const int y = (st.first + (KEYS ? j % st.per_head : j)) * kStream;      // first streamed row
        uint32_t s[2][32], d[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            tmem_ld_32x32b_x32(ts + 32 * c, s[c]);
            tmem_ld_32x32b_x32(td + 32 * c, d[c]);
        }
        tmem_ld_wait();
        // queries a key row sees start at i - shift; keys a query row sees end at limit
        const bool cut = __any_sync(0xffffffffu, KEYS ? P.causal && y < i - shift : y + kStream > limit);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t pp[16], pd[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float4 L = make_float4(lse2, lse2, lse2, lse2), T = make_float4(delta, delta, delta, delta);
                if (KEYS) {
                    L = *reinterpret_cast<const float4 *>(&B.stat[stage][0][32 * c + e]);
                    T = *reinterpret_cast<const float4 *>(&B.stat[stage][1][32 * c + e]);
                }
                const float l4[4] = {L.x, L.y, L.z, L.w}, t4[4] = {T.x, T.y, T.z, T.w};
                float p[4], q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = ex2(fmaf(__uint_as_float(s[c][e + k]), sl2, -l4[k]));
                    q[k] = p[k] * (__uint_as_float(d[c][e + k]) - t4[k]);
                    if (cut) {
                        const int col = y + 32 * c + e + k;
                        if (KEYS ? col < i - shift : col >= limit) p[k] = q[k] = 0.f;
                    }
                }
                pp[e / 2] = pack_bf16x2(p[0], p[1]);
                pp[e / 2 + 1] = pack_bf16x2(p[2], p[3]);
                pd[e / 2] = pack_bf16x2(q[0], q[1]);
                pd[e / 2 + 1] = pack_bf16x2(q[2], q[3]);
            }
            if (KEYS) tmem_st_x16(ts + 16 * c, pp);
            tmem_st_x16(td + 16 * c, pd);
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
    const uint32_t acc = B.tmem + lanes + (is_dv ? 256 : 384);
    const float f = is_dv ? 1.0f : P.scale;
    __nv_bfloat16 *out = KEYS ? (is_dv ? P.dv : P.dk).at(w.k0 + i, h) : P.dq.at(w.q0 + i, h);
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) {
        if (!KEYS && (c & 1) != g) continue;
        uint32_t o[16] = {0};
        if (st.n > 0) {
            tmem_ld_x16(acc + 16 * c, o);
            tmem_ld_wait();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pk[e] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * f, __uint_as_float(o[8 * q + 2 * e + 1]) * f);
            if (mine && 16 * c + 8 * q < P.D) st_global_v4(out + 16 * c + 8 * q, pk[0], pk[1], pk[2], pk[3]);
        }
    }
}

// mx0, mx1: maps of the kept tensors, my0, my1 of the streamed ones (boxes of 64 rows).
template <int DP, bool KEYS>
__global__ void __launch_bounds__(kBwdThreads, 1)
pe_attn_bwd_kernel(const __grid_constant__ CUtensorMap mx0, const __grid_constant__ CUtensorMap mx1,
                   const __grid_constant__ CUtensorMap my0, const __grid_constant__ CUtensorMap my1,
                   const __grid_constant__ AttnParams P) {
    constexpr int kC = kChunks<DP>;
    constexpr uint32_t kKept = kC * kChunkBytes, kOne = kC * kStreamChunk;     // bytes of one kept / streamed tile
    extern __shared__ uint8_t raw[];
    __shared__ BwdBars B;
    uint8_t *kept = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023), *ring = kept + 2 * kKept;
    volatile int *abort = &B.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, share = P.Hq / P.Hkv;
    if (warp == 9) {
        const Work w = find_work(P, KEYS, blockIdx.x, kTile);
        if (lane == 0) {
            B.w = w;
            B.abort = 0;
            for (int i = 0; i < kBwdStages; ++i) {
                mbar_init(smem_addr(&B.full[i]), KEYS ? 33 : 1);
                mbar_init(smem_addr(&B.empty[i]), 1);
            }
            mbar_init(smem_addr(&B.tail), 1);
            mbar_init(smem_addr(&B.xfull), 1);
            mbar_init(smem_addr(&B.acc_full), 1);
            mbar_init(smem_addr(&B.drain), 1);
            for (int t = 0; t < 2; ++t) mbar_init(smem_addr(&B.s_full[t]), 1), mbar_init(smem_addr(&B.d_full[t]), 4);
            fence_mbar_init();
            prefetch_tmap(&mx0);
            prefetch_tmap(&mx1);
            prefetch_tmap(&my0);
            prefetch_tmap(&my1);
        }
    }
    __syncthreads();
    const Work w = B.w;
    if (w.row < 0) return;
    if (warp == 8) {
        tmem_alloc(smem_addr(&B.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Stream st = stream_of<KEYS>(P, w);
    const int y_len = KEYS ? w.lq : w.lk;                   // streamed rows of the sequence
    if (warp < 8) {
        bwd_group<DP, KEYS>(P, B, w, st, warp >> 2, h);
    } else if (warp == 8 && st.n > 0) {
        // ---- loads
        const int x_row = (KEYS ? w.k0 : w.q0) + w.row, x_head = h;
        if (lane == 0) {
            mbar_arrive_expect_tx(smem_addr(&B.xfull), 2 * kKept);
            for (int t = 0; t < 2; ++t)
                for (int c = 0; c < kC; ++c)
                    for (int half = 0; half < 2; ++half)
                        tma_load_3d(smem_addr(kept + t * kKept + c * kChunkBytes + half * kStreamChunk), t ? &mx1 : &mx0,
                                    smem_addr(&B.xfull), 64 * c, x_head, x_row + half * kStream);
        }
        int f = 0, tails = 0;
        bool ok = true;
        for (; f < st.n; ++f) {
            const int slot = f % kBwdStages;
            ok = warp_wait(&B.empty[slot], ((f / kBwdStages) & 1) ^ 1, abort);
            if (!ok) break;
            const int row = (st.first + (KEYS ? f % st.per_head : f)) * kStream;
            const int y_head = KEYS ? h * share + f / st.per_head : h / share;
            const int y_row = (KEYS ? w.q0 : w.k0) + row;
            const int valid = min(y_len - row, kStream);
            uint8_t *dst = ring + slot * 2 * kOne;
            const bool clean = valid < kStream;             // the sequence's last tile: zeros behind it
            uint64_t *bar = clean ? &B.tail : &B.full[slot];
            if (KEYS) {
                const float *src = P.lse2 + (int64_t)y_head * P.Nq + y_row;
                const float *srd = P.delta + (int64_t)y_head * P.Nq + y_row;
#pragma unroll
                for (int e = lane; e < kStream; e += 32) {
                    const bool in = e < valid;
                    cp_async4(smem_addr(&B.stat[slot][0][e]), in ? src + e : src, in);
                    cp_async4(smem_addr(&B.stat[slot][1][e]), in ? srd + e : srd, in);
                }
                cp_async_arrive(smem_addr(&B.full[slot]));
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(smem_addr(bar), 2 * kOne);
                for (int t = 0; t < 2; ++t)
                    for (int c = 0; c < kC; ++c)
                        tma_load_3d(smem_addr(dst + t * kOne + c * kStreamChunk), t ? &my1 : &my0, smem_addr(bar), 64 * c,
                                    y_head, y_row);
            }
            __syncwarp();
            if (clean) {
                ok = warp_wait(&B.tail, tails & 1, abort);
                if (!ok) {
                    int never = 0;
                    mbar_wait(smem_addr(&B.tail), tails & 1, &never);
                    break;
                }
                ++tails;
                for (int t = 0; t < 2; ++t) zero_rows<kC, kStreamChunk>(dst + t * kOne, valid, (valid + 15) & ~15);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&B.full[slot]));
            }
        }
        if (!ok) {   // a wait gave up: the copies in flight still land before the block ends
            int never = 0;
            mbar_wait(smem_addr(&B.xfull), 0, &never);
            for (int s = max(f - kBwdStages, 0); s < f; ++s)
                mbar_wait(smem_addr(&B.full[s % kBwdStages]), (s / kBwdStages) & 1, &never);
        }
    } else if (warp == 9 && lane == 0 && st.n > 0) {
        // ---- MMAs
        constexpr uint32_t kIdS = idesc_bf16_f32(kTile, kStream), kIdA = idesc_b_mn(kTile, DP);
        const int ksteps = (P.D + 15) / 16;
        const uint32_t a0 = smem_addr(kept), r0 = smem_addr(ring);
        auto issue_s = [&](int j) {
            const uint32_t y = r0 + j % kBwdStages * 2 * kOne, d = B.tmem + (j & 1) * 128;
            for (int k = 0; k < ksteps; ++k)
                mma_ss(d, desc_k<kChunkBytes>(a0, k), desc_k<kStreamChunk>(y, k), kIdS, k > 0);
            for (int k = 0; k < ksteps; ++k)
                mma_ss(d + 64, desc_k<kChunkBytes>(a0 + kKept, k), desc_k<kStreamChunk>(y + kOne, k), kIdS, k > 0);
            mma_commit(&B.s_full[j & 1]);
        };
        auto wait_full = [&](int f) {
            return mbar_wait(smem_addr(&B.full[f % kBwdStages]), (f / kBwdStages) & 1, abort);
        };
        bool ok = mbar_wait(smem_addr(&B.xfull), 0, abort);
        for (int j = 0; j < 2 && j < st.n && ok; ++j) {
            ok = wait_full(j);
            tc_fence_after();
            if (ok) issue_s(j);
        }
        for (int j = 0; j < st.n && ok; ++j) {
            const int b = j & 1, row = (st.first + (KEYS ? j % st.per_head : j)) * kStream;
            const int steps = (min(y_len - row, kStream) + 15) / 16;
            const uint32_t y = r0 + j % kBwdStages * 2 * kOne, d = B.tmem + b * 128;
            ok = mbar_wait(smem_addr(&B.d_full[b]), (j >> 1) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            if (KEYS)
                for (int k = 0; k < steps; ++k)
                    mma_ts(B.tmem + 256, d + 8 * k, desc_mn<kStreamChunk>(y + kOne, k), kIdA, j > 0 || k > 0);
            for (int k = 0; k < steps; ++k)
                mma_ts(B.tmem + 384, d + 64 + 8 * k, desc_mn<kStreamChunk>(y, k), kIdA, j > 0 || k > 0);
            mma_commit(&B.empty[j % kBwdStages]);
            if (j + 1 == st.n) mma_commit(&B.acc_full);
            if (j + 2 < st.n) {
                ok = wait_full(j + 2);
                tc_fence_after();
                if (ok) issue_s(j + 2);
            }
        }
        if (!ok) {   // MMAs in flight finish before their tensor memory is freed
            int never = 0;
            mma_commit(&B.drain);
            mbar_wait(smem_addr(&B.drain), 0, &never);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && B.abort) atomicExch(P.err, (int)PE_ERR_DEVICE_TIMEOUT);
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(B.tmem, 512);
    }
}

}  // namespace pe
