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
    float *delta;                 // [Hq, Nq]
    int *err;
};

// Boundary s of a cumulative-length array, held inside [0, n] whatever it says.
__device__ __forceinline__ int boundary(const int32_t *cu, int s, int n) {
    const int v = cu[s];
    return v < 0 ? 0 : (v > n ? n : v);
}

// The last sequence that begins at or before row r, or -1.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n_seq, int r) {
    int lo = -1, hi = n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Four elements of a head per lane (D <= 128, a multiple of 8).
__device__ __forceinline__ void lane_load(const __nv_bfloat16 *p, int D, int lane, float (&v)[4]) {
    uint2 w = make_uint2(0, 0);
    if (4 * lane < D) w = *reinterpret_cast<const uint2 *>(p + 4 * lane);
    v[0] = bf16lo_to_f32(w.x), v[1] = bf16hi_to_f32(w.x), v[2] = bf16lo_to_f32(w.y), v[3] = bf16hi_to_f32(w.y);
}
__device__ __forceinline__ void lane_store(__nv_bfloat16 *p, int D, int lane, const float (&v)[4], float f) {
    if (4 * lane < D)
        *reinterpret_cast<uint2 *>(p + 4 * lane) = make_uint2(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f));
}
__device__ __forceinline__ float dot4(const float (&a)[4], const float (&b)[4]) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
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
template <int CHUNKS>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int valid, int end) {
    const int groups = (end - valid) * 8;
    for (int c = 0; c < CHUNKS; ++c)
        for (int i = threadIdx.x & 31; i < groups; i += 32)
            *reinterpret_cast<uint4 *>(tile + c * kChunkBytes + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// K-major operand (rows x 64-column chunks), k-step of 16 columns.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kstep) {
    return smem_desc(tile + (kstep >> 2) * kChunkBytes + (kstep & 3) * 32, 16, 1024, kLayoutSw128);
}
// The same tile read along its rows (MN-major): k-step of 16 rows, N = the columns.
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kstep) {
    return smem_desc(tile + kstep * 2048, kChunkBytes, 1024, kLayoutSw128);
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
                zero_rows<kC>(dst, valid, (valid + 15) & ~15);
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
                mma_ss(B.tmem + t * 128, desc_k(a_q + t * kTileBytes, k), desc_k(a_r + f % kFwdStages * kTileBytes, k), kIdS,
                       k > 0);
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
                               desc_mn(a_r + fv % kFwdStages * kTileBytes, k), kIdO, j > 0 || k > 0);
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

// delta and dq: one warp per query row and head.
__global__ void pe_attn_dq_simple(const AttnParams P) {
    const int lane = threadIdx.x & 31, r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), h = blockIdx.y;
    if (r >= P.Nq) return;
    const int s = sequence_of(P.cu_q, P.n_seq, r);
    if (s < 0) return;
    const int q0 = boundary(P.cu_q, s, P.Nq), q1 = boundary(P.cu_q, s + 1, P.Nq);
    const int k0 = boundary(P.cu_k, s, P.Nk), k1 = boundary(P.cu_k, s + 1, P.Nk);
    if (r >= q1) return;
    const int lk = k1 > k0 ? k1 - k0 : 0;
    int limit = lk;
    if (P.causal) limit = min(lk, max(0, r - q0 + 1 + lk - (q1 - q0)));
    const int hk = h / (P.Hq / P.Hkv);
    float q[4], o[4], g[4], dq[4] = {0.f, 0.f, 0.f, 0.f};
    lane_load(P.q.at(r, h), P.D, lane, q);
    lane_load(P.out.at(r, h), P.D, lane, o);
    lane_load(P.dout.at(r, h), P.D, lane, g);
    const float delta = warp_sum(dot4(g, o)), lse = P.lse[(int64_t)h * P.Nq + r];
    if (lane == 0) P.delta[(int64_t)h * P.Nq + r] = delta;
    for (int j = 0; j < limit; ++j) {
        float k[4], v[4];
        lane_load(P.k.at(k0 + j, hk), P.D, lane, k);
        lane_load(P.v.at(k0 + j, hk), P.D, lane, v);
        const float p = __expf(warp_sum(dot4(q, k)) * P.scale - lse), ds = p * (warp_sum(dot4(g, v)) - delta);
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[e] += ds * k[e];
    }
    lane_store(P.dq.at(r, h), P.D, lane, dq, P.scale);
}

// dk and dv: one warp per key row and key head, over the rows that see it and
// the query heads that share it.
__global__ void pe_attn_dkv_simple(const AttnParams P) {
    const int lane = threadIdx.x & 31, r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), hk = blockIdx.y;
    if (r >= P.Nk) return;
    const int s = sequence_of(P.cu_k, P.n_seq, r);
    if (s < 0) return;
    const int q0 = boundary(P.cu_q, s, P.Nq), q1 = boundary(P.cu_q, s + 1, P.Nq);
    const int k0 = boundary(P.cu_k, s, P.Nk), k1 = boundary(P.cu_k, s + 1, P.Nk);
    if (r >= k1) return;
    int first = 0;
    if (P.causal) first = max(0, r - k0 - ((k1 - k0) - (q1 - q0)));
    float k[4], v[4], dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
    lane_load(P.k.at(r, hk), P.D, lane, k);
    lane_load(P.v.at(r, hk), P.D, lane, v);
    const int share = P.Hq / P.Hkv;
    for (int h = hk * share; h < (hk + 1) * share; ++h)
        for (int i = q0 + first; i < q1; ++i) {
            float q[4], g[4];
            lane_load(P.q.at(i, h), P.D, lane, q);
            lane_load(P.dout.at(i, h), P.D, lane, g);
            const float p = __expf(warp_sum(dot4(q, k)) * P.scale - P.lse[(int64_t)h * P.Nq + i]);
            const float ds = p * (warp_sum(dot4(g, v)) - P.delta[(int64_t)h * P.Nq + i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dv[e] += p * g[e];
                dk[e] += ds * q[e];
            }
        }
    lane_store(P.dk.at(r, hk), P.D, lane, dk, P.scale);
    lane_store(P.dv.at(r, hk), P.D, lane, dv, 1.0f);
}

}  // namespace pe
