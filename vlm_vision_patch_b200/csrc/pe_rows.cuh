// Row-wise kernels of the vision tower: patch positions from grids, rotary
// positions, and layer norm with its gradient.  All are bound by HBM (or, on one
// image, by launch latency): each reads its rows once, with 16-byte accesses where
// sizes and strides allow (rotary positions take narrower ones elsewhere), and writes
// once.  Rows stay in registers in between, those of the layer norm's gradient in
// shared memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "pe_device.cuh"
#include "pe_packed.cuh"

namespace pe {

// ------------------------------------------------------------- positions

constexpr int kGridItems = 64;   // items per launch, carried in the launch parameters

struct GridItem {
    int row0, frame0, h, w;      // first row and frame of the item, frame size in patches
};
struct GridChunk {
    GridItem item[kGridItems];
    int n, row_end, frame_end;   // items; rows and frames before the chunk's end
    int last;                    // the last chunk also writes cu[F] = N
};

// Largest i with item[i].row0 <= r (items hold at least one row and frame each).
template <class Key>
__device__ __forceinline__ int find_item(const GridChunk &c, int r, Key key) {
    int lo = 0, hi = c.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (key(c.item[mid]) <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One thread per row (and per frame boundary).  Row r of a frame: window r / m^2,
// place r % m^2 inside it, both row-major.
__global__ void pe_positions_kernel(const __grid_constant__ GridChunk c, int m, int64_t N, int32_t *pos, int32_t *cu) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c.n == 0) {
        if (i == 0 && cu) cu[0] = 0;
        return;
    }
    const int64_t r = c.item[0].row0 + i;
    if (pos && r < c.row_end) {
        const GridItem g = c.item[find_item(c, (int)r, [](const GridItem &t) { return t.row0; })];
        const unsigned area = (unsigned)g.h * (unsigned)g.w, in_item = (unsigned)((int)r - g.row0);
        const unsigned f = in_item / area, in_frame = in_item - f * area;
        const unsigned m2 = (unsigned)(m * m), win = in_frame / m2, at = in_frame - win * m2;
        const unsigned across = (unsigned)(g.w / m), wr = win / across, wc = win - wr * across;
        const unsigned ar = at / (unsigned)m, ac = at - ar * (unsigned)m;
        pos[r] = (int32_t)f;
        pos[N + r] = (int32_t)(wr * (unsigned)m + ar);
        pos[2 * N + r] = (int32_t)(wc * (unsigned)m + ac);
    }
    const int64_t f = c.item[0].frame0 + i;
    if (cu && f < c.frame_end) {
        const GridItem g = c.item[find_item(c, (int)f, [](const GridItem &t) { return t.frame0; })];
        cu[f] = g.row0 + ((int)f - g.frame0) * (g.h * g.w);
    }
    if (cu && c.last && i == 0) cu[c.frame_end] = (int32_t)N;
}

// ------------------------------------------------------------- elements

// 8 consecutive elements as fp32.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo_to_f32(w[i]), v[2 * i + 1] = bf16hi_to_f32(w[i]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// 8 elements of a weight of either type, or `fill` without one.
__device__ __forceinline__ void load8_weight(const void *w, bool f32, int64_t e, float fill, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fill;
    } else if (f32) {
        load8(static_cast<const float *>(w) + e, v);
    } else {
        load8(static_cast<const __nv_bfloat16 *>(w) + e, v);
    }
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ------------------------------------------------------------- rotary positions

struct RopeSide {
    const void *in;
    void *out;
    int64_t in_row, in_head, out_row, out_head;   // strides in elements
    int heads;
};
struct RopeParams {
    RopeSide s[2];               // q, k
    const int32_t *pos;          // [axes, N]
    int64_t N;
    int pairs, tail;             // S, D - 2 S
    float sign;
    uint8_t axis[128];           // of pair i
    double turns[128];           // rate of pair i in turns: rate / (2 pi)
};

// VEC elements as one access, and as fp32.
template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        if constexpr (sizeof(T) == 2 && VEC > 1) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) f[2 * i] = bf16lo_to_f32(w[i]), f[2 * i + 1] = bf16hi_to_f32(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = to_f32(v[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        if constexpr (sizeof(T) == 2 && VEC > 1) {
            uint32_t *w = reinterpret_cast<uint32_t *>(v);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(f[i]);
        }
    }
};

constexpr int kRopeRows = 8;     // rows, and warps, of a block

// A warp turns a row.  Its cosines and sines are computed once for all heads of q
// and k: the angle in turns is a 64-bit product reduced to [-1/2, 1/2] exactly, so
// a position of a million costs no accuracy, and 64 bits are spent on S values a
// row, not on every element.  A lane keeps VEC of them in registers and takes the
// same VEC pairs of one head after the other, the lanes as many heads side by side
// as fit; two or four heads' loads are on their way ahead of the arithmetic, the
// first while the cosines are computed.
template <class T, int VEC>
__global__ void __launch_bounds__(32 * kRopeRows, 4) pe_rope_kernel(const __grid_constant__ RopeParams P) {
    extern __shared__ float2 all[];                      // [kRopeRows][pairs] (cos, sin)
    using V = Pack<T, VEC>;
    const int S = P.pairs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * kRopeRows + warp;
    if (row >= P.N) return;
    const int sv = S / VEC, per_head = sv + P.tail / VEC, across = per_head < 32 ? per_head : 32;
    const int step = 32 / across, h0 = lane / across, heads0 = P.s[0].heads, heads = heads0 + P.s[1].heads;
    const T *in0 = static_cast<const T *>(P.s[0].in) + row * P.s[0].in_row;
    const T *in1 = static_cast<const T *>(P.s[1].in) + row * P.s[1].in_row - heads0 * P.s[1].in_head;
    T *out0 = static_cast<T *>(P.s[0].out) + row * P.s[0].out_row;
    T *out1 = static_cast<T *>(P.s[1].out) + row * P.s[1].out_row - heads0 * P.s[1].out_head;
    auto source = [&](int h) { return h < heads0 ? in0 + h * P.s[0].in_head : in1 + h * P.s[1].in_head; };
    auto target = [&](int h) { return h < heads0 ? out0 + h * P.s[0].out_head : out1 + h * P.s[1].out_head; };
    constexpr int kAhead = sizeof(T) * VEC >= 16 ? 2 : 4;    // heads on their way
    V a[kAhead], b[kAhead];
    auto fetch = [&](V &x, V &y, int h, int v) {
        if (h >= heads || h0 >= step) return;
        const T *p = source(h) + (v < sv ? v * VEC : S + v * VEC);           // the tail begins at 2 S
        x = *reinterpret_cast<const V *>(p);
        if (v < sv) y = *reinterpret_cast<const V *>(p + S);
    };
    int v = lane - h0 * across;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(a[u], b[u], h0 + u * step, v);
    float2 *cs = all + warp * S;
    for (int p = lane; p < S; p += 32) {
        const double t = (double)P.pos[(int64_t)P.axis[p] * P.N + row] * P.turns[p];
        const float u = (float)(t - rint(t));
        float s, c;
        sincospif(2.0f * u, &s, &c);
        cs[p] = make_float2(c, P.sign * s);
    }
    __syncwarp();
    if (h0 >= step) return;
    for (; v < per_head; v += across) {
        const bool turn = v < sv;
        float2 t[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) t[e] = turn ? cs[v * VEC + e] : make_float2(1.f, 0.f);
        for (int h = h0; h < heads; h += kAhead * step) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (h + u * step >= heads) break;
                T *o = target(h + u * step) + (turn ? v * VEC : S + v * VEC);
                V x = a[u], y;
                if (turn) {
                    float f[VEC], g[VEC];
                    a[u].get(f);
                    b[u].get(g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        // the roundings are written out, so that every VEC gives the same bits
                        const float p = __fmaf_rn(f[e], t[e].x, -__fmul_rn(g[e], t[e].y));
                        g[e] = __fmaf_rn(g[e], t[e].x, __fmul_rn(f[e], t[e].y));
                        f[e] = p;
                    }
                    x.set(f);
                    y.set(g);
                    *reinterpret_cast<V *>(o + S) = y;
                }
                *reinterpret_cast<V *>(o) = x;
                fetch(a[u], b[u], h + (kAhead + u) * step, v);
            }
        }
        if (v + across < per_head) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(a[u], b[u], h0 + u * step, v + across);
        }
    }
}

// ------------------------------------------------------------- layer norm
//
// TPR threads share one row.  Forward, VPT groups of 8 elements per thread stay in
// registers: x is read once and the variance is taken from the deviations.
// Backward, the sums of the weight's gradients stay in registers, so the rows pass
// through shared memory: each thread copies its own 16-byte chunks there, rows
// ahead of the one it works on, and reads only what it copied itself (no barrier).

// Sum of v over the TPR threads of a row (all of them get it); blocks hold
// blockDim / TPR rows.  `red`: TPR / 32 floats per row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        __syncthreads();                                  // the last sum has been read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int base = threadIdx.x / TPR * (TPR / 32);
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += red[base + i];
    }
    return v;
}

// 16 bytes from global to shared memory, past L1 and without waiting.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's groups of copies are on their way.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A chunk of 16 bytes as fp32 pairs: 8 bf16 or 4 fp32.
template <class T>
constexpr int kPairs = 8 / (int)sizeof(T);

template <class T>
__device__ __forceinline__ void take_chunk(const uint8_t *p, float2 (&v)[kPairs<T>]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    if constexpr (sizeof(T) == 4) {
        v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    } else {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
    }
}
template <class T>
__device__ __forceinline__ void put_chunk(T *p, const float2 (&v)[kPairs<T>]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                   pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
    }
}

struct NormParams {
    const void *x, *dy, *gamma, *beta;
    void *y;                      // forward: y; backward: dx
    float *mean, *rstd;
    float *part;                  // backward: [gridDim][2][E] partial sums, or NULL
    int64_t N;
    int E, w_f32;
    float eps;
};

template <int TPR>
constexpr int kNormThreads = TPR > 128 ? TPR : 128;

template <class T, int TPR, int VPT>
__global__ void __launch_bounds__(kNormThreads<TPR>) pe_norm_fwd_kernel(const NormParams P) {
    __shared__ float red[kNormThreads<TPR> / 32];
    constexpr int kRows = kNormThreads<TPR> / TPR;
    const int t = threadIdx.x % TPR, nv = P.E / 8;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < P.N;                          // rows of several warps meet at barriers
    if (TPR == 32 && !live) return;
    const T *x = static_cast<const T *>(P.x) + row * P.E;
    float v[VPT][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (live && t + i * TPR < nv) {
            load8(x + 8 * (t + i * TPR), v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[i][e];
        }
    }
    const float mean = row_sum<TPR>(s, red) / (float)P.E;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (live && t + i * TPR < nv)
#pragma unroll
            for (int e = 0; e < 8; ++e) q += (v[i][e] - mean) * (v[i][e] - mean);
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red) / (float)P.E + P.eps);
    T *y = static_cast<T *>(P.y) + row * P.E;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (live && t + i * TPR < nv) {
            const int e0 = 8 * (t + i * TPR);
            float g[8], b[8];
            load8_weight(P.gamma, P.w_f32, e0, 1.f, g);
            load8_weight(P.beta, P.w_f32, e0, 0.f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = (v[i][e] - mean) * rstd * g[e] + b[e];
            store8(y + e0, v[i]);
        }
    }
    if (P.mean && live && t == 0) {
        P.mean[row] = mean;
        P.rstd[row] = rstd;
    }
}

template <int TPR, int CPT>
struct NormBwd {
    static constexpr int kThreads = kNormThreads<TPR>, kRows = kThreads / TPR;
    static constexpr int kTensor = CPT * kThreads * 16;                   // bytes of one tensor's rows
    static constexpr int kStages = 3 * 2 * kTensor <= 200 * 1024 ? 3 : 1; // rows on their way
    static constexpr int kSmem = kStages * 2 * kTensor;
    static constexpr int kResident = TPR <= 128 ? 3 : (TPR == 256 && CPT <= 4 ? 2 : 1);   // blocks of a SM
    static_assert(kResident * (kSmem + 1280) <= 228 * 1024, "shared memory");
};

// Each block takes rows blockIdx, blockIdx + gridDim, ... (in groups of its rows
// at once), writes dx, and keeps the sums over its rows of dy * xh and dy for
// its features in registers; they go to part[blockIdx] once.  No atomics: the
// order of every sum is fixed by the sizes.
template <class T, int TPR, int CPT>
__global__ void __launch_bounds__(NormBwd<TPR, CPT>::kThreads, NormBwd<TPR, CPT>::kResident)
pe_norm_bwd_kernel(const NormParams P) {
    using S = NormBwd<TPR, CPT>;
    constexpr int kRows = S::kRows, kStep = S::kThreads * 16, kP = kPairs<T>;
    extern __shared__ __align__(16) uint8_t ring[];       // [stage][x, dy][chunk][thread] of 16 bytes
    __shared__ float red[S::kThreads / 32];
    const int t = threadIdx.x % TPR, lane_row = threadIdx.x / TPR, chunks = P.E / (2 * kP);
    const float inv_e = 1.0f / (float)P.E;
    if (P.part) griddep_launch_dependents();              // the summing kernel
    float2 dg[CPT][kP], db[CPT][kP], gm[CPT][kP];
    // gamma stays in registers: every row passing by would push it out of L1
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int e = 0; e < kP; ++e) {
            dg[i][e] = db[i][e] = both(0.f);
            const int64_t at = 2 * (kP * (int64_t)(t + i * TPR) + e);
            gm[i][e] = both(1.f);
            if (P.gamma && t + i * TPR < chunks)
                gm[i][e] = P.w_f32 ? *reinterpret_cast<const float2 *>(static_cast<const float *>(P.gamma) + at)
                                   : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(
                                         static_cast<const __nv_bfloat16 *>(P.gamma) + at));
        }
    uint8_t *mine = ring + threadIdx.x * 16;
    const uint32_t mine_s = smem_addr(mine);
    auto fetch = [&](int64_t row, int stage) {
        if (row < P.N) {
            const T *px = static_cast<const T *>(P.x) + row * P.E, *py = static_cast<const T *>(P.dy) + row * P.E;
#pragma unroll
            for (int i = 0; i < CPT; ++i)
                if (t + i * TPR < chunks) {
                    const uint32_t dst = mine_s + stage * 2 * S::kTensor + i * kStep;
                    copy16(dst, px + 2 * kP * (t + i * TPR));
                    copy16(dst + S::kTensor, py + 2 * kP * (t + i * TPR));
                }
        }
        copy_commit();
    };
    const int64_t step = (int64_t)gridDim.x * kRows, first = (int64_t)blockIdx.x * kRows + lane_row;
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) fetch(first + s * step, s);
    int stage = 0;
    float mean_n = first < P.N ? P.mean[first] : 0.f, rstd_n = first < P.N ? P.rstd[first] : 0.f;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < P.N; r0 += step) {
        const int64_t row = r0 + lane_row;
        const bool live = row < P.N;
        const float mean = mean_n, rstd = rstd_n;
        if (row + step < P.N) {
            mean_n = P.mean[row + step];
            rstd_n = P.rstd[row + step];
        }
        fetch(row + (S::kStages - 1) * step, stage == 0 ? S::kStages - 1 : stage - 1);
        copy_wait<S::kStages - 1>();
        const uint8_t *xs = mine + stage * 2 * S::kTensor, *ys = xs + S::kTensor;
        const float2 off = both(-mean), scale = both(rstd);
        float2 p1 = both(0.f), p2 = both(0.f);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            if (live && t + i * TPR < chunks) {
                float2 x[kP], a[kP];
                take_chunk<T>(xs + i * kStep, x);
                take_chunk<T>(ys + i * kStep, a);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    const float2 xh = mul2(add2(x[e], off), scale);
                    dg[i][e] = fma2(a[e], xh, dg[i][e]);
                    db[i][e] = add2(db[i][e], a[e]);
                    a[e] = mul2(a[e], gm[i][e]);
                    p1 = add2(p1, a[e]);
                    p2 = fma2(a[e], xh, p2);
                }
            }
        }
        const float s1 = row_sum<TPR>(p1.x + p1.y, red) * inv_e;
        const float s2 = row_sum<TPR>(p2.x + p2.y, red) * inv_e;
        T *dx = static_cast<T *>(P.y) + row * P.E;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            if (live && t + i * TPR < chunks) {
                float2 x[kP], a[kP];
                take_chunk<T>(xs + i * kStep, x);
                take_chunk<T>(ys + i * kStep, a);
#pragma unroll
                for (int e = 0; e < kP; ++e) {
                    const float2 xh = mul2(add2(x[e], off), scale);
                    a[e] = mul2(scale, fma2(xh, both(-s2), fma2(a[e], gm[i][e], both(-s1))));
                }
                put_chunk<T>(dx + 2 * kP * (t + i * TPR), a);
            }
        }
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    if (!P.part) return;
    // the sums of the block's other rows go through shared memory, added in order
    float2 *sums = reinterpret_cast<float2 *>(ring), *out = reinterpret_cast<float2 *>(P.part + (int64_t)blockIdx.x * 2 * P.E);
    const int half = P.E / 2;
    if constexpr (kRows > 1) {
        copy_wait<0>();
        for (int r = 1; r < kRows; ++r) {
            __syncthreads();                              // the ring, or the last row's sums, are done with
            if (lane_row == r) {
#pragma unroll
                for (int i = 0; i < CPT; ++i)
                    if (t + i * TPR < chunks)
#pragma unroll
                        for (int e = 0; e < kP; ++e) {
                            sums[kP * (t + i * TPR) + e] = dg[i][e];
                            sums[half + kP * (t + i * TPR) + e] = db[i][e];
                        }
            }
            __syncthreads();
            if (lane_row == 0) {
#pragma unroll
                for (int i = 0; i < CPT; ++i)
                    if (t + i * TPR < chunks)
#pragma unroll
                        for (int e = 0; e < kP; ++e) {
                            dg[i][e] = add2(dg[i][e], sums[kP * (t + i * TPR) + e]);
                            db[i][e] = add2(db[i][e], sums[half + kP * (t + i * TPR) + e]);
                        }
            }
        }
        if (lane_row > 0) return;
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i)
        if (t + i * TPR < chunks)
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                out[kP * (t + i * TPR) + e] = dg[i][e];
                out[half + kP * (t + i * TPR) + e] = db[i][e];
            }
}

// dgamma and dbeta from `n` partial rows of 2 E: a block sums 32 columns, its 32
// warps every 32nd row each (four loads in flight), then the 32 sums in order.
__global__ void __launch_bounds__(1024) pe_norm_sum_kernel(const float *part, int n, int E, int w_f32, void *dgamma,
                                                           void *dbeta) {
    griddep_wait();                                       // for the kernel that wrote `part`
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < 2 * E)
        for (int r = w; r < n; r += 128)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + 32 * u < n) a[u] += part[(int64_t)(r + 32 * u) * 2 * E + col];
    s[w][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (w != 0 || col >= 2 * E) return;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][lane];
    void *dst = col < E ? dgamma : dbeta;
    const int e = col < E ? col : col - E;
    if (w_f32) static_cast<float *>(dst)[e] = v;
    else static_cast<__nv_bfloat16 *>(dst)[e] = __float2bfloat16_rn(v);
}

}  // namespace pe
