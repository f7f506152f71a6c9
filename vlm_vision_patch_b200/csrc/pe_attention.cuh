// Attention over packed sequences, forward and backward (include/pe.h has the
// formulas).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "pe_device.cuh"

namespace pe {

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

// One warp per query row and head, one pass over its keys with a running
// maximum and sum.
__global__ void pe_attn_fwd_simple(const AttnParams P) {
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
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    lane_load(P.q.at(r, h), P.D, lane, q);
    for (int j = 0; j < limit; ++j) {
        float k[4], v[4];
        lane_load(P.k.at(k0 + j, hk), P.D, lane, k);
        lane_load(P.v.at(k0 + j, hk), P.D, lane, v);
        const float x = warp_sum(dot4(q, k)) * P.scale;
        const float mn = fmaxf(m, x), f = __expf(m - mn), p = __expf(x - mn);
        l = l * f + p;
        m = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * f + p * v[e];
    }
    lane_store(P.out.at(r, h), P.D, lane, o, limit ? 1.0f / l : 0.f);
    if (P.lse && lane == 0) P.lse[(int64_t)h * P.Nq + r] = limit ? m + logf(l) : -INFINITY;
}

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
