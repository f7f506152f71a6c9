// C ABI of the vision-tower operators (see include/pe.h for the contract of
// every entry point): rotary positions, layer norm and attention.  Host side:
// argument validation, variant choice and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>
#include <type_traits>

#include "../../include/pe.h"
#include "pe_attention.cuh"
#include "pe_host_util.h"
#include "pe_rows.cuh"

using namespace pe;

struct pe_attention {
    int dev = -1;
    int Hq = 0, Hkv = 0, D = 0, causal = 0;
    float scale = 0.f;
    int num_sms = 0;
    int *err = nullptr;          // dev error word
};

namespace {

bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t size_of(pe_dtype dt) { return dt == PE_F32 ? 4 : 2; }

// Streaming multiprocessors of the current device (asked for once per device).
int current_sms() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// A kernel that waits (griddepcontrol) for the one before it on the stream: its
// blocks may start, and its set-up run, as that one's last blocks end.
template <class... K, class... A>
cudaError_t launch_after(void (*kern)(K...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Whether the heads of a tensor that is written do not overlap.
bool disjoint(const pe_heads &t, int64_t rows, int heads, int D) {
    const int64_t row = rows > 1 ? t.row_stride : INT64_MAX, head = heads > 1 ? t.head_stride : INT64_MAX;
    const int64_t inner = std::min(row, head), count = row < head ? rows : heads;
    if (inner == INT64_MAX) return true;                   // one row of one head
    if (inner < D) return false;
    const int64_t outer = std::max(row, head);
    return outer == INT64_MAX || (outer - D) / inner >= count - 1;
}

// ------------------------------------------------------------- rotary positions

// The widest access (at most 16 bytes) that divides the head's halves and tail,
// every stride in use and every base address.
int rope_vec(const RopeParams &P, size_t es) {
    int vec = (int)(16 / es);
    auto fits = [&](int v) {
        if (P.pairs % v || P.tail % v) return false;
        for (const RopeSide &s : P.s) {
            if (s.heads == 0) continue;
            if (!aligned_to(s.in, es * v) || !aligned_to(s.out, es * v)) return false;
            if (P.N > 1 && (s.in_row % v || s.out_row % v)) return false;
            if (s.heads > 1 && (s.in_head % v || s.out_head % v)) return false;
        }
        return true;
    };
    while (vec > 1 && !fits(vec)) vec /= 2;
    return vec;
}

template <class T, int VEC>
cudaError_t launch_rope(const RopeParams &P, cudaStream_t st) {
    const int64_t blocks = (P.N + kRopeRows - 1) / kRopeRows;
    pe_rope_kernel<T, VEC><<<(unsigned)blocks, 32 * kRopeRows, (size_t)kRopeRows * P.pairs * sizeof(float2), st>>>(P);
    return cudaGetLastError();
}

// ------------------------------------------------------------- layer norm

// Forward: a warp a row up to 1280 features, then 128 and 256 threads (8192 fp32
// features: 2.5 TB/s with 1024 threads, 5.8 with 256 fuller ones).
int norm_fwd_tpr(int E) { return E <= 1280 ? 32 : (E <= 4096 ? 128 : 256); }

int norm_rows(int tpr) { return tpr > 128 ? 1 : 128 / tpr; }          // rows per block

// Backward: as few threads as hold the row in 5 chunks of 16 bytes each (4 beyond
// 256 threads), so that the sums fit their registers.
struct NormBwdPlan {
    int tpr, cpt;
    int blocks;                  // as many as are resident: each writes one partial row of 2 E sums
};

NormBwdPlan plan_norm_bwd(int64_t N, int E, bool f32, int sms) {
    const int chunks = E * (f32 ? 4 : 2) / 16;
    NormBwdPlan p = {32, 0, 0};
    while (chunks > p.tpr * (p.tpr <= 256 ? 5 : 4)) p.tpr *= 2;
    p.cpt = (chunks + p.tpr - 1) / p.tpr;
    const int resident = p.tpr <= 128 ? 3 : (p.tpr == 256 && p.cpt <= 4 ? 2 : 1);
    p.blocks = (int)std::min<int64_t>((N + norm_rows(p.tpr) - 1) / norm_rows(p.tpr), (int64_t)sms * resident);
    return p;
}

template <class T, bool BACKWARD, int TPR, int PER>
cudaError_t launch_norm(const NormParams &P, int blocks, cudaStream_t st) {
    if constexpr (!BACKWARD) {
        pe_norm_fwd_kernel<T, TPR, PER><<<(unsigned)blocks, kNormThreads<TPR>, 0, st>>>(P);
    } else {
        using S = NormBwd<TPR, PER>;
        auto kern = pe_norm_bwd_kernel<T, TPR, PER>;
        if (S::kSmem > 40 * 1024) {                       // 48 KB with the static part
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
            if (e != cudaSuccess) return e;
        }
        kern<<<(unsigned)blocks, S::kThreads, S::kSmem, st>>>(P);
    }
    return cudaGetLastError();
}

// The kernel of LO .. HI groups or chunks per thread.
template <class T, bool BACKWARD, int TPR, int LO, int HI>
cudaError_t pick_norm(const NormParams &P, int per, int blocks, cudaStream_t st) {
    if constexpr (LO < HI) {
        if (per > LO) return pick_norm<T, BACKWARD, TPR, LO + 1, HI>(P, per, blocks, st);
    }
    return launch_norm<T, BACKWARD, TPR, LO>(P, blocks, st);
}

template <class T>
cudaError_t norm_forward(const NormParams &P, cudaStream_t st) {
    const int tpr = norm_fwd_tpr(P.E), vpt = (P.E / 8 + tpr - 1) / tpr, rows = norm_rows(tpr);
    const int blocks = (int)((P.N + rows - 1) / rows);
    if (tpr == 32) return pick_norm<T, false, 32, 1, 5>(P, vpt, blocks, st);
    if (tpr == 128) return pick_norm<T, false, 128, 2, 4>(P, vpt, blocks, st);
    return pick_norm<T, false, 256, 3, 8>(P, vpt, blocks, st);
}

template <class T>
cudaError_t norm_backward(const NormParams &P, const NormBwdPlan &p, cudaStream_t st) {
    switch (p.tpr) {
        case 32: return pick_norm<T, true, 32, 1, 5>(P, p.cpt, p.blocks, st);
        case 64: return pick_norm<T, true, 64, 3, 5>(P, p.cpt, p.blocks, st);
        case 128: return pick_norm<T, true, 128, 3, 5>(P, p.cpt, p.blocks, st);
        case 256: return pick_norm<T, true, 256, 3, 5>(P, p.cpt, p.blocks, st);
        case 512: return pick_norm<T, true, 512, 3, 4>(P, p.cpt, p.blocks, st);
    }
    if constexpr (sizeof(T) == 4) return pick_norm<T, true, 1024, 3, 4>(P, p.cpt, p.blocks, st);
    return cudaErrorInvalidValue;                         // bf16 rows end at 512 threads
}

pe_status check_norm(pe_dtype dt, pe_dtype w_dt, int64_t N, int E) {
    if (N < 0 || E < 1) return PE_ERR_INVALID_ARG;
    if (!valid_dtype(dt) || !valid_dtype(w_dt)) return PE_ERR_DTYPE;
    if (E % 8 || E > PE_LAYERNORM_MAX_E || N > INT32_MAX) return PE_ERR_UNSUPPORTED;
    return PE_OK;
}

// ------------------------------------------------------------- attention

// One [rows, heads, D] tensor: present, aligned, with strides a tensor map takes.
pe_status check_heads(const pe_heads &t, int64_t rows, int heads, int D) {
    if (!t.ptr) return PE_ERR_INVALID_ARG;
    if (!aligned16(t.ptr)) return PE_ERR_ALIGN;
    for (int a = 0; a < 2; ++a) {
        const int64_t n = a ? heads : rows, st = a ? t.head_stride : t.row_stride;
        if (n <= 1) continue;
        if (st < D || st >= ((int64_t)1 << 39)) return PE_ERR_SHAPE;
        if (st % 8) return PE_ERR_ALIGN;
    }
    return PE_OK;
}

HeadsPtr heads_ptr(const pe_heads &t, int64_t rows, int heads) {
    return {static_cast<__nv_bfloat16 *>(t.ptr), rows > 1 ? t.row_stride : 0, heads > 1 ? t.head_stride : 0};
}

// [rows, heads, D] bf16 in boxes of `box_rows` rows, `box_heads` heads and 64 elements, 128-byte
// swizzle; what lies outside reads as zero.
bool make_heads_tmap(CUtensorMap *m, const pe_heads &t, int64_t rows, int heads, int D, uint32_t box_rows,
                     uint32_t box_heads = 1) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t row = rows > 1 ? t.row_stride : (int64_t)heads * D, head = heads > 1 ? t.head_stride : D;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
    cuuint32_t box[3] = {64, box_heads, box_rows}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Calls f(std::integral_constant<int, DP>) with the head size rounded up to one
// the kernels are compiled for.
template <class F>
auto with_head_size(int D, F &&f) {
    if (D <= 64) return f(std::integral_constant<int, 64>());
    if (D <= 80) return f(std::integral_constant<int, 80>());
    if (D <= 96) return f(std::integral_constant<int, 96>());
    return f(std::integral_constant<int, 128>());
}

// Prepares an attention kernel.  Where its warpgroups divide the registers anew
// (setmaxnreg), more than it was launched with would be waited for without end, so
// a build that gave it fewer than `regs` is refused.  Once per kernel and
// device (`done`: a bit each); a second thread that does it again does no harm.
template <class Kernel>
bool ready_to_launch(Kernel kern, size_t smem, int dev, std::atomic<uint64_t> &done, int regs = kLaunchRegs) {
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    cudaFuncAttributes at;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaFuncGetAttributes(&at, kern) != cudaSuccess || at.numRegs < regs)
        return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Tiles of `rows` rows that n rows in n_seq sequences are given (find_work).
unsigned max_tiles(int64_t n, int n_seq, int rows) { return (unsigned)(n / rows + n_seq); }

// Sizes that do not depend on the buffers.
pe_status check_attention(const pe_attention *a, int n_seq, int64_t Nq, int64_t Nk) {
    if (!a || n_seq < 0 || Nq < 0 || Nk < 0) return PE_ERR_INVALID_ARG;
    if (Nq > INT32_MAX - 256 || Nk > INT32_MAX - 256 || n_seq > (1 << 24)) return PE_ERR_UNSUPPORTED;
    return PE_OK;
}

// How a forward call lays its rows and keys out over blocks, from the sizes alone.
struct FwdPlan {
    int groups, tiles, pack, splits;   // groups of softmax warps and query tiles a block
    unsigned blocks, rows;       // blocks of one head and split; heads or, packed, key heads
};

FwdPlan plan_forward(const pe_attention *a, int n_seq, int64_t Nq, int64_t Nk) {
    const int share = a->Hq / a->Hkv;
    FwdPlan p;
    // an average sequence's rows of all heads that share a key head fit one tile
    p.pack = share > 1 && share <= kTile && Nq * share <= (int64_t)kTile * n_seq ? share : 1;
    p.rows = (unsigned)(p.pack > 1 ? a->Hkv : a->Hq);
    // at least so many blocks of two tiles; one tile a block ends sooner while SMs are idle
    const int rows = kTile / p.pack;
    auto at_least = [&](int r) { return std::max<int64_t>((Nq + r - 1) / r, std::min<int64_t>(n_seq, Nq)) * p.rows; };
    p.tiles = at_least(2 * rows) * 2 <= a->num_sms ? 1 : 2;
    // Short sequences: blocks of one tile, two a SM, hide each other's start and end (925
    // sequences of 64 rows, 16 heads of 80: 815 -> 375 us; 115 of 512: 400 -> 339; 16 of 1024:
    // 183 -> 170).  Longer ones would read their keys twice as often (16 of 2048, heads of
    // 64: 492 -> 516), and fewer blocks than SMs would have less in flight each.
    p.groups = Nq <= (int64_t)8 * rows * n_seq && at_least(rows) > a->num_sms ? 1 : 2;
    if (p.groups == 1) p.tiles = 1;
    const int64_t blocks = at_least(p.tiles * rows);
    p.blocks = max_tiles(Nq, n_seq, p.tiles * rows);
    // With blocks for less than a quarter of the SMs the key axis is divided until there
    // is one a SM, but into no less than 4 tiles of an average sequence.  (The quarter is a
    // choice on one side measured: 128 blocks of a prompt lose by a division, 23.9 to 26.6 us.
    // Just above it long keys would gain: 18 single tokens over 12000 keys each, 12 heads on
    // 2, are 36 blocks and take 49 us, 19 of them 130.)
    const int64_t tiles = Nk / n_seq / 128;
    p.splits = 1;
    if (blocks * 4 <= a->num_sms)
        p.splits = (int)std::max<int64_t>(1, std::min(a->num_sms / blocks, std::min<int64_t>(tiles / 4, 64)));
    return p;
}

// Parts of the heads that share a key head, a block each, of the key kernel: when
// its blocks are fewer than two a SM, as long ones (the first keys of a causal
// sequence) would be all that runs in the end.
int plan_key_parts(const pe_attention *a, int n_seq, int64_t Nq, int64_t Nk) {
    if (n_seq == 0 || Nq == 0 || Nk == 0) return 1;
    const int64_t blocks = std::max<int64_t>((Nk + kTile - 1) / kTile, std::min<int64_t>(n_seq, Nk)) * a->Hkv;
    const int64_t want = (2 * (int64_t)a->num_sms + blocks - 1) / blocks;
    return (int)std::min<int64_t>(a->Hq / a->Hkv, want);
}

}  // namespace

extern "C" {

pe_status pe_vision_positions(int n, const int32_t *grid, int merge, int32_t *pos, int32_t *cu, pe_stream_t stream) {
    NvtxRange nvtx("pe_vision_positions");
    if (n < 0 || (n > 0 && !grid) || merge < 1 || merge > 4) return PE_ERR_INVALID_ARG;
    if (!aligned_to(pos, 4) || !aligned_to(cu, 4)) return PE_ERR_ALIGN;
    int64_t N = 0, F = 0;
    for (int i = 0; i < n; ++i) {
        const int32_t *g = grid + 3 * (int64_t)i;
        if (g[0] < 1 || g[1] < 1 || g[2] < 1 || g[1] % merge || g[2] % merge) return PE_ERR_SHAPE;
        const int64_t area = (int64_t)g[1] * g[2];
        if (area > INT32_MAX || area * g[0] > INT32_MAX - N) return PE_ERR_UNSUPPORTED;
        N += area * g[0];
        F += g[0];
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (!pos && !cu) return PE_OK;
    int64_t row = 0, frame = 0;
    int i = 0;
    do {
        GridChunk c;
        std::memset(&c, 0, sizeof(c));
        const int64_t row0 = row, frame0 = frame;
        for (; c.n < kGridItems && i < n; ++i, ++c.n) {
            const int32_t *g = grid + 3 * (int64_t)i;
            c.item[c.n] = {(int)row, (int)frame, g[1], g[2]};
            row += (int64_t)g[0] * g[1] * g[2];
            frame += g[0];
        }
        c.row_end = (int)row;
        c.frame_end = (int)frame;
        c.last = i == n;
        const int64_t threads = std::max<int64_t>(pos ? row - row0 : frame - frame0, 1);
        pe_positions_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(c, merge, N, pos, cu);
        if (cudaGetLastError() != cudaSuccess) return PE_ERR_CUDA;
    } while (i < n);
    return PE_OK;
}

pe_status pe_rope(pe_heads q, pe_heads k, pe_dtype dt, int64_t N, int Hq, int Hk, int D, const int32_t *pos, int axes,
                  const int32_t *sections, double theta, int axial, int inverse, pe_heads q_out, pe_heads k_out,
                  pe_stream_t stream) {
    NvtxRange nvtx("pe_rope");
    if (N < 0 || Hq < 1 || Hk < 0 || D < 1 || axes < 1 || !sections || (axial != 0 && axial != 1) ||
        (inverse != 0 && inverse != 1) || !(theta > 0.0) || !std::isfinite(theta))
        return PE_ERR_INVALID_ARG;
    if (!valid_dtype(dt)) return PE_ERR_DTYPE;
    if (axes > PE_ROPE_MAX_AXES || D > 1024 || N > INT32_MAX) return PE_ERR_UNSUPPORTED;
    int64_t S = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return PE_ERR_INVALID_ARG;
        S += sections[a];
    }
    if (S < 1 || 2 * S > D) return PE_ERR_SHAPE;
    if (S > PE_ROPE_MAX_PAIRS || (int64_t)Hq + Hk > 65536) return PE_ERR_UNSUPPORTED;
    // a position (below 2^31) times the largest rate is finite
    const double log2_theta = std::log2(theta);
    for (int a = 0; a < axes; ++a) {
        const double n = axial ? (double)sections[a] : (double)S;
        if (n > 0 && -(n - 1) / n * log2_theta > 990) return PE_ERR_UNSUPPORTED;
    }
    if (N == 0) return PE_OK;
    if (!pos) return PE_ERR_INVALID_ARG;
    if (!aligned_to(pos, 4)) return PE_ERR_ALIGN;
    const size_t es = size_of(dt);
    RopeParams P;
    std::memset(&P, 0, sizeof(P));
    const pe_heads *in[2] = {&q, &k}, *out[2] = {&q_out, &k_out};
    for (int i = 0; i < 2; ++i) {
        const int heads = i ? Hk : Hq;
        if (heads == 0) continue;
        if (!in[i]->ptr || !out[i]->ptr) return PE_ERR_INVALID_ARG;
        if (!aligned_to(in[i]->ptr, es) || !aligned_to(out[i]->ptr, es)) return PE_ERR_ALIGN;
        if (in[i]->row_stride < 0 || in[i]->head_stride < 0 || out[i]->row_stride < 0 || out[i]->head_stride < 0)
            return PE_ERR_INVALID_ARG;
        if (!disjoint(*out[i], N, heads, D)) return PE_ERR_SHAPE;
        P.s[i] = {in[i]->ptr, out[i]->ptr, in[i]->row_stride, in[i]->head_stride, out[i]->row_stride,
                  out[i]->head_stride, heads};
    }
    P.pos = pos;
    P.N = N;
    P.pairs = (int)S;
    P.tail = (int)(D - 2 * S);
    P.sign = inverse ? -1.f : 1.f;
    const double two_pi = 6.283185307179586476925286766559;
    for (int a = 0, i = 0; a < axes; ++a)
        for (int j = 0; j < sections[a]; ++j, ++i) {
            P.axis[i] = (uint8_t)a;
            P.turns[i] = std::exp2(-(axial ? (double)j / sections[a] : (double)i / (double)S) * log2_theta) / two_pi;
        }
    cudaStream_t st = (cudaStream_t)stream;
    const int vec = rope_vec(P, es);
    if (dt == PE_F32) {
        if (vec == 4) return finish(launch_rope<float, 4>(P, st));
        return finish(vec == 2 ? launch_rope<float, 2>(P, st) : launch_rope<float, 1>(P, st));
    }
    using bf16 = __nv_bfloat16;
    if (vec == 8) return finish(launch_rope<bf16, 8>(P, st));
    if (vec == 4) return finish(launch_rope<bf16, 4>(P, st));
    return finish(vec == 2 ? launch_rope<bf16, 2>(P, st) : launch_rope<bf16, 1>(P, st));
}

pe_status pe_layernorm_forward(const void *x, pe_dtype dt, int64_t N, int E, const void *gamma, const void *beta,
                               pe_dtype w_dt, float eps, void *y, float *mean, float *rstd, pe_stream_t stream) {
    NvtxRange nvtx("pe_layernorm_forward");
    if (!(eps >= 0.f) || !std::isfinite(eps) || (mean == nullptr) != (rstd == nullptr)) return PE_ERR_INVALID_ARG;
    if (pe_status s = check_norm(dt, w_dt, N, E); s != PE_OK) return s;
    if (N == 0) return PE_OK;
    if (!x || !y) return PE_ERR_INVALID_ARG;
    for (const void *p : {x, (const void *)y, gamma, beta})
        if (!aligned16(p)) return PE_ERR_ALIGN;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return PE_ERR_ALIGN;
    NormParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = x;
    P.gamma = gamma;
    P.beta = beta;
    P.y = y;
    P.mean = mean;
    P.rstd = rstd;
    P.N = N;
    P.E = E;
    P.w_f32 = w_dt == PE_F32;
    P.eps = eps;
    cudaStream_t st = (cudaStream_t)stream;
    return finish(dt == PE_F32 ? norm_forward<float>(P, st) : norm_forward<__nv_bfloat16>(P, st));
}

int64_t pe_layernorm_backward_workspace(int64_t N, int E) {
    if (check_norm(PE_F32, PE_F32, N, E) != PE_OK) return -1;
    const int sms = current_sms();
    return (int64_t)std::max(plan_norm_bwd(N, E, false, sms).blocks, plan_norm_bwd(N, E, true, sms).blocks) * 2 * E *
           (int64_t)sizeof(float);
}

pe_status pe_layernorm_backward(const void *dy, const void *x, pe_dtype dt, int64_t N, int E, const void *gamma,
                                pe_dtype w_dt, const float *mean, const float *rstd, void *dx, void *dgamma,
                                void *dbeta, void *ws, int64_t ws_bytes, pe_stream_t stream) {
    NvtxRange nvtx("pe_layernorm_backward");
    if ((dgamma == nullptr) != (dbeta == nullptr)) return PE_ERR_INVALID_ARG;
    if (pe_status s = check_norm(dt, w_dt, N, E); s != PE_OK) return s;
    if (N > 0 && (!dy || !x || !mean || !rstd || !dx)) return PE_ERR_INVALID_ARG;
    for (const void *p : {dy, x, gamma, (const void *)dx, (const void *)dgamma, (const void *)dbeta, (const void *)ws})
        if (!aligned16(p)) return PE_ERR_ALIGN;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return PE_ERR_ALIGN;
    const int sms = current_sms();
    if (sms < 1) return PE_ERR_CUDA;
    const NormBwdPlan plan = plan_norm_bwd(N, E, dt == PE_F32, sms);
    if (dgamma && N > 0) {
        if (!ws) return PE_ERR_INVALID_ARG;
        if (ws_bytes < (int64_t)plan.blocks * 2 * E * (int64_t)sizeof(float)) return PE_ERR_SHAPE;
    }
    NormParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = x;
    P.dy = dy;
    P.gamma = gamma;
    P.y = dx;
    P.mean = const_cast<float *>(mean);
    P.rstd = const_cast<float *>(rstd);
    P.part = dgamma ? static_cast<float *>(ws) : nullptr;
    P.N = N;
    P.E = E;
    P.w_f32 = w_dt == PE_F32;
    cudaStream_t st = (cudaStream_t)stream;
    if (N > 0) {
        const cudaError_t e = dt == PE_F32 ? norm_backward<float>(P, plan, st) : norm_backward<__nv_bfloat16>(P, plan, st);
        if (e != cudaSuccess) return PE_ERR_CUDA;
    }
    if (!dgamma) return PE_OK;
    return finish(launch_after(pe_norm_sum_kernel, dim3((unsigned)((2 * E + 31) / 32)), 1024, 0, st,
                               (const float *)P.part, plan.blocks, E, P.w_f32, dgamma, dbeta));
}

pe_status pe_attention_create(int Hq, int Hkv, int D, float scale, int causal, pe_attention **out) {
    if (!out) return PE_ERR_INVALID_ARG;
    *out = nullptr;
    if (Hq < 1 || Hkv < 1 || Hq % Hkv || D < 8 || D % 8 || !(scale > 0.f) || !std::isfinite(scale) ||
        (causal != 0 && causal != 1))
        return PE_ERR_INVALID_ARG;
    if (D > 128 || Hq > 65535 || scale < 1e-20f || scale > 1e20f) return PE_ERR_UNSUPPORTED;
    pe_attention *a = new (std::nothrow) pe_attention();
    if (!a) return PE_ERR_HOST_MEMORY;
    int major = 0, minor = 0;
    if (cudaGetDevice(&a->dev) != cudaSuccess) { delete a; return PE_ERR_CUDA; }
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, a->dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, a->dev);
    if (major != 10 || minor != 0) { delete a; return PE_ERR_UNSUPPORTED; }
    cudaDeviceGetAttribute(&a->num_sms, cudaDevAttrMultiProcessorCount, a->dev);
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->D = D;
    a->scale = scale;
    a->causal = causal;
    if (cudaMalloc(&a->err, sizeof(int)) != cudaSuccess || cudaMemset(a->err, 0, sizeof(int)) != cudaSuccess) {
        pe_attention_destroy(a);
        return PE_ERR_CUDA;
    }
    *out = a;
    return PE_OK;
}

void pe_attention_destroy(pe_attention *a) {
    if (!a) return;
    DeviceGuard g(a->dev);
    cudaDeviceSynchronize();
    if (a->err) cudaFree(a->err);
    delete a;
}

pe_status pe_attention_last_error(pe_attention *a) {
    if (!a) return PE_ERR_INVALID_ARG;
    DeviceGuard g(a->dev);
    int v = 0;
    if (cudaMemcpy(&v, a->err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return PE_ERR_CUDA;
    if (v != 0 && cudaMemset(a->err, 0, sizeof(int)) != cudaSuccess) return PE_ERR_CUDA;
    return v == 0 ? PE_OK : (pe_status)v;
}

int64_t pe_attention_workspace(const pe_attention *a, int n_seq, int64_t Nq, int64_t Nk, int backward) {
    if (check_attention(a, n_seq, Nq, Nk) != PE_OK || (backward != 0 && backward != 1)) return -1;
    if (backward) {
        const int parts = plan_key_parts(a, n_seq, Nq, Nk);
        return (int64_t)a->Hq * Nq * (int64_t)sizeof(uint4) +
               (parts > 1 ? (int64_t)parts * 2 * Nk * a->Hkv * a->D * (int64_t)sizeof(float) : 0);
    }
    if (n_seq == 0 || Nq == 0) return 0;
    const int splits = plan_forward(a, n_seq, Nq, Nk).splits;
    return splits > 1 ? (int64_t)splits * a->Hq * Nq * (a->D + 1) * (int64_t)sizeof(float) : 0;
}

static AttnParams attention_params(const pe_attention *a, int n_seq, const int32_t *cu_q, int64_t Nq,
                                   const int32_t *cu_k, int64_t Nk) {
    AttnParams P;
    std::memset(&P, 0, sizeof(P));
    P.cu_q = cu_q;
    P.cu_k = cu_k;
    P.n_seq = n_seq;
    P.Nq = (int)Nq;
    P.Nk = (int)Nk;
    P.Hq = a->Hq;
    P.Hkv = a->Hkv;
    P.D = a->D;
    P.causal = a->causal;
    P.scale = a->scale;
    P.err = a->err;
#ifdef PE_DEBUG_BOUNDS
    const char *ns = std::getenv("PE_TEST_WAIT_NS");      // two clock ticks each
    P.wait_clocks = ns ? 2 * std::atoll(ns) : kWaitClocks;
#endif
    return P;
}

pe_status pe_attention_forward(pe_attention *a, int n_seq, const int32_t *cu_q, int64_t Nq, const int32_t *cu_k,
                               int64_t Nk, pe_heads q, pe_heads k, pe_heads v, pe_heads out, float *lse, void *ws,
                               int64_t ws_bytes, pe_stream_t stream) {
    NvtxRange nvtx("pe_attention_forward");
    if (pe_status s = check_attention(a, n_seq, Nq, Nk); s != PE_OK) return s;
    if (n_seq == 0 || Nq == 0) return PE_OK;
    if (!cu_q || !cu_k) return PE_ERR_INVALID_ARG;
    if (!aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !aligned_to(lse, 4)) return PE_ERR_ALIGN;
    const int D = a->D;
    for (const pe_status s : {check_heads(q, Nq, a->Hq, D), check_heads(out, Nq, a->Hq, D)})
        if (s != PE_OK) return s;
    if (!disjoint(out, Nq, a->Hq, D)) return PE_ERR_SHAPE;
    if (Nk > 0)
        for (const pe_status s : {check_heads(k, Nk, a->Hkv, D), check_heads(v, Nk, a->Hkv, D)})
            if (s != PE_OK) return s;
    DeviceGuard g(a->dev);
    AttnParams P = attention_params(a, n_seq, cu_q, Nq, cu_k, Nk);
    P.q = heads_ptr(q, Nq, a->Hq);
    P.out = heads_ptr(out, Nq, a->Hq);
    P.k = heads_ptr(k, Nk, a->Hkv);
    P.v = heads_ptr(v, Nk, a->Hkv);
    P.lse = lse;
    const FwdPlan plan = plan_forward(a, n_seq, Nq, Nk);
    P.tiles = plan.tiles;
    P.pack = plan.pack;
    P.splits = plan.splits;
    P.n_tiles = plan.blocks;
    const int64_t all = (int64_t)plan.blocks * plan.rows * plan.splits;
    if (all > INT32_MAX) return PE_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)all);
    if (plan.splits > 1) {
        if (!ws) return PE_ERR_INVALID_ARG;
        if (!aligned16(ws)) return PE_ERR_ALIGN;
        if (ws_bytes < pe_attention_workspace(a, n_seq, Nq, Nk, 0)) return PE_ERR_SHAPE;
        P.part_out = static_cast<float *>(ws);
        P.part_lse2 = P.part_out + (int64_t)plan.splits * a->Hq * Nq * D;
    }
    cudaStream_t st = (cudaStream_t)stream;
    auto run = [&](auto dp, auto groups, auto causal) -> pe_status {
        constexpr int DP = decltype(dp)::value, G = decltype(groups)::value;
        using S = FwdShape<DP, G>;
        CUtensorMap mq, mk, mv;
        if (!make_heads_tmap(&mq, q, Nq, a->Hq, D, kTile / plan.pack, plan.pack)) return PE_ERR_CUDA;
        mk = mv = mq;                                       // without keys their maps are not read
        if (Nk > 0 && (!make_heads_tmap(&mk, k, Nk, a->Hkv, D, S::KT) || !make_heads_tmap(&mv, v, Nk, a->Hkv, D, S::KT)))
            return PE_ERR_CUDA;
        auto kern = pe_attn_fwd_kernel<DP, G, decltype(causal)::value>;
        static std::atomic<uint64_t> done{0};
        if (!ready_to_launch(kern, S::kSmem, a->dev, done, G == 1 ? 0 : kLaunchRegs)) return PE_ERR_CUDA;
        kern<<<grid, S::kThreads, S::kSmem, st>>>(mq, mk, mv, P);
        if (plan.splits > 1) {
            if (cudaGetLastError() != cudaSuccess) return PE_ERR_CUDA;
            return finish(launch_after(pe_attn_join_kernel, dim3((unsigned)(((int64_t)a->Hq * Nq + 7) / 8)), 256, 0, st, P));
        }
        return finish(cudaGetLastError());
    };
    return with_head_size(D, [&](auto dp) {
        auto of = [&](auto g) { return a->causal ? run(dp, g, std::true_type()) : run(dp, g, std::false_type()); };
        return plan.groups == 1 ? of(std::integral_constant<int, 1>()) : of(std::integral_constant<int, 2>());
    });
}

pe_status pe_attention_backward(pe_attention *a, int n_seq, const int32_t *cu_q, int64_t Nq, const int32_t *cu_k,
                                int64_t Nk, pe_heads q, pe_heads k, pe_heads v, pe_heads out, const float *lse,
                                pe_heads dout, pe_heads dq, pe_heads dk, pe_heads dv, void *ws, int64_t ws_bytes,
                                pe_stream_t stream) {
    NvtxRange nvtx("pe_attention_backward");
    if (pe_status s = check_attention(a, n_seq, Nq, Nk); s != PE_OK) return s;
    if (n_seq == 0 || (Nq == 0 && Nk == 0)) return PE_OK;
    if (!cu_q || !cu_k) return PE_ERR_INVALID_ARG;
    if (!aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !aligned_to(lse, 4)) return PE_ERR_ALIGN;
    const int D = a->D;
    if (Nq > 0) {
        if (!lse || !ws) return PE_ERR_INVALID_ARG;
        if (!aligned16(ws)) return PE_ERR_ALIGN;
        if (ws_bytes < pe_attention_workspace(a, n_seq, Nq, Nk, 1)) return PE_ERR_SHAPE;
        for (const pe_status s : {check_heads(q, Nq, a->Hq, D), check_heads(out, Nq, a->Hq, D),
                                  check_heads(dout, Nq, a->Hq, D), check_heads(dq, Nq, a->Hq, D)})
            if (s != PE_OK) return s;
        if (!disjoint(dq, Nq, a->Hq, D)) return PE_ERR_SHAPE;
    }
    if (Nk > 0)
        for (const pe_status s : {check_heads(k, Nk, a->Hkv, D), check_heads(v, Nk, a->Hkv, D),
                                  check_heads(dk, Nk, a->Hkv, D), check_heads(dv, Nk, a->Hkv, D)})
            if (s != PE_OK) return s;
    if (Nk > 0 && (!disjoint(dk, Nk, a->Hkv, D) || !disjoint(dv, Nk, a->Hkv, D))) return PE_ERR_SHAPE;
    DeviceGuard g(a->dev);
    AttnParams P = attention_params(a, n_seq, cu_q, Nq, cu_k, Nk);
    P.q = heads_ptr(q, Nq, a->Hq);
    P.out = heads_ptr(out, Nq, a->Hq);
    P.dout = heads_ptr(dout, Nq, a->Hq);
    P.dq = heads_ptr(dq, Nq, a->Hq);
    P.k = heads_ptr(k, Nk, a->Hkv);
    P.v = heads_ptr(v, Nk, a->Hkv);
    P.dk = heads_ptr(dk, Nk, a->Hkv);
    P.dv = heads_ptr(dv, Nk, a->Hkv);
    P.lse = const_cast<float *>(lse);
    P.stat = static_cast<uint4 *>(ws);
    P.splits = plan_key_parts(a, n_seq, Nq, Nk);
    P.n_tiles = max_tiles(Nk, n_seq, kTile);
    if ((int64_t)max_tiles(Nq, n_seq, kTile) * a->Hq > INT32_MAX || (int64_t)P.n_tiles * a->Hkv * P.splits > INT32_MAX)
        return PE_ERR_UNSUPPORTED;
    P.part_out = reinterpret_cast<float *>(P.stat + (int64_t)a->Hq * Nq);
    cudaStream_t st = (cudaStream_t)stream;
    CUtensorMap mq, mk, mv, md;
    if (Nq > 0 && (!make_heads_tmap(&mq, q, Nq, a->Hq, D, kStream) || !make_heads_tmap(&md, dout, Nq, a->Hq, D, kStream)))
        return PE_ERR_CUDA;
    if (Nk > 0 && (!make_heads_tmap(&mk, k, Nk, a->Hkv, D, kStream) || !make_heads_tmap(&mv, v, Nk, a->Hkv, D, kStream)))
        return PE_ERR_CUDA;
    // the maps of a side without rows are not read
    if (Nq == 0) mq = mk, md = mv;
    if (Nk == 0) mk = mq, mv = md;
    auto run = [&](auto dp, auto causal) -> pe_status {
        constexpr int DP = decltype(dp)::value;
        constexpr bool CAUSAL = decltype(causal)::value;
        auto dq_kern = pe_attn_bwd_kernel<DP, false, CAUSAL>;
        auto dkv_kern = pe_attn_bwd_kernel<DP, true, CAUSAL>;
        static std::atomic<uint64_t> dq_done{0}, dkv_done{0};
        if (!ready_to_launch(dq_kern, BwdShape<DP, false>::kSmem, a->dev, dq_done) ||
            !ready_to_launch(dkv_kern, BwdShape<DP, true>::kSmem, a->dev, dkv_done))
            return PE_ERR_CUDA;
        if (Nq > 0) {
            AttnParams Pq = P;
            Pq.splits = 1;
            Pq.n_tiles = max_tiles(Nq, n_seq, kTile);
            const dim3 grid(Pq.n_tiles * (unsigned)a->Hq);
            dq_kern<<<grid, kAttnThreads, BwdShape<DP, false>::kSmem, st>>>(mq, md, mk, mv, Pq);
            if (cudaGetLastError() != cudaSuccess) return PE_ERR_CUDA;
        }
        if (Nk > 0) {
            const dim3 grid(P.n_tiles * (unsigned)(a->Hkv * P.splits));
            const size_t smem = BwdShape<DP, true>::kSmem;
            if (Nq == 0) {
                dkv_kern<<<grid, kAttnThreads, smem, st>>>(mk, mv, mq, md, P);
                return finish(cudaGetLastError());
            }
            if (launch_after(dkv_kern, grid, kAttnThreads, smem, st, mk, mv, mq, md, P) != cudaSuccess) return PE_ERR_CUDA;
            if (P.splits > 1)
                return finish(launch_after(pe_attn_join_grads_kernel, dim3((unsigned)((Nk * a->Hkv + 7) / 8)), 256, 0, st, P));
        }
        return finish(cudaGetLastError());
    };
    return with_head_size(D, [&](auto dp) { return a->causal ? run(dp, std::true_type()) : run(dp, std::false_type()); });
}

}  // extern "C"
