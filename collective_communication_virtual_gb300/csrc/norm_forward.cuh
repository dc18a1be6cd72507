// norm_forward.cuh -- all-reduce, residual addition and RMS norm in one pass, with the
// output in the data's type or in 8 bits with scales.
//
//   h = sum_r x_r + residual          (fp32, ranks in order, then the residual)
//   rstd = 1 / sqrt(sum_j h_j^2 / hidden + eps)
//   y_j = h_j rstd w_j                (rounded once, from the fp32 h)
//   8 bits: amax = max_j |h_j w_j| rstd over the row or a group of 128 elements, at least
//   2^-64; scale = amax / 448; q_j = e4m3(h_j w_j (rstd 448 / amax))
//
// Every input byte is read once and every output byte written once: a thread keeps its part
// of h in registers across the row's reduction.  The maxima are taken of |h w| before rstd is
// known, so a row needs one reduction, not two.
//
// Bound by memory where rows are many: 8 ranks x 4096 x 4096 bf16 (604 MB) take 93 us, 0.96 of
// the measured copy rate; 1 x 16384 x 4096 to 8 bits (470 MB) 75 us, 0.93, and with a scale per 128
// elements, four shuffles a vector more, 91 us, 0.76.  Rows off 16 bytes
// take about twice the instructions and are bound by those (3 x 1537 x 2731 fp16, every rank at
// its own offset: 21 us, 0.47; 1 x 16000 x 2047 bf16: 59 us, 0.65).  One row over 8 ranks takes
// 3.7 us, a launch and two trips to memory.
#pragma once

#include "norm_stage.cuh"

namespace vc {

constexpr float kE4m3Max = 448.0f;
constexpr float kLeastAmax = 5.42101086242752217e-20f;   // 2^-64: keeps 448 / amax finite

// E values as e4m3 bytes: the low (and for E == 8 the high) word of the result.
template <int E>
__device__ __forceinline__ uint2 pack_e4m3(const float (&f)[E]) {
    uint32_t h[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; i++)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[E / 2 - 2] | (h[E / 2 - 1] << 16));
}
template <int E>
__device__ __forceinline__ void st_smem_e4m3(uint32_t p, const float (&f)[E]) {
    const uint2 q = pack_e4m3<E>(f);
    if (E == 8) asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(p), "r"(q.x), "r"(q.y) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" :: "r"(p), "r"(q.x) : "memory");
}

// A row's address, its team and the thread's place in it.
struct RowPlace {
    size_t row;
    bool live;                       // the row exists
    int t, part, col0;               // thread of the team, CTA of the cluster, its first column
    uint32_t buf;                    // GENERAL: the team's row buffers in shared memory
};

// What a row's team does once a thread has its part of h: the stream, the reduction, the scaled
// output.  weight(v, f) gives the weight's values for vector v, zeros behind the row's end.
// Q: 0 output in the data's type, 1 8 bits with one scale a row, 2 with one per 128 elements.
template <int DT, int V, bool GENERAL, int Q, typename Weight>
__device__ __forceinline__ void finish_row(const NormArgs& a, TeamScratch& red, const RowPlace& at, const RowVecs<DT, V>& rv,
                                           float (&h)[V][kVecElems<DT>], Weight weight) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const NormShape& sh = a.shape;
    const int columns = min(a.hidden - at.col0, sh.teamThreads * V * E);   // of this CTA
    const int mine = at.t * E;                         // the thread's first column of them
    // From here on a thread holds zeros behind the row's end, and only the stores ask for it.
    if (GENERAL) rv.mask(h);
    float2 two[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int v = 0; v < V; v++) {
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 x = make_float2(h[v][j], h[v][j + 1]);
            two[j / 2 & 1] = fma2(x, x, two[j / 2 & 1]);
        }
        if (!a.residualOut) continue;
        if (GENERAL) st_smem(at.buf + (uint32_t)((mine + v * rv.step) * ESZ), narrow_vec<DT>(h[v]));
        else if (at.live && rv.left[v] > 0)
            st_stream((char*)a.residualOut + (at.row * a.residualStride + rv.e0 + v * rv.step) * ESZ, narrow_vec<DT>(h[v]));
    }
    float sum = (two[0].x + two[0].y) + (two[1].x + two[1].y);

    // From here on h holds h w.
    float top = 0.0f, lead[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        weight(v, f);
        mul_by(h[v], f);
        if (!Q) continue;
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < E; j += 2) m = max_abs(m, h[v][j], h[v][j + 1]);
        if (Q == 1) {
            top = max_abs(top, m, 0.0f);
        } else {
            // a group lies in 128 / E neighbouring lanes, or a row in fewer: one vector a thread then
            const int lanes = min(kQuantGroup / E, sh.teamThreads);
            for (int o = lanes >> 1; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(~0u, m, o), 0.0f);
            lead[v] = m;
        }
    }
    if (GENERAL) __syncwarp();                         // a larger team's barrier is in its reduction
    team_reduce<Q == 1>(red, sh, sum, top);
    const float rstd = __frsqrt_rn(sum / (float)a.hidden + a.eps);
    if (a.rstd && at.live && at.t == 0 && at.part == 0) a.rstd[at.row] = rstd;
    if (GENERAL && a.residualOut && at.live)
        copy_out<ESZ>((char*)a.residualOut + (at.row * a.residualStride + at.col0) * ESZ, at.buf, columns * ESZ, at.t, sh.teamThreads);

    // A row (group) with a NaN has NaN as its scale.
    const auto amax_of = [&](float m) {
        const float f = m * rstd;
        return f < kLeastAmax ? kLeastAmax : f;
    };
    float amax[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (Q) amax[v] = amax_of(Q == 1 ? top : lead[v]);
        scale_by(h[v], Q ? rstd * (kE4m3Max / amax[v]) : rstd);
    }
    constexpr int OSZ = Q ? 1 : ESZ;
    if (GENERAL) {
        const size_t off = (at.row * a.recvStride + at.col0) * OSZ;
        const uint32_t buf = at.buf + (uint32_t)sh.rowBytes;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const uint32_t p = buf + (uint32_t)((mine + v * rv.step) * OSZ);
            if (Q) st_smem_e4m3<E>(p, h[v]);
            else st_smem(p, narrow_vec<DT>(h[v]));
        }
        if (sh.teamThreads > 32) __syncthreads();
        else __syncwarp();
        if (at.live) copy_out_all<OSZ>(a.recv, a.nOut, a.outSame, off, buf, columns * OSZ, at.t, sh.teamThreads);
    } else if (at.live) {
        for (int o = 0; o < a.nOut; o++) {
            char* p = (char*)a.recv[o] + (at.row * a.recvStride + rv.e0) * OSZ;
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (rv.left[v] == 0) continue;
                char* q = p + (size_t)v * rv.step * OSZ;
                if (Q == 0) {
                    st_stream(q, narrow_vec<DT>(h[v]));
                } else {
                    const uint2 b = pack_e4m3<E>(h[v]);
                    if (E == 8) *reinterpret_cast<uint2*>(q) = b;
                    else *reinterpret_cast<uint32_t*>(q) = b.x;
                }
            }
        }
    }
    if constexpr (Q == 1) {
        if (at.live && at.t == 0 && at.part == 0)
            for (int o = 0; o < a.nOut; o++) a.scales[o][at.row] = amax[0] / kE4m3Max;
    }
    if constexpr (Q == 2) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int e = rv.e0 + v * rv.step;
            if (!at.live || rv.left[v] == 0 || (e & (kQuantGroup - 1)) != 0) continue;     // a group's first vector
            for (int o = 0; o < a.nOut; o++) a.scales[o][at.row * (size_t)a.groups + e / kQuantGroup] = amax[v] / kE4m3Max;
        }
    }
}

// Few rows, or rows too long to stage: every team takes one row and loads it directly, one
// vector a thread where that reaches, split over a cluster of up to 8 CTAs while SMs are idle.
template <int DT, int V, bool GENERAL, int Q>
__global__ void __launch_bounds__(kNormMaxThreads, 1) k_allreduce_rmsnorm(const __grid_constant__ NormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red;
    const NormShape& sh = a.shape;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    RowPlace at;
    at.t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    at.part = sh.cluster > 1 ? (int)cluster_rank() : 0;
    at.col0 = at.part * sh.teamThreads * V * E;
    at.row = (size_t)(blockIdx.x / (unsigned)sh.cluster) * sh.rowsPerCta + team;
    at.live = at.row < a.rows;
    at.buf = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(2 * team * sh.rowBytes);
    if (sh.cluster > 1) cluster_arrive();
    const RowVecs<DT, V> rv(at.col0 + at.t * E, sh.teamThreads * E, a.hidden);

    // The weight's and the residual's loads are under way while the ranks' are awaited.
    float w[V][E];
    uint4 res[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = rv.e0 + v * rv.step;
        load_weight<DT, GENERAL>(a.weight, a.weightF32, e, rv.left[v], w[v]);
        res[v] = make_uint4(0u, 0u, 0u, 0u);
        if (a.residual && at.live && rv.left[v] > 0)
            res[v] = load_vec<ESZ, GENERAL>((const char*)a.residual + (at.row * a.residualStride + e) * ESZ, rv.left[v]);
    }
    if (GENERAL) rv.mask(w);
    float h[V][E];
    sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, (at.row * a.sendStride + rv.e0) * ESZ, at.live, rv, h);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        widen_vec<DT>(res[v], f);
        add_to(h[v], f);
    }
    finish_row<DT, V, GENERAL, Q>(a, red, at, rv, h, [&](int v, float (&f)[E]) {
#pragma unroll
        for (int j = 0; j < E; j++) f[j] = w[v][j];
    });
}

// Many rows: the next row's loads under way while one is finished.  A CTA takes sh.rounds rows
// (of each of its teams) one behind the other: CTAs start in order and stay near one another,
// which the memory rewards (1 x 16384 x 4096 bf16: 82 us; 97 us where as many CTAs stride over
// all rows and drift apart; 4 x 4096 x 8192: 102 and 114, 8 x 4096 x 4096: 93 and 95).  Only
// unaligned rows so long that one CTA fills an SM's share of the memory are strided over
// (sh.rounds 0), as what a CTA does before its first row costs most there (8 x 2000 x 4097: 60 us,
// 66 in rounds).
//
// SHARED: the CTAs of a cluster share a row that one cannot hold, and finish it together.  An
// instance of its own, as what it adds costs the others up to 2 % (3 x 1537 x 2731: 21.2 us, 20.9
// without).  1 x 4096 x 32768 bf16 takes 231 us (0.68 of the measured copy rate; 387 with direct
// loads), 8 x 1500 x 16384 148 us (0.88; 160): each row waits for two barriers of its cluster.
template <int DT, int V, bool GENERAL, int Q, bool SHARED>
__global__ void __launch_bounds__(kStageMaxThreads, V == 1 ? 2 : 1)
k_allreduce_rmsnorm_staged(const __grid_constant__ NormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    RowPlace at;
    at.t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    at.part = SHARED ? (int)cluster_rank() : 0;
    at.col0 = at.part * sh.teamThreads * V * E;
    if (SHARED) cluster_arrive();
    at.buf = base + (uint32_t)(sh.weightBytes + sh.stageBytes + 2 * team * sh.rowBytes);
    const RowVecs<DT, V> rv(at.col0 + at.t * E, sh.teamThreads * E, a.hidden);
    const StageAddr stage = stage_addr<GENERAL>(base + (uint32_t)sh.weightBytes, sh);
    const int N = a.nRanks, segments = N + (a.residual ? 1 : 0);

    const unsigned index = SHARED ? blockIdx.x / (unsigned)sh.cluster : blockIdx.x;
    const size_t first = (size_t)index * max(1, sh.rounds) * sh.rowsPerCta;
    const size_t step = (size_t)(sh.rounds ? 1 : sh.ctas) * sh.rowsPerCta;
    const size_t end = sh.rounds ? min(a.rows, first + (size_t)sh.rounds * sh.rowsPerCta) : a.rows;
    // address of a segment's element rv.e0: the ranks', then the residual's
    const auto segment = [&](int s, size_t row) {
        return s < N ? (const char*)a.send[s] + (row * a.sendStride + rv.e0) * ESZ
                     : (const char*)a.residual + (row * a.residualStride + rv.e0) * ESZ;
    };
    const auto fetch = [&](size_t row) {
        if (row < end)
            for (int s = 0; s < segments; s++) stage_segment<DT, V, GENERAL>(stage, s, segment(s, row), rv);
        copies_commit();
    };
    if (!GENERAL) stage_zeros<DT, V>(stage, segments, rv);
    fetch(first + team);
    stage_weight<DT, GENERAL>(a.weight, a.weightF32, at.col0, a.hidden, base, sh.weightBytes);
    copies_wait();
    __syncthreads();                                   // the weight, copied by all threads
    int flip = 0;
    // every team of a CTA, and every CTA of a cluster, runs the same number of rounds
    for (size_t row0 = first; row0 < end; row0 += step) {
        at.row = row0 + team;
        at.live = at.row < end;
        float h[V][E];
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] = 0.0f;
        copies_wait();
        if (GENERAL) __syncwarp();
#pragma unroll 2
        for (int s = 0; s < segments; s++)
            add_segment<DT, V, GENERAL>(stage, s, GENERAL ? (unsigned)(uintptr_t)segment(s, at.row) & 15u : 0u, h);
        if (GENERAL) __syncwarp();
        fetch(at.row + step);
        finish_row<DT, V, GENERAL, Q>(a, red[flip], at, rv, h, [&](int v, float (&f)[E]) {
            staged_weight<DT>(base, a.weightF32, at.t * E + v * rv.step, f);
        });
        if (SHARED) cluster_arrive();
        flip ^= 1;
    }
    if (SHARED) cluster_wait();
    copies_wait();
}

template <int DT, int V, bool GENERAL, int Q>
static cudaError_t norm_launch_g(const NormArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const auto kernel = !sh.staged       ? k_allreduce_rmsnorm<DT, V, GENERAL, Q>
                        : sh.cluster > 1 ? k_allreduce_rmsnorm_staged<DT, V, GENERAL, Q, true>
                                         : k_allreduce_rmsnorm_staged<DT, V, GENERAL, Q, false>;
    const cudaError_t e = allow_smem(kernel, sh.smemBytes);
    if (e != cudaSuccess) return e;
    const size_t teams = sh.staged ? (size_t)sh.ctas : (a.rows + sh.rowsPerCta - 1) / sh.rowsPerCta;
    return norm_launch(kernel, (unsigned)(teams * (size_t)sh.cluster), sh, sh.smemBytes, s, a);
}
template <int DT, int V, int Q>
static cudaError_t norm_launch_v(const NormArgs& a, cudaStream_t s) {
    return a.shape.general ? norm_launch_g<DT, V, true, Q>(a, s) : norm_launch_g<DT, V, false, Q>(a, s);
}
template <int DT, int Q>
static cudaError_t norm_launch_dt(const NormArgs& a, cudaStream_t s) {
    switch (a.shape.vecs) {
    case 1: return norm_launch_v<DT, 1, Q>(a, s);
    case 2: return norm_launch_v<DT, 2, Q>(a, s);
    default: return norm_launch_v<DT, 4, Q>(a, s);
    }
}
template <int Q>
static cudaError_t norm_launch_q(const NormArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return norm_launch_dt<kF32, Q>(a, s);
    case vFloat16: return norm_launch_dt<kF16, Q>(a, s);
    case vBFloat16: return norm_launch_dt<kBF16, Q>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
