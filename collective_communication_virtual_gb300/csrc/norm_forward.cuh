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
// of h and of the weight in registers across the row's reduction.  The maxima are taken of
// |h w| before rstd is known, so a row needs one reduction, not two.
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
__device__ __forceinline__ void store_e4m3(char* p, Span sp, bool whole, const float (&f)[E]) {
    const uint2 q = pack_e4m3<E>(f);
    if (whole && ((uintptr_t)p & (E - 1)) == 0) {
        if (E == 8) *reinterpret_cast<uint2*>(p) = q;
        else *reinterpret_cast<uint32_t*>(p) = q.x;
        return;
    }
#pragma unroll
    for (int j = 0; j < E; j++)
        if (sp.has(j)) *reinterpret_cast<uint8_t*>(p + j) = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
}
template <int E>
__device__ __forceinline__ void st_smem_e4m3(uint32_t p, const float (&f)[E]) {
    const uint2 q = pack_e4m3<E>(f);
    if (E == 8) asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(p), "r"(q.x), "r"(q.y) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" :: "r"(p), "r"(q.x) : "memory");
}

// What a row's team does once a thread has its part of h: the stream, the reduction, the scaled
// output.  weight(v, f) gives the weight's values for vector v.  groupMax: this row's maxima of
// the CTA's scale groups, zero on entry (GENERAL; aligned rows keep theirs in registers).
// rowBuf: the team's two row buffers in shared memory (its stream, then its output), 0 where
// every output's rows start at the frame's offset from 16 bytes.
// Q: 0 output in the data's type, 1 8 bits with one scale a row, 2 with one per 128 elements.
template <int DT, int V, bool GENERAL, int Q, typename Weight>
__device__ __forceinline__ void finish_row(const NormArgs& a, TeamScratch& red, uint32_t* groupMax, uint32_t rowBuf,
                                           size_t row, bool live, int t, int team, int part, const RowVecs<DT, V>& rv,
                                           float (&h)[V][kVecElems<DT>], Weight weight) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int e0 = rv.e0, step = rv.step;
    // columns of this CTA, and where its first one lies in a row buffer (elements)
    const int col0 = part * sh.teamThreads * V * E;
    const int columns = min(a.hidden - col0, clustered ? sh.teamThreads * V * E : a.hidden);
    const int bufShift = col0 + t * E - e0;
    const ptrdiff_t resOff = ((ptrdiff_t)(row * a.residualStride) + e0) * ESZ;
    const bool streamBuf = GENERAL && rowBuf && a.residualOut && ((uintptr_t)a.residualOut + resOff) & 15u;
    // Vectors outside the row hold zeros from here on, and only the stores ask for them.
    if (GENERAL) rv.mask(h);
    float2 two = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < V; v++) {
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 x = make_float2(h[v][j], h[v][j + 1]);
            two = fma2(x, x, two);
        }
        if (streamBuf) st_smem(rowBuf + (uint32_t)(v * sh.teamThreads + t) * 16u, narrow_vec<DT>(h[v]));
        else if (a.residualOut && rv.on[v])
            store_vec<DT, GENERAL>((char*)a.residualOut + resOff + (ptrdiff_t)v * step * ESZ, rv.sp[v], h[v]);
    }
    float sum = two.x + two.y;

    // From here on h holds h w.
    float top = 0.0f, lead[V];
    const int groupsHere = Q == 2 ? (a.hidden + kQuantGroup - 1) / kQuantGroup : 0;
    const int groupBase = !clustered ? team * groupsHere : -(part * sh.teamThreads * V * E / kQuantGroup);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        weight(v, f);
        mul_by(h[v], f);
    }
    if (GENERAL && Q) rv.mask(h);                      // the weight outside the row is undefined
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = e0 + v * step;
        if (Q == 1) {
#pragma unroll
            for (int j = 0; j < E; j += 2) top = max_abs(top, h[v][j], h[v][j + 1]);
        }
        if (Q == 2 && !GENERAL) {
            // a group lies in 128 / E neighbouring lanes (smaller teams take the general path)
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < E; j += 2) m = max_abs(m, h[v][j], h[v][j + 1]);
#pragma unroll
            for (int o = kQuantGroup / E / 2; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(~0u, m, o), 0.0f);
            lead[v] = m;
        }
        if (Q == 2 && GENERAL && rv.on[v]) {
            // m0 is of the group of element e + E - 1, m1 of the one before it
            float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
            for (int j = 0; j < E; j++) {
                if (((e + j) >> 7) != ((e + E - 1) >> 7)) m1 = max_abs(m1, h[v][j], 0.0f);
                else m0 = max_abs(m0, h[v][j], 0.0f);
            }
            const int last = (e + rv.sp[v].hi - 1) >> 7, first = (e + rv.sp[v].lo) >> 7;
            const int g0 = (e + E - 1) >> 7;
            // bits of non-negative floats order as the floats do, a NaN above all
            if (g0 <= last && g0 >= first) atomicMax(&groupMax[groupBase + g0], __float_as_uint(m0));
            if (g0 - 1 >= first && g0 - 1 <= last) atomicMax(&groupMax[groupBase + g0 - 1], __float_as_uint(m1));
        }
    }
    if (GENERAL) __syncwarp();                         // a larger team's barrier is in its reduction
    team_reduce<Q == 1>(red, sh, sum, top);
    const float rstd = __frsqrt_rn(sum / (float)a.hidden + a.eps);
    if (a.rstd && live && t == 0 && part == 0) a.rstd[row] = rstd;
    if (streamBuf && live)
        copy_out<ESZ>((char*)a.residualOut + ((ptrdiff_t)(row * a.residualStride) + col0) * ESZ,
                      rowBuf + (uint32_t)(bufShift * ESZ), columns * ESZ, t, sh.teamThreads);
    const uint32_t outBuf = rowBuf + (uint32_t)sh.rowBytes;
    const auto team_sync = [&]() {
        if (sh.teamThreads > 32) __syncthreads();
        else __syncwarp();
    };

    if (Q == 0) {
#pragma unroll
        for (int v = 0; v < V; v++) scale_by(h[v], rstd);
        const ptrdiff_t off = ((ptrdiff_t)(row * a.recvStride) + e0) * ESZ;
        if (GENERAL && rowBuf) {
#pragma unroll
            for (int v = 0; v < V; v++)
                st_smem(outBuf + (uint32_t)(v * sh.teamThreads + t) * 16u, narrow_vec<DT>(h[v]));
            team_sync();
        }
        for (int o = 0; o < a.nOut; o++) {
            char* p = (char*)a.recv[o] + off;
            if (GENERAL && rowBuf && ((uintptr_t)p & 15u)) {
                if (live)
                    copy_out<ESZ>((char*)a.recv[o] + ((ptrdiff_t)(row * a.recvStride) + col0) * ESZ,
                                  outBuf + (uint32_t)(bufShift * ESZ), columns * ESZ, t, sh.teamThreads);
                continue;
            }
#pragma unroll
            for (int v = 0; v < V; v++)
                if (rv.on[v]) store_vec<DT, GENERAL>(p + (ptrdiff_t)v * step * ESZ, rv.sp[v], h[v]);
        }
        return;
    }

    // A row (group) with a NaN has NaN as its scale.
    const auto amax_of = [&](float m) {
        const float f = m * rstd;
        return f < kLeastAmax ? kLeastAmax : f;
    };
    const ptrdiff_t off = (ptrdiff_t)(row * a.recvStride) + e0;
    float amax[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = e0 + v * step;
        if (Q == 1 || !GENERAL) {
            amax[v] = amax_of(Q == 1 ? top : lead[v]);
            scale_by(h[v], rstd * (kE4m3Max / amax[v]));
        } else if (rv.on[v]) {
            const int g0 = (e + E - 1) >> 7;
            const float k0 = rstd * (kE4m3Max / amax_of(__uint_as_float(groupMax[groupBase + min(g0, groupsHere - 1)])));
            const float k1 = g0 > 0 && (e >> 7) != g0 ? rstd * (kE4m3Max / amax_of(__uint_as_float(groupMax[groupBase + g0 - 1]))) : k0;
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] *= ((e + j) >> 7) != g0 ? k1 : k0;
        }
    }
    if (GENERAL && rowBuf) {
#pragma unroll
        for (int v = 0; v < V; v++) st_smem_e4m3<E>(outBuf + (uint32_t)((v * sh.teamThreads + t) * E), h[v]);
        team_sync();
    }
    for (int o = 0; o < a.nOut; o++) {
        if (GENERAL && rowBuf && (((uintptr_t)a.recv[o] + off) & (E - 1))) {
            if (live)
                copy_out<1>((char*)a.recv[o] + (ptrdiff_t)(row * a.recvStride) + col0, outBuf + (uint32_t)bufShift, columns,
                            t, sh.teamThreads);
            continue;
        }
#pragma unroll
        for (int v = 0; v < V; v++)
            if (rv.on[v])
                store_e4m3<E>((char*)a.recv[o] + off + (ptrdiff_t)v * step, rv.sp[v], !GENERAL || rv.sp[v].full(E), h[v]);
    }
    if (!live) return;
    if (Q == 1) {
        if (t == 0 && part == 0)
            for (int o = 0; o < a.nOut; o++) a.scales[o][row] = amax[0] / kE4m3Max;
    } else if (!GENERAL) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!rv.on[v] || (t & (kQuantGroup / E - 1)) != 0) continue;
            const size_t at = row * (size_t)a.groups + ((e0 + v * step) >> 7);
            for (int o = 0; o < a.nOut; o++) a.scales[o][at] = amax[v] / kE4m3Max;
        }
    } else {
        const int gFirst = clustered ? part * sh.teamThreads * V * E / kQuantGroup : 0;
        const int gEnd = clustered ? min(groupsHere, (part + 1) * sh.teamThreads * V * E / kQuantGroup) : groupsHere;
        for (int g = gFirst + t; g < gEnd; g += sh.teamThreads) {
            const float scale = amax_of(__uint_as_float(groupMax[groupBase + g])) / kE4m3Max;
            for (int o = 0; o < a.nOut; o++) a.scales[o][row * (size_t)a.groups + g] = scale;
        }
    }
}

// Offset of a row from a vector's boundary in the first output, in elements.
template <int DT, int OSZ>
__device__ __forceinline__ int frame_shift(const NormArgs& a, size_t row) {
    constexpr int E = kVecElems<DT>;
    return (int)(((uintptr_t)a.recv[0] + row * a.recvStride * OSZ) & (E * OSZ - 1)) / OSZ;
}

// Few rows, or rows too long to stage: every team takes one row and loads it directly.
template <int DT, int V, bool GENERAL, int Q>
__global__ void __launch_bounds__(kNormMaxThreads, 1) k_allreduce_rmsnorm(const __grid_constant__ NormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red;
    __shared__ uint32_t groupMax[Q == 2 && GENERAL ? kNormGroupSlots : 1];
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int part = clustered ? (int)cluster_rank() : 0;
    const size_t row = (size_t)(blockIdx.x / (unsigned)sh.cluster) * sh.rowsPerCta + team;
    const bool live = row < a.rows;
    if (clustered) cluster_arrive();
    if (Q == 2 && GENERAL) {
        for (int i = threadIdx.x; i < kNormGroupSlots; i += blockDim.x) groupMax[i] = 0u;
        __syncthreads();
    }
    // CTAs of a cluster cut the row at multiples of a vector from its start, so that a scale
    // group never spans two CTAs.
    const int shift = GENERAL && live && !clustered ? frame_shift<DT, Q ? 1 : ESZ>(a, row) : 0;
    RowVecs<DT, V> rv;
    rv.set((part * sh.teamThreads * V + t) * E - shift, sh.teamThreads * E, a.hidden, live);

    // The weight's and the residual's loads are under way while the ranks' are awaited.
    WeightVec<DT> w[V];
    uint4 res[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = rv.e0 + v * rv.step;
        if (rv.on[v]) w[v].template load<GENERAL>(a.weight, a.weightF32, e, rv.sp[v]);
        if (a.residual && rv.on[v])
            res[v] = load_vec<ESZ, GENERAL>((const char*)a.residual + ((ptrdiff_t)(row * a.residualStride) + e) * ESZ,
                                            rv.sp[v]);
    }
    float h[V][E];
    sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, ((ptrdiff_t)(row * a.sendStride) + rv.e0) * ESZ, rv, h);
    if (a.residual) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!rv.on[v]) continue;
            float f[E];
            widen_vec<DT>(res[v], f);
            add_to(h[v], f);
        }
    }
    const uint32_t rowBuf = GENERAL && sh.rowBytes ? (uint32_t)__cvta_generic_to_shared(smem) +
                                                         (uint32_t)(2 * team * sh.rowBytes) : 0u;
    finish_row<DT, V, GENERAL, Q>(a, red, groupMax, rowBuf, row, live, t, team, part, rv, h, [&](int v, float (&f)[E]) {
        if (rv.on[v]) {
            w[v].get(a.weightF32, f);
        } else {
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = 0.0f;
        }
    });
}

// Many rows: CTAs stride over them, the next row's loads under way while one is finished.
template <int V> constexpr int staged_min_ctas() { return V == 4 ? 1 : V == 2 ? 1 : 2; }
template <int DT, int V, bool GENERAL, int Q>
__global__ void __launch_bounds__(kStageMaxThreads, staged_min_ctas<V>())
k_allreduce_rmsnorm_staged(const __grid_constant__ NormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    __shared__ uint32_t groupMax[Q == 2 && GENERAL ? 3 * kNormGroupSlots : 1];
    const NormShape& sh = a.shape;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int N = a.nRanks;
    const int segments = N + (a.residual ? 1 : 0);
    const uint32_t base0 = (uint32_t)__cvta_generic_to_shared(smem);
    StageAddr stage;
    stage.pitch = blockDim.x * 16u;
    stage.base = base0 + (uint32_t)sh.weightBytes + threadIdx.x * 16u;
    stage.second = (uint32_t)segments * V * stage.pitch;
    const WeightSmem ws = stage_weight(a.weight, a.weightF32, a.weightF32 ? 4 : ESZ, a.hidden, base0,
                                       sh.weightBytes);
    const uint32_t rowBuf = GENERAL && sh.rowBytes
                                ? base0 + (uint32_t)(sh.weightBytes + sh.stageBytes + 2 * team * sh.rowBytes) : 0u;
    if (Q == 2 && GENERAL)
        for (int i = threadIdx.x; i < 3 * kNormGroupSlots; i += blockDim.x) groupMax[i] = 0u;

    const auto frame = [&](size_t row, RowVecs<DT, V>& rv) {
        const bool live = row < a.rows;
        const int shift = GENERAL && live ? frame_shift<DT, Q ? 1 : ESZ>(a, row) : 0;
        rv.set(t * E - shift, sh.teamThreads * E, a.hidden, live);
    };
    // address of a segment's element e0: the ranks', then the residual's
    const auto segment = [&](int s, size_t row, int e0) {
        return s < N ? (const char*)a.send[s] + ((ptrdiff_t)(row * a.sendStride) + e0) * ESZ
                     : (const char*)a.residual + ((ptrdiff_t)(row * a.residualStride) + e0) * ESZ;
    };
    // start a row's copies; none for a row past the end, whose vectors are all off
    const auto fetch = [&](size_t row) {
        RowVecs<DT, V> rv;
        frame(row, rv);
        for (int s = 0; s < segments; s++) stage_segment<DT, V, GENERAL>(stage, s, segment(s, row, rv.e0), rv);
        copies_commit();
    };
    const size_t first = (size_t)blockIdx.x * sh.rowsPerCta, stride = (size_t)gridDim.x * sh.rowsPerCta;
    if (!GENERAL) {
        RowVecs<DT, V> rv;
        frame(first + team, rv);
        stage_zeros<DT, V>(stage, segments, rv);
    }
    fetch(first + team);
    copies_wait();
    __syncthreads();                                   // the weight has been copied, by all threads
    int flip = 0, turn = 0;
    // every team of a CTA runs the same number of rounds
    for (size_t base = first; base < a.rows; base += stride) {
        const size_t row = base + team;
        RowVecs<DT, V> rv;
        frame(row, rv);
        float h[V][E];
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] = 0.0f;
        copies_wait();
#pragma unroll 2
        for (int s = 0; s < segments; s++)
            add_segment<DT, V, GENERAL>(stage, s, GENERAL ? (unsigned)(uintptr_t)segment(s, row, rv.e0) & 15u : 0u, rv, h);
        fetch(row + stride);
        uint32_t* groups = groupMax;
        if (Q == 2 && GENERAL) {
            // Three sets of maxima: this row's, the one the last row may still be read from, and
            // the next row's, which is cleared now.
            const int mine = (a.hidden + kQuantGroup - 1) / kQuantGroup, after = turn == 2 ? 0 : turn + 1;
            groups = groupMax + turn * kNormGroupSlots;
            for (int g = t; g < mine; g += sh.teamThreads) groupMax[after * kNormGroupSlots + team * mine + g] = 0u;
            turn = after;
        }
        finish_row<DT, V, GENERAL, Q>(a, red[flip], groups, rowBuf, row, row < a.rows, t, team, 0, rv, h,
                                      [&](int v, float (&f)[E]) { weight_vec<DT, GENERAL>(ws, rv.e0 + v * rv.step, f); });
        flip ^= 1;
    }
    copies_wait();
}

template <int DT, int V, bool GENERAL, int Q>
static cudaError_t norm_launch_g(const NormArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const cudaError_t e = sh.staged ? allow_smem(k_allreduce_rmsnorm_staged<DT, V, GENERAL, Q>, sh.smemBytes)
                                    : allow_smem(k_allreduce_rmsnorm<DT, V, GENERAL, Q>, sh.smemBytes);
    if (e != cudaSuccess) return e;
    if (sh.staged)
        return norm_launch(k_allreduce_rmsnorm_staged<DT, V, GENERAL, Q>, (unsigned)sh.ctas, sh, sh.smemBytes, s, a);
    const size_t ctas = (a.rows + sh.rowsPerCta - 1) / sh.rowsPerCta * (size_t)sh.cluster;
    return norm_launch(k_allreduce_rmsnorm<DT, V, GENERAL, Q>, (unsigned)ctas, sh, sh.smemBytes, s, a);
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
