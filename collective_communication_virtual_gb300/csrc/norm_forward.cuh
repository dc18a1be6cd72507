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

#include "norm.cuh"

namespace vc {

constexpr float kE4m3Max = 448.0f;
constexpr float kLeastAmax = 5.42101086242752217e-20f;   // 2^-64: keeps 448 / amax finite

template <int E>
__device__ __forceinline__ void store_e4m3(char* p, Span sp, bool whole, const float (&f)[E]) {
    uint16_t h[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; i++)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if (whole && ((uintptr_t)p & (E - 1)) == 0) {
        if (E == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | ((uint32_t)h[1] << 16),
                                                      h[E / 2 - 2] | ((uint32_t)h[E / 2 - 1] << 16));
        else
            *reinterpret_cast<uint32_t*>(p) = h[0] | ((uint32_t)h[1] << 16);
        return;
    }
#pragma unroll
    for (int j = 0; j < E; j++)
        if (sp.has(j)) *reinterpret_cast<uint8_t*>(p + j) = (uint8_t)(h[j >> 1] >> (8 * (j & 1)));
}

template <int V> constexpr int norm_cta_threads() { return V == 4 ? kNormMaxThreads : 512; }
template <int V> constexpr int norm_ctas_per_sm() { return V == 4 ? 1 : 2; }

// Q: 0 output in the data's type, 1 8 bits with one scale a row, 2 with one per 128 elements.
template <int DT, int V, bool GENERAL, int Q>
__global__ void __launch_bounds__(norm_cta_threads<V>(), norm_ctas_per_sm<V>())
k_allreduce_rmsnorm(const __grid_constant__ NormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    constexpr int OSZ = Q ? 1 : ESZ;
    __shared__ TeamScratch red;
    __shared__ uint32_t groupMax[Q == 2 ? kNormGroupSlots : 1];
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int part = clustered ? (int)cluster_rank() : 0;
    const size_t row = (size_t)(blockIdx.x / (unsigned)sh.cluster) * sh.rowsPerCta + team;
    const bool live = row < a.rows;
    if (clustered) cluster_arrive();
    if (Q == 2) {
        for (int i = threadIdx.x; i < kNormGroupSlots; i += blockDim.x) groupMax[i] = 0u;
        __syncthreads();
    }

    // The frame of the row's vectors.  CTAs of a cluster cut the row at multiples of a
    // vector from its start, so that a scale group never spans two CTAs.
    int shift = 0;
    if (GENERAL && live && !clustered)
        shift = (int)(((uintptr_t)a.recv[0] + row * a.recvStride * OSZ) & (E * OSZ - 1)) / OSZ;
    const int e0 = (part * sh.teamThreads * V + t) * E - shift;
    const int step = sh.teamThreads * E;               // elements between a thread's vectors
    Span sp[V];
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        sp[v] = span_of<E>(e0 + v * step, a.hidden);
        on[v] = live && sp[v].any();
    }

    // The weight's and the residual's loads are under way while the ranks' are awaited.
    WeightVec<DT> w[V];
    uint4 res[V];
    const ptrdiff_t resOff = ((ptrdiff_t)(row * a.residualStride) + e0) * ESZ;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (on[v]) w[v].template load<GENERAL>(a.weight, a.weightF32, e0 + v * step, sp[v]);
        if (a.residual && on[v])
            res[v] = load_vec<ESZ, GENERAL>((const char*)a.residual + resOff + (ptrdiff_t)v * step * ESZ, sp[v]);
    }
    float h[V][E];
    sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, ((ptrdiff_t)(row * a.sendStride) + e0) * ESZ, sp, on,
                              (ptrdiff_t)step * ESZ, h);
    float sum = 0.0f;
    uint32_t top = 0u;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (!on[v]) continue;
        if (a.residual) {
            float f[E];
            widen_vec<DT>(res[v], f);
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] += f[j];
        }
        if (GENERAL) {
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] = sp[v].has(j) ? h[v][j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < E; j++) sum = fmaf(h[v][j], h[v][j], sum);
        if (a.residualOut)
            store_vec<DT, GENERAL>((char*)a.residualOut + resOff + (ptrdiff_t)v * step * ESZ, sp[v], h[v]);
    }

    // From here on h holds h w.
    const int groupsHere = Q == 2 ? (a.hidden + kQuantGroup - 1) / kQuantGroup : 0;
    const int groupBase = Q == 2 && !clustered ? team * groupsHere
                          : -(part * sh.teamThreads * V * E / kQuantGroup);
#pragma unroll
    for (int v = 0; v < V; v++) {
        uint32_t m0 = 0u, m1 = 0u;                     // maxima of the vector's one or two groups
        const int e = e0 + v * step;
        if (on[v]) {
            float f[E];
            w[v].get(a.weightF32, f);
#pragma unroll
            for (int j = 0; j < E; j++) {
                h[v][j] = GENERAL ? (sp[v].has(j) ? h[v][j] * f[j] : 0.0f) : h[v][j] * f[j];
                if (Q) {
                    const uint32_t b = __float_as_uint(h[v][j]) & 0x7FFFFFFFu;
                    if (Q == 2 && GENERAL && ((e + j) >> 7) != ((e + E - 1) >> 7)) m1 = max(m1, b);
                    else m0 = max(m0, b);
                }
            }
        }
        if (Q == 1) top = max(top, m0);
        if (Q == 2 && !GENERAL) {
            // whole groups lie in 128 / E neighbouring lanes, but in the smallest teams
            const int lanes = min(kQuantGroup / E, sh.teamThreads);
            for (int o = lanes >> 1; o > 0; o >>= 1) m0 = max(m0, __shfl_xor_sync(~0u, m0, o));
            if (on[v] && (t & (lanes - 1)) == 0) atomicMax(&groupMax[groupBase + (e >> 7)], m0);
        }
        if (Q == 2 && GENERAL && on[v]) {
            const int last = (e + sp[v].hi - 1) >> 7, first = (e + sp[v].lo) >> 7;
            // m0 is the group of element e + E - 1, m1 the one before it
            const int g0 = (e + E - 1) >> 7;
            if (g0 <= last && g0 >= first) atomicMax(&groupMax[groupBase + g0], m0);
            if (g0 - 1 >= first && g0 - 1 <= last) atomicMax(&groupMax[groupBase + g0 - 1], m1);
        }
    }
    if (Q == 2) __syncthreads();
    team_reduce<Q == 1>(red, sh, sum, top);
    const float rstd = __frsqrt_rn(sum / (float)a.hidden + a.eps);
    if (a.rstd && live && t == 0 && part == 0) a.rstd[row] = rstd;

    if (Q == 0) {
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] *= rstd;
        const ptrdiff_t off = ((ptrdiff_t)(row * a.recvStride) + e0) * ESZ;
        for (int o = 0; o < a.nOut; o++) {
            char* p = (char*)a.recv[o] + off;
#pragma unroll
            for (int v = 0; v < V; v++)
                if (on[v]) store_vec<DT, GENERAL>(p + (ptrdiff_t)v * step * ESZ, sp[v], h[v]);
        }
        return;
    }

    // max() of the bits keeps a NaN: a row (group) with one has NaN as its scale.
    const auto amax_of = [&](uint32_t m) {
        const float f = __uint_as_float(m) * rstd;
        return f < kLeastAmax ? kLeastAmax : f;
    };
    const ptrdiff_t off = (ptrdiff_t)(row * a.recvStride) + e0;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = e0 + v * step;
        if (Q == 1) {
            const float k = rstd * (kE4m3Max / amax_of(top));
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] *= k;
        } else if (on[v]) {
            const int g0 = (e + E - 1) >> 7;
            const int gLast = groupsHere - 1;
            const float k0 = rstd * (kE4m3Max / amax_of(groupMax[groupBase + min(g0, gLast)]));
            const float k1 = GENERAL && g0 > 0 && (e >> 7) != g0 ? rstd * (kE4m3Max / amax_of(groupMax[groupBase + g0 - 1])) : k0;
#pragma unroll
            for (int j = 0; j < E; j++) h[v][j] *= GENERAL && ((e + j) >> 7) != g0 ? k1 : k0;
        }
    }
    for (int o = 0; o < a.nOut; o++) {
#pragma unroll
        for (int v = 0; v < V; v++)
            if (on[v]) store_e4m3<E>((char*)a.recv[o] + off + (ptrdiff_t)v * step, sp[v], !GENERAL || sp[v].full(E), h[v]);
    }
    if (!live) return;
    if (Q == 1) {
        if (t == 0 && part == 0)
            for (int o = 0; o < a.nOut; o++) a.scales[o][row] = amax_of(top) / kE4m3Max;
        return;
    }
    const int gFirst = clustered ? part * sh.teamThreads * V * E / kQuantGroup : 0;
    const int gEnd = clustered ? min(groupsHere, (part + 1) * sh.teamThreads * V * E / kQuantGroup) : groupsHere;
    for (int g = gFirst + t; g < gEnd; g += sh.teamThreads) {
        const float scale = amax_of(groupMax[groupBase + g]) / kE4m3Max;
        for (int o = 0; o < a.nOut; o++) a.scales[o][row * (size_t)a.groups + g] = scale;
    }
}

template <int DT, int V, int Q>
static cudaError_t norm_launch_v(const NormArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const size_t ctas = (a.rows + sh.rowsPerCta - 1) / sh.rowsPerCta * (size_t)sh.cluster;
    if (sh.general) return norm_launch(k_allreduce_rmsnorm<DT, V, true, Q>, (unsigned)ctas, sh, 0, s, a);
    return norm_launch(k_allreduce_rmsnorm<DT, V, false, Q>, (unsigned)ctas, sh, 0, s, a);
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
