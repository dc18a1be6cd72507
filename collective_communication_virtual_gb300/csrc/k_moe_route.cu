// k_moe_route.cu -- the router of a mixture of experts: logits, the topK best experts of every token
// and their weights.
//
//   l_te = sum_j x_tj router_ej,  score = l + bias
//   ids = the topK largest scores of the token, largest first, ties to the lower index
//   weight = exp(l_id) / sum of exp(l) over the chosen, or over all experts
//
// Two experts' scores may lie next to one another, and the choice between them is an integer.  So the
// logits come with a bound on their error: eight products at a time are added in fp32, at most 8 u of
// their magnitudes off (u = 2^-24), their sums as a value and its rounding error, and the lanes' sums
// in fp64.  Where that leaves open which of two scores is the larger, and one of the two is chosen,
// both logits are computed anew with every product and sum as a value and its error, some 2^-45 of the
// magnitudes off.
//
// A cluster of CTAs takes up to eight tokens, each CTA a share of the experts, a warp one expert at a
// time for all the tokens; the first CTA gathers the logits and picks, one warp a token.
#include "moe.h"
#include "norm.cuh"

namespace vc {

namespace {

// E consecutive values of a row from element e on, `left` of them inside the row (the rest zero).
template <int DT, int E, bool ALIGNED>
__device__ __forceinline__ void load_row(const void* row, int e, int left, float (&f)[E]) {
    constexpr int ESZ = DTypeOf<DT>::size, PER = 16 / ESZ;
    if (ALIGNED) {
#pragma unroll
        for (int i = 0; i < E; i += PER) {
            float part[PER];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (i < left) v = *reinterpret_cast<const uint4*>((const char*)row + (size_t)(e + i) * ESZ);
            widen_vec<DT>(v, part);
#pragma unroll
            for (int j = 0; j < PER; j++) f[i + j] = part[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i++) {
            f[i] = 0.0f;
            if (i >= left) continue;
            if (DT == kF32) f[i] = ((const float*)row)[e + i];
            else f[i] = widen16<DT>(((const uint16_t*)row)[e + i]);
        }
    }
}

// s + c stays the sum of everything added, c what s's roundings lost.
__device__ __forceinline__ void add_exactly(float& s, float& c, float x) {
    const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}

// The order of the choice: larger scores first, then lower indices; a NaN comes last.
__device__ __forceinline__ bool before(double a, int i, double b, int j) {
    const bool na = a != a, nb = b != b;
    if (na || nb) return na == nb ? i < j : nb;
    return a > b || (a == b && i < j);
}

// A logit by one warp, error-free products added error-free.
template <int DT, int WT, bool ALIGNED>
__device__ __noinline__ double exact_logit(const char* x, const char* w, int hidden) {
    constexpr int E = 8;
    const int lane = threadIdx.x & 31;
    float s = 0.0f, c = 0.0f;
    for (int j = lane * E; j < hidden; j += 32 * E) {
        float f[E], v[E];
        const int left = min(E, hidden - j);
        load_row<WT, E, ALIGNED>(w, j, left, f);
        load_row<DT, E, ALIGNED>(x, j, left, v);
#pragma unroll
        for (int i = 0; i < E; i++) {
            const float p = __fmul_rn(v[i], f[i]);
            add_exactly(s, c, p);
            c = __fadd_rn(c, __fmaf_rn(v[i], f[i], -p));
        }
    }
    double l = isfinite(s) ? (double)s + (double)c : (double)s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    return l;
}

template <int DT, int WT, int TOKENS, bool ALIGNED>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const __grid_constant__ RouteArgs a) {
    pdl_begin();
    constexpr int E = 8;
    extern __shared__ __align__(16) double logits[];   // of the first CTA: [TOKENS][experts]
    float* const errors = reinterpret_cast<float*>(logits + (size_t)TOKENS * a.experts);     // the same
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRouteThreads / 32;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    const int row0 = (int)(blockIdx.x / (unsigned)a.cluster) * TOKENS;
    if (a.cluster > 1) {
        cluster_arrive();
        cluster_wait();                                // every CTA of the cluster has started
    }
    const int last = min(a.experts, (rank + 1) * a.share);
    for (int e = rank * a.share + warp; e < last; e += warps) {
        const char* w = (const char*)a.router + (size_t)e * a.hidden * DTypeOf<WT>::size;
        float s[TOKENS], c[TOKENS], m[TOKENS];         // m: the products' magnitudes
#pragma unroll
        for (int t = 0; t < TOKENS; t++) s[t] = c[t] = m[t] = 0.0f;
#pragma unroll 2
        for (int j = lane * E; j < a.hidden; j += 32 * E) {
            float f[E];
            const int left = min(E, a.hidden - j);
            load_row<WT, E, ALIGNED>(w, j, left, f);
#pragma unroll
            for (int t = 0; t < TOKENS; t++) {
                const int row = min(row0 + t, a.rows - 1);
                float x[E];
                load_row<DT, E, ALIGNED>((const char*)a.x + (size_t)row * a.rowStride * DTypeOf<DT>::size, j, left, x);
                float p = x[0] * f[0];
#pragma unroll
                for (int i = 1; i < E; i++) p = fmaf(x[i], f[i], p);
#pragma unroll
                for (int i = 0; i < E; i++) m[t] = fmaf(fabsf(x[i]), fabsf(f[i]), m[t]);
                add_exactly(s[t], c[t], p);
            }
        }
#pragma unroll
        for (int t = 0; t < TOKENS; t++) {
            double l = isfinite(s[t]) ? (double)s[t] + (double)c[t] : (double)s[t];
            float off = m[t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                l += __shfl_xor_sync(~0u, l, o);
                off += __shfl_xor_sync(~0u, off, o);
            }
            if (lane != 0) continue;
            off *= 10 * 5.9604644775390625e-8f;        // 8 u, with room for the roundings of m itself
            const size_t at = (size_t)t * a.experts + e;
            if (a.cluster == 1) {
                logits[at] = l;
                errors[at] = off;
            } else {
                const unsigned long long bits = (unsigned long long)__double_as_longlong(l);
                st_cluster(logits + at, 0, (uint32_t)bits);
                st_cluster((const char*)(logits + at) + 4, 0, (uint32_t)(bits >> 32));
                st_cluster(errors + at, 0, __float_as_uint(off));
            }
        }
    }
    if (a.cluster > 1) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // One warp a token.  Each choice is the first in the order of all that come behind the one before.
    for (int t = warp; t < TOKENS; t += warps) {
        const int row = row0 + t;
        if (row >= a.rows) break;
        double* const l = logits + (size_t)t * a.experts;
        float* const error = errors + (size_t)t * a.experts;
        const auto score_of = [&](int e) { return a.bias ? l[e] + (double)a.bias[e] : l[e]; };
        double mine;                                   // lane k: the logit of choice k
        int id;
        for (bool again = true; again;) {
            again = false;
            mine = 0.0;
            id = 0;
            double lastScore = 0.0;
            int lastId = -1;
            for (int k = 0; k < a.topK; k++) {
                double best = 0.0;
                int at = -1;
                for (int e = lane; e < a.experts; e += 32) {
                    const double score = score_of(e);
                    if (lastId >= 0 && !before(lastScore, lastId, score, e)) continue;
                    if (at < 0 || before(score, e, best, at)) {
                        best = score;
                        at = e;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const double other = __shfl_xor_sync(~0u, best, o);
                    const int i = __shfl_xor_sync(~0u, at, o);
                    if (i >= 0 && (at < 0 || before(other, i, best, at))) {
                        best = other;
                        at = i;
                    }
                }
                lastScore = best;
                lastId = at;
                if (lane == k) {
                    id = at;
                    mine = l[at];
                }
            }
            // Scores that may change places with a chosen one: their logits anew, and the choice too.
            // An error of 0 marks a logit that is as good as it gets.
            for (int k = 0; k < a.topK; k++) {
                const int c = __shfl_sync(~0u, id, k);
                bool unsure = false;
                for (int e0 = 0; e0 < a.experts; e0 += 32) {
                    const int e = e0 + lane;
                    const float both = e < a.experts && e != c ? error[e] + error[c] : 0.0f;
                    const bool near = both > 0.0f && fabs(score_of(min(e, a.experts - 1)) - score_of(c)) <= (double)both;
                    unsure = unsure || near;
                    for (unsigned todo = __ballot_sync(~0u, near && error[e] > 0.0f); todo; todo &= todo - 1) {
                        const int i = e0 + __ffs(todo) - 1;
                        const double better = exact_logit<DT, WT, ALIGNED>(
                            (const char*)a.x + (size_t)row * a.rowStride * DTypeOf<DT>::size,
                            (const char*)a.router + (size_t)i * a.hidden * DTypeOf<WT>::size, a.hidden);
                        if (lane == 0) {
                            l[i] = better;
                            error[i] = 0.0f;
                        }
                        __syncwarp();
                    }
                }
                if (!__any_sync(~0u, unsure)) continue;
                again = true;
                if (error[c] > 0.0f) {
                    const double better = exact_logit<DT, WT, ALIGNED>(
                        (const char*)a.x + (size_t)row * a.rowStride * DTypeOf<DT>::size,
                        (const char*)a.router + (size_t)c * a.hidden * DTypeOf<WT>::size, a.hidden);
                    __syncwarp();
                    if (lane == 0) {
                        l[c] = better;
                        error[c] = 0.0f;
                    }
                }
                __syncwarp();
            }
        }
        // the largest chosen logit, and the sum that the weights are shares of
        double top = lane < a.topK ? mine : -INFINITY, sum = 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double other = __shfl_xor_sync(~0u, top, o);
            top = other > top || other != other ? other : top;
        }
        if (a.normalize) {
            sum = lane < a.topK ? (double)expf((float)(mine - top)) : 0.0;
        } else {
            for (int e = lane; e < a.experts; e += 32) sum += exp(l[e] - top);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane < a.topK) {
            a.ids[(size_t)row * a.topK + lane] = id;
            a.weights[(size_t)row * a.topK + lane] = (float)((double)expf((float)(mine - top)) / sum);
        }
    }
}

template <int DT, int WT, int TOKENS>
cudaError_t route_launch(const RouteArgs& a, cudaStream_t s) {
    const auto kernel = a.aligned ? k_moe_route<DT, WT, TOKENS, true> : k_moe_route<DT, WT, TOKENS, false>;
    const size_t smem = (size_t)TOKENS * a.experts * (sizeof(double) + sizeof(float));
    if (smem > 32 * 1024) {
        // one value for every launch, as host threads share the kernel's limit
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kRouteTokens * VCOMM_MAX_EXPERTS * (int)(sizeof(double) + sizeof(float)));
        if (e != cudaSuccess) return e;
    }
    NormShape sh = {};
    sh.threads = kRouteThreads;
    sh.cluster = a.cluster;
    return norm_launch(kernel, (unsigned)((a.rows + TOKENS - 1) / TOKENS * a.cluster), sh, smem, s, a);
}
template <int DT, int WT>
cudaError_t route_launch_t(const RouteArgs& a, cudaStream_t s) {
    switch (a.tokens) {
    case 1: return route_launch<DT, WT, 1>(a, s);
    case 2: return route_launch<DT, WT, 2>(a, s);
    case 4: return route_launch<DT, WT, 4>(a, s);
    default: return route_launch<DT, WT, 8>(a, s);
    }
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return route_launch_t<kF32, kF32>(a, s);
    case vFloat16: return a.routerF32 ? route_launch_t<kF16, kF32>(a, s) : route_launch_t<kF16, kF16>(a, s);
    case vBFloat16: return a.routerF32 ? route_launch_t<kBF16, kF32>(a, s) : route_launch_t<kBF16, kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
