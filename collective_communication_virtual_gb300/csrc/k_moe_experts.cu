// k_moe_experts.cu -- the experts' layer of a mixture of experts for a few tokens in fp32, the experts
// split over the ranks.
//
//   g = Wgate_e x_t,  u = Wlinear_e x_t,  a = silu(g) u,  silu(g) = g / (1 + exp(-g))
//   recv_r[t] = sum over the token's chosen experts e of rank r of weight_te Wdown_e a
//
// Two launches: the way up (a of every slot, a slot being one choice of one token, into the
// workspace) and the way down, whose last CTA of a tile of columns adds up every token's slots, in
// their order, for every rank.  A CTA takes one expert and a tile of output rows, finds the expert's
// slots in the router's list, and leaves at once if there are none.  A warp takes rows of the weights,
// one 16-byte vector a lane, against up to eight slots at a time.
//
// No tensor cores: theirs would round the factors to 11 bits.  16 tokens on 2 of 16 experts of 2048 x 1024
// take 128 us (355 MB, 2.8 TB/s: ten 16-byte loads a lane for 64 multiply-adds, which keep the load pipe busy),
// one token 31 us.
#include "moe.h"
#include "norm.cuh"

namespace vc {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;            // slots that a warp takes at once
constexpr int kRows = 2;             // rows of the weights that it takes at once
constexpr int kList = 1024;          // slots found before they are worked on

// The slots of expert e, in order, from position `from` on: fills `list` until it may be full, and
// returns where to go on (>= total: all found).  All threads of the CTA call it.
__device__ __forceinline__ int find_slots(const int* ids, int total, int e, int from, int* list, int* count) {
    __shared__ int perWarp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    while (from < total && n + kThreads <= kList) {
        const int i = from + (int)threadIdx.x;
        const bool hit = i < total && ids[i] == e;
        const unsigned in = __ballot_sync(~0u, hit);
        if (lane == 0) perWarp[warp] = __popc(in);
        __syncthreads();
        int at = n;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) at += perWarp[w];
            n += perWarp[w];
        }
        if (hit) list[at + __popc(in & ((1u << lane) - 1))] = i;
        from += kThreads;
        __syncthreads();
    }
    *count = n;
    return from;
}

// A lane's elements of one step along a row: ALIGNED a 16-byte vector from j on, else j + 32 i.
template <bool ALIGNED> constexpr int kElems = ALIGNED ? 4 : 8;
template <bool ALIGNED>
__device__ __forceinline__ void load_part(const float* row, int j, int width, float (&f)[kElems<ALIGNED>]) {
    if constexpr (ALIGNED) {
        widen_vec<kF32>(*reinterpret_cast<const uint4*>(row + j), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int e = j + 32 * i;
            f[i] = e < width ? row[e] : 0.0f;
        }
    }
}

// Dot products of R rows of the weights with n <= G vectors; every lane ends with all of them.
template <bool ALIGNED, int R, int G>
__device__ __forceinline__ void dots(const float* const (&w)[R], const float* const (&x)[G], int n, int width, float (&acc)[R][G]) {
    constexpr int E = kElems<ALIGNED>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int g = 0; g < G; g++) acc[r][g] = 0.0f;
    for (int j = ALIGNED ? lane * E : lane; j < width; j += 32 * E) {
        float f[R][E];
#pragma unroll
        for (int r = 0; r < R; r++) load_part<ALIGNED>(w[r], j, width, f[r]);
#pragma unroll
        for (int g = 0; g < G; g++) {
            if (g >= n) break;
            float v[E];
            load_part<ALIGNED>(x[g], j, width, v);
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int i = 0; i < E; i++) acc[r][g] = fmaf(f[r][i], v[i], acc[r][g]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[r][g] += __shfl_xor_sync(~0u, acc[r][g], o);
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_moe_up(const __grid_constant__ ExpertsArgs a) {
    pdl_begin();
    __shared__ int list[kList];
    const int e = (int)blockIdx.y, total = a.rows * a.topK;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && e == 0)
        for (int i = threadIdx.x; i < (a.hidden + a.tileDown - 1) / a.tileDown; i += kThreads) a.done[i] = 0;
    const float* base = (const float*)a.up[e / a.share] + (size_t)(e % a.share) * 2 * a.ffn * a.hidden;
    const int f0 = (int)blockIdx.x * a.tileUp, f1 = min(a.ffn, f0 + a.tileUp);
    for (int from = 0, n; from < total;) {
        from = find_slots(a.ids, total, e, from, list, &n);
        for (int g0 = 0; g0 < n; g0 += kGroup) {
            const int some = min(kGroup, n - g0);
            const float* x[kGroup];
#pragma unroll
            for (int g = 0; g < kGroup; g++)
                x[g] = (const float*)a.x + (size_t)(list[g0 + min(g, some - 1)] / a.topK) * a.rowStride;
            for (int f = f0 + warp; f < f1; f += kWarps) {
                const float* const w[kRows] = {base + (size_t)f * a.hidden, base + (size_t)(a.ffn + f) * a.hidden};
                float acc[kRows][kGroup];
                dots<ALIGNED>(w, x, some, a.hidden, acc);
#pragma unroll
                for (int g = 0; g < kGroup; g++) {
                    if (lane != g || g >= some) continue;
                    a.act[(size_t)list[g0 + g] * a.ffn + f] = acc[0][g] / (1.0f + expf(-acc[0][g])) * acc[1][g];
                }
            }
        }
        __syncthreads();
    }
}

// Columns [h0, h1) of every rank's output, from all slots' y.  What up to eight slots need is loaded
// together, whether it counts or not: the wait for memory is most of this.
__device__ __forceinline__ void combine(const ExpertsArgs& a, int h0, int h1) {
    constexpr int UN = 8;
    const int columns = h1 - h0;
    for (int i = threadIdx.x; i < a.rows * columns; i += kThreads) {
        const int t = i / columns, h = h0 + i % columns;
        for (int r0 = 0; r0 < a.nRanks; r0 = a.topK <= UN ? a.nRanks : r0 + 1) {
            // all ranks from one set of loads, or (more slots) a rank at a time
            float s = 0.0f;
            for (int k0 = 0; k0 < a.topK; k0 += UN) {
                int rank[UN];
                float w[UN], y[UN];
#pragma unroll
                for (int k = 0; k < UN; k++) {
                    const size_t slot = (size_t)t * a.topK + min(k0 + k, a.topK - 1);
                    const int e = a.ids[slot];
                    w[k] = a.weights[slot];
                    y[k] = __ldcg(a.y + slot * a.hidden + h);
                    rank[k] = k0 + k < a.topK && e >= 0 && e < a.experts ? e / a.share : -1;
                }
                for (int r = r0; r < (a.topK <= UN ? a.nRanks : r0 + 1); r++) {
                    if (k0 == 0) s = 0.0f;
#pragma unroll
                    for (int k = 0; k < UN; k++) s = rank[k] == r ? fmaf(w[k], y[k], s) : s;
                    if (k0 + UN >= a.topK) ((float*)a.recv[r])[(size_t)t * a.recvStride + h] = s;
                }
            }
        }
    }
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_moe_down(const __grid_constant__ ExpertsArgs a) {
    pdl_begin();
    __shared__ int list[kList];
    __shared__ unsigned seen[VCOMM_MAX_EXPERTS / 32];
    __shared__ int last;
    const int e = (int)blockIdx.y, total = a.rows * a.topK;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h0 = (int)blockIdx.x * a.tileDown, h1 = min(a.hidden, h0 + a.tileDown);
    const float* base = (const float*)a.down[e / a.share] + (size_t)(e % a.share) * a.hidden * a.ffn;
    int found = 0;
    for (int from = 0, n; from < total;) {
        from = find_slots(a.ids, total, e, from, list, &n);
        found += n;
        for (int g0 = 0; g0 < n; g0 += kGroup) {
            const int some = min(kGroup, n - g0);
            const float* x[kGroup];
#pragma unroll
            for (int g = 0; g < kGroup; g++) x[g] = a.act + (size_t)list[g0 + min(g, some - 1)] * a.ffn;
            for (int h = h0 + kRows * warp; h < h1; h += kRows * kWarps) {
                const float* const w[kRows] = {base + (size_t)h * a.ffn, base + (size_t)min(h + 1, h1 - 1) * a.ffn};
                float acc[kRows][kGroup];
                dots<ALIGNED>(w, x, some, a.ffn, acc);
#pragma unroll
                for (int g = 0; g < kGroup; g++) {
                    if (lane != g || g >= some) continue;
#pragma unroll
                    for (int r = 0; r < kRows; r++)
                        if (h + r < h1) a.y[(size_t)list[g0 + g] * a.hidden + h + r] = acc[r][g];
                }
            }
        }
        __syncthreads();
    }
    // The experts that some slot names; where there are none, the first CTA writes the zeros.
    for (int i = threadIdx.x; i < VCOMM_MAX_EXPERTS / 32; i += kThreads) seen[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int id = a.ids[i];
        if (id >= 0 && id < a.experts) atomicOr(&seen[id / 32], 1u << (id % 32));
    }
    __syncthreads();
    int active = 0;
    for (int i = 0; i < VCOMM_MAX_EXPERTS / 32; i++) active += __popc(seen[i]);
    if (found == 0 && !(active == 0 && e == 0)) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = active == 0 || atomicAdd(&a.done[blockIdx.x], 1u) == (unsigned)active - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    combine(a, h0, h1);
}

template <bool ALIGNED>
cudaError_t experts_launch(const ExpertsArgs& a, cudaStream_t s) {
    const auto run = [&](auto kernel, int columns, int tile) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((columns + tile - 1) / tile), (unsigned)a.experts);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pdl_enabled() ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, kernel, a);
    };
    const cudaError_t e = run(k_moe_up<ALIGNED>, a.ffn, a.tileUp);
    return e != cudaSuccess ? e : run(k_moe_down<ALIGNED>, a.hidden, a.tileDown);
}

}  // namespace

cudaError_t launch_moe_experts(const ExpertsArgs& a, cudaStream_t s) {
    return a.aligned ? experts_launch<true>(a, s) : experts_launch<false>(a, s);
}

}  // namespace vc
