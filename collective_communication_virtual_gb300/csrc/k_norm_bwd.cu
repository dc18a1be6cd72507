// k_norm_bwd.cu -- backward pass of the all-reduce + residual + RMS norm.
//
//   dy = sum_r dy_r                   (fp32, ranks in order: the all-reduce of the ranks'
//                                      partial gradients)
//   xhat = h rstd,  g = dy w,  c = sum_j g_j xhat_j / width
//   dh = rstd (g - xhat c) + dres     (rounded once; the gradient of the residual and, as h
//                                      is a plain sum, of every rank's partial sum)
//   dw_j = sum over rows of dy_j xhat_j
//
// dh needs one sum along the row, dw one down the columns.  A CTA (or cluster) strides over
// the rows and keeps its dw, in fp32; each writes its sums as one row of the workspace, and a
// second launch adds them up.  The order of the additions follows from the launch shape alone.
//
// Bound by memory: 8 ranks x 4096 x 4096 bf16 (604 MB) take 102 us, 0.87 of the measured copy
// rate (100 us without the second launch); 1 x 8192 x 2048 fp32 (268 MB) 49 us, 0.81 (45 us).
#include "norm_sums.cuh"

namespace vc {

// A row once a thread has its part: g holds dy on entry, hid the row that was normed, res the
// residual's gradient (zeros where there is none).  weight(v, f): zeros behind the row's end.
template <int DT, int V, bool GENERAL, typename Weight>
__device__ __forceinline__ void finish_row_backward(const NormBackwardArgs& a, TeamScratch& red, size_t row, bool live,
                                                    float rstd, int t, int col0, uint32_t buf, const RowVecs<DT, V>& rv,
                                                    WeightSums<DT, V>& dw, float (&g)[V][kVecElems<DT>],
                                                    const uint4 (&hid)[V], const uint4 (&res)[V], Weight weight) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const NormShape& sh = a.shape;
    float xhat[V][E];
#pragma unroll
    for (int v = 0; v < V; v++) {
        widen_vec<DT>(hid[v], xhat[v]);
        scale_by(xhat[v], rstd);
    }
    // From here on a thread holds zeros behind the row's end, and only the stores ask for it.
    if (GENERAL) {
        rv.mask(xhat);
        rv.mask(g);
    }
    float2 two[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (live) dw.add(v, g[v], xhat[v]);
        float f[E];
        weight(v, f);
        mul_by(g[v], f);
#pragma unroll
        for (int j = 0; j < E; j += 2)
            two[j / 2 & 1] = fma2(make_float2(g[v][j], g[v][j + 1]), make_float2(xhat[v][j], xhat[v][j + 1]), two[j / 2 & 1]);
    }
    float sum = (two[0].x + two[0].y) + (two[1].x + two[1].y), none = 0.0f;
    team_reduce<false>(red, sh, sum, none);
    const float c = -(sum / (float)a.width);
    const int mine = t * E;                            // the thread's first column of this CTA's
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        widen_vec<DT>(res[v], f);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 d = fma2(make_float2(xhat[v][j], xhat[v][j + 1]), make_float2(c, c),
                                  make_float2(g[v][j], g[v][j + 1]));
            const float2 r = fma2(d, make_float2(rstd, rstd), make_float2(f[j], f[j + 1]));
            g[v][j] = r.x;
            g[v][j + 1] = r.y;
        }
        if (GENERAL) st_smem(buf + (uint32_t)((mine + v * rv.step) * ESZ), narrow_vec<DT>(g[v]));
    }
    if (GENERAL) {
        if (sh.teamThreads > 32) __syncthreads();
        else __syncwarp();
        const int columns = min(a.width - col0, sh.teamThreads * V * E);
        const size_t off = (row * a.recvStride + col0) * ESZ;
        if (live) copy_out_all<ESZ>(a.recv, a.nOut, a.outSame, off, buf, columns * ESZ, t, sh.teamThreads);
        __syncwarp();                                  // a small team's buffer is free again
    } else if (live) {
        for (int o = 0; o < a.nOut; o++) {
            char* p = (char*)a.recv[o] + (row * a.recvStride + rv.e0) * ESZ;
#pragma unroll
            for (int v = 0; v < V; v++)
                if (rv.left[v] > 0) st_stream(p + (size_t)v * rv.step * ESZ, narrow_vec<DT>(g[v]));
        }
    }
}

// Few rows, or rows too long to stage: direct loads; a row may be split over a cluster.
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kNormMaxThreads, 1) k_rmsnorm_backward(const __grid_constant__ NormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int part = clustered ? (int)cluster_rank() : 0;
    const int col0 = part * sh.teamThreads * V * E;    // first column of this CTA
    if (clustered) cluster_arrive();
    WeightSums<DT, V> dw;
    dw.init(smem);
    const uint32_t buf = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(sh.extraBytes + team * sh.rowBytes);
    const RowVecs<DT, V> rv(col0 + t * E, sh.teamThreads * E, a.width);

    const size_t index = blockIdx.x / (unsigned)sh.cluster;
    const size_t stride = (size_t)(gridDim.x / (unsigned)sh.cluster) * sh.rowsPerCta;
    int flip = 0;
    // every team of a CTA runs the same number of rounds, as they share barriers
    for (size_t base = index * sh.rowsPerCta; base < a.rows; base += stride) {
        const size_t row = base + team;
        const bool live = row < a.rows;
        uint4 hid[V], res[V];
        float w[V][E];
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int e = rv.e0 + v * rv.step;
            const size_t off = (row * a.residualStride + e) * ESZ;
            hid[v] = res[v] = make_uint4(0u, 0u, 0u, 0u);
            load_weight<DT, GENERAL>(a.weight, a.weightF32, e, rv.left[v], w[v]);
            if (!live || rv.left[v] == 0) continue;
            hid[v] = load_vec<ESZ, GENERAL>((const char*)a.hidden + off, rv.left[v]);
            if (a.gradResidual) res[v] = load_vec<ESZ, GENERAL>((const char*)a.gradResidual + off, rv.left[v]);
        }
        if (GENERAL) rv.mask(w);
        const float rstd = live ? a.rstd[row] : 0.0f;
        float g[V][E];
        sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, (row * a.sendStride + rv.e0) * ESZ, live, rv, g);
        finish_row_backward<DT, V, GENERAL>(a, red[flip], row, live, rstd, t, col0, buf, rv, dw, g, hid, res,
                                            [&](int v, float (&f)[E]) {
#pragma unroll
                                                for (int j = 0; j < E; j++) f[j] = w[v][j];
                                            });
        if (clustered) cluster_arrive();
        flip ^= 1;
    }
    if (clustered) cluster_wait();
    dw.write(smem, sh, a.partials + index * a.width + col0, min(a.width - col0, sh.teamThreads * V * E));
}

// Many rows: CTAs stride over them, the next row's loads under way while one is finished.  A row
// that one CTA cannot hold is shared by the two of a cluster (8 x 2000 x 16384 bf16: 232 us, 0.75 of
// the measured copy rate, 277 with direct loads; 1 x 2000 x 16384 fp32: 121 us, 0.64, and 192).
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kStageMaxThreads, V == 1 ? 2 : 1)
k_rmsnorm_backward_staged(const __grid_constant__ NormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int N = a.nRanks, segments = N + 1 + (a.gradResidual ? 1 : 0);
    WeightSums<DT, V> dw;
    dw.init(smem);
    const uint32_t weight = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)sh.extraBytes;
    const uint32_t buf = weight + (uint32_t)(sh.weightBytes + sh.stageBytes + team * sh.rowBytes);
    const bool clustered = sh.cluster > 1;
    const int col0 = clustered ? (int)cluster_rank() * sh.teamThreads * V * E : 0;
    if (clustered) cluster_arrive();
    const RowVecs<DT, V> rv(col0 + t * E, sh.teamThreads * E, a.width);
    const StageAddr stage = stage_addr<GENERAL>(weight + (uint32_t)sh.weightBytes, sh);

    // address of a segment's element rv.e0: the ranks', the stream's, the residual's gradient
    const auto segment = [&](int s, size_t row) {
        if (s < N) return (const char*)a.send[s] + (row * a.sendStride + rv.e0) * ESZ;
        return (const char*)(s == N ? a.hidden : a.gradResidual) + (row * a.residualStride + rv.e0) * ESZ;
    };
    const auto fetch = [&](size_t row) {
        if (row < a.rows)
            for (int s = 0; s < segments; s++) stage_segment<DT, V, GENERAL>(stage, s, segment(s, row), rv);
        copies_commit();
    };
    const unsigned index = clustered ? blockIdx.x / (unsigned)sh.cluster : blockIdx.x;
    const size_t first = (size_t)index * sh.rowsPerCta, stride = (size_t)sh.ctas * sh.rowsPerCta;
    if (!GENERAL) stage_zeros<DT, V>(stage, segments, rv);
    fetch(first + team);
    float rstd = first + team < a.rows ? a.rstd[first + team] : 0.0f;
    stage_weight<DT, GENERAL>(a.weight, a.weightF32, col0, a.width, weight, sh.weightBytes);
    copies_wait();
    __syncthreads();                                   // the weight, copied by all threads
    int flip = 0;
    for (size_t base = first; base < a.rows; base += stride) {
        const size_t row = base + team;
        const float rstdNext = row + stride < a.rows ? a.rstd[row + stride] : 0.0f;
        float g[V][E];
        uint4 hid[V], res[V];
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) g[v][j] = 0.0f;
        const auto shift_of = [&](int s) { return GENERAL ? (unsigned)(uintptr_t)segment(s, row) & 15u : 0u; };
        copies_wait();
        if (GENERAL) __syncwarp();
#pragma unroll 2
        for (int s = 0; s < N; s++) add_segment<DT, V, GENERAL>(stage, s, shift_of(s), g);
        const unsigned shHid = shift_of(N), shRes = a.gradResidual ? shift_of(N + 1) : 0u;
        staged<V, GENERAL>(stage, N, shHid, hid);
#pragma unroll
        for (int v = 0; v < V; v++) res[v] = make_uint4(0u, 0u, 0u, 0u);
        if (a.gradResidual) staged<V, GENERAL>(stage, N + 1, shRes, res);
        if (GENERAL) __syncwarp();
        fetch(row + stride);
        finish_row_backward<DT, V, GENERAL>(a, red[flip], row, row < a.rows, rstd, t, col0, buf, rv, dw, g, hid, res,
                                            [&](int v, float (&f)[E]) {
                                                staged_weight<DT>(weight, a.weightF32, t * E + v * rv.step, f);
                                            });
        if (clustered) cluster_arrive();
        rstd = rstdNext;
        flip ^= 1;
    }
    if (clustered) cluster_wait();
    copies_wait();
    dw.write(smem, sh, a.partials + (size_t)index * a.width + col0, min(a.width - col0, sh.teamThreads * V * E));
}

// gradWeight[c] = sum of the partial rows' column c: 16 columns a CTA, the rows dealt to 32
// groups of its threads, whose sums are added in a fixed order.  CTAs of 512 threads: they become
// resident while the pass above still runs, and larger ones take the place of its next launch's.
constexpr int kSumColumns = 16;
constexpr int kSumGroups = 32;
constexpr int kSumThreads = kSumColumns * kSumGroups;
template <int DT>
__global__ void __launch_bounds__(kSumThreads) k_sum_columns(const float* partials, int rows, int width, void* out) {
    pdl_begin();
    __shared__ float part[kSumGroups][kSumColumns + 1];
    const int x = threadIdx.x % kSumColumns, y = threadIdx.x / kSumColumns;
    const int c = blockIdx.x * kSumColumns + x;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 8
        for (int r = y; r < rows; r += kSumGroups) s += partials[(size_t)r * width + c];
    }
    part[y][x] = s;
    __syncthreads();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s = part[lane][w];                                 // warp w: column w's 32 sums
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    const int cw = blockIdx.x * kSumColumns + w;
    if (lane == 0 && cw < width) st_elem<DTypeOf<DT>::size>(out, cw, f32_to_elem<DT>(s));
}
static_assert(kSumThreads / 32 == kSumColumns, "one warp per column");

template <int DT, int V, bool GENERAL>
static cudaError_t bwd_launch(const NormBackwardArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const cudaError_t e = sh.staged ? allow_smem(k_rmsnorm_backward_staged<DT, V, GENERAL>, sh.smemBytes)
                                    : allow_smem(k_rmsnorm_backward<DT, V, GENERAL>, sh.smemBytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(a.parts * sh.cluster);
    if (sh.staged) return norm_launch(k_rmsnorm_backward_staged<DT, V, GENERAL>, grid, sh, sh.smemBytes, s, a);
    return norm_launch(k_rmsnorm_backward<DT, V, GENERAL>, grid, sh, sh.smemBytes, s, a);
}
template <int DT>
static cudaError_t bwd_launch_dt(const NormBackwardArgs& a, cudaStream_t s) {
    cudaError_t e;
    const bool g = a.shape.general != 0;
    switch (a.shape.vecs) {
    case 1: e = g ? bwd_launch<DT, 1, true>(a, s) : bwd_launch<DT, 1, false>(a, s); break;
    case 2: e = g ? bwd_launch<DT, 2, true>(a, s) : bwd_launch<DT, 2, false>(a, s); break;
    default: e = g ? bwd_launch<DT, 4, true>(a, s) : bwd_launch<DT, 4, false>(a, s); break;
    }
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((a.width + kSumColumns - 1) / kSumColumns);
    if (a.weightF32)
        return pdl_launch(k_sum_columns<kF32>, grid, kSumThreads, 0, s, (const float*)a.partials, a.parts, a.width,
                          a.gradWeight);
    return pdl_launch(k_sum_columns<DT>, grid, kSumThreads, 0, s, (const float*)a.partials, a.parts, a.width,
                      a.gradWeight);
}

cudaError_t launch_rmsnorm_backward(const NormBackwardArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return bwd_launch_dt<kF32>(a, s);
    case vFloat16: return bwd_launch_dt<kF16>(a, s);
    case vBFloat16: return bwd_launch_dt<kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
