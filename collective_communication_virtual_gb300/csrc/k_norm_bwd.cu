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
// the rows and keeps its dw in shared memory, in fp32; each writes its sums as one row of the
// workspace, and a second launch adds those rows up.  No atomics: the order of the additions
// follows from the shapes alone.
#include "norm_stage.cuh"

namespace vc {

// A CTA's dw in shared memory.  Aligned rows: a thread holds the same columns of every row, so
// its sums are its own (float4 number (v E/4 + j/4) threads + thread).  GENERAL: a row's shift
// moves its columns among the threads of its team, and column c is at [c % E][c / E] of the
// team, so that the lanes of a warp touch neighbouring words; the barrier (or __syncwarp) of
// each row's reduction orders the additions to a column.
template <int DT, int V, bool GENERAL>
struct WeightSums {
    static constexpr int E = kVecElems<DT>;
    float* all;
    int slots;                       // vectors of a team's part of a row
    __device__ __forceinline__ void init(float* smem, const NormShape& sh) {
        all = smem;
        slots = sh.teamThreads * V;
        for (int i = threadIdx.x; i < slots * E * sh.rowsPerCta; i += blockDim.x) all[i] = 0.0f;
    }
    // dw += dy * xhat for vector v, whose first element is column e of this CTA's part
    __device__ __forceinline__ void add(int team, int v, int e, Span sp, const float (&dy)[E], const float (&xhat)[E]) {
        if (!GENERAL) {
            float4* p = reinterpret_cast<float4*>(all) + (size_t)v * (E / 4) * blockDim.x + threadIdx.x;
#pragma unroll
            for (int i = 0; i < E / 4; i++) {
                float4 s = p[i * blockDim.x];
                const float2 lo = fma2(make_float2(dy[4 * i], dy[4 * i + 1]), make_float2(xhat[4 * i], xhat[4 * i + 1]),
                                       make_float2(s.x, s.y));
                const float2 hi = fma2(make_float2(dy[4 * i + 2], dy[4 * i + 3]),
                                       make_float2(xhat[4 * i + 2], xhat[4 * i + 3]), make_float2(s.z, s.w));
                p[i * blockDim.x] = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
            return;
        }
        float* mine = all + (size_t)team * slots * E;
#pragma unroll
        for (int j = 0; j < E; j++) {
            if (!sp.has(j)) continue;
            float* p = &mine[((e + j) & (E - 1)) * slots + (e + j) / E];
            *p = fmaf(dy[j], xhat[j], *p);
        }
    }
    // One row of sums per CTA: its teams' in order.
    __device__ __forceinline__ void write(const NormShape& sh, float* out, int columns) const {
        for (int c = threadIdx.x; c < columns; c += blockDim.x) {
            float s = 0.0f;
            for (int k = 0; k < sh.rowsPerCta; k++) {
                if (GENERAL) {
                    s += all[(size_t)k * slots * E + (c & (E - 1)) * slots + c / E];
                } else {
                    const int vec = c / E, j = c & (E - 1);
                    const int v = vec / sh.teamThreads, t = vec - v * sh.teamThreads;
                    s += all[(((size_t)v * (E / 4) + j / 4) * blockDim.x + k * sh.teamThreads + t) * 4 + (j & 3)];
                }
            }
            out[c] = s;
        }
    }
};

// A row once a thread has its part: g holds dy on entry, hid the row that was normed, res the
// residual's gradient.
template <int DT, int V, bool GENERAL, typename Weight>
__device__ __forceinline__ void finish_row_backward(const NormBackwardArgs& a, TeamScratch& red, size_t row, float rstd,
                                                    bool live, int t, int team, int col0, uint32_t rowBuf,
                                                    const RowVecs<DT, V>& rv,
                                                    WeightSums<DT, V, GENERAL>& dw, float (&g)[V][kVecElems<DT>],
                                                    const uint4 (&hid)[V], const uint4 (&res)[V], Weight weight) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    // Vectors outside the row hold zeros from here on, and only the stores ask for them.
    float2 two = make_float2(0.0f, 0.0f);
    float xhat[V][E];
#pragma unroll
    for (int v = 0; v < V; v++) {
        widen_vec<DT>(hid[v], xhat[v]);
        scale_by(xhat[v], rstd);
    }
    if (GENERAL) {
        rv.mask(xhat);
        rv.mask(g);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (GENERAL ? rv.on[v] : live) dw.add(team, v, rv.e0 + v * rv.step - col0, rv.sp[v], g[v], xhat[v]);
        float f[E];
        weight(v, f);
        mul_by(g[v], f);
    }
    if (GENERAL) rv.mask(g);                           // the weight outside the row is undefined
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int j = 0; j < E; j += 2)
            two = fma2(make_float2(g[v][j], g[v][j + 1]), make_float2(xhat[v][j], xhat[v][j + 1]), two);
    float sum = two.x + two.y;
    float none = 0.0f;
    if (GENERAL) __syncwarp();
    team_reduce<false>(red, a.shape, sum, none);
    const float c = -(sum / (float)a.width);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        if (a.gradResidual) {
            widen_vec<DT>(res[v], f);
        } else {
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 d = fma2(make_float2(xhat[v][j], xhat[v][j + 1]), make_float2(c, c),
                                  make_float2(g[v][j], g[v][j + 1]));
            const float2 r = fma2(d, make_float2(rstd, rstd), make_float2(f[j], f[j + 1]));
            g[v][j] = r.x;
            g[v][j + 1] = r.y;
        }
    }
    const ptrdiff_t off = ((ptrdiff_t)(row * a.recvStride) + rv.e0) * ESZ;
    if (GENERAL && rowBuf) {
#pragma unroll
        for (int v = 0; v < V; v++)
            st_smem(rowBuf + (uint32_t)(v * a.shape.teamThreads + t) * 16u, narrow_vec<DT>(g[v]));
        if (a.shape.teamThreads > 32) __syncthreads();
        else __syncwarp();
    }
    for (int o = 0; o < a.nOut; o++) {
        char* p = (char*)a.recv[o] + off;
        if (GENERAL && rowBuf && ((uintptr_t)p & 15u)) {
            const int columns = min(a.width - col0, a.shape.cluster > 1 ? a.shape.teamThreads * V * E : a.width);
            if (live)
                copy_out<ESZ>((char*)a.recv[o] + ((ptrdiff_t)(row * a.recvStride) + col0) * ESZ,
                              rowBuf + (uint32_t)((col0 + t * E - rv.e0) * ESZ), columns * ESZ, t, a.shape.teamThreads);
            continue;
        }
#pragma unroll
        for (int v = 0; v < V; v++)
            if (rv.on[v]) store_vec<DT, GENERAL>(p + (ptrdiff_t)v * rv.step * ESZ, rv.sp[v], g[v]);
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
    WeightSums<DT, V, GENERAL> dw;
    dw.init(reinterpret_cast<float*>(smem), sh);
    __syncthreads();
    const uint32_t rowBuf = GENERAL && sh.rowBytes ? (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)sh.extraBytes +
                                                         (uint32_t)(team * sh.rowBytes) : 0u;

    const size_t index = blockIdx.x / (unsigned)sh.cluster;
    const size_t stride = (size_t)(gridDim.x / (unsigned)sh.cluster) * sh.rowsPerCta;
    int flip = 0;
    // every team of a CTA runs the same number of rounds, as they share barriers
    for (size_t base = index * sh.rowsPerCta; base < a.rows; base += stride) {
        const size_t row = base + team;
        const bool live = row < a.rows;
        int shift = 0;
        if (GENERAL && live && !clustered)
            shift = (int)(((uintptr_t)a.recv[0] + row * a.recvStride * ESZ) & 15u) / ESZ;
        RowVecs<DT, V> rv;
        rv.set(col0 + t * E - shift, sh.teamThreads * E, a.width, live);
        uint4 hid[V], res[V];
        WeightVec<DT> w[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
            hid[v] = res[v] = make_uint4(0u, 0u, 0u, 0u);
            if (!rv.on[v]) continue;
            const int e = rv.e0 + v * rv.step;
            const ptrdiff_t off = ((ptrdiff_t)(row * a.residualStride) + e) * ESZ;
            hid[v] = load_vec<ESZ, GENERAL>((const char*)a.hidden + off, rv.sp[v]);
            if (a.gradResidual) res[v] = load_vec<ESZ, GENERAL>((const char*)a.gradResidual + off, rv.sp[v]);
            w[v].template load<GENERAL>(a.weight, a.weightF32, e, rv.sp[v]);
        }
        const float rstd = live ? a.rstd[row] : 0.0f;
        float g[V][E];
        sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, ((ptrdiff_t)(row * a.sendStride) + rv.e0) * ESZ, rv, g);
        finish_row_backward<DT, V, GENERAL>(a, red[flip], row, rstd, live, t, team, col0, rowBuf, rv, dw, g, hid, res,
                                            [&](int v, float (&f)[E]) {
                                                if (rv.on[v]) {
                                                    w[v].get(a.weightF32, f);
                                                } else {
#pragma unroll
                                                    for (int j = 0; j < E; j++) f[j] = 0.0f;
                                                }
                                            });
        if (clustered) cluster_arrive();
        flip ^= 1;
    }
    if (clustered) cluster_wait();
    __syncthreads();
    dw.write(sh, a.partials + index * a.width + col0, min(dw.slots * E, a.width - col0));
}

// Many rows: the next row's loads are under way while one is finished.
template <int V> constexpr int staged_backward_min_ctas() { return V == 1 ? 2 : 1; }
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kStageMaxThreads, staged_backward_min_ctas<V>())
k_rmsnorm_backward_staged(const __grid_constant__ NormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int N = a.nRanks;
    const int segments = N + 1 + (a.gradResidual ? 1 : 0);
    WeightSums<DT, V, GENERAL> dw;
    dw.init(reinterpret_cast<float*>(smem), sh);
    const uint32_t base0 = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)sh.extraBytes;
    StageAddr stage;
    stage.pitch = blockDim.x * 16u;
    stage.base = base0 + (uint32_t)sh.weightBytes + threadIdx.x * 16u;
    stage.second = (uint32_t)segments * V * stage.pitch;
    const WeightSmem ws = stage_weight(a.weight, a.weightF32, a.weightF32 ? 4 : ESZ, a.width, base0,
                                       sh.weightBytes);
    const uint32_t rowBuf = GENERAL && sh.rowBytes
                                ? base0 + (uint32_t)(sh.weightBytes + sh.stageBytes + team * sh.rowBytes) : 0u;

    const auto frame = [&](size_t row, RowVecs<DT, V>& rv) {
        const bool live = row < a.rows;
        const int shift = GENERAL && live ? (int)(((uintptr_t)a.recv[0] + row * a.recvStride * ESZ) & 15u) / ESZ : 0;
        rv.set(t * E - shift, sh.teamThreads * E, a.width, live);
    };
    // address of a segment's element e0: the ranks', the stream's, the residual's gradient
    const auto segment = [&](int s, size_t row, int e0) {
        if (s < N) return (const char*)a.send[s] + ((ptrdiff_t)(row * a.sendStride) + e0) * ESZ;
        return (const char*)(s == N ? a.hidden : a.gradResidual) + ((ptrdiff_t)(row * a.residualStride) + e0) * ESZ;
    };
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
    float rstd = first + team < a.rows ? a.rstd[first + team] : 0.0f;
    copies_wait();
    __syncthreads();                                   // the weight has been copied, by all threads
    int flip = 0;
    for (size_t base = first; base < a.rows; base += stride) {
        const size_t row = base + team;
        RowVecs<DT, V> rv;
        frame(row, rv);
        const float rstdNext = row + stride < a.rows ? a.rstd[row + stride] : 0.0f;
        float g[V][E];
        uint4 hid[V], res[V];
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) g[v][j] = 0.0f;
        const auto shift_of = [&](int s) { return GENERAL ? (unsigned)(uintptr_t)segment(s, row, rv.e0) & 15u : 0u; };
        copies_wait();
#pragma unroll 2
        for (int s = 0; s < N; s++) add_segment<DT, V, GENERAL>(stage, s, shift_of(s), rv, g);
        const unsigned shHid = shift_of(N), shRes = a.gradResidual ? shift_of(N + 1) : 0u;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (GENERAL && !rv.on[v]) continue;
            hid[v] = staged<DT, V, GENERAL>(stage, N, v, shHid);
            if (a.gradResidual) res[v] = staged<DT, V, GENERAL>(stage, N + 1, v, shRes);
        }
        fetch(row + stride);
        finish_row_backward<DT, V, GENERAL>(a, red[flip], row, rstd, row < a.rows, t, team, 0, rowBuf, rv, dw, g, hid, res,
                                            [&](int v, float (&f)[E]) {
                                                weight_vec<DT, GENERAL>(ws, rv.e0 + v * rv.step, f);
                                            });
        rstd = rstdNext;
        flip ^= 1;
    }
    copies_wait();
    __syncthreads();
    dw.write(sh, a.partials + (size_t)blockIdx.x * a.width, a.width);
}

// gradWeight[c] = sum of the partial rows' column c: 32 columns a CTA, the rows dealt to its
// 32 warps and their sums added in warp order.
constexpr int kSumThreads = 1024;
template <int DT>
__global__ void __launch_bounds__(kSumThreads) k_sum_columns(const float* partials, int rows, int width, void* out) {
    pdl_begin();
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < width)
        for (int r = y; r < rows; r += 32) s += partials[(size_t)r * width + c];
    part[y][x] = s;
    __syncthreads();
    s = part[x][y];                                    // warp y: column y's 32 sums
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    const int cy = blockIdx.x * 32 + y;
    if (x == 0 && cy < width) st_elem<DTypeOf<DT>::size>(out, cy, f32_to_elem<DT>(s));
}

template <int DT, int V, bool GENERAL>
static cudaError_t bwd_launch(const NormBackwardArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const cudaError_t e = sh.staged ? allow_smem(k_rmsnorm_backward_staged<DT, V, GENERAL>, sh.smemBytes)
                                    : allow_smem(k_rmsnorm_backward<DT, V, GENERAL>, sh.smemBytes);
    if (e != cudaSuccess) return e;
    if (sh.staged) return norm_launch(k_rmsnorm_backward_staged<DT, V, GENERAL>, (unsigned)a.parts, sh, sh.smemBytes, s, a);
    return norm_launch(k_rmsnorm_backward<DT, V, GENERAL>, (unsigned)(a.parts * sh.cluster), sh, sh.smemBytes, s, a);
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
    const unsigned grid = (unsigned)((a.width + 31) / 32);
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
