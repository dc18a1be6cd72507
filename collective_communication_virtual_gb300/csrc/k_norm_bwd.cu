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
#include "norm.cuh"

namespace vc {

template <int V> constexpr int bwd_cta_threads() { return V == 4 ? kNormMaxThreads : 512; }
template <int V> constexpr int bwd_ctas_per_sm() { return V == 4 ? 1 : 2; }

// dw in shared memory: column c of a team at [c % E][c / E], so that the lanes of a warp,
// which hold neighbouring vectors, touch neighbouring words whatever the row's shift.
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(bwd_cta_threads<V>(), bwd_ctas_per_sm<V>())
k_rmsnorm_backward(const __grid_constant__ NormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ float dw[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int part = clustered ? (int)cluster_rank() : 0;
    const int slots = sh.teamThreads * V;              // vectors of a team's part of a row
    const int col0 = part * slots * E;                 // first column of this CTA
    float* mine = dw + (size_t)team * slots * E;
    if (clustered) cluster_arrive();
    for (int i = threadIdx.x; i < slots * E * sh.rowsPerCta; i += blockDim.x) dw[i] = 0.0f;
    __syncthreads();

    const int step = sh.teamThreads * E;
    const size_t ctas = gridDim.x / (unsigned)sh.cluster;
    const size_t stride = ctas * sh.rowsPerCta;
    int flip = 0;
    // every team of a CTA runs the same number of rounds, as they share barriers
    for (size_t base = (size_t)(blockIdx.x / (unsigned)sh.cluster) * sh.rowsPerCta; base < a.rows; base += stride) {
        const size_t row = base + team;
        const bool live = row < a.rows;
        int shift = 0;
        if (GENERAL && live && !clustered)
            shift = (int)(((uintptr_t)a.recv[0] + row * a.recvStride * ESZ) & 15u) / ESZ;
        const int e0 = col0 + t * E - shift;
        Span sp[V];
        bool on[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
            sp[v] = span_of<E>(e0 + v * step, a.width);
            on[v] = live && sp[v].any();
        }
        uint4 hid[V], res[V];
        WeightVec<DT> w[V];
        const ptrdiff_t resOff = ((ptrdiff_t)(row * a.residualStride) + e0) * ESZ;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!on[v]) continue;
            const ptrdiff_t off = resOff + (ptrdiff_t)v * step * ESZ;
            hid[v] = load_vec<ESZ, GENERAL>((const char*)a.hidden + off, sp[v]);
            if (a.gradResidual) res[v] = load_vec<ESZ, GENERAL>((const char*)a.gradResidual + off, sp[v]);
            w[v].template load<GENERAL>(a.weight, a.weightF32, e0 + v * step, sp[v]);
        }
        const float rstd = live ? a.rstd[row] : 0.0f;
        float g[V][E], xhat[V][E];
        sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, ((ptrdiff_t)(row * a.sendStride) + e0) * ESZ, sp, on,
                                  (ptrdiff_t)step * ESZ, g);
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!on[v]) continue;
            float f[E];
            widen_vec<DT>(hid[v], f);
#pragma unroll
            for (int j = 0; j < E; j++) {
                xhat[v][j] = f[j] * rstd;
                if (!GENERAL || sp[v].has(j)) {
                    const int c = e0 + v * step + j - col0;
                    float* p = GENERAL ? &mine[(c & (E - 1)) * slots + c / E] : &mine[j * slots + v * sh.teamThreads + t];
                    *p = fmaf(g[v][j], xhat[v][j], *p);
                }
            }
            w[v].get(a.weightF32, f);
#pragma unroll
            for (int j = 0; j < E; j++) {
                g[v][j] *= f[j];
                if (!GENERAL || sp[v].has(j)) sum = fmaf(g[v][j], xhat[v][j], sum);
            }
        }
        // With shifts that differ by row, a column passes from thread to thread: the barriers
        // of the row's reduction order its additions.
        uint32_t none = 0u;
        if (sh.teamThreads <= 32) __syncwarp();
        team_reduce<false>(red[flip], sh, sum, none);
        if (clustered) cluster_arrive();
        flip ^= 1;
        const float c = sum / (float)a.width;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!on[v]) continue;
            float f[E];
            if (a.gradResidual) widen_vec<DT>(res[v], f);
#pragma unroll
            for (int j = 0; j < E; j++) {
                g[v][j] = rstd * fmaf(-xhat[v][j], c, g[v][j]);
                if (a.gradResidual) g[v][j] += f[j];
            }
        }
        const ptrdiff_t off = ((ptrdiff_t)(row * a.recvStride) + e0) * ESZ;
        for (int o = 0; o < a.nOut; o++) {
            char* p = (char*)a.recv[o] + off;
#pragma unroll
            for (int v = 0; v < V; v++)
                if (on[v]) store_vec<DT, GENERAL>(p + (ptrdiff_t)v * step * ESZ, sp[v], g[v]);
        }
    }
    if (clustered) cluster_wait();

    // one row of sums per CTA (cluster): its teams in order
    __syncthreads();
    float* out = a.partials + (size_t)(blockIdx.x / (unsigned)sh.cluster) * a.width + col0;
    const int columns = min(slots * E, a.width - col0);
    for (int c = threadIdx.x; c < columns; c += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < sh.rowsPerCta; k++) s += dw[(size_t)k * slots * E + (c & (E - 1)) * slots + c / E];
        out[c] = s;
    }
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
    const size_t smem = (size_t)sh.teamThreads * V * kVecElems<DT> * sh.rowsPerCta * sizeof(float);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_rmsnorm_backward<DT, V, GENERAL>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return norm_launch(k_rmsnorm_backward<DT, V, GENERAL>, (unsigned)(a.parts * sh.cluster), sh, smem, s, a);
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
