// k_block_norm_bwd.cu -- backward pass of the block norm.
//
//   dy = sum_r dy_r                           (fp32, ranks in order)
//   x2 = h r2,  g2 = dy pre,  c2 = sum_j g2_j x2_j / width
//   dh = r2 (g2 - x2 c2) + dstream            (the stream's gradient; the residual's is alpha dh)
//   x1 = b r1,  g1 = dh (post gate),  c1 = sum_j g1_j x1_j / width
//   db = r1 (g1 - x1 c1)                      (of the block's output and, as that is a plain sum, of
//                                              every rank's partial sum)
//   dpre_j = sum over rows of dy_j x2_j,  q_j = sum over rows of dh_j x1_j
//   dpost_j = gate_j q_j,  dgate_j = post_j q_j
//
// The gate and the weight after the block stand side by side, so one sum down the columns serves
// both.  A CTA (or cluster) strides over the rows and keeps its two sums in fp32; each writes them as
// one row of the workspace, and a second launch adds them up and multiplies.  The order of the
// additions follows from the launch shape alone.
//
// Memory bounds aligned rows: 8 x 4096 x 4096 bf16 114 us (5.9 TB/s of 6.8; 105 the first launch alone).
// Rows off 16 bytes are bound by instructions: 3 x 1537 x 2731 fp16 46 us (1.8 TB/s), at 125 registers with both
// sums in shared memory, where every vector is shifted in and out and read and written back to the sums.  Rows too
// long to stage spill up to 652 bytes a thread with four vectors.
#include "block_norm.cuh"

namespace vc {

namespace {

// One vector a thread leaves registers for both sums; with more they are kept in shared memory.
template <int DT, int V> using Sums = WeightSums<DT, V, (V == 1)>;

template <int DT, int V>
struct Rows {                        // what the threads of a team hold of a row, in the storage type
    uint4 hidden[V], block[V], grad[V];
    float r1, r2;
};

// A row once a thread has its part: g holds dy on entry, `in` the rest (zeros for a gradient that
// there is none of).
template <int DT, int V, bool GENERAL, typename Scale, typename Pre>
__device__ __forceinline__ void finish(const BlockNormBackwardArgs& a, TeamScratch (&red)[2], size_t row, bool live, int t,
                                       int col0, uint32_t buf, const RowVecs<DT, V>& rv, Sums<DT, V>& dpre, Sums<DT, V>& q,
                                       float (&g)[V][kVecElems<DT>], const Rows<DT, V>& in, Scale scale, Pre pre) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const NormShape& sh = a.shape;
    const int columns = min(a.width - col0, sh.teamThreads * V * E), mine = t * E;
    const uint32_t bufOut = buf + (uint32_t)sh.rowBytes;
    const size_t off = row * a.residualStride;
    float none = 0.0f;
    // From here on a thread holds zeros behind the row's end, and only the stores ask for it.
    if (GENERAL) rv.mask(g);
    float x[V][E];
#pragma unroll
    for (int v = 0; v < V; v++) {
        widen_vec<DT>(in.hidden[v], x[v]);
        scale_by(x[v], in.r2);
    }
    if (GENERAL) rv.mask(x);
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (live) dpre.add(v, g[v], x[v]);
        float f[E];
        pre(v, f);
        mul_by(g[v], f);
    }
    float sum = dot(g, x);
    team_reduce<false>(red[0], sh, sum, none);
    if (sh.cluster > 1) cluster_arrive();              // for the next reduction
    const float c2 = -(sum / (float)a.width);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        widen_vec<DT>(in.grad[v], f);
        scale_add(x[v], c2, g[v]);                     // g2 - x2 c2
        scale_add(x[v], in.r2, f);
#pragma unroll
        for (int j = 0; j < E; j++) {
            g[v][j] = x[v][j];                         // dh
            x[v][j] *= a.scale;
        }
    }
    if (GENERAL) rv.mask(g);
    if (a.gradResidual) put_row<DT, V, GENERAL>(a.gradResidual, off, live, buf, mine, rv, x);
#pragma unroll
    for (int v = 0; v < V; v++) {
        widen_vec<DT>(in.block[v], x[v]);
        scale_by(x[v], in.r1);
    }
    if (GENERAL) rv.mask(x);
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (live) q.add(v, g[v], x[v]);
        float f[E];
        scale(v, f);
        mul_by(g[v], f);
    }
    sum = dot(g, x);
    if (GENERAL) __syncwarp();                         // a larger team's barrier is in its reduction
    team_reduce<false>(red[1], sh, sum, none);
    if (GENERAL && a.gradResidual && live)
        copy_out<ESZ>((char*)a.gradResidual + (off + col0) * ESZ, buf, columns * ESZ, t, sh.teamThreads);
    const float c1 = -(sum / (float)a.width);
#pragma unroll
    for (int v = 0; v < V; v++) {
        scale_add(x[v], c1, g[v]);
        scale_by(x[v], in.r1);
    }
    put_outputs<DT, V, GENERAL>(a.recv, a.nOut, a.outSame, row * a.recvStride, live, bufOut, t, col0, columns, sh, rv, x);
    if (GENERAL) __syncwarp();                         // a small team's buffers are free again
}

// One row of the workspace per CTA (cluster): dpre, then q.
template <int DT, int V>
__device__ __forceinline__ void write_sums(const BlockNormBackwardArgs& a, const unsigned char* smem, size_t index, int col0,
                                           Sums<DT, V>& dpre, Sums<DT, V>& q) {
    const NormShape& sh = a.shape;
    const int columns = min(a.width - col0, sh.teamThreads * V * kVecElems<DT>);
    float* out = a.partials + index * 2 * (size_t)a.width + col0;
    dpre.write(smem, sh, out, columns);
    q.write(smem + sh.extraBytes / 2, sh, out + a.width, columns);
}

// Few rows, or rows too long to stage: direct loads; a row may be split over a cluster.
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kNormMaxThreads, 1) k_block_norm_backward(const __grid_constant__ BlockNormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const bool clustered = sh.cluster > 1;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int col0 = clustered ? (int)cluster_rank() * sh.teamThreads * V * E : 0;     // first column of this CTA
    if (clustered) cluster_arrive();
    Sums<DT, V> dpre, q;
    dpre.init(smem);
    q.init(smem + sh.extraBytes / 2);
    const uint32_t buf = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(sh.extraBytes + 2 * team * sh.rowBytes);
    const RowVecs<DT, V> rv(col0 + t * E, sh.teamThreads * E, a.width);

    const size_t index = blockIdx.x / (unsigned)sh.cluster;
    const size_t stride = (size_t)(gridDim.x / (unsigned)sh.cluster) * sh.rowsPerCta;
    // every team of a CTA runs the same number of rounds, as they share barriers
    for (size_t base = index * sh.rowsPerCta; base < a.rows; base += stride) {
        const size_t row = base + team;
        const bool live = row < a.rows;
        Rows<DT, V> in;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const size_t off = (row * a.residualStride + rv.e0 + v * rv.step) * ESZ;
            in.hidden[v] = in.block[v] = in.grad[v] = make_uint4(0u, 0u, 0u, 0u);
            if (!live || rv.left[v] == 0) continue;
            in.hidden[v] = load_vec<ESZ, GENERAL>((const char*)a.hidden + off, rv.left[v]);
            in.block[v] = load_vec<ESZ, GENERAL>((const char*)a.block + off, rv.left[v]);
            if (a.gradStream) in.grad[v] = load_vec<ESZ, GENERAL>((const char*)a.gradStream + off, rv.left[v]);
        }
        in.r1 = live ? a.rstd[row] : 0.0f;
        in.r2 = live ? a.rstd[a.rows + row] : 0.0f;
        float g[V][E];
        sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, (row * a.sendStride + rv.e0) * ESZ, live, rv, g);
        finish<DT, V, GENERAL>(
            a, red, row, live, t, col0, buf, rv, dpre, q, g, in,
            [&](int v, float (&f)[E]) {
                load_scale<DT, GENERAL>(a.post, a.gate, a.weightF32, rv.e0 + v * rv.step, rv.left[v], f);
            },
            [&](int v, float (&f)[E]) {
                load_weight<DT, GENERAL>(a.pre, a.weightF32, rv.e0 + v * rv.step, rv.left[v], f);
                if (GENERAL) {
#pragma unroll
                    for (int j = 0; j < E; j++) f[j] = j < rv.left[v] ? f[j] : 0.0f;
                }
            });
        if (clustered) cluster_arrive();
    }
    if (clustered) cluster_wait();
    write_sums<DT, V>(a, smem, index, col0, dpre, q);
}

// Many rows: CTAs stride over them, the next row's loads under way while one is finished.  A row that
// one CTA cannot hold is shared by the CTAs of a cluster.
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kStageMaxThreads, 1)
k_block_norm_backward_staged(const __grid_constant__ BlockNormBackwardArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const int N = a.nRanks, segments = N + 2 + (a.gradStream ? 1 : 0);
    Sums<DT, V> dpre, q;
    dpre.init(smem);
    q.init(smem + sh.extraBytes / 2);
    // the weight before the next block in its own type, behind it post * gate in fp32
    const int scaleBytes = sh.teamThreads * V * E * 4, preBytes = sh.weightBytes - scaleBytes;
    const uint32_t weight = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)sh.extraBytes;
    const uint32_t scale = weight + (uint32_t)preBytes;
    const uint32_t buf = weight + (uint32_t)(sh.weightBytes + sh.stageBytes + 2 * team * sh.rowBytes);
    const bool clustered = sh.cluster > 1;
    const int col0 = clustered ? (int)cluster_rank() * sh.teamThreads * V * E : 0;
    if (clustered) cluster_arrive();
    const RowVecs<DT, V> rv(col0 + t * E, sh.teamThreads * E, a.width);
    const StageAddr stage = stage_addr<GENERAL>(weight + (uint32_t)sh.weightBytes, sh);

    // address of a segment's element rv.e0: the ranks', the stream's, the block's, the stream's gradient
    const auto segment = [&](int s, size_t row) {
        if (s < N) return (const char*)a.send[s] + (row * a.sendStride + rv.e0) * ESZ;
        return (const char*)(s == N ? a.hidden : s == N + 1 ? a.block : a.gradStream) + (row * a.residualStride + rv.e0) * ESZ;
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
    float r1 = first + team < a.rows ? a.rstd[first + team] : 0.0f;
    float r2 = first + team < a.rows ? a.rstd[a.rows + first + team] : 0.0f;
    stage_weight<DT, GENERAL>(a.pre, a.weightF32, col0, a.width, weight, preBytes);
    stage_scale<DT, GENERAL>(a.post, a.gate, a.weightF32, col0, a.width, scale, sh.teamThreads * V);
    copies_wait();
    __syncthreads();                                   // the weights, copied by all threads
    for (size_t base = first; base < a.rows; base += stride) {
        const size_t row = base + team, next = row + stride;
        const float r1Next = next < a.rows ? a.rstd[next] : 0.0f, r2Next = next < a.rows ? a.rstd[a.rows + next] : 0.0f;
        float g[V][E];
        Rows<DT, V> in;
        in.r1 = r1;
        in.r2 = r2;
#pragma unroll
        for (int v = 0; v < V; v++) {
            in.grad[v] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < E; j++) g[v][j] = 0.0f;
        }
        const auto shift_of = [&](int s) { return GENERAL ? (unsigned)(uintptr_t)segment(s, row) & 15u : 0u; };
        copies_wait();
        if (GENERAL) __syncwarp();
#pragma unroll 2
        for (int s = 0; s < N; s++) add_segment<DT, V, GENERAL>(stage, s, shift_of(s), g);
        staged<V, GENERAL>(stage, N, shift_of(N), in.hidden);
        staged<V, GENERAL>(stage, N + 1, shift_of(N + 1), in.block);
        if (a.gradStream) staged<V, GENERAL>(stage, N + 2, shift_of(N + 2), in.grad);
        if (GENERAL) __syncwarp();
        fetch(next);
        finish<DT, V, GENERAL>(
            a, red, row, row < a.rows, t, col0, buf, rv, dpre, q, g, in,
            [&](int v, float (&f)[E]) { staged_scale<DT>(scale, t * E + v * rv.step, f); },
            [&](int v, float (&f)[E]) { staged_weight<DT>(weight, a.weightF32, t * E + v * rv.step, f); });
        if (clustered) cluster_arrive();
        r1 = r1Next;
        r2 = r2Next;
    }
    if (clustered) cluster_wait();
    copies_wait();
    write_sums<DT, V>(a, smem, index, col0, dpre, q);
}

// The weights' gradients from the partial rows: 16 columns a CTA, the rows dealt to 32 groups of its
// threads, whose sums are added in a fixed order.  The first half of the grid adds dpre, the second q.
constexpr int kSumColumns = 16;
constexpr int kSumGroups = 32;
constexpr int kSumThreads = kSumColumns * kSumGroups;
template <int DT>
__global__ void __launch_bounds__(kSumThreads)
k_block_norm_weights(const float* partials, int rows, int width, const void* post, const void* gate, void* gradPre,
                     void* gradPost, void* gradGate) {
    pdl_begin();
    constexpr int ESZ = DTypeOf<DT>::size;
    __shared__ float part[kSumGroups][kSumColumns + 1];
    const int half = (int)gridDim.x / 2, ofQ = (int)blockIdx.x >= half;
    const int c0 = ((int)blockIdx.x - (ofQ ? half : 0)) * kSumColumns;
    const int x = threadIdx.x % kSumColumns, y = threadIdx.x / kSumColumns;
    const int c = c0 + x;
    const float* from = partials + (ofQ ? width : 0);
    float s = 0.0f;
    if (c < width) {
#pragma unroll 8
        for (int r = y; r < rows; r += kSumGroups) s += from[(size_t)r * 2 * width + c];
    }
    part[y][x] = s;
    __syncthreads();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s = part[lane][w];                                 // warp w: column w's 32 sums
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    const int cw = c0 + w;
    if (lane != 0 || cw >= width) return;
    const auto weight = [&](const void* p) {
        if (DT == kF32) return ((const float*)p)[cw];
        return widen16<DT>(((const uint16_t*)p)[cw]);
    };
    if (!ofQ) {
        st_elem<ESZ>(gradPre, cw, f32_to_elem<DT>(s));
        return;
    }
    st_elem<ESZ>(gradPost, cw, f32_to_elem<DT>(gate ? s * weight(gate) : s));
    if (gradGate) st_elem<ESZ>(gradGate, cw, f32_to_elem<DT>(s * weight(post)));
}
static_assert(kSumThreads / 32 == kSumColumns, "one warp per column");

template <int DT, int V, bool GENERAL>
cudaError_t bwd_launch(const BlockNormBackwardArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const auto kernel = sh.staged ? k_block_norm_backward_staged<DT, V, GENERAL> : k_block_norm_backward<DT, V, GENERAL>;
    const cudaError_t e = allow_smem(kernel, sh.smemBytes);
    if (e != cudaSuccess) return e;
    return norm_launch(kernel, (unsigned)(a.parts * sh.cluster), sh, sh.smemBytes, s, a);
}
template <int DT>
cudaError_t bwd_launch_dt(const BlockNormBackwardArgs& a, cudaStream_t s) {
    cudaError_t e;
    const bool g = a.shape.general != 0;
    switch (a.shape.vecs) {
    case 1: e = g ? bwd_launch<DT, 1, true>(a, s) : bwd_launch<DT, 1, false>(a, s); break;
    case 2: e = g ? bwd_launch<DT, 2, true>(a, s) : bwd_launch<DT, 2, false>(a, s); break;
    default: e = g ? bwd_launch<DT, 4, true>(a, s) : bwd_launch<DT, 4, false>(a, s); break;
    }
    if (e != cudaSuccess) return e;
    const unsigned grid = 2u * (unsigned)((a.width + kSumColumns - 1) / kSumColumns);
    const auto kernel = a.weightF32 ? k_block_norm_weights<kF32> : k_block_norm_weights<DT>;
    return pdl_launch(kernel, grid, kSumThreads, 0, s, (const float*)a.partials, a.parts, a.width, a.post, a.gate, a.gradPre,
                      a.gradPost, a.gradGate);
}

}  // namespace

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return bwd_launch_dt<kF32>(a, s);
    case vFloat16: return bwd_launch_dt<kF16>(a, s);
    case vBFloat16: return bwd_launch_dt<kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
