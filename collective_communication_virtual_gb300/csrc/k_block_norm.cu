// k_block_norm.cu -- all-reduce, the norm after a block, its gate, the scaled residual and the norm
// before the next block in one pass.
//
//   b = sum_r x_r                              (fp32, ranks in order)
//   r1 = 1 / sqrt(sum_j b_j^2 / hidden + eps)
//   h_j = alpha residual_j + b_j r1 (post_j gate_j)
//   r2 = 1 / sqrt(sum_j h_j^2 / hidden + eps)
//   y_j = h_j r2 pre_j                         (b, h and y rounded once each, from fp32)
//
// A row needs two reductions, one behind the other: r2 could be had from the sums of b^2, b h and
// residual^2 alone, but those cancel where the residual and the block's output nearly do.  A thread
// keeps its part of b, then of h, in registers, so every input byte is read once and every output
// byte written once: 18 of them a column and row of 8 ranks in bf16.  Memory bounds the long calls:
// 8 x 4096 x 4096 bf16 99 us, 6.4 TB/s of 6.8, where two warps of three wait for a load, a barrier of the row's
// reductions or shared memory; that is why many inputs get one vector a thread and two CTAs an SM, few
// inputs, where instructions count, four.  One row of 8192 takes 6 us, all launch and latency.  Rows too long to
// stage have four vectors a thread and 96 registers, of which up to 864 bytes are spilled.
#include "block_norm.cuh"

namespace vc {

namespace {

struct Place {
    size_t row;
    bool live;                       // the row exists
    int t, part, col0;               // thread of the team, CTA of the cluster, its first column
    uint32_t buf;                    // GENERAL: the team's three row buffers in shared memory
};

// A row once a thread has its part: b on entry the ranks' sum, res the residual (zeros where there is
// none).  scale(v, f) and pre(v, f) give post * gate and the next norm's weight, zeros behind the row's end.
template <int DT, int V, bool GENERAL, typename Scale, typename Pre>
__device__ __forceinline__ void finish(const BlockNormArgs& a, TeamScratch (&red)[2], const Place& at, const RowVecs<DT, V>& rv,
                                       float (&b)[V][kVecElems<DT>], const uint4 (&res)[V], Scale scale, Pre pre) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const NormShape& sh = a.shape;
    const int columns = min(a.hidden - at.col0, sh.teamThreads * V * E);   // of this CTA
    const int mine = at.t * E;                         // the thread's first column of them
    const size_t off = at.row * a.residualStride;
    const uint32_t bufBlock = at.buf, bufStream = at.buf + (uint32_t)sh.rowBytes, bufOut = at.buf + 2u * (uint32_t)sh.rowBytes;
    const bool leader = at.live && at.t == 0 && at.part == 0;
    float none = 0.0f;
    if (GENERAL) rv.mask(b);
    if (a.blockOut) put_row<DT, V, GENERAL>(a.blockOut, off, at.live, bufBlock, mine, rv, b);
    float sum = dot(b, b);
    if (GENERAL) __syncwarp();                         // a larger team's barrier is in its reduction
    team_reduce<false>(red[0], sh, sum, none);
    if (sh.cluster > 1) cluster_arrive();              // for the next reduction
    const float r1 = __frsqrt_rn(sum / (float)a.hidden + a.eps);
    if (a.rstd && leader) a.rstd[at.row] = r1;
    if (GENERAL && a.blockOut && at.live)
        copy_out<ESZ>((char*)a.blockOut + (off + at.col0) * ESZ, bufBlock, columns * ESZ, at.t, sh.teamThreads);

    // From here on b holds h.
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E], x[E];
        scale(v, f);
        scale_by(b[v], r1);
        mul_by(b[v], f);
        widen_vec<DT>(res[v], x);
        scale_add(x, a.scale, b[v]);
#pragma unroll
        for (int j = 0; j < E; j++) b[v][j] = a.residual ? x[j] : b[v][j];
    }
    if (GENERAL) rv.mask(b);
    if (a.residualOut) put_row<DT, V, GENERAL>(a.residualOut, off, at.live, bufStream, mine, rv, b);
    sum = dot(b, b);
    if (GENERAL) __syncwarp();
    team_reduce<false>(red[1], sh, sum, none);
    const float r2 = __frsqrt_rn(sum / (float)a.hidden + a.eps);
    if (a.rstd && leader) a.rstd[a.rows + at.row] = r2;
    if (GENERAL && a.residualOut && at.live)
        copy_out<ESZ>((char*)a.residualOut + (off + at.col0) * ESZ, bufStream, columns * ESZ, at.t, sh.teamThreads);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[E];
        pre(v, f);
        scale_by(b[v], r2);
        mul_by(b[v], f);
    }
    put_outputs<DT, V, GENERAL>(a.recv, a.nOut, a.outSame, at.row * a.recvStride, at.live, bufOut, at.t, at.col0, columns, sh,
                                rv, b);
}

// Few rows, or rows too long to stage: every team takes one row and loads it directly.
template <int DT, int V, bool GENERAL>
__global__ void __launch_bounds__(kNormMaxThreads, 1) k_block_norm(const __grid_constant__ BlockNormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    Place at;
    at.t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    at.part = sh.cluster > 1 ? (int)cluster_rank() : 0;
    at.col0 = at.part * sh.teamThreads * V * E;
    at.row = (size_t)(blockIdx.x / (unsigned)sh.cluster) * sh.rowsPerCta + team;
    at.live = at.row < a.rows;
    at.buf = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(3 * team * sh.rowBytes);
    if (sh.cluster > 1) cluster_arrive();
    const RowVecs<DT, V> rv(at.col0 + at.t * E, sh.teamThreads * E, a.hidden);

    // The weights' and the residual's loads are under way while the ranks' are awaited.
    float scale[V][E], pre[V][E];
    uint4 res[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = rv.e0 + v * rv.step;
        load_scale<DT, GENERAL>(a.post, a.gate, a.weightF32, e, rv.left[v], scale[v]);
        load_weight<DT, GENERAL>(a.pre, a.weightF32, e, rv.left[v], pre[v]);
        res[v] = make_uint4(0u, 0u, 0u, 0u);
        if (a.residual && at.live && rv.left[v] > 0)
            res[v] = load_vec<ESZ, GENERAL>((const char*)a.residual + (at.row * a.residualStride + e) * ESZ, rv.left[v]);
    }
    float b[V][E];
    sum_ranks<DT, V, GENERAL>(a.send, a.nRanks, (at.row * a.sendStride + rv.e0) * ESZ, at.live, rv, b);
    finish<DT, V, GENERAL>(
        a, red, at, rv, b, res,
        [&](int v, float (&f)[E]) {
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = scale[v][j];
        },
        [&](int v, float (&f)[E]) {
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = pre[v][j];
        });
}

// Many rows: the next row's loads under way while one is finished, sh.rounds rows (of each of its
// teams) one behind the other, or (rounds 0) as many as a stride over all rows brings.  SHARED: the
// CTAs of a cluster share a row that one cannot hold.
template <int DT, int V, bool GENERAL, bool SHARED>
__global__ void __launch_bounds__(kStageMaxThreads, V == 1 ? 2 : 1)
k_block_norm_staged(const __grid_constant__ BlockNormArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ TeamScratch red[2];
    const NormShape& sh = a.shape;
    const int team = sh.rowsPerCta > 1 ? (int)threadIdx.x / sh.teamThreads : 0;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    Place at;
    at.t = sh.rowsPerCta > 1 ? (int)threadIdx.x & (sh.teamThreads - 1) : (int)threadIdx.x;
    at.part = SHARED ? (int)cluster_rank() : 0;
    at.col0 = at.part * sh.teamThreads * V * E;
    if (SHARED) cluster_arrive();
    // the weight before the next block in its own type, behind it post * gate in fp32
    const int scaleBytes = sh.teamThreads * V * E * 4, preBytes = sh.weightBytes - scaleBytes;
    const uint32_t scale = base + (uint32_t)preBytes;
    at.buf = base + (uint32_t)(sh.weightBytes + sh.stageBytes + 3 * team * sh.rowBytes);
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
    stage_weight<DT, GENERAL>(a.pre, a.weightF32, at.col0, a.hidden, base, preBytes);
    stage_scale<DT, GENERAL>(a.post, a.gate, a.weightF32, at.col0, a.hidden, scale, sh.teamThreads * V);
    copies_wait();
    __syncthreads();                                   // the weights, copied by all threads
    // every team of a CTA, and every CTA of a cluster, runs the same number of rounds
    for (size_t row0 = first; row0 < end; row0 += step) {
        at.row = row0 + team;
        at.live = at.row < end;
        float b[V][E];
        uint4 res[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
            res[v] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < E; j++) b[v][j] = 0.0f;
        }
        const auto shift_of = [&](int s) { return GENERAL ? (unsigned)(uintptr_t)segment(s, at.row) & 15u : 0u; };
        copies_wait();
        if (GENERAL) __syncwarp();
#pragma unroll 2
        for (int s = 0; s < N; s++) add_segment<DT, V, GENERAL>(stage, s, shift_of(s), b);
        if (a.residual) staged<V, GENERAL>(stage, N, shift_of(N), res);
        if (GENERAL) __syncwarp();
        fetch(at.row + step);
        finish<DT, V, GENERAL>(
            a, red, at, rv, b, res, [&](int v, float (&f)[E]) { staged_scale<DT>(scale, at.t * E + v * rv.step, f); },
            [&](int v, float (&f)[E]) { staged_weight<DT>(base, a.weightF32, at.t * E + v * rv.step, f); });
        if (SHARED) cluster_arrive();
    }
    if (SHARED) cluster_wait();
    copies_wait();
}

template <int DT, int V, bool GENERAL>
cudaError_t launch_g(const BlockNormArgs& a, cudaStream_t s) {
    const NormShape& sh = a.shape;
    const auto kernel = !sh.staged       ? k_block_norm<DT, V, GENERAL>
                        : sh.cluster > 1 ? k_block_norm_staged<DT, V, GENERAL, true>
                                         : k_block_norm_staged<DT, V, GENERAL, false>;
    const cudaError_t e = allow_smem(kernel, sh.smemBytes);
    if (e != cudaSuccess) return e;
    const size_t teams = sh.staged ? (size_t)sh.ctas : (a.rows + sh.rowsPerCta - 1) / sh.rowsPerCta;
    return norm_launch(kernel, (unsigned)(teams * (size_t)sh.cluster), sh, sh.smemBytes, s, a);
}
template <int DT>
cudaError_t launch_dt(const BlockNormArgs& a, cudaStream_t s) {
    const bool g = a.shape.general != 0;
    switch (a.shape.vecs) {
    case 1: return g ? launch_g<DT, 1, true>(a, s) : launch_g<DT, 1, false>(a, s);
    case 2: return g ? launch_g<DT, 2, true>(a, s) : launch_g<DT, 2, false>(a, s);
    default: return g ? launch_g<DT, 4, true>(a, s) : launch_g<DT, 4, false>(a, s);
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return launch_dt<kF32>(a, s);
    case vFloat16: return launch_dt<kF16>(a, s);
    case vBFloat16: return launch_dt<kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
