// block_norm.cuh -- what the block norm's forward and backward pass share: the scale that the
// normed block output is multiplied by.
#pragma once

#include "norm_sums.cuh"

namespace vc {

// post * gate (gate may be NULL) of columns [e, e + E), `left` of them inside the row, in fp32;
// zeros behind the row's end.
template <int DT, bool GENERAL>
__device__ __forceinline__ void load_scale(const void* post, const void* gate, bool f32, int e, int left,
                                           float (&f)[kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    load_weight<DT, GENERAL>(post, f32, e, left, f);
    if (gate) {
        float g[E];
        load_weight<DT, GENERAL>(gate, f32, e, left, g);
        mul_by(f, g);
    }
    if (GENERAL) {
#pragma unroll
        for (int j = 0; j < E; j++) f[j] = j < left ? f[j] : 0.0f;
    }
}

// The CTA's part of that product in shared memory, `vecs` vectors of a row from column col0 on.
template <int DT, bool GENERAL>
__device__ __forceinline__ void stage_scale(const void* post, const void* gate, bool f32, int col0, int columns, uint32_t smem,
                                            int vecs) {
    constexpr int E = kVecElems<DT>;
    for (int i = threadIdx.x; i < vecs; i += blockDim.x) {
        const int e = col0 + i * E;
        float f[E];
        load_scale<DT, GENERAL>(post, gate, f32, e, max(0, min(E, columns - e)), f);
#pragma unroll
        for (int j = 0; j < E; j += 4)
            st_smem(smem + (uint32_t)((i * E + j) * 4), make_uint4(__float_as_uint(f[j]), __float_as_uint(f[j + 1]),
                                                                   __float_as_uint(f[j + 2]), __float_as_uint(f[j + 3])));
    }
}
template <int DT>
__device__ __forceinline__ void staged_scale(uint32_t smem, int e, float (&f)[kVecElems<DT>]) {
#pragma unroll
    for (int j = 0; j < kVecElems<DT>; j += 4) {
        const uint4 v = ld_smem(smem + (uint32_t)((e + j) * 4));
        f[j] = __uint_as_float(v.x);
        f[j + 1] = __uint_as_float(v.y);
        f[j + 2] = __uint_as_float(v.z);
        f[j + 3] = __uint_as_float(v.w);
    }
}

// x * y, summed over a thread's vectors.
template <int V, int E>
__device__ __forceinline__ float dot(const float (&x)[V][E], const float (&y)[V][E]) {
    float2 two[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int j = 0; j < E; j += 2)
            two[j / 2 & 1] = fma2(make_float2(x[v][j], x[v][j + 1]), make_float2(y[v][j], y[v][j + 1]), two[j / 2 & 1]);
    return (two[0].x + two[0].y) + (two[1].x + two[1].y);
}
// x * a + y
template <int E>
__device__ __forceinline__ void scale_add(float (&x)[E], float a, const float (&y)[E]) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 r = fma2(make_float2(x[j], x[j + 1]), make_float2(a, a), make_float2(y[j], y[j + 1]));
        x[j] = r.x;
        x[j + 1] = r.y;
    }
}

// A thread's part of a row in its storage type: straight to memory, or (GENERAL) into the team's
// row buffer `buf`, from which copy_out takes it after a barrier of the team.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void put_row(void* out, size_t off, bool live, uint32_t buf, int mine, const RowVecs<DT, V>& rv,
                                        const float (&x)[V][kVecElems<DT>]) {
    constexpr int ESZ = DTypeOf<DT>::size;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (GENERAL) st_smem(buf + (uint32_t)((mine + v * rv.step) * ESZ), narrow_vec<DT>(x[v]));
        else if (live && rv.left[v] > 0)
            st_stream((char*)out + (off + rv.e0 + v * rv.step) * ESZ, narrow_vec<DT>(x[v]));
    }
}
template <bool GENERAL>
__device__ __forceinline__ void team_sync(const NormShape& sh) {
    if (!GENERAL) return;
    if (sh.teamThreads > 32) __syncthreads();
    else __syncwarp();
}
// All wanted outputs of a row.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void put_outputs(void* const* recv, int nOut, bool same, size_t off, bool live, uint32_t buf, int t,
                                            int col0, int columns, const NormShape& sh, const RowVecs<DT, V>& rv,
                                            const float (&x)[V][kVecElems<DT>]) {
    constexpr int ESZ = DTypeOf<DT>::size;
    if (GENERAL) {
        put_row<DT, V, true>(nullptr, 0, live, buf, t * kVecElems<DT>, rv, x);
        team_sync<true>(sh);
        if (live) copy_out_all<ESZ>(recv, nOut, same, (off + col0) * ESZ, buf, columns * ESZ, t, sh.teamThreads);
    } else if (live) {
        uint4 w[V];
#pragma unroll
        for (int v = 0; v < V; v++) w[v] = narrow_vec<DT>(x[v]);
        for (int o = 0; o < nOut; o++) {
            char* p = (char*)recv[o] + (off + rv.e0) * ESZ;
#pragma unroll
            for (int v = 0; v < V; v++)
                if (rv.left[v] > 0) st_stream(p + (size_t)v * rv.step * ESZ, w[v]);
        }
    }
}

}  // namespace vc
