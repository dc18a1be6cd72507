// norm_sums.cuh -- sums down the columns of the rows that a CTA handles, for the weights' gradients
// in the backward passes.
#pragma once

#include "norm_stage.cuh"

namespace vc {

// The weight's gradient over a CTA's rows.  A thread holds the same columns of every row, so its
// sums are its own: in registers, or, where those are too few (REGS false), in shared memory (float4
// number (v E/4 + j/4) threads + thread), where the sums of all teams meet at the end.
template <int DT, int V, bool REGS = (V <= 2)>
struct WeightSums {
    static constexpr int E = kVecElems<DT>;
    static constexpr bool kRegs = REGS;
    float4* mine;
    float regs[kRegs ? V : 1][kRegs ? E : 1];
    __device__ __forceinline__ void init(unsigned char* smem) {
        mine = reinterpret_cast<float4*>(smem) + threadIdx.x;
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int j = 0; j < E; j++) {
                if (kRegs) regs[kRegs ? v : 0][kRegs ? j : 0] = 0.0f;
                else if (j % 4 == 0) mine[(v * (E / 4) + j / 4) * blockDim.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
    }
    // dw += dy * xhat for vector v
    __device__ __forceinline__ void add(int v, const float (&dy)[E], const float (&xhat)[E]) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            const float2 a0 = make_float2(dy[j], dy[j + 1]), a1 = make_float2(dy[j + 2], dy[j + 3]);
            const float2 b0 = make_float2(xhat[j], xhat[j + 1]), b1 = make_float2(xhat[j + 2], xhat[j + 3]);
            if (kRegs) {
                float* r = &regs[kRegs ? v : 0][kRegs ? j : 0];
                const float2 lo = fma2(a0, b0, make_float2(r[0], r[1])), hi = fma2(a1, b1, make_float2(r[2], r[3]));
                r[0] = lo.x;
                r[1] = lo.y;
                r[2] = hi.x;
                r[3] = hi.y;
            } else {
                float4* p = mine + (v * (E / 4) + j / 4) * blockDim.x;
                const float4 s = *p;
                const float2 lo = fma2(a0, b0, make_float2(s.x, s.y)), hi = fma2(a1, b1, make_float2(s.z, s.w));
                *p = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
    // One row of sums per CTA: its teams' in order.
    __device__ __forceinline__ void write(const unsigned char* smem, const NormShape& sh, float* out, int columns) {
        if (kRegs) {
#pragma unroll
            for (int v = 0; v < V; v++)
#pragma unroll
                for (int j = 0; j < E; j += 4) {
                    const float* r = &regs[kRegs ? v : 0][kRegs ? j : 0];
                    mine[(v * (E / 4) + j / 4) * blockDim.x] = make_float4(r[0], r[1], r[2], r[3]);
                }
        }
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(smem);
        for (int c = threadIdx.x; c < columns; c += blockDim.x) {
            const int vec = c / E, j = c & (E - 1);
            const int v = vec / sh.teamThreads, t = vec - v * sh.teamThreads;
            float s = 0.0f;
            for (int k = 0; k < sh.rowsPerCta; k++)
                s += all[(((size_t)v * (E / 4) + j / 4) * blockDim.x + k * sh.teamThreads + t) * 4 + (j & 3)];
            out[c] = s;
        }
    }
};

}  // namespace vc
