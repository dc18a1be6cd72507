// norm_stage.cuh -- rows staged through shared memory by asynchronous copies, for CTAs that
// handle many rows.
//
// A thread copies the 16-byte blocks of its part of the next row (of every input) into blocks
// of shared memory and reads them back when their turn comes.  Aligned rows: no thread reads
// another's blocks, so no barrier and no wait but for its own copies is needed.  GENERAL: a
// vector lies in two blocks, the thread's and its neighbour's in the warp, so the warp
// synchronises.  While one row is reduced, scaled and stored the next one's loads are under
// way, and they cost no registers.
#pragma once

#include "norm.cuh"

namespace vc {

__device__ __forceinline__ void copy_block_async(uint32_t smem, const char* p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem), "l"(p) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// The shared memory of a thread for one row: block (segment, v) at base + (segment * V + v) *
// pitch.  GENERAL: the blocks of a team's lanes of a warp lie side by side, with room for one
// more behind the last lane's.
struct StageAddr {
    uint32_t base, pitch;
    bool lastLane;                   // of the team's part of the warp
};
template <bool GENERAL>
__device__ __forceinline__ StageAddr stage_addr(uint32_t smem, const NormShape& sh) {
    StageAddr s;
    const int lanes = min(sh.teamThreads, 32);         // a power of two
    const int index = (int)threadIdx.x + (GENERAL ? (int)threadIdx.x / lanes : 0);
    s.base = smem + (uint32_t)index * 16u;
    s.pitch = (uint32_t)stage_blocks((int)blockDim.x, sh.teamThreads, GENERAL) * 16u;
    s.lastLane = ((int)threadIdx.x & (lanes - 1)) == lanes - 1;
    return s;
}

// Start the copies of one input's part of a row.  p: address of the row's element rv.e0.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void stage_segment(const StageAddr& s, int seg, const char* p, const RowVecs<DT, V>& rv) {
    constexpr int ESZ = DTypeOf<DT>::size;
    const uint32_t at = s.base + (uint32_t)(seg * V) * s.pitch;
    const unsigned sh = GENERAL ? (unsigned)((uintptr_t)p & 15u) : 0u;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (rv.left[v] == 0) continue;
        const char* q = p + (size_t)v * rv.step * ESZ;
        copy_block_async(at + v * s.pitch, GENERAL ? q - sh : q);
        // the second block, where it holds elements of the row and no neighbour copies it: its
        // vector lies in another warp, or behind the row
        if (GENERAL && sh != 0 && rv.left[v] > (int)(16u - sh) / ESZ && (s.lastLane || rv.last[v]))
            copy_block_async(at + v * s.pitch + 16, q - sh + 16);
    }
}
// One input's vectors back from shared memory.  GENERAL: elements outside the row are undefined;
// else a vector outside the row is zero.
template <int V, bool GENERAL>
__device__ __forceinline__ void staged(const StageAddr& s, int seg, unsigned sh, uint4 (&out)[V]) {
    const uint32_t at = s.base + (uint32_t)(seg * V) * s.pitch;
    if (!GENERAL || sh == 0) {
#pragma unroll
        for (int v = 0; v < V; v++) out[v] = ld_smem(at + v * s.pitch);
        return;
    }
    with_shift(sh, [&](auto shift) {
#pragma unroll
        for (int v = 0; v < V; v++) out[v] = shift(ld_smem(at + v * s.pitch), ld_smem(at + v * s.pitch + 16));
    });
}
// Aligned rows: the vectors of a thread that lie outside every row are never copied, and are
// zero from here on, so that nothing but the stores need ask for them.
template <int DT, int V>
__device__ __forceinline__ void stage_zeros(const StageAddr& s, int segments, const RowVecs<DT, V>& rv) {
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (rv.left[v] > 0) continue;
        for (int seg = 0; seg < segments; seg++)
            st_smem(s.base + (uint32_t)(seg * V + v) * s.pitch, make_uint4(0u, 0u, 0u, 0u));
    }
}

// One input's part of a row, back from shared memory and added.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void add_segment(const StageAddr& s, int seg, unsigned sh, float (&acc)[V][kVecElems<DT>]) {
    uint4 raw[V];
    staged<V, GENERAL>(s, seg, sh, raw);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[kVecElems<DT>];
        widen_vec<DT>(raw[v], f);
        add_to(acc[v], f);
    }
}

// The CTA's part of the weight, from column col0 on, in shared memory, in its own type, with
// zeros behind the row's end up to that of the team's last vector.  Starts copies that the caller
// waits for.
template <int DT, bool GENERAL>
__device__ __forceinline__ void stage_weight(const void* all, bool f32, int col0, int columns, uint32_t smem, int bytes) {
    const int size = f32 ? 4 : DTypeOf<DT>::size, per = 16 / size;
    const char* w = (const char*)all + (size_t)col0 * size;
    const int width = max(0, min(columns - col0, bytes / size));
    const bool aligned = !GENERAL || ((uintptr_t)w & 15u) == 0;
    const int whole = aligned ? width / per : 0;       // blocks that hold nothing else
    for (int i = threadIdx.x; i < whole; i += blockDim.x) copy_block_async(smem + 16 * i, w + (size_t)i * 16);
    for (int i = whole + (int)threadIdx.x; i < bytes / 16; i += blockDim.x) {
        const int left = width - i * per;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (left > 0) {
            const char* p = w + (size_t)i * 16;
            v = f32 ? load_vec<4, GENERAL, false>(p, left) : load_vec<DTypeOf<DT>::size, GENERAL, false>(p, left);
        }
        if (GENERAL && left > 0 && left < per) {       // zeros, not what follows the weight in memory
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int have = left * size - 4 * k;  // bytes of word k
                x[k] = have >= 4 ? x[k] : have == 2 ? x[k] & 0xFFFFu : 0u;
            }
            v = make_uint4(x[0], x[1], x[2], x[3]);
        }
        st_smem(smem + 16 * i, v);
    }
    copies_commit();
}
template <int DT>
__device__ __forceinline__ void staged_weight(uint32_t smem, bool f32, int e, float (&f)[kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    if constexpr (DT != kF32) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const uint4 v = ld_smem(smem + (uint32_t)((e + i) * 4));
                f[i] = __uint_as_float(v.x);
                f[i + 1] = __uint_as_float(v.y);
                f[i + 2] = __uint_as_float(v.z);
                f[i + 3] = __uint_as_float(v.w);
            }
            return;
        }
    }
    widen_vec<DT>(ld_smem(smem + (uint32_t)(e * DTypeOf<DT>::size)), f);
}

}  // namespace vc
