// operators.h -- argument blocks and launchers of the operators that run next to the
// collectives (all-reduce + residual + RMS norm, its backward pass, gradient norm and
// clipping), and the part of the communicator that their entry points use.
#pragma once

#include <functional>

#include "internal.h"

namespace vc {

// ---- the communicator, as the operators' entry points see it (vcomm.cpp) ----------------

struct CommView {
    int nRanks;
    int device;
    int smCount;
    bool debug;
    bool grouping;                   // between vcommGroupStart and vcommGroupEnd
};
// vInvalidArgument for a bad handle, the sticky error if there is one, else vSuccess.
vResult_t comm_view(vcomm_t c, CommView* v);
// Record a call of an open group; vcommGroupEnd runs it.
vResult_t comm_record(vcomm_t c, std::function<vResult_t()> call);
// Run `launch` with the communicator's device and launch mode, and take note of its error.
vResult_t comm_launch(vcomm_t c, const char* what, const std::function<cudaError_t()>& launch);

size_t dtype_size(int dt);           // 0 for a type that is none

// ---- RMS norm ----------------------------------------------------------------------------

// A row is handled by a team: the lanes of one warp's power-of-two part (teamThreads <= 32,
// several rows in a CTA), one CTA, or the CTAs of a cluster.  A thread of the team holds
// vecs vectors of 16 bytes of the row.
struct NormShape {
    int vecs;                        // 1, 2 or 4 vectors per thread
    int teamThreads;                 // threads of one CTA that share a row
    int rowsPerCta;                  // teams in a CTA
    int cluster;                     // CTAs that share a row
    int threads;                     // threads per CTA
    int general;                     // some row may start off a 16-byte boundary or end inside a vector
    int staged;                      // many rows: a CTA stages the next row while it finishes one
    int rounds;                      // staged, forward: rows that each team of a CTA takes; 0: the CTAs
                                     // stride over all rows, as in the backward pass
    int ctas;                        // staged: CTAs (clusters) of the grid
    int weightBytes;                 // dynamic shared memory: of the staged weight,
    int stageBytes;                  // of the staged row of every team,
    int rowBytes;                    // of a row buffer (GENERAL: two a team, the backward pass one),
    int extraBytes;                  // of the weight gradient's sums, in front,
    int smemBytes;                   // and altogether
};
constexpr int kStageMaxThreads = 512;
// 16-byte blocks of shared memory for one vector a thread of one input.  General: the blocks of
// a team's lanes of a warp lie side by side, with room for one more behind the last lane's.
#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr int stage_blocks(int threads, int teamThreads, bool general) {
    return !general ? threads : teamThreads >= 32 ? threads / 32 * 33 : threads / teamThreads * (teamThreads + 1);
}
constexpr int kQuantGroup = 128;
constexpr int kNormMaxThreads = 640;     // of a CTA that holds 4 vectors a thread
constexpr int kNormWarpCta = 128;        // threads of a CTA whose teams are parts of a warp
constexpr int kNormMaxCluster = 8;
constexpr int kNormStaticSmem = 768;                         // of a CTA, at most
constexpr int kNormMaxSmem = 227 * 1024 - kNormStaticSmem;   // dynamic, of a CTA
// What a launch has to be shaped for.
struct NormCall {
    size_t rows;
    int hidden, elemSize, weightSize;
    int segments;                    // inputs that every row is read from
    int smCount;
    bool general;                    // as in NormShape
    bool backward;
    bool groups;                     // 8-bit output with a scale per 128 elements
};
NormShape norm_shape(const NormCall& c);

struct NormArgs {
    const void* send[VCOMM_MAX_RANKS];
    void* recv[VCOMM_MAX_RANKS];     // the nOut outputs that are wanted, in rank order
    float* scales[VCOMM_MAX_RANKS];  // 8-bit output: scales of the output with that index
    const void* residual;            // may be NULL
    void* residualOut;               // may be NULL
    const void* weight;
    float* rstd;                     // may be NULL
    size_t rows;
    size_t sendStride, residualStride, recvStride;     // elements between rows
    int hidden;
    int nRanks;
    int nOut;
    int outSame;                     // the outputs all start at one offset from 16 bytes
    int weightF32;                   // the weight is fp32 (else the data's type)
    int groups;                      // 8-bit output: groups of 128 per row, 0: one scale a row
    float eps;
    NormShape shape;
};
cudaError_t launch_allreduce_rmsnorm(const NormArgs& a, vDataType_t dt, cudaStream_t s);
cudaError_t launch_allreduce_rmsnorm_quant(const NormArgs& a, vDataType_t dt, cudaStream_t s);

struct NormBackwardArgs {
    const void* send[VCOMM_MAX_RANKS];   // every rank's partial gradient of the normed output
    void* recv[VCOMM_MAX_RANKS];         // the nOut outputs that are wanted
    const void* hidden;                  // the stream that was normed
    const void* gradResidual;            // may be NULL
    const void* weight;
    const float* rstd;
    float* partials;                     // [parts][width]
    void* gradWeight;
    size_t rows;
    size_t sendStride, residualStride, recvStride;
    int width;
    int nRanks;
    int nOut;
    int outSame;
    int weightF32;
    int parts;                           // CTAs (clusters) that stride over the rows
    NormShape shape;
};
// CTAs (clusters) of the backward pass: its workspace holds one row of fp32 sums for each.
int norm_backward_parts(size_t rows, const NormShape& sh, int smCount);
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs& a, vDataType_t dt, cudaStream_t s);

// ---- gradient norm and clipping ----------------------------------------------------------

// A piece of one tensor of one rank, at most kGradChunkVecs vectors wherever it starts.
struct alignas(32) GradChunk {
    const char* in;
    char* out;
    int count;                       // elements
    int dt;                          // vDataType_t
    int pad[2];
};
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;         // vectors of a chunk that each thread holds
constexpr int kGradChunkVecs = kGradThreads * kGradVecs;   // 32 KiB
constexpr int kSquaresCtasPerSm = 4;

struct GradNormArgs {
    const GradChunk* chunks;         // those that count towards the norm
    unsigned int nChunks;
    unsigned int* done;              // CTAs that have written their sum: zero between calls
    double* partials;                // one sum of squares per CTA
    float* norm;
};
struct GradClipArgs {
    const GradChunk* chunks;
    unsigned int nChunks;
    const float* norm;
    float maxNorm;
};
cudaError_t launch_grad_norm(const GradNormArgs& a, int grid, cudaStream_t s);
cudaError_t launch_grad_clip(const GradClipArgs& a, cudaStream_t s);

}  // namespace vc
