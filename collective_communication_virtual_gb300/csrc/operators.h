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
    int general;                     // some buffer or row may start off a 16-byte boundary
};
// Elements that one 128-element scale group covers.
constexpr int kQuantGroup = 128;
constexpr int kNormMaxThreads = 640;     // of a CTA that holds 4 vectors a thread
constexpr int kNormWarpCta = 128;        // threads of a CTA whose teams are parts of a warp
constexpr int kNormMaxCluster = 8;
constexpr int kNormGroupSlots = 168;     // scale groups of one CTA: at most 640 * 4 * 8 / 128 + 1,
                                         // or 128 / team * (team * 4 * 8 / 128 + 1) of small teams
NormShape norm_shape(size_t rows, int hidden, int elemSize, int smCount, bool general);

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
    int weightF32;
    int parts;                           // CTAs (clusters) that stride over the rows
    NormShape shape;
};
// CTAs (clusters) of the backward pass: its workspace holds one row of fp32 sums for each.
int norm_backward_parts(size_t rows, const NormShape& sh, int smCount);
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs& a, vDataType_t dt, cudaStream_t s);

// ---- gradient norm and clipping ----------------------------------------------------------

// One tensor of one rank.  The table travels in the kernels' parameter block.
struct GradItem {
    const void* in;
    void* out;
    unsigned long long count;
    unsigned int chunk0;             // first chunk of this tensor in the launch
    unsigned int dt;                 // vDataType_t
};
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;         // vectors of a chunk that each thread holds
constexpr int kGradChunkVecs = kGradThreads * kGradVecs;   // 32 KiB
template <int CAP>
struct GradArgs {
    int nItems;
    unsigned int nChunks;
    double* partials;                // this launch's sums of squares
    const float* norm;               // clipping: the norm
    float maxNorm;
    int pad;
    GradItem items[CAP];
};
// Tables of two sizes: launching with a 4 KiB parameter block costs less host time.
constexpr int kGradItemsSmall = 120;
constexpr int kGradItemsLarge = 1000;
static_assert(sizeof(GradArgs<kGradItemsLarge>) <= 32764, "kernel parameters are limited to 32,764 bytes");
// Chunks that cover `count` elements wherever they start.
inline unsigned long long grad_chunks(unsigned long long count, size_t elemSize) {
    const unsigned long long e = 16 / elemSize;
    return (count + 2 * e - 2) / e / kGradChunkVecs + 1;
}

template <int CAP>
cudaError_t launch_grad_squares(const GradArgs<CAP>& a, int grid, cudaStream_t s);
cudaError_t launch_grad_norm(const double* partials, int n, float* norm, cudaStream_t s);
template <int CAP>
cudaError_t launch_grad_clip(const GradArgs<CAP>& a, cudaStream_t s);

}  // namespace vc
