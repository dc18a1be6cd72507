// moe.h -- argument blocks and launchers of the mixture-of-experts operators: the router, and the
// experts' layer for a few tokens.
#pragma once

#include "operators.h"

namespace vc {

constexpr int kRouteFew = 4;         // tokens of a cluster where a warp takes an expert's whole row
constexpr int kRouteTile = 8;        // where it takes a tile
constexpr int kRouteCluster = 8;     // CTAs of a cluster, at most,
constexpr int kRouteTileCluster = 4; // and for many tiles: larger ones do not fill the SMs at one CTA on each
constexpr int kRouteThreads = 256;
constexpr int kRouteTileThreads = 512;
constexpr int kRouteMaxSmem = 180 * 1024;

struct RouteArgs {
    const void* x;
    const void* router;              // [experts][hidden]
    const float* bias;               // may be NULL
    int* ids;                        // [rows][topK]
    float* weights;
    size_t rowStride;
    int rows, hidden, experts, topK;
    int few;                         // a warp takes an expert's whole row, for up to four tokens, else a tile
    int cluster;                     // CTAs that share the experts
    int share;                       // experts of a CTA
    int routerF32;
    int normalize;
    int aligned;                     // every row of x and of the router starts on 16 bytes and ends with a vector
};
cudaError_t launch_moe_route(const RouteArgs& a, vDataType_t dt, cudaStream_t s);

struct ExpertsArgs {
    const void* up[VCOMM_MAX_RANKS];     // [the rank's experts][2 ffn][hidden]: the gate's rows, then the linear part's
    const void* down[VCOMM_MAX_RANKS];   // [the rank's experts][hidden][ffn]
    void* recv[VCOMM_MAX_RANKS];         // [rows][hidden], rank r's part of the sum
    const void* x;
    const int* ids;                  // [rows][topK]
    const float* weights;
    float* act;                      // workspace: what goes into the way down, [rows * topK][ffn], or, of 16-bit types,
                                     // [rows * topK][2][moe_act_stride(ffn)] of them
    float* y;                        // workspace: every slot's output, [rows * topK][hidden], or [..][moe_y_stride(hidden)]
    unsigned int* done;              // workspace: experts that have finished a tile of columns
    size_t rowStride, recvStride;
    int rows, hidden, ffn, experts, topK;
    int nRanks;
    int share;                       // experts of a rank
    int aligned;                     // every row of x and of the weights starts on 16 bytes and ends with a vector
    int tileUp, tileDown;            // fp32: output columns of a CTA, 8 to 32, and 16 or 32
    int recvAligned;                 // every row of the outputs starts on 8 bytes
    int split;                       // tensor cores: CTAs of a cluster that share a tile's columns
    int stages;                      // the same: stages of a CTA
    int combineHere;                 // the same: the way down adds up the slots
    Status* status;                  // device copy
    volatile Status* statusHost;     // pinned mirror
    unsigned long long timeoutNs;    // limit of every wait
    int stallCta;                    // test hook: this CTA of both launches copies no stage (-1 = off)
};
constexpr int kMoeTile = 8;          // output columns of a CTA, at least
cudaError_t launch_moe_experts(const ExpertsArgs& a, cudaStream_t s);

// The same on the tensor cores, of 16-bit types.
constexpr int kMoeMaxStages = 8;
constexpr int kMoeMaxSmem = 225 * 1024;
struct MoeGroup {                    // tokens of one expert, as many as a tile takes
    uint16_t expert, first, count;   // first: of its slots in the list
};
#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr int moe_act_stride(int ffn) { return (ffn + 7) / 8 * 8; }
#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr int moe_y_stride(int hidden) { return (hidden + 3) / 4 * 4; }
#if defined(__CUDACC__)
__host__ __device__
#endif
constexpr int moe_groups(int experts, int slots, int tokens) {
    return (experts < slots ? experts : slots) + slots / tokens;
}
// Dynamic shared memory of a CTA: stages, the sums of the other CTAs of a cluster, and the lists.
constexpr int moe_stage_bytes(int tokens, bool up) { return 128 * 256 + (up ? 1 : 2) * tokens * 256; }
constexpr int moe_tiles_smem(int experts, int slots, int tokens, bool up, int split, int stages) {
    return 1024 + stages * moe_stage_bytes(tokens, up) + (split - 1) * tokens * 128 * 4 + experts * 4 +
           moe_groups(experts, slots, tokens) * (int)sizeof(MoeGroup) + slots * 2;
}
struct MoeTiles {
    int tokens;                      // of a tile: 16, 32 or 64
    int splitUp, splitDown;          // CTAs of a cluster that share a tile's columns: 1, 2 or 4
    int gridUp, gridDown;
    int stagesUp, stagesDown;
    int combineHere;                 // few tokens: no third launch
};
cudaError_t launch_moe_tiles(const ExpertsArgs& a, const MoeTiles& t, vDataType_t dt, cudaStream_t s);

}  // namespace vc
