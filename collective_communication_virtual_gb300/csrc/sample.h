// sample.h -- argument block and launcher of the sampling from split logits.
#pragma once

#include "operators.h"

namespace vc {

constexpr int kSampleThreads = 512;
constexpr int kSampleCluster = 8;
constexpr int kSampleBins = 2048;
constexpr int kSampleMaxSmem = 192 * 1024;
constexpr int kSamplePair = 9;       // blocks of a thread that leave an SM room for two CTAs
constexpr int kSampleList = 2560;    // values above a row's bound that one CTA takes

struct SampleArgs {
    const void* logits[VCOMM_MAX_RANKS];     // rank r: columns [r part, (r + 1) part) of every row
    int* tokens[VCOMM_MAX_RANKS];            // the nOut outputs that are wanted
    const float* temperature;                // these four may be NULL
    const int* topK;
    const float* topP;
    const float* minP;
    const float* uniform;
    float* logprob;                          // may be NULL
    size_t stride;                           // elements between rows
    int rows, vocab, part;
    int nParts;                              // ranks that hold columns below vocab
    int nOut;
    int cluster;                             // CTAs that share a row
    int each;                                // 16-byte blocks of it that a thread has, at most
};
cudaError_t launch_sample(const SampleArgs& a, vDataType_t dt, cudaStream_t s);

}  // namespace vc
