// sample.cpp -- entry point of the sampling from logits whose columns are split over the ranks.
#include <cstdio>
#include <vector>

#include "entry.h"
#include "sample.h"

namespace {

vResult_t sample(const vSampleDesc_t* desc, const void* const* logits, const float* temperature, const int* topK,
                 const float* topP, const float* minP, const float* uniform, int* const* tokens, float* logprob, vcomm_t c,
                 cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    if (!desc) return vInvalidArgument;
    vSampleDesc_t d = *desc;
    if (!is_float(d.datatype) || d.vocab < 1 || d.vocab > VCOMM_MAX_VOCAB || d.rows > VCOMM_MAX_SAMPLE_ROWS)
        return vInvalidArgument;
    if (d.part == 0) d.part = (d.vocab + v.nRanks - 1) / v.nRanks;
    if (d.part > VCOMM_MAX_VOCAB || d.part * v.nRanks < d.vocab) return vInvalidArgument;
    if (d.stride == 0) d.stride = d.part;
    if (d.stride < d.part || d.stride > ((size_t)1 << 62) / (4 * VCOMM_MAX_SAMPLE_ROWS)) return vInvalidArgument;
    if (v.grouping) {
        if (!logits || !tokens) return vInvalidArgument;
        const std::vector<const void*> l(logits, logits + v.nRanks);
        const std::vector<int*> o(tokens, tokens + v.nRanks);
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                return sample(&d, l.data(), temperature, topK, topP, minP, uniform, o.data(), logprob, c, stream);
            });
        });
    }
    if (d.rows == 0) return vSuccess;
    const size_t esz = vc::dtype_size(d.datatype), e = 16 / esz;
    if (!logits || !tokens || !uniform) return vInvalidArgument;
    for (const void* p : {(const void*)temperature, (const void*)topK, (const void*)topP, (const void*)minP,
                          (const void*)uniform, (const void*)logprob})
        if (!at(p, 4)) return vInvalidArgument;
    vc::SampleArgs a;
    a.nOut = a.nParts = 0;
    for (int k = 0; k < v.nRanks; k++) {
        a.logits[k] = logits[k];
        if (k * d.part < d.vocab) {                    // else it holds no column that counts
            if (!logits[k] || !at(logits[k], esz)) return vInvalidArgument;
            a.nParts++;
        }
        if (!tokens[k]) continue;
        if (!at(tokens[k], 4)) return vInvalidArgument;
        a.tokens[a.nOut++] = tokens[k];
    }
    if (a.nOut == 0) return vInvalidArgument;
    a.temperature = temperature;
    a.topK = topK;
    a.topP = topP;
    a.minP = minP;
    a.uniform = uniform;
    a.logprob = logprob;
    a.stride = d.stride;
    a.rows = (int)d.rows;
    a.vocab = (int)d.vocab;
    a.part = (int)d.part;
    // Blocks of a row, at most (a part may begin and end inside one), in equal shares for the warps of a
    // cluster and their lanes.  As many CTAs as leave an SM room for two, and more while SMs are idle.
    const size_t blocks = d.vocab / e + 2 * (size_t)a.nParts;
    const auto each = [&]() { return (int)(((blocks + 16 * a.cluster - 1) / (16 * a.cluster) + 31) / 32); };
    a.cluster = 1;
    while (a.cluster < vc::kSampleCluster &&
           (each() > vc::kSamplePair || (each() > 1 && d.rows * a.cluster < (size_t)v.smCount))) a.cluster *= 2;
    a.each = each();
    if (v.debug)
        std::fprintf(stderr, "vcomm INFO Sample rows=%d vocab=%d dt=%d N=%d cluster=%d each=%d\n", a.rows, a.vocab,
                     (int)d.datatype, v.nRanks, a.cluster, a.each);
    return comm_launch(c, "sample", [&]() { return vc::launch_sample(a, d.datatype, stream); });
}

}  // namespace

extern "C" {

vResult_t vSample(const vSampleDesc_t* desc, const void* const* logitbuffs, const float* temperature, const int32_t* topK,
                  const float* topP, const float* minP, const float* uniform, int32_t* const* tokenbuffs, float* logprob,
                  vcomm_t comm, cudaStream_t stream) {
    Range range("vSample");
    return guarded([&]() {
        return sample(desc, logitbuffs, temperature, topK, topP, minP, uniform, tokenbuffs, logprob, comm, stream);
    });
}

}  // extern "C"
