// decoder_host.cpp -- the entry points of the block norm, the mixture of experts and the sampling without
// a GPU: device memory is host memory, a launch keeps the arguments that it was given, and the
// communicator is the five functions below.
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#include "moe.h"
#include "operators.h"
#include "sample.h"

namespace {

int g_ranks = 1, g_grouping = 0, g_launches = 0, g_tracked = 0;
vc::BlockNormArgs g_block;
vc::BlockNormBackwardArgs g_back;
vc::RouteArgs g_route;
vc::ExpertsArgs g_experts;
vc::MoeTiles g_tiles;
vc::SampleArgs g_sample;
std::vector<std::function<vResult_t()>> g_recorded;

}  // namespace

namespace vc {

size_t dtype_size(int dt) { return dt == vFloat32 || dt == vInt32 ? 4 : dt == vFloat16 || dt == vBFloat16 ? 2 : 0; }

vResult_t comm_view(vcomm_t c, CommView* v) {
    if (!c) return vInvalidArgument;
    *v = {};
    v->nRanks = g_ranks;
    v->smCount = 152;
    v->grouping = g_grouping != 0;
    v->timeoutNs = 7654321;
    v->testStallRank = 5;
    return vSuccess;
}
vResult_t comm_record(vcomm_t, std::function<vResult_t()> call) {
    g_recorded.push_back(std::move(call));
    return vSuccess;
}
vResult_t comm_launch(vcomm_t, const char*, const std::function<cudaError_t()>& launch) {
    return launch() == cudaSuccess ? vSuccess : vUnhandledCudaError;
}
vResult_t comm_launch_tracked(vcomm_t, const char*, cudaStream_t, const std::function<cudaError_t()>& launch) {
    g_tracked++;
    return launch() == cudaSuccess ? vSuccess : vUnhandledCudaError;
}

cudaError_t launch_allreduce_rmsnorm(const NormArgs&, vDataType_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_allreduce_rmsnorm_quant(const NormArgs&, vDataType_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs&, vDataType_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_grad_norm(const GradNormArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_grad_clip(const GradClipArgs&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_block_norm(const BlockNormArgs& a, vDataType_t, cudaStream_t) { return g_launches++, g_block = a, cudaSuccess; }
cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs& a, vDataType_t, cudaStream_t) {
    return g_launches++, g_back = a, cudaSuccess;
}
cudaError_t launch_moe_route(const RouteArgs& a, vDataType_t, cudaStream_t) { return g_launches++, g_route = a, cudaSuccess; }
cudaError_t launch_moe_experts(const ExpertsArgs& a, cudaStream_t) {
    g_tiles = {};
    return g_launches++, g_experts = a, cudaSuccess;
}
cudaError_t launch_moe_tiles(const ExpertsArgs& a, const MoeTiles& t, vDataType_t, cudaStream_t) {
    return g_launches++, g_experts = a, g_tiles = t, cudaSuccess;
}
cudaError_t launch_sample(const SampleArgs& a, vDataType_t, cudaStream_t) { return g_launches++, g_sample = a, cudaSuccess; }

}  // namespace vc

extern "C" {

cudaError_t cudaMalloc(void** p, size_t n) { return *p = std::malloc(n), cudaSuccess; }
cudaError_t cudaFree(void* p) { return std::free(p), cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { return std::memcpy(d, s, n), cudaSuccess; }
cudaError_t cudaMemset(void* d, int v, size_t n) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }

void host_start(int ranks) {
    g_ranks = ranks;
    g_grouping = g_launches = g_tracked = 0;
    g_recorded.clear();
}
int host_launches() { return g_launches; }
int host_tracked() { return g_tracked; }
void host_group(int on) { g_grouping = on; }
int host_group_end() {
    g_grouping = 0;
    vResult_t first = vSuccess;
    for (auto& call : g_recorded) {
        const vResult_t r = call();
        if (r != vSuccess && first == vSuccess) first = r;
    }
    g_recorded.clear();
    return first;
}
static void put(int* out, const vc::NormShape& s) {
    const int fields[] = {s.vecs, s.teamThreads, s.rowsPerCta, s.cluster, s.threads, s.staged, s.rounds, s.ctas, s.smemBytes};
    std::memcpy(out, fields, sizeof(fields));
}
void host_block(int* out) { put(out, g_block.shape); }
void host_back(int* out) { put(out, g_back.shape), out[9] = g_back.parts; }
void host_route(int* out) {
    const int fields[] = {g_route.cluster, g_route.share, g_route.aligned};
    std::memcpy(out, fields, sizeof(fields));
}
void host_experts(int* out) {
    const vc::MoeTiles& t = g_tiles;
    const int slots = g_experts.rows * g_experts.topK;
    const int fields[] = {t.tokens, t.splitUp, t.splitDown, t.gridUp, t.gridDown, t.stagesUp, t.stagesDown, t.combineHere,
                          t.tokens ? vc::moe_tiles_smem(g_experts.experts, slots, t.tokens, true, t.splitUp, t.stagesUp) : 0,
                          t.tokens ? vc::moe_tiles_smem(g_experts.experts, slots, t.tokens, false, t.splitDown, t.stagesDown) : 0,
                          g_experts.aligned, g_experts.tileUp, g_experts.tileDown, g_experts.share};
    std::memcpy(out, fields, sizeof(fields));
}
long long host_experts_limit() { return (long long)g_experts.timeoutNs; }
int host_experts_stall() { return g_experts.stallCta; }
void host_sample(int* out) {
    const int fields[] = {g_sample.cluster, g_sample.each, g_sample.nParts, g_sample.nOut, g_sample.part};
    std::memcpy(out, fields, sizeof(fields));
}

}  // extern "C"
