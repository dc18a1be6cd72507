// operators_host.cpp -- the operators' entry points (csrc/operators.cpp) without a GPU: device
// memory is host memory, a launch is counted, and the communicator is the four functions below.
// That is all the operators may use of it: anything else leaves the link with an undefined name.
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <new>
#include <vector>

#include "operators.h"

namespace {

int g_ranks = 1, g_grouping = 0;
std::atomic<int> g_launches{0}, g_allocated{0};
std::vector<std::function<vResult_t()>> g_recorded;

}  // namespace

// Freed host objects keep their bytes, as they may under any allocator: a test that a handle is
// refused does not rest on what the next allocation writes.
void* operator new(size_t n) {
    if (void* p = std::malloc(n ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void*) noexcept {}
void operator delete(void*, size_t) noexcept {}

namespace vc {

size_t dtype_size(int dt) { return dt == vFloat32 || dt == vInt32 ? 4 : dt == vFloat16 || dt == vBFloat16 ? 2 : 0; }

vResult_t comm_view(vcomm_t c, CommView* v) {
    if (!c) return vInvalidArgument;
    v->nRanks = g_ranks;
    v->device = 0;
    v->smCount = 152;
    v->debug = false;
    v->grouping = g_grouping != 0;
    return vSuccess;
}
vResult_t comm_record(vcomm_t, std::function<vResult_t()> call) {
    g_recorded.push_back(std::move(call));
    return vSuccess;
}
vResult_t comm_launch(vcomm_t, const char*, const std::function<cudaError_t()>& launch) {
    return launch() == cudaSuccess ? vSuccess : vUnhandledCudaError;
}

cudaError_t launch_allreduce_rmsnorm(const NormArgs&, vDataType_t, cudaStream_t) { return g_launches++, cudaSuccess; }
cudaError_t launch_allreduce_rmsnorm_quant(const NormArgs&, vDataType_t, cudaStream_t) { return g_launches++, cudaSuccess; }
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs&, vDataType_t, cudaStream_t) { return g_launches++, cudaSuccess; }
cudaError_t launch_grad_norm(const GradNormArgs&, int, cudaStream_t) { return g_launches++, cudaSuccess; }
cudaError_t launch_grad_clip(const GradClipArgs&, cudaStream_t) { return g_launches++, cudaSuccess; }

}  // namespace vc

extern "C" {

cudaError_t cudaMalloc(void** p, size_t n) {
    g_allocated++;
    *p = std::malloc(n);
    return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
    g_allocated--;
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { return std::memcpy(d, s, n), cudaSuccess; }
cudaError_t cudaMemset(void* d, int v, size_t n) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }

void host_start(int ranks) {
    g_ranks = ranks;
    g_grouping = 0;
    g_launches = 0;
    g_recorded.clear();
}
int host_launches() { return g_launches; }
// The launch shape of a norm, as the fields that the tests read, in their order.
void host_norm_shape(size_t rows, int hidden, int elemSize, int weightSize, int segments, int general, int backward, int groups,
                     int* out) {
    vc::NormCall c = {};
    c.rows = rows;
    c.hidden = hidden;
    c.elemSize = elemSize;
    c.weightSize = weightSize;
    c.segments = segments;
    c.smCount = 152;
    c.general = general != 0;
    c.backward = backward != 0;
    c.groups = groups != 0;
    const vc::NormShape s = vc::norm_shape(c);
    const int fields[] = {s.vecs, s.teamThreads, s.rowsPerCta, s.cluster, s.threads, s.staged, s.rounds, s.ctas, s.smemBytes,
                          backward ? vc::norm_backward_parts(rows, s, 152) : 0};
    std::memcpy(out, fields, sizeof(fields));
}
int host_allocated() { return g_allocated; }
void host_group(int on) { g_grouping = on; }
// As vcommGroupEnd: runs what was recorded and returns the first error.
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

}  // extern "C"
