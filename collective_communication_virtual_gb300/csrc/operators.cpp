// operators.cpp -- entry points of the operators that run next to the collectives: argument
// checks, launch shapes and launches on the caller's stream.  Errors follow the collectives':
// a bad argument returns vInvalidArgument and launches nothing, the communicator's sticky
// error is returned by every call, and nothing is thrown through the C interface.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <vector>

#include "operators.h"

namespace vc {

// Launch shape of the norm kernels.
NormShape norm_shape(size_t rows, int hidden, int elemSize, int smCount, bool general) {
    const int E = 16 / elemSize;
    // a row that may start inside an aligned vector touches up to one vector more
    const int nv = general ? (hidden + 2 * E - 2) / E : hidden / E;
    NormShape s;
    s.general = general ? 1 : 0;
    s.cluster = 1;
    if (nv <= 128) {                 // a row fits 4 vectors of each lane of a warp
        s.vecs = nv <= 32 ? 1 : nv <= 64 ? 2 : 4;
        s.teamThreads = 1;
        while (s.teamThreads * s.vecs < nv) s.teamThreads *= 2;
        s.threads = kNormWarpCta;
        s.rowsPerCta = s.threads / s.teamThreads;
        return s;
    }
    // rows longer than a CTA's registers hold
    while ((nv + s.cluster - 1) / s.cluster > kNormMaxThreads * 4) s.cluster *= 2;
    // few rows: split each over more CTAs while SMs are idle
    while (s.cluster < kNormMaxCluster && rows * (size_t)s.cluster * 2 <= (size_t)smCount &&
           nv / (s.cluster * 2) >= 64)
        s.cluster *= 2;
    const int per = (nv + s.cluster - 1) / s.cluster;
    s.vecs = per <= 512 ? 1 : per <= 1024 ? 2 : 4;
    s.teamThreads = ((per + s.vecs - 1) / s.vecs + 31) / 32 * 32;
    s.threads = s.teamThreads;
    s.rowsPerCta = 1;
    return s;
}

int norm_backward_parts(size_t rows, const NormShape& sh, int smCount) {
    const int resident = sh.vecs == 1 ? 1024 : 512;    // threads of an SM, by their registers
    const int perSm = std::max(1, resident / sh.threads);
    const size_t most = std::max<size_t>(1, (size_t)smCount * perSm / sh.cluster);
    return (int)std::min(most, (rows + sh.rowsPerCta - 1) / sh.rowsPerCta);
}

}  // namespace vc

namespace {

using vc::comm_launch;
using vc::comm_view;
using vc::CommView;

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

bool is_float(int dt) { return dt == vFloat32 || dt == vFloat16 || dt == vBFloat16; }

bool at(const void* p, size_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

// Run `f`, giving vSystemError for a failed allocation.
template <typename F>
vResult_t guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return vSystemError;
    } catch (...) {
        return vInternalError;
    }
}

struct Checked {
    vRmsNormDesc_t d;                // strides filled in
    int esz;
};

vResult_t check_desc(const vRmsNormDesc_t* desc, Checked* k) {
    if (!desc) return vInvalidArgument;
    vRmsNormDesc_t& d = k->d;
    d = *desc;
    if (!is_float(d.datatype)) return vInvalidArgument;
    if (d.weightType != vFloat32 && d.weightType != d.datatype) return vInvalidArgument;
    if (d.hidden > VCOMM_MAX_HIDDEN || d.rows > 0x7FFFFFFFull) return vInvalidArgument;
    if (!(d.eps >= 0.0f) || std::isinf(d.eps)) return vInvalidArgument;
    if (d.quantGroup != 0 && d.quantGroup != vc::kQuantGroup) return vInvalidArgument;
    for (size_t* s : {&d.sendStride, &d.residualStride, &d.recvStride}) {
        if (*s == 0) *s = d.hidden;
        if (*s < d.hidden || *s > ((size_t)1 << 62) / (4 * std::max<size_t>(1, d.rows))) return vInvalidArgument;
    }
    k->esz = (int)vc::dtype_size(d.datatype);
    return vSuccess;
}

// The sends, the wanted outputs (compacted into `out`, their indices into `index`) and
// whether every vector of every row starts on a 16-byte boundary (an output of osz-byte
// elements: on one of its own vectors' size).
struct Buffers {
    int nOut = 0;
    bool aligned = true;
};
vResult_t check_buffers(const Checked& k, int nRanks, const void* const* send, void* const* recv, int osz,
                        const void** sendOut, void** out, int* index, Buffers* b) {
    const vRmsNormDesc_t& d = k.d;
    if (!send || !recv) return vInvalidArgument;
    const size_t e = 16 / (size_t)k.esz;
    b->aligned = d.hidden % e == 0 &&
                 (d.rows == 1 || (d.sendStride % e == 0 && d.residualStride % e == 0 && d.recvStride % e == 0));
    for (int r = 0; r < nRanks; r++) {
        if (!send[r] || !at(send[r], k.esz)) return vInvalidArgument;
        sendOut[r] = send[r];
        b->aligned = b->aligned && at(send[r], 16);
        if (!recv[r]) continue;
        if (!at(recv[r], osz)) return vInvalidArgument;
        b->aligned = b->aligned && at(recv[r], e * osz);
        if (index) index[b->nOut] = r;
        out[b->nOut++] = recv[r];
    }
    return b->nOut ? vSuccess : vInvalidArgument;
}

vResult_t check_weight(const Checked& k, const void* weight, Buffers* b) {
    if (!weight || !at(weight, vc::dtype_size(k.d.weightType))) return vInvalidArgument;
    b->aligned = b->aligned && at(weight, 16);
    return vSuccess;
}
vResult_t check_row_buffer(const Checked& k, const void* p, Buffers* b) {
    if (!p) return vSuccess;
    if (!at(p, k.esz)) return vInvalidArgument;
    b->aligned = b->aligned && at(p, 16);
    return vSuccess;
}

vResult_t norm_forward(const vRmsNormDesc_t* desc, const void* const* send, const void* residual, const void* weight,
                       void* residualOut, void* const* recv, float* const* scales, bool quant, float* rstd, vcomm_t c,
                       cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_desc(desc, &k)) != vSuccess) return r;
    if (v.grouping) {
        if (!send || !recv || (quant && !scales)) return vInvalidArgument;
        const vRmsNormDesc_t d = *desc;
        const std::vector<const void*> s(send, send + v.nRanks);
        const std::vector<void*> o(recv, recv + v.nRanks);
        const std::vector<float*> q = quant ? std::vector<float*>(scales, scales + v.nRanks) : std::vector<float*>();
        return vc::comm_record(c, [=]() {   // allocates nothing when it runs
            return norm_forward(&d, s.data(), residual, weight, residualOut, o.data(), q.data(), quant, rstd, c, stream);
        });
    }
    if (k.d.rows == 0 || k.d.hidden == 0) return vSuccess;
    vc::NormArgs a;
    int index[VCOMM_MAX_RANKS];
    Buffers b;
    if ((r = check_buffers(k, v.nRanks, send, recv, quant ? 1 : k.esz, a.send, a.recv, index, &b)) != vSuccess) return r;
    if ((r = check_weight(k, weight, &b)) != vSuccess) return r;
    if ((r = check_row_buffer(k, residual, &b)) != vSuccess) return r;
    if ((r = check_row_buffer(k, residualOut, &b)) != vSuccess) return r;
    if (!at(rstd, 4)) return vInvalidArgument;
    if (quant) {
        if (!scales) return vInvalidArgument;
        for (int o = 0; o < b.nOut; o++) {
            a.scales[o] = scales[index[o]];
            if (!a.scales[o] || !at(a.scales[o], 4)) return vInvalidArgument;
        }
    }
    a.residual = residual;
    a.residualOut = residualOut;
    a.weight = weight;
    a.rstd = rstd;
    a.rows = k.d.rows;
    a.sendStride = k.d.sendStride;
    a.residualStride = k.d.residualStride;
    a.recvStride = k.d.recvStride;
    a.hidden = (int)k.d.hidden;
    a.nRanks = v.nRanks;
    a.nOut = b.nOut;
    a.weightF32 = k.d.weightType == vFloat32;
    a.groups = k.d.quantGroup ? (int)((k.d.hidden + vc::kQuantGroup - 1) / vc::kQuantGroup) : 0;
    a.eps = k.d.eps;
    a.shape = vc::norm_shape(a.rows, a.hidden, k.esz, v.smCount, !b.aligned);
    return comm_launch(c, quant ? "allreduce rmsnorm quant" : "allreduce rmsnorm", [&]() {
        return quant ? vc::launch_allreduce_rmsnorm_quant(a, k.d.datatype, stream)
                     : vc::launch_allreduce_rmsnorm(a, k.d.datatype, stream);
    });
}

vResult_t norm_backward(const vRmsNormDesc_t* desc, const void* const* send, const void* hidden, const float* rstd,
                        const void* weight, const void* gradResidual, void* const* recv, void* gradWeight,
                        void* workspace, size_t workspaceBytes, vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_desc(desc, &k)) != vSuccess) return r;
    if (v.grouping) {
        if (!send || !recv) return vInvalidArgument;
        const vRmsNormDesc_t d = *desc;
        const std::vector<const void*> s(send, send + v.nRanks);
        const std::vector<void*> o(recv, recv + v.nRanks);
        return vc::comm_record(c, [=]() {
            return norm_backward(&d, s.data(), hidden, rstd, weight, gradResidual, o.data(), gradWeight, workspace,
                                 workspaceBytes, c, stream);
        });
    }
    if (k.d.hidden == 0) return vSuccess;
    const size_t wsz = vc::dtype_size(k.d.weightType);
    if (!gradWeight || !at(gradWeight, wsz)) return vInvalidArgument;
    if (k.d.rows == 0)               // a sum over no rows
        return comm_launch(c, "rmsnorm backward", [&]() {
            return cudaMemsetAsync(gradWeight, 0, k.d.hidden * wsz, stream);
        });
    vc::NormBackwardArgs a;
    Buffers b;
    if ((r = check_buffers(k, v.nRanks, send, recv, k.esz, a.send, a.recv, nullptr, &b)) != vSuccess) return r;
    if ((r = check_weight(k, weight, &b)) != vSuccess) return r;
    if (!hidden || !rstd || !at(rstd, 4)) return vInvalidArgument;
    if ((r = check_row_buffer(k, hidden, &b)) != vSuccess) return r;
    if ((r = check_row_buffer(k, gradResidual, &b)) != vSuccess) return r;
    a.hidden = hidden;
    a.gradResidual = gradResidual;
    a.weight = weight;
    a.rstd = rstd;
    a.partials = (float*)workspace;
    a.gradWeight = gradWeight;
    a.rows = k.d.rows;
    a.sendStride = k.d.sendStride;
    a.residualStride = k.d.residualStride;
    a.recvStride = k.d.recvStride;
    a.width = (int)k.d.hidden;
    a.nRanks = v.nRanks;
    a.nOut = b.nOut;
    a.weightF32 = k.d.weightType == vFloat32;
    a.shape = vc::norm_shape(a.rows, a.width, k.esz, v.smCount, !b.aligned);
    a.parts = vc::norm_backward_parts(a.rows, a.shape, v.smCount);
    if (!workspace || !at(workspace, 16) || workspaceBytes < (size_t)a.parts * k.d.hidden * sizeof(float))
        return vInvalidArgument;
    return comm_launch(c, "rmsnorm backward", [&]() { return vc::launch_rmsnorm_backward(a, k.d.datatype, stream); });
}

// ---- gradient norm and clipping ----------------------------------------------------------

// Partial sums of one launch.
constexpr int kSquaresCtasPerSm = 4;

vResult_t check_list(const vTensorList_t* l, int nRanks) {
    if (!l || l->nTensors < 0) return vInvalidArgument;
    if (l->nTensors == 0) return vSuccess;
    if (!l->counts || !l->datatypes || !l->grads || (size_t)l->nTensors > (size_t)0x7FFFFFFF / nRanks)
        return vInvalidArgument;
    const size_t most = (size_t)1 << 43;     // of all pieces together: their chunks fit one grid
    size_t total = 0;
    for (int t = 0; t < l->nTensors; t++) {
        if (!is_float(l->datatypes[t]) || l->counts[t] > (most - total) / nRanks) return vInvalidArgument;
        total += l->counts[t] * nRanks;
        if (l->counts[t] == 0) continue;
        const size_t esz = vc::dtype_size(l->datatypes[t]);
        for (int r = 0; r < nRanks; r++) {
            const size_t i = (size_t)r * l->nTensors + t;
            if (!l->grads[i] || !at(l->grads[i], esz)) return vInvalidArgument;
            if (l->outs && (!l->outs[i] || !at(l->outs[i], esz))) return vInvalidArgument;
        }
    }
    return vSuccess;
}

// Call f(item) for every piece that the norm counts (`all` false) or that is scaled.
template <typename F>
void each_item(const vTensorList_t* l, int nRanks, bool all, F f) {
    for (int r = 0; r < nRanks; r++)
        for (int t = 0; t < l->nTensors; t++) {
            if (l->counts[t] == 0 || (!all && r > 0 && l->replicated && l->replicated[t])) continue;
            const size_t i = (size_t)r * l->nTensors + t;
            vc::GradItem it;
            it.in = l->grads[i];
            it.out = l->outs ? l->outs[i] : const_cast<void*>(l->grads[i]);
            it.count = l->counts[t];
            it.chunk0 = 0;
            it.dt = (unsigned)l->datatypes[t];
            f(it);
        }
}

size_t count_items(const vTensorList_t* l, int nRanks, bool all) {
    size_t whole = 0, split = 0;
    for (int t = 0; t < l->nTensors; t++) {
        if (l->counts[t] == 0) continue;
        if (!all && l->replicated && l->replicated[t]) whole++;
        else split++;
    }
    return whole + split * (size_t)nRanks;
}

// Batches of the items in launches of at most CAP.
template <int CAP, typename F>
vResult_t batches(const vTensorList_t* l, int nRanks, bool all, F launch) {
    std::unique_ptr<vc::GradArgs<CAP>> a(new vc::GradArgs<CAP>);
    a->nItems = 0;
    unsigned long long chunks = 0;
    vResult_t res = vSuccess;
    const auto flush = [&]() {
        if (a->nItems == 0 || res != vSuccess) return;
        a->nChunks = (unsigned)chunks;
        res = launch(*a);
        a->nItems = 0;
        chunks = 0;
    };
    each_item(l, nRanks, all, [&](vc::GradItem it) {
        const unsigned long long n = vc::grad_chunks(it.count, vc::dtype_size((int)it.dt));
        if (a->nItems == CAP) flush();
        it.chunk0 = (unsigned)chunks;
        a->items[a->nItems++] = it;
        chunks += n;
    });
    flush();
    return res;
}

size_t squares_slots(const vTensorList_t* l, const CommView& v) {
    const size_t n = count_items(l, v.nRanks, false);
    return (n + vc::kGradItemsLarge - 1) / vc::kGradItemsLarge * (size_t)v.smCount * kSquaresCtasPerSm;
}

template <int CAP>
vResult_t enqueue_norm(const vTensorList_t* l, const CommView& v, double* partials, float* norm, vcomm_t c,
                       cudaStream_t stream) {
    int used = 0;
    const vResult_t r = batches<CAP>(l, v.nRanks, false, [&](vc::GradArgs<CAP>& a) {
        const int grid = (int)std::min<unsigned>(a.nChunks, (unsigned)(v.smCount * kSquaresCtasPerSm));
        a.partials = partials + used;
        used += grid;
        return comm_launch(c, "gradient squares", [&]() { return vc::launch_grad_squares<CAP>(a, grid, stream); });
    });
    if (r != vSuccess) return r;
    return comm_launch(c, "gradient norm", [&]() { return vc::launch_grad_norm(partials, used, norm, stream); });
}
template <int CAP>
vResult_t enqueue_clip(const vTensorList_t* l, const CommView& v, float maxNorm, const float* norm, vcomm_t c,
                       cudaStream_t stream) {
    return batches<CAP>(l, v.nRanks, true, [&](vc::GradArgs<CAP>& a) {
        a.norm = norm;
        a.maxNorm = maxNorm;
        return comm_launch(c, "gradient clip", [&]() { return vc::launch_grad_clip<CAP>(a, stream); });
    });
}

struct ListCopy {
    std::vector<size_t> counts;
    std::vector<vDataType_t> types;
    std::vector<unsigned char> replicated;
    std::vector<const void*> grads;
    std::vector<void*> outs;
    vTensorList_t list() const {
        vTensorList_t l;
        l.nTensors = (int)counts.size();
        l.counts = counts.data();
        l.datatypes = types.data();
        l.replicated = replicated.empty() ? nullptr : replicated.data();
        l.grads = grads.data();
        l.outs = outs.empty() ? nullptr : outs.data();
        return l;
    }
};

vResult_t grad_norm(const vTensorList_t* l, bool clip, float maxNorm, float* norm, void* workspace,
                    size_t workspaceBytes, vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    if ((r = check_list(l, v.nRanks)) != vSuccess) return r;
    if (!norm || !at(norm, 4)) return vInvalidArgument;
    if (clip && !(maxNorm >= 0.0f)) return vInvalidArgument;
    if (!workspace || !at(workspace, 16) || workspaceBytes < squares_slots(l, v) * sizeof(double))
        return vInvalidArgument;
    if (v.grouping) {
        auto k = std::make_shared<ListCopy>();
        const size_t n = (size_t)l->nTensors, all = n * v.nRanks;
        k->counts.assign(l->counts, l->counts + n);
        k->types.assign(l->datatypes, l->datatypes + n);
        if (l->replicated) k->replicated.assign(l->replicated, l->replicated + n);
        k->grads.assign(l->grads, l->grads + all);
        if (l->outs) k->outs.assign(l->outs, l->outs + all);
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                const vTensorList_t copy = k->list();
                return grad_norm(&copy, clip, maxNorm, norm, workspace, workspaceBytes, c, stream);
            });
        });
    }
    double* partials = (double*)workspace;
    r = count_items(l, v.nRanks, false) <= (size_t)vc::kGradItemsSmall
            ? enqueue_norm<vc::kGradItemsSmall>(l, v, partials, norm, c, stream)
            : enqueue_norm<vc::kGradItemsLarge>(l, v, partials, norm, c, stream);
    if (r != vSuccess || !clip) return r;
    return count_items(l, v.nRanks, true) <= (size_t)vc::kGradItemsSmall
               ? enqueue_clip<vc::kGradItemsSmall>(l, v, maxNorm, norm, c, stream)
               : enqueue_clip<vc::kGradItemsLarge>(l, v, maxNorm, norm, c, stream);
}

}  // namespace

extern "C" {

vResult_t vAllReduceRmsNorm(const vRmsNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                            const void* weight, void* residualOut, void* const* recvbuffs, float* rstd, vcomm_t comm,
                            cudaStream_t stream) {
    Range range("vAllReduceRmsNorm");
    return guarded([&]() {
        return norm_forward(desc, sendbuffs, residual, weight, residualOut, recvbuffs, nullptr, false, rstd, comm, stream);
    });
}

vResult_t vAllReduceRmsNormQuant(const vRmsNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                                 const void* weight, void* residualOut, void* const* recvbuffs,
                                 float* const* scalebuffs, float* rstd, vcomm_t comm, cudaStream_t stream) {
    Range range("vAllReduceRmsNormQuant");
    return guarded([&]() {
        return norm_forward(desc, sendbuffs, residual, weight, residualOut, recvbuffs, scalebuffs, true, rstd, comm, stream);
    });
}

vResult_t vRmsNormBackwardWorkspace(const vRmsNormDesc_t* desc, vcomm_t comm, size_t* bytes) {
    CommView v;
    vResult_t r = comm_view(comm, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_desc(desc, &k)) != vSuccess) return r;
    if (!bytes) return vInvalidArgument;
    *bytes = 16;
    if (k.d.rows == 0 || k.d.hidden == 0) return vSuccess;
    // whatever the buffers' alignment turns out to be
    for (const bool general : {false, true}) {
        if (!general && k.d.hidden % (16 / k.esz) != 0) continue;
        const vc::NormShape s = vc::norm_shape(k.d.rows, (int)k.d.hidden, k.esz, v.smCount, general);
        *bytes = std::max(*bytes, (size_t)vc::norm_backward_parts(k.d.rows, s, v.smCount) * k.d.hidden * sizeof(float));
    }
    return vSuccess;
}

vResult_t vAllReduceRmsNormBackward(const vRmsNormDesc_t* desc, const void* const* sendbuffs, const void* hiddenStates,
                                    const float* rstd, const void* weight, const void* gradResidual,
                                    void* const* recvbuffs, void* gradWeight, void* workspace, size_t workspaceBytes,
                                    vcomm_t comm, cudaStream_t stream) {
    Range range("vAllReduceRmsNormBackward");
    return guarded([&]() {
        return norm_backward(desc, sendbuffs, hiddenStates, rstd, weight, gradResidual, recvbuffs, gradWeight, workspace,
                             workspaceBytes, comm, stream);
    });
}

vResult_t vGradNormWorkspace(const vTensorList_t* list, vcomm_t comm, size_t* bytes) {
    CommView v;
    vResult_t r = comm_view(comm, &v);
    if (r != vSuccess) return r;
    if ((r = check_list(list, v.nRanks)) != vSuccess) return r;
    if (!bytes) return vInvalidArgument;
    *bytes = std::max<size_t>(16, squares_slots(list, v) * sizeof(double));
    return vSuccess;
}

vResult_t vGradNorm(const vTensorList_t* list, float* norm, void* workspace, size_t workspaceBytes, vcomm_t comm,
                    cudaStream_t stream) {
    Range range("vGradNorm");
    return guarded([&]() { return grad_norm(list, false, 0.0f, norm, workspace, workspaceBytes, comm, stream); });
}

vResult_t vClipGradNorm(const vTensorList_t* list, float maxNorm, float* norm, void* workspace, size_t workspaceBytes,
                        vcomm_t comm, cudaStream_t stream) {
    Range range("vClipGradNorm");
    return guarded([&]() { return grad_norm(list, true, maxNorm, norm, workspace, workspaceBytes, comm, stream); });
}

}  // extern "C"
