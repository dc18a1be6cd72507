// operators.cpp -- entry points of the operators that run next to the collectives: argument
// checks, launch shapes and launches on the caller's stream.  Errors follow the collectives':
// a bad argument returns vInvalidArgument and launches nothing, the communicator's sticky
// error is returned by every call, and nothing is thrown through the C interface.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "operators.h"

namespace vc {

namespace {

// Threads of a team that holds `vecs` vectors a thread of a row of nv vectors: part of a warp,
// or whole warps.
int team_threads(int nv, int vecs) {
    const int need = (nv + vecs - 1) / vecs;
    if (need > 32) return (need + 31) / 32 * 32;
    int t = 1;
    while (t < need) t *= 2;
    return t;
}
void set_team(NormShape* s, int nv, int vecs) {
    s->vecs = vecs;
    s->teamThreads = team_threads(nv, vecs);
    s->threads = s->teamThreads > 32 ? s->teamThreads : kNormWarpCta;
    s->rowsPerCta = s->threads / s->teamThreads;
}

}  // namespace

// Launch shape of the norm kernels.
NormShape norm_shape(const NormCall& c) {
    const int E = 16 / c.elemSize;
    const int nv = (c.hidden + E - 1) / E;
    NormShape s = {};
    s.general = c.general ? 1 : 0;
    s.cluster = 1;
    // Bytes of dynamic shared memory for the shape as it stands.
    const auto layout = [&]() {
        s.extraBytes = c.backward ? s.threads * s.vecs * E * (int)sizeof(float) : 0;
        s.weightBytes = s.staged ? s.teamThreads * s.vecs * E * c.weightSize : 0;
        s.stageBytes = s.staged ? (c.segments * s.vecs * stage_blocks(s.threads, s.teamThreads, c.general) + 1) * 16 : 0;
        // a row's vectors, and the block behind them that a realigned read may touch
        s.rowBytes = c.general ? s.teamThreads * s.vecs * 16 + 16 : 0;
        s.smemBytes = s.extraBytes + s.weightBytes + s.stageBytes + s.rowBytes * (c.backward ? 1 : 2) * s.rowsPerCta;
    };

    // Staged: more vectors a thread means fewer instructions and barriers a row, as long as the
    // last warp is not left half empty.  With few rows per SM and several inputs a row's latency
    // counts for more (3 x 1537 x 2731: 21 us with two vectors, 24 with four; but 1 x 1500 x 4096:
    // 13 and 11).  The backward pass keeps its sums in registers with two (1 x 16384 x 4096: 95 us,
    // 104 with four), but rows that fill a warp save more with four (1 x 16000 x 1024: 33 and 29).
    const bool few = c.rows <= (size_t)c.smCount * 16 && c.segments >= 4;
    const int most = 228 * 1024, overhead = 1024 + kNormStaticSmem;    // the SM's; a CTA's own and its static arrays
    const auto stage = [&]() {
        const int part = (nv + s.cluster - 1) / s.cluster;
        double best = 0;
        for (const int vecs : {4, 2, 1}) {
            const int team = team_threads(part, vecs);
            // a scale group is found in neighbouring lanes: no team of fewer lanes than it spans
            if (c.groups && vecs > 1 && team * E < kQuantGroup) continue;
            // a cluster's CTAs are whole teams of several warps
            if (team > kStageMaxThreads || (s.cluster > 1 && team <= 32)) continue;
            const bool four = !few && (!c.backward || team == 32);
            const double weight = vecs == 4 ? (four ? 1.0 : 0.8) : vecs == 2 ? 0.92 : 0.8;
            const double use = weight * part / ((double)team * vecs);
            if (use > best) {
                best = use;
                set_team(&s, part, vecs);
            }
        }
        if (best == 0) return false;
        layout();
        // CTAs of small teams: several rows each, but no more than keep the SM's CTAs several too
        while (s.teamThreads <= 32 && s.threads > 32 && s.threads > s.teamThreads && s.stageBytes > 40 * 1024) {
            s.threads /= 2;
            s.rowsPerCta = s.threads / s.teamThreads;
            layout();
        }
        return s.smemBytes + overhead <= most;
    };
    // A row too long for one CTA's threads or shared memory is shared by the CTAs of a cluster: of
    // eight in the forward pass, which leaves an SM several (8 x 1500 x 16384: 147 us, 162 of four,
    // 170 of two, 189 with direct loads); of two where the rows are strided over, as larger
    // clusters do not fill all SMs at once (backward, 1 x 2000 x 16384 fp32: 120 us, 300 of four,
    // 192 with direct loads).  Rows that direct loads hold with two vectors a thread are no faster
    // that way (32 x 2000 x 4096: 171 us, 195 of eight; backward, 16 x 2000 x 8192: 214, 226 of
    // two), unless they are unaligned (backward, 16 x 2000 x 9001: 299 us, 464 with direct loads).
    s.staged = 1;
    bool fits = stage();
    if (!fits && (c.general || nv > kNormMaxThreads * 2)) {
        s.cluster = c.backward || c.general ? 2 : kNormMaxCluster;
        fits = stage();
    }
    if (fits) {
        // Registers of a thread, at most: the launch bounds give 64 and 128, and the forward instances
        // with two vectors take 80 to 107 (in eights).
        const int regs = s.vecs == 1 ? 64 : s.vecs == 2 && !c.backward ? 112 : 128;
        const size_t groups = (c.rows + s.rowsPerCta - 1) / s.rowsPerCta;
        // About 72 KiB under way per SM: less leaves the memory waiting, more makes it slower
        // where the CTAs do not keep step.  (48 KiB in the backward pass with two vectors a thread.)
        const int goal = c.backward && s.vecs == 2 ? 48 * 1024 : 72 * 1024;
        const int aim = (goal + s.stageBytes - 1) / s.stageBytes;
        const int fit = std::max(1, std::min({most / (s.smemBytes + overhead), 65536 / (regs * s.threads), 16}));
        // unaligned rows take more instructions than one CTA issues while it waits (8 x 2000 x 4097:
        // 92 us with one, 67 with two)
        const int perSm = std::min(c.general ? std::max(2, aim) : aim, fit);
        const size_t wave = std::max<size_t>(1, (size_t)c.smCount * perSm / s.cluster);
        // few rows shared by eight CTAs: direct loads (8 x 150 x 16384: 17.5 us, staged 20)
        s.staged = groups > wave && (s.cluster <= 2 || c.rows > (size_t)c.smCount);
        if (c.backward || (c.general && aim == 1)) {
            // Every SM its share of the one wave: enough shared memory that no more fit, or CTAs
            // that arrive while another kernel still holds some SMs crowd on the others (two of
            // 152 CTAs on some SMs: 8 x 4096 x 4096 backward 102 -> 126 us).
            s.ctas = (int)wave;
            if (s.staged && perSm <= 6) s.smemBytes = std::max(s.smemBytes, 228 * 1024 / (perSm + 1));
        } else {
            // Up to four rows a CTA (cluster), or as many as make one wave of CTAs: a wave costs its
            // rows and a prologue of about 0.6 of one, and a wave that is nearly empty costs as much
            // as a full one (2 x 1500 x 8192, a wave of 304: 26 us with 3 or 5 rows a CTA, 31 with 4).
            // With two long rows an SM and many waves, two are enough (4 x 4096 x 5120: 65 us with
            // two, 68 with four; 1 x 16384 x 4096 to 8 bits, with more an SM: 79 and 74).
            const size_t resident = std::max<size_t>(1, (size_t)c.smCount * fit / s.cluster);
            const size_t one = (groups + resident - 1) / resident;
            const size_t cap = aim <= 2 && fit >= 2 && !c.general ? 2 : 4;
            double least = 0;
            for (size_t r = 1; r <= 6; r++) {
                if (r > cap && (r != one || s.cluster > 1)) continue;
                const double cost = (double)(((groups + r - 1) / r + resident - 1) / resident) * ((double)r + 0.6);
                if (s.rounds == 0 || cost < least) {
                    least = cost;
                    s.rounds = (int)r;
                }
            }
            s.ctas = (int)((groups + s.rounds - 1) / s.rounds);
        }
    }
    if (!fits || !s.staged) {        // few rows, or a row that not even a cluster can stage
        s.staged = 0;
        s.cluster = 1;
        if (nv <= 32) {              // one vector a thread, as the latency counts
            set_team(&s, nv, 1);
        } else {
            // rows longer than a CTA's registers hold
            while ((nv + s.cluster - 1) / s.cluster > kNormMaxThreads * 4) s.cluster *= 2;
            // few rows: split each over more CTAs while SMs are idle
            while (s.cluster < kNormMaxCluster && c.rows * (size_t)s.cluster * 2 <= (size_t)c.smCount &&
                   nv / (s.cluster * 2) >= 64)
                s.cluster *= 2;
            const int per = (nv + s.cluster - 1) / s.cluster;
            // One vector a thread where that makes one wave of CTAs at 72 registers a thread
            // (1 x 150 x 4096: 2.6 us, 3.1 with two), else two (1 x 300 x 4096: 3.1 us, 4.5 with one;
            // 32 x 2000 x 4096: 171 and 185).
            const int warps = (per + 31) / 32;
            const size_t wave = (size_t)c.smCount * std::max(1, 65536 / (72 * 32 * warps));
            const bool one = per <= kNormMaxThreads && (c.backward || c.rows * (size_t)s.cluster <= wave);
            s.vecs = one ? 1 : per <= kNormMaxThreads * 2 ? 2 : 4;
            s.teamThreads = ((per + s.vecs - 1) / s.vecs + 31) / 32 * 32;
            s.threads = s.teamThreads;
            s.rowsPerCta = 1;
        }
        layout();
    }
    return s;
}

int norm_backward_parts(size_t rows, const NormShape& sh, int smCount) {
    if (sh.staged) return sh.ctas;
    // direct loads: the launch bounds leave an SM room for kNormMaxThreads, at 96 registers a thread
    const int perSm = std::max(1, kNormMaxThreads / sh.threads);
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
    bool outSame = true;             // the outputs all start at one offset from 16 bytes
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
        b->outSame = b->outSame && at((const void*)((uintptr_t)recv[r] ^ (uintptr_t)out[0]), 16);
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

vc::NormCall norm_call(const Checked& k, const CommView& v, const Buffers& b) {
    vc::NormCall c = {};
    c.rows = k.d.rows;
    c.hidden = (int)k.d.hidden;
    c.elemSize = k.esz;
    c.weightSize = (int)vc::dtype_size(k.d.weightType);
    c.smCount = v.smCount;
    c.general = !b.aligned;
    return c;
}

void debug_norm(const CommView& v, const char* what, const Checked& k, const vc::NormShape& s) {
    if (!v.debug) return;
    std::fprintf(stderr,
                 "vcomm INFO %s rows=%zu hidden=%zu dt=%d N=%d vecs=%d team=%d rows/cta=%d cluster=%d general=%d staged=%d "
                 "rounds=%d smem=%d\n",
                 what, k.d.rows, k.d.hidden, (int)k.d.datatype, v.nRanks, s.vecs, s.teamThreads, s.rowsPerCta, s.cluster,
                 s.general, s.staged, s.rounds, s.smemBytes);
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
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                return norm_forward(&d, s.data(), residual, weight, residualOut, o.data(), q.data(), quant, rstd, c, stream);
            });
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
    a.outSame = b.outSame;
    a.weightF32 = k.d.weightType == vFloat32;
    a.groups = k.d.quantGroup ? (int)((k.d.hidden + vc::kQuantGroup - 1) / vc::kQuantGroup) : 0;
    a.eps = k.d.eps;
    vc::NormCall call = norm_call(k, v, b);
    call.segments = v.nRanks + (residual ? 1 : 0);
    call.groups = a.groups > 0;
    a.shape = vc::norm_shape(call);
    debug_norm(v, quant ? "AllReduceRmsNormQuant" : "AllReduceRmsNorm", k, a.shape);
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
            return guarded([&]() {
                return norm_backward(&d, s.data(), hidden, rstd, weight, gradResidual, o.data(), gradWeight, workspace,
                                     workspaceBytes, c, stream);
            });
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
    a.outSame = b.outSame;
    a.weightF32 = k.d.weightType == vFloat32;
    vc::NormCall call = norm_call(k, v, b);
    call.segments = v.nRanks + 1 + (gradResidual ? 1 : 0);
    call.backward = true;
    a.shape = vc::norm_shape(call);
    a.parts = vc::norm_backward_parts(a.rows, a.shape, v.smCount);
    if (!workspace || !at(workspace, 16) || workspaceBytes < (size_t)a.parts * k.d.hidden * sizeof(float))
        return vInvalidArgument;
    debug_norm(v, "AllReduceRmsNormBackward", k, a.shape);
    return comm_launch(c, "rmsnorm backward", [&]() { return vc::launch_rmsnorm_backward(a, k.d.datatype, stream); });
}

// ---- gradient norm and clipping ----------------------------------------------------------

size_t grad_partials(unsigned int chunks, int smCount) {
    return std::max<size_t>(1, std::min<size_t>(chunks, (size_t)smCount * vc::kSquaresCtasPerSm));
}

// Cut one rank's tensor into chunks.
void add_chunks(std::vector<vc::GradChunk>* v, const void* in, void* out, size_t count, vDataType_t dt) {
    const size_t esz = vc::dtype_size(dt), e = 16 / esz;
    // a chunk that starts off a 16-byte boundary touches one vector more than it fills
    const bool aligned = at(in, 16) && at(out, 16);
    const size_t most = (size_t)(aligned ? vc::kGradChunkVecs : vc::kGradChunkVecs - 1) * e;
    for (size_t i = 0; i < count; i += most) {
        vc::GradChunk c = {};
        c.in = (const char*)in + i * esz;
        c.out = (char*)out + i * esz;
        c.count = (int)std::min(most, count - i);
        c.dt = (int)dt;
        v->push_back(c);
    }
}

struct GradList {
    int nRanks;
    int device;
    vc::GradChunk* chunks;           // device: the counted ones, then the rest
    unsigned int* done;              // device: k_grad_norm's counter
    unsigned int nCounted, nChunks;
};

// The lists that exist.  A handle is a list's number, given once and never an address, so that
// the handle of a destroyed list is known for one without looking at freed memory.
struct GradLists {
    std::mutex lock;
    std::unordered_map<uintptr_t, GradList> live;
    uintptr_t last = 0;
};
GradLists& grad_lists() {
    static GradLists* lists = new GradLists;           // outlives the caller's own statics
    return *lists;
}

vResult_t list_create(vGradList_t* list, int nRanks, int nTensors, const size_t* counts, const vDataType_t* datatypes,
                      const unsigned char* replicated, const void* const* grads, void* const* outs) {
    if (!list) return vInvalidArgument;
    *list = nullptr;
    if (nRanks < 1 || nRanks > VCOMM_MAX_RANKS || nTensors < 0 || nTensors > 0x7FFFFFFF / nRanks) return vInvalidArgument;
    if (nTensors > 0 && (!counts || !datatypes || !grads)) return vInvalidArgument;
    const size_t most = (size_t)1 << 40;     // of all pieces together: their chunks fit one grid
    size_t total = 0;
    for (int t = 0; t < nTensors; t++) {
        if (!is_float(datatypes[t]) || counts[t] > (most - total) / nRanks) return vInvalidArgument;
        total += counts[t] * nRanks;
        if (counts[t] == 0) continue;
        const size_t esz = vc::dtype_size(datatypes[t]);
        for (int r = 0; r < nRanks; r++) {
            const size_t i = (size_t)r * nTensors + t;
            if (!grads[i] || !at(grads[i], esz) || (outs && (!outs[i] || !at(outs[i], esz)))) return vInvalidArgument;
        }
    }
    std::vector<vc::GradChunk> counted, rest;
    for (int r = 0; r < nRanks; r++)
        for (int t = 0; t < nTensors; t++) {
            const size_t i = (size_t)r * nTensors + t;
            if (counts[t] == 0) continue;
            add_chunks(r > 0 && replicated && replicated[t] ? &rest : &counted, grads[i],
                       outs ? outs[i] : const_cast<void*>(grads[i]), counts[t], datatypes[t]);
        }
    GradList l = {};
    l.nRanks = nRanks;
    l.nCounted = (unsigned)counted.size();
    counted.insert(counted.end(), rest.begin(), rest.end());
    l.nChunks = (unsigned)counted.size();
    cudaError_t e = cudaGetDevice(&l.device);
    struct Memory {
        void* p = nullptr;
        ~Memory() { if (p) cudaFree(p); }
    } own;
    void*& mem = own.p;
    const size_t bytes = counted.size() * sizeof(vc::GradChunk);
    if (e == cudaSuccess) e = cudaMalloc(&mem, bytes + 32);
    if (e == cudaSuccess && bytes) e = cudaMemcpy(mem, counted.data(), bytes, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemset((char*)mem + bytes, 0, 32);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return vUnhandledCudaError;
    }
    l.chunks = (vc::GradChunk*)mem;
    l.done = (unsigned int*)((char*)mem + bytes);
    GradLists& all = grad_lists();
    std::lock_guard<std::mutex> hold(all.lock);
    all.live.emplace(all.last + 1, l);
    mem = nullptr;
    *list = (vGradList_t)++all.last;
    return vSuccess;
}

vResult_t find_list(vGradList_t handle, const CommView& v, GradList* l) {
    GradLists& all = grad_lists();
    std::lock_guard<std::mutex> hold(all.lock);
    const auto i = all.live.find((uintptr_t)handle);
    if (i == all.live.end() || i->second.nRanks != v.nRanks || i->second.device != v.device) return vInvalidArgument;
    *l = i->second;
    return vSuccess;
}

vResult_t list_destroy(vGradList_t handle) {
    GradList l;
    {
        GradLists& all = grad_lists();
        std::lock_guard<std::mutex> hold(all.lock);
        const auto i = all.live.find((uintptr_t)handle);
        if (i == all.live.end()) return vInvalidArgument;
        l = i->second;
        all.live.erase(i);
    }
    int prev = -1;
    const bool other = cudaGetDevice(&prev) == cudaSuccess && prev != l.device;
    if (other) cudaSetDevice(l.device);
    const cudaError_t e = cudaFree(l.chunks);          // waits for the work that uses it
    if (other) cudaSetDevice(prev);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? vSuccess : vUnhandledCudaError;
}

vResult_t grad_norm(vGradList_t handle, bool clip, float maxNorm, float* norm, void* workspace, size_t workspaceBytes,
                    vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    GradList l;
    if ((r = find_list(handle, v, &l)) != vSuccess) return r;
    if (!norm || !at(norm, 4)) return vInvalidArgument;
    if (clip && !(maxNorm >= 0.0f)) return vInvalidArgument;
    const size_t parts = grad_partials(l.nCounted, v.smCount);
    if (!workspace || !at(workspace, 16) || workspaceBytes < parts * sizeof(double)) return vInvalidArgument;
    if (v.grouping)
        return vc::comm_record(c, [=]() {
            return guarded([&]() { return grad_norm(handle, clip, maxNorm, norm, workspace, workspaceBytes, c, stream); });
        });
    if (v.debug)
        std::fprintf(stderr, "vcomm INFO %s chunks=%u counted=%u N=%d\n", clip ? "ClipGradNorm" : "GradNorm", l.nChunks,
                     l.nCounted, v.nRanks);
    vc::GradNormArgs a;
    a.chunks = l.chunks;
    a.nChunks = l.nCounted;
    a.done = l.done;
    a.partials = (double*)workspace;
    a.norm = norm;
    r = comm_launch(c, "gradient norm", [&]() { return vc::launch_grad_norm(a, (int)parts, stream); });
    if (r != vSuccess || !clip || l.nChunks == 0) return r;
    vc::GradClipArgs k;
    k.chunks = l.chunks;
    k.nChunks = l.nChunks;
    k.norm = norm;
    k.maxNorm = maxNorm;
    return comm_launch(c, "gradient clip", [&]() { return vc::launch_grad_clip(k, stream); });
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
    // whatever the buffers' alignment turns out to be, with or without a residual's gradient
    for (int i = 0; i < 4; i++) {
        Buffers b;
        b.aligned = (i & 1) != 0;
        if (b.aligned && k.d.hidden % (16 / k.esz) != 0) continue;
        vc::NormCall call = norm_call(k, v, b);
        call.segments = v.nRanks + 1 + (i >> 1);
        call.backward = true;
        const int parts = vc::norm_backward_parts(k.d.rows, vc::norm_shape(call), v.smCount);
        *bytes = std::max(*bytes, (size_t)parts * k.d.hidden * sizeof(float));
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

vResult_t vGradListCreate(vGradList_t* list, int nRanks, int nTensors, const size_t* counts,
                          const vDataType_t* datatypes, const unsigned char* replicated, const void* const* grads,
                          void* const* outs) {
    return guarded([&]() { return list_create(list, nRanks, nTensors, counts, datatypes, replicated, grads, outs); });
}

vResult_t vGradListDestroy(vGradList_t list) {
    return guarded([&]() { return list_destroy(list); });
}

vResult_t vGradNormWorkspace(vGradList_t list, vcomm_t comm, size_t* bytes) {
    CommView v;
    vResult_t r = comm_view(comm, &v);
    if (r != vSuccess) return r;
    return guarded([&]() {
        GradList l;
        const vResult_t f = find_list(list, v, &l);
        if (f != vSuccess) return f;
        if (!bytes) return vInvalidArgument;
        *bytes = std::max<size_t>(16, grad_partials(l.nCounted, v.smCount) * sizeof(double));
        return vSuccess;
    });
}

vResult_t vGradNorm(vGradList_t list, float* norm, void* workspace, size_t workspaceBytes, vcomm_t comm,
                    cudaStream_t stream) {
    Range range("vGradNorm");
    return guarded([&]() { return grad_norm(list, false, 0.0f, norm, workspace, workspaceBytes, comm, stream); });
}

vResult_t vClipGradNorm(vGradList_t list, float maxNorm, float* norm, void* workspace, size_t workspaceBytes,
                        vcomm_t comm, cudaStream_t stream) {
    Range range("vClipGradNorm");
    return guarded([&]() { return grad_norm(list, true, maxNorm, norm, workspace, workspaceBytes, comm, stream); });
}

}  // extern "C"
