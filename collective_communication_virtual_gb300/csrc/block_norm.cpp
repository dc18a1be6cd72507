// block_norm.cpp -- entry points of the block norm (the norms after and before a block, its gate and
// the scaled residual, behind the ranks' all-reduce) and of its backward pass.
#include <cstdio>
#include <vector>

#include "entry.h"

namespace {

// The block norm's descriptor as an RMS norm's, whose checks it shares.
vResult_t check_block(const vBlockNormDesc_t* desc, Checked* k) {
    if (!desc) return vInvalidArgument;
    vRmsNormDesc_t d = {};
    d.rows = desc->rows;
    d.hidden = desc->hidden;
    d.sendStride = desc->sendStride;
    d.residualStride = desc->residualStride;
    d.recvStride = desc->recvStride;
    d.eps = desc->eps;
    d.datatype = desc->datatype;
    d.weightType = desc->weightType;
    if (!std::isfinite(desc->residualScale)) return vInvalidArgument;
    return check_desc(&d, k);
}

vc::NormCall block_call(const Checked& k, const CommView& v, const Buffers& b, bool backward, int segments) {
    vc::NormCall c = norm_call(k, v, b);
    c.weightSize += 4;               // beside the weight before the next block, post * gate in fp32
    c.extraRowBuffers = 1;
    c.backward = backward;
    c.segments = segments;
    // A row's two reductions, one behind the other, are waited for: with many inputs more threads a row
    // hide that (8 x 4096 x 4096 bf16: 99 us with one vector a thread, 102 with two, 113 with four;
    // 4 x 4096 x 4096: 65, 62 and 72), with few the instructions count (1 x 16384 x 4096: 150, 131 and
    // 112; 1 x 9000 x 1001: 41, 35 and 24).  Backward, one vector keeps both sums in registers, which pays
    // for long rows of several ranks (3 x 4000 x 4096: 69 us, 80 with two, 111 with four; but 8 x 8000 x
    // 1024: 82, 67 and 96; 1 x 16384 x 4096: 200, 158 and 282).
    const size_t vectors = k.d.hidden * k.esz / 16;
    if (backward) {
        c.extraSums = 1;
        c.regs = 128;
        c.vecs = segments >= 6 && vectors > 256 && !c.general ? 1 : 2;
    } else {
        c.vecs = segments <= (c.general ? 4 : 2) ? 4 : segments >= 7 && !c.general ? 1 : 2;
    }
    return c;
}

void debug_block(const CommView& v, const char* what, const Checked& k, const vc::NormShape& s) {
    if (!v.debug) return;
    std::fprintf(stderr,
                 "vcomm INFO %s rows=%zu hidden=%zu dt=%d N=%d vecs=%d team=%d rows/cta=%d cluster=%d general=%d staged=%d "
                 "rounds=%d smem=%d\n",
                 what, k.d.rows, k.d.hidden, (int)k.d.datatype, v.nRanks, s.vecs, s.teamThreads, s.rowsPerCta, s.cluster,
                 s.general, s.staged, s.rounds, s.smemBytes);
}

vResult_t block_forward(const vBlockNormDesc_t* desc, const void* const* send, const void* residual, const void* post,
                        const void* gate, const void* pre, void* blockOut, void* residualOut, void* const* recv, float* rstd,
                        vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_block(desc, &k)) != vSuccess) return r;
    if (v.grouping) {
        if (!send || !recv) return vInvalidArgument;
        const vBlockNormDesc_t d = *desc;
        const std::vector<const void*> s(send, send + v.nRanks);
        const std::vector<void*> o(recv, recv + v.nRanks);
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                return block_forward(&d, s.data(), residual, post, gate, pre, blockOut, residualOut, o.data(), rstd, c, stream);
            });
        });
    }
    if (k.d.rows == 0 || k.d.hidden == 0) return vSuccess;
    vc::BlockNormArgs a;
    Buffers b;
    if ((r = check_buffers(k, v.nRanks, send, recv, k.esz, a.send, a.recv, nullptr, &b)) != vSuccess) return r;
    if ((r = check_weight(k, post, &b)) != vSuccess) return r;
    if (gate && (r = check_weight(k, gate, &b)) != vSuccess) return r;
    if ((r = check_weight(k, pre, &b)) != vSuccess) return r;
    for (const void* p : {residual, (const void*)blockOut, (const void*)residualOut})
        if ((r = check_row_buffer(k, p, &b)) != vSuccess) return r;
    if (!at(rstd, 4)) return vInvalidArgument;
    a.residual = residual;
    a.post = post;
    a.gate = gate;
    a.pre = pre;
    a.blockOut = blockOut;
    a.residualOut = residualOut;
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
    a.eps = k.d.eps;
    a.scale = desc->residualScale;
    const vc::NormCall call = block_call(k, v, b, false, v.nRanks + (residual ? 1 : 0));
    a.shape = vc::norm_shape(call);
    debug_block(v, "AllReduceBlockNorm", k, a.shape);
    return comm_launch(c, "allreduce block norm", [&]() { return vc::launch_block_norm(a, k.d.datatype, stream); });
}

vResult_t block_backward(const vBlockNormDesc_t* desc, const void* const* send, const void* hidden, const void* block,
                         const float* rstd, const void* post, const void* gate, const void* pre, const void* gradStream,
                         void* gradResidual, void* const* recv, void* gradPost, void* gradGate, void* gradPre, void* workspace,
                         size_t workspaceBytes, vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_block(desc, &k)) != vSuccess) return r;
    if (v.grouping) {
        if (!send || !recv) return vInvalidArgument;
        const vBlockNormDesc_t d = *desc;
        const std::vector<const void*> s(send, send + v.nRanks);
        const std::vector<void*> o(recv, recv + v.nRanks);
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                return block_backward(&d, s.data(), hidden, block, rstd, post, gate, pre, gradStream, gradResidual, o.data(),
                                      gradPost, gradGate, gradPre, workspace, workspaceBytes, c, stream);
            });
        });
    }
    if (k.d.hidden == 0) return vSuccess;
    const size_t wsz = vc::dtype_size(k.d.weightType);
    if (!gradPost || !at(gradPost, wsz) || !gradPre || !at(gradPre, wsz)) return vInvalidArgument;
    if ((gate != nullptr) != (gradGate != nullptr) || !at(gradGate, wsz)) return vInvalidArgument;
    if (k.d.rows == 0)               // sums over no rows
        return comm_launch(c, "block norm backward", [&]() {
            for (void* p : {gradPost, gradGate, gradPre}) {
                if (!p) continue;
                const cudaError_t e = cudaMemsetAsync(p, 0, k.d.hidden * wsz, stream);
                if (e != cudaSuccess) return e;
            }
            return cudaSuccess;
        });
    vc::BlockNormBackwardArgs a;
    Buffers b;
    if ((r = check_buffers(k, v.nRanks, send, recv, k.esz, a.send, a.recv, nullptr, &b)) != vSuccess) return r;
    if ((r = check_weight(k, post, &b)) != vSuccess) return r;
    if (gate && (r = check_weight(k, gate, &b)) != vSuccess) return r;
    if ((r = check_weight(k, pre, &b)) != vSuccess) return r;
    if (!hidden || !block || !rstd || !at(rstd, 4)) return vInvalidArgument;
    for (const void* p : {hidden, block, gradStream, (const void*)gradResidual})
        if ((r = check_row_buffer(k, p, &b)) != vSuccess) return r;
    a.hidden = hidden;
    a.block = block;
    a.gradStream = gradStream;
    a.post = post;
    a.gate = gate;
    a.pre = pre;
    a.rstd = rstd;
    a.gradResidual = gradResidual;
    a.partials = (float*)workspace;
    a.gradPost = gradPost;
    a.gradGate = gradGate;
    a.gradPre = gradPre;
    a.rows = k.d.rows;
    a.sendStride = k.d.sendStride;
    a.residualStride = k.d.residualStride;
    a.recvStride = k.d.recvStride;
    a.width = (int)k.d.hidden;
    a.nRanks = v.nRanks;
    a.nOut = b.nOut;
    a.outSame = b.outSame;
    a.weightF32 = k.d.weightType == vFloat32;
    a.scale = desc->residualScale;
    const vc::NormCall call = block_call(k, v, b, true, v.nRanks + 2 + (gradStream ? 1 : 0));
    a.shape = vc::norm_shape(call);
    a.parts = vc::norm_backward_parts(a.rows, a.shape, v.smCount);
    if (!workspace || !at(workspace, 16) || workspaceBytes < (size_t)a.parts * 2 * k.d.hidden * sizeof(float))
        return vInvalidArgument;
    debug_block(v, "AllReduceBlockNormBackward", k, a.shape);
    return comm_launch(c, "block norm backward",
                       [&]() { return vc::launch_block_norm_backward(a, k.d.datatype, stream); });
}

}  // namespace

extern "C" {

vResult_t vAllReduceBlockNorm(const vBlockNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                              const void* postWeight, const void* gate, const void* preWeight, void* blockOut,
                              void* residualOut, void* const* recvbuffs, float* rstd, vcomm_t comm, cudaStream_t stream) {
    Range range("vAllReduceBlockNorm");
    return guarded([&]() {
        return block_forward(desc, sendbuffs, residual, postWeight, gate, preWeight, blockOut, residualOut, recvbuffs, rstd,
                             comm, stream);
    });
}

vResult_t vBlockNormBackwardWorkspace(const vBlockNormDesc_t* desc, vcomm_t comm, size_t* bytes) {
    CommView v;
    vResult_t r = comm_view(comm, &v);
    if (r != vSuccess) return r;
    Checked k;
    if ((r = check_block(desc, &k)) != vSuccess) return r;
    if (!bytes) return vInvalidArgument;
    *bytes = 16;
    if (k.d.rows == 0 || k.d.hidden == 0) return vSuccess;
    // whatever the buffers' alignment turns out to be, with or without a gradient of the stream
    for (int i = 0; i < 4; i++) {
        Buffers b;
        b.aligned = (i & 1) != 0;
        if (b.aligned && k.d.hidden % (16 / k.esz) != 0) continue;
        const vc::NormCall call = block_call(k, v, b, true, v.nRanks + 2 + (i >> 1));
        const int parts = vc::norm_backward_parts(k.d.rows, vc::norm_shape(call), v.smCount);
        *bytes = std::max(*bytes, (size_t)parts * 2 * k.d.hidden * sizeof(float));
    }
    return vSuccess;
}

vResult_t vAllReduceBlockNormBackward(const vBlockNormDesc_t* desc, const void* const* sendbuffs, const void* hiddenStates,
                                      const void* block, const float* rstd, const void* postWeight, const void* gate,
                                      const void* preWeight, const void* gradStream, void* gradResidual,
                                      void* const* recvbuffs, void* gradPostWeight, void* gradGate, void* gradPreWeight,
                                      void* workspace, size_t workspaceBytes, vcomm_t comm, cudaStream_t stream) {
    Range range("vAllReduceBlockNormBackward");
    return guarded([&]() {
        return block_backward(desc, sendbuffs, hiddenStates, block, rstd, postWeight, gate, preWeight, gradStream, gradResidual,
                              recvbuffs, gradPostWeight, gradGate, gradPreWeight, workspace, workspaceBytes, comm, stream);
    });
}

}  // extern "C"
