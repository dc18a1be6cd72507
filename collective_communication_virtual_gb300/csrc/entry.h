// entry.h -- what the operators' entry points share: the checks of a norm's descriptor and
// buffers, and the guards around a call.  Included by the translation units that define them.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "operators.h"

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

inline bool is_float(int dt) { return dt == vFloat32 || dt == vFloat16 || dt == vBFloat16; }

inline bool at(const void* p, size_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

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

inline vResult_t check_desc(const vRmsNormDesc_t* desc, Checked* k) {
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
inline vResult_t check_buffers(const Checked& k, int nRanks, const void* const* send, void* const* recv, int osz,
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

inline vResult_t check_weight(const Checked& k, const void* weight, Buffers* b) {
    if (!weight || !at(weight, vc::dtype_size(k.d.weightType))) return vInvalidArgument;
    b->aligned = b->aligned && at(weight, 16);
    return vSuccess;
}
inline vResult_t check_row_buffer(const Checked& k, const void* p, Buffers* b) {
    if (!p) return vSuccess;
    if (!at(p, k.esz)) return vInvalidArgument;
    b->aligned = b->aligned && at(p, 16);
    return vSuccess;
}

inline vc::NormCall norm_call(const Checked& k, const CommView& v, const Buffers& b) {
    vc::NormCall c = {};
    c.rows = k.d.rows;
    c.hidden = (int)k.d.hidden;
    c.elemSize = k.esz;
    c.weightSize = (int)vc::dtype_size(k.d.weightType);
    c.smCount = v.smCount;
    c.general = !b.aligned;
    return c;
}

}  // namespace
