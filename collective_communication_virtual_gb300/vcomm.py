"""ctypes binding of libvcomm (include/vcomm.h): the same entry points, argument
marshalling only.  Every collective runs in the library's CUDA kernels; there is no
Python or CPU fallback -- if the library is missing or a call fails, an exception is
raised.

Buffers may be given as torch tensors or as integer device addresses; ``datatype`` as a
torch dtype or a ``vDataType_t`` value; ``stream`` as a ``torch.cuda.Stream``, a raw
``cudaStream_t`` integer, or ``None`` for torch's current stream.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

# ---- enums (values of include/vcomm.h) ---------------------------------------------------
vSuccess, vUnhandledCudaError, vSystemError, vInternalError = 0, 1, 2, 3
vInvalidArgument, vInvalidUsage, vTimeout, vInProgress, vAborted = 4, 5, 6, 7, 8
vFloat32, vFloat16, vBFloat16, vInt32 = 0, 1, 2, 3
vSum, vProd, vMin, vMax = 0, 1, 2, 3
vProtoSimple, vProtoLL, vProtoLL128, vProtoAuto = 0, 1, 2, 3
vAlgoAuto, vAlgoOnePass, vAlgoRing, vAlgoTree = 0, 1, 2, 3
vCollAllReduce, vCollReduceScatter, vCollAllGather = 0, 1, 2
vCollBroadcast, vCollAllToAll, vCollAllToAllv = 3, 4, 5
vCollReduce, vCollGather, vCollScatter = 6, 7, 8
VCOMM_MAX_RANKS = 64

RESULT_NAMES = {0: "vSuccess", 1: "vUnhandledCudaError", 2: "vSystemError", 3: "vInternalError",
                4: "vInvalidArgument", 5: "vInvalidUsage", 6: "vTimeout", 7: "vInProgress",
                8: "vAborted"}
OPS = {"sum": vSum, "prod": vProd, "min": vMin, "max": vMax}
PROTOCOLS = {"simple": vProtoSimple, "ll": vProtoLL, "ll128": vProtoLL128, "auto": vProtoAuto}
ALGOS = {"auto": vAlgoAuto, "onepass": vAlgoOnePass, "ring": vAlgoRing, "tree": vAlgoTree}


class VcommError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {RESULT_NAMES.get(code, code)}")


class vPlanRequest_t(ctypes.Structure):
    _fields_ = [("nRanks", ctypes.c_int), ("nChannels", ctypes.c_int), ("proto", ctypes.c_int),
                ("algo", ctypes.c_int), ("coll", ctypes.c_int), ("datatype", ctypes.c_int),
                ("count", ctypes.c_size_t), ("chunkBytes", ctypes.c_size_t),
                ("aligned16", ctypes.c_int), ("smCount", ctypes.c_int), ("l2Bytes", ctypes.c_size_t),
                ("aligned32", ctypes.c_int), ("noBulkCopy", ctypes.c_int), ("persistentGrid", ctypes.c_int)]


class vPlanInfo_t(ctypes.Structure):
    _fields_ = [("algo", ctypes.c_int), ("proto", ctypes.c_int), ("nChannels", ctypes.c_int),
                ("ctasPerChannel", ctypes.c_int), ("gridCtas", ctypes.c_int),
                ("threadsPerCta", ctypes.c_int), ("vectorized", ctypes.c_int),
                ("launches", ctypes.c_int), ("blockElems", ctypes.c_size_t),
                ("channelElems", ctypes.c_size_t), ("chunkElems", ctypes.c_size_t),
                ("slotPayloadElems", ctypes.c_size_t), ("slotBytes", ctypes.c_size_t),
                ("fifoBytes", ctypes.c_size_t), ("minBytes", ctypes.c_double),
                ("busFactor", ctypes.c_double), ("vecBytes", ctypes.c_int), ("bulkCopy", ctypes.c_int),
                ("predictedUs", ctypes.c_double), ("tileBytes", ctypes.c_size_t), ("tmaStages", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class vRmsNormDesc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_size_t), ("hidden", ctypes.c_size_t), ("sendStride", ctypes.c_size_t),
                ("residualStride", ctypes.c_size_t), ("recvStride", ctypes.c_size_t), ("eps", ctypes.c_float),
                ("datatype", ctypes.c_int), ("weightType", ctypes.c_int), ("quantGroup", ctypes.c_int)]


class vBlockNormDesc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_size_t), ("hidden", ctypes.c_size_t), ("sendStride", ctypes.c_size_t),
                ("residualStride", ctypes.c_size_t), ("recvStride", ctypes.c_size_t), ("eps", ctypes.c_float),
                ("residualScale", ctypes.c_float), ("datatype", ctypes.c_int), ("weightType", ctypes.c_int)]


class vMoeDesc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_size_t), ("hidden", ctypes.c_size_t), ("ffn", ctypes.c_size_t), ("experts", ctypes.c_int),
                ("topK", ctypes.c_int), ("rowStride", ctypes.c_size_t), ("recvStride", ctypes.c_size_t),
                ("datatype", ctypes.c_int), ("routerType", ctypes.c_int), ("normalize", ctypes.c_int)]


class vSampleDesc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_size_t), ("vocab", ctypes.c_size_t), ("part", ctypes.c_size_t), ("stride", ctypes.c_size_t),
                ("datatype", ctypes.c_int)]


_lib = None

_SIGNATURES = {
    "vcommInit": ([ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int, ctypes.c_int], ctypes.c_int),
    "vcommDestroy": ([ctypes.c_void_p], ctypes.c_int),
    "vcommGetAsyncError": ([ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "vcommAbort": ([ctypes.c_void_p], ctypes.c_int),
    "vcommGetErrorString": ([ctypes.c_int], ctypes.c_char_p),
    "vcommSetAlgo": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "vcommGroupStart": ([ctypes.c_void_p], ctypes.c_int),
    "vcommGroupEnd": ([ctypes.c_void_p], ctypes.c_int),
    "vcommSetProtocol": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "vcommSetChunkBytes": ([ctypes.c_void_p, ctypes.c_size_t], ctypes.c_int),
    "vcommSetTimeoutMs": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "vcommTestSetStallRank": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "vcommQueryPlan": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                        ctypes.POINTER(vPlanInfo_t)], ctypes.c_int),
    "vPlanCompute": ([ctypes.POINTER(vPlanRequest_t), ctypes.POINTER(vPlanInfo_t)], ctypes.c_int),
    "vPlanTreeLinks": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                        ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "vPlanChannelRange": ([ctypes.POINTER(vPlanInfo_t), ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                           ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "vAllReduce": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                    ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vReduceScatter": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                        ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vReduceScatterScaleCast": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                                 ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vAllGather": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                    ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vBroadcast": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                    ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vAllToAll": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                   ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vcommCount": ([ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vcommTestSetJitterNs": ([ctypes.c_void_p, ctypes.c_uint], ctypes.c_int),
    "vcommTestSetBadFlagRank": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "vAllToAllv": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                    ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vReduce": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                 ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vGather": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                 ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vScatter": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                  ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "vAllReduceRmsNorm": ([ctypes.c_void_p] * 9, ctypes.c_int),
    "vAllReduceRmsNormQuant": ([ctypes.c_void_p] * 10, ctypes.c_int),
    "vRmsNormBackwardWorkspace": ([ctypes.c_void_p] * 3, ctypes.c_int),
    "vAllReduceRmsNormBackward": ([ctypes.c_void_p] * 9 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2, ctypes.c_int),
    "vAllReduceBlockNorm": ([ctypes.c_void_p] * 12, ctypes.c_int),
    "vBlockNormBackwardWorkspace": ([ctypes.c_void_p] * 3, ctypes.c_int),
    "vAllReduceBlockNormBackward": ([ctypes.c_void_p] * 15 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2, ctypes.c_int),
    "vMoeRoute": ([ctypes.c_void_p] * 8, ctypes.c_int),
    "vMoeExpertsWorkspace": ([ctypes.c_void_p] * 3, ctypes.c_int),
    "vMoeExperts": ([ctypes.c_void_p] * 8 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2, ctypes.c_int),
    "vSample": ([ctypes.c_void_p] * 11, ctypes.c_int),
    "vGradListCreate": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 5, ctypes.c_int),
    "vGradListDestroy": ([ctypes.c_void_p], ctypes.c_int),
    "vGradNormWorkspace": ([ctypes.c_void_p] * 3, ctypes.c_int),
    "vGradNorm": ([ctypes.c_void_p] * 3 + [ctypes.c_size_t] + [ctypes.c_void_p] * 2, ctypes.c_int),
    "vClipGradNorm": ([ctypes.c_void_p, ctypes.c_float] + [ctypes.c_void_p] * 2 + [ctypes.c_size_t]
                      + [ctypes.c_void_p] * 2, ctypes.c_int),
    "vAllReduceNoAlloc": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                           ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p], ctypes.c_int),
}


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libvcomm.so (built in-tree by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libvcomm.so is not built ({path}); run "
                               "collective_communication_virtual_gb300.build.build() first")
        L = ctypes.CDLL(path)
        for name, (args, res) in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


# ---- marshalling helpers -------------------------------------------------------------------

_DTYPE_CODES: dict = {}
_ARRAY_TYPES: dict = {}


def _dtype_code(dt) -> int:
    if isinstance(dt, int):
        return dt
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float32: vFloat32, torch.float16: vFloat16, torch.bfloat16: vBFloat16,
                             torch.int32: vInt32})
    return _DTYPE_CODES[dt]


def _op_code(op) -> int:
    return OPS[op] if isinstance(op, str) else int(op)


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


class Buffers:
    """What vBuffers makes: the C array of the addresses and where it lies."""
    __slots__ = ("array", "address", "count")

    def __init__(self, array):
        self.array, self.address, self.count = array, ctypes.addressof(array), len(array)


def _ptr_array(bufs, n_ranks: int):
    """A C array of the buffers' device addresses (None for NULL).  The library reads
    exactly n_ranks entries, so a list of another length is refused here."""
    made = type(bufs) is Buffers                    # by vBuffers
    n = bufs.count if made else len(bufs)
    if n != n_ranks:
        raise VcommError(vInvalidArgument, f"expected {n_ranks} buffers (one per rank), got {n}")
    if made:
        return bufs.address
    arr_t = _ARRAY_TYPES.get(n)
    if arr_t is None:
        arr_t = _ARRAY_TYPES[n] = ctypes.c_void_p * n
    return arr_t(*[None if b is None else (b if isinstance(b, int) else b.data_ptr()) for b in bufs])


_N_RANKS: dict = {}


def _handle(comm) -> int | None:
    return comm.value if isinstance(comm, ctypes.c_void_p) else comm


def _n_ranks(comm) -> int:
    """The communicator's rank count, asked of the library once per handle."""
    key = _handle(comm)
    n = _N_RANKS.get(key)
    if n is None:
        v = ctypes.c_int(0)
        _check(lib().vcommCount(comm, ctypes.byref(v)), "vcommCount")
        n = _N_RANKS[key] = v.value
    return n


def _pair(comm, sendbuffs, recvbuffs):
    n = _n_ranks(comm)
    return _ptr_array(sendbuffs, n), _ptr_array(recvbuffs, n)


_current_stream = None


def _find_current_stream():
    """torch's current stream as an address.  torch.cuda.current_stream() builds a Stream object
    (2.8 us of a 9.4 us call on Grace); the functions below it give the address in 0.2 us."""
    import torch
    get_device = getattr(torch._C, "_cuda_getDevice", None)
    get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get_device is None or get_stream is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: get_stream(get_device())


def _stream(stream) -> int | None:
    global _current_stream
    if stream is None:
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != vSuccess:
        raise VcommError(code, where)


# ---- the C ABI, one wrapper per entry point --------------------------------------------------

def vcommInit(n_ranks: int, n_channels: int = 1, protocol=vProtoSimple) -> ctypes.c_void_p:
    comm = ctypes.c_void_p()
    proto = PROTOCOLS[protocol] if isinstance(protocol, str) else protocol
    _check(lib().vcommInit(ctypes.byref(comm), n_ranks, n_channels, proto), "vcommInit")
    _N_RANKS[comm.value] = n_ranks
    return comm


def vcommDestroy(comm) -> None:
    _N_RANKS.pop(_handle(comm), None)
    _check(lib().vcommDestroy(comm), "vcommDestroy")


def vcommCount(comm) -> int:
    v = ctypes.c_int(0)
    _check(lib().vcommCount(comm, ctypes.byref(v)), "vcommCount")
    return v.value


def vcommGetAsyncError(comm) -> int:
    err = ctypes.c_int(0)
    _check(lib().vcommGetAsyncError(comm, ctypes.byref(err)), "vcommGetAsyncError")
    return err.value


def vcommAbort(comm) -> None:
    _check(lib().vcommAbort(comm), "vcommAbort")


def vcommGetErrorString(code: int) -> str:
    return lib().vcommGetErrorString(code).decode()


def vcommGroupStart(comm) -> None:
    _check(lib().vcommGroupStart(comm), "vcommGroupStart")


def vcommGroupEnd(comm) -> None:
    _check(lib().vcommGroupEnd(comm), "vcommGroupEnd")


def vcommSetAlgo(comm, algo) -> None:
    _check(lib().vcommSetAlgo(comm, ALGOS[algo] if isinstance(algo, str) else algo), "vcommSetAlgo")


def vcommSetProtocol(comm, protocol) -> None:
    proto = PROTOCOLS[protocol] if isinstance(protocol, str) else protocol
    _check(lib().vcommSetProtocol(comm, proto), "vcommSetProtocol")


def vcommSetChunkBytes(comm, chunk_bytes: int) -> None:
    _check(lib().vcommSetChunkBytes(comm, chunk_bytes), "vcommSetChunkBytes")


def vcommSetTimeoutMs(comm, ms: int) -> None:
    _check(lib().vcommSetTimeoutMs(comm, ms), "vcommSetTimeoutMs")


def vcommTestSetStallRank(comm, rank: int) -> None:
    _check(lib().vcommTestSetStallRank(comm, rank), "vcommTestSetStallRank")


def vcommTestSetBadFlagRank(comm, rank: int) -> None:
    _check(lib().vcommTestSetBadFlagRank(comm, rank), "vcommTestSetBadFlagRank")


def vcommTestSetJitterNs(comm, max_ns: int) -> None:
    _check(lib().vcommTestSetJitterNs(comm, max_ns), "vcommTestSetJitterNs")


def vcommQueryPlan(comm, coll: int, count: int, datatype, aligned: int = 32) -> dict:
    """The plan for buffers whose pointers share `aligned`-byte alignment (1..32)."""
    info = vPlanInfo_t()
    _check(lib().vcommQueryPlan(comm, coll, count, _dtype_code(datatype), int(aligned),
                                ctypes.byref(info)), "vcommQueryPlan")
    return info.as_dict()


def vPlanCompute(**req) -> vPlanInfo_t:
    q = vPlanRequest_t()
    for k, v in req.items():
        setattr(q, k, v)
    info = vPlanInfo_t()
    _check(lib().vPlanCompute(ctypes.byref(q), ctypes.byref(info)), "vPlanCompute")
    return info


def vPlanTreeLinks(n_ranks: int, rank: int, tree: int = 0) -> tuple[int, int, int]:
    u, a, b = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().vPlanTreeLinks(n_ranks, rank, tree, ctypes.byref(u), ctypes.byref(a), ctypes.byref(b)),
           "vPlanTreeLinks")
    return u.value, a.value, b.value


def vPlanChannelRange(plan: vPlanInfo_t, count: int, channel: int, block: int) -> tuple[int, int]:
    lo, hi = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().vPlanChannelRange(ctypes.byref(plan), count, channel, block, ctypes.byref(lo),
                                   ctypes.byref(hi)), "vPlanChannelRange")
    return lo.value, hi.value


def vAllReduce(sendbuffs, recvbuffs, count: int, datatype, op, comm, stream=None) -> None:
    _check(lib().vAllReduce(*_pair(comm, sendbuffs, recvbuffs), count, _dtype_code(datatype),
                            _op_code(op), comm, _stream(stream)), "vAllReduce")


def vReduceScatter(sendbuffs, recvbuffs, recvcount: int, datatype, op, comm, stream=None) -> None:
    _check(lib().vReduceScatter(*_pair(comm, sendbuffs, recvbuffs), recvcount,
                                _dtype_code(datatype), _op_code(op), comm, _stream(stream)), "vReduceScatter")


def vReduceScatterScaleCast(sendbuffs, recvbuffs, recvcount: int, datatype, op, out_type, scale: float,
                            comm, stream=None) -> None:
    _check(lib().vReduceScatterScaleCast(*_pair(comm, sendbuffs, recvbuffs), recvcount,
                                         _dtype_code(datatype), _op_code(op), _dtype_code(out_type),
                                         ctypes.c_float(scale), comm, _stream(stream)),
           "vReduceScatterScaleCast")


def vAllGather(sendbuffs, recvbuffs, sendcount: int, datatype, op, comm, stream=None) -> None:
    _check(lib().vAllGather(*_pair(comm, sendbuffs, recvbuffs), sendcount, _dtype_code(datatype),
                            _op_code(op), comm, _stream(stream)), "vAllGather")


def vBroadcast(sendbuffs, recvbuffs, count: int, datatype, op, root: int, comm, stream=None) -> None:
    _check(lib().vBroadcast(*_pair(comm, sendbuffs, recvbuffs), count, _dtype_code(datatype),
                            _op_code(op), root, comm, _stream(stream)), "vBroadcast")


def vAllToAll(sendbuffs, recvbuffs, count: int, datatype, op, comm, stream=None) -> None:
    _check(lib().vAllToAll(*_pair(comm, sendbuffs, recvbuffs), count, _dtype_code(datatype),
                           _op_code(op), comm, _stream(stream)), "vAllToAll")


def vReduce(sendbuffs, recvbuffs, count: int, datatype, op, root: int, comm, stream=None) -> None:
    _check(lib().vReduce(*_pair(comm, sendbuffs, recvbuffs), count, _dtype_code(datatype),
                         _op_code(op), root, comm, _stream(stream)), "vReduce")


def vGather(sendbuffs, recvbuffs, sendcount: int, datatype, root: int, comm, stream=None) -> None:
    _check(lib().vGather(*_pair(comm, sendbuffs, recvbuffs), sendcount, _dtype_code(datatype),
                         root, comm, _stream(stream)), "vGather")


def vScatter(sendbuffs, recvbuffs, recvcount: int, datatype, root: int, comm, stream=None) -> None:
    _check(lib().vScatter(*_pair(comm, sendbuffs, recvbuffs), recvcount, _dtype_code(datatype),
                          root, comm, _stream(stream)), "vScatter")


def vAllToAllv(sendbuffs, recvbuffs, counts, sdispls, rdispls, datatype, comm, stream=None) -> None:
    _check(lib().vAllToAllv(*_pair(comm, sendbuffs, recvbuffs), _addr(counts), _addr(sdispls),
                            _addr(rdispls), _dtype_code(datatype), comm, _stream(stream)), "vAllToAllv")


def vAllReduceNoAlloc(sendbuffs, recvbuffs, count: int, datatype, op, n_ranks: int, n_channels: int = 1,
                      protocol=vProtoSimple, stream=None) -> None:
    """The ring all-reduce that allocates nothing (see include/vcomm.h)."""
    proto = PROTOCOLS[protocol] if isinstance(protocol, str) else protocol
    _check(lib().vAllReduceNoAlloc(_ptr_array(sendbuffs, n_ranks), _ptr_array(recvbuffs, n_ranks), count, _dtype_code(datatype),
                                   _op_code(op), n_ranks, n_channels, proto, _stream(stream)),
           "vAllReduceNoAlloc")


# ---- operators next to the collectives -------------------------------------------------------

def vBuffers(bufs) -> Buffers:
    """The device addresses of a list of buffers (one per rank; None for NULL) as a C array,
    which every call here takes in place of the list: a caller whose buffers stay where they
    are marshals them once.  It holds addresses, not the tensors: the caller keeps those."""
    bufs = list(bufs)
    return Buffers(_ptr_array(bufs, len(bufs)))


def vRmsNormDesc(rows: int, hidden: int, datatype, weight_type=None, eps: float = 1e-6, send_stride: int = 0,
                 residual_stride: int = 0, recv_stride: int = 0, quant_group: int = 0) -> vRmsNormDesc_t:
    """Sizes, strides (in elements, 0 for ``hidden``) and types of an RMS norm's calls; the
    weight's type is the data's unless ``weight_type`` says float32."""
    dt = _dtype_code(datatype)
    return vRmsNormDesc_t(rows, hidden, send_stride, residual_stride, recv_stride, eps, dt,
                          dt if weight_type is None else _dtype_code(weight_type), quant_group)


def vAllReduceRmsNorm(desc, sendbuffs, residual, weight, residual_out, recvbuffs, rstd, comm, stream=None) -> None:
    """All-reduce + residual + RMS norm; residual, residual_out, rstd and entries of recvbuffs
    may be None."""
    n = _n_ranks(comm)
    _check(lib().vAllReduceRmsNorm(ctypes.addressof(desc), _ptr_array(sendbuffs, n), _addr(residual), _addr(weight),
                                   _addr(residual_out), _ptr_array(recvbuffs, n), _addr(rstd), comm, _stream(stream)),
           "vAllReduceRmsNorm")


def vAllReduceRmsNormQuant(desc, sendbuffs, residual, weight, residual_out, recvbuffs, scalebuffs, rstd, comm,
                           stream=None) -> None:
    """The same with e4m3 bytes in recvbuffs and their fp32 scales in scalebuffs."""
    n = _n_ranks(comm)
    _check(lib().vAllReduceRmsNormQuant(ctypes.addressof(desc), _ptr_array(sendbuffs, n), _addr(residual),
                                        _addr(weight), _addr(residual_out), _ptr_array(recvbuffs, n),
                                        _ptr_array(scalebuffs, n), _addr(rstd), comm, _stream(stream)),
           "vAllReduceRmsNormQuant")


def vRmsNormBackwardWorkspace(desc, comm) -> int:
    """Bytes of workspace that vAllReduceRmsNormBackward needs for this descriptor."""
    b = ctypes.c_size_t(0)
    _check(lib().vRmsNormBackwardWorkspace(ctypes.addressof(desc), comm, ctypes.addressof(b)),
           "vRmsNormBackwardWorkspace")
    return b.value


def _workspace(workspace) -> tuple[int | None, int]:
    """Address and bytes of a workspace: a tensor, or (address, bytes)."""
    if isinstance(workspace, tuple):
        return workspace
    return workspace.data_ptr(), workspace.nbytes


def vAllReduceRmsNormBackward(desc, sendbuffs, hidden_states, rstd, weight, grad_residual, recvbuffs, grad_weight,
                              workspace, comm, stream=None) -> None:
    n = _n_ranks(comm)
    _check(lib().vAllReduceRmsNormBackward(ctypes.addressof(desc), _ptr_array(sendbuffs, n), _addr(hidden_states),
                                           _addr(rstd), _addr(weight), _addr(grad_residual), _ptr_array(recvbuffs, n),
                                           _addr(grad_weight), *_workspace(workspace), comm, _stream(stream)),
           "vAllReduceRmsNormBackward")


def vBlockNormDesc(rows: int, hidden: int, datatype, weight_type=None, eps: float = 1e-6, residual_scale: float = 1.0,
                   send_stride: int = 0, residual_stride: int = 0, recv_stride: int = 0) -> vBlockNormDesc_t:
    """Sizes, strides (in elements, 0 for ``hidden``) and types of a block norm's calls; the weights'
    type is the data's unless ``weight_type`` says float32."""
    dt = _dtype_code(datatype)
    return vBlockNormDesc_t(rows, hidden, send_stride, residual_stride, recv_stride, eps, residual_scale, dt,
                            dt if weight_type is None else _dtype_code(weight_type))


def vAllReduceBlockNorm(desc, sendbuffs, residual, post_weight, gate, pre_weight, block_out, residual_out, recvbuffs, rstd,
                        comm, stream=None) -> None:
    """All-reduce, the norm after a block, its gate, the scaled residual and the norm before the next
    block; residual, gate, block_out, residual_out, rstd and entries of recvbuffs may be None."""
    n = _n_ranks(comm)
    _check(lib().vAllReduceBlockNorm(ctypes.addressof(desc), _ptr_array(sendbuffs, n), _addr(residual), _addr(post_weight),
                                     _addr(gate), _addr(pre_weight), _addr(block_out), _addr(residual_out),
                                     _ptr_array(recvbuffs, n), _addr(rstd), comm, _stream(stream)), "vAllReduceBlockNorm")


def vBlockNormBackwardWorkspace(desc, comm) -> int:
    """Bytes of workspace that vAllReduceBlockNormBackward needs for this descriptor."""
    b = ctypes.c_size_t(0)
    _check(lib().vBlockNormBackwardWorkspace(ctypes.addressof(desc), comm, ctypes.addressof(b)),
           "vBlockNormBackwardWorkspace")
    return b.value


def vAllReduceBlockNormBackward(desc, sendbuffs, hidden_states, block, rstd, post_weight, gate, pre_weight, grad_stream,
                                grad_residual, recvbuffs, grad_post_weight, grad_gate, grad_pre_weight, workspace, comm,
                                stream=None) -> None:
    """Backward pass of vAllReduceBlockNorm; grad_stream, grad_residual and entries of recvbuffs may be
    None, grad_gate exactly where gate is."""
    n = _n_ranks(comm)
    _check(lib().vAllReduceBlockNormBackward(ctypes.addressof(desc), _ptr_array(sendbuffs, n), _addr(hidden_states),
                                             _addr(block), _addr(rstd), _addr(post_weight), _addr(gate), _addr(pre_weight),
                                             _addr(grad_stream), _addr(grad_residual), _ptr_array(recvbuffs, n),
                                             _addr(grad_post_weight), _addr(grad_gate), _addr(grad_pre_weight),
                                             *_workspace(workspace), comm, _stream(stream)), "vAllReduceBlockNormBackward")


def vMoeDesc(rows: int, hidden: int, ffn: int, experts: int, top_k: int, datatype, router_type=None, normalize: bool = True,
             row_stride: int = 0, recv_stride: int = 0) -> vMoeDesc_t:
    """Sizes, strides (in elements, 0 for ``hidden``) and types of a mixture of experts; the router's
    type is the data's unless ``router_type`` says float32."""
    dt = _dtype_code(datatype)
    return vMoeDesc_t(rows, hidden, ffn, experts, top_k, row_stride, recv_stride, dt,
                      dt if router_type is None else _dtype_code(router_type), int(normalize))


def vMoeRoute(desc, x, router_weight, bias, expert_ids, expert_weights, comm, stream=None) -> None:
    """Every token's best experts (int32) and their weights (fp32); bias may be None."""
    _check(lib().vMoeRoute(ctypes.addressof(desc), _addr(x), _addr(router_weight), _addr(bias), _addr(expert_ids),
                           _addr(expert_weights), comm, _stream(stream)), "vMoeRoute")


def vMoeExpertsWorkspace(desc, comm) -> int:
    """Bytes of workspace that vMoeExperts needs for this descriptor."""
    b = ctypes.c_size_t(0)
    _check(lib().vMoeExpertsWorkspace(ctypes.addressof(desc), comm, ctypes.addressof(b)), "vMoeExpertsWorkspace")
    return b.value


def vMoeExperts(desc, x, expert_ids, expert_weights, upbuffs, downbuffs, recvbuffs, workspace, comm, stream=None) -> None:
    """Every rank's experts applied to the tokens that chose them: partial sums, one per rank."""
    n = _n_ranks(comm)
    _check(lib().vMoeExperts(ctypes.addressof(desc), _addr(x), _addr(expert_ids), _addr(expert_weights),
                             _ptr_array(upbuffs, n), _ptr_array(downbuffs, n), _ptr_array(recvbuffs, n),
                             *_workspace(workspace), comm, _stream(stream)), "vMoeExperts")


def vSampleDesc(rows: int, vocab: int, datatype, part: int = 0, stride: int = 0) -> vSampleDesc_t:
    """Sizes of a draw from split logits: ``part`` columns a rank (0: an equal share), rows ``stride``
    elements apart (0: ``part``)."""
    return vSampleDesc_t(rows, vocab, part, stride, _dtype_code(datatype))


def vSample(desc, logitbuffs, temperature, top_k, top_p, min_p, uniform, tokenbuffs, logprob, comm, stream=None) -> None:
    """One token a row; temperature, top_k, top_p, min_p, logprob and entries of tokenbuffs may be None."""
    n = _n_ranks(comm)
    _check(lib().vSample(ctypes.addressof(desc), _ptr_array(logitbuffs, n), _addr(temperature), _addr(top_k), _addr(top_p),
                         _addr(min_p), _addr(uniform), _ptr_array(tokenbuffs, n), _addr(logprob), comm, _stream(stream)),
           "vSample")


_dropped_lists: list[int] = []       # handles of lists that lost their last reference


class TensorList:
    """A vGradList_t: the gradients of a step by their addresses.  Made by vTensorList it holds
    the tensors, so that their memory is no other's while a call may still scale it; made from
    addresses it holds nothing.

    ``close`` destroys it.  One that loses its last reference is destroyed when the next list is
    made: destruction frees device memory and waits for the device, which is not allowed while a
    graph is being captured, and references are lost at any time."""
    handle = tensors = None
    on_host = False                  # tensors of host memory: no call takes the list

    def __init__(self, n_ranks: int, counts, datatypes, replicated, grads, outs):
        while True:
            try:
                dropped = _dropped_lists.pop()
            except IndexError:       # none, or another thread has just taken the last
                break
            _check(lib().vGradListDestroy(dropped), "vGradListDestroy")
        n = len(counts)
        arrays = ((ctypes.c_size_t * n)(*counts), (ctypes.c_int * n)(*datatypes),
                  None if replicated is None else (ctypes.c_ubyte * n)(*map(bool, replicated)),
                  (ctypes.c_void_p * (n * n_ranks))(*grads),
                  None if outs is None else (ctypes.c_void_p * (n * n_ranks))(*outs))
        handle = ctypes.c_void_p()
        self.n_ranks = n_ranks
        _check(lib().vGradListCreate(ctypes.addressof(handle), n_ranks, n,
                                     *(None if a is None else ctypes.addressof(a) for a in arrays)), "vGradListCreate")
        self.handle = handle.value

    def close(self) -> None:
        if self.handle is not None:
            handle, self.handle, self.tensors = self.handle, None, None
            _check(lib().vGradListDestroy(handle), "vGradListDestroy")

    def __del__(self, dropped=_dropped_lists):
        if self.handle is not None:
            dropped.append(self.handle)


def vTensorList(grads, outs=None, replicated=None) -> TensorList:
    """The gradients of a step: ``grads[r][t]`` is rank r's tensor t, ``outs`` (the clipped
    gradients; None: in place) the same, ``replicated[t]`` whether every rank holds all of
    tensor t (None: none).  The list is of these tensors, which it holds: it serves every step that
    fills them anew (``zero_grad(set_to_none=False)``, gradients in buffers of the caller's).  Where
    a step brings new tensors (``set_to_none=True``), it still is of the old ones, and a new list
    has to be made."""
    if not grads:
        raise VcommError(vInvalidArgument, "a tensor list of no ranks")
    first = grads[0]
    if replicated is not None and len(replicated) != len(first):
        raise VcommError(vInvalidArgument, f"replicated names {len(replicated)} tensors of {len(first)}")
    addresses = []
    try:
        counts, dtypes = [t.numel() for t in first], [t.dtype for t in first]
        devices = [t.get_device() for t in first]
        for side in (grads,) if outs is None else (grads, outs):
            if len(side) != len(grads):
                raise VcommError(vInvalidArgument, f"outputs of {len(side)} ranks for gradients of {len(grads)}")
            for tensors in side:
                if [t.numel() for t in tensors] != counts or [t.dtype for t in tensors] != dtypes:
                    raise VcommError(vInvalidArgument, "every rank's tensors have the same sizes and types")
                if [t.get_device() for t in tensors] != devices:
                    raise VcommError(vInvalidArgument, "a list's tensors lie on one device")
                if not all([t.is_contiguous() for t in tensors]):
                    raise VcommError(vInvalidArgument, "tensors of a list are contiguous")
            addresses.append([t.data_ptr() for tensors in side for t in tensors])
    except (AttributeError, TypeError):
        raise VcommError(vInvalidArgument, "a list's entries are tensors: leave out parameters without a gradient") from None
    if len(set(devices)) > 1:
        raise VcommError(vInvalidArgument, "a list's tensors lie on one device")
    device = devices[0] if devices else None
    if device is not None and device >= 0:
        import torch
        if device != torch.cuda.current_device():
            raise VcommError(vInvalidArgument, f"tensors on device {device}; a list lives on the current device")
    codes = {d: _dtype_code(d) for d in set(dtypes)}
    made = TensorList(len(grads), counts, [codes[d] for d in dtypes], replicated, addresses[0],
                      None if outs is None else addresses[1])
    made.tensors = [list(tensors) for side in (grads, outs or []) for tensors in side]
    made.on_host = device == -1
    return made


def _list(tensors: TensorList, comm) -> int | None:
    n = _n_ranks(comm)
    if tensors.n_ranks != n:
        raise VcommError(vInvalidArgument, f"a tensor list of {tensors.n_ranks} ranks on a communicator of {n}")
    if tensors.on_host:
        raise VcommError(vInvalidArgument, "the list's tensors are in host memory")
    return tensors.handle


def vGradNormWorkspace(tensors: TensorList, comm) -> int:
    """Bytes of workspace that vGradNorm and vClipGradNorm need for this list."""
    b = ctypes.c_size_t(0)
    _check(lib().vGradNormWorkspace(_list(tensors, comm), comm, ctypes.addressof(b)), "vGradNormWorkspace")
    return b.value


def vGradNorm(tensors: TensorList, norm, workspace, comm, stream=None) -> None:
    """norm[0] = the 2-norm of all the ranks' gradients together."""
    _check(lib().vGradNorm(_list(tensors, comm), _addr(norm), *_workspace(workspace), comm, _stream(stream)),
           "vGradNorm")


def vClipGradNorm(tensors: TensorList, max_norm: float, norm, workspace, comm, stream=None) -> None:
    """vGradNorm, then every gradient scaled by min(1, max_norm / (norm + 1e-6))."""
    _check(lib().vClipGradNorm(_list(tensors, comm), max_norm, _addr(norm), *_workspace(workspace), comm,
                               _stream(stream)), "vClipGradNorm")
