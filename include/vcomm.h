/*
 * vcomm.h -- collectives among N virtual ranks that all live in one GPU's memory.
 *
 * A communicator (vcomm_t) stands for N ranks whose send and receive buffers are
 * ordinary device allocations on the current GPU.  Each call moves or reduces data
 * between those buffers entirely on that GPU; no other GPU, process or network is
 * involved and no NCCL call is made.
 *
 * The interface follows the NCCL calls described in the NCCL book (aireadcode.com),
 * section 2.1 (communicator, async error) and chapter 6 (ncclAllReduce(sendbuff,
 * recvbuff, count, datatype, op, comm, stream) -> ncclInfo -> ncclEnqueueCheck), with
 * one change that the virtual ranks force: every rank's buffer is named at once, so
 * sendbuffs / recvbuffs are host arrays of N device pointers, rank r at index r.
 * The collectives' meaning is the collective table of "AI Systems Performance
 * Engineering (3)" (all-reduce, reduce-scatter, all-gather, broadcast, all-to-all).
 *
 * Stream contract ("NCCL Expert Course 29: ProcessGroupNCCL, Stream, Event and
 * Work"): every collective is enqueued on the caller's stream and returns as soon as
 * it is enqueued.  The caller keeps the device buffers alive and unmodified until the
 * stream work completes.  The host pointer arrays and tables are copied before the
 * call returns and may be freed right after it (as ncclInfo copies the user's config,
 * NCCL book chapter 6).
 *
 * Errors: a call returns vInvalidArgument for bad arguments and launches nothing.
 * Failures found on the device (a staged transfer that waits past its deadline, an
 * abort, a bad all-to-all table) are recorded in the communicator's sticky async
 * error (NCCL book section 2.1, asyncResult / ncclCommGetAsyncError); every later
 * call on that communicator returns that error without launching, and the
 * communicator must be destroyed.
 *
 * Threading: a communicator is used by one host thread at a time.  Staged ring transfers
 * on one communicator share its FIFOs, so they must not overlap on the GPU: issue them on
 * one stream or order the streams (NCCL orders a communicator's operations the same way).
 *
 * CUDA graphs: collectives may be captured into a graph.  A ring transfer can be
 * captured only after an eager ring call of at least the same size on the same
 * communicator (its FIFOs are allocated then; capturing it earlier returns
 * vInvalidUsage); the captured transfer clears its control words (and, for LL and LL128,
 * its FIFOs, whose lines carry the flags) before every replay.  Graph
 * replays are ordered by the caller: vcommDestroy waits only for eager launches.
 *
 * Launch: the one-pass kernels are launched with programmatic stream serialization
 * (programmatic dependent launch): a kernel may become resident while the previous
 * kernel on the stream finishes, and waits for that kernel's completion (and its memory)
 * before touching any buffer, so stream order is kept.  VCOMM_PDL=0 launches them
 * plainly.
 */
#ifndef VCOMM_H
#define VCOMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The CUDA runtime's stream handle, declared the same way cuda_runtime_api.h does. */
typedef struct CUstream_st* cudaStream_t;

#define VCOMM_MAX_RANKS 64
#define VCOMM_MAX_CHANNELS 64

typedef struct vcomm* vcomm_t;

/* Result codes.  vInvalidUsage = 5 matches NCCL's ncclInvalidUsage ("NCCL Expert
 * Course 17", duplicate-device probe, "code=5"). */
typedef enum {
    vSuccess = 0,
    vUnhandledCudaError = 1, /* a CUDA runtime call failed (no device, launch error, ...) */
    vSystemError = 2,        /* host allocation failed */
    vInternalError = 3,
    vInvalidArgument = 4,    /* bad pointer, size, type, op, root or communicator */
    vInvalidUsage = 5,       /* valid arguments the communicator cannot serve, e.g. a staged
                                protocol whose CTAs cannot all be resident at once */
    vTimeout = 6,            /* a staged transfer waited past its deadline (async) */
    vInProgress = 7,
    vAborted = 8             /* vcommAbort stopped a running staged transfer (async) */
} vResult_t;

typedef enum { vFloat32 = 0, vFloat16 = 1, vBFloat16 = 2, vInt32 = 3 } vDataType_t;

/* Reductions.  sum and prod on fp16/bf16 widen both operands to fp32, apply one fp32
 * operation (round to nearest even) and round back to the storage type; int32 sum and
 * prod wrap modulo 2^32; min/max keep the running partial unless the next element
 * compares strictly below/above it. */
typedef enum { vSum = 0, vProd = 1, vMin = 2, vMax = 3 } vRedOp_t;

/* Staging protocols of the ring path (NCCL book section 2.4, "protocol"):
 * Simple moves raw data through FIFO slots guarded by head/tail counters; LL packs
 * 4 bytes of data with a 4-byte flag in every 8-byte word (half the bandwidth); LL128
 * carries 120 bytes of data and an 8-byte flag in every 128-byte line.
 * vProtoAuto lets the planner choose the protocol its cost model predicts fastest for the
 * collective, size and channel count (a ring cost model in the form of the NCCL book's
 * ring.cc, latency + bytes / bandwidth per protocol and channel count, fitted to staged-ring
 * times measured on GB300 for every collective, protocol and size from 1 KiB to 1 GiB per
 * rank: 2.2 % median error, and a pick within 15 % of the fastest protocol measured). */
typedef enum { vProtoSimple = 0, vProtoLL = 1, vProtoLL128 = 2, vProtoAuto = 3 } vProto_t;

/* Algorithms.  vAlgoOnePass: one kernel reads every rank's buffer once and writes
 * every output once (the virtual-rank counterpart of NCCL's symmetric-memory kernels,
 * NCCL book chapter 5 section 5).  vAlgoRing: the literal ring of the NCCL book
 * section 2.3, N-1 reduce-scatter steps then N-1 all-gather steps, each hop staged
 * through a device FIFO with the communicator's protocol.  Both give identical bits.
 * vAlgoAuto picks the smaller predicted time (on GB300 the one-pass kernels are faster
 * at every size: about 2 us of latency against 8-55 us for the ring's steps).
 * vAlgoTree (all-reduce only; other collectives run one-pass): the double binary tree of
 * the NCCL book chapter 4 (ncclGetBtree / ncclGetDtree).  The first half of the buffer,
 * up to alignUp(ceil(count / 2), 16 / elemSize) elements, is reduced up tree 0, the rest
 * up tree 1; a tree node combines its own element, then child 0's partial, then child
 * 1's; every rank receives the root's result.  Its bits generally differ from the ring
 * order's (a different reduction order). */
typedef enum { vAlgoAuto = 0, vAlgoOnePass = 1, vAlgoRing = 2, vAlgoTree = 3 } vAlgo_t;

typedef enum {
    vCollAllReduce = 0, vCollReduceScatter = 1, vCollAllGather = 2,
    vCollBroadcast = 3, vCollAllToAll = 4, vCollAllToAllv = 5,
    vCollReduce = 6, vCollGather = 7, vCollScatter = 8
} vColl_t;

/* ------------------------------------------------------------------------------- */
/* Communicator lifecycle                                                           */
/* ------------------------------------------------------------------------------- */

/* Create a communicator of nRanks virtual ranks on the current CUDA device.
 * nRanks in [1, VCOMM_MAX_RANKS]; nChannels in [1, VCOMM_MAX_CHANNELS] is the number
 * of channels (independent CTA groups, each owning a contiguous sub-range of every
 * rank's block: NCCL book section 2.2, "each channel handles count/nChannels
 * elements"); protocol is the ring path's staging.  Out-of-range values give
 * vInvalidArgument and *comm is left NULL (as ncclCommInitRankDev rejects nranks < 1
 * with ncclInvalidArgument, "NCCL Expert Course 17").  No usable device gives
 * vUnhandledCudaError.  The communicator owns a small status block in pinned host
 * memory and, once a ring transfer is planned, its staging FIFOs in device memory.
 * Environment (read once here): VCOMM_ALGO=auto|onepass|ring|tree, VCOMM_CHUNK_BYTES,
 * VCOMM_TIMEOUT_MS, VCOMM_COPY_TMA=0|1 (0, the default: every thread loads and stores; 1:
 * all-gather, gather and broadcast stage tiles in shared memory with TMA bulk copies when
 * blocks are 16-byte aligned), VCOMM_GRID=flat|persistent (flat, the default: the
 * one-pass kernels launch one CTA per slice of work; persistent: about one resident wave
 * of CTAs striding over it), VCOMM_PDL=0|1 (1, the default: programmatic dependent
 * launch of the one-pass kernels), VCOMM_DEBUG=INFO (prints every plan to stderr). */
vResult_t vcommInit(vcomm_t* comm, int nRanks, int nChannels, vProto_t protocol);

/* Wait for the last enqueued work that uses the communicator's device memory (staged
 * ring transfers, variable all-to-all, bulk-copy fan-out, vMoeExperts of 16-bit types), then free everything it owns.
 * The other collectives touch only the caller's buffers and need not have finished.
 * A NULL or already destroyed communicator gives vInvalidArgument. */
vResult_t vcommDestroy(vcomm_t comm);

/* Store the communicator's rank count N in *nRanks: the length that every sendbuffs and
 * recvbuffs array of a call on it must have (the communicator's nRanks field, NCCL book
 * section 2.1).  Host only.  A NULL pointer or a bad communicator gives vInvalidArgument. */
vResult_t vcommCount(vcomm_t comm, int* nRanks);

/* Store the sticky asynchronous error (vSuccess if none) in *asyncError.  Reads host
 * memory that the kernels write; it does not synchronize any stream.  A vTimeout is
 * fatal for the stream it happened on: the outputs of that call are undefined, and after
 * a timed-out bulk-copy fan-out (VCOMM_COPY_TMA=1) a load that had still not landed when
 * its CTA gave up may write into shared memory that a later kernel on the GPU uses, so
 * no later result is to be trusted either. */
vResult_t vcommGetAsyncError(vcomm_t comm, vResult_t* asyncError);

/* Ask running and future ring transfers of this communicator to stop: their waits
 * return and the sticky error becomes vAborted. */
vResult_t vcommAbort(vcomm_t comm);

const char* vcommGetErrorString(vResult_t result);

/* Group batching (NCCL book chapter 6 ncclPrepareTasks and chapter 7 ncclGroupStart /
 * ncclGroupEnd).  Between vcommGroupStart and vcommGroupEnd every collective call on
 * this communicator is recorded (its pointer arrays copied) and nothing is enqueued.  An
 * all-reduce is checked at the call, so its argument errors are returned there; the other
 * collectives return vSuccess and are checked when vcommGroupEnd enqueues them.
 * vcommGroupEnd enqueues the recorded calls: one-pass all-reduces of the same type, op,
 * stream and vector width are fused into one kernel launch (each keeping its own block
 * order, so the bits equal separate calls); a launch holds as many as its 32 KiB
 * parameter block fits, 32,496 / (40 + 16 N) of them (193 at N = 8), and a larger batch
 * takes several launches.  Every other call is enqueued as its own launch,
 * in call order.  Calls in one group must not depend on each other's results.  Groups
 * nest; only the outermost end enqueues.  vcommGroupEnd returns the first error of the
 * recorded calls, or vInvalidUsage without a matching start.  The work table travels in
 * the launch's parameters: no device memory, no upload, and on a stream being captured
 * into a CUDA graph the fused launch is captured like any other. */
vResult_t vcommGroupStart(vcomm_t comm);
vResult_t vcommGroupEnd(vcomm_t comm);

/* Tuning knobs (host only, take effect for later calls).  chunkBytes is the ring
 * path's data bytes per rank per chunk (one chunk = 4 FIFO slots, one slice = 2 slots;
 * NCCL book chapter 6, ALLREDUCE_CHUNKSTEPS / ALLREDUCE_SLICESTEPS); a slot holds
 * chunkBytes / 4 data bytes in chunkBytes / 4 FIFO bytes (Simple), twice that (LL) or
 * 128-byte lines of 120 data bytes (LL128).  It must be a power of two in [4 KiB,
 * 64 MiB], or 0 for the planner's default: the largest power of two <= 1 MiB that keeps
 * all of the communicator's FIFOs (8 slots per channel and rank) within 1 GiB.
 * timeoutMs bounds every device-side wait that sees no progress (>= 1; default 2000). */
vResult_t vcommSetAlgo(vcomm_t comm, vAlgo_t algo);
vResult_t vcommSetProtocol(vcomm_t comm, vProto_t protocol);
vResult_t vcommSetChunkBytes(vcomm_t comm, size_t chunkBytes);
vResult_t vcommSetTimeoutMs(vcomm_t comm, int timeoutMs);

/* ------------------------------------------------------------------------------- */
/* Collectives.  sendbuffs / recvbuffs: host arrays of nRanks pointers to memory the */
/* device can access (device allocations, pinned or managed host memory: the kernels */
/* read and write it directly, so host buffers need no staging copies).              */
/* Any element-aligned pointer is accepted; when every pointer and the sizes allow   */
/* 16-byte (or 32-byte) vectors the vector path runs, otherwise an element path (for */
/* 2-byte types, 16-byte vectors realigned to the outputs where the offsets allow);  */
/* the output bits are the same.  The element paths read no byte outside the 16-byte */
/* aligned blocks that hold a buffer's own elements.  count == 0 returns vSuccess    */
/* and launches nothing (NCCL book chapter 6, taskAppend).  With nRanks == 1 every   */
/* collective is a copy.                                                             */
/* ------------------------------------------------------------------------------- */

/* All-reduce ("AI Systems Performance Engineering (3)", collective table, all-reduce row;
 * NCCL book section 2.3, the ring as reduce-scatter then all-gather):
 * recvbuffs[r][e] = the reduction over all ranks of sendbuffs[.][e], e < count, for
 * every rank r.  Element e belongs to block b = e / B with
 * B = alignUp(ceil(count / nRanks), 16 / elemSize) (the tail-chunk rule of
 * RingARAlgorithm::getNextSendAddr, NCCL book section 2.3), and block b is reduced in
 * ring order: ranks b+1, b+2, ..., b (mod nRanks), each partial rounded to the data
 * type.  In place (sendbuffs[r] == recvbuffs[r]) is allowed; other overlap is not. */
vResult_t vAllReduce(const void* const* sendbuffs, void* const* recvbuffs, size_t count,
                     vDataType_t datatype, vRedOp_t op, vcomm_t comm, cudaStream_t stream);

/* Reduce-scatter ("AI Systems Performance Engineering (3)", collective table,
 * reduce-scatter row: rank r ends with the reduction of block r; the reduce-scatter half
 * of the ring in the NCCL book section 2.3).
 * sendbuffs[r] holds nRanks * recvcount elements; recvbuffs[r][t] = the reduction of
 * sendbuffs[.][r * recvcount + t] in ring order ranks r+1, ..., r.  In place means
 * recvbuffs[r] == sendbuffs[r] + r * recvcount. */
vResult_t vReduceScatter(const void* const* sendbuffs, void* const* recvbuffs, size_t recvcount,
                         vDataType_t datatype, vRedOp_t op, vcomm_t comm, cudaStream_t stream);

/* vReduceScatter with a fused epilogue: recvbuffs[r][t] = (float)acc * scale computed
 * in fp32 (round to nearest even) and stored as outType, which is vFloat32 or the
 * input type.  datatype must be a floating type.  For gradient averaging scale is
 * 1/nRanks ("AI Systems Performance Engineering (3)", p.grad /= world_size). */
vResult_t vReduceScatterScaleCast(const void* const* sendbuffs, void* const* recvbuffs,
                                  size_t recvcount, vDataType_t datatype, vRedOp_t op,
                                  vDataType_t outType, float scale, vcomm_t comm,
                                  cudaStream_t stream);

/* All-gather ("AI Systems Performance Engineering (3)", collective table, all-gather row:
 * every rank ends with every rank's piece, in rank order; the ring all-gather of "NCCL
 * Expert Course 17" and NCCL book section 2.3 when staged):
 * recvbuffs[r][s * sendcount + t] = sendbuffs[s][t] for every r.  op is ignored (the
 * data is moved as bytes).  In place means sendbuffs[r] == recvbuffs[r] + r * sendcount. */
vResult_t vAllGather(const void* const* sendbuffs, void* const* recvbuffs, size_t sendcount,
                     vDataType_t datatype, vRedOp_t op, vcomm_t comm, cudaStream_t stream);

/* Broadcast ("AI Systems Performance Engineering (3)", collective table, broadcast row:
 * the root's buffer copied to every rank):
 * recvbuffs[r][0..count) = sendbuffs[root][0..count) for every r; root in [0, nRanks).
 * Only sendbuffs[root] is read; the other entries may be NULL.  op is ignored. */
vResult_t vBroadcast(const void* const* sendbuffs, void* const* recvbuffs, size_t count,
                     vDataType_t datatype, vRedOp_t op, int root, vcomm_t comm,
                     cudaStream_t stream);

/* Uniform all-to-all ("AI Systems Performance Engineering (3)", collective table,
 * all-to-all row: rank i's block j goes to rank j as its block i): count elements per
 * block, nRanks blocks per buffer;
 * recvbuffs[j][i * count + t] = sendbuffs[i][j * count + t].  op is ignored.
 * Send and receive buffers must not overlap. */
vResult_t vAllToAll(const void* const* sendbuffs, void* const* recvbuffs, size_t count,
                    vDataType_t datatype, vRedOp_t op, vcomm_t comm, cudaStream_t stream);

/* Variable all-to-all.  counts, sdispls and rdispls are DEVICE arrays of nRanks *
 * nRanks int32 values, in elements: counts[i * nRanks + j] elements go from
 * sendbuffs[i] + sdispls[i * nRanks + j] to recvbuffs[j] + rdispls[j * nRanks + i].
 * The caller guarantees that every block lies inside its buffers.  A rank that sends
 * (receives) nothing may pass a NULL send (receive) buffer, as an empty tensor has.  A
 * negative entry, or a positive count whose source or destination buffer is NULL, makes
 * the kernel skip that block and sets the sticky error vInvalidArgument.  Send and
 * receive buffers must not overlap.
 * Each call hands out its tiles from a pair of counters that the communicator owns.
 * Eager calls rotate through 64 pairs; a call captured into a CUDA graph keeps the pair
 * it was captured with, taken from a second set of 64 that eager calls never use.  So an
 * eager call may run on the GPU at the same time as a replay of a captured call, and up
 * to 64 eager calls may be in flight together; beyond that, vAllToAllv kernels on one
 * communicator must not overlap on the GPU (two replays of one graph, or of calls
 * captured 64 captured calls apart, share a pair). */
vResult_t vAllToAllv(const void* const* sendbuffs, void* const* recvbuffs, const int32_t* counts,
                     const int32_t* sdispls, const int32_t* rdispls, vDataType_t datatype,
                     vcomm_t comm, cudaStream_t stream);

/* Rooted collectives ("AI Systems Performance Engineering (3)", collective table:
 * reduce, gather and scatter rows).  root in [0, nRanks); recvbuffs / sendbuffs entries
 * that the call does not use may be NULL.
 *
 * vReduce: recvbuffs[root][e] = the reduction of sendbuffs[.][e] for e < count, every
 * element in the order of a ring chain that ends at the root: ranks root+1, ..., root
 * (the order block `root` of vAllReduce uses).  In place: recvbuffs[root] ==
 * sendbuffs[root].
 * vGather: recvbuffs[root][s * sendcount + t] = sendbuffs[s][t].  In place:
 * sendbuffs[root] == recvbuffs[root] + root * sendcount.
 * vScatter: recvbuffs[r][t] = sendbuffs[root][r * recvcount + t].  In place:
 * recvbuffs[root] == sendbuffs[root] + root * recvcount. */
vResult_t vReduce(const void* const* sendbuffs, void* const* recvbuffs, size_t count,
                  vDataType_t datatype, vRedOp_t op, int root, vcomm_t comm, cudaStream_t stream);
vResult_t vGather(const void* const* sendbuffs, void* const* recvbuffs, size_t sendcount,
                  vDataType_t datatype, int root, vcomm_t comm, cudaStream_t stream);
vResult_t vScatter(const void* const* sendbuffs, void* const* recvbuffs, size_t recvcount,
                   vDataType_t datatype, int root, vcomm_t comm, cudaStream_t stream);

/* ------------------------------------------------------------------------------- */
/* Operators next to the collectives: the all-reduce that ends a tensor-parallel     */
/* product fused with the residual's addition and the RMS norm behind it, its 8-bit  */
/* output and its backward pass, and the global gradient norm with clipping that     */
/* follows the gradients' reduction.  They take the communicator, the stream and the */
/* per-rank pointer arrays as the collectives do, return the same errors, may be     */
/* grouped and captured, and hold every sum, statistic and norm in fp32 or more.     */
/* Where one needs scratch memory, the caller passes it.                             */
/* ------------------------------------------------------------------------------- */

/* Longest row of the norms, in elements. */
#define VCOMM_MAX_HIDDEN 65536

typedef struct {
    size_t rows;               /* tokens, at most 2^31 - 1; 0 does nothing (the backward pass
                                  writes a zero weight gradient) */
    size_t hidden;             /* elements of a row, at most VCOMM_MAX_HIDDEN */
    size_t sendStride;         /* elements between the rows of every send buffer; 0: hidden */
    size_t residualStride;     /* the same of residual and residualOut, and of hiddenStates and
                                  gradResidual in the backward pass; 0: hidden */
    size_t recvStride;         /* the same of every receive buffer; 0: hidden */
    float eps;                 /* >= 0, added to the mean square */
    vDataType_t datatype;      /* vFloat32, vFloat16 or vBFloat16: of the sends, the residual, the
                                  stream and the outputs */
    vDataType_t weightType;    /* of the weight and its gradient: datatype or vFloat32 */
    int quantGroup;            /* 8-bit output: 0 for one scale a row, 128 for one per 128
                                  elements (the last group may be shorter) */
} vRmsNormDesc_t;

/* All-reduce, residual addition and RMS norm in one pass:
 *   h = sum over ranks of sendbuffs[r] (in rank order) + residual      per element, in fp32
 *   rstd = 1 / sqrt(mean over the row of h^2 + eps)
 *   recvbuffs[r] = h * rstd * weight      for every rank r, rounded once to the data type
 * residualOut gets h rounded to the data type, rstd (fp32, one per row) what the backward
 * pass needs.  The residual stream is the same on every rank, so it is passed once.
 * residual, residualOut and rstd may be NULL.  A rank whose recvbuffs entry is NULL gets no
 * copy of the output; at least one has to want it.  Unlike vAllReduce's, the partial sums
 * are not rounded to the data type from rank to rank.
 * In place: recvbuffs[r] == sendbuffs[r] with equal strides, and residualOut == residual;
 * no other overlap.  Any element-aligned pointer and stride is accepted: bytes between rows
 * are not written, and read only within the 16-byte aligned blocks that hold a row's own
 * elements.  An infinite or NaN element makes its own row NaN or zero as the formula has
 * it, no other row. */
vResult_t vAllReduceRmsNorm(const vRmsNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                            const void* weight, void* residualOut, void* const* recvbuffs, float* rstd,
                            vcomm_t comm, cudaStream_t stream);

/* The same with the normed output in 8 bits (e4m3: 4 exponent bits, 3 mantissa bits, no
 * infinity): recvbuffs[r] holds bytes, with recvStride bytes between rows, and scalebuffs[r]
 * the fp32 scales, one per row or ceil(hidden / 128) per row, without gaps:
 *   amax = max(2^-64, max |h * weight| * rstd) of the row or group, scale = amax / 448,
 *   recvbuffs[r] = h * weight * rstd / scale rounded to the nearest e4m3 value.
 * A NaN in a row or group makes its scale NaN.  A rank that wants the output wants its
 * scales. */
vResult_t vAllReduceRmsNormQuant(const vRmsNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                                 const void* weight, void* residualOut, void* const* recvbuffs,
                                 float* const* scalebuffs, float* rstd, vcomm_t comm, cudaStream_t stream);

/* Backward pass of vAllReduceRmsNorm.  sendbuffs[r] is rank r's partial gradient of the
 * normed output (its column-parallel product's input gradient), hiddenStates the stream that
 * was normed (residualOut), rstd what the forward pass stored, gradResidual (may be NULL) the
 * gradient that reaches the stream by another way:
 *   dy = sum over ranks of sendbuffs[r],  xhat = hiddenStates * rstd,  g = dy * weight
 *   recvbuffs[r] = rstd * (g - xhat * mean(g * xhat)) + gradResidual
 *   gradWeight = sum over rows of dy * xhat
 * The output is the gradient of the residual and, as the stream is a plain sum, of every
 * rank's partial sum too.  recvbuffs entries may be NULL, but not all.  In place:
 * recvbuffs[r] == sendbuffs[r] with equal strides, or one recvbuffs entry == gradResidual
 * with equal strides.  The workspace is at least the number of bytes that
 * vRmsNormBackwardWorkspace gives for the descriptor, 16-byte aligned, and used by nothing
 * else until the call's work is done; a smaller one gives vInvalidArgument.  The same call
 * (on buffers of the same offsets from 16 bytes) gives the same bits. */
vResult_t vRmsNormBackwardWorkspace(const vRmsNormDesc_t* desc, vcomm_t comm, size_t* bytes);
vResult_t vAllReduceRmsNormBackward(const vRmsNormDesc_t* desc, const void* const* sendbuffs,
                                    const void* hiddenStates, const float* rstd, const void* weight,
                                    const void* gradResidual, void* const* recvbuffs, void* gradWeight,
                                    void* workspace, size_t workspaceBytes, vcomm_t comm, cudaStream_t stream);

/* The norms after and before a block, with its gate and the residual's scale, behind the
 * all-reduce of the block's partial sums:
 *   b = sum over ranks of sendbuffs[r] (in rank order)               per element, in fp32
 *   n = b * rstd[0] * postWeight,  rstd[0] = 1 / sqrt(mean over the row of b^2 + eps)
 *   h = residualScale * residual + gate * n
 *   recvbuffs[r] = h * rstd[1] * preWeight,  rstd[1] = 1 / sqrt(mean over the row of h^2 + eps)
 * gate is one value per channel, shared by all rows.  blockOut gets b, residualOut h, each
 * rounded once to the data type; rstd (fp32, [2][rows]) first the block's values, then the
 * stream's: these are what the backward pass needs.  residual, gate (then 1), blockOut,
 * residualOut and rstd may be NULL, and so may recvbuffs entries, but not all.
 * In place: recvbuffs[r] == sendbuffs[r] with equal strides, and residualOut == residual; no
 * other overlap.  Pointers, strides and values as for vAllReduceRmsNorm. */
typedef struct {
    size_t rows;               /* as in vRmsNormDesc_t */
    size_t hidden;
    size_t sendStride;         /* elements between the rows of every send buffer; 0: hidden */
    size_t residualStride;     /* the same of residual, residualOut and blockOut, and of
                                  hiddenStates, block, gradStream and gradResidual */
    size_t recvStride;         /* the same of every receive buffer; 0: hidden */
    float eps;                 /* >= 0, added to both mean squares */
    float residualScale;       /* finite */
    vDataType_t datatype;      /* vFloat32, vFloat16 or vBFloat16 */
    vDataType_t weightType;    /* of both weights, the gate and their gradients: datatype or vFloat32 */
} vBlockNormDesc_t;
vResult_t vAllReduceBlockNorm(const vBlockNormDesc_t* desc, const void* const* sendbuffs, const void* residual,
                              const void* postWeight, const void* gate, const void* preWeight, void* blockOut,
                              void* residualOut, void* const* recvbuffs, float* rstd, vcomm_t comm, cudaStream_t stream);

/* Backward pass of vAllReduceBlockNorm.  sendbuffs[r] is rank r's partial gradient of the normed
 * output, hiddenStates and block what the forward pass stored (residualOut, blockOut), gradStream
 * (may be NULL) the gradient that reaches the stream h by another way:
 *   dy = sum over ranks of sendbuffs[r],  x2 = hiddenStates * rstd[1],  g2 = dy * preWeight
 *   dh = rstd[1] * (g2 - x2 * mean(g2 * x2)) + gradStream
 *   gradResidual = residualScale * dh
 *   x1 = block * rstd[0],  g1 = dh * gate * postWeight
 *   recvbuffs[r] = rstd[0] * (g1 - x1 * mean(g1 * x1))
 *   gradPreWeight = sum over rows of dy * x2,  gradPostWeight = gate * sum over rows of dh * x1,
 *   gradGate = postWeight * the same sum
 * The output is the gradient of every rank's partial sum.  gradResidual may be NULL, and so may
 * recvbuffs entries, but not all; gradGate is NULL exactly where gate is.  In place:
 * recvbuffs[r] == sendbuffs[r] with equal strides, gradResidual == gradStream; no other overlap.
 * rows == 0 writes zero weight gradients.  The workspace is at least what
 * vBlockNormBackwardWorkspace gives for the descriptor, 16-byte aligned, and used by nothing else
 * until the call's work is done; a smaller one gives vInvalidArgument.  The same call (on buffers
 * of the same offsets from 16 bytes) gives the same bits. */
vResult_t vBlockNormBackwardWorkspace(const vBlockNormDesc_t* desc, vcomm_t comm, size_t* bytes);
vResult_t vAllReduceBlockNormBackward(const vBlockNormDesc_t* desc, const void* const* sendbuffs, const void* hiddenStates,
                                      const void* block, const float* rstd, const void* postWeight, const void* gate,
                                      const void* preWeight, const void* gradStream, void* gradResidual,
                                      void* const* recvbuffs, void* gradPostWeight, void* gradGate, void* gradPreWeight,
                                      void* workspace, size_t workspaceBytes, vcomm_t comm, cudaStream_t stream);

/* A mixture of experts for a few tokens.  The tokens x are the same on every rank (a norm's output),
 * so they are passed once; the experts are split over the ranks: with share = ceil(experts /
 * nRanks), rank r holds experts [r * share, (r + 1) * share), the last ranks fewer or none. */
#define VCOMM_MAX_MOE_ROWS 1024
#define VCOMM_MAX_EXPERTS 1024
#define VCOMM_MAX_TOPK 32

typedef struct {
    size_t rows;               /* tokens, at most VCOMM_MAX_MOE_ROWS; 0 does nothing */
    size_t hidden;             /* elements of a token, at most VCOMM_MAX_HIDDEN */
    size_t ffn;                /* inner width of an expert, at most VCOMM_MAX_HIDDEN */
    int experts;               /* of all ranks together, at most VCOMM_MAX_EXPERTS */
    int topK;                  /* experts that a token goes to: at most VCOMM_MAX_TOPK, and experts */
    size_t rowStride;          /* elements between the rows of x; 0: hidden */
    size_t recvStride;         /* the same of every receive buffer; 0: hidden */
    vDataType_t datatype;      /* vFloat32, vFloat16 or vBFloat16: of x, the experts and the outputs */
    vDataType_t routerType;    /* of the router's weight: datatype or vFloat32 */
    int normalize;             /* the router's weights add up to 1 over the chosen experts (else over
                                  all experts) */
} vMoeDesc_t;

/* The router.  logits = x * routerWeight^T (routerWeight: [experts][hidden], without gaps), score =
 * logits + bias (fp32, [experts], may be NULL: it takes part in the choice alone).
 * expertIds[t][k] (int32, [rows][topK]) is the expert with the k-th largest score, ties to the lower
 * index and a NaN last; expertWeights[t][k] (fp32) = exp(logit of it) / sum of exp(logits), over
 * the chosen experts or all (normalize).  Where fp32 sums leave open which of two scores is the
 * larger, their logits are computed anew with twice the digits, so the choice is that of exact
 * sums but for scores closer than about 2^-45 of their products' magnitudes, or than 10^-24.  The
 * weights' logits are fp32 sums, off by at most 17 units of 2^-24 of their products' magnitudes. */
vResult_t vMoeRoute(const vMoeDesc_t* desc, const void* x, const void* routerWeight, const float* bias,
                    int32_t* expertIds, float* expertWeights, vcomm_t comm, cudaStream_t stream);

/* The experts' layer.  upbuffs[r] holds rank r's experts' [2 * ffn][hidden] matrices (the gate's rows
 * first, then the linear part's), downbuffs[r] their [hidden][ffn] ones, without gaps:
 *   g = gate_e * x[t],  u = linear_e * x[t],  a = g / (1 + exp(-g)) * u
 *   recvbuffs[r][t] = sum over k with expertIds[t][k] = e held by rank r of
 *                     expertWeights[t][k] * (down_e * a)
 * in the order of k and in fp32, rounded once: the ranks' partial sums, which vAllReduceRmsNorm or
 * vAllReduceBlockNorm adds up.  With 16-bit types the products are the tensor cores', whose fp32 sums may
 * cut off where others round, and a is held as two values of the type: right to 2^-18 of itself with bf16,
 * with fp16 to 2^-22 of itself or 2^-35, whichever is more, and infinite beyond 131008.  With fp32 all of it
 * is in fp32.  A token that goes to no expert of a rank gets zeros there.  An id outside [0, experts) is
 * no expert (padding); an expert named twice counts twice.  A rank that holds no expert may pass NULL
 * weights; every recvbuffs entry is written.  Outputs overlap no input.  The workspace is at least what
 * vMoeExpertsWorkspace gives for the descriptor, 16-byte aligned, and used by nothing else until the
 * call's work is done. */
vResult_t vMoeExpertsWorkspace(const vMoeDesc_t* desc, vcomm_t comm, size_t* bytes);
vResult_t vMoeExperts(const vMoeDesc_t* desc, const void* x, const int32_t* expertIds, const float* expertWeights,
                      const void* const* upbuffs, const void* const* downbuffs, void* const* recvbuffs,
                      void* workspace, size_t workspaceBytes, vcomm_t comm, cudaStream_t stream);

/* One token for every row of logits whose vocabulary is split over the ranks: logitbuffs[r] holds
 * columns [r * part, (r + 1) * part) of every row, those below vocab.  temperature, topP, minP and
 * uniform are fp32, topK int32, one value a row, in device memory; all but uniform may be NULL.
 *   e_i = exp((logit_i - max) / temperature), all filters in the order of the largest e, ties to the
 *   lower index: the topK first (<= 0: all); of those the shortest run whose sum reaches topP times
 *   theirs, at least one (topP >= 1 or NaN: all); of those the ones with e_i >= minP, which at most
 *   leaves the largest (<= 0 or NaN: all).
 *   token = the first kept index i, in the vocabulary's order, with
 *           (sum of kept e up to i) > uniform * (sum of kept e)
 * A temperature that is not above zero takes the largest logit, the first of equals, without a
 * draw.  uniform lies in [0, 1); other values act as the nearest one, a NaN as 0.  Sums are
 * taken in units of 2^-44, of e right to 2^-28.8 of itself (at temperatures from 10^-37 to 10^37), and the
 * same call gives the same tokens.
 * tokenbuffs[r] (int32, one a row) may be NULL for ranks that want none, but not all; logprob (fp32,
 * one a row, may be NULL) = log of the token's share of all e before the filters (temperature 1 where
 * the largest is taken); that sum is right to 2^-17 of itself where a filter is given, else as those
 * above.
 * Logits of minus infinity and NaN are never drawn; infinite ones share the draw alone.  A row in
 * which nothing is left gives the token -1 and a NaN. */
#define VCOMM_MAX_VOCAB 262144
#define VCOMM_MAX_SAMPLE_ROWS 16777216

typedef struct {
    size_t rows;               /* at most VCOMM_MAX_SAMPLE_ROWS; 0 does nothing */
    size_t vocab;              /* tokens to draw from, 1 to VCOMM_MAX_VOCAB */
    size_t part;               /* columns of a rank; 0: ceil(vocab / nRanks).  A rank all of whose columns
                                  lie behind vocab may pass a NULL buffer */
    size_t stride;             /* elements between the rows of every logit buffer; 0: part */
    vDataType_t datatype;      /* vFloat32, vFloat16 or vBFloat16 */
} vSampleDesc_t;
vResult_t vSample(const vSampleDesc_t* desc, const void* const* logitbuffs, const float* temperature,
                  const int32_t* topK, const float* topP, const float* minP, const float* uniform,
                  int32_t* const* tokenbuffs, float* logprob, vcomm_t comm, cudaStream_t stream);

/* The gradients that a norm is taken over: nTensors tensors on each of nRanks ranks.  A tensor
 * is either split (each rank holds a piece of counts[t] elements: reduce-scattered or
 * tensor-parallel) or replicated (each rank holds all of it: all-reduced).  Any number of
 * tensors, of any sizes, up to 2^40 elements in all.
 *   counts      [nTensors] elements on each rank; 0: skipped
 *   datatypes   [nTensors] vFloat32, vFloat16 or vBFloat16
 *   replicated  [nTensors], or NULL: all split
 *   grads       [nRanks * nTensors], rank r's tensor t at r * nTensors + t
 *   outs        the clipped gradients, in the same order and types; NULL: in place
 * The arrays are host memory and may be freed when the call returns.  The list lives on the
 * current device; it holds the tensors' addresses, so it serves every step for as long as they
 * stay where they are, and the only device memory that these operators allocate: a table of 32
 * bytes per 32 KiB of gradients.  Creating and destroying a list waits for the device, so
 * neither goes into a graph's capture.  vGradListCreate leaves *list NULL on an error.  A NULL
 * or destroyed list gives vInvalidArgument, from every call and from the end of a group that
 * recorded it while it lived; its handle is not given to another list.  A graph that captured a
 * call reads the list's table: the list has to outlive its last replay. */
typedef struct vgradlist* vGradList_t;
vResult_t vGradListCreate(vGradList_t* list, int nRanks, int nTensors, const size_t* counts,
                          const vDataType_t* datatypes, const unsigned char* replicated,
                          const void* const* grads, void* const* outs);
vResult_t vGradListDestroy(vGradList_t list);

/* *norm (device memory, fp32) = the 2-norm of all ranks' gradients together, a replicated
 * tensor counted once, by rank 0's copy.  Squares are taken and added in fp32 over at most
 * 64 elements, their sums in fp64, in an order that the sizes and the tensors' offsets from 16
 * bytes fix.  A square above fp32's range makes the norm infinite, one below it adds nothing.
 * vClipGradNorm then scales every rank's gradients by min(1, maxNorm / (norm + 1e-6)),
 * rounded once to their type (no element is rewritten in place where that factor is 1).  A
 * norm that is not finite scales as the formula has it: infinity by 0, NaN by NaN.  maxNorm
 * must be >= 0.  No tensor may overlap another, nor an output another tensor's gradient.
 * The list has as many ranks as the communicator and lives on its device; calls on one list
 * must not overlap on the GPU (they share its counter).  The workspace is at least what
 * vGradNormWorkspace gives for the list, 16-byte aligned, used by nothing else until the
 * call's work is done. */
vResult_t vGradNormWorkspace(vGradList_t list, vcomm_t comm, size_t* bytes);
vResult_t vGradNorm(vGradList_t list, float* norm, void* workspace, size_t workspaceBytes,
                    vcomm_t comm, cudaStream_t stream);
vResult_t vClipGradNorm(vGradList_t list, float maxNorm, float* norm, void* workspace,
                        size_t workspaceBytes, vcomm_t comm, cudaStream_t stream);

/* Ring all-reduce for callers that cannot allocate device memory.  The pages have no
 * counterpart to this call; it exists for code that must not call cudaMalloc (allocator
 * or memory-pool callbacks, which must not re-enter the allocator; runtimes that own all
 * device memory and hand it out themselves).  No communicator is needed and nothing is
 * allocated: the staging FIFOs and control words live in one fixed device array inside
 * this library (64 KiB + 8 MiB, held on every GPU that loads the library until the
 * process exits).
 * The result is bit-identical to vAllReduce.  The caller passes the buffers as for
 * vAllReduce plus nRanks (2..64), nChannels and protocol (Simple, LL or LL128); the
 * ring uses chunks of 64 KiB of data (32 KiB for LL and LL128, whose slots take more FIFO
 * bytes than they carry), so nRanks * nChannels may be at most 64 -- larger rings
 * return vInvalidArgument (as do the usual argument errors), and a ring whose CTAs
 * cannot all be resident returns vInvalidUsage.  The first call on a device looks up
 * the array's address (cudaGetSymbolAddress), so make it before any stream capture;
 * every call checks the kept address (cudaPointerGetAttributes) and looks it up again
 * after a cudaDeviceReset.
 * Every call clears and reuses the same array: calls whose kernels overlap on the GPU
 * (another stream, another thread) race and must be serialized by the caller.  Waits
 * inside the kernel still end after 2 s without progress, but such a failure is not
 * reported (there is no communicator to hold an error) and the output is then
 * undefined. */
vResult_t vAllReduceNoAlloc(const void* const* sendbuffs, void* const* recvbuffs, size_t count,
                            vDataType_t datatype, vRedOp_t op, int nRanks, int nChannels,
                            vProto_t protocol, cudaStream_t stream);

/* ------------------------------------------------------------------------------- */
/* Planner (host only; needs no GPU)                                                */
/* ------------------------------------------------------------------------------- */

typedef struct {
    int nRanks, nChannels;
    int proto;                 /* vProto_t requested */
    int algo;                  /* vAlgo_t requested */
    int coll;                  /* vColl_t */
    int datatype;              /* vDataType_t */
    size_t count;              /* elements: AR/BC/Reduce count, RS/Scatter recvcount,
                                  AG/Gather sendcount, A2A block */
    size_t chunkBytes;         /* ring chunk bytes per rank (0 = default) */
    int aligned16;             /* 1 if every buffer pointer is 16-byte aligned */
    int smCount;               /* streaming multiprocessors of the device */
    size_t l2Bytes;            /* L2 cache size of the device (kept for callers; the current
                                  plans do not depend on it) */
    int aligned32;             /* 1 if every buffer pointer is 32-byte aligned */
    int noBulkCopy;            /* 1: never use TMA bulk copies (a communicator sets it unless
                                  VCOMM_COPY_TMA=1) */
    int persistentGrid;        /* 1: one-pass grids of about one resident wave whose CTAs
                                  stride over their work (VCOMM_GRID=persistent); 0 (the
                                  default): one CTA per slice of work, dispatched in order */
} vPlanRequest_t;

typedef struct {
    int algo;                  /* vAlgo_t chosen: vAlgoOnePass or vAlgoRing */
    int proto;                 /* vProto_t used by the ring path */
    int nChannels;
    int ctasPerChannel;        /* one-pass: CTAs in each channel's group */
    int gridCtas;              /* CTAs launched */
    int threadsPerCta;
    int vectorized;            /* 1 when the 16-byte vector path runs */
    int launches;              /* kernel launches of the call */
    size_t blockElems;         /* B: elements of one rank block (AR rule, or RS/AG block) */
    size_t channelElems;       /* elements of each block that one channel owns */
    size_t chunkElems;         /* ring: elements per block per chunk */
    size_t slotPayloadElems;   /* ring: data elements carried by one FIFO slot */
    size_t slotBytes;          /* ring: bytes of one FIFO slot (payload + flags) */
    size_t fifoBytes;          /* ring: bytes of one (channel, rank) FIFO, 8 slots */
    double minBytes;           /* algorithmic minimum HBM bytes read + written */
    double busFactor;          /* busBW = algBW * busFactor (nSteps / nRanks) */
    int vecBytes;              /* bytes per vector access of the one-pass kernels: 0, 16, 32 */
    int bulkCopy;              /* 1: all-gather / gather / broadcast through TMA bulk copies */
    double predictedUs;        /* the planner's cost model for this plan (GB300 fit) */
    size_t tileBytes;          /* copies (load/store path): bytes each CTA moves per tile */
    int tmaStages;             /* bulk-copy fan-out: shared-memory tile stages per CTA */
} vPlanInfo_t;

/* Compute the plan a collective with these parameters would run.  Pure host
 * arithmetic; returns vInvalidArgument for out-of-range requests. */
vResult_t vPlanCompute(const vPlanRequest_t* request, vPlanInfo_t* plan);

/* The element range [*lo, *hi) of block `block` owned by `channel` under `plan`
 * (empty when *lo == *hi).  count is the request's total element count per rank
 * (AR count; nRanks * recvcount for RS).  Host only. */
vResult_t vPlanChannelRange(const vPlanInfo_t* plan, size_t count, int channel, int block,
                            size_t* lo, size_t* hi);

/* Test hook for failure detection: rank `rank` of every later ring transfer never
 * starts (its CTAs return at once), so its neighbours' bounded waits run out and the
 * transfer ends with the sticky error vTimeout.  In vMoeExperts of 16-bit types it is CTA `rank`
 * of both launches that copies nothing to its tensor core.  -1 turns the hook off. */
vResult_t vcommTestSetStallRank(vcomm_t comm, int rank);

/* Test hook for the LL128 line check: in every later LL128 ring transfer rank `rank`
 * expects wrong line flags (as if its predecessor had stored wrong ones; the per-warp
 * release flags it polls stay right), so it finds a line whose flag does not match after
 * the release flag did and ends the transfer with the sticky error vInternalError.  -1
 * turns the hook off. */
vResult_t vcommTestSetBadFlagRank(vcomm_t comm, int rank);

/* Test hook: staged ring transfers sleep for pseudo-random times of up to maxNs
 * nanoseconds (0 = off, at most 1,000,000) where a producer publishes a slot and where a
 * consumer observes one, so that tests exercise orderings of stores and flag reads that
 * rarely occur on their own.  Results must not change. */
vResult_t vcommTestSetJitterNs(vcomm_t comm, unsigned int maxNs);

/* Links of `rank` in tree `tree` (0 or 1) of the double binary tree over nRanks ranks
 * (NCCL book chapter 4, ncclGetBtree / ncclGetDtree): tree 0 hangs from rank 0, a
 * rank's lowest set bit fixes its level; tree 1 mirrors it (rank r -> nRanks-1-r) for an
 * even rank count and shifts it (r -> r+1) for an odd one.  -1 marks a missing link. */
vResult_t vPlanTreeLinks(int nRanks, int rank, int tree, int* parent, int* child0, int* child1);

/* vPlanCompute for this communicator's device and settings.  `aligned` is the largest
 * power-of-two alignment (in bytes, up to 32) shared by every buffer pointer. */
vResult_t vcommQueryPlan(vcomm_t comm, vColl_t coll, size_t count, vDataType_t datatype,
                         int aligned, vPlanInfo_t* plan);

#ifdef __cplusplus
}
#endif
#endif /* VCOMM_H */
