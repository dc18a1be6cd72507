// k_moe_tiles.cu -- the experts' layer for a few tokens on the tensor cores: 16-bit types.
//
// A tile of 128 rows of an expert's weights is the matrix A of the products, the tokens that chose the
// expert (up to NT of them) are B, so the weights are read from memory once and a product has as few
// columns as there are tokens.  Both launches read the weights at the memory's rate; everything else is
// there to keep it busy: a persistent CTA on every SM, or a cluster of CTAs that split a tile's columns
// where there are fewer tiles than SMs, walks over tiles of one (expert, tokens) group after another.
// Eight warps copy the next stages asynchronously, 128 columns each, into the swizzled layout; one
// thread issues the products; four warps take finished sums out of tensor memory, where two tiles' sums
// have room.  Rows that start off 16 bytes come through registers, a stage ahead, as the aligned words that
// hold them.
//
// Measured (bf16): 64 tokens on 8 of 128 experts of 4096 x 1536, 4.8 GB of weights, 757 to 773 us (6.2 TB/s; the
// way up 499), with 4095 x 1535 1735 (2.7); 8 tokens there 338 us (5.7 TB/s), one token 69 (4.4); one token on 4
// of 64 experts of 2048 x 1024 26 us (1.9), a chain of latencies: ids, weights, sums, ids, weights, sums.  The
// second launch gets onto an SM when the first has left it: registers (69 and 115 a thread) hold one CTA.
//
// The way up: the tile's rows are 64 of the gate and the 64 of the linear part that belong to them,
// sixteen and sixteen in turn, so that both sums of an element lie in one warp.  silu(g) u goes into the
// workspace as two values of the weights' type, the second what the first leaves out, for which the way
// down makes two products of every tile: in 16 bits alone the result would be as far off again as its own
// rounding.  In bf16 the two add up to the value, 2^-18 of it off.  fp16 has steps of 2^-24 at the least, so
// there the first is in units of 2 and the second in units of 2^-10, and each has sums of its own, which
// meet in fp32: 2^-22 of the value off, or 2^-35 where it is small; beyond 2 x 65504 it is infinite.  (Both in
// units of 1, one sum: 2^-25 off, more than the result's own rounding for values below 10^-4; the second sums
// cost 1 to 2 %, 96 tokens on 2 of 8 of 2048 x 1024 41.7 us in place of 40.9.)
// The way down: every slot's output goes into the workspace in fp32; for few tokens the last warp of a
// tile of columns adds them up, for more a third launch.
#include "moe.h"
#include "norm_stage.cuh"
#include "tcgen05.cuh"

namespace vc {

namespace {

constexpr int kEpilogueWarps = 4, kProducerWarps = 8;
constexpr int kIssuer = kEpilogueWarps;                // the warp that issues products
constexpr int kThreads = 32 * (kEpilogueWarps + 1 + kProducerWarps);
constexpr int kProducers = 32 * kProducerWarps;
constexpr int kM = 128;              // rows of a tile
constexpr int kK = 128;              // columns of a stage: two swizzled halves of 64
constexpr int kHalfA = kM * 128;     // bytes of a half of A
constexpr float kLargest = 0x1.FEp127f;                // of bf16
// fp16: what the two values of silu(g) u are in units of
constexpr float kFirstUnit = 2.0f, kSecondUnit = 0x1p-10f;
// Sums of a tile that the way down keeps apart, and columns of tensor memory, two tiles' (32 at least).
template <int DT, bool UP> constexpr int kSums = DT == kF16 && !UP ? 2 : 1;
template <int DT, int NT, bool UP> constexpr int kColumns = 2 * NT * kSums<DT, UP>;
static_assert(kProducers == 16 * 16, "a producer: one 16-byte chunk of a stage's row, sixteen rows apart");

struct Shared {
    uint64_t full[kMoeMaxStages], empty[kMoeMaxStages];
    uint64_t sumsFull[2], sumsEmpty[2];
    uint64_t partFull, partEmpty, drained;
    uint32_t tmem;
    int failed, nGroups;
    int warpSum[32];
};
// In dynamic shared memory, as long as the call needs them.
struct Lists {
    int* first;                      // of an expert's slots
    uint16_t* slots;                 // by expert
    MoeGroup* groups;
};

// The slots sorted by expert, and the groups.  All threads; `scratch` holds two bytes a warp and expert.
template <int NT>
__device__ __forceinline__ void make_lists(Shared& sh, const Lists& l, uint16_t* scratch, const ExpertsArgs& a) {
    const int total = a.rows * a.topK, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (total <= 32 && NT >= 16) {   // by one warp, experts in the order of their first slots
        if (warp == 0) {
            const int e = lane < total ? a.ids[lane] : -1;
            const bool counts = e >= 0 && e < a.experts;
            const unsigned same = __match_any_sync(~0u, counts ? e : -1), below = (1u << lane) - 1;
            const bool leads = counts && (same & below) == 0;
            const int n = __popc(same), mine = leads ? n | (n + NT - 1) / NT << 16 : 0;    // slots and groups
            int run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, run, o);
                if (lane >= o) run += v;
            }
            const int first = __shfl_sync(~0u, run - mine, __ffs(same) - 1) & 0xFFFF;
            if (counts) l.slots[first + __popc(same & below)] = (uint16_t)lane;
            if (leads)
                for (int j = 0; j < n; j += NT)
                    l.groups[((run - mine) >> 16) + j / NT] = MoeGroup{(uint16_t)e, (uint16_t)(first + j), (uint16_t)min(NT, n - j)};
            if (lane == 31) sh.nGroups = run >> 16;
        }
        __syncthreads();
        return;
    }
    // A stable sort by expert, every warp a run of the slots: how many of each expert it has, where they go,
    // and there they go, so that all CTAs agree on which slots a group has.
    constexpr int kWarps = kThreads / 32;
    for (int i = threadIdx.x; i < (kWarps * a.experts + 1) / 2; i += kThreads) reinterpret_cast<uint32_t*>(scratch)[i] = 0u;
    __syncthreads();
    uint16_t* const own = scratch + warp * a.experts;
    const int each = (total + 32 * kWarps - 1) / (32 * kWarps) * 32, from = warp * each, to = min(total, from + each);
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane, e = i < to ? a.ids[i] : -1;
        const bool counts = e >= 0 && e < a.experts;
        const unsigned same = __match_any_sync(~0u, counts ? e : -1);
        if (counts && lane == 31 - __clz((int)same)) own[e] += (uint16_t)__popc(same);
        __syncwarp();
    }
    __syncthreads();
    // running sums of slots and of groups, three experts a thread
    constexpr int PER = (VCOMM_MAX_EXPERTS + kThreads - 1) / kThreads;
    int n[PER], slots = 0, groups = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = (int)threadIdx.x * PER + i;
        n[i] = 0;
        if (e >= a.experts) break;
        for (int w = 0; w < kWarps; w++) {             // what a warp has, then what the warps before have
            const int m = scratch[w * a.experts + e];
            scratch[w * a.experts + e] = (uint16_t)n[i];
            n[i] += m;
        }
        slots += n[i];
        groups += (n[i] + NT - 1) / NT;
    }
    int run = slots | groups << 16;                    // neither above 2^15
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += v;
    }
    if (lane == 31) sh.warpSum[warp] = run;
    __syncthreads();
    int ahead = run - (slots | groups << 16), all = 0;
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) ahead += sh.warpSum[w];
        all += sh.warpSum[w];
    }
    int slot = ahead & 0xFFFF, group = ahead >> 16;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = (int)threadIdx.x * PER + i;
        if (e >= a.experts) break;
        for (int j = 0; j < n[i]; j += NT)
            l.groups[group++] = MoeGroup{(uint16_t)e, (uint16_t)(slot + j), (uint16_t)min(NT, n[i] - j)};
        l.first[e] = slot;
        slot += n[i];
    }
    if (threadIdx.x == 0) sh.nGroups = all >> 16;
    __syncthreads();
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane, e = i < to ? a.ids[i] : -1;
        const bool counts = e >= 0 && e < a.experts;
        const unsigned same = __match_any_sync(~0u, counts ? e : -1);
        const int at = counts ? own[e] : 0;
        __syncwarp();
        if (counts) {
            l.slots[l.first[e] + at + __popc(same & ((1u << lane) - 1))] = (uint16_t)i;
            if (lane == 31 - __clz((int)same)) own[e] = (uint16_t)(at + __popc(same));
        }
        __syncwarp();
    }
    __syncthreads();
}

__device__ __forceinline__ void copy_chunk(uint32_t to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}
// Eight elements that start anywhere, `left` of them inside their row (the rest zeros): the aligned words that
// hold some of them, and what they make.
__device__ __forceinline__ void load_words(const uint16_t* from, int left, uint32_t (&r)[5]) {
    const uintptr_t p = (uintptr_t)from;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p & ~(uintptr_t)3);
    const int ahead = (int)(p >> 1) & 1;               // elements of the first word before them
#pragma unroll
    for (int i = 0; i < 5; i++) {
        r[i] = 0u;
        if (2 * i - ahead < min(left, 8)) r[i] = w[i];
    }
}
__device__ __forceinline__ uint4 from_words(const uint16_t* from, int left, const uint32_t (&r)[5]) {
    const uint32_t shift = ((uint32_t)(uintptr_t)from & 2u) * 8u;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i] = __funnelshift_r(r[i], r[i + 1], shift);
        if (2 * i + 1 >= left) v[i] = 2 * i >= left ? 0u : v[i] & 0xFFFFu;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Columns [h, h + 4) of every rank's output for token t, from its slots' y.  What up to eight slots need is
// loaded together, whether it counts or not: the wait for memory is most of this.
template <int DT>
__device__ __forceinline__ void combine(const ExpertsArgs& a, int t, int h) {
    constexpr int ESZ = DTypeOf<DT>::size, UN = 8;
    static_assert(ESZ == 2, "the tensor cores' types");
    const auto put = [&](int r, const float (&s)[4]) {
        uint16_t* to = (uint16_t*)a.recv[r] + (size_t)t * a.recvStride + h;
        if (a.recvAligned && h + 4 <= a.hidden) {
            *reinterpret_cast<uint2*>(to) = make_uint2(narrow16<DT>(s[0]) | (uint32_t)narrow16<DT>(s[1]) << 16,
                                                       narrow16<DT>(s[2]) | (uint32_t)narrow16<DT>(s[3]) << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (h + j < a.hidden) to[j] = narrow16<DT>(s[j]);
        }
    };
    const auto add = [&](int k, float4& y, float& w, int& r) {
        const size_t slot = (size_t)t * a.topK + min(k, a.topK - 1);
        const int e = a.ids[slot];
        w = a.weights[slot];
        y = __ldcg(reinterpret_cast<const float4*>(a.y + slot * moe_y_stride(a.hidden) + h));
        r = k < a.topK && e >= 0 && e < a.experts ? e / a.share : -1;
    };
    if (a.topK <= UN) {
        float4 y[UN];
        float w[UN];
        int rank[UN];
#pragma unroll
        for (int k = 0; k < UN; k++) add(k, y[k], w[k], rank[k]);
        for (int r = 0; r < a.nRanks; r++) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < UN; k++) {
                if (rank[k] != r) continue;
                s[0] = fmaf(w[k], y[k].x, s[0]);
                s[1] = fmaf(w[k], y[k].y, s[1]);
                s[2] = fmaf(w[k], y[k].z, s[2]);
                s[3] = fmaf(w[k], y[k].w, s[3]);
            }
            put(r, s);
        }
        return;
    }
    for (int r = 0; r < a.nRanks; r++) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < a.topK; k++) {
            float4 y;
            float w;
            int rank;
            add(k, y, w, rank);
            if (rank != r) continue;
            s[0] = fmaf(w, y.x, s[0]);
            s[1] = fmaf(w, y.y, s[1]);
            s[2] = fmaf(w, y.z, s[2]);
            s[3] = fmaf(w, y.w, s[3]);
        }
        put(r, s);
    }
}

// UP: the way up, K = hidden, tiles of 64 of the ffn elements; else the way down, K = ffn, tiles of 128
// columns of the output.
template <int DT, int NT, bool UP, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1) k_moe_tiles(const __grid_constant__ ExpertsArgs a) {
    constexpr int COPIES = UP ? 1 : 2;                 // of B: the tokens, or both values of silu(g) u
    constexpr int kHalfB = NT * 128;
    constexpr int SUMS = kSums<DT, UP>, COLUMNS = kColumns<DT, NT, UP>;
    static_assert(COLUMNS >= 32 && (COLUMNS & (COLUMNS - 1)) == 0 && COLUMNS <= 256, "tensor memory comes in powers of two from 32 on");
    constexpr int kStage = 2 * kHalfA + 2 * COPIES * kHalfB;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    const uint32_t stages = (smem_at(raw) + 1023u) & ~1023u;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int split = a.split, rank = split > 1 ? (int)cluster_rank() : 0;
    const int nStages = a.stages;
    float* const parts = reinterpret_cast<float*>(raw + (stages - smem_at(raw)) + nStages * kStage);   // [split - 1][NT][128]
    Lists l;
    l.first = reinterpret_cast<int*>(parts + (split - 1) * NT * kM);
    l.groups = reinterpret_cast<MoeGroup*>(l.first + a.experts);
    l.slots = reinterpret_cast<uint16_t*>(l.groups + moe_groups(a.experts, a.rows * a.topK, NT));
    // The way up waits for what the calls before wrote, ids and tokens among it, before it lets the way
    // down start; so that one may read ids and weights at once, and what the way up writes after its wait.
    if (UP) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        const int tiles = (a.hidden + kM - 1) / kM;
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < tiles; i += kThreads) a.done[i] = 0;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < nStages; i++) {
            bar_init(&sh.full[i], ALIGNED || UP ? kProducers : 2 * kProducers);
            bar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(&sh.sumsFull[i], 1);
            bar_init(&sh.sumsEmpty[i], kEpilogueWarps);
        }
        bar_init(&sh.partFull, (split - 1) * kEpilogueWarps * 32 + (split == 1));
        bar_init(&sh.partEmpty, kEpilogueWarps);
        bar_init(&sh.drained, 1);
        sh.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) tmem_alloc(&sh.tmem, COLUMNS);
    make_lists<NT>(sh, l, reinterpret_cast<uint16_t*>(raw + (stages - smem_at(raw))), a);    // (no stage is in use yet)
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (split > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const uint32_t tmem = sh.tmem;
    const int K = UP ? a.hidden : a.ffn;
    const int tiles = UP ? (a.ffn + kM / 2 - 1) / (kM / 2) : (a.hidden + kM - 1) / kM;
    const int units = sh.nGroups * tiles;
    const int first = (int)blockIdx.x / split, step = (int)gridDim.x / split;
    const int chunks = (K + kK - 1) / kK, chunk0 = rank * chunks / split, chunk1 = (rank + 1) * chunks / split;

    if (warp > kIssuer) {
        // ---- producers: chunk `c` of rows r0, r0 + 16, ... of a stage
        const int t = (int)threadIdx.x - 32 * (kIssuer + 1), c = t & 15, r0 = t >> 4;
        const uint32_t column = (uint32_t)(c >> 3), swizzled = (uint32_t)(((c & 7) ^ (r0 & 7)) << 4);
        const auto weights = [&](const MoeGroup& g) {
            const size_t e = (size_t)(g.expert % a.share);
            return UP ? (const uint16_t*)a.up[g.expert / a.share] + e * 2 * a.ffn * K
                      : (const uint16_t*)a.down[g.expert / a.share] + e * a.hidden * K;
        };
        // Row 16 i + r0 of a tile; on the way up sixteen of the gate, sixteen of the linear part.
        const auto row = [&](int m, int i) { return UP ? m * (kM / 2) + (i >> 1) * 16 + r0 : m * kM + 16 * i + r0; };
        const auto first_of = [&](int n, int i) { return ((size_t)(UP && (i & 1) ? a.ffn : 0) + n) * K; };
        const int rows = UP ? a.ffn : a.hidden;
        const auto at_a = [&](int at) { return stages + (uint32_t)(at * kStage) + column * kHalfA + (uint32_t)r0 * 128 + swizzled; };
        const auto at_b = [&](int at) {
            return stages + (uint32_t)(at * kStage) + 2 * kHalfA + column * kHalfB + (uint32_t)r0 * 128 + swizzled;
        };
        const auto token = [&](const MoeGroup& g, int r) {
            return (const uint16_t*)a.x + (size_t)(l.slots[g.first + r] / a.topK) * a.rowStride;
        };
        // One stage's A, or B, asynchronously.
        const auto copy_a = [&](int u, int chunk, int at) {
            const MoeGroup g = l.groups[u / tiles];
            const int m = u % tiles, k = chunk * kK + c * 8;
            const uint32_t to = at_a(at);
            const uint16_t* w = weights(g) + k;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int n = row(m, i);
                const bool in = n < rows && k < K;
                copy_chunk(to + i * 16 * 128, in ? w + first_of(n, i) : w - k, in);
            }
        };
        const auto copy_b = [&](int u, int chunk, int at) {
            const MoeGroup g = l.groups[u / tiles];
            const int k = chunk * kK + c * 8, width = UP ? K : moe_act_stride(K);
            const uint32_t to = at_b(at);
            for (int r = r0; r < g.count; r += 16) {
                const bool in = k < width;
                if (UP) {
                    const uint16_t* x = token(g, r);
                    copy_chunk(to + (r - r0) * 128, in ? x + k : x, in);
                } else {
                    const uint16_t* x = (const uint16_t*)a.act + (size_t)l.slots[g.first + r] * 2 * width;
                    copy_chunk(to + (r - r0) * 128, in ? x + k : x, in);
                    copy_chunk(to + (r - r0) * 128 + 2 * kHalfB, in ? x + width + k : x, in);
                }
            }
        };
        // The same of rows that start anywhere: through registers, which hold one stage's ahead (two
        // stages': 1904 us against 1741 for 64 tokens on 8 of 128 experts of 4095 x 1535).
        struct Words {
            uint32_t a[ALIGNED ? 1 : 8][5], b[ALIGNED || !UP ? 1 : NT / 16][5];
        };
        const auto load_a = [&](int u, int chunk, Words& words) {
            if (ALIGNED || u >= units) return;
            const MoeGroup g = l.groups[u / tiles];
            const int m = u % tiles, k = chunk * kK + c * 8;
            const uint16_t* w = weights(g);
#pragma unroll
            for (int i = 0; i < (ALIGNED ? 1 : 8); i++) {
                const int n = row(m, i);
                const bool in = n < rows && k < K;
                load_words(in ? w + first_of(n, i) + k : w, in ? K - k : 0, words.a[i]);
            }
            if constexpr (UP && !ALIGNED) {
#pragma unroll
                for (int i = 0; i < NT / 16; i++) {
                    const int r = r0 + 16 * i;
                    const bool in = r < g.count && k < K;
                    load_words(in ? token(g, r) + k : w, in ? K - k : 0, words.b[i]);
                }
            }
        };
        const auto store_a = [&](int u, int chunk, int at, const Words& words) {
            const MoeGroup g = l.groups[u / tiles];
            const int m = u % tiles, k = chunk * kK + c * 8;
            const uint16_t* w = weights(g);
#pragma unroll
            for (int i = 0; i < (ALIGNED ? 1 : 8); i++)
                st_smem(at_a(at) + i * 16 * 128, from_words(w + first_of(row(m, i), i) + k, K - k, words.a[i]));
            if constexpr (UP && !ALIGNED) {
#pragma unroll
                for (int i = 0; i < NT / 16; i++) {
                    const int r = r0 + 16 * i;
                    if (r < g.count) st_smem(at_b(at) + i * 16 * 128, from_words(token(g, r) + k, K - k, words.b[i]));
                }
            }
        };
        const auto next = [&](int& u, int& chunk) {
            if (++chunk == chunk1) {
                chunk = chunk0;
                u += step;
            }
        };
        // The way down: the weights of the first stages need not wait for the way up.
        Words words;
        int early = 0, aheadU = first, aheadChunk = chunk0;            // of A: what is loaded next
        if (!UP) {
            for (; aheadU < units && early < nStages; early++) {
                if (ALIGNED) {
                    copy_a(aheadU, aheadChunk, early);
                } else {
                    load_a(aheadU, aheadChunk, words);
                    store_a(aheadU, aheadChunk, early, words);
                }
                next(aheadU, aheadChunk);
            }
        }
        load_a(aheadU, aheadChunk, words);
        if (!UP) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        }
        int at = 0, u = first, chunk = chunk0;
        uint32_t round = 0;                            // times that all stages have been filled
        // The next stage; false at the end.
        const auto fill = [&](bool early) {
            if (round > 0 && !__all_sync(~0u, bar_wait(&sh.empty[at], (round - 1) & 1u, &sh.failed, a.timeoutNs))) return false;
            if (ALIGNED && !early) copy_a(u, chunk, at);
            if (!ALIGNED) {
                if (!early) store_a(u, chunk, at, words);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&sh.full[at]);
            }
            if (ALIGNED || !UP) {
                copy_b(u, chunk, at);
                // arrives when this thread's copies are there; the issuer makes them visible to its products (a
                // fence here would wait for the stages under way: 816 us for the way up of 64 x 4096 x 1536, 499)
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_at(&sh.full[at])) : "memory");
            }
            if (!ALIGNED && !early) {
                next(aheadU, aheadChunk);
                load_a(aheadU, aheadChunk, words);
            }
            if (++at == nStages) {
                at = 0;
                round++;
            }
            next(u, chunk);
            return u < units;
        };
        bool more = u < units && (int)blockIdx.x != a.stallCta;
        for (; more && early > 0; early--) more = fill(true);
        while (more) more = fill(false);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kIssuer) {
        // ---- the issuer
        if (lane == 0) {
            // (no copy of B is under way before that: the limited waits below begin with it)
            if (!UP) asm volatile("griddepcontrol.wait;" ::: "memory");
            int at = 0, unit = 0;
            uint32_t round = 0;
            bool ok = true;
            for (int u = first; u < units && ok; u += step, unit++) {
                const int n = (l.groups[u / tiles].count + 15) & ~15, buffer = unit & 1;
                const uint32_t shape = product_shape<DT>(n), d = tmem + (uint32_t)(buffer * NT * SUMS);
                if (unit >= 2 && !(ok = bar_wait(&sh.sumsEmpty[buffer], (uint32_t)(unit / 2 - 1) & 1u, &sh.failed, a.timeoutNs))) break;
                tmem_fence_after();
                for (int chunk = chunk0; chunk < chunk1; chunk++) {
                    if (!(ok = bar_wait(&sh.full[at], round & 1u, &sh.failed, a.timeoutNs))) break;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tmem_fence_after();
                    const uint32_t sa = stages + (uint32_t)(at * kStage), sb = sa + 2 * kHalfA;
#pragma unroll
                    for (int i = 0; i < kK / 16; i++) {
                        const uint64_t opA = operand(sa + (i >> 2) * kHalfA + (i & 3) * 32);
#pragma unroll
                        for (int v = 0; v < COPIES; v++)
                            multiply(d + (SUMS > 1 ? v * NT : 0), opA, operand(sb + v * 2 * kHalfB + (i >> 2) * kHalfB + (i & 3) * 32),
                                     shape, chunk > chunk0 || i > 0 || (SUMS == 1 && v > 0));
                    }
                    products_done(&sh.empty[at]);
                    if (++at == nStages) {
                        at = 0;
                        round++;
                    }
                }
                if (ok) products_done(&sh.sumsFull[buffer]);
            }
            // nothing of this CTA's is under way when its tensor memory is given back
            products_done(&sh.drained);
            bar_drain(&sh.drained, 0, &sh.failed, a.timeoutNs);
        }
        __syncwarp();
    } else {
        // ---- sums out of tensor memory: lane `lane` of warp `warp` has row 32 warp + lane
        if (!UP) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int row = warp * 32 + lane;
        int unit = 0;
        for (int u = first; u < units; u += step, unit++) {
            const MoeGroup g = l.groups[u / tiles];
            const int m = u % tiles, buffer = unit & 1;
            bool ok = bar_wait(&sh.sumsFull[buffer], (uint32_t)(unit / 2) & 1u, &sh.failed, a.timeoutNs);
            if (rank > 0 && unit > 0) ok = ok && bar_wait(&sh.partEmpty, (uint32_t)(unit - 1) & 1u, &sh.failed, a.timeoutNs);
            if (split > 1 && rank == 0) ok = ok && bar_wait(&sh.partFull, (uint32_t)unit & 1u, &sh.failed, a.timeoutNs);
            if (!__all_sync(~0u, ok)) break;
            tmem_fence_after();
            for (int j0 = 0; j0 < g.count; j0 += 16) {
                float v[16];
                const uint32_t sums = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(buffer * NT * SUMS + j0);
                tmem_load(sums, v);
                if constexpr (SUMS > 1) {
                    float second[16];
                    tmem_load(sums + NT, second);
#pragma unroll
                    for (int j = 0; j < 16; j++) v[j] = fmaf(second[j], kSecondUnit, v[j] * kFirstUnit);
                }
                if (rank > 0) {      // to the first CTA of the cluster
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        st_cluster(parts + ((size_t)(rank - 1) * NT + j0 + j) * kM + row, 0, __float_as_uint(v[j]));
                    continue;
                }
                for (int s = 0; s < split - 1; s++)
#pragma unroll
                    for (int j = 0; j < 16; j++) v[j] += parts[((size_t)s * NT + j0 + j) * kM + row];
                if (UP) {
                    // lanes 0 to 15 hold the gate's sums, 16 to 31 the linear part's: the first take the
                    // even columns, the others the odd ones
                    const int f = m * (kM / 2) + warp * 16 + (lane & 15);
                    uint16_t* const act = (uint16_t*)a.act;
                    const int width = moe_act_stride(a.ffn);           // zeros from ffn on
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float other = __shfl_xor_sync(~0u, lane < 16 ? v[j + 1] : v[j], 16);
                        const float gate = lane < 16 ? v[j] : other, linear = lane < 16 ? other : v[j + 1];
                        const int column = j0 + j + (lane >> 4);
                        if (column >= g.count || f >= width) continue;
                        const float x = f < a.ffn ? gate / (1.0f + expf(-gate)) * linear : 0.0f;
                        uint16_t* to = act + (size_t)l.slots[g.first + column] * 2 * width + f;
                        if constexpr (DT == kF16) {    // (infinities and NaNs go into the first value)
                            const uint16_t first = narrow16<DT>(x * (1.0f / kFirstUnit));
                            const float near = widen16<DT>(first) * kFirstUnit;
                            to[0] = first;
                            to[width] = isfinite(near) ? narrow16<DT>((x - near) * (1.0f / kSecondUnit)) : (uint16_t)0;
                        } else {                       // (into the second)
                            const uint16_t first = narrow16<DT>(fminf(fmaxf(x, -kLargest), kLargest));
                            to[0] = first;
                            to[width] = narrow16<DT>(x - widen16<DT>(first));
                        }
                    }
                } else {
                    const int h = m * kM + row;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (j0 + j < g.count && h < a.hidden) a.y[(size_t)l.slots[g.first + j0 + j] * moe_y_stride(a.hidden) + h] = v[j];
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&sh.sumsEmpty[buffer]);
            if (rank > 0) bar_arrive_at(&sh.partFull, 0);
            if (split > 1 && rank == 0) {
                __syncwarp();
                if (lane > 0 && lane < split) bar_arrive_at(&sh.partEmpty, lane);
            }
            if (UP || rank > 0 || !a.combineHere) continue;
            // the last warp of the last group adds up the tile's columns
            __threadfence();
            __syncwarp();
            unsigned before = 0;
            if (lane == 0) before = atomicAdd(&a.done[m], 1u);
            if (__shfl_sync(~0u, before, 0) != (unsigned)(kEpilogueWarps * sh.nGroups) - 1) continue;
            __threadfence();
            if (m * kM + 4 * lane < a.hidden)
                for (int t = 0; t < a.rows; t++) combine<DT>(a, t, m * kM + 4 * lane);
        }
        // no expert at all: zeros
        if (!UP && a.combineHere && sh.nGroups == 0)
            for (int h = ((int)blockIdx.x * kM + row) * 4; h < a.hidden; h += (int)gridDim.x * kM * 4)
                for (int t = 0; t < a.rows; t++) combine<DT>(a, t, h);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kIssuer) tmem_free(tmem, COLUMNS);
    if (threadIdx.x == 0 && sh.failed) report_error(a.status, a.statusHost, vTimeout, blockIdx.x, 0, UP ? 0 : 1);
    if (split > 1) {                                   // another CTA may still arrive here
        cluster_arrive();
        cluster_wait();
    }
}

// Every token's slots added up, for many tokens: a thread four columns of a token.
constexpr int kCombineThreads = 128;
template <int DT>
__global__ void __launch_bounds__(kCombineThreads) k_moe_combine(const __grid_constant__ ExpertsArgs a) {
    pdl_begin();
    const int h = 4 * ((int)blockIdx.x * kCombineThreads + (int)threadIdx.x);
    if (h < a.hidden) combine<DT>(a, (int)blockIdx.y, h);
}

template <int DT, int NT, bool UP>
cudaError_t tiles_launch(const ExpertsArgs& a, const MoeTiles& t, cudaStream_t s) {
    const auto kernel = a.aligned ? k_moe_tiles<DT, NT, UP, true> : k_moe_tiles<DT, NT, UP, false>;
    // one value for every launch, as host threads share the kernel's limit
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeMaxSmem);
    if (e != cudaSuccess) return e;
    ExpertsArgs b = a;
    b.split = UP ? t.splitUp : t.splitDown;
    b.stages = UP ? t.stagesUp : t.stagesDown;
    b.combineHere = t.combineHere;
    // A wait for a tile's sums lasts as long as its stages take, under a microsecond each where the memory is not
    // shared with other work: 20 for each are no lack of progress.
    b.timeoutNs += 20000ull * (unsigned)(((UP ? a.hidden : a.ffn) + kK - 1) / kK);
    NormShape sh = {};
    sh.threads = kThreads;
    sh.cluster = b.split;
    return norm_launch(kernel, (unsigned)(UP ? t.gridUp : t.gridDown), sh,
                       (size_t)moe_tiles_smem(a.experts, a.rows * a.topK, NT, UP, b.split, b.stages), s, b);
}
template <int DT, int NT>
cudaError_t tiles_both(const ExpertsArgs& a, const MoeTiles& t, cudaStream_t s) {
    const cudaError_t e = tiles_launch<DT, NT, true>(a, t, s);
    return e != cudaSuccess ? e : tiles_launch<DT, NT, false>(a, t, s);
}
template <int DT>
cudaError_t tiles_dt(const ExpertsArgs& a, const MoeTiles& t, cudaStream_t s) {
    const cudaError_t e = t.tokens == 16   ? tiles_both<DT, 16>(a, t, s)
                          : t.tokens == 32 ? tiles_both<DT, 32>(a, t, s)
                                           : tiles_both<DT, 64>(a, t, s);
    if (e != cudaSuccess || t.combineHere) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.hidden + 4 * kCombineThreads - 1) / (4 * kCombineThreads)), (unsigned)a.rows);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_moe_combine<DT>, a);
}

}  // namespace

cudaError_t launch_moe_tiles(const ExpertsArgs& a, const MoeTiles& t, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat16: return tiles_dt<kF16>(a, t, s);
    case vBFloat16: return tiles_dt<kBF16>(a, t, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
