// k_sample.cu -- one token for every row of logits whose columns are split over the ranks.
//
//   z_i = logit_i / temperature,  e_i = exp(z_i - max z)
//   kept: the topK largest; of those the shortest run of largest whose sum reaches topP of theirs; of
//   those the ones with e_i >= minP.  Ties go to the lower index.
//   token = the first kept i, in the vocabulary's order, with (sum of kept e up to i) > u (sum of kept e)
//   logprob = z_token - max z - log(sum of all e)
//
// All filters keep a run of the largest logits, so what is kept is known by one value and how many of
// its equals are kept.  That value is found by counting, not by sorting: logits map to integers in
// their order, and a histogram of their distances from the largest, 2048 bins at a time, is refined
// until a bin is one value.  Bounds that cost nothing keep most logits out of the histograms: the
// topK-th largest is at least the smallest of topK disjoint groups' maxima, and weights below a share
// of the sum that all of them together could not fill lie outside topP.  Where few logits are left, they
// are held in registers and the value is found by halving its range, or, of at most 256, every one's
// place and what is kept before it by comparing it with all others.
//
// The draw is a comparison of sums, so these are exact: a weight is a 64-bit integer, 2^44 e, right to
// 2^-28.8 of itself (sample_weight.cuh), and the order of additions does not matter.  Where a filter is given,
// logprob's sum is one of fp32 exponentials, 2^-17 of itself off at most: a draw without filters, which sums
// exact weights, takes 126 us for 256 rows of 131072, one of topK 50 87.
//
// A row is read once, into the shared memory of a cluster's CTAs, which exchange maxima and sums there.
// What is above the bounds, where it is few, goes to the first of them, which decides alone, without the
// cluster's barriers (more than a microsecond each); else all decide together.
//
// A row's part on a rank is read by whole 16-byte blocks, wherever it starts; what a block holds besides
// counts as minus infinity.
//
// Instructions and the latencies between a row's reductions bound it, not memory (256 rows of 131072 bf16
// are read in 10 us): those take 68 us where the largest is taken, 88 with topK 50 and topP, 112 with topK
// 200, 126 without filters (a weight of every logit), 146 with topP 0.9 at temperature 0.6, where the
// nucleus fits the list, and 354 at 1.2, where it holds most of the row and the histograms decide; rows of all
// kinds 173.  One row takes 12 to 24 us on eight CTAs, 41 with topK 2000 and topP, and 50 with such a nucleus.  A
// CTA that streams its row from memory several times, a row a CTA, was slower (403 us for rows of all kinds).  Two
// CTAs an SM leave 64 registers a thread: 112 bytes of 16-bit types are spilled, 4 of fp32.
#include "norm_stage.cuh"
#include "sample.h"
#include "sample_weight.cuh"

namespace vc {

namespace {

constexpr int kWarps = kSampleThreads / 32;
constexpr int kWords = 4;            // that the CTAs of a cluster exchange at a time

constexpr int kSampleFew = 256;      // values that are compared with one another
struct alignas(16) FewValue {
    uint32_t d;                      // distance from the top
    int at;                          // place in the list
    u64 v;                           // weight
};
struct Shared {
    FewValue few[kSampleFew];
    int place[3][kSampleFew];
    u64 before[3][kSampleFew];
    uint32_t powers[32];
    float max[kWarps], low[kWarps];  // the largest value, and the smallest maximum of groups of lanes
    // the row's parts: the first block, the elements before the part in it, their number, and the blocks
    // of the parts before
    const uint4* part[VCOMM_MAX_RANKS];
    int shift[VCOMM_MAX_RANKS], length[VCOMM_MAX_RANKS], blocks[VCOMM_MAX_RANKS + 1];
    u64 warp[2][kWarps];
    u64 box[2][kSampleCluster][kWords];      // one line a CTA, written by all CTAs of the cluster
    u64 found[2][3];                 // bin, what lies before it, what lies in it
    int count[2][kWarps];
    unsigned mass[2][3][kWarps];
    u64 total;
    int settled;
};

// What the exchanges between the CTAs of a cluster need.
struct Team {
    int rank, size, flip, flipFound;
};
__device__ __forceinline__ void meet(const Team& team) {
    if (team.size > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}
__device__ __forceinline__ uint32_t ld_cluster(const void* local, unsigned rank) {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(local);
    uint32_t r, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
    return v;
}
// Every CTA's four words in box[.][its rank] of every CTA.  Called by all threads; `mine` is the same
// in all.  Two boxes in turn: a CTA writes one again only when all have met since it was read.
__device__ __forceinline__ const u64 (*exchange(Shared& sh, Team& team, const u64 (&mine)[kWords]))[kWords] {
    u64(*box)[kWords] = sh.box[team.flip];
    team.flip ^= 1;
    if (team.size == 1) {
        __syncthreads();
        if (threadIdx.x < 4) box[0][threadIdx.x] = mine[threadIdx.x];
        __syncthreads();
        return box;
    }
    if (threadIdx.x < 8u * (unsigned)team.size) {
        const int word = (int)threadIdx.x & 7;
        const u64 v = word < 2 ? mine[0] : word < 4 ? mine[1] : word < 6 ? mine[2] : mine[3];
        st_cluster((const char*)box[team.rank] + 4 * word, threadIdx.x >> 3, (uint32_t)(word & 1 ? v >> 32 : v));
    }
    meet(team);
    return box;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
// The CTA's sums of two values, in every thread.
__device__ __forceinline__ void block_sums(Shared& sh, u64& a, u64& b) {
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sh.warp[0][threadIdx.x >> 5] = a;
        sh.warp[1][threadIdx.x >> 5] = b;
    }
    __syncthreads();
    a = b = 0;
    for (int w = 0; w < kWarps; w++) {
        a += sh.warp[0][w];
        b += sh.warp[1][w];
    }
}

// Integers in the order of the values: of 16-bit types the bits that they have.
template <int DT> constexpr int kKeyShift = DT == kBF16 ? 16 : DT == kF16 ? 13 : 0;
template <int DT>
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);      // -0 is 0
    return (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) >> kKeyShift<DT>;
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t key) {
    const uint32_t o = key << kKeyShift<DT>;
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~(o | ((1u << kKeyShift<DT>) - 1)));
}

// e of a value: as an integer, and roughly.
struct Weights : FixedWeights {
    // The sum of E values' e, none of them the top's: 2^-20 off or so, and 0 below 2^-126.
    template <int E>
    __device__ __forceinline__ float rough(const float (&f)[E]) const {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 z = mul2(add2(make_float2(f[j], f[j + 1]), make_float2(-top, -top)), make_float2(ch, ch));
            float2 e;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
            sum = add2(sum, e);
        }
        return sum.x + sum.y;
    }
    __device__ __forceinline__ u64 fixed(float x) const {
        u64 a, b;
        fixed2(x, x, a, b);
        return a;
    }
    template <int E>
    __device__ __forceinline__ void fixed(const float (&f)[E], u64 (&v)[E]) const {
#pragma unroll
        for (int j = 0; j < E; j += 2) fixed2(f[j], f[j + 1], v[j], v[j + 1]);
    }
};

// 16-byte vectors of values.
template <int DT>
struct Vec {
    static constexpr int E = kVecElems<DT>;
    static constexpr int T = DT == kF32 ? kBF16 : DT;  // for what is only called with 16-bit types
    static __device__ __forceinline__ uint4 none() {
        const uint32_t w = DT == kF32 ? 0xFF800000u : DT == kBF16 ? 0xFF80FF80u : 0xFC00FC00u;
        return make_uint4(w, w, w, w);
    }
    // The largest value, by pairs in the 16-bit types.
    static __device__ __forceinline__ float largest(const uint4& v) {
        if (DT == kF32)
            return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(widen16<T>((uint16_t)m), widen16<T>((uint16_t)(m >> 16)));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        if (DT == kBF16) {
            const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
            return *reinterpret_cast<const uint32_t*>(&r);
        }
        const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    // Whether there may be a NaN: the sums are one then (infinities of both signs give one too).
    static __device__ __forceinline__ bool suspect(const uint4& v) {
        if (DT == kF32) {
            const float t = (__uint_as_float(v.x) + __uint_as_float(v.y)) + (__uint_as_float(v.z) + __uint_as_float(v.w));
            return t != t;
        }
        const uint32_t t = op_word<T, kSum>(op_word<T, kSum>(v.x, v.y), op_word<T, kSum>(v.z, v.w));
        const float a = widen16<T>((uint16_t)t), b = widen16<T>((uint16_t)(t >> 16));
        return a != a || b != b;
    }
    // Values before `from` and from `to` on, and NaNs, become minus infinity.
    static __device__ __noinline__ uint4 only(const uint4& v, int from, int to) {
        float f[E];
        widen_vec<DT>(v, f);
#pragma unroll
        for (int j = 0; j < E; j++) f[j] = j >= from && j < to && f[j] == f[j] ? f[j] : -INFINITY;
        return narrow_vec<DT>(f);
    }
};

// The parts of a row.  All threads.
template <int DT>
__device__ __forceinline__ void find_parts(const SampleArgs& a, Shared& sh, int row) {
    constexpr int E = kVecElems<DT>, ESZ = DTypeOf<DT>::size;
    if (threadIdx.x < 32) {
        int ahead = 0;
        for (int r0 = 0; r0 < a.nParts; r0 += 32) {
            const int r = r0 + (int)threadIdx.x;
            int n = 0;
            if (r < a.nParts) {
                const uintptr_t p = (uintptr_t)a.logits[r] + (size_t)row * a.stride * ESZ;
                const int shift = (int)(p & 15u) / ESZ, length = min(a.part, a.vocab - r * a.part);
                sh.part[r] = reinterpret_cast<const uint4*>(p & ~(uintptr_t)15);
                sh.shift[r] = shift;
                sh.length[r] = length;
                n = (shift + length + E - 1) / E;
            }
            int run = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, run, o);
                if ((int)threadIdx.x >= o) run += v;
            }
            if (r < a.nParts) sh.blocks[r + 1] = ahead + run;
            ahead += __shfl_sync(~0u, run, 31);
        }
        if (threadIdx.x == 0) sh.blocks[0] = 0;
    }
    __syncthreads();
}
// The part that holds a block, from part r on.
__device__ __forceinline__ int part_of(const Shared& sh, int block, int r) {
    while (block >= sh.blocks[r + 1]) r++;
    return r;
}
// Values in shared memory.  A warp has a run of blocks, each lane an equal share of them one behind the
// other, so that a lane's values follow those of the lanes before; the lanes lie an odd number of
// vectors apart, so that eight lanes' 16-byte loads touch all banks.
template <int DT>
struct Columns {
    static constexpr int E = kVecElems<DT>, kType = DT;
    using V = Vec<DT>;
    uint32_t at;                     // the thread's first vector
    int first, count;                // its number, and how many there are
    __device__ __forceinline__ Columns(uint32_t smem, int begin, int end, int each) {
        const int lane = (int)threadIdx.x & 31;
        at = smem + (uint32_t)(threadIdx.x * (unsigned)(each | 1)) * 16u;
        first = (end - begin) * lane / 32;
        count = (end - begin) * (lane + 1) / 32 - first;
        first += begin;
    }
    __device__ __forceinline__ uint4 raw(int k) const { return ld_smem(at + (uint32_t)k * 16u); }
    __device__ __forceinline__ void put(int k, const uint4& v) const { st_smem(at + (uint32_t)k * 16u, v); }
    // f(number of the vector, vector) for all of the thread's
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
        for (int k = 0; k < count; k++) f(k, raw(k));
    }
};

// The warp's blocks [begin, end) of a row into shared memory, by the warp.
template <int DT>
__device__ __forceinline__ void load_blocks(const Shared& sh, int parts, int begin, int end, int each, uint32_t smem) {
    constexpr int E = kVecElems<DT>;
    const int lane = (int)threadIdx.x & 31, stride = each | 1;
    const uint32_t base = smem + (threadIdx.x & ~31u) * (unsigned)stride * 16u;
    const int run = end - begin;
    const auto slot = [&](int i) {
        const int owner = (32 * (i + 1) - 1) / run;    // the lane l with run l / 32 <= i < run (l + 1) / 32
        return base + (uint32_t)(owner * stride + i - run * owner / 32) * 16u;
    };
    for (int i = lane, r = 0; i < run; i += 32) {
        r = part_of(sh, begin + i, r);
        copy_block_async(slot(i), reinterpret_cast<const char*>(sh.part[r] + (begin + i - sh.blocks[r])));
    }
    copies_commit();
    copies_wait();
    __syncwarp();
    // what the first and the last block of a part hold besides it
    for (int r = lane; r < parts; r += 32) {
        const int first = sh.blocks[r], last = sh.blocks[r + 1] - 1;
        const auto cut = [&](int b) {
            if (b < begin || b >= end) return;
            const int at = (b - first) * E - sh.shift[r];        // the first value's place in its part
            const uint32_t p = slot(b - begin);
            st_smem(p, Vec<DT>::only(ld_smem(p), -at, sh.length[r] - at));
        };
        cut(first);
        if (last > first) cut(last);
    }
    __syncwarp();
}

// The distance d from the largest key at which the running count (or, BY_MASS, the running sum of
// weights) reaches `target`: *before is what lies before d.  Looks at distances of at most `most`.
// False where all of them together do not reach it.
template <int DT, bool BY_MASS, typename Cols>
__device__ bool search(Shared& sh, Team& team, uint32_t* hist, const Cols& cols, const Weights& w, uint32_t keyTop,
                       uint32_t most, u64 target, uint32_t* at, u64* before) {
    constexpr int E = Cols::E;
    uint32_t* const low = hist;                        // counts, or the sums' low words
    uint32_t* const high = hist + kSampleBins;
    const int slice = kSampleBins / team.size, per = max(1, slice / kSampleThreads);
    uint32_t base = 0;
    u64 below = 0;
    int shift = max(0, 32 - __clz((int)most) - 11);
    for (;;) {
        const bool masses = BY_MASS && shift > 0;      // a bin of one value needs counts alone
        const float lowest = value_of<DT>(keyTop - most);
        for (int i = threadIdx.x; i < kSampleBins * (masses ? 2 : 1); i += kSampleThreads) hist[i] = 0;
        __syncthreads();
        cols.each([&](int, const uint4& v) {
            if (Cols::V::largest(v) < lowest) return;
            float f[E];
            widen_vec<Cols::kType>(v, f);
            u64 weight[E];
            if (masses) w.fixed(f, weight);
#pragma unroll
            for (int j = 0; j < E; j++) {
                const uint32_t d = keyTop - key_of<DT>(f[j]);
                if (d > most || d < base) continue;
                const uint32_t bin = (d - base) >> shift;
                if (!masses) {
                    atomicAdd(&low[bin], 1u);
                } else {
                    const u64 e = weight[j];
                    const uint32_t old = atomicAdd(&low[bin], (uint32_t)e);
                    const uint32_t carry = (uint32_t)(e >> 32) + (old + (uint32_t)e < old ? 1u : 0u);
                    if (carry) atomicAdd(&high[bin], carry);
                }
            }
        });
        meet(team);
        // This CTA's share of the bins, over all CTAs.
        u64 val[4], sum = 0;
        const int bin0 = team.rank * slice + (int)threadIdx.x * per;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            val[i] = 0;
            if (i >= per || (int)threadIdx.x * per >= slice) continue;
            for (int c = 0; c < team.size; c++) {
                if (team.size == 1) {
                    val[i] += low[bin0 + i];
                    if (masses) val[i] += (u64)high[bin0 + i] << 32;
                } else {
                    val[i] += ld_cluster(low + bin0 + i, c);
                    if (masses) val[i] += (u64)ld_cluster(high + bin0 + i, c) << 32;
                }
            }
            if (BY_MASS && !masses && val[i]) val[i] *= w.fixed(value_of<DT>(keyTop - (base + bin0 + i)));
            sum += val[i];
        }
        // exclusive prefix over the CTA's threads
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 v = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) sh.warp[0][warp] = run;
        __syncthreads();
        u64 all = 0, ahead = run - sum;
        for (int i = 0; i < kWarps; i++) {
            if (i < warp) ahead += sh.warp[0][i];
            all += sh.warp[0][i];
        }
        const u64 mine[kWords] = {all, 0, 0, 0};
        const u64(*box)[kWords] = exchange(sh, team, mine);
        u64 total = below;
        ahead += below;
        for (int c = 0; c < team.size; c++) {
            if (c < team.rank) ahead += box[c][0];
            total += box[c][0];
        }
        if (total < target) return false;
        u64* const found = sh.found[team.flipFound];
        team.flipFound ^= 1;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (ahead < target && ahead + val[i] >= target) {
                const uint32_t words[4] = {(uint32_t)(bin0 + i), 0u, (uint32_t)ahead, (uint32_t)(ahead >> 32)};
                for (int c = 0; c < team.size; c++)
                    for (int k = 0; k < 4; k++) {
                        if (team.size == 1) ((uint32_t*)found)[k] = words[k];
                        else st_cluster((const char*)found + 4 * k, c, words[k]);
                    }
            }
            ahead += val[i];
        }
        meet(team);
        base += (uint32_t)found[0] << shift;
        below = found[1];
        if (shift == 0) break;
        most = min(most, base + ((1u << shift) - 1));
        shift = max(0, shift - 11);
    }
    *at = base;
    *before = below;
    return true;
}

// x times f, f below 1, rounded down, or up: a product of 24 by 64 bits.
__device__ __forceinline__ u64 share_of(u64 x, float f, bool up) {
    if (!(f > 0.0f)) return 0;
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const u64 m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int down = 150 - (int)max(e, 1u);            // 24 or more
    const u64 lo = x * m, hi = __umul64hi(x, m);
    if (down >= 128) return up;
    const u64 whole = down >= 64 ? hi >> (down - 64) : hi << (64 - down) | lo >> down;
    const u64 rest = down >= 64 ? lo | (down > 64 ? hi << (128 - down) : 0) : lo << (64 - down);
    return whole + (up && rest ? 1 : 0);
}

// What the filters of a row ask for.
struct Filters {
    float heat, p, least;
    int k;                           // vocab: no limit
    bool greedy, limited, nucleus;
};

// The exact sum of all weights.
template <typename Cols>
__device__ u64 exact_sum(Shared& sh, Team& team, const Cols& cols, const Weights& w) {
    u64 s = 0, none = 0;
    cols.each([&](int, const uint4& v) {
        float f[Cols::E];
        u64 e[Cols::E];
        widen_vec<Cols::kType>(v, f);
        w.fixed(f, e);
#pragma unroll
        for (int j = 0; j < Cols::E; j++) s += e[j];
    });
    block_sums(sh, s, none);
    const u64 mine[kWords] = {s, 0, 0, 0};
    const u64(*box)[kWords] = exchange(sh, team, mine);
    u64 all = 0;
    for (int c = 0; c < team.size; c++) all += box[c][0];
    return all;
}

// The smallest value of weight `e`, with room for the roundings.
__device__ __forceinline__ float value_at(const Weights& w, float e) {
    const float x = w.top + (__log2f(e) - 0.01f) / w.ch;
    return x - 1e-5f * fabsf(x) - 1e-5f * fabsf(w.top);
}

// The token, from values that hold all that may be kept: none below kBound counts for topK, none below
// pBound for topP.  exact: the sum of all weights where topP is a share of it, else 0; total: of the
// weights before the filters, 0 where it is not known yet.  token_of gives a value's token.
template <int DT, typename Cols, typename TokenOf>
__device__ __forceinline__ void decide(const SampleArgs& a, const Filters& q, Shared& sh, Team& team, uint32_t* hist, const Cols& cols,
                                       const Weights& w, float kBound, float pBound, u64 exact, u64 total, int row, TokenOf token_of) {
    constexpr int E = Cols::E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float top = w.top;
    const uint32_t keyTop = key_of<DT>(top);
    // Distance of the smallest value that a value of at least x can have.
    const auto distance = [&](float x) { return x >= top ? 0u : keyTop - key_of<DT>(fmaxf(x, -3.40282347e38f)); };

    // What is kept: distances below `edge`, and the first `ties` values at it.
    uint32_t edge = 0xFFFFFFFFu;
    u64 ties = 0, before = 0;
    bool cut = false;
    if (q.k == 1) {                  // the first of the largest
        edge = 0;
        ties = 1;
        cut = true;
    } else if (q.limited) {
        cut = search<DT, false>(sh, team, hist, cols, w, keyTop, distance(kBound), (u64)q.k, &edge, &before);
        if (cut) ties = (u64)q.k - before;
    }
    if (q.nucleus) {
        uint32_t most;
        if (cut) {                   // the sum of the topK
            u64 s = 0, none = 0;
            cols.each([&](int, const uint4& v) {
                if (Cols::V::largest(v) < value_of<DT>(keyTop - edge)) return;
                float f[E];
                u64 weight[E];
                widen_vec<Cols::kType>(v, f);
                w.fixed(f, weight);
#pragma unroll
                for (int j = 0; j < E; j++)
                    if (keyTop - key_of<DT>(f[j]) < edge) s += weight[j];
            });
            block_sums(sh, s, none);
            const u64 mine[kWords] = {s, 0, 0, 0};
            const u64(*box)[kWords] = exchange(sh, team, mine);
            exact = ties * w.fixed(value_of<DT>(keyTop - edge));
            for (int c = 0; c < team.size; c++) exact += box[c][0];
            most = edge;
        } else {
            if (q.limited) exact = exact_sum(sh, team, cols, w);     // fewer than topK
            most = distance(pBound);
        }
        const u64 goal = max(1ull, share_of(exact, q.p, true));
        uint32_t at;
        if (search<DT, true>(sh, team, hist, cols, w, keyTop, most, goal, &at, &before)) {
            const u64 one = max(1ull, w.fixed(value_of<DT>(keyTop - at)));
            const u64 n = (goal - before + one - 1) / one;
            ties = cut && at == edge ? min(ties, n) : n;
            edge = at;
            cut = true;
        }
    }
    const u64 floorWeight = q.least >= 1.0f ? 1ull << kFix : share_of(1ull << kFix, q.least, true);
    const float floorValue = floorWeight ? value_at(w, fminf(q.least, 1.0f)) : -INFINITY;

    // Weights kept by every warp, its ties at the edge aside.
    u64 atEdge = cut ? w.fixed(value_of<DT>(keyTop - edge)) : 0;
    if (atEdge < floorWeight) atEdge = 0;
    const auto kept = [&](float x, u64 weight, bool* tie) {
        const uint32_t d = keyTop - key_of<DT>(x);
        *tie = cut && d == edge;
        return (cut && d >= edge) || weight < floorWeight ? 0ull : weight;
    };
    // What lies below this is not kept, and no tie.
    const float bottom = fmaxf(cut ? value_of<DT>(keyTop - edge) : -INFINITY, floorValue);
    u64 sum = 0, count = 0;
    cols.each([&](int, const uint4& v) {
        if (Cols::V::largest(v) < bottom) return;
        float f[E];
        u64 weight[E];
        widen_vec<Cols::kType>(v, f);
        w.fixed(f, weight);
#pragma unroll
        for (int j = 0; j < E; j++) {
            bool tie;
            sum += kept(f[j], weight[j], &tie);
            count += tie;
        }
    });
    u64 blockSum = sum, blockCount = count;
    block_sums(sh, blockSum, blockCount);              // leaves every warp's sums in sh.warp
    const u64 mine[kWords] = {blockSum, blockCount, 0, 0};
    const u64(*box)[kWords] = exchange(sh, team, mine);
    // From here on nothing touches another CTA's memory.  What is kept before this warp, and of its ties.
    u64 all = 0, ahead = 0, left = ties;
    {
        u64 rest = ties;
        for (int c = 0; c < team.size; c++) {
            const u64 n = min(rest, box[c][1]);
            if (c == team.rank) {
                ahead = all;
                left = rest;
            }
            all += box[c][0] + n * atEdge;
            rest -= n;
        }
        for (int i = 0; i < warp; i++) {
            const u64 n = min(left, sh.warp[1][i]);
            ahead += sh.warp[0][i] + n * atEdge;
            left -= n;
        }
    }
    const float u = a.uniform[row];
    const u64 goal = u >= 1.0f ? all - 1 : share_of(all, u, false);
    // The ties before this thread's, then what is kept before it.
    u64 runTies = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(~0u, runTies, o);
        if (lane >= o) runTies += x;
    }
    left -= min(left, runTies - count);
    sum += min(left, count) * atEdge;
    u64 run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += x;
    }
    ahead += run - sum;
    if (goal < ahead || goal >= ahead + sum) return;
    // The thread whose values hold the token goes through them in order, a vector's weights at a time (256 rows
    // of 131072 without filters 126 us; one weight behind the other 133).
    for (int k = 0; k < cols.count; k++) {
        const uint4 vec = cols.raw(k);
        if (Cols::V::largest(vec) < bottom) continue;
        float f[E], x = 0.0f;
        u64 weight[E];
        widen_vec<Cols::kType>(vec, f);
        w.fixed(f, weight);
        int at = -1;
#pragma unroll
        for (int j = 0; j < E; j++) {
            bool tie;
            u64 e = kept(f[j], weight[j], &tie);
            if (tie && left > 0) {
                left--;
                e = atEdge;
            }
            ahead += e;
            if (at >= 0 || goal >= ahead) continue;
            at = j;
            x = f[j];
        }
        if (at < 0) continue;
        const int token = token_of((cols.first + k) * E + at);
        for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = token;
        if (a.logprob) {
            const float z = x == top ? 0.0f : q.greedy ? x - top : (x - top) / q.heat;
            a.logprob[row] = z - log1pf((float)((total ? total : all) - (1ull << kFix)) * 0x1p-44f);
        }
        return;
    }
}

// A list's values, kPer a thread in their order.
constexpr int kPer = kSampleList / kSampleThreads;
static_assert(kPer * kSampleThreads == kSampleList, "the list is shared out");

// The CTA's sum, in every thread; `buffer` alternates from call to call.
__device__ __forceinline__ int block_count(Shared& sh, int v, int& buffer) {
    v = __reduce_add_sync(~0u, v);
    if ((threadIdx.x & 31) == 0) sh.count[buffer][threadIdx.x >> 5] = v;
    __syncthreads();
    const int w = (int)threadIdx.x & 31;
    v = __reduce_add_sync(~0u, w < kWarps ? sh.count[buffer][w] : 0);
    buffer ^= 1;
    return v;
}
// The same of numbers below 2^45 (at most kSampleList of them): three sums of 15 bits each.
__device__ __forceinline__ u64 block_mass(Shared& sh, const unsigned (&part)[3], int& buffer) {
    unsigned v[3];
#pragma unroll
    for (int i = 0; i < 3; i++) {
        v[i] = __reduce_add_sync(~0u, part[i]);
        if ((threadIdx.x & 31) == 0) sh.mass[buffer][i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
    const int w = (int)threadIdx.x & 31;
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < 3; i++) sum += (u64)__reduce_add_sync(~0u, w < kWarps ? sh.mass[buffer][i][w] : 0u) << (15 * i);
    buffer ^= 1;
    return sum;
}
__device__ __forceinline__ void add_mass(unsigned (&part)[3], u64 v) {
#pragma unroll
    for (int i = 0; i < 3; i++) part[i] += (unsigned)(v >> (15 * i)) & 0x7FFFu;
}

// As decide(), by one CTA, of the `n` values of its list that are no further than `most` from the top, each
// thread's distances in d.
template <int DT, typename TokenOf>
__device__ __forceinline__ bool decide_few(const SampleArgs& a, const Filters& q, Shared& sh, const float* values, const uint32_t (&d)[kPer],
                                           uint32_t most, int n, const Weights& w, u64 least, u64 exact, u64 total, int row,
                                           TokenOf token_of) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = (int)threadIdx.x * kPer;
    // in their order, one a thread
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; j++) mine += d[j] <= most;
    int to = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, to, o);
        if (lane >= o) to += x;
    }
    __syncthreads();
    if (lane == 31) sh.count[0][warp] = to;
    __syncthreads();
    to -= mine;
    for (int i = 0; i < warp; i++) to += sh.count[0][i];
#pragma unroll
    for (int j = 0; j < kPer; j++)
        if (d[j] <= most) sh.few[to++] = FewValue{d[j], first + j, w.fixed(values[first + j])};
    __syncthreads();
    // its place, and the sum of what lies before it, in the order of the filters; two or four threads a
    // value, each of which compares it with its share of all
    const int ways = n <= kSampleThreads / 4 ? 4 : 2, span = kSampleThreads / ways;
    const int i = (int)threadIdx.x % span, way = (int)threadIdx.x / span;
    FewValue own = {0xFFFFFFFFu, 0, 0};
    int place = 0;
    u64 before = 0;
    if (i < n) own = sh.few[i];
    if (i / 32 * 32 < n) {
#pragma unroll 4
        for (int j = n * way / ways; j < n * (way + 1) / ways; j++) {
            const FewValue other = sh.few[j];
            if (other.d < own.d + (j < i)) {
                place++;
                before += other.v;
            }
        }
    }
    if (way > 0) {
        sh.place[way - 1][i] = place;
        sh.before[way - 1][i] = before;
    }
    __syncthreads();
    if (way > 0) own = FewValue{0xFFFFFFFFu, 0, 0};
    for (int k = 0; k < (way == 0 ? ways - 1 : 0); k++) {
        place += sh.place[k][i];
        before += sh.before[k][i];
    }
    bool keep = way == 0 && i < n && place < q.k;
    if (q.nucleus) {
        if (q.limited) {             // the sum of the topK
            if (keep && (place == q.k - 1 || place == n - 1)) sh.total = before + own.v;
            __syncthreads();
            least = exact = sh.total;
        }
        keep = keep && before < max(1ull, share_of(exact, q.p, true));
        if (least != exact && __syncthreads_or(keep && before >= max(1ull, share_of(least, q.p, true)))) return false;
    }
    const u64 floorWeight = q.least >= 1.0f ? 1ull << kFix : share_of(1ull << kFix, q.least, true);
    const u64 sum = keep && own.v >= floorWeight ? own.v : 0;
    u64 run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += x;
    }
    if (lane == 31) sh.warp[0][warp] = run;
    __syncthreads();
    u64 all = 0, ahead = run - sum;
#pragma unroll
    for (int k = 0; k < kSampleFew / 32; k++) {
        const u64 x = sh.warp[0][k];
        if (k < warp) ahead += x;
        all += x;
    }
    const float u = a.uniform[row];
    const u64 goal = u >= 1.0f ? all - 1 : share_of(all, u, false);
    if (goal < ahead || goal >= ahead + sum) return true;
    const float x = values[own.at];
    const int token = token_of(own.at);
    for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = token;
    if (a.logprob) {
        const float z = x == w.top ? 0.0f : q.greedy ? x - w.top : (x - w.top) / q.heat;
        a.logprob[row] = z - log1pf((float)(total - (1ull << kFix)) * 0x1p-44f);
    }
    return true;
}

// As decide(), by one CTA, of the `few` values of its list, of which none is further than `most` from the top.
// The sum that topP is a share of lies between `least` and `exact`: false where that leaves open what is kept.
template <int DT, typename TokenOf>
__device__ __forceinline__ bool decide_list(const SampleArgs& a, const Filters& q, Shared& sh, const float* values, int few,
                                            const Weights& w, uint32_t most, u64 least, u64 exact, u64 total, int row,
                                            TokenOf token_of) {
    const float top = w.top;
    const uint32_t keyTop = key_of<DT>(top);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = (int)threadIdx.x * kPer;
    uint32_t d[kPer];
    u64 v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j++) d[j] = first + j < few ? keyTop - key_of<DT>(values[first + j]) : 0xFFFFFFFFu;
    int buffer = 0, within = 0;      // minus infinities are in the list where there is no bound
#pragma unroll
    for (int j = 0; j < kPer; j++) within += d[j] <= most;
    within = block_count(sh, within, buffer);
    // Few enough to compare all with all: those up to a distance that leaves at least k, or, of topP's
    // weights, rounded down to units of 2^-20, more than the goal.
    const bool byMass = q.nucleus && !q.limited;
    if (within <= kSampleFew || byMass || (q.limited && q.k <= kSampleFew)) {
        uint32_t lo = 0, hi = most;  // up to hi there are `n`, at least k of them where there are k
        int n = within;
        if (n > kSampleFew) {
            unsigned weight[kPer];
#pragma unroll
            for (int j = 0; j < kPer; j++) weight[j] = byMass && d[j] <= most ? (unsigned)(w.fixed(values[first + j]) >> (kFix - 20)) : 0u;
            const u64 goal = (share_of(exact, q.p, true) >> (kFix - 20)) + 1;
            while (n > kSampleFew && lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                int c = 0;
                unsigned sum = 0;
#pragma unroll
                for (int j = 0; j < kPer; j++) {
                    c += d[j] <= mid;
                    sum += d[j] <= mid ? weight[j] : 0u;
                }
                c = block_count(sh, c, buffer);
                if (byMass ? (unsigned)block_count(sh, (int)sum, buffer) >= goal : c >= q.k) {
                    hi = mid;
                    n = c;
                } else {
                    lo = mid + 1;
                }
            }
        }
        if (n <= kSampleFew)
            return decide_few<DT>(a, q, sh, values, d, hi, n, w, least, exact, total, row, token_of);
    }
    // What is kept: distances below `edge`, and the first `ties` values at it.
    uint32_t edge = most;
    u64 ties = ~0ull;
    if (q.limited && within >= q.k) {
        uint32_t lo = 0;             // fewer than k are nearer than lo: `below` of them
        int below = 0;
        while (lo < edge) {
            const uint32_t mid = lo + (edge - lo) / 2;
            int n = 0;
#pragma unroll
            for (int j = 0; j < kPer; j++) n += d[j] <= mid;
            n = block_count(sh, n, buffer);
            if (n >= q.k) {
                edge = mid;
            } else {
                lo = mid + 1;
                below = n;
            }
        }
        ties = (u64)(q.k - below);
    }
#pragma unroll
    for (int j = 0; j < kPer; j++) v[j] = d[j] <= edge ? w.fixed(values[first + j]) : 0;
    if (q.nucleus) {
        if (q.limited) {             // the sum of the topK
            unsigned part[3] = {};
#pragma unroll
            for (int j = 0; j < kPer; j++)
                if (d[j] < edge || ties == ~0ull) add_mass(part, v[j]);
            exact = block_mass(sh, part, buffer);
            if (ties != ~0ull) exact += ties * w.fixed(value_of<DT>(keyTop - edge));
            least = exact;
        }
        const u64 goal = max(1ull, share_of(exact, q.p, true));
        uint32_t lo = 0, hi = edge;
        u64 before = 0;              // the sum of what is nearer than lo, less than the goal
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            unsigned part[3] = {};
#pragma unroll
            for (int j = 0; j < kPer; j++)
                if (d[j] <= mid) add_mass(part, v[j]);
            const u64 sum = block_mass(sh, part, buffer);
            if (sum >= goal) {
                hi = mid;
            } else {
                lo = mid + 1;
                before = sum;
            }
        }
        const u64 one = max(1ull, w.fixed(value_of<DT>(keyTop - hi))), n = (goal - before + one - 1) / one;
        if (least != exact && max(1ull, share_of(least, q.p, true)) <= before + (n - 1) * one) return false;
        ties = hi == edge ? min(ties, n) : n;
        edge = hi;
    }
    const u64 floorWeight = q.least >= 1.0f ? 1ull << kFix : share_of(1ull << kFix, q.least, true);
    u64 sum = 0, atEdge = w.fixed(value_of<DT>(keyTop - edge));
    if (atEdge < floorWeight) atEdge = 0;
    int n = 0;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        n += d[j] == edge;
        v[j] = d[j] < edge && v[j] >= floorWeight ? v[j] : 0;
        sum += v[j];
    }
    // The ties before this thread's, then what is kept before it.
    int runTies = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, runTies, o);
        if (lane >= o) runTies += x;
    }
    __syncthreads();
    if (lane == 31) sh.count[0][warp] = runTies;
    __syncthreads();
    runTies -= n;
    for (int i = 0; i < warp; i++) runTies += sh.count[0][i];
    int mineLeft = (int)(ties > (u64)runTies ? min(ties - (u64)runTies, (u64)n) : 0);
    sum += (u64)mineLeft * atEdge;
    u64 run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += x;
    }
    if (lane == 31) sh.warp[0][warp] = run;
    __syncthreads();
    u64 all = 0, ahead = run - sum;
    for (int i = 0; i < kWarps; i++) {
        if (i < warp) ahead += sh.warp[0][i];
        all += sh.warp[0][i];
    }
    const float u = a.uniform[row];
    const u64 goal = u >= 1.0f ? all - 1 : share_of(all, u, false);
    if (goal < ahead || goal >= ahead + sum) return true;
    int pick = 0;
    bool done = false;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        u64 e = v[j];
        if (d[j] == edge && mineLeft > 0) {
            mineLeft--;
            e = atEdge;
        }
        ahead += e;
        if (!done && goal < ahead) {
            done = true;
            pick = j;
        }
    }
    const int token = token_of(first + pick);
    const float x = values[first + pick];
    for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = token;
    if (a.logprob) {
        const float z = x == top ? 0.0f : q.greedy ? x - top : (x - top) / q.heat;
        a.logprob[row] = z - log1pf((float)(total - (1ull << kFix)) * 0x1p-44f);
    }
    return true;
}

// From a row's values to its token.  top is this thread's largest value.
template <int DT, typename Cols, typename TokenOf>
__device__ __forceinline__ void draw(const SampleArgs& a, const Filters& q, Shared& sh, Team& team, uint32_t* hist,
                                     float* listValues, int* listTokens, const Cols& cols, float top, int row, TokenOf token_of) {
    constexpr int E = Cols::E;
    using V = typename Cols::V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // The largest value, and for topK the smallest maximum of at least k disjoint groups, of as many lanes
    // each as leave that many.
    const int groups = team.size * kWarps;
    int lanes = 32;
    while (lanes > 1 && q.k > groups * (32 / lanes)) lanes >>= 1;
    float kBound = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float other = __shfl_xor_sync(~0u, kBound, o);
        kBound = o < lanes ? fmaxf(kBound, other) : fminf(kBound, other);
    }
    if (lane == 0) {
        sh.max[warp] = top;
        sh.low[warp] = kBound;
    }
    __syncthreads();
    // (groups of several warps where fewer groups are enough: what is above their bound is less)
    int together = 1;
    while (together < kWarps && groups / (2 * together) >= q.k) together *= 2;
    kBound = INFINITY;
    float own = -INFINITY;
    for (int i = 0; i < kWarps; i++) {
        top = fmaxf(top, sh.max[i]);
        own = fmaxf(own, sh.low[i]);
        if (together == 1 || (i + 1) % together == 0) {
            kBound = fminf(kBound, own);
            own = -INFINITY;
        }
    }
    if (team.size > 1) cluster_wait();                 // every CTA of the cluster has started
    {
        const u64 mine[kWords] = {__float_as_uint(top), __float_as_uint(kBound), 0, 0};
        const u64(*box)[kWords] = exchange(sh, team, mine);
        for (int c = 0; c < team.size; c++) {
            top = fmaxf(top, __uint_as_float((uint32_t)box[c][0]));
            kBound = fminf(kBound, __uint_as_float((uint32_t)box[c][1]));
        }
        if (q.k > 32 * groups) kBound = -INFINITY;
    }
    if (top == -INFINITY) {                            // nothing to draw from
        if (threadIdx.x == 0 && team.rank == 0) {
            for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7FFFFFFF);
        }
        return;
    }

    Weights w;
    w.powers = sh.powers;
    w.set(top, q.greedy ? 1.0f : q.heat);

    // All that may be kept is at least `bound`: topK's is known, topP's follows from the sum of all weights,
    // minP's is a weight.  (pBound: weights below (1 - p) of the mean are outside topP, all of them together.)
    u64 exact = 0, total = 0;
    float bound = -INFINITY, pBound = -INFINITY;
    const bool share = q.nucleus && !q.limited;        // topP of all
    if (q.k == 1) bound = kBound = top;
    else if (q.limited) bound = kBound;
    if (!q.nucleus && q.least > 0.0f) bound = fmaxf(bound, value_at(w, fminf(q.least, 1.0f)));
    const auto within = [&](float b) { return b <= top ? b : b > top ? top : -INFINITY; };
    bound = within(bound);

    // The sum of all weights, roughly, and how many values are above the bound.
    u64 few = 0, ahead = 0, mine = 0;                  // of the row, of the CTAs before, of this thread
    // The rough sum of a vector's values, whose largest is m; of those that are at least `from`.
    const auto rough = [&](float (&f)[E], float m, float from) {
        u64 sum = 0;
        if (m == top || from > -INFINITY) {            // the largest apart: what is beside them may be small
#pragma unroll
            for (int j = 0; j < E; j++) {
                sum += f[j] == top ? 1ull << kFix : 0ull;
                f[j] = f[j] == top || f[j] < from ? -INFINITY : f[j];
            }
        }
        return sum + __float2ull_rn(w.rough(f) * (float)(1ull << kFix));
    };
    // Goes through all values: the rough sum of all, or of those above the bound, and their number.
    const auto go_through = [&](bool all, bool above, bool counts) {
        u64 sum = 0, count = 0;
        cols.each([&](int, const uint4& v) {
            const float m = V::largest(v);
            if (!all && m < bound) return;
            float f[E];
            widen_vec<DT>(v, f);
            if (counts && m >= bound) {
#pragma unroll
                for (int j = 0; j < E; j++) count += f[j] >= bound;
            }
            if (all || above) sum += rough(f, m, all ? -INFINITY : bound);
        });
        mine = count;
        block_sums(sh, sum, count);                    // leaves every warp's sums in sh.warp
        const u64 words[kWords] = {sum, count, 0, 0};
        const u64(*box)[kWords] = exchange(sh, team, words);
        u64 sums = 0;
        few = ahead = 0;
        for (int c = 0; c < team.size; c++) {
            sums += box[c][0];
            if (c < team.rank) ahead += box[c][1];
            few += box[c][1];
        }
        return sums;
    };
    // A weight of the rough sum is at most kRough of itself off: 45 units of the exponent rounded twice,
    // and the exponential's 2^-22.
    constexpr float kRough = 0x1p-17f;
    if (q.limited || q.nucleus || q.least > 0.0f) {
        if (a.logprob || share) total = go_through(true, false, !share);
        else go_through(false, false, true);
        bool listed = true;
        if (share) {
            // at most a list's worth of weights can be above a list's part of their sum; mostly they hold topP
            bound = within(value_at(w, (float)total * 0x1p-44f / (kSampleList - 64)));
            const u64 held = go_through(false, true, true);
            listed = (float)held * (1.0f - 4.0f * kRough) > fmaxf(q.p, 0.0f) * (float)total;
        }
        if (few > (u64)kSampleList) listed = false;
        if (listed) {
            // to the first CTA's list, in order
            int to = (int)mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, to, o);
                if (lane >= o) to += x;
            }
            to += (int)ahead - (int)mine;
            for (int i = 0; i < warp; i++) to += (int)sh.warp[1][i];
            if (mine) {
                cols.each([&](int k, const uint4& v) {
                    if (V::largest(v) < bound) return;
                    float f[E];
                    widen_vec<DT>(v, f);
#pragma unroll
                    for (int j = 0; j < E; j++) {
                        if (!(f[j] >= bound)) continue;
                        const int number = (cols.first + k) * E + j;
                        if (team.size == 1) {
                            listValues[to] = f[j];
                            listTokens[to] = number;
                        } else {
                            st_cluster(listValues + to, 0, __float_as_uint(f[j]));
                            st_cluster(listTokens + to, 0, (uint32_t)number);
                        }
                        to++;
                    }
                });
            }
            meet(team);
            if (!share && team.rank != 0) return;
            const auto token_at = [&](int i) { return token_of(listTokens[i]); };
            const uint32_t most = bound >= top ? 0u : key_of<DT>(top) - key_of<DT>(fmaxf(bound, -3.40282347e38f));
            if (!share) {
                decide_list<DT>(a, q, sh, listValues, (int)few, w, most, 0, 0, total, row, token_at);
                return;
            }
            // topP of a sum that is exact for what is listed and rough for the rest, a (1 - p)-th of it at most:
            // mostly that leaves nothing open.
            bool settled = false;
            if (team.rank == 0) {
                u64 own = 0, rough = 0;
                for (int i = threadIdx.x; i < (int)few; i += kSampleThreads) {
                    const float x = listValues[i], pair[2] = {x == top ? -INFINITY : x, -INFINITY};
                    own += w.fixed(x);
                    rough += x == top ? 1ull << kFix : __float2ull_rn(w.rough(pair) * (float)(1ull << kFix));
                }
                block_sums(sh, own, rough);
                const u64 rest = total > rough ? total - rough : 0;
                // (and for the rounding of both rough sums, a unit of 2^-23 a vector or value)
                const u64 off = (u64)((float)rest * kRough) + (u64)((float)total * 0x1p-21f) + (u64)a.vocab;
                const u64 least = own + (rest > off ? rest - off : 0), exactMost = own + rest + off;
                settled = decide_list<DT>(a, q, sh, listValues, (int)few, w, most, least, exactMost, total, row, token_at);
                if ((int)threadIdx.x < team.size) {
                    if (team.size == 1) sh.settled = settled;
                    else st_cluster(&sh.settled, threadIdx.x, (uint32_t)settled);
                }
            }
            meet(team);
            if (sh.settled) return;
            exact = total = exact_sum(sh, team, cols, w);
            if (team.rank == 0) decide_list<DT>(a, q, sh, listValues, (int)few, w, most, exact, exact, total, row, token_at);
            return;
        }
        if (share) {
            exact = total = exact_sum(sh, team, cols, w);
            pBound = value_at(w, (1.0f - fmaxf(q.p, 0.0f)) * 0.99f * ((float)exact * 0x1p-44f) / (float)a.vocab);
        }
    }
    decide<DT>(a, q, sh, team, hist, cols, w, kBound, pBound, exact, total, row, token_of);
}

__device__ __forceinline__ Filters filters_of(const SampleArgs& a, int row) {
    Filters q;
    q.heat = a.temperature ? a.temperature[row] : 1.0f;
    q.greedy = !(q.heat > 0.0f);
    q.k = q.greedy ? 1 : a.topK ? a.topK[row] : 0;
    if (q.k <= 0 || q.k >= a.vocab) q.k = a.vocab;
    q.p = a.topP && !q.greedy ? a.topP[row] : 1.0f;
    q.least = a.minP && !q.greedy ? a.minP[row] : 0.0f;
    q.limited = q.k < a.vocab;
    q.nucleus = q.p < 1.0f && q.k > 1;
    return q;
}

template <int DT>
__global__ void __launch_bounds__(kSampleThreads, 2) k_sample(const __grid_constant__ SampleArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ Shared sh;
    // either a list or a histogram
    uint32_t* const hist = reinterpret_cast<uint32_t*>(dynamic);
    float* const listValues = reinterpret_cast<float*>(dynamic);
    static_assert(2 * kSampleBins * 4 <= kSampleList * 8, "the histogram has room where the list is");
    int* const listTokens = reinterpret_cast<int*>(listValues + kSampleList);
    const uint32_t values = (uint32_t)__cvta_generic_to_shared(listTokens + kSampleList);
    Team team;
    team.size = a.cluster;
    team.rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    team.flip = team.flipFound = 0;
    if (team.size > 1) cluster_arrive();               // waited for before another CTA's memory is touched
    const int row = (int)(blockIdx.x / (unsigned)team.size), warp = (int)threadIdx.x >> 5;
    if (threadIdx.x < 32) sh.powers[threadIdx.x] = kPowers[threadIdx.x];
    const Filters q = filters_of(a, row);
    find_parts<DT>(a, sh, row);
    // every warp of the cluster the same share of the blocks, so that none is without a value
    const int total = sh.blocks[a.nParts], warps = team.size * kWarps;
    const auto share = [&](int w) { return (int)((long long)total * w / warps); };
    const int begin = share(team.rank * kWarps + warp), end = share(team.rank * kWarps + warp + 1);
    load_blocks<DT>(sh, a.nParts, begin, end, a.each, values);
    const Columns<DT> cols(values, begin, end, a.each);
    // a NaN counts as minus infinity, and is overwritten by it
    float top = -INFINITY;
    cols.each([&](int k, uint4 v) {
        if (Vec<DT>::suspect(v)) {
            v = Vec<DT>::only(v, 0, E);
            cols.put(k, v);
        }
        top = fmaxf(top, Vec<DT>::largest(v));
    });
    draw<DT>(a, q, sh, team, hist, listValues, listTokens, cols, top, row, [&](int number) {
        const int block = number / E, r = part_of(sh, block, 0);
        return r * a.part + (block - sh.blocks[r]) * E - sh.shift[r] + number % E;
    });
}

template <int DT>
cudaError_t sample_launch(const SampleArgs& a, cudaStream_t s) {
    const auto kernel = k_sample<DT>;
    // one value for every launch, as host threads share the kernel's limit
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleMaxSmem);
    if (e != cudaSuccess) return e;
    NormShape sh = {};
    sh.threads = kSampleThreads;
    sh.cluster = a.cluster;
    const size_t smem = kSampleList * 8 + (size_t)kSampleThreads * (a.each | 1) * 16;
    return norm_launch(kernel, (unsigned)a.rows * (unsigned)sh.cluster, sh, smem, s, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return sample_launch<kF32>(a, s);
    case vFloat16: return sample_launch<kF16>(a, s);
    case vBFloat16: return sample_launch<kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
