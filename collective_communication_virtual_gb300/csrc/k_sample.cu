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
// of the sum that all of them together could not fill lie outside topP.
//
// The draw is a comparison of sums, so these are exact: a weight is a 64-bit integer, 2^44 e, right to
// 2^-30 of itself, and the order of additions does not matter.
//
// A row is read once, into the shared memory of a cluster's CTAs, which exchange maxima, histograms
// and sums there.
#include "norm_stage.cuh"
#include "sample.h"

namespace vc {

namespace {

constexpr int kWarps = kSampleThreads / 32;
constexpr int kFix = 44;             // weights in units of 2^-44
typedef unsigned long long u64;

// 2^31 2^(k / 32), rounded
__constant__ uint32_t kPowers[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

struct Shared {
    uint32_t powers[32];
    float max[kWarps];
    float low[3][kWarps];            // smallest maximum of a warp, of its 8-lane groups, of its lanes
    u64 warp[2][kWarps];
    u64 box[2][kSampleCluster][4];   // one line a CTA, written by all CTAs of the cluster
    u64 found[2][3];                 // bin, what lies before it, what lies in it
    u64 target;
    int owner;
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
__device__ __forceinline__ const u64 (*exchange(Shared& sh, Team& team, const u64 (&mine)[4]))[4] {
    u64(*box)[4] = sh.box[team.flip];
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

// e of a value: x == top gives 1, also where both are infinite.
struct Weights {
    float top, ch, cl;               // ch + cl = log2(e) / temperature
    const uint32_t* powers;
    __device__ __forceinline__ float rough(float x) const { return exp2f((x - top) * ch); }
    // 2^44 e, as an integer: the difference and its product with ch + cl with their rounding errors,
    // 2^(k/32) from a table and 2^g, |g| <= 1/64, from its series.
    __device__ __forceinline__ u64 fixed(float x) const {
        if (x == top) return 1ull << kFix;
        const float dh = __fsub_rn(x, top);
        const float p = __fmul_rn(dh, ch);
        if (!(p >= -(float)kFix - 1.0f)) return 0;
        const float b = __fsub_rn(dh, x);
        const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(dh, b)), __fsub_rn(-top, b));
        const float pl = __fmaf_rn(dh, ch, -p) + __fmaf_rn(dh, cl, dl * ch);
        const float magic = 12582912.0f;               // 1.5 2^23: the sum's low bits are the integer
        const float r = __fadd_rn(p * 32.0f, magic);
        const int k = __float_as_int(r) - __float_as_int(magic);
        const float g = __fmaf_rn(__fsub_rn(r, magic), -0.03125f, p) + pl;
        const float q = g * fmaf(g, fmaf(g, fmaf(g, 0.009618129107628477f, 0.055504108664821576f), 0.2402265069591007f),
                                 0.6931471805599453f);
        const uint32_t t = powers[k & 31];
        const uint32_t m = t + (uint32_t)(int)(((long long)t * __float2int_rn(q * 4294967296.0f)) >> 32);
        const int down = -(k >> 5);
        return ((u64)m << (kFix - 31)) >> max(0, down);
    }
};

// A CTA's columns in shared memory: vector `step * 32 + lane` of a warp's run.
template <int DT>
struct Columns {
    static constexpr int E = kVecElems<DT>;
    uint32_t base;                   // the thread's first vector
    int first, steps;                // its first column within the CTA
    __device__ __forceinline__ Columns(uint32_t smem, int n) : steps(n) {
        const int vec = (int)(threadIdx.x >> 5) * 32 * n + (int)(threadIdx.x & 31);
        base = smem + (uint32_t)vec * 16u;
        first = vec * E;
    }
    // Values of a step; a NaN counts as minus infinity.
    __device__ __forceinline__ void get(int step, float (&f)[E]) const {
        widen_vec<DT>(ld_smem(base + (uint32_t)step * 512u), f);
#pragma unroll
        for (int j = 0; j < E; j++) f[j] = f[j] == f[j] ? f[j] : -INFINITY;
    }
};

// The CTA's columns [c0, c1) of a row into shared memory, minus infinity behind them.
template <int DT>
__device__ __forceinline__ void load_columns(const SampleArgs& a, int row, int c0, int columns, uint32_t smem) {
    constexpr int E = kVecElems<DT>, ESZ = DTypeOf<DT>::size;
    const int c1 = min(a.vocab, c0 + columns);
    const uint32_t none = DT == kF32 ? 0xFF800000u : DT == kBF16 ? 0xFF80u : 0xFC00u;
    const auto put = [&](int i, uint32_t v) {
        if (ESZ == 4) asm volatile("st.shared.u32 [%0], %1;" :: "r"(smem + 4u * i), "r"(v) : "memory");
        else asm volatile("st.shared.u16 [%0], %1;" :: "r"(smem + 2u * i), "h"((uint16_t)v) : "memory");
    };
    for (int i = max(0, c1 - c0) + (int)threadIdx.x; i < columns; i += kSampleThreads) put(i, none);
    for (int lo = c0; lo < c1;) {
        const int r = lo / a.part, hi = min(c1, (r + 1) * a.part);
        const char* from = (const char*)a.logits[r] + ((size_t)row * a.stride + (lo - r * a.part)) * ESZ;
        int done = 0;
        if (a.aligned) {             // lo is a multiple of E, as a part is
            const int whole = (hi - lo) / E;
            for (int i = threadIdx.x; i < whole; i += kSampleThreads)
                copy_block_async(smem + (uint32_t)(lo - c0) * ESZ + 16u * i, from + (size_t)i * 16);
            done = whole * E;
        }
#pragma unroll 4
        for (int i = done + (int)threadIdx.x; i < hi - lo; i += kSampleThreads)
            put(lo - c0 + i, ESZ == 4 ? ((const uint32_t*)from)[i] : (uint32_t)((const uint16_t*)from)[i]);
        lo = hi;
    }
    copies_commit();
    copies_wait();
    __syncthreads();
}

// The distance d from the largest key at which the running count (or, BY_MASS, the running sum of
// weights) reaches `target`: *before is what lies before d.  Looks at distances of at most `most`.
// False where all of them together do not reach it.
template <int DT, bool BY_MASS>
__device__ bool search(Shared& sh, Team& team, uint32_t* hist, const Columns<DT>& cols, const Weights& w, uint32_t keyTop,
                       uint32_t most, u64 target, uint32_t* at, u64* before) {
    constexpr int E = kVecElems<DT>;
    uint32_t* const low = hist;                        // counts, or the sums' low words
    uint32_t* const high = hist + kSampleBins;
    const int slice = kSampleBins / team.size, per = max(1, slice / kSampleThreads);
    uint32_t base = 0;
    u64 below = 0;
    int shift = max(0, 32 - __clz((int)most) - 11);
    for (;;) {
        const bool masses = BY_MASS && shift > 0;      // a bin of one value needs counts alone
        for (int i = threadIdx.x; i < kSampleBins * (masses ? 2 : 1); i += kSampleThreads) hist[i] = 0;
        __syncthreads();
        for (int s = 0; s < cols.steps; s++) {
            float f[E];
            cols.get(s, f);
#pragma unroll
            for (int j = 0; j < E; j++) {
                const uint32_t d = keyTop - key_of<DT>(f[j]);
                if (d > most || d < base) continue;
                const uint32_t bin = (d - base) >> shift;
                if (!masses) {
                    atomicAdd(&low[bin], 1u);
                } else {
                    const u64 v = w.fixed(f[j]);
                    const uint32_t old = atomicAdd(&low[bin], (uint32_t)v);
                    const uint32_t carry = (uint32_t)(v >> 32) + (old + (uint32_t)v < old ? 1u : 0u);
                    if (carry) atomicAdd(&high[bin], carry);
                }
            }
        }
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
        const u64 mine[4] = {all, 0, 0, 0};
        const u64(*box)[4] = exchange(sh, team, mine);
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

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) k_sample(const __grid_constant__ SampleArgs a) {
    pdl_begin();
    constexpr int E = kVecElems<DT>;
    extern __shared__ __align__(16) unsigned char dynamic[];
    __shared__ Shared sh;
    uint32_t* const hist = reinterpret_cast<uint32_t*>(dynamic);
    const uint32_t values = (uint32_t)__cvta_generic_to_shared(dynamic) + 2 * kSampleBins * 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Team team;
    team.size = a.cluster;
    team.rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    team.flip = team.flipFound = 0;
    const int row = (int)(blockIdx.x / (unsigned)a.cluster);
    const int columns = a.steps * kSampleThreads * E, c0 = team.rank * columns;
    if (threadIdx.x < 32) sh.powers[threadIdx.x] = kPowers[threadIdx.x];
    const float heat = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(heat > 0.0f);
    int k = greedy ? 1 : a.topK ? a.topK[row] : 0;
    if (k <= 0 || k >= a.vocab) k = a.vocab;           // no limit
    const float p = a.topP && !greedy ? a.topP[row] : 1.0f;
    const float least = a.minP && !greedy ? a.minP[row] : 0.0f;
    load_columns<DT>(a, row, c0, columns, values);
    const Columns<DT> cols(values, a.steps);

    // The largest value, and for topK the smallest maximum of disjoint groups.
    float top = -INFINITY;
    for (int s = 0; s < cols.steps; s++) {
        float f[E];
        cols.get(s, f);
#pragma unroll
        for (int j = 0; j < E; j++) top = fmaxf(top, f[j]);
    }
    float low[3];
    low[2] = top;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    low[1] = top;
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
    low[0] = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        low[1] = fminf(low[1], __shfl_xor_sync(~0u, low[1], o));
        low[2] = fminf(low[2], __shfl_xor_sync(~0u, low[2], o));
    }
    if (lane == 0) {
        sh.max[warp] = top;
        for (int i = 0; i < 3; i++) sh.low[i][warp] = low[i];
    }
    if (team.size > 1) meet(team);                     // every CTA of the cluster has started
    else __syncthreads();
    for (int i = 0; i < kWarps; i++) {
        top = fmaxf(top, sh.max[i]);
        for (int g = 0; g < 3; g++) low[g] = fminf(low[g], sh.low[g][i]);
    }
    {
        const u64 mine[4] = {__float_as_uint(top), __float_as_uint(low[0]), __float_as_uint(low[1]), __float_as_uint(low[2])};
        const u64(*box)[4] = exchange(sh, team, mine);
        for (int c = 0; c < team.size; c++) {
            top = fmaxf(top, __uint_as_float((uint32_t)box[c][0]));
            for (int g = 0; g < 3; g++) low[g] = fminf(low[g], __uint_as_float((uint32_t)box[c][1 + g]));
        }
    }
    if (top == -INFINITY) {                            // nothing to draw from
        if (threadIdx.x == 0 && team.rank == 0) {
            for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7FFFFFFF);
        }
        return;
    }

    Weights w;
    w.top = top;
    w.powers = sh.powers;
    {
        // log2(e) / temperature and what its rounding lost, kept off zero and infinity
        const float t = greedy ? 1.0f : heat, l2e = 1.44269504088896341f, l2eLow = 1.9259629911266175e-8f;
        const float r = __frcp_rn(t), c = __fmul_rn(l2e, r);
        w.ch = fminf(fmaxf(c, 1.17549435e-38f), 3.40282347e38f);
        w.cl = (__fmaf_rn(-c, t, l2e) + l2eLow) * r;
        if (w.ch != c || !(fabsf(w.cl) <= 1e-6f * c)) w.cl = 0.0f;
    }
    const uint32_t keyTop = key_of<DT>(top);
    // Distance of the smallest value that a value of at least x can have.
    const auto distance = [&](float x) { return x >= top ? 0u : keyTop - key_of<DT>(fmaxf(x, -3.40282347e38f)); };
    const bool limited = k < a.vocab, nucleus = p < 1.0f && k > 1;
    // The smallest value of weight `e`, with room for the roundings.
    const auto value_at = [&](float e) {
        const float x = top + (__log2f(e) - 0.01f) / w.ch;
        return x - 1e-5f * fabsf(x) - 1e-5f * fabsf(top);
    };

    // The sum of all weights: exactly, where topP is a share of it, or the draw goes through all.
    u64 total = 0, exact = 0;
    const auto sum_all = [&](bool exactly) {
        u64 s = 0, none = 0;
        for (int i = 0; i < cols.steps; i++) {
            float f[E];
            cols.get(i, f);
            if (exactly) {
#pragma unroll
                for (int j = 0; j < E; j++) s += w.fixed(f[j]);
            } else {
                float part = 0.0f;
#pragma unroll
                for (int j = 0; j < E; j++) {          // the largest apart: what is beside them may be small
                    part += f[j] == top ? 0.0f : w.rough(f[j]);
                    s += f[j] == top ? 1ull << kFix : 0ull;
                }
                s += __float2ull_rn(part * (float)(1ull << kFix));
            }
        }
        block_sums(sh, s, none);
        const u64 mine[4] = {s, 0, 0, 0};
        const u64(*box)[4] = exchange(sh, team, mine);
        u64 all = 0;
        for (int c = 0; c < team.size; c++) all += box[c][0];
        return all;
    };
    if (limited || least > 0.0f || !nucleus) total = sum_all(false);

    // What is kept: distances below `edge`, and the first `ties` columns at it.
    uint32_t edge = 0xFFFFFFFFu;
    u64 ties = 0, before = 0;
    bool cut = false;
    if (k == 1) {                    // the first of the largest
        edge = 0;
        ties = 1;
        cut = true;
    } else if (limited) {
        const int groups = team.size * kWarps;
        const float bound = k <= groups ? low[0] : k <= 4 * groups ? low[1] : k <= 32 * groups ? low[2] : -INFINITY;
        cut = search<DT, false>(sh, team, hist, cols, w, keyTop, distance(bound), (u64)k, &edge, &before);
        if (cut) ties = (u64)k - before;
    }
    if (nucleus) {
        uint32_t most;
        if (cut) {                   // the sum of the topK
            u64 s = 0, none = 0;
            for (int i = 0; i < cols.steps; i++) {
                float f[E];
                cols.get(i, f);
#pragma unroll
                for (int j = 0; j < E; j++)
                    if (keyTop - key_of<DT>(f[j]) < edge) s += w.fixed(f[j]);
            }
            block_sums(sh, s, none);
            const u64 mine[4] = {s, 0, 0, 0};
            const u64(*box)[4] = exchange(sh, team, mine);
            exact = ties * w.fixed(value_of<DT>(keyTop - edge));
            for (int c = 0; c < team.size; c++) exact += box[c][0];
            most = edge;
        } else {                     // weights below (1 - p) of the mean are outside, all of them together
            exact = sum_all(true);
            if (total == 0) total = exact;
            most = distance(value_at((1.0f - fmaxf(p, 0.0f)) * 0.99f * ((float)exact * 0x1p-44f) / (float)a.vocab));
        }
        const u64 goal = max(1ull, (u64)ceil((double)fmaxf(p, 0.0f) * (double)exact));
        uint32_t at;
        if (search<DT, true>(sh, team, hist, cols, w, keyTop, most, goal, &at, &before)) {
            const u64 one = max(1ull, w.fixed(value_of<DT>(keyTop - at)));
            const u64 n = (goal - before + one - 1) / one;
            ties = cut && at == edge ? min(ties, n) : n;
            edge = at;
            cut = true;
        }
    }
    if (total == 0) total = exact;
    const u64 floorWeight = least > 0.0f ? (u64)ceil((double)fminf(least, 1.0f) * (double)(1ull << kFix)) : 0;
    const float floorValue = floorWeight ? value_at(fminf(least, 1.0f)) : -INFINITY;

    // Weights kept by every warp, its ties at the edge aside.
    u64 atEdge = cut ? w.fixed(value_of<DT>(keyTop - edge)) : 0;
    if (atEdge < floorWeight) atEdge = 0;
    const auto kept = [&](float x, bool* tie) {
        const uint32_t d = keyTop - key_of<DT>(x);
        *tie = cut && d == edge;
        if ((cut && d >= edge) || x < floorValue) return 0ull;
        const u64 v = w.fixed(x);
        return v >= floorWeight ? v : 0ull;
    };
    u64 sum = 0, count = 0;
    for (int s = 0; s < cols.steps; s++) {
        float f[E];
        cols.get(s, f);
#pragma unroll
        for (int j = 0; j < E; j++) {
            bool tie;
            sum += kept(f[j], &tie);
            count += tie;
        }
    }
    u64 blockSum = sum, blockCount = count;
    block_sums(sh, blockSum, blockCount);              // leaves every warp's sums in sh.warp
    const u64 mine[4] = {blockSum, blockCount, 0, 0};
    const u64(*box)[4] = exchange(sh, team, mine);
    // From here on nothing touches another CTA's memory.
    if (threadIdx.x == 0) {
        u64 all = 0, ahead = 0, left = ties, leftHere = ties;
        for (int c = 0; c < team.size; c++) {
            const u64 n = min(left, box[c][1]);
            if (c == team.rank) {
                ahead = all;
                leftHere = left;
            }
            all += box[c][0] + n * atEdge;
            left -= n;
        }
        const float u = a.uniform[row];
        u64 goal = u > 0.0f ? (u64)((double)u * (double)all) : 0;
        goal = min(goal, all - 1);
        sh.owner = -1;
        for (int i = 0; i < kWarps && goal >= ahead; i++) {
            const u64 n = min(leftHere, sh.warp[1][i]), here = sh.warp[0][i] + n * atEdge;
            if (goal < ahead + here) {
                sh.owner = i;
                sh.target = goal - ahead;
                sh.box[0][0][0] = leftHere;            // nobody reads the boxes any more but this thread
                break;
            }
            ahead += here;
            leftHere -= n;
        }
    }
    __syncthreads();
    if (warp != sh.owner) return;

    // The warp whose columns hold the token goes through them in order.
    u64 goal = sh.target, left = sh.box[0][0][0];
    for (int s = 0; s < cols.steps; s++) {
        float f[E];
        cols.get(s, f);
        u64 v[E], own = 0, n = 0;
        bool tie[E];
#pragma unroll
        for (int j = 0; j < E; j++) {
            v[j] = kept(f[j], &tie[j]);
            own += v[j];
            n += tie[j];
        }
        u64 runTies = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(~0u, runTies, o);
            if (lane >= o) runTies += x;
        }
        u64 mineLeft = left - min(left, runTies - n);  // ties that may still be kept, from this lane on
        own += min(mineLeft, n) * atEdge;
        u64 run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += x;
        }
        const bool here = goal >= run - own && goal < run;
        if (here) {
            u64 ahead = run - own;
            int pick = 0;
            float x = f[0];
            bool done = false;
#pragma unroll
            for (int j = 0; j < E; j++) {
                u64 e = v[j];
                if (tie[j] && mineLeft > 0) {
                    mineLeft--;
                    e = atEdge;
                }
                ahead += e;
                if (!done && goal < ahead) {
                    done = true;
                    pick = j;
                    x = f[j];
                }
            }
            const int token = c0 + cols.first + s * 32 * E + pick;
            for (int o = 0; o < a.nOut; o++) a.tokens[o][row] = token;
            if (a.logprob) {
                const float z = x == top ? 0.0f : greedy ? x - top : (x - top) / heat;
                a.logprob[row] = z - log1pf((float)(total - (1ull << kFix)) * 0x1p-44f);
            }
        }
        if (__any_sync(~0u, here)) return;
        goal -= __shfl_sync(~0u, run, 31);
        left -= min(left, __shfl_sync(~0u, runTies, 31));
    }
}

template <int DT>
cudaError_t sample_launch(const SampleArgs& a, cudaStream_t s) {
    const size_t smem = 2 * kSampleBins * 4 + (size_t)a.steps * kSampleThreads * 16;
    if (smem > 32 * 1024) {
        // one value for every launch, as host threads share the kernel's limit
        const cudaError_t e = cudaFuncSetAttribute(k_sample<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != cudaSuccess) return e;
    }
    NormShape sh = {};
    sh.threads = kSampleThreads;
    sh.cluster = a.cluster;
    return norm_launch(k_sample<DT>, (unsigned)a.rows * (unsigned)a.cluster, sh, smem, s, a);
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
