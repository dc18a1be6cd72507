// k_moe_route.cu -- the router of a mixture of experts: logits, the topK best experts of every token
// and their weights.
//
//   l_te = sum_j x_tj router_ej,  score = l + bias
//   ids = the topK largest scores of the token, largest first, ties to the lower index
//   weight = exp(l_id) / sum of exp(l) over the chosen, or over all experts
//
// Two experts' scores may lie next to one another, and the choice between them is an integer.  So the
// logits come as a value and a rest, with a bound on their error: a few products at a time are added in
// fp32, off by at most a unit u = 2^-24 of their magnitudes for each addition, and their sums error-free.
// Where that leaves open which of two scores is the larger, and one of the two is chosen, both logits
// are computed anew with every product and sum as a value and its error, some 2^-45 of the magnitudes
// off.  No fp64: its rate here is a 64th of fp32's (256 x 4096 of 128 experts with the choice in fp64:
// 164 us, 30 as it is).
//
// A cluster of CTAs takes a few tokens, each CTA a share of the experts.  Few tokens: up to four a
// cluster, a warp takes an expert, its lanes stride along the row (1 x 4096 of 64: 6 us, most of it launch and
// latency).  More: eight tokens, a warp four of them by four experts, so that what it loads serves four
// times (256 x 4096 of 128, fp32 router: 30 us, of which the loop over the columns takes 15, bound by its
// instructions, near 390 a warp and 256 columns, and logits computed anew 7; tiles staged in shared
// memory and read by threads that share rows 67, the same warp's tiles from stages copied ahead 37).  All 128
// registers are taken: 28 to 64 bytes a thread are spilled around that loop, 236 to 284 of unaligned rows.  The
// logits go to the CTA that picks for their token.
#include "moe.h"
#include "norm_stage.cuh"

namespace vc {

namespace {

constexpr float kUnit = 5.9604644775390625e-8f;        // 2^-24

// E consecutive values of a row from element e on, `left` of them inside the row (the rest zero).
template <int DT, int E, bool ALIGNED>
__device__ __forceinline__ void load_row(const void* row, int e, int left, float (&f)[E]) {
    constexpr int ESZ = DTypeOf<DT>::size, PER = 16 / ESZ;
    if (ALIGNED) {
#pragma unroll
        for (int i = 0; i < E; i += PER) {
            float part[PER];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (i < left) v = *reinterpret_cast<const uint4*>((const char*)row + (size_t)(e + i) * ESZ);
            widen_vec<DT>(v, part);
#pragma unroll
            for (int j = 0; j < PER; j++) f[i + j] = part[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i++) {
            f[i] = 0.0f;
            if (i >= left) continue;
            if (DT == kF32) f[i] = ((const float*)row)[e + i];
            else f[i] = widen16<DT>(((const uint16_t*)row)[e + i]);
        }
    }
}

// s + c stays the sum of everything added, c what s's roundings lost.
__device__ __forceinline__ void add_exactly(float& s, float& c, float x) {
    const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}
// The same sum with c below half a unit of s, so that sums compare by s, then by c.  A sum that is not
// finite has no rest.
__device__ __forceinline__ float2 settle(float s, float c) {
    const float t = __fadd_rn(s, c), b = __fsub_rn(t, s);
    const float rest = __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(c, b));
    return isfinite(s) ? make_float2(t, rest + 0.0f) : make_float2(s, 0.0f);
}
// The lanes' sums together.
__device__ __forceinline__ float2 warp_total(float s, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float s2 = __shfl_xor_sync(~0u, s, o), c2 = __shfl_xor_sync(~0u, c, o);
        add_exactly(s, c, s2);
        c = __fadd_rn(c, c2);
    }
    // lanes added in different orders: one of them speaks for all
    return settle(__shfl_sync(~0u, s, 0), __shfl_sync(~0u, c, 0));
}

// A warp's part of a logit, error-free products added error-free in two chains: stretches of 256 columns,
// dealt to half of the CTA's warps.
template <int DT, int WT, bool ALIGNED, int THREADS>
__device__ __noinline__ float2 exact_part(const char* x, const char* w, int hidden) {
    constexpr int E = 8;
    float s[2] = {0.0f, 0.0f}, c[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int j = (int)threadIdx.x % (THREADS / 2) * E; j < hidden; j += THREADS / 2 * E) {
        float f[E], v[E];
        const int left = min(E, hidden - j);
        load_row<WT, E, ALIGNED>(w, j, left, f);
        load_row<DT, E, ALIGNED>(x, j, left, v);
#pragma unroll
        for (int i = 0; i < E; i++) {
            const float p = __fmul_rn(v[i], f[i]);
            add_exactly(s[i & 1], c[i & 1], p);
            c[i & 1] = __fadd_rn(c[i & 1], __fmaf_rn(v[i], f[i], -p));
        }
    }
    add_exactly(s[0], c[0], s[1]);
    return warp_total(s[0], __fadd_rn(c[0], c[1]));
}

// Integers in the order of the choice: a larger score has the larger (x, y); a NaN comes last, (0, 0)
// behind it.
__device__ __forceinline__ uint32_t order(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint2 key_of(float2 v) {
    return v.x != v.x ? make_uint2(1u, 0u) : make_uint2(order(v.x), order(v.y));
}

__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
__device__ __forceinline__ float2 value_of(uint2 key) {
    return key.x == 1u ? make_float2(__int_as_float(0x7FFFFFFF), 0.0f) : make_float2(value_of(key.x), value_of(key.y));
}

// What a CTA keeps of the tokens that it picks for: [token][expert] logits, scores' keys and the logits'
// bounds.
struct Picks {
    float2* logit;
    uint2* key;
    float* error;
};
constexpr int kRedo = 32;            // logits computed anew at a time
struct Redo {
    int count;
    uint16_t entry[kRouteFew * VCOMM_MAX_EXPERTS];     // token slot * experts + expert
    float2 part[kRedo][kRouteTileThreads / 64];
    int id[kRouteTile][VCOMM_MAX_TOPK];                // the choices as they stand
};
__host__ __device__ constexpr int pick_bytes(int tokens, int experts) { return tokens * experts * 20; }
__device__ __forceinline__ Picks picks_at(unsigned char* smem, int tokens, int experts) {
    Picks p;
    p.logit = reinterpret_cast<float2*>(smem);
    p.key = reinterpret_cast<uint2*>(p.logit + (size_t)tokens * experts);
    p.error = reinterpret_cast<float*>(p.key + (size_t)tokens * experts);
    return p;
}
__device__ __forceinline__ void send(const Picks& p, size_t at, int rank, int cluster, float2 logit, float error) {
    if (cluster == 1) {
        p.logit[at] = logit;
        p.error[at] = error;
        return;
    }
    st_cluster(&p.logit[at].x, rank, __float_as_uint(logit.x));
    st_cluster(&p.logit[at].y, rank, __float_as_uint(logit.y));
    st_cluster(&p.error[at], rank, __float_as_uint(error));
}

// The score of an expert: logit + bias.
__device__ __forceinline__ float2 score_of(const RouteArgs& a, const float2* l, int e) {
    float2 v = l[e];
    if (!a.bias) return v;
    add_exactly(v.x, v.y, a.bias[e]);
    return settle(v.x, v.y);
}

// One warp's choice for the token of slot `at`, into redo.id, and the logits that it hangs on and that
// are not exact yet, into redo.entry.
__device__ void choose(const RouteArgs& a, const Picks& all, Redo& redo, int at) {
    const int lane = threadIdx.x & 31, E = a.experts;
    const float2* const l = all.logit + (size_t)at * E;
    uint2* const key = all.key + (size_t)at * E;
    const float* const error = all.error + (size_t)at * E;
    int* const id = redo.id[at];
    const int more = min(a.topK + 1, E);               // one more than are chosen, to see how near it is
    float worst = 0.0f;
    for (int e = lane; e < E; e += 32) {
        key[e] = key_of(score_of(a, l, e));
        worst = fmaxf(worst, error[e]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) worst = fmaxf(worst, __shfl_xor_sync(~0u, worst, o));
    unsigned taken = 0;                                // bit b: expert 32 b + lane is chosen
    unsigned long long near = 0;                       // bit k: choice k and the next may change places
    float2 last = make_float2(0.0f, 0.0f);
    for (int k = 0; k < more; k++) {
        uint2 best = make_uint2(0u, 0u);
        int e0 = 0x7FFFFFFF;
        for (int e = lane, b = 0; e < E; e += 32, b++) {
            const uint2 v = key[e];
            const bool more = v.x > best.x || (v.x == best.x && v.y > best.y);
            if (more && !(taken >> b & 1)) {
                best = v;
                e0 = e;
            }
        }
        const uint32_t hi = __reduce_max_sync(~0u, best.x);
        const uint32_t lo = __reduce_max_sync(~0u, best.x == hi ? best.y : 0u);
        const int c = __reduce_min_sync(~0u, best.x == hi && best.y == lo ? e0 : 0x7FFFFFFF);
        const float2 score = value_of(make_uint2(hi, lo));
        if (k > 0 && fabsf((last.x - score.x) + (last.y - score.y)) <= 2.0f * worst) near |= 1ull << (k - 1);
        last = score;
        if (lane == (c & 31)) taken |= 1u << (c >> 5);
        if (k < a.topK && lane == 0) id[k] = c;
    }
    __syncwarp();
    if (!near || worst == 0.0f) return;
    unsigned flags = 0;                                // bit b: expert 32 b + lane may change places with a chosen one
    for (int k = 0; k < a.topK; k++) {
        // what is that near a choice is behind or before a neighbour that is nearer still
        if (!((near | near << 1) >> k & 1)) continue;
        const int c = id[k];
        const float2 chosen = value_of(key[c]);
        bool unsure = false;
        for (int e = lane; e < E; e += 32) {
            const float both = error[e] + error[c];
            const float2 other = value_of(key[e]);
            if (e == c || !(both > 0.0f && fabsf((other.x - chosen.x) + (other.y - chosen.y)) <= both)) continue;
            unsure = true;
            flags |= 1u << (e >> 5);
        }
        if (__any_sync(~0u, unsure) && lane == (c & 31)) flags |= 1u << (c >> 5);
    }
    for (; flags; flags &= flags - 1) {
        const int e = 32 * (__ffs(flags) - 1) + lane;
        if (error[e] > 0.0f) redo.entry[atomicAdd(&redo.count, 1)] = (uint16_t)(at * E + e);
    }
}

// All threads of a CTA pick for its `mine` tokens, whose rows are row_of(slot), < 0 for none.
template <int DT, int WT, bool ALIGNED, int THREADS, typename RowOf>
__device__ __forceinline__ void pick(const RouteArgs& a, const Picks& all, Redo& redo, int mine, RowOf row_of) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = THREADS / 32, E = a.experts;
    for (;;) {
        if (threadIdx.x == 0) redo.count = 0;
        __syncthreads();
        for (int at = warp; at < mine; at += warps)
            if (row_of(at) >= 0) choose(a, all, redo, at);
        __syncthreads();
        const int n = redo.count;
        if (n == 0) break;
        // These logits anew, by all warps together; a bound of 0 marks one that is as good as it gets, so
        // this ends.
        for (int i0 = 0; i0 < n; i0 += kRedo) {
            const int some = min(kRedo, n - i0);
            for (int i = warp / (warps / 2); i < some; i += 2) {
                const int entry = redo.entry[i0 + i], at = entry / E, e = entry % E;
                const float2 v = exact_part<DT, WT, ALIGNED, THREADS>(
                    (const char*)a.x + (size_t)row_of(at) * a.rowStride * DTypeOf<DT>::size,
                    (const char*)a.router + (size_t)e * a.hidden * DTypeOf<WT>::size, a.hidden);
                if (lane == 0) redo.part[i][warp % (warps / 2)] = v;
            }
            __syncthreads();
            if ((int)threadIdx.x < some) {
                float2 v = redo.part[threadIdx.x][0];
                for (int w = 1; w < warps / 2; w++) {
                    const float2 p = redo.part[threadIdx.x][w];
                    add_exactly(v.x, v.y, p.x);
                    v.y = __fadd_rn(v.y, p.y);
                }
                const int entry = redo.entry[i0 + threadIdx.x];
                all.logit[entry] = settle(v.x, v.y);
                all.error[entry] = 0.0f;
            }
            __syncthreads();
        }
    }
    for (int at = warp; at < mine; at += warps) {
        const int row = row_of(at);
        if (row < 0) continue;
        // The weights: differences from the largest chosen logit, a NaN's wherever there is one.
        const float2* const l = all.logit + (size_t)at * E;
        const int id = lane < a.topK ? redo.id[at][lane] : 0;
        const float2 own = l[id];
        float top = lane < a.topK ? own.x : -INFINITY, sum = 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float other = __shfl_xor_sync(~0u, top, o);
            top = other > top || other != other ? other : top;
        }
        const auto share = [&](float2 v) { return expf((v.x - top) + v.y); };
        if (a.normalize) {
            sum = lane < a.topK ? share(own) : 0.0f;
        } else {
            for (int e = lane; e < E; e += 32) sum += share(l[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane < a.topK) {
            a.ids[(size_t)row * a.topK + lane] = id;
            a.weights[(size_t)row * a.topK + lane] = share(own) / sum;
        }
    }
}

// ---- up to four tokens a cluster: a warp an expert, lanes along its row --------------------------

template <int DT, int WT, int TOKENS, bool ALIGNED>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route_few(const __grid_constant__ RouteArgs a) {
    pdl_begin();
    constexpr int E = 8, STEPS = TOKENS == 1 ? 4 : 2;  // steps whose loads are under way together
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Redo redo;
    const Picks picks = picks_at(smem, TOKENS, a.experts);       // of the first CTA
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRouteThreads / 32;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    if (a.cluster > 1) cluster_arrive();
    bool started = a.cluster == 1;
    const int row0 = (int)(blockIdx.x / (unsigned)a.cluster) * TOKENS;
    const int last = min(a.experts, (rank + 1) * a.share);
    for (int e = rank * a.share + warp; e < last; e += warps) {
        const char* w = (const char*)a.router + (size_t)e * a.hidden * DTypeOf<WT>::size;
        float s[TOKENS], c[TOKENS], m[TOKENS];         // m: the products' magnitudes
#pragma unroll
        for (int t = 0; t < TOKENS; t++) s[t] = c[t] = m[t] = 0.0f;
        for (int j0 = lane * E; j0 < a.hidden; j0 += 32 * E * STEPS) {
            float f[STEPS][E];
#pragma unroll
            for (int i = 0; i < STEPS; i++) {
                const int j = j0 + i * 32 * E;
                load_row<WT, E, ALIGNED>(w, j, max(0, min(E, a.hidden - j)), f[i]);
            }
#pragma unroll
            for (int t = 0; t < TOKENS; t++) {
                const int row = min(row0 + t, a.rows - 1);
                const char* x = (const char*)a.x + (size_t)row * a.rowStride * DTypeOf<DT>::size;
                float v[STEPS][E];
#pragma unroll
                for (int i = 0; i < STEPS; i++) {
                    const int j = j0 + i * 32 * E;
                    load_row<DT, E, ALIGNED>(x, j, max(0, min(E, a.hidden - j)), v[i]);
                }
#pragma unroll
                for (int i = 0; i < STEPS; i++) {
                    float p = v[i][0] * f[i][0];
#pragma unroll
                    for (int k = 1; k < E; k++) p = fmaf(v[i][k], f[i][k], p);
#pragma unroll
                    for (int k = 0; k < E; k++) m[t] = fmaf(fabsf(v[i][k]), fabsf(f[i][k]), m[t]);
                    add_exactly(s[t], c[t], p);
                }
            }
        }
        if (!started) {                                // every CTA of the cluster has
            cluster_wait();
            started = true;
        }
#pragma unroll
        for (int t = 0; t < TOKENS; t++) {
            const float2 l = warp_total(s[t], c[t]);
            float off = m[t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) off += __shfl_xor_sync(~0u, off, o);
            // eight roundings a product, with room for those of m itself
            if (lane == 0) send(picks, (size_t)t * a.experts + e, 0, a.cluster, l, off * (10.0f * kUnit));
        }
    }
    if (a.cluster > 1) {
        if (!started) cluster_wait();
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    pick<DT, WT, ALIGNED, kRouteThreads>(a, picks, redo, min(TOKENS, a.rows - row0), [&](int at) { return row0 + at; });
}

// ---- more: tiles of eight tokens and thirty-two experts -----------------------------------------

constexpr int kSide = 4;             // a warp's tile: four tokens by four experts, lanes along their rows
constexpr int kPass = kRouteTileThreads / 32 / (kRouteTile / kSide) * kSide;   // experts of a CTA at a time
// Vectors of eight products that a lane adds, in two fp32 chains, before the error-free sum: 17 roundings a
// product, with one vector five.  Ids do not depend on it; a weight whose logit is not computed anew is off by up to
// that many units of its products' magnitudes (10^-7 of the norm measured, 256 x 4096 of 128), and one vector would
// take 31.2 us there in place of 30.2, 34.5 in place of 31.9 for 1024 x 2048 of 64.
constexpr int kFold = 4;

// How far off a logit of a tile is at most, from the squared norms of its token and expert: seventeen
// roundings a product, and the magnitudes' sum is at most the product of the norms.  Squares below 2^-149 are
// lost: with room for them no norm is too small, and none is zero beside an infinite one.  Scores closer
// than 10^-24 are not told apart, which leaves tokens and experts of zeros at that.
__device__ __noinline__ float bound_of(float token, float expert, int hidden) {
    const float lost = (float)hidden * 0x1p-149f;
    const float off = 20.0f * kUnit * sqrtf(token + lost) * sqrtf(expert + lost);
    return off < 0x1p-81f ? 0.0f : off;
}

template <int DT, int WT, bool ALIGNED>
__global__ void __launch_bounds__(kRouteTileThreads, 1) k_moe_route(const __grid_constant__ RouteArgs a) {
    pdl_begin();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Redo redo;
    __shared__ float tokenNorm[kRouteTile];             // squared
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
    const int mine = (kRouteTile + a.cluster - 1) / a.cluster;   // tokens that a CTA picks for
    const Picks picks = picks_at(smem, mine, a.experts);
    const int row0 = (int)(blockIdx.x / (unsigned)a.cluster) * kRouteTile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.cluster > 1) cluster_arrive();
    const int last = min(a.experts, (rank + 1) * a.share);
    const int t0 = warp % (kRouteTile / kSide) * kSide;
    const char* x[kSide];
#pragma unroll
    for (int t = 0; t < kSide; t++) x[t] = (const char*)a.x + (size_t)min(row0 + t0 + t, a.rows - 1) * a.rowStride * DTypeOf<DT>::size;
    bool started = a.cluster == 1;
    const int group = warp / (kRouteTile / kSide);
    for (int pass = rank * a.share; pass < last; pass += kPass) {
        const int e0 = pass + group * kSide;
        const char* w[kSide];
#pragma unroll
        for (int e = 0; e < kSide; e++) w[e] = (const char*)a.router + (size_t)min(e0 + e, last - 1) * a.hidden * DTypeOf<WT>::size;
        float s[kSide][kSide] = {}, c[kSide][kSide] = {};
        float2 p[kSide][kSide] = {}, square[kSide] = {}, token = {};
        int folded = 0;
        for (int j = lane * 8; j < a.hidden; j += 256) {
            const int left = min(8, a.hidden - j);
            float f[kSide][8], v[kSide][8];
#pragma unroll
            for (int e = 0; e < kSide; e++) load_row<WT, 8, ALIGNED>(w[e], j, left, f[e]);
#pragma unroll
            for (int t = 0; t < kSide; t++) {
                load_row<DT, 8, ALIGNED>(x[t], j, left, v[t]);
                if (group != t) continue;              // the token's norm, by one warp
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 two = make_float2(v[t][i], v[t][i + 1]);
                    token = fma2(two, two, token);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
#pragma unroll
                for (int e = 0; e < kSide; e++) {
                    const float2 two = make_float2(f[e][i], f[e][i + 1]);
                    square[e] = fma2(two, two, square[e]);
#pragma unroll
                    for (int t = 0; t < kSide; t++) p[t][e] = fma2(make_float2(v[t][i], v[t][i + 1]), two, p[t][e]);
                }
            }
            if (++folded % kFold) continue;
#pragma unroll
            for (int t = 0; t < kSide; t++)
#pragma unroll
                for (int e = 0; e < kSide; e++) {
                    add_exactly(s[t][e], c[t][e], __fadd_rn(p[t][e].x, p[t][e].y));
                    p[t][e] = make_float2(0.0f, 0.0f);
                }
        }
        // The lanes' sums, halving the tile with every step: lane (t, e) ends with logit (t, e), and both
        // halves of the warp with the same.
        float sum[kSide * kSide], rest[kSide * kSide];
#pragma unroll
        for (int i = 0; i < kSide * kSide; i++) {
            add_exactly(s[i / kSide][i % kSide], c[i / kSide][i % kSide], __fadd_rn(p[i / kSide][i % kSide].x, p[i / kSide][i % kSide].y));
            sum[i] = s[i / kSide][i % kSide];
            rest[i] = c[i / kSide][i % kSide];
        }
#pragma unroll
        for (int half = kSide * kSide / 2; half > 0; half >>= 1) {
            const bool upper = (lane & half) != 0;
#pragma unroll
            for (int i = 0; i < half; i++) {
                const float sGive = upper ? sum[i] : sum[i + half], cGive = upper ? rest[i] : rest[i + half];
                sum[i] = upper ? sum[i + half] : sum[i];
                rest[i] = upper ? rest[i + half] : rest[i];
                const float s2 = __shfl_xor_sync(~0u, sGive, half), c2 = __shfl_xor_sync(~0u, cGive, half);
                add_exactly(sum[i], rest[i], s2);
                rest[i] = __fadd_rn(rest[i], c2);
            }
        }
        const float s2 = __shfl_xor_sync(~0u, sum[0], 16), c2 = __shfl_xor_sync(~0u, rest[0], 16);
        add_exactly(sum[0], rest[0], s2);
        rest[0] = __fadd_rn(rest[0], c2);
        float norm = 0.0f;           // of expert e0 + lane % 4, squared
#pragma unroll
        for (int e = 0; e < kSide; e++) {
            float q = square[e].x + square[e].y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
            if ((lane & 3) == e) norm = q;
        }
        float q = token.x + token.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
        if (pass == rank * a.share && group < kSide && lane == 0) tokenNorm[t0 + group] = q;
        __syncthreads();
        if (!started) {                                // every CTA of the cluster has
            cluster_wait();
            started = true;
        }
        // bits 3 and 2 of the lane chose the token, bits 1 and 0 the expert
        const int t = t0 + (lane >> 2 & 3), e = e0 + (lane & 3);
        if (lane < 16 && row0 + t < a.rows && e < last) {
            send(picks, (size_t)(t / a.cluster) * a.experts + e, t % a.cluster, a.cluster, settle(sum[0], rest[0]),
                 bound_of(tokenNorm[t], norm, a.hidden));
        }
    }
    if (a.cluster > 1) {
        if (!started) cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    pick<DT, WT, ALIGNED, kRouteTileThreads>(a, picks, redo, mine, [&](int at) {
        const int t = at * a.cluster + rank;
        return t < kRouteTile && row0 + t < a.rows ? row0 + t : -1;
    });
}

template <typename K>
cudaError_t route_start(K kernel, const RouteArgs& a, int threads, int groups, size_t smem, cudaStream_t s) {
    if (smem > 32 * 1024) {
        // one value for every launch, as host threads share the kernel's limit
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteMaxSmem);
        if (e != cudaSuccess) return e;
    }
    NormShape sh = {};
    sh.threads = threads;
    sh.cluster = a.cluster;
    return norm_launch(kernel, (unsigned)(groups * a.cluster), sh, smem, s, a);
}
template <int DT, int WT, bool ALIGNED>
cudaError_t route_launch(const RouteArgs& a, cudaStream_t s) {
    if (!a.few) {
        return route_start(k_moe_route<DT, WT, ALIGNED>, a, kRouteTileThreads, (a.rows + kRouteTile - 1) / kRouteTile,
                           pick_bytes((kRouteTile + a.cluster - 1) / a.cluster, a.experts), s);
    }
    if (a.rows == 1) return route_start(k_moe_route_few<DT, WT, 1, ALIGNED>, a, kRouteThreads, 1, pick_bytes(1, a.experts), s);
    if (a.rows == 2) return route_start(k_moe_route_few<DT, WT, 2, ALIGNED>, a, kRouteThreads, 1, pick_bytes(2, a.experts), s);
    return route_start(k_moe_route_few<DT, WT, 4, ALIGNED>, a, kRouteThreads, (a.rows + 3) / 4, pick_bytes(4, a.experts), s);
}
template <int DT, int WT>
cudaError_t route_launch_a(const RouteArgs& a, cudaStream_t s) {
    return a.aligned ? route_launch<DT, WT, true>(a, s) : route_launch<DT, WT, false>(a, s);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, vDataType_t dt, cudaStream_t s) {
    switch (dt) {
    case vFloat32: return route_launch_a<kF32, kF32>(a, s);
    case vFloat16: return a.routerF32 ? route_launch_a<kF16, kF32>(a, s) : route_launch_a<kF16, kF16>(a, s);
    case vBFloat16: return a.routerF32 ? route_launch_a<kBF16, kF32>(a, s) : route_launch_a<kBF16, kBF16>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vc
