// moe.cpp -- entry points of the mixture-of-experts operators.
#include <cstdio>
#include <vector>

#include "entry.h"
#include "moe.h"

namespace {

struct Moe {
    vMoeDesc_t d;                    // strides filled in
    int esz;
    int share;                       // experts of a rank
    size_t slots;
};

vResult_t check_moe(const vMoeDesc_t* desc, int nRanks, Moe* m) {
    if (!desc) return vInvalidArgument;
    vMoeDesc_t& d = m->d;
    d = *desc;
    if (!is_float(d.datatype)) return vInvalidArgument;
    if (d.routerType != vFloat32 && d.routerType != d.datatype) return vInvalidArgument;
    if (d.rows > VCOMM_MAX_MOE_ROWS || d.hidden > VCOMM_MAX_HIDDEN || d.ffn > VCOMM_MAX_HIDDEN) return vInvalidArgument;
    if (d.experts < 1 || d.experts > VCOMM_MAX_EXPERTS) return vInvalidArgument;
    if (d.topK < 1 || d.topK > VCOMM_MAX_TOPK || d.topK > d.experts) return vInvalidArgument;
    for (size_t* s : {&d.rowStride, &d.recvStride}) {
        if (*s == 0) *s = d.hidden;
        if (*s < d.hidden || *s > ((size_t)1 << 62) / (4 * VCOMM_MAX_MOE_ROWS)) return vInvalidArgument;
    }
    m->esz = (int)vc::dtype_size(d.datatype);
    m->share = (d.experts + nRanks - 1) / nRanks;
    m->slots = d.rows * (size_t)d.topK;
    return vSuccess;
}

// Bytes of the workspace's parts, in their order: act, y, the tiles' counters.
struct Layout {
    size_t act, y, done;
    explicit Layout(const Moe& m)
        : act((m.slots * vc::moe_act_stride((int)m.d.ffn) * 4 + 255) / 256 * 256),
          y((m.slots * vc::moe_y_stride((int)m.d.hidden) * 4 + 255) / 256 * 256),
          done((m.d.hidden + vc::kMoeTile - 1) / vc::kMoeTile * 4) {}
    size_t total() const { return act + y + done + 16; }
};

// Shapes of the tensor core launches.
vc::MoeTiles moe_tiles(const vc::ExpertsArgs& a, int smCount) {
    vc::MoeTiles t = {};
    const int slots = a.rows * a.topK;
    // Most experts' tokens in one group: a second one reads the expert's weights again.
    const double mean = (double)slots / a.experts;
    t.tokens = a.rows <= 16 || mean <= 6 ? 16 : a.rows <= 32 || mean <= 18 ? 32 : 64;
    const int groups = std::min(a.experts, slots);
    const auto shape = [&](int tiles, int columns, int* split, int* grid) {
        // rounds of tiles by the stages of one, and one more for a sum that is put together
        const int chunks = (columns + 127) / 128;
        double least = 0;
        for (const int s : {1, 2, 4}) {
            if (s > 1 && (t.tokens > 16 || s > chunks)) break;
            const int clusters = std::max(1, smCount / s);
            const double cost = (double)((groups * tiles + clusters - 1) / clusters) * ((double)((chunks + s - 1) / s) + (s > 1));
            if (s > 1 && cost >= least) continue;
            least = cost;
            *split = s;
            *grid = std::min(clusters, std::max(1, (groups + slots / t.tokens) * tiles)) * s;
        }
    };
    shape((a.ffn + 63) / 64, a.hidden, &t.splitUp, &t.gridUp);
    shape((a.hidden + 127) / 128, a.ffn, &t.splitDown, &t.gridDown);
    // All stages that an SM has room for: its registers hold one CTA of either launch.  (72 registers a thread
    // and 124 and 100 KiB hold one of each, the second's first weights on their way while the first runs, but
    // spill: one token on 4 of 64 experts of 2048 x 1024 26.7 us, 26.2 so; on 8 of 128 of 4096 x 1536 71.4 and
    // 69.0; on 2 of 8 of 6144 x 4096 74.7 and 83.7.)
    const auto stages = [&](bool up, int split) {
        int n = 2;
        while (n < vc::kMoeMaxStages && vc::moe_tiles_smem(a.experts, slots, t.tokens, up, split, n + 1) <= vc::kMoeMaxSmem) n++;
        return n;
    };
    t.stagesUp = stages(true, t.splitUp);
    t.stagesDown = stages(false, t.splitDown);
    t.combineHere = a.rows <= 4;
    return t;
}

vResult_t route(const vMoeDesc_t* desc, const void* x, const void* router, const float* bias, int* ids, float* weights,
                vcomm_t c, cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Moe m;
    if ((r = check_moe(desc, v.nRanks, &m)) != vSuccess) return r;
    if (v.grouping) {
        const vMoeDesc_t d = *desc;
        return vc::comm_record(c, [=]() {
            return guarded([&]() { return route(&d, x, router, bias, ids, weights, c, stream); });
        });
    }
    if (m.d.rows == 0) return vSuccess;
    if (m.d.hidden == 0) return vInvalidArgument;
    const size_t wsz = vc::dtype_size(m.d.routerType);
    if (!x || !at(x, m.esz) || !router || !at(router, wsz) || !at(bias, 4)) return vInvalidArgument;
    if (!ids || !at(ids, 4) || !weights || !at(weights, 4)) return vInvalidArgument;
    vc::RouteArgs a;
    a.x = x;
    a.router = router;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.rowStride = m.d.rowStride;
    a.rows = (int)m.d.rows;
    a.hidden = (int)m.d.hidden;
    a.experts = m.d.experts;
    a.topK = m.d.topK;
    // An expert for every warp, or a pass of experts for every CTA, as far as a cluster goes.  A warp an
    // expert for up to four tokens, and for more while there is an SM for every CTA and no warp has more than two
    // experts (bf16, us against tiles: 32 x 4096 of 128 experts 18 against 22.5, 64 x 2048 of 64 10 against 14, 5 x
    // 4096 of 16 9 against 19; but 64 x 4096 of 256 54 against 28, 128 x 8192 fp32 of 128 89 against 55).  Tiles:
    // larger clusters only where that leaves no SM twice as much to do (64 x 4096 of 256: 28 against 44).
    const auto cluster = [&](int each, int most) {
        int c = 1;
        while (c < most && c * each < a.experts) c *= 2;
        return c;
    };
    const int warps = vc::kRouteThreads / 32, fours = (a.rows + 3) / 4, tiles = (a.rows + vc::kRouteTile - 1) / vc::kRouteTile;
    a.cluster = cluster(warps, vc::kRouteCluster);
    a.few = a.rows <= vc::kRouteFew || (a.experts <= 2 * a.cluster * warps && fours * a.cluster <= v.smCount);
    if (!a.few)
        a.cluster = cluster(vc::kRouteTileThreads / 16,
                            vc::kRouteCluster * tiles <= v.smCount / 2 ? vc::kRouteCluster : vc::kRouteTileCluster);
    a.share = (a.experts + a.cluster - 1) / a.cluster;
    a.routerF32 = m.d.routerType == vFloat32;
    a.normalize = m.d.normalize != 0;
    const size_t e = 16 / (size_t)m.esz;
    a.aligned = m.d.hidden % 8 == 0 && (a.rows == 1 || m.d.rowStride % e == 0) && at(x, 16) && at(router, 16);
    if (v.debug)
        std::fprintf(stderr, "vcomm INFO MoeRoute rows=%d hidden=%d experts=%d topK=%d cluster=%d aligned=%d\n", a.rows,
                     a.hidden, a.experts, a.topK, a.cluster, a.aligned);
    return comm_launch(c, "moe route", [&]() { return vc::launch_moe_route(a, m.d.datatype, stream); });
}

vResult_t experts(const vMoeDesc_t* desc, const void* x, const int* ids, const float* weights, const void* const* up,
                  const void* const* down, void* const* recv, void* workspace, size_t workspaceBytes, vcomm_t c,
                  cudaStream_t stream) {
    CommView v;
    vResult_t r = comm_view(c, &v);
    if (r != vSuccess) return r;
    Moe m;
    if ((r = check_moe(desc, v.nRanks, &m)) != vSuccess) return r;
    if (v.grouping) {
        if (!up || !down || !recv) return vInvalidArgument;
        const vMoeDesc_t d = *desc;
        const std::vector<const void*> u(up, up + v.nRanks), w(down, down + v.nRanks);
        const std::vector<void*> o(recv, recv + v.nRanks);
        return vc::comm_record(c, [=]() {
            return guarded([&]() {
                return experts(&d, x, ids, weights, u.data(), w.data(), o.data(), workspace, workspaceBytes, c, stream);
            });
        });
    }
    if (m.d.rows == 0 || m.d.hidden == 0) return vSuccess;
    if (m.d.ffn == 0) return vInvalidArgument;
    if (!x || !at(x, m.esz) || !ids || !at(ids, 4) || !weights || !at(weights, 4) || !up || !down || !recv)
        return vInvalidArgument;
    vc::ExpertsArgs a;
    const size_t e = 16 / (size_t)m.esz;
    a.aligned = m.d.hidden % e == 0 && m.d.ffn % e == 0 && (m.d.rows == 1 || m.d.rowStride % e == 0) && at(x, 16);
    a.recvAligned = m.d.rows == 1 || m.d.recvStride * m.esz % 8 == 0;
    for (int k = 0; k < v.nRanks; k++) {
        const bool holds = k * m.share < m.d.experts;  // else its weights are not looked at
        if (holds && (!up[k] || !at(up[k], m.esz) || !down[k] || !at(down[k], m.esz))) return vInvalidArgument;
        if (!recv[k] || !at(recv[k], m.esz)) return vInvalidArgument;
        a.up[k] = up[k];
        a.down[k] = down[k];
        a.recv[k] = recv[k];
        a.recvAligned = a.recvAligned && at(recv[k], 8);
        if (holds) a.aligned = a.aligned && at(up[k], 16) && at(down[k], 16);
    }
    const Layout l(m);
    if (!workspace || !at(workspace, 16) || workspaceBytes < l.total()) return vInvalidArgument;
    a.x = x;
    a.ids = ids;
    a.weights = weights;
    a.act = (float*)workspace;
    a.y = (float*)((char*)workspace + l.act);
    a.done = (unsigned int*)((char*)workspace + l.act + l.y);
    a.rowStride = m.d.rowStride;
    a.recvStride = m.d.recvStride;
    a.rows = (int)m.d.rows;
    a.hidden = (int)m.d.hidden;
    a.ffn = (int)m.d.ffn;
    a.experts = m.d.experts;
    a.topK = m.d.topK;
    a.nRanks = v.nRanks;
    a.share = m.share;
    a.split = 1;
    a.combineHere = 1;
    a.status = v.status;
    a.statusHost = v.statusHost;
    a.timeoutNs = v.timeoutNs;
    a.stallCta = v.testStallRank;
    if (m.esz == 2) {
        const vc::MoeTiles t = moe_tiles(a, v.smCount);
        if (v.debug)
            std::fprintf(stderr, "vcomm INFO MoeExperts rows=%d hidden=%d ffn=%d experts=%d topK=%d N=%d aligned=%d tokens=%d split=%d,%d grid=%d,%d\n",
                         a.rows, a.hidden, a.ffn, a.experts, a.topK, a.nRanks, a.aligned, t.tokens, t.splitUp, t.splitDown, t.gridUp, t.gridDown);
        return vc::comm_launch_tracked(c, "moe experts", stream, [&]() { return vc::launch_moe_tiles(a, t, m.d.datatype, stream); });
    }
    // A warp one row of the weights (two on the way down), and more where there are CTAs enough: each looks
    // through the router's list first (13 tokens on 10 experts of 1001 x 333, when fp16 came here: 54 us with four
    // a warp, 28 so).
    const size_t groups = std::min<size_t>(a.experts, m.slots), enough = 24 * (size_t)v.smCount;
    a.tileUp = vc::kMoeTile;
    while (a.tileUp < 32 && groups * a.ffn / a.tileUp > enough) a.tileUp *= 2;
    a.tileDown = 2 * vc::kMoeTile;
    while (a.tileDown < 32 && groups * a.hidden / a.tileDown > enough) a.tileDown *= 2;
    if (v.debug)
        std::fprintf(stderr, "vcomm INFO MoeExperts rows=%d hidden=%d ffn=%d experts=%d topK=%d N=%d aligned=%d\n", a.rows,
                     a.hidden, a.ffn, a.experts, a.topK, a.nRanks, a.aligned);
    return comm_launch(c, "moe experts", [&]() { return vc::launch_moe_experts(a, stream); });
}

}  // namespace

extern "C" {

vResult_t vMoeRoute(const vMoeDesc_t* desc, const void* x, const void* routerWeight, const float* bias, int32_t* expertIds,
                    float* expertWeights, vcomm_t comm, cudaStream_t stream) {
    Range range("vMoeRoute");
    return guarded([&]() { return route(desc, x, routerWeight, bias, expertIds, expertWeights, comm, stream); });
}

vResult_t vMoeExpertsWorkspace(const vMoeDesc_t* desc, vcomm_t comm, size_t* bytes) {
    CommView v;
    vResult_t r = comm_view(comm, &v);
    if (r != vSuccess) return r;
    Moe m;
    if ((r = check_moe(desc, v.nRanks, &m)) != vSuccess) return r;
    if (!bytes) return vInvalidArgument;
    *bytes = Layout(m).total();
    return vSuccess;
}

vResult_t vMoeExperts(const vMoeDesc_t* desc, const void* x, const int32_t* expertIds, const float* expertWeights,
                      const void* const* upbuffs, const void* const* downbuffs, void* const* recvbuffs, void* workspace,
                      size_t workspaceBytes, vcomm_t comm, cudaStream_t stream) {
    Range range("vMoeExperts");
    return guarded([&]() {
        return experts(desc, x, expertIds, expertWeights, upbuffs, downbuffs, recvbuffs, workspace, workspaceBytes, comm, stream);
    });
}

}  // extern "C"
