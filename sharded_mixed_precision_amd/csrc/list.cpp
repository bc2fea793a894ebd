// Host side of a tensor list: sizes, arena offsets, tiles and workspace map.
#include "list.h"

#include <algorithm>
#include <cstring>
#include <new>

namespace dopt {

// More elements than any GPU holds; every 32-bit field of a tile descriptor
// and every byte offset then fits (block index < 2^38 / 128 + 2^24).
constexpr int64_t kListMaxNumel = int64_t(1) << 38;
constexpr int64_t kListMaxTensors = int64_t(1) << 24;

static int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

static bool known_dtype(int32_t d) { return d == DOPT_F32 || d == DOPT_BF16 || d == DOPT_F16; }

// Ranges of about as many consecutive tensors, at most `most`, and at most
// `launch` tiles of a class (a tensor of more tiles lies in several).
static void cut(const ListClass &C, int most, int64_t launch, std::vector<ListRange> &out) {
    const int32_t n = static_cast<int32_t>(C.tensors.size());
    const int32_t parts = (n + most - 1) / most, slots = (n + parts - 1) / parts;
    const int64_t n_tiles = static_cast<int64_t>(C.tiles.size());
    int64_t t = 0;
    for (int32_t f = 0; f < n; f += slots) {
        ListRange r;
        r.first = f;
        r.count = std::min(slots, n - f);
        while (t < n_tiles && C.tiles[static_cast<size_t>(t)].index < uint32_t(f + r.count)) {
            r.t0 = t;
            while (t < n_tiles && t - r.t0 < launch && C.tiles[static_cast<size_t>(t)].index < uint32_t(f + r.count))
                ++t;
            r.t1 = t;
            out.push_back(r);
        }
    }
}

static int plan(dopt_list &P) {
    int64_t blocks = 0, numel = 0;
    for (size_t i = 0; i < P.tensors.size(); ++i) {
        ListTensor &T = P.tensors[i];
        if (T.numel < 0 || T.numel > kListMaxNumel || !known_dtype(T.pd) || !known_dtype(T.gd) || T.hgroup < 0 ||
            T.hgroup >= DOPT_MAX_HGROUPS)
            return fail(DOPT_ERR_INVALID, "tensor " + std::to_string(i) + ": bad numel, dtype or hgroup");
        T.arena = blocks * kListBlock;
        T.xoff = numel;
        numel += T.numel;
        P.grad_bytes += T.numel * (T.gd == DOPT_F32 ? 4 : 2);
        if (numel > kListMaxNumel) return fail(DOPT_ERR_INVALID, "the tensors hold more than 2^38 elements in total");
        blocks += (T.numel + kListBlock - 1) / kListBlock;
        P.max_hgroup = std::max(P.max_hgroup, T.hgroup);
        if (T.pd != DOPT_F32) P.has_master = true;
        if (T.numel == 0) continue;
        size_t c = 0;
        while (c < P.classes.size() && !(P.classes[c].pd == T.pd && P.classes[c].gd == T.gd)) ++c;
        if (c == P.classes.size()) {
            P.classes.emplace_back();
            P.classes.back().pd = T.pd;
            P.classes.back().gd = T.gd;
        }
        ListClass &C = P.classes[c];
        const uint32_t index = static_cast<uint32_t>(C.tensors.size());
        C.tensors.push_back(static_cast<int64_t>(i));
        C.xoff.push_back(T.xoff);
        for (int64_t e = 0; e < T.numel; e += kTile) {
            const int64_t n = std::min<int64_t>(kTile, T.numel - e);
            C.tiles.push_back(ListTile{static_cast<uint32_t>(e / kTile), index,
                                       static_cast<uint32_t>((T.arena + e) / kListBlock),
                                       static_cast<uint32_t>(n) | static_cast<uint32_t>(T.hgroup) << 16});
        }
    }
    P.numel = numel;
    P.arena_numel = blocks * kListBlock;
    int32_t partials = 0;
    for (ListClass &C : P.classes) {
        cut(C, kListSlots, list_launch_tiles(P.state_kind), C.apply);
        cut(C, kListGradSlots, kListStatsLaunch, C.stats);
        for (ListRange &r : C.apply) r.grid = static_cast<int32_t>(r.t1 - r.t0);
        for (ListRange &r : C.stats) {
            r.grid = list_stats_grid(r.t1 - r.t0);
            r.partial_base = partials;
            partials += r.grid;
        }
    }
    P.total_partials = partials;
    for (const ListClass &C : P.classes) P.total_tiles += static_cast<int64_t>(C.tiles.size());
    int64_t ws = kWsPartials + up(int64_t(partials) * 16, 256);
    for (ListClass &C : P.classes) {
        C.ws_tiles = ws;
        ws += up(int64_t(C.tiles.size()) * int64_t(sizeof(ListTile)), 256);
        C.ws_xoff = ws;
        ws += up(int64_t(C.xoff.size()) * 8, 256);
        C.ws_addr = ws;
        ws += up(int64_t(C.tensors.size()) * int64_t(sizeof(dopt_list_ptrs)), 256);
    }
    P.ws_bytes = ws;
    return DOPT_OK;
}

// Builds a list from tensors that `fill` puts into it.
template <class Fill>
static int make_list(int32_t state_kind, dopt_list **out, Fill fill) {
    *out = nullptr;
    if (state_kind != DOPT_STATE_F32 && state_kind != DOPT_STATE_E4M3 && state_kind != DOPT_STATE_E4M3_SR)
        return fail(DOPT_ERR_INVALID, "bad state kind");
    dopt_list *P = new (std::nothrow) dopt_list();
    if (!P) return fail(DOPT_ERR_NOMEM, "out of host memory");
    int rc;
    try {
        P->state_kind = state_kind;
        fill(P->tensors);
        rc = plan(*P);
    } catch (const std::bad_alloc &) {
        rc = fail(DOPT_ERR_NOMEM, "out of host memory");
    }
    if (rc != DOPT_OK) {
        delete P;
        return rc;
    }
    *out = P;
    return DOPT_OK;
}

}  // namespace dopt

using namespace dopt;

extern "C" {

int dopt_list_build(const dopt_tensor_desc *tensors, int64_t n, int32_t state_kind, dopt_list **out) {
    if (!out || (n > 0 && !tensors)) return fail(DOPT_ERR_INVALID, "null argument");
    if (n < 0 || n > kListMaxTensors) return fail(DOPT_ERR_INVALID, "the number of tensors must be in [0, 2^24]");
    return make_list(state_kind, out, [&](std::vector<ListTensor> &ts) {
        ts.resize(static_cast<size_t>(n));
        for (int64_t i = 0; i < n; ++i) {
            ListTensor &T = ts[static_cast<size_t>(i)];
            T.numel = tensors[i].numel;
            T.pd = tensors[i].param_dtype;
            T.gd = tensors[i].grad_dtype;
            T.hgroup = tensors[i].hgroup;
        }
    });
}

int dopt_list_from_layout(const dopt_layout *L, int32_t state_kind, dopt_list **out) {
    if (!L || !out) return fail(DOPT_ERR_INVALID, "null argument");
    if (static_cast<int64_t>(L->params.size()) > kListMaxTensors)
        return fail(DOPT_ERR_INVALID, "the layout holds more than 2^24 params");
    return make_list(state_kind, out, [&](std::vector<ListTensor> &ts) {
        for (size_t p = 0; p < L->params.size(); ++p) {
            const Param &q = L->params[p];
            if (!q.has_shard) continue;
            ListTensor T;
            T.numel = q.local.end - q.local.start;
            T.pd = q.pd;
            T.gd = q.gd;
            T.hgroup = q.hgroup;
            T.param = static_cast<int64_t>(p);
            ts.push_back(T);
        }
    });
}

void dopt_list_free(dopt_list *list) { delete list; }

int dopt_list_query(const dopt_list *P, dopt_list_info *out) {
    if (!P || !out) return fail(DOPT_ERR_INVALID, "null argument");
    std::memset(out, 0, sizeof *out);
    out->n_tensors = static_cast<int64_t>(P->tensors.size());
    out->numel = P->numel;
    out->arena_numel = P->arena_numel;
    out->n_blocks = P->arena_numel / kListBlock;
    out->workspace_bytes = P->ws_bytes;
    out->stats_record_offset = kWsRecord;
    out->state_kind = P->state_kind;
    out->has_master = P->has_master ? 1 : 0;
    return DOPT_OK;
}

int dopt_list_tensor(const dopt_list *P, int64_t i, dopt_list_tensor_info *out) {
    if (!P || !out) return fail(DOPT_ERR_INVALID, "null argument");
    if (i < 0 || i >= static_cast<int64_t>(P->tensors.size())) return fail(DOPT_ERR_RANGE, "tensor index");
    const ListTensor &T = P->tensors[static_cast<size_t>(i)];
    std::memset(out, 0, sizeof *out);
    out->numel = T.numel;
    out->arena_offset = T.arena;
    out->export_offset = T.xoff;
    out->param = T.param;
    out->param_dtype = T.pd;
    out->grad_dtype = T.gd;
    out->hgroup = T.hgroup;
    return DOPT_OK;
}

}  // extern "C"
