// Driver for running the host side of a tensor list under AddressSanitizer and
// UndefinedBehaviorSanitizer (built by tests/test_list_plan.py with g++; no
// device code is involved).  Builds seeded lists, from descriptors and from
// layouts, and checks what the kernels take for granted: every tile in exactly
// one launch of each pass, a launch's tensors within its argument slots, grids
// and partials that match, state offsets that match the tiles, and workspace
// regions that do not meet.  Prints a line per list; exits 1 at the first
// violation.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "dopt_list.h"
#include "list.h"

using namespace dopt;

#define CHECK(cond)                                                 \
    do {                                                            \
        if (!(cond)) {                                              \
            printf("violated at line %d: %s\n", __LINE__, #cond);   \
            exit(1);                                                \
        }                                                           \
    } while (0)

static void check_ranges(const ListClass &C, const std::vector<ListRange> &ranges, int slots, int64_t launch) {
    int64_t t = 0;
    for (const ListRange &r : ranges) {
        CHECK(r.t0 == t && r.t1 > r.t0 && r.t1 - r.t0 <= launch);
        CHECK(r.count >= 1 && r.count <= slots);
        for (int64_t i = r.t0; i < r.t1; ++i) {
            const int64_t index = C.tiles[static_cast<size_t>(i)].index;
            CHECK(index >= r.first && index < r.first + r.count);
        }
        CHECK(r.first + r.count <= static_cast<int64_t>(C.tensors.size()));
        t = r.t1;
    }
    CHECK(t == static_cast<int64_t>(C.tiles.size()));
}

static void check(const dopt_list *P) {
    dopt_list_info info;
    CHECK(dopt_list_query(P, &info) == 0);
    int64_t numel = 0, blocks = 0, tiles = 0, ws = kWsPartials, n_in = 0;
    for (int64_t i = 0; i < info.n_tensors; ++i) {
        dopt_list_tensor_info t;
        CHECK(dopt_list_tensor(P, i, &t) == 0);
        CHECK(t.arena_offset == blocks * DOPT_LIST_BLOCK && t.export_offset == numel);
        numel += t.numel;
        blocks += (t.numel + DOPT_LIST_BLOCK - 1) / DOPT_LIST_BLOCK;
        n_in += t.numel > 0;
    }
    CHECK(info.numel == numel && info.n_blocks == blocks && info.arena_numel == blocks * DOPT_LIST_BLOCK);
    int32_t partials = 0;
    int64_t seen = 0;
    for (const ListClass &C : P->classes) {
        check_ranges(C, C.apply, kListSlots, list_launch_tiles(P->state_kind));
        check_ranges(C, C.stats, kListGradSlots, kListStatsLaunch);
        for (const ListRange &r : C.apply) CHECK(r.grid == r.t1 - r.t0);
        for (const ListRange &r : C.stats) {
            CHECK(r.grid == list_stats_grid(r.t1 - r.t0) && r.grid >= 1 && r.partial_base == partials);
            partials += r.grid;
        }
        size_t t = 0;
        for (size_t k = 0; k < C.tensors.size(); ++k) {
            const ListTensor &T = P->tensors[static_cast<size_t>(C.tensors[k])];
            CHECK(T.pd == C.pd && T.gd == C.gd && T.numel > 0 && C.xoff[k] == T.xoff);
            for (int64_t e = 0; e < T.numel; e += kTile, ++t) {
                const ListTile &d = C.tiles[t];
                CHECK(d.index == k && int64_t(d.tile) * kTile == e && int64_t(d.block) * kListBlock == T.arena + e);
                CHECK(int64_t(d.packed & 0xffff) == std::min<int64_t>(kTile, T.numel - e));
                CHECK(int32_t(d.packed >> 16) == T.hgroup && T.hgroup <= P->max_hgroup);
            }
            ++seen;
        }
        CHECK(t == C.tiles.size());
        tiles += static_cast<int64_t>(t);
    }
    CHECK(seen == n_in && partials == P->total_partials && tiles == P->total_tiles);
    ws += int64_t(partials) * 16;
    for (const ListClass &C : P->classes) {
        CHECK(C.ws_tiles >= ws && C.ws_tiles % 256 == 0);
        ws = C.ws_tiles + static_cast<int64_t>(C.tiles.size() * sizeof(ListTile));
        CHECK(C.ws_xoff >= ws && C.ws_xoff % 256 == 0);
        ws = C.ws_xoff + static_cast<int64_t>(C.xoff.size()) * 8;
        CHECK(C.ws_addr >= ws && C.ws_addr % 256 == 0);
        ws = C.ws_addr + static_cast<int64_t>(C.tensors.size() * sizeof(dopt_list_ptrs));
    }
    CHECK(info.workspace_bytes >= ws && P->classes.size() <= size_t(kDtypes * kDtypes));
    printf("%" PRId64 " tensors, %" PRId64 " elements, %zu classes, %" PRId64 " tiles, %d partials\n", info.n_tensors, numel,
           P->classes.size(), tiles, partials);
}

static void build(const std::vector<dopt_tensor_desc> &d, int kind) {
    dopt_list *P = nullptr;
    CHECK(dopt_list_build(d.data(), static_cast<int64_t>(d.size()), kind, &P) == 0);
    check(P);
    dopt_list_free(P);
}

int main() {
    std::mt19937_64 rng(5);
    auto draw = [&](int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % uint64_t(hi - lo + 1)); };
    for (int kind = 0; kind < 2; ++kind) {
        build({}, kind);
        for (int64_t n : {0, 1, 127, 128, 129, 2047, 2048, 2049, 8192, 8193, 1 << 20})
            build({dopt_tensor_desc{n, 1, 1, 0, 0}}, kind);
        for (int64_t count : {479, 480, 481, 799, 800, 801, 961, 5000})
            for (int64_t most : {1, 3000, 9000}) {
                std::vector<dopt_tensor_desc> d;
                for (int64_t i = 0; i < count; ++i) {
                    const int32_t mixed = count % 2 ? 1 : 0;
                    d.push_back(dopt_tensor_desc{draw(0, most), mixed ? int32_t(draw(0, 2)) : 1,
                                                 mixed ? int32_t(draw(0, 2)) : 1, int32_t(draw(0, 15)), 0});
                }
                build(d, kind);
            }
        // more tiles than a launch takes, in one tensor and between two, and all 16-bit block indices passed
        build({dopt_tensor_desc{(int64_t(1) << 28) + 77, 1, 0, 3, 0}}, kind);
        build({dopt_tensor_desc{100000001, 2, 2, 0, 0}, dopt_tensor_desc{50000000, 2, 2, 1, 0}, dopt_tensor_desc{1, 2, 2, 0, 0}},
              kind);
        dopt_list *P = nullptr;
        for (int i = 0; i < 20; ++i) {
            std::vector<dopt_param_desc> ps;
            for (int64_t k = draw(1, 30); k > 0; --k)
                ps.push_back(dopt_param_desc{draw(1, 20000), int32_t(draw(0, 2)), int32_t(draw(0, 2)), int32_t(draw(0, 9) == 0),
                                             int32_t(draw(0, 4))});
            const int32_t n = int32_t(draw(1, 9));
            const dopt_shard_cfg cfg{n, int32_t(draw(0, n - 1)), draw(0, 1) * 9000, 0, 1};
            dopt_layout *L = nullptr;
            CHECK(dopt_build_ranges(ps.data(), static_cast<int64_t>(ps.size()), &cfg, &L) == 0);
            CHECK(dopt_list_from_layout(L, kind, &P) == 0);
            check(P);
            CHECK(P->numel == L->state_numel);
            dopt_list_free(P);
            dopt_layout_free(L);
        }
        const dopt_tensor_desc bad[] = {{-1, 1, 1, 0, 0}, {(int64_t(1) << 38) + 1, 1, 1, 0, 0}, {1, 3, 1, 0, 0},
                                        {1, 1, -1, 0, 0}, {1, 1, 1, 16, 0}, {1, 1, 1, -1, 0}, {INT64_MAX, 1, 1, 0, 0}};
        for (const dopt_tensor_desc &b : bad) CHECK(dopt_list_build(&b, 1, kind, &P) == DOPT_ERR_INVALID && !P);
        CHECK(dopt_list_build(bad, -1, kind, &P) == DOPT_ERR_INVALID);
        CHECK(dopt_list_build(nullptr, 1, kind, &P) == DOPT_ERR_INVALID);
        CHECK(dopt_list_build(bad, 1, 7, &P) == DOPT_ERR_INVALID);
        CHECK(dopt_list_build(bad, (int64_t(1) << 24) + 1, kind, &P) == DOPT_ERR_INVALID);
    }
    printf("ok\n");
    return 0;
}
