// A list of tensors cut into tiles: shared by the plan (list.cpp) and the
// kernels (list.hip).  Not part of the ABI.
#pragma once

#include <cstdint>
#include <vector>

#include "dopt_list.h"
#include "internal.h"

namespace dopt {

constexpr int kListBlock = DOPT_LIST_BLOCK;
static_assert(kTile % kListBlock == 0, "a tile holds whole blocks");

// One tile: up to kTile consecutive elements of one tensor, from a multiple
// of kTile.  32-bit fields keep a descriptor at 16 bytes, one scalar load;
// the plan refuses lists beyond them.
struct ListTile {
    uint32_t tile;    // index within the tensor
    uint32_t index;   // the tensor's index in its class
    uint32_t block;   // arena offset of the tile's first element / kListBlock
    uint32_t packed;  // elements (1 .. kTile) | hyper-group << 16
};

// Tensor addresses reach a kernel by value, in its arguments: nothing is
// copied from the host, the addresses may change from call to call, and a
// captured call keeps its own.  The arguments hold 4 KB; as 32-bit distances
// from the lowest address of the launch, in units of what divides them all
// (512 bytes for tensors of PyTorch's allocator, which reach 2 TB that way),
// that is kListSlots param and grad pairs, or kListGradSlots grads beside
// pass 1's own arguments.  A class of more tensors takes more launches, of
// about as many tensors each.  If tensors of a launch lie further apart (8 GB
// for 2-byte units), k_list_put writes the class's addresses into the
// workspace first, kListPut at a time (448 tensors of 30,000 elements: 54.2 us
// a step, 49.9 without): the launches and the order of the sums stay the same.
// 500 tensors of 1.8e7 elements in all were stepped in 77.6 us on MI355X, 86.0
// with full addresses in the arguments (240 to a launch); the statistics of
// 1500 tensors of 1.3e7 took 19.0 and 26.0 us.
constexpr int kListSlots = 480;
constexpr int kListGradSlots = 800;
constexpr int kListPut = 240;

// Tiles of one launch.  The XCDs take their workgroups of a long launch at
// slightly different rates and drift apart along the arrays; pass 2 and the
// copies, which write as much as they read, are therefore launched piece by
// piece, of about 2e9 bytes.  On MI355X, per launch 2^20 / 2^18 / 2^17 / 2^16 /
// 2^15 tiles (with 256 threads to a tile; with 512 the last three order alike):
// pass 2 of 1.1e9 bf16 params with fp32 moments 5.25 / 5.24 / 5.12 / 5.05 / 5.03 ms, of
// 1.2e8 fp32 params 0.592 (to 2^16) / 0.576; with e4m3 moments 1.0e9 params and fp32
// grads 2.94 / 2.90 / 2.88 / 2.90 / 2.94, 1.2e8 bf16 0.333 (to 2^16) / 0.338; export of 1.0e9
// 3.25 / 3.15 / 3.03 / 2.96 / 2.95.  Pass 1 only reads and loses by it (1.1e9 bf16 grads 328 us
// in one launch, 435 at 2^15): it takes a new launch, with partials of its own, after
// 2^31 elements of a type pair only.  Its grid is bounded without that (list_stats_grid).
constexpr int64_t kListStatsLaunch = int64_t(1) << 20;
inline int64_t list_launch_tiles(int state_kind) { return int64_t(1) << (state_kind != DOPT_STATE_F32 ? 16 : 15); }

// Pass 2 and the copies take one workgroup per tile.  A workgroup of pass 1
// reads kListStatsTiles tiles at a time and grid-strides, about 8 times on
// the largest lists: on MI355X 1.1e9 bf16 grads took 329 us with 16384
// workgroups and 342 with 4096, 1.2e8 took 51 and 47.5 (the finish adds a
// partial of each).  A function of the list only, so the reduction order is
// too.
constexpr int kListStatsTiles = 4;
inline int32_t list_stats_grid(int64_t tiles) {
    const int64_t n = (tiles + kListStatsTiles - 1) / kListStatsTiles;
    const int64_t most = n / 8 < 4096 ? 4096 : n / 8 > 16384 ? 16384 : n / 8;
    return static_cast<int32_t>(n < most ? n : most);
}

// Up to this many partials, pass 1's last workgroup adds them: a launch less.
// Each workgroup pays for it with a release and a count that all XCDs share,
// so a larger list keeps a finish of its own.  dopt_list_prepare on MI355X,
// with and without: 6.7 / 8.6 us at 8 partials, 7.7 / 8.2 at 64, 8.5 / 8.2 at
// 100, 10.8 / 8.2 at 200.
constexpr int32_t kListFused = 64;
// Pass 1 reads grads of at most this many bytes (twice the last-level cache)
// with ordinary loads, which leave them to pass 2, and more of them with
// nontemporal ones, which read faster.  A step on MI355X, nontemporal / ordinary
// loads, at 160 / 320 / 640 / 960 MB of grads: fp32 grads with e4m3 moments 148 / 137,
// 282 / 270, 561 / 555, 826 / 833 us; bf16 ones with e4m3 moments 243 / 235, 477 / 469,
// 943 / 947 us to 640 MB, with fp32 moments 397 / 375, 788 / 753, 1641 / 1619 us.
// Pass 1 alone: 160 MB in 31 / 34 us, 2 GB in 293 / 330.  dopt_list_stats, which does not
// know whether dopt_list_apply follows, goes by the same rule: a call for the norm alone
// pays the 3 us, a step in parts gains the 7 to 11.
constexpr int64_t kListKeep = int64_t(512) << 20;
// Where the workspace counts pass 1's finished workgroups.
constexpr int64_t kWsListDone = kWsRecord + 64;
// The seed of a list that rounds its moments by chance.
constexpr int64_t kWsListSeed = kWsRecord + 128;
static_assert(kWsListSeed + 8 <= kWsPartials, "the records end before the partials");

struct ListRange {  // tiles [t0, t1) of `count` consecutive tensors of a class, from tensor `first`
    int32_t first = 0, count = 0;
    int64_t t0 = 0, t1 = 0;
    int32_t grid = 0;  // workgroups: one per tile in pass 2 and the copies, as above in pass 1
    int32_t partial_base = 0;
};

constexpr int kDtypes = 3;

// The tensors of one (param dtype, grad dtype), empty ones left out.
struct ListClass {
    int32_t pd = 0, gd = 0;
    std::vector<int64_t> tensors;  // indices in the list, ascending
    std::vector<ListTile> tiles;
    std::vector<int64_t> xoff;     // export offset per tensor of the class
    std::vector<ListRange> apply, stats;
    int64_t ws_tiles = 0, ws_xoff = 0, ws_addr = 0;  // byte offsets in the workspace
};

// A list of at most this many tiles is stepped by one launch of one workgroup
// (k_list_small).
constexpr int kSmallTiles = 4;

struct ListTensor {
    int64_t numel = 0, arena = 0, xoff = 0, param = -1;
    int32_t pd = 0, gd = 0, hgroup = 0;
};

}  // namespace dopt

struct dopt_list {
    int32_t state_kind = 0, max_hgroup = 0;
    bool has_master = false;
    std::vector<dopt::ListTensor> tensors;
    std::vector<dopt::ListClass> classes;
    int64_t numel = 0, arena_numel = 0, ws_bytes = 0, grad_bytes = 0;
    int32_t total_partials = 0;
    int64_t total_tiles = 0;
};
