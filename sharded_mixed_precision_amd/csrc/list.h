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

// Tensor addresses reach a kernel by value, in its arguments (4 KB hold
// kListSlots param and grad pairs, or kListGradSlots grads beside pass 1's own);
// a list of more tensors of one class takes a launch for each so many.  Nothing is copied
// from the host and the addresses may change from call to call.
constexpr int kListSlots = 240;
constexpr int kListGradSlots = 400;

// Tiles of one launch: 2^28 threads, below the 2^32 a launch may have.
constexpr int64_t kListLaunchTiles = int64_t(1) << 20;

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
// Where the workspace counts pass 1's finished workgroups.
constexpr int64_t kWsListDone = kWsRecord + 64;

struct ListRange {  // tiles [t0, t1) of `count` consecutive tensors of a class, from tensor `first`
    int32_t first = 0, count = 0;
    int64_t t0 = 0, t1 = 0;
    int32_t grid = 0;  // workgroups: one per tile in pass 2 and the copies, as above in pass 1
    int32_t partial_base = 0;
};

// The tensors of one (param dtype, grad dtype), empty ones left out.
struct ListClass {
    int32_t pd = 0, gd = 0;
    std::vector<int64_t> tensors;  // indices in the list, ascending
    std::vector<ListTile> tiles;
    std::vector<int64_t> xoff;     // export offset per tensor of the class
    std::vector<ListRange> apply, stats;
    int64_t ws_tiles = 0, ws_xoff = 0;  // byte offsets in the workspace
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
    int64_t numel = 0, arena_numel = 0, ws_bytes = 0;
    int32_t total_partials = 0;
    int64_t total_tiles = 0;
};
