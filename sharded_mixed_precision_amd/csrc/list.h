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
// kListSlots param and grad pairs, or kListGradSlots grads); a list of more
// tensors of one class takes a launch for each so many.  Nothing is copied
// from the host and the addresses may change from call to call.
constexpr int kListSlots = 240;
constexpr int kListGradSlots = 2 * kListSlots;

// Tiles of one launch: 2^28 threads, below the 2^32 a launch may have.
constexpr int64_t kListLaunchTiles = int64_t(1) << 20;

// Pass 2 and the copies take one workgroup per tile; pass 1 one per
// kListStatsTiles tiles up to a fixed number, which then grid-stride (the
// finish adds a partial of each).  A function of the list only, so the
// reduction order is too.
constexpr int kListStatsTiles = 4;
constexpr int64_t kListStatsBlocks = 4096;
inline int32_t list_stats_grid(int64_t tiles) {
    const int64_t n = (tiles + kListStatsTiles - 1) / kListStatsTiles;
    return static_cast<int32_t>(n < kListStatsBlocks ? n : kListStatsBlocks);
}

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
};
