// What the files of the low-rank adapters share: the plan's table and the buffers' layout.
#pragma once

#include "common.cuh"

namespace dit6 {
namespace lora {

constexpr int TILE_ROWS = 128;           // rows of a tile: the M of one tensor-core instruction
constexpr int SMALL_ROWS = 16;           // rows of a small tile
constexpr int SMALL_INTS = 4 + SMALL_ROWS;
constexpr int SMALL_RUN = 32;            // serving: a run of up to this many rows goes to small tiles
constexpr int MAX_RANK = 128;
constexpr int64_t MAX_ROWS = 0x7fffff00;
constexpr int64_t MAX_TILES = 1 << 26;

// The table: n_tiles x {first row, rows, adapter, 0}; n_adapters + 1 indices of each adapter's
// first tile (tiles are in the adapters' order); from a multiple of 4 on, n_small x {adapter,
// rows, -1, -1, 16 row indices}.
inline int64_t off_first(const dit_adapter_plan_t& p) { return 4 * (int64_t)p.n_tiles; }
inline int64_t off_small(const dit_adapter_plan_t& p) { return (off_first(p) + p.n_adapters + 1 + 3) / 4 * 4; }

// h and e: for each 128-row tile of the plan, 128 rows of rank values (the rank rounded up to
// 16), rows past the tile's own zero.
inline int padded_rank(int rank) { return (rank + 15) / 16 * 16; }
inline size_t held_bytes(int64_t n_tiles, int rank) { return (size_t)n_tiles * TILE_ROWS * padded_rank(rank) * 4; }

struct Tile {
  int row0, rows, g;
};
// A tile of the table; one outside the batch or the bank has no rows and raises the status word.
__device__ __forceinline__ Tile load_tile(const int32_t* table, int t, int64_t rows, int n_adapters, void* ws) {
  const int4 v = reinterpret_cast<const int4*>(table)[t];
  Tile o{v.x, v.y, v.z};
  if (o.row0 < 0 || o.rows <= 0 || o.rows > TILE_ROWS || (int64_t)o.row0 + o.rows > rows || o.g < 0 || o.g >= n_adapters) {
    raise_status(ws, DIT_ERR_INVALID_ARG);
    o = Tile{0, 0, 0};
  }
  return o;
}

bool plan_ok(const dit_adapter_plan_t* p);
dit_status check_common(const dit_adapter_plan_t* plan, const int32_t* table, const void* x, const void* a,
                        const void* b, const float* scale, int rank, int64_t k, int64_t n, const void* scratch,
                        size_t scratch_bytes, const void* ws, size_t ws_bytes);

}  // namespace lora
}  // namespace dit6
