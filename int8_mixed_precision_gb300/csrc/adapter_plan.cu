// Host side of the low-rank adapters: the plan (tiles of rows that share an adapter), buffer
// sizes and the checks of arguments that both directions share.
#include <new>
#include <vector>

#include "adapters.cuh"

namespace dit6 {
namespace lora {

// A run is a maximal stretch of consecutive rows with one adapter (adjacent requests of the
// same adapter are one run; empty requests do not break it).
struct Run {
  int32_t row0;
  int32_t rows;
};

static dit_status make_plan(const int64_t* lengths, const int32_t* adapters, int64_t requests, int n_adapters,
                            int training, dit_adapter_plan_t* plan, int32_t* table, int64_t table_ints) {
  if (!plan || requests < 0 || n_adapters <= 0 || (requests > 0 && (!lengths || !adapters))) return DIT_ERR_INVALID_ARG;
  if (n_adapters > MAX_ADAPTERS) return DIT_ERR_UNSUPPORTED;
  std::vector<std::vector<Run>> runs((size_t)n_adapters);
  int64_t rows = 0;
  int32_t last = -1;
  for (int64_t i = 0; i < requests; ++i) {
    const int32_t g = adapters[i];
    if (lengths[i] < 0 || lengths[i] > MAX_ROWS || g < -1 || g >= n_adapters) return DIT_ERR_INVALID_ARG;
    if (lengths[i] == 0) continue;
    if (rows + lengths[i] > MAX_ROWS) return DIT_ERR_INVALID_ARG;
    if (g >= 0) {
      if (g == last)
        runs[(size_t)g].back().rows += (int32_t)lengths[i];
      else
        runs[(size_t)g].push_back({(int32_t)rows, (int32_t)lengths[i]});
    }
    last = g;
    rows += lengths[i];
  }
  // Serving plans: runs of few rows go to small tiles, which share a tile among runs and are one launch beside those
  // of the large ones (12 to 17 us).  Where there are some large tiles and few short runs, each run gets a large
  // tile of its own instead: at 1920 -> 7680 and rank 64 in bf16, 4 runs beside 16 large tiles take 22.0 us (33.8 with
  // the launch), 16 beside 64 65.2 (72.9), and in long batches 0.55 us a run, which is the launch's time at
  // about 30: 34 beside 276 take 215.5, 69 take 230.1 (209.7).
  constexpr int64_t FEW = 24;
  int64_t large = 0, shorts = 0;
  for (const auto& rs : runs)
    for (const Run& r : rs) (r.rows <= SMALL_RUN ? shorts : large) += r.rows <= SMALL_RUN ? 1 : (r.rows + TILE_ROWS - 1) / TILE_ROWS;
  const bool no_small = training || (4 * shorts <= large && shorts <= FEW);
  int64_t n_tiles = 0, n_small = 0, most = 0;
  for (const auto& rs : runs) {
    int64_t few = 0;
    const int64_t before = n_tiles;
    for (const Run& r : rs) {
      if (!no_small && r.rows <= SMALL_RUN)
        few += r.rows;
      else
        n_tiles += (r.rows + TILE_ROWS - 1) / TILE_ROWS;
    }
    n_small += (few + SMALL_ROWS - 1) / SMALL_ROWS;
    if (n_tiles - before > most) most = n_tiles - before;
  }
  if (n_tiles > MAX_TILES || n_small > MAX_TILES) return DIT_ERR_UNSUPPORTED;
  plan->rows = rows;
  plan->n_adapters = n_adapters;
  plan->training = training ? 1 : 0;
  plan->n_tiles = (int32_t)n_tiles;
  plan->n_small = (int32_t)n_small;
  plan->most_tiles = (int32_t)most;
  plan->reserved = 0;
  plan->table_ints = off_small(*plan) + (int64_t)SMALL_INTS * n_small;
  if (!table) return DIT_OK;
  if (table_ints < plan->table_ints) return DIT_ERR_INVALID_ARG;
  for (int64_t i = 0; i < plan->table_ints; ++i) table[i] = -1;
  int32_t* tile = table;
  int32_t* first = table + off_first(*plan);
  int32_t* small = table + off_small(*plan);
  int32_t t = 0;
  for (int32_t g = 0; g < n_adapters; ++g) {
    first[g] = t;
    int32_t* s = nullptr;  // the adapter's small tile that is being filled
    for (const Run& r : runs[(size_t)g]) {
      if (!no_small && r.rows <= SMALL_RUN) {
        for (int32_t i = 0; i < r.rows; ++i) {
          if (!s || s[1] == SMALL_ROWS) {
            s = small;
            small += SMALL_INTS;
            s[0] = g;
            s[1] = 0;
          }
          s[4 + s[1]++] = r.row0 + i;
        }
        continue;
      }
      for (int32_t o = 0; o < r.rows; o += TILE_ROWS, ++t, tile += 4) {
        tile[0] = r.row0 + o;
        tile[1] = r.rows - o < TILE_ROWS ? r.rows - o : TILE_ROWS;
        tile[2] = g;
        tile[3] = 0;
      }
    }
  }
  first[n_adapters] = t;
  return DIT_OK;
}

bool plan_ok(const dit_adapter_plan_t* p) {
  return p && p->rows >= 0 && p->rows <= MAX_ROWS && p->n_adapters > 0 && p->n_adapters <= MAX_ADAPTERS && p->n_tiles >= 0 && p->n_tiles <= MAX_TILES &&
         p->n_small >= 0 && p->n_small <= MAX_TILES && p->most_tiles >= 0 && p->most_tiles <= p->n_tiles && p->table_ints == off_small(*p) + (int64_t)SMALL_INTS * p->n_small;
}

dit_status check_common(const dit_adapter_plan_t* plan, const int32_t* table, const void* x, const void* a,
                        const void* b, const float* scale, int rank, int64_t k, int64_t n, const void* scratch,
                        size_t scratch_bytes, const void* ws, size_t ws_bytes) {
  if (!plan_ok(plan) || !table || !a || !b || !scale || !ws || ws_bytes < WS_BYTES) return DIT_ERR_INVALID_ARG;
  if ((!x && plan->rows > 0) || k <= 0 || n <= 0 || k > MAX_WIDTH || n > MAX_WIDTH || rank <= 0) return DIT_ERR_INVALID_ARG;
  if (rank > MAX_RANK || rank % 8 || k % 8 || n % 8) return DIT_ERR_UNSUPPORTED;
  if (scratch_bytes < dit_adapter_scratch_bytes(plan, rank, k, n) || (scratch_bytes && !scratch)) return DIT_ERR_INVALID_ARG;
  if (!aligned32(x) || !aligned32(a) || !aligned32(b) || !aligned32(ws) || !aligned32(scratch) ||
      (reinterpret_cast<uintptr_t>(table) & 15) || (reinterpret_cast<uintptr_t>(scale) & 3))
    return DIT_ERR_ALIGNMENT;
  return DIT_OK;
}

}  // namespace lora
}  // namespace dit6

extern "C" dit_status dit_adapter_plan(const int64_t* lengths, const int32_t* adapters, int64_t requests, int n_adapters,
                                       int training, dit_adapter_plan_t* plan, int32_t* table, int64_t table_ints) {
  try {
    return dit6::lora::make_plan(lengths, adapters, requests, n_adapters, training, plan, table, table_ints);
  } catch (...) {  // out of host memory
    return DIT_ERR_UNSUPPORTED;
  }
}

extern "C" size_t dit_adapter_saved_bytes(const dit_adapter_plan_t* plan, int rank) {
  if (!dit6::lora::plan_ok(plan) || rank <= 0 || rank > dit6::lora::MAX_RANK) return 0;
  return dit6::lora::held_bytes(plan->n_tiles, rank);
}

extern "C" size_t dit_adapter_scratch_bytes(const dit_adapter_plan_t* plan, int rank, int64_t k, int64_t n) {
  using namespace dit6::lora;
  if (!plan_ok(plan) || rank <= 0 || rank > MAX_RANK || k <= 0 || n <= 0 || !plan->n_tiles) return 0;
  return held_bytes(plan->n_tiles, rank) + slot_bytes(padded_rank(rank), plan->training != 0);
}
