// What the files of the low-rank adapters share: the plan's table, the buffers' layout, how work is
// cut over CTAs, and the tensor-core instructions of one CTA.
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
constexpr int64_t MAX_TILES = 1 << 23;   // 2^30 rows of h: a tensor map's extents stay below 2^32
constexpr int MAX_ADAPTERS = 1 << 20;
constexpr int64_t MAX_WIDTH = 1 << 30;   // of k and n
constexpr int MAX_CTAS = 160;            // of the persistent kernels (GB300 has 152 SMs)

// The table: n_tiles x {first row, rows, adapter, 0}; n_adapters + 1 indices of each adapter's
// first tile (tiles are in the adapters' order); from a multiple of 4 on, n_small x {adapter,
// rows, -1, -1, 16 row indices}.
inline int64_t off_first(const dit_adapter_plan_t& p) { return 4 * (int64_t)p.n_tiles; }
inline int64_t off_small(const dit_adapter_plan_t& p) { return (off_first(p) + p.n_adapters + 1 + 3) / 4 * 4; }

// h and e ("held"): for each tile of the plan 128 rows (those past the tile's own are zeros) of
// PARTS x rp bf16 (rp: the rank rounded up to 16; columns past the rank are zeros).  A value is held
// as the sum of its parts, each the bf16 nearest to what the earlier ones leave: three parts
// carry 24 significant bits, for the gradients and for fp32 outputs, two carry 16, for bf16 outputs.  There
// they cost at most 2^-17 of the sum of |h B|, less than the output's own rounding (2^-9 of it) unless y all
// but cancels, to less than 2^-8 of that sum; a third part would make half as many MMAs more.  All parts are operands of the bf16 tensor pipe, whose
// products of two bf16 values are exact.
constexpr int PARTS = 3;
inline int padded_rank(int rank) { return (rank + 15) / 16 * 16; }
inline size_t round_256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t held_bytes(int64_t n_tiles, int rank) {
  return round_256((size_t)n_tiles * TILE_ROWS * padded_rank(rank) * 2 * PARTS);
}

// Work is a list of `units` that `ctas` CTAs take in contiguous shares of equal numbers of grains
// (`grain` units each).  The CTAs of an output whose units fall to several write partial results, which a
// second kernel adds up in the order of the CTAs.  A CTA has at most two shared outputs (its
// first and its last), hence two slots.
struct Split {
  int64_t units, grain;
  int ctas;
};
inline Split split_units(int64_t units, int64_t grain, int64_t least_per_cta, int sms) {
  int64_t c = units / least_per_cta;
  if (c < 1) c = 1;
  if (c > units / grain) c = units / grain;
  if (c > sms) c = sms;
  if (c > MAX_CTAS) c = MAX_CTAS;
  return Split{units, grain, (int)c};
}
__host__ __device__ __forceinline__ int64_t first_unit(const Split& s, int cta) {
  return s.units / s.grain * cta / s.ctas * s.grain;
}
__host__ __device__ __forceinline__ int cta_of(const Split& s, int64_t unit) {
  return (int)(((unit / s.grain + 1) * s.ctas - 1) / (s.units / s.grain));
}

// Partial results: 128 rows by the rank of h and e; up to 512 columns by the rank of the gradients.
inline size_t slot_bytes(int rp, bool training) {
  return (size_t)2 * MAX_CTAS * TILE_ROWS * (training ? (rp <= 64 ? 4 : 2) : 1) * rp * 4;
}

struct Tile {
  int row0, rows, g;
};
// A tile of the table; one outside the batch or the bank has no rows and raises the status word.
__device__ __forceinline__ Tile check_tile(const int4& v, int64_t rows, int n_adapters, void* ws) {
  Tile o{v.x, v.y, v.z};
  if (o.row0 < 0 || o.rows <= 0 || o.rows > TILE_ROWS || (int64_t)o.row0 + o.rows > rows || o.g < 0 || o.g >= n_adapters) {
    raise_status(ws, DIT_ERR_INVALID_ARG);
    o = Tile{0, 0, 0};
  }
  return o;
}
__device__ __forceinline__ Tile load_tile(const int32_t* table, int64_t t, int64_t rows, int n_adapters, void* ws) {
  return check_tile(reinterpret_cast<const int4*>(table)[t], rows, n_adapters, ws);
}

// The counter that hands out jobs (k_from_rank), in the workspace; k_to_rank, which precedes it in each
// call, sets it to zero.
constexpr size_t WS_JOBS = 33280;
static_assert(WS_JOBS >= WS_PARTIALS + 32 * MAX_RED_CTAS && WS_JOBS + 4 <= WS_BYTES, "");

bool plan_ok(const dit_adapter_plan_t* p);
dit_status small_tiles(const dit_adapter_plan_t& plan, const int32_t* table, const void* x, const void* a, const void* b,
                       const float* scale, int rank, int64_t k, int64_t n, void* y, dit_dtype y_dt, void* ws,
                       cudaStream_t st);
dit_status check_common(const dit_adapter_plan_t* plan, const int32_t* table, const void* x, const void* a,
                        const void* b, const float* scale, int rank, int64_t k, int64_t n, const void* scratch,
                        size_t scratch_bytes, const void* ws, size_t ws_bytes);

// ---------------------------------------------------------------------------------------
// tcgen05 of one CTA: operands in 128-byte swizzled shared memory, bf16 x bf16 -> fp32
// ---------------------------------------------------------------------------------------
// Operand descriptors.  Their upper words are constants and the lower ones advance by bytes / 16, so the
// issuing thread makes a tile's descriptors by one addition each: it issues an instruction every
// few dozen cycles, and forming 64-bit descriptors anew cost more than the MMAs themselves.
//
// K-major: rows of 64 bf16 along the contraction, in groups of 8 rows (1024 bytes); a step of 16
// along the contraction is 32 bytes.  MN-major: rows of 64 bf16 along M or N, one for each index
// of the contraction, in groups of 8; the next 64 of M or N are `chunk` bytes on; a step of 16
// along the contraction is 16 rows, 2048 bytes.
constexpr uint32_t DESC_HI = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t chunk) {
  return (saddr & 0x3FFFFu) >> 4 | (chunk >> 4) << 16;
}
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// What becomes of the A operand in the tensor core's buffer: consecutive MMAs with one A read it from
// shared memory once (the first keeps it, the middle ones use it, the last one uses and drops it).
enum Keep { KEEP_NOT, KEEP_FIRST, KEEP_MIDDLE, KEEP_LAST };
#define DIT_LORA_MMA(collector)                                                                                  \
  asm volatile(                                                                                                  \
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %4, 0; mov.b64 x, {%1, %5}; mov.b64 y, {%2, %5};\n"        \
      "tcgen05.mma.cta_group::1.kind::f16" collector " [%0], x, y, %3, p; }" ::"r"(d),                           \
      "r"(a), "r"(b), "r"(id), "r"(accumulate ? 1u : 0u), "n"(DESC_HI)                                           \
      : "memory")
template <int KEEP = KEEP_NOT>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
  if (KEEP == KEEP_FIRST)
    DIT_LORA_MMA(".collector::a::fill");
  else if (KEEP == KEEP_MIDDLE)
    DIT_LORA_MMA(".collector::a::use");
  else if (KEEP == KEEP_LAST)
    DIT_LORA_MMA(".collector::a::lastuse");
  else
    DIT_LORA_MMA("");
}
#undef DIT_LORA_MMA
// A value that all lanes of the warp share, so that the compiler keeps what follows from it in uniform
// registers: instructions that want them (MMAs, TMA) otherwise pay for moving every operand.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}
// arrives on `bar` when every MMA issued so far by this thread has completed
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// eight accumulator columns of this thread's row; complete after tmem_wait()
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// keeps uses of eight loaded columns behind the wait
__device__ __forceinline__ void pin8(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
// a box of shared memory to global memory, and the waits for this thread's boxes
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tma_store_read_wait() {  // all but the last N have left shared memory
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The cluster's CTAs meet without ordering what they wrote (only its lifetime is at stake).  The barrier wants
// converged warps, and lanes leave the loops before it after different numbers of rounds.
__device__ __forceinline__ void cluster_leave() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// A bounded wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, void* ws, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ws, abort));
}

}  // namespace lora
}  // namespace dit6
