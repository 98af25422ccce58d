// What the files of the attention share: the plan's table, which keys a query sees, and the instructions of
// one CTA that the adapters' files do not have.
#pragma once

#include "adapters.cuh"

namespace dit6 {
namespace attn {

constexpr int TILE = 128;                 // rows of the stationary operand: the M of one instruction
constexpr int MAX_DIM = 128;
constexpr int MAX_HEADS = 4096;
constexpr int MAX_GROUP = 128;            // query heads to a key head
constexpr int64_t MAX_ROWS = 0x7fffff00;
constexpr int64_t MAX_DOCUMENTS = 1 << 22;
enum List { FORWARD, JOIN, GRAD_Q, GRAD_KV };

// The head's dimensions as the tensor cores see them (columns behind dim are zeros that TMA fills in), and the
// streamed operand's rows to a tile: as many as tensor memory holds beside the accumulators.
__host__ __device__ constexpr int padded_dim(int dim) { return dim <= 64 ? 64 : 128; }
// Floats of a row's partial result: its dimensions, the maximum and the sum, in whole 16 bytes.
__host__ __device__ constexpr int partial_floats(int padded) { return padded + 4; }
constexpr int FORWARD_COLS = 128, BACK_COLS = 64;

// The table, in int32: the items of the four lists behind one another.  An item has its document with it, so that one load brings all
// that a CTA asks of the plan.
struct Doc {
  int32_t q0, queries, k0, keys, prefix;
  int32_t tile0;  // its first padded row / 128
};
struct Item {
  Doc doc;
  int32_t row0;         // rows of the document: queries, or keys (GRAD_KV)
  int32_t begin, end;   // tiles of the streamed operand; JOIN: the first partial row, the pieces
  int32_t slot;         // FORWARD: the first partial row, -1: the output itself; JOIN: the rows
  int32_t turns;        // FORWARD: one block of rows whose tiles the CTA's two halves take in turn, each with a partial result
  int32_t unused[5];
};
constexpr int ITEM_INTS = 16;
static_assert(sizeof(Item) == 4 * ITEM_INTS, "");
__host__ __device__ inline int64_t first_item(const dit_attention_plan_t& p, int list) {
  int64_t n = 0;
  for (int i = 0; i < list; ++i) n += p.items[i];
  return ITEM_INTS * n;
}
// The keys [0, end) that query `row` of a document sees, and the first query that sees key `key` (monotone both).
__host__ __device__ inline int64_t seen_end(const Doc& d, int64_t frame, int64_t row) {
  if (frame == 0) return d.keys;
  const int64_t t = row + d.keys - d.queries;
  if (t < 0) return 0;
  const int64_t e = t < d.prefix ? (int64_t)d.prefix : d.prefix + ((t - d.prefix) / frame + 1) * frame;
  return e < d.keys ? e : d.keys;
}
__host__ __device__ inline int64_t seen_from(const Doc& d, int64_t frame, int64_t key) {
  if (frame == 0) return 0;
  const int64_t t = key < d.prefix ? 0 : d.prefix + (key - d.prefix) / frame * frame;
  const int64_t row = t - ((int64_t)d.keys - d.queries);
  return row < 0 ? 0 : row;
}

// Query heads of one key head share a forward tile: its rows are (query, head of the group), so that a key's
// tile is read once for all of them.
__host__ __device__ inline int rows_per_tile(int group) { return TILE / group; }

// A tensor of heads, strides in elements.
struct Heads {
  __nv_bfloat16* ptr;
  int64_t row, head;
};

// What a CTA works at: an item and a head.  Items of like cost are a bucket, the costliest first; within one a
// head's items follow one another and share its keys in L2.
struct Work {
  Doc doc;
  int32_t row0, begin, end, slot, turns;
  int32_t head;
  bool ok;  // the entry fits the plan
};
__device__ __forceinline__ bool fits(const Work& w, const dit_attention_plan_t& p, int list) {
  const Doc& d = w.doc;
  // the CTA's own rows begin in the document, with queries' gradients at a whole tile: the statistics of all its rows are written
  if (w.row0 < 0 || w.row0 >= (list == GRAD_KV ? d.keys : d.queries) || (list == GRAD_Q && w.row0 % TILE != 0)) return false;
  // the streamed operand's tiles lie in the document
  const int64_t cols = list == FORWARD ? FORWARD_COLS : BACK_COLS, rows = list == GRAD_KV ? d.queries : d.keys;
  if (list == FORWARD && w.slot >= 0 && p.items[JOIN] == 0) return false;  // a piece that nothing joins
  if (w.begin < 0 || (list != JOIN && (w.end < w.begin || (w.end > w.begin && (int64_t)w.end * cols >= rows + cols)))) return false;
  return d.q0 >= 0 && d.queries >= 0 && (int64_t)d.q0 + d.queries <= p.q_rows && d.k0 >= 0 && d.keys >= 0 && (int64_t)d.k0 + d.keys <= p.k_rows &&
         d.prefix >= 0 && d.tile0 >= 0 && (int64_t)d.tile0 * TILE + d.queries <= p.padded_rows;
}
// The work of this CTA.
__device__ __forceinline__ Work find_work(const int32_t* table, const dit_attention_plan_t& p, int list, int heads, void* ws) {
  Work w = {};
  const int64_t at = blockIdx.x;
  int i = -1;
  for (int b = 0; b < p.buckets[list]; ++b) {  // a few, out of the kernel's arguments
    const int first = p.bucket[list][2 * b], many = p.bucket[list][2 * b + 1];
    const int64_t r = at - (int64_t)first * heads;
    if (first >= 0 && many > 0 && r >= 0 && r < (int64_t)many * heads) {
      w.head = (int)((uint32_t)r / (uint32_t)many);
      i = first + (int)((uint32_t)r % (uint32_t)many);
    }
  }
  if (i >= 0 && i < p.items[list]) {
    const int4* it = reinterpret_cast<const int4*>(table + first_item(p, list)) + (ITEM_INTS / 4) * (int64_t)i;
    const int4 a = __ldg(it), b = __ldg(it + 1), c = __ldg(it + 2);
    w.doc = Doc{a.x, a.y, a.z, a.w, b.x, b.y};
    w.row0 = b.z, w.begin = b.w, w.end = c.x, w.slot = c.y, w.turns = c.z;
    w.ok = fits(w, p, list);
  }
  if (!w.ok && threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
  __syncwarp();
  // What follows from these is the same for all lanes: in uniform registers, where the MMAs and TMA want their operands.
  w.doc.q0 = lora::uniform(w.doc.q0);
  w.doc.queries = lora::uniform(w.doc.queries);
  w.doc.k0 = lora::uniform(w.doc.k0);
  w.doc.keys = lora::uniform(w.doc.keys);
  w.doc.prefix = lora::uniform(w.doc.prefix);
  w.doc.tile0 = lora::uniform(w.doc.tile0);
  w.row0 = lora::uniform(w.row0);
  w.begin = lora::uniform(w.begin);
  w.end = lora::uniform(w.end);
  w.slot = lora::uniform(w.slot);
  w.turns = lora::uniform(w.turns);
  w.head = lora::uniform(w.head);
  w.ok = lora::uniform(w.ok);
  return w;
}

bool plan_ok(const dit_attention_plan_t* p);
dit_status check_view(const dit_heads_t* v, int heads, int64_t rows, int dim, Heads* o);
dit_status check_output(const dit_heads_t* v, int heads, int64_t rows, int dim, Heads* o);  // its heads lie apart too
bool buffers_apart(const dit_attention_plan_t& p, const void* saved, const void* scratch, const void* ws);
bool map_heads(CUtensorMap* map, const Heads& t, int dim, int heads, int64_t rows, int box_heads, int box_rows);

// ---------------------------------------------------------------------------------------
// A CTA of warpgroups that load and issue and of HOLD (two) that hold a tile's rows in registers and take over what the first
// ones need not.  The block is launched with so many registers a thread and the shares add up to those: taking
// more than the launch brought would wait for ever, so the host checks what the kernel was compiled to.
// ---------------------------------------------------------------------------------------
template <int WARPGROUPS, int LAUNCH, int ISSUE, int ROWS, int HOLD = 2>
struct Registers {
  static constexpr int THREADS = 128 * WARPGROUPS, LAUNCHED = LAUNCH, FIRST_ROWS = 4 * (WARPGROUPS - HOLD);
  static_assert((WARPGROUPS - HOLD) * ISSUE + HOLD * ROWS <= WARPGROUPS * LAUNCH && THREADS * LAUNCH <= 65536, "");
  static __device__ __forceinline__ void give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ISSUE)); }
  static __device__ __forceinline__ void take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(ROWS)); }
};
template <typename R, typename... KArgs>
cudaError_t prepare_kernel(OncePerDevice& checked, OncePerDevice& once, void (*kern)(KArgs...), int smem) {
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const cudaError_t fits = checked.run(device, [&] {
    cudaFuncAttributes a;
    const cudaError_t got = cudaFuncGetAttributes(&a, kern);
    return got != cudaSuccess ? got : a.numRegs == R::LAUNCHED ? cudaSuccess : cudaErrorInvalidKernelImage;
  });
  return fits == cudaSuccess ? opt_in_smem(once, kern, smem) : fits;
}

// ---------------------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------------------
// D += A B with A in tensor memory (its 16 bf16 of a step are eight columns)
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %4, 0; mov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate ? 1u : 0u), "n"(lora::DESC_HI)
      : "memory");
}
// The row warps (of THREADS with their relay) and the relay meet.  Looking at an mbarrier takes a warp 130 to 160 cycles even where its phase
// has long completed; a warp of its own does that ahead of the row warps, whose barrier costs them a few dozen.
template <int THREADS>
__device__ __forceinline__ void meet(int barrier) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(barrier), "n"(THREADS) : "memory");
}
// The relay: passes on the completion of `n` phases.  It meets the row warps in each round, whatever its waits say, so
// that none is left behind; they look at the flag at the end.
template <int THREADS>
__device__ __forceinline__ void relay_one(uint32_t bar, int barrier, int j, void* ws, volatile int* abort) {
  if (!__any_sync(0xffffffffu, *abort)) lora::warp_wait(bar, j & 1, ws, abort);
  lora::fence_after();
  lora::fence_before();
  __syncwarp();
  meet<THREADS>(barrier);
}
template <int THREADS>
__device__ __forceinline__ void relay(uint32_t bar, int barrier, int n, void* ws, volatile int* abort) {
  for (int j = 0; j < n; ++j) relay_one<THREADS>(bar, barrier, j, ws, abort);
}
// 32 accumulator columns of this thread's row and the largest of them (NaN counts for nothing); complete after lora::tmem_wait()
// and pin()
__device__ __forceinline__ void tmem_ld32_max(uint32_t addr, uint32_t* r, float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
      : "r"(addr));
}
// 32 accumulator columns of this thread's row; complete after lora::tmem_wait() and pin()
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
  static_assert(N % 8 == 0, "");
#pragma unroll
  for (int i = 0; i < N; i += 8) lora::pin8(r + i);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Zeroes rows [from, rows) of a tile of 64-column chunks in shared memory (a row of a chunk is 128 bytes, whatever the
// swizzle), by a whole warp: what lies behind a document's end must not meet the zeros of p or ds in a product, which
// NaN or infinity would turn into NaN.
__device__ __forceinline__ void zero_rows(uint32_t tile, int chunk_bytes, int chunks, int from, int rows) {
  for (int c = 0; c < chunks; ++c)
    for (int i = from * 128 + (threadIdx.x & 31) * 16; i < rows * 128; i += 512)
      lora::sts128(tile + c * chunk_bytes + i, make_uint4(0, 0, 0, 0));
  fence_proxy_async();
  __syncwarp();
}
// Rows of CH x 16 bytes, a row to each lane, to `dst` of each lane (if it is live; `chunks` of a row are stored).  By way of the warp's own
// 512 CH bytes of shared memory, so that a store instruction writes whole lines: straight from the lanes each
// instruction touched 32 lines, 1900 cycles for two blocks of 128 x 64 bf16.
template <int CH>
__device__ __forceinline__ void store_rows(uint32_t smem, const uint4 (&v)[CH], void* dst, bool live, int chunks) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int c = 0; c < CH; ++c) lora::sts128(smem + lane * CH * 16 + ((c ^ (lane & (CH - 1))) << 4), v[c]);
  __syncwarp();
  const uint64_t at = live ? reinterpret_cast<uint64_t>(dst) : 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int row = i * (32 / CH) + lane / CH, c = lane % CH;
    const uint4 x = lora::lds128(smem + row * CH * 16 + ((c ^ (row & (CH - 1))) << 4));
    const uint64_t to = __shfl_sync(0xffffffffu, at, row);
    if (to && c < chunks) reinterpret_cast<uint4*>(to)[c] = x;
  }
  __syncwarp();
}
// Eight columns of fp32 as bf16, 16 bytes.
__device__ __forceinline__ uint4 pack8(const uint32_t* r, float f) {
  const float* v = reinterpret_cast<const float*>(r);
  return make_uint4(f2_to_bf16x2(v[0] * f, v[1] * f), f2_to_bf16x2(v[2] * f, v[3] * f), f2_to_bf16x2(v[4] * f, v[5] * f),
                    f2_to_bf16x2(v[6] * f, v[7] * f));
}

}  // namespace attn
}  // namespace dit6
