// Low-rank adapters of many requests beside one shared projection: forward and backward.
//
//   h = scale (x A^T),  y += h B^T;   e = scale (dy B),  dx += e A,  dA = e^T x,  dB = dy^T h
//
// Bound by memory: with ranks of 8 to 128 a product does 2 rank operations for each 2-byte element of x, y or
// dy that it reads, far below what the tensor cores do meanwhile.  So each product streams its wide
// operand once through shared memory by TMA and runs on tcgen05 with everything of the rank's
// size on chip.  Three kernels of one CTA per SM, and two short ones that add up partial results:
//
//   k_to_rank    h, e: units are (128 rows, 64 columns of x or dy).  35552 x 1920 at rank 64: 31 us, 4.4 TB/s
//                of x; 17776 x 7680: 51 us, 5.4 TB/s.  What keeps it below the copy rate is the weights'
//                way from L2 (half as many bytes again at rank 64).
//   k_from_rank  y, dx: jobs are (128 rows, a few blocks of 128 columns), read, added to and written once.
//                35552 x 7680 in bf16 at rank 64: 168 us, 6.5 TB/s, 0.96 of the copy rate.
//   k_over_rows  dA, dB: units are (128 to 512 columns, 128 rows), both gradients in one launch.  17776 rows of
//                7680 + 1920 columns at rank 64: 81 us, 4.2 TB/s of x and dy, on 114 SMs, while the other 38
//                begin with dx (on all SMs 69 us, but with 20 MB of partial results to add up).
//
// Weights are read as they lie: A [rank x k] and B [n x rank] serve both the product along their
// rows (K-major operand) and the one across them (MN-major operand), so no transposed copies are kept.
//
// The tensor cores' fp32 accumulation truncates (measured: a relative error of 1.1e-9 per
// element of the contraction, 4.4e-6 over 4096), so sums are drained to registers every CHUNK
// elements and added there with rounding to nearest.
//
// Ahead of the stream.  Each kernel lets the next one launch only after its own wait for the one before, so a kernel
// that has started finds everything but its immediate predecessor complete and in global memory (the wait returns when
// the grids before have completed and flushed their results), and waits for that one
// where it first reads what it made (h and e) or writes what it reads: k_from_rank's first weights and
// old values and k_over_rows' units of dB come in before, and dx, which needs nothing of k_over_rows, is
// updated beside it; its e is two kernels back.  The instruction's own text speaks of a grid and its direct
// predecessors, so a new kernel in between has to keep the order of wait and trigger.  Every kernel waits before it
// ends, so the stream's order holds for whatever follows.
//
// Warps: 0 loads (TMA), 1 issues the MMAs, the others drain and store.  Every wait is bounded.  Loads and MMAs
// are issued by an elected lane of a converged warp, from values that the warp shares: otherwise the
// compiler moves every operand to uniform registers first, 50 ns an MMA.
#include <stdio.h>
#include <stdlib.h>

#include "adapters.cuh"

namespace dit6 {
namespace lora {

constexpr int EPI_WARPS = 8, EPI_THREADS = 32 * EPI_WARPS;
constexpr int THREADS = 64 + EPI_THREADS;
constexpr int CHUNK = 256;                  // elements of a contraction between drains
constexpr int RING_BYTES = 220 * 1024;      // shared memory for operands
constexpr int SMEM_BYTES = RING_BYTES + 1024 + 1024;
constexpr int MAX_STAGES = 12;
constexpr int MAX_PANELS = 8;               // k_from_rank: 128 rows x 128 bytes of the output each
constexpr int ACCS = 4;                     // accumulators in turn in k_from_rank (two in the other kernels)

struct Args {
  const int32_t* table;
  int64_t rows;  // of the batch
  int n_adapters, n_tiles;
  int rank, rp;
  int parts;     // of held that are written (k_to_rank) or read (k_from_rank)
  int stages;
  Split split;
  void* ws;
  int stall;
};

constexpr int JOBS = 4;                     // announced ahead in k_from_rank

// Barriers and flags behind the operands in shared memory.
struct Control {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t dfull[ACCS], dempty[ACCS];  // accumulators
  uint64_t hfull[2], hempty[2];        // tiles of held (k_from_rank)
  uint64_t jfull[JOBS], jempty[JOBS];  // jobs (k_from_rank)
  uint64_t yfull[MAX_PANELS], ydone[MAX_PANELS], yempty[MAX_PANELS];  // panels of the output: loaded, updated, stored
  uint64_t done;
  uint32_t tmem;
  int abort;
  int job[JOBS];
  int valid[MAX_STAGES];               // rows of a stage that belong to its tile (k_over_rows)
};

static_assert(sizeof(Control) <= 1024, "");

struct Frame {
  uint32_t smem;  // operands, 1024-byte aligned
  Control* c;
};
__device__ __forceinline__ Frame frame(uint8_t* raw) {
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  return Frame{smem_u32(base), reinterpret_cast<Control*>(base + RING_BYTES)};
}
__device__ __forceinline__ void start(const Frame& f, int stages, uint32_t cols, int epi_warps = EPI_WARPS) {
  Control* c = f.c;
  if (threadIdx.x < 32) {  // some barriers to a lane: sixty in a row take half a microsecond
    const int i = threadIdx.x;
    if (i < stages) {
      mbar_init(smem_u32(&c->full[i]), 1);
      mbar_init(smem_u32(&c->empty[i]), 1);
    }
    if (i < ACCS) {
      mbar_init(smem_u32(&c->dfull[i]), 1);
      mbar_init(smem_u32(&c->dempty[i]), epi_warps);
    }
    if (i < MAX_PANELS) {
      mbar_init(smem_u32(&c->yfull[i]), 1);
      mbar_init(smem_u32(&c->ydone[i]), epi_warps);
      mbar_init(smem_u32(&c->yempty[i]), 1);
    }
    if (i < 2) {
      mbar_init(smem_u32(&c->hfull[i]), 1);
      mbar_init(smem_u32(&c->hempty[i]), 1);
    }
    if (i < JOBS) {
      mbar_init(smem_u32(&c->jfull[i]), 1);
      mbar_init(smem_u32(&c->jempty[i]), 2 + epi_warps);  // the MMA, epilogue and store warps
    }
    if (i == 0) {
      mbar_init(smem_u32(&c->done), 1);
      c->abort = 0;
    }
    fence_barrier_init();
  }
  if (threadIdx.x / 32 == 1) {
    tmem_alloc(smem_u32(&c->tmem), cols);
    fence_before();
  }
  __syncthreads();
  fence_after();
}
__device__ __forceinline__ void finish(const Frame& f, uint32_t cols) {
  fence_before();
  __syncthreads();
  if (threadIdx.x / 32 == 1) {
    fence_after();
    tmem_free(f.c->tmem, cols);
  }
}
// A producer that gave up waits for its own copies in flight; `n` were started.
__device__ __forceinline__ void await_copies(const Frame& f, int stages, uint32_t n, void* ws) {
  volatile int never = 0;
  for (uint32_t i = n > (uint32_t)stages ? n - stages : 0; i < n; ++i)
    mbar_wait(smem_u32(&f.c->full[i % stages]), (i / stages) & 1, ws, &never);
}
// The MMA issuer's end: everything that it issued has completed.
__device__ __forceinline__ void await_mmas(const Frame& f, void* ws) {
  volatile int never = 0;
  mma_commit(smem_u32(&f.c->done));
  mbar_wait(smem_u32(&f.c->done), 0, ws, &never);
}
// The slot of CTA `cta`'s partial result for an output that CTAs c0 and later ones share.
__device__ __forceinline__ int slot_of(int cta, int c0) { return 2 * cta + (cta == c0 ? 1 : 0); }

// The sum over CTAs c0 to c1 of their partial results at float4 index e, in the CTAs' order.
__device__ __forceinline__ float4 sum_slots(const float* slots, int64_t slot, int c0, int c1, int e) {
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = c0; k <= c1; k += 4) {  // four loads in flight
    float4 v[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      v[h] = k + h <= c1 ? __ldcg(reinterpret_cast<const float4*>(slots + slot_of(k + h, c0) * slot) + e)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      sum.x += v[h].x;
      sum.y += v[h].y;
      sum.z += v[h].z;
      sum.w += v[h].w;
    }
  }
  return sum;
}

// A value's parts: each the bf16 nearest to what is left.  An infinite or NaN first part stands alone.
template <int N>
__device__ __forceinline__ void split_parts(float v, float (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = __bfloat162float(__float2bfloat16_rn(v));
    v = isfinite(part[i]) ? v - part[i] : 0.f;
  }
}

// ---------------------------------------------------------------------------------------
// To the rank: held = scale * (in W^T), in [rows x width] along its rows, W K-major (A) or
// MN-major (B).
// ---------------------------------------------------------------------------------------
struct ToRank {
  const float* scale;
  __nv_bfloat16* held;
  float* slots;
  int blocks;   // of 64 along the contraction
  int cluster;  // CTAs to a tile (CLUSTER)
};

// Four columns of row r of tile ti of held, from their sums.
__device__ __forceinline__ void store_held(const Args& p, const ToRank& o, const Tile& t, float scale, int64_t ti, int r, int col,
                                           const float4& sum) {
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
  float part[4][PARTS];
#pragma unroll
  for (int h = 0; h < 4; ++h) split_parts(r < t.rows && col + h < p.rank ? v[h] * scale : 0.f, part[h]);
  __nv_bfloat16* held = o.held + (ti * TILE_ROWS + r) * (int64_t)(p.parts * p.rp) + col;
#pragma unroll
  for (int h = 0; h < PARTS; ++h)
    if (h < p.parts)
      *reinterpret_cast<uint2*>(held + h * p.rp) = make_uint2(f2_to_bf16x2(part[0][h], part[1][h]), f2_to_bf16x2(part[2][h], part[3][h]));
}

// A tile falls to one CTA, to a cluster that splits its contraction (few tiles), or to the CTAs whose equal
// shares of all units it meets; the cluster sums its partial results through distributed shared memory,
// the others' are summed by k_to_rank_sum.

template <bool MN, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 1)
    k_to_rank(const __grid_constant__ CUtensorMap m_in, const __grid_constant__ CUtensorMap m_w, Args p, ToRank o) {
  extern __shared__ uint8_t raw[];
  const Frame f = frame(raw);
  Control* c = f.c;
  volatile int* abort = &c->abort;
  constexpr uint32_t COLS = 256;  // two accumulators of up to 128 columns
  if (threadIdx.x == 0) {
    prefetch_tmap(&m_in);
    prefetch_tmap(&m_w);
  }
  start(f, p.stages, COLS);
  const uint32_t tmem = c->tmem;
  pdl_wait();
  pdl_launch_dependents();  // not before: see above, ahead of the stream
  if (blockIdx.x == 0 && threadIdx.x == 0) *ws_u32(p.ws, WS_JOBS) = 0;  // for the next k_from_rank

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int w_chunks = MN ? (p.rank + 63) / 64 : 1;
  const uint32_t w_bytes = MN ? w_chunks * 8192 : p.rp * 128;
  const uint32_t stage_bytes = 16384 + w_bytes;
  const int in_cluster = CLUSTER ? (int)cluster_rank() : 0;
  const int64_t tile0 = CLUSTER ? blockIdx.x / o.cluster * (int64_t)o.blocks : 0;
  const int64_t u0 = CLUSTER ? tile0 + (int64_t)o.blocks * in_cluster / o.cluster : first_unit(p.split, blockIdx.x);
  const int64_t u1 = CLUSTER ? tile0 + (int64_t)o.blocks * (in_cluster + 1) / o.cluster : first_unit(p.split, blockIdx.x + 1);

  if (warp == 0) {
    if (!p.stall) {
      uint32_t n = 0, parity = 1;
      bool ok = true;
      Tile t{0, 0, 0};
      int64_t ti = u0 / o.blocks;
      int kb = (int)(u0 % o.blocks), s = 0;
      for (int64_t u = u0; u < u1; ++u, ++n) {
        if (u == u0 || kb == 0) t = load_tile(p.table, ti, p.rows, p.n_adapters, p.ws);
        if (!warp_wait(smem_u32(&c->empty[s]), parity, p.ws, abort)) {
          ok = false;
          break;
        }
        const uint32_t full = smem_u32(&c->full[s]), dst = f.smem + s * stage_bytes;
        if (elect_one()) {
          mbar_expect_tx(full, stage_bytes);
          tma_load_2d(dst, &m_in, full, kb * 64, t.row0);
          if (MN) {
            for (int i = 0; i < w_chunks; ++i) tma_load_3d(dst + 16384 + i * 8192, &m_w, full, i * 64, kb * 64, t.g);
          } else {
            tma_load_3d(dst + 16384, &m_w, full, kb * 64, 0, t.g);
          }
        }
        __syncwarp();
        if (++kb == o.blocks) {
          kb = 0;
          ++ti;
        }
        if (++s == p.stages) {
          s = 0;
          parity ^= 1;
        }
      }
      if (!ok) await_copies(f, p.stages, n, p.ws);
    }
  } else if (warp == 1) {
    const uint32_t id = idesc(128, p.rp, false, MN);
    uint32_t chunk = 0, parity = 0;
    int s = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const int64_t end = min(u1, (u / o.blocks + 1) * o.blocks);  // of this tile's share
      for (; u < end && ok; ++chunk) {
        const int buf = chunk & 1;
        if (!warp_wait(smem_u32(&c->dempty[buf]), ((chunk >> 1) & 1) ^ 1, p.ws, abort)) {
          ok = false;
          break;
        }
        const int64_t stop = min(end, u + CHUNK / 64);
        for (int64_t first = u; u < stop; ++u) {
          if (!warp_wait(smem_u32(&c->full[s]), parity, p.ws, abort)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            fence_after();
            const uint32_t at = f.smem + s * stage_bytes;
            const uint32_t a = desc_k(at), b = MN ? desc_mn(at + 16384, 8192) : desc_k(at + 16384);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma(tmem + buf * 128, a + j * (32 >> 4), b + j * ((MN ? 2048 : 32) >> 4), id, u > first || j > 0);
            mma_commit(smem_u32(&c->empty[s]));
            if (u + 1 == stop) mma_commit(smem_u32(&c->dfull[buf]));
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
    }
    if (elect_one()) await_mmas(f, p.ws);
    __syncwarp();
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    const int nc = p.rp / 2, col0 = half * nc;  // this thread's columns (a multiple of 8)
    uint32_t chunk = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const int64_t ti = u / o.blocks;
      const int64_t end = min(u1, (ti + 1) * o.blocks);
      const bool whole = u == ti * o.blocks && end == (ti + 1) * o.blocks;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (; u < end; u = min(end, u + CHUNK / 64), ++chunk) {
        const int buf = chunk & 1;
        if (!warp_wait(smem_u32(&c->dfull[buf]), (chunk >> 1) & 1, p.ws, abort)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 128 + col0;
        uint32_t r[64];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * i < nc) tmem_ld8(at + 8 * i, r + 8 * i);
        tmem_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * i < nc) {
            pin8(r + 8 * i);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[8 * i + j] += __uint_as_float(r[8 * i + j]);
          }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c->dempty[buf]));
      }
      if (!ok) break;
      if (CLUSTER) {  // every MMA of this CTA has read its operands: their place takes the partial result
        const uint32_t mine = f.smem + (row * (p.rp + 4) + col0) * 4;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (4 * i < nc)
            sts128(mine + 16 * i, make_uint4(__float_as_uint(acc[4 * i]), __float_as_uint(acc[4 * i + 1]),
                                             __float_as_uint(acc[4 * i + 2]), __float_as_uint(acc[4 * i + 3])));
        continue;
      }
      const Tile t = load_tile(p.table, ti, p.rows, p.n_adapters, p.ws);
      if (!whole) {
        const int c0 = cta_of(p.split, ti * o.blocks);
        float* mine = o.slots + slot_of(blockIdx.x, c0) * ((int64_t)TILE_ROWS * p.rp) + (int64_t)row * p.rp + col0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (4 * i < nc) reinterpret_cast<float4*>(mine)[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        continue;
      }
      const float scale = o.scale[t.g];
      __nv_bfloat16* held = o.held + (ti * TILE_ROWS + row) * (int64_t)(p.parts * p.rp) + col0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * i < nc) {
          uint32_t w[PARTS][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo[PARTS], hi[PARTS];
            const int col = col0 + 8 * i + 2 * j;
            split_parts(row < t.rows && col < p.rank ? acc[8 * i + 2 * j] * scale : 0.f, lo);
            split_parts(row < t.rows && col + 1 < p.rank ? acc[8 * i + 2 * j + 1] * scale : 0.f, hi);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) w[q][j] = f2_to_bf16x2(lo[q], hi[q]);
          }
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            if (q < p.parts) *reinterpret_cast<uint4*>(held + q * p.rp + 8 * i) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        }
    }
  }
  if (CLUSTER) {
    // Each CTA sums a share of the rows over the cluster's shared memories.
    const int64_t ti = blockIdx.x / o.cluster;
    const Tile t = load_tile(p.table, ti, p.rows, p.n_adapters, p.ws);  // while the others come
    const float scale = o.scale[t.g];
    __syncthreads();
    cluster_sync();
    const int quads = p.rp / 4, row0 = TILE_ROWS * in_cluster / o.cluster, row1 = TILE_ROWS * (in_cluster + 1) / o.cluster;
    for (int e = threadIdx.x; e < (row1 - row0) * quads; e += THREADS) {
      const int r = row0 + e / quads, col = e % quads * 4;
      const uint32_t at = f.smem + (r * (p.rp + 4) + col) * 4;
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < o.cluster ? ld_cluster_f4(mapa_rank(at, k)) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 sum = v[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) sum = make_float4(sum.x + v[k].x, sum.y + v[k].y, sum.z + v[k].z, sum.w + v[k].w);
      store_held(p, o, t, scale, ti, r, col, sum);
    }
    cluster_leave();  // nobody still reads this CTA's shared memory
  }
  finish(f, COLS);
}

// The tiles that several CTAs share: four columns of a row to a thread.
__global__ void __launch_bounds__(256) k_to_rank_sum(Args p, ToRank o) {
  pdl_wait();
  pdl_launch_dependents();
  const int quads = p.rp / 4, ctas = TILE_ROWS * quads / 256;  // rp is a multiple of 16
  const int64_t ti = blockIdx.x / ctas;
  const int e = blockIdx.x % ctas * 256 + threadIdx.x, r = e / quads, col = e % quads * 4;
  const int c0 = cta_of(p.split, ti * o.blocks), c1 = cta_of(p.split, (ti + 1) * o.blocks - 1);
  if (c0 == c1) return;
  const Tile t = load_tile(p.table, ti, p.rows, p.n_adapters, p.ws);
  store_held(p, o, t, o.scale[t.g], ti, r, col, sum_slots(o.slots, (int64_t)TILE_ROWS * p.rp, c0, c1, e));
}

// ---------------------------------------------------------------------------------------
// The gradients' output tiles (see k_over_rows)
// ---------------------------------------------------------------------------------------
struct Grad {
  float* out;
  int64_t width;
  int64_t blocks;  // of the output, along the width
};
struct OverRows {
  Grad g[2];       // dB [n x rank], dA [rank x k]
  const int32_t* first;
  float* slots;
  int mtiles;      // 1, 2 or 4
  int whole;       // whole output tiles to each CTA, else equal shares of the units
  int cluster;     // CTAs to an output tile (CLUSTER)
  Split split;     // of the units
};

// Output tile `i` of all: its problem, adapter, columns and units (none if its adapter has no tiles, or the
// plan's table is wrong).
struct Output {
  bool second;
  int64_t g, block, first, count;
};
__device__ __forceinline__ Output output_at(const Args& p, const OverRows& o, int64_t i) {
  Output r;
  const int64_t outputs0 = o.g[0].blocks * p.n_adapters;
  r.second = i >= outputs0;
  const int64_t blocks = r.second ? o.g[1].blocks : o.g[0].blocks, v = r.second ? i - outputs0 : i;
  r.g = v / blocks;
  r.block = v % blocks;
  const int64_t f0 = o.first[r.g], f1 = o.first[r.g + 1];
  const bool fine = f0 >= 0 && f0 <= f1 && f1 <= p.n_tiles;
  if (!fine && threadIdx.x == 0) raise_status(p.ws, DIT_ERR_INVALID_ARG);
  r.count = fine ? f1 - f0 : 0;
  r.first = (r.second ? o.g[0].blocks * p.n_tiles : 0) + (fine ? blocks * f0 + r.block * r.count : 0);
  return r;
}
// Four values of an output tile of m_all columns: e counts them as the output lies, columns along memory for dA,
// the rank for dB.
__device__ __forceinline__ void store_grad(const Args& p, const OverRows& o, const Output& r, int m_all, int e, const float4& v) {
  if (r.second) {
    const int64_t width = o.g[1].width, col = r.block * m_all + e % (m_all / 4) * 4;
    const int j = e / (m_all / 4);
    if (j < p.rank && col < width) *reinterpret_cast<float4*>(o.g[1].out + (r.g * p.rank + j) * width + col) = v;
  } else {
    const int64_t width = o.g[0].width, col = r.block * m_all + e / (p.rp / 4);
    const int j = e % (p.rp / 4) * 4;
    if (col < width && j < p.rank) *reinterpret_cast<float4*>(o.g[0].out + (r.g * width + col) * p.rank + j) = v;
  }
}

// Adds up the output tiles that several CTAs of k_over_rows share, in the order of the CTAs; this CTA is number
// `cta` of `ctas`, with N threads.  A thread has the loads of four CTAs' values at PLACES places in flight: where
// few threads do it, behind k_from_rank, one place at a time took 10 us for one video's gradients.
template <int N, int PLACES>
__device__ __forceinline__ void add_up_grads(const Args& p, const OverRows& o, int cta, int ctas) {
  const int m_all = o.mtiles * 128, quads = m_all * p.rp / 4, chunks = (quads + PLACES * N - 1) / (PLACES * N);
  const int64_t slot = (int64_t)m_all * p.rp, all = (o.g[0].blocks + o.g[1].blocks) * p.n_adapters * chunks;
  for (int64_t c = cta; c < all; c += ctas) {
    const Output r = output_at(p, o, c / chunks);
    if (!r.count) continue;
    const int c0 = cta_of(o.split, r.first), c1 = cta_of(o.split, r.first + r.count - 1);
    if (c0 == c1) continue;
    const int first = (int)(c % chunks) * PLACES * N + threadIdx.x;
    float4 sum[PLACES];
#pragma unroll
    for (int i = 0; i < PLACES; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = c0; k <= c1; k += 4) {
      float4 v[4][PLACES];
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < PLACES; ++i)
          v[h][i] = k + h <= c1 && first + i * N < quads
                        ? __ldcg(reinterpret_cast<const float4*>(o.slots + slot_of(k + h, c0) * slot) + first + i * N)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < PLACES; ++i)
          sum[i] = make_float4(sum[i].x + v[h][i].x, sum[i].y + v[h][i].y, sum[i].z + v[h][i].z, sum[i].w + v[h][i].w);
    }
#pragma unroll
    for (int i = 0; i < PLACES; ++i)
      if (first + i * N < quads) store_grad(p, o, r, m_all, first + i * N, sum[i]);
  }
}

// ---------------------------------------------------------------------------------------
// From the rank: out += held W, out [rows x width], W = B^T (K-major) or A (MN-major).
//
// A job is a few consecutive blocks of columns of one tile.  CTAs take jobs from a counter: with equal
// shares the fastest SM was done after 138 us and the slowest after 190 (two videos), since SMs
// differ in their way to memory.  The tile of held stays in shared memory for its job; weights
// come through a ring, and so do the output's panels (128 rows x 128 bytes): loaded by TMA well
// ahead of the accumulators, updated in place and stored by TMA, so that neither direction waits
// for the other.  With a row to each thread, loads and stores straight to global memory took one
// wavefront per 32 bytes and the kernel ran at 3.6 TB/s, bound by them.  Panels of a tile that
// ends inside them are stored row by row, so that rows of other requests are never written.
// ---------------------------------------------------------------------------------------
struct FromRank {
  void* out;
  int64_t width;
  int nb, n_blocks;  // columns of a block (64 or 128), blocks along the width
  int per_job;       // blocks
  int64_t jobs, tile_jobs;  // all, and of a tile
  int panels, helds; // of the rings
  // The kernel before it is k_over_rows, whose gradients are no business of this one: its jobs fill the SMs that
  // are done there, without a wait for the others.  Not where out is what that kernel still reads.
  int early;
  int sums;  // behind k_over_rows: this kernel adds up what k_over_rows left in parts (no launch of its own for that)
};
// Where a job begins, and its blocks.
struct Job {
  int64_t tile;
  int block, blocks;
  __device__ __forceinline__ Job(const FromRank& o, int64_t j) {
    tile = j / o.tile_jobs;
    block = (int)(j % o.tile_jobs) * o.per_job;
    blocks = min(o.per_job, o.n_blocks - block);
  }
};
// The jobs as a consuming warp sees them: the next one's number, or -1 (no more, or a wait ran out).
struct JobQueue {
  Control* c;
  void* ws;
  uint32_t n;
  __device__ __forceinline__ int next() {
    const int s = n % JOBS;
    if (!warp_wait(smem_u32(&c->jfull[s]), (n / JOBS) & 1, ws, &c->abort)) return -1;
    const int job = *reinterpret_cast<volatile int*>(&c->job[s]);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&c->jempty[s]));
    ++n;
    return job;
  }
};

constexpr int FROM_THREADS = THREADS + 32;  // and a warp that stores

template <bool MN, bool BF16>
__global__ void __launch_bounds__(FROM_THREADS, 1)
    k_from_rank(const __grid_constant__ CUtensorMap m_held, const __grid_constant__ CUtensorMap m_w,
                const __grid_constant__ CUtensorMap m_out, Args p, FromRank o, OverRows rows) {
  extern __shared__ uint8_t raw[];
  const Frame f = frame(raw);
  Control* c = f.c;
  volatile int* abort = &c->abort;
  constexpr uint32_t COLS = 512;  // four accumulators of up to 128 columns
  if (threadIdx.x == 0) {
    prefetch_tmap(&m_held);
    prefetch_tmap(&m_w);
    prefetch_tmap(&m_out);
  }
  start(f, p.stages, COLS);
  const uint32_t tmem = c->tmem;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int steps = p.parts * p.rp / 16;           // of the contraction
  const int h_boxes = (p.parts * p.rp + 63) / 64;  // of 128 rows x 64 columns, 16 KB each
  const int w_boxes = MN ? o.nb / 64 : (p.rank + 63) / 64;
  const uint32_t box_bytes = MN ? p.rp * 128 : o.nb * 128;
  const uint32_t w_bytes = w_boxes * box_bytes, h_bytes = h_boxes * 16384;
  const uint32_t ring = f.smem + o.helds * h_bytes, panels = ring + p.stages * w_bytes;
  constexpr int ES = BF16 ? 2 : 4, PC = 128 / ES;  // columns of a panel
  // panels of a block (the last one may have fewer)
  auto panels_of = [&](int b) { return (int)min((int64_t)o.nb / PC, (o.width - (int64_t)b * o.nb + PC - 1) / PC); };

  if (warp == 0) {
    if (!p.stall) {
      uint32_t n = 0, tiles = 0, np = 0, announced = 0;
      int s = 0, q = 0;
      uint32_t sp = 1, qp = 1;  // parities of the rings' next waits
      bool ok = true, waited = o.early != 0;
      if (waited) pdl_launch_dependents();
      int64_t job = blockIdx.x;
      while (ok) {
        const int js = announced % JOBS;
        if (!warp_wait(smem_u32(&c->jempty[js]), ((announced / JOBS) & 1) ^ 1, p.ws, abort)) {
          ok = false;
          break;
        }
        const bool more = job < o.jobs;
        // the job after this one: its number is on its way while this one is loaded
        unsigned next = 0;
        if (lane == 0) {
          c->job[js] = more ? (int)job : -1;
          mbar_arrive(smem_u32(&c->jfull[js]));
        }
        ++announced;
        if (!more) break;
        const Job j(o, job);
        const Tile t = load_tile(p.table, j.tile, p.rows, p.n_adapters, p.ws);
        auto load_w = [&](int b) {
          const int n0 = b * o.nb;
          const uint32_t full = smem_u32(&c->full[s]);
          if (elect_one()) {
            mbar_expect_tx(full, w_bytes);
            for (int i = 0; i < w_boxes; ++i)
              tma_load_3d(ring + s * w_bytes + i * box_bytes, &m_w, full, MN ? n0 + i * 64 : i * 64, MN ? 0 : n0, t.g);
          }
          __syncwarp();
          ++n;
          if (++s == p.stages) {
            s = 0;
            sp ^= 1;
          }
        };
        auto load_panel = [&](int b, int i) {
          if (elect_one()) {
            mbar_expect_tx(smem_u32(&c->yfull[q]), 16384);
            tma_load_2d(panels + q * 16384, &m_out, smem_u32(&c->yfull[q]), b * o.nb + i * PC, t.row0);
          }
          __syncwarp();
          ++np;
          if (++q == o.panels) {
            q = 0;
            qp ^= 1;
          }
        };
        // Weights and old values of the first block are nobody's business that may still run: they come in while
        // the last of h is made.
        int done = 0;  // panels of the first block
        if (!waited) {
          load_w(j.block);
          for (const int all = min(panels_of(j.block), o.panels); done < all; ++done) load_panel(j.block, done);
          waited = true;
          pdl_wait();
          pdl_launch_dependents();
        }
        if (lane == 0) next = atomicAdd(ws_u32(p.ws, WS_JOBS), 1u);
        const int hs = tiles % o.helds;
        if (!warp_wait(smem_u32(&c->hempty[hs]), ((tiles / o.helds) & 1) ^ 1, p.ws, abort)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(smem_u32(&c->hfull[hs]), h_bytes);
          for (int i = 0; i < h_boxes; ++i)
            tma_load_2d(f.smem + hs * h_bytes + i * 16384, &m_held, smem_u32(&c->hfull[hs]), i * 64, (int)(j.tile * TILE_ROWS));
        }
        __syncwarp();
        ++tiles;
        for (int b = j.block; b < j.block + j.blocks && ok; ++b) {
          if (done == 0) {
            if (!warp_wait(smem_u32(&c->empty[s]), sp, p.ws, abort)) {
              ok = false;
              break;
            }
            load_w(b);
          }
          for (const int all = panels_of(b); done < all; ++done) {
            if (!warp_wait(smem_u32(&c->yempty[q]), qp, p.ws, abort)) {
              ok = false;
              break;
            }
            load_panel(b, done);
          }
          done = 0;
        }
        job = (int64_t)__shfl_sync(0xffffffffu, next, 0) + gridDim.x;
      }
      if (!ok) {
        await_copies(f, p.stages, n, p.ws);
        volatile int never = 0;
        for (uint32_t i = tiles > (uint32_t)o.helds ? tiles - o.helds : 0; i < tiles; ++i)
          mbar_wait(smem_u32(&c->hfull[i % o.helds]), (i / o.helds) & 1, p.ws, &never);
        for (uint32_t i = np > (uint32_t)o.panels ? np - o.panels : 0; i < np; ++i)
          mbar_wait(smem_u32(&c->yfull[i % o.panels]), (i / o.panels) & 1, p.ws, &never);
      }
    }
  } else if (warp == 1) {
    const uint32_t id = idesc(128, o.nb, false, MN);
    uint32_t n = 0, tiles = 0;
    const int rank_steps = p.rp / 16;
    JobQueue queue{c, p.ws, 0};
    bool ok = true;
    for (int job; ok && (job = queue.next()) >= 0; ++tiles) {
      const Job j(o, job);
      const int hs = tiles % o.helds;
      if (!warp_wait(smem_u32(&c->hfull[hs]), (tiles / o.helds) & 1, p.ws, abort)) break;
      for (int i = 0; i < j.blocks; ++i, ++n) {
        const int buf = n % ACCS, s = n % p.stages;
        if (!warp_wait(smem_u32(&c->dempty[buf]), ((n / ACCS) & 1) ^ 1, p.ws, abort) ||
            !warp_wait(smem_u32(&c->full[s]), (n / p.stages) & 1, p.ws, abort)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          fence_after();
          const uint32_t b0 = MN ? desc_mn(ring + s * w_bytes, box_bytes) : desc_k(ring + s * w_bytes);
          const uint32_t a0 = desc_k(f.smem + hs * h_bytes);
          // Every part meets the same weights; the small parts first, while truncation takes little of the sum.
          int k = rank_steps - 1;
          for (int q = steps - 1; q >= 0; --q) {
            const uint32_t b = b0 + (MN ? k * (2048 >> 4) : (k / 4) * (box_bytes >> 4) + (k % 4) * (32 >> 4));
            mma(tmem + buf * 128, a0 + (q / 4) * (16384 >> 4) + (q % 4) * (32 >> 4), b, id, q < steps - 1);
            if (--k < 0) k = rank_steps - 1;
          }
          mma_commit(smem_u32(&c->empty[s]));
          mma_commit(smem_u32(&c->dfull[buf]));
          if (i + 1 == j.blocks) mma_commit(smem_u32(&c->hempty[hs]));
        }
        __syncwarp();
      }
    }
    if (elect_one()) await_mmas(f, p.ws);
    __syncwarp();
  } else if (warp < 2 + EPI_WARPS) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    uint32_t n = 0;
    int q = 0;
    uint32_t qp = 0;
    JobQueue queue{c, p.ws, 0};
    bool ok = true;
    for (int job; ok && (job = queue.next()) >= 0;) {
      const Job j(o, job);
      for (int b = j.block; b < j.block + j.blocks && ok; ++b, ++n) {
        const int buf = n % ACCS, all = panels_of(b);
        if (!warp_wait(smem_u32(&c->dfull[buf]), (n / ACCS) & 1, p.ws, abort)) {
          ok = false;
          break;
        }
        fence_after();
        for (int i = 0; i < all; ++i) {
          __syncwarp();  // lane 0 is back from its arrival: the loads want all lanes
          constexpr int MINE = PC / 2;  // this thread's columns of the panel
          uint32_t r[MINE];
          const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 128 + i * PC + half * MINE;
#pragma unroll
          for (int k = 0; k < MINE / 8; ++k) tmem_ld8(at + 8 * k, r + 8 * k);
          if (!warp_wait(smem_u32(&c->yfull[q]), qp, p.ws, abort)) {
            ok = false;
            break;
          }
          tmem_wait();
#pragma unroll
          for (int k = 0; k < MINE / 8; ++k) pin8(r + 8 * k);
          if (i == all - 1) {  // everything is in registers: the accumulator is free
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c->dempty[buf]));
          }
          const uint32_t line = panels + q * 16384 + row * 128;
#pragma unroll
          for (int h = 0; h < 4; ++h) {  // 16-byte pieces of the row, swizzled as TMA lays them
            const uint32_t addr = line + (((half * 4 + h) ^ (row & 7)) << 4);
            uint4 v = lds128(addr);
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (BF16) {
                const float2 was = bf16x2_to_f2(w[k]);
                w[k] = f2_to_bf16x2(was.x + __uint_as_float(r[8 * h + 2 * k]), was.y + __uint_as_float(r[8 * h + 2 * k + 1]));
              } else {
                w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(r[4 * h + k]));
              }
            }
            sts128(addr, v);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&c->ydone[q]));
          if (++q == o.panels) {
            q = 0;
            qp ^= 1;
          }
        }
      }
    }
  } else {
    int q = 0;
    uint32_t qp = 0;
    int pending = -1;  // the panel that the last TMA store reads
    JobQueue queue{c, p.ws, 0};
    bool ok = true;
    for (int job; ok && (job = queue.next()) >= 0;) {
      const Job j(o, job);
      const Tile t = load_tile(p.table, j.tile, p.rows, p.n_adapters, p.ws);
      for (int b = j.block; b < j.block + j.blocks && ok; ++b)
        for (int i = 0, all = panels_of(b); i < all; ++i) {
          if (!warp_wait(smem_u32(&c->ydone[q]), qp, p.ws, abort)) {
            ok = false;
            break;
          }
          const int64_t col = (int64_t)b * o.nb + i * PC;
          const uint32_t src = panels + q * 16384;
          if (t.rows == TILE_ROWS) {
            if (lane == 0) {
              tma_store_2d(&m_out, src, (int)col, t.row0);
              if (pending >= 0) {
                tma_store_read_wait<1>();
                mbar_arrive(smem_u32(&c->yempty[pending]));
              }
            }
            pending = q;
          } else {
            const int piece = lane & 7;
            char* out = reinterpret_cast<char*>(o.out) + ((int64_t)t.row0 * o.width + col) * ES + piece * 16;
            if (col + piece * (16 / ES) < o.width)
              for (int r = lane >> 3; r < t.rows; r += 4)
                *reinterpret_cast<uint4*>(out + (int64_t)r * o.width * ES) = lds128(src + r * 128 + ((piece ^ (r & 7)) << 4));
            __syncwarp();
            if (lane == 0) {
              if (pending >= 0) {
                tma_store_read_wait<0>();
                mbar_arrive(smem_u32(&c->yempty[pending]));
              }
              mbar_arrive(smem_u32(&c->yempty[q]));
            }
            pending = -1;
          }
          if (++q == o.panels) {
            q = 0;
            qp ^= 1;
          }
        }
    }
    if (lane == 0) tma_store_wait();
  }
  pdl_wait();
  if (MN && o.sums) add_up_grads<FROM_THREADS, 4>(p, rows, blockIdx.x, gridDim.x);
  finish(f, COLS);
}

// ---------------------------------------------------------------------------------------
// Over the rows: dA[g] = e^T x and dB[g] = dy^T h over the rows of every adapter g.
//
// An output tile is 128 mtiles columns of x (or dy) by the whole rank; its units are the adapter's
// tiles of 128 rows.  The columns are M of the instructions (MN-major: x as it lies), the rank is N,
// and the parts of e (or h) are three instructions into one accumulator.  What bounds it is the
// traffic into shared memory: e is read again for every output tile, so the tiles are as wide as
// tensor memory holds twice over (512 columns up to rank 64, 256 above); accumulators are
// drained after every 128 rows, 24 instructions, while the other ones fill.
// ---------------------------------------------------------------------------------------
constexpr int ROW_EPI_WARPS = 16, ROW_THREADS = 96 + 32 * ROW_EPI_WARPS;  // and a warp that lets the next kernel launch
constexpr int ROW_STAGE = 32;       // rows of a stage
constexpr int ROW_BOX = ROW_STAGE * 128;  // bytes of a box of 64 columns

// The boxes of a stage of e or h: where parts lie side by side in 64 columns (ranks of 16, 32 and 64 and
// 128 after padding) they are loaded so, otherwise each part begins a box of its own, since an
// operand's chunks of 64 columns start at its first column.
struct HeldBoxes {
  int boxes, per_part, rp;
  __device__ __forceinline__ explicit HeldBoxes(int rp_) : rp(rp_) {
    per_part = 64 % rp == 0 ? 0 : (rp + 63) / 64;
    boxes = per_part ? PARTS * per_part : (PARTS * rp + 63) / 64;
  }
  __device__ __forceinline__ uint32_t offset(int part) const {
    return per_part ? part * per_part * ROW_BOX : part * rp / 64 * ROW_BOX + part * rp % 64 * 2;
  }
};

// A unit of k_over_rows: its output tile (problem, adapter, columns) and tile of rows.
struct RowsUnit {
  bool ok;
  int problem, g;
  int64_t block;         // of columns
  int64_t tile;          // of the plan
  int64_t first, count;  // first unit and units of the output tile
};
__device__ __forceinline__ RowsUnit rows_unit(const Args& p, const OverRows& o, int64_t u) {
  RowsUnit r;
  const int64_t units0 = o.g[0].blocks * p.n_tiles;
  r.problem = u >= units0;  // 0: dB, 1: dA
  const int64_t base = r.problem ? units0 : 0, blocks = r.problem ? o.g[1].blocks : o.g[0].blocks, v = u - base;
  // An adapter's units follow one another and its tiles are [f0, f1): v / blocks is one of its tiles.
  r.g = p.table[4 * (v / blocks) + 2];
  r.ok = r.g >= 0 && r.g < p.n_adapters;
  if (!r.ok) return r;
  const int64_t f0 = o.first[r.g], f1 = o.first[r.g + 1];
  r.ok = f0 >= 0 && f0 <= v / blocks && v / blocks < f1 && f1 <= p.n_tiles;
  if (!r.ok) return r;
  r.count = f1 - f0;
  r.block = (v - blocks * f0) / r.count;
  r.first = base + blocks * f0 + r.block * r.count;
  r.tile = f0 + (u - r.first);
  return r;
}
// MT: tiles of 128 columns, 1, 2 or 4.  An output tile's rows fall to one CTA, to a cluster (CLUSTER: few output
// tiles; the partial results are summed through distributed shared memory), or to the CTAs whose equal
// shares of all units it meets (summed by k_over_rows_sum).
template <int MT, bool CLUSTER>
__global__ void __launch_bounds__(ROW_THREADS, 1)
    k_over_rows(const __grid_constant__ CUtensorMap m_x, const __grid_constant__ CUtensorMap m_e,
                const __grid_constant__ CUtensorMap m_dy, const __grid_constant__ CUtensorMap m_h, Args p, OverRows o) {
  extern __shared__ uint8_t raw[];
  const Frame f = frame(raw);
  Control* c = f.c;
  volatile int* abort = &c->abort;
  constexpr uint32_t COLS = 512;
  if (threadIdx.x == 0) {
    prefetch_tmap(&m_x);
    prefetch_tmap(&m_e);
    prefetch_tmap(&m_dy);
    prefetch_tmap(&m_h);
  }
  start(f, p.stages, COLS, ROW_EPI_WARPS);
  const uint32_t tmem = c->tmem;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const HeldBoxes hb(p.rp);
  const int a_boxes = 2 * MT;
  const uint32_t stage_bytes = (a_boxes + hb.boxes) * ROW_BOX;
  int64_t u0, u1;
  Output mine{};
  const int in_cluster = CLUSTER ? (int)cluster_rank() : 0;
  if (CLUSTER) {
    mine = output_at(p, o, blockIdx.x / o.cluster);
    u0 = mine.first + mine.count * in_cluster / o.cluster;
    u1 = mine.first + mine.count * (in_cluster + 1) / o.cluster;
  } else if (o.whole) {
    const int64_t outputs = (o.g[0].blocks + o.g[1].blocks) * p.n_adapters;
    const int64_t i = outputs * (blockIdx.x + 1) / gridDim.x;
    u0 = output_at(p, o, outputs * blockIdx.x / gridDim.x).first;
    u1 = i < outputs ? output_at(p, o, i).first : p.split.units;
  } else {
    u0 = first_unit(p.split, blockIdx.x);
    u1 = first_unit(p.split, blockIdx.x + 1);
  }

  if (warp == 0) {
    if (!p.stall) {
      uint32_t parity = 1, n = 0;
      int s = 0;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok;) {
        const RowsUnit r = rows_unit(p, o, u);
        if (!r.ok) {
          raise_status(p.ws, DIT_ERR_INVALID_ARG);
          ++u;
          continue;
        }
        if (r.problem) pdl_wait();  // e is the previous kernel's
        const int64_t end = min(u1, r.first + r.count);
        const int4* entry = reinterpret_cast<const int4*>(p.table) + r.tile;
        const CUtensorMap *wide = r.problem ? &m_x : &m_dy, *narrow = r.problem ? &m_e : &m_h;
        const int col = (int)(r.block * a_boxes) * 64;
        int held_row = (int)(r.tile * TILE_ROWS);
        int4 next = *entry;
        for (; u < end && ok; ++u) {
          const Tile t = check_tile(next, p.rows, p.n_adapters, p.ws);
          if (u + 1 < end) next = *++entry;  // used a tile later
          for (int h = 0; h < TILE_ROWS; h += ROW_STAGE, held_row += ROW_STAGE, ++n) {
            if (!warp_wait(smem_u32(&c->empty[s]), parity, p.ws, abort)) {
              ok = false;
              break;
            }
            const uint32_t full = smem_u32(&c->full[s]);
            if (elect_one()) {
              c->valid[s] = min(ROW_STAGE, max(0, t.rows - h));
              mbar_expect_tx(full, stage_bytes);
              uint32_t dst = f.smem + s * stage_bytes;
              for (int i = 0; i < a_boxes; ++i, dst += ROW_BOX) tma_load_2d(dst, wide, full, col + i * 64, t.row0 + h);
              if (hb.per_part) {
                for (int q = 0; q < PARTS; ++q)
                  for (int i = 0; i < hb.per_part; ++i, dst += ROW_BOX)
                    tma_load_2d(dst, narrow, full, q * p.rp + i * 64, held_row);
              } else {
                for (int i = 0; i < hb.boxes; ++i, dst += ROW_BOX) tma_load_2d(dst, narrow, full, i * 64, held_row);
              }
            }
            __syncwarp();
            if (++s == p.stages) {
              s = 0;
              parity ^= 1;
            }
          }
        }
      }
      if (!ok) await_copies(f, p.stages, n, p.ws);
    }
  } else if (warp == 1) {
    const uint32_t id = idesc(128, p.rp, true, true);
    const uint32_t part_at[PARTS] = {hb.offset(0) >> 4, hb.offset(1) >> 4, hb.offset(2) >> 4};
    uint32_t parity = 0, chunk = 0;
    int s = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const RowsUnit r = rows_unit(p, o, u);
      if (!r.ok) {
        ++u;
        continue;
      }
      const int todo = uniform((int)(min(u1, r.first + r.count) - u));
      u += todo;
      for (int t = 0; t < todo && ok; ++t, ++chunk) {
        const uint32_t buf = chunk & 1, d = tmem + buf * MT * p.rp;
        if (!warp_wait(smem_u32(&c->dempty[buf]), ((chunk >> 1) & 1) ^ 1, p.ws, abort)) {
          ok = false;
          break;
        }
        fence_after();
#pragma unroll
        for (int h = 0; h < TILE_ROWS / ROW_STAGE; ++h) {
          if (!warp_wait(smem_u32(&c->full[s]), parity, p.ws, abort)) {
            ok = false;
            break;
          }
          const uint32_t a = f.smem + s * stage_bytes;
          const int valid = uniform(c->valid[s]);
          if (valid < ROW_STAGE) {
            // rows of other requests behind the tile's own: zeros, so that what they hold stays out
            for (int k = valid * 8 + lane; k < ROW_STAGE * 8; k += 32)
              for (int q = 0; q < a_boxes; ++q) sts128(a + q * ROW_BOX + k * 16, make_uint4(0, 0, 0, 0));
            fence_proxy_async();
            __syncwarp();
          }
          if (elect_one()) {
            fence_after();
            const uint32_t ad = desc_mn(a, ROW_BOX), bd = desc_mn(a + a_boxes * ROW_BOX, ROW_BOX);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int j = 0; j < ROW_STAGE / 16; ++j) {  // the small parts first
                const uint32_t dd = d + mt * p.rp, aj = ad + (mt * 2 * ROW_BOX + j * 2048) / 16, bj = bd + j * (2048 / 16);
                static_assert(PARTS == 3, "three MMAs with one A");
                mma<KEEP_FIRST>(dd, aj, bj + part_at[2], id, h > 0 || j > 0);
                mma<KEEP_MIDDLE>(dd, aj, bj + part_at[1], id, true);
                mma<KEEP_LAST>(dd, aj, bj + part_at[0], id, true);
              }
            mma_commit(smem_u32(&c->empty[s]));
            if (h + 1 == TILE_ROWS / ROW_STAGE) mma_commit(smem_u32(&c->dfull[buf]));
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
    }
    if (elect_one()) await_mmas(f, p.ws);
    __syncwarp();
  } else if (warp == 2 + ROW_EPI_WARPS) {
    pdl_wait();
    pdl_launch_dependents();
  } else {
    // Sixteen warps: four to the quarters of 128 columns; the four groups take an M tile each (mtiles 4), half
    // the rank of two, or half of one (then two groups have nothing).
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    const int mt = MT == 4 ? group : MT == 2 ? group >> 1 : 0;
    const int nc = MT == 4 ? p.rp : MT == 2 || group < 2 ? p.rp / 2 : 0;
    const int col0 = MT == 4 ? 0 : (group & 1) * nc;
    const int m = mt * 128 + quarter * 32 + lane;  // column of x or dy within the output tile
    const int m_all = MT * 128;
    uint32_t chunk = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const RowsUnit r = rows_unit(p, o, u);
      if (!r.ok) {
        ++u;
        continue;
      }
      const int64_t end = min(u1, r.first + r.count);
      const bool whole = u == r.first && end == r.first + r.count;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (; u < end; ++u, ++chunk) {
        const uint32_t buf = chunk & 1;
        if (!warp_wait(smem_u32(&c->dfull[buf]), (chunk >> 1) & 1, p.ws, abort)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (buf * MT + mt) * p.rp + col0;
#pragma unroll
        for (int i = 0; i < 64; i += 16) {
          if (i >= nc) break;
          uint32_t v[16];
          tmem_ld8(at + i, v);
          if (i + 8 < nc) tmem_ld8(at + i + 8, v + 8);
          tmem_wait();
          pin8(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i + j] += __uint_as_float(v[j]);
          if (i + 8 < nc) {
            pin8(v + 8);
#pragma unroll
            for (int j = 8; j < 16; ++j) acc[i + j] += __uint_as_float(v[j]);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c->dempty[buf]));
      }
      if (!ok) break;
      pdl_wait();  // what is written from here on may still be read by the previous kernel
      if (CLUSTER) {  // every MMA of this CTA has read its operands: their place takes the partial result
        if (!r.problem) {
          const uint32_t at = f.smem + (m * (p.rp + 4) + col0) * 4;
#pragma unroll
          for (int i = 0; i < 64; i += 4)
            if (i < nc)
              sts128(at + 4 * i, make_uint4(__float_as_uint(acc[i]), __float_as_uint(acc[i + 1]), __float_as_uint(acc[i + 2]),
                                            __float_as_uint(acc[i + 3])));
        } else {
          const uint32_t at = f.smem + (col0 * m_all + m) * 4;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < nc) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * i * m_all), "f"(acc[i]) : "memory");
        }
        continue;
      }
      if (!whole) {
        const int c0 = cta_of(p.split, r.first);
        const int64_t slot = (int64_t)m_all * p.rp;
        // as the output lies: columns along memory for dA, the rank for dB
        float* mine = o.slots + slot_of(blockIdx.x, c0) * slot;
        if (!r.problem) {
          mine += (int64_t)m * p.rp + col0;
#pragma unroll
          for (int i = 0; i < 64; i += 4)
            if (i < nc) *reinterpret_cast<float4*>(mine + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        } else {
          mine += col0 * m_all + m;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < nc) mine[i * m_all] = acc[i];
        }
        continue;
      }
      const int64_t col = r.block * m_all + m, width = r.problem ? o.g[1].width : o.g[0].width;
      if (col < width) {
        float* out = (r.problem ? o.g[1].out : o.g[0].out) + (int64_t)r.g * p.rank * width;
        if (!r.problem) {  // dB: the rank runs along memory, and is a multiple of 8
          out += col * p.rank + col0;
#pragma unroll
          for (int i = 0; i < 64; i += 4)
            if (i < nc && col0 + i < p.rank) *reinterpret_cast<float4*>(out + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        } else {
          out += col + col0 * width;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < nc && col0 + i < p.rank) out[i * width] = acc[i];
        }
      }
    }
  }
  if (CLUSTER) {
    // Each CTA sums a share of the output tile over the shared memories of the CTAs that have units of it.
    __syncthreads();
    cluster_sync();
    constexpr int m_all = MT * 128;
    const int all = m_all * p.rp / 4, quads = p.rp / 4;
    uint32_t with = 0;
    for (int k = 0; k < o.cluster; ++k)
      if (mine.count * (k + 1) / o.cluster > mine.count * k / o.cluster) with |= 1u << k;
    if (with)
      for (int e = all * in_cluster / o.cluster + threadIdx.x; e < all * (in_cluster + 1) / o.cluster; e += ROW_THREADS) {
        const uint32_t at = f.smem + (mine.second ? e * 16 : (e / quads * (p.rp + 4) + e % quads * 4) * 4);
        float4 v[8], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = with >> k & 1 ? ld_cluster_f4(mapa_rank(at, k)) : sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = make_float4(sum.x + v[k].x, sum.y + v[k].y, sum.z + v[k].z, sum.w + v[k].w);
        store_grad(p, o, mine, m_all, e, sum);
      }
  }
  pdl_wait();
  // adapters without rows
  for (int g = blockIdx.x; g < p.n_adapters; g += gridDim.x) {
    if (o.first[g] != o.first[g + 1]) continue;
    for (int q = 0; q < 2; ++q) {
      const int64_t n = p.rank * (q ? o.g[1].width : o.g[0].width);
      float4* out = reinterpret_cast<float4*>((q ? o.g[1].out : o.g[0].out) + g * n);
      for (int64_t i = threadIdx.x; i < n / 4; i += ROW_THREADS) out[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if (CLUSTER) {
    cluster_leave();  // nobody still reads this CTA's shared memory
  }
  finish(f, COLS);
}

__global__ void __launch_bounds__(256) k_over_rows_sum(Args p, OverRows o) {
  pdl_launch_dependents();
  pdl_wait();
  add_up_grads<256, 1>(p, o, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------------
static Args args_of(const dit_adapter_plan_t& plan, const int32_t* table, int rank, void* ws) {
  Args p = {};
  p.table = table;
  p.rows = plan.rows;
  p.n_adapters = plan.n_adapters;
  p.n_tiles = plan.n_tiles;
  p.rank = rank;
  p.rp = padded_rank(rank);
  p.ws = ws;
  p.stall = test_stall();
  return p;
}
static int stages_for(uint32_t room, uint32_t stage_bytes) {
  const uint32_t s = room / stage_bytes;
  return (int)(s < (uint32_t)MAX_STAGES ? s : (uint32_t)MAX_STAGES);
}
template <auto KERN>
static bool allow_smem() {
  static OncePerDevice once;
  return opt_in_smem(once, KERN, SMEM_BYTES) == cudaSuccess;
}
static bool map_rows(CUtensorMap* m, const void* base, int64_t width, int64_t rows, uint32_t box_rows) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<void*>(base), (uint64_t)width, (uint64_t)rows,
                        (uint64_t)width * 2, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// What the cuts of the work are chosen by: a CTA's own time for its largest share at an SM's rate, or
// all CTAs' at the device's, whichever is longer; shared outputs add a kernel that sums them, which
// takes longer the more CTAs have shared.
// (12000 rows of 1920 columns at rank 32 took 6 us less a forward call with whole tiles than with equal shares,
// though those keep only 94 SMs busy; 4160 rows 3 us less, and 4 less again in clusters of four; 130 rows
// take 13.5 us in equal shares, 15.7 whole, and 9.6 in clusters of eight.)
constexpr double SM_BYTES_NS = 90, DEVICE_BYTES_NS = 6500;
constexpr double CLUSTER_NS = 2000, CLUSTER_ROWS_NS = 3000;  // what a cluster takes to sum h or e, or a gradient
static double shared_ns(int ctas) { return 3700 + 12.0 * ctas; }
static double time_ns(double share_ns, double bytes) {
  const double all = bytes / DEVICE_BYTES_NS;
  return share_ns > all ? share_ns : all;
}
// how many clusters of 2 to 8 CTAs the device runs at a time
struct Clusters {
  int most[7];
};
struct RankSplit {
  Split split;
  int cluster;  // 0: the sizes do not allow what is forced
};
// Test hook: DIT6_TEST_CUT="cut,n,width" forces the cut of the work of k_to_rank and k_over_rows, where the sizes allow
// it (else the call is DIT_ERR_UNSUPPORTED): 1 whole outputs to n CTAs, 2 equal shares of the units to n CTAs (0: as
// many as there are), 3 clusters of n CTAs; and the columns of k_over_rows' output tiles, 128 times width (0: chosen).
enum { CUT_CHOSEN, CUT_WHOLE, CUT_SHARES, CUT_CLUSTERS };
struct ForcedCut {
  int cut, n, width;
};
static ForcedCut forced_cut() {
  ForcedCut f{CUT_CHOSEN, 0, 0};
  const char* e = getenv("DIT6_TEST_CUT");
  if (e && sscanf(e, "%d,%d,%d", &f.cut, &f.n, &f.width) != 3) f = ForcedCut{CUT_CHOSEN, 0, 0};
  return f;
}
static RankSplit split_to_rank(int64_t tiles, int64_t blocks, int64_t unit_bytes, const Clusters& clusters,
                               const ForcedCut& force) {
  constexpr int64_t LEAST = 4;  // units of an equal share
  const int64_t sms = num_sms();
  if (force.cut != CUT_CHOSEN) {
    const int64_t grain = force.cut == CUT_WHOLE ? blocks : 1;
    const int ctas = force.cut != CUT_CLUSTERS && force.n > 0 && force.n < sms ? force.n : (int)sms, c = force.n;
    const bool fits = force.cut != CUT_CLUSTERS || (c >= 2 && c <= 8 && blocks >= c && tiles <= clusters.most[c - 2]);
    return RankSplit{split_units(tiles * blocks, grain, grain, ctas), !fits ? 0 : force.cut == CUT_CLUSTERS ? c : 1};
  }
  const Split s = split_units(tiles * blocks, 1, LEAST, (int)sms);
  const double unit_ns = (double)unit_bytes / SM_BYTES_NS;
  const double bytes = (double)s.units * (16384 + (unit_bytes - 16384) / 2.5);  // the weights come out of L2, faster
  const double whole = time_ns((double)((tiles + sms - 1) / sms * blocks) * unit_ns, bytes);
  const double shared = time_ns((double)s.units / s.ctas * unit_ns, bytes) + shared_ns(s.ctas);
  RankSplit best{whole <= shared ? split_units(s.units, blocks, blocks, (int)sms) : s, 1};
  double ns = whole <= shared ? whole : shared;
  for (int i = 0; i < 7; ++i) {
    const int c = 2 + i;
    const double t = time_ns((double)((blocks + c - 1) / c) * unit_ns, bytes) + CLUSTER_NS;
    if (tiles <= clusters.most[i] && blocks >= 2 * c && t < ns) {
      ns = t;
      best.cluster = c;
    }
  }
  return best;
}
template <auto KERN, int N_THREADS>
static Clusters max_clusters() {
  static Clusters of_device[OncePerDevice::DEVICES];
  static OncePerDevice once;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= OncePerDevice::DEVICES) return Clusters{};
  const cudaError_t e = once.run(device, [device] {
    if (!allow_smem<KERN>()) return cudaErrorInvalidValue;
    for (int i = 0; i < 7; ++i) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2u + i;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(num_sms() / (2 + i) * (2 + i));
      cfg.blockDim = dim3(N_THREADS);
      cfg.dynamicSmemBytes = SMEM_BYTES;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      const cudaError_t bad = cudaOccupancyMaxActiveClusters(&of_device[device].most[i], KERN, &cfg);
      if (bad != cudaSuccess) return bad;
    }
    return cudaSuccess;
  });
  return e == cudaSuccess ? of_device[device] : Clusters{};
}

// held = scale * (in W^T); MN: w is [n_adapters][width][rank], else [n_adapters][rank][width]
template <bool MN>
static dit_status to_rank(Args p, const void* in, int64_t width, const void* w, const float* scale, void* held, int parts,
                          void* slots, const ForcedCut& force, cudaStream_t st) {
  CUtensorMap m_in, m_w;
  const bool maps = map_rows(&m_in, in, width, p.rows, TILE_ROWS) &&
                    (MN ? encode_tmap_bf16_3d(&m_w, w, p.rank, width, p.n_adapters, 64)
                        : encode_tmap_bf16_3d(&m_w, w, width, p.rank, p.n_adapters, p.rp));
  if (!maps) return DIT_ERR_CUDA;
  ToRank o{scale, reinterpret_cast<__nv_bfloat16*>(held), reinterpret_cast<float*>(slots), (int)((width + 63) / 64), 1};
  p.parts = parts;
  const uint32_t stage_bytes = 16384 + (MN ? (p.rank + 63) / 64 * 8192 : p.rp * 128);
  p.stages = stages_for(RING_BYTES, stage_bytes);
  const RankSplit cut = split_to_rank(p.n_tiles, o.blocks, stage_bytes, max_clusters<k_to_rank<MN, true>, THREADS>(), force);
  if (!cut.cluster) return DIT_ERR_UNSUPPORTED;
  p.split = cut.split;
  o.cluster = cut.cluster;
  if (!(cut.cluster > 1 ? allow_smem<k_to_rank<MN, true>>() : allow_smem<k_to_rank<MN, false>>())) return DIT_ERR_CUDA;
  if (cut.cluster > 1)
    return launch_pdl(k_to_rank<MN, true>, dim3((unsigned)(p.n_tiles * cut.cluster)), dim3(THREADS), SMEM_BYTES, st,
                      (unsigned)cut.cluster, m_in, m_w, p, o) == cudaSuccess
               ? DIT_OK
               : DIT_ERR_CUDA;
  if (launch_pdl(k_to_rank<MN, false>, dim3(p.split.ctas), dim3(THREADS), SMEM_BYTES, st, 1, m_in, m_w, p, o) != cudaSuccess)
    return DIT_ERR_CUDA;
  if (p.split.grain == 1 && p.split.ctas > 1 &&  // shares may end inside tiles
      launch_pdl(k_to_rank_sum, dim3((unsigned)(p.n_tiles * (TILE_ROWS * p.rp / 1024))), dim3(256), 0, st, 1, p, o) != cudaSuccess)
    return DIT_ERR_CUDA;
  return DIT_OK;
}

// out += held W; MN: w is [n_adapters][rank][width], else [n_adapters][width][rank]; held has `held_parts` parts
template <bool MN, bool BF16>
static dit_status from_rank(Args p, const void* held, int held_parts, const void* w, void* out, int64_t width, const OverRows* after,
                            bool early, cudaStream_t st) {
  const int64_t sms = num_sms();
  FromRank o{out, width, 128, 0, 1, 0, 0, 0, 1, early ? 1 : 0, after && !after->whole && after->split.ctas > 1 ? 1 : 0};
  p.parts = BF16 ? 2 : PARTS;
  const uint32_t h_bytes = (p.parts * p.rp + 63) / 64 * 16384;
  auto bytes_of = [&](int nb) { return (uint32_t)(MN ? nb / 64 * p.rp * 128 : (p.rank + 63) / 64 * nb * 128); };
  // narrower blocks where all of them run at once, or where wide ones leave the panels too little room
  if ((int64_t)p.n_tiles * ((width + 63) / 64) <= sms || RING_BYTES < h_bytes + 2 * bytes_of(128) + 5 * 16384) o.nb = 64;
  const uint32_t w_bytes = bytes_of(o.nb);
  p.stages = 2;
  // two tiles of held if that leaves six panels; then up to four stages of weights
  if (RING_BYTES >= 2 * h_bytes + p.stages * w_bytes + 6 * 16384) o.helds = 2;
  const uint32_t room = RING_BYTES - o.helds * h_bytes;
  while (p.stages < 4 && room >= (p.stages + 1) * w_bytes + MAX_PANELS * 16384) ++p.stages;
  o.panels = (int)((room - p.stages * w_bytes) / 16384);
  if (o.panels > MAX_PANELS) o.panels = MAX_PANELS;
  o.n_blocks = (int)((width + o.nb - 1) / o.nb);
  // Jobs of up to eight blocks, sixteen jobs to an SM where there are that many blocks; but enough blocks to a
  // job that its tile of held (read again for each job) stays behind what it updates, as long as
  // every SM has two jobs.  (17776 x 1920 in fp32 at rank 128: 90 us with one block, 79 with four.)  At least two
  // blocks even where the tile of held is small, since a job's number is a round trip to memory
  // (12000 x 1920 in bf16 at rank 32, forward: 37.4 us with one block, 34.1 with two, 35.4 with three).
  const int64_t blocks = (int64_t)p.n_tiles * o.n_blocks, even = blocks / (16 * sms), two = blocks / (2 * sms);
  int64_t per_job = 1 + h_bytes / (o.nb * TILE_ROWS * (BF16 ? 2 : 4));
  if (per_job < 2) per_job = 2;
  if (per_job > two) per_job = two;
  if (per_job < even) per_job = even;
  o.per_job = per_job < 1 ? 1 : per_job > 8 ? 8 : (int)per_job;
  o.tile_jobs = (o.n_blocks + o.per_job - 1) / o.per_job;
  o.jobs = p.n_tiles * o.tile_jobs;
  if (o.jobs > 0x7fffff00) return DIT_ERR_UNSUPPORTED;
  const int64_t ctas = o.jobs < sms ? o.jobs : sms;
  CUtensorMap m_held, m_w, m_out;
  const bool maps = encode_tmap_2d(&m_out, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out,
                                   (uint64_t)width, (uint64_t)p.rows, (uint64_t)width * (BF16 ? 2 : 4), BF16 ? 64 : 32,
                                   TILE_ROWS, CU_TENSOR_MAP_SWIZZLE_128B) &&
                    map_rows(&m_held, held, held_parts * p.rp, (int64_t)p.n_tiles * TILE_ROWS, TILE_ROWS) &&
                    (MN ? encode_tmap_bf16_3d(&m_w, w, width, p.rank, p.n_adapters, p.rp)
                        : encode_tmap_bf16_3d(&m_w, w, p.rank, width, p.n_adapters, o.nb));
  if (!maps || !allow_smem<k_from_rank<MN, BF16>>()) return DIT_ERR_CUDA;
  return launch_pdl(k_from_rank<MN, BF16>, dim3((unsigned)ctas), dim3(FROM_THREADS), SMEM_BYTES, st, 1, m_held, m_w, m_out, p,
                    o, after ? *after : OverRows{}) == cudaSuccess
             ? DIT_OK
             : DIT_ERR_CUDA;
}
template <bool MN>
static dit_status from_rank(const Args& p, const void* held, int held_parts, const void* w, void* out, dit_dtype dt,
                            int64_t width, const OverRows* after, bool early, cudaStream_t st) {
  return dt == DIT_BF16 ? from_rank<MN, true>(p, held, held_parts, w, out, width, after, early, st)
                        : from_rank<MN, false>(p, held, held_parts, w, out, width, after, early, st);
}

}  // namespace lora
}  // namespace dit6

using namespace dit6;
using namespace dit6::lora;

extern "C" dit_status dit_lora_forward(const dit_adapter_plan_t* plan, const int32_t* table, const void* x, const void* a,
                                       const void* b, const float* scale, int rank, int64_t k, int64_t n, void* y,
                                       dit_dtype y_dt, void* saved, size_t saved_bytes, void* scratch,
                                       size_t scratch_bytes, void* ws, size_t ws_bytes, dit_stream_t stream) {
  const dit_status bad = check_common(plan, table, x, a, b, scale, rank, k, n, scratch, scratch_bytes, ws, ws_bytes);
  if (bad != DIT_OK) return bad;
  if ((!y && plan->rows > 0) || (y_dt != DIT_F32 && y_dt != DIT_BF16)) return DIT_ERR_INVALID_ARG;
  if (saved && (!plan->training || saved == scratch || saved_bytes < held_bytes(plan->n_tiles, rank)))
    return DIT_ERR_INVALID_ARG;
  if (!aligned32(y) || !aligned32(saved)) return DIT_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  dit_status s = DIT_OK;
  if (plan->n_tiles) {
    const Args p = args_of(*plan, table, rank, ws);
    void* held = saved ? saved : scratch;
    char* slots = reinterpret_cast<char*>(scratch) + held_bytes(plan->n_tiles, rank);
    const int parts = saved || y_dt == DIT_F32 ? PARTS : 2;
    s = to_rank<false>(p, x, k, a, scale, held, parts, slots, forced_cut(), st);
    if (s == DIT_OK) s = from_rank<false>(p, held, parts, b, y, y_dt, n, nullptr, false, st);
  }
  if (s == DIT_OK) s = small_tiles(*plan, table, x, a, b, scale, rank, k, n, y, y_dt, ws, st);
  return s;
}

extern "C" dit_status dit_lora_backward(const dit_adapter_plan_t* plan, const int32_t* table, const void* x,
                                        const void* dy, const void* a, const void* b, const float* scale, int rank,
                                        int64_t k, int64_t n, const void* saved, size_t saved_bytes, void* dx,
                                        dit_dtype dx_dt, float* da, float* db, void* scratch, size_t scratch_bytes,
                                        void* ws, size_t ws_bytes, dit_stream_t stream) {
  const dit_status bad = check_common(plan, table, x, a, b, scale, rank, k, n, scratch, scratch_bytes, ws, ws_bytes);
  if (bad != DIT_OK) return bad;
  if (!plan->training || (!dy && plan->rows > 0) || !da || !db || (dx_dt != DIT_F32 && dx_dt != DIT_BF16) ||
      saved_bytes < held_bytes(plan->n_tiles, rank) || (plan->n_tiles > 0 && (!saved || saved == scratch)))
    return DIT_ERR_INVALID_ARG;
  if (!aligned32(dy) || !aligned32(saved) || !aligned32(dx) || !aligned32(da) || !aligned32(db)) return DIT_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Args plain = args_of(*plan, table, rank, ws);
  Args p = plain;
  char* slots = reinterpret_cast<char*>(scratch) + held_bytes(plan->n_tiles, rank);
  if (!plan->n_tiles) {  // no row has an adapter: every gradient is zero
    const bool ok = cudaMemsetAsync(da, 0, (size_t)plan->n_adapters * rank * k * 4, st) == cudaSuccess &&
                    cudaMemsetAsync(db, 0, (size_t)plan->n_adapters * rank * n * 4, st) == cudaSuccess;
    return ok ? DIT_OK : DIT_ERR_CUDA;
  }
  const ForcedCut force = forced_cut();
  dit_status s = to_rank<true>(p, dy, n, b, scale, scratch, PARTS, slots, force, st);
  if (s != DIT_OK) return s;

  OverRows o{};
  o.first = table + off_first(*plan);
  o.slots = reinterpret_cast<float*>(slots);
  // The widths of the output tiles, and whole output tiles to each CTA or equal shares of the units.  A unit takes
  // its bytes' time or its 24 MMAs' for each 128 columns (25 ns measured up to rank 64, 50 at 128).
  {
    const int64_t sms = num_sms(), boxes = 64 % p.rp == 0 ? (PARTS * p.rp + 63) / 64 : PARTS * ((p.rp + 63) / 64);
    const Clusters clusters = max_clusters<k_over_rows<2, true>, ROW_THREADS>();
    double best = -1;
    for (int mt = p.rp <= 64 ? 4 : 2; mt >= 1; mt /= 2) {
      if (force.width && mt != force.width) continue;
      const int64_t bk = (k + 128 * mt - 1) / (128 * mt), bn = (n + 128 * mt - 1) / (128 * mt);
      const int64_t unit = (2 * mt + boxes) * 16384, outputs = (bk + bn) * p.n_adapters, units = (bk + bn) * p.n_tiles;
      const double mma_ns = mt * 24 * (p.rp <= 64 ? 25.0 : 25.0 * p.rp / 64), load_ns = (double)unit / SM_BYTES_NS;
      const double unit_ns = mma_ns > load_ns ? mma_ns : load_ns;
      const double bytes = (double)units * 16384 * (2 * mt + boxes / 2.5);  // e and h come out of L2, faster
      const Split s = split_units(units, 1, 1, (int)sms);
      const double partial = 2.0 * s.ctas * mt * 128 * p.rp * 4;  // written and read again
      const double cost[2] = {time_ns((double)units / s.ctas * unit_ns, bytes) + shared_ns(s.ctas) + partial / 3000,
                              time_ns((double)((outputs + sms - 1) / sms * plan->most_tiles) * unit_ns, bytes)};
      auto take = [&](double ns, int whole, int cluster, int64_t ctas) {
        if (best >= 0 && ns >= best) return;
        best = ns;
        o.mtiles = mt;
        o.whole = whole;
        o.cluster = cluster;
        o.g[0] = Grad{db, n, bn};
        o.g[1] = Grad{da, k, bk};
        p.split = s;
        p.split.ctas = (int)ctas;
      };
      if (force.cut != CUT_CHOSEN) {
        const int ctas = force.n > 0 && force.n < sms ? force.n : (int)sms, c = force.n;
        if (force.cut == CUT_WHOLE) take(0, 1, 1, outputs < ctas ? outputs : ctas);
        if (force.cut == CUT_SHARES) take(0, 0, 1, split_units(units, 1, 1, ctas).ctas);
        if (force.cut == CUT_CLUSTERS && c >= 2 && c <= 8 && outputs <= clusters.most[c - 2]) take(0, 1, c, outputs * c);
        continue;
      }
      take(cost[0], 0, 1, s.ctas);
      take(cost[1], 1, 1, outputs < s.ctas ? outputs : s.ctas);
      for (int i = 0; i < 7; ++i) {
        const int64_t c = 2 + i;
        if (outputs <= clusters.most[i] && plan->most_tiles >= c)
          take(time_ns((double)((plan->most_tiles + c - 1) / c) * unit_ns, bytes) + CLUSTER_ROWS_NS, 1, (int)c, outputs * c);
      }
    }
  }
  if (!o.mtiles) return DIT_ERR_UNSUPPORTED;  // what is forced does not fit
  const int64_t sum_chunks = (o.g[0].blocks + o.g[1].blocks) * p.n_adapters * (o.mtiles * 128 * p.rp / 1024);
  const int64_t sum_ctas = sum_chunks < 65536 ? sum_chunks : 65536;
  CUtensorMap m_x, m_e, m_dy, m_h;
  const int64_t held_rows = (int64_t)p.n_tiles * TILE_ROWS;
  if (!map_rows(&m_x, x, k, p.rows, ROW_STAGE) || !map_rows(&m_e, scratch, PARTS * p.rp, held_rows, ROW_STAGE) ||
      !map_rows(&m_dy, dy, n, p.rows, ROW_STAGE) || !map_rows(&m_h, saved, PARTS * p.rp, held_rows, ROW_STAGE))
    return DIT_ERR_CUDA;
  struct Kernel {
    void (*run)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Args, OverRows);
    bool (*allowed)();
  };
  static const Kernel kernels[2][3] = {{{k_over_rows<1, false>, allow_smem<k_over_rows<1, false>>},
                                        {k_over_rows<2, false>, allow_smem<k_over_rows<2, false>>},
                                        {k_over_rows<4, false>, allow_smem<k_over_rows<4, false>>}},
                                       {{k_over_rows<1, true>, allow_smem<k_over_rows<1, true>>},
                                        {k_over_rows<2, true>, allow_smem<k_over_rows<2, true>>},
                                        {k_over_rows<4, true>, allow_smem<k_over_rows<4, true>>}}};
  const Kernel& kern = kernels[o.cluster > 1][o.mtiles / 2];
  if (!kern.allowed()) return DIT_ERR_CUDA;
  const int h_boxes = 64 % p.rp == 0 ? (PARTS * p.rp + 63) / 64 : PARTS * ((p.rp + 63) / 64);
  p.stages = stages_for(RING_BYTES, (2 * o.mtiles + h_boxes) * ROW_BOX);
  if (launch_pdl(kern.run, dim3(p.split.ctas), dim3(ROW_THREADS), SMEM_BYTES, st, (unsigned)o.cluster, m_x, m_e, m_dy, m_h, p, o) != cudaSuccess)
    return DIT_ERR_CUDA;
  // dx after the gradients of the factors: dy, which the first product has just read, is still in L2 for them
  // where it fits.
  o.split = p.split;
  if (dx) {
    // dx may be dy itself (a residual's gradient), or x: then k_over_rows has to be done with it first.
    auto apart = [&](const void* in, int64_t width) {
      const char *d = reinterpret_cast<const char*>(dx), *i = reinterpret_cast<const char*>(in);
      return d + plan->rows * k * (dx_dt == DIT_BF16 ? 2 : 4) <= i || i + plan->rows * width * 2 <= d;
    };
    return from_rank<true>(plain, scratch, PARTS, a, dx, dx_dt, k, &o, apart(x, k) && apart(dy, n), st);
  }
  if (!o.whole && p.split.ctas > 1 &&
      launch_pdl(k_over_rows_sum, dim3((unsigned)sum_ctas), dim3(256), 0, st, 1, p, o) != cudaSuccess)
    return DIT_ERR_CUDA;
  return DIT_OK;
}
