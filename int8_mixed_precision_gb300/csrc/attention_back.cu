// Attention, backward: dq = scale ds k, dk = scale ds^T q, dv = p^T do, with p = exp(s - lse), ds = p (do v^T - delta),
// delta = sum over dim of do o.
//
// Two kernels of one form, so that every gradient is a sum in a fixed order that ends in one rounding: neither atomics
// nor an fp32 copy of dq in memory.  The price is that s and do v^T are made twice, seven products instead of five.  A CTA
// keeps 128 rows of a pair (X1, X2) and streams tiles of a pair (Y1, Y2):
//
//   S = X1 Y1^T,  T = X2 Y2^T,  ds = p (T - delta),  A += ds Y1,  B += p Y2
//
//   queries stay: X = (q, do), Y = (k, v):  A = dq / scale
//   keys stay:    X = (k, v), Y = (q, do):  A = dk / scale, B = dv; S, T, p and ds are the transposed ones, and the
//                                           queries of all heads that share the keys pass by
//
// S and T lie in tensor memory; p and ds go back there in bf16 as A operands of the next products (each rounding at most 2^-8 of its
// value), so nothing but the streamed tiles passes through shared memory.  The next tile's S and T are made while the
// warps work at the present one's.  Where tensor memory holds two of everything, the two warpgroups work at tiles in turn
// (STREAMS 2), so that one's exponentials hide the other's waits; else they share each tile's columns.
//
// Ahead of the stream.  The kernel of dk and dv needs nothing of the one of dq before it and starts on the SMs that one leaves.  That one
// lets it launch only after its own wait, so that the inputs, lse and delta are then complete and in global memory; and
// it waits itself before it ends, so for what follows on the stream the order is that of plain launches.  The kernels of delta
// and of dk and dv let their successors launch before they have waited: those wait before they read anything.
//
// Bound by the row warps' chains and the MMAs, which do not quite hide each other.  17,776 rows of 30 heads of 64, seconds of it under
// the power cap: 2.79 ms where queries stay (at 1965 MHz) and 3.38 where keys do (1935 MHz; their columns' lse and delta
// come from shared memory), apart.  To two tiles of 64 columns that is 1435 and 1720 cycles, a CTA's start and end included, for
// MMAs of 1024 and 1280: the tensor pipe has work for 71 and 74 % of the time.  The whole backward pass takes 6.3 ms so and 6.1
// among other work, 995 TFLOP/s of the formulas' ten operations; 4096 rows of 9 heads of 128: 216 us, 893.  With one stream in
// each the pass took 7.6 ms.
//
// Warps: 0 loads; 1 and 6 issue S and T of a stream each; 2 issues A, 3 B; 4, 5 and 7 relay the MMAs' completion; the others hold
// the rows and take over most of the first ones' registers.  Every wait on memory is bounded.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "attention.cuh"

namespace dit6 {
namespace attn {

using namespace lora;

constexpr int BACK_STAGES = 10;  // most
using Regs = Registers<4, 128, 56, 200>;

template <int PD, bool KEYS>
struct Back {
  static constexpr int COLS = BACK_COLS;
  static constexpr int STREAMS = PD == 64 || !KEYS ? 2 : 1;
  static constexpr int MINE = COLS * STREAMS / 2;  // columns of a thread
  static constexpr int CHUNKS = PD / 64;
  static constexpr int X_CHUNK = TILE * 128, X_BYTES = CHUNKS * X_CHUNK;
  static constexpr int Y_CHUNK = COLS * 128, Y_BYTES = CHUNKS * Y_CHUNK;
  static constexpr int STAGES = PD == 64 ? 10 : 4;
  static constexpr int STATS = 2 * X_BYTES + 2 * STAGES * Y_BYTES;  // lse and delta of a stage's columns
  static constexpr int STAT_BYTES = 2 * COLS * 4;
  static constexpr int CONTROL = STATS + STAGES * STAT_BYTES;
  static constexpr int SMEM = CONTROL + 1024 + 1024;
  // tensor memory: S and T of each stream, p and dS of each stream, A, B
  static constexpr uint32_t S = 0, T = COLS, S_STEP = 2 * COLS, P = STREAMS * S_STEP, DS = P + COLS / 2, P_STEP = COLS, A = P + STREAMS * P_STEP, B = A + PD;
  static constexpr int MMA_WARPS = STREAMS + 1 + KEYS, ROW_WARPS = 8 / STREAMS, MEET = 32 + 32 * ROW_WARPS;
  static_assert((KEYS ? B : A) + PD <= 512 && SMEM <= 227 * 1024 && Regs::THREADS * Regs::LAUNCHED == 65536, "");
};

struct BackControl {
  uint64_t xfull, done, sfull[2], sfree[2], pready[2], pdone[2];
  uint64_t yfull[BACK_STAGES], yempty[BACK_STAGES];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(BackControl) <= 1024, "");

struct BackArgs {
  dit_attention_plan_t plan;
  const int32_t* table;
  const float* lse;   // [heads][padded rows], in base 2
  float* delta;       // the same
  Heads out, dout;
  Heads a, b;         // dq; dk and dv
  void* ws;
  float c, scale;     // scale log2(e); scale
  int group;
  int ahead;  // the kernel before is the gradient of the queries
  int stall;
};

// delta of 128 queries of a head, sixteen bytes to a lane.  Bound by memory: 17,776 rows of 30 heads of 64 take 40 us, 3.4 TB/s.
__global__ void __launch_bounds__(256) k_attention_delta(const __grid_constant__ BackArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  const Work w = find_work(p.table, p.plan, GRAD_Q, p.plan.heads, p.ws);
  if (!w.ok) return;
  const int lane = threadIdx.x % 16, dim = p.plan.dim;
#pragma unroll
  for (int i = 0; i < TILE / 16; ++i) {  // all loads at once
    const int r = threadIdx.x / 16 + 16 * i;
    const int64_t row = (int64_t)w.row0 + r;
    const bool mine = row < w.doc.queries;
    float sum = 0.f;
    if (mine && 8 * lane < dim) {
      const int64_t at = w.doc.q0 + row;
      const uint4 o = __ldg(reinterpret_cast<const uint4*>(p.out.ptr + at * p.out.row + w.head * p.out.head + 8 * lane));
      const uint4 g = __ldg(reinterpret_cast<const uint4*>(p.dout.ptr + at * p.dout.row + w.head * p.dout.head + 8 * lane));
      const uint32_t a[4] = {o.x, o.y, o.z, o.w}, b[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = bf16x2_to_f2(a[k]), y = bf16x2_to_f2(b[k]);
        sum += x.x * y.x + x.y * y.y;
      }
    }
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    // the rows that pad a document to whole tiles are written too
    if (lane == 0) p.delta[(int64_t)w.head * p.plan.padded_rows + (int64_t)w.doc.tile0 * TILE + row] = sum;
  }
}

template <int PD, bool KEYS>
__global__ void __launch_bounds__(Regs::THREADS, 1)
    k_attention_back(const __grid_constant__ CUtensorMap mx1, const __grid_constant__ CUtensorMap mx2,
                     const __grid_constant__ CUtensorMap my1, const __grid_constant__ CUtensorMap my2, const __grid_constant__ BackArgs p) {
  if (!KEYS) {  // before the next kernel starts, everything that it reads is there
    pdl_wait();
    pdl_launch_dependents();
  }
  using F = Back<PD, KEYS>;
  constexpr int COLS = F::COLS, STREAMS = F::STREAMS, MINE = F::MINE;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_u32(base);
  BackControl* c = reinterpret_cast<BackControl*>(base + F::CONTROL);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  if (warp == 0) {
    if (lane < F::STAGES) {
      mbar_init(smem_u32(&c->yfull[lane]), 1);
      mbar_init(smem_u32(&c->yempty[lane]), KEYS ? 2 : 1);
    } else if (lane >= 16 && lane < 18) {
      const int w = lane - 16;
      mbar_init(smem_u32(&c->sfull[w]), 1);
      mbar_init(smem_u32(&c->sfree[w]), F::ROW_WARPS);
      mbar_init(smem_u32(&c->pready[w]), F::ROW_WARPS);
      mbar_init(smem_u32(&c->pdone[w]), KEYS ? 2 : 1);
    } else if (lane == 18) {
      mbar_init(smem_u32(&c->xfull), 1);
      mbar_init(smem_u32(&c->done), F::MMA_WARPS);
      c->abort = 0;
    }
    fence_barrier_init();
    __syncwarp();
  } else if (warp == 2) {
    if (lane < 4) prefetch_tmap(lane == 0 ? &mx1 : lane == 1 ? &mx2 : lane == 2 ? &my1 : &my2);
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&c->tmem), 512);
    fence_before();
  }
  if (KEYS) {
    if (!p.ahead) pdl_wait();
    pdl_launch_dependents();
  }
  const Work w = find_work(p.table, p.plan, KEYS ? GRAD_KV : GRAD_Q, KEYS ? p.plan.kv_heads : p.plan.heads, p.ws);
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(c->tmem);
  volatile int* abort = &c->abort;
  const Doc& d = w.doc;
  const int row0 = w.row0;
  const int x_rows = KEYS ? d.keys : d.queries, y_rows = KEYS ? d.queries : d.keys;  // of the document
  const int x0 = KEYS ? d.k0 : d.q0, y0 = KEYS ? d.q0 : d.k0;
  const int tiles = w.ok && w.end > w.begin ? w.end - w.begin : 0;
  const int n = tiles * (KEYS ? p.group : 1);

  const int w_begin = w.begin;
  if (warp < Regs::FIRST_ROWS) Regs::give();
  const uint32_t ring = smem + 2 * F::X_BYTES;
  if (warp == 0) {
    if (n > 0 && elect_one()) {
      int s = 0, parity = 1, issued = 0;
      bool ok = true;
      if (!p.stall) {
        mbar_expect_tx(smem_u32(&c->xfull), 2 * F::X_BYTES);
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < F::CHUNKS; ++k)
            tma_load_3d(smem + i * F::X_BYTES + k * F::X_CHUNK, i ? &mx2 : &mx1, smem_u32(&c->xfull), k * 64, w.head, x0 + row0);
      }
      int tile = 0, head = KEYS ? w.head * p.group : w.head / p.group;
      for (int j = 0; j < n; ++j) {
        if (j >= F::STAGES && !mbar_wait(smem_u32(&c->yempty[s]), parity, p.ws, abort)) {
          ok = false;
          break;
        }
        if (!p.stall) {
          const uint32_t full = smem_u32(&c->yfull[s]), to = ring + s * F::Y_BYTES, stats = smem + F::STATS + s * F::STAT_BYTES;
          const int row = (w.begin + tile) * COLS;
          mbar_expect_tx(full, 2 * F::Y_BYTES + (KEYS ? F::STAT_BYTES : 0));
#pragma unroll
          for (int k = 0; k < F::CHUNKS; ++k) {
            tma_load_3d(to + k * F::Y_CHUNK, &my1, full, k * 64, head, y0 + row);
            tma_load_3d(to + F::STAGES * F::Y_BYTES + k * F::Y_CHUNK, &my2, full, k * 64, head, y0 + row);
          }
          if (KEYS) {
            const int64_t at = (int64_t)head * p.plan.padded_rows + (int64_t)d.tile0 * TILE + row;
            bulk_load(stats, p.lse + at, COLS * 4, full);
            bulk_load(stats + COLS * 4, p.delta + at, COLS * 4, full);
          }
          issued = j + 1;
        }
        if (++s == F::STAGES) s = 0, parity ^= 1;
        if (++tile == tiles) tile = 0, head += KEYS;
      }
      if ((!ok || *abort) && !p.stall) {  // its own copies land before the CTA ends
        volatile int never = 0;
        mbar_wait(smem_u32(&c->xfull), 0, p.ws, &never);
        for (int i = issued > F::STAGES ? issued - F::STAGES : 0; i < issued; ++i) mbar_wait(smem_u32(&c->yfull[i % F::STAGES]), (i / F::STAGES) & 1, p.ws, &never);
      }
    }
  } else if (warp == 1 || (warp == 6 && STREAMS == 2)) {
    if (n > 0) {  // S and T of every tile of a stream, once the rows' warps have the tile before in registers
      constexpr uint32_t id = idesc(128, COLS, false, false);
      const int w = warp == 6;
      const uint32_t sfull = smem_u32(&c->sfull[w]), sfree = smem_u32(&c->sfree[w]), to = tmem + F::S + w * F::S_STEP;
      bool ok = warp_wait(smem_u32(&c->xfull), 0, p.ws, abort);
      int s = w, parity = 0, tile = tiles > 1 ? w : 0;
      for (int j = w, i = 0; j < n && ok; j += STREAMS, ++i) {
        const uint32_t y = ring + s * F::Y_BYTES;
        ok = warp_wait(smem_u32(&c->yfull[s]), parity, p.ws, abort);
        const int left = y_rows - (w_begin + tile) * COLS;
        if (ok && left < COLS) {
          zero_rows(y, F::Y_CHUNK, F::CHUNKS, left, COLS);
          zero_rows(y + F::STAGES * F::Y_BYTES, F::Y_CHUNK, F::CHUNKS, left, COLS);
        }
        if (i > 0) ok = ok && warp_wait(sfree, (i - 1) & 1, p.ws, abort);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = desc_k(smem + h * F::X_BYTES), b = desc_k(y + h * F::STAGES * F::Y_BYTES);
#pragma unroll
            for (int k = 0; k < PD / 16; ++k)
              mma(to + h * COLS, a + (k / 4) * (F::X_CHUNK >> 4) + (k % 4) * 2, b + (k / 4) * (F::Y_CHUNK >> 4) + (k % 4) * 2, id, k > 0);
          }
          mma_commit(sfull);
        }
        __syncwarp();
        s += STREAMS;
        if (s >= F::STAGES) s -= F::STAGES, parity ^= 1;
        tile += STREAMS;
        while (tile >= tiles) tile -= tiles;
      }
      if (elect_one()) mma_commit(smem_u32(&c->done));
      __syncwarp();
    }
  } else if (warp < 4) {
    const bool second = warp == 3;  // B += P Y2, else A += dS Y1
    if (n > 0 && (KEYS || !second)) {
      const uint32_t id = idesc(128, (p.plan.dim + 15) / 16 * 16, false, true);
      const uint32_t a0 = tmem + (second ? F::P : F::DS), to = tmem + (second ? F::B : F::A), y = ring + (second ? F::STAGES * F::Y_BYTES : 0);
      bool ok = true;
      int s = 0, w = 0, parity = 0;
      for (int j = 0; j < n; ++j) {
        ok = warp_wait(smem_u32(&c->pready[w]), parity, p.ws, abort);  // the tile has long been there: S and T were made of it
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint32_t a = a0 + w * F::P_STEP, b = desc_mn(y + s * F::Y_BYTES, F::Y_CHUNK);
#pragma unroll
          for (int k = 0; k < COLS / 16; ++k) mma_ta(to, a + k * 8, b + k * (2048 >> 4), id, j > 0 || k > 0);
          mma_commit(smem_u32(&c->pdone[w]));
          mma_commit(smem_u32(&c->yempty[s]));
        }
        __syncwarp();
        if (++s == F::STAGES) s = 0;
        if (++w == STREAMS) w = 0, parity ^= 1;
      }
      if (elect_one()) mma_commit(smem_u32(&c->done));
      __syncwarp();
    }
  } else if (warp < Regs::FIRST_ROWS) {
    if (n > 0) {
      if (warp == 4 || (warp == 5 && STREAMS == 2)) {
        const int w = warp - 4;
        relay<F::MEET>(smem_u32(&c->sfull[w]), 1 + w, (n - w + STREAMS - 1) / STREAMS, p.ws, abort);
        if (w == 0) {  // every MMA has completed before the rows' warps read the results, and before the CTA ends
          volatile int never = 0;
          warp_wait(smem_u32(&c->done), 0, p.ws, &never);
          fence_after();
          fence_before();
          __syncwarp();
          meet<288>(5);
        }
      } else if (warp == 7) {  // of each stream's tiles but its last
        for (int j = 0; j < n - STREAMS; ++j) {
          const int w = j % STREAMS;
          if (!__any_sync(0xffffffffu, *abort)) warp_wait(smem_u32(&c->pdone[w]), (j / STREAMS) & 1, p.ws, abort);
          fence_after();
          fence_before();
          __syncwarp();
          meet<F::MEET>(3 + w);
        }
      }
    }
  } else {
    Regs::take();
    const int half = (warp - Regs::FIRST_ROWS) / 4;  // of the columns; STREAMS 2: the stream
    const int stream = STREAMS == 2 ? half : 0, col = STREAMS == 2 ? 0 : half * MINE;
    const int r = (warp % 4) * 32 + lane;
    const int row = row0 + r;
    const bool live = w.ok && row < x_rows;
    const uint32_t at = tmem + ((uint32_t)(warp % 4) << 21);
    // the columns that this row meets; rows behind the last one: whatever they hold is not stored
    int lo = 0, hi = INT_MAX - COLS;
    if (live && KEYS) {
      lo = (int)min(seen_from(d, p.plan.frame, row), (int64_t)d.queries);
      hi = d.queries;
    } else if (live) {
      hi = (int)seen_end(d, p.plan.frame, row);
    }
    // tiles that every row of the warp meets whole
    const int whole_from = __reduce_max_sync(0xffffffffu, lo / COLS + (lo % COLS != 0));
    const int whole_to = __reduce_min_sync(0xffffffffu, hi / COLS);
    float lse = 0.f, delta = 0.f;
    if (!KEYS && live) {
      const int64_t i = (int64_t)w.head * p.plan.padded_rows + (int64_t)d.tile0 * TILE + row;
      lse = -p.lse[i];
      delta = -p.delta[i];
    }
    const uint32_t s_at = at + F::S + stream * F::S_STEP + col, t_at = s_at + COLS;
    const uint32_t p_at = at + F::P + stream * F::P_STEP + col / 2, ds_at = p_at + COLS / 2;
    const uint32_t sfree = smem_u32(&c->sfree[stream]), pready = smem_u32(&c->pready[stream]);
    const float2 c2 = make_float2(p.c, p.c);
    int stage = stream, tile = tiles > 1 ? stream : 0;
    for (int j = stream; j < n; j += STREAMS) {
      __syncwarp();
      meet<F::MEET>(1 + stream);
      fence_after();
      uint32_t s[MINE], g[MINE];
#pragma unroll
      for (int k = 0; k < MINE; k += 32) {
        tmem_ld32(s_at + k, s + k);
        tmem_ld32(t_at + k, g + k);
      }
      tmem_wait();
      pin(s);
      pin(g);
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfree);
      const uint32_t stats = smem + F::STATS + stage * F::STAT_BYTES + col * 4;
      float l4[4] = {lse, lse, lse, lse}, d4[4] = {delta, delta, delta, delta};
#pragma unroll
      for (int i = 0; i < MINE; i += 4) {
        if (KEYS) {  // the columns' own
          const uint4 l = lds128(stats + i * 4), d = lds128(stats + COLS * 4 + i * 4);
          l4[0] = -__uint_as_float(l.x), l4[1] = -__uint_as_float(l.y), l4[2] = -__uint_as_float(l.z), l4[3] = -__uint_as_float(l.w);
          d4[0] = -__uint_as_float(d.x), d4[1] = -__uint_as_float(d.y), d4[2] = -__uint_as_float(d.z), d4[3] = -__uint_as_float(d.w);
        }
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(s[i + h]), __uint_as_float(s[i + h + 1])), c2, make_float2(l4[h], l4[h + 1]));
          const float2 t = add2(make_float2(__uint_as_float(g[i + h]), __uint_as_float(g[i + h + 1])), make_float2(d4[h], d4[h + 1]));
          s[i + h] = __float_as_uint(exp2_approx(x.x));
          s[i + h + 1] = __float_as_uint(exp2_approx(x.y));
          g[i + h] = __float_as_uint(t.x);
          g[i + h + 1] = __float_as_uint(t.y);
        }
      }
      const int at_tile = w.begin + tile;
      if (at_tile < whole_from || at_tile >= whole_to) {  // masked pairs: p and ds are zero, whatever was there
        const int col0 = at_tile * COLS + col, from = lo - col0, to = hi - col0;
#pragma unroll
        for (int i = 0; i < MINE; ++i)
          if (i < from || i >= to) s[i] = g[i] = 0u;
      }
      __syncwarp();
      if (j >= STREAMS) {  // the products that read p and dS are done
        meet<F::MEET>(3 + stream);
        fence_after();
      }
#pragma unroll
      for (int k = 0; k < MINE / 2; k += 16) {
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 e = make_float2(__uint_as_float(s[2 * (k + i)]), __uint_as_float(s[2 * (k + i) + 1]));
          const float2 t = mul2(e, make_float2(__uint_as_float(g[2 * (k + i)]), __uint_as_float(g[2 * (k + i) + 1])));
          if (KEYS) pk[i] = f2_to_bf16x2(e.x, e.y);
          dk[i] = f2_to_bf16x2(t.x, t.y);
        }
        if (KEYS) tmem_st16(p_at + k, pk);
        tmem_st16(ds_at + k, dk);
      }
      tmem_st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready);
      stage += STREAMS;
      if (stage >= F::STAGES) stage -= F::STAGES;
      tile += STREAMS;
      while (tile >= tiles) tile -= tiles;
    }
    if (n > 0) {
      __syncwarp();
      meet<288>(5);
      fence_after();
    }
    const bool ok = !__any_sync(0xffffffffu, *abort);
    if (ok) {  // one warpgroup to each of dk and dv, or to each half of dq's columns
      const Heads& to = KEYS && half ? p.b : p.a;
      const float f = KEYS && half ? 1.f : p.scale;
      constexpr int WIDTH = KEYS ? PD : PD / 2, CH = WIDTH < 64 ? 4 : 8;  // columns of a warp, and chunks of eight at a time
      const int first = KEYS ? 0 : half * WIDTH;
      const uint32_t stage = smem + (warp - Regs::FIRST_ROWS) * 4096;  // what stayed is done with
      __nv_bfloat16* dst = to.ptr + (int64_t)(x0 + row) * to.row + w.head * to.head + first;
#pragma unroll
      for (int k = 0; k < WIDTH; k += 8 * CH) {
        uint32_t o[8 * CH];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8 * CH; i += 32) tmem_ld32(at + (KEYS && half ? F::B : F::A) + first + k + i, o + i);
        tmem_wait();
        pin(o);
        uint4 v[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) v[i] = n == 0 ? make_uint4(0, 0, 0, 0) : pack8(o + 8 * i, f);
        store_rows<CH>(stage, v, dst + k, live, (p.plan.dim - first - k + 7) / 8);
      }
    }
  }
  if (KEYS) pdl_wait();  // whoever follows finds the gradient of the queries complete too
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

struct Inputs {
  Heads q, k, v, dout;
};

template <int PD, bool KEYS>
static dit_status launch(BackArgs a, const Inputs& in, cudaStream_t st) {
  using F = Back<PD, KEYS>;
  static OncePerDevice checked, once;
  const dit_attention_plan_t& p = a.plan;
  const int items = p.items[KEYS ? GRAD_KV : GRAD_Q], heads = KEYS ? p.kv_heads : p.heads;
  if (!items) return DIT_OK;
  // Without queries or without keys nothing is loaded: any tensor makes a map.
  const bool q_any = p.q_rows > 0, k_any = p.k_rows > 0;
  auto map = [&](CUtensorMap* m, const Heads& own, const Heads& other, bool query, int rows) {
    const bool mine = query ? q_any : k_any, of_query = mine ? query : !query;
    return map_heads(m, mine ? own : other, p.dim, of_query ? p.heads : p.kv_heads, of_query ? p.q_rows : p.k_rows, 1, rows);
  };
  CUtensorMap mq, mo, mk, mv;
  const int q_box = KEYS ? F::COLS : TILE, k_box = KEYS ? TILE : F::COLS;
  if (!map(&mq, in.q, in.k, true, q_box) || !map(&mo, in.dout, in.v, true, q_box) || !map(&mk, in.k, in.q, false, k_box) || !map(&mv, in.v, in.dout, false, k_box))
    return DIT_ERR_CUDA;
  if (prepare_kernel<Regs>(checked, once, k_attention_back<PD, KEYS>, F::SMEM) != cudaSuccess) return DIT_ERR_CUDA;
  const cudaError_t e = KEYS ? launch_pdl(k_attention_back<PD, KEYS>, dim3((unsigned)(items * heads)), dim3(Regs::THREADS), F::SMEM, st, 1, mk, mv, mq, mo, a)
                             : launch_pdl(k_attention_back<PD, KEYS>, dim3((unsigned)(items * heads)), dim3(Regs::THREADS), F::SMEM, st, 1, mq, mo, mk, mv, a);
  return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

template <int PD>
static dit_status backward(BackArgs a, const Inputs& in, const Heads& dq, const Heads& dk, const Heads& dv, cudaStream_t st) {
  if (a.plan.items[GRAD_Q] &&
      launch_pdl(k_attention_delta, dim3((unsigned)(a.plan.items[GRAD_Q] * a.plan.heads)), dim3(256), 0, st, 1, a) != cudaSuccess)
    return DIT_ERR_CUDA;
  a.a = dq;
  const dit_status e = launch<PD, false>(a, in, st);
  if (e != DIT_OK) return e;
  a.a = dk;
  a.b = dv;
  a.ahead = a.plan.items[GRAD_Q] > 0;
  return launch<PD, true>(a, in, st);
}

}  // namespace attn
}  // namespace dit6

using namespace dit6;

extern "C" dit_status dit_attention_backward(const dit_attention_plan_t* plan, const int32_t* table, const dit_heads_t* q,
                                             const dit_heads_t* k, const dit_heads_t* v, const dit_heads_t* out,
                                             const dit_heads_t* dout, const dit_heads_t* dq, const dit_heads_t* dk,
                                             const dit_heads_t* dv, double scale, const void* saved, size_t saved_bytes,
                                             void* scratch, size_t scratch_bytes, void* ws, size_t ws_bytes,
                                             dit_stream_t stream) {
  using namespace attn;
  if (!plan_ok(plan) || (!table && plan->table_ints > 0) || !ws || ws_bytes < WS_BYTES || !(scale > 0.0) || !isfinite(scale) || !plan->training) return DIT_ERR_INVALID_ARG;
  if (saved_bytes < (size_t)plan->saved_bytes || (plan->saved_bytes && !saved)) return DIT_ERR_INVALID_ARG;
  if (scratch_bytes < (size_t)plan->scratch_bytes || (plan->scratch_bytes && !scratch)) return DIT_ERR_INVALID_ARG;
  BackArgs a = {};
  Inputs in;
  Heads hdq, hdk, hdv;
  const int h = plan->heads, hk = plan->kv_heads, dim = plan->dim;
  dit_status e = check_view(q, h, plan->q_rows, dim, &in.q);
  if (e == DIT_OK) e = check_view(k, hk, plan->k_rows, dim, &in.k);
  if (e == DIT_OK) e = check_view(v, hk, plan->k_rows, dim, &in.v);
  if (e == DIT_OK) e = check_view(out, h, plan->q_rows, dim, &a.out);
  if (e == DIT_OK) e = check_view(dout, h, plan->q_rows, dim, &a.dout);
  if (e == DIT_OK) e = check_output(dq, h, plan->q_rows, dim, &hdq);
  if (e == DIT_OK) e = check_output(dk, hk, plan->k_rows, dim, &hdk);
  if (e == DIT_OK) e = check_output(dv, hk, plan->k_rows, dim, &hdv);
  if (e != DIT_OK) return e;
  if (!aligned32(ws) || (reinterpret_cast<uintptr_t>(table) & 15) || (reinterpret_cast<uintptr_t>(saved) & 15) || (reinterpret_cast<uintptr_t>(scratch) & 15))
    return DIT_ERR_ALIGNMENT;
  in.dout = a.dout;
  a.plan = *plan;
  a.table = table;
  a.lse = reinterpret_cast<const float*>(saved);
  a.delta = reinterpret_cast<float*>(scratch);
  a.ws = ws;
  a.c = (float)(scale * 1.4426950408889634);
  a.scale = (float)scale;
  a.group = h / hk;
  a.stall = test_stall();
  if (!(a.c >= FLT_MIN && a.c <= FLT_MAX)) return DIT_ERR_INVALID_ARG;  // in fp32 too
  if (!buffers_apart(*plan, saved, scratch, ws)) return DIT_ERR_INVALID_ARG;
  return dim <= 64 ? backward<64>(a, in, hdq, hdk, hdv, stream) : backward<128>(a, in, hdq, hdk, hdv, stream);
}
