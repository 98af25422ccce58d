// Attention, forward: o = softmax(scale q k^T) v over the keys that each query sees.
//
// One pass over the keys with the running maximum and sum of the softmax.  A block is 128 rows (a row is a query and a head of
// the group that shares the keys); keys and values stream through shared memory by TMA.  S = Q K^T goes to tensor
// memory, a thread to each row turns it into P (in bf16, back to tensor memory as the A operand of the next product) and
// O += P V stays there.  While the warps of one block work at their softmax the tensor cores have another block's products,
// and S of the next tile is made as soon as the present one is in registers.
//
// The running maximum moves only when it grows by more than 2^GROWTH: until then P is larger than 1 by at
// most that factor, which neither bf16 nor fp32 sums mind, and O need not be rescaled.  The final division takes the
// same maximum out again.
//
// P is rounded to bf16 (an operand of the bf16 tensor pipe), 2^-8 of each weight at most; the sum of the weights is of the unrounded
// ones.  Scores are scaled inside the exponent's multiply-add, in base 2.
//
// Two blocks.  With 64 dimensions a CTA has two blocks, which share the keys and a ring of six tiles, and the SM to itself; with
// 128, and where no item has many tiles, it has one, and an SM two CTAs: the start and end of one hide behind the other's tiles.
// With 128 P lies over S, so the next S waits for the product with V, and a ring of one tile loses nothing beside that: 17,776
// rows of 30 heads take 3.35 ms, two blocks to a CTA took 3.47; 5 documents of 2000 (16 heads) 150 us and 167.
//
// Few rows.  Where the keys of an item are cut into pieces and a CTA of two blocks has one alone, its halves take its tiles
// in turn, two blocks of the same rows: a tile's chain of waits is then half as long for two.
//
// Bound by the row warps' chain of a tile: with 64 dimensions 1740 cycles for two blocks, 1024 of them exponentials and as many
// MMAs beside those.  17,776 rows of 30 heads: 1.77 ms, 1370 TFLOP/s, with 128 dimensions 3.35 ms, 1450; 4096 rows of 9 heads 33
// us and 59.
//
// Warps: 0 loads, 1 issues S, 2 and 3 issue O += P V of a block each, 4 to 7 relay the MMAs' completion to the rows' warps, which are
// 8 to 11 and 12 to 15, a thread to each row, and take over most of the others' registers.  With one block 3 relays, and
// 4 to 7 have the rows.  Every wait on memory is bounded.
#include <float.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "attention.cuh"

namespace dit6 {
namespace attn {

using namespace lora;

constexpr float GROWTH = 8.f;
constexpr int FWD_STAGES = 6;  // most

// BLOCKS: blocks of rows to a CTA.  One, and two CTAs to an SM, with 128 dimensions and for short items.
template <int PD, int BLOCKS>
struct Fwd {
  using Regs = Registers<2 * BLOCKS, 128, 48, 208, BLOCKS>;
  static constexpr int COLS = FORWARD_COLS;
  static constexpr int CHUNKS = PD / 64;
  static constexpr bool OVER_S = PD > 64;  // P takes the place of S
  static constexpr int Q_CHUNK = TILE * 128, Q_BYTES = CHUNKS * Q_CHUNK;
  static constexpr int KV_CHUNK = COLS * 128, KV_BYTES = CHUNKS * KV_CHUNK;
  static constexpr int STAGES = BLOCKS == 2 ? 6 : PD == 64 ? 2 : 1;
  static constexpr int RING = BLOCKS * Q_BYTES;
  static constexpr int CONTROL = RING + 2 * STAGES * KV_BYTES;
  static constexpr int SMEM = CONTROL + 1024 + 1024;
  // tensor memory: S and P of each block, then O
  static constexpr uint32_t S = 0, P = OVER_S ? S : BLOCKS * COLS, P_STEP = OVER_S ? COLS : COLS / 2, O = P + BLOCKS * P_STEP;
  static constexpr uint32_t COLUMNS = BLOCKS == 2 ? 512 : 256;
  static_assert(O + BLOCKS * PD <= COLUMNS && (3 - BLOCKS) * (SMEM + 1024) <= 228 * 1024, "");
  // A kernel starts early and takes its tensor memory before it waits for the one before, whose last CTAs may not have taken theirs: CTAs
  // that fit an SM together must find columns together, or they wait for one another.  The library's kernels with 512 columns
  // leave less than 64 KB of shared memory or no registers, and those with 256 need a third of an SM's or more.
  static_assert(COLUMNS == 512 ? Regs::THREADS * Regs::LAUNCHED == 65536 : SMEM >= 64 * 1024 && 3 * (SMEM + 1024) > 228 * 1024, "");
};

struct FwdControl {
  uint64_t qfull, done;
  uint64_t kfull[FWD_STAGES], kempty[FWD_STAGES], vfull[FWD_STAGES], vempty[FWD_STAGES];
  uint64_t sfull[2], sfree[2], pready[2], pdone[2], tail;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(FwdControl) <= 1024, "");

template <int PD>
constexpr int PARTIAL = partial_floats(PD);

struct FwdArgs {
  dit_attention_plan_t plan;
  const int32_t* table;
  Heads out;
  float* lse;       // [heads][padded rows], in base 2, or nullptr
  float* partial;   // [heads][slots][PARTIAL]: o unnormalised, the maximum (in base 2) and the sum
  void* ws;
  float c;          // scale log2(e)
  int group, rows;  // heads of a group, queries of a block
  int stall;
};

// SPLIT: some items are pieces of a longer one, whose results are partial.  A kernel that has none is
// 1.76 ms instead of 1.79 at 17,776 rows of 30 heads of 64.
template <int PD, bool SPLIT, int BLOCKS>
__global__ void __launch_bounds__(Fwd<PD, BLOCKS>::Regs::THREADS, 3 - BLOCKS)
    k_attention(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const __grid_constant__ FwdArgs p) {
  pdl_launch_dependents();
  using F = Fwd<PD, BLOCKS>;
  using Regs = typename F::Regs;
  constexpr int COLS = F::COLS;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_u32(base);
  FwdControl* c = reinterpret_cast<FwdControl*>(base + F::CONTROL);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  if (warp == 0) {
    if (lane < F::STAGES) {
      mbar_init(smem_u32(&c->kfull[lane]), 1);
      mbar_init(smem_u32(&c->kempty[lane]), 1);
      mbar_init(smem_u32(&c->vfull[lane]), 1);
      mbar_init(smem_u32(&c->vempty[lane]), 2);
    } else if (lane >= 8 && lane < 10) {
      const int t = lane - 8;
      mbar_init(smem_u32(&c->sfull[t]), 1);
      mbar_init(smem_u32(&c->sfree[t]), 4);
      mbar_init(smem_u32(&c->pready[t]), 4);
      mbar_init(smem_u32(&c->pdone[t]), 1);
    } else if (lane == 10) {
      mbar_init(smem_u32(&c->qfull), 1);
      mbar_init(smem_u32(&c->done), 1 + BLOCKS);
      mbar_init(smem_u32(&c->tail), 1);
      c->abort = 0;
    }
    fence_barrier_init();
    __syncwarp();
  } else if (warp == 2) {
    if (lane < 3) prefetch_tmap(lane == 0 ? &mq : lane == 1 ? &mk : &mv);
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&c->tmem), F::COLUMNS);
    fence_before();
  }
  pdl_wait();
  const Work w = find_work(p.table, p.plan, FORWARD, p.plan.kv_heads, p.ws);
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(c->tmem);
  volatile int* abort = &c->abort;
  const Doc& d = w.doc;
  const int row0 = w.row0;
  const int n = uniform(w.ok ? w.end - w.begin : 0);  // tiles
  // Two blocks of rows, one, or one whose tiles both halves of the CTA take in turn, as two blocks of the same rows.
  const bool turns = SPLIT && BLOCKS == 2 && w.ok && w.turns && w.slot >= 0;
  const int blocks = BLOCKS == 2 && w.ok && (turns || row0 + p.rows < d.queries) ? 2 : 1, step = turns ? 2 : 1;
  auto first_of = [&](int t) { return turns ? t : 0; };
  auto tiles_of = [&](int t) { return t < blocks ? (n - first_of(t) + step - 1) / step : 0; };
  const bool work = n > 0;

  if (warp < Regs::FIRST_ROWS) Regs::give();
  if (warp == 0) {
    if (work && elect_one()) {
      const uint32_t ring = smem + F::RING;
      int s = 0, parity = 1, issued = 0;  // of K; V has as many or one less
      bool ok = true;
      if (!p.stall) {
        const int loads = turns ? 1 : blocks;
        mbar_expect_tx(smem_u32(&c->qfull), loads * F::CHUNKS * p.rows * p.group * 128);
        for (int t = 0; t < loads; ++t)
#pragma unroll
          for (int k = 0; k < F::CHUNKS; ++k)
            tma_load_3d(smem + t * F::Q_BYTES + k * F::Q_CHUNK, &mq, smem_u32(&c->qfull), k * 64, w.head * p.group, d.q0 + row0 + t * p.rows);
      }
      int row = d.k0 + w.begin * COLS;
      for (int j = 0; j < n; ++j, row += COLS) {
        if (j >= F::STAGES && !mbar_wait(smem_u32(&c->kempty[s]), parity, p.ws, abort)) {
          ok = false;
          break;
        }
        if (!p.stall) {
          const uint32_t full = smem_u32(&c->kfull[s]), at = ring + s * F::KV_BYTES;
          mbar_expect_tx(full, F::KV_BYTES);
#pragma unroll
          for (int k = 0; k < F::CHUNKS; ++k) tma_load_3d(at + k * F::KV_CHUNK, &mk, full, k * 64, w.head, row);
          issued = 2 * j + 1;
        }
        if (j >= F::STAGES && !mbar_wait(smem_u32(&c->vempty[s]), parity, p.ws, abort)) {
          ok = false;
          break;
        }
        if (!p.stall) {
          const uint32_t full = smem_u32(&c->vfull[s]), at = ring + (F::STAGES + s) * F::KV_BYTES;
          mbar_expect_tx(full, F::KV_BYTES);
#pragma unroll
          for (int k = 0; k < F::CHUNKS; ++k) tma_load_3d(at + k * F::KV_CHUNK, &mv, full, k * 64, w.head, row);
          issued = 2 * j + 2;
        }
        if (++s == F::STAGES) s = 0, parity ^= 1;
      }
      if ((!ok || *abort) && !p.stall) {  // its own copies land before the CTA ends
        volatile int never = 0;
        mbar_wait(smem_u32(&c->qfull), 0, p.ws, &never);
        for (int i = issued > 2 * F::STAGES ? issued - 2 * F::STAGES : 0; i < issued; ++i) {
          const int j = i / 2;
          mbar_wait(smem_u32(i % 2 ? &c->vfull[j % F::STAGES] : &c->kfull[j % F::STAGES]), (j / F::STAGES) & 1, p.ws, &never);
        }
      }
    }
  } else if (warp == 1) {
    if (work) {  // S of each tile and block, once its warps have the tile before in registers (OVER_S: once P is used up)
      constexpr uint32_t id = idesc(128, COLS, false, false);
      const uint32_t ring = smem + F::RING;
      bool ok = warp_wait(smem_u32(&c->qfull), 0, p.ws, abort);
      int s = 0, parity = 0;
      for (int j = 0; j < n && ok; ++j) {
        ok = warp_wait(smem_u32(&c->kfull[s]), parity, p.ws, abort);
        for (int t = turns ? j & 1 : 0; t < (turns ? (j & 1) + 1 : blocks) && ok; ++t) {
          const int i = turns ? j >> 1 : j;
          if (i > 0) ok = warp_wait(smem_u32(F::OVER_S ? &c->pdone[t] : &c->sfree[t]), (i - 1) & 1, p.ws, abort);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t a = desc_k(smem + (turns ? 0 : t * F::Q_BYTES)), b = desc_k(ring + s * F::KV_BYTES), to = tmem + F::S + t * COLS;
#pragma unroll
            for (int k = 0; k < PD / 16; ++k) mma(to, a + (k / 4) * (F::Q_CHUNK >> 4) + (k % 4) * 2, b + (k / 4) * (F::KV_CHUNK >> 4) + (k % 4) * 2, id, k > 0);
            mma_commit(smem_u32(&c->sfull[t]));
            if (turns || t == blocks - 1) mma_commit(smem_u32(&c->kempty[s]));
          }
          __syncwarp();
        }
        if (++s == F::STAGES) s = 0, parity ^= 1;
      }
      if (elect_one()) mma_commit(smem_u32(&c->done));
      __syncwarp();
    }
  } else if (warp < 2 + BLOCKS) {
    const int t = warp - 2;
    if (work && t < blocks) {  // O += P V of a block
      const uint32_t id = idesc(128, (p.plan.dim + 15) / 16 * 16, false, true);
      const uint32_t a = tmem + F::P + t * F::P_STEP, to = tmem + F::O + t * PD;
      bool ok = true;
      int s = first_of(t), parity = 0;
      int left = d.keys - (w.begin + s) * COLS;  // keys from this tile's first on
      const int many = tiles_of(t);
      for (int j = 0; j < many && ok; ++j, left -= step * COLS) {
        const uint32_t v = smem + F::RING + (F::STAGES + s) * F::KV_BYTES;
        ok = warp_wait(smem_u32(&c->vfull[s]), parity, p.ws, abort);
        if (ok && left < COLS) {  // the document's last tile, for both blocks
          if (t == 0 || turns) {
            zero_rows(v, F::KV_CHUNK, F::CHUNKS, left, COLS);
            if (!turns && lane == 0) mbar_arrive(smem_u32(&c->tail));
            __syncwarp();
          } else {
            ok = warp_wait(smem_u32(&c->tail), 0, p.ws, abort);
          }
        }
        ok = ok && warp_wait(smem_u32(&c->pready[t]), j & 1, p.ws, abort);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint32_t b = desc_mn(v, F::KV_CHUNK);
#pragma unroll
          for (int k = 0; k < COLS / 16; ++k) mma_ta(to, a + k * 8, b + k * (2048 >> 4), id, j > 0 || k > 0);
          mma_commit(smem_u32(&c->pdone[t]));
          mma_commit(smem_u32(&c->vempty[s]));
          if (blocks == 1 || turns) mma_commit(smem_u32(&c->vempty[s]));
        }
        __syncwarp();
        s += step;
        if (s >= F::STAGES) s -= F::STAGES, parity ^= 1;
      }
    }
    if (work) {
      if (elect_one()) mma_commit(smem_u32(&c->done));
      __syncwarp();
      if (t == 0) {  // every MMA has completed before the CTA ends
        volatile int never = 0;
        warp_wait(smem_u32(&c->done), 0, p.ws, &never);
      }
    }
  } else if (BLOCKS == 1 && warp < Regs::FIRST_ROWS) {  // one relay for both, in the order in which the rows' warps ask
    if (work)
      for (int j = 0; j <= n; ++j) {
        if (j < n) relay_one<160>(smem_u32(&c->sfull[0]), 1, j, p.ws, abort);
        if (j > 0) relay_one<160>(smem_u32(&c->pdone[0]), 3, j - 1, p.ws, abort);
      }
  } else if (warp < Regs::FIRST_ROWS) {
    const int t = warp % 2, what = (warp - 4) / 2;
    if (work) relay<160>(smem_u32(what ? &c->pdone[t] : &c->sfull[t]), 1 + what * 2 + t, tiles_of(t), p.ws, abort);
  } else {
    Regs::take();
    const int t = (warp - Regs::FIRST_ROWS) / 4;
    const int r = (warp % 4) * 32 + lane;  // this thread's row: a lane of tensor memory
    const int row = row0 + (turns ? 0 : t * p.rows) + r / p.group, head = w.head * p.group + r % p.group;
    const bool live = w.ok && t < blocks && r < p.rows * p.group && row < d.queries;
    const bool any = __any_sync(0xffffffffu, live);
    const uint32_t at = tmem + ((uint32_t)(warp % 4) << 21);
    // rows behind the last one: nothing is masked and nothing stored
    const int hi = live ? (int)seen_end(d, p.plan.frame, row) : INT_MAX - COLS;
    const int first = w.begin + first_of(t), many = uniform(work ? tiles_of(t) : 0);
    // tiles up to the first one that some row does not see whole
    const int whole = uniform((max(__reduce_min_sync(0xffffffffu, hi / COLS) - first, 0) + step - 1) / step);
    float m = -INFINITY, mc = 0.f, l = 0.f;  // the maximum in use, -m c, and the sum
    if (many > 0) {
      const uint32_t s_at = at + F::S + t * COLS, p_at = at + F::P + t * F::P_STEP, o_at = at + F::O + t * PD;
      const uint32_t sfree = smem_u32(&c->sfree[t]), pready = smem_u32(&c->pready[t]);
      for (int j = 0; j < many && !any; ++j) {  // rows behind the last one alone: nothing to do but to keep step
        __syncwarp();
        meet<160>(1 + t);
        if (lane == 0) mbar_arrive(sfree);
        __syncwarp();
        if (j > 0) meet<160>(3 + t);
        if (lane == 0) mbar_arrive(pready);
      }
      for (int j = 0; j < many && any; ++j) {
        __syncwarp();
        meet<160>(1 + t);
        fence_after();
        uint32_t s[COLS];
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_max(s_at + k * 32, s + k * 32, mx[k]);
        tmem_wait();
        pin(s);
        asm volatile("" : "+f"(mx[0]), "+f"(mx[1]), "+f"(mx[2]), "+f"(mx[3]));
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree);
        if (j >= whole) {
          const int upto = hi - (first + j * step) * COLS;
#pragma unroll
          for (int i = 0; i < COLS; ++i)
            if (i >= upto) s[i] = 0xff800000u;  // -infinity
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = -INFINITY;
#pragma unroll
          for (int i = 0; i < COLS; i += 2) mx[i / 2 % 4] = max3(mx[i / 2 % 4], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        }
        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        const bool moves = __any_sync(0xffffffffu, (top - m) * p.c > GROWTH);  // also from no maximum to any
        if (j > 0) {  // the products that read P and write O are done
          meet<160>(3 + t);
          fence_after();
        }
        if (moves) {
          const float next = (top - m) * p.c > GROWTH ? top : m;
          const float grow = next == m ? 1.f : exp2_approx((m - next) * p.c);
          m = next;
          mc = m == -INFINITY ? 0.f : -m * p.c;
          l *= grow;
          if (j > 0) {
#pragma unroll
            for (int k = 0; k < PD; k += 32) {
              uint32_t o[32];
              tmem_ld32(o_at + k, o);
              tmem_wait();
              pin(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * grow);
              tmem_st16(o_at + k, o);
              tmem_st16(o_at + k + 16, o + 16);
            }
          }
        }
        const float2 c2 = make_float2(p.c, p.c), m2 = make_float2(mc, mc);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int k = 0; k < COLS / 2; k += 16) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 x = fma2(make_float2(__uint_as_float(s[2 * (k + i)]), __uint_as_float(s[2 * (k + i) + 1])), c2, m2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            sum[i % 2] = add2(sum[i % 2], x);
            pk[i] = f2_to_bf16x2(x.x, x.y);
          }
          tmem_st16(p_at + k, pk);
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready);
      }
      __syncwarp();
      meet<160>(3 + t);
      fence_after();
    }
    bool ok = !__any_sync(0xffffffffu, *abort);
    // the other half's products read the same queries, whose place the results pass through
    if (turns && work) ok = warp_wait(smem_u32(&c->done), 0, p.ws, abort) && ok;
    if (ok && any) {  // a warp's loads of tensor memory are whole; what is not live is not stored
      const bool empty = !live || hi == 0 || many == 0;
      const float inv = 1.f / l;
      const int64_t at_row = (int64_t)d.q0 + row;
      __nv_bfloat16* out = p.out.ptr + at_row * p.out.row + head * p.out.head;
      const bool part = SPLIT && w.slot >= 0;
      const int64_t slot = (int64_t)w.slot + row - row0 + (turns && t ? min(p.rows, d.queries - row0) : 0);
      const bool room = !part || slot < p.plan.slots;
      float* mine = part ? p.partial + ((int64_t)head * p.plan.slots + slot) * PARTIAL<PD> : nullptr;
      const uint32_t stage = smem + t * F::Q_BYTES + (warp % 4) * 4096;  // the queries are done with
#pragma unroll
      for (int k = 0; k < PD; k += 64) {
        uint32_t o[64];
        __syncwarp();
        tmem_ld32(at + F::O + t * PD + k, o);
        tmem_ld32(at + F::O + t * PD + k + 32, o + 32);
        tmem_wait();
        pin(o);
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (empty) o[i] = 0u;
        uint4 v[8];
        if (part) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = make_uint4(o[32 * h + 4 * i], o[32 * h + 4 * i + 1], o[32 * h + 4 * i + 2], o[32 * h + 4 * i + 3]);
            store_rows<8>(stage, v, mine + k + 32 * h, live && room, 8);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = pack8(o + 8 * i, empty ? 0.f : inv);
          store_rows<8>(stage, v, out + k, live, (p.plan.dim - k + 7) / 8);
        }
      }
      const float mc = m == -INFINITY ? -INFINITY : m * p.c;
      if (live && part && room) *reinterpret_cast<float2*>(mine + PD) = make_float2(empty ? -INFINITY : mc, empty ? 0.f : l);
      if (live && !part && p.lse) p.lse[(int64_t)head * p.plan.padded_rows + (int64_t)d.tile0 * TILE + row] = empty ? -INFINITY : mc + log2_approx(l);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free(tmem, F::COLUMNS);
  }
}

// The pieces of a split item, joined: o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i in the pieces' order.  Bound by latency: a lane
// holds the maximum and the sum of every 32nd piece, and those and the first pieces' values are asked for at once.  Two rows
// of a head to a warp, or, where an item has few rows, several warps to a row, each with a share of its pieces.  4 us for 64 rows of
// 18 pieces of 128 dimensions behind single tokens; 81,000 partial rows of 64, 22 MB, 13 us.
constexpr int JOIN_WARPS = 8, JOIN_ROWS = 2 * JOIN_WARPS;  // of a CTA
template <int PD>
using JoinVec = typename std::conditional<PD == 64, float2, float4>::type;  // a lane's dimensions

// Rows r0 to r0 + EACH - 1, pieces [begin, end): their part of o and of the sum, under the row's maximum over all pieces.
template <int PD, int EACH, int AHEAD>
struct Joined {
  float m[EACH], sum[EACH], o[EACH][PD / 32];
  __device__ __forceinline__ Joined(const FwdArgs& p, const Work& w, int r0, int begin, int end) {
    const int rows = w.slot, pieces = w.end, lane = threadIdx.x % 32;
    const int64_t step = (int64_t)rows * PARTIAL<PD>;
    const float* from = p.partial + ((int64_t)w.head * p.plan.slots + w.begin + r0) * PARTIAL<PD>;
    auto stat = [&](int r, int i) {  // maximum and sum of piece i; none: no key seen
      return r0 + r < rows && i < pieces ? __ldcg(reinterpret_cast<const float2*>(from + r * PARTIAL<PD> + i * step + PD)) : make_float2(-INFINITY, 0.f);
    };
    auto value = [&](int r, int i) {
      return r0 + r < rows && i < end ? __ldcg(reinterpret_cast<const JoinVec<PD>*>(from + r * PARTIAL<PD> + i * step) + lane) : JoinVec<PD>{};
    };
    JoinVec<PD> v[EACH][AHEAD];
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      m[r] = stat(r, lane).x;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) v[r][k] = value(r, begin + k);
    }
    float2 ml[EACH];
#pragma unroll
    for (int r = 0; r < EACH; ++r) {
      ml[r] = begin + lane < end ? stat(r, begin + lane) : make_float2(-INFINITY, 0.f);
      for (int i = lane + 32; i < pieces; i += 32) m[r] = fmaxf(m[r], stat(r, i).x);
      m[r] = warp_max_f(m[r]);
      sum[r] = 0.f;
#pragma unroll
      for (int e = 0; e < PD / 32; ++e) o[r][e] = 0.f;
    }
    for (int first = begin; first < end; first += 32) {
      float f[EACH], l[EACH];
#pragma unroll
      for (int r = 0; r < EACH; ++r) {
        if (first > begin) ml[r] = first + lane < end ? stat(r, first + lane) : make_float2(-INFINITY, 0.f);
        f[r] = ml[r].x == -INFINITY ? 0.f : exp2_approx(ml[r].x - m[r]);
        l[r] = ml[r].x == -INFINITY ? ml[r].y : f[r] * ml[r].y;
        if (ml[r].x == -INFINITY && ml[r].y == 0.f) f[r] = -1.f;  // it has seen no key of this row
      }
      const int many = min(32, end - first);
      for (int i = 0; i < many; i += AHEAD) {
#pragma unroll
        for (int r = 0; r < EACH; ++r) {
          if (first + i > begin)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[r][k] = value(r, first + i + k);
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {  // lanes behind the last piece have f -1 and l 0
            const float g = __shfl_sync(0xffffffffu, f[r], i + k);
            sum[r] += __shfl_sync(0xffffffffu, l[r], i + k);
            const float* b = reinterpret_cast<const float*>(&v[r][k]);
#pragma unroll
            for (int e = 0; e < PD / 32; ++e)
              if (!(g < 0.f)) o[r][e] += g * b[e];
          }
        }
      }
    }
  }
};

template <int PD>
__device__ __forceinline__ void store_joined(const FwdArgs& p, const Work& w, int r, float m, float sum, const float (&o)[PD / 32]) {
  constexpr int EACH = PD / 32;
  const int lane = threadIdx.x % 32;
  const int64_t row = (int64_t)w.row0 + r;
  const bool empty = seen_end(w.doc, p.plan.frame, row) == 0;  // a query that sees no key
  __nv_bfloat16* out = p.out.ptr + (w.doc.q0 + row) * p.out.row + w.head * p.out.head + lane * EACH;
  const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
  for (int k = 0; k < EACH; k += 2)
    if (lane * EACH + k < p.plan.dim) *reinterpret_cast<uint32_t*>(out + k) = f2_to_bf16x2(o[k] * inv, o[k + 1] * inv);
  if (lane == 0 && p.lse) p.lse[(int64_t)w.head * p.plan.padded_rows + (int64_t)w.doc.tile0 * TILE + row] = empty ? -INFINITY : m + log2_approx(sum);
}

template <int PD>
__global__ void __launch_bounds__(32 * JOIN_WARPS) k_attention_join(const __grid_constant__ FwdArgs p) {
  pdl_launch_dependents();
  __shared__ float parts[JOIN_WARPS][PD + 1];
  pdl_wait();
  const Work w = find_work(p.table, p.plan, JOIN, p.plan.heads, p.ws);
  if (!w.ok) return;
  const int rows = w.slot, pieces = w.end, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (rows <= 0 || pieces <= 0 || (int64_t)w.row0 + rows > w.doc.queries || (int64_t)w.begin + (int64_t)rows * pieces > p.plan.slots) {
    if (threadIdx.x == 0) raise_status(p.ws, DIT_ERR_INVALID_ARG);
    return;
  }
  if (rows >= JOIN_WARPS) {
    const int r0 = blockIdx.y * JOIN_ROWS + warp * 2;
    if (r0 >= rows) return;
    const Joined<PD, 2, 4> j(p, w, r0, 0, pieces);
    store_joined<PD>(p, w, r0, j.m[0], j.sum[0], j.o[0]);
    if (r0 + 1 < rows) store_joined<PD>(p, w, r0 + 1, j.m[1], j.sum[1], j.o[1]);
    return;
  }
  if (blockIdx.y > 0) return;
  const int each = rows > 4 ? 1 : rows > 2 ? 2 : rows > 1 ? 4 : 8;  // warps to a row
  const int r = warp / each, part = warp % each, per = (pieces + each - 1) / each;
  float m = 0.f, sum = 0.f, o[PD / 32] = {};
  if (r < rows) {
    const Joined<PD, 1, 8> j(p, w, r, min(part * per, pieces), min((part + 1) * per, pieces));
    m = j.m[0], sum = j.sum[0];
#pragma unroll
    for (int e = 0; e < PD / 32; ++e) o[e] = j.o[0][e];
  }
#pragma unroll
  for (int e = 0; e < PD / 32; ++e) parts[warp][lane * (PD / 32) + e] = o[e];
  if (lane == 0) parts[warp][PD] = sum;
  __syncthreads();
  if (r >= rows || part) return;
  for (int k = 1; k < each; ++k) {  // in the pieces' order
    sum += parts[warp + k][PD];
#pragma unroll
    for (int e = 0; e < PD / 32; ++e) o[e] += parts[warp + k][lane * (PD / 32) + e];
  }
  store_joined<PD>(p, w, r, m, sum, o);
}

template <int PD, bool SPLIT, int BLOCKS>
static dit_status launch(FwdArgs& a, const Heads& q, const Heads& k, const Heads& v, cudaStream_t st) {
  using F = Fwd<PD, BLOCKS>;
  using Regs = typename F::Regs;
  static OncePerDevice checked, once;
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded: any tensor makes a map
  const bool keys = a.plan.k_rows > 0;
  const int64_t k_rows = keys ? a.plan.k_rows : a.plan.q_rows;
  const int k_heads = keys ? a.plan.kv_heads : a.plan.heads;
  if (!map_heads(&mq, q, a.plan.dim, a.plan.heads, a.plan.q_rows, a.group, a.rows) ||
      !map_heads(&mk, keys ? k : q, a.plan.dim, k_heads, k_rows, 1, F::COLS) || !map_heads(&mv, keys ? v : q, a.plan.dim, k_heads, k_rows, 1, F::COLS))
    return DIT_ERR_CUDA;
  if (prepare_kernel<Regs>(checked, once, k_attention<PD, SPLIT, BLOCKS>, F::SMEM) != cudaSuccess) return DIT_ERR_CUDA;
  if (launch_pdl(k_attention<PD, SPLIT, BLOCKS>, dim3((unsigned)(a.plan.items[FORWARD] * a.plan.kv_heads)), dim3(Regs::THREADS), F::SMEM, st, 1, mq, mk, mv, a) != cudaSuccess)
    return DIT_ERR_CUDA;
  if (SPLIT && launch_pdl(k_attention_join<PD>, dim3((unsigned)(a.plan.items[JOIN] * a.plan.heads), (unsigned)(2 * a.rows + JOIN_ROWS - 1) / JOIN_ROWS), dim3(32 * JOIN_WARPS), 0, st, 1, a) != cudaSuccess)
    return DIT_ERR_CUDA;
  return DIT_OK;
}

}  // namespace attn
}  // namespace dit6

using namespace dit6;

extern "C" dit_status dit_attention(const dit_attention_plan_t* plan, const int32_t* table, const dit_heads_t* q, const dit_heads_t* k,
                                    const dit_heads_t* v, const dit_heads_t* out, double scale, void* saved, size_t saved_bytes,
                                    void* scratch, size_t scratch_bytes, void* ws, size_t ws_bytes, dit_stream_t stream) {
  using namespace attn;
  if (!plan_ok(plan) || (!table && plan->table_ints > 0) || !ws || ws_bytes < WS_BYTES || !(scale > 0.0) || !isfinite(scale)) return DIT_ERR_INVALID_ARG;
  if (saved && !plan->training) return DIT_ERR_INVALID_ARG;
  if (saved && saved_bytes < (size_t)plan->saved_bytes) return DIT_ERR_INVALID_ARG;
  if (scratch_bytes < (size_t)plan->scratch_bytes || (plan->scratch_bytes && !scratch)) return DIT_ERR_INVALID_ARG;
  Heads hq, hk, hv, ho;
  dit_status e = check_view(q, plan->heads, plan->q_rows, plan->dim, &hq);
  if (e == DIT_OK) e = check_view(k, plan->kv_heads, plan->k_rows, plan->dim, &hk);
  if (e == DIT_OK) e = check_view(v, plan->kv_heads, plan->k_rows, plan->dim, &hv);
  if (e == DIT_OK) e = check_output(out, plan->heads, plan->q_rows, plan->dim, &ho);
  if (e != DIT_OK) return e;
  if (!aligned32(ws) || (reinterpret_cast<uintptr_t>(table) & 15) || (reinterpret_cast<uintptr_t>(saved) & 15) || (reinterpret_cast<uintptr_t>(scratch) & 15))
    return DIT_ERR_ALIGNMENT;
  if (plan->items[FORWARD] == 0) return DIT_OK;
  FwdArgs a = {};
  a.plan = *plan;
  a.table = table;
  a.out = ho;
  a.lse = reinterpret_cast<float*>(saved);
  a.partial = reinterpret_cast<float*>(scratch);
  a.ws = ws;
  a.c = (float)(scale * 1.4426950408889634);
  a.group = plan->heads / plan->kv_heads;
  a.rows = rows_per_tile(a.group);
  a.stall = test_stall();
  if (!(a.c >= FLT_MIN && a.c <= FLT_MAX)) return DIT_ERR_INVALID_ARG;  // in fp32 too
  if (!buffers_apart(*plan, saved, scratch, ws)) return DIT_ERR_INVALID_ARG;
  const bool split = plan->items[JOIN] > 0;
  if (plan->dim > 64) return split ? launch<128, true, 1>(a, hq, hk, hv, stream) : launch<128, false, 1>(a, hq, hk, hv, stream);
  if (plan->row_blocks == 1) return launch<64, false, 1>(a, hq, hk, hv, stream);
  return split ? launch<64, true, 2>(a, hq, hk, hv, stream) : launch<64, false, 2>(a, hq, hk, hv, stream);
}
