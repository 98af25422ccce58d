// Attention, forward: o = softmax(scale q k^T) v over the keys that each query sees.
//
// One pass over the keys with the running maximum and sum of the softmax.  A CTA holds two blocks of 128 rows (a row is
// a query and a head of the group that shares the keys) and streams keys and values through shared memory by
// TMA.  S = Q K^T goes to tensor memory, a thread to each row turns it into P (in bf16, back to tensor memory as
// the A operand of the next product) and O += P V stays there.  While the warps of one block work at their softmax
// the tensor cores have the other block's products, and S of the next tile is made as soon as the present one is in
// registers.
//
// The running maximum moves only when it grows by more than 2^GROWTH: until then P is larger than 1 by at
// most that factor, which neither bf16 nor fp32 sums mind, and O need not be rescaled.  The final division takes the
// same maximum out again.
//
// P is rounded to bf16 (an operand of the bf16 tensor pipe), 2^-8 of each weight at most; the sum of the weights is of the unrounded
// ones.  Scores are scaled inside the exponent's multiply-add, in base 2.
//
// Warps: 0 loads, 1 issues the MMAs, 4 to 7 and 8 to 11 are the blocks' rows and take over most of the first four
// warps' registers.  Every wait is bounded.
#include <math.h>

#include "attention.cuh"

namespace dit6 {
namespace attn {

using namespace lora;

constexpr float GROWTH = 8.f;
constexpr int FWD_STAGES = 6;  // most

template <int PD>
struct Fwd {
  static constexpr int COLS = tile_cols(PD);
  static constexpr int CHUNKS = PD / 64;
  static constexpr int Q_CHUNK = TILE * 128, Q_BYTES = CHUNKS * Q_CHUNK;
  static constexpr int KV_CHUNK = COLS * 128, KV_BYTES = CHUNKS * KV_CHUNK;
  static constexpr int STAGES = PD == 64 ? 6 : 5;
  static constexpr int CONTROL = 2 * Q_BYTES + 2 * STAGES * KV_BYTES;
  static constexpr int SMEM = CONTROL + 1024 + 1024;
  // tensor memory: S and P of each block, then O
  static constexpr uint32_t S = 0, P = 2 * COLS, O = 3 * COLS;
  static_assert(3 * COLS + 2 * PD <= 512 && SMEM <= 227 * 1024, "");
};

struct FwdControl {
  uint64_t qfull, done;
  uint64_t kfull[FWD_STAGES], kempty[FWD_STAGES], vfull[FWD_STAGES], vempty[FWD_STAGES];
  uint64_t sfull[2], sfree[2], pready[2], pdone[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(FwdControl) <= 1024, "");

struct FwdArgs {
  dit_attention_plan_t plan;
  const int32_t* table;
  Heads out;
  float* lse;       // [heads][padded rows], in base 2, or nullptr
  float* partial;   // [heads][slots][PD + 2]
  void* ws;
  float c;          // scale log2(e)
  int group, rows;  // heads of a group, queries of a block
  int stall;
};

template <int PD>
__global__ void __launch_bounds__(THREADS, 1)
    k_attention(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const __grid_constant__ FwdArgs p) {
  pdl_launch_dependents();
  using F = Fwd<PD>;
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
      mbar_init(smem_u32(&c->vempty[lane]), 1);
    } else if (lane >= 8 && lane < 10) {
      const int t = lane - 8;
      mbar_init(smem_u32(&c->sfull[t]), 1);
      mbar_init(smem_u32(&c->sfree[t]), 4);
      mbar_init(smem_u32(&c->pready[t]), 4);
      mbar_init(smem_u32(&c->pdone[t]), 1);
    } else if (lane == 10) {
      mbar_init(smem_u32(&c->qfull), 1);
      mbar_init(smem_u32(&c->done), 1);
      c->abort = 0;
    }
    fence_barrier_init();
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&c->tmem), 512);
    fence_before();
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = c->tmem;
  volatile int* abort = &c->abort;
  pdl_wait();

  const Work w = find_work(p.table, p.plan, FORWARD, p.plan.kv_heads, p.ws);
  const Doc& d = w.doc;
  const int row0 = w.item.row0;
  const int n = w.ok ? w.item.end - w.item.begin : 0;  // tiles
  const int blocks = w.ok && row0 + p.rows < d.queries ? 2 : 1;
  const bool work = n > 0 && (int64_t)w.item.end * COLS < (int64_t)d.keys + COLS;

  if (warp < 4) give_registers();
  if (warp == 0) {
    if (work && elect_one()) {
      uint32_t nk = 0, nv = 0;
      bool ok = true;
      if (!p.stall) {
        mbar_expect_tx(smem_u32(&c->qfull), blocks * F::CHUNKS * p.rows * p.group * 128);
        for (int t = 0; t < blocks; ++t)
          for (int k = 0; k < F::CHUNKS; ++k)
            tma_load_3d(smem + t * F::Q_BYTES + k * F::Q_CHUNK, &mq, smem_u32(&c->qfull), k * 64, w.head * p.group, d.q0 + row0 + t * p.rows);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int s = j % F::STAGES;
        const int row = d.k0 + (w.item.begin + j) * COLS;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const uint32_t full = smem_u32(kv ? &c->vfull[s] : &c->kfull[s]), empty = smem_u32(kv ? &c->vempty[s] : &c->kempty[s]);
          if (j >= F::STAGES && !mbar_wait(empty, ((j / F::STAGES) - 1) & 1, p.ws, abort)) {
            ok = false;
            break;
          }
          if (p.stall) continue;
          mbar_expect_tx(full, F::KV_BYTES);
          for (int k = 0; k < F::CHUNKS; ++k)
            tma_load_3d(smem + 2 * F::Q_BYTES + (kv * F::STAGES + s) * F::KV_BYTES + k * F::KV_CHUNK, kv ? &mv : &mk, full, k * 64, w.head, row);
          ++(kv ? nv : nk);
        }
      }
      if (!ok || *abort) {  // its own copies land before the CTA ends
        volatile int never = 0;
        if (!p.stall) mbar_wait(smem_u32(&c->qfull), 0, p.ws, &never);
        for (uint32_t i = nk > F::STAGES ? nk - F::STAGES : 0; i < nk; ++i) mbar_wait(smem_u32(&c->kfull[i % F::STAGES]), (i / F::STAGES) & 1, p.ws, &never);
        for (uint32_t i = nv > F::STAGES ? nv - F::STAGES : 0; i < nv; ++i) mbar_wait(smem_u32(&c->vfull[i % F::STAGES]), (i / F::STAGES) & 1, p.ws, &never);
      }
    }
  } else if (warp == 1) {
    if (work) {
      const uint32_t id_s = idesc(128, COLS, false, false);
      const uint32_t id_o = idesc(128, (p.plan.dim + 15) / 16 * 16, false, true);
      const int steps = (p.plan.dim + 15) / 16;
      bool ok = warp_wait(smem_u32(&c->qfull), 0, p.ws, abort);
      auto scores = [&](int j) {  // S of tile j for each block
        const int s = j % F::STAGES;
        ok = ok && warp_wait(smem_u32(&c->kfull[s]), (j / F::STAGES) & 1, p.ws, abort);
        for (int t = 0; t < blocks && ok; ++t) {
          if (j > 0) ok = warp_wait(smem_u32(&c->sfree[t]), (j - 1) & 1, p.ws, abort);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t a = desc_k(smem + t * F::Q_BYTES), b = desc_k(smem + 2 * F::Q_BYTES + s * F::KV_BYTES);
#pragma unroll
            for (int k = 0; k < PD / 16; ++k)
              if (k < steps)
                mma(tmem + F::S + t * COLS, a + (k / 4) * (F::Q_CHUNK >> 4) + (k % 4) * 2, b + (k / 4) * (F::KV_CHUNK >> 4) + (k % 4) * 2, id_s, k > 0);
            mma_commit(smem_u32(&c->sfull[t]));
            if (t == blocks - 1) mma_commit(smem_u32(&c->kempty[s]));
          }
          __syncwarp();
        }
      };
      scores(0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) scores(j + 1);
        const int s = j % F::STAGES;
        const uint32_t v = smem + 2 * F::Q_BYTES + (F::STAGES + s) * F::KV_BYTES;
        ok = ok && warp_wait(smem_u32(&c->vfull[s]), (j / F::STAGES) & 1, p.ws, abort);
        const int64_t left = (int64_t)d.keys - (int64_t)(w.item.begin + j) * COLS;
        if (ok && left < COLS) zero_rows(v, F::KV_CHUNK, F::CHUNKS, (int)left, COLS);
        for (int t = 0; t < blocks && ok; ++t) {
          ok = warp_wait(smem_u32(&c->pready[t]), j & 1, p.ws, abort);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t a = tmem + F::P + t * (COLS / 2), b = desc_mn(v, F::KV_CHUNK);
#pragma unroll
            for (int k = 0; k < COLS / 16; ++k) mma_ta(tmem + F::O + t * PD, a + k * 8, b + k * (2048 >> 4), id_o, j > 0 || k > 0);
            mma_commit(smem_u32(&c->pdone[t]));
            if (t == blocks - 1) mma_commit(smem_u32(&c->vempty[s]));
          }
          __syncwarp();
        }
      }
      volatile int never = 0;
      if (elect_one()) mma_commit(smem_u32(&c->done));
      __syncwarp();
      warp_wait(smem_u32(&c->done), 0, p.ws, &never);
    }
  } else if (warp >= 4) {
    take_registers();
    const int t = (warp - 4) / 4;
    const int r = (warp % 4) * 32 + lane;  // this thread's row: a lane of tensor memory
    const int row = row0 + t * p.rows + r / p.group, head = w.head * p.group + r % p.group;
    const bool live = w.ok && t < blocks && r < p.rows * p.group && row < d.queries;
    const bool any = __any_sync(0xffffffffu, live);
    const uint32_t at = tmem + ((uint32_t)(warp % 4) << 21);
    // rows behind the last one: nothing is masked and nothing stored
    const int64_t hi = live ? seen_end(d, p.plan.frame, row) : INT64_MAX;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (work && t < blocks) {
      for (int j = 0; j < n; ++j) {
        ok = warp_wait(smem_u32(&c->sfull[t]), j & 1, p.ws, abort);
        if (!ok) break;
        fence_after();
        uint32_t s[COLS];
        if (any) {
#pragma unroll
          for (int k = 0; k < COLS; k += 32) tmem_ld32(at + F::S + t * COLS + k, s + k);
          tmem_wait();
          pin(s);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c->sfree[t]));
        uint32_t pk[COLS / 2];
        float grow = 1.f;
        bool rescale = false;
        if (any) {
          const int col0 = (w.item.begin + j) * COLS;
          if (!__all_sync(0xffffffffu, hi >= (int64_t)col0 + COLS)) mask_cols(s, col0, 0, hi);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < COLS; ++i) mx[i % 4] = fmaxf(mx[i % 4], __uint_as_float(s[i]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if ((top - m) * p.c > GROWTH || (m == -INFINITY && top > m)) {
            grow = exp2_approx((m - top) * p.c);
            m = top;
            l *= grow;
          }
          rescale = j > 0 && __any_sync(0xffffffffu, grow != 1.f);
          const float mc = m == -INFINITY ? 0.f : -m * p.c;
          const float2 c2 = make_float2(p.c, p.c), m2 = make_float2(mc, mc);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) {
            float2 x = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, m2);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            sum[i % 2] = add2(sum[i % 2], x);
            pk[i] = f2_to_bf16x2(x.x, x.y);
          }
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
        }
        if (j > 0) {
          ok = warp_wait(smem_u32(&c->pdone[t]), (j - 1) & 1, p.ws, abort);
          if (!ok) break;
          fence_after();
        }
        __syncwarp();
        if (rescale) {
#pragma unroll
          for (int k = 0; k < PD; k += 32) {
            uint32_t o[32];
            tmem_ld32(at + F::O + t * PD + k, o);
            tmem_wait();
            pin(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * grow);
            tmem_st16(at + F::O + t * PD + k, o);
            tmem_st16(at + F::O + t * PD + k + 16, o + 16);
          }
        }
        if (any) {
#pragma unroll
          for (int k = 0; k < COLS / 2; k += 16) tmem_st16(at + F::P + t * (COLS / 2) + k, pk + k);
          tmem_st_wait();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c->pready[t]));
      }
      if (ok) {
        ok = warp_wait(smem_u32(&c->pdone[t]), (n - 1) & 1, p.ws, abort);
        fence_after();
      }
    }
    if (ok && any) {  // a warp's loads of tensor memory are whole; what is not live is not stored
      const bool empty = !live || hi == 0 || !work;
      const float inv = 1.f / l;
      const int64_t at_row = (int64_t)d.q0 + row;
      __nv_bfloat16* out = p.out.ptr + at_row * p.out.row + head * p.out.head;
      const bool part = w.item.slot >= 0;
      const bool room = !part || (int64_t)w.item.slot + row - row0 < p.plan.slots;
      float* mine = part ? p.partial + ((int64_t)head * p.plan.slots + w.item.slot + row - row0) * (PD + 2) : nullptr;
#pragma unroll
      for (int k = 0; k < PD; k += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(at + F::O + t * PD + k, o);
        tmem_wait();
        pin(o);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (empty) o[i] = 0u;
        if (live && part && room) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) *reinterpret_cast<uint2*>(mine + k + i) = make_uint2(o[i], o[i + 1]);
        } else if (live && !part) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            if (k + i < p.plan.dim) *reinterpret_cast<uint4*>(out + k + i) = pack8(o + i, empty ? 0.f : inv);
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
    tmem_free(tmem, 512);
  }
}

// The pieces of a split item, joined: o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i in the pieces' order, a warp to each row
// and head.
template <int PD>
__global__ void __launch_bounds__(256) k_attention_join(const __grid_constant__ FwdArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  const Work w = find_work(p.table, p.plan, JOIN, p.plan.heads, p.ws);
  if (!w.ok) return;
  const int rows = w.item.slot, pieces = w.item.end, lane = threadIdx.x % 32;
  if (rows <= 0 || (int64_t)w.item.row0 + rows > w.doc.queries || (int64_t)w.item.begin + (int64_t)rows * pieces > p.plan.slots) {
    if (threadIdx.x == 0) raise_status(p.ws, DIT_ERR_INVALID_ARG);
    return;
  }
  constexpr int EACH = PD / 32;
  for (int r = threadIdx.x / 32; r < rows; r += 8) {
    const float* from = p.partial + ((int64_t)w.head * p.plan.slots + w.item.begin + r) * (PD + 2);
    const int64_t step = (int64_t)rows * (PD + 2);
    float m = -INFINITY;
    for (int i = 0; i < pieces; ++i) m = fmaxf(m, __ldcg(from + i * step + PD));
    float sum = 0.f, o[EACH] = {};
    const bool empty = m == -INFINITY;
    for (int i = 0; i < pieces && !empty; ++i) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + i * step + PD));
      const float f = exp2_approx(ml.x - m);
      sum += f * ml.y;
      if (ml.x == -INFINITY) continue;
#pragma unroll
      for (int k = 0; k < EACH; k += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(from + i * step + lane * EACH + k));
        o[k] += f * v.x;
        o[k + 1] += f * v.y;
      }
    }
    const int64_t row = (int64_t)w.item.row0 + r;
    __nv_bfloat16* out = p.out.ptr + (w.doc.q0 + row) * p.out.row + w.head * p.out.head;
    const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < EACH; k += 2)
      if (lane * EACH + k < p.plan.dim) *reinterpret_cast<uint32_t*>(out + lane * EACH + k) = f2_to_bf16x2(o[k] * inv, o[k + 1] * inv);
    if (lane == 0 && p.lse) p.lse[(int64_t)w.head * p.plan.padded_rows + (int64_t)w.doc.tile0 * TILE + row] = empty ? -INFINITY : m + log2_approx(sum);
  }
}

template <int PD>
static dit_status launch(FwdArgs& a, const Heads& q, const Heads& k, const Heads& v, cudaStream_t st) {
  using F = Fwd<PD>;
  static OncePerDevice checked, once;
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded: any tensor makes a map
  const bool keys = a.plan.k_rows > 0;
  const int64_t k_rows = keys ? a.plan.k_rows : a.plan.q_rows;
  const int k_heads = keys ? a.plan.kv_heads : a.plan.heads;
  if (!map_heads(&mq, q, a.plan.dim, a.plan.heads, a.plan.q_rows, a.group, a.rows) ||
      !map_heads(&mk, keys ? k : q, a.plan.dim, k_heads, k_rows, 1, F::COLS) || !map_heads(&mv, keys ? v : q, a.plan.dim, k_heads, k_rows, 1, F::COLS))
    return DIT_ERR_CUDA;
  if (prepare_kernel(checked, once, k_attention<PD>, F::SMEM) != cudaSuccess) return DIT_ERR_CUDA;
  if (launch_pdl(k_attention<PD>, dim3((unsigned)(a.plan.items[FORWARD] * a.plan.kv_heads)), dim3(THREADS), F::SMEM, st, 1, mq, mk, mv, a) != cudaSuccess)
    return DIT_ERR_CUDA;
  if (a.plan.items[JOIN] && launch_pdl(k_attention_join<PD>, dim3((unsigned)(a.plan.items[JOIN] * a.plan.heads)), dim3(256), 0, st, 1, a) != cudaSuccess)
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
  if (!plan_ok(plan) || !table || !ws || ws_bytes < WS_BYTES || !(scale > 0.0) || !isfinite(scale)) return DIT_ERR_INVALID_ARG;
  if (saved && !plan->training) return DIT_ERR_INVALID_ARG;
  if (saved && saved_bytes < (size_t)plan->saved_bytes) return DIT_ERR_INVALID_ARG;
  if (scratch_bytes < (size_t)plan->scratch_bytes || (plan->scratch_bytes && !scratch)) return DIT_ERR_INVALID_ARG;
  Heads hq, hk, hv, ho;
  dit_status e = check_view(q, plan->heads, plan->q_rows, plan->dim, &hq);
  if (e == DIT_OK) e = check_view(k, plan->kv_heads, plan->k_rows, plan->dim, &hk);
  if (e == DIT_OK) e = check_view(v, plan->kv_heads, plan->k_rows, plan->dim, &hv);
  if (e == DIT_OK) e = check_view(out, plan->heads, plan->q_rows, plan->dim, &ho);
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
  return plan->dim <= 64 ? launch<64>(a, hq, hk, hv, stream) : launch<128>(a, hq, hk, hv, stream);
}
