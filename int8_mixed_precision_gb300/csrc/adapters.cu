// Low-rank adapters of many requests beside one shared projection: forward and backward.
//
//   h = scale (x A^T),  y += h B^T;   e = scale (dy B),  dx += e A,  dA = e^T x,  dB = dy^T h
//
// One product kernel in fp32 on the CUDA cores, 64 x 64 outputs per CTA, in three modes: to the
// rank (h, e), from the rank (y, dx) and over the rows (dA, dB).
#include "adapters.cuh"

namespace dit6 {
namespace lora {

enum Mode { TO_RANK, FROM_RANK, OVER_ROWS };

struct Args {
  const int32_t* table;
  const int32_t* first;
  int64_t rows;      // of the batch
  int n_adapters, n_tiles;
  const __nv_bfloat16* in;  // x or dy [rows x width]
  const __nv_bfloat16* w;   // A or B; element (rank j, column c) of adapter g at g * wg + j * wj + c * wc
  int64_t wg, wj, wc;
  const float* scale;
  float* held;       // h or e [n_tiles * 128 x rp]
  void* out;         // y or dx [rows x width] (FROM_RANK), dA or dB (OVER_ROWS, laid out like w)
  int out_bf16;
  int rank, rp;
  int64_t width;     // k or n
  void* ws;
};

template <int MODE>
__global__ void __launch_bounds__(256) k_lora_product(Args p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  // the CTA's tile and place: outputs [m0, m0 + 64) x [n0, n0 + 64)
  const int m0 = MODE == TO_RANK || MODE == FROM_RANK ? (blockIdx.x & 1) * 64 : (int)blockIdx.z * 64;
  const int64_t n0 = (int64_t)blockIdx.y * 64;
  int t0, t1, g;
  if (MODE == OVER_ROWS) {
    g = blockIdx.x;
    t0 = p.first[g];
    t1 = p.first[g + 1];
    if (t0 < 0 || t1 < t0 || t1 > p.n_tiles) {
      raise_status(p.ws, DIT_ERR_INVALID_ARG);
      t0 = t1 = 0;
    }
  } else {
    t0 = blockIdx.x >> 1;
    t1 = t0 + 1;
  }
  float acc[4][4] = {};
  Tile t{0, 0, 0};
  for (int ti = t0; ti < t1; ++ti) {
    t = load_tile(p.table, ti, p.rows, p.n_adapters, p.ws);
    if (MODE == OVER_ROWS && t.g != g) continue;
    const int64_t depth = MODE == TO_RANK ? p.width : MODE == FROM_RANK ? p.rank : t.rows;
    for (int64_t k0 = 0; k0 < depth; k0 += 16) {
      for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        // the faster index runs along memory
        const int kk = MODE == OVER_ROWS ? i / 64 : i % 16, mm = MODE == OVER_ROWS ? i % 64 : i / 16;
        const int64_t k = k0 + kk;
        float va = 0.f, vb = 0.f;
        if (k < depth) {
          const int m = m0 + mm;
          const int64_t n = n0 + mm;
          if (MODE == TO_RANK) {
            if (m < t.rows) va = __bfloat162float(p.in[((int64_t)t.row0 + m) * p.width + k]);
            if (n < p.rank) vb = __bfloat162float(p.w[t.g * p.wg + n * p.wj + k * p.wc]);
          } else if (MODE == FROM_RANK) {
            if (m < t.rows) va = p.held[((int64_t)ti * TILE_ROWS + m) * p.rp + k];
            if (n < p.width) vb = __bfloat162float(p.w[t.g * p.wg + k * p.wj + n * p.wc]);
          } else {
            if (m < p.rank) va = p.held[((int64_t)ti * TILE_ROWS + k) * p.rp + m];
            if (n < p.width) vb = __bfloat162float(p.in[((int64_t)t.row0 + k) * p.width + n]);
          }
        }
        sa[kk][mm] = va;
        sb[kk][mm] = vb;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 16; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty + 16 * i], sb[kk][tx + 16 * j], acc[i][j]);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i;
      const int64_t n = n0 + tx + 16 * j;
      if (MODE == TO_RANK) {
        if (n < p.rp)
          p.held[((int64_t)t0 * TILE_ROWS + m) * p.rp + n] = m < t.rows && n < p.rank ? acc[i][j] * p.scale[t.g] : 0.f;
      } else if (MODE == FROM_RANK) {
        if (m < t.rows && n < p.width) {
          const int64_t o = ((int64_t)t.row0 + m) * p.width + n;
          if (p.out_bf16) {
            __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.out);
            y[o] = __float2bfloat16_rn(__bfloat162float(y[o]) + acc[i][j]);
          } else {
            reinterpret_cast<float*>(p.out)[o] += acc[i][j];
          }
        }
      } else if (m < p.rank && n < p.width) {
        reinterpret_cast<float*>(p.out)[g * p.wg + m * p.wj + n * p.wc] = acc[i][j];
      }
    }
}

// A small tile: up to 16 rows anywhere in the batch; one CTA, h in shared memory.
__global__ void __launch_bounds__(256) k_lora_small(Args p, const int32_t* small, int64_t k, const __nv_bfloat16* b) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float h[SMALL_ROWS][MAX_RANK];
  __shared__ int rows[SMALL_ROWS];
  const int32_t* s = small + (int64_t)blockIdx.x * SMALL_INTS;
  const int g = s[0], count = s[1];
  bool bad = g < 0 || g >= p.n_adapters || count < 0 || count > SMALL_ROWS;
  for (int i = 0; i < count && !bad; ++i) bad = s[4 + i] < 0 || s[4 + i] >= p.rows;
  if (bad) {
    if (threadIdx.x == 0) raise_status(p.ws, DIT_ERR_INVALID_ARG);
    return;
  }
  if (threadIdx.x < count) rows[threadIdx.x] = s[4 + threadIdx.x];
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int o = warp; o < count * p.rank; o += 8) {
    const int i = o / p.rank, j = o % p.rank;
    const __nv_bfloat16* xr = p.in + (int64_t)rows[i] * k;
    const __nv_bfloat16* ar = p.w + g * p.wg + j * p.wj;
    float v = 0.f;
    for (int64_t c = lane; c < k; c += 32) v = fmaf(__bfloat162float(xr[c]), __bfloat162float(ar[c]), v);
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0) h[i][j] = v * p.scale[g];
  }
  __syncthreads();
  for (int64_t c = threadIdx.x; c < p.width; c += 256)
    for (int i = 0; i < count; ++i) {
      float v = 0.f;
      for (int j = 0; j < p.rank; ++j) v = fmaf(h[i][j], __bfloat162float(b[((int64_t)g * p.width + c) * p.rank + j]), v);
      const int64_t o = (int64_t)rows[i] * p.width + c;
      if (p.out_bf16) {
        __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.out);
        y[o] = __float2bfloat16_rn(__bfloat162float(y[o]) + v);
      } else {
        reinterpret_cast<float*>(p.out)[o] += v;
      }
    }
}

template <int MODE>
static dit_status product(const Args& a, cudaStream_t st) {
  if (MODE != OVER_ROWS && a.n_tiles == 0) return DIT_OK;
  const int64_t cols = MODE == TO_RANK ? a.rp : a.width;
  dim3 grid(MODE == OVER_ROWS ? a.n_adapters : 2 * a.n_tiles, (unsigned)((cols + 63) / 64),
            MODE == OVER_ROWS ? (a.rank + 63) / 64 : 1);
  return launch_pdl(k_lora_product<MODE>, grid, dim3(256), 0, st, 1, a) == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
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
  if (saved && (!plan->training || saved_bytes < held_bytes(plan->n_tiles, rank))) return DIT_ERR_INVALID_ARG;
  if (!aligned32(y) || !aligned32(saved)) return DIT_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Args p = {};
  p.table = table;
  p.first = table + off_first(*plan);
  p.rows = plan->rows;
  p.n_adapters = plan->n_adapters;
  p.n_tiles = plan->n_tiles;
  p.scale = scale;
  p.held = reinterpret_cast<float*>(saved ? saved : scratch);
  p.rank = rank;
  p.rp = padded_rank(rank);
  p.ws = ws;
  p.out = y;
  p.out_bf16 = y_dt == DIT_BF16;
  p.in = reinterpret_cast<const __nv_bfloat16*>(x);
  p.w = reinterpret_cast<const __nv_bfloat16*>(a);
  p.wg = rank * k;
  p.wj = k;
  p.wc = 1;
  p.width = k;
  dit_status s = product<TO_RANK>(p, st);
  Args q = p;
  q.w = reinterpret_cast<const __nv_bfloat16*>(b);
  q.wg = rank * n;
  q.wj = 1;
  q.wc = rank;
  q.width = n;
  if (s == DIT_OK) s = product<FROM_RANK>(q, st);
  if (s == DIT_OK && plan->n_small) {
    p.width = n;
    if (launch_pdl(k_lora_small, dim3(plan->n_small), dim3(256), 0, st, 1, p, table + off_small(*plan), k,
                   reinterpret_cast<const __nv_bfloat16*>(b)) != cudaSuccess)
      s = DIT_ERR_CUDA;
  }
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
      saved_bytes < held_bytes(plan->n_tiles, rank) || (!saved && plan->n_tiles > 0))
    return DIT_ERR_INVALID_ARG;
  if (!aligned32(dy) || !aligned32(saved) || !aligned32(dx) || !aligned32(da) || !aligned32(db)) return DIT_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Args p = {};
  p.table = table;
  p.first = table + off_first(*plan);
  p.rows = plan->rows;
  p.n_adapters = plan->n_adapters;
  p.n_tiles = plan->n_tiles;
  p.scale = scale;
  p.held = reinterpret_cast<float*>(scratch);
  p.rank = rank;
  p.rp = padded_rank(rank);
  p.ws = ws;
  Args along_n = p, along_k = p;
  along_n.in = reinterpret_cast<const __nv_bfloat16*>(dy);
  along_n.w = reinterpret_cast<const __nv_bfloat16*>(b);
  along_n.wg = rank * n;
  along_n.wj = 1;
  along_n.wc = rank;
  along_n.width = n;
  along_k.in = reinterpret_cast<const __nv_bfloat16*>(x);
  along_k.w = reinterpret_cast<const __nv_bfloat16*>(a);
  along_k.wg = rank * k;
  along_k.wj = k;
  along_k.wc = 1;
  along_k.width = k;
  dit_status s = product<TO_RANK>(along_n, st);
  along_k.out = dx;
  along_k.out_bf16 = dx_dt == DIT_BF16;
  if (s == DIT_OK && dx) s = product<FROM_RANK>(along_k, st);
  along_k.out = da;
  if (s == DIT_OK) s = product<OVER_ROWS>(along_k, st);
  along_n.out = db;
  along_n.held = reinterpret_cast<float*>(const_cast<void*>(saved));
  if (s == DIT_OK) s = product<OVER_ROWS>(along_n, st);
  return s;
}
