// Low-rank adapters for short requests: y[t] += scale (x[t] A^T) B^T for tiles of up to 16 rows that
// share an adapter, wherever in the batch they are (single tokens of a serving batch above all).
//
// Bound by latency (one token, 1920 -> 5760 at rank 16: 5.9 us a call, 5.4 in a graph; 64 tokens over 16 adapters,
// 1920 -> 7680 at rank 32: 9.6 us, 1.2 TB/s), and then by reading each adapter's A and B once: 16 rows reuse a weight far too
// little to fill a 128-row tcgen05 instruction, so the products run on mma.sync (16 x 8 x 16) with
// both operands loaded from global memory straight into fragments; a product's contraction
// index may be permuted freely, so every lane loads 16 (or 8) contiguous bytes and takes them for the
// elements that the fragment wants of it.
//
// One launch: a cluster of CTAs takes a tile.  Each CTA contracts its share of k and leaves a partial h in
// its shared memory; after one cluster barrier every CTA sums all of them (in the CTAs' order, so
// all get the same bits) and takes its share of the n columns, whose weights and old values are
// loaded 16 or 32 columns of a warp ahead, the first ones before the barrier.
#include "adapters.cuh"

namespace dit6 {
namespace lora {

constexpr int SMALL_WARPS = 8, SMALL_THREADS = 32 * SMALL_WARPS;

struct Small {
  const int32_t* tiles;
  const __nv_bfloat16 *x, *a, *b;
  const float* scale;
  void* y;
  int64_t rows, k, n;
  int n_adapters, rank, rp, cluster;
  void* ws;
};

// d += a b: a 16 x 16 (row), b 16 x 8 (col)
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();  // the barriers want converged warps
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same about the lifetime of what other CTAs read alone
__device__ __forceinline__ void cluster_arrive_relaxed() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// What a lane loads for 16 columns of the result: its share of their weights and its four old values of two
// rows.  Tile t of the two has the columns n0 + 4 (s / 2) + 2 t + s % 2 in its slots s, so that a
// lane's two pairs of results are four consecutive columns.
template <int RT, bool BF16>
struct Columns {
  static constexpr int STEPS = (RT + 3) / 4;  // of 32 along the rank
  uint4 w0[STEPS], w1[STEPS], was_lo, was_hi;
  __device__ __forceinline__ void load(const Small& p, const __nv_bfloat16* b, int64_t n0, int64_t n_last, int row_lo,
                                       int row_hi, bool has_lo, bool has_hi) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, c4 = lane & 3;
    const int64_t b0 = n0 + 4 * (g8 >> 1) + (g8 & 1), b1 = b0 + 2, col = n0 + c4 * 4;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int k = j * 32 + c4 * 8;  // the rank is a multiple of 8
      w0[j] = w1[j] = make_uint4(0, 0, 0, 0);
      if (n0 < n_last && k < p.rank && b0 < p.n) w0[j] = *reinterpret_cast<const uint4*>(b + b0 * p.rank + k);
      if (n0 < n_last && k < p.rank && b1 < p.n) w1[j] = *reinterpret_cast<const uint4*>(b + b1 * p.rank + k);
    }
    was_lo = was_hi = make_uint4(0, 0, 0, 0);
    if (n0 >= n_last || col >= p.n) return;
    if (has_lo) was_lo = old(p, row_lo, col);
    if (has_hi) was_hi = old(p, row_hi, col);
  }
  static __device__ __forceinline__ uint4 old(const Small& p, int row, int64_t col) {
    if (!BF16) return *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p.y) + (int64_t)row * p.n + col);
    const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p.y) + (int64_t)row * p.n + col);
    return make_uint4(v.x, v.y, 0, 0);
  }
  static __device__ __forceinline__ void store(const Small& p, int row, int64_t col, const uint4& was, float v0, float v1,
                                               float v2, float v3) {
    if (BF16) {
      const float2 e = bf16x2_to_f2(was.x), f = bf16x2_to_f2(was.y);
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.y) + (int64_t)row * p.n + col) =
          make_uint2(f2_to_bf16x2(e.x + v0, e.y + v1), f2_to_bf16x2(f.x + v2, f.y + v3));
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.y) + (int64_t)row * p.n + col) =
          make_float4(__uint_as_float(was.x) + v0, __uint_as_float(was.y) + v1, __uint_as_float(was.z) + v2,
                      __uint_as_float(was.w) + v3);
    }
  }
};

// RT: tiles of 8 of the rank at least (a bound on registers)
template <int RT, bool BF16>
__global__ void __launch_bounds__(SMALL_THREADS) k_small(Small p) {
  extern __shared__ float sm[];
  float* part = sm;                                // [warps][16][rp], then this CTA's h in the first [16][rp]
  float* sum = sm + SMALL_WARPS * 16 * p.rp;       // this CTA's partial h [16][rp], read by the cluster
  const int P = BF16 ? 2 : PARTS;                  // parts of h (see adapters.cuh)
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(sum + 16 * p.rp);  // [P][16][rp + 8]
  const int hp = p.rp + 8;                         // rows 16 bytes apart in banks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, c4 = lane & 3;
  const uint32_t rank_in = p.cluster > 1 ? cluster_rank() : 0;
  pdl_wait();
  const int32_t* tile = p.tiles + (int64_t)(blockIdx.x / p.cluster) * SMALL_INTS;
  const int4 head = *reinterpret_cast<const int4*>(tile);
  const int g = head.x, count = head.y;
  // every lane looks at one row of the tile; the whole cluster comes to the same verdict
  const int mine = lane < 16 ? tile[4 + lane] : 0;
  const bool bad = g < 0 || g >= p.n_adapters || count < 0 || count > SMALL_ROWS ||
                   __any_sync(0xffffffffu, lane < count && (mine < 0 || mine >= p.rows));
  if (bad) {
    if (threadIdx.x == 0) raise_status(p.ws, DIT_ERR_INVALID_ARG);
    return;
  }
  const int row_lo = __shfl_sync(0xffffffffu, mine, g8), row_hi = __shfl_sync(0xffffffffu, mine, g8 + 8);
  const bool has_lo = g8 < count, has_hi = g8 + 8 < count;

  const float scale = p.scale[g];

  // this CTA's share of the columns, in groups of 16
  const int64_t groups = (p.n + 15) / 16;
  const int64_t n_first = groups * rank_in / p.cluster * 16, n_last = min(p.n, groups * (rank_in + 1) / p.cluster * 16);
  const __nv_bfloat16* b = p.b + (int64_t)g * p.n * p.rank;

  // ---- h over this CTA's share of k, 32 elements of it to a warp at a time
  float acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  const int64_t steps = (p.k + 31) / 32;
  const int64_t k_first = steps * rank_in / p.cluster, k_last = steps * (rank_in + 1) / p.cluster;
  const __nv_bfloat16* a = p.a + (int64_t)g * p.rank * p.k;
  const int tiles8 = p.rank / 8;
  // The tensor cores' additions cut their sums to 24 bits, so every DRAIN steps (256 elements) the sums are added to
  // those of before, with rounding to nearest, where the warp's share of h is left at the end anyway.
  constexpr int DRAIN = 8;
  bool drained = false;
  auto drain = [&](bool again) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (i < tiles8) {
        float2* at = reinterpret_cast<float2*>(part + ((int64_t)warp * 16 + g8) * p.rp + i * 8 + c4 * 2);
#pragma unroll
        for (int half = 0; half < 2; ++half, at += 4 * p.rp) {
          float2 sum = make_float2(acc[i][2 * half], acc[i][2 * half + 1]);
          if (again) sum = make_float2(at->x + sum.x, at->y + sum.y);
          *at = sum;
        }
      }
  };
  int64_t s = k_first + warp;
  for (int64_t stop = k_first + DRAIN * SMALL_WARPS;; stop += DRAIN * SMALL_WARPS) {
    for (; s < min(k_last, stop); s += SMALL_WARPS) {
      const int64_t k = s * 32 + c4 * 8;  // this lane's eight elements: four of each 16-deep step
      const bool in = k < p.k;
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (in && has_lo) lo = *reinterpret_cast<const uint4*>(p.x + (int64_t)row_lo * p.k + k);
      if (in && has_hi) hi = *reinterpret_cast<const uint4*>(p.x + (int64_t)row_hi * p.k + k);
      uint4 w[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (in && i < tiles8) w[i] = *reinterpret_cast<const uint4*>(a + (int64_t)(i * 8 + g8) * p.k + k);
      }
      const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
      for (int i = 0; i < RT; ++i)
        if (i < tiles8) {
          mma_16816(acc[i], a0, w[i].x, w[i].y);
          mma_16816(acc[i], a1, w[i].z, w[i].w);
        }
    }
    if (stop >= k_last) break;
    drain(drained);
    drained = true;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  }
  // The next kernel's CTAs come in from here on: earlier, they would take issue slots and L1 from this one's
  // loads (64 tokens over 16 adapters: 14.9 us a call, against 11.3).
  pdl_launch_dependents();
  // The first columns' weights and old values, while the partial sums meet.
  constexpr int AHEAD = RT <= 8 ? 2 : 1;  // more costs registers and code: 64 tokens 9.4 us with two, 10.5 with four
  constexpr int STRIDE = SMALL_WARPS * 16;
  Columns<RT, BF16> ahead[AHEAD];
  int64_t n0 = n_first + warp * 16;
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) ahead[d].load(p, b, n0 + d * STRIDE, n_last, row_lo, row_hi, has_lo, has_hi);
  if (drained)
    drain(true);
  else
    drain(false);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * p.rp; i += SMALL_THREADS) {
    float v = 0.f;
    if (i % p.rp < p.rank)
      for (int w = 0; w < SMALL_WARPS; ++w) v += part[w * 16 * p.rp + i];
    sum[i] = v;
  }
  if (p.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 16 * p.rp; i += SMALL_THREADS) {
    float v = 0.f;
    if (p.cluster > 1) {
      const uint32_t at = smem_u32(sum + i);
      float other[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) other[c] = c < p.cluster ? ld_cluster_f32(mapa_rank(at, c)) : 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) v += other[c];
    } else {
      v = sum[i];
    }
    v *= scale;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      if (q >= P) break;
      const __nv_bfloat16 first = __float2bfloat16_rn(v);
      h[(q * 16 + i / p.rp) * hp + i % p.rp] = first;
      const float f = __bfloat162float(first);
      v = isfinite(f) ? v - f : 0.f;
    }
  }
  if (p.cluster > 1) cluster_arrive_relaxed();  // this CTA has read the others' sums
  __syncthreads();

  // ---- y: 16 columns to a warp at a time; a lane ends with four consecutive ones of two rows
  while (n0 < n_last) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (n0 >= n_last) break;
      const Columns<RT, BF16> now = ahead[d];
      ahead[d].load(p, b, n0 + AHEAD * STRIDE, n_last, row_lo, row_hi, has_lo, has_hi);
      float d0[4] = {}, d1[4] = {};
      // The small parts first: an addition cuts the sum to 24 bits, and then only those of the largest parts meet
      // it at its full size.
#pragma unroll
      for (int q = PARTS - 1; q >= 0; --q) {
        if (q >= P) continue;
#pragma unroll
        for (int j = 0; j < Columns<RT, BF16>::STEPS; ++j) {
          const int k = j * 32 + c4 * 8;  // this lane's eight elements: four of each 16-deep step
          if (j * 32 >= p.rp) break;
          uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
          if (k < p.rp) {
            lo = *reinterpret_cast<const uint4*>(h + (q * 16 + g8) * hp + k);
            hi = *reinterpret_cast<const uint4*>(h + (q * 16 + g8 + 8) * hp + k);
          }
          const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
          mma_16816(d0, a0, now.w0[j].x, now.w0[j].y);
          mma_16816(d1, a0, now.w1[j].x, now.w1[j].y);
          mma_16816(d0, a1, now.w0[j].z, now.w0[j].w);
          mma_16816(d1, a1, now.w1[j].z, now.w1[j].w);
        }
      }
      const int64_t col = n0 + c4 * 4;
      if (has_lo && col < p.n) now.store(p, row_lo, col, now.was_lo, d0[0], d0[1], d1[0], d1[1]);
      if (has_hi && col < p.n) now.store(p, row_hi, col, now.was_hi, d0[2], d0[3], d1[2], d1[3]);
      n0 += STRIDE;
    }
  }
  if (p.cluster > 1) cluster_wait();  // nobody still reads this CTA's shared memory
}

template <int RT, bool BF16>
static cudaError_t launch_small(const Small& p, int tiles, cudaStream_t st) {
  const size_t smem = (size_t)(SMALL_WARPS + 1) * 16 * p.rp * 4 + (size_t)PARTS * 16 * (p.rp + 8) * 2;
  static OncePerDevice once;
  const cudaError_t allowed = opt_in_smem(once, k_small<RT, BF16>, 96 * 1024);
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(k_small<RT, BF16>, dim3((unsigned)(tiles * p.cluster)), dim3(SMALL_THREADS), smem, st,
                    (unsigned)p.cluster, p);
}

// The small tiles of a plan.
dit_status small_tiles(const dit_adapter_plan_t& plan, const int32_t* table, const void* x, const void* a, const void* b,
                       const float* scale, int rank, int64_t k, int64_t n, void* y, dit_dtype y_dt, void* ws,
                       cudaStream_t st) {
  if (!plan.n_small) return DIT_OK;
  Small p{table + off_small(plan), reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(a),
          reinterpret_cast<const __nv_bfloat16*>(b), scale, y, plan.rows, k, n, plan.n_adapters, rank, padded_rank(rank), 8,
          ws};
  // CTAs to a tile: as many as the SMs allow
  while (p.cluster > 1 && (int64_t)plan.n_small * p.cluster > 2 * num_sms()) p.cluster /= 2;
  const bool bf16 = y_dt == DIT_BF16;
  cudaError_t e;
  if (rank <= 16)
    e = bf16 ? launch_small<2, true>(p, plan.n_small, st) : launch_small<2, false>(p, plan.n_small, st);
  else if (rank <= 32)
    e = bf16 ? launch_small<4, true>(p, plan.n_small, st) : launch_small<4, false>(p, plan.n_small, st);
  else if (rank <= 64)
    e = bf16 ? launch_small<8, true>(p, plan.n_small, st) : launch_small<8, false>(p, plan.n_small, st);
  else
    e = bf16 ? launch_small<16, true>(p, plan.n_small, st) : launch_small<16, false>(p, plan.n_small, st);
  return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

}  // namespace lora
}  // namespace dit6
