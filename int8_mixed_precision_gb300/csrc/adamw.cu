// One AdamW step over many tensors, with the moments in 32 or in 8 bits.
//
// Bound by memory: per element 2 x p + g + 4 x moment (+ copy) bytes and about 16 operations.  (32-bit moments,
// fp32 parameters, bf16 gradients, 265 M elements: 1.00 ms, 6.9 TB/s, the copy rate.)  One
// launch covers all tensors: a CTA takes one chunk of 4096 consecutive elements of one tensor
// from a table, a warp 256 of them at a time (8 to a lane: 32-byte vectors of fp32), which is
// also the block that shares a scale of the 8-bit moments, so its largest magnitude is
// a warp reduction and no element is read twice.  Each operation is rounded to fp32 on its own
// (no contraction), so that the moments' codes are reproducible by any fp32 program.
#include <math.h>

#include "common.cuh"

namespace dit6 {
namespace adamw {

constexpr int CHUNK = DIT_ADAMW_CHUNK;
constexpr int BLOCK = 256;    // elements that share a scale
constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr float E4M3_MAX = 448.f;
constexpr float TINY = 7.8886090522101181e-31f;  // 2^-100

struct Factors {
  float beta1, one_beta1, beta2, one_beta2, decay, rate, root, eps;
};

struct V8 {
  float v[8];
};

// eight elements from i on; the first `count` of them exist (vectors when all do)
template <typename T>
__device__ __forceinline__ V8 load8(const void* base, int64_t i, int count);
template <>
__device__ __forceinline__ V8 load8<float>(const void* base, int64_t i, int count) {
  V8 o;
  const float* p = reinterpret_cast<const float*>(base) + i;
  if (count == 8) {
    const U8x32 r = ld256(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = __uint_as_float(r.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = j < count ? p[j] : 0.f;
  }
  return o;
}
template <>
__device__ __forceinline__ V8 load8<__nv_bfloat16>(const void* base, int64_t i, int count) {
  V8 o;
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(base) + i;
  if (count == 8) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = bf16x2_to_f2(w[j]);
      o.v[2 * j] = f.x;
      o.v[2 * j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = j < count ? __bfloat162float(p[j]) : 0.f;
  }
  return o;
}
template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t i, int count, const V8& o);
template <>
__device__ __forceinline__ void store8<float>(void* base, int64_t i, int count, const V8& o) {
  float* p = reinterpret_cast<float*>(base) + i;
  if (count == 8) {
    U8x32 r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(o.v[j]);
    st256(p, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) p[j] = o.v[j];
  }
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(void* base, int64_t i, int count, const V8& o) {
  __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(base) + i;
  if (count == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(f2_to_bf16x2(o.v[0], o.v[1]), f2_to_bf16x2(o.v[2], o.v[3]),
                                              f2_to_bf16x2(o.v[4], o.v[5]), f2_to_bf16x2(o.v[6], o.v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) p[j] = __float2bfloat16_rn(o.v[j]);
  }
}

// E4M3 codes: two values per 16-bit half (the first in its low byte)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_values(uint32_t code) {
  uint32_t h2;
  const uint16_t c = (uint16_t)code;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  return make_float2(__half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu))),
                     __half2float(__ushort_as_half((unsigned short)(h2 >> 16))));
}
__device__ __forceinline__ uint2 load_codes(const void* base, int64_t i, int count) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + i;
  if (count == 8) return *reinterpret_cast<const uint2*>(p);
  uint2 c = make_uint2(0, 0);
  for (int j = 0; j < count; ++j) {
    const uint32_t b = (uint32_t)p[j] << (8 * (j & 3));
    if (j < 4)
      c.x |= b;
    else
      c.y |= b;
  }
  return c;
}
__device__ __forceinline__ V8 codes8(uint2 c, float scale) {
  V8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = e4m3x2_values((j < 2 ? c.x : c.y) >> (16 * (j & 1)));
    const float2 x = mul2(f, make_float2(scale, scale));
    o.v[2 * j] = x.x;
    o.v[2 * j + 1] = x.y;
  }
  return o;
}
__device__ __forceinline__ V8 load8_codes(const void* base, int64_t i, int count, float scale) {
  return codes8(load_codes(base, i, count), scale);
}
// Codes of eight values of a block whose largest magnitude is amax; ROOT: no nonzero value gets code 0.
template <bool ROOT>
__device__ __forceinline__ void store8_codes(void* base, int64_t i, int count, const V8& v, float amax) {
  const bool fine = amax >= TINY;
  const float to_code = fine ? __fdiv_rn(E4M3_MAX, amax) : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 x = mul2(make_float2(v.v[2 * j], v.v[2 * j + 1]), make_float2(to_code, to_code));
    if (ROOT && fine) {  // values below the smallest code are lifted to it, zeros (and NaN) stay
      x.x = v.v[2 * j] > 0.f ? fmaxf(x.x, 0x1p-9f) : v.v[2 * j];
      x.y = v.v[2 * j + 1] > 0.f ? fmaxf(x.y, 0x1p-9f) : v.v[2 * j + 1];
    }
    w[j / 2] |= e4m3x2(x.x, x.y) << (16 * (j & 1));
  }
  uint8_t* p = reinterpret_cast<uint8_t*>(base) + i;
  if (count == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    for (int j = 0; j < count; ++j) p[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}
__device__ __forceinline__ float warp_amax(const V8& v) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v.v[j]));
  return warp_max_f(m);
}

// A CTA's share of the chunk table is contiguous; a walk takes it as ranges, each a stretch of
// consecutive chunks of one tensor.  A range that points nowhere has no elements and raises the
// status word.
struct Walk {
  const dit_adamw_tensor* descs;
  const int2* chunks;
  int64_t n_tensors, at, last;
  dit_adamw_tensor d;
  int64_t begin, end;  // elements

  __device__ __forceinline__ Walk(const dit_adamw_tensor* descs_, int64_t n_tensors_, const int2* chunks_, int64_t n_chunks)
      : descs(descs_), chunks(chunks_), n_tensors(n_tensors_) {
    at = n_chunks * blockIdx.x / gridDim.x;
    last = n_chunks * (blockIdx.x + 1) / gridDim.x;
  }
  __device__ __forceinline__ bool step(void* ws) {
    if (at >= last) return false;
    const int2 c = chunks[at];
    begin = end = 0;
    if (c.x < 0 || c.x >= n_tensors || c.y < 0) {
      if (threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
      ++at;
      return true;
    }
    d = descs[c.x];
    begin = (int64_t)c.y * CHUNK;
    if (begin >= d.n && threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
    // the rest of the tensor or of the share, if the table's last entry of it says the same
    int64_t n = min(last - at, (d.n - begin + CHUNK - 1) / CHUNK);
    if (n > 1) {
      const int2 e = chunks[at + n - 1];
      if (e.x != c.x || e.y != c.y + (int)(n - 1)) n = 1;
    }
    if (n < 1) n = 1;
    end = min(begin + n * CHUNK, d.n);
    at += n;
    return true;
  }
};

// p, m, v and u = sqrt(v) of eight elements after the step.  Each product and sum is rounded on its own.
// With 32-bit moments, where memory leaves time for it, the quotient is too; with 8-bit ones it is the
// hardware's approximation (within 2 units in the last place), which only the step of p sees.
__device__ __forceinline__ float div_approx(float a, float b) {
  float r;
  asm("div.approx.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <bool CODES>
__device__ __forceinline__ void update8(V8& p, const V8& g, V8& m, V8& v, V8& u, float gs, const Factors& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = __fmul_rn(g.v[j], gs);
    m.v[j] = __fadd_rn(__fmul_rn(m.v[j], f.beta1), __fmul_rn(gj, f.one_beta1));
    v.v[j] = __fadd_rn(__fmul_rn(v.v[j], f.beta2), __fmul_rn(__fmul_rn(gj, gj), f.one_beta2));
    u.v[j] = __fsqrt_rn(v.v[j]);
    const float top = __fmul_rn(m.v[j], f.rate), under = __fadd_rn(__fmul_rn(u.v[j], f.root), f.eps);
    // The decay goes into the step, not into a factor of p: 1 - lr wd in fp32 comes in steps of 2^-24, which at a
    // rate of 1e-5 and a decay of 0.01 makes it 19 % too large, and at 1e-6 nothing.
    p.v[j] = __fsub_rn(p.v[j], __fadd_rn(__fmul_rn(p.v[j], f.decay), CODES ? div_approx(top, under) : __fdiv_rn(top, under)));
  }
}

template <typename P, typename G>
__global__ void __launch_bounds__(THREADS)
    k_adamw(const dit_adamw_tensor* __restrict__ descs, int64_t n_tensors, const int2* __restrict__ chunks, int64_t n_chunks,
            Factors f, const float* __restrict__ grad_scale, void* ws) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk w(descs, n_tensors, chunks, n_chunks);
  const float gs = grad_scale ? *grad_scale : 1.f;
  while (w.step(ws)) {
    const dit_adamw_tensor& d = w.d;
    for (int64_t b0 = w.begin + warp * BLOCK; b0 < w.end; b0 += WARPS * BLOCK) {
      const int64_t i = b0 + lane * 8;
      const int count = (int)max((int64_t)0, min((int64_t)8, w.end - i));
      V8 g = load8<G>(d.g, i, count), p = load8<P>(d.p, i, count), m = load8<float>(d.m, i, count),
         v = load8<float>(d.v, i, count), u;
      update8<false>(p, g, m, v, u, gs, f);
      store8<P>(d.p, i, count, p);
      if (d.copy) store8<__nv_bfloat16>(d.copy, i, count, p);
      store8<float>(d.m, i, count, m);
      store8<float>(d.v, i, count, v);
    }
  }
}

// The step with 8-bit moments moves 10 to 18 bytes an element for about 60 instructions.  With a CTA to
// each chunk its dependent chain (table entry, descriptor, data) bound it, 392 us for 59 M elements in
// fp32 with copies; with persistent CTAs and plain loads the warps of an SM waited together and then
// computed together, 238.  Here persistent CTAs take every gridDim-th chunk and everything is
// fetched ahead: a chunk's table entry three chunks before its turn, its descriptor two (a word to
// each lane), its elements one, by cp.async into the warp's own shared memory.  179 us, 5.9 TB/s.
constexpr int BLOCKS = CHUNK / BLOCK / WARPS;  // of a chunk to a warp
constexpr int DEPTH = 2;                       // chunks in shared memory
template <typename P, typename G>
struct Stage {  // one block, as it lies in memory
  uint4 p[sizeof(P) / 2 * 32], g[sizeof(G) / 2 * 32];
  uint2 m[32], v[32];
  float scale[2];
};
template <int N>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ V8 staged8(const uint4* s, int lane) {
  V8 o;
  if (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 r = s[2 * lane + h];
      o.v[4 * h] = __uint_as_float(r.x);
      o.v[4 * h + 1] = __uint_as_float(r.y);
      o.v[4 * h + 2] = __uint_as_float(r.z);
      o.v[4 * h + 3] = __uint_as_float(r.w);
    }
  } else {
    const uint4 r = s[lane];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = bf16x2_to_f2(w[j]);
      o.v[2 * j] = f.x;
      o.v[2 * j + 1] = f.y;
    }
  }
  return o;
}

// A chunk as a warp holds it: word l of the descriptor in lane l, and the chunk's elements.
struct Ahead {
  uint32_t word;
  int64_t begin, end;
  __device__ __forceinline__ void load(const dit_adamw_tensor* descs, int64_t n_tensors, int2 entry, bool there, void* ws) {
    begin = end = 0;
    word = 0;
    if (!there) return;
    if (entry.x < 0 || entry.x >= n_tensors || entry.y < 0) {
      if (threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
      return;
    }
    const int lane = threadIdx.x & 31;
    if (lane < (int)(sizeof(dit_adamw_tensor) / 4)) word = reinterpret_cast<const uint32_t*>(descs + entry.x)[lane];
    begin = (int64_t)entry.y * CHUNK;
    end = begin + CHUNK;  // the tensor's size is not there yet
  }
  __device__ __forceinline__ uint64_t field(int i) const {
    return (uint64_t)__shfl_sync(0xffffffffu, word, 2 * i + 1) << 32 | __shfl_sync(0xffffffffu, word, 2 * i);
  }
  __device__ __forceinline__ void clip(void* ws) {
    const int64_t n = (int64_t)field(9);
    if (end > begin && n <= begin && threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
    end = max(begin, min(end, n));
  }
};
static_assert(sizeof(dit_adamw_tensor) == 80, "ten words of 64 bits");

template <typename P, typename G>
__global__ void __launch_bounds__(THREADS, 2)
    k_adamw_codes(const dit_adamw_tensor* __restrict__ descs, int64_t n_tensors, const int2* __restrict__ chunks,
                  int64_t n_chunks, Factors f, const float* __restrict__ grad_scale, void* ws) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ uint4 raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Stage<P, G>* stages = reinterpret_cast<Stage<P, G>*>(raw) + warp * DEPTH * BLOCKS;
  const int64_t step = gridDim.x;
  auto entry_at = [&](int64_t t) { return t < n_chunks ? chunks[t] : make_int2(0, 0); };
  int64_t at = blockIdx.x;
  const int2 e0 = entry_at(at), e1 = entry_at(at + step);
  int2 e2 = entry_at(at + 2 * step);
  const float gs = grad_scale ? *grad_scale : 1.f;
  Ahead now, next, later;
  now.load(descs, n_tensors, e0, at < n_chunks, ws);
  next.load(descs, n_tensors, e1, at + step < n_chunks, ws);
  now.clip(ws);

  // whole blocks go through shared memory, a tensor's last partial one does not
  auto fetch = [&](const Ahead& c, Stage<P, G>* to) {
    const char *p = reinterpret_cast<const char*>(c.field(0)), *g = reinterpret_cast<const char*>(c.field(1)),
               *m = reinterpret_cast<const char*>(c.field(2)), *v = reinterpret_cast<const char*>(c.field(3));
    const float *ms = reinterpret_cast<const float*>(c.field(4)), *vs = reinterpret_cast<const float*>(c.field(5));
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
      const int64_t b0 = c.begin + (k * WARPS + warp) * BLOCK;
      if (b0 + BLOCK > c.end) continue;
      Stage<P, G>& t = to[k];  // 16 (or 8) consecutive bytes to a lane: whole lines to an instruction
#pragma unroll
      for (int h = 0; h < (int)sizeof(P) / 2; ++h) copy_async<16>(&t.p[h * 32 + lane], p + b0 * sizeof(P) + 512 * h + 16 * lane);
#pragma unroll
      for (int h = 0; h < (int)sizeof(G) / 2; ++h) copy_async<16>(&t.g[h * 32 + lane], g + b0 * sizeof(G) + 512 * h + 16 * lane);
      copy_async<8>(&t.m[lane], m + b0 + 8 * lane);
      copy_async<8>(&t.v[lane], v + b0 + 8 * lane);
      if (lane < 2) copy_async<4>(&t.scale[lane], (lane ? vs : ms) + b0 / BLOCK);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(now, stages);
  for (int s = 0; at < n_chunks; at += step, s ^= 1) {
    later.load(descs, n_tensors, e2, at + 2 * step < n_chunks, ws);
    e2 = entry_at(at + 3 * step);
    next.clip(ws);
    fetch(next, stages + (s ^ 1) * BLOCKS);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();  // the other lanes' copies too
    void *dp = reinterpret_cast<void*>(now.field(0)), *dm = reinterpret_cast<void*>(now.field(2)),
         *dv = reinterpret_cast<void*>(now.field(3)), *copy = reinterpret_cast<void*>(now.field(6));
    const void* dg = reinterpret_cast<const void*>(now.field(1));
    float *m_scale = reinterpret_cast<float*>(now.field(4)), *v_scale = reinterpret_cast<float*>(now.field(5));
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
      const int64_t b0 = now.begin + (k * WARPS + warp) * BLOCK, i = b0 + lane * 8;
      if (b0 >= now.end) continue;
      const int count = (int)max((int64_t)0, min((int64_t)8, now.end - i));
      V8 g, p, m, v, u;
      if (b0 + BLOCK <= now.end) {
        const Stage<P, G>& t = stages[s * BLOCKS + k];
        g = staged8<G>(t.g, lane);
        p = staged8<P>(t.p, lane);
        m = codes8(t.m[lane], t.scale[0]);
        v = codes8(t.v[lane], t.scale[1]);
      } else {
        g = load8<G>(dg, i, count);
        p = load8<P>(dp, i, count);
        m = load8_codes(dm, i, count, m_scale[b0 / BLOCK]);
        v = load8_codes(dv, i, count, v_scale[b0 / BLOCK]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v.v[j] = __fmul_rn(v.v[j], v.v[j]);
      update8<true>(p, g, m, v, u, gs, f);
      store8<P>(dp, i, count, p);
      if (copy) store8<__nv_bfloat16>(copy, i, count, p);
      // elements past the tensor's end are zeros here (0 gradient, 0 moments)
      const float am = warp_amax(m), au = warp_amax(u);
      store8_codes<false>(dm, i, count, m, am);
      store8_codes<true>(dv, i, count, u, au);
      if (lane == 0) {
        m_scale[b0 / BLOCK] = am >= TINY ? __fmul_rn(am, 1.f / E4M3_MAX) : 0.f;
        v_scale[b0 / BLOCK] = au >= TINY ? __fmul_rn(au, 1.f / E4M3_MAX) : 0.f;
      }
    }
    now = next;
    next = later;
    __syncwarp();  // every lane has read what the next copies overwrite
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Bound by memory and then by latency: four blocks' loads of a warp are in flight together, from four chunks
// to a CTA where there are enough (59 M elements: 56 us, 6.3 TB/s; 64 with a few persistent CTAs, whose
// distant streams cost DRAM more), from one where there are few (1 M elements: 4 us against 6).
__global__ void __launch_bounds__(THREADS)
    k_adamw_moments(const dit_adamw_tensor* __restrict__ descs, int64_t n_tensors, const int2* __restrict__ chunks,
                    int64_t n_chunks, void* ws) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk w(descs, n_tensors, chunks, n_chunks);
  constexpr int AHEAD = 4;
  while (w.step(ws)) {
    const dit_adamw_tensor& d = w.d;
    for (int64_t b0 = w.begin + warp * BLOCK; b0 < w.end; b0 += AHEAD * WARPS * BLOCK) {
      uint2 m[AHEAD], v[AHEAD];
      float ms[AHEAD], vs[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int64_t b = b0 + a * WARPS * BLOCK, i = b + lane * 8;
        const int count = (int)max((int64_t)0, min((int64_t)8, w.end - i));
        m[a] = v[a] = make_uint2(0, 0);
        ms[a] = vs[a] = 0.f;
        if (count > 0 && d.m_values) {
          m[a] = load_codes(d.m, i, count);
          ms[a] = d.m_scale[b / BLOCK];
        }
        if (count > 0 && d.v_values) {
          v[a] = load_codes(d.v, i, count);
          vs[a] = d.v_scale[b / BLOCK];
        }
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int64_t i = b0 + a * WARPS * BLOCK + lane * 8;
        const int count = (int)max((int64_t)0, min((int64_t)8, w.end - i));
        if (d.m_values) store8<__nv_bfloat16>(d.m_values, i, count, codes8(m[a], ms[a]));
        if (d.v_values) {
          V8 u = codes8(v[a], vs[a]);
#pragma unroll
          for (int j = 0; j < 8; ++j) u.v[j] = __fmul_rn(u.v[j], u.v[j]);
          store8<__nv_bfloat16>(d.v_values, i, count, u);
        }
      }
    }
  }
}

static dit_status check_tables(const void* descs, int64_t n_tensors, const void* chunks, int64_t n_chunks, const void* ws,
                               size_t ws_bytes) {
  if (n_tensors < 0 || n_chunks < 0 || n_tensors > 0x7fffffff || n_chunks > 0x7fffffff || !ws || ws_bytes < WS_BYTES)
    return DIT_ERR_INVALID_ARG;
  if (n_chunks && (!descs || !chunks || !n_tensors)) return DIT_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(descs) & 15) || (reinterpret_cast<uintptr_t>(chunks) & 7) || !aligned32(ws))
    return DIT_ERR_ALIGNMENT;
  return DIT_OK;
}

static unsigned few(int64_t n_chunks, int ctas_per_sm) {
  const int64_t most = (int64_t)num_sms() * ctas_per_sm;
  return (unsigned)(n_chunks < most ? n_chunks : most);
}
// 32-bit moments: a CTA to each chunk (265 M elements: 0.99 ms, against 1.07 with persistent CTAs); 8-bit
// moments: persistent CTAs, so that the loads run ahead through many blocks.
template <typename P, typename G>
static cudaError_t launch(bool codes, const dit_adamw_tensor* descs, int64_t n_tensors, const int2* chunks, int64_t n_chunks,
                          const Factors& f, const float* gs, void* ws, cudaStream_t st) {
  if (!codes)
    return launch_pdl(k_adamw<P, G>, dim3((unsigned)n_chunks), dim3(THREADS), 0, st, 1, descs, n_tensors, chunks, n_chunks, f,
                      gs, ws);
  constexpr int SMEM = sizeof(Stage<P, G>) * DEPTH * BLOCKS * WARPS;
  static OncePerDevice once;
  const cudaError_t allowed = opt_in_smem(once, k_adamw_codes<P, G>, SMEM);
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(k_adamw_codes<P, G>, dim3(few(n_chunks, 2)), dim3(THREADS), SMEM, st, 1, descs, n_tensors, chunks, n_chunks,
                    f, gs, ws);
}

}  // namespace adamw
}  // namespace dit6

extern "C" int64_t dit_adamw_chunks(const int64_t* sizes, int64_t n_tensors, int32_t* table, int64_t n_chunks) {
  if (n_tensors < 0 || n_tensors > 0x7fffffff || (n_tensors > 0 && !sizes)) return -1;
  int64_t count = 0;
  for (int64_t t = 0; t < n_tensors; ++t) {
    if (sizes[t] < 0 || sizes[t] > ((int64_t)1 << 42)) return -1;
    const int64_t c = (sizes[t] + DIT_ADAMW_CHUNK - 1) / DIT_ADAMW_CHUNK;
    if (count + c > 0x7fffffff) return -1;
    if (table)
      for (int64_t i = 0; i < c; ++i) {
        if (count + i >= n_chunks) return -1;
        table[2 * (count + i)] = (int32_t)t;
        table[2 * (count + i) + 1] = (int32_t)i;
      }
    count += c;
  }
  return count;
}

extern "C" dit_status dit_adamw_step(const dit_adamw_tensor* descs, int64_t n_tensors, const int32_t* chunks,
                                     int64_t n_chunks, dit_dtype p_dt, dit_dtype g_dt, int moment_bits,
                                     const dit_adamw_args* args, const float* grad_scale, void* ws, size_t ws_bytes,
                                     dit_stream_t stream) {
  using namespace dit6;
  using namespace dit6::adamw;
  const dit_status bad = check_tables(descs, n_tensors, chunks, n_chunks, ws, ws_bytes);
  if (bad != DIT_OK) return bad;
  if (!args || args->step < 1 || (moment_bits != 8 && moment_bits != 32)) return DIT_ERR_INVALID_ARG;
  if ((p_dt != DIT_F32 && p_dt != DIT_BF16) || (g_dt != DIT_F32 && g_dt != DIT_BF16)) return DIT_ERR_INVALID_ARG;
  if (!(args->beta1 >= 0 && args->beta1 < 1) || !(args->beta2 >= 0 && args->beta2 < 1) || !(args->eps >= 0) ||
      !isfinite(args->lr) || !isfinite(args->weight_decay))
    return DIT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(grad_scale) & 3) return DIT_ERR_ALIGNMENT;
  if (n_chunks == 0) return DIT_OK;
  Factors f;
  f.beta1 = (float)args->beta1;
  f.one_beta1 = (float)(1.0 - args->beta1);
  f.beta2 = (float)args->beta2;
  f.one_beta2 = (float)(1.0 - args->beta2);
  f.decay = (float)(args->lr * args->weight_decay);
  f.rate = (float)(args->lr / (1.0 - pow(args->beta1, (double)args->step)));
  f.root = (float)(1.0 / sqrt(1.0 - pow(args->beta2, (double)args->step)));
  f.eps = (float)args->eps;
  const int2* ch = reinterpret_cast<const int2*>(chunks);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool codes = moment_bits == 8;
  using B = __nv_bfloat16;
  cudaError_t e;
  if (p_dt == DIT_F32)
    e = g_dt == DIT_F32 ? launch<float, float>(codes, descs, n_tensors, ch, n_chunks, f, grad_scale, ws, st)
                        : launch<float, B>(codes, descs, n_tensors, ch, n_chunks, f, grad_scale, ws, st);
  else
    e = g_dt == DIT_F32 ? launch<B, float>(codes, descs, n_tensors, ch, n_chunks, f, grad_scale, ws, st)
                        : launch<B, B>(codes, descs, n_tensors, ch, n_chunks, f, grad_scale, ws, st);
  return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

extern "C" dit_status dit_adamw_moments(const dit_adamw_tensor* descs, int64_t n_tensors, const int32_t* chunks,
                                        int64_t n_chunks, void* ws, size_t ws_bytes, dit_stream_t stream) {
  using namespace dit6;
  using namespace dit6::adamw;
  const dit_status bad = check_tables(descs, n_tensors, chunks, n_chunks, ws, ws_bytes);
  if (bad != DIT_OK) return bad;
  if (n_chunks == 0) return DIT_OK;
  const int64_t ctas = n_chunks <= 8 * num_sms() ? n_chunks : (n_chunks + 3) / 4;
  return launch_pdl(k_adamw_moments, dim3((unsigned)ctas), dim3(THREADS), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                    descs, n_tensors, reinterpret_cast<const int2*>(chunks), n_chunks, ws) == cudaSuccess
             ? DIT_OK
             : DIT_ERR_CUDA;
}
