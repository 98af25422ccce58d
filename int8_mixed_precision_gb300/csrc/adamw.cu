// One AdamW step over many tensors, with the moments in 32 or in 8 bits.
//
// Bound by memory: per element 2 x p + g + 4 x moment (+ copy) bytes and about 15 operations.  One
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
constexpr int THREADS = 256;  // 8 warps, two blocks each
constexpr float E4M3_MAX = 448.f;
constexpr float TINY = 7.8886090522101181e-31f;  // 2^-100

struct Factors {
  float beta1, one_beta1, beta2, one_beta2, keep, rate, root, eps;
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
__device__ __forceinline__ V8 load8_codes(const void* base, int64_t i, int count, float scale) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + i;
  uint2 c = make_uint2(0, 0);
  if (count == 8) {
    c = __ldcs(reinterpret_cast<const uint2*>(p));
  } else {
    for (int j = 0; j < count; ++j) {
      const uint32_t b = (uint32_t)p[j] << (8 * (j & 3));
      if (j < 4)
        c.x |= b;
      else
        c.y |= b;
    }
  }
  V8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = e4m3x2_values((j < 2 ? c.x : c.y) >> (16 * (j & 1)));
    o.v[2 * j] = __fmul_rn(f.x, scale);
    o.v[2 * j + 1] = __fmul_rn(f.y, scale);
  }
  return o;
}
// Codes of eight values of a block whose largest magnitude is amax; ROOT: no nonzero value gets code 0.
template <bool ROOT>
__device__ __forceinline__ void store8_codes(void* base, int64_t i, int count, const V8& v, float amax) {
  const bool fine = amax >= TINY;
  const float to_code = fine ? __fdiv_rn(E4M3_MAX, amax) : 0.f;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t c = e4m3x2(__fmul_rn(v.v[2 * j], to_code), __fmul_rn(v.v[2 * j + 1], to_code));
    if (ROOT && fine) {
      if (!(c & 0x00ffu) && v.v[2 * j] > 0.f) c |= 1u;
      if (!(c & 0xff00u) && v.v[2 * j + 1] > 0.f) c |= 0x100u;
    }
    w[j / 2] |= c << (16 * (j & 1));
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

// The chunk of this CTA: its descriptor, and [begin, end) of its elements (empty if the table is wrong).
__device__ __forceinline__ bool load_chunk(const dit_adamw_tensor* descs, int64_t n_tensors, const int2* chunks,
                                           dit_adamw_tensor& d, int64_t& begin, int64_t& end, void* ws) {
  const int2 c = chunks[blockIdx.x];
  if (c.x < 0 || c.x >= n_tensors || c.y < 0) {
    if (threadIdx.x == 0) raise_status(ws, DIT_ERR_INVALID_ARG);
    return false;
  }
  d = descs[c.x];
  begin = (int64_t)c.y * CHUNK;
  end = min(begin + CHUNK, d.n);
  return true;
}

template <typename P, typename G, bool CODES>
__global__ void __launch_bounds__(THREADS) k_adamw(const dit_adamw_tensor* __restrict__ descs, int64_t n_tensors,
                                                   const int2* __restrict__ chunks, Factors f,
                                                   const float* __restrict__ grad_scale, void* ws) {
  pdl_launch_dependents();
  pdl_wait();
  dit_adamw_tensor d;
  int64_t begin, end;
  if (!load_chunk(descs, n_tensors, chunks, d, begin, end, ws)) return;
  const float gs = grad_scale ? *grad_scale : 1.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t b0 = begin + warp * BLOCK; b0 < end; b0 += (THREADS / 32) * BLOCK) {
    const int64_t i = b0 + lane * 8;
    const int count = (int)max((int64_t)0, min((int64_t)8, end - i));
    V8 g = load8<G>(d.g, i, count), p = load8<P>(d.p, i, count), m, v;
    if (CODES) {
      m = load8_codes(d.m, i, count, d.m_scale[b0 / BLOCK]);
      v = load8_codes(d.v, i, count, d.v_scale[b0 / BLOCK]);
    } else {
      m = load8<float>(d.m, i, count);
      v = load8<float>(d.v, i, count);
    }
    V8 u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = __fmul_rn(g.v[j], gs);
      if (CODES) v.v[j] = __fmul_rn(v.v[j], v.v[j]);
      m.v[j] = __fadd_rn(__fmul_rn(m.v[j], f.beta1), __fmul_rn(gj, f.one_beta1));
      v.v[j] = __fadd_rn(__fmul_rn(v.v[j], f.beta2), __fmul_rn(__fmul_rn(gj, gj), f.one_beta2));
      u.v[j] = __fsqrt_rn(v.v[j]);
      const float step = __fdiv_rn(__fmul_rn(m.v[j], f.rate), __fadd_rn(__fmul_rn(u.v[j], f.root), f.eps));
      p.v[j] = __fsub_rn(__fmul_rn(p.v[j], f.keep), step);
    }
    store8<P>(d.p, i, count, p);
    if (d.copy) store8<__nv_bfloat16>(d.copy, i, count, p);
    if (CODES) {
      // elements past the tensor's end are zeros here (0 gradient, 0 moments)
      const float am = warp_amax(m), au = warp_amax(u);
      store8_codes<false>(d.m, i, count, m, am);
      store8_codes<true>(d.v, i, count, u, au);
      if (lane == 0) {
        d.m_scale[b0 / BLOCK] = am >= TINY ? __fmul_rn(am, 1.f / E4M3_MAX) : 0.f;
        d.v_scale[b0 / BLOCK] = au >= TINY ? __fmul_rn(au, 1.f / E4M3_MAX) : 0.f;
      }
    } else {
      store8<float>(d.m, i, count, m);
      store8<float>(d.v, i, count, v);
    }
  }
}

__global__ void __launch_bounds__(THREADS) k_adamw_moments(const dit_adamw_tensor* __restrict__ descs, int64_t n_tensors,
                                                           const int2* __restrict__ chunks, void* ws) {
  pdl_launch_dependents();
  pdl_wait();
  dit_adamw_tensor d;
  int64_t begin, end;
  if (!load_chunk(descs, n_tensors, chunks, d, begin, end, ws)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t b0 = begin + warp * BLOCK; b0 < end; b0 += (THREADS / 32) * BLOCK) {
    const int64_t i = b0 + lane * 8;
    const int count = (int)max((int64_t)0, min((int64_t)8, end - i));
    if (d.m_values) store8<__nv_bfloat16>(d.m_values, i, count, load8_codes(d.m, i, count, d.m_scale[b0 / BLOCK]));
    if (d.v_values) {
      V8 u = load8_codes(d.v, i, count, d.v_scale[b0 / BLOCK]);
#pragma unroll
      for (int j = 0; j < 8; ++j) u.v[j] = __fmul_rn(u.v[j], u.v[j]);
      store8<__nv_bfloat16>(d.v_values, i, count, u);
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

template <typename P, typename G>
static cudaError_t launch(bool codes, const dit_adamw_tensor* descs, int64_t n_tensors, const int2* chunks, int64_t n_chunks,
                          const Factors& f, const float* gs, void* ws, cudaStream_t st) {
  return launch_pdl(codes ? k_adamw<P, G, true> : k_adamw<P, G, false>, dim3((unsigned)n_chunks), dim3(THREADS), 0, st, 1,
                    descs, n_tensors, chunks, f, gs, ws);
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
  f.keep = (float)(1.0 - args->lr * args->weight_decay);
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
  return launch_pdl(k_adamw_moments, dim3((unsigned)n_chunks), dim3(THREADS), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                    descs, n_tensors, reinterpret_cast<const int2*>(chunks), ws) == cudaSuccess
             ? DIT_OK
             : DIT_ERR_CUDA;
}
