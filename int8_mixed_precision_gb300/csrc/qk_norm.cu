// Norms of query and key heads with the position rotation in the same pass, and the gradients.
//
//   n = (x - mean) r w + b (layer), x r w (RMS);  y = n turned by its token's angles;
//   dn = dy turned back;  dx = r (g - mean(g) - xhat mean(g xhat)), g = dn w;  dw = sum dn xhat, db = sum dn
//
// Bound by memory: 4 bytes an element forward, 6 backward, and some 10 fp32 operations.  A head's row is
// spread over `lanes` lanes (a power of two, eight dimensions to a lane), so that a warp's loads are whole
// lines, its statistics are a few shuffles and both dimensions of a pair meet in one thread: a lane takes
// eight neighbouring dimensions where pairs are neighbours, else four of the first half of the turned
// dimensions and the four that pair with them.  A group of lanes stays with one token and walks over its heads, so
// the weights, the sines and the cosines are read once and stay in registers.
//
// Angles.  A pair's frequency is held in turns as a 64-bit fraction; position times frequency modulo 2^64 is
// the angle's fraction of a turn, by two integer multiplications, with no loss at far positions.
#include <math.h>

#include "common.cuh"

namespace dit6 {
namespace qk {

constexpr int THREADS = 256;
constexpr int MAX_DIM = 256;
constexpr int AHEAD = 4;         // heads of a thread in flight
constexpr int BACK_AHEAD = 2;
constexpr int MAX_CTAS = 152 * 2;  // of the backward pass, for each of q and k
constexpr int64_t MAX_TOKENS = 0x7fffff00;

struct Pair {
  uint64_t turn;  // turns a position, times 2^64
  int32_t axis;
  int32_t unused;
};
static_assert(sizeof(Pair) == 16, "");

struct View {
  const __nv_bfloat16* ptr;
  int64_t token, head;  // strides
};
struct Side {           // q or k
  View x, dy, y;        // backward: input, gradient of the output, gradient of the input
  const float *w, *b;
  float *dw, *db;
  int heads;
};
struct Args {
  Side side[2];
  int64_t tokens;
  const Pair* table;
  const int32_t* positions;
  float* partials;
  void* ws;
  int dim, pairs, axes, interleaved;
  int lanes, per_token, ctas;  // lanes to a row, groups of lanes to a token, CTAs to a side
  int sides;
  float eps;
  int want;  // gradients of the parameters
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The eight dimensions of lane `c`: four from d0 on and four from d1 on.
struct Place {
  int d0, d1;
  int pair;     // its first pair; pairs >= the rotation's number are not turned
  bool split;   // the two parts are halves of the same four pairs
  bool active;
};
__device__ __forceinline__ Place place_of(const Args& p, int c) {
  Place o;
  o.active = 8 * c < p.dim;
  o.split = !p.interleaved && 8 * c < 2 * p.pairs;
  o.d0 = o.split ? 4 * c : 8 * c;
  o.d1 = o.split ? 4 * c + p.pairs : 8 * c + 4;
  o.pair = 4 * c;
  return o;
}
template <bool SPLIT>
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* row, const Place& at) {
  if (!at.active) return make_uint4(0, 0, 0, 0);
  if (!SPLIT || !at.split) return load16(row + at.d0);
  const uint2 a = load8(row + at.d0), b = load8(row + at.d1);
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool SPLIT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const Place& at, const float (&v)[8]) {
  if (!at.active) return;
  const uint4 o = make_uint4(f2_to_bf16x2(v[0], v[1]), f2_to_bf16x2(v[2], v[3]), f2_to_bf16x2(v[4], v[5]), f2_to_bf16x2(v[6], v[7]));
  if (!SPLIT || !at.split) {
    *reinterpret_cast<uint4*>(row + at.d0) = o;
  } else {
    *reinterpret_cast<uint2*>(row + at.d0) = make_uint2(o.x, o.y);
    *reinterpret_cast<uint2*>(row + at.d1) = make_uint2(o.z, o.w);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load_weights(const float* w, const Place& at, float (&v)[8], float other) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w && at.active ? __ldg(w + (i < 4 ? at.d0 + i : at.d1 + i - 4)) : other;
}
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum of eight as a tree.
__device__ __forceinline__ float sum8(const float (&v)[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
// Turns the thread's four pairs forward (BACK: back).
template <bool SPLIT, bool BACK>
__device__ __forceinline__ void turn(float (&v)[8], const float2 (&cs)[4], const Place& at) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = cs[i].x, s = BACK ? -cs[i].y : cs[i].y;
    if (SPLIT && at.split) {
      const float a = v[i], b = v[i + 4];
      v[i] = a * c - b * s;
      v[i + 4] = a * s + b * c;
    } else {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * c - b * s;
      v[2 * i + 1] = a * s + b * c;
    }
  }
}
// xhat in v, returns r.
template <int NORM>
__device__ __forceinline__ float normalise(float (&v)[8], const Args& p, const Place& at, float inv) {
  if (NORM == DIT_NORM_NONE) return 1.f;
  float sq[8];
  if (NORM == DIT_NORM_LAYER) {
    const float mean = group_sum(sum8(v), p.lanes) * inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at.active ? v[i] - mean : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sq[i] = v[i] * v[i];
  const float r = 1.f / sqrtf(group_sum(sum8(sq), p.lanes) * inv + p.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= r;
  return r;
}
// cos and sin of the tokens of a CTA, one thread to a pair.
__device__ __forceinline__ void fill_angles(const Args& p, float2* cs, int64_t token0, int tokens) {
  for (int i = threadIdx.x; i < tokens * p.pairs; i += THREADS) {
    const int t = i / p.pairs, pair = i - t * p.pairs;
    float s = 0.f, c = 1.f;
    if (token0 + t < p.tokens) {
      const uint4 e = __ldg(reinterpret_cast<const uint4*>(p.table) + pair);
      const uint64_t freq = (uint64_t)e.y << 32 | e.x;
      const int64_t pos = __ldg(p.positions + (token0 + t) * p.axes + (int)e.z);
      const uint64_t turns = (uint64_t)pos * freq;                  // modulo a turn, of either sign
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);  // [-1/2, 1/2) of a turn, to 2^-25 of it
    }
    cs[i] = make_float2(c, s);
  }
}
__device__ __forceinline__ void load_angles(const Args& p, const float2* cs, int t, const Place& at, float2 (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = at.active && at.pair + i < p.pairs ? cs[t * p.pairs + at.pair + i] : make_float2(1.f, 0.f);
}

template <int NORM, bool SPLIT>
__global__ void __launch_bounds__(THREADS) k_norm_rope(Args p) {
  pdl_launch_dependents();
  __shared__ float2 cs[THREADS * 4];
  pdl_wait();
  const Side& s = p.side[blockIdx.y];
  const int groups = THREADS / p.lanes, tokens = groups / p.per_token;
  const int g = threadIdx.x / p.lanes, t = g / p.per_token, h0 = g - t * p.per_token;
  const Place at = place_of(p, threadIdx.x & (p.lanes - 1));
  const int64_t token0 = (int64_t)blockIdx.x * tokens, token = token0 + t;
  const bool live = token < p.tokens;
  const __nv_bfloat16* x = s.x.ptr + token * s.x.token;
  __nv_bfloat16* y = const_cast<__nv_bfloat16*>(s.y.ptr) + token * s.y.token;
  uint4 raw[AHEAD];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) {
    const int h = h0 + j * p.per_token;
    if (live && h < s.heads) raw[j] = load_row<SPLIT>(x + h * s.x.head, at);
  }
  fill_angles(p, cs, token0, tokens);
  __syncthreads();
  float2 a[4];
  load_angles(p, cs, t, at, a);
  float w[8], b[8];
  if (NORM != DIT_NORM_NONE) load_weights(s.w, at, w, 1.f);
  if (NORM == DIT_NORM_LAYER) load_weights(s.b, at, b, 0.f);
  const float inv = 1.f / (float)p.dim;
  // every thread makes every round: the sums' shuffles want whole warps
  for (int base = 0; base < s.heads; base += AHEAD * p.per_token) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int h = base + h0 + j * p.per_token;
      const bool mine = live && h < s.heads;
      float v[8];
      unpack(raw[j], v);
      if (mine && h + AHEAD * p.per_token < s.heads) raw[j] = load_row<SPLIT>(x + (h + AHEAD * p.per_token) * s.x.head, at);
      normalise<NORM>(v, p, at, inv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (NORM == DIT_NORM_RMS) v[i] *= w[i];
        if (NORM == DIT_NORM_LAYER) v[i] = v[i] * w[i] + b[i];
      }
      turn<SPLIT, false>(v, a, at);
      if (mine) store_row<SPLIT>(y + h * s.y.head, at, v);
    }
  }
}

// Tokens are dealt to the CTAs in turn; each thread sums its parameters' gradients over all of its rows, the CTA adds
// them up over its groups, and the CTA that finishes last over the CTAs, always in the same order.
template <int NORM, bool SPLIT>
__global__ void __launch_bounds__(THREADS) k_norm_rope_back(Args p) {
  pdl_launch_dependents();
  __shared__ float2 cs[THREADS * 4];
  __shared__ float sums[THREADS * 8];
  __shared__ bool last;
  pdl_wait();
  const Side& s = p.side[blockIdx.y];
  const int groups = THREADS / p.lanes, tokens = groups / p.per_token;
  const int g = threadIdx.x / p.lanes, t = g / p.per_token, h0 = g - t * p.per_token;
  const Place at = place_of(p, threadIdx.x & (p.lanes - 1));
  const float inv = 1.f / (float)p.dim;
  float w[8], dw[8], db[8];
  if (NORM != DIT_NORM_NONE) load_weights(s.w, at, w, 1.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
  const int64_t blocks = (p.tokens + tokens - 1) / tokens;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t token0 = blk * tokens, token = token0 + t;
    const bool live = token < p.tokens;
    const __nv_bfloat16* x = s.x.ptr + token * s.x.token;
    const __nv_bfloat16* dy = s.dy.ptr + token * s.dy.token;
    __nv_bfloat16* dx = const_cast<__nv_bfloat16*>(s.y.ptr) + token * s.y.token;
    uint4 rx[BACK_AHEAD], rd[BACK_AHEAD];
#pragma unroll
    for (int j = 0; j < BACK_AHEAD; ++j) {
      const int h = h0 + j * p.per_token;
      if (live && h < s.heads) {
        rd[j] = load_row<SPLIT>(dy + h * s.dy.head, at);
        if (NORM != DIT_NORM_NONE) rx[j] = load_row<SPLIT>(x + h * s.x.head, at);
      }
    }
    __syncthreads();  // the angles of the round before have been read
    fill_angles(p, cs, token0, tokens);
    __syncthreads();
    float2 a[4];
    load_angles(p, cs, t, at, a);
    for (int base = 0; base < s.heads; base += BACK_AHEAD * p.per_token) {
#pragma unroll
      for (int j = 0; j < BACK_AHEAD; ++j) {
        const int h = base + h0 + j * p.per_token;
        const bool mine = live && h < s.heads;
        float v[8], d[8];
        unpack(rd[j], d);
        if (NORM != DIT_NORM_NONE) unpack(rx[j], v);
        const int next = h + BACK_AHEAD * p.per_token;
        if (mine && next < s.heads) {
          rd[j] = load_row<SPLIT>(dy + next * s.dy.head, at);
          if (NORM != DIT_NORM_NONE) rx[j] = load_row<SPLIT>(x + next * s.x.head, at);
        }
        turn<SPLIT, true>(d, a, at);
        if (NORM != DIT_NORM_NONE) {
          const float r = normalise<NORM>(v, p, at, inv);
          float e[8];
          if (mine && at.active) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dw[i] += d[i] * v[i];
              if (NORM == DIT_NORM_LAYER) db[i] += d[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            d[i] = at.active ? d[i] * w[i] : 0.f;
            e[i] = d[i] * v[i];
          }
          const float me = group_sum(sum8(e), p.lanes) * inv;
          const float m = NORM == DIT_NORM_LAYER ? group_sum(sum8(d), p.lanes) * inv : 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = (d[i] - m - v[i] * me) * r;
        }
        if (mine) store_row<SPLIT>(dx + h * s.y.head, at, d);
      }
    }
  }
  if (NORM == DIT_NORM_NONE || !p.want) return;
  constexpr int ROWS = NORM == DIT_NORM_LAYER ? 2 : 1;
  const int outs = ROWS * p.dim;  // of one side
  float* mine = p.partials + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * outs;
#pragma unroll
  for (int row = 0; row < ROWS; ++row) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.active) sums[g * p.lanes * 8 + (i < 4 ? at.d0 + i : at.d1 + i - 4)] = row ? db[i] : dw[i];
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += THREADS) {
      float v = 0.f;
      for (int k = 0; k < groups; ++k) v += sums[k * p.lanes * 8 + d];
      __stcg(mine + row * p.dim + d, v);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ws_u32(p.ws, WS_TICKET), 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int o = threadIdx.x; o < p.sides * outs; o += THREADS) {
    const int side = o / outs, e = o - side * outs;
    const float* from = p.partials + (int64_t)side * gridDim.x * outs + e;
    float v[8] = {};
    for (int c = 0; c < (int)gridDim.x; c += 8)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < (int)gridDim.x) v[i] += __ldcg(from + (int64_t)(c + i) * outs);
    (e < p.dim ? p.side[side].dw : p.side[side].db)[e < p.dim ? e : e - p.dim] = sum8(v);
  }
  if (threadIdx.x == 0) *ws_u32(p.ws, WS_TICKET) = 0u;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A view's checks, with strides that are not used replaced.
static dit_status view_of(const dit_heads_t* v, int heads, int64_t tokens, int dim, View* o) {
  if (!v || (!v->ptr && tokens > 0) || v->heads != heads) return DIT_ERR_INVALID_ARG;
  *o = View{reinterpret_cast<const __nv_bfloat16*>(v->ptr), tokens > 1 ? v->token_stride : 0, heads > 1 ? v->head_stride : 0};
  if (!aligned16(v->ptr) || o->token % 8 || o->head % 8) return DIT_ERR_ALIGNMENT;
  return DIT_OK;
}

static int lanes_of(int dim) {
  int l = 1;
  while (8 * l < dim) l *= 2;
  return l;
}

static dit_status fill(Args& p, const dit_heads_t* q, const dit_heads_t* k, const dit_heads_t* dq_out, const dit_heads_t* dk_out,
                       const dit_heads_t* q_out, const dit_heads_t* k_out, int64_t tokens, int dim, int norm,
                       const float* params, double eps, const dit_rotary_t* rot, const int32_t* positions, bool back) {
  if (tokens < 0 || tokens > MAX_TOKENS || dim <= 0 || norm < DIT_NORM_NONE || norm > DIT_NORM_LAYER || !q) return DIT_ERR_INVALID_ARG;
  if (norm != DIT_NORM_NONE && (!params || !(eps >= 0.0) || !isfinite(eps))) return DIT_ERR_INVALID_ARG;
  if (dim % 8 || dim > MAX_DIM) return DIT_ERR_UNSUPPORTED;
  if (rot && (rot->pairs < 0 || 2 * (int64_t)rot->pairs > dim || rot->axes < 1 || rot->axes > DIT_MAX_AXES || (rot->pairs && (!rot->table || (!positions && tokens)))))
    return DIT_ERR_INVALID_ARG;
  if (rot && !rot->interleaved && rot->pairs % 4) return DIT_ERR_UNSUPPORTED;
  if (rot && rot->pairs && (!aligned16(rot->table) || (reinterpret_cast<uintptr_t>(positions) & 3))) return DIT_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(params) & 3) return DIT_ERR_ALIGNMENT;
  if (!k != !k_out || (back && !k != !dk_out)) return DIT_ERR_INVALID_ARG;
  const int rows = norm == DIT_NORM_LAYER ? 2 : 1;
  p.sides = k ? 2 : 1;
  for (int i = 0; i < p.sides; ++i) {
    Side& s = p.side[i];
    s.heads = (i ? k : q)->heads;
    if (s.heads < 1 || s.heads > (1 << 20)) return DIT_ERR_INVALID_ARG;
    dit_status e = view_of(i ? k : q, s.heads, tokens, dim, &s.x);
    if (e == DIT_OK) e = view_of(i ? k_out : q_out, s.heads, tokens, dim, &s.y);
    if (e == DIT_OK && back) e = view_of(i ? dk_out : dq_out, s.heads, tokens, dim, &s.dy);
    if (e != DIT_OK) return e;
    if (norm != DIT_NORM_NONE) {
      s.w = params + (int64_t)i * rows * dim;
      s.b = s.w + dim;
    }
  }
  p.tokens = tokens;
  p.dim = dim;
  p.eps = (float)eps;
  p.pairs = rot ? rot->pairs : 0;
  p.axes = rot ? rot->axes : 1;
  p.interleaved = rot ? rot->interleaved != 0 : 1;
  p.table = rot ? reinterpret_cast<const Pair*>(rot->table) : nullptr;
  p.positions = positions;
  p.lanes = lanes_of(dim);
  // About AHEAD heads to a group of lanes: the angles and weights are then read once for four rows.  Batches that
  // fill less than two CTAs an SM get more groups to a token.
  const int groups = THREADS / p.lanes;
  const int heads = p.sides == 2 && p.side[1].heads > p.side[0].heads ? p.side[1].heads : p.side[0].heads;
  p.per_token = 1;
  while (p.per_token < groups && p.per_token * AHEAD < heads) p.per_token *= 2;
  while (p.per_token < groups && p.per_token < heads && tokens * p.per_token < (int64_t)groups * 2 * num_sms()) p.per_token *= 2;
  return DIT_OK;
}

template <bool BACK, int NORM>
static cudaError_t launch(const Args& p, dim3 grid, cudaStream_t st) {
  const bool split = !p.interleaved && p.pairs;
  if (BACK) return split ? launch_pdl(k_norm_rope_back<NORM, true>, grid, dim3(THREADS), 0, st, 1, p) : launch_pdl(k_norm_rope_back<NORM, false>, grid, dim3(THREADS), 0, st, 1, p);
  return split ? launch_pdl(k_norm_rope<NORM, true>, grid, dim3(THREADS), 0, st, 1, p) : launch_pdl(k_norm_rope<NORM, false>, grid, dim3(THREADS), 0, st, 1, p);
}
template <bool BACK>
static dit_status launch(const Args& p, int norm, int64_t ctas, cudaStream_t st) {
  const dim3 grid((unsigned)ctas, (unsigned)p.sides);
  const cudaError_t e = norm == DIT_NORM_LAYER ? launch<BACK, DIT_NORM_LAYER>(p, grid, st)
                        : norm == DIT_NORM_RMS ? launch<BACK, DIT_NORM_RMS>(p, grid, st)
                                               : launch<BACK, DIT_NORM_NONE>(p, grid, st);
  return e == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

}  // namespace qk
}  // namespace dit6

using namespace dit6;

extern "C" dit_status dit_rotary_table(const int32_t* dims, int axes, double theta, const double* scale, void* table, size_t table_bytes) {
  if (!dims || !scale || !table || axes < 1 || axes > DIT_MAX_AXES || !(theta > 0.0) || !isfinite(theta)) return DIT_ERR_INVALID_ARG;
  int64_t pairs = 0;
  for (int a = 0; a < axes; ++a) {
    if (dims[a] < 0 || dims[a] % 2 || dims[a] > qk::MAX_DIM || !isfinite(scale[a])) return DIT_ERR_INVALID_ARG;
    pairs += dims[a] / 2;
  }
  if (2 * pairs > qk::MAX_DIM) return DIT_ERR_UNSUPPORTED;
  if (table_bytes < pairs * sizeof(qk::Pair)) return DIT_ERR_INVALID_ARG;
  qk::Pair* o = reinterpret_cast<qk::Pair*>(table);
  const double two_pi = 6.283185307179586476925;
  for (int a = 0; a < axes; ++a)
    for (int i = 0; i < dims[a] / 2; ++i) {
      const double turns = scale[a] * pow(theta, -2.0 * i / dims[a]) / two_pi;
      const double part = turns - floor(turns);  // whole turns a position change nothing
      *o++ = qk::Pair{part < 1.0 ? (uint64_t)ldexp(part, 64) : 0, a, 0};
    }
  return DIT_OK;
}

extern "C" size_t dit_qk_norm_scratch_bytes(int dim) {
  if (dim <= 0 || dim > qk::MAX_DIM) return 0;
  return (size_t)2 * qk::MAX_CTAS * 2 * dim * sizeof(float);
}

extern "C" dit_status dit_qk_norm_rope(const dit_heads_t* q, const dit_heads_t* k, const dit_heads_t* q_out, const dit_heads_t* k_out,
                                       int64_t tokens, int dim, int norm, const float* params, double eps,
                                       const dit_rotary_t* rot, const int32_t* positions, dit_stream_t stream) {
  qk::Args p = {};
  const dit_status e = qk::fill(p, q, k, nullptr, nullptr, q_out, k_out, tokens, dim, norm, params, eps, rot, positions, false);
  if (e != DIT_OK || tokens == 0) return e;
  const int per_cta = qk::THREADS / p.lanes / p.per_token;
  return qk::launch<false>(p, norm, (tokens + per_cta - 1) / per_cta, stream);
}

extern "C" dit_status dit_qk_norm_rope_backward(const dit_heads_t* q, const dit_heads_t* k, const dit_heads_t* dq_out,
                                                const dit_heads_t* dk_out, const dit_heads_t* dq, const dit_heads_t* dk,
                                                int64_t tokens, int dim, int norm, const float* params, double eps,
                                                const dit_rotary_t* rot, const int32_t* positions, float* dparams,
                                                void* scratch, size_t scratch_bytes, void* ws, size_t ws_bytes,
                                                dit_stream_t stream) {
  qk::Args p = {};
  const dit_status e = qk::fill(p, q, k, dq_out, dk_out, dq, dk, tokens, dim, norm, params, eps, rot, positions, true);
  if (e != DIT_OK) return e;
  if (!ws || ws_bytes < WS_BYTES) return DIT_ERR_INVALID_ARG;
  if (!aligned32(ws)) return DIT_ERR_ALIGNMENT;
  if (dparams) {
    if (norm == DIT_NORM_NONE || !scratch || scratch_bytes < dit_qk_norm_scratch_bytes(dim)) return DIT_ERR_INVALID_ARG;
    if (!qk::aligned16(scratch) || (reinterpret_cast<uintptr_t>(dparams) & 3)) return DIT_ERR_ALIGNMENT;
    const int rows = norm == DIT_NORM_LAYER ? 2 : 1;
    for (int i = 0; i < p.sides; ++i) {
      p.side[i].dw = dparams + (int64_t)i * rows * dim;
      p.side[i].db = p.side[i].dw + dim;
    }
    p.want = 1;
  }
  p.partials = reinterpret_cast<float*>(scratch);
  p.ws = ws;
  if (tokens == 0 && !p.want) return DIT_OK;
  const int per_cta = qk::THREADS / p.lanes / p.per_token;
  int64_t ctas = (tokens + per_cta - 1) / per_cta;
  if (ctas > qk::MAX_CTAS) ctas = qk::MAX_CTAS;
  if (ctas < 1) ctas = 1;  // no tokens: the parameters' gradients are zeros
  return qk::launch<true>(p, norm, ctas, stream);
}
