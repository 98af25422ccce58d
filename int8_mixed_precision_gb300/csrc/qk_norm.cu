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

constexpr int THREADS = 256, BACK_THREADS = 512;
constexpr int MAX_DIM = 256;
constexpr int AHEAD = 4, BACK_AHEAD = 2;  // rows of a thread in flight
constexpr int CTAS_PER_SM = 3;            // forward
constexpr int BACK_CTAS = 152;  // of the backward pass, most: one to an SM, divided between q and k by their heads
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
  int per_token, ctas;  // groups of lanes to a token, CTAs
};
struct Args {
  Side side[2];
  int64_t tokens;
  const Pair* table;
  const int32_t* positions;
  float* partials;
  void* ws;
  int dim, pairs, axes, interleaved;
  int lanes;  // to a row
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

// The eight dimensions of lane `c` (a lane without any neither loads nor stores, and holds zeros): four from d0 on and four from d1 on.
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
  if (!SPLIT || !at.split) return load16(row + at.d0);
  const uint2 a = load8(row + at.d0), b = load8(row + at.d1);
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool SPLIT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const Place& at, const float2 (&v)[4]) {
  const uint4 o = make_uint4(f2_to_bf16x2(v[0].x, v[0].y), f2_to_bf16x2(v[1].x, v[1].y), f2_to_bf16x2(v[2].x, v[2].y), f2_to_bf16x2(v[3].x, v[3].y));
  if (!SPLIT || !at.split) {
    *reinterpret_cast<uint4*>(row + at.d0) = o;
  } else {
    *reinterpret_cast<uint2*>(row + at.d0) = make_uint2(o.x, o.y);
    *reinterpret_cast<uint2*>(row + at.d1) = make_uint2(o.z, o.w);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float2 (&v)[4]) {
  v[0] = bf16x2_to_f2(u.x);
  v[1] = bf16x2_to_f2(u.y);
  v[2] = bf16x2_to_f2(u.z);
  v[3] = bf16x2_to_f2(u.w);
}
__device__ __forceinline__ void load_weights(const float* w, const Place& at, float2 (&v)[4], float other) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* from = w + (i < 2 ? at.d0 + 2 * i : at.d1 + 2 * i - 4);
    v[i] = at.active ? make_float2(__ldg(from), __ldg(from + 1)) : make_float2(other, other);
  }
}
// Sum over the lanes of a row; LANES 0: `lanes` of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, int lanes) {
  if (LANES) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  } else {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}
__device__ __forceinline__ float sum8(const float2 (&v)[4]) {
  const float2 s = add2(add2(v[0], v[1]), add2(v[2], v[3]));
  return s.x + s.y;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// Turns the thread's four pairs forward (BACK: back).  cs: cosines and sines of pairs 0 and 1, 2 and 3.
struct Angles {
  float2 c[2], s[2];
};
template <bool SPLIT, bool BACK>
__device__ __forceinline__ void turn(float2 (&v)[4], const Angles& a, const Place& at) {
  const float2 s[2] = {BACK ? make_float2(-a.s[0].x, -a.s[0].y) : a.s[0], BACK ? make_float2(-a.s[1].x, -a.s[1].y) : a.s[1]};
  if (SPLIT && at.split) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = v[i], y = v[i + 2];
      v[i] = fma2(make_float2(-y.x, -y.y), s[i], mul2(x, a.c[i]));
      v[i + 2] = fma2(x, s[i], mul2(y, a.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float cc = i % 2 ? a.c[i / 2].y : a.c[i / 2].x, ss = i % 2 ? s[i / 2].y : s[i / 2].x;
      const float x = v[i].x, y = v[i].y;
      v[i] = make_float2(x * cc - y * ss, x * ss + y * cc);
    }
  }
}
// xhat in v, returns r (to 2 units of fp32).
template <int NORM, int LANES>
__device__ __forceinline__ float normalise(float2 (&v)[4], const Args& p, const Place& at, float inv) {
  if (NORM == DIT_NORM_NONE) return 1.f;
  if (NORM == DIT_NORM_LAYER) {
    const float mean = row_sum<LANES>(sum8(v), p.lanes) * inv;
    const float2 m = both(at.active ? -mean : 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], m);
  }
  const float2 q = fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0]))));
  const float r = rsqrtf(row_sum<LANES>(q.x + q.y, p.lanes) * inv + p.eps);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(r));
  return r;
}
// cos and sin of the tokens of a CTA, one thread to a pair.
template <int THREADS>
__device__ __forceinline__ void fill_angles(const Args& p, float2* cs, int64_t token0, int tokens) {
  for (int i = threadIdx.x; i < tokens * p.pairs; i += THREADS) {
    const int t = i / p.pairs, pair = i - t * p.pairs;
    float s = 0.f, c = 1.f;
    if (token0 + t < p.tokens) {
      const uint4 e = __ldg(reinterpret_cast<const uint4*>(p.table) + pair);
      const uint64_t freq = (uint64_t)e.y << 32 | e.x;
      if (e.z < (uint32_t)p.axes) {  // an axis that the positions do not have turns nothing
        const int64_t pos = __ldg(p.positions + (token0 + t) * p.axes + (int)e.z);
        const uint64_t turns = (uint64_t)pos * freq;                  // modulo a turn, of either sign
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);  // [-1/2, 1/2) of a turn, to 2^-25 of it
      }
    }
    cs[i] = make_float2(c, s);
  }
}
__device__ __forceinline__ Angles load_angles(const Args& p, const float2* cs, int t, const Place& at) {
  float2 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = at.active && at.pair + i < p.pairs ? cs[t * p.pairs + at.pair + i] : make_float2(1.f, 0.f);
  return Angles{{make_float2(o[0].x, o[1].x), make_float2(o[2].x, o[3].x)}, {make_float2(o[0].y, o[1].y), make_float2(o[2].y, o[3].y)}};
}

// CTAs are persistent and take every ctas-th block of tokens; a thread's next rows are always on their way, into the next block, and
// the angles of that block are made during the present one.  104,746 tokens of 30 + 30 heads of 64: 308 us with the RMS norm, 5.2
// TB/s.  17,776 tokens with the layer norm: 65 us, 4.2 TB/s; neither memory (40 % of the DRAM's) nor the issue slots (62 %, some 190
// instructions to eight dimensions of a row) are full there: six warps to a scheduler wait for fixed latencies, the blocks' barrier and
// memory in about equal parts.
template <int NORM, bool SPLIT, int LANES>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) k_norm_rope(const __grid_constant__ Args p) {
  pdl_launch_dependents();
  __shared__ float2 cs[2][THREADS * 4];
  pdl_wait();
  const int which = (int)blockIdx.x >= p.side[0].ctas, cta = blockIdx.x - (which ? p.side[0].ctas : 0);
  const Side& s = p.side[which];
  const int lanes = LANES ? LANES : p.lanes;
  const int groups = THREADS / lanes, tokens = groups / s.per_token;
  const int g = threadIdx.x / lanes, t = g / s.per_token, h0 = g - t * s.per_token;
  const Place at = place_of(p, threadIdx.x & (lanes - 1));
  const int rounds = (s.heads + AHEAD * s.per_token - 1) / (AHEAD * s.per_token);  // of AHEAD rows of a thread
  const int64_t stride = (int64_t)s.ctas * tokens, first = (int64_t)cta * tokens;
  const int64_t x_step = s.per_token * s.x.head, y_step = s.per_token * s.y.head;
  int64_t token = first + t;  // whose rows are asked for
  const __nv_bfloat16* x = s.x.ptr + token * s.x.token + h0 * s.x.head;
  int ask_h = h0;
  bool ask_live = at.active && token < p.tokens;
  uint4 raw[AHEAD] = {};
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) {
    if (ask_live && ask_h < s.heads) raw[j] = load_row<SPLIT>(x, at);
    x += x_step;
    ask_h += s.per_token;
  }
  fill_angles<THREADS>(p, cs[0], first, tokens);
  const float inv = 1.f / (float)p.dim;
  float2 w[4], b[4];
  if (NORM != DIT_NORM_NONE) load_weights(s.w, at, w, 1.f);
  if (NORM == DIT_NORM_LAYER) load_weights(s.b, at, b, 0.f);
  // every thread makes every round: the sums' shuffles want whole warps, the barrier whole CTAs
  int buf = 0;
#pragma unroll 1
  for (int64_t block = first; block < p.tokens; block += stride, buf ^= 1) {
    __syncthreads();  // this block's angles are there, and those of the block before have been read
    const Angles a = load_angles(p, cs[buf], t, at);
    fill_angles<THREADS>(p, cs[buf ^ 1], block + stride, tokens);
    __nv_bfloat16* y = const_cast<__nv_bfloat16*>(s.y.ptr) + (block + t) * s.y.token + h0 * s.y.head;
    const int heads = at.active && block + t < p.tokens ? s.heads : 0;
    int h = h0;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      if (round + 1 == rounds) {  // from here on the next block's rows are asked for
        token += stride;
        ask_live = at.active && token < p.tokens;
        ask_h = h0;
        x = s.x.ptr + token * s.x.token + h0 * s.x.head;
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        float2 v[4];
        unpack(raw[j], v);
        if (ask_live && ask_h < s.heads) raw[j] = load_row<SPLIT>(x, at);
        x += x_step;
        ask_h += s.per_token;
        normalise<NORM, LANES>(v, p, at, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (NORM == DIT_NORM_RMS) v[i] = mul2(v[i], w[i]);
          if (NORM == DIT_NORM_LAYER) v[i] = fma2(v[i], w[i], b[i]);
        }
        turn<SPLIT, false>(v, a, at);
        if (h < heads) store_row<SPLIT>(y, at, v);
        y += y_step;
        h += s.per_token;
      }
    }
  }
}

// Each thread sums its parameters' gradients over all of its rows, the CTA adds them up over its groups, and the CTA that finishes
// last over the CTAs, always in the same order.  One CTA of 512 threads to an SM makes few rows for that last sum; with 608 it took 27 us.
// 17,776 tokens of 30 + 30 heads of 64, layer norm: 109 us, 3.8 TB/s, 42 % of the issue slots and 40 % of the DRAM's.  It is bound by
// latency: with four warps to a scheduler and two rows of a thread on their way a warp waits 2.2 of some 8 cycles between its
// instructions for memory and 1.4 at the blocks' barriers.
template <int NORM, bool SPLIT, int LANES>
__global__ void __launch_bounds__(BACK_THREADS, 1) k_norm_rope_back(const __grid_constant__ Args p) {
  pdl_launch_dependents();
  __shared__ float2 cs[2][BACK_THREADS * 4];
  __shared__ bool last;
  float* sums = reinterpret_cast<float*>(&cs[0][0]);  // once the angles are done with
  pdl_wait();
  const int which = (int)blockIdx.x >= p.side[0].ctas, cta = blockIdx.x - (which ? p.side[0].ctas : 0);
  const Side& s = p.side[which];
  const int lanes = LANES ? LANES : p.lanes;
  const int groups = BACK_THREADS / lanes, tokens = groups / s.per_token;
  const int g = threadIdx.x / lanes, t = g / s.per_token, h0 = g - t * s.per_token;
  const Place at = place_of(p, threadIdx.x & (lanes - 1));
  const int rounds = (s.heads + BACK_AHEAD * s.per_token - 1) / (BACK_AHEAD * s.per_token);  // of BACK_AHEAD rows of a thread
  const int64_t stride = (int64_t)s.ctas * tokens, first = (int64_t)cta * tokens;
  const int64_t x_step = s.per_token * s.x.head, y_step = s.per_token * s.y.head, d_step = s.per_token * s.dy.head;
  int64_t token = first + t;  // whose rows are asked for
  const __nv_bfloat16* x = s.x.ptr + token * s.x.token + h0 * s.x.head;
  const __nv_bfloat16* dy = s.dy.ptr + token * s.dy.token + h0 * s.dy.head;
  int ask_h = h0;
  bool ask_live = at.active && token < p.tokens;
  uint4 rx[BACK_AHEAD] = {}, rd[BACK_AHEAD] = {};
#pragma unroll
  for (int j = 0; j < BACK_AHEAD; ++j) {
    if (ask_live && ask_h < s.heads) {
      rd[j] = load_row<SPLIT>(dy, at);
      if (NORM != DIT_NORM_NONE) rx[j] = load_row<SPLIT>(x, at);
    }
    x += x_step;
    dy += d_step;
    ask_h += s.per_token;
  }
  fill_angles<BACK_THREADS>(p, cs[0], first, tokens);
  const float inv = 1.f / (float)p.dim;
  float2 w[4], dw[4], db[4];
  if (NORM != DIT_NORM_NONE) load_weights(s.w, at, w, 1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = db[i] = make_float2(0.f, 0.f);
  // every thread makes every round: the sums' shuffles want whole warps, the barrier whole CTAs
  int buf = 0;
#pragma unroll 1
  for (int64_t block = first; block < p.tokens; block += stride, buf ^= 1) {
    __syncthreads();  // this block's angles are there, and those of the block before have been read
    const Angles a = load_angles(p, cs[buf], t, at);
    fill_angles<BACK_THREADS>(p, cs[buf ^ 1], block + stride, tokens);
    __nv_bfloat16* y = const_cast<__nv_bfloat16*>(s.y.ptr) + (block + t) * s.y.token + h0 * s.y.head;
    const int heads = at.active && block + t < p.tokens ? s.heads : 0;
    int h = h0;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      if (round + 1 == rounds) {  // from here on the next block's rows are asked for
        token += stride;
        ask_live = at.active && token < p.tokens;
        ask_h = h0;
        x = s.x.ptr + token * s.x.token + h0 * s.x.head;
        dy = s.dy.ptr + token * s.dy.token + h0 * s.dy.head;
      }
#pragma unroll
      for (int j = 0; j < BACK_AHEAD; ++j) {
        float2 v[4], d[4];
        unpack(rd[j], d);
        if (NORM != DIT_NORM_NONE) unpack(rx[j], v);
        if (ask_live && ask_h < s.heads) {
          rd[j] = load_row<SPLIT>(dy, at);
          if (NORM != DIT_NORM_NONE) rx[j] = load_row<SPLIT>(x, at);
        }
        x += x_step;
        dy += d_step;
        ask_h += s.per_token;
        turn<SPLIT, true>(d, a, at);
        if (NORM != DIT_NORM_NONE) {
          const float r = normalise<NORM, LANES>(v, p, at, inv);
          float2 e[4];
          if (h < heads) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dw[i] = fma2(d[i], v[i], dw[i]);
              if (NORM == DIT_NORM_LAYER) db[i] = add2(db[i], d[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            d[i] = mul2(d[i], w[i]);
            e[i] = mul2(d[i], v[i]);
          }
          const float me = -row_sum<LANES>(sum8(e), p.lanes) * inv;
          const float m = NORM == DIT_NORM_LAYER ? -row_sum<LANES>(sum8(d), p.lanes) * inv : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (NORM == DIT_NORM_LAYER) d[i] = add2(d[i], both(m));
            d[i] = mul2(fma2(v[i], both(me), d[i]), both(r));
          }
        }
        if (h < heads) store_row<SPLIT>(y, at, d);
        y += y_step;
        h += s.per_token;
      }
    }
  }
  if (NORM == DIT_NORM_NONE || !p.want) return;
  constexpr int ROWS = NORM == DIT_NORM_LAYER ? 2 : 1;
  const int outs = ROWS * p.dim;  // of one side
  float* mine = p.partials + (int64_t)blockIdx.x * outs;
#pragma unroll
  for (int row = 0; row < ROWS; ++row) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.active) {
        const float2 v = row ? db[i / 2] : dw[i / 2];
        sums[g * lanes * 8 + (i < 4 ? at.d0 + i : at.d1 + i - 4)] = i % 2 ? v.y : v.x;
      }
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += BACK_THREADS) {
      float v = 0.f;
      for (int k = 0; k < groups; ++k) v += sums[k * lanes * 8 + d];
      __stcg(mine + row * p.dim + d, v);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ws_u32(p.ws, WS_TICKET), 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int o = threadIdx.x; o < p.sides * outs; o += BACK_THREADS) {
    const int side = o / outs, e = o - side * outs, many = p.side[side].ctas;
    const float* from = p.partials + (int64_t)(side ? p.side[0].ctas : 0) * outs + e;
    float v[16] = {};
    for (int c = 0; c < many; c += 16)  // sixteen loads in flight
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < many) v[i] += __ldcg(from + (int64_t)(c + i) * outs);
#pragma unroll
    for (int w = 8; w > 0; w >>= 1)
#pragma unroll
      for (int i = 0; i < w; ++i) v[i] += v[i + w];
    (e < p.dim ? p.side[side].dw : p.side[side].db)[e < p.dim ? e : e - p.dim] = v[0];
  }
  if (threadIdx.x == 0) *ws_u32(p.ws, WS_TICKET) = 0u;
}

// A number as the sum of two doubles, 106 bits (Dekker, 1971; Knuth): what a rotation's frequencies are made in.  A frequency's
// fraction of a turn is wanted to 2^-64, and plain doubles leave 2^-53 of the whole frequency.
struct Wide {
  double hi, lo;
};
static Wide sum_of(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
static Wide product_of(Wide a, Wide b) {
  const double p = a.hi * b.hi;
  return sum_of(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
// theta^(-1/m): a step of Newton's method on theta x^m = 1 doubles the bits that a double has, a second one is for m's sake.  Products
// with the smallest thetas are made 2^300 times as large, so that their low parts are held.
static Wide root_of(double theta, int m) {
  const int up = theta < 0x1p-600 ? 300 : 0;
  Wide x = {pow(theta, -1.0 / m), 0.0};
  for (int step = 0; step < 2; ++step) {
    Wide t = {ldexp(theta, up), 0.0};
    for (int i = 0; i < m; ++i) t = product_of(t, x);
    x = sum_of(x.hi, x.lo - x.hi * ((ldexp(t.hi, -up) - 1.0) + ldexp(t.lo, -up)) / m);
  }
  return x;
}
// The fraction of a number of turns, times 2^64.
static uint64_t fraction_of(Wide turns) {
  const double a = ldexp(turns.hi - nearbyint(turns.hi), 64), b = ldexp(turns.lo - nearbyint(turns.lo), 64), whole = floor(a);
  return (uint64_t)((__int128)whole + (__int128)nearbyint((a - whole) + b));
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
    if (e == DIT_OK && !heads_apart(tokens, s.heads, dim, s.y.token, s.y.head)) e = DIT_ERR_INVALID_ARG;
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
  // CTAs for q and for k in the proportion of their heads, no more than there are blocks of tokens.  About AHEAD heads go to a group
  // of lanes: the angles and weights are then read once for four rows.  Batches that leave CTAs without a block get more
  // groups to a token.
  const int groups = (back ? BACK_THREADS : THREADS) / p.lanes;
  const int64_t most = back ? BACK_CTAS : (int64_t)CTAS_PER_SM * num_sms();
  for (int i = 0; i < p.sides; ++i) {
    Side& s = p.side[i];
    int64_t n = most;
    if (p.sides == 2) {
      const int64_t q = most * p.side[0].heads / ((int64_t)p.side[0].heads + p.side[1].heads);
      n = q < 1 ? 1 : q > most - 1 ? most - 1 : q;
      if (i) n = most - n;
    }
    s.per_token = 1;
    while (s.per_token < groups && s.per_token * AHEAD < s.heads) s.per_token *= 2;
    while (s.per_token < groups && s.per_token < s.heads && tokens * s.per_token < groups * n) s.per_token *= 2;
    const int64_t blocks = (tokens * s.per_token + groups - 1) / groups;
    s.ctas = (int)(blocks < 1 ? 1 : blocks < n ? blocks : n);
  }
  return DIT_OK;
}

// Heads of 40 to 64 and of 72 to 128 dimensions have kernels of their own, whose sums over a row's lanes are unrolled.
template <bool BACK, int NORM, bool SPLIT>
static cudaError_t launch(const Args& p, dim3 grid, cudaStream_t st) {
  auto go = [&](auto* kernel) { return launch_pdl(kernel, grid, dim3(BACK ? BACK_THREADS : THREADS), 0, st, 1, p); };
  if (BACK) return p.lanes == 8 ? go(k_norm_rope_back<NORM, SPLIT, 8>) : p.lanes == 16 ? go(k_norm_rope_back<NORM, SPLIT, 16>) : go(k_norm_rope_back<NORM, SPLIT, 0>);
  return p.lanes == 8 ? go(k_norm_rope<NORM, SPLIT, 8>) : p.lanes == 16 ? go(k_norm_rope<NORM, SPLIT, 16>) : go(k_norm_rope<NORM, SPLIT, 0>);
}
template <bool BACK, int NORM>
static cudaError_t launch(const Args& p, dim3 grid, cudaStream_t st) {
  return !p.interleaved && p.pairs ? launch<BACK, NORM, true>(p, grid, st) : launch<BACK, NORM, false>(p, grid, st);
}
template <bool BACK>
static dit_status launch(const Args& p, int norm, cudaStream_t st) {
  const dim3 grid((unsigned)(p.side[0].ctas + (p.sides == 2 ? p.side[1].ctas : 0)));
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
  const qk::Wide turns_a_radian = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
  for (int a = 0; a < axes; ++a) {
    const int m = dims[a] / 2;
    const qk::Wide root = m ? qk::root_of(theta, m) : qk::Wide{};
    qk::Wide turns = qk::product_of(turns_a_radian, {scale[a], 0.0});
    for (int i = 0; i < m; ++i, turns = qk::product_of(turns, root)) {
      if (!isfinite(turns.hi) || !isfinite(turns.lo)) return DIT_ERR_INVALID_ARG;
      *o++ = qk::Pair{qk::fraction_of(turns), a, 0};
    }
  }
  return DIT_OK;
}

extern "C" size_t dit_qk_norm_scratch_bytes(int dim) {
  if (dim <= 0 || dim > qk::MAX_DIM) return 0;
  return (size_t)qk::BACK_CTAS * 2 * dim * sizeof(float);
}

extern "C" dit_status dit_qk_norm_rope(const dit_heads_t* q, const dit_heads_t* k, const dit_heads_t* q_out, const dit_heads_t* k_out,
                                       int64_t tokens, int dim, int norm, const float* params, double eps,
                                       const dit_rotary_t* rot, const int32_t* positions, dit_stream_t stream) {
  qk::Args p = {};
  const dit_status e = qk::fill(p, q, k, nullptr, nullptr, q_out, k_out, tokens, dim, norm, params, eps, rot, positions, false);
  if (e != DIT_OK || tokens == 0) return e;
  return qk::launch<false>(p, norm, stream);
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
    const size_t sums = dit_qk_norm_scratch_bytes(dim), all = sizeof(float) * p.sides * rows * dim;
    if (!bytes_apart(scratch, sums, dparams, all) || !bytes_apart(scratch, sums, params, all) || !bytes_apart(scratch, sums, ws, WS_BYTES) ||
        !bytes_apart(dparams, all, ws, WS_BYTES) || (p.pairs && !bytes_apart(scratch, sums, positions, sizeof(int32_t) * tokens * p.axes)))
      return DIT_ERR_INVALID_ARG;
    for (int i = 0; i < p.sides; ++i) {
      p.side[i].dw = dparams + (int64_t)i * rows * dim;
      p.side[i].db = p.side[i].dw + dim;
    }
    p.want = 1;
  }
  p.partials = reinterpret_cast<float*>(scratch);
  p.ws = ws;
  if (tokens == 0 && !p.want) return DIT_OK;
  return qk::launch<true>(p, norm, stream);  // without tokens a CTA of each side still writes the parameters' gradients, zeros
}
