// Grouped-query attention in which each query sees an interval of its sequence's keys, with capped
// scores and a bias that falls with the distance, forward and backward, on the tcgen05 tensor cores:
//   t_ij = cap tanh(scale q_i k_j / cap) (or scale q_i k_j) - slope_h |i - j|,  lo_i <= j < hi_i;
//   P = softmax_j(t), o_i = sum_j P_ij v_j, lse_i = log sum_j e^(t_ij); a row that sees nothing: o = 0, lse = -inf.
//   Backward with dP = do v, D_i = sum_j P_ij dP_ij: dS = P (dP - D) (1 - tanh^2), dq = scale dS k, dk = scale dS^T q,
//   dv = P^T do.
// Intervals say causal, packed documents, prefixes, windows and padding alike, and their extremes over
// 128-row tiles say which tiles of keys a tile of queries needs at all and which need no mask. That is the plan
// (attention_plan): made once for a batch and read by every layer's forward and backward.
#include <cuda_bf16.h>
#include <type_traits>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "sl_attn.cuh"
#include "sl_packed.h"

namespace sl {

namespace {

// Every wait is for one phase of a barrier by its parity, so no barrier may complete a phase before everyone who waits for
// the last one has passed: each producer below is held back by an answer of its consumers, or has a second barrier
// to alternate with.
constexpr int kFwdThreads = 384;  // warp 0 TMA, warps 1 and 2 MMA (warp 1 allocates TMEM), warps 4..11 softmax
constexpr int kBwdThreads = 640;  // dq: warp 0 loads, warps 1, 2 and 3 MMA, warps 4..19 compute
// dk, dv: warp 0 loads, warps 1, 2 and 3 MMA, the others compute
template <bool CAP>
constexpr int kDkvThreads = CAP ? 384 : 640;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------------------------------- plan

constexpr int kPlanHeader = 16;          // int32 words
constexpr int32_t kPlanMagic = 0x534c504c;

struct Plan {
  const int32_t* header;   // magic, n_seq, S
  const int32_t *lo, *hi;  // [T], within [0, S]; a row that sees nothing has lo = hi = 0
  // [n_seq * n_t], n_t = ceil(S / 128). q_range: key tiles [x, y) that any row of the query tile sees (never
  // empty: [0, 1) when none does), and [z, w) that all of its rows see whole; k_range: query tiles [x, y) that
  // see any of the key tile (never empty)
  const int4* q_range;
  const int2* k_range;
  const int2* q2_range;  // key tiles of query tiles 2 i and 2 i + 1 together (sequence * ceil(n_t / 2) + i)
  // {tile or pair, range x, range y, 0}, the longest ranges first
  const int4 *q_order, *k_order, *q2_order;
};

int64_t plan_tiles(int n_seq, int S) { return (int64_t)n_seq * ((S + kTile - 1) / kTile); }

// Carves a plan out of a buffer (16-byte aligned) and returns its bytes.
int64_t carve_plan(void* buf, int n_seq, int S, Plan* out) {
  const int64_t T = (int64_t)n_seq * S, nt = plan_tiles(n_seq, S);
  uint8_t* b = static_cast<uint8_t*>(buf);
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = b ? b + off : nullptr;
    off += (bytes + 15) & ~int64_t(15);
    return p;
  };
  Plan p;
  p.header = reinterpret_cast<int32_t*>(take(kPlanHeader * 4));
  p.lo = reinterpret_cast<int32_t*>(take(T * 4));
  p.hi = reinterpret_cast<int32_t*>(take(T * 4));
  p.q_range = reinterpret_cast<int4*>(take(nt * 16));
  p.k_range = reinterpret_cast<int2*>(take(nt * 8));
  p.q_order = reinterpret_cast<int4*>(take(nt * 16));
  p.k_order = reinterpret_cast<int4*>(take(nt * 16));
  const int64_t n2 = (int64_t)n_seq * (((S + kTile - 1) / kTile + 1) / 2);
  p.q2_range = reinterpret_cast<int2*>(take(n2 * 8));
  p.q2_order = reinterpret_cast<int4*>(take(n2 * 16));
  if (out) *out = p;
  return off;
}

// Whether the buffer holds a plan of these sizes (else the error word is set and nothing is computed).
__device__ __forceinline__ bool plan_fits(const Plan& p, int n_seq, int S, int* err) {
  const int4 h = *reinterpret_cast<const int4*>(p.header);
  const bool ok = h.x == kPlanMagic && h.y == n_seq && h.z == S;
  if (!ok && threadIdx.x == 0 && blockIdx.x == 0) record_error(err, DEV_BAD_PLAN);
  return ok;
}

constexpr int kPlanThreads = 1024;

// Rows of the tiles (sequence * n_t + tile) first, first + step, ...: a warp per tile.
__device__ void plan_rows(const Plan& p, const int32_t* row_lo, const int32_t* row_hi, int n_seq, int S, int64_t first,
                          int64_t step, int4* q_range) {
  const int n_t = (S + kTile - 1) / kTile, lane = threadIdx.x & 31;
  int32_t *lo = const_cast<int32_t*>(p.lo), *hi = const_cast<int32_t*>(p.hi);
  for (int64_t at = first; at < (int64_t)n_seq * n_t; at += step) {
    const int t = (int)(at % n_t);
    const int64_t b = at / n_t;
    int l_min = S, l_max = 0, h_min = S, h_max = 0;
    bool any_empty = false;
    for (int r = lane; r < kTile; r += 32) {
      const int q = t * kTile + r;
      if (q >= S) continue;
      const int64_t row = b * S + q;
      int l = max(0, row_lo ? row_lo[row] : 0), h = min(S, row_hi ? row_hi[row] : q + 1);
      if (l >= h) {
        l = h = 0;
        any_empty = true;
      } else {
        l_min = min(l_min, l);
        l_max = max(l_max, l);
        h_min = min(h_min, h);
        h_max = max(h_max, h);
      }
      lo[row] = l;
      hi[row] = h;
    }
    l_min = __reduce_min_sync(0xffffffffu, l_min);
    l_max = __reduce_max_sync(0xffffffffu, l_max);
    h_min = __reduce_min_sync(0xffffffffu, h_min);
    h_max = __reduce_max_sync(0xffffffffu, h_max);
    any_empty = __any_sync(0xffffffffu, any_empty);
    if (lane == 0) {
      int4 v = h_max == 0 ? make_int4(0, 1, 0, 0)
                          : make_int4(l_min / kTile, (h_max + kTile - 1) / kTile, (l_max + kTile - 1) / kTile, h_min / kTile);
      if (any_empty) v.z = v.w = 0;
      q_range[at] = v;
    }
  }
}

// Tiles by the lengths of their ranges, the longest first (equal ones in no set order: the order only
// says when a unit starts). hist: n_t + 2 counters.
template <typename R>
__device__ void plan_order(const R* range, int64_t n, int n_t, int4* order, int32_t* hist, int32_t* carry) {
  for (int i = threadIdx.x; i < n_t + 2; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t at = threadIdx.x; at < n; at += kPlanThreads) atomicAdd(&hist[n_t - (range[at].y - range[at].x)], 1);
  __syncthreads();
  // exclusive sums, 1024 counters at a time
  if (threadIdx.x == 0) *carry = 0;
  __syncthreads();
  __shared__ int32_t warp_sum[32];
  for (int base = 0; base < n_t + 2; base += kPlanThreads) {
    const int i = base + threadIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int v = i < n_t + 2 ? hist[i] : 0;
    int inc = v;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sum[w] = inc;
    __syncthreads();
    int before = *carry;
    for (int k = 0; k < w; ++k) before += warp_sum[k];
    if (i < n_t + 2) hist[i] = before + inc - v;
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) *carry = before + inc;
    __syncthreads();
  }
  for (int64_t at = threadIdx.x; at < n; at += kPlanThreads) {
    const R v = range[at];
    order[atomicAdd(&hist[n_t - (v.y - v.x)], 1)] = make_int4((int)at, v.x, v.y, 0);
  }
  __syncthreads();
}

// Key tiles' ranges from the query tiles', and both orders. One block, and two atomics per pair of a query tile and a key
// tile that it sees: with the rows' kernel 17 us for one causal sequence of 16512 tokens, 76 for 65536, 262 for 131072,
// 15.7 ms for 2^20 (once per batch, beside attention that grows the same way).
__device__ void plan_tiles_and_order(const Plan& p, int n_seq, int S, int32_t* hist, int32_t* carry) {
  const int n_t = (S + kTile - 1) / kTile;
  const int64_t n = (int64_t)n_seq * n_t;
  int2* kr = const_cast<int2*>(p.k_range);
  for (int64_t at = threadIdx.x; at < n; at += kPlanThreads) kr[at] = make_int2(n_t, 0);
  __syncthreads();
  for (int64_t at = threadIdx.x; at < n; at += kPlanThreads) {
    const int4 v = p.q_range[at];
    const int t = (int)(at % n_t);
    const int64_t seq0 = at - t;
    for (int j = v.x; j < v.y; ++j) {
      atomicMin(&kr[seq0 + j].x, t);
      atomicMax(&kr[seq0 + j].y, t + 1);
    }
  }
  __syncthreads();
  for (int64_t at = threadIdx.x; at < n; at += kPlanThreads)
    if (kr[at].y == 0) kr[at] = make_int2(0, 1);
  const int n_t2 = (n_t + 1) / 2;
  const int64_t n2 = (int64_t)n_seq * n_t2;
  for (int64_t at = threadIdx.x; at < n2; at += kPlanThreads) {
    const int i = (int)(at % n_t2);
    const int4 a = p.q_range[at / n_t2 * n_t + 2 * i];
    int2 v = make_int2(a.x, a.y);
    if (2 * i + 1 < n_t) {
      const int4 c = p.q_range[at / n_t2 * n_t + 2 * i + 1];
      v = make_int2(min(v.x, c.x), max(v.y, c.y));
    }
    const_cast<int2*>(p.q2_range)[at] = v;
  }
  __syncthreads();
  plan_order(p.q2_range, n2, n_t, const_cast<int4*>(p.q2_order), hist, carry);
  plan_order(p.q_range, n, n_t, const_cast<int4*>(p.q_order), hist, carry);
  plan_order(p.k_range, n, n_t, const_cast<int4*>(p.k_order), hist, carry);
  if (threadIdx.x < 3) const_cast<int32_t*>(p.header)[threadIdx.x] = threadIdx.x == 0 ? kPlanMagic : threadIdx.x == 1 ? n_seq : S;
}

__global__ void __launch_bounds__(kPlanThreads) plan_rows_kernel(Plan p, const int32_t* lo, const int32_t* hi, int n_seq, int S) {
  pdl_wait();
  const int64_t warp = ((int64_t)blockIdx.x * kPlanThreads + threadIdx.x) >> 5;
  plan_rows(p, lo, hi, n_seq, S, warp, (int64_t)gridDim.x * (kPlanThreads / 32), const_cast<int4*>(p.q_range));
}

__global__ void __launch_bounds__(kPlanThreads) plan_tiles_kernel(Plan p, int n_seq, int S) {
  extern __shared__ int32_t hist[];
  __shared__ int32_t carry;
  pdl_wait();
  plan_tiles_and_order(p, n_seq, S, hist, &carry);
}

// A plan of at most kPlanSmall tiles in one block and one launch: ranges in shared memory, and each tile's place by
// counting the longer ones (equal ones stand by their number).
constexpr int kPlanSmall = 128;
__global__ void __launch_bounds__(kPlanThreads) plan_small_kernel(Plan p, const int32_t* lo, const int32_t* hi, int n_seq, int S) {
  __shared__ int4 q[kPlanSmall];
  __shared__ int2 k[kPlanSmall], q2[kPlanSmall];
  pdl_wait();
  const int n_t = (S + kTile - 1) / kTile, n = n_seq * n_t, n_t2 = (n_t + 1) / 2, n2 = n_seq * n_t2, at = threadIdx.x;
  if (at < n) k[at] = make_int2(n_t, 0);
  plan_rows(p, lo, hi, n_seq, S, threadIdx.x >> 5, kPlanThreads / 32, q);
  __syncthreads();
  if (at < n) {
    const int t = at % n_t, seq0 = at - t;
    for (int j = q[at].x; j < q[at].y; ++j) {
      atomicMin(&k[seq0 + j].x, t);
      atomicMax(&k[seq0 + j].y, t + 1);
    }
  } else if (at >= kPlanSmall && at - kPlanSmall < n2) {
    const int i = at - kPlanSmall, a = i / n_t2 * n_t + i % n_t2 * 2;
    int2 v = make_int2(q[a].x, q[a].y);
    if (i % n_t2 * 2 + 1 < n_t) v = make_int2(min(v.x, q[a + 1].x), max(v.y, q[a + 1].y));
    q2[i] = v;
  }
  __syncthreads();
  if (at < n && k[at].y == 0) k[at] = make_int2(0, 1);
  __syncthreads();
  auto place = [&](int me, int count, auto range_of, int4* order) {
    const int2 r = range_of(me);
    const int len = r.y - r.x;
    int rank = 0;
    for (int j = 0; j < count; ++j) {
      const int2 o = range_of(j);
      rank += o.y - o.x > len || (o.y - o.x == len && j < me);
    }
    order[rank] = make_int4(me, r.x, r.y, 0);
  };
  const int which = at / kPlanSmall, me = at % kPlanSmall;
  if (which == 0 && me < n) place(me, n, [&](int j) { return make_int2(q[j].x, q[j].y); }, const_cast<int4*>(p.q_order));
  if (which == 1 && me < n) place(me, n, [&](int j) { return k[j]; }, const_cast<int4*>(p.k_order));
  if (which == 2 && me < n2) place(me, n2, [&](int j) { return q2[j]; }, const_cast<int4*>(p.q2_order));
  if (which == 3 && me < n) {
    const_cast<int4*>(p.q_range)[me] = q[me];
    const_cast<int2*>(p.k_range)[me] = k[me];
    if (me < n2) const_cast<int2*>(p.q2_range)[me] = q2[me];
  }
  if (at < 3) const_cast<int32_t*>(p.header)[at] = at == 0 ? kPlanMagic : at == 1 ? n_seq : S;
}

// ----------------------------------------------------------------------------------------- scores

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in a 64-bit register: multiply-adds, sums and products of both in one instruction, which halves
// the issue slots of the element-wise work (each element counts: a tile has 128 per thread and only two warps share a
// scheduler).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pk(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2 pku(uint32_t a, uint32_t b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ f2 both(float a) { return pk(a, a); }
__device__ __forceinline__ void un(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ void unu(f2 v, uint32_t& a, uint32_t& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Maxima that are NaN where one of the values is
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 2^x of two values on the multiply-add units: x = n + f with a whole n and |f| <= 1/2, 2^f a polynomial of degree 5 (least
// maximum of the relative error with the constant 1: 1.1e-7, 1.7e-7 with fp32 arithmetic, about ex2.approx's), n added
// to its exponent. From -127 down: 0 (the exponent of 1 less 127 leaves no bit). 1.5 * 2^23 + x keeps n in its low
// bits. NaN gives some number: the row's maximum keeps it. A quarter of the forward's exponentials, which otherwise wait for the exponential unit (8192 tokens with a bias 537 against 576 us, 4096 causal 131 against 135;
// an eighth 555, three eighths 543, half 585); with a cap, whose tanh is on the same units, and in the backward it gains nothing.
__device__ __forceinline__ void ex2_poly(f2 x, float& y0, float& y1) {
  float x0, x1;
  un(x, x0, x1);
  x = pk(fmaxf(x0, -127.f), fmaxf(x1, -127.f));
  const f2 t = add2(x, both(12582912.f)), f = fma2(add2(t, both(-12582912.f)), both(-1.f), x);
  f2 r = fma2(f, both(0.0013264727f), both(0.009671513f));
  r = fma2(f, r, both(0.055507336f));
  r = fma2(f, r, both(0.24022242f));
  r = fma2(f, r, both(0.693147f));
  r = fma2(f, r, both(1.f));
  uint32_t n0, n1, r0, r1;
  unu(t, n0, n1);
  unu(r, r0, r1);
  y0 = __uint_as_float(r0 + (n0 << 23));
  y1 = __uint_as_float(r1 + (n1 << 23));
}
// tanh of N raw products times mul (= scale / cap), in place. Up to 0.75 an odd polynomial (a least-maximum
// fit of tanh(u) / u in u^2, relative error 6.5e-8, 1.6e-7 with fp32 arithmetic): 7 multiply-adds, and small
// scores keep their relative exactness. Above, for the whole warp: 1 - 2 / (2^(2 log2(e) u) + 1), error
// about 1e-7 of 1 (2^x = inf gives 1, 0 gives -1), on the exponential unit, which the softmax needs too.
// tanh.approx would be off by 5e-4 of the value.
template <int N>
__device__ __forceinline__ void tanh_n(uint32_t (&v)[N], float mul) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N; e += 2) top = fmaxf(fmaxf(top, fabsf(__uint_as_float(v[e]))), fabsf(__uint_as_float(v[e + 1])));
  if (__any_sync(0xffffffffu, !(top * mul <= 0.75f))) {
    const float mul2x = mul * (2.f * kLog2e);
#pragma unroll
    for (int e = 0; e < N; ++e)
      v[e] = __float_as_uint(fmaf(-2.f, rcp(ex2(__uint_as_float(v[e]) * mul2x) + 1.f), 1.f));
  } else {
    const f2 m = both(mul), c5 = both(-0.0047162557f), c4 = both(0.019582905f), c3 = both(-0.053344428f),
             c2 = both(0.13325407f), c1 = both(-0.33332959f), c0 = both(1.f);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const f2 u = mul2(pku(v[e], v[e + 1]), m), w = mul2(u, u);
      f2 r = fma2(w, c5, c4);
      r = fma2(w, r, c3);
      r = fma2(w, r, c2);
      r = fma2(w, r, c1);
      unu(mul2(u, fma2(w, r, c0)), v[e], v[e + 1]);
    }
  }
}

__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
  return max2(max3(mx[0], mx[1], mx[2]), mx[3]);
}

// The score in powers of two from a raw product (with a cap: its tanh) v: mul = log2(e) scale, or log2(e) cap. away:
// the distance, of either sign.
template <bool BIAS>
__device__ __forceinline__ float score(uint32_t v, float mul, float slope, float away) {
  const float y = __uint_as_float(v) * mul;
  return BIAS ? fmaf(-slope, fabsf(away), y) : y;
}

// Biased scores of 32 raw products (or their tanh) in place, powers of two: v mul - slope |away - e|. side: 1 where
// away - e >= 0 for the whole warp, -1 where it is <= 0 (the distance then needs no absolute value), else 0.
__device__ __forceinline__ void bias32(uint32_t (&v)[32], float mul, float slope, float away, int side) {
  if (side) {
    const float sl = side > 0 ? slope : -slope;
    const f2 m = both(mul), s = both(sl), a = both(-sl * away);
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      unu(fma2(pku(v[e], v[e + 1]), m, fma2(s, pk((float)e, (float)(e + 1)), a)), v[e], v[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(score<true>(v[e], mul, slope, away - (float)e));
  }
}

// Bits of the columns [first, end) of 32
__device__ __forceinline__ uint32_t see_bits(int first, int end) {
  const int a = min(max(first, 0), 32), b = min(max(end, 0), 32);
  return a >= b ? 0u : (0xffffffffu << a) & (0xffffffffu >> (32 - b));
}

// -inf in the columns whose bit is 0
__device__ __forceinline__ void mask32(uint32_t (&v)[32], uint32_t see) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(see & (1u << e))) v[e] = 0xff800000u;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T: A is 128 rows (lanes) of 16 bf16, two per 32-bit column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The 16-element steps of one product, unrolled: the descriptors of a step are the first one's plus a constant (address
// fields count 16 bytes). One thread issues them all, and with descriptors built anew in a loop over the steps its own
// instructions, not the tensor cores, set the pace.
// A and B K-major tiles (N steps over the head dimension, four per 16 KB chunk):
template <int N, int B_CHUNK>
__device__ __forceinline__ void mma_kk(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    umma_bf16(d, a + (k >> 2) * (kChunk >> 4) + (k & 3) * 2, b + (k >> 2) * (B_CHUNK >> 4) + (k & 3) * 2, id, k > 0 ? 1u : 0u);
}
template <int B_CHUNK = kChunk>  // bytes from one 64-column chunk of B to the next
__device__ __forceinline__ void mma_kk_nd(int nd, uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  if (nd == 2) mma_kk<8, B_CHUNK>(d, a, b, id);
  else mma_kk<4, B_CHUNK>(d, a, b, id);
}
// A in TMEM (8 columns per step, STRIDE columns from one 32-element piece to the next), B MN-major (16 token rows, 2 KB,
// per step); N steps over tokens:
template <int N, int STRIDE = 16>
__device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    umma_bf16_ts(d, a + 8 * (k & 1) + STRIDE * (k >> 1), b + k * 128, id, (k > 0 || add) ? 1u : 0u);
}

// One arrival for the whole warp (32 of its threads' own would take turns at the barrier's word, 512 of a block longer than
// the step that they end): after every lane's tensor-memory accesses are complete and fenced.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// mbar_wait_soon whose tries tell the hardware that they may sleep for as long as 20 us: a waiting warp then takes fewer
// issue slots from the warps that compute (forward, 8192 tokens: 579 against 589 us; dq, 4096 tokens, its loading and
// issuing warps alone: 281 against 296). The key-major kernel loses by it (287 against 284 us and more).
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
  }
  return mbar_wait(bar, parity, abort, err, code);
}

// Streams of a forward unit: two heads of a group at one query tile, two neighbouring query tiles of a head, or one alone
enum : int32_t { kTwoHeads = 0, kTwoTiles = 1, kAlone = 2 };

struct MaskedFwdParams {
  CUtensorMap qmap, kmap, vmap;  // [head_dim, heads, seq_len, n_seq], boxes 64 x 1 x 128 x 1
  Plan plan;
  const float* slopes;           // [hq]
  __nv_bfloat16* o;
  int64_t ldo;
  float* lse;                    // [n_q_heads][n_seq * seq_len]
  int32_t n_seq, S, hq, hkv, hd, nd;
  int32_t n_units, kind;         // of a unit's streams
  float mul, cap_mul;            // see score() and tanh_n()
  int* err;
};

struct MaskedBwdParams {
  CUtensorMap qmap, kmap, vmap, domap;  // boxes as in the forward
  CUtensorMap qmap64, domap64;          // of half the rows
  Plan plan;
  const float* slopes;
  const float* lse;              // [hq][T]
  float* delta;                  // [hq][T]: D per query row (written by the dq kernel, read by the dk, dv kernel)
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  int32_t n_seq, S, hq, hkv, hd, nd;
  int32_t n_units;               // of the dq kernel
  int32_t split;                 // CTAs (1 or 2, a cluster) that share a unit of the dk, dv kernel
  float scale, mul, cap_mul;
  int* err;
};

// Barrier of the 512 threads of the backward's compute warps that also returns whether `ok` holds in all of them.
__device__ __forceinline__ bool bar_and_compute(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred q, a;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred a, 1, 512, q;\n\t"
      "selp.u32 %0, 1, 0, a;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// ------------------------------------------------------------------------------------ forward

// Persistent CTAs, one per SM, over units of two streams that share their keys and values: two heads of a group at one
// tile of 128 queries (an even number of heads per group: the streams see the same key tiles), else two
// neighbouring query tiles of one head. Warp 0 loads each stream's Q and, for both, K and V (two stages each); warps 1 and 2
// issue the products of stream 0 and 1; warps 4-7 and 8-11 are the softmax of stream 0 and 1, a query row per thread. A step is
// half a key tile (64 keys): each stream has two S buffers in TMEM, so while the softmax works on step h, S of step h + 1
// is there or on its way, and the order of a stream's products is O_x += P_x V of step h, S_x of step h + 2 (into the same
// buffer). Keys run from the last to the first: with a bias by distance the largest scores mostly come first, and O
// is rescaled rarely (from the first key on, steep slopes rescaled it in every step: 1076 against 908 us at 8192
// tokens). With whole tiles and one S buffer per stream the softmax waited for a P V and an S in
// each step, 40% of its time. P replaces S in TMEM (bf16, the first operand of P V) and never passes through
// shared memory. Each stream has an issuing warp of its own: one thread for both is busy with waits and commits for as long
// as with products, and the tensor cores, which queue about five, run dry (8192 tokens: 908 us with one, 613 with two);
// a third one for S alone loses what a stream's order gives (604 against 589). TMEM: S_x / P_x of step h at
// 128 x + 64 (h & 1), O_x at 256 + 128 x.
//
// Measured (32 query, 8 key/value heads of 128): one sequence of 8192 tokens with a prefix and a bias 537 us (1040 TFLOP/s
// over the visible pairs, 0.63 of a library bf16 product's rate), 4096 tokens causal 131 us, with a cap 131 us (its
// documents see fewer tiles), 8 x 512 tokens 38 us. The tensor pipe is busy half of the time; the rest are waits between
// the products and the softmax, 64 exponentials per row and step.
struct Unit {
  int qt0, qt1, h0, h1, b, j0, j1;
  __device__ __forceinline__ int qt(int x) const { return x ? qt1 : qt0; }
  __device__ __forceinline__ int h(int x) const { return x ? h1 : h0; }
};

// Unit number of a CTA's i-th unit: the units stand longest first, and a CTA goes through them there and back, so
// that every CTA gets long and short ones.
__device__ __forceinline__ int unit_number(int i) {
  return (i & 1) ? (i + 1) * (int)gridDim.x - 1 - (int)blockIdx.x : i * (int)gridDim.x + (int)blockIdx.x;
}

// A unit's entry of the plan, read a unit ahead, and what it says (apart, so that nothing waits for the read).
__device__ __forceinline__ int4 unit_entry(const MaskedFwdParams& p, int u) {
  if (u >= p.n_units) return make_int4(0, 0, 0, 0);
  if (p.kind == kTwoTiles) return p.plan.q2_order[u / p.hq];
  return p.plan.q_order[u / (p.kind == kTwoHeads ? p.hq >> 1 : p.hq)];
}

__device__ __forceinline__ Unit unit_of(const MaskedFwdParams& p, int u, const int4& e) {
  Unit r;
  if (p.kind != kTwoTiles) {
    const int n_qt = (p.S + kTile - 1) / kTile, heads = p.kind == kTwoHeads ? p.hq >> 1 : p.hq;
    r.b = e.x / n_qt;
    r.qt0 = r.qt1 = e.x % n_qt;
    r.h0 = r.h1 = u % heads;
    if (p.kind == kTwoHeads) {
      r.h0 *= 2;
      r.h1 = r.h0 + 1;
    }
    r.j0 = e.y;
    r.j1 = e.z;
  } else {
    const int n_t2 = ((p.S + kTile - 1) / kTile + 1) >> 1;
    r.b = e.x / n_t2;
    r.qt0 = 2 * (e.x % n_t2);
    r.qt1 = r.qt0 + 1;
    r.h0 = r.h1 = u % p.hq;
    r.j0 = e.y;
    r.j1 = e.z;
  }
  return r;
}

// Each thread of the warp writes 16 consecutive 32-bit columns of its TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Stores 32 bf16 columns of 32 rows, a row per lane (w: 16 packed pairs), row `lane` at out + lane * ld: four lanes trade
// 16-byte pieces (a 4 x 4 transposition) so that each store writes 64 consecutive bytes of eight rows instead of 16
// bytes of 32. Rows from n_rows on and columns from n_cols (a multiple of 8) on are not written.
__device__ __forceinline__ void store_rows32(__nv_bfloat16* out, int64_t ld, uint32_t (&w)[16], int n_rows, int n_cols) {
  const int lane = threadIdx.x & 31, sub = lane & 3;
  // pieces i of this row; stage 1 trades pieces 0 <-> 1, 2 <-> 3 with lane ^ 1, stage 2 pieces 0 <-> 2, 1 <-> 3 with lane ^ 2
#pragma unroll
  for (int st = 1; st <= 2; st <<= 1) {
    const bool upper = (sub & st) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & st) continue;
      const int k = i | st;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t give = upper ? w[4 * i + q] : w[4 * k + q];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, st);
        if (upper) w[4 * i + q] = got;
        else w[4 * k + q] = got;
      }
    }
  }
  // now piece i of this lane is piece `sub` of row (lane & ~3) + i
  if (8 * sub < n_cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (lane & ~3) + i;
      if (row < n_rows)
        *reinterpret_cast<uint4*>(out + row * ld + 8 * sub) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kFwdThreads, 1) masked_fwd_kernel(const __grid_constant__ MaskedFwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nd = p.nd;
  uint8_t* sq = smem;                     // Q of stream x: nd chunks at 2 x chunks
  uint8_t* sk = smem + 4 * kChunk;        // [2] stages of K, 2 chunks each
  uint8_t* sv = smem + 8 * kChunk;        // [2] stages of V
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 12 * kChunk);
  uint64_t* q_full = bars;         // [2] by stream
  uint64_t* q_empty = bars + 2;    // [2]
  uint64_t* kv_full = bars + 4;    // [2] by stage
  uint64_t* kv_empty = bars + 6;   // [2]
  uint64_t* s_full = bars + 12;    // [2 x + buffer]
  uint64_t* p_full = bars + 16;    // [2 x + buffer]
  uint64_t* pv_done = bars + 20;   // [2 x + buffer]: P V of a unit's last two steps
  uint64_t* drain = bars + 24;     // [2] by stream
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hpg = p.hq / p.hkv, n_streams = p.kind == kAlone ? 1 : 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], n_streams);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&pv_done[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.qmap);
    tma_prefetch_desc(&p.kmap);
    tma_prefetch_desc(&p.vmap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  int4 e0 = unit_entry(p, unit_number(0)), e1 = unit_entry(p, unit_number(1));  // this unit and the next
  const bool plan_ok = plan_fits(p.plan, p.n_seq, p.S, p.err);

  if (warp == 0) {
    if (lane == 0) {
      bool ok = plan_ok;
      int i = 0, t = 0, n_q[2] = {0, 0};  // units, key tiles loaded, each stream's query tiles
      for (; ok && unit_number(i) < p.n_units; ++i) {
        const Unit un = unit_of(p, unit_number(i), e0);
        e0 = e1;
        e1 = unit_entry(p, unit_number(i + 2));
        const int g = un.h0 / hpg;
        for (int x = 0; x < n_streams && ok; ++x) {
          if (i > 0) ok = mbar_wait_idle(&q_empty[x], (i - 1) & 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full[x], nd * kChunk);
          for (int c = 0; c < nd; ++c)
            tma_load_4d(sq + (2 * x + c) * kChunk, &p.qmap, &q_full[x], 64 * c, un.h(x), un.qt(x) * kTile, un.b);
          ++(x ? n_q[1] : n_q[0]);
        }
        for (int j = un.j1 - 1; ok && j >= un.j0; --j, ++t) {
          const int s = t & 1;
          ok = mbar_wait_idle(&kv_empty[s], ((t >> 1) & 1) ^ 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(&kv_full[s], 2 * nd * kChunk);
          for (int c = 0; c < nd; ++c)
            tma_load_4d(sk + (2 * s + c) * kChunk, &p.kmap, &kv_full[s], 64 * c, g, j * kTile, un.b);
          for (int c = 0; c < nd; ++c)
            tma_load_4d(sv + (2 * s + c) * kChunk, &p.vmap, &kv_full[s], 64 * c, g, j * kTile, un.b);
        }
      }
      // every copy lands before the CTA may exit
      if (n_q[0]) mbar_wait(&q_full[0], (n_q[0] - 1) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
      if (n_q[1]) mbar_wait(&q_full[1], (n_q[1] - 1) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
      for (int k = max(0, t - 2); k < t; ++k) mbar_wait(&kv_full[k & 1], (k >> 1) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    }
  } else if (warp <= n_streams) {
    if (lane == 0) {
      const int x = warp - 1;  // stream
      const uint32_t id_s = idesc_bf16(128, 64, 0, 0);         // S = Q K^T: both K-major over d
      const uint32_t id_pv = idesc_bf16(128, 64 * nd, 0, 1);   // O += P V: P in TMEM, V MN-major
      const uint64_t dq0 = kmajor_desc(smem_u32(sq + 2 * x * kChunk), 0), dk0 = kmajor_desc(smem_u32(sk), 0),
                     dv0 = mnmajor_desc(smem_u32(sv), 0);
      // S of key tile t, half buf (the second half of the keys first); first: of its unit, last: the unit's last tile
      auto issue_s = [&](int t, int buf, bool last) {
        const int s = t & 1;
        mma_kk_nd(nd, tmem + 128 * x + 64 * buf, dq0, dk0 + s * (2 * kChunk >> 4) + (buf ^ 1) * (kChunk / 2 >> 4), id_s);
        umma_commit(&s_full[2 * x + buf]);
        if (last && buf) umma_commit(&q_empty[x]);
      };
      auto arrived = [&](int t, int i, bool first) -> bool {  // K and V of tile t, and its unit's Q
        return (!first || mbar_wait_idle(&q_full[x], i & 1, abort_flag, p.err, DEV_TIMEOUT_MMA)) &&
               mbar_wait_idle(&kv_full[t & 1], (t >> 1) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
      };
      int n = e0.z - e0.y, n_next = e1.z - e1.y, i = 0, j = 0;  // tiles of this unit and the next (0: none), unit, tile in it
      int4 e2 = unit_entry(p, unit_number(2));
      bool ok = plan_ok && n > 0 && arrived(0, 0, true);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0, n == 1);
        issue_s(0, 1, n == 1);
      }
      for (int t = 0; ok; ++t) {
        // P V of tile t, and S of tile t + 1 a tile ahead; S of the next unit, whose Q is on its way, behind both P V
        const bool last = j == n - 1, more = !last || n_next > 0;
        const int s = t & 1;
#pragma unroll
        for (int buf = 0; buf < 2; ++buf) {
          ok = mbar_wait_idle(&p_full[2 * x + buf], t & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
          if (!ok) break;
          tc_fence_after();
          mma_tm<4>(tmem + 256 + 128 * x, tmem + 128 * x + 64 * buf, dv0 + s * (2 * kChunk >> 4) + (buf ^ 1) * 512, id_pv,
                    j > 0 || buf > 0);
          if (last) umma_commit(&pv_done[2 * x + buf]);
          if (buf) umma_commit(&kv_empty[s]);
          if (!last) {
            if (buf == 0) {
              ok = arrived(t + 1, i, false);
              if (!ok) break;
              tc_fence_after();
            }
            issue_s(t + 1, buf, j + 1 == n - 1);
          }
        }
        if (!more || !ok) break;
        if (last) {
          ++i;
          j = 0;
          n = n_next;
          n_next = e2.z - e2.y;
          e2 = unit_entry(p, unit_number(i + 2));
          ok = arrived(t + 1, i, true);
          if (!ok) break;
          tc_fence_after();
          issue_s(t + 1, 0, n == 1);
          issue_s(t + 1, 1, n == 1);
        } else {
          ++j;
        }
      }
      umma_commit(&drain[x]);
      mbar_wait(&drain[x], 0, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    }
  } else if (warp >= 4 && warp < 4 + 4 * n_streams) {
    const int x = warp >= 8;                         // stream
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;               // query row in the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + 128 * x, o_tm = s_tm + 256;
    bool ok = plan_ok, more = plan_ok && unit_number(0) < p.n_units;
    int t = 0;
    Unit me, nx;
    int lo = 0, hi = 0, nlo = 0, nhi = 0;            // the keys [lo, hi) that this row sees (rows past the sequence: none)
    auto rows_of = [&](const Unit& w, int& l, int& h) {
      const int q = w.qt(x) * kTile + r;
      l = h = 0;
      if (q < p.S) {
        l = p.plan.lo[(int64_t)w.b * p.S + q];
        h = p.plan.hi[(int64_t)w.b * p.S + q];
      }
    };
    if (more) {
      nx = unit_of(p, unit_number(0), e0);
      rows_of(nx, nlo, nhi);
    }
    for (int i = 0; ok && more; ++i) {
      me = nx;
      lo = nlo;
      hi = nhi;
      more = unit_number(i + 1) < p.n_units;
      if (more) {
        nx = unit_of(p, unit_number(i + 1), e1);
        e1 = unit_entry(p, unit_number(i + 2));
      }
      const int qt = me.qt(x), h = me.h(x);
      const int qpos = qt * kTile + r;               // position in the sequence
      const float slope = BIAS ? p.slopes[h] * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int k0 = me.j1 * kTile - 64; k0 >= me.j0 * kTile; k0 -= 64, ++t) {
        const int buf = t & 1;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_idle(&s_full[2 * x + buf], (t >> 1) & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[2][32];
        tmem_ld32(s_tm + 64 * buf, s[0]);
        tmem_ld32(s_tm + 64 * buf + 32, s[1]);
        tmem_ld_wait_regs(s[0]);
        regs_after_wait(s[1]);
        if (CAP) {
          tanh_n(s[0], p.cap_mul);
          tanh_n(s[1], p.cap_mul);
        }
        // With a bias the score itself is formed here (mul = 1 below), else scores stay raw products
        if (BIAS) {
          const int side = qt * kTile + 32 * quarter >= k0 + 63;
#pragma unroll
          for (int c = 0; c < 2; ++c) bias32(s[c], p.mul, slope, (float)(qpos - k0 - 32 * c), side);
        }
        const float mul = BIAS ? 1.f : p.mul;
        if (__any_sync(0xffffffffu, lo > k0 || hi < k0 + 64)) {
          mask32(s[0], see_bits(lo - k0, hi - k0));
          mask32(s[1], see_bits(lo - k0 - 32, hi - k0 - 32));
        }
        // A NaN or +inf score makes its row's maximum NaN, and with it o and lse, whatever ex2_poly makes of it.
        float mj = max2(max32(s[0]), max32(s[1])) * mul;
        if (mj == INFINITY) mj = NAN;
        // The running maximum moves only when a row's maximum grows by more than 2^8: the exponentials then
        // stay below 256 and O and l keep one common reference, so O is rescaled rarely.
        const float m_cand = max2(m, mj);
        const bool grow = !(m_cand - m <= 8.0f);  // also from a row that has seen nothing, and to NaN
        const float m_new = grow ? m_cand : m;
        const float mb = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
        const float corr = grow && m != -INFINITY ? ex2(m - mb) : 1.f;  // O and l of a row that saw nothing are 0
        f2 rs[2] = {0, 0};
        const f2 mul_2 = both(mul), mb_2 = both(-mb);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            const f2 x = fma2(pku(s[c][e], s[c][e + 1]), mul_2, mb_2);
            if (!CAP && (e & 6) == 4) {
              ex2_poly(x, x0, x1);
            } else {
              un(x, x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
            }
            rs[(e >> 1) & 1] = add2(rs[(e >> 1) & 1], pk(x0, x1));
            pw[e / 2] = pack2(x0, x1);
          }
          tmem_st16(s_tm + 64 * buf + 16 * c, pw);
        }
        if (k0 < me.j1 * kTile - 64 && __any_sync(0xffffffffu, corr != 1.f)) {
          // O of the steps before is complete once their last P V is: S of the next step stands behind it in the tensor
          // pipe; after a unit's last S its own barrier tells
          uint64_t* bar = k0 > me.j0 * kTile ? &s_full[2 * x + (buf ^ 1)] : &pv_done[2 * x];
          const uint32_t phase = k0 > me.j0 * kTile ? ((t + 1) >> 1) & 1 : i & 1;
          ok = __all_sync(0xffffffffu, mbar_wait_idle(bar, phase, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 2 * nd; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_tm + 32 * c, ov);
            tmem_ld_wait_regs(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
            tmem_st32(o_tm + 32 * c, ov);
          }
        }
        float r0, r1;
        un(add2(rs[0], rs[1]), r0, r1);
        l = l * corr + (r0 + r1);
        m = m_new;
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&p_full[2 * x + buf], lane);
      }
      if (!ok) break;
      if (more) rows_of(nx, nlo, nhi);
      ok = __all_sync(0xffffffffu, mbar_wait_idle(&pv_done[2 * x + 1], i & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
      if (!ok) break;
      // O / l as bf16; the next unit's first P V waits for this softmax's next P
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing: o = 0
      const int64_t row0 = (int64_t)me.b * p.S + qt * kTile + 32 * quarter;  // row of lane 0
      const int n_rows = p.S - (qt * kTile + 32 * quarter);
#pragma unroll 1
      for (int c = 0; c < 2 * nd; c += 2) {
        uint32_t ov[2][32], w[2][16];
        tmem_ld32(o_tm + 32 * c, ov[0]);
        tmem_ld32(o_tm + 32 * c + 32, ov[1]);
        tmem_ld_wait_regs(ov[0]);
        regs_after_wait(ov[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            w[k][e / 2] = pack2(__uint_as_float(ov[k][e]) * inv, __uint_as_float(ov[k][e + 1]) * inv);
          store_rows32(p.o + row0 * p.ldo + (int64_t)h * p.hd + 32 * (c + k), p.ldo, w[k], n_rows, p.hd - 32 * (c + k));
        }
      }
      tc_fence_before();
      if (qpos < p.S)
        p.lse[(int64_t)h * p.n_seq * p.S + row0 + lane] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------------------------------- backward

// Two kernels. dq: per tile of queries, D and then dQ, over the key tiles that it sees; dk, dv: per tile of keys, over
// the query tiles that see it. Each forms S and dP for itself (nine products of a tile pair where one kernel for
// all would have five and a sum for D), but no partial sum leaves the chip and every sum has a fixed order. With dQ
// added up across key tiles in global memory (64 KB of fp32 reductions per tile pair, a kernel for D before it and a pass
// that rounds after it) dq's last bits depended on the order. As first built that form took 161 us at 8 x 512 tokens and
// 631 at 4096 capped ones, this one 129 and 609 (115 and 534 by what came later, which the other form has not had).
//
// D_i = sum_j P_ij dP_ij (= dO_i . o_i) is formed from P and dP in fp32 and not from the stored o: that one is rounded to
// bf16, and its error, the same for all keys of a row, is as large as all other roundings of dq and dk
// together where a row's weight lies on few keys (relative error of dq over 4e-3 with 8 keys, against 2.3e-3).

// dS = P (dP - D) (1 - tanh^2) of 32 columns: from raw products s and dp; c1: -lse (powers of two), c2: -D, each
// one per row (ROW) or read per column from shared memory. P as packed bf16 in pw (when wanted), dS in dw; FINE: and behind
// it what the rounding left of dS, as bf16 again.
//
// Rounded once, dS costs dq and dk about as much as their own rounding does: the error of both together is 1.41 times the
// latter's alone, 1.35 to 1.47 for heads of 72 to 128 with documents or windows of any length from two tokens on. It grows
// where few terms make a result: heads of 8 have up to 1.7, and single batches of a few tokens any value up to 2.4
// (their mean is 1.4 too). With the rest as a second first operand of dQ += dS K and dK += dS^T Q nothing of that is left.
// fine_grads() takes it for heads up to 64, whose products are half as wide, and for sequences of one tile, where it
// costs little (4096 causal tokens of 128: dq 324 against 281 us with it, dk and dv 294 against 264).
bool fine_grads(int hd, int S) { return hd <= 64 || S <= kTile; }

template <bool CAP, bool BIAS, bool ROW, bool WANT_P, bool FINE>
__device__ __forceinline__ void grad32(uint32_t (&s)[32], uint32_t (&dp)[32], float mul, float cap_mul, float slope,
                                       float away, int side, bool part, uint32_t see, float c1, float c2,
                                       const float* col1, const float* col2, uint32_t (&pw)[16],
                                       uint32_t (&dw)[FINE ? 32 : 16]) {
  uint32_t th[CAP ? 32 : 2];
  if (CAP) {
    tanh_n(s, cap_mul);
#pragma unroll
    for (int e = 0; e < 32; ++e) th[e] = s[e];
  }
  if (BIAS) bias32(s, mul, slope, away, side);
  if (part) mask32(s, see);  // -inf: P = 0
  const f2 m = both(BIAS ? 1.f : mul), one = both(1.f);
  const f2 r1 = both(c1), r2 = both(c2);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    f2 a1[2], a2[2];
    if (ROW) {
      a1[0] = a1[1] = r1;
      a2[0] = a2[1] = r2;
    } else {
      const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(col1 + e), d = *reinterpret_cast<const ulonglong2*>(col2 + e);
      a1[0] = l.x, a1[1] = l.y, a2[0] = d.x, a2[1] = d.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = e + 2 * k;
      float x0, x1;
      un(fma2(pku(s[i], s[i + 1]), m, a1[k]), x0, x1);
      x0 = ex2(x0);
      x1 = ex2(x1);
      const f2 pe = pk(x0, x1);
      f2 ds = mul2(pe, add2(pku(dp[i], dp[i + 1]), a2[k]));
      if (CAP) {
        const f2 t = pku(th[i], th[i + 1]);
        ds = mul2(ds, fma2(mul2(t, both(-1.f)), t, one));
      }
      float d0, d1;
      un(ds, d0, d1);
      if (WANT_P) pw[i / 2] = pack2(x0, x1);
      const uint32_t d = pack2(d0, d1);
      dw[i / 2] = d;
      if (FINE) dw[16 + i / 2] = pack2(d0 - __uint_as_float(d << 16), d1 - __uint_as_float(d & 0xffff0000u));
    }
  }
}

// dq: persistent CTAs over units (query tile, head). Q and dO stay, K streams through three stages and V through two, for D
// and then, from the last key tile to the first, for dQ. S, dP and K of the last two tiles are kept, so the second pass forms
// them again only from the third on (documents of up to 256 keys: once). Warp 0 loads; warps 1, 2 and 3 issue
// S = Q K^T, dP = dO V^T and dQ += dS K, S and dP ahead of the compute warps. Warps 4-19 hold a query row and 32 of
// the 128 key columns per thread. With n key tiles in unit i, step m < n of the first pass has S in buffer (i + m) & 1, the
// k-th of the second pass (kept or formed again) in buffer (i + n - 1 + k) & 1, where dS takes its place. TMEM: S / dS at
// 128 and 256, dP at 384 and, in the first pass, every other one at 0, the last tile's among them (of two or more):
// dQ is added up there once that one has been read. K has three stages, since it stays until dS K is done, V two.
//
// Measured (32 query, 8 key/value heads of 128): 4096 causal tokens 282 us (1200 TFLOP/s of the products done), capped documents
// 265 us, 8 x 512 tokens 62 us. S and dP formed twice for every tile: 349, 318 and 69 us; K and V in two common stages: 353,
// 298, 66 (a stage is held from its load to the end of dS K, and the next load waits); dP without its second place: 299.
// What is left between the products is the chain from a dS over its product to the S that takes its buffer. The 104 registers
// of a compute thread (96 as compiled) do not hold all: 116 bytes per thread are spilled without a cap, 224 with one, 252
// with a bias too. (Eight compute warps, which spill nothing, are not measured here.)
template <bool CAP, bool BIAS, bool FINE>
__global__ void __launch_bounds__(kBwdThreads, 1) masked_dq_kernel(const __grid_constant__ MaskedBwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_dq[];
  const int nd = p.nd;
  uint8_t* sq = smem_dq;                    // Q, then dO: 2 chunks each
  uint8_t* sk = smem_dq + 4 * kChunk;       // [3] stages of K
  uint8_t* sv = smem_dq + 10 * kChunk;      // [2] stages of V
  float* s_part = reinterpret_cast<float*>(smem_dq + 14 * kChunk);  // [4][128]: the quarters' sums of D
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_part + 512);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* v_full = bars + 2;     // [2]
  uint64_t* v_empty = bars + 4;    // [2]
  uint64_t* s_full = bars + 6;     // [2] by buffer
  uint64_t* s_read = bars + 8;     // [2]: S is in registers and not kept
  uint64_t* ds_full = bars + 10;   // [2]: dS in the buffer
  uint64_t* ds_done = bars + 12;   // [2]: dQ has read it
  uint64_t* dp_full = bars + 14;   // [2]: dP in its place, in dQ's place
  uint64_t* dp_read = bars + 16;   // [2]: dP is in registers and not kept
  uint64_t* dq_done = bars + 18;   // a unit's dQ
  uint64_t* dq_read = bars + 19;   // it is in registers
  uint64_t* drain = bars + 20;     // [3]
  uint64_t* k_full = bars + 23;    // [3]
  uint64_t* k_empty = bars + 26;   // [3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 29);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_qt = (p.S + kTile - 1) / kTile;
  const int hpg = p.hq / p.hkv;
  auto entry = [&](int i) -> int4 {  // of this CTA's unit i, read ahead (no key tiles: there is no such unit)
    const int u = unit_number(i);
    return u < p.n_units ? p.plan.q_order[u / p.hq] : make_int4(0, 0, 0, 0);
  };
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);  // S, dP
    for (int s = 0; s < 2; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_read[s], 16);
      mbar_init(&ds_full[s], 16);
      mbar_init(&ds_done[s], 1);
      mbar_init(&dp_full[s], 1);
      mbar_init(&dp_read[s], 16);
    }
    mbar_init(dq_done, 1);
    mbar_init(dq_read, 16);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&drain[s], 1);
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);  // S of the first pass, or dQ
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.qmap);
    tma_prefetch_desc(&p.kmap);
    tma_prefetch_desc(&p.vmap);
    tma_prefetch_desc(&p.domap);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  int4 e = entry(0);
  const bool plan_ok = plan_fits(p.plan, p.n_seq, p.S, p.err);

  // 640 threads start with 96 registers each; 56 in the first four warps and 104 in the others stay within their sum
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      bool ok = plan_ok;
      int n_q = 0, n_k = 0, n_v = 0;  // query tiles, K, V loaded
      for (int i = 0; ok && e.z > e.y; ++i) {
        const int qt0 = e.x % n_qt * kTile, b = e.x / n_qt, h = unit_number(i) % p.hq, j0 = e.y, j1 = e.z;
        e = entry(i + 1);
        if (i > 0 && !mbar_wait_idle(q_empty, (i - 1) & 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER)) break;
        mbar_arrive_expect_tx(q_full, 2 * nd * kChunk);
        for (int c = 0; c < nd; ++c) {
          tma_load_4d(sq + c * kChunk, &p.qmap, q_full, 64 * c, h, qt0, b);
          tma_load_4d(sq + (2 + c) * kChunk, &p.domap, q_full, 64 * c, h, qt0, b);
        }
        ++n_q;
        const int n = j1 - j0, steps = 2 * n - min(2, n), g = h / hpg;
        for (int m = 0; m < steps; ++m) {
          const int j = m < n ? j0 + m : j1 - 3 - (m - n), sk_ = n_k % 3, sv_ = n_v & 1;
          ok = mbar_wait_idle(&k_empty[sk_], ((n_k / 3) & 1) ^ 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(&k_full[sk_], nd * kChunk);
          for (int c = 0; c < nd; ++c)
            tma_load_4d(sk + (2 * sk_ + c) * kChunk, &p.kmap, &k_full[sk_], 64 * c, g, j * kTile, b);
          ++n_k;
          ok = mbar_wait_idle(&v_empty[sv_], ((n_v >> 1) & 1) ^ 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(&v_full[sv_], nd * kChunk);
          for (int c = 0; c < nd; ++c)
            tma_load_4d(sv + (2 * sv_ + c) * kChunk, &p.vmap, &v_full[sv_], 64 * c, g, j * kTile, b);
          ++n_v;
        }
      }
      // every copy lands before the CTA may exit
      if (n_q) mbar_wait(q_full, (n_q - 1) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
      for (int l = max(0, n_k - 3); l < n_k; ++l) mbar_wait(&k_full[l % 3], (l / 3) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
      for (int l = max(0, n_v - 2); l < n_v; ++l) mbar_wait(&v_full[l & 1], (l >> 1) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    } else if (warp > 0 && lane == 0) {
      bool ok = plan_ok;
      if (warp == 3) {
        const uint32_t id = idesc_bf16(128, 64 * nd, 0, 1);
        const uint64_t dk0 = mnmajor_desc(smem_u32(sk), 0);
        int l0 = 0;            // the unit's first load
        int used[2] = {0, 0};  // dS in each buffer so far
        for (int i = 0; ok && e.z > e.y; ++i) {
          const int n = e.z - e.y;
          e = entry(i + 1);
          for (int k = 0; k < n; ++k) {
            const int b = (i + n - 1 + k) & 1;
            // the step's K has come (its S has read it), and the first dS is written when dP has been read in dQ's place
            ok = mbar_wait_idle(&ds_full[b], (b ? used[1]++ : used[0]++) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
            if (!ok) break;
            tc_fence_after();
            const int s = (l0 + (k < min(2, n) ? n - 1 - k : n - 2 + k)) % 3;
            mma_tm<8, 32>(tmem, tmem + 128 + 128 * b, dk0 + s * (2 * kChunk >> 4), id, k > 0);
            if (FINE) mma_tm<8, 32>(tmem, tmem + 144 + 128 * b, dk0 + s * (2 * kChunk >> 4), id, true);
            umma_commit(&ds_done[b]);
            umma_commit(&k_empty[s]);
          }
          if (ok) umma_commit(dq_done);
          l0 += 2 * n - min(2, n);
        }
      } else {
        // warp 1: S, warp 2: dP of every step
        const bool is_s = warp == 1;
        const uint32_t id = idesc_bf16(128, 128, 0, 0);
        const uint64_t a0 = kmajor_desc(smem_u32(sq), 0) + (is_s ? 0 : 2 * kChunk >> 4),
                       b0 = kmajor_desc(smem_u32(is_s ? sk : sv), 0);
        int l = 0;                       // steps so far
        int used[2] = {0, 0};            // of each number
        int read[2] = {0, 0}, done[2] = {0, 0};  // S of each buffer that were read once, that became a dS
        bool held[2] = {false, false};   // the buffer's last S becomes a dS
        int n_dp[2] = {0, 0};            // dP in each place that were read and not kept
        for (int i = 0; ok && e.z > e.y; ++i) {
          const int n = e.z - e.y, kept = min(2, n), steps = 2 * n - kept;
          e = entry(i + 1);
          ok = mbar_wait_idle(q_full, i & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
          for (int m = 0; ok && m < steps; ++m, ++l) {
            const int b = (i + m + (m >= n)) & 1;
            const bool once = m < n - kept, in_dq = n > 1 && m < n && !((n - 1 - m) & 1);
            const int u = b ? used[1]++ : used[0]++, s = is_s ? l % 3 : l & 1;
            ok = mbar_wait_idle(is_s ? &k_full[s] : &v_full[s], (is_s ? l / 3 : l >> 1) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
            if (ok && is_s) {
              if (u > 0) {
                const bool ds = b ? held[1] : held[0];
                int& c = ds ? (b ? done[1] : done[0]) : (b ? read[1] : read[0]);
                ok = mbar_wait_idle(ds ? &ds_done[b] : &s_read[b], c++ & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
              }
              (b ? held[1] : held[0]) = !once;
            } else if (ok && in_dq) {
              // behind the unit's dP two steps ago, or the last unit's dQ
              if (m >= 2) ok = mbar_wait_idle(&dp_read[1], n_dp[1]++ & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
              else if (i > 0) ok = mbar_wait_idle(dq_read, (i - 1) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
            } else if (ok && (i > 0 || m >= 2)) {
              ok = mbar_wait_idle(&dp_read[0], n_dp[0]++ & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
            }
            if (!ok) break;
            tc_fence_after();
            mma_kk_nd(nd, is_s ? tmem + 128 + 128 * b : (in_dq ? tmem : tmem + 384), a0, b0 + s * (2 * kChunk >> 4), id);
            umma_commit(is_s ? &s_full[b] : &dp_full[in_dq]);
            if (!is_s) umma_commit(&v_empty[s]);
            else if (once) umma_commit(&k_empty[s]);
            if (m == steps - 1) umma_commit(q_empty);
          }
          // each phase of dq_read is waited for once, also where dQ's place held no dP
          if (ok && !is_s && n == 1 && i > 0) ok = mbar_wait_idle(dq_read, (i - 1) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
        }
      }
      umma_commit(&drain[warp - 1]);
      mbar_wait(&drain[warp - 1], 0, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int quarter = warp & 3, cq = (warp - 4) >> 2;  // rows (TMEM lanes); 32 of the 128 key columns
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t dq_tm = tmem + lane_off + 32 * cq, s_tm = dq_tm + 128, dp_tm = dq_tm + 384;
    bool ok = plan_ok, live = plan_ok && e.z > e.y;
    uint32_t phases = 0;  // of s_full (bits 0, 1) and dp_full (2, 3), turned with each wait
    int nlo = 0, nhi = 0;
    float nlse = 0.f;
    const int64_t T = (int64_t)p.n_seq * p.S;
    auto rows_of = [&](int i) {  // what the row of unit i (entry e) sees, and its lse in powers of two
      const int q = e.x % n_qt * kTile + r, row = e.x / n_qt * p.S + q;
      const bool in = q < p.S;
      nlo = in ? p.plan.lo[row] : 0;
      nhi = in ? p.plan.hi[row] : 0;
      nlse = in ? p.lse[(int64_t)(unit_number(i) % p.hq) * T + row] * kLog2e : 0.f;
    };
    if (live) rows_of(0);
    for (int i = 0; ok && live; ++i) {
      const int lo = nlo, hi = nhi, qt0 = e.x % n_qt * kTile, first = e.x / n_qt * p.S + qt0, h = unit_number(i) % p.hq;
      const int j0 = e.y, j1 = e.z;
      const float nl = lo < hi ? -nlse : -INFINITY;  // a row that sees nothing: P = 0 whatever its score
      e = entry(i + 1);
      const float slope = BIAS ? p.slopes[h] * kLog2e : 0.f;
      // a row that sees one key: P = 1 and D = dP to the bit, so that its dS is 0 and not a rounding's rest
      const bool single = hi - lo == 1;
      const bool singles = __any_sync(0xffffffffu, single);
      const int n = j1 - j0, kept = min(2, n);
      // S and dP of a step in registers; fresh: they have to be waited for
      uint32_t s[32], dp[32];
      auto take = [&](int bf, bool in_dq, bool fresh) {
        if (fresh) {
          ok = __all_sync(0xffffffffu, mbar_wait_soon(&s_full[bf], (phases >> bf) & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE) &&
                                           mbar_wait_soon(&dp_full[in_dq], (phases >> (2 + in_dq)) & 1, abort_flag, p.err,
                                                          DEV_TIMEOUT_EPILOGUE));
          if (!ok) return;
          phases ^= 1u << bf | 4u << in_dq;
          tc_fence_after();
        }
        tmem_ld32(s_tm + 128 * bf, s);
        tmem_ld32(in_dq ? dq_tm : dp_tm, dp);
        tmem_ld_wait_regs(s);
        regs_after_wait(dp);
        tc_fence_before();
        __syncwarp();
      };
      f2 acc[2] = {0, 0};
      float only = 0.f;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int bf = (i + k) & 1;
        const bool in_dq = n > 1 && !((n - 1 - k) & 1);
        take(bf, in_dq, true);
        if (!ok) break;
        if (lane == 0 && k < n - kept) {
          mbar_arrive(&dp_read[in_dq]);
          mbar_arrive(&s_read[bf]);
        }
        const int k0 = (j0 + k) * kTile + 32 * cq;  // key of this thread's first column
        if (CAP) tanh_n(s, p.cap_mul);
        if (BIAS) bias32(s, p.mul, slope, (float)(qt0 + r - k0), qt0 + 32 * quarter >= k0 + 31);
        if (__any_sync(0xffffffffu, lo > k0 || hi < k0 + 32)) {
          const uint32_t see = see_bits(lo - k0, hi - k0);
          mask32(s, see);
          if (singles) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (see & (1u << e)) only = __uint_as_float(dp[e]);
          }
        }
        const f2 m = both(BIAS ? 1.f : p.mul), l2 = both(nl);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1;
          un(fma2(pku(s[e], s[e + 1]), m, l2), x0, x1);
          acc[(e >> 1) & 1] = fma2(pk(ex2(x0), ex2(x1)), pku(dp[e], dp[e + 1]), acc[(e >> 1) & 1]);
        }
      }
      float a0, a1;
      un(add2(acc[0], acc[1]), a0, a1);
      s_part[cq * 128 + r] = single ? only : a0 + a1;
      ok = bar_and_compute(ok);
      const float sum = (s_part[r] + s_part[128 + r]) + (s_part[256 + r] + s_part[384 + r]);
      if (ok && cq == 0 && qt0 + r < p.S) p.delta[(int64_t)h * T + first + r] = sum;
#pragma unroll 1
      for (int k = 0; ok && k < n; ++k) {
        const int bf = (i + n - 1 + k) & 1;
        const bool in_dq = n > 1 && k == 0;
        take(bf, in_dq, k >= kept);
        if (!ok) break;
        if (lane == 0 && !in_dq) mbar_arrive(&dp_read[0]);
        const int k0 = (j1 - 1 - k) * kTile + 32 * cq;
        const bool part = __any_sync(0xffffffffu, lo > k0 || hi < k0 + 32);
        uint32_t pw[16], dw[FINE ? 32 : 16];
        grad32<CAP, BIAS, true, false, FINE>(s, dp, p.mul, p.cap_mul, slope, (float)(qt0 + r - k0), qt0 + 32 * quarter >= k0 + 31,
                                       part, see_bits(lo - k0, hi - k0), nl, -sum, nullptr, nullptr, pw, dw);
        // over the scores that this warp itself has read
        if constexpr (FINE) tmem_st32(s_tm + 128 * bf, dw);
        else tmem_st16(s_tm + 128 * bf, dw);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&ds_full[bf], lane);
      }
      live = e.z > e.y;
      if (ok && live) rows_of(i + 1);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_soon(dq_done, i & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
      ok = bar_and_compute(ok);  // also: s_part is free for the next unit
      if (!ok) break;
      tc_fence_after();
      const int64_t row0 = first + 32 * quarter;
      const int n_rows = p.S - qt0 - 32 * quarter;
      if (cq < 2 * nd) {
        uint32_t v[32], pk16[16];
        tmem_ld32(dq_tm, v);
        tmem_ld_wait_regs(v);
        tc_fence_before();
        warp_arrive(dq_read, lane);
#pragma unroll
        for (int e = 0; e < 32; e += 2) pk16[e / 2] = pack2(__uint_as_float(v[e]) * p.scale, __uint_as_float(v[e + 1]) * p.scale);
        store_rows32(p.dq + row0 * p.lddq + (int64_t)h * p.hd + 32 * cq, p.lddq, pk16, n_rows, p.hd - 32 * cq);
      } else {
        warp_arrive(dq_read, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// dk, dv: one CTA per (key tile, key/value head) in the plan's order, over (query head of the group, query tile). K and V
// stay, Q and dO stream through five stages of half a query tile. A step is such a half (64 queries): S^T = K Q^T and
// dP^T = V dO^T of step t + 1 run while the compute warps work on step t; P^T and dS^T replace them in TMEM (bf16, first
// operands of dV += P^T dO and dK += dS^T Q). Warp 0 loads, the query rows' lse, D and intervals too; warps 1, 2 and 3 issue
// S^T, dP^T, and dV and dK (a thread that issues also waits and commits, and meanwhile the tensor cores, which queue
// about five products, run dry: 340 us at 4096 causal tokens with one such thread, 320 with two, 277 with three); the
// others compute, one half for the even and one for the odd steps, a key row and 32 query columns per thread at a time:
// 16 warps (40 to 52 bytes spilled), or 8 where a cap's tanh needs the registers (none; with 16 it spilled: 335 against 318
// us at 4096 capped tokens; without a cap 16 gained 10%). TMEM: S^T of buffer x at 64 x, dP^T at 128 + 64 x, dV at 256, dK at 384.
//
// Measured (32 query, 8 key/value heads of 128): 4096 causal tokens 264 us (1070 TFLOP/s of four products per tile pair; 286
// with two stages of whole query tiles), capped 269 us, 8 x 512 tokens 53 us. The products alone take 2640 of a query
// tile's 3900 cycles (64 columns cost 50 cycles per 16-element step, 128 cost 65); whole tiles do not fit the TMEM.
constexpr int kQdStages = 5;

// Both CTAs of a cluster: what each wrote to the other's shared memory before it is there behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(uint32_t smem, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <bool CAP, bool BIAS, bool FINE>
__global__ void __launch_bounds__(kDkvThreads<CAP>, 1) masked_dkv_kernel(const __grid_constant__ MaskedBwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_dkv[];
  const int nd = p.nd;
  constexpr int kWarps = (kDkvThreads<CAP> - 128) / 32, kCols = kWarps == 16 ? 1 : 2;  // 32-column pieces per thread and step
  uint8_t* sk = smem_dkv;                   // K, then V: 2 chunks each
  uint8_t* sqd = smem_dkv + 4 * kChunk;     // stage s of half a query tile: Q (2 half chunks), then dO
  float* s_lse = reinterpret_cast<float*>(smem_dkv + 14 * kChunk);  // [2][64]: -lse in powers of two
  float* s_del = s_lse + 128;                                       // [2][64]: -D
  int2* s_see = reinterpret_cast<int2*>(s_del + 128);               // [2][64]: keys that the query sees
  int* s_whole = reinterpret_cast<int*>(s_see + 128);               // [2]: all of the tile's queries see all of the key tile
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_whole + 4);
  uint64_t* kv_full = bars;
  uint64_t* qd_full = bars + 1;     // [5] by stage
  uint64_t* qd_empty = bars + 6;    // [5]
  uint64_t* rows_full = bars + 11;  // [2] by half
  uint64_t* rows_empty = bars + 13; // [2]
  uint64_t* sd_full = bars + 15;    // [2] by buffer = half
  uint64_t* pd_full = bars + 17;    // [2]
  uint64_t* pd_done = bars + 19;    // [2]
  uint64_t* drain = bars + 21;      // [3]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_t = (p.S + kTile - 1) / kTile;
  const int unit = blockIdx.x / p.split, rank = blockIdx.x % p.split, g = unit % p.hkv;
  const int hpg = p.hq / p.hkv;
  const int64_t T = (int64_t)p.n_seq * p.S;
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < kQdStages; ++s) {
      mbar_init(&qd_full[s], 1);
      mbar_init(&qd_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&rows_full[s], 1);
      mbar_init(&rows_empty[s], kWarps / 2);
      mbar_init(&sd_full[s], 2);  // S^T, dP^T
      mbar_init(&pd_full[s], kWarps / 2);
      mbar_init(&pd_done[s], 1);
    }
    for (int s = 0; s < 3; ++s) mbar_init(&drain[s], 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.qmap64);
    tma_prefetch_desc(&p.kmap);
    tma_prefetch_desc(&p.vmap);
    tma_prefetch_desc(&p.domap64);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // (key tile, sequence) in the plan's order, and the query tiles q0 .. q1 - 1 that see any of it (at least
  // one, so that a tile that nobody sees takes the same path and gets zeros)
  const bool plan_ok = plan_fits(p.plan, p.n_seq, p.S, p.err);
  const int4 entry = plan_ok ? p.plan.k_order[unit / p.hkv] : make_int4(0, 0, 0, 0);
  const int kt = entry.x % n_t, b = entry.x / n_t;
  // this CTA's steps: all of the unit's, or the first or second half (which may be none)
  const int q0 = entry.y, n_unit = hpg * (entry.z - q0), it0 = rank ? (n_unit + 1) / 2 : 0;
  const int n_it = p.split == 1 ? n_unit : rank ? n_unit / 2 : (n_unit + 1) / 2;
  auto it_head = [&](int it) { return g * hpg + (it0 + it) % hpg; };
  auto it_qtile = [&](int it) { return q0 + (it0 + it) / hpg; };

  // 640 threads start with 96 registers each; 56 in the first four warps and 104 in the others stay within their sum
  if (warp < 4) {
    if (kWarps == 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (!plan_ok) {
      // nothing is issued
    } else if (warp == 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(kv_full, 2 * nd * kChunk);
        for (int c = 0; c < nd; ++c) {
          tma_load_4d(sk + c * kChunk, &p.kmap, kv_full, 64 * c, g, kt * kTile, b);
          tma_load_4d(sk + (2 + c) * kChunk, &p.vmap, kv_full, 64 * c, g, kt * kTile, b);
        }
      }
      // the rows' values of a half tile, read one ahead: nothing waits for them then
      float l[2], d[2];
      int2 see[2];
      int4 range;
      auto read_rows = [&](int t) {
        const int it = t >> 1, qt = it_qtile(it), h = it_head(it);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int qp = min(qt * kTile + 64 * (t & 1) + 32 * k + lane, p.S - 1);
          const int64_t row = (int64_t)b * p.S + qp, at = (int64_t)h * T + row;
          see[k] = make_int2(p.plan.lo[row], p.plan.hi[row]);
          l[k] = p.lse[at];
          d[k] = p.delta[at];
        }
        range = p.plan.q_range[b * n_t + qt];
      };
      if (n_it > 0) read_rows(0);
      int t = 0;  // half tiles loaded
      for (; t < 2 * n_it; ++t) {
        const int it = t >> 1, x = t & 1, s = t % kQdStages, first = it_qtile(it) * kTile + 64 * x;
        if (!__all_sync(0xffffffffu, mbar_wait_soon(&qd_empty[s], ((t / kQdStages) & 1) ^ 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&qd_full[s], nd * kChunk);
          uint8_t* st = sqd + s * 2 * kChunk;
          for (int c = 0; c < nd; ++c) {
            tma_load_4d(st + c * (kChunk / 2), &p.qmap64, &qd_full[s], 64 * c, it_head(it), first, b);
            tma_load_4d(st + (2 + c) * (kChunk / 2), &p.domap64, &qd_full[s], 64 * c, it_head(it), first, b);
          }
        }
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait_soon(&rows_empty[x], (it & 1) ^ 1, abort_flag, p.err, DEV_TIMEOUT_PRODUCER))) {
          ++t;
          break;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // a row that sees nothing or lies past the sequence: 2^-inf, P = 0 whatever its score
          const bool in = first + 32 * k + lane < p.S, sees = in && see[k].x < see[k].y;
          s_lse[x * 64 + 32 * k + lane] = sees ? -l[k] * kLog2e : -INFINITY;
          s_del[x * 64 + 32 * k + lane] = sees ? -d[k] : 0.f;
          s_see[x * 64 + 32 * k + lane] = sees ? see[k] : make_int2(0, 0);
        }
        if (lane == 0) s_whole[x] = range.z <= kt && kt < range.w;
        __syncwarp();
        if (lane == 0) mbar_arrive(&rows_full[x]);
        if (t + 1 < 2 * n_it) read_rows(t + 1);
      }
      // every copy lands before the CTA may exit
      if (lane == 0) {
        mbar_wait(kv_full, 0, nullptr, p.err, DEV_TIMEOUT_DRAIN);
        for (int k = max(0, t - kQdStages); k < t; ++k)
          mbar_wait(&qd_full[k % kQdStages], (k / kQdStages) & 1, nullptr, p.err, DEV_TIMEOUT_DRAIN);
      }
    } else if (warp < 3 && lane == 0) {
      // warp 1: S^T = K Q^T; warp 2: dP^T = V dO^T
      const int w = warp - 1;
      const uint32_t id = idesc_bf16(128, 64, 0, 0), d0 = tmem + 128 * w;
      const uint64_t a0 = kmajor_desc(smem_u32(sk), 0) + w * (2 * kChunk >> 4), b0 = kmajor_desc(smem_u32(sqd), 0) + w * (kChunk >> 4);
      bool ok = mbar_wait_soon(kv_full, 0, abort_flag, p.err, DEV_TIMEOUT_MMA);
      for (int it = 0; ok && it < n_it; ++it) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = 2 * it + x, s = t % kQdStages;
          if (ok) ok = mbar_wait_soon(&qd_full[s], (t / kQdStages) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
          if (ok && it > 0) ok = mbar_wait_soon(&pd_done[x], (it - 1) & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
          if (!ok) break;
          tc_fence_after();
          mma_kk_nd<kChunk / 2>(nd, d0 + 64 * x, a0, b0 + s * (2 * kChunk >> 4), id);
          umma_commit(&sd_full[x]);
        }
      }
      umma_commit(&drain[w]);
      mbar_wait(&drain[w], 0, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    } else if (warp == 3 && lane == 0) {
      const uint32_t id = idesc_bf16(128, 64 * nd, 0, 1);  // P^T, dS^T in TMEM; dO, Q MN-major
      const uint64_t dqm0 = smem_desc_sw128(smem_u32(sqd), kChunk / 2, 1024);  // 64-column pieces 8 KB apart
      bool ok = true;
      for (int it = 0; ok && it < n_it; ++it) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // the step's queries have come: its S^T and dP^T have read them
          ok = mbar_wait_soon(&pd_full[x], it & 1, abort_flag, p.err, DEV_TIMEOUT_MMA);
          if (!ok) break;
          tc_fence_after();
          const int s = (2 * it + x) % kQdStages;
          const uint64_t bq = dqm0 + s * (2 * kChunk >> 4);
          mma_tm<4, 32>(tmem + 256, tmem + 64 * x, bq + (kChunk >> 4), id, it > 0 || x > 0);
          mma_tm<4, 32>(tmem + 384, tmem + 128 + 64 * x, bq, id, it > 0 || x > 0);
          if (FINE) mma_tm<4, 32>(tmem + 384, tmem + 144 + 64 * x, bq, id, true);
          umma_commit(&pd_done[x]);
          umma_commit(&qd_empty[s]);
        }
      }
      umma_commit(&drain[2]);
      mbar_wait(&drain[2], 0, nullptr, p.err, DEV_TIMEOUT_DRAIN);
    }
    if (p.split == 2) {  // see the end of the compute warps
      __syncwarp();
      cluster_barrier();
      cluster_barrier();
    }
  } else {
    if (kWarps == 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // x: buffer, half of each query tile; c0: first 32 columns of it
    const int quarter = warp & 3, x = (warp - 4) / (kWarps / 2), c0 = kCols == 1 ? ((warp - 4) >> 2) & 1 : 0;
    const int r = quarter * 32 + lane;                  // key row of the tile
    const int kpos = kt * kTile + r;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + 64 * x, dp_tm = s_tm + 128;
    bool ok = plan_ok;
    for (int it = 0; ok && it < n_it; ++it) {
      const int qt0 = it_qtile(it) * kTile + 64 * x;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&rows_full[x], it & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE) &&
                                       mbar_wait_soon(&sd_full[x], it & 1, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
      if (!ok) break;
      tc_fence_after();
      const bool part = !s_whole[x];
      const float slope = BIAS ? p.slopes[it_head(it)] * kLog2e : 0.f;
      const int side = qt0 >= kt * kTile + 32 * quarter + 31 ? -1 : 0;
#pragma unroll 1
      for (int c = c0; c < c0 + kCols; ++c) {
        uint32_t sv[32], dp[32], pw[16], dw[FINE ? 32 : 16];
        tmem_ld32(s_tm + 32 * c, sv);
        tmem_ld32(dp_tm + 32 * c, dp);
        tmem_ld_wait_regs(sv);
        regs_after_wait(dp);
        const int col = 64 * x + 32 * c;
        uint32_t see = 0xffffffffu;
        if (part) {
          see = 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int2 w = s_see[col + e];
            see |= (uint32_t)(w.x <= kpos && kpos < w.y) << e;
          }
        }
        grad32<CAP, BIAS, false, true, FINE>(sv, dp, p.mul, p.cap_mul, slope, (float)(kpos - qt0 - 32 * c), side, part, see, 0.f,
                                       0.f, s_lse + col, s_del + col, pw, dw);
        tmem_st16(s_tm + 32 * c, pw);  // over the scores and products that this warp itself has read
        if constexpr (FINE) tmem_st32(dp_tm + 32 * c, dw);
        else tmem_st16(dp_tm + 32 * c, dw);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&pd_full[x], lane);
      if (lane == 0) mbar_arrive(&rows_empty[x]);
    }
    // dV (first group), dK (second) once every product is done
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_soon(&drain[2], 0, abort_flag, p.err, DEV_TIMEOUT_EPILOGUE));
    // Two CTAs: the first finishes dV, the second dK; each sends the other one's share, fp32, to the other's stages of Q and dO,
    // which nothing reads any more.
    const uint32_t acc_tm = tmem + lane_off + 256 + 128 * x;
    float* share = reinterpret_cast<float*>(sqd);  // [column][row]
    if (p.split == 2) {
      __syncwarp();
      cluster_barrier();
      if (x != rank) {
        const uint32_t to = peer_address(smem_u32(share), rank ^ 1) + 4 * r;
        tc_fence_after();
#pragma unroll 1
        for (int k = c0; k < 2 * nd; k += kCols == 1 ? 2 : 1) {
          uint32_t v[32];
          tmem_ld32(acc_tm + 32 * k, v);
          tmem_ld_wait_regs(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) st_peer(to + (32 * k + e) * 512, n_it ? v[e] : 0u);
        }
      }
      cluster_barrier();
    }
    if (ok && (p.split == 1 || x == rank)) {
      tc_fence_after();
      const int64_t row0 = (int64_t)b * p.S + kt * kTile + 32 * quarter;
      const int n_rows = p.S - kt * kTile - 32 * quarter;
      const int64_t ld = x ? p.lddk : p.lddv;
      __nv_bfloat16* out = (x ? p.dk : p.dv) + row0 * ld + (int64_t)g * p.hd;
      const float mul = x ? p.scale : 1.f;
#pragma unroll 1
      for (int k = c0; k < 2 * nd; k += kCols == 1 ? 2 : 1) {
        uint32_t v[32], w[16];
        tmem_ld32(acc_tm + 32 * k, v);
        tmem_ld_wait_regs(v);
        if (p.split == 2) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float other = share[(32 * k + e) * 128 + r];
            v[e] = __float_as_uint(n_it ? __uint_as_float(v[e]) + other : other);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) w[e / 2] = pack2(__uint_as_float(v[e]) * mul, __uint_as_float(v[e + 1]) * mul);
        store_rows32(out + 32 * k, ld, w, n_rows, p.hd - 32 * k);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------- host side

// Shared memory of a launch: sized for head_dim 128 whatever the head dimension, which also keeps
// one CTA per SM (each CTA allocates all 512 TMEM columns).
int fwd_smem() { return 1024 + 12 * kChunk + 256; }
int dq_smem() { return 14 * kChunk + 2048 + 256; }
int dkv_smem() { return 14 * kChunk + 2048 + 16 + 256; }

// Raises a kernel's shared-memory limit once per device.
template <typename K>
bool smem_limit(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

template <bool CAP, bool BIAS>
int fwd_launch(const MaskedFwdParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  if (!smem_limit(masked_fwd_kernel<CAP, BIAS>, fwd_smem(), done)) return 5;
  const int n_sm = sm_count();
  if (n_sm <= 0) return 5;
  launch_kernel(masked_fwd_kernel<CAP, BIAS>, (unsigned)std::min(p.n_units, n_sm), kFwdThreads, fwd_smem(), s, p);
  if (launch_failed("sl_attention_masked")) return 5;
  note_launch();
  return 0;
}

template <bool CAP, bool BIAS, bool FINE>
int bwd_launch(const MaskedBwdParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done_q{0}, done_kv{0};
  if (!smem_limit(masked_dq_kernel<CAP, BIAS, FINE>, dq_smem(), done_q) ||
      !smem_limit(masked_dkv_kernel<CAP, BIAS, FINE>, dkv_smem(), done_kv))
    return 5;
  const int n_sm = sm_count();
  if (n_sm <= 0) return 5;
  launch_kernel(masked_dq_kernel<CAP, BIAS, FINE>, (unsigned)std::min(p.n_units, n_sm), kBwdThreads, dq_smem(), s, p);
  if (launch_failed("sl_attention_masked")) return 5;
  note_launch();
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan_tiles(p.n_seq, p.S) * p.hkv * p.split));
  cfg.blockDim = dim3(kDkvThreads<CAP>);
  cfg.dynamicSmemBytes = dkv_smem();
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  cudaLaunchKernelEx(&cfg, masked_dkv_kernel<CAP, BIAS, FINE>, p);
  if (launch_failed("sl_attention_masked")) return 5;
  note_launch();
  return 0;
}
template <bool CAP, bool BIAS>
int bwd_launch(const MaskedBwdParams& p, cudaStream_t s) {
  return fine_grads(p.hd, p.S) ? bwd_launch<CAP, BIAS, true>(p, s) : bwd_launch<CAP, BIAS, false>(p, s);
}

}  // namespace

void masked_score_constants(float scale, float cap, int hd, float* sc, float* mul, float* cap_mul) {
  const double s = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)hd);
  *sc = (float)s;
  *mul = (float)(1.4426950408889634 * (cap > 0.f ? (double)cap : s));
  *cap_mul = cap > 0.f ? (float)(s / cap) : 0.f;
}

int64_t attention_plan_bytes(int n_seq, int S) { return carve_plan(nullptr, n_seq, S, nullptr); }

int attention_plan(const int32_t* row_lo, const int32_t* row_hi, int n_seq, int S, void* plan, cudaStream_t s) {
  Plan p;
  carve_plan(plan, n_seq, S, &p);
  const int64_t tiles = plan_tiles(n_seq, S);
  if (tiles <= kPlanSmall) {
    launch_kernel(plan_small_kernel, 1u, kPlanThreads, 0, s, p, row_lo, row_hi, n_seq, S);
    if (launch_failed("sl_attention_plan")) return 5;
    note_launch();
    return 0;
  }
  launch_kernel(plan_rows_kernel, (unsigned)std::min<int64_t>((tiles + 31) / 32, 148), kPlanThreads, 0, s, p, row_lo, row_hi,
                n_seq, S);
  if (launch_failed("sl_attention_plan")) return 5;
  note_launch();
  launch_kernel(plan_tiles_kernel, 1u, kPlanThreads, ((size_t)(S + kTile - 1) / kTile + 2) * 4, s, p, n_seq, S);
  if (launch_failed("sl_attention_plan")) return 5;
  note_launch();
  return 0;
}

int attention_masked_fwd(const MaskedArgs& a, cudaStream_t s) {
  MaskedFwdParams p;
  memset(&p, 0, sizeof(p));
  if (!head_map(&p.qmap, a.q, a.ldq, a.n_seq, a.S, a.hq, a.hd) || !head_map(&p.kmap, a.k, a.ldk, a.n_seq, a.S, a.hkv, a.hd) ||
      !head_map(&p.vmap, a.v, a.ldv, a.n_seq, a.S, a.hkv, a.hd))
    return 2;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.ldo = a.ldo;
  const bool pairs = (a.hq / a.hkv) % 2 == 0;
  const int n_t = (a.S + kTile - 1) / kTile;
  // as few units as SMs: each stream has one to itself (3 x 333 tokens, 6 heads: 16.6 against 20 us)
  p.kind = (int64_t)a.n_seq * n_t * a.hq <= sm_count() ? kAlone : pairs ? kTwoHeads : kTwoTiles;
  p.n_units = p.kind == kTwoTiles ? a.n_seq * ((n_t + 1) / 2) * a.hq : a.n_seq * n_t * (p.kind == kTwoHeads ? a.hq / 2 : a.hq);
  carve_plan(const_cast<void*>(a.plan), a.n_seq, a.S, &p.plan);
  p.slopes = a.slopes;
  p.lse = const_cast<float*>(a.lse);
  p.n_seq = a.n_seq;
  p.S = a.S;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.hd = a.hd;
  p.nd = (a.hd + 63) / 64;
  float scale;
  masked_score_constants(a.scale, a.cap, a.hd, &scale, &p.mul, &p.cap_mul);
  p.err = a.err;
  if (a.cap > 0.f) return a.slopes ? fwd_launch<true, true>(p, s) : fwd_launch<true, false>(p, s);
  return a.slopes ? fwd_launch<false, true>(p, s) : fwd_launch<false, false>(p, s);
}

size_t attention_masked_scratch(int n_seq, int S, int hq) { return (size_t)n_seq * S * hq * 4; }

int attention_masked_bwd(const MaskedArgs& a, cudaStream_t s) {
  MaskedBwdParams p;
  memset(&p, 0, sizeof(p));
  if (!head_map(&p.qmap, a.q, a.ldq, a.n_seq, a.S, a.hq, a.hd) || !head_map(&p.kmap, a.k, a.ldk, a.n_seq, a.S, a.hkv, a.hd) ||
      !head_map(&p.vmap, a.v, a.ldv, a.n_seq, a.S, a.hkv, a.hd) || !head_map(&p.domap, a.d_o, a.lddo, a.n_seq, a.S, a.hq, a.hd) ||
      !head_map(&p.qmap64, a.q, a.ldq, a.n_seq, a.S, a.hq, a.hd, 64) ||
      !head_map(&p.domap64, a.d_o, a.lddo, a.n_seq, a.S, a.hq, a.hd, 64))
    return 2;
  carve_plan(const_cast<void*>(a.plan), a.n_seq, a.S, &p.plan);
  p.slopes = a.slopes;
  p.lse = a.lse;
  p.delta = static_cast<float*>(a.scratch);
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.lddq = a.lddq;
  p.lddk = a.lddk;
  p.lddv = a.lddv;
  p.n_seq = a.n_seq;
  p.S = a.S;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.hd = a.hd;
  p.nd = (a.hd + 63) / 64;
  p.n_units = (int)(plan_tiles(a.n_seq, a.S) * a.hq);
  // units that leave half of the SMs free are shared by two CTAs each (3 x 333 tokens, 27 units: 20.3 against 28.6 us; one
  // key tile, two steps: 9.9 against 10.3)
  p.split = 2 * plan_tiles(a.n_seq, a.S) * a.hkv <= sm_count() ? 2 : 1;
  masked_score_constants(a.scale, a.cap, a.hd, &p.scale, &p.mul, &p.cap_mul);
  p.err = a.err;
  if (a.cap > 0.f) return a.slopes ? bwd_launch<true, true>(p, s) : bwd_launch<true, false>(p, s);
  return a.slopes ? bwd_launch<false, true>(p, s) : bwd_launch<false, false>(p, s);
}

}  // namespace sl
