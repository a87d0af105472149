// Per-head RMSNorm of q and k with gains, and the position rotation, in one pass over both,
// forward and backward. For a head's row x of hd elements at position p:
//   n = x * rstd * g, rstd = 1 / sqrt(mean(x^2) + eps);  (a, b) the members of rotated pair i:
//   y_a = n_a cos(p f_i) - n_b sin(p f_i),  y_b = n_b cos(p f_i) + n_a sin(p f_i);  the rest: y = n.
// Backward: dn = (rotation by -p f_i) dy;  dg = sum over rows of dn x rstd;
//   dx = rstd (g dn) - x rstd^3 mean_j(x_j g_j dn_j).
//
// Both passes move each element once and are bound by memory. A warp takes one token and a share of
// its heads; a group of lanes holds one head, each lane two vectors of it that contain both
// members of its pairs, so the rotation needs no exchange and the norm one short shuffle sum. The
// token's cosines and sines are computed once per warp and serve all its heads.
// Angles: p f_i in turns as a 64-bit fraction (f_i / 2 pi scaled by 2^64, times p, wrapping), so
// far positions lose nothing to the range reduction; one rounding to fp32 before sincospi.
#include <cuda_bf16.h>

#include <algorithm>

#include "sl_internal.h"

namespace sl {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotWarps = kRotThreads / 32;

struct RotParams {
  const __nv_bfloat16 *xq, *xk;    // inputs (backward: the forward's inputs; null without the norm)
  const __nv_bfloat16 *dyq, *dyk;  // backward: gradients of the outputs
  __nv_bfloat16 *oq, *ok;          // outputs (backward: gradients of the inputs)
  int64_t ldxq, ldxk, lddq, lddk, ldoq, ldok;
  const int32_t* pos;
  const float* inv_freq;
  const __nv_bfloat16 *gq, *gk;  // gains (null without the norm)
  float* partial;                // [gridDim.x][2][hd] sums of dg (backward with gain gradients)
  float eps, inv_hd, sign;       // sign: +1 forward, -1 backward
  int64_t n_tok;
  int32_t hq, hkv, hd, rot, group, split;
};

template <int V>
struct Raw {
  uint32_t w[V / 2];
};
template <int V>
__device__ __forceinline__ void ld_raw(Raw<V>& r, const __nv_bfloat16* p) {
  if constexpr (V == 8) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    r.w[0] = t.x; r.w[1] = t.y; r.w[2] = t.z; r.w[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    r.w[0] = t.x; r.w[1] = t.y;
  }
}
template <int V>
__device__ __forceinline__ void st_raw(__nv_bfloat16* p, const Raw<V>& r) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}
template <int V>
__device__ __forceinline__ void widen(const Raw<V>& r, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    f[2 * i] = __uint_as_float(r.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
template <int V>
__device__ __forceinline__ void narrow(Raw<V>& r, const float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// f / (2 pi) as a fraction of a turn in 64 bits; ok = false for a frequency that is not finite.
__device__ __forceinline__ uint64_t turn_step(float f, bool& ok) {
  double t = (double)f * 0.15915494309189533576888;
  ok = f - f == 0.f;
  t -= floor(t);
  return ok ? (uint64_t)__double2ull_rz(t * 18446744073709551616.0) : 0;
}

// V: elements per vector (8, or 4 where half the rotated width is no multiple of 8). PAIRS: pair i
// is (2 i, 2 i + 1), else (i, i + rot / 2). BWD: the norm's backward (without the norm the backward
// is the forward kernel with the sign of the sines turned).
template <int V, bool NORM, bool PAIRS, bool BWD>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (p.group - 1), gi = lane / p.group, n_groups = 32 / p.group;
  // this lane's two vectors of a head
  const int half = p.rot >> 1;
  int off0, off1;
  bool on0, on1, turn0, turn1;
  if (PAIRS) {
    off0 = 2 * V * sub;
    off1 = off0 + V;
    on0 = off0 < p.hd;
    on1 = off1 < p.hd;
    turn0 = off0 < p.rot;
    turn1 = off1 < p.rot;
  } else {
    const int n_pair = half / V;
    turn0 = turn1 = sub < n_pair;
    off0 = turn0 ? V * sub : p.rot + 2 * V * (sub - n_pair);
    off1 = turn0 ? off0 + half : off0 + V;
    on0 = off0 < p.hd;
    on1 = off1 < p.hd;
  }
  // the lane's V pairs: pair index, step in turns
  uint64_t step[V];
  bool fine[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int i = PAIRS ? (e < V / 2 ? off0 : off1) / 2 + e % (V / 2) : off0 + e;
    const bool t = PAIRS ? (e < V / 2 ? turn0 : turn1) : turn0;
    step[e] = turn_step(t ? p.inv_freq[i] : 0.f, fine[e]);
  }
  const int nh = p.hq + p.hkv;
  const int per = (nh + p.split - 1) / p.split;
  float dgq[NORM && BWD ? 2 * V : 1], dgk[NORM && BWD ? 2 * V : 1];
  if constexpr (NORM && BWD) {
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) dgq[e] = dgk[e] = 0.f;
  }
  const int64_t n_items = p.n_tok * p.split;
  for (int64_t item = (int64_t)blockIdx.x * kRotWarps + warp; item < n_items; item += (int64_t)gridDim.x * kRotWarps) {
    const int64_t tok = item / p.split;
    const int h0 = (int)(item % p.split) * per, h1 = min(nh, h0 + per);
    float cs[V], sn[V];
    if (p.rot > 0) {
      const int64_t pos = p.pos[tok];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float turns = (float)(int64_t)(step[e] * (uint64_t)pos) * 5.421010862427522e-20f;  // 2^-64
        sincospif(2.f * turns, &sn[e], &cs[e]);
        sn[e] *= p.sign;
        if (!fine[e]) cs[e] = sn[e] = __int_as_float(0x7fffffff);
      }
    }
    for (int h = h0 + gi; h < h1 + gi; h += n_groups) {  // the same trips for every group of the warp
      const bool live = h < h1;
      const bool is_q = h < p.hq;
      const int hh = is_q ? h : h - p.hq;
      const int64_t at = (int64_t)hh * p.hd;
      const bool l0 = live && on0, l1 = live && on1;
      Raw<V> r0, r1;
      float x0[V], x1[V], y0[V], y1[V];
#pragma unroll
      for (int e = 0; e < V; ++e) x0[e] = x1[e] = y0[e] = y1[e] = 0.f;
      float rs = 1.f;
      if (!BWD || NORM) {
        const __nv_bfloat16* x = (is_q ? p.xq + tok * p.ldxq : p.xk + tok * p.ldxk) + at;
        if (l0) { ld_raw(r0, x + off0); widen(r0, x0); }
        if (l1) { ld_raw(r1, x + off1); widen(r1, x1); }
      }
      float g0[V], g1[V];
      if constexpr (NORM) {
        const __nv_bfloat16* g = is_q ? p.gq : p.gk;
#pragma unroll
        for (int e = 0; e < V; ++e) g0[e] = g1[e] = 0.f;
        if (on0) { ld_raw(r0, g + off0); widen(r0, g0); }
        if (on1) { ld_raw(r1, g + off1); widen(r1, g1); }
      }
      if constexpr (BWD) {
        const __nv_bfloat16* dy = (is_q ? p.dyq + tok * p.lddq : p.dyk + tok * p.lddk) + at;
        if (l0) { ld_raw(r0, dy + off0); widen(r0, y0); }
        if (l1) { ld_raw(r1, dy + off1); widen(r1, y1); }
      }
      if constexpr (NORM && !BWD) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
        for (int o = p.group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * p.inv_hd + p.eps);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y0[e] = x0[e] * rs * g0[e];
          y1[e] = x1[e] * rs * g1[e];
        }
      }
      if constexpr (!NORM && !BWD) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y0[e] = x0[e];
          y1[e] = x1[e];
        }
      }
      // the rotation of (y0, y1)
      if (PAIRS) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          if (turn0) {
            const float a = y0[2 * e], b = y0[2 * e + 1];
            y0[2 * e] = a * cs[e] - b * sn[e];
            y0[2 * e + 1] = b * cs[e] + a * sn[e];
          }
          if (turn1) {
            const float a = y1[2 * e], b = y1[2 * e + 1];
            y1[2 * e] = a * cs[V / 2 + e] - b * sn[V / 2 + e];
            y1[2 * e + 1] = b * cs[V / 2 + e] + a * sn[V / 2 + e];
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float a = y0[e], b = y1[e];
          y0[e] = a * cs[e] - b * sn[e];
          y1[e] = b * cs[e] + a * sn[e];
        }
      }
      if constexpr (NORM && BWD) {
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
          dot = fmaf(x0[e], g0[e] * y0[e], fmaf(x1[e], g1[e] * y1[e], dot));
        }
        for (int o = p.group >> 1; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        rs = rsqrtf(ss * p.inv_hd + p.eps);
        if (live) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float a = y0[e] * x0[e] * rs, b = y1[e] * x1[e] * rs;
            if (is_q) { dgq[e] += a; dgq[V + e] += b; }
            else { dgk[e] += a; dgk[V + e] += b; }
          }
        }
        const float c = rs * rs * dot * p.inv_hd;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y0[e] = rs * (g0[e] * y0[e] - x0[e] * c);
          y1[e] = rs * (g1[e] * y1[e] - x1[e] * c);
        }
      }
      __nv_bfloat16* o = (is_q ? p.oq + tok * p.ldoq : p.ok + tok * p.ldok) + at;
      if (l0) { narrow(r0, y0); st_raw(o + off0, r0); }
      if (l1) { narrow(r1, y1); st_raw(o + off1, r1); }
    }
  }
  if constexpr (NORM && BWD) {
    if (p.partial) {
      // every group of the block adds its share in a fixed order: [warp and group][2][hd]
      extern __shared__ float s_dg[];
      float* mine = s_dg + (size_t)(warp * n_groups + gi) * 2 * p.hd;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (on0) { mine[off0 + e] = dgq[e]; mine[p.hd + off0 + e] = dgk[e]; }
        if (on1) { mine[off1 + e] = dgq[V + e]; mine[p.hd + off1 + e] = dgk[V + e]; }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * p.hd; c += kRotThreads) {
        float s = 0.f;
        for (int w = 0; w < kRotWarps * n_groups; ++w) s += s_dg[(size_t)w * 2 * p.hd + c];
        p.partial[(int64_t)blockIdx.x * 2 * p.hd + c] = s;
      }
    }
  }
}

// dg[c] = sum over the blocks' partials, 32 columns per block; 32 interleaved sums per column, then
// one tree: a fixed order.
__global__ void __launch_bounds__(1024) rotary_gain_kernel(const float* __restrict__ partial, int n_part, int hd,
                                                          float* __restrict__ dgq, float* __restrict__ dgk) {
  pdl_wait();
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float v = 0.f;
  if (c < 2 * hd)
    for (int i = r; i < n_part; i += 32) v += partial[(int64_t)i * 2 * hd + c];
  s[r][threadIdx.x & 31] = v;
  __syncthreads();
  v = s[threadIdx.x & 31][r];  // lane = partial sum, warp = column
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + r;
  if ((threadIdx.x & 31) == 0 && col < 2 * hd) {
    float* out = col < hd ? dgq : dgk;
    if (out) out[col < hd ? col : col - hd] = v;
  }
}

template <int V, bool NORM, bool BWD>
auto pick_style(bool pairs) {
  return pairs ? rotary_kernel<V, NORM, true, BWD> : rotary_kernel<V, NORM, false, BWD>;
}

// Blocks of a launch: enough to fill the SMs, tokens strided over them.
int64_t rot_blocks(int64_t n_items) { return std::min<int64_t>((n_items + kRotWarps - 1) / kRotWarps, 148 * 8); }

}  // namespace

int64_t rotary_partial_floats(int64_t n_tok, int hd) {
  return std::min<int64_t>(rot_blocks(n_tok * 64), 148 * 8) * 2 * hd;
}

int rotary(const RotaryArgs& a, cudaStream_t s) {
  RotParams p = {};
  const bool norm = a.gq != nullptr, bwd = a.dyq != nullptr && norm;
  p.xq = static_cast<const __nv_bfloat16*>(a.dyq && !norm ? a.dyq : a.xq);
  p.xk = static_cast<const __nv_bfloat16*>(a.dyq && !norm ? a.dyk : a.xk);
  p.ldxq = a.dyq && !norm ? a.lddq : a.ldxq;
  p.ldxk = a.dyq && !norm ? a.lddk : a.ldxk;
  p.dyq = static_cast<const __nv_bfloat16*>(a.dyq);
  p.dyk = static_cast<const __nv_bfloat16*>(a.dyk);
  p.lddq = a.lddq;
  p.lddk = a.lddk;
  p.oq = static_cast<__nv_bfloat16*>(a.oq);
  p.ok = static_cast<__nv_bfloat16*>(a.ok);
  p.ldoq = a.ldoq;
  p.ldok = a.ldok;
  p.pos = a.pos;
  p.inv_freq = a.inv_freq;
  p.gq = static_cast<const __nv_bfloat16*>(a.gq);
  p.gk = static_cast<const __nv_bfloat16*>(a.gk);
  p.eps = a.eps;
  p.inv_hd = 1.f / (float)a.hd;
  p.sign = a.dyq ? -1.f : 1.f;
  p.n_tok = a.n_tok;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.hd = a.hd;
  p.rot = a.rot;
  const int V = a.pairs || a.rot % 16 == 0 ? 8 : 4;
  // lanes per head: one slot of two vectors each
  const int slots = a.pairs ? (a.hd + 2 * V - 1) / (2 * V) : a.rot / 2 / V + (a.hd - a.rot + 2 * V - 1) / (2 * V);
  int group = 1;
  while (group < slots) group *= 2;
  p.group = group;
  // few tokens: the heads of a token are spread over several warps
  const int nh = a.hq + a.hkv, n_groups = 32 / group;
  int split = 1;
  while (split * n_groups < nh && a.n_tok * split < 148 * 16) split *= 2;
  p.split = std::min(split, 64);
  const int64_t grid = rot_blocks(a.n_tok * p.split);
  const bool gains = bwd && (a.dgq || a.dgk);
  p.partial = gains ? a.partial : nullptr;
  const size_t smem = gains ? (size_t)kRotWarps * n_groups * 2 * a.hd * 4 : 0;
  auto kernel = V == 8 ? (norm ? (bwd ? pick_style<8, true, true>(a.pairs) : pick_style<8, true, false>(a.pairs))
                               : pick_style<8, false, false>(a.pairs))
                       : (norm ? (bwd ? rotary_kernel<4, true, false, true> : rotary_kernel<4, true, false, false>)
                               : rotary_kernel<4, false, false, false>);
  launch_kernel(kernel, (unsigned)grid, kRotThreads, smem, s, p);
  if (launch_failed("sl_qk_norm_rope")) return 5;
  note_launch();
  if (gains) {
    launch_kernel(rotary_gain_kernel, (unsigned)((2 * a.hd + 31) / 32), 1024, 0, s, (const float*)a.partial, (int)grid,
                  a.hd, a.dgq, a.dgk);
    if (launch_failed("sl_qk_norm_rope")) return 5;
    note_launch();
  }
  return 0;
}

}  // namespace sl
