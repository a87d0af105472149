// Per-head RMSNorm of q and k with gains, and the position rotation, in one pass over both,
// forward and backward. For a head's row x of hd elements at position p:
//   n = x * rstd * g, rstd = 1 / sqrt(mean(x^2) + eps);  (a, b) the members of rotated pair i:
//   y_a = n_a cos(p f_i) - n_b sin(p f_i),  y_b = n_b cos(p f_i) + n_a sin(p f_i);  the rest: y = n.
// Backward: dn = (rotation by -p f_i) dy;  dg = sum over rows of dn x rstd;
//   dx = rstd (g dn) - x rstd^3 mean_j(x_j g_j dn_j).
//
// Both passes move each element once and are bound by memory. A warp takes tokens in turn, and of each the heads of q
// or of k; a group of lanes holds one head, each lane two vectors of it that contain both members of its
// pairs, so the rotation needs no exchange and the norm one short shuffle sum. The token's cosines and sines are
// computed a pair per lane and serve all its heads through shared memory; the next heads' vectors are on their way
// meanwhile. (One block per token, each lane one head: 400 of 616 instructions a warp went into set-up, and the
// forward was bound by issue at 1.8 TB/s.) Blocks of q stand before blocks of k.
// Measured beside library copies of the same bytes: rotation of 4096 tokens of 40 heads of 128 (84 MB) 18.6 us, a copy 15.0;
// norm and rotation of 20011 tokens of 30 heads of 96 (231 MB) 57, a copy 41.5; its backward (346 MB) 97, a sum of two tensors
// 51.5. The vectors in flight are held in registers (64, 72 and 125 to 128 a thread); in the forward with norm the sum and
// the products with gains stand between a vector's arrival and its store, and issue slots are three quarters full.
// Angles: p f_i in turns as a 64-bit fraction (f_i / 2 pi scaled by 2^64, times p, wrapping), so
// far positions lose nothing to the range reduction; one rounding to fp32 before sincospi.
#include <cuda_bf16.h>

#include <algorithm>

#include "sl_packed.h"

namespace sl {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotMaxPairs = 128;  // of a head: head_dim <= 256

struct RotSide {
  const __nv_bfloat16* x;   // inputs (backward: the forward's inputs; not read without the norm)
  const __nv_bfloat16* dy;  // backward: gradients of the outputs
  __nv_bfloat16* o;         // outputs (backward: gradients of the inputs)
  const __nv_bfloat16* g;   // gains
  int64_t ldx, lddy, ldo;
  int32_t heads;
  int32_t trips, split;     // trips of a warp over a token's heads, and the warps that share them
  int32_t blocks;
};

struct RotParams {
  RotSide side[2];  // q, k
  const int32_t* pos;
  const float* inv_freq;
  float* partial;   // [q's blocks, then k's][hd] sums of dg (backward with gain gradients)
  float eps, inv_hd, sign;  // sign: +1 forward, -1 backward
  int64_t n_tok;
  int32_t hd, rot, group;
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

// Blocks that an SM holds at once: what is in flight bounds the kernel, so as many as leave no register spilled (rotation
// alone, 4096 tokens: 18.7 us with 8 against 20.3 with 6; forward with norm, 20011 tokens: 57 with 7 against 60 with 6,
// 75 with 8; backward: 96 with 4 against 117 with 3, 199 with 5).
constexpr int rot_blocks_per_sm(bool norm, bool bwd) { return bwd ? 4 : norm ? 7 : 8; }

// V: elements per vector (8, or 4 where half the rotated width is no multiple of 8). PAIRS: pair i
// is (2 i, 2 i + 1), else (i, i + rot / 2). BWD: the norm's backward (without the norm the backward
// is the forward kernel with the sign of the sines turned).
template <int V, bool NORM, bool PAIRS, bool BWD>
__global__ void __launch_bounds__(kRotThreads, rot_blocks_per_sm(NORM, BWD)) rotary_kernel(const __grid_constant__ RotParams p) {
  __shared__ uint64_t s_step[kRotMaxPairs];              // a pair's angle per position; bit 0: not finite
  __shared__ float2 s_turn[kRotWarps][kRotMaxPairs];     // the warp's token: (cos, sin) per pair
  extern __shared__ float s_dg[];                        // at the end the groups' sums of dg
  pdl_wait();
  const bool is_k = blockIdx.x >= (unsigned)p.side[0].blocks;
  const RotSide& sd = p.side[is_k];
  const int block = blockIdx.x - (is_k ? p.side[0].blocks : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (p.group - 1), gi = lane / p.group, n_groups = 32 / p.group;
  const int half = p.rot >> 1;
  // this lane's two vectors of a head
  int off0, off1;
  bool turn0, turn1;
  if (PAIRS) {
    off0 = 2 * V * sub;
    off1 = off0 + V;
    turn0 = off0 < p.rot;
    turn1 = off1 < p.rot;
  } else {
    const int n_pair = half / V;
    turn0 = turn1 = sub < n_pair;
    off0 = turn0 ? V * sub : p.rot + 2 * V * (sub - n_pair);
    off1 = turn0 ? off0 + half : off0 + V;
  }
  const bool on0 = off0 < p.hd, on1 = off1 < p.hd;
  Raw<V> gr0 = {}, gr1 = {};
  if constexpr (NORM) {
    if (on0) ld_raw(gr0, sd.g + off0);
    if (on1) ld_raw(gr1, sd.g + off1);
  }
  float dg[NORM && BWD ? 2 * V : 1];
  if constexpr (NORM && BWD) {
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) dg[e] = 0.f;
  }
  // raw vectors of this trip, then of the next (two trips ahead gained nothing)
  struct Head {
    Raw<V> x0, x1, d0, d1;
  };
  Head raw = {};
  auto fetch = [&](int64_t tok, int trip, Head& r) {
    const int h = trip * n_groups + gi;
    if (h >= sd.heads) return;
    if (!BWD || NORM) {
      const __nv_bfloat16* x = sd.x + tok * sd.ldx + (int64_t)h * p.hd;
      if (on0) ld_raw(r.x0, x + off0);
      if (on1) ld_raw(r.x1, x + off1);
    }
    if constexpr (BWD) {
      const __nv_bfloat16* dy = sd.dy + tok * sd.lddy + (int64_t)h * p.hd;
      if (on0) ld_raw(r.d0, dy + off0);
      if (on1) ld_raw(r.d1, dy + off1);
    }
  };
  // items: (token, share of its trips)
  const int64_t n_items = p.n_tok * sd.split, stride = (int64_t)sd.blocks * kRotWarps;
  const int per = (sd.trips + sd.split - 1) / sd.split;
  int64_t item = (int64_t)block * kRotWarps + warp;
  int64_t tok = item / sd.split;
  int trip = (int)(item % sd.split) * per;
  int pos = 0;
  if (item < n_items) {
    fetch(tok, trip, raw);
    if (half) pos = p.pos[tok];
  }
  for (int i = threadIdx.x; i < half; i += kRotThreads) {
    bool fine;
    const uint64_t f = turn_step(p.inv_freq[i], fine) & ~1ull;
    s_step[i] = fine ? f : 1ull;
  }
  __syncthreads();
  for (; item < n_items; item += stride) {
    const int64_t next = item + stride, tok_next = next / sd.split;
    const int trip_next = (int)(next % sd.split) * per;
    const int end = min(sd.trips, trip + per);
    if (half) {
      __syncwarp();  // the last token's table has been read
      for (int i = lane; i < half; i += 32) {
        const uint64_t f = s_step[i];
        float2 v;
        sincospif(2.f * ((float)(int64_t)(f * (uint64_t)(int64_t)pos) * 5.421010862427522e-20f), &v.y, &v.x);  // 2^-64
        v.y *= p.sign;
        if (f & 1) v.x = v.y = __int_as_float(0x7fffffff);
        s_turn[warp][i] = v;
      }
      __syncwarp();
      if (next < n_items) pos = p.pos[tok_next];
    }
    const float2* mine = s_turn[warp];
    for (; trip < end; ++trip) {
      const int h = trip * n_groups + gi;
      const bool live = h < sd.heads;
      float x0[V], x1[V], y0[V], y1[V];
      widen(raw.x0, x0);
      widen(raw.x1, x1);
      if constexpr (BWD) {
        widen(raw.d0, y0);
        widen(raw.d1, y1);
      }
      if (trip + 1 < end) fetch(tok, trip + 1, raw);
      else if (next < n_items) fetch(tok_next, trip_next, raw);
      float rs = 1.f;
      if constexpr (NORM && !BWD) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
        for (int o = p.group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * p.inv_hd + p.eps);
        float g[V];
        widen(gr0, g);
#pragma unroll
        for (int e = 0; e < V; ++e) y0[e] = x0[e] * rs * g[e];
        widen(gr1, g);
#pragma unroll
        for (int e = 0; e < V; ++e) y1[e] = x1[e] * rs * g[e];
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
            const float2 t = mine[off0 / 2 + e];
            const float a = y0[2 * e], b = y0[2 * e + 1];
            y0[2 * e] = a * t.x - b * t.y;
            y0[2 * e + 1] = b * t.x + a * t.y;
          }
          if (turn1) {
            const float2 t = mine[off1 / 2 + e];
            const float a = y1[2 * e], b = y1[2 * e + 1];
            y1[2 * e] = a * t.x - b * t.y;
            y1[2 * e + 1] = b * t.x + a * t.y;
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 t = mine[off0 + e];
          const float a = y0[e], b = y1[e];
          y0[e] = a * t.x - b * t.y;
          y1[e] = b * t.x + a * t.y;
        }
      }
      if constexpr (NORM && BWD) {
        // y is dn here
        float ss = 0.f, dot = 0.f;
        float g0[V], g1[V];
        widen(gr0, g0);
        widen(gr1, g1);
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
        if (live && p.partial) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dg[e] += y0[e] * x0[e] * rs;
            dg[V + e] += y1[e] * x1[e] * rs;
          }
        }
        const float c = rs * rs * dot * p.inv_hd;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y0[e] = rs * (g0[e] * y0[e] - x0[e] * c);
          y1[e] = rs * (g1[e] * y1[e] - x1[e] * c);
        }
      }
      if (live) {
        __nv_bfloat16* o = sd.o + tok * sd.ldo + (int64_t)h * p.hd;
        Raw<V> w;
        if (on0) { narrow(w, y0); st_raw(o + off0, w); }
        if (on1) { narrow(w, y1); st_raw(o + off1, w); }
      }
    }
    tok = tok_next;
    trip = trip_next;
  }
  if constexpr (NORM && BWD) {
    if (p.partial) {
      // every group of the block adds its share in a fixed order: [group][hd]
      float* out = s_dg + (size_t)(threadIdx.x / p.group) * p.hd;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (on0) out[off0 + e] = dg[e];
        if (on1) out[off1 + e] = dg[V + e];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.hd; c += kRotThreads) {
        float v = 0.f;
        for (int w = 0; w < kRotThreads / p.group; ++w) v += s_dg[(size_t)w * p.hd + c];
        p.partial[(int64_t)blockIdx.x * p.hd + c] = v;
      }
    }
  }
}

// dg[c] = sum over the blocks' partials: rows [0, n_q) for q, [n_q, n_q + n_k) for k (blockIdx.y), eight columns (32
// bytes) per block; 128 interleaved sums per column, then one tree: a fixed order.
constexpr int kGainCols = 8;
__global__ void __launch_bounds__(1024) rotary_gain_kernel(const float* __restrict__ partial, int n_q, int n_k, int hd,
                                                          float* __restrict__ dgq, float* __restrict__ dgk) {
  pdl_wait();
  __shared__ float s[32][kGainCols];
  const int k = threadIdx.x % kGainCols, c = blockIdx.x * kGainCols + k;  // hd is a multiple of eight
  const int row0 = blockIdx.y ? n_q : 0, n = blockIdx.y ? n_k : n_q;
  float v = 0.f;
#pragma unroll 8
  for (int i = threadIdx.x / kGainCols; i < n; i += 1024 / kGainCols) v += partial[(int64_t)(row0 + i) * hd + c];
  for (int o = 16; o >= kGainCols; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);  // the warp's four rows
  if ((threadIdx.x & 31) < kGainCols) s[threadIdx.x >> 5][k] = v;
  __syncthreads();
  if (threadIdx.x >= 32 * kGainCols) return;
  v = s[threadIdx.x & 31][threadIdx.x >> 5];  // lane = partial sum, warp = column
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  float* out = blockIdx.y ? dgk : dgq;
  if ((threadIdx.x & 31) == 0 && out) out[blockIdx.x * kGainCols + (threadIdx.x >> 5)] = v;
}

template <int V, bool NORM, bool BWD>
auto pick_style(bool pairs) {
  return pairs ? rotary_kernel<V, NORM, true, BWD> : rotary_kernel<V, NORM, false, BWD>;
}

// Blocks of a launch: several times what the SMs hold at once, so that those that end early make room (20011 tokens:
// forward 60 against 66 us, backward 97 against 104 with one load; rotation alone, 4096 tokens, 18.7 with three loads against
// 19.2 with two or four); with gain gradients each leaves one row of partial sums.
constexpr int kRotBwdBlocks = 148 * 8;
int64_t rot_blocks(bool norm, bool bwd) { return bwd ? kRotBwdBlocks : norm ? 148 * 28 : 148 * 24; }

}  // namespace

int64_t rotary_partial_floats(int64_t n_tok, int hd) { return (int64_t)(kRotBwdBlocks + 2) * hd; }

int rotary(const RotaryArgs& a, cudaStream_t s) {
  RotParams p = {};
  const bool norm = a.gq != nullptr, bwd = a.dyq != nullptr && norm;
  const bool turn_back = a.dyq && !norm;  // without the norm the gradient is rotated like an input
  const int V = a.pairs || a.rot % 16 == 0 ? 8 : 4;
  // lanes per head: one slot of two vectors each
  const int slots = a.pairs ? (a.hd + 2 * V - 1) / (2 * V) : a.rot / 2 / V + (a.hd - a.rot + 2 * V - 1) / (2 * V);
  int group = 1;
  while (group < slots) group *= 2;
  const bool gains = bwd && (a.dgq || a.dgk);
  for (int k = 0; k < 2; ++k) {
    RotSide& d = p.side[k];
    d.x = static_cast<const __nv_bfloat16*>(turn_back ? (k ? a.dyk : a.dyq) : (k ? a.xk : a.xq));
    d.ldx = turn_back ? (k ? a.lddk : a.lddq) : (k ? a.ldxk : a.ldxq);
    d.dy = static_cast<const __nv_bfloat16*>(k ? a.dyk : a.dyq);
    d.lddy = k ? a.lddk : a.lddq;
    d.o = static_cast<__nv_bfloat16*>(k ? a.ok : a.oq);
    d.ldo = k ? a.ldok : a.ldoq;
    d.g = static_cast<const __nv_bfloat16*>(k ? a.gk : a.gq);
    d.heads = k ? a.hkv : a.hq;
    d.trips = (d.heads * group + 31) / 32;
    // the blocks in proportion to the heads; few tokens: a token's trips over several warps
    const int64_t share = std::max<int64_t>(1, rot_blocks(norm, bwd) * d.heads / (a.hq + a.hkv));
    int split = 1;
    while (split < d.trips && a.n_tok * split * 2 <= share * kRotWarps) split *= 2;
    d.split = std::min(split, d.trips);
    d.blocks = (int)std::min((a.n_tok * d.split + kRotWarps - 1) / kRotWarps, share);
  }
  p.pos = a.pos;
  p.inv_freq = a.inv_freq;
  p.eps = a.eps;
  p.inv_hd = 1.f / (float)a.hd;
  p.sign = a.dyq ? -1.f : 1.f;
  p.n_tok = a.n_tok;
  p.hd = a.hd;
  p.rot = a.rot;
  p.group = group;
  p.partial = gains ? a.partial : nullptr;
  const size_t smem = gains ? (size_t)(kRotThreads / group) * a.hd * 4 : 0;
  auto kernel = V == 8 ? (norm ? (bwd ? pick_style<8, true, true>(a.pairs) : pick_style<8, true, false>(a.pairs))
                               : pick_style<8, false, false>(a.pairs))
                       : (norm ? (bwd ? rotary_kernel<4, true, false, true> : rotary_kernel<4, true, false, false>)
                               : rotary_kernel<4, false, false, false>);
  launch_kernel(kernel, (unsigned)(p.side[0].blocks + p.side[1].blocks), kRotThreads, smem, s, p);
  if (launch_failed("sl_qk_norm_rope")) return 5;
  note_launch();
  if (gains) {
    launch_kernel(rotary_gain_kernel, dim3((unsigned)(a.hd / kGainCols), 2), 1024, 0, s, (const float*)a.partial,
                  p.side[0].blocks, p.side[1].blocks, a.hd, a.dgq, a.dgk);
    if (launch_failed("sl_qk_norm_rope")) return 5;
    note_launch();
  }
  return 0;
}

}  // namespace sl
