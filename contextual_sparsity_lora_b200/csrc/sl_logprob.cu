// Log probabilities of given tokens, the entropy of each row's distribution and its most likely
// tokens, from one pass over logits z [rows, vocab], and the gradient of the first two:
//   lse = log sum_j e^(z_j);  logp = z_t - lse;  H = -sum_j p_j log p_j, p_j = e^(z_j - lse);
//   d logp / d z_j = [j = t] - p_j;  d H / d z_j = -p_j (log p_j + H).
//
// Sums run in powers of two: x_j = z_j log2(e) - r with r a whole number at or above the running
// maximum of z log2(e), s = sum 2^x, w = sum 2^x x. With r whole, x has one rounding and moving
// r multiplies the sums by exact powers of two; logp = ln 2 (x_t - log2 s), H = ln 2 (log2 s - w / s).
// (r, log2 s) of each row go to the backward, which needs nothing else: p_j = 2^(x_j - log2 s).
//
// r is a whole number only as far as fp32 holds one next to it: z log2(e) rounds to r by up to half a unit u of r, and
// the largest x is then not in (-1, 0] but that rest (64 at most where |r| < 2^31: sums below 2^89, nothing lost, log2 s
// contains it). From |r| >= 2^31 on it would overflow the sums, or empty them; but there two different logits are at
// least 128 apart, and e^-128 is 0 in fp32 beside 1: the distribution is the maximum's ties alone. A row whose maximum
// is such a far logit m (masked by -1e10 or -1e30 throughout, or 1e10 itself) keeps r = 4 m, an exact number that
// stands beyond every near r and in the order of m, with s = w = 0 until the ties are counted at the end, in a second
// pass over the row. Others pay nothing: one comparison stands for the two with the ends of the range.
//
// The top k (k <= 32): while the sums are taken, the maximum of every 16 consecutive logits goes to
// shared memory. The k largest logits lie in k of these chunks: those whose maximum exceeds the k-th
// largest maximum, and the first of those that equal it. Their 16 k logits are read again and
// ranked by (value, lowest index first). The k-th largest maximum itself is looked for only where many are equal
// (local_top); mostly a bound close below it does (local_top_few), from one value per thread.
//
// The forward reads each logit once, the backward reads and writes it once. Measured on 128256 bf16 logits a row: backward,
// 1024 rows, 88 us (6.0 TB/s, 0.91 of the copy rate); forward with entropy, 1024 rows 61 us, 4096 rows with 20
// alternatives 213 us (4.9 TB/s, 0.75): its issue slots are four fifths full, with a range check, a maximum, a
// conversion, an exponential and two sums per logit (a second maximum that keeps NaN cost 224 us; NaN shows in
// the sums). Few rows: a cluster of up to 8 CTAs shares a row, each with a contiguous part of the
// vocabulary, and the first CTA joins sums and candidates through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "sl_packed.h"

namespace sl {

namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpChunk = 16;    // logits per chunk
constexpr int kLpMaxTop = 32;
constexpr int kLpFewChunks = 128;
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.693147181f;
constexpr float kHuge = 10633823966279326983230456482242756608.f;  // 2^123: logits below -kHuge count as -infinity; one above kHuge makes its row NaN
constexpr float kNothing = -3e38f;  // reference of sums that hold nothing
constexpr float kFar = 2147483648.f;  // 2^31, of |z log2(e)|: see above
constexpr float kFarLogit = 1488522240.f;  // the smallest z whose z log2(e) rounds to 2^31

struct LpParams {
  const void* z;
  int64_t ld, rows, vocab, seg;  // seg: columns per CTA of a cluster
  const int32_t* target;
  float* logp;
  float2* stats;
  float* entropy;
  int32_t* top_ids;
  float* top_logp;
  int32_t k;
};

struct Sums {
  float r, s, w;  // reference (whole, in powers of two; of far logits 4 m), sum of 2^x, sum of 2^x x
};

// z log2(e) rounded to fp32, for itself (not contracted into a multiply-add).
__device__ __forceinline__ float in_twos(float z) { return __fmul_rn(z, kLog2e); }
__device__ __forceinline__ bool is_far(float r) { return fabsf(r) >= kFar; }
// Two neighbouring far logits may round to the same z log2(e) (the factor is below 2), never three. Whether the next
// larger fp32 number than z does as z:
__device__ __forceinline__ bool next_same(float z) {
  const int b = __float_as_int(z);
  return in_twos(__int_as_float(b + (b < 0 ? -1 : 1))) == in_twos(z);
}

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void move_ref(Sums& a, float r) {
  const float d = a.r - r, c = lp_ex2(d);
  a.w = c * (a.w + a.s * fmaxf(d, -1000.f));
  a.s *= c;
  a.r = r;
}

__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float r = fmaxf(a.r, b.r);
  move_ref(a, r);
  move_ref(b, r);
  a.s += b.s;
  a.w += b.w;
  return a;
}

// Order of logits as unsigned numbers: larger logit, larger number; -0 as 0; NaN below all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return z != z ? 0u : ((int32_t)b < 0 ? ~b : b | 0x80000000u);
}
__device__ __forceinline__ float from_order_key(uint32_t k) {
  return k == 0 ? __int_as_float(0x7fffffff) : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// 16 consecutive logits as they lie in memory, and the reads of two chunks of them in flight at once.
template <typename T>
struct Chunk {
  uint4 w[sizeof(T)];
};
// Columns at n and behind read as -inf.
template <typename T>
__device__ __forceinline__ void load16(const T* row, int64_t c, int64_t n, Chunk<T>& q) {
  if (c + kLpChunk <= n) {
#pragma unroll
    for (int v = 0; v < (int)sizeof(T); ++v) q.w[v] = *(reinterpret_cast<const uint4*>(row + c) + v);
  } else {
    T* e = reinterpret_cast<T*>(q.w);
#pragma unroll
    for (int i = 0; i < kLpChunk; ++i) e[i] = c + i < n ? row[c + i] : (T)(-INFINITY);
  }
}

typedef unsigned long long f2;  // two fp32 values: one instruction for both
__device__ __forceinline__ f2 pk(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void un(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Raises a chunk's logits to -kHuge at least (so that 2^x x is 0, not NaN, where the logit is -infinity); NaN stays, and
// makes the sums NaN. Returns the largest logit that is a number, as it was (NaN: there is none).
__device__ __forceinline__ float clamp_max(Chunk<__nv_bfloat16>& q) {
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(q.w);
  const __nv_bfloat162 low = __float2bfloat162_rn(-kHuge);
  __nv_bfloat162 t = h[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) t = __hmax2(t, h[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = __hmax2_nan(h[i], low);
  return fmaxf(__low2float(t), __high2float(t));
}
__device__ __forceinline__ float clamp_max(Chunk<float>& q) {
  float* z = reinterpret_cast<float*>(q.w);
  float top = z[0];
#pragma unroll
  for (int i = 0; i < kLpChunk; ++i) {
    top = fmaxf(top, z[i]);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(z[i]) : "f"(-kHuge));
  }
  return top;
}
__device__ __forceinline__ void pair_of(const Chunk<__nv_bfloat16>& q, int i, float& a, float& b) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(q.w)[i];
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void pair_of(const Chunk<float>& q, int i, float& a, float& b) {
  a = reinterpret_cast<const float*>(q.w)[2 * i];
  b = reinterpret_cast<const float*>(q.w)[2 * i + 1];
}

template <typename T>
using KeyOf = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
// A chunk's maximum as a key of the logits' own width.
template <typename T>
__device__ __forceinline__ KeyOf<T> chunk_key(float m) {
  if constexpr (sizeof(T) == 2) return (uint16_t)(order_key(m) >> 16);
  else return order_key(m);
}

struct LpShared {
  Sums part[kLpWarps];
  Sums mine;                                    // this CTA's sums
  int count[2][kLpWarps];
  int pick[kLpMaxTop];                          // chosen chunks
  int few[kLpFewChunks];                        // chunks that reach the bound
  int n_pick, n_cand;
  unsigned long long cand[kLpMaxTop * kLpChunk];  // (key, ~index) of candidates
  unsigned long long best[kLpMaxTop];           // this CTA's top k, best first (0: none)
};

// Sum over the block of one count per thread; `turn` alternates between calls.
__device__ __forceinline__ int block_count(LpShared& sh, int turn, int v) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) sh.count[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) s += sh.count[turn][w];
  return s;
}

// Ranks n distinct candidates; the k largest go to out[0..k), best first, the rest of out is 0.
__device__ __forceinline__ void rank_into(const unsigned long long* cand, int n, int k, unsigned long long* out) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long me = cand[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += cand[j] > me;
    if (rank < k) out[rank] = me;
  }
}

// The same from few chunks: the k-th largest of the threads' own largest keys (to 16 bits) is a bound that k chunks reach, and
// hardly more do. Only the threads that reach it look for theirs, and only those chunks are read again. False when
// more chunks or logits reach the bound than there is room for (many equal ones): nothing is done then.
template <typename T>
__device__ bool local_top_few(LpShared& sh, const KeyOf<T>* keys, KeyOf<T> top_key, const T* row, int64_t c0, int64_t n, int k) {
  constexpr int kShift = 8 * (int)sizeof(KeyOf<T>) - 16;
  const int n_chunk = (int)((n + kLpChunk - 1) / kLpChunk);
  if (min(n_chunk, kLpThreads) <= k) return false;
  const uint32_t mine = (uint32_t)top_key >> kShift;
  if (threadIdx.x == 0) sh.n_pick = sh.n_cand = 0;
  if (threadIdx.x < kLpMaxTop) sh.best[threadIdx.x] = 0;
  uint32_t bound = 0;
#pragma unroll 1
  for (int b = 15; b >= 0; --b)
    if (__syncthreads_count(mine >= (bound | (1u << b))) >= k) bound |= 1u << b;
  if (mine >= bound)
    for (int c = threadIdx.x; c < n_chunk; c += kLpThreads)
      if ((uint32_t)keys[c] >> kShift >= bound) {
        const int at = atomicAdd(&sh.n_pick, 1);
        if (at < kLpFewChunks) sh.few[at] = c;
      }
  __syncthreads();
  const int n_pick = sh.n_pick;
  if (n_pick > kLpFewChunks) return false;
  for (int i = threadIdx.x; i < n_pick * kLpChunk; i += kLpThreads) {
    const int64_t c = c0 + (int64_t)sh.few[i / kLpChunk] * kLpChunk + i % kLpChunk;
    if (c >= c0 + n) continue;
    const uint32_t key = order_key((float)row[c]);
    if (key >> 16 >= bound) {
      const int at = atomicAdd(&sh.n_cand, 1);
      if (at < kLpMaxTop * kLpChunk) sh.cand[at] = ((unsigned long long)key << 32) | (uint32_t)~(uint32_t)c;
    }
  }
  __syncthreads();
  const int n_cand = sh.n_cand;
  if (n_cand > kLpMaxTop * kLpChunk) return false;
  rank_into(sh.cand, n_cand, k, sh.best);
  __syncthreads();
  return true;
}

// This CTA's k largest logits of columns [c0, c0 + n) into sh.best, from the chunks' keys.
template <typename T>
__device__ void local_top(LpShared& sh, const KeyOf<T>* keys, const T* row, int64_t c0, int64_t n, int k) {
  const int n_chunk = (int)((n + kLpChunk - 1) / kLpChunk);
  __syncthreads();
  const int per = (n_chunk + kLpThreads - 1) / kLpThreads;
  const int a = min(n_chunk, (int)threadIdx.x * per), e = min(n_chunk, a + per);
  if (threadIdx.x == 0) sh.n_pick = sh.n_cand = 0;
  if (threadIdx.x < kLpMaxTop) sh.best[threadIdx.x] = 0;
  uint32_t tau = 0;  // the k-th largest key (0 when there are no more than k chunks)
  int turn = 0;
  __syncthreads();
  if (n_chunk > k) {
    for (int b = 8 * (int)sizeof(KeyOf<T>) - 1; b >= 0; --b, turn ^= 1) {
      const uint32_t cand = tau | (1u << b);
      int c = 0;
      for (int i = a; i < e; ++i) c += keys[i] >= cand;
      if (block_count(sh, turn, c) >= k) tau = cand;
    }
  }
  int above = 0, equal = 0;
  for (int i = a; i < e; ++i) {
    above += keys[i] > tau;
    equal += keys[i] == tau;
  }
  const int n_above = block_count(sh, turn, above);
  turn ^= 1;
  // exclusive count of the equal ones before this thread's, in the order of the columns
  int inc = equal;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh.count[turn][warp] = inc;
  __syncthreads();
  int before = inc - equal;
  for (int w = 0; w < warp; ++w) before += sh.count[turn][w];
  const int room = k - n_above;  // chunks still to take of the equal ones: the first
  for (int i = a; i < e; ++i) {
    bool take = keys[i] > tau;
    if (keys[i] == tau) take = before++ < room;
    if (take) sh.pick[atomicAdd(&sh.n_pick, 1)] = i;
  }
  __syncthreads();
  const int n_pick = sh.n_pick;
  for (int i = threadIdx.x; i < n_pick * kLpChunk; i += kLpThreads) {
    const int64_t c = c0 + (int64_t)sh.pick[i / kLpChunk] * kLpChunk + i % kLpChunk;
    if (c >= c0 + n) continue;
    const uint32_t key = order_key((float)row[c]);
    const uint32_t cut = sizeof(T) == 2 ? tau << 16 : tau;
    if (key >= cut) sh.cand[atomicAdd(&sh.n_cand, 1)] = ((unsigned long long)key << 32) | (uint32_t)~(uint32_t)c;
  }
  __syncthreads();
  rank_into(sh.cand, sh.n_cand, k, sh.best);
  __syncthreads();
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(kLpThreads) logprob_fwd_kernel(const __grid_constant__ LpParams p) {
  extern __shared__ uint4 s_keys_raw[];
  KeyOf<T>* keys = reinterpret_cast<KeyOf<T>*>(s_keys_raw);
  __shared__ LpShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t r = blockIdx.x / n_cta;
  pdl_wait();
  const T* row = static_cast<const T*>(p.z) + r * p.ld;
  const int64_t c0 = min(p.vocab, (int64_t)rank * p.seg), c1 = min(p.vocab, c0 + p.seg), n = c1 - c0;
  const int k = p.k;

  // The sums of this thread's chunks; of bf16 the next chunk's logits are on their way (32 bits: the 16 registers are worth
  // a third block per SM, 301 rows of 32003 15.8 against 19.4 us, 1000 rows of 64000 66 against 68).
  constexpr bool kAhead = sizeof(T) == 2;
  Sums a = {kNothing, 0.f, 0.f};
  const int n_chunk = (int)((n + kLpChunk - 1) / kLpChunk);
  KeyOf<T> top_key = 0;  // of this thread's chunks
  float z_max = -kHuge;  // the largest logit so far; a.r follows from it
  Chunk<T> q, q_next;
  if (kAhead && (int)threadIdx.x < n_chunk) load16(row, c0 + (int64_t)threadIdx.x * kLpChunk, c1, q_next);
  for (int c = threadIdx.x; c < n_chunk; c += kLpThreads) {
    if (kAhead) q = q_next;
    else load16(row, c0 + (int64_t)c * kLpChunk, c1, q);
    if (kAhead && c + kLpThreads < n_chunk) load16(row, c0 + (int64_t)(c + kLpThreads) * kLpChunk, c1, q_next);
    const float top = clamp_max(q), m = fmaxf(top, -kHuge), z_new = fmaxf(z_max, m);
    if (k > 0) {
      const KeyOf<T> key = chunk_key<T>(top);
      keys[c] = key;
      top_key = max(top_key, key);
    }
    if (fabsf(m) >= kFarLogit) {  // a far maximum, nothing here (all raised to -kHuge), or NaN
#pragma unroll
      for (int i = 0; i < kLpChunk / 2; ++i) {
        float z0, z1;
        pair_of(q, i, z0, z1);
        if (z0 != z0 || z1 != z1) a.s = __int_as_float(0x7fffffff);
      }
      z_max = z_new;
      continue;
    }
    const float ref_new = ceilf(in_twos(z_new));
    if (z_new > z_max) {
      a.r = ceilf(in_twos(z_max));
      move_ref(a, ref_new);
    }
    z_max = z_new;
    f2 s[2] = {0, 0}, w[2] = {0, 0};
    const f2 l2e = pk(kLog2e, kLog2e), ref = pk(-ref_new, -ref_new);
#pragma unroll
    for (int i = 0; i < kLpChunk / 2; ++i) {
      float z0, z1;
      pair_of(q, i, z0, z1);
      const f2 x = fma2(pk(z0, z1), l2e, ref);
      un(x, z0, z1);
      const f2 e = pk(lp_ex2(z0), lp_ex2(z1));
      s[i & 1] = add2(s[i & 1], e);
      if (ENT) w[i & 1] = fma2(e, x, w[i & 1]);
    }
    float s0, s1;
    un(add2(s[0], s[1]), s0, s1);
    a.s += s0 + s1;
    if (ENT) {
      un(add2(w[0], w[1]), s0, s1);
      a.w += s0 + s1;
    }
  }
  if (fabsf(z_max) >= kFarLogit) {  // what was summed is 0 beside a far logit (NaN stays)
    a.r = z_max > -kHuge ? 4.f * z_max : kNothing;
    a.s *= z_max > kHuge ? __int_as_float(0x7fffffff) : 0.f;
    a.w *= 0.f;
  } else {
    a.r = ceilf(in_twos(z_max));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.r = __shfl_xor_sync(0xffffffffu, a.r, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.w = __shfl_xor_sync(0xffffffffu, a.w, o);
    a = join(a, b);
  }
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kLpWarps; ++w) a = join(a, sh.part[w]);
    sh.mine = a;
  }
  __syncthreads();
  if (k > 0 && !local_top_few<T>(sh, keys, top_key, row, c0, n, k)) local_top<T>(sh, keys, row, c0, n, k);

  if (n_cta > 1) {
    cluster.sync();
    if (rank == 0) {
      if (threadIdx.x == 0) {
        a = sh.mine;
        for (int i = 1; i < n_cta; ++i) a = join(a, *cluster.map_shared_rank(&sh.mine, i));
        sh.part[0] = a;
      }
      if (threadIdx.x < n_cta * k) {
        const int i = threadIdx.x / k, j = threadIdx.x % k;
        sh.cand[threadIdx.x] = cluster.map_shared_rank(sh.best, i)[j];
      }
      __syncthreads();
      if (threadIdx.x == 0) sh.mine = sh.part[0];
      if (k > 0) {
        // entries that a short part left empty (0) are not distinct: they rank behind every other
        if (threadIdx.x < n_cta * k) {
          const unsigned long long me = sh.cand[threadIdx.x];
          int place = 0;
          for (int j = 0; j < n_cta * k; ++j) place += sh.cand[j] > me;
          if (me != 0 && place < k) sh.best[place] = me;
        }
      }
      __syncthreads();
    }
    cluster.sync();  // the others' shared memory has been read
    if (rank != 0) return;
  }
  Sums t = sh.mine;
  if (t.s == 0.f && t.r > kNothing) {  // a far row: the maximum's ties
    int ties = 0;
    for (int64_t c = threadIdx.x; c < p.vocab; c += kLpThreads) ties += (float)row[c] == 0.25f * t.r;
    t.s = (float)block_count(sh, 0, ties);
  }
  const bool none = t.s == 0.f;  // the row has no logit above -infinity
  const bool far = t.s >= 1.f && is_far(t.r);  // neither empty nor NaN
  const float l2s = none ? 0.f : log2f(t.s), m = 0.25f * t.r;  // m: of a far row
  auto log_p = [&](float z) {
    return none ? -INFINITY : far ? fmaf(-kLn2, l2s, z - m) : (fmaf(z, kLog2e, -t.r) - l2s) * kLn2;
  };
  if (threadIdx.x == 0) {
    const int32_t tg = p.target[r];
    float lp = 0.f;
    if (tg >= 0 && tg < p.vocab) lp = log_p((float)row[tg]);
    p.logp[r] = lp;
    // of a far row m log2(e); log2 s, which is not negative there, has the sign bit when m is the smaller one of two
    // logits with this value (what that takes from the log sum is below its rounding)
    p.stats[r] = far ? make_float2(in_twos(m), next_same(m) ? -l2s : l2s) : make_float2(none ? -INFINITY : t.r, l2s);
    if (ENT) p.entropy[r] = none ? 0.f : (l2s - t.w / t.s) * kLn2;
  }
  if (threadIdx.x < k) {
    const unsigned long long b = sh.best[threadIdx.x];
    const float z = from_order_key((uint32_t)(b >> 32));
    p.top_ids[r * k + threadIdx.x] = (int32_t)~(uint32_t)b;
    p.top_logp[r * k + threadIdx.x] = log_p(z);
  }
}

struct LpBwdParams {
  const void* z;
  int64_t ld, rows, vocab, ldd, seg;
  const int32_t* target;
  const float2* stats;
  const float* g_logp;
  const float* g_entropy;
  const float* entropy;
  void* dz;
};

// dz_j = [j = t] g - p_j (g + gH (log p_j + H)) = [j = t] g - 2^x (A + B x): one column range of a row per block.
template <typename T>
__global__ void __launch_bounds__(256) logprob_bwd_kernel(const __grid_constant__ LpBwdParams p) {
  pdl_wait();
  constexpr int kVec = 16 / sizeof(T);
  const int64_t r = blockIdx.x;
  const T* row = static_cast<const T*>(p.z) + r * p.ld;
  T* out = static_cast<T*>(p.dz) + r * p.ldd;
  const int64_t c0 = (int64_t)blockIdx.y * p.seg, c1 = min(p.vocab, c0 + p.seg);
  const int32_t t = p.target[r];
  const bool has = t >= 0 && t < p.vocab;
  const float2 st = p.stats[r];
  const float g = has ? p.g_logp[r] : 0.f;
  const float gh = p.g_entropy ? p.g_entropy[r] : 0.f;
  const bool none = st.x == -INFINITY || (g == 0.f && gh == 0.f);
  const bool far = !none && is_far(st.x) && st.y == st.y;  // see logprob_fwd_kernel's stats
  const float l2s = far ? fabsf(st.y) : st.y;
  const float inv = lp_ex2(-l2s);
  const float h = gh != 0.f ? p.entropy[r] : 0.f;
  const float A = inv * (g + gh * (h - l2s * kLn2)), B = inv * gh * kLn2;
  auto grad = [&](float z, int64_t c) {
    const float x = fmaf(z, kLog2e, -st.x);
    const float e = lp_ex2(x);
    const float d = -e * fmaf(B, fmaxf(x, -1000.f), A);
    return c == t ? d + g : d;
  };
  if (far) {
    const bool lower = signbit(st.y);
    for (int64_t c = c0 + threadIdx.x; c < c1; c += 256) {
      const float z = (float)row[c];
      const float d = in_twos(z) == st.x && (lower || !next_same(z)) ? -A : 0.f;
      out[c] = (T)(c == t ? d + g : d);
    }
    return;
  }
  for (int64_t c = c0 + (int64_t)threadIdx.x * kVec; c < c1; c += 256 * kVec) {
    if (c + kVec <= c1) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (!none) {
        w = *reinterpret_cast<const uint4*>(row + c);
        uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162 d = __floats2bfloat162_rn(grad(__uint_as_float(v[i] << 16), c + 2 * i),
                                                           grad(__uint_as_float(v[i] & 0xffff0000u), c + 2 * i + 1));
            v[i] = *reinterpret_cast<const uint32_t*>(&d);
          } else {
            v[i] = __float_as_uint(grad(__uint_as_float(v[i]), c + i));
          }
        }
        w = make_uint4(v[0], v[1], v[2], v[3]);
      }
      *reinterpret_cast<uint4*>(out + c) = w;
    } else {
      for (int64_t j = c; j < c1; ++j) out[j] = none ? (T)0.f : (T)grad((float)row[j], j);
    }
  }
}

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

constexpr int kLpMaxKeysBytes = 200 * 1024;

template <typename T, bool ENT>
int fwd_launch(const LpParams& p, int n_cta, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  auto kernel = logprob_fwd_kernel<T, ENT>;
  if (!smem_limit(kernel, kLpMaxKeysBytes, done)) return 5;
  const size_t smem = p.k > 0 ? (size_t)((p.seg + kLpChunk - 1) / kLpChunk) * sizeof(KeyOf<T>) : 0;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * n_cta));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kernel, p);
  if (launch_failed("sl_token_logprobs")) return 5;
  note_launch();
  return 0;
}

}  // namespace

int token_logprobs_fwd(const LogprobArgs& a, cudaStream_t s) {
  LpParams p = {};
  p.z = a.z;
  p.ld = a.ld;
  p.rows = a.rows;
  p.vocab = a.vocab;
  p.target = a.target;
  p.logp = a.logp;
  p.stats = reinterpret_cast<float2*>(a.stats);
  p.entropy = a.entropy;
  p.top_ids = a.top_ids;
  p.top_logp = a.top_logp;
  p.k = a.k;
  // CTAs per row: a cluster where the rows alone do not fill the SMs and each part keeps a pass of the block
  int n_cta = 1;
  while (n_cta < 8 && a.rows * n_cta * 2 <= 2 * 148 && a.vocab / (2 * n_cta) >= kLpThreads * kLpChunk / 2) n_cta *= 2;
  // the chunks' keys of a part have to fit the shared memory of a CTA
  const int64_t key = a.fp32 ? 4 : 2;
  auto seg_of = [&](int n) { return ((a.vocab + n - 1) / n + kLpChunk - 1) / kLpChunk * kLpChunk; };
  while (a.k > 0 && n_cta < 8 && seg_of(n_cta) / kLpChunk * key > kLpMaxKeysBytes) n_cta *= 2;
  if (a.k > 0 && seg_of(n_cta) / kLpChunk * key > kLpMaxKeysBytes) return 1;
  p.seg = seg_of(n_cta);
  if (a.rows * n_cta > 0x7fffffff) return 1;
  if (a.fp32) return a.entropy ? fwd_launch<float, true>(p, n_cta, s) : fwd_launch<float, false>(p, n_cta, s);
  return a.entropy ? fwd_launch<__nv_bfloat16, true>(p, n_cta, s) : fwd_launch<__nv_bfloat16, false>(p, n_cta, s);
}

int token_logprobs_bwd(const LogprobArgs& a, cudaStream_t s) {
  LpBwdParams p = {};
  p.z = a.z;
  p.ld = a.ld;
  p.rows = a.rows;
  p.vocab = a.vocab;
  p.ldd = a.ldd;
  p.target = a.target;
  p.stats = reinterpret_cast<const float2*>(a.stats);
  p.g_logp = a.g_logp;
  p.g_entropy = a.g_entropy;
  p.entropy = a.entropy;
  p.dz = a.dz;
  const int64_t step = 256 * (a.fp32 ? 4 : 8);  // columns of one trip of a block
  // column ranges: whole trips, more of them while the blocks do not fill the SMs a few times over
  int64_t n_seg = 1;
  while (a.rows * n_seg < 148 * 16 && a.vocab / (n_seg * 2) >= step) n_seg *= 2;
  p.seg = ((a.vocab + n_seg - 1) / n_seg + step - 1) / step * step;
  n_seg = (a.vocab + p.seg - 1) / p.seg;
  if (a.rows > 0x7fffffff || n_seg > 65535) return 1;
  launch_kernel(a.fp32 ? logprob_bwd_kernel<float> : logprob_bwd_kernel<__nv_bfloat16>,
                dim3((unsigned)a.rows, (unsigned)n_seg), 256, 0, s, p);
  if (launch_failed("sl_token_logprobs")) return 5;
  note_launch();
  return 0;
}

}  // namespace sl
