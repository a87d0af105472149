// Device and host pieces that the attention kernels share: 4-D tensor copies, TMEM stores, operand
// descriptors of 128-token tiles, and the tensor maps of heads.
#pragma once
#include <cuda_bf16.h>

#include "sl_internal.h"
#include "sl_ptx.cuh"

namespace sl {

namespace {

constexpr int kTile = 128;           // tokens per tile (TMEM lanes)
constexpr int kChunk = 128 * 64 * 2;  // one 128-token x 64-element bf16 tile chunk (16 KB)

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Each thread of the warp writes 32 consecutive fp32 columns of its TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Shared-memory descriptors of a tile stored as nc chunks (16 KB apart) of 128 token rows x 128 B.
// K-major use (contraction over the head dimension, or over the 128 columns of a P-like tile):
// 16-element step t lies in chunk t / 4 at byte 32 (t % 4) of each row.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base, int t) {
  return smem_desc_sw128(base + (uint32_t)(t >> 2) * kChunk + (uint32_t)(t & 3) * 32, 16, 1024);
}
// MN-major use (contraction over the 128 token rows): step t covers rows 16 t .. 16 t + 15; the
// 64-wide chunks of the other dimension are 16 KB apart.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t base, int t) {
  return smem_desc_sw128(base + (uint32_t)t * 2048, kChunk, 1024);
}

// Writes 32 bf16 values (v[0..31] as 16 packed pairs) of row r into a 128-byte-swizzled K-major
// tile (the layout the tensor maps produce): element c of the row sits in chunk c / 64, 16-byte
// unit ((c % 64) / 8) ^ (r % 8).
__device__ __forceinline__ void st_swizzled_row32(uint8_t* tile, int r, int c0, const uint32_t (&w)[16]) {
  uint8_t* row = tile + (c0 >> 6) * kChunk + r * 128;
  const int u0 = (c0 & 63) >> 3;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int u = (u0 + q) ^ (r & 7);
    *reinterpret_cast<uint4*>(row + u * 16) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
}

// Writes row r of a box of 32-element fp32 rows (128-byte swizzle: 16-byte unit u of row r sits at
// unit u ^ (r % 8); the box starts on a 1024-byte boundary) from 32 raw fp32 values, each
// multiplied by `mul`.
__device__ __forceinline__ void st_dq_box_row(uint8_t* box, int r, const uint32_t (&v)[32], float mul) {
  uint8_t* row = box + r * 128;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<float4*>(row + ((u ^ (r & 7)) * 16)) =
        make_float4(__uint_as_float(v[4 * u]) * mul, __uint_as_float(v[4 * u + 1]) * mul,
                    __uint_as_float(v[4 * u + 2]) * mul, __uint_as_float(v[4 * u + 3]) * mul);
}

// Bulk tensor store of a shared-memory box through a 4-D tensor map (elements outside the tensor
// are not written), tracked in the issuing thread's bulk async-groups.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, const void* smem_src, int32_t c0, int32_t c1,
                                             int32_t c2, int32_t c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// Adds a shared-memory box to global memory through a 4-D tensor map (fp32 add in L2; elements
// outside the tensor are skipped), tracked in the issuing thread's bulk async-groups.
__device__ __forceinline__ void tma_reduce_add_4d(const CUtensorMap* m, const void* smem_src, int32_t c0, int32_t c1,
                                                  int32_t c2, int32_t c3) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.4d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// mbar_wait that reads the clock only after a number of tries: a read of the nanosecond timer takes longer than the
// waits of a running pipeline, and each wait that is not over at once would pay it.
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, err, code);
}

// ---- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* ptr = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

// [hd, heads, S, n_seq] view of a [n_seq * S, ld] bf16 matrix whose head h occupies columns
// [h hd, (h + 1) hd); boxes of 64 x 1 x box_rows x 1, 128-byte swizzle, zero fill outside.
bool head_map(CUtensorMap* m, const void* ptr, int64_t ld, int n_seq, int S, int heads, int hd, int box_rows = 128) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)S, (cuuint64_t)n_seq};
  cuuint64_t strides[3] = {(cuuint64_t)hd * 2, (cuuint64_t)ld * 2, (cuuint64_t)S * ld * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [hd, heads, S, n_seq] view of the [n_seq * S, heads * hd] fp32 dQ accumulator; boxes of
// 32 x 1 x 32 x 1 (32 rows of 128 bytes: one warp's rows), 128-byte swizzle.
bool dq_acc_map(CUtensorMap* m, float* ptr, int n_seq, int S, int heads, int hd) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)S, (cuuint64_t)n_seq};
  cuuint64_t strides[3] = {(cuuint64_t)hd * 4, (cuuint64_t)heads * hd * 4, (cuuint64_t)S * heads * hd * 4};
  cuuint32_t box[4] = {32, 1, 32, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace sl
