// What the tensor-core attention kernels share: packed fp32 arithmetic, the
// split of a number into two 8-bit ones, and the tensor maps of the KV pool.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "internal.cuh"

namespace dsa {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// f16x2 -> hi = E4M3(x) and lo = E4M3(x - hi) as byte pairs (low half ->
// low byte).  x - hi is exact in fp16: hi is x rounded to 4 significant bits.
__device__ __forceinline__ void split_e4m3x2(uint32_t h2, uint32_t& hi, uint32_t& lo) {
  unsigned short a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h2));
  uint32_t back;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h2), *reinterpret_cast<const __half2*>(&back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(*reinterpret_cast<const uint32_t*>(&r)));
  hi = a;
  lo = b;
}
// f16x2 -> hi = E4M3(x) and lo = E5M2(x - hi): 3 significant bits of the
// residual, down to 2^-17 where E4M3 ends at 2^-10.
__device__ __forceinline__ void split_e4m3_e5m2x2(uint32_t h2, uint32_t& hi, uint32_t& lo) {
  unsigned short a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h2));
  uint32_t back;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h2), *reinterpret_cast<const __half2*>(&back));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(b) : "r"(*reinterpret_cast<const uint32_t*>(&r)));
  hi = a;
  lo = b;
}
// Two-wide fp32 arithmetic, each lane rounded as its scalar .rn form.
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float x0, float x1) {
  const __half2 h = __floats2half2_rn(x0, x1);  // x0 in the low half
  return *reinterpret_cast<const uint32_t*>(&h);
}

// cuTensorMapEncodeTiled, looked up once from the driver
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The KV pool as a 2-D byte tensor [slots][row_bytes], in boxes of box_rows
// rows (1 for tile::gather4), box_cols wide from any column.
inline bool make_kv_map(CUtensorMap* map, const MlaArgs& a, uint32_t row_bytes, uint32_t box_cols, uint32_t box_rows,
                        CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)a.num_pages * (cuuint64_t)a.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows}, elem[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.kv), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 rows [n, groups, d] behind strides (in elements), in boxes of 64 columns, one
// group and box_rows rows, 128-byte swizzle; what a box takes from outside is zero.
inline bool make_rows_map(CUtensorMap* map, const void* p, int64_t n, int64_t groups, int64_t d, int64_t row_stride,
                          int64_t group_stride, uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  // (a stride that is never taken is any valid one)
  const cuuint64_t any = (cuuint64_t)((d * 2 + 15) / 16 * 16);
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)groups, (cuuint64_t)n};
  const cuuint64_t strides[2] = {groups > 1 ? (cuuint64_t)group_stride * 2 : any, n > 1 ? (cuuint64_t)row_stride * 2 : any};
  const cuuint32_t box[3] = {64, 1, box_rows}, elem[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dsa
