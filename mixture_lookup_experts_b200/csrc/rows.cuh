// rows.cuh -- access to rows of D elements by groups of threads, 8 columns a
// thread, fp32 or bf16: shared by the embedding (embed.cu) and the block norms
// (norm.cu).
#pragma once

#include "common.cuh"

namespace mole {
namespace {

template <class T>
__device__ __forceinline__ float ld1(const T* p);
template <>
__device__ __forceinline__ float ld1<float>(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float ld1<uint16_t>(const uint16_t* p) {
  return to_f32(*p);
}
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ __forceinline__ void ld_vec8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void ld_vec8(const uint16_t* p, float (&f)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
  f[4] = bf16_lo(a.z); f[5] = bf16_hi(a.z); f[6] = bf16_lo(a.w); f[7] = bf16_hi(a.w);
}
__device__ __forceinline__ void st_vec8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi)) << 16);
}
__device__ __forceinline__ void st_vec8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// A thread's 8 columns of a row: consecutive (kVec; col0 = 8 * thread), or
// spaced by `step` from col0 = thread, those past D left out.
template <bool kVec, class T>
__device__ __forceinline__ void ld_cols(const T* row, int col0, int step, int D, float (&f)[8]) {
  if constexpr (kVec) {
    ld_vec8(row + col0, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = col0 + k * step < D ? ld1(row + col0 + k * step) : 0.f;
  }
}
template <bool kVec, class T>
__device__ __forceinline__ void st_cols(T* row, int col0, int step, int D, const float (&f)[8]) {
  if constexpr (kVec) {
    st_vec8(row + col0, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col0 + k * step < D) st1(row + col0 + k * step, f[k]);
  }
}

// How a row of D columns is spread: groups of tx threads, each thread 8
// columns, `slices` groups side by side.
struct RowSplit {
  int tx, slices;
};
RowSplit row_split(int64_t D, int max_tx) {
  const int64_t units = (D + 7) / 8;
  int tx = 1;
  while (tx < max_tx && tx < units) tx *= 2;
  return {tx, (int)((units + tx - 1) / tx)};
}

// Pointers aligned to n bytes (a power of two).
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace mole
