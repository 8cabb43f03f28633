// rows.cuh -- access to rows of D elements, fp32 or bf16, by groups of threads,
// in units of 4 elements: shared by the embedding (embed.cu), the block norms
// (norm.cu) and the optimizer (adamw.cu).
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// How a group of `step` threads holds the columns of a row, C a thread: with
// vector accesses (kVec: D a multiple of 4, rows aligned to 4 elements) in
// units of 4 columns, unit u of thread i at 4 (i + u step), so that every access
// of a warp is contiguous; else column k of thread i at i + k step.  `col0` is
// the thread's first column, and what lies at or past D is left out.

// Loads of a unit of 4 columns, and their values.
__device__ __forceinline__ void ld_unit(const float* p, float (&f)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void ld_unit(const uint16_t* p, float (&f)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
}
__device__ __forceinline__ void st_unit(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void st_unit(uint16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

// (kSure: how many of the thread's first units lie in the row for every thread.)
template <bool kVec, int C, class T, int kSure = 0>
__device__ __forceinline__ void ld_cols(const T* row, int col0, int step, int D, float (&f)[C]) {
  if constexpr (kVec) {
#pragma unroll
    for (int u = 0; u < C / 4; ++u) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (u < kSure || col0 + 4 * u * step < D) ld_unit(row + col0 + 4 * u * step, x);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[4 * u + k] = x[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < C; ++k) f[k] = col0 + k * step < D ? ld1(row + col0 + k * step) : 0.f;
  }
}
template <bool kVec, int C, class T, int kSure = 0>
__device__ __forceinline__ void st_cols(T* row, int col0, int step, int D, const float (&f)[C]) {
  if constexpr (kVec) {
#pragma unroll
    for (int u = 0; u < C / 4; ++u)
      if (u < kSure || col0 + 4 * u * step < D)
        st_unit(row + col0 + 4 * u * step, f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (col0 + k * step < D) st1(row + col0 + k * step, f[k]);
  }
}

// A thread's C columns of a row as loaded: converted when they are used, so that
// a load in flight holds no more registers than its bytes; single bf16 columns
// have a register each (packing two of them waits for both: the gradient of 16384
// x 1001 bf16 61.5 us, so 46.8).
template <bool kVec, class T, int C>
struct RowUnit {
  static constexpr int kWords = kVec ? C * (int)sizeof(T) / 4 : C;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* row, int col0, int step, int D) {
    if constexpr (kVec) {
#pragma unroll
      for (int u = 0; u < C / 4; ++u) {
        if (col0 + 4 * u * step >= D) continue;
        if constexpr (sizeof(T) == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(row + col0 + 4 * u * step);
          w[4 * u] = x.x; w[4 * u + 1] = x.y; w[4 * u + 2] = x.z; w[4 * u + 3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(row + col0 + 4 * u * step);
          w[2 * u] = x.x; w[2 * u + 1] = x.y;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = col0 + k * step;
        if constexpr (sizeof(T) == 4)
          w[k] = c < D ? __float_as_uint(row[c]) : 0u;
        else
          w[k] = c < D ? (uint32_t)row[c] : 0u;
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[C]) const {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if constexpr (sizeof(T) == 4)
        f[k] = __uint_as_float(w[k]);
      else
        f[k] = !kVec ? bf16_lo(w[k]) : k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
    }
  }
};

// Asynchronous copies (8 or 16 bytes) into shared memory, in groups of the
// thread's own.  kPart: of the first `bytes` bytes only, zeros for the rest.
template <int kBytes, bool kPart = false>
__device__ __forceinline__ void cp_async(void* smem, const void* global, int bytes = kBytes) {
  if constexpr (kPart && kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem)), "l"(global), "r"(bytes)
                 : "memory");
  else if constexpr (kPart)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(smem)), "l"(global), "r"(bytes)
                 : "memory");
  else if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// How a row of D columns is spread: groups of tx threads, each thread `unit`
// columns, `slices` groups side by side.  tx is a power of two below a warp, else
// whole warps, as many as leave the slices alike (lookup of 16384 x 2049 bf16 in
// two slices of 160 threads 39 us, of 256 and little in the second 47).
struct RowSplit {
  int tx, slices;
};
RowSplit row_split(int64_t D, int unit, int max_tx) {
  const int64_t units = (D + unit - 1) / unit, slices = (units + max_tx - 1) / max_tx;
  const int64_t per = (units + slices - 1) / slices;
  int tx = 1;
  while (tx < per && tx < 32) tx *= 2;
  if (tx < per) tx = (int)((per + 31) / 32 * 32);
  return {tx, (int)((units + tx - 1) / tx)};
}

// Lets `kern` have up to kMaxSmem of dynamic shared memory: always the same
// number, so that calls from several host threads do not lower each other's.
constexpr size_t kMaxSmem = 220 * 1024;
template <class K>
cudaError_t allow_smem(K kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
}

// Whether vector accesses (units of 4 columns) can start at p.
bool aligned_rows(const void* p, bool bf16) { return bf16 ? aligned8(p) : aligned16(p); }

// Pointers aligned to n bytes (a power of two).
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace mole
