// adamw.cu -- one AdamW step over a list of tensors (mole.h states the
// formulas).  MoLE page, 训练阶段: the layer is trained end to end; this is the
// step that consumes the gradients which the backward calls add up in fp32.
//
// Elementwise, so bound by HBM: per element the gradient (4 or 2 bytes), the
// weight (bf16 with an fp32 master: 10 bytes moved, fp32: 8, bf16 alone: 4) and
// the states (fp32: 16, 8 bits: 4 + 16 / 128).  One launch serves up to 128
// tensors: their addresses travel in the kernel's parameters, and the work is
// cut into chunks of kAdamChunk elements, each inside one tensor.
//
// A thread has kAdamUnits units of 4 elements, so that a warp's unit is 128
// consecutive ones: every access is contiguous, and it is one block of 8-bit
// states, whose largest value takes one warp reduction (of the bits: values
// that are not negative order like their bits, NaN above all).  m and sqrt(v)
// are e4m3 times an fp32 scale; keeping the root halves the exponents that the
// codes must span.  In between everything is fp32.  m, v and the quantiser use
// separately rounded products and sums (no contraction): which code an element
// gets then depends on its inputs alone.
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>
#include <vector>

#include "rows.cuh"

namespace mole {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnits = 2;                              // units of 4 elements a thread
constexpr int kAdamChunk = 4 * kAdamUnits * kAdamThreads;  // elements a CTA
constexpr int kAdamBlock = 128;                            // elements per scale
constexpr int kAdamTensors = 128;                          // per launch (10 KB of parameters)
constexpr float kInvE4m3Max = (float)(1.0 / 448.0);
constexpr float kScaleFloor = 0x1p-120f;                   // its reciprocal is finite
constexpr float kE4m3Tiny = 0x1p-9f;                       // the smallest nonzero code
constexpr float kEpsMin = 0x1p-126f, kEpsMax = 0x1p125f;   // well inside what fast_rcp has

struct AdamTensor {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float weight_decay;
  int param_bf16, grad_bf16, vec;
};

struct AdamArgs {
  AdamTensor t[kAdamTensors];
  unsigned first[kAdamTensors + 1];  // first chunk of each tensor, and the total
  int n_tensors;
  float b1, omb1, b2, omb2, eps;
  double lr_host, beta1, beta2;  // with step_dev or lr_dev
  float lr, step_size, root;  // lr; lr / (1 - b1^t); 1 / sqrt(1 - b2^t)
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
};

// b^t for t >= 0 by squaring (the same products on the host and the device).
__host__ __device__ inline double int_pow(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

__host__ __device__ inline void step_factors(double lr, double beta1, double beta2, int64_t t, float* step_size,
                                             float* root) {
  *step_size = (float)(lr / (1.0 - int_pow(beta1, t)));
  *root = (float)(1.0 / sqrt(1.0 - int_pow(beta2, t)));
}

// The unit's elements [0, cnt): all 4 with vector accesses (kFull), or one by
// one (a tensor's last elements, tensors of other alignment).
template <bool kFull, class T>
__device__ __forceinline__ void load_unit(const T* p, int cnt, float (&f)[4]) {
  if constexpr (kFull) {
    ld_unit(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = k < cnt ? ld1(p + k) : 0.f;
  }
}
template <bool kFull, class T>
__device__ __forceinline__ void store_unit(T* p, int cnt, const float (&f)[4]) {
  if constexpr (kFull) {
    st_unit(p, f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < cnt) st1(p + k, f[k]);
  }
}

// Four e4m3 codes.
template <bool kFull>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int cnt) {
  if constexpr (kFull) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < cnt) w |= (uint32_t)p[k] << (8 * k);
  return w;
}
template <bool kFull>
__device__ __forceinline__ void store_codes(uint8_t* p, int cnt, uint32_t w) {
  if constexpr (kFull) {
    *reinterpret_cast<uint32_t*>(p) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < cnt) p[k] = (uint8_t)(w >> (8 * k));
  }
}
__device__ __forceinline__ void decode(uint32_t w, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3)));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ uint32_t encode(const float (&f)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 1 / x for x that is infinite, NaN or in [2^-126, 2^126] (1 ulp); subnormal x
// count as zero.
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The scale of a block whose largest magnitude has these bits (a NaN stays one).
__device__ __forceinline__ float block_scale(unsigned bits) {
  const float s = __fmul_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, bits)), kInvE4m3Max);
  return s < kScaleFloor ? kScaleFloor : s;
}

// The tensor of chunk c: the last one whose first chunk is not behind it.
__device__ __forceinline__ int tensor_of(const AdamArgs& a, unsigned c) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < kAdamTensors; i += 32) {
    const int j = i + (threadIdx.x & 31);
    n += __popc(__ballot_sync(0xffffffffu, j < a.n_tensors && a.first[j] <= c));
  }
  return n - 1;
}

// The step's factors: lr, lr / (1 - b1^t), 1 / sqrt(1 - b2^t), the gradients' one.
struct Factors {
  float lr, step_size, root, grad;
};

// The thread's units of a chunk whose first element it has is e0.  kFull: the
// whole chunk lies in the tensor, with vector accesses; its types are template
// parameters then (tests per unit made the 8-bit kernel issue-bound: 89
// instructions an element, 67 now).
template <bool kState8, bool kFull, bool kGradBf16, bool kParamBf16, bool kMaster>
__device__ __forceinline__ void step_chunk(const AdamArgs& a, const AdamTensor& t, const Factors& w, int64_t e0) {
  using G = std::conditional_t<kGradBf16, uint16_t, float>;
  using P = std::conditional_t<kParamBf16, uint16_t, float>;
  float g[kAdamUnits][4], p[kAdamUnits][4], m[kAdamUnits][4], v[kAdamUnits][4];
  uint32_t mc[kAdamUnits], vc[kAdamUnits];
  float sm[kAdamUnits], sv[kAdamUnits];
  int cnt[kAdamUnits];
#pragma unroll
  for (int u = 0; u < kAdamUnits; ++u) {
    const int64_t e = e0 + 4 * u * kAdamThreads;
    cnt[u] = kFull ? 4 : (int)std::min<int64_t>(4, std::max<int64_t>(0, t.n - e));
    load_unit<kFull>(static_cast<const G*>(t.grad) + e, cnt[u], g[u]);
    if constexpr (kMaster)
      load_unit<kFull>(t.master + e, cnt[u], p[u]);
    else
      load_unit<kFull>(static_cast<const P*>(t.param) + e, cnt[u], p[u]);
    if constexpr (kState8) {
      mc[u] = load_codes<kFull>(static_cast<const uint8_t*>(t.m) + e, cnt[u]);
      vc[u] = load_codes<kFull>(static_cast<const uint8_t*>(t.v) + e, cnt[u]);
      sm[u] = cnt[u] > 0 ? t.m_scale[e / kAdamBlock] : 0.f;
      sv[u] = cnt[u] > 0 ? t.v_scale[e / kAdamBlock] : 0.f;
    } else {
      load_unit<kFull>(static_cast<const float*>(t.m) + e, cnt[u], m[u]);
      load_unit<kFull>(static_cast<const float*>(t.v) + e, cnt[u], v[u]);
    }
  }
  const float decay = w.lr * t.weight_decay;
  float r[kAdamUnits][4];
#pragma unroll
  for (int u = 0; u < kAdamUnits; ++u) {
    const int64_t e = e0 + 4 * u * kAdamThreads;
    unsigned m_max = 0, r_max = 0;
    if constexpr (kState8) {
      decode(mc[u], m[u]);
      decode(vc[u], v[u]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (kState8) {
        m[u][k] = __fmul_rn(m[u][k], sm[u]);
        v[u][k] = __fmul_rn(v[u][k], sv[u]);
        v[u][k] = __fmul_rn(v[u][k], v[u][k]);
      }
      g[u][k] *= w.grad;
      m[u][k] = __fadd_rn(__fmul_rn(m[u][k], a.b1), __fmul_rn(g[u][k], a.omb1));
      v[u][k] = __fadd_rn(__fmul_rn(v[u][k], a.b2), __fmul_rn(__fmul_rn(g[u][k], g[u][k]), a.omb2));
      r[u][k] = __fsqrt_rn(v[u][k]);
      // (eps is in [2^-126, 2^125], and the root, up to 2^64, and its factor, up to
      // 2^27, add to it: the reciprocal is finite and not zero but for a v that is
      // not finite, and an m of zero makes a step of zero whatever v and eps)
      const float step = m[u][k] * fast_rcp(fmaf(r[u][k], w.root, a.eps));
      p[u][k] = fmaf(-w.step_size, step, fmaf(-decay, p[u][k], p[u][k]));
      if constexpr (kState8) {
        m_max = max(m_max, __float_as_uint(fabsf(m[u][k])));
        r_max = max(r_max, __float_as_uint(r[u][k]));
      }
    }
    if constexpr (kMaster) store_unit<kFull>(t.master + e, cnt[u], p[u]);
    store_unit<kFull>(static_cast<P*>(t.param) + e, cnt[u], p[u]);
    if constexpr (kState8) {
      sm[u] = block_scale(m_max);
      sv[u] = block_scale(r_max);
    } else {
      store_unit<kFull>(static_cast<float*>(t.m) + e, cnt[u], m[u]);
      store_unit<kFull>(static_cast<float*>(t.v) + e, cnt[u], v[u]);
    }
  }
  if constexpr (kState8) {
    // the scales' reciprocals, correctly rounded: one division for the warp's
    // blocks, a lane each
    static_assert(kAdamUnits == 2, "four scales");
    const int lane = threadIdx.x & 31;
    const float own = lane & 1 ? (lane & 2 ? sv[1] : sv[0]) : (lane & 2 ? sm[1] : sm[0]);
    const float inv = __frcp_rn(own);
#pragma unroll
    for (int u = 0; u < kAdamUnits; ++u) {
      const int64_t e = e0 + 4 * u * kAdamThreads;
      const float im = __shfl_sync(0xffffffffu, inv, 2 * u), iv = __shfl_sync(0xffffffffu, inv, 2 * u + 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[u][k] = __fmul_rn(m[u][k], im);
        const float q = __fmul_rn(r[u][k], iv);
        v[u][k] = r[u][k] > 0.f && q < kE4m3Tiny ? kE4m3Tiny : q;
      }
      store_codes<kFull>(static_cast<uint8_t*>(t.m) + e, cnt[u], encode(m[u]));
      store_codes<kFull>(static_cast<uint8_t*>(t.v) + e, cnt[u], encode(v[u]));
      if (cnt[u] > 0 && lane == 0) {
        t.m_scale[e / kAdamBlock] = sm[u];
        t.v_scale[e / kAdamBlock] = sv[u];
      }
    }
  }
}

template <bool kState8, bool kFull>
__device__ __forceinline__ void step_types(const AdamArgs& a, const AdamTensor& t, const Factors& w, int64_t e0) {
  if (t.grad_bf16) {
    if (t.master)
      step_chunk<kState8, kFull, true, true, true>(a, t, w, e0);
    else if (t.param_bf16)
      step_chunk<kState8, kFull, true, true, false>(a, t, w, e0);
    else
      step_chunk<kState8, kFull, true, false, false>(a, t, w, e0);
  } else {
    if (t.master)
      step_chunk<kState8, kFull, false, true, true>(a, t, w, e0);
    else if (t.param_bf16)
      step_chunk<kState8, kFull, false, true, false>(a, t, w, e0);
    else
      step_chunk<kState8, kFull, false, false, false>(a, t, w, e0);
  }
}

// CTAs per SM (the registers that a thread gets): 185 M elements, one step on an
// idle GPU and (in brackets) steps without a pause, at the clocks that the power
// limit leaves.  8-bit states: 524 us (582) at 4 (64 registers), 510 (561) at 5
// (48, 120 bytes of spill stores), 612 (695) at 6 (40, 624 bytes); two elements an
// instruction (fp32x2) is slower, (640).  fp32 states: 813 us (815) at 3, 821
// (822) at 4, 836 (840) at 5.
template <bool kState8>
__global__ void __launch_bounds__(kAdamThreads, kState8 ? 5 : 3) adamw_kernel(const __grid_constant__ AdamArgs a) {
  __shared__ float factors[3];
  Factors w{a.lr, a.step_size, a.root, a.grad_scale ? *a.grad_scale : 1.f};
  if (a.step_dev || a.lr_dev) {
    if (threadIdx.x == 0) {
      const double l = a.lr_dev ? (double)*a.lr_dev : a.lr_host;
      factors[0] = (float)l;
      step_factors(l, a.beta1, a.beta2, a.step_dev ? *a.step_dev : a.step, &factors[1], &factors[2]);
    }
    __syncthreads();
    w.lr = factors[0];
    w.step_size = factors[1];
    w.root = factors[2];
  }
  const unsigned total = a.first[a.n_tensors];
  for (unsigned c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = tensor_of(a, c);
    const AdamTensor& t = a.t[i];
    const int64_t start = (int64_t)(c - a.first[i]) * kAdamChunk;
    if (t.vec && start + kAdamChunk <= t.n)
      step_types<kState8, true>(a, t, w, start + 4 * threadIdx.x);
    else
      step_types<kState8, false>(a, t, w, start + 4 * threadIdx.x);
  }
}

struct Range {
  uintptr_t lo, hi;
  bool written;
};

// Whether memory that the step writes overlaps any other of its memory.
bool overlapping(std::vector<Range>& r) {
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
  uintptr_t written_to = 0, used_to = 0;  // ends of the ranges so far
  for (const Range& x : r) {
    if (x.lo < written_to || (x.written && x.lo < used_to)) return true;
    used_to = std::max(used_to, x.hi);
    if (x.written) written_to = std::max(written_to, x.hi);
  }
  return false;
}

mole_status check_adamw(const mole_adamw_tensor* tensors, int32_t n_tensors, const mole_adamw_config* c) {
  if (n_tensors < 0 || !c || (n_tensors > 0 && !tensors)) return MOLE_ERR_ARG;
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0) ||
      !(c->eps >= 0.0 && c->eps <= (double)kEpsMax))
    return MOLE_ERR_ARG;
  if (!c->step_dev && c->step < 1) return MOLE_ERR_ARG;
  if (c->state8 != 0 && c->state8 != 1) return MOLE_ERR_ARG;
  if (!aligned_to(c->step_dev, 8) || !aligned_to(c->lr_dev, 4) || !aligned_to(c->grad_scale_dev, 4))
    return MOLE_ERR_ALIGN;
  std::vector<Range> ranges;
  ranges.reserve((size_t)n_tensors * 7 + 3);
  auto add = [&ranges](const void* p, int64_t bytes, bool written) {
    if (p) ranges.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes, written});
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    const mole_adamw_tensor& t = tensors[i];
    if (t.n < 0 || (t.dt_param != MOLE_F32 && t.dt_param != MOLE_BF16) ||
        (t.dt_grad != MOLE_F32 && t.dt_grad != MOLE_BF16))
      return MOLE_ERR_ARG;
    if (t.n == 0) continue;
    if (t.n > ((int64_t)1 << 40)) return MOLE_ERR_UNSUPPORTED;
    if (!t.param || !t.grad || !t.m || !t.v || (t.master && t.dt_param == MOLE_F32)) return MOLE_ERR_ARG;
    if (c->state8 ? (!t.m_scale || !t.v_scale) : (t.m_scale || t.v_scale)) return MOLE_ERR_ARG;
    const int64_t sp = t.dt_param == MOLE_BF16 ? 2 : 4, sg = t.dt_grad == MOLE_BF16 ? 2 : 4, ss = c->state8 ? 1 : 4;
    if (!aligned_to(t.param, sp) || !aligned_to(t.grad, sg) || !aligned_to(t.master, 4) || !aligned_to(t.m, ss) ||
        !aligned_to(t.v, ss) || !aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4))
      return MOLE_ERR_ALIGN;
    add(t.param, t.n * sp, true);
    add(t.grad, t.n * sg, false);
    add(t.master, t.n * 4, true);
    add(t.m, t.n * ss, true);
    add(t.v, t.n * ss, true);
    const int64_t blocks = (t.n + kAdamBlock - 1) / kAdamBlock;
    add(t.m_scale, blocks * 4, true);
    add(t.v_scale, blocks * 4, true);
  }
  add(c->step_dev, 8, false);
  add(c->lr_dev, 4, false);
  add(c->grad_scale_dev, 4, false);
  return overlapping(ranges) ? MOLE_ERR_ARG : MOLE_OK;
}

mole_status run_adamw(const mole_adamw_tensor* tensors, int32_t n_tensors, const mole_adamw_config* c, int n_sm,
                      cudaStream_t stream) {
  AdamArgs a{};
  a.b1 = (float)c->beta1;
  a.omb1 = (float)(1.0 - c->beta1);
  a.b2 = (float)c->beta2;
  a.omb2 = (float)(1.0 - c->beta2);
  a.eps = std::max((float)c->eps, kEpsMin);
  a.beta1 = c->beta1;
  a.beta2 = c->beta2;
  a.lr_host = c->lr;
  a.lr = (float)c->lr;
  a.step = c->step;
  a.step_dev = c->step_dev;
  a.lr_dev = c->lr_dev;
  a.grad_scale = c->grad_scale_dev;
  if (!c->step_dev && !c->lr_dev) step_factors(c->lr, c->beta1, c->beta2, c->step, &a.step_size, &a.root);
  const size_t state_align = c->state8 ? 4 : 16;  // of a unit's 4 elements
  auto launch = [&]() -> mole_status {
    if (a.n_tensors == 0) return MOLE_OK;
    const unsigned grid = std::min<unsigned>(a.first[a.n_tensors], (unsigned)n_sm * 256u);
    if (c->state8)
      adamw_kernel<true><<<grid, kAdamThreads, 0, stream>>>(a);
    else
      adamw_kernel<false><<<grid, kAdamThreads, 0, stream>>>(a);
    a.n_tensors = 0;
    return cuda_status(cudaGetLastError());
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    const mole_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t chunks = (t.n + kAdamChunk - 1) / kAdamChunk;
    if (a.n_tensors == kAdamTensors || (a.n_tensors > 0 && a.first[a.n_tensors] + chunks > (int64_t)INT32_MAX)) {
      const mole_status st = launch();
      if (st != MOLE_OK) return st;
    }
    AdamTensor& d = a.t[a.n_tensors];
    d = {t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay, t.dt_param == MOLE_BF16,
         t.dt_grad == MOLE_BF16,
         aligned_rows(t.param, t.dt_param == MOLE_BF16) && aligned_rows(t.grad, t.dt_grad == MOLE_BF16) &&
             aligned16(t.master) && aligned_to(t.m, state_align) && aligned_to(t.v, state_align)};
    a.first[a.n_tensors + 1] = a.first[a.n_tensors] + (unsigned)chunks;
    ++a.n_tensors;
  }
  return launch();
}

}  // namespace
}  // namespace mole

extern "C" mole_status mole_adamw_step(const mole_adamw_tensor* tensors, int32_t n_tensors,
                                       const mole_adamw_config* config, cudaStream_t stream) {
  try {
    mole_status st = mole::check_adamw(tensors, n_tensors, config);
    if (st != MOLE_OK || n_tensors == 0) return st;
    st = mole::check_device();
    if (st != MOLE_OK) return st;
    const int n_sm = mole::num_sms();
    if (n_sm <= 0) return MOLE_ERR_NO_DEVICE;
    return mole::run_adamw(tensors, n_tensors, config, n_sm, stream);
  } catch (...) {  // no host memory for the check's list
    return MOLE_ERR_CUDA;
  }
}
