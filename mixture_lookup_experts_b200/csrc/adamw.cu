// adamw.cu -- one AdamW step over a list of tensors (mole.h states the
// formulas).  MoLE page, 训练阶段: the layer is trained end to end; this is the
// step that consumes the gradients which the backward calls add up in fp32.
//
// Elementwise, so bound by HBM: per element the gradient (4 or 2 bytes), the
// weight (bf16 with an fp32 master: 10 bytes moved, fp32: 8, bf16 alone: 4) and
// the states (fp32: 16, 8 bits: 4 + 16 / 128).  One launch serves up to 64
// tensors: their addresses travel in the kernel's parameters, and the work is
// cut into chunks of kChunk elements, each inside one tensor.
//
// 8-bit states: a block of 128 consecutive elements is 16 lanes of 8 elements,
// so its largest value takes four shuffles.  m and sqrt(v) are e4m3 times an
// fp32 scale; keeping the root halves the exponents that the codes must span.
// The update of a block reads codes and writes codes; in between everything is
// fp32.  m, v and the quantiser use separately rounded products and sums (no
// contraction): which code an element gets then depends on its inputs alone.
#include <cuda_fp8.h>

#include <cmath>
#include <vector>

#include "rows.cuh"

namespace mole {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = 8;                          // elements a thread
constexpr int kAdamChunk = kAdamThreads * kAdamUnit;  // elements a CTA
constexpr int kAdamBlock = 128;                       // elements per scale
constexpr int kAdamTensors = 64;                      // per launch
constexpr float kInvE4m3Max = (float)(1.0 / 448.0);
constexpr float kScaleFloor = 0x1p-120f;              // its reciprocal is finite
constexpr float kE4m3Tiny = 0x1p-9f;                  // the smallest nonzero code

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

// Elements [0, cnt) of the thread's 8 (cnt = 8 unless the tensor ends here).
template <class T>
__device__ __forceinline__ void load_unit(const T* p, int cnt, bool vec, float (&f)[8]) {
  if (vec && cnt == 8) {
    ld_vec8(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < cnt ? ld1(p + k) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store_unit(T* p, int cnt, bool vec, const float (&f)[8]) {
  if (vec && cnt == 8) {
    st_vec8(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cnt) st1(p + k, f[k]);
  }
}

__device__ __forceinline__ float2 e4m3_pair(uint16_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
  return __half22float2(__half2(h));
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int cnt, bool vec, float (&f)[8]) {
  uint32_t w[2] = {0, 0};
  if (vec && cnt == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cnt) w[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = e4m3_pair((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int cnt, bool vec, const float (&f)[8]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= c << (16 * (i & 1));
  }
  if (vec && cnt == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cnt) p[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
}

// The largest of a block's values (16 lanes; NaN where one is NaN).
__device__ __forceinline__ float block_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = (u > v || u != u) ? u : v;
  }
  return v;
}

template <bool kState8>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamArgs a) {
  __shared__ float factors[3];
  if (threadIdx.x == 0) {
    float lr = a.lr, step_size = a.step_size, root = a.root;
    if (a.step_dev || a.lr_dev) {
      const double l = a.lr_dev ? (double)*a.lr_dev : a.lr_host;
      lr = (float)l;
      step_factors(l, a.beta1, a.beta2, a.step_dev ? *a.step_dev : a.step, &step_size, &root);
    }
    factors[0] = lr;
    factors[1] = step_size;
    factors[2] = root;
  }
  __syncthreads();
  const float lr = factors[0], step_size = factors[1], root = factors[2];
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const unsigned total = a.first[a.n_tensors];
  for (unsigned c = blockIdx.x; c < total; c += gridDim.x) {
    int i = 0, end = a.n_tensors;  // the tensor i with first[i] <= c < first[i + 1]
    while (end - i > 1) {
      const int mid = (i + end) >> 1;
      if (a.first[mid] <= c)
        i = mid;
      else
        end = mid;
    }
    const AdamTensor& t = a.t[i];
    const int64_t e0 = (int64_t)(c - a.first[i]) * kAdamChunk + kAdamUnit * threadIdx.x;
    const int cnt = (int)std::min<int64_t>(kAdamUnit, std::max<int64_t>(0, t.n - e0));
    const bool vec = t.vec != 0;
    float g[8], p[8], m[8], v[8];
    if (t.grad_bf16)
      load_unit(static_cast<const uint16_t*>(t.grad) + e0, cnt, vec, g);
    else
      load_unit(static_cast<const float*>(t.grad) + e0, cnt, vec, g);
    if (t.master)
      load_unit(t.master + e0, cnt, vec, p);
    else if (t.param_bf16)
      load_unit(static_cast<const uint16_t*>(t.param) + e0, cnt, vec, p);
    else
      load_unit(static_cast<const float*>(t.param) + e0, cnt, vec, p);
    const int64_t block = e0 / kAdamBlock;
    if constexpr (kState8) {
      load_codes(static_cast<const uint8_t*>(t.m) + e0, cnt, vec, m);
      load_codes(static_cast<const uint8_t*>(t.v) + e0, cnt, vec, v);
      const float sm = cnt > 0 ? t.m_scale[block] : 0.f, sv = cnt > 0 ? t.v_scale[block] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = __fmul_rn(m[k], sm);
        v[k] = __fmul_rn(v[k], sv);
        v[k] = __fmul_rn(v[k], v[k]);
      }
    } else {
      load_unit(static_cast<const float*>(t.m) + e0, cnt, vec, m);
      load_unit(static_cast<const float*>(t.v) + e0, cnt, vec, v);
    }
    const float decay = lr * t.weight_decay;
    float m_max = 0.f, r_max = 0.f;
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] *= gs;
      m[k] = __fadd_rn(__fmul_rn(m[k], a.b1), __fmul_rn(g[k], a.omb1));
      v[k] = __fadd_rn(__fmul_rn(v[k], a.b2), __fmul_rn(__fmul_rn(g[k], g[k]), a.omb2));
      r[k] = __fsqrt_rn(v[k]);
      p[k] = p[k] - p[k] * decay - step_size * (m[k] / fmaf(r[k], root, a.eps));
      if constexpr (kState8) {
        const float am = fabsf(m[k]);
        m_max = (am > m_max || am != am) ? am : m_max;
        r_max = (r[k] > r_max || r[k] != r[k]) ? r[k] : r_max;
      }
    }
    if (t.master) store_unit(t.master + e0, cnt, vec, p);
    if (t.param_bf16)
      store_unit(static_cast<uint16_t*>(t.param) + e0, cnt, vec, p);
    else
      store_unit(static_cast<float*>(t.param) + e0, cnt, vec, p);
    if constexpr (kState8) {
      m_max = __fmul_rn(block_max(m_max), kInvE4m3Max);
      r_max = __fmul_rn(block_max(r_max), kInvE4m3Max);
      const float sm = m_max < kScaleFloor ? kScaleFloor : m_max, sv = r_max < kScaleFloor ? kScaleFloor : r_max;
      const float im = __frcp_rn(sm), iv = __frcp_rn(sv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = __fmul_rn(m[k], im);
        const float q = __fmul_rn(r[k], iv);
        v[k] = r[k] > 0.f && q < kE4m3Tiny ? kE4m3Tiny : q;
      }
      store_codes(static_cast<uint8_t*>(t.m) + e0, cnt, vec, m);
      store_codes(static_cast<uint8_t*>(t.v) + e0, cnt, vec, v);
      if (cnt > 0 && (threadIdx.x & 15) == 0) {
        t.m_scale[block] = sm;
        t.v_scale[block] = sv;
      }
    } else {
      store_unit(static_cast<float*>(t.m) + e0, cnt, vec, m);
      store_unit(static_cast<float*>(t.v) + e0, cnt, vec, v);
    }
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
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0) || !(c->eps >= 0.0))
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
  a.eps = (float)c->eps;
  a.beta1 = c->beta1;
  a.beta2 = c->beta2;
  a.lr_host = c->lr;
  a.lr = (float)c->lr;
  a.step = c->step;
  a.step_dev = c->step_dev;
  a.lr_dev = c->lr_dev;
  a.grad_scale = c->grad_scale_dev;
  if (!c->step_dev && !c->lr_dev) step_factors(c->lr, c->beta1, c->beta2, c->step, &a.step_size, &a.root);
  const size_t state_align = c->state8 ? 8 : 16;
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
         aligned16(t.param) && aligned16(t.grad) && aligned16(t.master) && aligned_to(t.m, state_align) &&
             aligned_to(t.v, state_align)};
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
