// norm.cu -- the norms around a block, with its gate and the residual scale,
// forward and backward (mole.h states the formulas).  MoLE page, 训练阶段: a
// layer's router and shared expert read the previous layer's output; what lies
// between two blocks' GEMMs is one pass over the token rows:
//     y = w_post f / rms(f),  x' = beta x + gate y,  h = w_pre x' / rms(x')
// A token's row is held in registers, up to 16 columns a thread, by a CTA of one
// to 16 warps; the row's sums are reduced by shuffles and (beyond one warp)
// shared memory.  Each tensor is read and written once: both kernels are bound
// by HBM (16384 x 2048 fp32: forward 73 to 76 us, backward 127 to 129 us and 6 us
// for the weight gradients' join; 71.7 and 123 us at the copy rate).
//
// Backward, per token (n = D, r = 1/rms):
//     G  = dx' + r_x (a - x^ <a, x^>/n)      a = dh w_pre,  x^ = x' r_x
//     dx = beta G
//     df = r_f (b - f^ <b, f^>/n)            b = gate G w_post,  f^ = f r_f
//     dgate = <G w_post, f^>
// so two reductions: (sum x'^2, sum a x', sum f^2), then <G w_post, f>.  The
// norms' statistics come from the rows themselves (they are read anyway); no
// forward state is kept.  dw_pre and dw_post: a thread adds its columns over
// its CTA's rows in registers; the CTAs' sums go to the workspace and
// norm_reduce_kernel adds them in order.
#include "rows.cuh"

namespace mole {
namespace {

constexpr int kRowThreads = 256, kMaxRowThreads = 512;  // a row's threads, up to 4096 columns and beyond
constexpr int64_t kMaxNormD = 16 * kMaxRowThreads;
constexpr int kStages = 2;
constexpr int64_t kFewRows = 148 * 16;
constexpr int kReduceUnits = 8, kReduceRows = 128;  // 32 columns and 32 warps a CTA

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of K <= 4 values over the CTA's threads (a multiple of 32), in a fixed
// order.  `red` holds a float4 per warp of the CTA (K == 1: a float); a call
// that reuses it comes at least one other call (one barrier) later.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float4* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5;
  if constexpr (K == 1) {
    // (what pads the warps to a multiple of 4 is left out of the sum)
    const int quads = (warps + 3) >> 2;
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(red)[warp] = v[0];
    __syncthreads();
    float sum = 0.f;
    for (int q = 0; q < quads; ++q) {
      const float4 x = red[q];
      sum += x.x;
      if (4 * q + 1 < warps) sum += x.y;
      if (4 * q + 2 < warps) sum += x.z;
      if (4 * q + 3 < warps) sum += x.w;
    }
    v[0] = sum;
  } else {
    if ((threadIdx.x & 31) == 0)
      red[warp] = make_float4(v[0], v[1], K > 2 ? v[K > 2 ? 2 : 0] : 0.f, K > 3 ? v[K > 3 ? 3 : 0] : 0.f);
    __syncthreads();
    float4 sum = red[0];
    for (int w = 1; w < warps; ++w) {
      const float4 x = red[w];
      sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
    }
    const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = out[k];
  }
}

// How the threads have a row's columns: as single elements, or in units of 4
// with vector accesses (rows.cuh).  kUnits: every row starts on a unit (D a
// multiple of 4).  kShifted: the tensors do but not every row: units are those
// of the memory, the first one of a row begins up to 3 columns before it, and
// the last one ends behind it.  The shift is (t D) mod 4, so a CTA whose rows
// are a multiple of 4 apart has one shift, and a thread the same columns, for
// all of them.
enum Form { kElements, kShifted, kUnits };

// The CTA's shift.
template <Form kForm>
__device__ __forceinline__ int first_column(int D) {
  if (kForm == kElements) return (int)threadIdx.x;
  return 4 * (int)threadIdx.x - (kForm == kShifted ? (int)(((int64_t)blockIdx.x * D) & 3) : 0);
}

// A thread's columns of a row on their way through shared memory (cp.async;
// each thread reads back its own copies only).  at: the thread's place in the
// stage's area of this tensor, which lies there as in the row; row: the row's
// first element.  What lies behind the row is neither read nor left to chance (0);
// what lies before it is the end of the row before, left out by stage_get.
template <Form kForm, int kSure, int C, class T>
__device__ __forceinline__ void stage_put(uint8_t* at, const T* row, int col0, int step, int D) {
#pragma unroll
  for (int u = 0; u < C / 4; ++u) {
    const int col = col0 + 4 * u * step;
    if (u < kSure)
      cp_async<4 * sizeof(T)>(at + u * step * 4 * sizeof(T), row + col);
    else if (col < D)
      cp_async<4 * sizeof(T), kForm == kShifted>(at + u * step * 4 * sizeof(T), row + col,
                                                 (int)sizeof(T) * std::min(4, D - col));
  }
}
template <Form kForm, int kSure, int C, class T>
__device__ __forceinline__ void stage_get(const uint8_t* at, int col0, int step, int D, float (&f)[C]) {
#pragma unroll
  for (int u = 0; u < C / 4; ++u) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (u < kSure || col0 + 4 * u * step < D) ld_unit(reinterpret_cast<const T*>(at + u * step * 4 * sizeof(T)), x);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[4 * u + k] = kForm == kShifted && u == 0 && col0 + k < 0 ? 0.f : x[k];
  }
}

// A weight vector, whose units are not those of the rows where these are
// shifted: the thread's columns then lie in shared memory (`at`), as the stages'.
template <Form kForm, int C>
__device__ __forceinline__ void weight_put(uint8_t* at, const float* w, int col0, int step, int D) {
  if constexpr (kForm == kShifted) {
    if (!w) return;
#pragma unroll
    for (int u = 0; u < C / 4; ++u) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = col0 + 4 * u * step + k;
        x[k] = col >= 0 && col < D ? w[col] : 0.f;
      }
      st_unit(reinterpret_cast<float*>(at + u * step * 16), x[0], x[1], x[2], x[3]);
    }
  }
}
template <Form kForm, int kSure, int C>
__device__ __forceinline__ void weight_get(const uint8_t* at, const float* w, int col0, int step, int D,
                                           float (&f)[C]) {
  if constexpr (kForm == kShifted) {
#pragma unroll
    for (int u = 0; u < C / 4; ++u) {
      float x[4];
      ld_unit(reinterpret_cast<const float*>(at + u * step * 16), x);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[4 * u + k] = x[k];
    }
  } else {
    ld_cols<kForm == kUnits, C, float, kSure>(w, col0, step, D, f);
  }
}

// The thread's columns to a row whose first element is at `row`.
template <Form kForm, int kSure, int C, class T>
__device__ __forceinline__ void store_row(T* row, int col0, int step, int D, const float (&f)[C]) {
  if constexpr (kForm == kShifted) {
#pragma unroll
    for (int u = 0; u < C / 4; ++u) {
      const int col = col0 + 4 * u * step;
      if ((u > 0 || col >= 0) && (u < kSure || col + 4 <= D)) {
        st_unit(row + col, f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (col + k >= 0 && col + k < D) st1(row + col + k, f[4 * u + k]);
      }
    }
  } else {
    st_cols<kForm == kUnits, C, T, kSure>(row, col0, step, D, f);
  }
}

struct NormFwd {
  const void* x;
  const void* f;
  const float* w_post;
  const float* gate;
  const float* w_pre;
  float res_scale, eps;
  int64_t T;
  int D;
  void* x_out;
  void* h;
};

// A CTA has a row at a time, C columns a thread.  kStages > 0: rows come through
// shared memory, kStages - 1 of them ahead of the one in work (loads of a row
// then overlap the sums and stores of the one before); kStages == 0: straight
// into registers.  Stages and registers together: rows of 16 columns a thread
// have 3 stages (16384 x 2048 fp32 75 to 76 us whatever the tensors' addresses;
// with 2, 74 to 86), fewer columns 2 (16384 x 768 32.5 us, with 3 34.2); 85
// registers a thread leave room for 6 CTAs of 4 warps.
template <Form kForm, int C, int kStages, int kThreads, class X, class F, class H>
__global__ void __launch_bounds__(kThreads, kThreads == kMaxRowThreads ? 1 : kForm == kElements ? 4 : 3)
    norm_forward_kernel(const NormFwd a) {
  constexpr int kSure = kForm != kElements ? C / 4 - 1 : 0;
  static_assert(kForm != kShifted || kStages > 0, "shifted units only through shared memory");
  __shared__ float4 red[2][2][kMaxRowThreads / 32];
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const int step = blockDim.x, D = a.D;
  const int c0 = first_column<kForm>(D);
  const float inv_d = 1.f / (float)D;
  const X* x_in = static_cast<const X*>(a.x);
  const F* f_in = static_cast<const F*>(a.f);
  const int stage_bytes = step * C * (int)(sizeof(X) + sizeof(F));
  const int at0 = 4 * (int)threadIdx.x, x_at = at0 * (int)sizeof(X),
            f_at = step * C * (int)sizeof(X) + at0 * (int)sizeof(F);
  [[maybe_unused]] uint8_t* post_at = norm_smem + kStages * stage_bytes + 4 * at0;  // kShifted: the weights
  [[maybe_unused]] uint8_t* pre_at = post_at + step * C * 4;
  const int64_t stride = gridDim.x;
  int64_t t = blockIdx.x;
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.T) {
      uint8_t* at = norm_smem + stage * stage_bytes;
      stage_put<kForm, kSure, C>(at + x_at, x_in + row * D, c0, step, D);
      if (f_in) stage_put<kForm, kSure, C>(at + f_at, f_in + row * D, c0, step, D);
    }
    cp_async_commit();
  };
  if constexpr (kStages > 0) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(t + k * stride, k);
  }
  weight_put<kForm, C>(post_at, a.w_post, c0, step, D);
  weight_put<kForm, C>(pre_at, a.w_pre, c0, step, D);
  int stage = 0, parity = 0;
  for (; t < a.T; t += stride, parity ^= 1) {
    float x[C], f[C];
    float s[1] = {0.f};
    if constexpr (kStages > 0) {
      fetch(t + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_wait<kStages - 1>();
      const uint8_t* at = norm_smem + stage * stage_bytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      stage_get<kForm, kSure, C, X>(at + x_at, c0, step, D, x);
      if (f_in) stage_get<kForm, kSure, C, F>(at + f_at, c0, step, D, f);
    } else {
      ld_cols<kForm == kUnits, C, X, kSure>(x_in + t * D, c0, step, D, x);
      if (f_in) ld_cols<kForm == kUnits, C, F, kSure>(f_in + t * D, c0, step, D, f);
    }
    if (f_in) {
      const float g = a.gate ? a.gate[t] : 1.f;
      if (a.w_post) {
        float w[C];
        weight_get<kForm, kSure>(post_at, a.w_post, c0, step, D, w);
#pragma unroll
        for (int k = 0; k < C; ++k) s[0] = fmaf(f[k], f[k], s[0]);
        row_sums(s, red[parity][0]);
        const float r = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
        for (int k = 0; k < C; ++k) f[k] = f[k] * r * w[k];
      }
#pragma unroll
      for (int k = 0; k < C; ++k) x[k] = fmaf(g, f[k], a.res_scale * x[k]);
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) x[k] *= a.res_scale;
    }
    if (a.x_out) store_row<kForm, kSure>(static_cast<X*>(a.x_out) + t * D, c0, step, D, x);
    if (a.h) {
      float w[C];
      weight_get<kForm, kSure>(pre_at, a.w_pre, c0, step, D, w);
      s[0] = 0.f;
#pragma unroll
      for (int k = 0; k < C; ++k) s[0] = fmaf(x[k], x[k], s[0]);
      row_sums(s, red[parity][1]);
      const float r = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
      for (int k = 0; k < C; ++k) w[k] *= x[k] * r;
      store_row<kForm, kSure>(static_cast<H*>(a.h) + t * D, c0, step, D, w);
    }
  }
  if constexpr (kStages > 0) cp_async_wait<0>();
}

// The CTA's sums to its row of the partial ones (if there are such), each of
// which starts on a unit: shifted columns go there one by one.
template <Form kForm, int C>
__device__ __forceinline__ void store_part(float* part, int col0, int step, int D, const float (&f)[C]) {
  if (!part) return;
  float* row = part + (int64_t)blockIdx.x * ((D + 3) & ~3);
  if constexpr (kForm == kShifted) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int col = col0 + 4 * (k / 4) * step + k % 4;
      if (col >= 0 && col < D) row[col] = f[k];
    }
  } else {
    st_cols<kForm == kUnits>(row, col0, step, D, f);
  }
}

struct NormBwd {
  const void* x;
  const void* f;
  const float* w_post;
  const float* gate;
  const float* w_pre;
  float res_scale, eps;
  int64_t T;
  int D;
  const float* dx_out;
  const float* dh;
  float* dx;
  float* df;
  float* dgate;
  float* part_post;  // [gridDim.x][D rounded up to 4] or null
  float* part_pre;
};

// kAll: every input but the gate is there, and dx and df are wanted (a training
// step's call; fewer tests).
template <Form kForm, bool kAll, int C, int kStages, int kThreads, class X, class F>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormBwd a) {
  constexpr int kSure = kForm != kElements ? C / 4 - 1 : 0;
  static_assert(kForm != kShifted || kStages > 0, "shifted units only through shared memory");
  __shared__ float4 red[2][2][kMaxRowThreads / 32];
  extern __shared__ __align__(16) uint8_t norm_smem[];
  // norm_reduce_kernel may take its place (only it: another kernel behind this
  // one might not wait for it)
  if (a.part_pre || a.part_post) pdl_trigger();
  const int step = blockDim.x, D = a.D;
  const int c0 = first_column<kForm>(D);
  const float inv_d = 1.f / (float)D;
  const bool has_h = kAll || a.dh, has_xo = kAll || a.dx_out, has_f = kAll || a.f, post = kAll || a.w_post;
  const X* x_in = static_cast<const X*>(a.x);
  const F* f_in = static_cast<const F*>(a.f);
  // a stage: dh, dx_out, x, f
  const int at0 = 4 * (int)threadIdx.x, h_at = 4 * at0, g_at = step * C * 4 + 4 * at0,
            x_at = step * C * 8 + at0 * (int)sizeof(X),
            f_at = step * C * (8 + (int)sizeof(X)) + at0 * (int)sizeof(F),
            stage_bytes = step * C * (8 + (int)(sizeof(X) + sizeof(F)));
  [[maybe_unused]] uint8_t* post_at = norm_smem + kStages * stage_bytes + 4 * at0;  // kShifted: the weights
  [[maybe_unused]] uint8_t* pre_at = post_at + step * C * 4;
  const int64_t stride = gridDim.x;
  int64_t t = blockIdx.x;
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.T) {
      uint8_t* at = norm_smem + stage * stage_bytes;
      const int64_t off = row * D;
      if (has_h) {
        stage_put<kForm, kSure, C>(at + h_at, a.dh + off, c0, step, D);
        stage_put<kForm, kSure, C>(at + x_at, x_in + off, c0, step, D);
      }
      if (has_xo) stage_put<kForm, kSure, C>(at + g_at, a.dx_out + off, c0, step, D);
      if (has_f) stage_put<kForm, kSure, C>(at + f_at, f_in + off, c0, step, D);
    }
    cp_async_commit();
  };
  if constexpr (kStages > 0) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(t + k * stride, k);
  }
  weight_put<kForm, C>(post_at, a.w_post, c0, step, D);
  weight_put<kForm, C>(pre_at, a.w_pre, c0, step, D);
  float acc_pre[C], acc_post[C];
#pragma unroll
  for (int k = 0; k < C; ++k) acc_pre[k] = acc_post[k] = 0.f;
  int stage = 0, parity = 0;
  for (; t < a.T; t += stride, parity ^= 1) {
    float x[C], f[C], dh[C], G[C];
    if constexpr (!kAll) {
#pragma unroll
      for (int k = 0; k < C; ++k) x[k] = f[k] = dh[k] = G[k] = 0.f;
    }
    if constexpr (kStages > 0) {
      fetch(t + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_wait<kStages - 1>();
      const uint8_t* at = norm_smem + stage * stage_bytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (has_h) {
        stage_get<kForm, kSure, C, float>(at + h_at, c0, step, D, dh);
        stage_get<kForm, kSure, C, X>(at + x_at, c0, step, D, x);
      }
      if (has_xo) stage_get<kForm, kSure, C, float>(at + g_at, c0, step, D, G);
      if (has_f) stage_get<kForm, kSure, C, F>(at + f_at, c0, step, D, f);
    } else {
      if (has_h) {
        ld_cols<kForm == kUnits, C, float, kSure>(a.dh + t * D, c0, step, D, dh);
        ld_cols<kForm == kUnits, C, X, kSure>(x_in + t * D, c0, step, D, x);
      }
      if (has_xo) ld_cols<kForm == kUnits, C, float, kSure>(a.dx_out + t * D, c0, step, D, G);
      if (has_f) ld_cols<kForm == kUnits, C, F, kSure>(f_in + t * D, c0, step, D, f);
    }
    const float g = a.gate ? a.gate[t] : 1.f;
    float w[C];
    float s[3] = {0.f, 0.f, 0.f};
    if (has_h) {
      weight_get<kForm, kSure>(pre_at, a.w_pre, c0, step, D, w);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        s[0] = fmaf(x[k], x[k], s[0]);
        w[k] *= dh[k];
        s[1] = fmaf(w[k], x[k], s[1]);
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) s[2] = fmaf(f[k], f[k], s[2]);
    row_sums(s, red[parity][0]);
    const float rf = post ? rsqrtf(fmaf(s[2], inv_d, a.eps)) : 1.f;
    if (has_h) {
      const float rx = rsqrtf(fmaf(s[0], inv_d, a.eps));
      const float cx = rx * rx * (s[1] * inv_d);  // <a, x^> / n = rx s1 / n; x^ = rx x'
#pragma unroll
      for (int k = 0; k < C; ++k) {
        acc_pre[k] = fmaf(dh[k], x[k] * rx, acc_pre[k]);
        G[k] = fmaf(rx, fmaf(-cx, x[k], w[k]), G[k]);
      }
    }
    // f becomes f^ (f itself without a post-norm); dh becomes G w_post
    if (post) {
      weight_get<kForm, kSure>(post_at, a.w_post, c0, step, D, w);
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) w[k] = 1.f;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < C; ++k) {
      f[k] *= rf;
      acc_post[k] = fmaf(g * G[k], f[k], acc_post[k]);
      dh[k] = G[k] * w[k];
      q[0] = fmaf(dh[k], f[k], q[0]);
    }
    if (kAll || a.dx) {
#pragma unroll
      for (int k = 0; k < C; ++k) G[k] *= a.res_scale;
      store_row<kForm, kSure>(a.dx + t * D, c0, step, D, G);
    }
    if (has_f) {
      row_sums(q, red[parity][1]);
      if (a.dgate && threadIdx.x == 0) a.dgate[t] = q[0];
    }
    if (kAll || a.df) {
      const float cf = post ? -(q[0] * inv_d) : 0.f, gr = g * rf;
#pragma unroll
      for (int k = 0; k < C; ++k) dh[k] = gr * fmaf(cf, f[k], dh[k]);
      store_row<kForm, kSure>(a.df + t * D, c0, step, D, dh);
    }
  }
  if constexpr (kStages > 0) cp_async_wait<0>();
  store_part<kForm>(a.part_pre, c0, step, D, acc_pre);
  store_part<kForm>(a.part_post, c0, step, D, acc_post);
}

// dw[d] += sum over the CTAs' rows, in a fixed order: 4 columns a thread, 128
// rows side by side, then 32 sums per column from shared memory.  blockIdx.y:
// 0 = dw_pre, 1 = dw_post.  Rows are `ld` floats apart (a multiple of 4).
__global__ void __launch_bounds__(kReduceUnits* kReduceRows)
    norm_reduce_kernel(const float* part_pre, const float* part_post, int rows, int D, int ld, float* dw_pre,
                       float* dw_post) {
  constexpr int kCols = 4 * kReduceUnits;
  __shared__ float s[kCols][kCols + 1];  // [warp][column]
  const float* part = blockIdx.y ? part_post : part_pre;
  float* dw = blockIdx.y ? dw_post : dw_pre;
  if (!part) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = lane & (kReduceUnits - 1), row = threadIdx.x / kReduceUnits;
  const int d = blockIdx.x * kCols + 4 * unit;
  pdl_wait();
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (d < D) {
#pragma unroll 4
    for (int r = row; r < rows; r += kReduceRows) {
      const float4 x = *reinterpret_cast<const float4*>(part + (int64_t)r * ld + d);
      acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = kReduceUnits; o < 32; o *= 2) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
    if (lane < kReduceUnits) s[warp][4 * lane + k] = acc[k];
  }
  __syncthreads();
  const float sum = warp_sum(s[lane][warp]);  // warp = column
  if (lane == 0 && blockIdx.x * kCols + warp < D) dw[blockIdx.x * kCols + warp] += sum;
}

// A row's threads, a multiple of 32, and columns per thread.  Vector rows: as few
// threads as have the row in 4 units of 4 columns (the sums over the threads then
// cost the fewest instructions per column: at 2048 columns 2 units 78.7 us
// forward, 4 units 76.2; backward 143 and 128), and as few units as these need:
// every unit but the last is whole for all threads and needs no tests (backward of
// 16384 x 2048 with tests 168 us, without 130).  The backward of few rows, which
// is bound by latency, has 2 units (1237 x 1001 bf16 12.8 us, with 4 16.1; 2500 x
// 1000 17.9 and 18.5; but 60000 x 301 90 and 67).  Rows of single elements are
// bound by latency too: 4 columns a thread (backward of 6946 x 1911 bf16 with 4
// 100 us, with 8 122; forward of 60000 x 301 70 and 80), the forward of over 512
// columns 8 with 4 CTAs on an SM (6946 x 1911 46 us, with 4 62), rows of over
// 2048 columns 16.  (The same rows by shifted units: 54 us, 39 and 29.)
struct RowPlan {
  int threads, cols;
};
RowPlan row_plan(Form form, bool forward, int64_t T, int64_t D) {
  if (form == kElements) {
    const int cols = D > 4 * kMaxRowThreads ? 16 : forward && D > 512 ? 8 : 4;
    return {(int)(((D + cols - 1) / cols + 31) / 32 * 32), cols};
  }
  const int64_t span = D + (form == kShifted ? 3 : 0);
  const int64_t per_warp = !forward && T <= kFewRows && span <= 8 * kRowThreads ? 256 : 512;
  int threads = (int)((span + per_warp - 1) / per_warp * 32), units;
  // (where the span, but not the row, begins a unit: more threads, fewer units)
  while ((units = (int)((span + 4 * threads - 1) / (4 * threads))), (units - 1) * 4 * threads > D) threads += 32;
  return {threads, 4 * units};
}

// Shared memory of a vector form with kStages' rows of `row` bytes a column.
size_t stage_bytes(Form form, int stages, const RowPlan& p, size_t row) {
  return (size_t)p.threads * p.cols * (stages * row + (form == kShifted ? 8 : 0));
}

// The form for rows of D columns from tensors which all start on a unit or not;
// `row`: bytes a column of a stage.  Shifted rows need room for their stages.
Form row_form(bool units, int64_t T, int64_t D, size_t row) {
  if (units && D % 4 == 0) return kUnits;
  return units && D + 3 <= kMaxNormD && stage_bytes(kShifted, kStages, row_plan(kShifted, true, T, D), row) <= kMaxSmem
             ? kShifted
             : kElements;
}

// The backward's CTAs, each with a row of partial sums: up to 1024 threads on
// each of 148 SMs, and no more than 16 CTAs there.
int64_t max_backward_ctas(int threads) { return 148 * std::min(16, 1024 / threads); }

// CTAs of a persistent launch: as many as fit the GPU at once.
template <class K>
cudaError_t resident_ctas(K kern, int threads, size_t smem, int n_sm, int64_t most, unsigned* grid) {
  *grid = (unsigned)std::min<int64_t>(most, n_sm);
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = allow_smem(kern);
  if (most <= n_sm || e != cudaSuccess) return e;
  int occ = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, threads, smem);
  if (e == cudaSuccess && occ < 1) e = cudaErrorInvalidConfiguration;
  *grid = (unsigned)std::min<int64_t>(most, (int64_t)n_sm * occ);
  return e;
}

// Rows of a CTA a multiple of 4 apart, unless it has one only.
unsigned shifted_grid(unsigned grid, int64_t T) { return grid < T ? grid / 4 * 4 : grid; }

template <Form kForm, int C, int kStages, int kThreads, class X, class F, class H>
cudaError_t forward_launch(const NormFwd& a, const RowPlan& p, int n_sm, cudaStream_t stream) {
  auto kern = norm_forward_kernel<kForm, C, kStages, kThreads, X, F, H>;
  const size_t smem = stage_bytes(kForm, kStages, p, sizeof(X) + sizeof(F));
  unsigned grid = 0;
  const cudaError_t e = resident_ctas(kern, p.threads, smem, n_sm, a.T, &grid);
  if (e != cudaSuccess) return e;
  kern<<<kForm == kShifted ? shifted_grid(grid, a.T) : grid, p.threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <Form kForm, class X, class F, class H>
cudaError_t forward_units(const NormFwd& a, int n_sm, cudaStream_t stream) {
  const RowPlan p = row_plan(kForm, true, a.T, a.D);
  if (p.threads > kRowThreads)
    return forward_launch<kForm, 16, kStages, kMaxRowThreads, X, F, H>(a, p, n_sm, stream);
  switch (p.cols) {
    case 4: return forward_launch<kForm, 4, kStages, kRowThreads, X, F, H>(a, p, n_sm, stream);
    case 8: return forward_launch<kForm, 8, kStages, kRowThreads, X, F, H>(a, p, n_sm, stream);
    case 12: return forward_launch<kForm, 12, kStages, kRowThreads, X, F, H>(a, p, n_sm, stream);
    default: return forward_launch<kForm, 16, kStages + 1, kRowThreads, X, F, H>(a, p, n_sm, stream);
  }
}

template <class X, class F, class H>
cudaError_t forward_form(const NormFwd& a, bool units, int n_sm, cudaStream_t stream) {
  const Form form = row_form(units, a.T, a.D, sizeof(X) + sizeof(F));
  if (form == kUnits) return forward_units<kUnits, X, F, H>(a, n_sm, stream);
  if (form == kShifted) return forward_units<kShifted, X, F, H>(a, n_sm, stream);
  const RowPlan p = row_plan(kElements, true, a.T, a.D);
  return p.cols == 4   ? forward_launch<kElements, 4, 0, kRowThreads, X, F, H>(a, p, n_sm, stream)
         : p.cols == 8 ? forward_launch<kElements, 8, 0, kRowThreads, X, F, H>(a, p, n_sm, stream)
                       : forward_launch<kElements, 16, 0, kMaxRowThreads, X, F, H>(a, p, n_sm, stream);
}

template <class X>
cudaError_t forward_types(const NormFwd& a, bool f_bf16, bool h_bf16, bool units, int n_sm, cudaStream_t stream) {
  if (f_bf16)
    return h_bf16 ? forward_form<X, uint16_t, uint16_t>(a, units, n_sm, stream)
                  : forward_form<X, uint16_t, float>(a, units, n_sm, stream);
  return h_bf16 ? forward_form<X, float, uint16_t>(a, units, n_sm, stream)
                : forward_form<X, float, float>(a, units, n_sm, stream);
}

template <Form kForm, bool kAll, int C, int kStages, int kThreads, class X, class F>
cudaError_t backward_launch(const NormBwd& a, const RowPlan& p, int n_sm, int* ctas, cudaStream_t stream) {
  auto kern = norm_backward_kernel<kForm, kAll, C, kStages, kThreads, X, F>;
  const size_t smem = stage_bytes(kForm, kStages, p, 8 + sizeof(X) + sizeof(F));
  unsigned grid = 0;
  const cudaError_t e =
      resident_ctas(kern, p.threads, smem, n_sm, std::min<int64_t>(a.T, max_backward_ctas(p.threads)), &grid);
  if (e != cudaSuccess) return e;
  if (kForm == kShifted) grid = shifted_grid(grid, a.T);
  *ctas = (int)grid;
  kern<<<grid, p.threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <Form kForm, bool kAll, class X, class F>
cudaError_t backward_staged(const NormBwd& a, const RowPlan& p, int n_sm, int* ctas, cudaStream_t stream) {
  switch (p.cols) {
    case 4: return backward_launch<kForm, kAll, 4, kStages, kRowThreads, X, F>(a, p, n_sm, ctas, stream);
    case 8: return backward_launch<kForm, kAll, 8, kStages, kRowThreads, X, F>(a, p, n_sm, ctas, stream);
    case 12: return backward_launch<kForm, kAll, 12, kStages, kRowThreads, X, F>(a, p, n_sm, ctas, stream);
    default: return backward_launch<kForm, kAll, 16, kStages, kRowThreads, X, F>(a, p, n_sm, ctas, stream);
  }
}

template <Form kForm, class X, class F>
cudaError_t backward_units(const NormBwd& a, int n_sm, int* ctas, cudaStream_t stream) {
  const RowPlan p = row_plan(kForm, false, a.T, a.D);
  if (p.threads > kRowThreads) {
    if constexpr (kForm == kUnits)  // (two rows of over 6656 columns, fp32, do not fit shared memory)
      if (stage_bytes(kForm, kStages, p, 8 + sizeof(X) + sizeof(F)) > kMaxSmem)
        return backward_launch<kForm, false, 16, 0, kMaxRowThreads, X, F>(a, p, n_sm, ctas, stream);
    return backward_launch<kForm, false, 16, kStages, kMaxRowThreads, X, F>(a, p, n_sm, ctas, stream);
  }
  return a.dh && a.dx_out && a.f && a.w_post && a.dx && a.df
             ? backward_staged<kForm, true, X, F>(a, p, n_sm, ctas, stream)
             : backward_staged<kForm, false, X, F>(a, p, n_sm, ctas, stream);
}

template <class X, class F>
cudaError_t backward_form(const NormBwd& a, bool units, int n_sm, int* ctas, cudaStream_t stream) {
  const Form form = row_form(units, a.T, a.D, 8 + sizeof(X) + sizeof(F));
  if (form == kUnits) return backward_units<kUnits, X, F>(a, n_sm, ctas, stream);
  if (form == kShifted) return backward_units<kShifted, X, F>(a, n_sm, ctas, stream);
  const RowPlan p = row_plan(kElements, false, a.T, a.D);
  return p.cols == 4 ? backward_launch<kElements, false, 4, 0, kMaxRowThreads, X, F>(a, p, n_sm, ctas, stream)
                     : backward_launch<kElements, false, 16, 0, kMaxRowThreads, X, F>(a, p, n_sm, ctas, stream);
}

bool valid(mole_dtype dt) { return dt == MOLE_F32 || dt == MOLE_BF16; }
size_t size_of(mole_dtype dt) { return dt == MOLE_BF16 ? 2 : 4; }

// Rows of partial sums of each weight gradient, 16-byte aligned.
int64_t part_ld(int64_t D) { return (D + 3) / 4 * 4; }
size_t partial_bytes(int64_t T, int64_t D) {
  const int most = (int)max_backward_ctas(row_plan(kUnits, true, T, D).threads);  // (with the fewest threads)
  const int64_t rows = std::min<int64_t>(T, most);
  return ((size_t)rows * (size_t)part_ld(D) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace mole

extern "C" mole_status mole_block_norm_forward(const void* x, mole_dtype dt_x, const void* f, mole_dtype dt_f,
                                               const float* w_post, const float* gate, float res_scale,
                                               const float* w_pre, float eps, int64_t T, int64_t D, void* x_out,
                                               void* h, mole_dtype dt_h, cudaStream_t stream) {
  using namespace mole;
  if (!valid(dt_x) || !valid(dt_f) || !valid(dt_h) || T < 0 || D <= 0 || !(eps > 0.f)) return MOLE_ERR_ARG;
  if (T > INT32_MAX || D > kMaxNormD) return MOLE_ERR_UNSUPPORTED;
  if (T == 0) return MOLE_OK;
  if (!x || (!x_out && !h) || (h && !w_pre) || (!f && (w_post || gate))) return MOLE_ERR_ARG;
  if (!aligned_to(x, size_of(dt_x)) || !aligned_to(x_out, size_of(dt_x)) || !aligned_to(f, size_of(dt_f)) ||
      !aligned_to(h, size_of(dt_h)) || !aligned_to(w_post, 4) || !aligned_to(w_pre, 4) || !aligned_to(gate, 4))
    return MOLE_ERR_ALIGN;
  mole_status st = check_device();
  if (st != MOLE_OK) return st;
  const int n_sm = num_sms();
  if (n_sm <= 0) return MOLE_ERR_NO_DEVICE;
  const bool units = aligned_rows(x, dt_x == MOLE_BF16) && aligned_rows(f, dt_f == MOLE_BF16) &&
                   aligned_rows(x_out, dt_x == MOLE_BF16) && aligned_rows(h, dt_h == MOLE_BF16) &&
                   aligned16(w_post) && aligned16(w_pre);
  const NormFwd a{x, f, w_post, gate, w_pre, res_scale, eps, T, (int)D, x_out, h};
  const bool fb = dt_f == MOLE_BF16, hb = dt_h == MOLE_BF16;
  return cuda_status(dt_x == MOLE_BF16 ? forward_types<uint16_t>(a, fb, hb, units, n_sm, stream)
                                       : forward_types<float>(a, fb, hb, units, n_sm, stream));
}

extern "C" size_t mole_block_norm_backward_workspace(int64_t T, int64_t D) {
  if (T <= 0 || T > INT32_MAX || D <= 0 || D > mole::kMaxNormD) return 0;
  return 2 * mole::partial_bytes(T, D);
}

extern "C" mole_status mole_block_norm_backward(const void* x_out, mole_dtype dt_x, const void* f, mole_dtype dt_f,
                                                const float* w_post, const float* gate, float res_scale,
                                                const float* w_pre, float eps, int64_t T, int64_t D,
                                                const float* dx_out, const float* dh, float* dx, float* df,
                                                float* dgate, float* dw_post, float* dw_pre, void* workspace,
                                                size_t ws_bytes, cudaStream_t stream) {
  using namespace mole;
  if (!valid(dt_x) || !valid(dt_f) || T < 0 || D <= 0 || !(eps > 0.f)) return MOLE_ERR_ARG;
  if (T > INT32_MAX || D > kMaxNormD) return MOLE_ERR_UNSUPPORTED;
  if (T == 0) return MOLE_OK;
  if ((!dx_out && !dh) || (!dx && !df && !dgate && !dw_post && !dw_pre)) return MOLE_ERR_ARG;
  if (dh && (!w_pre || !x_out)) return MOLE_ERR_ARG;
  if (dw_pre && !dh) return MOLE_ERR_ARG;
  if (!f && (w_post || dgate)) return MOLE_ERR_ARG;
  if (dw_post && !w_post) return MOLE_ERR_ARG;
  if (!aligned_to(x_out, size_of(dt_x)) || !aligned_to(f, size_of(dt_f)) || !aligned_to(w_post, 4) ||
      !aligned_to(w_pre, 4) || !aligned_to(gate, 4) || !aligned_to(dx_out, 4) || !aligned_to(dh, 4) ||
      !aligned_to(dx, 4) || !aligned_to(df, 4) || !aligned_to(dgate, 4) || !aligned_to(dw_post, 4) ||
      !aligned_to(dw_pre, 4))
    return MOLE_ERR_ALIGN;
  float *part_pre = nullptr, *part_post = nullptr;
  if (dw_pre || dw_post) {
    const size_t half = partial_bytes(T, D);
    if (!workspace || ws_bytes < 2 * half) return MOLE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOLE_ERR_ALIGN;
    if (dw_pre) part_pre = static_cast<float*>(workspace);
    if (dw_post) part_post = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + half);
  }
  mole_status st = check_device();
  if (st != MOLE_OK) return st;
  const int n_sm = num_sms();
  if (n_sm <= 0) return MOLE_ERR_NO_DEVICE;
  const bool units = aligned_rows(x_out, dt_x == MOLE_BF16) && aligned_rows(f, dt_f == MOLE_BF16) &&
                   aligned16(w_post) && aligned16(w_pre) && aligned16(dx_out) && aligned16(dh) && aligned16(dx) &&
                   aligned16(df);
  const NormBwd a{x_out, f,  w_post, gate, w_pre, res_scale, eps,       T, (int)D,
                  dx_out, dh, dx,     df,   dgate, part_post, part_pre};
  int ctas = 0;
  cudaError_t e;
  if (dt_x == MOLE_BF16)
    e = dt_f == MOLE_BF16 ? backward_form<uint16_t, uint16_t>(a, units, n_sm, &ctas, stream)
                          : backward_form<uint16_t, float>(a, units, n_sm, &ctas, stream);
  else
    e = dt_f == MOLE_BF16 ? backward_form<float, uint16_t>(a, units, n_sm, &ctas, stream)
                          : backward_form<float, float>(a, units, n_sm, &ctas, stream);
  if (e != cudaSuccess) return MOLE_ERR_CUDA;
  if (part_pre || part_post) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((D + 4 * kReduceUnits - 1) / (4 * kReduceUnits)), 2);
    cfg.blockDim = dim3(kReduceUnits * kReduceRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto join = [&](const float* pre, const float* post) {
      return cudaLaunchKernelEx(&cfg, norm_reduce_kernel, pre, post, ctas, (int)D, (int)part_ld(D), dw_pre, dw_post);
    };
    if (dw_pre != dw_post)
      e = join(part_pre, part_post);
    else if ((e = join(part_pre, nullptr)) == cudaSuccess)  // one gradient for both: one sum, then the other
      e = join(nullptr, part_post);
    if (e != cudaSuccess) return MOLE_ERR_CUDA;
  }
  return MOLE_OK;
}
