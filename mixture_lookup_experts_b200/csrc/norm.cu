// norm.cu -- the norms around a block, with its gate and the residual scale,
// forward and backward (mole.h states the formulas).  MoLE page, 训练阶段: a
// layer's router and shared expert read the previous layer's output; what lies
// between two blocks' GEMMs is one pass over the token rows:
//     y = w_post f / rms(f),  x' = beta x + gate y,  h = w_pre x' / rms(x')
// A token's row is held in registers, 8 columns a thread, by a group of one to
// 16 warps; the row's sums are reduced by shuffles and (beyond one warp) shared
// memory.  Each tensor is read and written once: both kernels are bound by HBM.
//
// Backward, per token (n = D, r = 1/rms):
//     G  = dx' + r_x (a - x^ <a, x^>/n)      a = dh w_pre,  x^ = x' r_x
//     dx = beta G
//     df = r_f (b - f^ <b, f^>/n)            b = gate G w_post,  f^ = f r_f
//     dgate = <G w_post, f^>
// so two reductions: (sum x'^2, sum a x', sum f^2), then <G w_post, f>.  The
// norms' statistics come from the rows themselves (they are read anyway); no
// forward state is kept.  dw_pre and dw_post: a thread adds its columns over
// its group's rows in registers; the CTAs' sums go to the workspace and
// norm_reduce_kernel adds them in order.
#include "rows.cuh"

namespace mole {
namespace {

constexpr int kMaxRowThreads = 512;   // leaves 128 registers a thread
constexpr int kNormThreads = 256;     // CTA size while a row needs no more
constexpr int64_t kMaxNormD = 2 * 8 * kMaxRowThreads;
constexpr int kMaxNormCtas = 1024;    // rows of partial sums in the workspace
constexpr int kReduceCols = 32, kReduceRows = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of K values over a row's group of threads (blockDim.x, a multiple of
// 32), in a fixed order.  `red` holds K floats per warp of the CTA and serves
// one call between two barriers of the row loop.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5;
  float* mine = red + (size_t)threadIdx.y * warps * K;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) mine[warp * K + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += mine[w * K + k];
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

// First column and column step of a thread's unit v of 8 columns.
template <bool kVec>
__device__ __forceinline__ int unit_col(int v) {
  return 8 * v * (int)blockDim.x + (kVec ? 4 : 1) * (int)threadIdx.x;
}

// blockDim = (threads per row, rows per CTA); kUnits units of 8 columns a thread.
template <bool kVec, int kUnits, class X, class F, class H>
__global__ void __launch_bounds__(kMaxRowThreads) norm_forward_kernel(const NormFwd a) {
  __shared__ float red[2][kMaxRowThreads / 32];
  const int step = blockDim.x, D = a.D;
  const float inv_d = 1.f / (float)D;
  for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < a.T; t0 += (int64_t)gridDim.x * blockDim.y) {
    const int64_t t = t0 + threadIdx.y;
    const bool in = t < a.T;
    float x[kUnits][8], f[kUnits][8];
    float s[1] = {0.f};
    const X* xr = static_cast<const X*>(a.x) + t * D;
    const F* fr = static_cast<const F*>(a.f) + t * D;
#pragma unroll
    for (int v = 0; v < kUnits; ++v) {
      const int c = unit_col<kVec>(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[v][k] = f[v][k] = 0.f;
      if (in && c < D) {
        ld_cols<kVec>(xr, c, step, D, x[v]);
        if (a.f) ld_cols<kVec>(fr, c, step, D, f[v]);
      }
    }
    float g = 1.f;
    if (a.f) {
      if (a.gate && in) g = a.gate[t];
      if (a.w_post) {
#pragma unroll
        for (int v = 0; v < kUnits; ++v)
#pragma unroll
          for (int k = 0; k < 8; ++k) s[0] = fmaf(f[v][k], f[v][k], s[0]);
        row_sums(s, red[0]);
        const float r = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
        for (int v = 0; v < kUnits; ++v) {
          const int c = unit_col<kVec>(v);
          float w[8];
          if (c < D) {
            ld_cols<kVec>(a.w_post, c, step, D, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[v][k] = f[v][k] * r * w[k];
          }
        }
      }
    }
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < kUnits; ++v) {
      const int c = unit_col<kVec>(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[v][k] = a.f ? fmaf(g, f[v][k], a.res_scale * x[v][k]) : a.res_scale * x[v][k];
        s[0] = fmaf(x[v][k], x[v][k], s[0]);
      }
      if (in && a.x_out && c < D) st_cols<kVec>(static_cast<X*>(a.x_out) + t * D, c, step, D, x[v]);
    }
    if (a.h) {
      row_sums(s, red[1]);
      const float r = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
      for (int v = 0; v < kUnits; ++v) {
        const int c = unit_col<kVec>(v);
        if (in && c < D) {
          float w[8];
          ld_cols<kVec>(a.w_pre, c, step, D, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] *= x[v][k] * r;
          st_cols<kVec>(static_cast<H*>(a.h) + t * D, c, step, D, w);
        }
      }
    }
    if (blockDim.x > 32) __syncthreads();  // red's readers are done
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
  float* part_post;  // [gridDim.x][D] or null
  float* part_pre;
};

template <bool kVec, int kUnits, class X, class F>
__global__ void __launch_bounds__(kMaxRowThreads) norm_backward_kernel(const NormBwd a) {
  __shared__ float red[2][3 * (kMaxRowThreads / 32)];
  extern __shared__ float fold[];  // several rows per CTA: their sums before one is written
  const int step = blockDim.x, D = a.D;
  const float inv_d = 1.f / (float)D;
  float acc_pre[kUnits][8], acc_post[kUnits][8];
#pragma unroll
  for (int v = 0; v < kUnits; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc_pre[v][k] = acc_post[v][k] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < a.T; t0 += (int64_t)gridDim.x * blockDim.y) {
    const int64_t t = t0 + threadIdx.y;
    const bool in = t < a.T;
    float x[kUnits][8], f[kUnits][8], dh[kUnits][8], G[kUnits][8];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kUnits; ++v) {
      const int c = unit_col<kVec>(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[v][k] = f[v][k] = dh[v][k] = G[v][k] = 0.f;
      if (in && c < D) {
        if (a.dh) {
          ld_cols<kVec>(static_cast<const X*>(a.x) + t * D, c, step, D, x[v]);
          ld_cols<kVec>(a.dh + t * D, c, step, D, dh[v]);
        }
        if (a.f) ld_cols<kVec>(static_cast<const F*>(a.f) + t * D, c, step, D, f[v]);
        if (a.dx_out) ld_cols<kVec>(a.dx_out + t * D, c, step, D, G[v]);
      }
    }
    const float g = a.gate && in ? a.gate[t] : 1.f;
#pragma unroll
    for (int v = 0; v < kUnits; ++v) {
      const int c = unit_col<kVec>(v);
      float w[8];
      if (a.dh && c < D) {
        ld_cols<kVec>(a.w_pre, c, step, D, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s[0] = fmaf(x[v][k], x[v][k], s[0]);
          s[1] = fmaf(dh[v][k] * w[k], x[v][k], s[1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s[2] = fmaf(f[v][k], f[v][k], s[2]);
    }
    row_sums(s, red[0]);
    const float rf = a.w_post ? rsqrtf(fmaf(s[2], inv_d, a.eps)) : 1.f;
    float q[1] = {0.f};
    if (a.dh) {
      const float rx = rsqrtf(fmaf(s[0], inv_d, a.eps));
      const float cx = rx * rx * (s[1] * inv_d);  // <a, x^> / n = rx s1 / n; x^ = rx x'
#pragma unroll
      for (int v = 0; v < kUnits; ++v) {
        const int c = unit_col<kVec>(v);
        if (c < D) {
          float w[8];
          ld_cols<kVec>(a.w_pre, c, step, D, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            acc_pre[v][k] = fmaf(dh[v][k], x[v][k] * rx, acc_pre[v][k]);
            G[v][k] += rx * fmaf(-cx, x[v][k], dh[v][k] * w[k]);
          }
        }
      }
    }
    // f becomes f^ (f itself without a post-norm); dh becomes dy w_post / gate = G w_post
#pragma unroll
    for (int v = 0; v < kUnits; ++v) {
      const int c = unit_col<kVec>(v);
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.f;
      if (a.w_post && c < D) ld_cols<kVec>(a.w_post, c, step, D, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[v][k] *= rf;
        acc_post[v][k] = fmaf(g * G[v][k], f[v][k], acc_post[v][k]);
        dh[v][k] = G[v][k] * w[k];
        q[0] = fmaf(dh[v][k], f[v][k], q[0]);
      }
      if (in && a.dx && c < D) {
#pragma unroll
        for (int k = 0; k < 8; ++k) G[v][k] *= a.res_scale;
        st_cols<kVec>(a.dx + t * D, c, step, D, G[v]);
      }
    }
    if (a.f) {
      row_sums(q, red[1]);
      if (in && a.dgate && threadIdx.x == 0) a.dgate[t] = q[0];
    }
    if (a.df && in) {
      const float cf = a.w_post ? q[0] * inv_d : 0.f;
#pragma unroll
      for (int v = 0; v < kUnits; ++v) {
        const int c = unit_col<kVec>(v);
        if (c < D) {
#pragma unroll
          for (int k = 0; k < 8; ++k) dh[v][k] = g * rf * fmaf(-cf, f[v][k], dh[v][k]);
          st_cols<kVec>(a.df + t * D, c, step, D, dh[v]);
        }
      }
    }
    if (blockDim.x > 32) __syncthreads();  // red's readers are done
  }
  // the CTA's sums over its rows: group by group into one row of the workspace
  for (int which = 0; which < 2; ++which) {
    float* part = which ? a.part_post : a.part_pre;
    if (!part) continue;
    for (int r = 0; r < (int)blockDim.y; ++r) {
      if ((int)threadIdx.y == r) {
#pragma unroll
        for (int v = 0; v < kUnits; ++v) {
          const int c = unit_col<kVec>(v);
          if (c >= D) continue;
          float w[8];
          if (r > 0) {
            ld_cols<kVec>(fold, c, step, D, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] += which ? acc_post[v][k] : acc_pre[v][k];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = which ? acc_post[v][k] : acc_pre[v][k];
          }
          if (r == (int)blockDim.y - 1)
            st_cols<kVec>(part + (int64_t)blockIdx.x * D, c, step, D, w);
          else
            st_cols<kVec>(fold, c, step, D, w);
        }
      }
      if (blockDim.y > 1) __syncthreads();
    }
  }
}

// dw[d] += sum over the CTAs' rows, in order: a thread takes every
// kReduceRows-th row of its column, then the 32 sums are added in order.
// blockIdx.y: 0 = dw_pre, 1 = dw_post.
__global__ void __launch_bounds__(kReduceCols* kReduceRows)
    norm_reduce_kernel(const float* part_pre, const float* part_post, int rows, int D, float* dw_pre, float* dw_post) {
  __shared__ float s[kReduceRows][kReduceCols + 1];
  pdl_wait();
  const float* part = blockIdx.y ? part_post : part_pre;
  float* dw = blockIdx.y ? dw_post : dw_pre;
  if (!part) return;
  const int d = blockIdx.x * kReduceCols + threadIdx.x;
  float acc = 0.f;
  if (d < D)
    for (int r = threadIdx.y; r < rows; r += kReduceRows) acc += part[(int64_t)r * D + d];
  s[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.y == 0 && d < D) {
    float sum = 0.f;
    for (int r = 0; r < kReduceRows; ++r) sum += s[r][threadIdx.x];
    dw[d] += sum;
  }
}

// How rows are spread over a CTA: threads per row (a multiple of 32), rows per
// CTA, units of 8 columns per thread.
struct RowPlan {
  int tx, rows, units;
};
RowPlan row_plan(int64_t D) {
  const int units = D > 8 * kMaxRowThreads ? 2 : 1;
  const int64_t threads = (D + 8 * units - 1) / (8 * units);
  const int tx = (int)((threads + 31) / 32 * 32);
  return {tx, std::max(1, kNormThreads / tx), units};
}

template <bool kVec, int kUnits, class X, class F, class H>
cudaError_t forward_launch(const NormFwd& a, const RowPlan& p, int n_sm, cudaStream_t stream) {
  const int64_t ctas = (a.T + p.rows - 1) / p.rows;
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)n_sm * 8);
  norm_forward_kernel<kVec, kUnits, X, F, H><<<grid, dim3(p.tx, p.rows), 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool kVec, int kUnits, class X, class F>
cudaError_t forward_h(const NormFwd& a, bool h_bf16, const RowPlan& p, int n_sm, cudaStream_t stream) {
  return h_bf16 ? forward_launch<kVec, kUnits, X, F, uint16_t>(a, p, n_sm, stream)
                : forward_launch<kVec, kUnits, X, F, float>(a, p, n_sm, stream);
}

template <bool kVec, int kUnits>
cudaError_t forward_xf(const NormFwd& a, bool x_bf16, bool f_bf16, bool h_bf16, const RowPlan& p, int n_sm,
                       cudaStream_t stream) {
  if (x_bf16)
    return f_bf16 ? forward_h<kVec, kUnits, uint16_t, uint16_t>(a, h_bf16, p, n_sm, stream)
                  : forward_h<kVec, kUnits, uint16_t, float>(a, h_bf16, p, n_sm, stream);
  return f_bf16 ? forward_h<kVec, kUnits, float, uint16_t>(a, h_bf16, p, n_sm, stream)
                : forward_h<kVec, kUnits, float, float>(a, h_bf16, p, n_sm, stream);
}

int backward_ctas(int64_t T, const RowPlan& p, int n_sm) {
  return (int)std::min<int64_t>((T + p.rows - 1) / p.rows, std::min(kMaxNormCtas, n_sm * 4));
}

template <bool kVec, int kUnits, class X, class F>
cudaError_t backward_launch(const NormBwd& a, const RowPlan& p, int n_sm, cudaStream_t stream) {
  const int grid = backward_ctas(a.T, p, n_sm);
  const size_t smem = p.rows > 1 ? (size_t)a.D * 4 : 0;
  norm_backward_kernel<kVec, kUnits, X, F><<<grid, dim3(p.tx, p.rows), smem, stream>>>(a);
  return cudaGetLastError();
}

template <bool kVec, int kUnits>
cudaError_t backward_xf(const NormBwd& a, bool x_bf16, bool f_bf16, const RowPlan& p, int n_sm, cudaStream_t stream) {
  if (x_bf16)
    return f_bf16 ? backward_launch<kVec, kUnits, uint16_t, uint16_t>(a, p, n_sm, stream)
                  : backward_launch<kVec, kUnits, uint16_t, float>(a, p, n_sm, stream);
  return f_bf16 ? backward_launch<kVec, kUnits, float, uint16_t>(a, p, n_sm, stream)
                : backward_launch<kVec, kUnits, float, float>(a, p, n_sm, stream);
}

bool valid(mole_dtype dt) { return dt == MOLE_F32 || dt == MOLE_BF16; }
size_t size_of(mole_dtype dt) { return dt == MOLE_BF16 ? 2 : 4; }

// Rows of partial sums of each weight gradient.
size_t partial_bytes(int64_t T, int64_t D) {
  const RowPlan p = row_plan(D);
  const size_t rows = (size_t)std::min<int64_t>((T + p.rows - 1) / p.rows, kMaxNormCtas);
  return (rows * (size_t)D * 4 + 255) / 256 * 256;
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
  const bool vec = D % 4 == 0 && aligned_rows(x, dt_x == MOLE_BF16) && aligned_rows(f, dt_f == MOLE_BF16) &&
                   aligned_rows(x_out, dt_x == MOLE_BF16) && aligned_rows(h, dt_h == MOLE_BF16) &&
                   aligned16(w_post) && aligned16(w_pre);
  const NormFwd a{x, f, w_post, gate, w_pre, res_scale, eps, T, (int)D, x_out, h};
  const RowPlan p = row_plan(D);
  const bool xb = dt_x == MOLE_BF16, fb = dt_f == MOLE_BF16, hb = dt_h == MOLE_BF16;
  cudaError_t e;
  if (p.units == 1)
    e = vec ? forward_xf<true, 1>(a, xb, fb, hb, p, n_sm, stream) : forward_xf<false, 1>(a, xb, fb, hb, p, n_sm, stream);
  else
    e = vec ? forward_xf<true, 2>(a, xb, fb, hb, p, n_sm, stream) : forward_xf<false, 2>(a, xb, fb, hb, p, n_sm, stream);
  return cuda_status(e);
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
  const bool vec = D % 4 == 0 && aligned_rows(x_out, dt_x == MOLE_BF16) && aligned_rows(f, dt_f == MOLE_BF16) &&
                   aligned16(w_post) && aligned16(w_pre) && aligned16(dx_out) && aligned16(dh) && aligned16(dx) && aligned16(df);
  const NormBwd a{x_out, f, w_post, gate, w_pre, res_scale, eps, T, (int)D, dx_out, dh, dx, df, dgate, part_post, part_pre};
  const RowPlan p = row_plan(D);
  const bool xb = dt_x == MOLE_BF16, fb = dt_f == MOLE_BF16;
  cudaError_t e;
  if (p.units == 1)
    e = vec ? backward_xf<true, 1>(a, xb, fb, p, n_sm, stream) : backward_xf<false, 1>(a, xb, fb, p, n_sm, stream);
  else
    e = vec ? backward_xf<true, 2>(a, xb, fb, p, n_sm, stream) : backward_xf<false, 2>(a, xb, fb, p, n_sm, stream);
  if (e != cudaSuccess) return MOLE_ERR_CUDA;
  if (part_pre || part_post) {
    norm_reduce_kernel<<<dim3((unsigned)((D + kReduceCols - 1) / kReduceCols), 2), dim3(kReduceCols, kReduceRows), 0,
                         stream>>>(part_pre, part_post, backward_ctas(T, p, n_sm), (int)D, dw_pre, dw_post);
    if (cudaGetLastError() != cudaSuccess) return MOLE_ERR_CUDA;
  }
  return MOLE_OK;
}
