// embed.cu -- the model's input embedding in training: the scaled lookup and
// its gradient.  MoLE page, 训练阶段: the embedding matrix feeds the model and
// the routed experts, so its gradient has two parts; mole_train_backward adds
// the experts' part to dE and this file the lookup's.
//
// Forward: out[t] = s E[ids[t]], bound by the rows read and written.
//
// Gradient: dE[v] += s sum_{t: ids[t] = v} dout[t].  Text repeats ids heavily
// (one of 50304 ids takes one token in seven of a Zipf batch), so the work is
// split over the tokens in id order, not over the ids:
//   1. embed_sort_kernel: (id, t) sorted by id, stably (ascending t inside an
//      id), by a radix sort of 8-bit digits run by ONE cluster of 8 CTAs: the
//      digit counts of its 256 warps meet in distributed shared memory, so a
//      pass costs two cluster barriers instead of two kernel boundaries.
//   2. embed_chunk_kernel: fixed chunks of the sorted order, one group of
//      threads per (chunk, slice of columns); runs of equal ids inside a chunk
//      go to dE, the runs that cross a chunk border leave partial sums.
//   3. embed_join_kernel: per crossing run, its partial sums in chunk order.
// Every sum has one order, fixed by the ids alone: the result has the same
// bits on every run.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace mole {
namespace {

namespace cg = cooperative_groups;

constexpr int kEmbedThreads = 256;
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;
constexpr int kChunkThreads = 128;
constexpr int kRowsInFlight = 8;

// ---- forward ----
// blockDim = (tx, 256 / tx): a row slice per group, rows in grid order.
template <bool kVec, class In, class Out>
__global__ void __launch_bounds__(kEmbedThreads) embed_forward_kernel(const int32_t* __restrict__ ids, int64_t T,
                                                                      const In* __restrict__ E, int64_t V, int D,
                                                                      float scale, Out* __restrict__ out,
                                                                      unsigned* err) {
  const int tx = blockDim.x;
  const int slice0 = blockIdx.y * tx * 8;
  const int col0 = kVec ? slice0 + 8 * threadIdx.x : slice0 + threadIdx.x;
  if (col0 >= D) return;
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < T; t += (int64_t)gridDim.x * blockDim.y) {
    const int32_t id = __ldg(ids + t);
    float f[8];
    if (id < 0 || (int64_t)id >= V) {
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(err, kErrIndex);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = NAN;
    } else {
      ld_cols<kVec>(E + (int64_t)id * D, col0, tx, D, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
    }
    st_cols<kVec>(out + t * D, col0, tx, D, f);
  }
}

// ---- gradient, step 1: the stable sort ----
struct SortArgs {
  const int32_t* ids;
  int64_t T, V;
  int2* buf[2];  // {id, t}; the last pass writes buf[0]
  int passes;
  unsigned* err;
};

// Key of a bad id: V, behind every row (keys fit 31 bits + 1: V <= 2^31 - 1).
__device__ __forceinline__ int2 sort_input(const SortArgs& a, int pass, int64_t i) {
  if (pass == 0) {
    const int32_t id = __ldg(a.ids + i);
    const bool ok = id >= 0 && (int64_t)id < a.V;
    return make_int2(ok ? id : (int)a.V, (int)i);
  }
  return __ldcg(a.buf[(a.passes - pass) & 1] + i);  // another CTA wrote it: past L1
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const SortArgs a) {
  __shared__ int hist[kSortWarps][kDigits];  // per warp: its count of a digit, then its offset inside the CTA
  __shared__ int tot[kDigits];               // per digit: the CTA's count (read by the cluster)
  __shared__ int base[kDigits];              // per digit: first position of the CTA's elements
  __shared__ int wsum[kDigits / 32];
  pdl_trigger();  // the chunk kernel may take its place on the other SMs
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // each warp owns a contiguous range of the input, so that warp order is input order
  const int64_t per = ((a.T + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const int64_t lo = std::min<int64_t>(a.T, per * (cta * kSortWarps + warp));
  const int64_t hi = std::min<int64_t>(a.T, lo + per);
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 8 * pass;
    for (int d = lane; d < kDigits; d += 32) hist[warp][d] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const bool in = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int2 e = sort_input(a, pass, i0 + lane);
        if (pass == 0 && (int64_t)e.x == a.V) atomicOr(a.err, kErrIndex);
        const int d = ((unsigned)e.x >> shift) & (kDigits - 1);
        const unsigned same = __match_any_sync(act, d);
        if (lane == __ffs(same) - 1) hist[warp][d] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      int run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = hist[w][threadIdx.x];
        hist[w][threadIdx.x] = run;
        run += c;
      }
      tot[threadIdx.x] = run;
    }
    cluster.sync();
    int before = 0, all = 0, incl = 0;
    if (threadIdx.x < kDigits) {
      for (int c = 0; c < kSortCtas; ++c) {
        const int x = cluster.map_shared_rank(tot, c)[threadIdx.x];
        if (c < cta) before += x;
        all += x;
      }
      incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) wsum[warp] = incl;
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      int off = incl - all + before;
      for (int w = 0; w < warp; ++w) off += wsum[w];
      base[threadIdx.x] = off;
    }
    __syncthreads();
    int2* dst = a.buf[(a.passes - 1 - pass) & 1];
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const bool in = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int2 e = sort_input(a, pass, i0 + lane);
        const int d = ((unsigned)e.x >> shift) & (kDigits - 1);
        const unsigned same = __match_any_sync(act, d);
        const int off = hist[warp][d];
        __syncwarp(act);
        if (lane == __ffs(same) - 1) hist[warp][d] = off + __popc(same);
        __stcg(dst + base[d] + off + __popc(same & ((1u << lane) - 1u)), e);
      }
      __syncwarp();
    }
    // the pass's output (global) and the readers of tot are done
    cluster.sync();
  }
}

// ---- gradient, steps 2 and 3 ----
struct SumArgs {
  const int2* sorted;  // {id, t}, id == V: a bad id
  int64_t T, V;
  int D, chunk;
  int64_t n_chunks;
  const void* dout;
  float scale;
  float* dE;
  float* part;  // [n_chunks][2][D]: sums of the run that enters the chunk, of the run that leaves it
};

template <bool kVec>
__device__ __forceinline__ void add_row(float* row, int col0, int step, int D, float scale, const float (&acc)[8]) {
  float f[8];
  ld_cols<kVec>(row, col0, step, D, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = fmaf(scale, acc[k], f[k]);
  st_cols<kVec>(row, col0, step, D, f);
}

// blockDim = (tx, 128 / tx): threadIdx.y = chunk inside the CTA, blockIdx.y = slice.
template <bool kVec, class In>
__global__ void __launch_bounds__(kChunkThreads) embed_chunk_kernel(const SumArgs a) {
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int step = blockDim.x;
  const int col0 = blockIdx.y * step * 8 + (kVec ? 8 : 1) * (int)threadIdx.x;
  pdl_wait();
  if (c >= a.n_chunks || col0 >= a.D) return;
  const In* dout = static_cast<const In*>(a.dout);
  const int64_t p0 = c * a.chunk, p1 = std::min<int64_t>(a.T, p0 + a.chunk);
  const int V = (int)a.V;
  const int enters = c > 0 ? a.sorted[p0 - 1].x : -1;   // id of the run that may enter the chunk
  const int leaves = p1 < a.T ? a.sorted[p1].x : -1;     // id of the run that may leave it
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  int cur = a.sorted[p0].x;
  bool entered = cur == enters;
  auto flush = [&](bool at_end) {
    if (cur == V) return;
    float* part = a.part + 2 * c * a.D;
    if (entered)
      st_cols<kVec>(part, col0, step, a.D, acc);
    else if (at_end && cur == leaves)
      st_cols<kVec>(part + a.D, col0, step, a.D, acc);
    else
      add_row<kVec>(a.dE + (int64_t)cur * a.D, col0, step, a.D, a.scale, acc);
  };
  for (int64_t p = p0; p < p1; p += kRowsInFlight) {
    int2 e[kRowsInFlight];
    float f[kRowsInFlight][8];
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) e[q] = p + q < p1 ? a.sorted[p + q] : make_int2(V, 0);
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q)
      if (e[q].x != V) ld_cols<kVec>(dout + (int64_t)e[q].y * a.D, col0, step, a.D, f[q]);
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) {
      if (p + q >= p1) break;
      if (e[q].x != cur) {
        flush(false);
        cur = e[q].x;
        entered = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
      }
      if (cur != V)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[q][k];
    }
  }
  flush(true);
}

// One group of threads per (chunk, slice): where a run starts in the chunk and
// leaves it, the sum of its parts.
template <bool kVec>
__global__ void __launch_bounds__(kChunkThreads) embed_join_kernel(const SumArgs a) {
  const int64_t c = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int step = blockDim.x;
  const int col0 = blockIdx.y * step * 8 + (kVec ? 8 : 1) * (int)threadIdx.x;
  pdl_wait();
  if (c + 1 >= a.n_chunks || col0 >= a.D) return;
  const int64_t next = (c + 1) * a.chunk;
  const int id = a.sorted[next].x;
  if (id == (int)a.V || a.sorted[next - 1].x != id) return;               // no run leaves this chunk
  if (c > 0 && a.sorted[c * a.chunk - 1].x == id) return;                 // it began earlier
  // the chunks that it enters: those after c whose first id is the run's
  int64_t lo = c + 1, hi = a.n_chunks;  // first id of lo is the run's, of hi (if any) behind it
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.sorted[mid * a.chunk].x == id)
      lo = mid;
    else
      hi = mid;
  }
  float acc[8];
  ld_cols<kVec>(a.part + (2 * c + 1) * a.D, col0, step, a.D, acc);
  for (int64_t k0 = c + 1; k0 <= lo; k0 += kRowsInFlight) {
    float f[kRowsInFlight][8];
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q)
      if (k0 + q <= lo) ld_cols<kVec>(a.part + 2 * (k0 + q) * a.D, col0, step, a.D, f[q]);
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q)
      if (k0 + q <= lo)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[q][k];
  }
  add_row<kVec>(a.dE + (int64_t)id * a.D, col0, step, a.D, a.scale, acc);
}

// Tokens per chunk: enough (chunk, slice) groups to fill the GPU several times
// over, few enough partial sums (2 rows of D per chunk) to stay small beside
// the gradient rows.
int chunk_tokens(int64_t T, int64_t D) {
  const int64_t groups = 2048;
  const int64_t slices = row_split(D, kChunkThreads).slices;
  int chunk = 16;
  while (chunk < 256 && T * slices > groups * chunk) chunk *= 2;
  return chunk;
}

struct EmbedWs {
  int2* buf[2];
  float* part;
};

size_t carve_embed(void* ws, int64_t T, int64_t D, EmbedWs* w) {
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const int64_t chunk = chunk_tokens(T, D);
  const size_t o_a = take(8 * (size_t)T), o_b = take(8 * (size_t)T);
  const size_t o_p = take(8 * (size_t)((T + chunk - 1) / chunk) * (size_t)D);
  if (w != nullptr) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    w->buf[0] = reinterpret_cast<int2*>(b + o_a);
    w->buf[1] = reinterpret_cast<int2*>(b + o_b);
    w->part = reinterpret_cast<float*>(b + o_p);
  }
  return off;
}

template <bool kVec, class In>
cudaError_t launch_sums(const SumArgs& a, dim3 grid, dim3 block, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, embed_chunk_kernel<kVec, In>, a);
  if (e != cudaSuccess || a.n_chunks == 1) return e;
  return cudaLaunchKernelEx(&cfg, embed_join_kernel<kVec>, a);
}

template <bool kVec, class In>
void launch_forward(const int32_t* ids, int64_t T, const void* E, int64_t V, int D, float scale, bool out_bf16,
                    void* out, unsigned* err, dim3 grid, dim3 block, cudaStream_t stream) {
  if (out_bf16)
    embed_forward_kernel<kVec><<<grid, block, 0, stream>>>(ids, T, static_cast<const In*>(E), V, D, scale,
                                                           static_cast<uint16_t*>(out), err);
  else
    embed_forward_kernel<kVec><<<grid, block, 0, stream>>>(ids, T, static_cast<const In*>(E), V, D, scale,
                                                           static_cast<float*>(out), err);
}

}  // namespace

mole_status embed_forward(const int32_t* ids, int64_t T, const void* E, int64_t V, int64_t D, float scale,
                          bool E_bf16, void* out, bool out_bf16, cudaStream_t stream) {
  unsigned* err = error_word();
  const int n_sm = num_sms();
  if (!err || n_sm <= 0) return MOLE_ERR_CUDA;
  const bool vec = D % 8 == 0 && aligned16(E) && aligned16(out);
  const RowSplit s = row_split(D, kEmbedThreads);
  const dim3 block(s.tx, kEmbedThreads / s.tx);
  const dim3 grid((unsigned)std::min<int64_t>((T + block.y - 1) / block.y, 1 << 20), s.slices);
  if (E_bf16)
    (vec ? launch_forward<true, uint16_t> : launch_forward<false, uint16_t>)(ids, T, E, V, (int)D, scale, out_bf16, out,
                                                                            err, grid, block, stream);
  else
    (vec ? launch_forward<true, float> : launch_forward<false, float>)(ids, T, E, V, (int)D, scale, out_bf16, out, err,
                                                                      grid, block, stream);
  return cuda_status(cudaGetLastError());
}

size_t embed_backward_bytes(int64_t T, int64_t D) { return carve_embed(nullptr, T, D, nullptr); }

mole_status embed_backward(const int32_t* ids, int64_t T, const void* dout, bool bf16, int64_t V, int64_t D,
                           float scale, float* dE, void* ws, cudaStream_t stream) {
  unsigned* err = error_word();
  if (!err) return MOLE_ERR_CUDA;
  EmbedWs w{};
  carve_embed(ws, T, D, &w);
  int bits = 0;  // of the keys 0 .. V
  while (bits < 32 && (V >> bits) != 0) ++bits;
  SortArgs sa{ids, T, V, {w.buf[0], w.buf[1]}, (bits + 7) / 8, err};
  embed_sort_kernel<<<kSortCtas, kSortThreads, 0, stream>>>(sa);
  if (cudaGetLastError() != cudaSuccess) return MOLE_ERR_CUDA;
  const int chunk = chunk_tokens(T, D);
  SumArgs a{w.buf[0], T, V, (int)D, chunk, (T + chunk - 1) / chunk, dout, scale, dE, w.part};
  const RowSplit s = row_split(D, kChunkThreads);
  const dim3 block(s.tx, kChunkThreads / s.tx);
  const dim3 grid((unsigned)((a.n_chunks + block.y - 1) / block.y), s.slices);
  const bool vec = D % 8 == 0 && aligned16(dout) && aligned16(dE);
  cudaError_t e;
  if (bf16)
    e = vec ? launch_sums<true, uint16_t>(a, grid, block, stream) : launch_sums<false, uint16_t>(a, grid, block, stream);
  else
    e = vec ? launch_sums<true, float>(a, grid, block, stream) : launch_sums<false, float>(a, grid, block, stream);
  return cuda_status(e);
}

}  // namespace mole

namespace {
// Shared checks of the two entry points.
mole_status check_embed(const int32_t* ids, int64_t T, const void* rows, mole_dtype dt_rows, int64_t V, int64_t D,
                        const void* to, mole_dtype dt_to) {
  if (dt_rows != MOLE_F32 && dt_rows != MOLE_BF16) return MOLE_ERR_ARG;
  if (dt_to != MOLE_F32 && dt_to != MOLE_BF16) return MOLE_ERR_ARG;
  if (T < 0 || V <= 0 || D <= 0) return MOLE_ERR_ARG;
  if (T > 0 && (!ids || !rows || !to)) return MOLE_ERR_ARG;
  if (T > INT32_MAX || V > INT32_MAX || D > (1 << 20)) return MOLE_ERR_UNSUPPORTED;
  if (!mole::aligned_to(ids, 4) || !mole::aligned_to(rows, dt_rows == MOLE_BF16 ? 2 : 4) ||
      !mole::aligned_to(to, dt_to == MOLE_BF16 ? 2 : 4))
    return MOLE_ERR_ALIGN;
  return MOLE_OK;
}
}  // namespace

extern "C" mole_status mole_embed_forward(const int32_t* ids, int64_t T, const void* E, int64_t V, int64_t D,
                                          float scale, mole_dtype dt_E, void* out, mole_dtype dt_out,
                                          cudaStream_t stream) {
  mole_status st = check_embed(ids, T, E, dt_E, V, D, out, dt_out);
  if (st != MOLE_OK || T == 0) return st;
  st = mole::check_device();
  if (st != MOLE_OK) return st;
  return mole::embed_forward(ids, T, E, V, D, scale, dt_E == MOLE_BF16, out, dt_out == MOLE_BF16, stream);
}

extern "C" size_t mole_embed_backward_workspace(int64_t T, int64_t D) {
  if (T <= 0 || T > INT32_MAX || D <= 0 || D > (1 << 20)) return 0;
  return mole::embed_backward_bytes(T, D);
}

extern "C" mole_status mole_embed_backward(const int32_t* ids, int64_t T, const void* dout, mole_dtype dt, int64_t V,
                                           int64_t D, float scale, float* dE, void* workspace, size_t ws_bytes,
                                           cudaStream_t stream) {
  mole_status st = check_embed(ids, T, dout, dt, V, D, dE, MOLE_F32);
  if (st != MOLE_OK || T == 0) return st;
  if (!workspace || ws_bytes < mole::embed_backward_bytes(T, D)) return MOLE_ERR_WORKSPACE;
  if (!mole::aligned16(workspace)) return MOLE_ERR_ALIGN;
  st = mole::check_device();
  if (st != MOLE_OK) return st;
  return mole::embed_backward(ids, T, dout, dt == MOLE_BF16, V, D, scale, dE, workspace, stream);
}
