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
//      id), by a radix sort of 8-bit digits run by ONE cluster of 16 CTAs: the
//      digit counts of its 512 warps meet in distributed shared memory, so a
//      pass costs two cluster barriers instead of two kernel boundaries (up to
//      kOneCtaTokens by one CTA).
//   2. embed_chunk_kernel: fixed chunks of the sorted order, one group of
//      threads per (chunk, slice of columns); the runs of equal ids go to dE,
//      but those longer than a chunk leave partial sums.
//   3. embed_join_kernel: per long run, its partial sums in chunk order.
// Batches of up to kSmallTokens do all of it in one launch (embed_small_kernel).
// Every sum has one order, fixed by the ids alone: the result has the same
// bits on every run.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace mole {
namespace {

namespace cg = cooperative_groups;

constexpr int kEmbedThreads = 256;
constexpr int kSortCtas = 16;  // 16 measured against 8: 12.1 -> 11.6 us at 16384 tokens, 37 -> 24 at 65536
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;
constexpr int kParts = kSortThreads / kDigits;  // groups of warps in a scan over them
constexpr int kChunkThreads = 128;
constexpr int kJoinThreads = 256;
constexpr int kChunkUnits = 2, kChunkSlots = 5, kScalarCols = 4;
constexpr int64_t kChunkGroups = 1776;  // chunks times slices: 12 CTAs for each of 148 SMs
constexpr int kSmallTokens = 1024, kSmallBatch = 8;
constexpr int kOneCtaTokens = 2048;

// ---- forward ----
// blockDim = (tx, 256 / tx): a row slice per group of tx threads, kRows rows in
// flight each (their ids are loaded together, then their rows: two waits for
// memory per kRows rows).
template <bool kVec, class In, class Out, int kRows>
__global__ void __launch_bounds__(kEmbedThreads) embed_forward_kernel(const int32_t* __restrict__ ids, int64_t T,
                                                                      const In* __restrict__ E, int64_t V, int D,
                                                                      float scale, Out* __restrict__ out,
                                                                      unsigned* err) {
  const int tx = blockDim.x;
  const int slice0 = blockIdx.y * tx * 8;
  const int col0 = slice0 + (kVec ? 4 : 1) * (int)threadIdx.x;
  if (col0 >= D) return;
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * kRows;
  int32_t id[kRows];
  RowUnit<kVec, In, 8> row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) id[r] = t0 + r < T ? __ldg(ids + t0 + r) : 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (t0 + r < T && id[r] >= 0 && (int64_t)id[r] < V) row[r].load(E + (int64_t)id[r] * D, col0, tx, D);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (t0 + r >= T) return;
    float f[8];
    if (id[r] >= 0 && (int64_t)id[r] < V) {
      row[r].get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
    } else {
      if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(err, kErrIndex);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = NAN;
    }
    st_cols<kVec>(out + (t0 + r) * D, col0, tx, D, f);
  }
}

// Rows of a bf16 table that start inside a unit of 4 columns (D no multiple of
// 4), table and output starting on one: the units are those of out, shifted by up
// to 3 columns, so that stores are whole but at a row's ends; a unit's columns
// come from the two units of E that they lie in (the second one is the next
// thread's first: one read of memory), joined by the row's distance.  Half the
// accesses of single columns: 16384 x 2049 to bf16 38 us, by those 55; to fp32 47
// and 61.  (With an fp32 table the second unit costs more than it saves: 72 and 52.)

// The unit at element i (a multiple of 4) of E's n elements; what lies outside
// is not read.
__device__ __forceinline__ uint2 load_inside(const uint16_t* E, int64_t i, int64_t n) {
  if (i >= 0 && i + 4 <= n) return *reinterpret_cast<const uint2*>(E + i);
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = i + k >= 0 && i + k < n ? E[i + k] : 0;
  return make_uint2(x[0] | (x[1] << 16), x[2] | (x[3] << 16));
}

// Columns d .. d + 3 of two units.
__device__ __forceinline__ void join_units(uint2 x, uint2 next, int d, float (&f)[4]) {
  const uint32_t a[3] = {d & 2 ? x.y : x.x, d & 2 ? next.x : x.y, d & 2 ? next.y : next.x};
  const uint32_t lo = d & 1 ? __funnelshift_r(a[0], a[1], 16) : a[0];
  const uint32_t hi = d & 1 ? __funnelshift_r(a[1], a[2], 16) : a[1];
  f[0] = bf16_lo(lo); f[1] = bf16_hi(lo); f[2] = bf16_lo(hi); f[3] = bf16_hi(hi);
}

template <class Out, int kRows>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_forward_shifted_kernel(const int32_t* __restrict__ ids, int64_t T, const uint16_t* __restrict__ E, int64_t V,
                                 int D, float scale, Out* __restrict__ out, unsigned* err) {
  const int tx = blockDim.x;
  const int unit0 = blockIdx.y * tx * 8 + 4 * (int)threadIdx.x;  // the first unit's place; the second: 4 tx on
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * kRows, n = V * D;
  int32_t id[kRows];
  uint2 x[kRows][2], next[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) id[r] = t0 + r < T ? __ldg(ids + t0 + r) : -1;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (id[r] < 0 || (int64_t)id[r] >= V) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int col = unit0 + 4 * u * tx - (int)(((t0 + r) * D) & 3);
      if (col >= D) continue;
      const int64_t first = (int64_t)id[r] * D + col;
      x[r][u] = load_inside(E, first & ~(int64_t)3, n);
      if (first & 3) next[r][u] = load_inside(E, (first & ~(int64_t)3) + 4, n);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (t0 + r >= T) return;
    const bool ok = id[r] >= 0 && (int64_t)id[r] < V;
    if (!ok && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(err, kErrIndex);
    const int shift = (int)(((t0 + r) * D) & 3), d = (int)(((int64_t)id[r] * D - shift) & 3);
    Out* row = out + (t0 + r) * D;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int col = unit0 + 4 * u * tx - shift;
      if (col >= D) continue;
      float f[4];
      join_units(x[r][u], next[r][u], d, f);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = ok ? f[k] * scale : NAN;
      if (col >= 0 && col + 4 <= D) {
        st_unit(row + col, f[0], f[1], f[2], f[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (col + k >= 0 && col + k < D) st1(row + col + k, f[k]);
      }
    }
  }
}

// ---- gradient, step 1: the stable sort ----
struct SortArgs {
  const int32_t* ids;
  int64_t T, V;
  int2* to;      // {id, t}: the sorted elements
  int2* other;   // the second buffer of the global passes, which end in `to`
  int passes;
  int* n_runs;   // cleared for the chunk kernel
  unsigned* err;
};

// Key of a bad id: V, behind every row (keys fit 31 bits: V <= 2^31 - 1).
__device__ __forceinline__ int2 sort_key(const int32_t* ids, int64_t V, int64_t i) {
  const int32_t id = __ldg(ids + i);
  return make_int2(id >= 0 && (int64_t)id < V ? id : (int)V, (int)i);
}

// Digits and counts of a radix pass run by one CTA (of kSortWarps warps).
struct SortSmem {
  int hist[kSortWarps][kDigits];  // per warp: its count of a digit, then its offset inside the CTA
  int psum[kParts][kDigits];
  int tot[kSortCtas][kDigits];    // per digit: the CTAs' counts (by rank; one CTA: [0])
  int base[kDigits];              // per digit: position of the CTA's first element
  int wsum[kDigits / 32];
};

// Ranks of a warp's tiles e[j] (elements 32 j + lane < n of its range) among
// the elements of equal digit that the warp has seen; hist counts on.  The
// lanes of equal digit come from one ballot per bit (__match_any_sync took
// 1.1 us a tile with 32 warps on the SM).
template <int kHold>
__device__ __forceinline__ void rank_tiles(const int2 (&e)[kHold], int (&rank)[kHold], int64_t n, int shift,
                                           int* hist) {
  const int lane = threadIdx.x & 31;
  const unsigned lower = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    if (32 * j >= n) break;
    const bool in = 32 * j + lane < n;
    const int d = in ? ((unsigned)e[j].x >> shift) & (kDigits - 1) : 0;
    unsigned same = __ballot_sync(0xffffffffu, in);  // the lanes of this lane's digit
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const unsigned ones = __ballot_sync(0xffffffffu, (d >> b) & 1);
      same &= (d >> b) & 1 ? ones : ~ones;
    }
    const int off = hist[d];
    __syncwarp();
    if (in) {
      rank[j] = off + __popc(same & lower);
      if ((same & lower) == 0) hist[d] = off + __popc(same);
    }
    __syncwarp();
  }
}

// hist (counts per warp) to offsets inside the CTA; returns the CTA's count of
// the thread's digit (threadIdx.x % kDigits).
__device__ __forceinline__ int scan_warps(SortSmem& s) {
  constexpr int kPartWarps = kSortWarps / kParts;
  const int digit = threadIdx.x & (kDigits - 1), part = threadIdx.x / kDigits;
  int c[kPartWarps], run = 0;
#pragma unroll
  for (int w = 0; w < kPartWarps; ++w) {
    c[w] = run;
    run += s.hist[part * kPartWarps + w][digit];
  }
  s.psum[part][digit] = run;
  __syncthreads();
  int start = 0, all = 0;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    if (p == part) start = all;
    all += s.psum[p][digit];
  }
#pragma unroll
  for (int w = 0; w < kPartWarps; ++w) s.hist[part * kPartWarps + w][digit] = start + c[w];
  return all;
}

// base[d] = sum of `all` over the digits before d, plus `before` (threads below
// kDigits hold their digit's values).
__device__ __forceinline__ void scan_digits(SortSmem& s, int all, int before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = all;
  if (threadIdx.x < kDigits) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s.wsum[warp] = incl;
  }
  __syncthreads();
  if (threadIdx.x < kDigits) {
    int off = incl - all + before;
#pragma unroll
    for (int w = 0; w < kDigits / 32; ++w)
      if (w < warp) off += s.wsum[w];
    s.base[threadIdx.x] = off;
  }
  __syncthreads();
}

// The sort by one CTA of up to 32 * H * kSortWarps tokens, in its shared memory:
// `sorted` has the result.
template <int H>
__device__ __forceinline__ void cta_sort(SortSmem& s, const int32_t* ids, int T, int64_t V, int passes, int2* sorted,
                                         unsigned* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lo = 32 * H * warp;
  int2 e[H];
  int rank[H];
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const int i = lo + 32 * j + lane;
    if (i < T) {
      e[j] = sort_key(ids, V, i);
      if (blockIdx.x == 0 && (int64_t)e[j].x == V) atomicOr(err, kErrIndex);
    }
  }
  for (int pass = 0; pass < passes; ++pass) {
    for (int d = lane; d < kDigits; d += 32) s.hist[warp][d] = 0;
    __syncwarp();
    rank_tiles<H>(e, rank, T - lo, 8 * pass, s.hist[warp]);
    __syncthreads();
    scan_digits(s, scan_warps(s), 0);
#pragma unroll
    for (int j = 0; j < H; ++j)
      if (lo + 32 * j + lane < T) {
        const int d = ((unsigned)e[j].x >> (8 * pass)) & (kDigits - 1);
        sorted[s.base[d] + s.hist[warp][d] + rank[j]] = e[j];
      }
    __syncthreads();
    if (pass + 1 < passes) {
#pragma unroll
      for (int j = 0; j < H; ++j)
        if (lo + 32 * j + lane < T) e[j] = sorted[lo + 32 * j + lane];
    }
  }
}

// Up to kOneCtaTokens tokens: one CTA, no cluster barriers (the gradient of 1500
// tokens of 2048 16.2 us, by the cluster 18.5; of 4096 of 512 18.4 and 16.4).
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_one_kernel(const SortArgs a) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  SortSmem& s = *reinterpret_cast<SortSmem*>(sort_smem);
  int2* sorted = reinterpret_cast<int2*>(sort_smem + sizeof(SortSmem));  // [kOneCtaTokens]
  pdl_trigger();  // the chunk kernel may take its place on the other SMs
  if (threadIdx.x == 0) *a.n_runs = 0;
  cta_sort<kOneCtaTokens / kSortThreads>(s, a.ids, (int)a.T, a.V, a.passes, sorted, a.err);
  for (int i = threadIdx.x; i < (int)a.T; i += kSortThreads) a.to[i] = sorted[i];
}

// Where the sort's elements live between passes: while a CTA's share fits its
// shared memory (kHold > 0: kHold tiles of 32 a warp, held in registers inside
// a pass) the passes exchange them through distributed shared memory, else
// through the two global buffers, in batches of 8 tiles.
template <int kHold>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const SortArgs a) {
  constexpr bool kLocal = kHold > 0;
  constexpr int H = kLocal ? kHold : 8;
  extern __shared__ __align__(16) uint8_t sort_smem[];
  SortSmem& s = *reinterpret_cast<SortSmem*>(sort_smem);
  int2* mine = reinterpret_cast<int2*>(sort_smem + sizeof(SortSmem));  // kLocal: this CTA's elements
  pdl_trigger();  // the chunk kernel may take its place on the other SMs
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // waited for before the first access to another CTA's memory
  const int cta = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cta == 0 && threadIdx.x == 0) *a.n_runs = 0;
  // each warp owns a contiguous range of the input, so that warp order is input order
  const int64_t per = kLocal ? 32 * H : ((a.T + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const int64_t lo = std::min<int64_t>(a.T, per * (cta * kSortWarps + warp));
  const int64_t hi = std::min<int64_t>(a.T, lo + per);
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 8 * pass;
    const bool last = pass == a.passes - 1;
    int2 e[H];
    int rank[H];
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        if (i >= hi) continue;
        if (pass == 0)
          e[j] = sort_key(a.ids, a.V, i);
        else if (kLocal)
          e[j] = mine[i - per * kSortWarps * cta];
        else
          e[j] = __ldcg(((a.passes - pass) & 1 ? a.other : a.to) + i);  // another CTA wrote it: past L1
      }
    };
    for (int d = lane; d < kDigits; d += 32) s.hist[warp][d] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * H) {
      load(i0);
      if (pass == 0) {
#pragma unroll
        for (int j = 0; j < H; ++j)
          if (i0 + 32 * j + lane < hi && (int64_t)e[j].x == a.V) atomicOr(a.err, kErrIndex);
      }
      rank_tiles<H>(e, rank, hi - i0, shift, s.hist[warp]);
    }
    __syncthreads();
    // the CTA's counts to every CTA of the cluster: written, not read, across
    // it, so that their way is part of the barrier's
    const int count = scan_warps(s);
    if (pass == 0) cluster.barrier_wait(std::move(started));
#pragma unroll
    for (int r = 0; r < kSortCtas / kParts; ++r)
      cluster.map_shared_rank(&s.tot[cta][0], (threadIdx.x / kDigits) * (kSortCtas / kParts) + r)[threadIdx.x &
                                                                                               (kDigits - 1)] = count;
    cluster.sync();  // (and every element of `mine` is in registers)
    int before = 0, all = 0;
    if (threadIdx.x < kDigits) {
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const int x = s.tot[r][threadIdx.x];
        if (r < cta) before += x;
        all += x;
      }
    }
    scan_digits(s, all, before);
    int2* dst = (a.passes - 1 - pass) & 1 ? a.other : a.to;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * H) {
      if (!kLocal) {  // hist runs on from the warp's offset: rank counts from the CTA's first element
        load(i0);
        rank_tiles<H>(e, rank, hi - i0, shift, s.hist[warp]);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) {
        if (i0 + 32 * j + lane >= hi) continue;
        const int d = ((unsigned)e[j].x >> shift) & (kDigits - 1);
        const int pos = s.base[d] + rank[j] + (kLocal ? s.hist[warp][d] : 0);
        if (kLocal && !last) {
          const int share = 32 * H * kSortWarps;
          cluster.map_shared_rank(mine, pos / share)[pos % share] = e[j];
        } else {
          __stcg(dst + pos, e[j]);
        }
      }
    }
    // the pass's output is there, and tot has been read (the last pass's output
    // goes to global memory, and no CTA touches another's memory after it)
    if (!last) cluster.sync();
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
  float* part;  // [n_chunks][2][D]: sums of the part that entered the chunk, of the part that leaves it
  int* n_runs;  // runs with parts: how many,
  int2* runs;   // and of each {chunk where it begins, id}, in any order
};

// Rows of dout in order of their runs, column by column (any width and
// alignment): batches of kQ tokens have the loads of their rows in flight, and
// with them those rows of dE whose run ends in the batch (a load inside the sums
// would stall them once per run).  `at(p)` gives the sorted element p < end;
// runs that end in [p0, p1) go to dE, `head` takes the sum of a part that
// entered, `tail` of one that leaves.
template <class In, int C, int kQ, class At, class Head, class Tail>
__device__ __forceinline__ void sum_runs(const In* dout, float* dE, int D, float scale, int V, int p0, int p1, int end,
                                         int enters, int col0, int step, At at, Head head, Tail tail) {
  float acc[C];
  int cur = -1;
  int2 e[kQ + 1];
#pragma unroll
  for (int q = 0; q <= kQ; ++q) e[q] = p0 + q < end ? at(p0 + q) : make_int2(-1, 0);
  for (int p = p0; p < p1; p += kQ) {
    RowUnit<false, In, C> row[kQ];
    RowUnit<false, float, C> grad[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (p + q < p1 && e[q].x != V) {
        row[q].load(dout + (int64_t)e[q].y * D, col0, step, D);
        if (e[q].x != e[q + 1].x && e[q].x != enters) grad[q].load(dE + (int64_t)e[q].x * D, col0, step, D);
      }
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (p + q >= p1 || e[q].x == V) break;
      float f[C];
      row[q].get(f);
#pragma unroll
      for (int k = 0; k < C; ++k) acc[k] = e[q].x == cur ? acc[k] + f[k] : f[k];
      cur = e[q].x;
      const bool ends = e[q].x != e[q + 1].x;
      if (cur == enters) {
        if (ends || p + q + 1 == p1) head(acc);
      } else if (ends) {
        float g[C];
        grad[q].get(g);
#pragma unroll
        for (int k = 0; k < C; ++k) g[k] = fmaf(scale, acc[k], g[k]);
        st_cols<false>(dE + (int64_t)cur * D, col0, step, D, g);
      } else if (p + q + 1 == p1) {
        tail(cur, acc);
      }
    }
#pragma unroll
    for (int q = 0; q <= kQ; ++q) e[q] = p + kQ + q < end ? at(p + kQ + q) : make_int2(-1, 0);
  }
}

// Step 2.  blockDim = (tx, 128 / tx): threadIdx.y = chunk inside the CTA,
// blockIdx.y = slice of columns.  A chunk's share is its own tokens, with one
// change at each border so that only runs longer than a chunk have parts: a run
// that crosses one border belongs whole to the chunk where it begins.
struct Share {
  int begin, end;  // tokens of the share, from the chunk's first one; end may pass the chunk
  int enters;      // the id (or -1) of a part that entered the chunk
};

// `id(i)`: id of the i-th token from the chunk's first, -1 outside the batch,
// for i from -chunk - 1 to 2 * chunk; n tokens in the chunk.
template <class Id>
__device__ __forceinline__ Share chunk_share(int n, int chunk, Id id) {
  Share s{0, n, -1};
  const int first = id(0), last = id(n - 1);
  if (id(-1) == first) {
    // one border crossed: it begins in the chunk before this one and ends here
    if (id(-chunk - 1) != first && id(chunk) != first) {
      while (s.begin < n && id(s.begin) == first) ++s.begin;
    } else {
      s.enters = first;
    }
  }
  // (a run that reaches behind the next chunk leaves a part)
  if (n == chunk && id(n) == last && s.enters != last && id(2 * chunk) != last)
    while (id(s.end) == last) ++s.end;
  return s;
}

// After the sort: the tokens of the chunk and of the next one into es[0] ..
// es[2 * chunk - 1], and those at -1, 2 * chunk and (es[-2]) -chunk - 1.  Returns
// the number of tokens in the chunk; all threads of the CTA take part.
__device__ __forceinline__ int load_share(const SumArgs& a, int64_t c, int2* es) {
  const int64_t p0 = c * a.chunk;
  const int n = c < a.n_chunks ? (int)std::min<int64_t>(a.chunk, a.T - p0) : 0;
  pdl_wait();
  if (n > 0)
    for (int i = (int)threadIdx.x - 2; i <= 2 * a.chunk; i += blockDim.x) {
      const int64_t p = i == -2 ? p0 - a.chunk - 1 : p0 + i;
      es[i] = p >= 0 && p < a.T ? a.sorted[p] : make_int2(-1, 0);
    }
  __syncthreads();
  return n;
}

__device__ __forceinline__ void leave_run(const SumArgs& a, int64_t c, int id) {
  if (threadIdx.x == 0 && blockIdx.y == 0) a.runs[atomicAdd(a.n_runs, 1)] = make_int2((int)c, id);
}

// Vector rows: a thread streams its columns of the chunk's rows through a ring
// of kSlots slots of its own in shared memory (cp.async; nothing is shared
// between threads), so that kSlots rows are in flight per thread whatever the
// registers; with a row come the columns of dE where its run ends.  A thread
// has kUnits units of 4 columns, 4 * blockDim.x apart: accesses to dout and to
// dE are both contiguous over a warp, and the bookkeeping of a token serves all
// of them.  (Loads into registers, 8 tokens at a time: 47 us for 16384 Zipf
// tokens of 2048 fp32, this form 34; 1, 2 and 4 units and 4 to 14 slots: 2 and 5
// are the fastest together.)  Bound by HBM for ids that hardly repeat (65536 x
// 1024 bf16: 67 us against 66 at the copy rate), for text by the last CTAs: 9 us
// each, which nothing overlaps at the end.
template <class In, int kUnits, int kSlots>
__global__ void __launch_bounds__(kChunkThreads) embed_chunk_kernel(const SumArgs a) {
  constexpr int kIn = 4 * sizeof(In), kUnitBytes = kIn + 16, kSlotBytes = kUnits * kUnitBytes * kChunkThreads;
  extern __shared__ __align__(16) uint8_t chunk_smem[];
  // slot: per unit the threads' columns of dout, then their columns of dE
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  int2* es = reinterpret_cast<int2*>(chunk_smem + (size_t)kSlots * kSlotBytes) +
             (size_t)threadIdx.y * (2 * a.chunk + 3) + 2;
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int step = blockDim.x;
  const int col0 = blockIdx.y * step * 4 * kUnits + 4 * (int)threadIdx.x;
  const int n = load_share(a, c, es);
  if (n == 0 || col0 >= a.D) return;
  const Share share = chunk_share(n, a.chunk, [&](int i) { return es[i < -1 ? -2 : i].x; });
  const int units = std::min(kUnits, (a.D - col0 + 4 * step - 1) / (4 * step));  // those that begin inside the row
  const In* dout = static_cast<const In*>(a.dout) + col0;
  float* dE = a.dE + col0;
  const int V = (int)a.V;
  float* part = a.part + 2 * c * a.D + col0;
  auto fetch = [&](int i, int at) {
    if (i < share.end && es[i].x != V) {
      uint8_t* slot = chunk_smem + at * kSlotBytes;
      const int2 e = es[i];
      const In* row = dout + (int64_t)e.y * a.D;
      const bool whole = e.x != es[i + 1].x && e.x != share.enters;
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (u < units) {
          cp_async<kIn>(slot + (u * kChunkThreads + tid) * kIn, row + u * 4 * step);
          if (whole)
            cp_async<16>(slot + kUnits * kChunkThreads * kIn + (u * kChunkThreads + tid) * 16,
                         dE + (int64_t)e.x * a.D + u * 4 * step);
        }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) fetch(share.begin + i, i);
  float acc[kUnits][4];
  int cur = -1, at = 0;
  for (int i = share.begin; i < share.end; ++i) {
    const int id = es[i].x;
    if (id == V) break;
    fetch(i + kSlots - 1, at == 0 ? kSlots - 1 : at - 1);
    cp_async_wait<kSlots - 1>();
    const uint8_t* slot = chunk_smem + at * kSlotBytes;
    at = at + 1 == kSlots ? 0 : at + 1;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float f[4];
      ld_unit(reinterpret_cast<const In*>(slot + (u * kChunkThreads + tid) * kIn), f);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[u][k] = id == cur ? acc[u][k] + f[k] : f[k];
    }
    cur = id;
    const bool ends = id != es[i + 1].x;
    if (!ends && i + 1 != share.end) continue;
    float* to = part;  // a part that entered
    if (id != share.enters) {
      if (ends) {
        to = dE + (int64_t)id * a.D;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const float4 x = *reinterpret_cast<const float4*>(slot + kUnits * kChunkThreads * kIn +
                                                            (u * kChunkThreads + tid) * 16);
          acc[u][0] = fmaf(a.scale, acc[u][0], x.x);
          acc[u][1] = fmaf(a.scale, acc[u][1], x.y);
          acc[u][2] = fmaf(a.scale, acc[u][2], x.z);
          acc[u][3] = fmaf(a.scale, acc[u][3], x.w);
        }
      } else {
        to = part + a.D;
        leave_run(a, c, id);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (u < units) st_unit(to + u * 4 * step, acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
  }
  cp_async_wait<0>();
}

// Rows of any width and alignment.
template <class In>
__global__ void __launch_bounds__(kChunkThreads) embed_chunk_scalar_kernel(const SumArgs a) {
  constexpr int C = kScalarCols, kQ = 2;
  extern __shared__ __align__(16) uint8_t chunk_smem[];
  int2* es = reinterpret_cast<int2*>(chunk_smem) + (size_t)threadIdx.y * (2 * a.chunk + 3) + 2;
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int step = blockDim.x;
  const int col0 = blockIdx.y * step * C + (int)threadIdx.x;
  const int n = load_share(a, c, es);
  if (n == 0 || col0 >= a.D) return;
  const Share share = chunk_share(n, a.chunk, [&](int i) { return es[i < -1 ? -2 : i].x; });
  float* part = a.part + 2 * c * a.D;
  sum_runs<In, C, kQ>(
      static_cast<const In*>(a.dout), a.dE, a.D, a.scale, (int)a.V, share.begin, share.end, 2 * a.chunk + 1,
      share.enters, col0, step, [&](int i) { return es[i]; },
      [&](const float(&acc)[C]) { st_cols<false>(part, col0, step, a.D, acc); },
      [&](int id, const float(&acc)[C]) {
        st_cols<false>(part + a.D, col0, step, a.D, acc);
        leave_run(a, c, id);
      });
}

// Number of chunks after c that the run of `id` enters (sorted ids: a prefix of
// them), by a warp: 1024 chunks in two probes, 31 in one.
__device__ __forceinline__ int64_t chunks_entered(const SumArgs& a, int64_t c, int id) {
  const int lane = threadIdx.x & 31;
  auto enters = [&](int64_t k) { return k < a.n_chunks && a.sorted[k * a.chunk].x == id; };
  int64_t n = 0;  // chunks c + 1 .. c + n are entered
  for (;;) {
    const bool far = enters(c + n + 32 * (lane + 1)), near = enters(c + n + 1 + lane);
    const int blocks = __popc(__ballot_sync(0xffffffffu, far)), rest = __popc(__ballot_sync(0xffffffffu, near));
    if (blocks == 0) return n + rest;
    n += 32 * blocks;
  }
}

// Step 3: the parts of the long runs, in chunk order, onto dE.  (The order of
// the list of runs does not matter: each has its own row.)  Item = (run, 128
// columns), a CTA each: its warps take the parts in contiguous shares, whose
// sums are added in order.  Bound by the chain of loads; 8 warps a CTA: 9600
// tokens of 544 ids 23.2 us, 4 warps 25.6, 16 warps 22.6 (but text 55 against 53).
template <bool kVec>
__global__ void __launch_bounds__(kJoinThreads, 4) embed_join_kernel(const SumArgs a) {
  constexpr int C = 4, kWarpsJ = kJoinThreads / 32, kQ = 8;
  __shared__ float sums[kWarpsJ][C][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned slices = (a.D + 32 * C - 1) / (32 * C);
  int2 r = a.runs[blockIdx.x / slices];  // with the count: used if there is such a run
  const unsigned items = (unsigned)*a.n_runs * slices;
  for (unsigned it = blockIdx.x; it < items; it += gridDim.x, r = it < items ? a.runs[it / slices] : r) {
    const int col0 = (int)(it % slices) * 32 * C + (kVec ? C : 1) * lane;
    const int64_t c = r.x;
    float* to = a.dE + (int64_t)r.y * a.D;
    RowUnit<kVec, float, C> grad;
    if (warp == 0 && col0 < a.D) grad.load(to, col0, 32, a.D);
    // part 0 left chunk c, part k entered chunk c + k
    const int64_t n = 1 + chunks_entered(a, c, r.y);
    const int64_t k1 = n * (warp + 1) / kWarpsJ;
    float acc[C];
#pragma unroll
    for (int k = 0; k < C; ++k) acc[k] = 0.f;
    if (col0 < a.D)
      for (int64_t k0 = n * warp / kWarpsJ; k0 < k1; k0 += kQ) {
        RowUnit<kVec, float, C> f[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q)
          if (k0 + q < k1) f[q].load(a.part + (2 * (c + k0 + q) + (k0 + q == 0)) * a.D, col0, 32, a.D);
#pragma unroll
        for (int q = 0; q < kQ; ++q)
          if (k0 + q < k1) {
            float x[C];
            f[q].get(x);
#pragma unroll
            for (int k = 0; k < C; ++k) acc[k] += x[k];
          }
      }
#pragma unroll
    for (int k = 0; k < C; ++k) sums[warp][k][lane] = acc[k];
    __syncthreads();
    if (warp == 0 && col0 < a.D) {
      for (int w = 1; w < kWarpsJ; ++w)
#pragma unroll
        for (int k = 0; k < C; ++k) acc[k] += sums[w][k][lane];
      float g[C];
      grad.get(g);
#pragma unroll
      for (int k = 0; k < C; ++k) g[k] = fmaf(a.scale, acc[k], g[k]);
      st_cols<kVec>(to, col0, 32, a.D, g);
    }
    __syncthreads();
  }
}

// ---- gradient of a small batch (T <= kSmallTokens): one launch ----
// CTA = a strip of G columns, one a lane (any width and alignment).  Every CTA
// sorts the whole batch in its shared memory (a few us; the other strips do the
// same beside it), its kSortThreads / G groups of G lanes sum equal shares of the
// sorted tokens, and the runs that cross a share are joined from shared memory.
template <class In, int G>
__global__ void __launch_bounds__(kSortThreads, 1)
    embed_small_kernel(const int32_t* __restrict__ ids, int T, int64_t V, int passes, const In* __restrict__ dout,
                       int D, float scale, float* dE, unsigned* err) {
  constexpr int kShares = kSortThreads / G;
  extern __shared__ __align__(16) uint8_t sort_smem[];
  SortSmem& s = *reinterpret_cast<SortSmem*>(sort_smem);
  int2* sorted = reinterpret_cast<int2*>(sort_smem + sizeof(SortSmem));  // [kSmallTokens]
  float* part = reinterpret_cast<float*>(sorted + kSmallTokens);         // [kShares][2][G]
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  cta_sort<kSmallTokens / kSortThreads>(s, ids, T, V, passes, sorted, err);
  const int col = blockIdx.x * G + lane;
  auto begin = [&](int w) { return (int)((int64_t)T * w / kShares); };
  const int p0 = begin(group), p1 = begin(group + 1);
  float* entering = part + group * 2 * G + lane;
  float* leaving = entering + G;
  int owner = -1;  // the id of the run that begins in this share and leaves it
  if (p0 < p1 && col < D)
    sum_runs<In, 1, kSmallBatch>(
        dout, dE, D, scale, (int)V, p0, p1, T, p0 > 0 ? sorted[p0 - 1].x : -1, col, G,
        [&](int p) { return sorted[p]; }, [&](const float(&acc)[1]) { *entering = acc[0]; },
        [&](int id, const float(&acc)[1]) {
          owner = id;
          *leaving = acc[0];
        });
  __syncthreads();
  if (owner < 0) return;
  float* to = dE + (int64_t)owner * D + col;
  const float before = *to;
  float acc = *leaving;
  for (int w = group + 1; w < kShares; ++w) {
    const int q0 = begin(w);
    if (q0 == begin(w + 1)) continue;  // an empty share
    if (sorted[q0].x != owner) break;
    acc += part[w * 2 * G + lane];
  }
  *to = fmaf(scale, acc, before);
}

// Tokens per chunk: enough (chunk, slice) groups to fill the GPU several times
// over (888 to 2368 groups measured within 5 % of each other at 16384 x 2048 and
// 65536 x 1024).  At least 8, so that the partial sums (2 fp32 rows of D per chunk)
// take no more workspace than T D bytes (half of a bf16 dout).  At most 256, since
// one group works through a chunk alone, and no more than leave room for the CTA's
// groups' tokens in 64 KB of shared memory (narrow rows: up to 128 groups).
int chunk_tokens(int64_t T, int64_t D) {
  const RowSplit r = row_split(D, 4 * kChunkUnits, kChunkThreads);
  const int64_t groups = std::max<int64_t>(1, kChunkGroups * (kChunkThreads / r.tx) / r.slices);
  const int64_t room = (64 * 1024 / 8 / (kChunkThreads / r.tx) - 3) / 2;
  return (int)std::min<int64_t>(std::min<int64_t>(256, room), std::max<int64_t>(8, (T + groups - 1) / groups));
}

struct EmbedWs {
  int2* buf[2];  // [T] sorted elements
  int* n_runs;
  int2* runs;    // [n_chunks]
  float* part;   // [n_chunks][2][D]
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
  const size_t n_chunks = (size_t)((T + chunk - 1) / chunk);
  const size_t o_r = take(16 + 8 * n_chunks);
  const size_t o_p = take(8 * n_chunks * (size_t)D);
  if (w != nullptr) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    w->buf[0] = reinterpret_cast<int2*>(b + o_a);
    w->buf[1] = reinterpret_cast<int2*>(b + o_b);
    w->n_runs = reinterpret_cast<int*>(b + o_r);
    w->runs = reinterpret_cast<int2*>(b + o_r + 16);
    w->part = reinterpret_cast<float*>(b + o_p);
  }
  return off;
}

template <bool kVec, class In>
cudaError_t launch_sums(const SumArgs& a, int n_sm, cudaStream_t stream) {
  const RowSplit s = row_split(a.D, kVec ? 4 * kChunkUnits : kScalarCols, kChunkThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(s.tx, kChunkThreads / s.tx);
  cfg.gridDim = dim3((unsigned)((a.n_chunks + cfg.blockDim.y - 1) / cfg.blockDim.y), s.slices);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  const size_t share_bytes = (size_t)cfg.blockDim.y * (2 * a.chunk + 3) * 8;
  if constexpr (kVec) {
    auto kern = embed_chunk_kernel<In, kChunkUnits, kChunkSlots>;
    cfg.dynamicSmemBytes = (size_t)kChunkSlots * kChunkUnits * (4 * sizeof(In) + 16) * kChunkThreads + share_bytes;
    e = allow_smem(kern);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, a);
  } else {
    auto kern = embed_chunk_scalar_kernel<In>;
    cfg.dynamicSmemBytes = share_bytes;
    e = allow_smem(kern);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, a);
  }
  if (e != cudaSuccess) return e;
  // Always launched (more than kSmallTokens make at least 4 chunks): the chunk
  // kernel lets the kernel behind it start early, which must be one that waits.
  // A run with parts enters a whole chunk: at most one per two chunks.
  const int64_t items = (a.n_chunks / 2) * ((a.D + 127) / 128);
  return launch_pdl(embed_join_kernel<kVec>, (unsigned)std::min<int64_t>(items, (int64_t)n_sm * 4), kJoinThreads, 0,
                    stream, a);
}

template <int kHold>
cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream) {
  const int smem = (int)sizeof(SortSmem) + kHold * kSortThreads * (int)sizeof(int2);
  cudaError_t e = allow_smem(embed_sort_kernel<kHold>);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(embed_sort_kernel<kHold>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  embed_sort_kernel<kHold><<<kSortCtas, kSortThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_sort_one(const SortArgs& a, cudaStream_t stream) {
  const cudaError_t e = allow_smem(embed_sort_one_kernel);
  if (e != cudaSuccess) return e;
  embed_sort_one_kernel<<<1, kSortThreads, sizeof(SortSmem) + kOneCtaTokens * sizeof(int2), stream>>>(a);
  return cudaGetLastError();
}

// Strips of 16 columns where shares of 32-column strips take more than a batch of
// tokens and an SM has one strip at most: the shares are half as long then (777
// tokens of 1001 bf16 10.3 us, by 32 columns 12.3; 1024 of 1000 10.9 and 14.4;
// but 40 of 1272 7.5 and 6.8).  Strips of 8 gain no more (10.3).
template <class In>
cudaError_t launch_small(const int32_t* ids, int64_t T, int64_t V, int passes, const void* dout, int D, float scale,
                         float* dE, unsigned* err, int n_sm, cudaStream_t stream) {
  const int smem = (int)sizeof(SortSmem) + kSmallTokens * 8 + kSortThreads * 2 * 4;
  const int G = T > kSmallBatch * 32 && D <= 16 * n_sm ? 16 : 32;
  auto kern = G == 16 ? embed_small_kernel<In, 16> : embed_small_kernel<In, 32>;
  const cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((D + G - 1) / G), kSortThreads, smem, stream>>>(ids, (int)T, V, passes,
                                                                    static_cast<const In*>(dout), D, scale, dE, err);
  return cudaGetLastError();
}

// Rows per thread: 4 (2 of the shifted form, whose rows take twice the registers)
// once that leaves a CTA for every SM.
template <class In, class Out>
void launch_forward(const int32_t* ids, int64_t T, const In* E, int64_t V, int D, float scale, Out* out, unsigned* err,
                    int n_sm, cudaStream_t stream) {
  constexpr bool kBf16 = sizeof(In) == 2;
  const bool units = aligned_rows(E, kBf16) && aligned_rows(out, sizeof(Out) == 2), vec = units && D % 4 == 0;
  const bool shifted = units && !vec && kBf16;
  const RowSplit s = row_split(D + (shifted ? 3 : 0), 8, kEmbedThreads);
  const dim3 block(s.tx, kEmbedThreads / s.tx);
  const bool many = T * s.slices >= (int64_t)n_sm * 4 * block.y;
  const unsigned rows = block.y * (many ? shifted ? 2 : 4 : 1);
  const dim3 grid((unsigned)((T + rows - 1) / rows), s.slices);
  auto kern = vec    ? many ? embed_forward_kernel<true, In, Out, 4> : embed_forward_kernel<true, In, Out, 1>
              : many ? embed_forward_kernel<false, In, Out, 4>
                     : embed_forward_kernel<false, In, Out, 1>;
  if constexpr (kBf16) {
    if (shifted) kern = many ? embed_forward_shifted_kernel<Out, 2> : embed_forward_shifted_kernel<Out, 1>;
  }
  kern<<<grid, block, 0, stream>>>(ids, T, E, V, D, scale, out, err);
}

}  // namespace

mole_status embed_forward(const int32_t* ids, int64_t T, const void* E, int64_t V, int64_t D, float scale,
                          bool E_bf16, void* out, bool out_bf16, cudaStream_t stream) {
  unsigned* err = error_word();
  const int n_sm = num_sms();
  if (!err || n_sm <= 0) return MOLE_ERR_CUDA;
  auto rows = [&](auto* e, auto* o) { launch_forward(ids, T, e, V, (int)D, scale, o, err, n_sm, stream); };
  auto types = [&](auto* e) { out_bf16 ? rows(e, static_cast<uint16_t*>(out)) : rows(e, static_cast<float*>(out)); };
  E_bf16 ? types(static_cast<const uint16_t*>(E)) : types(static_cast<const float*>(E));
  return cuda_status(cudaGetLastError());
}

size_t embed_backward_bytes(int64_t T, int64_t D) { return carve_embed(nullptr, T, D, nullptr); }

mole_status embed_backward(const int32_t* ids, int64_t T, const void* dout, bool bf16, int64_t V, int64_t D,
                           float scale, float* dE, void* ws, cudaStream_t stream) {
  unsigned* err = error_word();
  if (!err) return MOLE_ERR_CUDA;
  const int n_sm = num_sms();
  if (n_sm <= 0) return MOLE_ERR_NO_DEVICE;
  EmbedWs w{};
  carve_embed(ws, T, D, &w);
  int bits = 0;  // of the keys 0 .. V
  while (bits < 32 && (V >> bits) != 0) ++bits;
  const int passes = (bits + 7) / 8;
  const bool vec = D % 4 == 0 && aligned_rows(dout, bf16) && aligned16(dE);
  cudaError_t e;
  if (T <= kSmallTokens)
    return cuda_status((bf16 ? launch_small<uint16_t> : launch_small<float>)(ids, T, V, passes, dout, (int)D, scale, dE,
                                                                            err, n_sm, stream));
  const SortArgs sa{ids, T, V, w.buf[0], w.buf[1], passes, w.n_runs, err};
  if (T <= kOneCtaTokens)
    e = launch_sort_one(sa, stream);
  else if (T <= kSortCtas * kSortThreads)
    e = launch_sort<1>(sa, stream);
  else if (T <= 4 * kSortCtas * kSortThreads)
    e = launch_sort<4>(sa, stream);
  else
    e = launch_sort<0>(sa, stream);
  if (e != cudaSuccess) return MOLE_ERR_CUDA;
  const int chunk = chunk_tokens(T, D);
  const SumArgs a{w.buf[0], T, V, (int)D, chunk, (T + chunk - 1) / chunk, dout, scale, dE, w.part, w.n_runs, w.runs};
  if (bf16)
    e = vec ? launch_sums<true, uint16_t>(a, n_sm, stream) : launch_sums<false, uint16_t>(a, n_sm, stream);
  else
    e = vec ? launch_sums<true, float>(a, n_sm, stream) : launch_sums<false, float>(a, n_sm, stream);
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
