// Embedding lookup with scaling, and its gradient by sorted tokens, summed
// straight into the flat, partitioned FP32 accumulation buffer.
//
// The gradient of row v is the sum of dout over the tokens with id v.  Token
// ids repeat with a long tail (a few rows get thousands of tokens, most get
// none or one), so adding with atomics would serialise on the frequent rows
// and make the sum's order, and its bits, depend on timing.  Instead:
//   k_embed_sort   sorts (id, position) by id, stably (radix, 9 bits a pass,
//                  one cluster of thread blocks);
//   k_embed_sum    walks the sorted tokens in blocks of kRun: a run of equal
//                  ids inside a block goes straight to its row of accum, a run
//                  that crosses blocks leaves partial sums;
//   k_embed_join   adds the partial sums of each crossing run in block order.
// So every sum has one fixed order, and the work is balanced whatever the ids.
#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include <cooperative_groups.h>

#include "token_ops.cuh"

namespace muon {
namespace {

namespace cg = cooperative_groups;
using tok::Vec;

__device__ int g_embedding_err;

int efail(int code, const std::string& msg) {
  set_last_error(msg.c_str());
  return code;
}

// ------------------------------------------------------------------ lookup

struct Lookup {
  const void* table;
  const void* ids;
  void* out;
  int64_t stride, ostride, n;
  int rows, cols, ids64;
  float scale;
};

__device__ __forceinline__ int lookup_id(const void* ids, int ids64, int64_t t, int rows) {
  const int id = tok::load_index(ids, ids64, t);
  if (id >= rows) {
    atomicCAS(&g_embedding_err, 0, kErrIndex);
    return -1;
  }
  return id < 0 ? -1 : id;
}

// blockDim.y tokens per block, blockDim.x threads along a row.  VEC: 16 bytes
// of the table per thread and step (rows of both arrays 16-byte aligned).
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256) k_lookup(const Lookup a) {
  constexpr int N = VEC ? Vec<TI>::N : 1;
  const int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.n) return;
  const int id = lookup_id(a.ids, a.ids64, t, a.rows);
  const TI* src = static_cast<const TI*>(a.table) + int64_t(id < 0 ? 0 : id) * a.stride;
  TO* dst = static_cast<TO*>(a.out) + t * a.ostride;
  const float scale = a.scale;
  const int nvec = a.cols / N;
#pragma unroll 4
  for (int i = threadIdx.x; i < nvec; i += blockDim.x) {
    float f[N];
    if constexpr (VEC) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (id >= 0) v = *reinterpret_cast<const uint4*>(src + i * N);
      Vec<TI>::unpack(v, f);
    } else {
      f[0] = id >= 0 ? tok::to_float(src[i]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = id >= 0 ? f[k] * scale : 0.f;
    if constexpr (VEC && sizeof(TI) == sizeof(TO)) {
      *reinterpret_cast<uint4*>(dst + i * N) = Vec<TO>::pack(f);
    } else if constexpr (VEC && sizeof(TO) == 4) {
      float4* d = reinterpret_cast<float4*>(dst + i * N);
      d[0] = make_float4(f[0], f[1], f[2], f[3]);
      d[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else if constexpr (VEC) {
      *reinterpret_cast<uint2*>(dst + i * N) =
          make_uint2(Vec<TO>::pack2(f[0], f[1]), Vec<TO>::pack2(f[2], f[3]));
    } else {
      dst[i] = tok::from_float<TO>(f[0]);
    }
  }
  for (int c = nvec * N + threadIdx.x; c < a.cols; c += blockDim.x)
    dst[c] = tok::from_float<TO>(id >= 0 ? tok::to_float(src[c]) * scale : 0.f);
}

template <typename TI, typename TO>
void launch_lookup(const Lookup& a, cudaStream_t s) {
  auto whole = [](const void* p, int64_t stride, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
  };
  const bool vec = whole(a.table, a.stride, sizeof(TI)) && whole(a.out, a.ostride, sizeof(TO)) &&
                   a.cols >= Vec<TI>::N;
  const int steps = vec ? a.cols / Vec<TI>::N : a.cols;
  int tx = 32;
  while (tx < 256 && tx * 4 < steps) tx *= 2;   // up to four loads in flight per thread
  const dim3 block(tx, 256 / tx);
  const unsigned grid = static_cast<unsigned>((a.n + block.y - 1) / block.y);
  if (vec) k_lookup<TI, TO, true><<<grid, block, 0, s>>>(a);
  else k_lookup<TI, TO, false><<<grid, block, 0, s>>>(a);
}

// ------------------------------------------------------------------ gradient

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kRun = 32;             // sorted tokens per block of k_embed_sum
constexpr int kSumX = 128;           // threads of k_embed_sum and k_embed_join

struct SortArgs {
  const void* ids;
  int ids64;
  int n, rows;
  int passes, bits;      // bits per pass
  int *key0, *val0;      // the result
  int *key1, *val1;
};

// Stable radix sort of (id, position) by id, tokens without a row last (key =
// rows).  One cluster; block r takes the r-th contiguous share of the tokens
// and each warp a contiguous share of that, so ranks in order of (bin, block,
// warp, token) keep the sort stable.  Per pass: each warp counts its tokens'
// bins (equal bins within a warp found by match_any, so no atomics), the
// counts become offsets, and each warp places its tokens.
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const SortArgs a) {
  __shared__ int count[kSortWarps][kSortBins];   // 32 KB
  __shared__ int total[kSortBins];               // this block's tokens per bin
  __shared__ int scan[kSortWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int nb = cl.num_blocks(), rank = cl.block_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int share = (a.n + nb * kSortWarps - 1) / (nb * kSortWarps);
  const int64_t from = int64_t(rank * kSortWarps + warp) * share;
  const int lo = static_cast<int>(from < a.n ? from : a.n);
  const int hi = static_cast<int>(from + share < a.n ? from + share : a.n);
  const unsigned below = (1u << lane) - 1;
  const int mask = (1 << a.bits) - 1;
  for (int p = 0; p < a.passes; ++p) {
    const bool to0 = ((a.passes - 1 - p) & 1) == 0;
    const int* ki = to0 ? a.key1 : a.key0;
    const int* vi = to0 ? a.val1 : a.val0;
    int* ko = to0 ? a.key0 : a.key1;
    int* vo = to0 ? a.val0 : a.val1;
    auto load = [&](int t) -> int {
      if (p) return ki[t];
      const int id = tok::load_index(a.ids, a.ids64, t);
      if (id >= a.rows) atomicCAS(&g_embedding_err, 0, kErrIndex);
      return id < 0 || id >= a.rows ? a.rows : id;
    };
    const int shift = p * a.bits;
    for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) (&count[0][0])[i] = 0;
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32) {
      const int t = t0 + lane;
      const unsigned on = __ballot_sync(0xffffffffu, t < hi);
      if (t < hi) {
        const int bin = static_cast<int>(static_cast<unsigned>(load(t)) >> shift) & mask;
        const unsigned same = __match_any_sync(on, bin);
        if ((same & below) == 0) count[warp][bin] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    // per bin: offsets of the warps within the block, and the block's total
    const int bin = threadIdx.x;   // kSortThreads == kSortBins
    int run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = count[w][bin];
      count[w][bin] = run;
      run += c;
    }
    total[bin] = run;
    cl.sync();
    int all = 0, before = 0;
    for (int b = 0; b < nb; ++b) {
      const int c = *cl.map_shared_rank(&total[bin], b);
      if (b < rank) before += c;
      all += c;
    }
    int incl = all;   // exclusive sum over the bins of the cluster's totals
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int base = incl - all + before;
    for (int w = 0; w < warp; ++w) base += scan[w];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) count[w][bin] += base;
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32) {
      const int t = t0 + lane;
      const unsigned on = __ballot_sync(0xffffffffu, t < hi);
      if (t < hi) {
        const int key = load(t);
        const int b = static_cast<int>(static_cast<unsigned>(key) >> shift) & mask;
        const unsigned same = __match_any_sync(on, b);
        const int at = count[warp][b] + __popc(same & below);
        __syncwarp(on);
        if ((same & below) == 0) count[warp][b] += __popc(same);
        ko[at] = key;
        vo[at] = p ? vi[t] : t;
      }
      __syncwarp();
    }
    cl.sync();   // the other blocks read ko / vo, and total, in the next pass
  }
}

// The parameter's runs in storage: elements [rel[i], rel[i + 1]) of the
// parameter start at storage index at[i].
struct Segments {
  int n;
  int64_t rel[MUON_EMBEDDING_MAX_SEGMENTS];
  int64_t at[MUON_EMBEDDING_MAX_SEGMENTS];
  int64_t numel;

  __device__ __forceinline__ int find(int64_t i) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (rel[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // storage index of element i, and how many elements follow in one piece
  __device__ __forceinline__ int64_t place(int64_t i, int64_t* room) const {
    const int k = find(i);
    *room = (k + 1 < n ? rel[k + 1] : numel) - i;
    return at[k] + (i - rel[k]);
  }
};

struct Grad {
  float* accum;
  const void* dout;
  int64_t dstride;
  int n, rows, cols;
  float scale;
  int overwrite;
  const int* key;
  const int* val;
  float* partial;   // two rows of `cols` per block of kRun tokens
  int blocks;       // blocks of kRun tokens
  int slabs;        // blocks of columns
  int fill_rows;    // rows of the table per filling block (overwrite)
};

// Thread columns.  VEC: N consecutive columns, moved as 16 bytes; else N
// columns kSumX apart (each access of a warp then covers consecutive ones).
template <int N, bool VEC>
__device__ __forceinline__ int column(int slab, int k) {
  return VEC ? (slab * kSumX + int(threadIdx.x)) * N + k
             : slab * kSumX * N + k * kSumX + int(threadIdx.x);
}

// accum[row] = old + scale * f
template <int N, bool VEC>
__device__ __forceinline__ void add_row(const Grad& g, const Segments& sg, int row, int slab,
                                        const float* f) {
  if constexpr (VEC) {
    const int c = column<N, VEC>(slab, 0);
    if (c >= g.cols) return;
    int64_t room;
    float* d = g.accum + sg.place(int64_t(row) * g.cols + c, &room);
    if (room >= N && (reinterpret_cast<uintptr_t>(d) & 15) == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        float4* q = reinterpret_cast<float4*>(d + k);
        float4 o = g.overwrite ? make_float4(0.f, 0.f, 0.f, 0.f) : *q;
        o.x += g.scale * f[k]; o.y += g.scale * f[k + 1];
        o.z += g.scale * f[k + 2]; o.w += g.scale * f[k + 3];
        *q = o;
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = column<N, VEC>(slab, k);
    if (c >= g.cols) continue;
    int64_t room;
    float* d = g.accum + sg.place(int64_t(row) * g.cols + c, &room);
    *d = (g.overwrite ? 0.f : *d) + g.scale * f[k];
  }
}

template <int N, bool VEC>
__device__ __forceinline__ float* partial_at(const Grad& g, int block, int which, int slab, int k) {
  return g.partial + (int64_t(block) * 2 + which) * g.cols + column<N, VEC>(slab, k);
}

// Rows that no token names, in [r0, r1): zeros.
__device__ void fill_rows(const Grad& g, const Segments& sg, int r0, int r1) {
  int lo = 0, hi = g.n;   // first sorted token with id >= r0
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (g.key[mid] < r0) lo = mid + 1; else hi = mid;
  }
  for (int r = r0; r < r1; ++r) {
    bool named = false;
    while (lo < g.n && g.key[lo] <= r) {
      named = true;
      // step over the run of r
      int a = lo, b = g.n;
      while (a < b) {
        const int mid = a + (b - a) / 2;
        if (g.key[mid] <= r) a = mid + 1; else b = mid;
      }
      lo = a;
    }
    if (named) continue;
    int64_t room;
    for (int c = threadIdx.x; c < g.cols; c += kSumX)
      g.accum[sg.place(int64_t(r) * g.cols + c, &room)] = 0.f;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumX) k_embed_sum(const Grad g, const __grid_constant__ Segments sg) {
  constexpr int N = Vec<T>::N;
  constexpr int U = 4;    // rows in flight
  if (blockIdx.x >= unsigned(g.blocks) * g.slabs) {
    const int r0 = (blockIdx.x - g.blocks * g.slabs) * g.fill_rows;
    return fill_rows(g, sg, r0, min(g.rows, r0 + g.fill_rows));
  }
  __shared__ int key[kRun + 2], val[kRun];   // key[0], key[n + 1]: the neighbours' ids
  const int block = blockIdx.x / g.slabs, slab = blockIdx.x % g.slabs;
  const int t0 = block * kRun, n = min(kRun, g.n - t0);
  for (int i = threadIdx.x; i < n + 2; i += kSumX) {
    const int t = t0 + i - 1;
    key[i] = t >= 0 && t < g.n ? g.key[t] : -1;
    if (i >= 1 && i <= n) val[i - 1] = g.val[t];
  }
  __syncthreads();
  if (key[1] >= g.rows) return;   // only tokens without a row from here on
  const T* dout = static_cast<const T*>(g.dout);
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  bool from_before = key[0] == key[1];
  auto flush = [&](int id, bool goes_on) {
    if (from_before || goes_on) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (column<N, VEC>(slab, k) < g.cols)
          *partial_at<N, VEC>(g, block, from_before ? 0 : 1, slab, k) = acc[k];
    } else {
      add_row<N, VEC>(g, sg, id, slab, acc);
    }
    from_before = false;
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
  };
  for (int j0 = 0; j0 < n; j0 += U) {
    float f[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      const bool on = j < n && key[j + 1] < g.rows;
      const T* row = dout + (on ? int64_t(val[j]) : 0) * g.dstride;
      if constexpr (VEC) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const int c = column<N, VEC>(slab, 0);
        if (on && c < g.cols) v = *reinterpret_cast<const uint4*>(row + c);
        Vec<T>::unpack(v, f[u]);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int c = column<N, VEC>(slab, k);
          f[u][k] = on && c < g.cols ? tok::to_float(row[c]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      if (j >= n || key[j + 1] >= g.rows) break;
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += f[u][k];
      const int next = key[j + 2];
      if (j + 1 == n || next != key[j + 1]) flush(key[j + 1], j + 1 == n && next == key[j + 1]);
    }
  }
}

// Block b joins the run that starts inside block b of tokens and goes on past
// it (if there is one).
template <int N, bool VEC>
__global__ void __launch_bounds__(kSumX) k_embed_join(const Grad g, const __grid_constant__ Segments sg) {
  const int block = blockIdx.x / g.slabs, slab = blockIdx.x % g.slabs;
  const int t0 = block * kRun, last = t0 + kRun - 1;
  if (last + 1 >= g.n) return;
  const int id = g.key[last];
  if (id >= g.rows || g.key[last + 1] != id) return;
  if (t0 > 0 && g.key[t0] == id && g.key[t0 - 1] == id) return;   // started earlier
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    acc[k] = column<N, VEC>(slab, k) < g.cols ? *partial_at<N, VEC>(g, block, 1, slab, k) : 0.f;
  for (int b = block + 1; b < g.blocks && g.key[b * kRun] == id; ++b)
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (column<N, VEC>(slab, k) < g.cols) acc[k] += *partial_at<N, VEC>(g, b, 0, slab, k);
  add_row<N, VEC>(g, sg, id, slab, acc);
}

struct Workspace {
  size_t key0, val0, key1, val1, partial, bytes;
};

int64_t token_blocks(int64_t n) { return (n + kRun - 1) / kRun; }

Workspace workspace_of(int64_t n, int cols) {
  Workspace w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~size_t(255);
    return p;
  };
  w.key0 = take(n * sizeof(int));
  w.val0 = take(n * sizeof(int));
  w.key1 = take(n * sizeof(int));
  w.val1 = take(n * sizeof(int));
  w.partial = take(size_t(token_blocks(n)) * 2 * cols * sizeof(float));
  w.bytes = at;
  return w;
}

// The parameter's pieces in storage, in flat order.
int segments_of(const muon_param_t& p, const muon_partition_t* parts, int nparts, Segments* out) {
  const int64_t numel = int64_t(p.rows) * p.cols;
  out->numel = numel;
  if (nparts == 0) {
    out->n = 1;
    out->rel[0] = 0;
    out->at[0] = p.offset;
    return MUON_OK;
  }
  std::vector<std::pair<int64_t, int64_t>> st;
  for (int i = 0; i < nparts; ++i) {
    const muon_partition_t& q = parts[i];
    if (q.flat_begin < 0 || q.flat_end < q.flat_begin || q.storage_offset < 0)
      return efail(MUON_ERR_INVALID, "partition " + std::to_string(i) + " has a bad range");
    if (i > 0 && parts[i - 1].flat_end > q.flat_begin)
      return efail(MUON_ERR_INVALID, "partitions must be sorted by flat_begin and must not overlap (at " +
                                         std::to_string(i) + ")");
    if (q.flat_end > q.flat_begin)
      st.push_back({q.storage_offset, q.storage_offset + q.flat_end - q.flat_begin});
  }
  std::sort(st.begin(), st.end());
  for (size_t i = 1; i < st.size(); ++i)
    if (st[i - 1].second > st[i].first) return efail(MUON_ERR_INVALID, "partitions overlap in storage");
  int64_t cursor = 0;
  out->n = 0;
  for (int i = 0; i < nparts && cursor < numel; ++i) {
    const muon_partition_t& q = parts[i];
    const int64_t lo = std::max(p.offset, q.flat_begin) - p.offset;
    const int64_t hi = std::min(p.offset + numel, q.flat_end) - p.offset;
    if (lo >= hi) continue;
    if (lo != cursor) break;
    if (out->n == MUON_EMBEDDING_MAX_SEGMENTS)
      return efail(MUON_ERR_UNSUPPORTED, "the parameter lies in more than MUON_EMBEDDING_MAX_SEGMENTS partitions");
    out->rel[out->n] = lo;
    out->at[out->n++] = q.storage_offset + (p.offset + lo - q.flat_begin);
    cursor = hi;
  }
  if (cursor != numel) return efail(MUON_ERR_INVALID, "the parameter is not covered by the partitions");
  return MUON_OK;
}

int launch_sort(const SortArgs& a, cudaStream_t s) {
  // one warp per 128 tokens, up to a cluster of eight blocks
  int blocks = 1;
  while (blocks < 8 && a.n > blocks * 2048) blocks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_embed_sort, a) == cudaSuccess;
}

template <typename T>
int launch_grad(Grad g, const Segments& sg, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  bool vec = reinterpret_cast<uintptr_t>(g.dout) % 16 == 0 && g.dstride * sizeof(T) % 16 == 0 &&
             g.cols % N == 0;
  for (int i = 0; i < sg.n && vec; ++i) vec = (sg.at[i] - sg.rel[i]) % 4 == 0 && sg.rel[i] % 4 == 0;
  g.slabs = (g.cols + kSumX * N - 1) / (kSumX * N);
  g.fill_rows = std::max(1, 16384 / g.cols);
  const int64_t fills = g.overwrite ? (g.rows + g.fill_rows - 1) / g.fill_rows : 0;
  const int64_t grid = int64_t(g.blocks) * g.slabs + fills;
  if (grid > 0x7fffffff) return -1;
  int k = 0;
  if (grid > 0) {
    if (vec) k_embed_sum<T, true><<<static_cast<unsigned>(grid), kSumX, 0, s>>>(g, sg);
    else k_embed_sum<T, false><<<static_cast<unsigned>(grid), kSumX, 0, s>>>(g, sg);
    ++k;
  }
  if (g.blocks > 1) {
    const unsigned jg = static_cast<unsigned>(int64_t(g.blocks) * g.slabs);
    if (vec) k_embed_join<N, true><<<jg, kSumX, 0, s>>>(g, sg);
    else k_embed_join<N, false><<<jg, kSumX, 0, s>>>(g, sg);
    ++k;
  }
  return k;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

size_t dtype_bytes(int dtype) {
  return dtype == MUON_DTYPE_BF16 ? 2 : dtype == MUON_DTYPE_FP32 ? 4 : 0;
}

// The checks the lookup and its gradient share.  x: the rows of `cols`
// elements per token (out or dout).
int check_tokens(int rows, int cols, const void* ids, int ids_type, int64_t n, float scale,
                 const void* x, int x_dtype, int64_t x_stride, const char* name) {
  if (ids_type != MUON_INDEX_INT32 && ids_type != MUON_INDEX_INT64)
    return efail(MUON_ERR_INVALID, "unknown ids_type");
  if (!dtype_bytes(x_dtype)) return efail(MUON_ERR_INVALID, std::string("unknown ") + name + "_dtype");
  if (rows < 1 || cols < 1) return efail(MUON_ERR_INVALID, "rows or cols < 1");
  if (cols > (1 << 30)) return efail(MUON_ERR_UNSUPPORTED, "cols > 2^30");
  if (n < 0 || n > (int64_t(1) << 30)) return efail(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30]");
  if (x_stride < cols) return efail(MUON_ERR_INVALID, std::string(name) + "_stride must be >= cols");
  if (!std::isfinite(scale)) return efail(MUON_ERR_INVALID, "scale must be finite");
  if (n > 0 && (!ids || !x)) return efail(MUON_ERR_INVALID, std::string("ids or ") + name + " is NULL");
  if (misaligned(ids, ids_type == MUON_INDEX_INT64 ? 8 : 4) || misaligned(x, dtype_bytes(x_dtype)))
    return efail(MUON_ERR_INVALID, std::string("ids or ") + name + " is not aligned to its type");
  return MUON_OK;
}

int begin_call() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return efail(MUON_ERR_CUDA, "cudaGetDevice failed");
  note_token_device(dev);
  return MUON_OK;
}

int end_call(int launches) {
  count_launches(launches);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return efail(MUON_ERR_CUDA, std::string("kernel launch: ") + cudaGetErrorString(e));
  return MUON_OK;
}

}  // namespace

int embedding_take_device_error() { return take_flag(g_embedding_err); }

}  // namespace muon

using namespace muon;

extern "C" int muon_embedding(const void* table, int table_dtype, int64_t table_stride, int rows,
                              int cols, const void* ids, int ids_type, int64_t n_tokens,
                              float scale, void* out, int out_dtype, int64_t out_stride,
                              void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_embedding");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    int rc = check_tokens(rows, cols, ids, ids_type, n_tokens, scale, out, out_dtype, out_stride, "out");
    if (rc != MUON_OK) return rc;
    const size_t te = dtype_bytes(table_dtype), oe = dtype_bytes(out_dtype);
    if (!te) return efail(MUON_ERR_INVALID, "unknown table_dtype");
    if (table_stride < cols) return efail(MUON_ERR_INVALID, "table_stride must be >= cols");
    if (n_tokens == 0) return MUON_OK;
    if (!table || misaligned(table, te)) return efail(MUON_ERR_INVALID, "table is NULL or misaligned");
    const uintptr_t t0 = reinterpret_cast<uintptr_t>(table), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t t1 = t0 + (int64_t(rows - 1) * table_stride + cols) * te;
    const uintptr_t o1 = o0 + ((n_tokens - 1) * out_stride + cols) * oe;
    if (t0 < o1 && o0 < t1) return efail(MUON_ERR_INVALID, "out overlaps the table");
    if ((rc = begin_call()) != MUON_OK) return rc;
    const Lookup a{table, ids, out, table_stride, out_stride, n_tokens, rows, cols,
                   ids_type == MUON_INDEX_INT64, scale};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (te == 2 && oe == 2) launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, s);
    else if (te == 2) launch_lookup<__nv_bfloat16, float>(a, s);
    else if (oe == 2) launch_lookup<float, __nv_bfloat16>(a, s);
    else launch_lookup<float, float>(a, s);
    return end_call(1);
  });
}

extern "C" int muon_embedding_grad_workspace(int64_t n_tokens, int cols, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    if (n_tokens < 0 || n_tokens > (int64_t(1) << 30) || cols < 1 || cols > (1 << 30) || !bytes)
      return efail(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30], cols in [1, 2^30] and bytes non-NULL");
    *bytes = workspace_of(n_tokens, cols).bytes;
    return MUON_OK;
  });
}

extern "C" int muon_embedding_grad(float* accum, const void* dout, int dout_dtype,
                                   int64_t dout_stride, const void* ids, int ids_type,
                                   int64_t n_tokens, float scale, int overwrite,
                                   const muon_param_t* param, const muon_partition_t* parts,
                                   int nparts, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_embedding_grad");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    if (!param) return efail(MUON_ERR_INVALID, "param is NULL");
    int rc = check_tokens(param->rows, param->cols, ids, ids_type, n_tokens, scale, dout, dout_dtype,
                          dout_stride, "dout");
    if (rc != MUON_OK) return rc;
    if (param->offset < 0) return efail(MUON_ERR_INVALID, "the parameter's offset < 0");
    if (overwrite != 0 && overwrite != 1) return efail(MUON_ERR_INVALID, "overwrite must be 0 or 1");
    if (!accum || misaligned(accum, 16)) return efail(MUON_ERR_INVALID, "accum must be 16-byte aligned");
    if (nparts < 0 || (nparts > 0 && !parts)) return efail(MUON_ERR_INVALID, "parts is NULL");
    Segments sg;
    if ((rc = segments_of(*param, parts, nparts, &sg)) != MUON_OK) return rc;
    const Workspace w = workspace_of(n_tokens, param->cols);
    if (w.bytes > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < w.bytes))
      return efail(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
    if (n_tokens == 0 && !overwrite) return MUON_OK;
    if ((rc = begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    auto ints = [&](size_t at) { return reinterpret_cast<int*>(base + at); };
    SortArgs so{};
    so.ids = ids;
    so.ids64 = ids_type == MUON_INDEX_INT64;
    so.n = static_cast<int>(n_tokens);
    so.rows = param->rows;
    int bits = 1;
    while (bits < 32 && (int64_t(1) << bits) <= param->rows) ++bits;   // keys 0 .. rows
    so.passes = (bits + kSortBits - 1) / kSortBits;
    so.bits = (bits + so.passes - 1) / so.passes;
    so.key0 = ints(w.key0);
    so.val0 = ints(w.val0);
    so.key1 = ints(w.key1);
    so.val1 = ints(w.val1);
    int launches = 0;
    if (n_tokens > 0) {
      if (!launch_sort(so, s)) return end_call(0);
      ++launches;
    }
    Grad g{};
    g.accum = accum;
    g.dout = dout;
    g.dstride = dout_stride;
    g.n = so.n;
    g.rows = param->rows;
    g.cols = param->cols;
    g.scale = scale;
    g.overwrite = overwrite;
    g.key = so.key0;
    g.val = so.val0;
    g.partial = reinterpret_cast<float*>(base + w.partial);
    g.blocks = static_cast<int>(token_blocks(n_tokens));
    const int k = dout_dtype == MUON_DTYPE_BF16 ? launch_grad<__nv_bfloat16>(g, sg, s)
                                                : launch_grad<float>(g, sg, s);
    if (k < 0) return efail(MUON_ERR_UNSUPPORTED, "too many tokens and columns for one launch");
    return end_call(launches + k);
  });
}
