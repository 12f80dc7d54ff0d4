// Embedding lookup with scaling, and its gradient by sorted tokens, summed
// straight into the flat, partitioned FP32 accumulation buffer.
//
// The gradient of row v is the sum of dout over the tokens with id v.  Token
// ids repeat with a long tail (a few rows get thousands of tokens, most get
// none or one), so adding with atomics would serialise on the frequent rows
// and make the sum's order, and its bits, depend on timing.  Instead:
//   k_embed_sort   sorts (id, position) by id, stably (radix, up to 9 bits a
//                  pass, one cluster of thread blocks);
//   k_embed_sum    walks the sorted tokens in blocks: a run of equal ids goes
//                  straight to its row of accum, one that covers a block or
//                  more leaves partial sums;
//   k_embed_join   adds the partial sums of each such run in block order.
// Up to 1024 tokens k_embed_few does all of it in one launch.
// So every sum has one fixed order, and the work is balanced whatever the ids.
#include <algorithm>
#include <cmath>
#include <string>

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

constexpr int kTokens = 2;   // k_lookup: rows a thread has under way

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

// kTokens * blockDim.y tokens per block, blockDim.x threads along a row, each
// with kTokens rows under way at once.  VEC: 16 bytes of the table per thread
// and step (rows of both arrays 16-byte aligned); else eight elements,
// blockDim.x apart, so that a warp's accesses lie together.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256) k_lookup(const Lookup a) {
  const TI* src[kTokens];
  TO* dst[kTokens];
  bool on[kTokens], in[kTokens];
#pragma unroll
  for (int q = 0; q < kTokens; ++q) {
    const int64_t t = (int64_t(blockIdx.x) * kTokens + q) * blockDim.y + threadIdx.y;
    in[q] = t < a.n;
    const int id = in[q] ? lookup_id(a.ids, a.ids64, t, a.rows) : -1;
    on[q] = id >= 0;
    src[q] = static_cast<const TI*>(a.table) + int64_t(on[q] ? id : 0) * a.stride;
    dst[q] = static_cast<TO*>(a.out) + t * a.ostride;
  }
  const float scale = a.scale;
  int done = 0;
  if constexpr (VEC) {
    constexpr int N = Vec<TI>::N;
    const int nvec = a.cols / N;
#pragma unroll 2
    for (int i = threadIdx.x; i < nvec; i += blockDim.x) {
      uint4 v[kTokens];
#pragma unroll
      for (int q = 0; q < kTokens; ++q)
        v[q] = on[q] ? *reinterpret_cast<const uint4*>(src[q] + i * N) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < kTokens; ++q) {
        if (!in[q]) continue;
        float f[N];
        Vec<TI>::unpack(v[q], f);
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = on[q] ? f[k] * scale : 0.f;
        if constexpr (sizeof(TI) == sizeof(TO)) {
          __stcs(reinterpret_cast<uint4*>(dst[q] + i * N), Vec<TO>::pack(f));
        } else if constexpr (sizeof(TO) == 4) {
          float4* d = reinterpret_cast<float4*>(dst[q] + i * N);
          __stcs(d, make_float4(f[0], f[1], f[2], f[3]));
          __stcs(d + 1, make_float4(f[4], f[5], f[6], f[7]));
        } else {
          __stcs(reinterpret_cast<uint2*>(dst[q] + i * N),
                 make_uint2(Vec<TO>::pack2(f[0], f[1]), Vec<TO>::pack2(f[2], f[3])));
        }
      }
    }
    done = nvec * N;
  }
  constexpr int U = VEC ? 1 : 8;
  for (int c0 = done + threadIdx.x; c0 < a.cols; c0 += U * blockDim.x) {
    float f[kTokens][U];
#pragma unroll
    for (int q = 0; q < kTokens; ++q)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * blockDim.x;
        f[q][k] = on[q] && c < a.cols ? tok::to_float(src[q][c]) * scale : 0.f;
      }
#pragma unroll
    for (int q = 0; q < kTokens; ++q)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * blockDim.x;
        if (in[q] && c < a.cols) dst[q][c] = tok::from_float<TO>(f[q][k]);
      }
  }
}

template <typename TI, typename TO>
void launch_lookup(const Lookup& a, cudaStream_t s) {
  auto whole = [](const void* p, int64_t stride, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
  };
  const bool vec = whole(a.table, a.stride, sizeof(TI)) && whole(a.out, a.ostride, sizeof(TO)) &&
                   a.cols >= Vec<TI>::N;
  const int steps = vec ? a.cols / Vec<TI>::N : a.cols;
  const int per = vec ? 4 : 8;   // steps of a thread; a thread per step of a short row
  int tx = 1;
  while (tx < steps && (tx < 32 || (tx < 256 && tx * per < steps))) tx *= 2;
  const dim3 block(tx, std::max(1, 128 / tx));
  const unsigned grid = static_cast<unsigned>((a.n + block.y * kTokens - 1) / (block.y * kTokens));
  if (vec) k_lookup<TI, TO, true><<<grid, block, 0, s>>>(a);
  else k_lookup<TI, TO, false><<<grid, block, 0, s>>>(a);
}

// ------------------------------------------------------------------ gradient

constexpr int kSms = 152;
constexpr int kSortThreads = 512;
constexpr int kSortBlocks = 16;      // most blocks of its cluster
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortItems = 4;        // tokens a thread has in hand (8 spill at two blocks per SM)
constexpr int kSortShared = kSortWarps * kSortBins * int(sizeof(int));
constexpr int kRunMost = 32;         // sorted tokens per block of k_embed_sum, at most
constexpr int kSumX = 128;           // its threads, at most
constexpr int kJoinGroups = 8;       // k_embed_join: warps of a block, each adding every 8th partial sum
constexpr int kFew = 1024;           // tokens up to which k_embed_few is taken
constexpr int kFewX = 256;
constexpr int kFillX = 256;
constexpr int kFillBlocks = 4;       // per SM

struct Grad {
  float* accum;
  const void* dout;
  const void* ids;
  int64_t dstride;
  int ids64;
  int n, rows, cols;
  float scale;
  int overwrite;
  const int2* sorted;   // (id, position) of the tokens, by id
  float* partial;   // two rows of `cols` per block of `run` tokens
  int* crossing;    // [0]: how many runs have partial sums; then the blocks they start in
  int run;          // tokens per block
  int blocks;       // blocks of tokens
  int slabs;        // blocks of columns
};

__device__ __forceinline__ int grad_id(const Grad& g, int t) {
  return lookup_id(g.ids, g.ids64, t, g.rows);
}

// Where row `row` of the parameter lies; NULL if it is cut by partitions.
__device__ __forceinline__ float* row_of(const Grad& g, const Segments& sg, int row) {
  int64_t room;
  float* p = g.accum + sg.place(int64_t(row) * g.cols, &room);
  return room >= g.cols ? p : nullptr;
}

// A thread's columns within a block of `width` threads.  VEC: N consecutive
// ones, moved as 16 bytes; else N columns `width` apart (each access of a warp
// then covers consecutive ones).
template <int N, bool VEC>
__device__ __forceinline__ int column(int slab, int width, int x, int k) {
  return VEC ? (slab * width + x) * N + k : slab * width * N + k * width + x;
}

// One token's columns of dout as they lie in memory.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = Vec<T>::N;
  uint4 v;                     // VEC
  float f[VEC ? 1 : N];
  __device__ __forceinline__ void load(const Grad& g, int64_t t, int slab, int width, int x, bool on) {
    const T* row = static_cast<const T*>(g.dout) + t * g.dstride;
    if constexpr (VEC) {
      const int c = column<N, true>(slab, width, x, 0);
      v = make_uint4(0, 0, 0, 0);
      if (on && c < g.cols) v = *reinterpret_cast<const uint4*>(row + c);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = column<N, false>(slab, width, x, k);
        f[k] = on && c < g.cols ? tok::to_float(row[c]) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void add_to(float* acc) const {
    if constexpr (VEC) {
      float u[N];
      Vec<T>::unpack(v, u);
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += u[k];
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += f[k];
    }
  }
};

// A thread's columns of a row that lies in one piece at p.  ADD: scale * sum
// added to accum, or put in its place; else a partial sum.  All old values are
// fetched before the first store: the compiler cannot move a load over a store
// that may be to its address, and each would wait for the one before.
template <int N, bool VEC, bool ADD>
__device__ __forceinline__ void put(const Grad& g, float* p, int slab, int width, int x, const float* sum) {
  float out[N];
  const bool add = ADD && !g.overwrite;
  const float scale = ADD ? g.scale : 1.f;
  if constexpr (VEC) {
    const int c = column<N, VEC>(slab, width, x, 0);
    if (c >= g.cols) return;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const float4 o = add ? *reinterpret_cast<const float4*>(p + c + k) : make_float4(0.f, 0.f, 0.f, 0.f);
      out[k] = o.x; out[k + 1] = o.y; out[k + 2] = o.z; out[k + 3] = o.w;
    }
#pragma unroll
    for (int k = 0; k < N; k += 4)
      *reinterpret_cast<float4*>(p + c + k) =
          make_float4(out[k] + scale * sum[k], out[k + 1] + scale * sum[k + 1], out[k + 2] + scale * sum[k + 2],
                      out[k + 3] + scale * sum[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = column<N, VEC>(slab, width, x, k);
      out[k] = add && c < g.cols ? p[c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = column<N, VEC>(slab, width, x, k);
      if (c < g.cols) p[c] = out[k] + scale * sum[k];
    }
  }
}

// The same for any row of accum (p = NULL: cut by partitions, then element by
// element).  Where rows do not all start on 16 bytes (ALIGNED false) the
// columns of a VEC thread are exchanged through `stage` for ones that a warp
// stores side by side.  `lanes` threads (a block or a warp) hold a row's
// columns.
template <int N, bool VEC, bool ALIGNED, typename Sync>
__device__ __forceinline__ void put_any(const Grad& g, const Segments& sg, float* p, int id, int slab, int lanes,
                                        int x, float* sum, float* stage, Sync sync) {
  constexpr bool kDirect = !VEC || ALIGNED;
  if (kDirect && p) return put<N, VEC, true>(g, p, slab, lanes, x, sum);
#pragma unroll
  for (int k = 0; k < N; ++k) stage[column<N, VEC>(0, lanes, x, k)] = sum[k];
  sync();
  if (!kDirect && p) {
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = stage[column<N, false>(0, lanes, x, k)];
    put<N, false, true>(g, p, slab, lanes, x, sum);
  } else {
#pragma unroll 1
    for (int i = x; i < lanes * N; i += lanes) {
      const int c = slab * lanes * N + i;
      if (c >= g.cols) break;
      int64_t room;
      float* q = g.accum + sg.place(int64_t(id) * g.cols + c, &room);
      *q = (g.overwrite ? 0.f : *q) + g.scale * stage[i];
    }
  }
  sync();
}

// What k_embed_sum does after a token.
enum { kGoOn = 0, kCommit = 1, kPartial = 2 };
struct __align__(16) Step {
  float* p;
  int act;
};

// Zeros in the whole parameter (overwrite).  One resident wave of blocks, so
// that the sort is scheduled beside it and costs no time of its own.  The rows
// of tokens are written twice.  Zeroing only the other rows beside
// k_embed_sum, once the sort is done, took 55 us instead of 53 for 5003 tokens
// of a 50001 x 1001 table, and 183 instead of 202 for 16384 of a 131072 x 2048
// one, with twice the code (zeroing alone: 30 us and 165 us).
__global__ void __launch_bounds__(kFillX) k_embed_fill(float* accum, const __grid_constant__ Segments sg) {
  tok::allow_next();
  for (int i = 0; i < sg.n; ++i) {
    float* p = accum + sg.at[i];
    const int64_t n = (i + 1 < sg.n ? sg.rel[i + 1] : sg.numel) - sg.rel[i];
    const int64_t head = min(n, int64_t(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / 4));
    const int64_t quads = (n - head) / 4;
    const int64_t x = int64_t(blockIdx.x) * kFillX + threadIdx.x;
    if (x < head) p[x] = 0.f;
    for (int64_t q = x; q < quads; q += int64_t(gridDim.x) * kFillX)
      __stcs(reinterpret_cast<float4*>(p + head) + q, make_float4(0.f, 0.f, 0.f, 0.f));
    if (head + 4 * quads + x < n) p[head + 4 * quads + x] = 0.f;
  }
}

// ---- few tokens: one launch, no sort

// One block per token and block of columns.  The block of an id's first token
// finds the others (every block reads all the ids: at most 8 KB, from L2),
// adds them in order of position and writes the row; the others leave.
template <typename T, bool VEC, bool ALIGNED>
__global__ void __launch_bounds__(kFewX) k_embed_few(const Grad g, const __grid_constant__ Segments sg) {
  constexpr int N = Vec<T>::N;
  constexpr int U = 4;
  constexpr int F = 8;    // ids in flight
  __shared__ unsigned found[kFew / 32];
  __shared__ int list[kFew];
  __shared__ float stage[kFewX * N];
  const int x = threadIdx.x, lane = x % 32, width = blockDim.x;
  const int t = blockIdx.x / g.slabs, slab = blockIdx.x % g.slabs;
  const int id = grad_id(g, t);
  for (int j0 = x; j0 - lane < g.n; j0 += F * width) {
    int other[F];
#pragma unroll
    for (int k = 0; k < F; ++k)
      other[k] = j0 + k * width < g.n ? tok::load_index(g.ids, g.ids64, j0 + k * width) : -1;
#pragma unroll
    for (int k = 0; k < F; ++k) {
      const unsigned same = __ballot_sync(0xffffffffu, other[k] == id);
      if (lane == 0 && j0 + k * width < g.n) found[(j0 + k * width) / 32] = same;
    }
  }
  tok::wait_before();   // zeros first (overwrite)
  if (id < 0) return;
  __syncthreads();
  int count = 0;
  for (int w = 0; w < (g.n + 31) / 32; ++w) {
    const unsigned m = found[w];
    if (w == t / 32 ? (m & ((1u << (t % 32)) - 1)) != 0 : w < t / 32 && m != 0) return;   // not the first
    if (x < 32 && (m >> lane & 1)) list[count + __popc(m & ((1u << lane) - 1))] = w * 32 + lane;
    count += __popc(m);
  }
  __syncthreads();
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  for (int j0 = 0; j0 < count; j0 += U) {
    Piece<T, VEC> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u].load(g, list[min(j0 + u, count - 1)], slab, width, x, j0 + u < count);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u < count) p[u].add_to(acc);
  }
  put_any<N, VEC, ALIGNED>(g, sg, row_of(g, sg, id), id, slab, width, x, acc, stage, [] { __syncthreads(); });
}

// ---- more tokens: sort, sum runs, join the runs that cross blocks

struct SortArgs {
  const void* ids;
  int ids64;
  int n, rows;
  int passes, bits;      // bits per pass
  int2* sorted;          // (id, position): the result
  int2* other;
  int* crossing;
};

// Stable radix sort of (id, position) by id, tokens without a row last (key =
// rows).  One cluster; block r takes the r-th contiguous share of the tokens
// and each warp a contiguous share of that, so ranks in order of (bin, block,
// warp, token) keep the sort stable.  Per pass: each warp counts its tokens'
// bins (equal bins within a warp found by one ballot per bit, so no atomics;
// match_any took 3 times as long), the counts become offsets, and each warp
// places its tokens.  A thread fetches kSortItems tokens at a time; up to
// 32768 tokens they stay in registers, with their ranks, from the count to the
// placing.  Bound by latency (two trips to L2, two scans and a cluster barrier
// per pass): 14 us for 32768 tokens of 131072 ids, 19 by 8 blocks of twice the
// threads.
__global__ void __launch_bounds__(kSortThreads, 2) k_embed_sort(const SortArgs a) {
  extern __shared__ int count[];                  // kSortWarps x kSortBins
  __shared__ int total[kSortBlocks][kSortBins];   // every block's tokens per bin
  __shared__ int scan[kSortBins / 32];
  cg::cluster_group cl = cg::this_cluster();
  const int nb = cl.num_blocks(), rank = cl.block_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  tok::allow_next();
  if (rank == 0 && threadIdx.x == 0) a.crossing[0] = 0;
  // Every block has to have started before `total` is written from outside.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int share = (a.n + nb * kSortWarps - 1) / (nb * kSortWarps);
  const int64_t from = int64_t(rank * kSortWarps + warp) * share;
  const int lo = static_cast<int>(from < a.n ? from : a.n);
  const int hi = static_cast<int>(from + share < a.n ? from + share : a.n);
  const bool once = share <= 32 * kSortItems;
  const unsigned below = (1u << lane) - 1;
  const int mask = (1 << a.bits) - 1;
  int* mine = count + warp * kSortBins;
  int key[kSortItems], val[kSortItems], rank_in[kSortItems];
  for (int p = 0; p < a.passes; ++p) {
    const bool to0 = ((a.passes - 1 - p) & 1) == 0;
    const int2* src = to0 ? a.other : a.sorted;
    int2* dst = to0 ? a.sorted : a.other;
    auto fetch = [&](int t0) {
#pragma unroll
      for (int i = 0; i < kSortItems; ++i) {
        const int t = t0 + 32 * i + lane;
        key[i] = val[i] = 0;
        if (t < hi) {
          if (p) {
            const int2 q = src[t];
            key[i] = q.x;
            val[i] = q.y;
          } else {
            const int id = lookup_id(a.ids, a.ids64, t, a.rows);
            key[i] = id < 0 ? a.rows : id;
            val[i] = t;
          }
        }
      }
    };
    const int shift = p * a.bits;
    auto bin_of = [&](int i) { return static_cast<int>(static_cast<unsigned>(key[i]) >> shift) & mask; };
    // each token's place among its bin's, counted on from mine[]
    auto place = [&](int t0) {
#pragma unroll
      for (int i = 0; i < kSortItems; ++i) {
        if (t0 + 32 * i >= hi) break;
        const bool in = t0 + 32 * i + lane < hi;
        const int b = bin_of(i);
        unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
        for (int q = 0; q < kSortBits; ++q) {
          const unsigned set = __ballot_sync(0xffffffffu, b >> q & 1);
          same &= (b >> q & 1) ? set : ~set;
        }
        if (in) rank_in[i] = mine[b] + __popc(same & below);
        __syncwarp();
        if (in && (same & below) == 0) mine[b] += __popc(same);
        __syncwarp();
      }
    };
    fetch(lo);
    for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) count[i] = 0;
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32 * kSortItems) {
      if (t0 > lo) fetch(t0);
      place(t0);
    }
    __syncthreads();
    // per bin: the warps' offsets within the block, and the block's total
    static_assert(kSortThreads == kSortBins, "one bin per thread");
    const int bin = threadIdx.x;
    int run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = count[w * kSortBins + bin];
      count[w * kSortBins + bin] = run;
      run += c;
    }
    if (p == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
    for (int b = 0; b < kSortBlocks; ++b)
      if (b < nb) *cl.map_shared_rank(&total[rank][bin], b) = run;
    cl.sync();
    int all = 0, before = 0;
#pragma unroll
    for (int b = 0; b < kSortBlocks; ++b) {
      const int c = b < nb ? total[b][bin] : 0;
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
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) base += w < warp ? scan[w] : 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) count[w * kSortBins + bin] += base;
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32 * kSortItems) {
      if (!once) {
        fetch(t0);
        place(t0);
      }
#pragma unroll
      for (int i = 0; i < kSortItems; ++i)
        if (t0 + 32 * i + lane < hi)
          dst[rank_in[i] + (once ? mine[bin_of(i)] : 0)] = make_int2(key[i], val[i]);
    }
    if (p + 1 < a.passes) cl.sync();   // dst is complete, and total read everywhere
  }
  tok::wait_before();   // k_embed_fill beside it (overwrite): the next kernel waits for this one alone
}

// One block per `run` sorted tokens and block of columns: each thread adds its
// columns of the tokens, four of them on their way at once, and at the end of a
// run adds the sum to the row.  Bound by memory: 32768 tokens of 4096 bf16
// columns, 12000 different ones, move 660 MB in 99 us (6.6 TB/s).  Plain loads
// and stores of accum are faster than reductions at L2 (102 us against 118),
// and loading pieces into shared memory by bulk copies is not (120): more of
// them are under way, but fewer warps are there to add them.
template <typename T, bool VEC, bool ALIGNED>
__global__ void __launch_bounds__(kSumX) k_embed_sum(const Grad g, const __grid_constant__ Segments sg) {
  constexpr int N = Vec<T>::N;
  constexpr int U = 4;    // tokens in flight
  __shared__ int key[2 * kRunMost + 1], val[2 * kRunMost];   // this block's tokens and the next one's
  __shared__ int edge[3];   // ids of the token before, the one before the block before, the one after the next
  __shared__ Step step[2 * kRunMost];
  __shared__ float stage[kSumX * N];
  const int width = blockDim.x;
  tok::wait_before();
  tok::allow_next();
  const int block = blockIdx.x / g.slabs, slab = blockIdx.x % g.slabs;
  const int x = threadIdx.x;
  const int64_t t0 = int64_t(block) * g.run;
  auto key_at = [&](int64_t t) { return t >= 0 && t < g.n ? g.sorted[t].x : -1; };
  for (int i = x; i < 2 * g.run; i += width) {
    const int2 q = t0 + i < g.n ? g.sorted[t0 + i] : make_int2(-1, 0);
    key[i] = q.x;
    val[i] = q.y;
  }
  if (x >= width - 3) {
    const int e = x - (width - 3);
    edge[e] = key_at(e == 0 ? t0 - 1 : e == 1 ? t0 - g.run - 1 : t0 + 2 * g.run);
  }
  __syncthreads();
  const int n = static_cast<int>(min(int64_t(g.run), g.n - t0));
  const int id0 = key[0], id1 = key[n - 1];
  if (id0 >= g.rows) return;   // only tokens without a row from here on
  const int lane = x % 32;
  auto count = [&](int from, int id) {   // tokens of `id` among the g.run from `from` on
    return __popc(__ballot_sync(0xffffffffu, lane < g.run && key[from + min(lane, g.run - 1)] == id));
  };
  // The first run, where it comes from an earlier block: its tokens here.
  const int begun = edge[0] == id0 ? count(0, id0) : 0;
  // The last run, where it goes on into the next block: its tokens there.
  const int beyond = n == g.run && id1 < g.rows && key[g.run] == id1 ? count(g.run, id1) : 0;
  // A run over one border belongs to the block it starts in; a longer one
  // leaves a partial sum in every block (slot 1 where it starts, else 0).
  const bool begun_long = begun > 0 && (edge[1] == id0 || (begun == n && beyond > 0));
  const bool last_starts = begun < n;
  const bool last_long = beyond == g.run && edge[2] == id1;
  const int from = begun > 0 && !begun_long ? begun : 0;
  int end = last_starts && !last_long ? n + beyond : n;
  if (slab == 0 && x == 0 && last_starts && last_long) g.crossing[1 + atomicAdd(g.crossing, 1)] = block;
  while (end > from && key[end - 1] >= g.rows) --end;   // tokens without a row are the last
  // What to do after each token, worked out once per block: finding a row
  // among the partitions costs more than adding a token's columns.
  for (int j = from + x; j < end; j += width) {
    Step st{nullptr, kGoOn};
    if (j + 1 == end || key[j + 1] != key[j]) {
      const bool first_part = j < begun, last_part = j + 1 == end && last_starts && last_long;
      if (first_part || last_part) {
        st = {g.partial + (int64_t(block) * 2 + (first_part ? 0 : 1)) * g.cols, kPartial};
      } else {
        st = {row_of(g, sg, key[j]), kCommit};
      }
    }
    step[j] = st;
  }
  __syncthreads();
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  for (int j0 = from; j0 < end; j0 += U) {
    Piece<T, VEC> p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u].load(g, val[min(j0 + u, end - 1)], slab, width, x, j0 + u < end);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u >= end) break;
      p[u].add_to(acc);
      const Step st = step[j0 + u];
      if (st.act == kGoOn) continue;
      if (st.act == kPartial) put<N, VEC, false>(g, st.p, slab, width, x, acc);
      else put_any<N, VEC, ALIGNED>(g, sg, st.p, key[j0 + u], slab, width, x, acc, stage, [] { __syncthreads(); });
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = 0.f;
    }
  }
}

// Each run with partial sums: that of the block it starts in,
// then those of the blocks it goes on through.  Warp w of kJoinGroups adds
// every kJoinGroups-th of them, and the warps' sums are added in order.
template <bool VEC>
__global__ void __launch_bounds__(32 * kJoinGroups) k_embed_join(const Grad g, const __grid_constant__ Segments sg,
                                                                 int slabs) {
  constexpr int U = 4;
  constexpr int N = 4;     // columns of a lane: partial sums are FP32 whatever dout is
  __shared__ float sum[kJoinGroups][N][32];
  tok::wait_before();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t tasks = int64_t(g.crossing[0]) * slabs;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int block = g.crossing[1 + task / slabs], slab = static_cast<int>(task % slabs);
    const int id = g.sorted[block * g.run + g.run - 1].x;
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    bool more = true;
    for (int64_t i0 = warp; more; i0 += kJoinGroups * U) {   // the run's i-th block
      float f[U][N];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t b = block + i0 + u * kJoinGroups;
        on[u] = b == block || (b < g.blocks && g.sorted[b * g.run].x == id);
        const float* partial = g.partial + (b * 2 + (b == block)) * g.cols;
#pragma unroll
        for (int k = 0; k < N; ++k)
          f[u][k] = on[u] && column<N, VEC>(slab, 32, lane, k) < g.cols
                        ? partial[column<N, VEC>(slab, 32, lane, k)] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += f[u][k];
      more = on[U - 1];
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sum[warp][k][lane] = acc[k];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kJoinGroups; ++w)
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += sum[w][k][lane];
      put_any<N, VEC, VEC>(g, sg, row_of(g, sg, id), id, slab, 32, lane, acc, &sum[0][0][0], [] { __syncwarp(); });
    }
    __syncthreads();
  }
}

struct Workspace {
  size_t sorted, other, crossing, partial, bytes;
};

// Sorted tokens per block of k_embed_sum: 32, so that few runs leave partial
// sums, or down to 8 where that would leave too few blocks to fill the SMs
// (20000 tokens of 1001 bf16 columns, the whole call: 81 us at 8, 98 at 16, 158 at 32).
int run_of(int64_t n, int cols) {
  const int64_t slabs = (int64_t(cols) + 1023) / 1024;
  int run = kRunMost;
  while (run > 8 && (n + run - 1) / run * slabs < 12 * kSms) run /= 2;
  return run;
}

int64_t token_blocks(int64_t n, int cols) {
  const int run = run_of(n, cols);
  return (n + run - 1) / run;
}

Workspace workspace_of(int64_t n, int cols) {
  Workspace w{};
  if (n <= kFew) return w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~size_t(255);
    return p;
  };
  w.sorted = take(n * sizeof(int2));
  w.other = take(n * sizeof(int2));
  w.crossing = take((token_blocks(n, cols) + 1) * sizeof(int));
  w.partial = take(size_t(token_blocks(n, cols)) * 2 * cols * sizeof(float));
  w.bytes = at;
  return w;
}

cudaError_t launch_sort(const SortArgs& a, bool early, cudaStream_t s) {
  // 2048 tokens per block (4 per thread), up to a cluster of 16 blocks
  int blocks = 1;
  while (blocks < kSortBlocks && a.n > blocks * 2048) blocks *= 2;
  if (blocks > 8) {
    const cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortShared);
  if (e != cudaSuccess) return e;
  return launch(k_embed_sort, blocks, kSortThreads, blocks, early, s, kSortShared, a);
}

// Threads along a row of k_embed_few or k_embed_sum, `per` columns each: as
// many as it has columns for.
int row_threads(bool few, int cols, int per) {
  int width = few ? 64 : 32;
  while (width < (few ? kFewX : kSumX) && width * per < cols) width *= 2;
  return width;
}

// The gradient's kernels after the sort, or the one for few tokens; *launches
// counts them.
template <typename T>
cudaError_t launch_grad(const Grad& g, const Segments& sg, bool few, cudaStream_t s, int* launches) {
  constexpr int N = Vec<T>::N;
  const bool vec = reinterpret_cast<uintptr_t>(g.dout) % 16 == 0 && g.dstride * sizeof(T) % 16 == 0 &&
                   g.cols % N == 0;
  bool aligned = g.cols % 4 == 0;   // every row of accum (and of partial sums) starts on 16 bytes
  for (int i = 0; i < sg.n && aligned; ++i) aligned = (sg.at[i] - sg.rel[i]) % 4 == 0 && sg.rel[i] % 4 == 0;
  const int width = row_threads(few, g.cols, N);
  const unsigned blocks = static_cast<unsigned>((few ? g.n : g.blocks) * g.slabs);
  ++*launches;
  if (few)
    return launch(!vec ? k_embed_few<T, false, false> : aligned ? k_embed_few<T, true, true> : k_embed_few<T, true, false>,
                  blocks, width, 1, g.overwrite, s, 0, g, sg);
  cudaError_t e =
      launch(!vec ? k_embed_sum<T, false, false> : aligned ? k_embed_sum<T, true, true> : k_embed_sum<T, true, false>,
             blocks, width, 1, true, s, 0, g, sg);
  if (e != cudaSuccess) return e;
  ++*launches;
  const int slabs = static_cast<int>((int64_t(g.cols) + 127) / 128);
  const unsigned join = static_cast<unsigned>(std::min<int64_t>(int64_t(g.blocks) * slabs, 8 * kSms));
  return launch(aligned ? k_embed_join<true> : k_embed_join<false>, join, 32 * kJoinGroups, 1, true, s, 0, g, sg, slabs);
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

int end_call(int launches, cudaError_t e) {
  count_launches(launches);
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
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
    return end_call(1, cudaSuccess);
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

extern "C" int muon_embedding_grad(float* accum, int64_t accum_elems, const void* dout,
                                   int dout_dtype, int64_t dout_stride, const void* ids, int ids_type,
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
    for (int i = 0; i < sg.n; ++i)
      if (sg.at[i] + ((i + 1 < sg.n ? sg.rel[i + 1] : sg.numel) - sg.rel[i]) > accum_elems)
        return efail(MUON_ERR_INVALID, "accum_elems is less than the tables describe");
    const Workspace w = workspace_of(n_tokens, param->cols);
    if (w.bytes > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < w.bytes))
      return efail(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
    const bool few = n_tokens <= kFew;
    const int64_t blocks = token_blocks(n_tokens, param->cols);
    const int per = dout_dtype == MUON_DTYPE_BF16 ? Vec<__nv_bfloat16>::N : Vec<float>::N;
    const int slab = per * row_threads(few, param->cols, per);
    const int64_t slabs = (int64_t(param->cols) + slab - 1) / slab;
    if ((few ? n_tokens : blocks) * slabs > 0x7fffffff)
      return efail(MUON_ERR_UNSUPPORTED, "too many tokens of rows this long for one call");
    if (n_tokens == 0 && !overwrite) return MUON_OK;
    if ((rc = begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    SortArgs so{};
    so.ids = ids;
    so.ids64 = ids_type == MUON_INDEX_INT64;
    so.n = static_cast<int>(n_tokens);
    so.rows = param->rows;
    int bits = 1;
    while (bits < 32 && (int64_t(1) << bits) <= param->rows) ++bits;   // keys 0 .. rows
    so.passes = (bits + kSortBits - 1) / kSortBits;
    so.bits = (bits + so.passes - 1) / so.passes;
    so.sorted = reinterpret_cast<int2*>(base + w.sorted);
    so.other = reinterpret_cast<int2*>(base + w.other);
    so.crossing = reinterpret_cast<int*>(base + w.crossing);
    int launches = 0;
    if (overwrite) {
      const cudaError_t e = launch(k_embed_fill, unsigned(std::min<int64_t>(kFillBlocks * kSms, sg.numel / 1024 + 1)),
                                   kFillX, 1, false, s, 0, accum, sg);
      if (e != cudaSuccess) return end_call(0, e);
      ++launches;
    }
    if (n_tokens == 0) return end_call(launches, cudaSuccess);
    if (!few) {
      const cudaError_t e = launch_sort(so, overwrite, s);
      if (e != cudaSuccess) return end_call(launches, e);
      ++launches;
    }
    Grad g{};
    g.accum = accum;
    g.dout = dout;
    g.ids = ids;
    g.ids64 = so.ids64;
    g.dstride = dout_stride;
    g.n = so.n;
    g.rows = param->rows;
    g.cols = param->cols;
    g.scale = scale;
    g.overwrite = overwrite;
    g.sorted = so.sorted;
    g.partial = reinterpret_cast<float*>(base + w.partial);
    g.crossing = so.crossing;
    g.run = run_of(n_tokens, param->cols);
    g.blocks = static_cast<int>(blocks);
    g.slabs = static_cast<int>(slabs);
    const cudaError_t e = dout_dtype == MUON_DTYPE_BF16
                              ? launch_grad<__nv_bfloat16>(g, sg, few, s, &launches)
                              : launch_grad<float>(g, sg, few, s, &launches);
    return end_call(launches, e);
  });
}
