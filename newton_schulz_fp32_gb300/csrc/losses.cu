// Log-probabilities of target tokens, the clipped policy loss with a KL term
// and the preference loss of paired log ratios, with the gradient of the
// logits.
//
// With z a row of logits, s the scale, y its target, m = max z:
//     e_v  = exp(s (z_v - m)),   S = sum_v e_v
//     logp = s (z_y - m) - log S
// and for a loss that depends on the row through logp alone,
//     dz_v = s c (1[v = y] - e_v / S),   c = d loss / d logp.
// (Any m near the maximum serves.)  Subtracting m before scaling keeps rows of
// the type's lowest value and of minus infinities right without a branch: m
// starts at the lowest finite FP32 value, so minus infinity always gives e = 0,
// and a row of nothing else has S = 0 and logp NaN.
//
// Maxima, sums and e are FP32 whatever the logits' type; sums over tokens are
// kept as two FP32 values, in a fixed order.
//
// Which kernel takes a row is a matter of its size, and of whether its gradient
// is written (launch_rows_of):
//   k_held    a cluster of blocks holds the row in shared memory: read once,
//             gradient and all.  Bound by memory: 8192 rows of 131072 bf16, 5%
//             of them masked, with their gradient 660 us the whole call, 6.35
//             TB/s of reads and writes.
//   k_rows    one block streams the row; for many rows without a gradient
//             (8192 of 131072 bf16, 10% left out: 265 us, 7.3 TB/s) and for rows too long to
//             be held, whose gradient takes a second pass.
//   k_given   the gradient from statistics taken before: the preference loss
//             needs all of a pair's rows before any of their gradients, so it
//             reads the logits twice (statistics 224 us, gradient 555 us for
//             8192 rows of 131072 bf16, both at the copy rate).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <string>

#include <cooperative_groups.h>

#include "tc_common.cuh"
#include "token_ops.cuh"

namespace muon {
namespace {

namespace cg = cooperative_groups;
using tok::Vec;

__device__ int g_losses_err;

constexpr int kRowLoads = 8;         // k_rows: 16-byte loads of a thread in flight
constexpr int kSumThreads = 1024;    // k_policy_sum
constexpr int kHeldThreads = 256;    // k_held: most threads of a block,
constexpr int kHeldBlocks = 6;       // blocks per SM,
constexpr int kHeldLoads = 2;        // vectors a thread adds at once,
constexpr int kHeldVecs = 2048;      // 16-byte vectors of a block before a row takes more blocks,
constexpr int kHeldMost = 13824;     // and at most (216 KB)
constexpr int kHeldRow = 8192;       // bytes of a row up to which it is held without a gradient too
constexpr int kSms = 152;
constexpr int kPairThreads = 1024;   // k_pairs: most threads of a pair
constexpr int kGivenThreads = 256;   // k_given: most threads of a block
constexpr int kGivenVecs = 8;        // 16-byte vectors of its threads

int lfail(int code, const std::string& msg) {
  set_last_error(msg.c_str());
  return code;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What every row kernel takes.
struct Rows {
  const void* logits;
  int64_t stride;
  int64_t n;
  int vocab;
  int targets64;
  const void* targets;
  float scale;     // s
  float scale2;    // s log2(e): exp(s x) = 2^(scale2 x)
  float first, second;   // the same as a product
  float slack;     // 8 / s
  float* logp;
  void* dlogits;   // NULL: no gradient
  int64_t dstride;
};

// The policy loss's inputs of one token.
struct Policy {
  const float* advantages;
  const float* weights;
  const float* old_logp;
  const float* ref_logp;
  float clip_low, clip_high, kl_coef;
};

struct Token {
  float a, w, old, ref;
};

struct PolicyTerms {
  float term, kl;
  float coef;   // d (term + kl_coef kl) / d logp
  bool cut;
};

__device__ __forceinline__ Token load_token(const Policy& p, int64_t t) {
  return {p.advantages[t], p.weights[t], p.old_logp ? p.old_logp[t] : 0.f,
          p.ref_logp ? p.ref_logp[t] : 0.f};
}

__device__ __forceinline__ PolicyTerms policy_terms(const Token& k, const Policy& p, float logp) {
  PolicyTerms o;
  const float r = p.old_logp ? expf(logp - k.old) : (logp == logp ? 1.f : logp);
  const float free = k.a == 0.f && r > FLT_MAX ? 0.f : r * k.a;   // an r past the range is a number all the same
  const float held = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * k.a;
  o.cut = free > held;
  o.term = o.cut ? -held : -free;
  o.coef = o.cut ? 0.f : -free;
  o.kl = 0.f;
  if (p.ref_logp) {
    const float q = k.ref - logp;
    const float g = expm1f(q);
    o.kl = q > FLT_MAX ? q : g - q;
    if (p.kl_coef != 0.f) o.coef -= p.kl_coef * g;   // 0 times infinity would spoil the gradient
  }
  return o;
}

// The target of row t, or -1 where the row takes no part.
__device__ __forceinline__ int row_target(const Rows& a, int64_t t) {
  const int y = tok::load_index(a.targets, a.targets64, t);
  if (y >= a.vocab) {
    if (threadIdx.x == 0) atomicCAS(&g_losses_err, 0, kErrIndex);
    return -1;
  }
  return y < 0 ? -1 : y;
}

// Joins the softmax statistics (m, s) of two parts of a row.  Three joins, one
// in another, end in log S: by expf, since the errors of ex2.approx lie on one
// side (2e-8 on average).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float scale) {
  const float top = fmaxf(m, m2);
  s = s * expf((m - top) * scale) + s2 * expf((m2 - top) * scale);
  m = top;
}

__device__ __forceinline__ void warp_join(float& m, float& s, float scale) {
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  s *= expf((m - top) * scale);
  m = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}

// A row's elements as `head` single ones up to a 16-byte boundary, `nvec`
// 16-byte vectors, and the rest.
template <typename T>
struct RowShape {
  int head, nvec, tail0;   // tail0: the first element after the vectors
  __device__ __forceinline__ RowShape(const T* p, int vocab) {
    head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int(sizeof(T));
    if (head > vocab) head = vocab;
    nvec = (vocab - head) / Vec<T>::N;
    tail0 = head + nvec * Vec<T>::N;
  }
  // This thread's element before or after the vectors, or -1: fewer than 8 of
  // either.  (A vocabulary may end at the last int: tail0 + a thread's number
  // need not fit in one.)
  __device__ __forceinline__ int single(int vocab) const {
    const int k = int(threadIdx.x) - 8;
    return int(threadIdx.x) < head ? int(threadIdx.x) : k >= 0 && k < vocab - tail0 ? tail0 + k : -1;
  }
};

template <typename T>
__device__ __forceinline__ float vec_max(const uint4& v) {
  if constexpr (sizeof(T) == 2) {
    auto pair = [](uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); };
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

// Two FP32 lanes per instruction.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// e of 16 bytes of logits, in pairs: 2^((z - m) scale2).
template <typename T>
__device__ __forceinline__ void vec_exp(const uint4& v, uint64_t minus_m, uint64_t scale2,
                                        uint64_t (&e)[Vec<T>::N / 2]) {
  float f[Vec<T>::N];
  Vec<T>::unpack(v, f);
#pragma unroll
  for (int j = 0; j < Vec<T>::N / 2; ++j) {
    float lo, hi;
    split(mul2(add2(two(f[2 * j], f[2 * j + 1]), minus_m), scale2), lo, hi);
    e[j] = two(ex2(lo), ex2(hi));
  }
}

// A thread's running sum of e = exp(s (z - m)).  m is not its maximum but one
// that it reached: it moves when a logit is past it by more than 8 / s, which
// FP32 has room for, so that most threads take it from their first vector and
// never rescale (a warp whose lanes follow the maximum rescales at nearly every
// vector: 279 us became 324 with rescales exact enough to be worth having).
// Any m serves in the formulas above.  The exponents are formed in two products
// (Rows::first, second), see make_rows.
template <typename T>
struct Softmax {
  float m = -FLT_MAX;
  uint64_t s[2] = {0, 0};
  template <int U>
  __device__ __forceinline__ void add(const uint4 (&v)[U], const Rows& a) {
    float top = vec_max<T>(v[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) top = fmaxf(top, vec_max<T>(v[u]));
    if (top - m > a.slack) {
      const float k = expf((m - top) * a.scale);
      s[0] = mul2(s[0], two(k, k));
      s[1] = mul2(s[1], two(k, k));
      m = top;
    }
    const uint64_t mm = two(-m, -m), p = two(a.first, a.first), q = two(a.second, a.second);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[Vec<T>::N];
      Vec<T>::unpack(v[u], f);
#pragma unroll
      for (int j = 0; j < Vec<T>::N / 2; ++j) {
        float lo, hi;
        split(mul2(mul2(add2(two(f[2 * j], f[2 * j + 1]), mm), p), q), lo, hi);
        s[j & 1] = add2(s[j & 1], two(ex2(lo), ex2(hi)));
      }
    }
  }
  __device__ __forceinline__ float sum() const {
    float lo, hi;
    split(add2(s[0], s[1]), lo, hi);
    return lo + hi;
  }
};

enum RowMode {
  kLogp = 0,     // logp
  kStats = 1,    // logp and (m, 1/S) for k_given
  kPolicy = 2    // logp and the policy loss's gradient
};

struct Extra {
  Policy policy;
  float2* stats;      // kStats: (m, 1/S) per row
  float* coef;        // kStats: c per row, zero here (k_pairs writes it)
  float* logp_lo;     // kStats: log-probability - logp
};

// What a row's log-probability loses when it is rounded to FP32.  Margins are
// differences of sums of hundreds of them, so the preference loss adds it
// back: one FP64 logarithm per row, by one thread.
__device__ __noinline__ float logp_rest(float scale, float zy, float m, float s, float logp) {
  const double v = double(scale) * (double(zy) - double(m)) - log(double(s)) - double(logp);
  return fabs(v) <= 1.0 ? static_cast<float>(v) : 0.f;   // 0 beside infinities and NaN
}

// Writes one row's gradient: g = s c, e scaled by -g / S, plus g at y.
template <typename T>
__device__ __forceinline__ void write_grad(const Rows& a, const T* row, T* drow, int y, float m,
                                           float inv, float g) {
  constexpr int N = Vec<T>::N;
  const RowShape<T> sh(row, a.vocab);
  const float ga = -g * inv;
  auto one = [&](int v, float z) {
    float d = ga * ex2((z - m) * a.scale2);
    return v == y ? d + g : d;
  };
  const bool aligned =
      ((reinterpret_cast<uintptr_t>(drow) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
  const int u = sh.single(a.vocab);
  if (u >= 0) drow[u] = tok::from_float<T>(one(u, tok::to_float(row[u])));
  for (int i = threadIdx.x; i < sh.nvec; i += blockDim.x) {
    const int v0 = sh.head + i * N;
    float f[N];
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + v0), f);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = one(v0 + k, f[k]);
    if (aligned) {
      *reinterpret_cast<uint4*>(drow + v0) = Vec<T>::pack(f);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) drow[v0 + k] = tok::from_float<T>(f[k]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void write_zeros(const Rows& a, T* drow) {
  const RowShape<T> sh(drow, a.vocab);
  const int u = sh.single(a.vocab);
  if (u >= 0) drow[u] = tok::from_float<T>(0.f);
  for (int i = threadIdx.x; i < sh.nvec; i += blockDim.x)
    *reinterpret_cast<uint4*>(drow + sh.head + i * Vec<T>::N) = make_uint4(0, 0, 0, 0);
}

// One block of W threads per row: a pass for (m, S), kRowLoads loads per thread
// in flight, and for the gradient a second one that reads the row again.  The second pass
// comes from L2 (the rows in flight are a few tens of MB) but is not free: the
// SMs' traffic with L2 is the bound then (8192 rows of 131072 bf16 with their
// gradient: 887 us).
template <typename T, int MODE, int W>
__global__ void __launch_bounds__(W) k_rows(const Rows a, const Extra x) {
  constexpr int N = Vec<T>::N;
  __shared__ float sm[W / 32], ss[W / 32];
  tok::allow_next();
  const int64_t t = blockIdx.x;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
  T* drow = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
  const int y = row_target(a, t);
  if (y < 0 || (MODE == kPolicy && x.policy.weights[t] == 0.f)) {
    if (threadIdx.x == 0) {
      a.logp[t] = 0.f;
      if (MODE == kStats) {
        x.coef[t] = 0.f;
        x.logp_lo[t] = 0.f;
      }
    }
    if (MODE == kPolicy && drow) write_zeros<T>(a, drow);
    return;
  }
  const RowShape<T> sh(row, a.vocab);
  Softmax<T> part;
  int i = threadIdx.x;
  for (; i + (kRowLoads - 1) * W < sh.nvec; i += kRowLoads * W) {
    uint4 v[kRowLoads];
#pragma unroll
    for (int u = 0; u < kRowLoads; ++u)
      v[u] = *reinterpret_cast<const uint4*>(row + sh.head + (i + u * W) * N);
    part.add(v, a);
  }
  for (; i < sh.nvec; i += W) {
    const uint4 v[1] = {*reinterpret_cast<const uint4*>(row + sh.head + i * N)};
    part.add(v, a);
  }
  float m = part.m, s = part.sum();
  if (threadIdx.x < sh.head) join(m, s, tok::to_float(row[threadIdx.x]), 1.f, a.scale);
  if (int(threadIdx.x) < a.vocab - sh.tail0) join(m, s, tok::to_float(row[sh.tail0 + threadIdx.x]), 1.f, a.scale);
  const float zy = tok::to_float(row[y]);
  warp_join(m, s, a.scale);
  if (threadIdx.x % 32 == 0) {
    sm[threadIdx.x / 32] = m;
    ss[threadIdx.x / 32] = s;
  }
  __syncthreads();
  m = sm[0];
  s = ss[0];
  for (int w = 1; w < W / 32; ++w) join(m, s, sm[w], ss[w], a.scale);
  const float logp = a.scale * (zy - m) - logf(s);
  if (threadIdx.x == 0) {
    a.logp[t] = logp;
    if (MODE == kStats) {
      x.stats[t] = make_float2(m, 1.f / s);
      x.coef[t] = 0.f;
      x.logp_lo[t] = logp_rest(a.scale, zy, m, s, logp);
    }
  }
  if (MODE == kPolicy && drow) {
    const float c = x.policy.weights[t] * policy_terms(load_token(x.policy, t), x.policy, logp).coef;
    if (c == 0.f) return write_zeros<T>(a, drow);
    write_grad<T>(a, row, drow, y, m, 1.f / s, a.scale * c);
  }
}

// The sum over the cluster's threads, valid in thread 0 of its first block.
// sh: one entry per warp and quantity; every block of the cluster calls it.
template <int NT, int Q>
__device__ __forceinline__ void cluster_sum(tok::Two (&v)[Q], tok::Two (*sh)[NT / 32]) {
  cg::cluster_group cl = cg::this_cluster();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    v[q].warp_sum();
    if (lane == 0) sh[q][warp] = v[q];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      v[q] = lane < NT / 32 ? sh[q][lane] : tok::Two();
      v[q].warp_sum();
    }
    __syncwarp();
    if (lane == 0)
#pragma unroll
      for (int q = 0; q < Q; ++q) sh[q][0] = v[q];
  }
  cl.sync();
  if (cl.block_rank() == 0 && threadIdx.x == 0)
    for (int b = 1; b < int(cl.num_blocks()); ++b)
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q].add(*cl.map_shared_rank(&sh[q][0], b));
  cl.sync();   // no block leaves while its sums are read
}

// The policy loss's statistics from the tokens' logp.  One cluster: up to
// 8 x 1024 tokens at once.
__global__ void __launch_bounds__(kSumThreads) k_policy_sum(const Rows a, const Policy p,
                                                            float* stats) {
  __shared__ tok::Two sh[3][kSumThreads / 32];
  tok::Two v[3];   // term, kl, cut
  tok::wait_before();
  for (int64_t t = blockIdx.x * kSumThreads + threadIdx.x; t < a.n; t += int64_t(gridDim.x) * kSumThreads) {
    const int y = tok::load_index(a.targets, a.targets64, t);
    const float w = p.weights[t];
    if (y < 0 || y >= a.vocab || w == 0.f) continue;
    const PolicyTerms o = policy_terms(load_token(p, t), p, a.logp[t]);
    v[0].add(w * o.term);
    v[1].add(w * o.kl);
    if (o.cut) v[2].add(w);
  }
  cluster_sum<kSumThreads, 3>(v, sh);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const float term = v[0].value(), kl = v[1].value();
    if (p.kl_coef != 0.f) {
      v[0].add(p.kl_coef * v[1].hi);
      v[0].lo += p.kl_coef * v[1].lo;
    }
    stats[0] = v[0].value();
    stats[1] = term;
    stats[2] = kl;
    stats[3] = v[2].value();
  }
}

struct Pairs {
  const void* offsets;
  int offsets64;
  int n;
  const float* ref_logp;
  const float* weights;
  float beta, smoothing;
  const float* logp_lo;   // what the tokens' logp lost when it was rounded
  float* margins;
  float* coef;            // c per token; NULL: no gradient
};

// log(1 + exp(x)) and 1 / (1 + exp(-x)) without overflow.
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return x >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
}

__device__ __forceinline__ void sequence(const Rows& a, const Pairs& q, int i, int64_t& b, int64_t& e) {
  auto at = [&](int k) -> int64_t {
    return q.offsets64 ? reinterpret_cast<const int64_t*>(q.offsets)[k]
                       : reinterpret_cast<const int32_t*>(q.offsets)[k];
  };
  b = at(i);
  e = at(i + 1);
  if (b < 0 || e < b || e > a.n) {
    if (threadIdx.x == 0) atomicCAS(&g_losses_err, 0, kErrOffsets);
    b = b < 0 ? 0 : b > a.n ? a.n : b;
    e = e < b ? b : e > a.n ? a.n : e;
  }
}

// One block per pair: the two sequences' sums, the margin, and c of every
// token of the pair.
__global__ void __launch_bounds__(kPairThreads) k_pairs(const Rows a, const Pairs q) {
  constexpr int U = 4;   // tokens of a thread under way
  __shared__ tok::Two sh[2][kPairThreads / 32];
  __shared__ float grad;
  const int width = blockDim.x;
  tok::wait_before();
  tok::allow_next();
  tok::Two sum[2];
  int64_t b[2], e[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    sequence(a, q, blockIdx.x + j * q.n, b[j], e[j]);
    for (int64_t t0 = b[j] + threadIdx.x; t0 < e[j]; t0 += U * width) {
      float hi[U], lo[U], ref[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * width;
        const int y = t < e[j] ? tok::load_index(a.targets, a.targets64, t) : -1;
        const bool on = y >= 0 && y < a.vocab;
        hi[u] = on ? a.logp[t] : 0.f;
        lo[u] = on ? q.logp_lo[t] : 0.f;
        ref[u] = on && q.ref_logp ? q.ref_logp[t] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        sum[j].add(hi[u]);
        sum[j].lo += lo[u];
        sum[j].add(-ref[u]);
      }
    }
    sum[j].warp_sum();
    if (threadIdx.x % 32 == 0) sh[j][threadIdx.x / 32] = sum[j];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      sum[j] = sh[j][0];
      for (int w = 1; w < width / 32; ++w) sum[j].add(sh[j][w]);
    }
    float h;
    if (fabsf(sum[0].hi) <= FLT_MAX && fabsf(sum[1].hi) <= FLT_MAX) {
      sum[0].add(-sum[1].hi);
      sum[0].lo -= sum[1].lo;
      h = q.beta * sum[0].value();
    } else {
      h = q.beta * (sum[0].hi - sum[1].hi);
    }
    q.margins[blockIdx.x] = h;
    const float w = q.weights ? q.weights[blockIdx.x] : 1.f / q.n;
    // d loss / d h = sigmoid(h) - (1 - smoothing), written so that neither term cancels
    const float dh = q.smoothing * sigmoid(h) - (1.f - q.smoothing) * sigmoid(-h);
    grad = w == 0.f ? 0.f : w * q.beta * dh;
  }
  if (!q.coef) return;
  __syncthreads();
  const float g = grad;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    for (int64_t t = b[j] + threadIdx.x; t < e[j]; t += width) q.coef[t] = j ? -g : g;
}

// The preference loss's statistics from the margins, by the block's first
// warp: one order of sums, whatever block calls it.
__device__ __forceinline__ void pair_sum(const Pairs& q, float* stats) {
  if (threadIdx.x >= 32) return;
  tok::Two v[4];   // loss, margin, won, weight
  for (int i = threadIdx.x; i < q.n; i += 32) {
    const float w = q.weights ? q.weights[i] : 1.f;
    if (w == 0.f) continue;
    const float h = q.margins[i];
    float l = 0.f;
    if (q.smoothing < 1.f) l += (1.f - q.smoothing) * softplus(-h);
    if (q.smoothing > 0.f) l += q.smoothing * softplus(h);
    v[0].add(w * l);
    v[1].add(w * h);
    if (h > 0.f) v[2].add(w);
    v[3].add(w);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k].warp_sum();
    if (threadIdx.x == 0) stats[k] = v[k].value() / (q.weights || q.n == 0 ? 1.f : float(q.n));
  }
}

__global__ void __launch_bounds__(32) k_pair_sum(const Pairs q, float* stats) {
  tok::wait_before();
  pair_sum(q, stats);
}

// The gradient from (m, 1/S) and c of every row.  Block 0 sums the
// statistics; the others take kGivenVecs vectors per thread of a row each, the
// last rows first: the statistics pass read those last, so some are in L2 yet.
template <typename T, int W>
__global__ void __launch_bounds__(W) k_given(const Rows a, const Extra x, const Pairs q,
                                                         float* stats, int slices) {
  constexpr int N = Vec<T>::N;
  constexpr int NV = kGivenVecs;
  tok::wait_before();
  if (blockIdx.x == 0) return pair_sum(q, stats);
  const unsigned task = gridDim.x - 1 - blockIdx.x;
  const int64_t t = task / slices;
  const int slice = task % slices;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
  T* drow = static_cast<T*>(a.dlogits) + t * a.dstride;
  const int y = row_target(a, t);
  const float c = x.coef[t];
  const bool on = y >= 0 && c != 0.f;   // else zeros, and the row is not read
  const float2 st = x.stats[t];
  const float g = a.scale * c, ga = -g * st.y, m = st.x;
  const bool aligned =
      ((reinterpret_cast<uintptr_t>(drow) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
  const RowShape<T> sh(on || aligned ? row : drow, a.vocab);
  const int i0 = slice * NV * W + threadIdx.x;
  uint4 v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    v[k] = make_uint4(0, 0, 0, 0);
    const int i = i0 + k * W;
    if (on && i < sh.nvec) v[k] = __ldcs(reinterpret_cast<const uint4*>(row + sh.head + i * N));
  }
  auto one = [&](int u, float z) {
    const float d = ga * ex2((z - m) * a.scale2);
    return !on ? 0.f : u == y ? d + g : d;
  };
  if (slice == 0) {   // the elements before and after the vectors
    // RowShape::single, written out: 48 registers and five blocks per SM, 56 and four by the call
    const int k = int(threadIdx.x) - 8;
    const bool before = int(threadIdx.x) < sh.head;
    if (before || (k >= 0 && k < a.vocab - sh.tail0)) {
      const int u = before ? int(threadIdx.x) : sh.tail0 + k;
      drow[u] = tok::from_float<T>(one(u, on ? tok::to_float(row[u]) : 0.f));
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * W;
    if (i >= sh.nvec) break;
    const int v0 = sh.head + i * N;
    float f[N];
    Vec<T>::unpack(v[k], f);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = one(v0 + j, f[j]);
    if (aligned || !on) {
      __stcs(reinterpret_cast<uint4*>(drow + v0), Vec<T>::pack(f));
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) drow[v0 + j] = tok::from_float<T>(f[j]);
    }
  }
}

template <typename T>
cudaError_t launch_given(const Rows& a, const Extra& x, const Pairs& q, float* stats, int width, int slices,
                         cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.n * slices + 1);
  auto go = [&](auto kernel) { return launch(kernel, grid, width, 1, true, s, 0, a, x, q, stats, slices); };
  return width == 32 ? go(k_given<T, 32>) : width == 64 ? go(k_given<T, 64>)
         : width == 128 ? go(k_given<T, 128>) : go(k_given<T, 256>);
}

int sum_blocks(int64_t n) {
  int blocks = 1;
  while (blocks < 8 && n > blocks * int64_t(kSumThreads)) blocks *= 2;
  return blocks;
}

// ---- a row held on chip

// The blocks of a cluster have started (arrive, then wait before the first
// write to another's shared memory).  Relaxed: it orders no data.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// Sends (m, s) and z to `slot` in block `rank`, counted in bytes on its
// barrier there.  A release barrier of the whole cluster instead makes every warp wait
// for its own earlier memory operations: 23% longer for 8192 rows of 131072
// bf16 with their gradient.
__device__ __forceinline__ void send(uint32_t slot, uint32_t bar, int rank, float m, float s, float z) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          tc::mapa_shared(slot, rank)),
      "r"(__float_as_uint(m)), "r"(__float_as_uint(s)), "r"(__float_as_uint(z)), "r"(0),
      "r"(tc::mapa_shared(bar, rank))
      : "memory");
}

// After a wait that ran out, once more and for longer than any other block's
// waits before its stores: no copy or remote store may find its block gone.
__device__ __noinline__ void wait_again(uint32_t bar) {
  const unsigned long long t0 = tc::globaltimer();
  while (!tc::mbar_try_wait(bar, 0) && tc::globaltimer() - t0 < 2 * tc::kTimeoutNs) {
  }
}

// Zeros in vectors [v0, v1) of a row, and around them in block 0.
template <typename T>
__device__ __forceinline__ void zero_share(const Rows& a, T* drow, int v0, int per_block, int rank) {
  const RowShape<T> sh(drow, a.vocab);
  const int u = rank == 0 ? sh.single(a.vocab) : -1;
  if (u >= 0) drow[u] = tok::from_float<T>(0.f);
  const int v1 = min(sh.nvec, v0 + per_block);
  for (int i = v0 + threadIdx.x; i < v1; i += blockDim.x)
    __stcs(reinterpret_cast<uint4*>(drow + sh.head + i * Vec<T>::N), make_uint4(0, 0, 0, 0));
}

// A row held on chip: one cluster of blocks per row, each with `per_block` of
// the row's 16-byte vectors in shared memory, brought there by a bulk copy.
// The row is read from memory exactly once, also where its gradient is
// written, and a row is spread over up to eight SMs, so a call with few rows is
// short (one row of 131072 bf16: 3.3 us, 7.3 by one block).  Blocks of
// different rows on one SM overlap one row's loads with another's arithmetic
// and writes; holding rows in shared memory leaves registers for six of them
// (in registers, four: 18% longer for 8192 rows of 131072 bf16 with their
// gradient).  Instructions come next: arithmetic on pairs of values.
template <typename T, int MODE>
__global__ void __launch_bounds__(kHeldThreads, kHeldBlocks) k_held(const Rows a, const Extra x, int per_block) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 held[];
  __shared__ __align__(8) uint64_t full, joined;
  __shared__ float2 warp_part[kHeldThreads / 32];
  __shared__ __align__(16) float4 part[8];   // (m, s, the target's logit or minus infinity) of every block
  __shared__ float2 out;         // (-g / S, g)
  __shared__ float out_m;
  __shared__ int stopped;
  tok::allow_next();
  cg::cluster_group cl = cg::this_cluster();
  const int c = cl.num_blocks(), rank = cl.block_rank();
  const int64_t t = blockIdx.x / unsigned(c);
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
  T* drow = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int base = rank * per_block;
  const int y = row_target(a, t);
  Token tk{};
  if (MODE == kPolicy) tk = load_token(x.policy, t);
  if (y < 0 || (MODE == kPolicy && tk.w == 0.f)) {   // the same for the whole cluster
    if (rank == 0 && threadIdx.x == 0) {
      a.logp[t] = 0.f;
      if (MODE == kStats) {
        x.coef[t] = 0.f;
        x.logp_lo[t] = 0.f;
      }
    }
    if (MODE == kPolicy && drow) zero_share<T>(a, drow, base, per_block, rank);
    return;
  }
  const RowShape<T> sh(row, a.vocab);
  const int mine = max(0, min(per_block, sh.nvec - base));   // this block's vectors
  if (threadIdx.x == 0) {
    stopped = 0;
    tc::mbar_init(tc::smem_u32(&full), 1);
    tc::mbar_init(tc::smem_u32(&joined), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (c > 1) tc::mbar_expect_tx(tc::smem_u32(&joined), c * 16);
    tc::mbar_expect_tx(tc::smem_u32(&full), mine * 16);
    if (mine > 0)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              tc::smem_u32(held)),
          "l"(row + sh.head + int64_t(base) * N), "r"(mine * 16), "r"(tc::smem_u32(&full))
          : "memory");
  }
  __syncthreads();
  if (c > 1) cluster_arrive();   // waited for before the first write to another block
  // elements before and after the vectors: one per thread of the first block
  const int single = rank == 0 ? sh.single(a.vocab) : -1;
  const float zs = single >= 0 ? tok::to_float(row[single]) : -INFINITY;
  // The target's logit is read by the block that writes its gradient alone, and
  // goes to the others with (m, s): the sums' exchange orders no other load, so
  // another block's could come after that write where the gradient replaces
  // the logits.
  const bool ours = y < sh.head || y >= sh.tail0 ? rank == 0 : unsigned((y - sh.head) / N - base) < unsigned(mine);
  float zy = warp == 0 && ours ? tok::to_float(row[y]) : -INFINITY;
  Softmax<T> share;
  tc::mbar_wait(tc::smem_u32(&full), 0, &stopped, &g_losses_err, 1);
  int at = threadIdx.x;
  for (; at + (kHeldLoads - 1) * int(blockDim.x) < mine; at += kHeldLoads * blockDim.x) {
    uint4 v[kHeldLoads];
#pragma unroll
    for (int u = 0; u < kHeldLoads; ++u) v[u] = held[at + u * blockDim.x];
    share.add(v, a);
  }
  for (; at < mine; at += blockDim.x) {
    const uint4 v[1] = {held[at]};
    share.add(v, a);
  }
  float m = share.m, s = share.sum();
  if (single >= 0) join(m, s, zs, 1.f, a.scale);
  warp_join(m, s, a.scale);
  if (lane == 0) warp_part[warp] = make_float2(m, s);
  __syncthreads();
  if (warp == 0) {
    const bool on = lane < int(blockDim.x) / 32;
    m = on ? warp_part[lane].x : -FLT_MAX;
    s = on ? warp_part[lane].y : 0.f;
    warp_join(m, s, a.scale);
  }
  if (c > 1) {
    cluster_wait();
    if (warp == 0) {
      if (lane < c) send(tc::smem_u32(&part[rank]), tc::smem_u32(&joined), lane, m, s, zy);
      if (!tc::mbar_wait_cluster(tc::smem_u32(&joined), 0, &stopped, &g_losses_err, 4))
        wait_again(tc::smem_u32(&joined));
      const float4 p = lane < c ? part[lane] : make_float4(-FLT_MAX, 0.f, -INFINITY, 0.f);
      m = p.x;
      s = p.y;
      zy = p.z;   // a NaN is lost here, but is in s as well
      warp_join(m, s, a.scale);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) zy = fmaxf(zy, __shfl_xor_sync(0xffffffffu, zy, o));
    }
  }
  if (warp == 0 && lane == 0) {
    const float logp = a.scale * (zy - m) - logf(s);
    if (rank == 0) {
      a.logp[t] = logp;
      if (MODE == kStats) {
        x.stats[t] = make_float2(m, 1.f / s);
        x.coef[t] = 0.f;
        x.logp_lo[t] = logp_rest(a.scale, zy, m, s, logp);
      }
    }
    if (MODE == kPolicy) {
      const float g = a.scale * (tk.w * policy_terms(tk, x.policy, logp).coef);
      out = make_float2(-g / s, g);
      out_m = m;
    }
  }
  __syncthreads();   // no thread leaves while the others' values are still on their way here
  if (stopped) return wait_again(tc::smem_u32(&full));
  if (MODE != kPolicy || !drow) return;
  const float ga = out.x, g = out.y;
  m = out_m;
  if (g == 0.f) return zero_share<T>(a, drow, base, per_block, rank);
  if (single >= 0) {
    const float d = ga * ex2((zs - m) * a.scale2);
    drow[single] = tok::from_float<T>(single == y ? d + g : d);
  }
  const bool aligned =
      ((reinterpret_cast<uintptr_t>(drow) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
  const uint64_t mm = two(-m, -m), ss = two(a.scale2, a.scale2), gg = two(ga, ga);
#pragma unroll 2
  for (int i = threadIdx.x; i < mine; i += blockDim.x) {
    const int v0 = sh.head + (base + i) * N;
    float f[N];
    uint64_t e[N / 2];
    vec_exp<T>(held[i], mm, ss, e);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) split(mul2(e[j], gg), f[2 * j], f[2 * j + 1]);
    if (unsigned(y - v0) < unsigned(N)) {
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] += y - v0 == j ? g : 0.f;
    }
    if (aligned) {
      __stcs(reinterpret_cast<uint4*>(drow + v0), Vec<T>::pack(f));
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) drow[v0 + j] = tok::from_float<T>(f[j]);
    }
  }
}

// How a row is held: c blocks of `threads` with `vecs` vectors each; c = 0:
// it does not fit.
struct Hold {
  int c, vecs, threads;
};

Hold hold_of(int64_t n, int vocab, int per_vec) {
  const int nvec = std::max(1, vocab / per_vec);
  int c = 1;
  while (c < 8 && (nvec + c - 1) / c > kHeldVecs) c *= 2;
  while (c < 8 && n * c * 2 <= kSms && nvec / c > 64) c *= 2;   // few rows: use the SMs that there are
  const int vecs = (nvec + c - 1) / c;
  if (vecs > kHeldMost) return {0, 0, 0};
  // Few rows: as many threads as help.  Many rows: 16 vectors per thread, so that
  // an SM has blocks of more rows to turn to (16384 rows of 8192 bf16: 41 us, 57
  // at 4 vectors); 8 where shared memory limits the blocks (8192 rows of
  // 131072 bf16 with their gradient: 6% longer at 16).
  const int per_thread = n * c < 4 * kSms ? 2 : vecs * 7 > kHeldMost ? 8 : 16;
  int threads = 32;
  while (threads < kHeldThreads && threads * per_thread < vecs) threads *= 2;
  return {c, vecs, threads};
}

template <typename T, int MODE>
cudaError_t launch_held(const Rows& a, const Extra& x, Hold h, cudaStream_t s) {
  const int bytes = h.vecs * 16;
  if (bytes > 40 * 1024) {   // beyond what a launch may ask without it
    const cudaError_t e = cudaFuncSetAttribute(k_held<T, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kHeldMost * 16);
    if (e != cudaSuccess) return e;
  }
  return launch(k_held<T, MODE>, static_cast<unsigned>(a.n * h.c), h.threads, h.c, false, s, bytes, a, x, h.vecs);
}

template <typename T, int MODE>
cudaError_t launch_rows_of(const Rows& a, const Extra& x, cudaStream_t s) {
  const Hold h = hold_of(a.n, a.vocab, Vec<T>::N);
  const bool grad = MODE == kPolicy && a.dlogits;
  // Without a gradient many rows are read faster by streams of loads, all but
  // the shortest (8192 rows of 131072 bf16 265 us, held 350; 16384 of 16384 73
  // us, held 82; 32768 of 2000 39 us, held 37).
  const int64_t bytes = int64_t(a.vocab) * int64_t(sizeof(T));
  const bool stream = !grad && a.n >= 2 * kSms && bytes > kHeldRow;
  if (h.c && !stream && a.n * h.c <= 0x7fffffff) return launch_held<T, MODE>(a, x, h, s);
  // A thread's loads in flight are to be a small part of its row: for rows of
  // 8192 / 32768 / 131072 bf16, blocks of 64 threads take 39 / 141 / - us, of 128
  // 42 / 136 / 284 and of 256 68 / 138 / 266.
  auto go = [&](auto kernel, int w) { return launch(kernel, static_cast<unsigned>(a.n), w, 1, false, s, 0, a, x); };
  return bytes <= 16384    ? go(k_rows<T, MODE, 64>, 64)
         : bytes <= 131072 ? go(k_rows<T, MODE, 128>, 128)
                           : go(k_rows<T, MODE, 256>, 256);
}

template <int MODE>
cudaError_t launch_rows(const Rows& a, const Extra& x, int dtype, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  return dtype == MUON_DTYPE_BF16 ? launch_rows_of<__nv_bfloat16, MODE>(a, x, s)
                                  : launch_rows_of<float, MODE>(a, x, s);
}

// ------------------------------------------------------------------ arguments

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int check_rows(const void* logits, int dtype, int64_t stride, int64_t n, int vocab,
               const void* targets, int targets_type, float scale, const float* logp) {
  if (dtype != MUON_DTYPE_BF16 && dtype != MUON_DTYPE_FP32)
    return lfail(MUON_ERR_INVALID, "unknown dtype");
  if (targets_type != MUON_INDEX_INT32 && targets_type != MUON_INDEX_INT64)
    return lfail(MUON_ERR_INVALID, "unknown targets_type");
  if (n < 0 || n > (int64_t(1) << 30))
    return lfail(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30]");
  if (vocab < 1) return lfail(MUON_ERR_INVALID, "vocab must be >= 1");
  if (stride < vocab) return lfail(MUON_ERR_INVALID, "stride must be >= vocab");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return lfail(MUON_ERR_INVALID, "logit_scale must be > 0 and finite");
  if (n > 0 && (!logits || !targets || !logp))
    return lfail(MUON_ERR_INVALID, "logits, targets or logp is NULL");
  if (misaligned(logits, dtype == MUON_DTYPE_BF16 ? 2 : 4) || misaligned(logp, 4) ||
      misaligned(targets, targets_type == MUON_INDEX_INT64 ? 8 : 4))
    return lfail(MUON_ERR_INVALID, "logits, targets or logp is not aligned to its type");
  return MUON_OK;
}

int check_grad(const void* logits, int dtype, int64_t stride, int64_t n, int vocab,
               const void* d, int64_t dstride) {
  if (!d) return MUON_OK;
  const size_t es = dtype == MUON_DTYPE_BF16 ? 2 : 4;
  if (misaligned(d, es)) return lfail(MUON_ERR_INVALID, "dlogits is not aligned to its type");
  if (dstride < vocab) return lfail(MUON_ERR_INVALID, "dlogits_stride must be >= vocab");
  if (n == 0) return MUON_OK;
  if (d == logits && (dstride == stride || n == 1)) return MUON_OK;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(logits), b0 = reinterpret_cast<uintptr_t>(d);
  const uintptr_t a1 = a0 + ((n - 1) * stride + vocab) * es, b1 = b0 + ((n - 1) * dstride + vocab) * es;
  if (a0 < b1 && b0 < a1)
    return lfail(MUON_ERR_INVALID, "dlogits overlaps the logits without being the same rows");
  return MUON_OK;
}

Rows make_rows(const void* logits, int64_t stride, int64_t n, int vocab, const void* targets,
               int targets_type, float scale, float* logp, void* d, int64_t dstride) {
  Rows a{};
  a.logits = logits;
  a.stride = stride;
  a.n = n;
  a.vocab = vocab;
  a.targets64 = targets_type == MUON_INDEX_INT64;
  a.targets = targets;
  a.scale = scale;
  const double scale2 = double(scale) * 1.4426950408889634;
  a.scale2 = static_cast<float>(scale2);
  a.slack = static_cast<float>(std::min(8.0 / double(scale), 1e38));
  // Rounded to FP32, s log2(e) makes every exponent too large or too small by
  // up to 6e-8 of itself, in every row alike, and sums of log-probabilities over
  // a sequence show it (3e-7 a token at s = 0.8).  Of the factors k / 64 one
  // leaves a second factor that is exact to about 1e-9.
  double best = 1.0;
  for (int k = 64; k < 128; ++k) {
    const double first = k / 64.0, second = static_cast<float>(scale2 / first);
    const double off = std::fabs(first * second / scale2 - 1.0);
    if (off < best) {
      best = off;
      a.first = static_cast<float>(first);
      a.second = static_cast<float>(second);
    }
  }
  a.logp = logp;
  a.dlogits = d;
  a.dstride = dstride;
  return a;
}

int begin_call() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return lfail(MUON_ERR_CUDA, "cudaGetDevice failed");
  note_token_device(dev);
  return MUON_OK;
}

int end_call(int launches, cudaError_t e) {
  count_launches(launches);
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
  if (e != cudaSuccess)
    return lfail(MUON_ERR_CUDA, std::string("kernel launch: ") + cudaGetErrorString(e));
  return MUON_OK;
}

size_t preference_bytes(int64_t n) { return (size_t(n) * (sizeof(float2) + 2 * sizeof(float)) + 15) & ~size_t(15); }

}  // namespace

int losses_take_device_error() { return take_flag(g_losses_err); }

}  // namespace muon

using namespace muon;

extern "C" int muon_token_logprobs(const void* logits, int dtype, int64_t stride, int64_t n_tokens,
                                   int vocab, const void* targets, int targets_type,
                                   float logit_scale, float* logp, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_token_logprobs");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    int rc = check_rows(logits, dtype, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp);
    if (rc != MUON_OK) return rc;
    if (n_tokens == 0) return MUON_OK;
    if ((rc = begin_call()) != MUON_OK) return rc;
    const Rows a = make_rows(logits, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp,
                             nullptr, 0);
    return end_call(1, launch_rows<kLogp>(a, Extra{}, dtype, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int muon_policy_loss(const void* logits, int dtype, int64_t stride, int64_t n_tokens,
                                int vocab, const void* targets, int targets_type,
                                const float* advantages, const float* weights,
                                const float* old_logp, const float* ref_logp, float clip_low,
                                float clip_high, float kl_coef, float logit_scale, float* stats,
                                float* logp, void* dlogits, int64_t dlogits_stride, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_policy_loss");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    int rc = check_rows(logits, dtype, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp);
    if (rc == MUON_OK) rc = check_grad(logits, dtype, stride, n_tokens, vocab, dlogits, dlogits_stride);
    if (rc != MUON_OK) return rc;
    if (!stats || misaligned(stats, 4)) return lfail(MUON_ERR_INVALID, "stats is NULL or misaligned");
    if (n_tokens > 0 && (!advantages || !weights))
      return lfail(MUON_ERR_INVALID, "advantages or weights is NULL");
    if (misaligned(advantages, 4) || misaligned(weights, 4) || misaligned(old_logp, 4) || misaligned(ref_logp, 4))
      return lfail(MUON_ERR_INVALID, "a per-token array is not 4-byte aligned");
    if (!(clip_low >= 0.f) || !(clip_high >= 0.f) || !(kl_coef >= 0.f) || !std::isfinite(clip_low) ||
        !std::isfinite(clip_high) || !std::isfinite(kl_coef))
      return lfail(MUON_ERR_INVALID, "clip_low, clip_high and kl_coef must be finite and >= 0");
    if (kl_coef > 0.f && !ref_logp && n_tokens > 0)
      return lfail(MUON_ERR_INVALID, "kl_coef > 0 needs ref_logp");
    if ((rc = begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Rows a = make_rows(logits, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp,
                             dlogits, dlogits_stride);
    Extra x{};
    x.policy = {advantages, weights, old_logp, ref_logp, clip_low, clip_high, kl_coef};
    cudaError_t e = launch_rows<kPolicy>(a, x, dtype, s);
    const int blocks = sum_blocks(n_tokens);
    if (e == cudaSuccess)
      e = launch(k_policy_sum, blocks, kSumThreads, blocks, n_tokens > 0, s, 0, a, x.policy, stats);
    return end_call((n_tokens > 0) + 1, e);
  });
}

extern "C" int muon_preference_loss_workspace(int64_t n_tokens, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    if (n_tokens < 0 || n_tokens > (int64_t(1) << 30) || !bytes)
      return lfail(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30] and bytes non-NULL");
    *bytes = preference_bytes(n_tokens);
    return MUON_OK;
  });
}

extern "C" int muon_preference_loss(const void* logits, int dtype, int64_t stride, int64_t n_tokens,
                                    int vocab, const void* targets, int targets_type,
                                    const void* offsets, int offsets_type, int n_pairs,
                                    const float* ref_logp, const float* pair_weights, float beta,
                                    float label_smoothing, float logit_scale, float* stats,
                                    float* margins, float* logp, void* dlogits,
                                    int64_t dlogits_stride, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_preference_loss");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    int rc = check_rows(logits, dtype, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp);
    if (rc == MUON_OK) rc = check_grad(logits, dtype, stride, n_tokens, vocab, dlogits, dlogits_stride);
    if (rc != MUON_OK) return rc;
    if (!stats || misaligned(stats, 4)) return lfail(MUON_ERR_INVALID, "stats is NULL or misaligned");
    if (n_pairs < 0 || n_pairs > (1 << 30)) return lfail(MUON_ERR_INVALID, "n_pairs must be in [0, 2^30]");
    if (offsets_type != MUON_INDEX_INT32 && offsets_type != MUON_INDEX_INT64)
      return lfail(MUON_ERR_INVALID, "unknown offsets_type");
    if (n_pairs > 0 && (!offsets || !margins))
      return lfail(MUON_ERR_INVALID, "offsets or margins is NULL");
    if (misaligned(offsets, offsets_type == MUON_INDEX_INT64 ? 8 : 4) || misaligned(margins, 4) ||
        misaligned(ref_logp, 4) || misaligned(pair_weights, 4))
      return lfail(MUON_ERR_INVALID, "offsets, margins, ref_logp or pair_weights is misaligned");
    if (!std::isfinite(beta)) return lfail(MUON_ERR_INVALID, "beta must be finite");
    if (!(label_smoothing >= 0.f && label_smoothing <= 1.f))
      return lfail(MUON_ERR_INVALID, "label_smoothing must be in [0, 1]");
    const int vec = dtype == MUON_DTYPE_BF16 ? Vec<__nv_bfloat16>::N : Vec<float>::N;
    const int nvec = std::max(1, vocab / vec);
    int given = 32;   // k_given's threads: a short row in one block of them
    while (given < kGivenThreads && given * kGivenVecs < nvec) given *= 2;
    const int slices = (nvec + given * kGivenVecs - 1) / (given * kGivenVecs);
    if (n_tokens * slices >= 0x7fffffff)
      return lfail(MUON_ERR_UNSUPPORTED, "too many tokens of a vocabulary this large for one call");
    if (n_tokens > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < preference_bytes(n_tokens)))
      return lfail(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
    if ((rc = begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Rows a = make_rows(logits, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp,
                             dlogits, dlogits_stride);
    Extra x{};
    x.stats = static_cast<float2*>(workspace);
    x.coef = reinterpret_cast<float*>(x.stats + n_tokens);
    x.logp_lo = x.coef + n_tokens;
    const Pairs q{offsets, offsets_type == MUON_INDEX_INT64, n_pairs, ref_logp, pair_weights, beta,
                  label_smoothing, x.logp_lo, margins, dlogits ? x.coef : nullptr};
    cudaError_t e = launch_rows<kStats>(a, x, dtype, s);
    int width = 64;   // a pair's mean sequence in one round of its threads
    while (width < kPairThreads && int64_t(width) * 8 * n_pairs < n_tokens) width *= 2;
    if (e == cudaSuccess && n_pairs > 0) e = launch(k_pairs, n_pairs, width, 1, n_tokens > 0, s, 0, a, q);
    if (e == cudaSuccess && dlogits && n_tokens > 0) {
      e = dtype == MUON_DTYPE_BF16 ? launch_given<__nv_bfloat16>(a, x, q, stats, given, slices, s)
                                   : launch_given<float>(a, x, q, stats, given, slices, s);
    } else if (e == cudaSuccess) {
      e = launch(k_pair_sum, 1, 32, 1, n_tokens > 0 || n_pairs > 0, s, 0, q, stats);
    }
    return end_call((n_tokens > 0) + (n_pairs > 0) + 1, e);
  });
}
