// Log-probabilities of target tokens, the clipped policy loss with a KL term
// and the preference loss of paired log ratios, with the gradient of the
// logits.
//
// With z a row of logits, s the scale, y its target, m = max z:
//     e_v  = exp(s (z_v - m)),   S = sum_v e_v
//     logp = s (z_y - m) - log S
// and for a loss that depends on the row through logp alone,
//     dz_v = s c (1[v = y] - e_v / S),   c = d loss / d logp.
// Subtracting m before scaling keeps rows of the type's lowest value and of
// minus infinities right without a branch: the running maximum starts at the
// lowest finite FP32 value, so minus infinity always gives e = 0, and a row of
// nothing else has S = 0 and logp NaN.
//
// Maxima, sums and e are FP32 whatever the logits' type; sums over tokens are
// FP64 (a few thousand terms, off the hot path) in a fixed order.
#include <cfloat>
#include <cmath>
#include <string>

#include "token_ops.cuh"

namespace muon {
namespace {

using tok::Vec;

__device__ int g_losses_err;

constexpr int kRowThreads = 512;     // k_rows: threads of a row
constexpr int kSumThreads = 1024;
constexpr int kPairThreads = 256;

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

struct PolicyTerms {
  float term, kl;
  float coef;   // d (term + kl_coef kl) / d logp
  bool cut;
};

__device__ __forceinline__ PolicyTerms policy_terms(const Policy& p, int64_t t, float logp) {
  PolicyTerms o;
  const float a = p.advantages[t];
  const float r = p.old_logp ? expf(logp - p.old_logp[t]) : (logp == logp ? 1.f : logp);
  const float free = r * a;
  const float held = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * a;
  o.cut = free > held;
  o.term = o.cut ? -held : -free;
  o.coef = o.cut ? 0.f : -free;
  o.kl = 0.f;
  if (p.ref_logp) {
    const float q = p.ref_logp[t] - logp;
    const float g = expm1f(q);
    o.kl = g - q;
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

// Joins the softmax statistics (m, s) of two parts of a row.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float scale2) {
  const float top = fmaxf(m, m2);
  s = s * ex2((m - top) * scale2) + s2 * ex2((m2 - top) * scale2);
  m = top;
}

__device__ __forceinline__ void warp_join(float& m, float& s, float scale2) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2, scale2);
  }
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
};

enum RowMode {
  kLogp = 0,     // logp
  kStats = 1,    // logp and (m, 1/S) for a later gradient pass
  kPolicy = 2,   // logp and the policy loss's gradient
  kGiven = 3     // the gradient alone, from (m, 1/S) and c
};

struct Extra {
  Policy policy;
  float2* stats;      // kStats, kGiven: (m, 1/S) per row
  float* coef;        // kGiven: c per row; kStats zeroes it
};

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
  if (threadIdx.x < sh.head)
    drow[threadIdx.x] = tok::from_float<T>(one(threadIdx.x, tok::to_float(row[threadIdx.x])));
  for (int v = sh.tail0 + threadIdx.x; v < a.vocab; v += blockDim.x)
    drow[v] = tok::from_float<T>(one(v, tok::to_float(row[v])));
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
  const T zero = tok::from_float<T>(0.f);
  if (threadIdx.x < sh.head) drow[threadIdx.x] = zero;
  for (int v = sh.tail0 + threadIdx.x; v < a.vocab; v += blockDim.x) drow[v] = zero;
  for (int i = threadIdx.x; i < sh.nvec; i += blockDim.x)
    *reinterpret_cast<uint4*>(drow + sh.head + i * Vec<T>::N) = make_uint4(0, 0, 0, 0);
}

// One block per row: a pass for (m, S), and for the gradient a second one
// that reads the row again (from L2: the rows in flight are a few tens of MB).
template <typename T, int MODE>
__global__ void __launch_bounds__(kRowThreads) k_rows(const Rows a, const Extra x) {
  constexpr int N = Vec<T>::N;
  __shared__ float sm[kRowThreads / 32], ss[kRowThreads / 32];
  const int64_t t = blockIdx.x;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
  T* drow = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
  const int y = row_target(a, t);
  if (MODE == kGiven) {
    const float c = x.coef[t];
    if (y < 0 || c == 0.f) return write_zeros<T>(a, drow);
    const float2 st = x.stats[t];
    return write_grad<T>(a, row, drow, y, st.x, st.y, a.scale * c);
  }
  if (y < 0 || (MODE == kPolicy && x.policy.weights[t] == 0.f)) {
    if (threadIdx.x == 0) {
      a.logp[t] = 0.f;
      if (MODE == kStats) x.coef[t] = 0.f;
    }
    if (MODE == kPolicy && drow) write_zeros<T>(a, drow);
    return;
  }
  const RowShape<T> sh(row, a.vocab);
  float m = -FLT_MAX, s = 0.f;
  auto take = [&](float z) { join(m, s, z, 1.f, a.scale2); };
  if (threadIdx.x < sh.head) take(tok::to_float(row[threadIdx.x]));
  for (int v = sh.tail0 + threadIdx.x; v < a.vocab; v += kRowThreads) take(tok::to_float(row[v]));
#pragma unroll 4
  for (int i = threadIdx.x; i < sh.nvec; i += kRowThreads) {
    float f[N];
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + sh.head + i * N), f);
    float top = m;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, f[k]);
    s *= ex2((m - top) * a.scale2);
    m = top;
#pragma unroll
    for (int k = 0; k < N; ++k) s += ex2((f[k] - m) * a.scale2);
  }
  const float zy = tok::to_float(row[y]);
  warp_join(m, s, a.scale2);
  if (threadIdx.x % 32 == 0) {
    sm[threadIdx.x / 32] = m;
    ss[threadIdx.x / 32] = s;
  }
  __syncthreads();
  m = sm[0];
  s = ss[0];
  for (int w = 1; w < kRowThreads / 32; ++w) join(m, s, sm[w], ss[w], a.scale2);
  const float logp = a.scale * (zy - m) - logf(s);
  if (threadIdx.x == 0) {
    a.logp[t] = logp;
    if (MODE == kStats) {
      x.stats[t] = make_float2(m, 1.f / s);
      x.coef[t] = 0.f;
    }
  }
  if (MODE == kPolicy && drow) {
    const float c = x.policy.weights[t] * policy_terms(x.policy, t, logp).coef;
    if (c == 0.f) return write_zeros<T>(a, drow);
    write_grad<T>(a, row, drow, y, m, 1.f / s, a.scale * c);
  }
}

template <int NT>
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < NT / 32; ++w) v += sh[w];
  return v;
}

// The policy loss's statistics from the tokens' logp.
__global__ void __launch_bounds__(kSumThreads) k_policy_sum(const Rows a, const Policy p,
                                                            float* stats) {
  __shared__ double sh[kSumThreads / 32];
  double term = 0.0, kl = 0.0, cut = 0.0;
  for (int64_t t = threadIdx.x; t < a.n; t += kSumThreads) {
    const int y = tok::load_index(a.targets, a.targets64, t);
    const float w = p.weights[t];
    if (y < 0 || y >= a.vocab || w == 0.f) continue;
    const PolicyTerms o = policy_terms(p, t, a.logp[t]);
    term += double(w) * o.term;
    kl += double(w) * o.kl;
    if (o.cut) cut += w;
  }
  term = block_sum<kSumThreads>(term, sh);
  kl = block_sum<kSumThreads>(kl, sh);
  cut = block_sum<kSumThreads>(cut, sh);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(p.kl_coef != 0.f ? term + double(p.kl_coef) * kl : term);
    stats[1] = static_cast<float>(term);
    stats[2] = static_cast<float>(kl);
    stats[3] = static_cast<float>(cut);
  }
}

struct Pairs {
  const void* offsets;
  int offsets64;
  int n;
  const float* ref_logp;
  const float* weights;
  float beta, smoothing;
  float* margins;
  float* coef;
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
  __shared__ double sh[kPairThreads / 32];
  double sum[2];
  int64_t b[2], e[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    sequence(a, q, blockIdx.x + j * q.n, b[j], e[j]);
    double v = 0.0;
    for (int64_t t = b[j] + threadIdx.x; t < e[j]; t += kPairThreads)
      if (row_target(a, t) >= 0) v += double(a.logp[t]) - (q.ref_logp ? double(q.ref_logp[t]) : 0.0);
    sum[j] = block_sum<kPairThreads>(v, sh);
  }
  const float h = static_cast<float>(double(q.beta) * (sum[0] - sum[1]));
  if (threadIdx.x == 0) q.margins[blockIdx.x] = h;
  if (!q.coef) return;
  const float w = q.weights ? q.weights[blockIdx.x] : 1.f / q.n;
  // d loss / d h = sigmoid(h) - (1 - smoothing), written so that neither term cancels
  const float dh = q.smoothing * sigmoid(h) - (1.f - q.smoothing) * sigmoid(-h);
  const float g = w == 0.f ? 0.f : w * q.beta * dh;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    for (int64_t t = b[j] + threadIdx.x; t < e[j]; t += kPairThreads) q.coef[t] = j ? -g : g;
}

__global__ void __launch_bounds__(kSumThreads) k_pair_sum(const Pairs q, float* stats) {
  __shared__ double sh[kSumThreads / 32];
  double loss = 0.0, mean = 0.0, won = 0.0, weight = 0.0;
  for (int i = threadIdx.x; i < q.n; i += kSumThreads) {
    const double w = q.weights ? double(q.weights[i]) : 1.0 / q.n;
    if (w == 0.0) continue;
    const float h = q.margins[i];
    float l = 0.f;
    if (q.smoothing < 1.f) l += (1.f - q.smoothing) * softplus(-h);
    if (q.smoothing > 0.f) l += q.smoothing * softplus(h);
    loss += w * l;
    mean += w * h;
    won += h > 0.f ? w : 0.0;
    weight += w;
  }
  loss = block_sum<kSumThreads>(loss, sh);
  mean = block_sum<kSumThreads>(mean, sh);
  won = block_sum<kSumThreads>(won, sh);
  weight = block_sum<kSumThreads>(weight, sh);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(loss);
    stats[1] = static_cast<float>(mean);
    stats[2] = static_cast<float>(won);
    stats[3] = static_cast<float>(weight);
  }
}

template <int MODE>
int launch_rows(const Rows& a, const Extra& x, int dtype, cudaStream_t s) {
  if (a.n == 0) return 0;
  if (dtype == MUON_DTYPE_BF16)
    k_rows<__nv_bfloat16, MODE><<<static_cast<unsigned>(a.n), kRowThreads, 0, s>>>(a, x);
  else
    k_rows<float, MODE><<<static_cast<unsigned>(a.n), kRowThreads, 0, s>>>(a, x);
  return 1;
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
  a.scale2 = static_cast<float>(double(scale) * 1.4426950408889634);
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

int end_call(int launches) {
  count_launches(launches);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return lfail(MUON_ERR_CUDA, std::string("kernel launch: ") + cudaGetErrorString(e));
  return MUON_OK;
}

size_t preference_bytes(int64_t n) { return (size_t(n) * (sizeof(float2) + sizeof(float)) + 15) & ~size_t(15); }

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
    return end_call(launch_rows<kLogp>(a, Extra{}, dtype, static_cast<cudaStream_t>(stream)));
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
    const int k = launch_rows<kPolicy>(a, x, dtype, s);
    k_policy_sum<<<1, kSumThreads, 0, s>>>(a, x.policy, stats);
    return end_call(k + 1);
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
    if (n_tokens > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < preference_bytes(n_tokens)))
      return lfail(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
    if ((rc = begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Rows a = make_rows(logits, stride, n_tokens, vocab, targets, targets_type, logit_scale, logp,
                             dlogits, dlogits_stride);
    Extra x{};
    x.stats = static_cast<float2*>(workspace);
    x.coef = reinterpret_cast<float*>(x.stats + n_tokens);
    Pairs q{offsets, offsets_type == MUON_INDEX_INT64, n_pairs, ref_logp, pair_weights, beta,
            label_smoothing, margins, dlogits ? x.coef : nullptr};
    int k = dlogits ? launch_rows<kStats>(a, x, dtype, s) : launch_rows<kLogp>(a, x, dtype, s);
    if (n_pairs > 0) {
      k_pairs<<<n_pairs, kPairThreads, 0, s>>>(a, q);
      ++k;
    }
    k_pair_sum<<<1, kSumThreads, 0, s>>>(q, stats);
    if (dlogits) k += launch_rows<kGiven>(a, x, dtype, s);
    return end_call(k + 1);
  });
}
