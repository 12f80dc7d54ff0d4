// Shared by the operators of a model's layers (linear.cu, layers.cu): the
// draws of dropout, activations, host checks.
#pragma once

#include <cmath>

#include "token_ops.cuh"

namespace muon {
namespace lay {

// ------------------------------------------------------------------ dropout

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products, the key
// raised by two constants after each.  One call gives eight elements their 16
// bits, about 7 instructions an element.
__device__ __forceinline__ uint4 philox(uint4 c, uint2 k) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = uint64_t(0xD2511F53u) * c.x, q = uint64_t(0xCD9E8D57u) * c.z;
    c = make_uint4(uint32_t(q >> 32) ^ c.y ^ k.x, uint32_t(q), uint32_t(p >> 32) ^ c.w ^ k.y, uint32_t(p));
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

// What an element is multiplied by: 0 where its 16 bits are below `least`, else
// `gain`.  least = 0: no dropout.
struct Dropout {
  const int64_t* rng;   // seed, step
  uint32_t site;
  uint32_t least;
  float gain;
};

// The two words a thread needs of rng, read once.
struct Draw {
  uint2 key;
  uint32_t step;
  __device__ __forceinline__ void init(const Dropout& d) {
    if (d.least == 0) return;
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]);
    key = make_uint2(uint32_t(seed), uint32_t(seed >> 32));
    step = static_cast<uint32_t>(d.rng[1]);
  }
  // Columns [8 group, 8 group + 8) of a row, four words of two elements each.
  __device__ __forceinline__ uint4 at(uint32_t row, uint32_t group, uint32_t site) const {
    return philox(make_uint4(group, row, site, step), key);
  }
};

__device__ __forceinline__ uint32_t draw_of(const uint4& w, int j) {
  const uint32_t u = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return j & 1 ? u >> 16 : u & 0xffffu;
}

__device__ __forceinline__ float dropped(float x, uint32_t bits, const Dropout& d) {
  return bits < d.least ? 0.f : x * d.gain;   // a select: what is left out may be infinite or NaN
}

// ------------------------------------------------------------------ activations

// u (1 + tanh(h)) / 2 = u / (1 + exp(-2 h)) with h = sqrt(2 / pi) (u + 0.044715 u^3).
constexpr float kGelu1 = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.07135481627260025f;   // 0.044715 of it

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// CUDA bounds __expf's error by 2 + floor(|1.173 x|) units and __fdividef's by 2, so
// that the sigmoid is off by (4 + 1.2 |x|) 2^-23 of itself at most where it is small,
// by less than that next to 1.  Where 1 + exp(-x) passes 2^126 (x < -87.3), __fdividef
// gives 0 for what is below 2^-126.
__device__ __forceinline__ float activation(float u, int kind) {
  switch (kind) {
    case MUON_ACT_RELU: return u > 0.f ? u : u == u ? 0.f : u;
    case MUON_ACT_RELU2: return u > 0.f ? u * u : u == u ? 0.f : u;
    case MUON_ACT_GELU: return u * sigmoid(u * (kGelu1 + kGelu3 * u * u));
    case MUON_ACT_SILU: return u * sigmoid(u);
    default: return u;
  }
}

__device__ __forceinline__ float slope(float u, int kind) {
  switch (kind) {
    case MUON_ACT_RELU: return u > 0.f ? 1.f : u == u ? 0.f : u;
    case MUON_ACT_RELU2: return u > 0.f ? 2.f * u : u == u ? 0.f : u;
    case MUON_ACT_GELU: {
      u = u > 20.f ? 20.f : u < -20.f ? -20.f : u;   // 0 and 1 from there on, and u^2 stays finite
      const float s = sigmoid(u * (kGelu1 + kGelu3 * u * u));
      return s + u * s * (1.f - s) * (kGelu1 + 3.f * kGelu3 * u * u);
    }
    case MUON_ACT_SILU: {
      u = u > 80.f ? 80.f : u < -80.f ? -80.f : u;   // NaN stays: both comparisons are false
      const float s = sigmoid(u);
      return s * (1.f + u * (1.f - s));
    }
    default: return 1.f;
  }
}

// ------------------------------------------------------------------ host checks

// Bytes from a tensor's first to behind its last element.
struct Span {
  uintptr_t begin = 0, end = 0;
  Span() = default;
  Span(const void* p, int64_t rows, int64_t stride, int64_t cols, size_t es) {
    if (!p || rows <= 0) return;
    begin = reinterpret_cast<uintptr_t>(p);
    end = begin + (uintptr_t(rows - 1) * stride + cols) * es;
  }
  bool meets(const Span& o) const { return begin < o.end && o.begin < end; }
};

inline bool same(const void* a, int64_t sa, const void* b, int64_t sb) { return a == b && sa == sb; }

// Strides such that rows * stride * es stays far from wrapping.
inline bool stride_fits(int64_t rows, int64_t stride) {
  return stride >= 0 && (rows <= 1 || stride <= (int64_t(1) << 58) / rows);
}

// dropout's rate, site and generator; `least` = 0 where nothing is left out.
inline int make_dropout(float rate, const int64_t* rng, uint32_t site, Dropout* out) {
  if (!(rate >= 0.f && rate < 1.f)) return fail_with(MUON_ERR_INVALID, "the dropout rate must be in [0, 1)");
  const uint32_t least = static_cast<uint32_t>(std::floor(double(rate) * 65536.0 + 0.5));
  if (least > 65535) return fail_with(MUON_ERR_INVALID, "the dropout rate must be less than 1 - 2^-17");
  if (least > 0 && (!rng || misaligned(rng, 8)))
    return fail_with(MUON_ERR_INVALID, "rng is NULL or not aligned to 8 bytes");
  *out = {rng, site, least, 65536.f / (65536.f - float(least))};
  return MUON_OK;
}

inline int begin_call() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail_with(MUON_ERR_CUDA, "cudaGetDevice failed");
  note_token_device(dev);
  return MUON_OK;
}

inline int end_call(int launches, cudaError_t e) {
  count_launches(launches);
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
  if (e != cudaSuccess)
    return fail_with(MUON_ERR_CUDA, std::string("kernel launch: ") + cudaGetErrorString(e));
  return MUON_OK;
}

// A parameter's place in accum: its pieces, checked as muon_embedding_grad checks them.
inline int place_param(const muon_param_t& p, const float* accum, int64_t accum_elems,
                       const muon_partition_t* parts, int nparts, Segments* sg) {
  if (p.offset < 0) return fail_with(MUON_ERR_INVALID, "the parameter's offset < 0");
  if (p.rows < 1 || p.cols < 1) return fail_with(MUON_ERR_INVALID, "the parameter's rows or cols < 1");
  if (!accum || misaligned(accum, 16)) return fail_with(MUON_ERR_INVALID, "accum must be 16-byte aligned");
  if (nparts < 0 || (nparts > 0 && !parts)) return fail_with(MUON_ERR_INVALID, "parts is NULL");
  const int rc = segments_of(p, parts, nparts, sg);
  if (rc != MUON_OK) return rc;
  for (int i = 0; i < sg->n; ++i)
    if (sg->at[i] + ((i + 1 < sg->n ? sg->rel[i + 1] : sg->numel) - sg->rel[i]) > accum_elems)
      return fail_with(MUON_ERR_INVALID, "accum_elems is less than the tables describe");
  return MUON_OK;
}

inline bool flat_overlap(const muon_param_t& a, const muon_param_t& b) {
  const int64_t na = int64_t(a.rows) * a.cols, nb = int64_t(b.rows) * b.cols;
  return a.offset < b.offset + nb && b.offset < a.offset + na;
}

}  // namespace lay
}  // namespace muon
