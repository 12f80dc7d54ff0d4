// Shared by the operators at the two ends of a language model (embedding.cu,
// losses.cu) and of its layers (linear.cu, layers.cu): element types, token
// indexes, where a parameter lies in storage, the device error flag.
#pragma once

#include <algorithm>
#include <limits>
#include <string>
#include <vector>

#include <cuda_bf16.h>

#include "muon_internal.h"

namespace muon {

// Codes these operators record for muon_device_error.
constexpr int kErrIndex = 17;     // a token id or target >= the table's rows / the vocabulary
constexpr int kErrOffsets = 18;   // sequence offsets that decrease or leave [0, tokens]

namespace tok {

// 16 bytes of T as floats and back.
template <typename T> struct Vec;

template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack2(uint32_t u, float* f) {
    f[0] = __uint_as_float(u << 16);
    f[1] = __uint_as_float(u & 0xffff0000u);
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    unpack2(v.x, f); unpack2(v.y, f + 2); unpack2(v.z, f + 4); unpack2(v.w, f + 6);
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Token indexes: int32 or int64.  Values above INT32_MAX are kept apart from
// the valid ones by saturating, those below 0 all mean "no token".
__device__ __forceinline__ int load_index(const void* p, int is64, int64_t i) {
  if (!is64) return reinterpret_cast<const int32_t*>(p)[i];
  const int64_t v = reinterpret_cast<const int64_t*>(p)[i];
  return v < 0 ? -1 : v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v);
}

// Sums of FP32 values kept as hi + lo (Knuth's two-sum), about 48 bits: FP64
// adds run at 1/64 of the FP32 rate here (a block's sum of 1024 doubles took
// 10 us).  An infinite or NaN hi is the sum.
struct Two {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Two& o) {
    add(o.hi);
    lo += o.lo;
  }
  __device__ __forceinline__ float value() const { return fabsf(hi) <= 3.402823466e38f ? hi + lo : hi; }
  __device__ __forceinline__ void warp_sum() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Two b;
      b.hi = __shfl_xor_sync(0xffffffffu, hi, o);
      b.lo = __shfl_xor_sync(0xffffffffu, lo, o);
      // the lanes of a pair add the same two values in the same order
      const bool up = (threadIdx.x & o) != 0;
      Two x = up ? b : *this;
      x.add(up ? *this : b);
      *this = x;
    }
  }
};

// Programmatic dependent launch: wait until the kernels before this one in
// the stream have written what they write; let the next one be scheduled.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace tok

// The parameter's runs in storage: elements [rel[i], rel[i + 1]) of the
// parameter start at storage index at[i].
struct Segments {
  int n;
  int64_t rel[MUON_EMBEDDING_MAX_SEGMENTS];
  int64_t at[MUON_EMBEDDING_MAX_SEGMENTS];
  int64_t numel;

  // storage index of element i, and how many elements follow in one piece
  __device__ __forceinline__ int64_t place(int64_t i, int64_t* room) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (rel[mid] <= i) lo = mid; else hi = mid - 1;
    }
    *room = (lo + 1 < n ? rel[lo + 1] : numel) - i;
    return at[lo] + (i - rel[lo]);
  }
};

// Launches `kernel` in clusters of `cluster` blocks; early: it may be
// scheduled while the kernel before it drains (it then calls wait_before).
template <typename... A, typename... B>
cudaError_t launch(void (*kernel)(A...), unsigned grid, dim3 block, int cluster, bool early,
                   cudaStream_t s, int shared_bytes, B... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.dynamicSmemBytes = shared_bytes;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (early) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, A(args)...);
}

// Runs the body of a C entry point: no C++ exception leaves it (the only ones
// that can arise are failed host allocations).
template <typename F>
int entry(F&& body) {
  try {
    return body();
  } catch (...) {
    return MUON_ERR_OOM;
  }
}

inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline size_t dtype_bytes(int dtype) {
  return dtype == MUON_DTYPE_BF16 ? 2 : dtype == MUON_DTYPE_FP32 ? 4 : 0;
}

inline int fail_with(int code, const std::string& msg) {
  set_last_error(msg.c_str());
  return code;
}

// The parameter's pieces in storage, in flat order.
inline int segments_of(const muon_param_t& p, const muon_partition_t* parts, int nparts, Segments* out) {
  const int64_t numel = int64_t(p.rows) * p.cols;
  out->numel = numel;
  if (p.offset > std::numeric_limits<int64_t>::max() - numel)
    return fail_with(MUON_ERR_INVALID, "the parameter's end is past the range of an index");
  if (nparts == 0) {
    out->n = 1;
    out->rel[0] = 0;
    out->at[0] = p.offset;
    return MUON_OK;
  }
  std::vector<std::pair<int64_t, int64_t>> st;
  bool rising = true;   // in storage too: nothing to sort
  int64_t end = 0;
  for (int i = 0; i < nparts; ++i) {
    const muon_partition_t& q = parts[i];
    if (q.flat_begin < 0 || q.flat_end < q.flat_begin || q.storage_offset < 0 ||
        q.storage_offset > std::numeric_limits<int64_t>::max() - (q.flat_end - q.flat_begin))
      return fail_with(MUON_ERR_INVALID, "partition " + std::to_string(i) + " has a bad range");
    if (i > 0 && parts[i - 1].flat_end > q.flat_begin)
      return fail_with(MUON_ERR_INVALID, "partitions must be sorted by flat_begin and must not overlap (at " +
                                         std::to_string(i) + ")");
    if (q.flat_end == q.flat_begin) continue;
    rising = rising && q.storage_offset >= end;
    end = q.storage_offset + (q.flat_end - q.flat_begin);
  }
  for (int i = 0; i < nparts && !rising; ++i)
    if (parts[i].flat_end > parts[i].flat_begin)
      st.push_back({parts[i].storage_offset, parts[i].storage_offset + parts[i].flat_end - parts[i].flat_begin});
  std::sort(st.begin(), st.end());
  for (size_t i = 1; i < st.size(); ++i)
    if (st[i - 1].second > st[i].first) return fail_with(MUON_ERR_INVALID, "partitions overlap in storage");
  int64_t cursor = 0;
  out->n = 0;
  for (int i = 0; i < nparts && cursor < numel; ++i) {
    const muon_partition_t& q = parts[i];
    const int64_t lo = std::max(p.offset, q.flat_begin) - p.offset;
    const int64_t hi = std::min(p.offset + numel, q.flat_end) - p.offset;
    if (lo >= hi) continue;
    if (lo != cursor) break;
    if (out->n == MUON_EMBEDDING_MAX_SEGMENTS)
      return fail_with(MUON_ERR_UNSUPPORTED, "the parameter lies in more than MUON_EMBEDDING_MAX_SEGMENTS partitions");
    out->rel[out->n] = lo;
    out->at[out->n++] = q.storage_offset + (p.offset + lo - q.flat_begin);
    cursor = hi;
  }
  if (cursor != numel) return fail_with(MUON_ERR_INVALID, "the parameter is not covered by the partitions");
  return MUON_OK;
}

// Host side.  Which devices have run these operators (bit per device; the
// caller holds the library lock), so that muon_device_error reads their flags.
void note_token_device(int dev);
// The first nonzero code among the devices noted, cleared once read; the
// others' wait for the next query.
int embedding_take_device_error();
int losses_take_device_error();
int linear_take_device_error();
uint64_t token_devices();

// `symbol`: the TU's own __device__ int.
template <typename S>
int take_flag(S& symbol) {
  int v = 0, now = 0;
  if (!token_devices() || cudaGetDevice(&now) != cudaSuccess) return 0;
  for (int d = 0; d < 64 && !v; ++d) {
    if (!(token_devices() >> d & 1)) continue;
    const int zero = 0;
    if (cudaSetDevice(d) != cudaSuccess || (d != now && cudaDeviceSynchronize() != cudaSuccess) ||
        cudaMemcpyFromSymbol(&v, symbol, sizeof(int)) != cudaSuccess)
      v = 0;
    if (v) cudaMemcpyToSymbol(symbol, &zero, sizeof(int));
  }
  cudaSetDevice(now);
  return v;
}

}  // namespace muon
