// Dropout from a counter, and the norm and rotation of query and key heads
// with its gradients.  Both are bound by memory: every element is read once
// and written once.
#include "layers.cuh"

namespace muon {
namespace {

using tok::Vec;
using lay::Draw;
using lay::Dropout;
using lay::Span;

constexpr int kSms = 152;

// ------------------------------------------------------------------ dropout

constexpr int kDropThreads = 256;
constexpr int kDropRows = 2;   // rows a thread has under way

struct DropArgs {
  const void* x;
  const void* residual;
  void* out;
  int64_t xs, rs, os, rows;
  int cols;
  Dropout d;
};

// Eight elements of a row as floats.  VEC: 16-byte accesses (rows of every
// tensor start on 16 bytes and cols % 8 = 0).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int left, float* f) {
  if constexpr (VEC) {
    constexpr int N = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(p + i)), f + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < left ? tok::to_float(p[i]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int left, const float* f) {
  if constexpr (VEC) {
    constexpr int N = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) __stcs(reinterpret_cast<uint4*>(p + i), Vec<T>::pack(f + i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = tok::from_float<T>(f[i]);
  }
}

// blockDim.x threads along a row, eight columns (one draw of 128 bits) each.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const DropArgs a) {
  Draw draw;
  draw.init(a.d);
  const int64_t r0 = (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * kDropRows;
  const int groups = (a.cols + 7) / 8;
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    const int c = g * 8, left = a.cols - c;
    float f[kDropRows][8], add[kDropRows][8];
#pragma unroll
    for (int q = 0; q < kDropRows; ++q) {
      if (r0 + q >= a.rows) continue;
      load8<T, VEC>(static_cast<const T*>(a.x) + (r0 + q) * a.xs + c, left, f[q]);
      if (a.residual) load8<T, VEC>(static_cast<const T*>(a.residual) + (r0 + q) * a.rs + c, left, add[q]);
    }
#pragma unroll
    for (int q = 0; q < kDropRows; ++q) {
      if (r0 + q >= a.rows) continue;
      if (a.d.least) {
        const uint4 w = draw.at(uint32_t(r0 + q), g, a.d.site);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[q][j] = lay::dropped(f[q][j], lay::draw_of(w, j), a.d);
      }
      if (a.residual) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[q][j] += add[q][j];
      }
      store8<T, VEC>(static_cast<T*>(a.out) + (r0 + q) * a.os + c, left, f[q]);
    }
  }
}

template <typename T>
cudaError_t launch_dropout(const DropArgs& a, cudaStream_t s) {
  auto whole = [](const void* p, int64_t stride) {
    return !misaligned(p, 16) && stride * int64_t(sizeof(T)) % 16 == 0;
  };
  const bool vec = a.cols % 8 == 0 && whole(a.x, a.xs) && whole(a.out, a.os) &&
                   (!a.residual || whole(a.residual, a.rs));
  const int groups = (a.cols + 7) / 8;
  int tx = 1;
  while (tx < groups && tx < kDropThreads) tx *= 2;
  const dim3 block(tx, kDropThreads / tx);
  const unsigned grid = unsigned((a.rows + int64_t(block.y) * kDropRows - 1) / (int64_t(block.y) * kDropRows));
  if (vec) k_dropout<T, true><<<grid, block, 0, s>>>(a);
  else k_dropout<T, false><<<grid, block, 0, s>>>(a);
  return cudaSuccess;
}

// ------------------------------------------------------------------ norm and rotation

constexpr int kMaxPairs = MUON_MAX_HEAD_DIM / 2;
constexpr int kRotWarps = 8;
constexpr int kGradBlocks = 4 * kSms;   // blocks of the gradient, each with its own partial sums

// One of the tensors of a group: element d of head h of token t at
// t * stride + h * head + d.
struct Heads {
  const void* p;
  int64_t stride, head;
};

struct Group {
  Heads in;    // x, or dout of the gradient
  Heads x;     // the gradient's x
  Heads out;
  const void* weight;
  int heads;
};

struct RotArgs {
  Group group[2];
  int groups;
  int64_t n;
  int dim, pairs, axes, interleaved, pos64;
  float eps;
  const void* positions;
  float* partial;              // the gradient: [block][group][dim]
  int want[2];                 // groups whose weight's gradient is wanted
  int split[2], share[2];      // pieces a token's heads are cut into, and heads in a piece
  uint64_t turns[kMaxPairs];   // turns per position, in units of 2^-64
  uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ int64_t position(const RotArgs& a, int64_t t, int axis) {
  const int64_t i = t * a.axes + axis;
  return a.pos64 ? reinterpret_cast<const int64_t*>(a.positions)[i]
                 : reinterpret_cast<const int32_t*>(a.positions)[i];
}

// cos and sin of pair i: position * turns wraps at whole turns by itself; its
// upper 32 bits, as a signed fraction, are the angle in half turns / 2^31.
__device__ __forceinline__ void angle(const RotArgs& a, int64_t t, int i, float* c, float* s) {
  const uint64_t whole = uint64_t(position(a, t, a.axis[i])) * a.turns[i];
  const float half_turns = float(int32_t((whole + 0x80000000u) >> 32)) * 4.656612873077393e-10f;
  sincospif(half_turns, s, c);
}

// A lane's share of a head: NU units of 2 * P elements.  Rotated units hold P
// pairs: P elements and their P partners; the rest holds 2 * P consecutive ones.
template <int P>
struct Place {
  int a, b;      // first element of either half
  int na, nb;    // how many of them there are
  int pair;      // first pair; -1: not turned
  __device__ __forceinline__ void of(const RotArgs& r, int unit) {
    const int turned = r.pairs / P;
    pair = -1;
    if (unit < turned) {
      pair = unit * P;
      a = r.interleaved ? unit * 2 * P : unit * P;
      b = r.interleaved ? a + P : r.pairs + unit * P;
      na = nb = P;
    } else {
      a = 2 * r.pairs + (unit - turned) * 2 * P;
      b = a + P;
      na = max(0, min(P, r.dim - a));
      nb = max(0, min(P, r.dim - b));
    }
  }
};

// P elements as floats (0 beyond n).  P = 4: one access of 8 or 16 bytes, all
// or nothing.
template <typename T, int P>
__device__ __forceinline__ void load_part(const T* p, int n, float* f) {
  if constexpr (P == 4) {
    if constexpr (sizeof(T) == 2) {
      uint2 v = make_uint2(0, 0);
      if (n) v = *reinterpret_cast<const uint2*>(p);
      Vec<T>::unpack2(v.x, f);
      Vec<T>::unpack2(v.y, f + 2);
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (n) v = *reinterpret_cast<const uint4*>(p);
      Vec<T>::unpack(v, f);
    }
  } else {
    static_assert(P == 1, "one pair or four");
    f[0] = n ? tok::to_float(*p) : 0.f;
  }
}

template <typename T, int P>
__device__ __forceinline__ void store_part(T* p, int n, const float* f) {
  if (!n) return;
  if constexpr (P == 4) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(Vec<T>::pack2(f[0], f[1]), Vec<T>::pack2(f[2], f[3]));
    else
      *reinterpret_cast<uint4*>(p) = Vec<T>::pack(f);
  } else {
    *p = tok::from_float<T>(f[0]);
  }
}

// Pairs of a unit turned in place: (a, b) -> (a c - b s, b c + a s).  f: the
// unit's 2 * P elements, those at `a` first.
template <int P>
__device__ __forceinline__ void turn(float* f, const float* c, const float* s, bool interleaved) {
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (interleaved && P > 1) {
      const float x = f[2 * k], y = f[2 * k + 1];
      f[2 * k] = x * c[k] - y * s[k];
      f[2 * k + 1] = y * c[k] + x * s[k];
    } else {
      const float x = f[k], y = f[P + k];
      f[k] = x * c[k] - y * s[k];
      f[P + k] = y * c[k] + x * s[k];
    }
  }
}

// Sum over the `lanes` lanes that hold a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp takes a token's heads of one group, or a piece of them where tokens
// are few; `lanes` lanes hold a head, 32 / lanes heads go at once.  The
// token's cosines and sines stay in registers over its heads.
template <typename T, int P, int NU, bool NORM>
__global__ void __launch_bounds__(32 * kRotWarps) k_norm_rotary(const __grid_constant__ RotArgs a, int lanes) {
  const int lane = threadIdx.x % 32, in_head = lane % lanes, first = lane / lanes, step = 32 / lanes;
  const int tasks = a.split[0] + a.split[1];
  const int64_t task = int64_t(blockIdx.x) * kRotWarps + threadIdx.x / 32;
  const int64_t t = task / tasks;
  if (t >= a.n) return;
  int piece = static_cast<int>(task % tasks);
  const int which = piece >= a.split[0];
  if (which) piece -= a.split[0];
  const Group& g = a.group[which];
  const int h0 = piece * a.share[which], h1 = min(g.heads, h0 + a.share[which]);
  bool on = true;
  if (a.pairs)
    for (int x = 0; x < a.axes; ++x) on = on && position(a, t, x) >= 0;
  Place<P> at[NU];
  float c[NU][P], s[NU][P], w[NU][2 * P];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    at[u].of(a, in_head + u * lanes);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      c[u][k] = 1.f;
      s[u][k] = 0.f;
      if (at[u].pair >= 0 && on) angle(a, t, at[u].pair + k, &c[u][k], &s[u][k]);
    }
    if constexpr (NORM) {
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) w[u][k] = 1.f;
      if (g.weight) {
        load_part<T, P>(static_cast<const T*>(g.weight) + at[u].a, at[u].na, w[u]);
        load_part<T, P>(static_cast<const T*>(g.weight) + at[u].b, at[u].nb, w[u] + P);
      }
    }
  }
  const T* in = static_cast<const T*>(g.in.p) + t * g.in.stride;
  T* out = static_cast<T*>(const_cast<void*>(g.out.p)) + t * g.out.stride;
  constexpr int U = NU == 1 ? 2 : 1;   // heads a lane has under way
  for (int b = h0; b < h1; b += U * step) {
    float f[U][NU][2 * P];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int h = b + v * step + first;
      const bool here = on && h < h1;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        load_part<T, P>(in + h * g.in.head + at[u].a, here ? at[u].na : 0, f[v][u]);
        load_part<T, P>(in + h * g.in.head + at[u].b, here ? at[u].nb : 0, f[v][u] + P);
      }
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int h = b + v * step + first;
      if constexpr (NORM) {
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int k = 0; k < 2 * P; ++k) sum += f[v][u][k] * f[v][u][k];
        const float r = rsqrtf(head_sum(sum, lanes) / float(a.dim) + a.eps);
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int k = 0; k < 2 * P; ++k) f[v][u][k] = on ? f[v][u][k] * r * w[u][k] : 0.f;
      }
      if (h >= h1) continue;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        turn<P>(f[v][u], c[u], s[u], a.interleaved);
        store_part<T, P>(out + h * g.out.head + at[u].a, at[u].na, f[v][u]);
        store_part<T, P>(out + h * g.out.head + at[u].b, at[u].nb, f[v][u] + P);
      }
    }
  }
}

// The gradient: g = dout turned back; with r = 1 / rms and n = x r,
//     dw += g n,   dx = r (g w - n mean(g w n)).
// A lane keeps its columns' dw over all tokens of its warp; blocks leave
// partial sums, which k_norm_join adds in order.
template <typename T, int P, int NU, bool NORM>
__global__ void __launch_bounds__(32 * kRotWarps) k_norm_rotary_grad(const __grid_constant__ RotArgs a, int lanes) {
  __shared__ float sums[kRotWarps][MUON_MAX_HEAD_DIM];
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32, in_head = lane % lanes, first = lane / lanes, step = 32 / lanes;
  Place<P> at[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) at[u].of(a, in_head + u * lanes);
  for (int which = 0; which < a.groups; ++which) {
    const Group& g = a.group[which];
    float w[NU][2 * P], dw[NU][2 * P];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) w[u][k] = 1.f, dw[u][k] = 0.f;
      if (NORM && g.weight) {
        load_part<T, P>(static_cast<const T*>(g.weight) + at[u].a, at[u].na, w[u]);
        load_part<T, P>(static_cast<const T*>(g.weight) + at[u].b, at[u].nb, w[u] + P);
      }
    }
    const int split = a.split[which], share = a.share[which];
    for (int64_t task = int64_t(blockIdx.x) * kRotWarps + warp; task < a.n * split;
         task += int64_t(gridDim.x) * kRotWarps) {
      const int64_t t = task / split;
      const int h0 = static_cast<int>(task % split) * share, h1 = min(g.heads, h0 + share);
      bool on = true;
      if (a.pairs)
        for (int x = 0; x < a.axes; ++x) on = on && position(a, t, x) >= 0;
      float c[NU][P], s[NU][P];
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          c[u][k] = 1.f;
          s[u][k] = 0.f;
          if (at[u].pair >= 0 && on) angle(a, t, at[u].pair + k, &c[u][k], &s[u][k]);
          s[u][k] = -s[u][k];
        }
      for (int b = h0; b < h1; b += step) {
        const int h = b + first;
        const bool here = on && h < h1;
        float d[NU][2 * P], x[NU][2 * P];
        const T* din = static_cast<const T*>(g.in.p) + t * g.in.stride + h * g.in.head;
        const T* xin = static_cast<const T*>(g.x.p) + t * g.x.stride + h * g.x.head;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          load_part<T, P>(din + at[u].a, here ? at[u].na : 0, d[u]);
          load_part<T, P>(din + at[u].b, here ? at[u].nb : 0, d[u] + P);
          if constexpr (NORM) {
            load_part<T, P>(xin + at[u].a, here ? at[u].na : 0, x[u]);
            load_part<T, P>(xin + at[u].b, here ? at[u].nb : 0, x[u] + P);
          }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) turn<P>(d[u], c[u], s[u], a.interleaved);
        if constexpr (NORM) {
          float sq = 0.f, dot = 0.f;
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int k = 0; k < 2 * P; ++k) {
              sq += x[u][k] * x[u][k];
              dot += x[u][k] * (d[u][k] * w[u][k]);
            }
          const float inv = 1.f / float(a.dim);
          const float r = rsqrtf(head_sum(sq, lanes) * inv + a.eps);
          const float m = head_sum(dot, lanes) * r * inv;   // mean of g w n
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int k = 0; k < 2 * P; ++k) {
              const float n = x[u][k] * r;
              if (here) dw[u][k] += d[u][k] * n;
              d[u][k] = r * (d[u][k] * w[u][k] - n * m);
            }
        }
        if (h >= h1) continue;
        T* out = static_cast<T*>(const_cast<void*>(g.out.p)) + t * g.out.stride + h * g.out.head;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          if (!on) {
#pragma unroll
            for (int k = 0; k < 2 * P; ++k) d[u][k] = 0.f;
          }
          store_part<T, P>(out + at[u].a, at[u].na, d[u]);
          store_part<T, P>(out + at[u].b, at[u].nb, d[u] + P);
        }
      }
    }
    if (!NORM || !a.want[which]) continue;
    // lanes of the same columns, then the block's warps
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) {
        float v = dw[u][k];
        for (int o = lanes; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int i = k < P ? at[u].a + k : at[u].b + (k - P);
        const bool there = k < P ? k < at[u].na : k - P < at[u].nb;
        if (first == 0 && there) sums[warp][i] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < a.dim; i += 32 * kRotWarps) {
      float v = 0.f;
      for (int q = 0; q < kRotWarps; ++q) v += sums[q][i];
      a.partial[(int64_t(blockIdx.x) * 2 + which) * a.dim + i] = v;
    }
  }
}

struct JoinArgs {
  const float* partial;
  int blocks, dim;
  float* accum;
  float scale;
  int overwrite;
  int want[2];
};

constexpr int kJoinWarps = 16;

// The weights' gradients: 32 columns per block, every 16th partial sum per warp.
__global__ void __launch_bounds__(32 * kJoinWarps)
k_norm_join(const JoinArgs a, const __grid_constant__ Segments s0, const __grid_constant__ Segments s1) {
  __shared__ float sums[kJoinWarps][32];
  const int slabs = (a.dim + 31) / 32;
  const int which = blockIdx.x / slabs, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = blockIdx.x % slabs * 32 + lane;
  if (!a.want[which]) return;
  float v = 0.f;
  if (i < a.dim)
    for (int b = warp; b < a.blocks; b += kJoinWarps) v += a.partial[(int64_t(b) * 2 + which) * a.dim + i];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp || i >= a.dim) return;
  for (int q = 1; q < kJoinWarps; ++q) v += sums[q][lane];
  int64_t room;
  float* p = a.accum + (which ? s1 : s0).place(i, &room);
  *p = (a.overwrite ? 0.f : *p) + a.scale * v;
}

// ---- host

int grad_blocks(int64_t n) {
  return static_cast<int>(std::min<int64_t>(kGradBlocks, std::max<int64_t>(1, (n + kRotWarps - 1) / kRotWarps)));
}

// Whether element d of any head of two tensors can share memory: apart as
// spans, or interleaved rows of one stride whose windows are apart (queries and
// keys of one packed projection).
struct HeadsView {
  const void* p;
  int64_t stride, head, n, heads, dim;
  size_t es;
  int64_t window() const { return (heads - 1) * head + dim; }
  Span span() const { return Span(p, n, stride, window(), es); }
};

bool apart(const HeadsView& a, const HeadsView& b) {
  if (!a.p || !b.p || !a.span().meets(b.span())) return true;
  if (a.stride != b.stride || a.es != b.es || a.stride < 1 || a.window() > a.stride || b.window() > b.stride)
    return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const int64_t bytes = static_cast<int64_t>(pb - pa);   // one address space: fits
  if (bytes % int64_t(a.es)) return false;
  const int64_t gap = ((bytes / int64_t(a.es)) % a.stride + a.stride) % a.stride;   // b's window within a's row
  return gap >= a.window() && a.stride - gap >= b.window();
}

int check_heads(const void* p, int64_t stride, int64_t head, int64_t n, int heads, int dim, size_t es, bool written,
                const char* name) {
  if (!p || misaligned(p, es)) return fail_with(MUON_ERR_INVALID, std::string(name) + " is NULL or misaligned");
  if (stride < 0 || head < 0 || !lay::stride_fits(n, stride) || !lay::stride_fits(heads, head))
    return fail_with(MUON_ERR_INVALID, std::string(name) + "'s strides are negative or too large");
  if (written) {
    const bool by_token = heads <= 1 || head >= dim, rows = n <= 1 || stride >= (heads - 1) * head + dim;
    const bool by_head = n <= 1 || stride >= dim, cols = heads <= 1 || head >= (n - 1) * stride + dim;
    if (!(by_token && rows) && !(by_head && cols))
      return fail_with(MUON_ERR_INVALID, std::string(name) + "'s heads overlap one another");
  }
  return MUON_OK;
}

// Arguments both directions share.
int make_rotation(RotArgs* a, int n_groups, int dtype, int64_t n_tokens, int head_dim, int norm, float eps,
                  const void* positions, int positions_type, int axes, const double* inv_freq, const int32_t* axis,
                  int pairs, int interleaved) {
  if (n_groups != 1 && n_groups != 2) return fail_with(MUON_ERR_INVALID, "n_groups must be 1 or 2");
  if (!dtype_bytes(dtype)) return fail_with(MUON_ERR_INVALID, "unknown dtype");
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 30))
    return fail_with(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30]");
  if (head_dim < 1 || head_dim > MUON_MAX_HEAD_DIM)
    return fail_with(MUON_ERR_INVALID, "head_dim must be in [1, MUON_MAX_HEAD_DIM]");
  if (norm != 0 && norm != 1) return fail_with(MUON_ERR_INVALID, "norm must be 0 or 1");
  if (norm && !(eps >= 0.f && std::isfinite(eps))) return fail_with(MUON_ERR_INVALID, "eps must be >= 0 and finite");
  if (pairs < 0 || 2 * int64_t(pairs) > head_dim)
    return fail_with(MUON_ERR_INVALID, "2 * pairs must be in [0, head_dim]");
  if (interleaved != 0 && interleaved != 1) return fail_with(MUON_ERR_INVALID, "interleaved must be 0 or 1");
  a->groups = n_groups;
  a->n = n_tokens;
  a->dim = head_dim;
  a->pairs = pairs;
  a->eps = eps;
  a->interleaved = interleaved;
  if (!pairs) return MUON_OK;
  if (positions_type != MUON_INDEX_INT32 && positions_type != MUON_INDEX_INT64)
    return fail_with(MUON_ERR_INVALID, "unknown positions_type");
  if (axes < 1 || axes > MUON_MAX_AXES) return fail_with(MUON_ERR_INVALID, "axes must be in [1, MUON_MAX_AXES]");
  if (n_tokens > 0 && (!positions || misaligned(positions, positions_type == MUON_INDEX_INT64 ? 8 : 4)))
    return fail_with(MUON_ERR_INVALID, "positions is NULL or misaligned");
  if (!inv_freq) return fail_with(MUON_ERR_INVALID, "inv_freq is NULL");
  a->positions = positions;
  a->pos64 = positions_type == MUON_INDEX_INT64;
  a->axes = axes;
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(inv_freq[i])) return fail_with(MUON_ERR_INVALID, "inv_freq must be finite");
    if (axis && (axis[i] < 0 || axis[i] >= axes)) return fail_with(MUON_ERR_INVALID, "axis must be in [0, axes)");
    // turns per position, of which the whole ones do not matter
    const double turns = inv_freq[i] / 6.283185307179586476925;
    const double part = std::ldexp(turns - std::floor(turns), 64);
    a->turns[i] = part >= 18446744073709551615.0 ? 0 : static_cast<uint64_t>(part);
    a->axis[i] = static_cast<uint8_t>(axis ? axis[i] : 0);
  }
  return MUON_OK;
}

bool on16(const Heads& h, size_t es) {
  return !h.p || (!misaligned(h.p, 16) && h.stride * int64_t(es) % 16 == 0 && h.head * int64_t(es) % 16 == 0);
}

// Four pairs to a unit where every access is then aligned: rows of 16 bytes,
// and neither the pairs nor what is behind them ends inside a unit.
bool wide(const RotArgs& a, size_t es) {
  if (a.pairs % 4 || (a.dim - 2 * a.pairs) % 8) return false;
  for (int i = 0; i < a.groups; ++i)
    if (!on16(a.group[i].in, es) || !on16(a.group[i].x, es) || !on16(a.group[i].out, es) ||
        misaligned(a.group[i].weight, 16))
      return false;
  return true;
}

// Lanes that hold a head of so many units.
int lanes_of(const RotArgs& a, int per) {
  const int units = a.pairs / per + (a.dim - 2 * a.pairs + 2 * per - 1) / (2 * per);
  int lanes = 1;
  while (lanes < units && lanes < 32) lanes *= 2;
  return lanes;
}

// A token's heads in one piece, or in more where tokens are too few to fill the
// SMs with a warp each.
void split_heads(RotArgs* a, int lanes) {
  const int step = 32 / lanes;
  int64_t total = 0;
  for (int i = 0; i < a->groups; ++i) total += a->group[i].heads;
  int share = int(std::max<int64_t>(step, std::min<int64_t>(total * a->n / (32 * kSms), 1 << 20)));
  share = (share + step - 1) / step * step;
  for (int i = 0; i < 2; ++i) {
    a->share[i] = share;
    a->split[i] = i < a->groups ? (a->group[i].heads + share - 1) / share : 0;
  }
}

template <typename T>
cudaError_t launch_rotary(RotArgs& a, bool norm, cudaStream_t s) {
  const bool v = wide(a, sizeof(T));
  const int lanes = lanes_of(a, v ? 4 : 1);
  split_heads(&a, lanes);
  const int64_t tasks = a.n * (a.split[0] + a.split[1]);
  auto k = v ? (norm ? k_norm_rotary<T, 4, 1, true> : k_norm_rotary<T, 4, 1, false>)
             : (norm ? k_norm_rotary<T, 1, 4, true> : k_norm_rotary<T, 1, 4, false>);
  return launch(k, unsigned((tasks + kRotWarps - 1) / kRotWarps), 32 * kRotWarps, 1, false, s, 0, a, lanes);
}

template <typename T>
cudaError_t launch_rotary_grad(RotArgs& a, bool norm, int blocks, cudaStream_t s) {
  const bool v = wide(a, sizeof(T));
  const int lanes = lanes_of(a, v ? 4 : 1);
  split_heads(&a, lanes);
  auto k = v ? (norm ? k_norm_rotary_grad<T, 4, 1, true> : k_norm_rotary_grad<T, 4, 1, false>)
             : (norm ? k_norm_rotary_grad<T, 1, 4, true> : k_norm_rotary_grad<T, 1, 4, false>);
  return launch(k, unsigned(blocks), 32 * kRotWarps, 1, false, s, 0, a, lanes);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" int muon_dropout(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, void* out,
                            int64_t out_stride, int dtype, int64_t rows, int cols, float rate, const int64_t* rng,
                            uint32_t site, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_dropout");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    const size_t es = dtype_bytes(dtype);
    if (!es) return fail_with(MUON_ERR_INVALID, "unknown dtype");
    if (rows < 0 || rows > (int64_t(1) << 30)) return fail_with(MUON_ERR_INVALID, "rows must be in [0, 2^30]");
    if (cols < 1 || cols > (1 << 30)) return fail_with(MUON_ERR_INVALID, "cols must be in [1, 2^30]");
    if (x_stride < cols || out_stride < cols || (residual && residual_stride < cols) ||
        !lay::stride_fits(rows, x_stride) || !lay::stride_fits(rows, out_stride) ||
        (residual && !lay::stride_fits(rows, residual_stride)))
      return fail_with(MUON_ERR_INVALID, "strides must be >= cols, and not past what memory can hold");
    DropArgs a{};
    int rc = lay::make_dropout(rate, rng, site, &a.d);
    if (rc != MUON_OK) return rc;
    if (rows == 0) return MUON_OK;
    if (!x || !out || misaligned(x, es) || misaligned(out, es) || misaligned(residual, es))
      return fail_with(MUON_ERR_INVALID, "x or out is NULL, or a tensor is not aligned to its type");
    const Span o(out, rows, out_stride, cols, es);
    if ((o.meets(Span(x, rows, x_stride, cols, es)) && !lay::same(x, x_stride, out, out_stride)) ||
        (residual && o.meets(Span(residual, rows, residual_stride, cols, es)) &&
         !lay::same(residual, residual_stride, out, out_stride)) ||
        (a.d.least && o.meets(Span(rng, 1, 2, 2, 8))))
      return fail_with(MUON_ERR_INVALID, "out overlaps x, the residual or rng");
    if ((rc = lay::begin_call()) != MUON_OK) return rc;
    a.x = x;
    a.residual = residual;
    a.out = out;
    a.xs = x_stride;
    a.rs = residual_stride;
    a.os = out_stride;
    a.rows = rows;
    a.cols = cols;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return lay::end_call(1, es == 2 ? launch_dropout<__nv_bfloat16>(a, s) : launch_dropout<float>(a, s));
  });
}

extern "C" int muon_norm_rotary(const muon_heads_t* groups, int n_groups, int dtype, int64_t n_tokens, int head_dim,
                                int norm, float eps, const void* positions, int positions_type, int axes,
                                const double* inv_freq, const int32_t* axis, int pairs, int interleaved,
                                void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_norm_rotary");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    RotArgs a{};
    int rc = make_rotation(&a, n_groups, dtype, n_tokens, head_dim, norm, eps, positions, positions_type, axes,
                           inv_freq, axis, pairs, interleaved);
    if (rc != MUON_OK) return rc;
    if (!groups) return fail_with(MUON_ERR_INVALID, "groups is NULL");
    const size_t es = dtype_bytes(dtype);
    int64_t total = 0;
    HeadsView in[2], out[2];
    for (int i = 0; i < n_groups; ++i) {
      const muon_heads_t& g = groups[i];
      if (g.heads < 1 || g.heads > (1 << 20) || g.reserved != 0)
        return fail_with(MUON_ERR_INVALID, "heads must be in [1, 2^20] and reserved 0");
      if (n_tokens == 0) continue;
      if ((rc = check_heads(g.x, g.x_stride, g.x_head_stride, n_tokens, g.heads, head_dim, es, false, "x")) ||
          (rc = check_heads(g.out, g.out_stride, g.out_head_stride, n_tokens, g.heads, head_dim, es, true, "out")))
        return rc;
      if (misaligned(g.weight, es)) return fail_with(MUON_ERR_INVALID, "weight is not aligned to its type");
      in[i] = {g.x, g.x_stride, g.x_head_stride, n_tokens, g.heads, head_dim, es};
      out[i] = {g.out, g.out_stride, g.out_head_stride, n_tokens, g.heads, head_dim, es};
      a.group[i] = {{g.x, g.x_stride, g.x_head_stride}, {}, {g.out, g.out_stride, g.out_head_stride},
                    norm ? g.weight : nullptr, g.heads};
      total += g.heads;
    }
    if (n_tokens == 0) return MUON_OK;
    if (n_tokens * total > (int64_t(1) << 33))
      return fail_with(MUON_ERR_UNSUPPORTED, "too many heads for one launch");
    const Span pos(positions, pairs ? n_tokens : 0, axes, axes, a.pos64 ? 8 : 4);
    for (int i = 0; i < n_groups; ++i) {
      for (int j = 0; j < n_groups; ++j) {
        const bool in_place = i == j && in[j].p == out[i].p && in[j].stride == out[i].stride &&
                              in[j].head == out[i].head;
        if ((!in_place && !apart(in[j], out[i])) || (j != i && !apart(out[j], out[i])))
          return fail_with(MUON_ERR_INVALID, "an out overlaps another tensor, or its x in another layout");
        if (out[i].span().meets(Span(a.group[j].weight, 1, head_dim, head_dim, es)))
          return fail_with(MUON_ERR_INVALID, "an out overlaps a weight");
      }
      if (out[i].span().meets(pos)) return fail_with(MUON_ERR_INVALID, "an out overlaps the positions");
    }
    if ((rc = lay::begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return lay::end_call(1, es == 2 ? launch_rotary<__nv_bfloat16>(a, norm, s) : launch_rotary<float>(a, norm, s));
  });
}

extern "C" int muon_norm_rotary_grad_workspace(int64_t n_tokens, int head_dim, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    if (n_tokens < 0 || n_tokens > (int64_t(1) << 30) || head_dim < 1 || head_dim > MUON_MAX_HEAD_DIM || !bytes)
      return fail_with(MUON_ERR_INVALID,
                       "n_tokens must be in [0, 2^30], head_dim in [1, MUON_MAX_HEAD_DIM] and bytes non-NULL");
    *bytes = n_tokens ? size_t(grad_blocks(n_tokens)) * 2 * head_dim * sizeof(float) : 0;
    return MUON_OK;
  });
}

extern "C" int muon_norm_rotary_grad(const muon_heads_grad_t* groups, int n_groups, int dtype, int64_t n_tokens,
                                     int head_dim, int norm, float eps, const void* positions, int positions_type,
                                     int axes, const double* inv_freq, const int32_t* axis, int pairs,
                                     int interleaved, float* accum, int64_t accum_elems,
                                     const muon_partition_t* parts, int nparts, float scale, int overwrite,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_norm_rotary_grad");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    RotArgs a{};
    int rc = make_rotation(&a, n_groups, dtype, n_tokens, head_dim, norm, eps, positions, positions_type, axes,
                           inv_freq, axis, pairs, interleaved);
    if (rc != MUON_OK) return rc;
    if (!groups) return fail_with(MUON_ERR_INVALID, "groups is NULL");
    if (overwrite != 0 && overwrite != 1) return fail_with(MUON_ERR_INVALID, "overwrite must be 0 or 1");
    if (!std::isfinite(scale)) return fail_with(MUON_ERR_INVALID, "scale must be finite");
    const size_t es = dtype_bytes(dtype);
    Segments sg[2];
    sg[0].n = sg[1].n = 0;
    JoinArgs j{};
    int64_t total = 0;
    bool any = false;
    HeadsView din[2], x[2], dx[2];
    for (int i = 0; i < n_groups; ++i) {
      const muon_heads_grad_t& g = groups[i];
      if (g.heads < 1 || g.heads > (1 << 20) || g.reserved != 0)
        return fail_with(MUON_ERR_INVALID, "heads must be in [1, 2^20] and reserved 0");
      if (g.param) {
        if (!norm) return fail_with(MUON_ERR_INVALID, "a param without norm");
        if (int64_t(g.param->rows) * g.param->cols != head_dim)
          return fail_with(MUON_ERR_INVALID, "a param must have head_dim elements");
        if ((rc = lay::place_param(*g.param, accum, accum_elems, parts, nparts, &sg[i])) != MUON_OK) return rc;
        if (i == 1 && groups[0].param && lay::flat_overlap(*groups[0].param, *g.param))
          return fail_with(MUON_ERR_INVALID, "the two params overlap");
        a.want[i] = j.want[i] = 1;
        any = true;
      }
      if (n_tokens == 0) continue;
      if ((rc = check_heads(g.dout, g.dout_stride, g.dout_head_stride, n_tokens, g.heads, head_dim, es, false,
                            "dout")) ||
          (norm && (rc = check_heads(g.x, g.x_stride, g.x_head_stride, n_tokens, g.heads, head_dim, es, false,
                                     "x"))) ||
          (rc = check_heads(g.dx, g.dx_stride, g.dx_head_stride, n_tokens, g.heads, head_dim, es, true, "dx")))
        return rc;
      if (misaligned(g.weight, es)) return fail_with(MUON_ERR_INVALID, "weight is not aligned to its type");
      const void* xp = norm ? g.x : nullptr;
      din[i] = {g.dout, g.dout_stride, g.dout_head_stride, n_tokens, g.heads, head_dim, es};
      x[i] = {xp, g.x_stride, g.x_head_stride, n_tokens, g.heads, head_dim, es};
      dx[i] = {g.dx, g.dx_stride, g.dx_head_stride, n_tokens, g.heads, head_dim, es};
      a.group[i] = {{g.dout, g.dout_stride, g.dout_head_stride}, {xp, g.x_stride, g.x_head_stride},
                    {g.dx, g.dx_stride, g.dx_head_stride}, norm ? g.weight : nullptr, g.heads};
      total += g.heads;
    }
    const int blocks = n_tokens ? grad_blocks(n_tokens) : 0;
    const size_t need = any ? size_t(blocks) * 2 * head_dim * sizeof(float) : 0;
    if (need && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
      return fail_with(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
    if (n_tokens * total > (int64_t(1) << 33))
      return fail_with(MUON_ERR_UNSUPPORTED, "too many heads for one launch");
    const Span pos(positions, pairs ? n_tokens : 0, axes, axes, a.pos64 ? 8 : 4);
    const Span work(workspace, need ? 1 : 0, int64_t(need), int64_t(need), 1);
    const Span sums(accum, any ? 1 : 0, accum_elems, accum_elems, 4);
    if (work.meets(sums) || work.meets(pos) || sums.meets(pos))
      return fail_with(MUON_ERR_INVALID, "workspace, accum and positions overlap");
    for (int i = 0; n_tokens && i < n_groups; ++i) {
      for (int k = 0; k < n_groups; ++k) {
        auto in_place = [&](const HeadsView& v) {
          return i == k && v.p == dx[i].p && v.stride == dx[i].stride && v.head == dx[i].head;
        };
        if ((!in_place(din[k]) && !apart(din[k], dx[i])) || (!in_place(x[k]) && !apart(x[k], dx[i])) ||
            (k != i && !apart(dx[k], dx[i])))
          return fail_with(MUON_ERR_INVALID, "a dx overlaps another tensor, or its dout or x in another layout");
        const Span w(a.group[k].weight, 1, head_dim, head_dim, es);
        if (dx[i].span().meets(w) || work.meets(w) || sums.meets(w))
          return fail_with(MUON_ERR_INVALID, "a weight overlaps what is written");
      }
      for (const Span& v : {din[i].span(), x[i].p ? x[i].span() : Span(), dx[i].span()})
        if (v.meets(work) || v.meets(sums))
          return fail_with(MUON_ERR_INVALID, "workspace or accum overlaps a tensor of heads");
      if (dx[i].span().meets(pos)) return fail_with(MUON_ERR_INVALID, "a dx overlaps the positions");
    }
    if (n_tokens == 0 && !(any && overwrite)) return MUON_OK;
    if ((rc = lay::begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (n_tokens) {
      a.partial = static_cast<float*>(workspace);
      e = es == 2 ? launch_rotary_grad<__nv_bfloat16>(a, norm, blocks, s)
                  : launch_rotary_grad<float>(a, norm, blocks, s);
      if (e != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
    }
    if (any) {
      j.partial = static_cast<const float*>(workspace);
      j.blocks = blocks;
      j.dim = head_dim;
      j.accum = accum;
      j.scale = scale;
      j.overwrite = overwrite;
      e = launch(k_norm_join, unsigned(2 * ((head_dim + 31) / 32)), 32 * kJoinWarps, 1, false, s, 0, j, sg[0], sg[1]);
      ++launches;
    }
    return lay::end_call(launches, e);
  });
}
