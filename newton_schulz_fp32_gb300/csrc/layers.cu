// Dropout from a counter, and the norm and rotation of query and key heads
// with its gradients.  Both are bound by memory: every element is read once
// and written once.
#include <type_traits>

#include "layers.cuh"

namespace muon {
namespace {

using tok::Vec;
using lay::Draw;
using lay::Dropout;
using lay::Span;

constexpr int kSms = 152;

// ------------------------------------------------------------------ dropout

constexpr int kDropThreads = 128;

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

// blockDim.x threads along a row, eight columns (one draw of 128 bits) each.  Bound
// by memory: 16384 x 4096 bf16 with a residual in 61 us, 6.6 TB/s of reads and
// writes; issue slots are 56% busy behind it.  One row per thread and blocks of 128
// threads were the best of a sweep (65 us then; two rows 84, four 121; 256 threads 72).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const DropArgs a) {
  tok::wait_before();
  tok::allow_next();
  Draw draw;
  draw.init(a.d);
  const int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (r >= a.rows) return;
  const int groups = (a.cols + 7) / 8;
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    const int c = g * 8, left = a.cols - c;
    float f[8], add[8];
    load8<T, VEC>(static_cast<const T*>(a.x) + r * a.xs + c, left, f);
    if (a.residual) load8<T, VEC>(static_cast<const T*>(a.residual) + r * a.rs + c, left, add);
    if (a.d.least) {
      const uint4 w = draw.at(uint32_t(r), g, a.d.site);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = lay::dropped(f[j], lay::draw_of(w, j), a.d);
    }
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += add[j];
    }
    store8<T, VEC>(static_cast<T*>(a.out) + r * a.os + c, left, f);
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
  const unsigned grid = unsigned((a.rows + block.y - 1) / block.y);
  return launch(vec ? k_dropout<T, true> : k_dropout<T, false>, grid, block, 1, true, s, 0, a);
}

// ------------------------------------------------------------------ norm and rotation
//
// For a head x with weight w, position p and frequencies f:
//     n = x / sqrt(mean x^2 + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin) with the angle p f.
// Both directions are bound by memory, each element moved once (16384 tokens of 40
// heads of 128 bf16: 57 us, 5.9 TB/s; the gradients 103 us, 4.9 TB/s, issue slots 60%
// busy), and short of it by latency: 16 warps per SM hold what is on its way in
// registers.

constexpr int kMaxPairs = MUON_MAX_HEAD_DIM / 2;
constexpr int kRotWarps = 8;
constexpr int kGradBlocks = 2 * kSms;   // most blocks of the gradient, each with its own partial sums

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

// How a head is laid over lanes.  A unit is P pairs (elements of both halves, or
// 2 P neighbours if interleaved), or 2 P elements behind the pairs; a lane has NU
// units.  P = 4 and 2 need accesses of P and 2 P elements aligned (see wide()).
template <int P_, int NU_, bool FIXED_, bool NORM_, bool INTER_>
struct Shape {
  static constexpr int P = P_, NU = NU_;
  // Norm and order of pairs known when compiled, and every lane with a turned unit (all
  // of a head is turned, and it is a power of two long).
  static constexpr bool kFixed = FIXED_;
  static __device__ __forceinline__ bool norm(int n) { return kFixed ? NORM_ : n != 0; }
  static __device__ __forceinline__ bool inter(int i) { return kFixed ? INTER_ : i != 0; }
};

struct RotArgs {
  Group group[2];
  int groups;
  int64_t n;
  int dim, pairs, axes, norm, interleaved, pos64;
  float eps, inv_dim;
  const void* positions;
  float* partial;              // the gradient: [block][group][dim]
  int want[2];                 // groups whose weight's gradient is wanted
  int split, share;            // pieces a token's heads (of both groups, one after the other) are cut into, and heads in a piece
  uint64_t turns[kMaxPairs];   // turns per position, in units of 2^-64
  uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ int64_t position(const RotArgs& a, int64_t t, int axis) {
  const int64_t i = t * a.axes + axis;
  return a.pos64 ? reinterpret_cast<const int64_t*>(a.positions)[i]
                 : reinterpret_cast<const int32_t*>(a.positions)[i];
}

// A token's position on axis `lane`; 0 behind the axes (of which there are none without positions).
__device__ __forceinline__ int64_t lane_position(const RotArgs& a, int64_t t, int lane) {
  return lane < a.axes ? position(a, t, lane) : 0;
}

// cos and sin of a pair's angle: position * turns wraps at whole turns by itself;
// its upper 32 bits, as a signed fraction, are the angle in half turns / 2^31.
__device__ __forceinline__ void angle(int64_t pos, uint64_t turns, float* c, float* s) {
  const uint64_t whole = uint64_t(pos) * turns;
  const float half_turns = float(int32_t((whole + 0x80000000u) >> 32)) * 4.656612873077393e-10f;
  sincospif(half_turns, s, c);
}

// P elements as they lie in memory.  P > 1: one access, always (what a lane has no
// part in is not added up or stored); P = 1: 0 where n is 0.
template <typename T, int P>
struct Part {
  static constexpr int kBytes = P * int(sizeof(T));
  using Raw = std::conditional_t<kBytes == 16, uint4, std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;
  Raw raw;
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (P == 1) {
      raw = Raw{};
      if (n) raw = *reinterpret_cast<const Raw*>(p);
    } else {
      raw = *reinterpret_cast<const Raw*>(p);
    }
  }
  __device__ __forceinline__ void to(float* f) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = __uint_as_float(u[i]);
    } else if constexpr (P == 1) {
      f[0] = __uint_as_float(uint32_t(raw) << 16);
    } else {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) Vec<T>::unpack2(u[i], f + 2 * i);
    }
  }
  __device__ __forceinline__ void from(const float* f) {
    if constexpr (sizeof(T) == 4) {
      uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < P; ++i) u[i] = __float_as_uint(f[i]);
    } else if constexpr (P == 1) {
      const __nv_bfloat16 h = __float2bfloat16_rn(f[0]);
      raw = *reinterpret_cast<const uint16_t*>(&h);
    } else {
      uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) u[i] = Vec<T>::pack2(f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void store(T* p, int n) const {
    if (n) *reinterpret_cast<Raw*>(p) = raw;
  }
};

// A lane's units of a head as pairs: f[2 k] and f[2 k + 1] are pair k's two
// elements (of what is not turned, any two).
template <typename T, class S>
__device__ __forceinline__ void to_pairs(const Part<T, S::P>& a, const Part<T, S::P>& b, bool inter, float* f) {
  constexpr int P = S::P;
  float x[2 * P];
  a.to(x);
  b.to(x + P);
#pragma unroll
  for (int k = 0; k < P; ++k) {
    f[2 * k] = inter ? x[2 * k] : x[k];
    f[2 * k + 1] = inter ? x[2 * k + 1] : x[P + k];
  }
}

template <typename T, class S>
__device__ __forceinline__ void from_pairs(Part<T, S::P>& a, Part<T, S::P>& b, bool inter, const float* f) {
  constexpr int P = S::P;
  float x[2 * P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    x[inter ? 2 * k : k] = f[2 * k];
    x[inter ? 2 * k + 1 : P + k] = f[2 * k + 1];
  }
  a.from(x);
  b.from(x + P);
}

// How fast pairs turn and by which axis, in shared memory (lanes that read
// different kernel arguments wait for one another).
struct Turns {
  uint64_t turns[kMaxPairs];
  uint8_t axis[kMaxPairs];
  __device__ __forceinline__ void init(const RotArgs& a) {
    for (int i = threadIdx.x; i < a.pairs; i += blockDim.x) {
      turns[i] = a.turns[i];
      axis[i] = a.axis[i];
    }
    if (!a.pairs && threadIdx.x == 0) axis[0] = 0;
    __syncthreads();
  }
};

// What a lane keeps over all tokens: where its units lie.
template <class S>
struct Units {
  static constexpr int P = S::P, NU = S::NU;
  __device__ __forceinline__ bool turns(int u) const { return S::kFixed || turned[u]; }
  __device__ __forceinline__ int first_half(int u) const { return S::kFixed ? P : na[u]; }
  __device__ __forceinline__ int second_half(int u) const { return S::kFixed ? P : nb[u]; }
  int at[NU], gap[NU];     // first element, and how far behind it the other P are
  int na[NU], nb[NU];      // how many there are of either
  bool turned[NU];
  int pair[NU];            // the first

  __device__ __forceinline__ void init(const RotArgs& a, int in_head, int lanes) {
    const int whole = a.pairs / P;
    const bool inter = S::inter(a.interleaved);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int unit = in_head + u * lanes;
      turned[u] = unit < whole;
      if (turned[u]) {
        at[u] = inter ? unit * 2 * P : unit * P;
        gap[u] = inter ? P : a.pairs;
        na[u] = nb[u] = P;
      } else {
        at[u] = 2 * a.pairs + (unit - whole) * 2 * P;
        gap[u] = P;
        na[u] = max(0, min(P, a.dim - at[u]));
        nb[u] = max(0, min(P, a.dim - at[u] - P));
        if (P > 1 && !na[u]) at[u] = 0;   // a lane without a unit reads along with the first
      }
      pair[u] = unit * P;
    }
  }
  // position: lane x holds the token's position on axis x.
  __device__ __forceinline__ void turn_by(const Turns& q, int64_t position, float (&c)[NU][P], float (&s)[NU][P]) const {
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int i = turned[u] ? pair[u] + k : 0;
        const int64_t at = __shfl_sync(0xffffffffu, position, q.axis[i]);
        c[u][k] = 1.f;
        s[u][k] = 0.f;
        if (turned[u]) angle(at, q.turns[i], &c[u][k], &s[u][k]);
      }
  }
  // The weight's elements, as pairs.
  template <typename T>
  __device__ __forceinline__ void weights(const RotArgs& a, const void* p, float (&w)[NU][2 * P]) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) w[u][k] = 1.f;
      if (!p || !na[u]) continue;
      Part<T, P> x, y;
      x.load(static_cast<const T*>(p) + at[u], na[u]);
      y.load(static_cast<const T*>(p) + at[u] + gap[u], nb[u]);
      to_pairs<T, S>(x, y, turned[u] && S::inter(a.interleaved), w[u]);
    }
  }
};

// Sums over the `lanes` lanes that hold a head, of several heads at once.
template <int U>
__device__ __forceinline__ void head_sums(float (&v)[U], int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Where a warp is in its work: tokens (or pieces of their heads), in each the two
// groups, in each batches of heads.  What comes next is fetched before what is
// there is worked on, across batches, groups and tokens (16384 tokens of 40
// heads, when that was the last step: 64 us against 70 with a fresh start at each
// token and group).
struct Cursor {
  int64_t task, t;
  int which, h0, h1;   // group, and its heads in this piece
  int left;            // heads from this lane's on
  bool first;          // of its token

  __device__ __forceinline__ bool valid(const RotArgs& a) const { return task < a.n * a.split; }
  // The group's range of heads in the piece; false if it has none.
  __device__ __forceinline__ bool range(const RotArgs& a, int in_step) {
    const int piece = a.split == 1 ? 0 : static_cast<int>(task - t * a.split);
    const int before = which ? a.group[0].heads : 0;
    h0 = max(0, piece * a.share - before);
    h1 = min(a.group[which].heads, (piece + 1) * a.share - before);
    left = h1 - h0 - in_step;
    return h0 < h1;
  }
  __device__ __forceinline__ void start(const RotArgs& a, int64_t at, int in_step) {
    task = at;
    t = a.split == 1 ? task : task / a.split;
    which = 0;
    first = true;
    if (!range(a, in_step)) {   // a piece of the second group alone
      which = 1;
      range(a, in_step);
    }
  }
  // The next batch of `heads` heads.
  __device__ __forceinline__ void next(const RotArgs& a, int heads, int in_step) {
    first = false;
    left -= heads;
    if (left + in_step > 0) return;
    if (which + 1 < a.groups) {
      which = 1;
      if (range(a, in_step)) return;
    }
    start(a, task + int64_t(gridDim.x) * kRotWarps, in_step);
  }
};

// A warp takes a token's heads, both groups', or a piece of them where tokens are
// few; `lanes` lanes hold a head, 32 / lanes heads go at once and U of those are
// under way.  What a token's pairs are multiplied by, cosines and sines with the
// weight in them, stays in registers over its heads.
template <typename T, class S>
__global__ void __launch_bounds__(32 * kRotWarps, 2) k_norm_rotary(const __grid_constant__ RotArgs a, int lanes) {
  constexpr int P = S::P, NU = S::NU, U = NU > 1 ? 1 : P == 4 ? 4 : 2;
  const int lane = threadIdx.x % 32, first = lane / lanes, step = 32 / lanes;
  const bool inter = S::inter(a.interleaved);
  __shared__ Turns turns;
  turns.init(a);
  Units<S> units;
  units.init(a, lane % lanes, lanes);
  tok::wait_before();
  tok::allow_next();
  Part<T, P> nx[U][NU], ny[U][NU];   // heads on their way
  int64_t position = 0;              // of the token on its way
  auto fetch = [&](const Cursor& c) {
    const Group& g = a.group[c.which];
    const T* base = static_cast<const T*>(g.in.p) + c.t * g.in.stride + (c.h1 - first - c.left) * g.in.head;
    const T* in = base + first * g.in.head;
    if (c.first) position = lane_position(a, c.t, lane);
#pragma unroll
    for (int v = 0; v < U; ++v, in += step * g.in.head) {
      const T* head = v * step < c.left ? in : base;   // behind the last head: one that is there
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const T* q = head + units.at[u];
        nx[v][u].load(q, units.first_half(u));
        ny[v][u].load(q + units.gap[u], units.second_half(u));
      }
    }
  };
  Cursor now, then;
  then.start(a, int64_t(blockIdx.x) * kRotWarps + threadIdx.x / 32, first);
  if (!then.valid(a)) return;
  fetch(then);
  float c[NU][P], s[NU][P];
  float ac[NU][P], bs[NU][P], bc[NU][P], as[NU][P];   // (a, b) -> r (a ac - b bs, b bc + a as)
  bool on = true;
  do {
    now = then;
    const int64_t here = position;
    Part<T, P> x[U][NU], y[U][NU];
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        x[v][u] = nx[v][u];
        y[v][u] = ny[v][u];
      }
    then.next(a, U * step, first);
    if (then.valid(a)) fetch(then);
    const Group& g = a.group[now.which];
    T* out = static_cast<T*>(const_cast<void*>(g.out.p)) + now.t * g.out.stride + (now.h1 - now.left) * g.out.head;
    if (now.first) {
      on = __all_sync(0xffffffffu, here >= 0);
      units.turn_by(turns, here, c, s);
    }
    if (!on) {   // the warp's
#pragma unroll
      for (int v = 0; v < U; ++v, out += step * g.out.head)
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const Part<T, P> zero{};
          zero.store(out + units.at[u], v * step < now.left ? units.first_half(u) : 0);
          zero.store(out + units.at[u] + units.gap[u], v * step < now.left ? units.second_half(u) : 0);
        }
      continue;
    }
    if (now.first || now.left + first == now.h1 - now.h0) {
      float w[NU][2 * P];
      units.template weights<T>(a, g.weight, w);
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          ac[u][k] = w[u][2 * k] * c[u][k];
          as[u][k] = w[u][2 * k] * s[u][k];
          bc[u][k] = w[u][2 * k + 1] * c[u][k];
          bs[u][k] = w[u][2 * k + 1] * s[u][k];
        }
    }
    float r[U];
    if (S::norm(a.norm)) {
#pragma unroll
      for (int v = 0; v < U; ++v) {
        r[v] = 0.f;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          float f[2 * P];
          x[v][u].to(f);
          y[v][u].to(f + P);
#pragma unroll
          for (int k = 0; k < 2 * P; ++k) r[v] += f[k] * f[k];
        }
        if (P > 1 && !units.first_half(0)) r[v] = 0.f;   // (NU is 1)
      }
      head_sums<U>(r, lanes);
#pragma unroll
      for (int v = 0; v < U; ++v) r[v] = rsqrtf(r[v] * a.inv_dim + a.eps);
    } else {
#pragma unroll
      for (int v = 0; v < U; ++v) r[v] = 1.f;
    }
#pragma unroll
    for (int v = 0; v < U; ++v, out += step * g.out.head) {
      if (v * step >= now.left) continue;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const bool in_pairs = units.turns(u) && inter;
        float f[2 * P], o[2 * P];
        to_pairs<T, S>(x[v][u], y[v][u], in_pairs, f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          o[2 * k] = r[v] * (f[2 * k] * ac[u][k] - f[2 * k + 1] * bs[u][k]);
          o[2 * k + 1] = r[v] * (f[2 * k + 1] * bc[u][k] + f[2 * k] * as[u][k]);
        }
        if (!units.turns(u)) {   // neighbours, not a pair: an infinite one leaves the other alone
#pragma unroll
          for (int k = 0; k < P; ++k) {
            o[2 * k] = r[v] * (f[2 * k] * ac[u][k]);
            o[2 * k + 1] = r[v] * (f[2 * k + 1] * bc[u][k]);
          }
        }
        Part<T, P> p, q;
        from_pairs<T, S>(p, q, in_pairs, o);
        T* to = out + units.at[u];
        p.store(to, units.first_half(u));
        q.store(to + units.gap[u], units.second_half(u));
      }
    }
  } while (then.valid(a));
}

// The gradient: g = dout turned back; with r = 1 / rms and n = x r,
//     dw += g n,   dx = r (g w - n mean(g w n)).
// A lane keeps its columns' dw over all tokens of its warp; blocks leave
// partial sums, which k_norm_join adds in order.  (Fetching ahead across tokens, as
// k_norm_rotary does, took longer here: 8% with the groups one after the other, 30%
// with sums of both chosen from.)
template <typename T, class S>
__global__ void __launch_bounds__(32 * kRotWarps, 2) k_norm_rotary_grad(const __grid_constant__ RotArgs a, int lanes) {
  constexpr int P = S::P, NU = S::NU, U = NU > 1 ? 1 : 2;
  __shared__ float sums[kRotWarps][MUON_MAX_HEAD_DIM];
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32, first = lane / lanes, step = 32 / lanes;
  const bool inter = S::inter(a.interleaved);
  __shared__ Turns turns;
  turns.init(a);
  Units<S> units;
  units.init(a, lane % lanes, lanes);
  tok::wait_before();
  tok::allow_next();
  float dw[2][NU][2 * P] = {};
  const int64_t tasks = a.n * a.split;
  for (int64_t task = int64_t(blockIdx.x) * kRotWarps + warp; task < tasks; task += int64_t(gridDim.x) * kRotWarps) {
    const int64_t t = a.split == 1 ? task : task / a.split;
    const int piece = a.split == 1 ? 0 : static_cast<int>(task - t * a.split);
    const int64_t position = lane_position(a, t, lane);
    const bool on = __all_sync(0xffffffffu, position >= 0);
    float c[NU][P], s[NU][P];
    units.turn_by(turns, position, c, s);
#pragma unroll
    for (int which = 0; which < 2; ++which) {   // unrolled: dw stays in registers
      const Group& g = a.group[which];
      const int before = which ? a.group[0].heads : 0;
      const int h0 = max(0, piece * a.share - before), h1 = min(g.heads, (piece + 1) * a.share - before);
      if (which >= a.groups || h0 >= h1) continue;
      float w[NU][2 * P];
      units.template weights<T>(a, g.weight, w);
      const int64_t dby = g.in.head * step, xby = g.x.head * step, oby = g.out.head * step;
      const T* dbase = static_cast<const T*>(g.in.p) + t * g.in.stride + h0 * g.in.head;   // for what is behind the last head
      const T* xbase = static_cast<const T*>(g.x.p) + t * g.x.stride + h0 * g.x.head;
      const T *din = dbase + first * g.in.head, *xin = xbase + first * g.x.head;
      T* out = static_cast<T*>(const_cast<void*>(g.out.p)) + t * g.out.stride + (h0 + first) * g.out.head;
      Part<T, P> p[U][NU], q[U][NU], y[U][NU], z[U][NU];   // heads on their way
      auto fetch = [&](int left) {
#pragma unroll
        for (int v = 0; v < U; ++v, din += dby, xin += xby) {
          const bool here = v * step < left;
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            const T* i = (here ? din : dbase) + units.at[u];
            p[v][u].load(i, units.first_half(u));
            q[v][u].load(i + units.gap[u], units.second_half(u));
            if (S::norm(a.norm)) {
              i = (here ? xin : xbase) + units.at[u];
              y[v][u].load(i, units.first_half(u));
              z[v][u].load(i + units.gap[u], units.second_half(u));
            }
          }
        }
      };
      fetch(h1 - h0 - first);
#pragma unroll 1
      for (int left = h1 - h0 - first; left + first > 0; left -= U * step) {
        float d[U][NU][2 * P], x[U][NU][2 * P];
        {
#pragma unroll
          for (int v = 0; v < U; ++v)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              const bool in_pairs = units.turns(u) && inter;
              float f[2 * P];
              to_pairs<T, S>(p[v][u], q[v][u], in_pairs, f);
#pragma unroll
              for (int k = 0; k < P; ++k) {
                d[v][u][2 * k] = f[2 * k] * c[u][k] + f[2 * k + 1] * s[u][k];
                d[v][u][2 * k + 1] = f[2 * k + 1] * c[u][k] - f[2 * k] * s[u][k];
              }
              if (!units.turns(u)) {
#pragma unroll
                for (int k = 0; k < 2 * P; ++k) d[v][u][k] = f[k];
              }
              if (S::norm(a.norm)) to_pairs<T, S>(y[v][u], z[v][u], in_pairs, x[v][u]);
            }
        }
        if (left + first > U * step) fetch(left - U * step);
        if (S::norm(a.norm)) {
          float r[U], m[U];
#pragma unroll
          for (int v = 0; v < U; ++v) {
            r[v] = m[v] = 0.f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
              for (int k = 0; k < 2 * P; ++k) {
                r[v] += x[v][u][k] * x[v][u][k];
                m[v] += x[v][u][k] * (d[v][u][k] * w[u][k]);
              }
            if (P > 1 && !units.first_half(0)) r[v] = m[v] = 0.f;   // (NU is 1)
          }
          head_sums<U>(r, lanes);
          head_sums<U>(m, lanes);
#pragma unroll
          for (int v = 0; v < U; ++v) {
            r[v] = rsqrtf(r[v] * a.inv_dim + a.eps);
            m[v] = m[v] * r[v] * a.inv_dim;   // mean of g w n
            const bool counts = on && v * step < left;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
              for (int k = 0; k < 2 * P; ++k) {
                const float n = x[v][u][k] * r[v];
                if (counts) dw[which][u][k] += d[v][u][k] * n;
                d[v][u][k] = r[v] * (d[v][u][k] * w[u][k] - n * m[v]);
              }
          }
        }
#pragma unroll
        for (int v = 0; v < U; ++v, out += oby) {
          if (v * step >= left) continue;
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            Part<T, P> i, j;
            from_pairs<T, S>(i, j, units.turns(u) && inter, d[v][u]);
            if (!on) i = j = Part<T, P>{};
            T* to = out + units.at[u];
            i.store(to, units.first_half(u));
            j.store(to + units.gap[u], units.second_half(u));
          }
        }
      }
    }
  }
  if (!S::norm(a.norm)) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!a.want[which]) continue;
    // lanes of the same columns, then the block's warps
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const bool in_pairs = units.turns(u) && inter;
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) {
        float v = dw[which][u][k];
        for (int o = lanes; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        // the k-th of the lane's values is one of pair k / 2
        const int j = in_pairs ? k : k % 2 * P + k / 2, i = units.at[u] + (j < P ? j : units.gap[u] + (j - P));
        const bool there = j < P ? j < units.first_half(u) : j - P < units.second_half(u);
        if (first == 0 && there) sums[warp][i] = v;
      }
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
  tok::wait_before();
  tok::allow_next();
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

// Blocks of the gradient: all of them from 64 tokens on (a token's heads are then cut into pieces).
int grad_blocks(int64_t n) { return static_cast<int>(std::min<int64_t>(kGradBlocks, 5 * n)); }

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
  a->norm = norm;
  a->eps = eps;
  a->inv_dim = 1.f / float(head_dim);
  a->interleaved = interleaved;
  if (!pairs && !positions) return MUON_OK;
  if (positions_type != MUON_INDEX_INT32 && positions_type != MUON_INDEX_INT64)
    return fail_with(MUON_ERR_INVALID, "unknown positions_type");
  if (axes < 1 || axes > MUON_MAX_AXES) return fail_with(MUON_ERR_INVALID, "axes must be in [1, MUON_MAX_AXES]");
  if (n_tokens > 0 && (!positions || misaligned(positions, positions_type == MUON_INDEX_INT64 ? 8 : 4)))
    return fail_with(MUON_ERR_INVALID, "positions is NULL or misaligned");
  if (pairs && !inv_freq) return fail_with(MUON_ERR_INVALID, "inv_freq is NULL");
  a->positions = positions;
  a->pos64 = positions_type == MUON_INDEX_INT64;
  a->axes = axes;
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(inv_freq[i])) return fail_with(MUON_ERR_INVALID, "inv_freq must be finite");
    if (axis && (axis[i] < 0 || axis[i] >= axes)) return fail_with(MUON_ERR_INVALID, "axis must be in [0, axes)");
    // turns per position, of which the whole ones do not matter; those of a pair that turns backwards are taken from a
    // whole turn in fixed point, where a small one's last bits stay
    const double turns = std::fabs(inv_freq[i]) / 6.283185307179586476925;
    const uint64_t part = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));   // below 2^64: turns is not
    a->turns[i] = inv_freq[i] < 0 ? ~part + 1 : part;                                         // below 0
    a->axis[i] = static_cast<uint8_t>(axis ? axis[i] : 0);
  }
  return MUON_OK;
}

// Whether units of `per` pairs fit: every access of a unit aligned (neighbours go
// as two accesses, so rows on `per` elements are enough), and neither the
// pairs nor what is behind them ending inside a unit.
bool fits(const RotArgs& a, int per, size_t es) {
  const int64_t unit = per * int64_t(es);
  auto on = [&](const Heads& h) {
    return !h.p || (!misaligned(h.p, unit) && h.stride * int64_t(es) % unit == 0 && h.head * int64_t(es) % unit == 0);
  };
  if (a.pairs % per || (a.dim - 2 * a.pairs) % (2 * per)) return false;
  for (int i = 0; i < a.groups; ++i)
    if (!on(a.group[i].in) || !on(a.group[i].x) || !on(a.group[i].out) || misaligned(a.group[i].weight, unit))
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
// SMs with a warp each (pieces of at least `least` heads).
void split_heads(RotArgs* a, int least) {
  int64_t total = 0;
  for (int i = 0; i < a->groups; ++i) total += a->group[i].heads;
  int64_t share = std::max<int64_t>(least, std::min<int64_t>(total, total * a->n / (24 * kSms)));
  share = (share + least - 1) / least * least;
  a->share = static_cast<int>(share);
  a->split = static_cast<int>((total + share - 1) / share);
}

// Four pairs to a unit, two where four do not fit (heads of up to 128 elements: 32
// lanes), else one.
template <typename T, template <typename, class> class KERNEL>
cudaError_t launch_heads(RotArgs& a, int blocks, cudaStream_t s) {
  const int per = fits(a, 4, sizeof(T)) ? 4 : fits(a, 2, sizeof(T)) && a.dim <= 128 ? 2 : 1;
  const int lanes = lanes_of(a, per);
  split_heads(&a, 32 / lanes);
  const bool whole = a.norm && 2 * a.pairs == a.dim && lanes * 8 == a.dim;
  void (*k)(RotArgs, int) = KERNEL<T, Shape<1, 4, false, false, false>>::kernel;
  if (per == 2) k = KERNEL<T, Shape<2, 1, false, false, false>>::kernel;
  else if (per == 4 && whole && a.interleaved) k = KERNEL<T, Shape<4, 1, true, true, true>>::kernel;
  else if (per == 4 && whole) k = KERNEL<T, Shape<4, 1, true, true, false>>::kernel;
  else if (per == 4) k = KERNEL<T, Shape<4, 1, false, false, false>>::kernel;
  if (!blocks) blocks = int(std::min<int64_t>((a.n * a.split + kRotWarps - 1) / kRotWarps, 2 * kSms));
  return launch(k, unsigned(blocks), 32 * kRotWarps, 1, true, s, 0, a, lanes);
}

template <typename T, class S>
struct There {
  static constexpr auto kernel = k_norm_rotary<T, S>;
};

template <typename T, class S>
struct Back {
  static constexpr auto kernel = k_norm_rotary_grad<T, S>;
};

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
    const Span pos(a.positions, n_tokens, a.axes, a.axes, a.pos64 ? 8 : 4);
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
    return lay::end_call(1, es == 2 ? launch_heads<__nv_bfloat16, There>(a, 0, s) : launch_heads<float, There>(a, 0, s));
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
    const Span pos(a.positions, n_tokens, a.axes, a.axes, a.pos64 ? 8 : 4);
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
      e = es == 2 ? launch_heads<__nv_bfloat16, Back>(a, blocks, s) : launch_heads<float, Back>(a, blocks, s);
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
      e = launch(k_norm_join, unsigned(2 * ((head_dim + 31) / 32)), 32 * kJoinWarps, 1, true, s, 0, j, sg[0], sg[1]);
      ++launches;
    }
    return lay::end_call(launches, e);
  });
}
