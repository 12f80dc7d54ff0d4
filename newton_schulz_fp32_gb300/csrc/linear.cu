// A dense layer: the product of tokens and weight with bias, activation,
// dropout and residual, and its gradients: dx through the activation before the
// layer, and the weight's and bias's summed straight into the flat,
// partitioned FP32 accumulation buffer.
//
//     u = x W^T + b,  out = residual + drop(act(u));
//     dx = (d W) act'(pre),  accum[W] (+)= s d^T x,  accum[b] (+)= s sum d.
//
// All three products are bf16 x bf16 with FP32 sums on the tensor cores; an
// operand is read as it lies, with its k contiguous or its rows.  Which kernel
// takes a product is a matter of its sizes (offers_of, plan_few, takes_rows):
//   k_linear_pair   tiles of 256 x 256 or 256 x 128 on pairs of SMs, persistent.
//                   Bound by the tensor cores (92% active): 8192 x 4096 -> 14336 in
//                   495 us, 1945 TFLOP/s, as fast as the library's product alone;
//                   in long runs by the power limit (604 us with silu and its
//                   argument kept).
//   k_linear_split  tiles of 128 x 128 on single SMs, the K blocks shared out in a
//                   cluster, for products of few tiles; tiles of 128 features x
//                   32 or 64 tokens for few tokens (4096 -> 14336, 32 tokens 23 us,
//                   5.1 TB/s of weight).
//   k_linear_rows   one or two tokens (up to four of a small weight): multiply-adds
//                   over the weight's rows (one token through 4096 -> 14336 20 us,
//                   5.8 TB/s).
//   k_linear_pack   operands whose rows do not start on 16 bytes, copied first.
//   k_bias_grad     sums of dout's columns.
#include <type_traits>

#include "layers.cuh"
#include "tc_common.cuh"

namespace muon {
namespace {

using lay::Draw;
using lay::Dropout;
using lay::Span;
using namespace tc;

__device__ int g_linear_err;

// The kernels of one call follow one another by programmatic launch.  The first
// waits for what was in the stream before it, and lets the next one start; one
// that needs nothing of the kernels before it in the call (late) runs beside them
// and waits for them only at its end, so that what comes after the call waits for
// all of it.
__device__ __forceinline__ void begin_kernel(int late) {
  if (!late) tok::wait_before();
  tok::allow_next();
}
__device__ __forceinline__ void end_kernel(int late) {
  if (late) tok::wait_before();
}

// ------------------------------------------------------------------ epilogues
//
// A warp takes a chunk of 32 rows x 32 columns of the result.  Its lane has, in
// turn, eight consecutive columns of row 8 i + lane / 4, i = 0 .. 3: 16 bytes of
// bf16 and the eight elements that one draw of dropout serves.  What is added to
// the chunk or multiplies it (residual, argument of the activation) is fetched
// ahead by asynchronous copies into slots of the lane's own.

constexpr int kSlotBytes = 4096;    // a warp's slots: a chunk of FP32, or two of bf16
constexpr int kChunkBytes = 4096;   // a chunk of FP32 sums

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint4 slot16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// A chunk of sums in shared memory: 32 rows of 128 bytes, their 16-byte pieces
// exchanged by the row's low bits, so that neither a lane's row nor eight lanes'
// pieces meet in a bank.
__device__ __forceinline__ uint32_t piece(int row, int granule) {
  return uint32_t(row) * 128u + (uint32_t(granule ^ (row & 7)) << 4);
}

__device__ __forceinline__ float at_column(uint32_t stage, int row, int lane) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(stage + piece(row, lane >> 2) + (lane & 3) * 4) : "memory");
  return x;
}
__device__ __forceinline__ void put_column(uint32_t stage, int row, int lane, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + piece(row, lane >> 2) + (lane & 3) * 4), "f"(x) : "memory");
}

// A matrix that is read or written beside the sums.
struct Matrix {
  void* p;
  int64_t stride;
  int fp32;
  int wide;   // every row starts on 16 bytes

  __device__ __forceinline__ char* at(int64_t r, int64_t c) const {
    return static_cast<char*>(p) + (r * stride + c) * (fp32 ? 4 : 2);
  }
  __device__ __forceinline__ int64_t step() const { return 8 * stride * (fp32 ? 4 : 2); }   // bytes between the lane's rows
  // The lane's eight elements at q, `left` of them inside the row.
  __device__ __forceinline__ void load(const char* q, int left, float* f) const {
    if (fp32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = j < left ? reinterpret_cast<const float*>(q)[j] : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = j < left ? tok::to_float(reinterpret_cast<const __nv_bfloat16*>(q)[j]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(char* q, int left, const float* f) const {
    if (wide && left >= 8) {
      uint4* u = reinterpret_cast<uint4*>(q);
      if (fp32) {
        u[0] = tok::Vec<float>::pack(f);
        u[1] = tok::Vec<float>::pack(f + 4);
      } else {
        u[0] = tok::Vec<__nv_bfloat16>::pack(f);
      }
    } else if (fp32) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) reinterpret_cast<float*>(q)[j] = f[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) reinterpret_cast<__nv_bfloat16*>(q)[j] = __float2bfloat16_rn(f[j]);
    }
  }
  // Fetches the lane's part of a chunk into its slots; bf16 chunks alternate
  // between two halves.
  __device__ __forceinline__ void fetch(uint32_t slots, int half, int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                        int lane) const {
    const int64_t c = c0 + (lane & 3) * 8, r = r0 + (lane >> 2);
    if (!wide || cols - c < 8) return;
    const char* q = at(r, c);
    const int64_t by = step();
#pragma unroll
    for (int i = 0; i < 4; ++i, q += by) {
      if (r + 8 * i >= rows) break;
      if (fp32) {
        copy16(slots + (2 * i) * 512 + lane * 16, q);
        copy16(slots + (2 * i + 1) * 512 + lane * 16, q + 16);
      } else {
        copy16(slots + half * 2048 + i * 512 + lane * 16, q);
      }
    }
  }
  // A whole chunk of rows that start anywhere, for a converged warp: a row of 32
  // elements at once (eight elements of four rows at once, as above, would be 32
  // pieces of memory to each access: 35 us instead of 9 for 1001 x 1001 -> 763).
  // raw: column c0 + lane of the rows, all of them on their way at once.
  __device__ __forceinline__ void load_column(int64_t r0, int64_t c0, int64_t rows, int64_t cols, int lane,
                                              float (&raw)[32]) const {
    const int here = c0 + lane < cols ? int(min(int64_t(32), rows - r0)) : 0;
    const char* q = at(r0, c0 + lane);
    const int64_t by = stride * (fp32 ? 4 : 2);
    if (fp32) {
#pragma unroll
      for (int r = 0; r < 32; ++r, q += by) raw[r] = r < here ? *reinterpret_cast<const float*>(q) : 0.f;
    } else {
#pragma unroll
      for (int r = 0; r < 32; ++r, q += by)
        raw[r] = r < here ? tok::to_float(*reinterpret_cast<const __nv_bfloat16*>(q)) : 0.f;
    }
  }
  // The lane's pieces of what its warp has loaded that way.
  static __device__ __forceinline__ void pieces_of(uint32_t stage, int lane, const float (&raw)[32], float (&f)[4][8]) {
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; ++r) put_column(stage, r, lane, raw[r]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        tok::Vec<float>::unpack(slot16(stage + piece(8 * i + (lane >> 2), 2 * (lane & 3) + h)), f[i] + 4 * h);
    __syncwarp();
  }
  __device__ __forceinline__ void store_rows(uint32_t stage, int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                             int lane, const float (&f)[4][8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + piece(8 * i + (lane >> 2), 2 * (lane & 3) + h)),
                     "f"(f[i][4 * h]), "f"(f[i][4 * h + 1]), "f"(f[i][4 * h + 2]), "f"(f[i][4 * h + 3])
                     : "memory");
    __syncwarp();
    const int here = int(min(int64_t(32), rows - r0));
    const bool in = c0 + lane < cols;
    char* q = at(r0, c0 + lane);
    const int64_t by = stride * (fp32 ? 4 : 2);
#pragma unroll 8
    for (int r = 0; r < 32; ++r, q += by) {
      const float x = at_column(stage, r, lane);
      if (!in || r >= here) continue;
      if (fp32) *reinterpret_cast<float*>(q) = x;
      else *reinterpret_cast<__nv_bfloat16*>(q) = __float2bfloat16_rn(x);
    }
    __syncwarp();
  }
  __device__ __forceinline__ void fetched(uint32_t slots, int half, int i, const char* q, int left, int lane,
                                          float* f) const {
    if (left < 8) return load(q, left, f);
    if (fp32) {
      tok::Vec<float>::unpack(slot16(slots + (2 * i) * 512 + lane * 16), f);
      tok::Vec<float>::unpack(slot16(slots + (2 * i + 1) * 512 + lane * 16), f + 4);
    } else {
      tok::Vec<__nv_bfloat16>::unpack(slot16(slots + half * 2048 + i * 512 + lane * 16), f);
    }
  }
};

template <int KIND>
__device__ __forceinline__ void act32(float (&v)[4][8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = lay::activation(v[i][j], KIND);
}

template <int KIND>
__device__ __forceinline__ void slope32(float (&v)[4][8], const float (&u)[4][8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= lay::slope(u[i][j], KIND);
}

// A lane's four rows of a chunk go through each step together: four independent
// chains hide the latency that one warp has nothing else to hide behind (one
// row at a time, the results of a 256 x 256 tile took 12 us, longer than the
// sums of 4096 terms; now 3 us).

// out = residual + dropout(activation(acc + bias)), pre = acc + bias.
struct Forward {
  const void* bias;
  Matrix out, pre, residual;   // p = NULL: none
  int64_t rows;                // tokens
  int cols, bias32, act;
  Dropout drop;

  // A result in FP32 is summed in passes of kDepth K blocks, not kDepthRounded.
  __device__ __forceinline__ bool exact() const { return out.fp32; }
  __device__ __forceinline__ bool halves() const { return !residual.fp32; }
  __device__ __forceinline__ void fetch(uint32_t slots, int half, int64_t t0, int64_t n0, int lane) const {
    if (residual.p) residual.fetch(slots, half, t0, n0, rows, cols, lane);
  }
  // Eight columns of one token.
  __device__ __forceinline__ void piece8(float (&v)[8], int64_t t, int64_t n, const Draw& draw) const {
    const int left = int(min(int64_t(8), cols - n));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (bias && j < left)
        v[j] += bias32 ? static_cast<const float*>(bias)[n + j]
                       : tok::to_float(static_cast<const __nv_bfloat16*>(bias)[n + j]);
    if (pre.p) pre.store(pre.at(t, n), left, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = lay::activation(v[j], act);
    if (drop.least) {
      const uint4 w = draw.at(uint32_t(t), uint32_t(n / 8), drop.site);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = lay::dropped(v[j], lay::draw_of(w, j), drop);
    }
    if (residual.p) {
      float r[8];
      residual.load(residual.at(t, n), left, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    out.store(out.at(t, n), left, v);
  }
  template <typename Read>
  __device__ __forceinline__ void chunk(const Read& read, uint32_t slots, int half, int64_t t0, int64_t n0, int lane,
                                        const Draw& draw) const {
    const int64_t n = n0 + (lane & 3) * 8, t = t0 + (lane >> 2);
    const int left = int(min(int64_t(8), cols - n));                                      // of its columns
    const int live = left <= 0 ? 0 : int(min(int64_t(4), (rows - t + 7) >> 3));   // of its rows
    float v[4][8], raw[32];
    const bool late = residual.p && !residual.wide;   // its rows start anywhere
    if (late) residual.load_column(t0, n0, rows, cols, lane, raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) read(8 * i + (lane >> 2), lane & 3, v[i]);
    if (bias) {
      float b[8];
      if (bias32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = j < left ? static_cast<const float*>(bias)[n + j] : 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          b[j] = j < left ? tok::to_float(static_cast<const __nv_bfloat16*>(bias)[n + j]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += b[j];
    }
    // The conditions on `wide` are the warp's.
    if (pre.p) {
      if (pre.wide) {
        char* q = pre.at(t, n);
        const int64_t by = pre.step();
#pragma unroll
        for (int i = 0; i < 4; ++i, q += by)
          if (i < live) pre.store(q, left, v[i]);
      } else {
        __syncwarp();   // the sums have been read
        pre.store_rows(read.at, t0, n0, rows, cols, lane, v);
      }
    }
    switch (act) {
      case MUON_ACT_RELU: act32<MUON_ACT_RELU>(v); break;
      case MUON_ACT_RELU2: act32<MUON_ACT_RELU2>(v); break;
      case MUON_ACT_GELU: act32<MUON_ACT_GELU>(v); break;
      case MUON_ACT_SILU: act32<MUON_ACT_SILU>(v); break;
      default: break;
    }
    if (drop.least) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = draw.at(uint32_t(t + 8 * i), uint32_t(n / 8), drop.site);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = lay::dropped(v[i][j], lay::draw_of(w, j), drop);
      }
    }
    if (residual.p) {
      if (!late) {
        const char* q = residual.at(t, n);
        const int64_t by = residual.step();
#pragma unroll
        for (int i = 0; i < 4; ++i, q += by) {
          if (i >= live) break;
          float r[8];
          residual.fetched(slots, half, i, q, left, lane, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        }
      } else {
        float r[4][8];
        Matrix::pieces_of(read.at, lane, raw, r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += r[i][j];
      }
    }
    if (out.wide) {
      char* q = out.at(t, n);
      const int64_t by = out.step();
#pragma unroll
      for (int i = 0; i < 4; ++i, q += by)
        if (i < live) out.store(q, left, v[i]);
    } else {
      __syncwarp();
      out.store_rows(read.at, t0, n0, rows, cols, lane, v);
    }
  }
};

// dx = acc * activation'(pre).
struct InputGrad {
  Matrix dx, pre;
  int64_t rows;
  int cols, act;
  Dropout drop;   // none

  __device__ __forceinline__ bool exact() const { return false; }
  __device__ __forceinline__ bool halves() const { return true; }
  __device__ __forceinline__ void fetch(uint32_t slots, int half, int64_t t0, int64_t n0, int lane) const {
    if (act != MUON_ACT_NONE) pre.fetch(slots, half, t0, n0, rows, cols, lane);
  }
  template <typename Read>
  __device__ __forceinline__ void chunk(const Read& read, uint32_t slots, int half, int64_t t0, int64_t n0, int lane,
                                        const Draw&) const {
    const int64_t n = n0 + (lane & 3) * 8, t = t0 + (lane >> 2);
    const int left = int(min(int64_t(8), cols - n));
    const int live = left <= 0 ? 0 : int(min(int64_t(4), (rows - t + 7) >> 3));
    float v[4][8], raw[32];
    const bool late = act != MUON_ACT_NONE && !pre.wide;
    if (late) pre.load_column(t0, n0, rows, cols, lane, raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) read(8 * i + (lane >> 2), lane & 3, v[i]);
    if (act != MUON_ACT_NONE) {
      float u[4][8];
      if (!late) {
        const char* q = pre.at(t, n);
        const int64_t by = pre.step();
#pragma unroll
        for (int i = 0; i < 4; ++i, q += by)
          if (i < live) pre.fetched(slots, half, i, q, left, lane, u[i]);
      } else {
        Matrix::pieces_of(read.at, lane, raw, u);
      }
      switch (act) {
        case MUON_ACT_RELU: slope32<MUON_ACT_RELU>(v, u); break;
        case MUON_ACT_RELU2: slope32<MUON_ACT_RELU2>(v, u); break;
        case MUON_ACT_GELU: slope32<MUON_ACT_GELU>(v, u); break;
        default: slope32<MUON_ACT_SILU>(v, u); break;
      }
    }
    if (dx.wide) {
      char* q = dx.at(t, n);
      const int64_t by = dx.step();
#pragma unroll
      for (int i = 0; i < 4; ++i, q += by)
        if (i < live) dx.store(q, left, v[i]);
    } else {
      __syncwarp();
      dx.store_rows(read.at, t0, n0, rows, cols, lane, v);
    }
  }
};

// accum = (overwrite ? 0 : accum) + scale * acc, at the parameter's place.
//
// A warp's 32 rows x 32 columns: a lane's row lies in shared memory, 144 bytes from
// the next, shifted as its place in accum is against 16 bytes, and goes out as one
// bulk copy, added at L2 or put in place, so that a warp needs no load of the old
// sums and waits for nothing.  What lies before the first and behind the last
// 16-byte piece, up to three elements each, goes by itself: added or stored, once
// for each element of the gradient, so that the order of the sums is one.  Rows
// that a partition cuts go element by element.
constexpr int kRowBytes = 144;

__device__ __forceinline__ void bulk_add(float* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_put(float* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void add_one(float* dst, float x) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(dst), "f"(x) : "memory");
}
__device__ __forceinline__ float shared_float(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

struct WeightGrad {
  float* accum;
  int64_t rows;
  int cols, overwrite;
  float scale;
  Dropout drop;   // none
  Segments sg;

  __device__ __forceinline__ bool exact() const { return true; }
  __device__ __forceinline__ void put(float* p, float x) const {
    if (overwrite) *p = x;
    else add_one(p, x);
  }

  // x: columns c0 .. c0 + 31 of row r0 + lane.  room: the warp's, 32 * kRowBytes.
  __device__ __forceinline__ void put_rows(uint32_t room, int64_t r0, int64_t c0, int lane, const float (&x)[32]) const {
    const int64_t r = r0 + lane;
    const int width = int(min(int64_t(32), cols - c0));
    int64_t piece = 0;
    float* p = r < rows ? accum + sg.place(r * cols + c0, &piece) : nullptr;
    const bool whole = p && piece >= width;
    const int shift = whole ? int(reinterpret_cast<uintptr_t>(p) >> 2) & 3 : 0;
    const uint32_t mine = room + uint32_t(lane * kRowBytes);
    tma_store_wait_read();   // this lane's row before
    if (__all_sync(0xffffffffu, shift == 0)) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + g * 16), "f"(scale * x[4 * g]),
                     "f"(scale * x[4 * g + 1]), "f"(scale * x[4 * g + 2]), "f"(scale * x[4 * g + 3])
                     : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + uint32_t(shift + j) * 4), "f"(scale * x[j]) : "memory");
    }
    if (whole) {
      const int head = min((4 - shift) & 3, width), mid = (width - head) & ~3;
      if (mid) {
        fence_async_smem();
        const uint32_t from = mine + uint32_t(shift + head) * 4;
        if (overwrite) bulk_put(p + head, from, mid * 4);
        else bulk_add(p + head, from, mid * 4);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (j < head) put(p + j, shared_float(mine + uint32_t(shift + j) * 4));
        const int c = head + mid + j;
        if (c < width) put(p + c, shared_float(mine + uint32_t(shift + c) * 4));
      }
    }
    for (uint32_t cut = __ballot_sync(0xffffffffu, p && !whole); cut; cut &= cut - 1) {
      const int row = __ffs(cut) - 1;   // its columns to the warp's lanes
      __syncwarp();
      int64_t left;
      if (lane < width)
        put(accum + sg.place((r0 + row) * cols + c0 + lane, &left), shared_float(room + uint32_t(row * kRowBytes + lane * 4)));
    }
    __syncwarp();
  }
  __device__ __forceinline__ void fetch(uint32_t, int, int64_t, int64_t, int) const {}
  // A chunk whose sums lie in several blocks, or this one: rows of them, then as above.
  template <typename Read>
  __device__ __forceinline__ void chunk(const Read& read, uint32_t room, int, int64_t r0, int64_t c0, int lane,
                                        const Draw&) const {
    float v[4][8], x[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) read(8 * i + (lane >> 2), lane & 3, v[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(read.at + piece(8 * i + (lane >> 2), 2 * (lane & 3) + h)),
                     "f"(v[i][4 * h]), "f"(v[i][4 * h + 1]), "f"(v[i][4 * h + 2]), "f"(v[i][4 * h + 3])
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 8; ++g) tok::Vec<float>::unpack(slot16(read.at + piece(lane, g)), x + 4 * g);
    put_rows(room, r0, c0, lane, x);
  }
};

__device__ __forceinline__ void stage_rows(uint32_t at, int lane, const float* x) {   // lane: the row
#pragma unroll
  for (int g = 0; g < 8; ++g)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + piece(lane, g)), "f"(x[4 * g]),
                 "f"(x[4 * g + 1]), "f"(x[4 * g + 2]), "f"(x[4 * g + 3])
                 : "memory");
}

__device__ __forceinline__ void stage_columns(uint32_t at, int lane, const float* x) {   // lane: the column
#pragma unroll
  for (int r = 0; r < 32; ++r)
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + piece(r, lane >> 2) + (lane & 3) * 4), "f"(x[r]) : "memory");
}

struct ReadOwn {
  uint32_t at;
  __device__ __forceinline__ void operator()(int row, int quarter, float* v) const {
    tok::Vec<float>::unpack(slot16(at + piece(row, 2 * quarter)), v);
    tok::Vec<float>::unpack(slot16(at + piece(row, 2 * quarter + 1)), v + 4);
  }
};

// The same chunk's sums from every block of the cluster, added in their order.
struct ReadAll {
  uint32_t at;
  int blocks;
  __device__ __forceinline__ void operator()(int row, int quarter, float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) {
      const uint32_t far = tc::mapa_shared(at, b);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x, y, z, w;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x), "=f"(y), "=f"(z), "=f"(w)
                     : "r"(far + piece(row, 2 * quarter + h)));
        v[4 * h] += x;
        v[4 * h + 1] += y;
        v[4 * h + 2] += z;
        v[4 * h + 3] += w;
      }
    }
  }
};

// ------------------------------------------------------------------ products

// One lane of a converged warp.  The compiler knows that elect.sync leaves one
// thread: behind `lane == 0` it issued each copy and each product through a loop
// over the lanes that might be there, 125 cycles apiece, and a K block took 0.45
// us instead of 0.28 at 256 x 256, 0.3 instead of 0.1 at 128 x 32.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

// Bounded wait, timed by the SM's own clock.
constexpr long long kMostCycles = 4000000000ll;   // about 2 s

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kMostCycles) {
      *abort_flag = 1;
      atomicExch(err, code);
      return false;
    }
  }
}

// D[m][n] = sum over k of A[m][k] B[n][k].  An operand lies with its k
// contiguous, or (mn) with its rows contiguous, k rows apart.
struct Product {
  CUtensorMap a, b;
  int64_t m, n;
  int k;                  // blocks of 64
  int tiles_m, tiles_n;
  int a_mn, b_mn;
};

template <class E>
struct One {
  Product p;
  int tiles;
  E e;
};

constexpr int BK = 64;

// Tensor memory adds 16 terms at a time and cuts off instead of rounding, all in one
// direction: about half a unit of 2^-23 of the sum a step at first, and more once the
// sum is 2^8 times a term and the last of a product's 16 bits lie below its unit.  Of
// terms of one sign one pass loses 3.8e-7 of its sum (256 terms), 2.2e-6 (1024), 1.4e-5
// (4096), 8.3e-5 (16384), 3.9e-4 (65536).  So a sum is formed in passes of so many K
// blocks of 64 terms, which FP32 registers add up: 16 for a result in FP32 and for
// accum; 64 for what is rounded to bf16, by up to 3.9e-3 (8192 x 14336 -> 4096 takes 2%
// longer than in one pass; in passes of 16 8192 x 4096 -> 14336 would take 5% longer, with
// a residual 15%); 4 for gradients of up to 2048 tokens, the more exact ones, where a K
// block of 256 x 256 takes 0.345 us instead of 0.26.
constexpr int kDepth = 16, kDepthRounded = 64, kDepthFew = 4, kFewBlocks = 32;

__device__ __forceinline__ uint32_t idesc_of(const Product& p, int m, int n) {
  return make_idesc(p.b_mn != 0, m, n) | (p.a_mn ? 1u << 15 : 0u);
}

// K block `kb` of `rows` (64 or 128) rows of an operand from row0.
template <int ROWS, bool PAIR>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int mn, int kb, int row0,
                                             uint32_t bar) {
  auto one = [&](uint32_t d, int x, int y) {
    if constexpr (PAIR) tma_load_2d_pair(d, map, x, y, bar);
    else tma_load_2d(d, map, x, y, bar);
  };
  if (!mn) {
    one(dst, kb * BK, row0);
  } else {
    constexpr int W = ROWS < 64 ? ROWS : 64;
#pragma unroll
    for (int j = 0; j < ROWS / W; ++j) one(dst + j * (W * BK * 2), row0 + j * W, kb * BK);
  }
}

// Descriptor of the first 16 of its terms, and what the next 16 and the next
// stage add to it (its low bits are the address / 16, below 2^14).  One thread
// issues every product: building descriptors anew for each took it 0.45 us a K
// block, where the tensor cores take 0.28.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at, int mn) {
  return mn ? make_desc(at, 64 * BK * 2, 1024, kSwizzle128) : make_desc(at, 16, 1024, kSwizzle128);
}
__device__ __forceinline__ uint32_t operand_step(int mn) { return mn ? 16 * 128 / 16 : 32 / 16; }

// 32 lanes x 16 columns of FP32 from tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t at, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}

// Tiles in groups of eight rows of tiles, column by column: what is under way
// at one time shares its operands in L2.
__device__ __forceinline__ void tile_of(const Product& p, int i, int* tm, int* tn) {
  const int per = 8 * p.tiles_n, g = i / per, first = g * 8, rows = min(8, p.tiles_m - first), r = i - g * per;
  *tm = first + r % rows;
  *tn = r / rows;
}

constexpr int kPairThreads = 320;
constexpr int kPairWarps = 8;   // of the epilogue

template <int BN, class E>
struct PairShape {
  static constexpr bool kSums = std::is_same_v<E, WeightGrad>;
  static constexpr int kA = 128 * BK * 2, kB = BN / 2 * BK * 2, kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kBars = 2 * kStages + 4;
  static constexpr int kWarpBytes = kSums ? 32 * kRowBytes : kChunkBytes + kSlotBytes;
  static constexpr int kShared = 1024 + kStages * kStage + kPairWarps * kWarpBytes + 8 * kBars + 16;
};

// Tiles of 256 x BN on pairs of SMs (tcgen05 cta_group::2): each block of the
// pair loads its half of either operand and holds 128 rows of the result.
// Warp 0 loads, warp 1 of the even block issues the products, eight warps of
// each block add up the partial sums and write the results of one tile while
// the next one's are formed.
template <int BN, class E>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
k_linear_pair(const __grid_constant__ One<E> w, int late, int* err) {
  using S = PairShape<BN, E>;
  extern __shared__ uint8_t raw_shared[];
  const uint32_t base = (smem_u32(raw_shared) + 1023u) & ~1023u;
  const uint32_t epi = base + S::kStages * S::kStage;
  const uint32_t bars = epi + kPairWarps * S::kWarpBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
  auto tfull = [&](int i) { return bars + 8u * (2 * S::kStages + i); };
  auto tempty = [&](int i) { return bars + 8u * (2 * S::kStages + 2 + i); };
  uint8_t* tail = raw_shared + (bars + 8u * S::kBars - smem_u32(raw_shared));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail) + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const Product& p = w.p;
  const int nk = p.k;
  const bool exact = w.e.exact();
  const int depth = !exact ? kDepthRounded : S::kSums && nk <= kFewBlocks ? kDepthFew : kDepth;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), 2 * kPairWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  begin_kernel(late);

  if (warp == 0) {
    if (elect_one()) {
      const int a_mn = p.a_mn, b_mn = p.b_mn;
      const CUtensorMap *ma = &p.a, *mb = &p.b;
      int s = 0;
      uint32_t ph = 0;
      for (int tile = first; tile < w.tiles && !*abort_flag; tile += step) {
        int tm, tn;
        tile_of(p, tile, &tm, &tn);
        const int row0 = tm * 256 + int(rank) * 128, col0 = tn * BN + int(rank) * (BN / 2);
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait(empty(s), ph ^ 1u, abort_flag, err, ERR_TIMEOUT_PRODUCER)) break;
          const uint32_t sa = base + s * S::kStage, fb = mapa_shared(full(s), 0);
          if (rank == 0) mbar_expect_tx(full(s), 2 * S::kStage);
          load_operand<128, true>(sa, ma, a_mn, kb, row0, fb);
          load_operand<BN / 2, true>(sa + S::kA, mb, b_mn, kb, col0, fb);
          if (++s == S::kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      const uint32_t idesc = idesc_of(p, 256, BN);
      const uint64_t a0 = operand_desc(base, p.a_mn), b0 = operand_desc(base + S::kA, p.b_mn);
      const uint32_t a_step = operand_step(p.a_mn), b_step = operand_step(p.b_mn);
      for (int tile = first; ok && tile < w.tiles; tile += step) {
        for (int k0 = 0; ok && k0 < nk; k0 += depth) {
          if (!wait(tempty(acc), acc_ph ^ 1u, abort_flag, err, ERR_TIMEOUT_MMA)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + uint32_t(acc * BN);
          const int k1 = min(nk, k0 + depth);
          for (int kb = k0; kb < k1; ++kb) {
            if (!wait(full(s), ph, abort_flag, err, ERR_TIMEOUT_MMA)) { ok = false; break; }
            tc_fence_after();
            uint64_t ad = a0 + uint32_t(s * (S::kStage / 16)), bd = b0 + uint32_t(s * (S::kStage / 16));
#pragma unroll
            for (int k = 0; k < BK / 16; ++k, ad += a_step, bd += b_step)
              umma_bf16_pair(d, ad, bd, idesc, kb > k0 || k > 0);
            umma_commit_pair(empty(s), 0x3);
            if (++s == S::kStages) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          umma_commit_pair(tfull(acc), 0x3);
          acc ^= 1;
          if (acc == 0) acc_ph ^= 1u;
        }
      }
    }
  } else {
    const int ew = warp - 2, q = warp & 3, side = ew >> 2;
    const uint32_t stage = epi + ew * S::kWarpBytes, slots = stage + kChunkBytes;
    constexpr int N = BN / 64;   // chunks of a warp
    Draw draw;
    draw.init(w.e.drop);
    int acc = 0;
    uint32_t acc_ph = 0;
    const uint32_t mine = tmem + uint32_t(side * (BN / 2)) + (uint32_t(q * 32) << 16);
    bool ok = true;
    auto next = [&] {   // hands the accumulator back
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    };
    auto ready = [&] {
      const bool r = wait(tfull(acc), acc_ph, abort_flag, err, ERR_TIMEOUT_EPILOGUE);
      __syncwarp();
      tc_fence_after();
      return r;
    };
    for (int tile = first; ok && tile < w.tiles; tile += step) {
      int tm, tn;
      tile_of(p, tile, &tm, &tn);
      const int64_t m0 = int64_t(tm) * 256 + rank * 128 + q * 32, n0 = int64_t(tn) * BN + side * (BN / 2);
      const bool here = m0 < p.m && n0 < p.n;
      if constexpr (S::kSums) {
        // adds up the partial sums of the tile's K blocks in registers
        float sum[N][32];
#pragma unroll
        for (int c = 0; c < N; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
        for (int k0 = 0; ok && k0 < nk; k0 += depth) {
          if (!ready()) { ok = false; break; }
          if (here) {
#pragma unroll
            for (int c = 0; c < 2 * N; ++c) {   // 16 columns at once: 32 more registers would spill
              float x[16];
              tmem_ld16(mine + uint32_t(acc * BN + c * 16), x);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[c / 2][c % 2 * 16 + j] += x[j];
            }
          }
          next();
        }
        if (!ok || !here) continue;
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (n0 + 32 * c < p.n) w.e.put_rows(stage, m0, n0 + 32 * c, lane, sum[c]);
      } else {
        if (here) w.e.fetch(slots, 0, m0, n0, lane);
        if (nk > depth) {
          // as above, and the sums back to where the last of them lay
          float sum[2 * N][16];
#pragma unroll
          for (int c = 0; c < 2 * N; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c][j] = 0.f;
          for (int k0 = 0; k0 < nk; k0 += depth) {
            if (!ready()) { ok = false; break; }
            if (here) {
#pragma unroll
              for (int c = 0; c < 2 * N; ++c) {
                float x[16];
                tmem_ld16(mine + uint32_t(acc * BN + c * 16), x);
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[c][j] += x[j];
              }
            }
            if (k0 + depth < nk) next();
          }
          if (!ok) break;
          if (here) {
#pragma unroll
            for (int c = 0; c < 2 * N; ++c) tmem_st16(mine + uint32_t(acc * BN + c * 16), sum[c]);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
        } else if (!ready()) {
          ok = false;
          break;
        }
        if (here) {
#pragma unroll 1
          for (int c = 0; c < N && n0 + 32 * c < p.n; ++c) {
            float x[32];
            tmem_ld32(mine + uint32_t(acc * BN + c * 32), x);
            stage_rows(stage, lane, x);
            copies_done();
            __syncwarp();
            // the other half of bf16 slots is refilled before this one is read, FP32
            // slots behind that
            const bool ahead = c + 1 < N && n0 + 32 * (c + 1) < p.n, halves = w.e.halves();
            if (ahead && halves) w.e.fetch(slots, (c + 1) & 1, m0, n0 + 32 * (c + 1), lane);
            w.e.chunk(ReadOwn{stage}, slots, c & 1, m0, n0 + 32 * c, lane, draw);
            if (ahead && !halves) w.e.fetch(slots, (c + 1) & 1, m0, n0 + 32 * (c + 1), lane);
            __syncwarp();
          }
        }
        next();
      }
    }
    if constexpr (S::kSums) tma_store_wait_all();
  }
  if (*abort_flag) {
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 20000000ull) __nanosleep(100000);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
  end_kernel(late);
}

constexpr int kSplitThreads = 192;
constexpr int kSplitWarps = 4;   // of the epilogue
constexpr int kMostSplits = 4;   // blocks of a cluster

template <int BN>
struct SplitShape {
  static constexpr int kA = 128 * BK * 2, kB = BN * BK * 2, kStage = kA + kB;
  static constexpr int kStages = BN == 128 ? 6 : BN == 64 ? 9 : 11;
  static constexpr int kBars = 2 * kStages + 4;
  static constexpr int kChunks = kSplitWarps * (BN / 32);
  static constexpr int kShared = 1024 + kStages * kStage + 8 * kBars + 16;
  static constexpr int kRoom = 32 * kRowBytes;   // a warp's slots, or its rows on their way to accum
  static_assert(kRoom >= kSlotBytes && kChunks * kChunkBytes + kSplitWarps * kRoom <= kStages * kStage,
                "sums and slots take the operands' place");
};

// One tile of 128 x BN per cluster, whose blocks share out the K blocks and add
// their sums through distributed shared memory, in the order of the blocks.
// SWAP: the rows of the product are the result's columns (features, of which
// there are many) and its columns the result's rows (few tokens), so that few
// tokens leave no part of a tile's 128 rows empty.
template <int BN, bool SWAP, class E>
__global__ void __launch_bounds__(kSplitThreads, 1)
k_linear_split(const __grid_constant__ One<E> w, int splits, int late, int* err) {
  using S = SplitShape<BN>;
  extern __shared__ uint8_t raw_shared[];
  const uint32_t base = (smem_u32(raw_shared) + 1023u) & ~1023u;
  const uint32_t bars = base + S::kStages * S::kStage;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
  auto tfull = [&](int i) { return bars + 8u * (2 * S::kStages + i); };
  auto tempty = [&](int i) { return bars + 8u * (2 * S::kStages + 2 + i); };
  uint8_t* tail = raw_shared + (bars + 8u * S::kBars - smem_u32(raw_shared));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail) + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / splits, rank = blockIdx.x % splits;   // clusters are consecutive blocks
  const Product& p = w.p;
  int tm, tn;
  tile_of(p, tile, &tm, &tn);
  const int kb0 = int(int64_t(p.k) * rank / splits), kb1 = int(int64_t(p.k) * (rank + 1) / splits);

  const bool loader = warp == 0 && elect_one();
  auto load = [&](int kb, int s) {
    const uint32_t sa = base + s * S::kStage;
    mbar_expect_tx(full(s), S::kStage);
    load_operand<128, false>(sa, &p.a, p.a_mn, kb, tm * 128, full(s));
    load_operand<BN, false>(sa + S::kA, &p.b, p.b_mn, kb, tn * BN, full(s));
  };
  if (loader) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), kSplitWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    // the first loads are on their way before tensor memory is there (1 us)
    begin_kernel(late);
    for (int s = 0; s < S::kStages && kb0 + s < kb1; ++s) load(kb0 + s, s);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!loader) begin_kernel(late);

  const int ew = warp - 2, q = warp & 3;
  const uint32_t slots = base + S::kChunks * kChunkBytes + ew * S::kRoom;   // once the operands are read
  constexpr int N = BN / 32;
  // where chunk (quarter of the rows, 32 columns) lies in the result
  auto row_of = [&](int quarter, int c) { return SWAP ? int64_t(tn) * BN + 32 * c : int64_t(tm) * 128 + 32 * quarter; };
  auto col_of = [&](int quarter, int c) { return SWAP ? int64_t(tm) * 128 + 32 * quarter : int64_t(tn) * BN + 32 * c; };
  auto inside = [&](int quarter, int c) {
    return int64_t(tm) * 128 + 32 * quarter < p.m && int64_t(tn) * BN + 32 * c < p.n;
  };
  bool ok = true;
  if (warp == 0) {
    if (loader) {
      int s = 0;
      uint32_t ph = 0;
      for (int kb = kb0 + S::kStages; kb < kb1; ++kb) {
        if (!wait(empty(s), ph, abort_flag, err, ERR_TIMEOUT_PRODUCER)) break;
        load(kb, s);
        if (++s == S::kStages) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      const uint32_t idesc = idesc_of(p, 128, BN);
      const uint64_t a0 = operand_desc(base, p.a_mn), b0 = operand_desc(base + S::kA, p.b_mn);
      const uint32_t a_step = operand_step(p.a_mn), b_step = operand_step(p.b_mn);
      for (int k0 = kb0; ok && k0 < kb1; k0 += kDepthFew) {
        if (!wait(tempty(acc), acc_ph ^ 1u, abort_flag, err, ERR_TIMEOUT_MMA)) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc * BN);
        const int k1 = min(kb1, k0 + kDepthFew);
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait(full(s), ph, abort_flag, err, ERR_TIMEOUT_MMA)) { ok = false; break; }
          tc_fence_after();
          uint64_t ad = a0 + uint32_t(s * (S::kStage / 16)), bd = b0 + uint32_t(s * (S::kStage / 16));
#pragma unroll
          for (int k = 0; k < BK / 16; ++k, ad += a_step, bd += b_step)
            umma_bf16(d, ad, bd, idesc, kb > k0 || k > 0);
          umma_commit(empty(s));
          if (++s == S::kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(tfull(acc));
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1u;
      }
    }
  } else {
    int acc = 0;
    uint32_t acc_ph = 0;
    float sum[N][32];
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
    for (int k0 = kb0; k0 < kb1; k0 += kDepthFew) {
      if (!wait(tfull(acc), acc_ph, abort_flag, err, ERR_TIMEOUT_EPILOGUE)) { ok = false; break; }
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < N; ++c) {
        float x[32];
        tmem_ld32(tmem + uint32_t(acc * BN + c * 32) + (uint32_t(q * 32) << 16), x);
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[c][j] += x[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(acc));
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    }
    // Every product has read its operands: the sums take their place.  (All of
    // a block's loads have landed, since its products waited for them.)
    if (ok) {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const uint32_t at = base + uint32_t((q * N + c) * kChunkBytes);
        if (SWAP) stage_columns(at, lane, sum[c]);
        else stage_rows(at, lane, sum[c]);
      }
    }
  }
  __syncwarp();
  if (splits > 1) cluster_sync();
  else __syncthreads();
  // every block's status: a block that gave up has staged nothing
  bool good = !*abort_flag;
  if (splits > 1)
    for (int b = 0; b < splits; ++b) {
      uint32_t v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(tail), b)));
      good = good && v == 0;
    }
  if (warp >= 2 && good) {
    Draw draw;
    draw.init(w.e.drop);
    // the cluster's blocks, and their warps, take chunks in turn
    for (int i = rank + splits * ew; i < S::kChunks; i += splits * kSplitWarps) {
      const int quarter = i / N, c = i % N;
      if (!inside(quarter, c)) continue;
      const uint32_t at = base + uint32_t(i * kChunkBytes);
      const int64_t r = row_of(quarter, c), n = col_of(quarter, c);
      w.e.fetch(slots, 0, r, n, lane);
      copies_done();
      if (splits > 1) w.e.chunk(ReadAll{at, splits}, slots, 0, r, n, lane, draw);
      else w.e.chunk(ReadOwn{at}, slots, 0, r, n, lane, draw);
    }
    if constexpr (std::is_same_v<E, WeightGrad>) tma_store_wait_all();
  }
  if (*abort_flag) {
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 20000000ull) __nanosleep(100000);
  }
  __syncwarp();
  tc_fence_before();
  if (splits > 1) cluster_sync();   // nobody leaves while its sums may be read
  else __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
  end_kernel(late);
}

// ------------------------------------------------------------------ a few tokens

constexpr int kRowWarps = 8;

// Whether k_linear_rows takes the product: one or two tokens, or up to four of a
// weight of at most 2^22 elements, whose rows start on 16 bytes.  Measured, one
// after another with other weights each time, against tiles on single SMs: 4096 x
// 4096, 1 token 7.4 us against 11.2, 2 tokens 11.0 against 11.2, 4 tokens 12.6 against
// 11.5; 768 x 2304, 4 tokens 3.3 against 5.5; rows at odd places 9.3 against 6.7
// (copied first).
constexpr int kRowTokens = 4;
bool takes_rows(int64_t tokens, int64_t in, int64_t out, bool aligned) {
  return aligned && (tokens <= 2 || (tokens <= kRowTokens && in * out <= (1 << 22)));
}

struct RowArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  int64_t x_stride, w_stride;
  int k;
  Forward f;
};

// Eight features for up to T tokens per block, whose warps share out K; sums by
// FP32 multiply-adds, lanes and warps joined in a fixed order.  Bound by the
// weight's bytes: every lane has eight loads of 16 bytes on their way, and
// nothing is set up before them (the tensor cores' way to the same place takes
// 5 us more: tensor memory, maps, a cluster's sums).  The first pieces of the
// weight are asked for into L2, where that is always safe, before the kernel
// waits for the one before it.
template <int T>
__global__ void __launch_bounds__(32 * kRowWarps) k_linear_rows(const __grid_constant__ RowArgs a) {
  __shared__ float sums[kRowWarps][T * 8];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t n0 = int64_t(blockIdx.x) * 8;
  const int features = int(min(int64_t(8), a.f.cols - n0));
  const int tokens = int(a.f.rows);
  const __nv_bfloat16* w = a.w + n0 * a.w_stride;
  constexpr int kPiece = 256;   // elements of a warp's step
  const int first = warp * kPiece + lane * 8;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < features && first < a.k) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + r * a.w_stride + first));
  begin_kernel(0);
  float acc[T][8] = {};
  for (int k = first; k < a.k; k += kRowWarps * kPiece) {
    float f[8], g[T][8];
    if (k + 8 <= a.k) {
      uint4 raw[8], xs[T];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        raw[r] = make_uint4(0, 0, 0, 0);
        if (r < features) raw[r] = __ldcs(reinterpret_cast<const uint4*>(w + r * a.w_stride + k));
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        xs[t] = make_uint4(0, 0, 0, 0);
        if (t < tokens) xs[t] = *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + k);
      }
#pragma unroll
      for (int t = 0; t < T; ++t) tok::Vec<__nv_bfloat16>::unpack(xs[t], g[t]);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        tok::Vec<__nv_bfloat16>::unpack(raw[r], f);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[t][r] += f[j] * g[t][j];
      }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          g[t][j] = t < tokens && k + j < a.k ? tok::to_float(a.x[t * a.x_stride + k + j]) : 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          f[j] = r < features && k + j < a.k ? tok::to_float(w[r * a.w_stride + k + j]) : 0.f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[t][r] += f[j] * g[t][j];
      }
    }
  }
  // 8 T sums over the warp's lanes
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t][r] += __shfl_xor_sync(0xffffffffu, acc[t][r], o);
      if (lane == 0) sums[warp][t * 8 + r] = acc[t][r];
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= T || t >= tokens) return;
  float v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    v[r] = 0.f;
#pragma unroll
    for (int q = 0; q < kRowWarps; ++q) v[r] += sums[q][t * 8 + r];
  }
  Draw draw;
  draw.init(a.f.drop);
  a.f.piece8(v, t, n0, draw);
}

// ------------------------------------------------------------------ operands that are copied first

constexpr int kPackThreads = 256;
constexpr int kPackMost = 3;   // operands of a call

struct Pack {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t stride, rows;
  int cols;
};

struct Packs {
  Pack p[kPackMost];
  int64_t end[kPackMost];   // pieces of the operands up to this one
  int n;
};

// Rows of `cols` elements at any stride to rows that start on 16 bytes; eight
// elements per thread, all of a call's operands in one launch (words instead of
// elements, or two pieces per thread, gained 0.2 of 20 us).  What a row's last piece
// holds beyond cols is not read.
__global__ void __launch_bounds__(kPackThreads) k_linear_pack(const __grid_constant__ Packs a) {
  begin_kernel(0);
  for (int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x; i < a.end[kPackMost - 1];
       i += int64_t(gridDim.x) * kPackThreads) {
    const int which = i < a.end[0] ? 0 : i < a.end[1] ? 1 : 2;
    const Pack& p = a.p[which];
    const int pieces = (p.cols + 7) / 8;
    const int64_t j = which ? i - a.end[which - 1] : i, r = j / pieces;
    const int c = int(j - r * pieces) * 8;
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p.in) + r * p.stride + c;
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = c + 2 * k < p.cols ? q[2 * k] : 0u, hi = c + 2 * k + 1 < p.cols ? q[2 * k + 1] : 0u;
      v[k] = lo | hi << 16;
    }
    *reinterpret_cast<uint4*>(p.out + (r * pieces + (c >> 3)) * 8) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// ------------------------------------------------------------------ bias

struct BiasGrad {
  const __nv_bfloat16* dout;
  int64_t stride, tokens;
  int cols;
  float* accum;
  float scale;
  int overwrite;
};

constexpr int kBiasThreads = 256;
constexpr int kBiasColumns = 64;   // of a block: 128 bytes of a row, eight threads
constexpr int kBiasRows = kBiasThreads / 8;
constexpr int kBiasLoads = 8;      // rows a thread has under way

// Sums of dout's columns.  A cluster of blocks shares out the tokens of 64
// columns; their sums meet in the first block, in the order of the blocks.  VEC:
// rows start on 16 bytes.  Bound by memory: 8192 x 8192 in 26 us (5.2 TB/s), 16384 x
// 2304 in 20 (13 where dout lies in L2).
template <bool VEC>
__global__ void __launch_bounds__(kBiasThreads)
k_bias_grad(const BiasGrad a, const __grid_constant__ Segments sg, int blocks) {
  __shared__ float sums[kBiasRows][kBiasColumns + 4];
  __shared__ float all[kBiasColumns];
  begin_kernel(0);   // the call's first, but for copies of operands
  const int slab = blockIdx.x / blocks, rank = blockIdx.x % blocks;
  const int x = threadIdx.x % 8, y = threadIdx.x / 8;
  const int64_t c = int64_t(slab) * kBiasColumns + x * 8;
  const int left = int(min(int64_t(8), a.cols - c));
  const int64_t t0 = a.tokens * rank / blocks, t1 = a.tokens * (rank + 1) / blocks;
  float v[8] = {};
  for (int64_t t = t0 + y; t < t1; t += kBiasRows * kBiasLoads) {
    if constexpr (VEC) {
      uint4 raw[kBiasLoads];
#pragma unroll
      for (int u = 0; u < kBiasLoads; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (left >= 8 && t + u * kBiasRows < t1)
          raw[u] = __ldg(reinterpret_cast<const uint4*>(a.dout + (t + u * kBiasRows) * a.stride + c));
      }
#pragma unroll
      for (int u = 0; u < kBiasLoads; ++u) {
        float f[8];
        tok::Vec<__nv_bfloat16>::unpack(raw[u], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
      }
    }
    if (!VEC || left < 8)
#pragma unroll 1
      for (int u = 0; u < kBiasLoads; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left && t + u * kBiasRows < t1) v[j] += tok::to_float(a.dout[(t + u * kBiasRows) * a.stride + c + j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[y][x * 8 + j] = v[j];
  __syncthreads();
  const int i = threadIdx.x;
  if (i < kBiasColumns) {
    float s = 0.f;
#pragma unroll 8
    for (int r = 0; r < kBiasRows; ++r) s += sums[r][i];
    all[i] = s;
  }
  __syncwarp();
  if (blocks > 1) cluster_sync();
  const int64_t col = int64_t(slab) * kBiasColumns + i;
  if (rank == 0 && i < kBiasColumns && col < a.cols) {
    float s = all[i];
    for (int b = 1; b < blocks; ++b) {
      float f;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(mapa_shared(smem_u32(&all[i]), b)));
      s += f;
    }
    int64_t room;
    float* p = a.accum + sg.place(col, &room);
    *p = (a.overwrite ? 0.f : *p) + a.scale * s;
  }
  __syncwarp();
  if (blocks > 1) cluster_sync();
}

cudaError_t launch_bias(const BiasGrad& a, const Segments& sg, cudaStream_t s) {
  const int slabs = (a.cols + kBiasColumns - 1) / kBiasColumns;
  // up to eight blocks of at least 64 tokens to 64 columns, four per SM
  int blocks = 1;
  while (blocks < 8 && int64_t(blocks) * 2 * slabs <= 4 * 152 && a.tokens >= 64 * 2 * blocks) blocks *= 2;
  const bool vec = !misaligned(a.dout, 16) && (a.tokens <= 1 || a.stride % 8 == 0);
  return launch(vec ? k_bias_grad<true> : k_bias_grad<false>, unsigned(slabs) * blocks, kBiasThreads, blocks, true, s, 0, a, sg,
                blocks);
}

// ------------------------------------------------------------------ host

constexpr int kMostFeatures = 1 << 24;
constexpr int kSms = 152, kPairs = kSms / 2;
constexpr int kLeast = 16;        // SMs that a kernel beside another is given at least
constexpr int kFourfold = 144;   // blocks that run at once as clusters of four (of eight: 120, of three: 138)

// An operand of a product: rows x cols, bf16.
struct Operand {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, stride = 0;
  size_t packed = 0;   // bytes of its copy in the workspace; 0: read where it lies

  Operand() = default;
  Operand(const void* q, int64_t r, int64_t c, int64_t s) : p(q), rows(r), cols(c), stride(s) {
    if (r <= 1) stride = (c + 7) / 8 * 8;   // a single row's stride says nothing
    // what the copies of tiles take: rows that start on 16 bytes, strides below 2^40 bytes
    if (q && (misaligned(q, 16) || stride % 8 || stride >= (int64_t(1) << 39)))
      packed = (size_t(r) * ((c + 7) / 8 * 16) + 255) & ~size_t(255);
  }
  // Adds its copy to a launch's, where it needs one; *at moves behind the copy.
  void pack(char** at, Packs* all) {
    if (packed) {
      const int64_t to = (cols + 7) / 8 * 8;
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(*at);
      all->p[all->n] = {static_cast<const __nv_bfloat16*>(p), out, stride, rows, int(cols)};
      const int64_t before = all->n ? all->end[all->n - 1] : 0;
      for (int i = all->n; i < kPackMost; ++i) all->end[i] = before + rows * (to / 8);
      ++all->n;
      *at += packed;
      p = out;
      stride = to;
    }
  }
};

cudaError_t launch_packs(const Packs& all, cudaStream_t s, int* launches) {
  if (!all.n) return cudaSuccess;
  const int64_t blocks = (all.end[kPackMost - 1] + kPackThreads - 1) / kPackThreads;
  const cudaError_t e = launch(k_linear_pack, unsigned(std::min<int64_t>(blocks, 16 * kSms)), kPackThreads, 1, true, s, 0, all);
  ++*launches;
  return e;
}

// How a product is run: pairs of SMs and tiles of 256 x bn, or single ones, 128 x
// bn, with the K blocks shared out to `splits` blocks.
struct Plan {
  bool pairs = false, swap = false;
  int bn = 0, splits = 1;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The plan of least estimated time for D[m][n] with k terms on `sms` SMs.  An SM takes in 64
// bytes a cycle, which is what a K block of 64 costs: 0.28 us on a pair at 256
// columns (there the tensor cores take as long), 0.20 at 128, 0.30 on a single SM.
// Starting, the first operands' latency and the results cost 7.2, 4.7 and 4.5 us, a
// cluster's sums 2 more.  Sums into accum (a weight's gradient, both operands along
// their rows, each row a piece of bulk copies) cost 8.8, 5.7 and 8.5, however many
// blocks share them out, and passes of kDepthFew K blocks more for each.  Measured
// on pairs at 128 / pairs at 256 / single SMs without a split / by 2 / by 4 (us,
// chosen: *): 1024 x 768 -> 768 7.8* / 12.0 / 8.9 / 9.4 / 16.5; 512 x 4096 -> 1024
// 18.0 / 25.5 / 20.8 / 15.1 / 12.0*; 1024 x 1024 -> 4096 13.0* / 13.9 / 19.5 / 38 / 66;
// 2048^3 19.4 / 18.2* / 27 / 45 / 74; their weights' gradients of 512 x 768 -> 768
// 7.6* / 11.1 / 10.7 / 9.3 / 9.0; 2048 x 768 -> 768 13.9 / 19.7 / 16.9 / 12.4 / 10.7*;
// 2048 x 1024 -> 1024 14.3 / 19.9 / 17.1 / 12.9* / 20.3; 2048^3 26.0 / 21.2* / 35 / 50 / 77.
struct Offer {
  Plan plan;
  double us;
  int64_t sms;   // that it holds
};

constexpr int kOffers = 5;

// more: results have something done to them (us for each tile that an SM or a pair forms).
int offers_of(int64_t m, int64_t n, int64_t k, bool sums, bool more, int sms, Offer* out) {
  const double kb = double(ceil_div(k, 64));
  int count = 0;
  auto offer = [&](bool pairs, int bn, int splits, int64_t tiles, double us) {
    Offer& o = out[count++];
    o.plan.pairs = pairs;
    o.plan.bn = bn;
    o.plan.splits = splits;
    o.us = us;
    o.sms = std::min<int64_t>(sms, tiles * (pairs ? 2 : splits));
  };
  for (int bn : {256, 128}) {
    const int64_t tiles = ceil_div(m, 256) * ceil_div(n, bn);
    const double waves = double(ceil_div(tiles, sms / 2)), worked = more ? waves * (bn == 256 ? 3.7 : 1.8) : 0.0;
    double block = bn == 256 ? 0.28 : 0.20, again = 0.5, start = bn == 256 ? 7.2 : 4.7;
    if (sums) {
      block = kb > kFewBlocks ? (bn == 256 ? 0.26 : 0.20) : bn == 256 ? 0.345 : 0.27;
      again = bn == 256 ? 4.0 : 3.1;
      start = bn == 256 ? 8.8 : 5.7;
    }
    offer(true, bn, 1, tiles, waves * kb * block + (waves - 1) * again + start + worked);
  }
  const int64_t tiles = ceil_div(m, 128) * ceil_div(n, 128);
  for (int s = 1; s <= kMostSplits && (s == 1 || kb >= 2 * s); s *= 2) {
    const double waves = double(ceil_div(tiles * s, s > 2 ? std::max(4, sms - (kSms - kFourfold)) : sms));
    offer(false, 128, s, tiles, sums ? waves * (double(ceil_div(int64_t(kb), s)) * 0.27 + 8.2) + 0.3
                                     : waves * (double(ceil_div(int64_t(kb), s)) * 0.30 + 2.0 + (more ? 3.2 / s : 0.0)) +
                                           2.5 + (s > 1 ? 2.0 : 0.0));
  }
  return count;
}

Offer offer_of(int64_t m, int64_t n, int64_t k, bool sums, bool more, int sms) {
  Offer all[kOffers];
  const int count = offers_of(m, n, k, sums, more, sms, all);
  return *std::min_element(all, all + count, [](const Offer& a, const Offer& b) { return a.us < b.us; });
}

// Few tokens: features are the rows of the tiles, and the K blocks are shared out
// while there are SMs for it (a block that holds tensor memory has its SM for
// itself): what counts is how many bytes of the weight are on their way.
Plan plan_few(int64_t tokens, int64_t features, int64_t k) {
  Plan p;
  p.swap = true;
  p.bn = tokens <= 32 ? 32 : 64;
  const int64_t tiles = ceil_div(features, 128) * ceil_div(tokens, p.bn), kb = ceil_div(k, 64);
  while (p.splits < kMostSplits && tiles * p.splits * 2 <= kFourfold && kb >= 4 * p.splits) p.splits *= 2;
  return p;
}

constexpr int kFewTokens = 64;

// The plans of both gradients: the weight's beside the inputs', on the SMs that one
// leaves, where that is quicker than one after the other, which saves 2 us of starting
// (us, with the bias's; one after the other: 2048 x 768 -> 768 15.5 and 18.7; 4096 x 512
// -> 512 14.9 and 19.5; 1024 x 768 -> 768 12.7 and 17.4; 16384 x 256 -> 256 with a slope
// 28.8 and 38.2).
void plan_both(int64_t tokens, int64_t in, int64_t out, bool slope, Plan* dx, Plan* dw) {
  Offer first[kOffers];
  int count = 1;
  if (tokens <= kFewTokens) {
    first[0].plan = plan_few(tokens, in, out);
    first[0].sms = ceil_div(in, 128) * ceil_div(tokens, first[0].plan.bn) * first[0].plan.splits;
    first[0].us = 7.0;
  } else {
    count = offers_of(tokens, in, out, false, slope, kSms, first);
  }
  const Offer after = offer_of(out, in, tokens, true, false, kSms);
  double least = 0;
  for (int i = 0; i < count; ++i) {
    const int left = int(std::max<int64_t>(0, kSms - first[i].sms)) / 2 * 2;
    double us = first[i].us + after.us - 2.0;
    Plan second = after.plan;
    if (left >= kLeast) {
      const Offer beside = offer_of(out, in, tokens, true, false, left);
      if (std::max(first[i].us, beside.us) < us) {
        us = std::max(first[i].us, beside.us);
        second = beside.plan;
      }
    }
    if (i == 0 || us < least) {
      least = us;
      *dx = first[i].plan;
      *dw = second;
    }
  }
}

// The product of a and b, whose k lies along their columns (or, mn, along their
// rows), as the plan's tiles.  False: the driver refuses a map.
bool make_product(const Plan& plan, const Operand& a, bool a_mn, const Operand& b, bool b_mn, Product* p) {
  p->m = a_mn ? a.cols : a.rows;
  p->n = b_mn ? b.cols : b.rows;
  const int64_t k = a_mn ? a.rows : a.cols;
  p->k = int(ceil_div(k, BK));
  p->a_mn = a_mn;
  p->b_mn = b_mn;
  p->tiles_m = int(ceil_div(p->m, plan.pairs ? 256 : 128));
  p->tiles_n = int(ceil_div(p->n, plan.bn));
  if (k == 0) return true;   // nothing is loaded
  auto map = [](CUtensorMap* m, const Operand& o, bool mn, int rows) {
    return encode_2d(m, o.p, 2, o.cols, o.rows, o.stride, mn ? uint32_t(std::min(rows, 64)) : BK,
                     mn ? BK : uint32_t(rows), CU_TENSOR_MAP_SWIZZLE_128B);
  };
  return map(&p->a, a, a_mn, 128) && map(&p->b, b, b_mn, plan.pairs ? plan.bn / 2 : plan.bn);
}

template <auto KERNEL, class... A>
cudaError_t launch_shared(unsigned grid, unsigned block, int cluster, int bytes, cudaStream_t s, const A&... args) {
  static uint64_t done = 0;   // devices that know how much shared memory this kernel takes
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(done >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done |= uint64_t(1) << (dev & 63);
  }
  return launch(KERNEL, grid, block, cluster, true, s, bytes, args...);
}

// Where the current device's error flag lies.
cudaError_t error_flag(int** out) {
  static int* at[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!at[dev & 63]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_linear_err);
    at[dev & 63] = static_cast<int*>(p);
  }
  *out = at[dev & 63];
  return e;
}

template <int BN, class E>
cudaError_t launch_pair(const One<E>& w, int late, cudaStream_t s) {
  int* err;
  const cudaError_t e = error_flag(&err);
  if (e != cudaSuccess) return e;
  return launch_shared<k_linear_pair<BN, E>>(2 * unsigned(std::min(w.tiles, kPairs)), kPairThreads, 1,
                                             PairShape<BN, E>::kShared, s, w, late, err);
}

template <int BN, bool SWAP, class E>
cudaError_t launch_split(const One<E>& w, int splits, int late, cudaStream_t s) {
  int* err;
  const cudaError_t e = error_flag(&err);
  if (e != cudaSuccess) return e;
  return launch_shared<k_linear_split<BN, SWAP, E>>(unsigned(w.tiles) * splits, kSplitThreads, splits,
                                                    SplitShape<BN>::kShared, s, w, splits, late, err);
}

// A product's kernel arguments; false: the driver refuses a map.
template <class E>
bool prepare(const Plan& plan, const Operand& a, bool a_mn, const Operand& b, bool b_mn, const E& e, One<E>* w) {
  w->e = e;
  if (!make_product(plan, a, a_mn, b, b_mn, &w->p)) return false;
  w->tiles = w->p.tiles_m * w->p.tiles_n;
  return true;
}

template <class E>
cudaError_t launch_one(const Plan& plan, const One<E>& w, int late, cudaStream_t s) {
  if (plan.pairs) return plan.bn == 256 ? launch_pair<256>(w, late, s) : launch_pair<128>(w, late, s);
  if constexpr (!std::is_same_v<E, WeightGrad>) {
    if (plan.swap && plan.bn == 32) return launch_split<32, true>(w, plan.splits, late, s);
    if (plan.swap) return launch_split<64, true>(w, plan.splits, late, s);
  }
  return launch_split<128, false>(w, plan.splits, late, s);
}

cudaError_t launch_rows(const Operand& x, const Operand& w, const Forward& f, cudaStream_t s) {
  const RowArgs a{static_cast<const __nv_bfloat16*>(x.p), static_cast<const __nv_bfloat16*>(w.p), x.stride, w.stride,
                  int(w.cols), f};
  const int64_t t = f.rows;
  auto k = t == 1 ? k_linear_rows<1> : t == 2 ? k_linear_rows<2> : k_linear_rows<kRowTokens>;
  return launch(k, unsigned(ceil_div(w.rows, 8)), 32 * kRowWarps, 1, true, s, 0, a);
}

// The sum of launches' tiles stays below 2^31 (each plan has no more than this).
int check_sizes(int64_t tokens, int in, int out, int act) {
  if (tokens < 0 || tokens > (int64_t(1) << 30)) return fail_with(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30]");
  if (in < 1 || out < 1 || in > kMostFeatures || out > kMostFeatures)
    return fail_with(MUON_ERR_INVALID, "in_features and out_features must be in [1, 2^24]");
  if (act < MUON_ACT_NONE || act > MUON_ACT_SILU) return fail_with(MUON_ERR_INVALID, "unknown activation");
  auto tiles = [](int64_t a, int64_t b) { return ceil_div(a, 128) * ceil_div(b, 128) * kMostSplits; };
  if (tiles(tokens, out) + tiles(tokens, in) + tiles(in, out) > 0x7fffffff)
    return fail_with(MUON_ERR_UNSUPPORTED, "too many tokens and features for one launch");
  return MUON_OK;
}

int check_matrix(const void* p, int64_t stride, int64_t rows, int64_t cols, size_t es, const char* name) {
  if (rows == 0) return MUON_OK;
  if (!p || misaligned(p, es)) return fail_with(MUON_ERR_INVALID, std::string(name) + " is NULL or misaligned");
  if (stride < cols || !lay::stride_fits(rows, stride))
    return fail_with(MUON_ERR_INVALID, std::string(name) + "_stride is less than its columns or too large");
  return MUON_OK;
}

int check_forward(const muon_linear_args_t* a, Forward* f) {
  if (!a || a->struct_size != int32_t(sizeof(muon_linear_args_t)))
    return fail_with(MUON_ERR_INVALID, "args is NULL or its struct_size is wrong");
  const int64_t T = a->n_tokens;
  const int K = a->in_features, N = a->out_features;
  int rc = check_sizes(T, K, N, a->activation);
  if (rc != MUON_OK) return rc;
  const size_t es = dtype_bytes(a->out_dtype);
  if (!es) return fail_with(MUON_ERR_INVALID, "unknown out_dtype");
  if ((rc = lay::make_dropout(a->dropout, a->rng, a->site, &f->drop)) != MUON_OK) return rc;
  if ((rc = check_matrix(a->x, a->x_stride, T, K, 2, "x")) || (rc = check_matrix(a->weight, a->weight_stride, N, K, 2, "weight")) ||
      (rc = check_matrix(a->out, a->out_stride, T, N, es, "out")) ||
      (a->pre && (rc = check_matrix(a->pre, a->pre_stride, T, N, 2, "pre"))) ||
      (a->residual && (rc = check_matrix(a->residual, a->residual_stride, T, N, es, "residual"))))
    return rc;
  const size_t be = dtype_bytes(a->bias_dtype);
  if (a->bias && (!be || misaligned(a->bias, be)))
    return fail_with(MUON_ERR_INVALID, "bias is misaligned or of unknown bias_dtype");
  const Span x(a->x, T, a->x_stride, K, 2), w(a->weight, N, a->weight_stride, K, 2), b(a->bias, 1, N, N, be),
      res(a->residual, T, a->residual_stride, N, es), out(a->out, T, a->out_stride, N, es),
      pre(a->pre, T, a->pre_stride, N, 2), rng(f->drop.least ? a->rng : nullptr, 1, 2, 2, 8);
  for (const Span& v : {x, w, b, rng})
    if (v.meets(out) || v.meets(pre)) return fail_with(MUON_ERR_INVALID, "out or pre overlaps an input");
  if (out.meets(pre) || pre.meets(res) ||
      (out.meets(res) && !lay::same(a->residual, a->residual_stride, a->out, a->out_stride)))
    return fail_with(MUON_ERR_INVALID, "out, pre and the residual overlap");
  auto matrix = [&](const void* p, int64_t stride, size_t size) {
    return Matrix{const_cast<void*>(p), stride, size == 4, !misaligned(p, 16) && (T <= 1 || stride * int64_t(size) % 16 == 0)};
  };
  f->bias = a->bias;
  f->bias32 = a->bias_dtype == MUON_DTYPE_FP32;
  f->out = matrix(a->out, a->out_stride, es);
  f->pre = matrix(a->pre, a->pre_stride, 2);
  f->residual = matrix(a->residual, a->residual_stride, es);
  f->rows = T;
  f->cols = N;
  f->act = a->activation;
  return MUON_OK;
}

struct GradPlaces {
  Segments weight, bias;
};

int check_grad(const muon_linear_grad_args_t* a, GradPlaces* at) {
  if (!a || a->struct_size != int32_t(sizeof(muon_linear_grad_args_t)) || a->reserved != 0)
    return fail_with(MUON_ERR_INVALID, "args is NULL, its struct_size is wrong or reserved is not 0");
  const int64_t T = a->n_tokens;
  const int K = a->in_features, N = a->out_features;
  int rc = check_sizes(T, K, N, a->activation);
  if (rc != MUON_OK) return rc;
  if (a->overwrite != 0 && a->overwrite != 1) return fail_with(MUON_ERR_INVALID, "overwrite must be 0 or 1");
  if (!std::isfinite(a->scale)) return fail_with(MUON_ERR_INVALID, "scale must be finite");
  const bool slope = a->dx && a->activation != MUON_ACT_NONE;
  if ((rc = check_matrix(a->dout, a->dout_stride, T, N, 2, "dout")) ||
      (a->param && (rc = check_matrix(a->x, a->x_stride, T, K, 2, "x"))) ||
      (a->dx && ((rc = check_matrix(a->weight, a->weight_stride, N, K, 2, "weight")) ||
                 (rc = check_matrix(a->dx, a->dx_stride, T, K, 2, "dx")))) ||
      (slope && (rc = check_matrix(a->pre, a->pre_stride, T, K, 2, "pre"))))
    return rc;
  if (a->param) {
    if (a->param->rows != N || a->param->cols != K)
      return fail_with(MUON_ERR_INVALID, "param must be out_features x in_features");
    if ((rc = lay::place_param(*a->param, a->accum, a->accum_elems, a->parts, a->nparts, &at->weight))) return rc;
  }
  if (a->bias) {
    if (int64_t(a->bias->rows) * a->bias->cols != N)
      return fail_with(MUON_ERR_INVALID, "bias must have out_features elements");
    if ((rc = lay::place_param(*a->bias, a->accum, a->accum_elems, a->parts, a->nparts, &at->bias))) return rc;
    if (a->param && lay::flat_overlap(*a->param, *a->bias))
      return fail_with(MUON_ERR_INVALID, "param and bias overlap");
  }
  const Span dx(a->dx, T, a->dx_stride, K, 2), sums(a->param || a->bias ? a->accum : nullptr, 1, a->accum_elems,
                                                   a->accum_elems, 4);
  for (const Span& v : {Span(a->dout, T, a->dout_stride, N, 2), Span(a->param ? a->x : nullptr, T, a->x_stride, K, 2),
                        Span(a->dx ? a->weight : nullptr, N, a->weight_stride, K, 2),
                        Span(slope ? a->pre : nullptr, T, a->pre_stride, K, 2)})
    if (v.meets(dx) || v.meets(sums)) return fail_with(MUON_ERR_INVALID, "dx or accum overlaps an input");
  if (dx.meets(sums)) return fail_with(MUON_ERR_INVALID, "dx overlaps accum");
  return MUON_OK;
}

// The operands of the gradients' products.
struct GradOperands {
  Operand dout, weight, x;
  size_t bytes() const { return dout.packed + weight.packed + x.packed; }
};

GradOperands grad_operands(const muon_linear_grad_args_t& a) {
  GradOperands o;
  if (a.n_tokens == 0) {   // sums of nothing: extents only
    o.dout = Operand(nullptr, 0, a.out_features, a.out_features);
    o.x = Operand(nullptr, 0, a.in_features, a.in_features);
    return o;
  }
  if (a.dx || a.param) o.dout = Operand(a.dout, a.n_tokens, a.out_features, a.dout_stride);
  if (a.dx) o.weight = Operand(a.weight, a.out_features, a.in_features, a.weight_stride);
  if (a.param) o.x = Operand(a.x, a.n_tokens, a.in_features, a.x_stride);
  return o;
}

}  // namespace

int linear_take_device_error() { return take_flag(g_linear_err); }

}  // namespace muon

using namespace muon;

namespace {

// Where the workspace is too small for `need` bytes.
int check_workspace(const void* workspace, size_t bytes, size_t need, std::initializer_list<Span> others) {
  if (!need) return MUON_OK;
  if (!workspace || misaligned(workspace, 16) || bytes < need)
    return fail_with(MUON_ERR_INVALID, "workspace is NULL, misaligned or too small");
  const Span work(workspace, 1, int64_t(need), int64_t(need), 1);
  for (const Span& v : others)
    if (v.meets(work)) return fail_with(MUON_ERR_INVALID, "workspace overlaps another tensor");
  return MUON_OK;
}

}  // namespace

extern "C" int muon_linear_workspace(const muon_linear_args_t* args, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    Forward f{};
    const int rc = check_forward(args, &f);
    if (rc != MUON_OK) return rc;
    if (!bytes) return fail_with(MUON_ERR_INVALID, "bytes is NULL");
    const Operand x(args->x, args->n_tokens, args->in_features, args->x_stride),
        w(args->weight, args->out_features, args->in_features, args->weight_stride);
    *bytes = args->n_tokens ? x.packed + w.packed : 0;
    return MUON_OK;
  });
}

extern "C" int muon_linear(const muon_linear_args_t* args, void* workspace, size_t workspace_bytes, void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_linear");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    Forward f{};
    int rc = check_forward(args, &f);
    if (rc != MUON_OK) return rc;
    const muon_linear_args_t& a = *args;
    const int64_t T = a.n_tokens;
    const int K = a.in_features, N = a.out_features;
    if (T == 0) return MUON_OK;
    Operand x(a.x, T, K, a.x_stride), w(a.weight, N, K, a.weight_stride);
    if (takes_rows(T, K, N, !x.packed && !w.packed)) {
      if ((rc = lay::begin_call()) != MUON_OK) return rc;
      return lay::end_call(1, launch_rows(x, w, f, static_cast<cudaStream_t>(stream)));
    }
    const size_t es = dtype_bytes(a.out_dtype);
    if ((rc = check_workspace(workspace, workspace_bytes, x.packed + w.packed,
                              {Span(a.x, T, a.x_stride, K, 2), Span(a.weight, N, a.weight_stride, K, 2),
                               Span(a.bias, 1, N, N, dtype_bytes(a.bias_dtype)),
                               Span(a.residual, T, a.residual_stride, N, es), Span(a.out, T, a.out_stride, N, es),
                               Span(a.pre, T, a.pre_stride, N, 2),
                               Span(f.drop.least ? a.rng : nullptr, 1, 2, 2, 8)})) != MUON_OK ||
        (rc = lay::begin_call()) != MUON_OK)
      return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* at = static_cast<char*>(workspace);
    int launches = 0;
    Packs packs{};
    x.pack(&at, &packs);
    w.pack(&at, &packs);
    static One<Forward> product;   // large; this call holds the library lock
    const bool few = T <= kFewTokens;
    const bool more = a.activation != MUON_ACT_NONE || f.drop.least || a.pre || a.residual;
    const Plan plan = few ? plan_few(T, N, K) : offer_of(T, N, K, false, more, kSms).plan;
    if (!(few ? prepare(plan, w, false, x, false, f, &product) : prepare(plan, x, false, w, false, f, &product)))
      return fail_with(MUON_ERR_CUDA, "the driver refuses a map of x or weight");
    cudaError_t e = launch_packs(packs, s, &launches);
    if (e != cudaSuccess) return lay::end_call(launches, e);
    e = launch_one(plan, product, 0, s);
    return lay::end_call(launches + 1, e);
  });
}

extern "C" int muon_linear_grad_workspace(const muon_linear_grad_args_t* args, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    GradPlaces at;
    const int rc = check_grad(args, &at);
    if (rc != MUON_OK) return rc;
    if (!bytes) return fail_with(MUON_ERR_INVALID, "bytes is NULL");
    *bytes = grad_operands(*args).bytes();
    return MUON_OK;
  });
}

extern "C" int muon_linear_grad(const muon_linear_grad_args_t* args, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_linear_grad");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    GradPlaces places;
    int rc = check_grad(args, &places);
    if (rc != MUON_OK) return rc;
    const muon_linear_grad_args_t& a = *args;
    const int64_t T = a.n_tokens;
    const int K = a.in_features, N = a.out_features;
    const bool sums = a.param || a.bias, slope = a.dx && a.activation != MUON_ACT_NONE;
    if (T == 0 && !(sums && a.overwrite)) return MUON_OK;
    GradOperands o = grad_operands(a);
    if ((rc = check_workspace(workspace, workspace_bytes, o.bytes(),
                              {Span(a.dout, T, a.dout_stride, N, 2), Span(a.param ? a.x : nullptr, T, a.x_stride, K, 2),
                               Span(a.dx ? a.weight : nullptr, N, a.weight_stride, K, 2),
                               Span(slope ? a.pre : nullptr, T, a.pre_stride, K, 2), Span(a.dx, T, a.dx_stride, K, 2),
                               Span(sums ? a.accum : nullptr, 1, a.accum_elems, a.accum_elems, 4)})) != MUON_OK ||
        (rc = lay::begin_call()) != MUON_OK)
      return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* at = static_cast<char*>(workspace);
    int launches = 0;
    Packs packs{};
    o.dout.pack(&at, &packs);
    o.weight.pack(&at, &packs);
    o.x.pack(&at, &packs);
    InputGrad f{};
    auto matrix = [&](const void* p, int64_t stride) {
      return Matrix{const_cast<void*>(p), stride, 0, !misaligned(p, 16) && (T <= 1 || stride % 8 == 0)};
    };
    f.dx = matrix(a.dx, a.dx_stride);
    f.pre = matrix(a.pre, a.pre_stride);
    f.rows = T;
    f.cols = K;
    f.act = a.activation;
    WeightGrad g{};
    g.accum = a.accum;
    g.rows = N;
    g.cols = K;
    g.overwrite = a.overwrite;
    g.scale = a.scale;
    if (a.param) g.sg = places.weight;
    const bool dx = a.dx && T, dw = a.param, few = T <= kFewTokens;
    Plan plans[2];
    static One<InputGrad> first;    // large; this call holds the library lock
    static One<WeightGrad> second;
    bool fine = true;
    if (dx && dw) plan_both(T, K, N, slope, &plans[0], &plans[1]);
    else if (dx) plans[0] = few ? plan_few(T, K, N) : offer_of(T, K, N, false, slope, kSms).plan;
    else if (dw) plans[1] = offer_of(N, K, T, true, false, kSms).plan;
    if (dx)
      fine = few ? prepare(plans[0], o.weight, true, o.dout, false, f, &first)
                 : prepare(plans[0], o.dout, false, o.weight, true, f, &first);
    if (dw && fine) fine = prepare(plans[1], o.dout, true, o.x, true, g, &second);
    if (!fine) return fail_with(MUON_ERR_CUDA, "the driver refuses a map of an operand");
    cudaError_t e = launch_packs(packs, s, &launches);
    if (e != cudaSuccess) return lay::end_call(launches, e);
    // The call's kernels depend on copies of the operands alone: behind the first
    // that waits for those, they run beside one another.
    int late = 0;
    if (a.bias) {
      const BiasGrad b{static_cast<const __nv_bfloat16*>(o.dout.p ? o.dout.p : a.dout), o.dout.p ? o.dout.stride : a.dout_stride,
                       T, N, a.accum, a.scale, a.overwrite};
      if ((e = launch_bias(b, places.bias, s)) != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
      late = 1;
    }
    if (dx) {
      if ((e = launch_one(plans[0], first, late, s)) != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
      late = 1;
    }
    if (dw) {
      e = launch_one(plans[1], second, late, s);
      ++launches;
    }
    return lay::end_call(launches, e);
  });
}
