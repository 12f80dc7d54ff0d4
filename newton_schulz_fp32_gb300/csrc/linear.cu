// A dense layer: the product of tokens and weight with bias, activation,
// dropout and residual, and its gradients: dx through the activation before the
// layer, and the weight's and bias's summed straight into the flat,
// partitioned FP32 accumulation buffer.
#include "layers.cuh"

namespace muon {
namespace {

using lay::Draw;
using lay::Dropout;
using lay::Span;

__device__ int g_linear_err;

// ------------------------------------------------------------------ epilogues

// out = residual + dropout(activation(acc + bias)), pre = acc + bias.
struct Forward {
  const void* bias;
  __nv_bfloat16* pre;
  const void* residual;
  void* out;
  int64_t pre_stride, res_stride, out_stride;
  int bias32, out32, act;
  Dropout drop;

  __device__ __forceinline__ void put(float v, int64_t t, int64_t n, const Draw& draw) const {
    if (bias) v += bias32 ? static_cast<const float*>(bias)[n]
                          : tok::to_float(static_cast<const __nv_bfloat16*>(bias)[n]);
    if (pre) pre[t * pre_stride + n] = __float2bfloat16_rn(v);
    v = lay::activation(v, act);
    if (drop.least)
      v = lay::dropped(v, lay::draw_of(draw.at(uint32_t(t), uint32_t(n / 8), drop.site), int(n % 8)), drop);
    if (out32) {
      if (residual) v += static_cast<const float*>(residual)[t * res_stride + n];
      static_cast<float*>(out)[t * out_stride + n] = v;
    } else {
      if (residual) v += tok::to_float(static_cast<const __nv_bfloat16*>(residual)[t * res_stride + n]);
      static_cast<__nv_bfloat16*>(out)[t * out_stride + n] = __float2bfloat16_rn(v);
    }
  }
};

// dx = acc * activation'(pre).
struct InputGrad {
  const __nv_bfloat16* pre;
  __nv_bfloat16* dx;
  int64_t pre_stride, dx_stride;
  int act;

  __device__ __forceinline__ void put(float v, int64_t t, int64_t k, const Draw&) const {
    if (act != MUON_ACT_NONE) v *= lay::slope(tok::to_float(pre[t * pre_stride + k]), act);
    dx[t * dx_stride + k] = __float2bfloat16_rn(v);
  }
};

// accum = (overwrite ? 0 : accum) + scale * acc, at the parameter's place.
struct WeightGrad {
  float* accum;
  int64_t cols;
  float scale;
  int overwrite;
  Segments sg;

  __device__ __forceinline__ void put(float v, int64_t n, int64_t k, const Draw&) const {
    int64_t room;
    float* p = accum + sg.place(n * cols + k, &room);
    *p = (overwrite ? 0.f : *p) + scale * v;
  }
};

// ------------------------------------------------------------------ product

// acc[m][n] = sum over k of A(m, k) B(n, k); element (r, k) of an operand lies at
// r * row + k * col.
struct Operands {
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  int64_t arow, acol, brow, bcol;
  int64_t m, n, k;
};

constexpr int kTile = 64, kDepth = 16;

template <typename Epilogue>
__global__ void __launch_bounds__(256) k_product(const Operands p, const __grid_constant__ Epilogue e,
                                                 const Dropout drop) {
  __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
  const int64_t tiles_n = (p.n + kTile - 1) / kTile;
  const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
      const int r = i / kDepth, k = i % kDepth;
      const bool in = k0 + k < p.k;
      sa[k][r] = in && m0 + r < p.m ? tok::to_float(p.a[(m0 + r) * p.arow + (k0 + k) * p.acol]) : 0.f;
      sb[k][r] = in && n0 + r < p.n ? tok::to_float(p.b[(n0 + r) * p.brow + (k0 + k) * p.bcol]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
    __syncthreads();
  }
  Draw draw;
  draw.init(drop);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < p.m && n < p.n) e.put(acc[i][j], m, n, draw);
    }
}

template <typename Epilogue>
cudaError_t launch_product(const Operands& p, const Epilogue& e, const Dropout& drop, cudaStream_t s) {
  const int64_t blocks = ((p.m + kTile - 1) / kTile) * ((p.n + kTile - 1) / kTile);
  return launch(k_product<Epilogue>, unsigned(blocks), 256, 1, false, s, 0, p, e, drop);
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

__global__ void __launch_bounds__(1024) k_bias_grad(const BiasGrad a, const __grid_constant__ Segments sg) {
  __shared__ float sums[32][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + x;
  float v = 0.f;
  if (c < a.cols)
    for (int64_t t = y; t < a.tokens; t += 32) v += tok::to_float(a.dout[t * a.stride + c]);
  sums[y][x] = v;
  __syncthreads();
  if (y || c >= a.cols) return;
  for (int q = 1; q < 32; ++q) v += sums[q][x];
  int64_t room;
  float* p = a.accum + sg.place(c, &room);
  *p = (a.overwrite ? 0.f : *p) + a.scale * v;
}

// ------------------------------------------------------------------ host

constexpr int kMostFeatures = 1 << 24;

int check_sizes(int64_t tokens, int in, int out, int act) {
  if (tokens < 0 || tokens > (int64_t(1) << 30)) return fail_with(MUON_ERR_INVALID, "n_tokens must be in [0, 2^30]");
  if (in < 1 || out < 1 || in > kMostFeatures || out > kMostFeatures)
    return fail_with(MUON_ERR_INVALID, "in_features and out_features must be in [1, 2^24]");
  if (act < MUON_ACT_NONE || act > MUON_ACT_SILU) return fail_with(MUON_ERR_INVALID, "unknown activation");
  auto tiles = [](int64_t a, int64_t b) { return ((a + kTile - 1) / kTile) * ((b + kTile - 1) / kTile); };
  if (tiles(tokens, out) > 0x7fffffff || tiles(tokens, in) > 0x7fffffff || tiles(in, out) > 0x7fffffff)
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
  f->bias = a->bias;
  f->bias32 = a->bias_dtype == MUON_DTYPE_FP32;
  f->pre = static_cast<__nv_bfloat16*>(a->pre);
  f->pre_stride = a->pre_stride;
  f->residual = a->residual;
  f->res_stride = a->residual_stride;
  f->out = a->out;
  f->out_stride = a->out_stride;
  f->out32 = es == 4;
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

}  // namespace

int linear_take_device_error() { return take_flag(g_linear_err); }

}  // namespace muon

using namespace muon;

extern "C" int muon_linear_workspace(const muon_linear_args_t* args, size_t* bytes) {
  return entry([&]() -> int {
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    Forward f{};
    const int rc = check_forward(args, &f);
    if (rc != MUON_OK) return rc;
    if (!bytes) return fail_with(MUON_ERR_INVALID, "bytes is NULL");
    *bytes = 0;
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
    if (args->n_tokens == 0) return MUON_OK;
    if ((rc = lay::begin_call()) != MUON_OK) return rc;
    const Operands p{static_cast<const __nv_bfloat16*>(args->x), static_cast<const __nv_bfloat16*>(args->weight),
                     args->x_stride, 1, args->weight_stride, 1, args->n_tokens, args->out_features,
                     args->in_features};
    return lay::end_call(1, launch_product(p, f, f.drop, static_cast<cudaStream_t>(stream)));
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
    *bytes = 0;
    return MUON_OK;
  });
}

extern "C" int muon_linear_grad(const muon_linear_grad_args_t* args, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return entry([&]() -> int {
    NvtxRange nvtx_("muon_linear_grad");
    std::lock_guard<std::mutex> lk(library_mutex());
    set_last_error(nullptr);
    GradPlaces at;
    int rc = check_grad(args, &at);
    if (rc != MUON_OK) return rc;
    const muon_linear_grad_args_t& a = *args;
    const bool sums = a.param || a.bias;
    if (a.n_tokens == 0 && !(sums && a.overwrite)) return MUON_OK;
    if ((rc = lay::begin_call()) != MUON_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const __nv_bfloat16 *d = static_cast<const __nv_bfloat16*>(a.dout), *x = static_cast<const __nv_bfloat16*>(a.x),
                        *w = static_cast<const __nv_bfloat16*>(a.weight);
    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (a.dx && a.n_tokens) {
      const InputGrad f{static_cast<const __nv_bfloat16*>(a.pre), static_cast<__nv_bfloat16*>(a.dx), a.pre_stride,
                        a.dx_stride, a.activation};
      const Operands p{d, w, a.dout_stride, 1, 1, a.weight_stride, a.n_tokens, a.in_features, a.out_features};
      if ((e = launch_product(p, f, Dropout{}, s)) != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
    }
    if (a.param) {
      const WeightGrad f{a.accum, a.in_features, a.scale, a.overwrite, at.weight};
      const Operands p{d, x, 1, a.dout_stride, 1, a.x_stride, a.out_features, a.in_features, a.n_tokens};
      if ((e = launch_product(p, f, Dropout{}, s)) != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
    }
    if (a.bias) {
      const BiasGrad b{d, a.dout_stride, a.n_tokens, a.out_features, a.accum, a.scale, a.overwrite};
      e = launch(k_bias_grad, unsigned((a.out_features + 31) / 32), 1024, 1, false, s, 0, b, at.bias);
      if (e != cudaSuccess) return lay::end_call(launches, e);
      ++launches;
    }
    return lay::end_call(launches, cudaSuccess);
  });
}
