// gated.cu -- act(x Wg^T + bg) * (x Wu^T + bu), and its gradients.
//
// Backward, with a = x Wg^T + bg and b = x Wu^T + bu computed anew:
//   da = grad b act'(a), db = grad act(a)
//   dx = da Wg + db Wu, dWg = da^T x, dWu = db^T x, dbg and dbu the sums of da and db over rows.
#include <climits>

#include "activate.cuh"
#include "half.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace lm {
namespace {

constexpr int kTile = 32;

struct GatedParams {
  const void *x, *wg, *wu, *bg, *bu, *grad;
  void *out;          // y, or [rows][2][n]: da and db
  float *columns;     // [row tiles][2][n], sums of da and db, or null
  int64_t rows, k, n, x_row, g_row, u_row, out_row, grad_row;
  int32_t bias_f32, act;
};

template <typename T>
__device__ __forceinline__ float bias_of(const void *b, int f32, int64_t i) {
  if (!b) return 0.0f;
  return f32 ? static_cast<const float *>(b)[i] : to_f32(static_cast<const T *>(b)[i]);
}

// A CTA a tile of 32 x 32 outputs, 256 threads.
template <typename T, bool BACKWARD>
__global__ void __launch_bounds__(256) gated_tile(const GatedParams p) {
  __shared__ float sx[kTile][kTile + 1], sg[kTile][kTile + 1], su[kTile][kTile + 1];
  pdl_launch();
  pdl_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int c = threadIdx.x % 32, r = threadIdx.x / 32;
  float a[4] = {}, b[4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += kTile) {
    for (int i = r; i < kTile; i += 8) {
      const bool in = k0 + c < p.k;
      sx[i][c] = in && row0 + i < p.rows ? to_f32(static_cast<const T *>(p.x)[(row0 + i) * p.x_row + k0 + c]) : 0.0f;
      sg[i][c] = in && n0 + i < p.n ? to_f32(static_cast<const T *>(p.wg)[(n0 + i) * p.g_row + k0 + c]) : 0.0f;
      su[i][c] = in && n0 + i < p.n ? to_f32(static_cast<const T *>(p.wu)[(n0 + i) * p.u_row + k0 + c]) : 0.0f;
    }
    __syncthreads();
    for (int j = 0; j < kTile; ++j)
      for (int i = 0; i < 4; ++i) {
        a[i] = fmaf(sx[r + 8 * i][j], sg[c][j], a[i]);
        b[i] = fmaf(sx[r + 8 * i][j], su[c][j], b[i]);
      }
    __syncthreads();
  }
  const int64_t n = n0 + c;
  float sa = 0.0f, sb = 0.0f;
  for (int i = 0; i < 4 && n < p.n; ++i) {
    const int64_t row = row0 + r + 8 * i;
    if (row >= p.rows) break;
    const float za = a[i] + bias_of<T>(p.bg, p.bias_f32, n), zb = b[i] + bias_of<T>(p.bu, p.bias_f32, n);
    if (BACKWARD) {
      float slope;
      const float y = activate_slope_any(za, p.act, slope);
      const float g = to_f32(static_cast<const T *>(p.grad)[row * p.grad_row + n]);
      const float da = g * zb * slope, db = g * y;
      sa += da;
      sb += db;
      static_cast<T *>(p.out)[row * p.out_row + n] = from_f32<T>(da);
      static_cast<T *>(p.out)[row * p.out_row + p.n + n] = from_f32<T>(db);
    } else {
      static_cast<T *>(p.out)[row * p.out_row + n] = from_f32<T>(activate_any(za, p.act) * zb);
    }
  }
  if (!BACKWARD || !p.columns) return;
  sx[r][c] = sa;
  sg[r][c] = sb;
  __syncthreads();
  if (r >= 2 || n >= p.n) return;
  float s = 0.0f;
  for (int i = 0; i < 8; ++i) s += r == 0 ? sx[i][c] : sg[i][c];
  p.columns[(static_cast<int64_t>(blockIdx.y) * 2 + r) * p.n + n] = s;
}

// out[i][j] = sum over t of a[i][t] b[t][j], over two pairs of operands one after the other.
struct SumParams {
  const void *a[2], *b[2];
  void *out;
  int64_t rows, cols, terms, a_row, a_term, b_term[2], out_row;
  int32_t pairs;
};

template <typename T>
__global__ void __launch_bounds__(256) sum_tile(const SumParams p) {
  __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
  pdl_launch();
  pdl_wait();
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile, j0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int c = threadIdx.x % 32, r = threadIdx.x / 32;
  float s[4] = {};
  for (int q = 0; q < p.pairs; ++q)
    for (int64_t t0 = 0; t0 < p.terms; t0 += kTile) {
      for (int i = r; i < kTile; i += 8) {
        sa[i][c] = t0 + c < p.terms && i0 + i < p.rows
                       ? to_f32(static_cast<const T *>(p.a[q])[(i0 + i) * p.a_row + (t0 + c) * p.a_term]) : 0.0f;
        sb[i][c] = t0 + i < p.terms && j0 + c < p.cols
                       ? to_f32(static_cast<const T *>(p.b[q])[(t0 + i) * p.b_term[q] + j0 + c]) : 0.0f;
      }
      __syncthreads();
      for (int t = 0; t < kTile; ++t)
        for (int i = 0; i < 4; ++i) s[i] = fmaf(sa[r + 8 * i][t], sb[t][c], s[i]);
      __syncthreads();
    }
  for (int i = 0; i < 4; ++i)
    if (i0 + r + 8 * i < p.rows && j0 + c < p.cols)
      static_cast<T *>(p.out)[(i0 + r + 8 * i) * p.out_row + j0 + c] = from_f32<T>(s[i]);
}

// Joins the tiles' sums of da and db in their order.
template <typename T>
__global__ void __launch_bounds__(256) columns_kernel(const float *columns, int64_t tiles, int64_t n, void *dbg, void *dbu,
                                                      int f32) {
  pdl_launch();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= 2 * n) return;
  void *const to = i < n ? dbg : dbu;
  if (!to) return;
  float s = 0.0f;
  for (int64_t t = 0; t < tiles; ++t) s += columns[t * 2 * n + i];
  const int64_t at = i < n ? i : i - n;
  if (f32) {
    static_cast<float *>(to)[at] = s;
  } else {
    static_cast<T *>(to)[at] = from_f32<T>(s);
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

lm_status check(const lm_gated_args *a) {
  if (!a || a->rows < 0 || a->k < 0 || a->n < 0 || a->x_row_stride < 0 || a->gate_row_stride < 0 ||
      a->up_row_stride < 0 || a->out_row_stride < 0)
    return LM_ERR_INVALID_ARG;
  if (a->activation < LM_ACT_NONE || a->activation > LM_ACT_SIGMOID) return LM_ERR_INVALID_ARG;
  if (a->dtype != LM_F16 && a->dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if ((a->b_gate || a->b_up) && a->bias_dtype != LM_F32 && a->bias_dtype != a->dtype) return LM_ERR_UNSUPPORTED;
  const int64_t most = INT_MAX - 512;
  if (a->rows > most || a->n > most / 2 || a->k > most) return LM_ERR_UNSUPPORTED;
  for (const int64_t s : {a->x_row_stride, a->gate_row_stride, a->up_row_stride, a->out_row_stride})
    if (s > (1ll << 38)) return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

lm_status check_pointers(const lm_gated_args &a, const void *workspace) {
  if (a.k > 0 && (!a.x || !a.w_gate || !a.w_up)) return LM_ERR_INVALID_ARG;
  const size_t bias = a.bias_dtype == LM_F32 ? 4 : 2;
  if (!aligned(a.x, 2) || !aligned(a.w_gate, 2) || !aligned(a.w_up, 2) || !aligned(a.b_gate, bias) ||
      !aligned(a.b_up, bias) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  return LM_OK;
}

bool meets_inputs(const lm_gated_args &a, ByteRows out) {
  const int64_t bias = a.bias_dtype == LM_F32 ? 4 : 2;
  return (a.k > 0 && (rows_meet(out, {a.x, a.rows, a.x_row_stride * 2, a.k * 2}) ||
                      rows_meet(out, {a.w_gate, a.n, a.gate_row_stride * 2, a.k * 2}) ||
                      rows_meet(out, {a.w_up, a.n, a.up_row_stride * 2, a.k * 2}))) ||
         (a.b_gate && rows_meet(out, {a.b_gate, 1, 0, a.n * bias})) ||
         (a.b_up && rows_meet(out, {a.b_up, 1, 0, a.n * bias}));
}

GatedParams params(const lm_gated_args &a) {
  GatedParams p = {};
  p.x = a.x;
  p.wg = a.w_gate;
  p.wu = a.w_up;
  p.bg = a.b_gate;
  p.bu = a.b_up;
  p.rows = a.rows;
  p.k = a.k;
  p.n = a.n;
  p.x_row = a.x_row_stride;
  p.g_row = a.gate_row_stride;
  p.u_row = a.up_row_stride;
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.act = a.activation;
  return p;
}

lm_status tiles_of(int64_t rows, int64_t cols, dim3 *grid) {
  if (up(rows, kTile) > 65535) return LM_ERR_UNSUPPORTED;
  *grid = dim3(static_cast<unsigned>(up(cols, kTile)), static_cast<unsigned>(up(rows, kTile)));
  return LM_OK;
}

template <typename T>
lm_status sum(const SumParams &p, cudaStream_t s) {
  dim3 grid;
  if (p.rows == 0 || p.cols == 0) return LM_OK;
  if (lm_status st = tiles_of(p.rows, p.cols, &grid); st != LM_OK) return st;
  return launch_dependent(sum_tile<T>, grid, 256, 0, s, 1, p);
}

template <typename T>
lm_status backward(const lm_gated_backward_args &a, char *scratch, cudaStream_t s) {
  const lm_gated_args &f = a.forward;
  T *const da = reinterpret_cast<T *>(scratch);
  float *const columns = reinterpret_cast<float *>(scratch + up(f.rows * f.n * 4, 256) * 256);
  GatedParams p = params(f);
  p.out = da;
  p.out_row = 2 * f.n;
  p.grad = a.grad;
  p.grad_row = a.grad_row_stride;
  p.columns = a.db_gate || a.db_up ? columns : nullptr;
  dim3 grid;
  if (f.rows > 0 && f.n > 0) {
    if (lm_status st = tiles_of(f.rows, f.n, &grid); st != LM_OK) return st;
    if (lm_status st = launch_dependent(gated_tile<T, true>, grid, 256, 0, s, 1, p); st != LM_OK) return st;
  }
  if (a.dx) {
    SumParams q = {{da, da + f.n}, {f.w_gate, f.w_up}, a.dx, f.rows, f.k, f.n, 2 * f.n, 1,
                   {f.gate_row_stride, f.up_row_stride}, f.k, 2};
    if (lm_status st = sum<T>(q, s); st != LM_OK) return st;
  }
  for (int i = 0; i < 2; ++i)
    if (void *const dw = i ? a.dw_up : a.dw_gate) {
      SumParams q = {{da + i * f.n}, {f.x}, dw, f.n, f.k, f.rows, 1, 2 * f.n, {f.x_row_stride}, f.k, 1};
      if (lm_status st = sum<T>(q, s); st != LM_OK) return st;
    }
  if (p.columns && f.n > 0)
    return launch_dependent(columns_kernel<T>, dim3(static_cast<unsigned>(up(2 * f.n, 256))), 256, 0, s, 1, p.columns,
                            up(f.rows, kTile), f.n, a.db_gate, a.db_up, p.bias_f32);
  return LM_OK;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_gated_linear_workspace_size(const lm_gated_args *args, size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(args); st != LM_OK) return st;
  *bytes = 256;
  return LM_OK;
}

extern "C" lm_status lm_gated_linear(const lm_gated_args *args, void *workspace, size_t workspace_bytes,
                                     lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_gated_linear_workspace_size(args, &need); st != LM_OK) return st;
  const lm_gated_args &a = *args;
  if (a.rows == 0 || a.n == 0) return LM_OK;
  if (!a.out) return LM_ERR_INVALID_ARG;
  if (lm_status st = check_pointers(a, workspace); st != LM_OK) return st;
  if (!aligned(a.out, 2)) return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  if ((a.rows > 1 && a.out_row_stride < a.n) || meets_inputs(a, {a.out, a.rows, a.out_row_stride * 2, a.n * 2}))
    return LM_ERR_INVALID_ARG;
  GatedParams p = params(a);
  p.out = a.out;
  p.out_row = a.out_row_stride;
  dim3 grid;
  if (lm_status st = tiles_of(a.rows, a.n, &grid); st != LM_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launch_dependent(a.dtype == LM_F16 ? gated_tile<__half, false> : gated_tile<__nv_bfloat16, false>, grid, 256, 0,
                          s, 1, p);
}

extern "C" lm_status lm_gated_linear_backward_workspace_size(const lm_gated_backward_args *args, size_t *bytes) {
  using namespace lm;
  if (!args || !bytes || args->grad_row_stride < 0) return LM_ERR_INVALID_ARG;
  const lm_gated_args &f = args->forward;
  if (lm_status st = check(&f); st != LM_OK) return st;
  if (args->grad_row_stride > (1ll << 38)) return LM_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(256 + up(f.rows * f.n * 4, 256) * 256 + up(f.rows, kTile) * f.n * 8);
  return LM_OK;
}

extern "C" lm_status lm_gated_linear_backward(const lm_gated_backward_args *args, void *workspace,
                                              size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_gated_linear_backward_workspace_size(args, &need); st != LM_OK) return st;
  const lm_gated_backward_args &a = *args;
  const lm_gated_args &f = a.forward;
  void *const outs[] = {a.dx, a.dw_gate, a.dw_up, a.db_gate, a.db_up};
  const int64_t bias = f.bias_dtype == LM_F32 ? 4 : 2;
  const int64_t sizes[] = {f.rows * f.k * 2, f.n * f.k * 2, f.n * f.k * 2, f.n * bias, f.n * bias};
  bool any = false;
  for (int i = 0; i < 5; ++i) any = any || (outs[i] && sizes[i] > 0);
  if (!any) return LM_OK;
  if (f.rows > 0 && f.n > 0) {
    if (!a.grad) return LM_ERR_INVALID_ARG;
    if (lm_status st = check_pointers(f, workspace); st != LM_OK) return st;
  }
  if ((a.db_gate || a.db_up) && f.bias_dtype != LM_F32 && f.bias_dtype != f.dtype) return LM_ERR_UNSUPPORTED;
  for (int i = 0; i < 5; ++i)
    if (!aligned(outs[i], i < 3 ? 2 : static_cast<size_t>(bias))) return LM_ERR_MISALIGNED;
  if (!aligned(a.grad, 2) || !aligned(workspace, 16)) return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  for (int i = 0; i < 5; ++i) {
    if (!outs[i]) continue;
    const ByteRows out{outs[i], 1, 0, sizes[i]};
    if (meets_inputs(f, out) || rows_meet(out, {a.grad, f.rows, a.grad_row_stride * 2, f.n * 2})) return LM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[j] && rows_meet(out, {outs[j], 1, 0, sizes[j]})) return LM_ERR_INVALID_ARG;
  }
  char *const scratch = static_cast<char *>(workspace) + 256;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return f.dtype == LM_F16 ? backward<__half>(a, scratch, s) : backward<__nv_bfloat16>(a, scratch, s);
}
