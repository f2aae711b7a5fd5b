// C-ABI entry points of the residual norm, the gated linear recurrence and the
// orthogonalised update (declared in include/m2rnn.h): argument validation,
// workspace carving and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "around.cuh"

using namespace m2rnn;

namespace {

bool dtype_ok(int dt) { return dt == M2RNN_F32 || dt == M2RNN_BF16; }
size_t elem(int dt) { return dt == M2RNN_BF16 ? 2 : dt == M2RNN_E4M3 ? 1 : 4; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool given16(const void* p) { return p != nullptr && aligned(p, 16); }
bool opt16(const void* p) { return p == nullptr || aligned(p, 16); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? M2RNN_OK : M2RNN_ERR_CUDA; }

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uint64_t x = reinterpret_cast<uint64_t>(a), y = reinterpret_cast<uint64_t>(b);
  return x < y + nb && y < x + na;
}

// A piece of memory that a call reads or writes; none where p is null.
struct Span {
  const void* p;
  uint64_t bytes;
};

// Whether an output overlaps an input or another output; outs[0] may be ins[0]
// itself where `in_place` allows it.
template <int kOuts, int kIns>
bool clobbers(const Span (&outs)[kOuts], const Span (&ins)[kIns], bool in_place) {
  for (int o = 0; o < kOuts; ++o) {
    for (int i = 0; i < kIns; ++i)
      if (!(o == 0 && i == 0 && in_place && outs[0].p == ins[0].p) &&
          overlap(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes))
        return true;
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o].p, outs[o].bytes, outs[i].p, outs[i].bytes)) return true;
  }
  return false;
}

// Bytes from the first to behind the last element of `rows` rows.
uint64_t span(int64_t rows, int64_t stride, int64_t width, size_t e) {
  return static_cast<uint64_t>((rows - 1) * stride + width) * e;
}

// Rows that may be a column slice: given, aligned to an element, not overlapping.
bool rows_ok(const void* p, int64_t stride, int64_t width, size_t e) {
  return p != nullptr && aligned(p, e) && stride >= width && stride <= INT_MAX / 8;
}

int norm_dims(int64_t rows, int64_t D) {
  if (rows < 1 || D < 1) return M2RNN_ERR_INVALID_ARG;
  if (D > kNormMaxWidth || rows > INT_MAX / 8) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

bool eps_ok(float eps) { return eps >= 0.f && std::isfinite(eps); }

int linear_dims(int64_t B, int64_t T, int64_t C, int dt) {
  if (!dtype_ok(dt) || B < 1 || T < 1 || C < 1) return M2RNN_ERR_INVALID_ARG;
  if (B > INT_MAX / 8 || T > INT_MAX / 8 || C > INT_MAX / 8) return M2RNN_ERR_UNSUPPORTED;
  if (B * T > INT_MAX || B * ((C + 31) / 32) > INT_MAX / 32) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

LinearArgs linear_args(const void* x, int64_t x_stride, const void* a, int64_t a_stride, const float* alpha,
                       const float* beta, const float* H_0, const int32_t* lengths, int64_t B, int64_t T, int64_t C,
                       m2rnn_dtype dtype) {
  LinearArgs r{};
  r.x = x; r.a = a; r.alpha = alpha; r.beta = beta; r.H_0 = H_0; r.lengths = lengths;
  r.x_stride = x_stride; r.a_stride = a_stride;
  r.B = static_cast<int>(B); r.T = static_cast<int>(T); r.C = static_cast<int>(C);
  r.bf16 = dtype == M2RNN_BF16;
  return r;
}

bool linear_inputs_ok(const LinearArgs& a) {
  const size_t e = a.bf16 ? 2 : 4;
  return rows_ok(a.x, a.x_stride, a.C, e) && rows_ok(a.a, a.a_stride, a.C, e) && given16(a.alpha) && opt16(a.beta) &&
         opt16(a.H_0) && (a.lengths == nullptr || aligned(a.lengths, 4));
}

int ortho_dims(int64_t n, int64_t rows, int64_t cols) {
  if (n < 1 || rows < 1 || cols < 1) return M2RNN_ERR_INVALID_ARG;
  if (n > 65535 || rows > kOrthoMaxDim || cols > kOrthoMaxDim || n * rows * cols > (1ll << 38)) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

}  // namespace

extern "C" {

int m2rnn_residual_norm(const void* x, int64_t x_stride, const void* residual, const float* w, float eps, void* h, void* y,
                        float* scale, int64_t rows, int64_t D, m2rnn_dtype x_dtype, m2rnn_dtype h_dtype,
                        m2rnn_dtype y_dtype, void* cuda_stream) {
  const int st = norm_dims(rows, D);
  if (st != M2RNN_OK) return st;
  if (!dtype_ok(x_dtype) || !dtype_ok(h_dtype) || (!dtype_ok(y_dtype) && y_dtype != M2RNN_E4M3) || !eps_ok(eps))
    return M2RNN_ERR_INVALID_ARG;
  if (!rows_ok(x, x_stride, D, elem(x_dtype)) || !opt16(residual) || !given16(w) || !opt16(h) || !given16(y) ||
      !opt16(scale) || (scale != nullptr) != (y_dtype == M2RNN_E4M3) || (residual == nullptr && h != nullptr))
    return M2RNN_ERR_INVALID_ARG;
  const uint64_t n = static_cast<uint64_t>(rows) * D, nh = n * elem(h_dtype);
  const Span outs[] = {{h, nh}, {y, n * elem(y_dtype)},
                       {scale, static_cast<uint64_t>(rows) * ((D + kScaleBlock - 1) / kScaleBlock) * 4}};
  const Span ins[] = {{residual, nh}, {x, span(rows, x_stride, D, elem(x_dtype))}, {w, static_cast<uint64_t>(D) * 4}};
  if (clobbers(outs, ins, true)) return M2RNN_ERR_INVALID_ARG;
  NormRowsArgs a{};
  a.x = x; a.residual = residual; a.w = w; a.h = h; a.y = y; a.scale = scale;
  a.rows = rows; a.x_stride = x_stride; a.D = static_cast<int>(D); a.eps = eps;
  a.x_bf16 = x_dtype == M2RNN_BF16; a.h_bf16 = h_dtype == M2RNN_BF16; a.y_type = y_dtype;
  return cuda_status(launch_residual_norm(a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_residual_norm_backward_workspace_size(int64_t rows, int64_t D) {
  if (norm_dims(rows, D) != M2RNN_OK) return 0;
  return sizeof(float) * static_cast<size_t>(norm_rows_parts(rows, D)) * D;
}

int m2rnn_residual_norm_backward(const void* h, const float* w, const void* dy, const float* dh, float eps, float* dx,
                                 float* dw, int64_t rows, int64_t D, m2rnn_dtype h_dtype, m2rnn_dtype dy_dtype,
                                 void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const int st = norm_dims(rows, D);
  if (st != M2RNN_OK) return st;
  if (!dtype_ok(h_dtype) || !dtype_ok(dy_dtype) || !eps_ok(eps) || !given16(h) || !given16(w) || !given16(dy) ||
      !opt16(dh) || !given16(dx) || !given16(dw))
    return M2RNN_ERR_INVALID_ARG;
  const size_t need = m2rnn_residual_norm_backward_workspace_size(rows, D);
  if (!given16(workspace) || workspace_bytes < need) return M2RNN_ERR_WORKSPACE;
  const uint64_t n = static_cast<uint64_t>(rows) * D;
  const Span outs[] = {{dx, n * 4}, {dw, static_cast<uint64_t>(D) * 4}, {workspace, need}};
  const Span ins[] = {{dh, n * 4}, {h, n * elem(h_dtype)}, {w, static_cast<uint64_t>(D) * 4}, {dy, n * elem(dy_dtype)}};
  if (clobbers(outs, ins, true)) return M2RNN_ERR_INVALID_ARG;
  NormRowsArgs a{};
  a.h = const_cast<void*>(h); a.w = w; a.dy = dy; a.dh = dh; a.dx = dx; a.dw = dw; a.part = static_cast<float*>(workspace);
  a.rows = rows; a.D = static_cast<int>(D); a.eps = eps;
  a.h_bf16 = h_dtype == M2RNN_BF16; a.dy_bf16 = dy_dtype == M2RNN_BF16;
  return cuda_status(launch_residual_norm_backward(a, static_cast<cudaStream_t>(cuda_stream)));
}

int m2rnn_linear_scan(const void* x, int64_t x_stride, const void* a, int64_t a_stride, const float* alpha,
                      const float* beta, const float* H_0, const int32_t* lengths, void* y, float* H_T, int64_t B,
                      int64_t T, int64_t C, m2rnn_dtype dtype, void* cuda_stream) {
  const int st = linear_dims(B, T, C, dtype);
  if (st != M2RNN_OK) return st;
  LinearArgs r = linear_args(x, x_stride, a, a_stride, alpha, beta, H_0, lengths, B, T, C, dtype);
  if (!linear_inputs_ok(r) || !given16(y) || !opt16(H_T)) return M2RNN_ERR_INVALID_ARG;
  const size_t e = elem(dtype);
  const uint64_t state = static_cast<uint64_t>(B) * C * 4, chan = static_cast<uint64_t>(C) * 4;
  const Span outs[] = {{H_T, state}, {y, static_cast<uint64_t>(B) * T * C * e}};
  const Span ins[] = {{H_0, state}, {x, span(B * T, x_stride, C, e)}, {a, span(B * T, a_stride, C, e)}, {alpha, chan},
                      {beta, chan}, {lengths, static_cast<uint64_t>(B) * 4}};
  if (clobbers(outs, ins, true)) return M2RNN_ERR_INVALID_ARG;
  r.y = y; r.H_T = H_T;
  return cuda_status(launch_linear_forward(r, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_linear_backward_workspace_size(int64_t B, int64_t T, int64_t C) {
  return linear_dims(B, T, C, M2RNN_F32) != M2RNN_OK ? 0 : linear_backward_scratch_bytes(B, T, C);
}

int m2rnn_linear_scan_backward(const void* x, int64_t x_stride, const void* a, int64_t a_stride, const float* alpha,
                               const float* beta, const float* H_0, const int32_t* lengths, const void* dy,
                               const float* dH_T, float* dx, float* da, float* dalpha, float* dbeta, float* dH_0,
                               int64_t B, int64_t T, int64_t C, m2rnn_dtype dtype, void* workspace,
                               size_t workspace_bytes, void* cuda_stream) {
  const int st = linear_dims(B, T, C, dtype);
  if (st != M2RNN_OK) return st;
  LinearArgs r = linear_args(x, x_stride, a, a_stride, alpha, beta, H_0, lengths, B, T, C, dtype);
  if (!linear_inputs_ok(r) || !given16(dy) || !opt16(dH_T) || !given16(dx) || !given16(da) || !given16(dalpha) ||
      !opt16(dbeta) || !opt16(dH_0))
    return M2RNN_ERR_INVALID_ARG;
  const size_t e = elem(dtype), need = m2rnn_linear_backward_workspace_size(B, T, C);
  if (!given16(workspace) || workspace_bytes < need) return M2RNN_ERR_WORKSPACE;
  const uint64_t n = static_cast<uint64_t>(B) * T * C, state = static_cast<uint64_t>(B) * C * 4,
                 chan = static_cast<uint64_t>(C) * 4;
  const Span outs[] = {{dH_0, state}, {dx, n * 4}, {da, n * 4}, {dalpha, chan}, {dbeta, chan}, {workspace, need}};
  const Span ins[] = {{dH_T, state}, {x, span(B * T, x_stride, C, e)}, {a, span(B * T, a_stride, C, e)}, {alpha, chan},
                      {beta, chan}, {H_0, state}, {lengths, static_cast<uint64_t>(B) * 4}, {dy, n * e}};
  if (clobbers(outs, ins, true)) return M2RNN_ERR_INVALID_ARG;
  r.dy = dy; r.dH_T = dH_T; r.dx = dx; r.da = da; r.dalpha = dalpha; r.dbeta = dbeta; r.dH_0 = dH_0; r.ws = workspace;
  return cuda_status(launch_linear_backward(r, static_cast<cudaStream_t>(cuda_stream)));
}

int m2rnn_linear_step(float* H, const void* x, int64_t x_stride, const void* a, int64_t a_stride, const float* alpha,
                      const float* beta, void* y, int64_t B, int64_t C, m2rnn_dtype dtype, void* cuda_stream) {
  const int st = linear_dims(B, 1, C, dtype);
  if (st != M2RNN_OK) return st;
  LinearArgs r = linear_args(x, x_stride, a, a_stride, alpha, beta, nullptr, nullptr, B, 1, C, dtype);
  if (!linear_inputs_ok(r) || !given16(H) || !given16(y)) return M2RNN_ERR_INVALID_ARG;
  const size_t e = elem(dtype);
  const uint64_t n = static_cast<uint64_t>(B) * C, chan = static_cast<uint64_t>(C) * 4;
  const Span outs[] = {{H, n * 4}, {y, n * e}};
  const Span ins[] = {{x, span(B, x_stride, C, e)}, {a, span(B, a_stride, C, e)}, {alpha, chan}, {beta, chan}};
  if (clobbers(outs, ins, false)) return M2RNN_ERR_INVALID_ARG;
  r.y = y;
  return cuda_status(launch_linear_step(H, r, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_orthogonalize_workspace_size(int64_t n, int64_t rows, int64_t cols) {
  if (ortho_dims(n, rows, cols) != M2RNN_OK) return 0;
  return sizeof(StatusBlock) + ortho_scratch_bytes(n, rows, cols);
}

int m2rnn_orthogonalize(const void* g, void* out, int64_t n, int64_t rows, int64_t cols, int steps, float eps,
                        m2rnn_dtype dtype, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const int st = ortho_dims(n, rows, cols);
  if (st != M2RNN_OK) return st;
  if (!dtype_ok(dtype) || !given16(g) || !given16(out) || steps < 1 || steps > kOrthoMaxSteps || !eps_ok(eps))
    return M2RNN_ERR_INVALID_ARG;
  const uint64_t count = static_cast<uint64_t>(n) * rows * cols;
  if (!(out == g && dtype == M2RNN_BF16) && overlap(out, count * 2, g, count * elem(dtype))) return M2RNN_ERR_INVALID_ARG;
  const size_t need = m2rnn_orthogonalize_workspace_size(n, rows, cols);
  if (!given16(workspace) || workspace_bytes < need) return M2RNN_ERR_WORKSPACE;
  if (overlap(workspace, need, g, count * elem(dtype)) || overlap(workspace, need, out, count * 2))
    return M2RNN_ERR_INVALID_ARG;
  OrthoArgs a{};
  a.g = g; a.out = static_cast<uint16_t*>(out); a.status = static_cast<StatusBlock*>(workspace);
  a.ws = static_cast<char*>(workspace) + sizeof(StatusBlock);
  a.n = n; a.rows = static_cast<int>(rows); a.cols = static_cast<int>(cols); a.steps = steps; a.eps = eps;
  a.bf16 = dtype == M2RNN_BF16;
  return cuda_status(launch_orthogonalize(a, static_cast<cudaStream_t>(cuda_stream)));  // (clears the status block)
}

}  // extern "C"
