// C-ABI entry points of the hybrid layer's operators (declared in
// include/m2rnn.h): argument validation, workspace carving and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include "layer.cuh"

using namespace m2rnn;

namespace {

constexpr int kMaxDim = 128;
constexpr int64_t kMaxBlocks = INT_MAX;

bool dtype_ok(int dt) { return dt == M2RNN_F32 || dt == M2RNN_BF16; }
size_t elem(int dt) { return dt == M2RNN_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool given16(const void* p) { return p != nullptr && aligned(p, 16); }
bool opt16(const void* p) { return p == nullptr || aligned(p, 16); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? M2RNN_OK : M2RNN_ERR_CUDA; }

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uint64_t x = reinterpret_cast<uint64_t>(a), y = reinterpret_cast<uint64_t>(b);
  return x < y + nb && y < x + na;
}

// Bytes from the first to behind the last element of `rows` rows.
uint64_t span(int64_t rows, int64_t stride, int64_t width, size_t e) {
  return static_cast<uint64_t>((rows - 1) * stride + width) * e;
}

// M2RNN_OK, or what the call returns.
int conv_dims(int64_t B, int64_t T, int64_t C, int64_t W, int dt) {
  if (!dtype_ok(dt) || B < 1 || T < 1 || C < 1 || W < 1) return M2RNN_ERR_INVALID_ARG;
  if (B > INT_MAX / 8 || T > INT_MAX / 8 || C > INT_MAX / 8) return M2RNN_ERR_INVALID_ARG;
  if (W > kConvMaxWidth) return M2RNN_ERR_UNSUPPORTED;
  if (B * T > kMaxBlocks || B * T > INT64_MAX / 16 / C) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

int ssm_dims(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V, int dt) {
  if (!dtype_ok(dt) || B < 1 || T < 1 || N < 1 || G < 1 || K < 1 || V < 1) return M2RNN_ERR_INVALID_ARG;
  if (B > INT_MAX / 8 || T > INT_MAX / 8 || N > INT_MAX / 8 || N % G != 0) return M2RNN_ERR_INVALID_ARG;
  if (K > kMaxDim || V > kMaxDim) return M2RNN_ERR_UNSUPPORTED;
  if (B * N > INT_MAX / 8 || (T + 31) / 32 > kMaxBlocks / (B * N)) return M2RNN_ERR_UNSUPPORTED;
  return M2RNN_OK;
}

// The column-sliced inputs: given, aligned to an element, rows that do not overlap.
bool rows_ok(const void* p, int64_t stride, int64_t width, size_t e) {
  return p != nullptr && aligned(p, e) && stride >= width && stride <= INT_MAX / 8;
}

bool ssm_inputs_ok(const SsmArgs& a) {
  const size_t e = a.bf16 ? 2 : 4;
  return rows_ok(a.q, a.q_stride, static_cast<int64_t>(a.G) * a.K, e) &&
         rows_ok(a.k, a.k_stride, static_cast<int64_t>(a.G) * a.K, e) &&
         rows_ok(a.v, a.v_stride, static_cast<int64_t>(a.N) * a.V, e) && rows_ok(a.dt, a.dt_stride, a.N, e) &&
         given16(a.A) && opt16(a.dt_bias) && opt16(a.w_r) && opt16(a.H_0) &&
         (a.lengths == nullptr || aligned(a.lengths, 4));
}

// Whether an output overlaps the q, k, v that other blocks still read.
bool ssm_clobbers(const SsmArgs& a, const void* out, uint64_t bytes) {
  const size_t e = a.bf16 ? 2 : 4;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  return overlap(a.q, span(rows, a.q_stride, static_cast<int64_t>(a.G) * a.K, e), out, bytes) ||
         overlap(a.k, span(rows, a.k_stride, static_cast<int64_t>(a.G) * a.K, e), out, bytes) ||
         overlap(a.v, span(rows, a.v_stride, static_cast<int64_t>(a.N) * a.V, e), out, bytes);
}

SsmArgs ssm_args(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const void* dt, int64_t dt_stride, const float* A, const float* dt_bias, const void* w_r,
                 const float* H_0, const int32_t* lengths, int64_t B, int64_t T, int64_t N, int64_t G, int64_t K,
                 int64_t V, m2rnn_dtype dtype, void* ws) {
  SsmArgs a{};
  a.q = q; a.k = k; a.v = v; a.dt = dt; a.A = A; a.dt_bias = dt_bias; a.w_r = w_r; a.H_0 = H_0; a.lengths = lengths;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.dt_stride = dt_stride;
  a.B = static_cast<int>(B); a.T = static_cast<int>(T); a.N = static_cast<int>(N); a.G = static_cast<int>(G);
  a.K = static_cast<int>(K); a.V = static_cast<int>(V);
  a.bf16 = dtype == M2RNN_BF16;
  a.ws = ws;
  return a;
}

}  // namespace

extern "C" {

int m2rnn_causal_conv(const void* x, int64_t x_stride, const void* w, const void* bias, const void* x0,
                      const int32_t* lengths, void* y, void* x_T, int64_t B, int64_t T, int64_t C, int64_t W, int silu,
                      m2rnn_dtype dtype, void* cuda_stream) {
  const int st = conv_dims(B, T, C, W, dtype);
  if (st != M2RNN_OK) return st;
  const size_t e = elem(dtype);
  if (!rows_ok(x, x_stride, C, e) || !given16(w) || !opt16(bias) || !opt16(x0) || !given16(y) || !opt16(x_T) ||
      (lengths != nullptr && !aligned(lengths, 4)) || (silu != 0 && silu != 1))
    return M2RNN_ERR_INVALID_ARG;
  const uint64_t nx = span(B * T, x_stride, C, e), ny = static_cast<uint64_t>(B * T * C) * e,
                 ns = static_cast<uint64_t>(B * (W - 1) * C) * e;
  if (overlap(x, nx, y, ny) || overlap(x0, ns, y, ny) || overlap(x, nx, x_T, ns) || overlap(x0, ns, x_T, ns))
    return M2RNN_ERR_INVALID_ARG;
  ConvArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.x0 = x0; a.lengths = lengths; a.y = y; a.x_T = x_T; a.x_stride = x_stride;
  a.B = static_cast<int>(B); a.T = static_cast<int>(T); a.C = static_cast<int>(C); a.W = static_cast<int>(W);
  a.silu = silu != 0; a.bf16 = dtype == M2RNN_BF16;
  return cuda_status(launch_conv_forward(a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_causal_conv_backward_workspace_size(int64_t B, int64_t T, int64_t C, int64_t W) {
  if (conv_dims(B, T, C, W, M2RNN_F32) != M2RNN_OK) return 0;
  return sizeof(float) * static_cast<size_t>(conv_backward_parts(B, T, C)) * (W + 1) * C;
}

int m2rnn_causal_conv_backward(const void* x, int64_t x_stride, const void* w, const void* bias, const void* x0,
                               const int32_t* lengths, const float* dy, const float* dx_T, float* dx, float* dw,
                               float* db, float* dx0, int64_t B, int64_t T, int64_t C, int64_t W, int silu,
                               m2rnn_dtype dtype, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const int st = conv_dims(B, T, C, W, dtype);
  if (st != M2RNN_OK) return st;
  const size_t e = elem(dtype);
  if (!rows_ok(x, x_stride, C, e) || !given16(w) || !opt16(bias) || !opt16(x0) || !given16(dy) || !opt16(dx_T) ||
      !given16(dx) || !given16(dw) || !opt16(db) || !opt16(dx0) || (lengths != nullptr && !aligned(lengths, 4)) ||
      (silu != 0 && silu != 1))
    return M2RNN_ERR_INVALID_ARG;
  const uint64_t n = static_cast<uint64_t>(B * T * C) * 4, ns = static_cast<uint64_t>(B * (W - 1) * C) * 4;
  if (overlap(x, span(B * T, x_stride, C, e), dx, n) || overlap(dy, n, dx, n) || overlap(dx_T, ns, dx0, ns) || overlap(dx_T, ns, dx, n) || overlap(dy, n, dx0, ns))
    return M2RNN_ERR_INVALID_ARG;
  if (!given16(workspace) || workspace_bytes < m2rnn_causal_conv_backward_workspace_size(B, T, C, W))
    return M2RNN_ERR_WORKSPACE;
  ConvArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.x0 = x0; a.lengths = lengths; a.dy = dy; a.dx_T = dx_T; a.dx = dx; a.dw = dw;
  a.db = db; a.dx0 = dx0; a.x_stride = x_stride; a.part = static_cast<float*>(workspace);
  a.B = static_cast<int>(B); a.T = static_cast<int>(T); a.C = static_cast<int>(C); a.W = static_cast<int>(W);
  a.silu = silu != 0; a.bf16 = dtype == M2RNN_BF16;
  return cuda_status(launch_conv_backward(a, static_cast<cudaStream_t>(cuda_stream)));
}

int m2rnn_causal_conv_step(void* state, const void* x, int64_t x_stride, const void* w, const void* bias, void* y,
                           int64_t B, int64_t C, int64_t W, int silu, m2rnn_dtype dtype, void* cuda_stream) {
  const int st = conv_dims(B, 1, C, W, dtype);
  if (st != M2RNN_OK) return st;
  const size_t e = elem(dtype);
  if (!rows_ok(x, x_stride, C, e) || !given16(w) || !opt16(bias) || !given16(y) || (W > 1 && !given16(state)) ||
      (silu != 0 && silu != 1))
    return M2RNN_ERR_INVALID_ARG;
  const uint64_t nx = span(B, x_stride, C, e), ny = static_cast<uint64_t>(B * C) * e, ns = ny * (W - 1);
  if (overlap(state, ns, x, nx) || overlap(state, ns, y, ny) || overlap(x, nx, y, ny)) return M2RNN_ERR_INVALID_ARG;
  ConvArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.y = y; a.x_stride = x_stride;
  a.B = static_cast<int>(B); a.T = 1; a.C = static_cast<int>(C); a.W = static_cast<int>(W);
  a.silu = silu != 0; a.bf16 = dtype == M2RNN_BF16;
  return cuda_status(launch_conv_step(state, a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_ssm_workspace_size(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V, m2rnn_dtype dtype) {
  if (ssm_dims(B, T, N, G, K, V, dtype) != M2RNN_OK) return 0;
  return ssm_forward_scratch_bytes(B, T, N, K, V, dtype == M2RNN_BF16);
}

int m2rnn_ssm_scan(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                   const void* dt, int64_t dt_stride, const float* A, const float* dt_bias, const void* w_r,
                   const float* H_0, const int32_t* lengths, void* y, float* H_T, int64_t B, int64_t T, int64_t N,
                   int64_t G, int64_t K, int64_t V, m2rnn_dtype dtype, void* workspace, size_t workspace_bytes,
                   void* cuda_stream) {
  const int st = ssm_dims(B, T, N, G, K, V, dtype);
  if (st != M2RNN_OK) return st;
  SsmArgs a = ssm_args(q, q_stride, k, k_stride, v, v_stride, dt, dt_stride, A, dt_bias, w_r, H_0, lengths, B, T, N, G,
                       K, V, dtype, workspace);
  if (!ssm_inputs_ok(a) || !given16(y) || !opt16(H_T)) return M2RNN_ERR_INVALID_ARG;
  if (ssm_clobbers(a, y, static_cast<uint64_t>(B * T) * N * V * elem(dtype))) return M2RNN_ERR_INVALID_ARG;
  if (!given16(workspace) || workspace_bytes < m2rnn_ssm_workspace_size(B, T, N, G, K, V, dtype))
    return M2RNN_ERR_WORKSPACE;
  a.y = y;
  a.H_T = H_T;
  return cuda_status(launch_ssm_forward(a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_ssm_backward_workspace_size(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V,
                                         m2rnn_dtype dtype) {
  if (ssm_dims(B, T, N, G, K, V, dtype) != M2RNN_OK) return 0;
  return ssm_backward_scratch_bytes(B, T, N, G, K, V, dtype == M2RNN_BF16);
}

int m2rnn_ssm_scan_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const void* dt, int64_t dt_stride, const float* A, const float* dt_bias,
                            const void* w_r, const float* H_0, const int32_t* lengths, const void* dy,
                            const float* dH_T, float* dq, float* dk, float* dv, float* ddt, float* dA, float* ddt_bias,
                            float* dw_r, float* dH_0, int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V,
                            m2rnn_dtype dtype, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  const int st = ssm_dims(B, T, N, G, K, V, dtype);
  if (st != M2RNN_OK) return st;
  SsmArgs a = ssm_args(q, q_stride, k, k_stride, v, v_stride, dt, dt_stride, A, dt_bias, w_r, H_0, lengths, B, T, N, G,
                       K, V, dtype, workspace);
  const void* req[] = {dy, dq, dk, dv, ddt, dA};
  const void* opt[] = {dH_T, ddt_bias, dw_r, dH_0};
  if (!ssm_inputs_ok(a)) return M2RNN_ERR_INVALID_ARG;
  for (const void* p : req)
    if (!given16(p)) return M2RNN_ERR_INVALID_ARG;
  for (const void* p : opt)
    if (!opt16(p)) return M2RNN_ERR_INVALID_ARG;
  const uint64_t rows = static_cast<uint64_t>(B * T), nqk = rows * G * K * 4, nv = rows * N * V * 4;
  const uint64_t ny = rows * N * V * elem(dtype);
  if (ssm_clobbers(a, dq, nqk) || ssm_clobbers(a, dk, nqk) || ssm_clobbers(a, dv, nv) || overlap(dy, ny, dq, nqk) ||
      overlap(dy, ny, dk, nqk) || overlap(dy, ny, dv, nv))
    return M2RNN_ERR_INVALID_ARG;
  if (!given16(workspace) || workspace_bytes < m2rnn_ssm_backward_workspace_size(B, T, N, G, K, V, dtype))
    return M2RNN_ERR_WORKSPACE;
  a.dy = dy; a.dH_T = dH_T; a.dq = dq; a.dk = dk; a.dv = dv; a.ddt = ddt; a.dA = dA; a.ddt_bias = ddt_bias;
  a.dw_r = dw_r; a.dH_0 = dH_0;
  return cuda_status(launch_ssm_backward(a, static_cast<cudaStream_t>(cuda_stream)));
}

int m2rnn_ssm_step(float* H, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, const void* dt, int64_t dt_stride, const float* A, const float* dt_bias,
                   const void* w_r, void* y, int64_t B, int64_t N, int64_t G, int64_t K, int64_t V, m2rnn_dtype dtype,
                   void* cuda_stream) {
  const int st = ssm_dims(B, 1, N, G, K, V, dtype);
  if (st != M2RNN_OK) return st;
  SsmArgs a = ssm_args(q, q_stride, k, k_stride, v, v_stride, dt, dt_stride, A, dt_bias, w_r, nullptr, nullptr, B, 1, N,
                       G, K, V, dtype, nullptr);
  if (!ssm_inputs_ok(a) || !given16(H) || !given16(y)) return M2RNN_ERR_INVALID_ARG;
  a.y = y;
  return cuda_status(launch_ssm_step(H, a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t m2rnn_grad_plan_size(int64_t n, const int64_t* counts) {
  if (n < 0 || (n > 0 && counts == nullptr)) return 0;
  int64_t chunks = 1;  // the first entry holds the number of pieces
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || counts[i] > INT64_MAX / 64) return 0;
    chunks += (counts[i] + kGradChunk - 1) / kGradChunk;
    if (chunks > kMaxBlocks) return 0;
  }
  return static_cast<size_t>(chunks) * sizeof(GradChunk);
}

int m2rnn_grad_plan_build(int64_t n, const void* const* grads, void* const* outs, const int64_t* counts,
                          const int32_t* dtypes, void* plan, size_t plan_bytes) {
  const size_t need = m2rnn_grad_plan_size(n, counts);
  if (need == 0 || plan == nullptr || (n > 0 && (grads == nullptr || dtypes == nullptr))) return M2RNN_ERR_INVALID_ARG;
  if (plan_bytes < need) return M2RNN_ERR_WORKSPACE;
  GradChunk* at = static_cast<GradChunk*>(plan);
  std::memset(at, 0, sizeof(GradChunk));
  ++at;
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    if (!dtype_ok(dtypes[i])) return M2RNN_ERR_INVALID_ARG;
    const size_t e = elem(dtypes[i]);
    const char* in = static_cast<const char*>(grads[i]);
    char* out = outs != nullptr ? static_cast<char*>(outs[i]) : const_cast<char*>(in);
    if (in == nullptr || out == nullptr || !aligned(in, e) || !aligned(out, e)) return M2RNN_ERR_INVALID_ARG;
    if (in != out && overlap(in, counts[i] * e, out, counts[i] * e)) return M2RNN_ERR_INVALID_ARG;
    for (int64_t o = 0; o < counts[i]; o += kGradChunk, ++at) {
      const int64_t c = counts[i] - o < kGradChunk ? counts[i] - o : kGradChunk;
      *at = GradChunk{in + o * e, out + o * e, static_cast<int32_t>(c), dtypes[i] == M2RNN_BF16 ? 1 : 0, 0};
    }
  }
  return M2RNN_OK;
}

size_t m2rnn_grad_workspace_size(void) { return grad_clip_scratch_bytes(); }

}  // extern "C"

namespace {

int grad_call(const void* plan, size_t plan_bytes, float max_norm, bool clip, float* norm, void* workspace,
              size_t workspace_bytes, void* cuda_stream) {
  if (!given16(plan) || plan_bytes < sizeof(GradChunk) || plan_bytes % sizeof(GradChunk) != 0 || norm == nullptr ||
      !aligned(norm, 4) || !(max_norm > 0.f))
    return M2RNN_ERR_INVALID_ARG;
  if (!given16(workspace) || workspace_bytes < grad_clip_scratch_bytes()) return M2RNN_ERR_WORKSPACE;
  return cuda_status(launch_grad_clip(static_cast<const GradChunk*>(plan) + 1,
                                      static_cast<int64_t>(plan_bytes / sizeof(GradChunk)) - 1, max_norm, clip, norm,
                                      workspace, static_cast<cudaStream_t>(cuda_stream)));
}

}  // namespace

extern "C" {

int m2rnn_grad_norm(const void* plan, size_t plan_bytes, float* norm, void* workspace, size_t workspace_bytes,
                    void* cuda_stream) {
  return grad_call(plan, plan_bytes, 1.f, false, norm, workspace, workspace_bytes, cuda_stream);
}

int m2rnn_grad_clip(const void* plan, size_t plan_bytes, float max_norm, float* norm, void* workspace,
                    size_t workspace_bytes, void* cuda_stream) {
  return grad_call(plan, plan_bytes, max_norm, true, norm, workspace, workspace_bytes, cuda_stream);
}

}  // extern "C"
