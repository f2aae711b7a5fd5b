// Gated linear recurrence on a vector state, per batch element and channel,
// from H_0, with the gate of the matrix-state scans (gate.cuh):
//     f_t = exp(-alpha softplus(a_t + beta)),
//     h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t.
// Backward, with dh the gradient of h:
//     dh_t = dy_t + f_{t+1} dh_{t+1},   dx_t = (1 - f_t) dh_t,
//     g_t = dh_t f_t (h_{t-1} - x_t)  (= dL / d log f_t),
//     da_t = -alpha sigmoid(a_t + beta) g_t,
//     dalpha = -sum softplus(a_t + beta) g_t,  dbeta = sum da_t,
//     dH_0 = f_1 dh_1.
// A thread per channel.
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;

struct Gate {
  float f, e, soft, sig;  // e = 1 - f
};
__device__ __forceinline__ Gate gate_of(float z, float alpha) {
  Gate g;
  const float t = expf(-fabsf(z));
  g.soft = fmaxf(z, 0.f) + log1pf(t);
  g.sig = (z >= 0.f ? 1.f : t) / (1.f + t);
  g.e = -expm1f(-alpha * g.soft);
  g.f = expf(-alpha * g.soft);
  return g;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) linear_forward_kernel(LinearArgs A) {
  const int per = (A.C + kThreads - 1) / kThreads, b = blockIdx.x / per;
  const int c = (blockIdx.x - b * per) * kThreads + threadIdx.x;
  if (c >= A.C) return;
  const int len = A.lengths != nullptr ? min(max(A.lengths[b], 0), A.T) : A.T;
  const E* x = static_cast<const E*>(A.x) + static_cast<int64_t>(b) * A.T * A.x_stride + c;
  const E* a = static_cast<const E*>(A.a) + static_cast<int64_t>(b) * A.T * A.a_stride + c;
  E* y = static_cast<E*>(A.y) + static_cast<int64_t>(b) * A.T * A.C + c;
  const float alpha = A.alpha[c], beta = A.beta != nullptr ? A.beta[c] : 0.f;
  float h = A.H_0 != nullptr ? A.H_0[static_cast<int64_t>(b) * A.C + c] : 0.f;
  for (int t = 0; t < len; ++t) {
    const Gate g = gate_of(to_f32(a[t * A.a_stride]) + beta, alpha);
    h = fmaf(g.f, h, g.e * to_f32(x[t * A.x_stride]));
    y[static_cast<int64_t>(t) * A.C] = from_f32<E>(h);
  }
  for (int t = len; t < A.T; ++t) y[static_cast<int64_t>(t) * A.C] = from_f32<E>(0.f);
  if (A.H_T != nullptr) A.H_T[static_cast<int64_t>(b) * A.C + c] = h;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) linear_backward_kernel(LinearArgs A) {
  const int per = (A.C + kThreads - 1) / kThreads, b = blockIdx.x / per;
  const int c = (blockIdx.x - b * per) * kThreads + threadIdx.x;
  if (c >= A.C) return;
  const int len = A.lengths != nullptr ? min(max(A.lengths[b], 0), A.T) : A.T;
  const E* x = static_cast<const E*>(A.x) + static_cast<int64_t>(b) * A.T * A.x_stride + c;
  const E* a = static_cast<const E*>(A.a) + static_cast<int64_t>(b) * A.T * A.a_stride + c;
  const int64_t at = static_cast<int64_t>(b) * A.T * A.C + c, state = static_cast<int64_t>(b) * A.C + c;
  const float alpha = A.alpha[c], beta = A.beta != nullptr ? A.beta[c] : 0.f;
  float h = A.H_0 != nullptr ? A.H_0[state] : 0.f;
  for (int t = 0; t < len; ++t) {  // dx holds h_{t-1} - x_t until its own turn
    const Gate g = gate_of(to_f32(a[t * A.a_stride]) + beta, alpha);
    const float v = to_f32(x[t * A.x_stride]);
    A.dx[at + static_cast<int64_t>(t) * A.C] = h - v;
    h = fmaf(g.f, h, g.e * v);
  }
  float carry = A.dH_T != nullptr ? A.dH_T[state] : 0.f, sa = 0.f, sb = 0.f;
  for (int t = A.T - 1; t >= len; --t) A.dx[at + static_cast<int64_t>(t) * A.C] = A.da[at + static_cast<int64_t>(t) * A.C] = 0.f;
  for (int t = len - 1; t >= 0; --t) {
    const int64_t i = at + static_cast<int64_t>(t) * A.C;
    const Gate g = gate_of(to_f32(a[t * A.a_stride]) + beta, alpha);
    const float dh = to_f32(static_cast<const E*>(A.dy)[i]) + carry;
    carry = g.f * dh;
    const float lf = carry * A.dx[i];
    A.dx[i] = g.e * dh;
    A.da[i] = -alpha * g.sig * lf;
    sb += A.da[i];
    sa -= g.soft * lf;
  }
  if (A.dH_0 != nullptr) A.dH_0[state] = carry;
  float* part = static_cast<float*>(A.ws) + static_cast<int64_t>(b) * 2 * A.C;
  part[c] = sa;
  part[A.C + c] = sb;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(float* H, LinearArgs A) {
  const int per = (A.C + kThreads - 1) / kThreads, b = blockIdx.x / per;
  const int c = (blockIdx.x - b * per) * kThreads + threadIdx.x;
  if (c >= A.C) return;
  const float beta = A.beta != nullptr ? A.beta[c] : 0.f;
  const Gate g = gate_of(to_f32(static_cast<const E*>(A.a)[b * A.a_stride + c]) + beta, A.alpha[c]);
  const int64_t i = static_cast<int64_t>(b) * A.C + c;
  const float h = fmaf(g.f, H[i], g.e * to_f32(static_cast<const E*>(A.x)[b * A.x_stride + c]));
  H[i] = h;
  static_cast<E*>(A.y)[i] = from_f32<E>(h);
}

__global__ void __launch_bounds__(256) sum_parts_kernel(const float* part, float* out, float* out2, int parts, int64_t D,
                                                        int64_t width) {
  wait_previous();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= width) return;
  float t = 0.f;
  for (int p = 0; p < parts; ++p) t += part[p * width + j];
  if (j < D)
    out[j] = t;
  else if (out2 != nullptr)
    out2[j - D] = t;
}

}  // namespace

size_t linear_backward_scratch_bytes(int64_t B, int64_t T, int64_t C) { return static_cast<size_t>(B) * 2 * C * 4; }

cudaError_t launch_sum_parts(const float* part, float* out, float* out2, bool two, int parts, int64_t D,
                             cudaStream_t s) {
  const int64_t width = two ? 2 * D : D;
  sum_parts_kernel<<<static_cast<unsigned>((width + 255) / 256), 256, 0, s>>>(part, out, out2, parts, D, width);
  return cudaGetLastError();
}

cudaError_t launch_linear_forward(const LinearArgs& a, cudaStream_t s) {
  const int grid = (a.C + kThreads - 1) / kThreads * a.B;
  if (a.bf16)
    linear_forward_kernel<uint16_t><<<grid, kThreads, 0, s>>>(a);
  else
    linear_forward_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s) {
  const int grid = (a.C + kThreads - 1) / kThreads * a.B;
  if (a.bf16)
    linear_backward_kernel<uint16_t><<<grid, kThreads, 0, s>>>(a);
  else
    linear_backward_kernel<float><<<grid, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_sum_parts(static_cast<const float*>(a.ws), a.dalpha, a.dbeta, true, a.B, a.C, s);
}

cudaError_t launch_linear_step(float* H, const LinearArgs& a, cudaStream_t s) {
  const int grid = (a.C + kThreads - 1) / kThreads * a.B;
  if (a.bf16)
    linear_step_kernel<uint16_t><<<grid, kThreads, 0, s>>>(H, a);
  else
    linear_step_kernel<float><<<grid, kThreads, 0, s>>>(H, a);
  return cudaGetLastError();
}

}  // namespace m2rnn
