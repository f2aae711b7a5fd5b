// Short causal depthwise convolution with bias and SiLU, the layer that makes
// q, k and v from their projections ("M2RNN: Non-Linear RNNs with Matrix-
// Valued States for Scalable Language Modeling", Eq. 14-23 of the reading
// notes; width 4 there).  With xs = [x0 | x] along time (x0: the W - 1 inputs
// before the sequence, zero when not given), per channel c,
//     pre_t = b[c] + sum_w w[c][w] xs[t + w],   y_t = pre_t sigmoid(pre_t),
// and, with g_t = dy_t act'(pre_t) for t < length (0 behind it),
//     dxs[s] = sum_w w[c][w] g[s - w],  dw[c][w] = sum_{b,t} g_t xs[t + w],
//     db[c] = sum_{b,t} g_t.
#include <cuda_runtime.h>

#include <cstdint>

#include "layer.cuh"

namespace m2rnn {
namespace {

// x sigmoid(x); __expf and __fdividef are good to a few units of fp32 here.
__device__ __forceinline__ float silu_f(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// One thread per (b, t, c): the plain kernel.
template <typename T>
__global__ void conv_forward_kernel(ConvArgs A) {
  const int64_t n = static_cast<int64_t>(A.B) * A.T * A.C;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int c = static_cast<int>(i % A.C);
  const int64_t bt = i / A.C;
  const int t = static_cast<int>(bt % A.T), b = static_cast<int>(bt / A.T);
  const int len = A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
  const T* x = static_cast<const T*>(A.x) + static_cast<int64_t>(b) * A.T * A.x_stride + c;
  const T* x0 = static_cast<const T*>(A.x0);
  auto at = [&](int s) -> float {  // xs at x index s >= -(W - 1)
    if (s >= 0) return to_f32(x[s * A.x_stride]);
    return x0 ? to_f32(x0[(static_cast<int64_t>(b) * (A.W - 1) + s + A.W - 1) * A.C + c]) : 0.f;
  };
  float r = 0.f;
  if (t < len) {
    float p = A.bias ? to_f32(static_cast<const T*>(A.bias)[c]) : 0.f;
    for (int w = 0; w < A.W; ++w) p += to_f32(static_cast<const T*>(A.w)[c * A.W + w]) * at(t + w - (A.W - 1));
    r = A.silu ? silu_f(p) : p;
  }
  static_cast<T*>(A.y)[i] = from_f32<T>(r);
  if (A.x_T != nullptr && t == 0)
    for (int j = 0; j < A.W - 1; ++j)
      static_cast<T*>(A.x_T)[(static_cast<int64_t>(b) * (A.W - 1) + j) * A.C + c] = from_f32<T>(at(len + j - (A.W - 1)));
}

constexpr int kBwdStrip = 64;  // steps of one partial sum of dw, db

// One thread per (channel, strip of kBwdStrip steps).
template <typename T>
__global__ void conv_backward_kernel(ConvArgs A) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= A.C) return;
  const int strips = (A.T + kBwdStrip - 1) / kBwdStrip;
  const int b = blockIdx.y / strips, strip = blockIdx.y % strips;
  const int t0 = strip * kBwdStrip, t1 = min(A.T, t0 + kBwdStrip);
  const int len = A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
  const int W = A.W;
  const T* x = static_cast<const T*>(A.x) + static_cast<int64_t>(b) * A.T * A.x_stride + c;
  const T* x0 = static_cast<const T*>(A.x0);
  const float* dy = A.dy + static_cast<int64_t>(b) * A.T * A.C + c;
  float w[kConvMaxWidth], dw[kConvMaxWidth], db = 0.f;
  for (int j = 0; j < W; ++j) {
    w[j] = to_f32(static_cast<const T*>(A.w)[c * W + j]);
    dw[j] = 0.f;
  }
  const float bias = A.bias ? to_f32(static_cast<const T*>(A.bias)[c]) : 0.f;
  auto at = [&](int s) -> float {
    if (s >= 0) return to_f32(x[s * A.x_stride]);
    return x0 ? to_f32(x0[(static_cast<int64_t>(b) * (W - 1) + s + W - 1) * A.C + c]) : 0.f;
  };
  auto grad = [&](int t, bool add) -> float {
    if (t < 0 || t >= len) return 0.f;
    float p = bias;
    for (int j = 0; j < W; ++j) p += w[j] * at(t + j - (W - 1));
    float g = dy[static_cast<int64_t>(t) * A.C];
    if (A.silu) {
      const float sg = 1.f / (1.f + __expf(-p));
      g *= sg * (1.f + p * (1.f - sg));
    }
    if (add) {
      db += g;
      for (int j = 0; j < W; ++j) dw[j] += g * at(t + j - (W - 1));
    }
    return g;
  };
  // x index s gets sum over t = s .. s + W - 1 of g_t w[s - t + W - 1].
  for (int s = strip == 0 ? -(W - 1) : t0; s < t1; ++s) {
    float d = 0.f;
    for (int t = s; t < s + W; ++t) d += grad(t, t == s) * w[s - t + W - 1];
    if (A.dx_T != nullptr && s < len && s >= len - (W - 1))
      d += A.dx_T[(static_cast<int64_t>(b) * (W - 1) + s - len + W - 1) * A.C + c];
    if (s >= 0)
      A.dx[(static_cast<int64_t>(b) * A.T + s) * A.C + c] = d;
    else if (A.dx0 != nullptr)
      A.dx0[(static_cast<int64_t>(b) * (W - 1) + s + W - 1) * A.C + c] = d;
  }
  float* part = A.part + static_cast<int64_t>(blockIdx.y) * (W + 1) * A.C + c;
  for (int j = 0; j < W; ++j) part[static_cast<int64_t>(j) * A.C] = dw[j];
  part[static_cast<int64_t>(W) * A.C] = db;
}

// Fixed-order sum of the partials: thread (j, c) of [W + 1][C].
__global__ void conv_sum_parts_kernel(const float* part, float* dw, float* db, int parts, int C, int W) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, j = blockIdx.y;
  if (c >= C) return;
  float t = 0.f;
  for (int p = 0; p < parts; ++p) t += part[(static_cast<int64_t>(p) * (W + 1) + j) * C + c];
  if (j < W)
    dw[static_cast<int64_t>(c) * W + j] = t;
  else if (db != nullptr)
    db[c] = t;
}

template <typename T>
__global__ void conv_step_kernel(T* state, const T* x, int64_t x_stride, const T* w, const T* bias, T* y, int B, int C,
                                 int W, bool silu) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(B) * C) return;
  const int c = static_cast<int>(i % C), b = static_cast<int>(i / C);
  T* st = state + static_cast<int64_t>(b) * (W - 1) * C + c;
  const T xn = x[b * x_stride + c];
  float p = bias ? to_f32(bias[c]) : 0.f;
  for (int j = 0; j < W - 1; ++j) p += to_f32(w[c * W + j]) * to_f32(st[static_cast<int64_t>(j) * C]);
  p += to_f32(w[c * W + W - 1]) * to_f32(xn);
  for (int j = 0; j + 1 < W - 1; ++j) st[static_cast<int64_t>(j) * C] = st[static_cast<int64_t>(j + 1) * C];
  if (W > 1) st[static_cast<int64_t>(W - 2) * C] = xn;
  y[i] = from_f32<T>(silu ? silu_f(p) : p);
}

}  // namespace

int conv_backward_parts(int64_t B, int64_t T) { return static_cast<int>(B * ((T + kBwdStrip - 1) / kBwdStrip)); }

cudaError_t launch_conv_forward(const ConvArgs& a, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(a.B) * a.T * a.C;
  const unsigned grid = static_cast<unsigned>((n + 255) / 256);
  if (a.bf16)
    conv_forward_kernel<uint16_t><<<grid, 256, 0, s>>>(a);
  else
    conv_forward_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_conv_backward(const ConvArgs& a, cudaStream_t s) {
  const int parts = conv_backward_parts(a.B, a.T);
  const dim3 grid((a.C + 127) / 128, parts);
  if (a.bf16)
    conv_backward_kernel<uint16_t><<<grid, 128, 0, s>>>(a);
  else
    conv_backward_kernel<float><<<grid, 128, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  conv_sum_parts_kernel<<<dim3((a.C + 127) / 128, a.W + 1), 128, 0, s>>>(a.part, a.dw, a.db, parts, a.C, a.W);
  return cudaGetLastError();
}

cudaError_t launch_conv_step(void* state, const void* x, int64_t x_stride, const void* w, const void* bias, void* y,
                             int B, int C, int W, bool silu, bool bf16, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(B) * C + 127) / 128);
  if (bf16)
    conv_step_kernel<uint16_t><<<grid, 128, 0, s>>>(static_cast<uint16_t*>(state), static_cast<const uint16_t*>(x),
                                                    x_stride, static_cast<const uint16_t*>(w),
                                                    static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), B, C,
                                                    W, silu);
  else
    conv_step_kernel<float><<<grid, 128, 0, s>>>(static_cast<float*>(state), static_cast<const float*>(x), x_stride,
                                                 static_cast<const float*>(w), static_cast<const float*>(bias),
                                                 static_cast<float*>(y), B, C, W, silu);
  return cudaGetLastError();
}

}  // namespace m2rnn
