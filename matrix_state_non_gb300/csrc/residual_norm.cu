// Root-mean-square norm of the residual stream, with the branch's addition:
//     h = x + residual,  s = (sum_j h_j^2 / D + eps)^(-1/2),  y = w (*) h s,
// y in bf16, fp32, or e4m3 with a scale for each 128 values of a row; and its
// backward, with p = w (*) dy and r = sum_j p_j h_j per row:
//     dx = s p - r s^3 h / D + dh,   dw = sum over rows of dy (*) h s.
// A block per row; sums run in a fixed order.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256, kMaxPer = kNormMaxWidth / kThreads;

__device__ __forceinline__ float load_as(const void* p, int64_t i, bool bf16) {
  return bf16 ? to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_as(void* p, int64_t i, bool bf16, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = from_f32<uint16_t>(v);
  else
    static_cast<float*>(p)[i] = v;
}

__device__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) t += red[i];
  return t;
}

__global__ void __launch_bounds__(kThreads) residual_norm_kernel(NormRowsArgs A) {
  extern __shared__ float row[];
  __shared__ float red[kThreads / 32];
  for (int64_t i = blockIdx.x; i < A.rows; i += gridDim.x) {
    float ss = 0.f;
    for (int j = threadIdx.x; j < A.D; j += kThreads) {
      float v = load_as(A.x, i * A.x_stride + j, A.x_bf16);
      if (A.residual != nullptr) v += load_as(A.residual, i * A.D + j, A.h_bf16);
      if (A.h != nullptr) store_as(A.h, i * A.D + j, A.h_bf16, v);
      row[j] = v;
      ss += v * v;
    }
    const float s = rsqrtf(block_sum(ss, red) / static_cast<float>(A.D) + A.eps);
    if (A.y_type != M2RNN_E4M3) {
      for (int j = threadIdx.x; j < A.D; j += kThreads)
        store_as(A.y, i * A.D + j, A.y_type == M2RNN_BF16, row[j] * s * A.w[j]);
    } else {
      const int lane = threadIdx.x & 31, blocks = (A.D + kScaleBlock - 1) / kScaleBlock;
      for (int b = threadIdx.x >> 5; b < blocks; b += kThreads / 32) {
        float v[kScaleBlock / 32], most = 0.f;
        for (int e = 0; e < kScaleBlock / 32; ++e) {
          const int j = b * kScaleBlock + e * 32 + lane;
          v[e] = j < A.D ? row[j] * s * A.w[j] : 0.f;
          most = fmaxf(most, fabsf(v[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float scale = fmaxf(most / 448.f, 0x1p-126f);
        for (int e = 0; e < kScaleBlock / 32; ++e) {
          const int j = b * kScaleBlock + e * 32 + lane;
          if (j < A.D)
            static_cast<uint8_t*>(A.y)[i * A.D + j] = __nv_cvt_float_to_fp8(v[e] / scale, __NV_SATFINITE, __NV_E4M3);
        }
        if (lane == 0) A.scale[i * blocks + b] = scale;
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) residual_norm_backward_kernel(NormRowsArgs A) {
  __shared__ float red[kThreads / 32];
  float dw[kMaxPer];
  for (int e = 0; e < kMaxPer; ++e) dw[e] = 0.f;
  for (int64_t i = blockIdx.x; i < A.rows; i += gridDim.x) {
    float ss = 0.f, rr = 0.f;
    for (int j = threadIdx.x; j < A.D; j += kThreads) {
      const float h = load_as(A.h, i * A.D + j, A.h_bf16), d = load_as(A.dy, i * A.D + j, A.dy_bf16);
      ss += h * h;
      rr += h * (d * A.w[j]);
    }
    const float s = rsqrtf(block_sum(ss, red) / static_cast<float>(A.D) + A.eps);
    const float c = block_sum(rr, red) * s * s * s / static_cast<float>(A.D);
    for (int e = 0, j = threadIdx.x; j < A.D; ++e, j += kThreads) {
      const float h = load_as(A.h, i * A.D + j, A.h_bf16), d = load_as(A.dy, i * A.D + j, A.dy_bf16);
      const float up = A.dh != nullptr ? A.dh[i * A.D + j] : 0.f;
      A.dx[i * A.D + j] = s * (d * A.w[j]) - c * h + up;
      dw[e] += d * (h * s);
    }
  }
  for (int e = 0, j = threadIdx.x; j < A.D; ++e, j += kThreads) A.part[static_cast<int64_t>(blockIdx.x) * A.D + j] = dw[e];
}

}  // namespace

int norm_rows_parts(int64_t rows, int64_t D) { return static_cast<int>(rows < 304 ? rows : 304); }

cudaError_t launch_residual_norm(const NormRowsArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(residual_norm_kernel), kNormMaxWidth * 4, ready);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(a.rows < 152 * 8 ? a.rows : 152 * 8);
  residual_norm_kernel<<<grid, kThreads, a.D * 4, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_residual_norm_backward(const NormRowsArgs& a, cudaStream_t s) {
  const int parts = norm_rows_parts(a.rows, a.D);
  residual_norm_backward_kernel<<<parts, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_sum_parts(a.part, a.dw, nullptr, false, parts, a.D, s);
}

}  // namespace m2rnn
