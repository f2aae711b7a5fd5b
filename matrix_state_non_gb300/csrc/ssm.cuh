// Shared by the selective state space scan's kernel files.
#pragma once

#include "layer.cuh"

namespace m2rnn {

// Where a chunk's gradients go: dq, dk [B,T,qk_heads,K] (qk_heads = N: per
// value head, summed over shared heads afterwards where G < N), per-chunk
// partials of dw_r [chunks][V] (or null) and of (dA, ddt_bias) [chunks].
struct SsmGradOut {
  float* dq;
  float* dk;
  float* wr_part;
  float2* ab_part;
  int qk_heads;
};

__device__ __forceinline__ int ssm_len(const SsmArgs& A, int b) {
  return A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
}

// log a = D A.  From -1e4 down, where a is 0 many times over, the same: sums of it stay finite, and what small steps
// add to them is not lost beside a huge one.
template <typename T>
__device__ __forceinline__ T log_decay(T D, T A) {
  const T x = D * A;
  return x < T(-1e4) ? T(-1e4) : x;
}

// A running sum as hi + lo, good to about twice fp32.  (Adding in fp64 would do as well; its unit is slow here.)
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {  // two-sum: the rounding of hi + x goes into lo
    const float s = hi + x, w = s - hi;
    lo += (hi - (s - w)) + (x - w);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& x) {
    add(x.hi);
    lo += x.lo;
  }
  __device__ __forceinline__ void subtract(const Sum2& x) {
    add(-x.hi);
    lo -= x.lo;
  }
  __device__ __forceinline__ Sum2 across(int mask) const {
    return Sum2{__shfl_xor_sync(0xffffffffu, hi, mask), __shfl_xor_sync(0xffffffffu, lo, mask)};
  }
  __device__ __forceinline__ Sum2 after(int n) const {  // of the lane n further; zero behind the last
    const Sum2 x{__shfl_down_sync(0xffffffffu, hi, n), __shfl_down_sync(0xffffffffu, lo, n)};
    return static_cast<int>(threadIdx.x & 31) + n < 32 ? x : Sum2{};
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

// The CUDA-core kernels (fp32 inputs).
size_t ssm_f32_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V);
size_t ssm_f32_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V);
cudaError_t launch_ssm_f32_forward(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_ssm_f32_backward(const SsmArgs& a, cudaStream_t s);

// The tensor-core kernels (bf16 inputs).
size_t ssm_mma_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V);
cudaError_t launch_ssm_mma_forward(const SsmArgs& a, cudaStream_t s);
size_t ssm_mma_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V);
cudaError_t launch_ssm_mma_backward(const SsmArgs& a, cudaStream_t s);

// The fixed-order sums behind the chunks' gradients: dA, ddt_bias, dw_r from
// their partials over the chunks, dq, dk from the value heads' where G < N.
cudaError_t launch_ssm_grad_sums(const SsmArgs& a, const SsmGradOut& o, int nc, cudaStream_t s);

}  // namespace m2rnn
