// Global norm of many gradient tensors, and clipping by it:
//     norm = sqrt(sum over every tensor of x^2),
//     out  = x c,  c = min(1, max_norm / (norm + 1e-6)).
// A plan lists the tensors in pieces of at most kGradChunk elements; block b
// takes pieces b, b + grid, ...  Squares are summed in fp32 within a piece
// (each thread its own elements in order, then a fixed tree) and in fp64
// across pieces and blocks, in a fixed order: results are bitwise
// reproducible.
#include <cuda_runtime.h>

#include <cstdint>

#include "layer.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBlocks = 608;  // 4 per SM

struct ClipScratch {
  double part[kMaxBlocks];
  float coef;
  unsigned int ticket;
};

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ float square_sum(const T* x, int n) {
  float s = 0.f;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float v = to_f32(x[i]);
    s = fmaf(v, v, s);
  }
  return s;
}

// The same in fp64, for a piece whose squares leave the fp32 range.
template <typename T>
__device__ double square_sum_wide(const T* x, int n) {
  double s = 0.;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const double v = to_f32(x[i]);
    s += v * v;
  }
  return s;
}

__device__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.;
  for (int i = 0; i < kThreads / 32; ++i) t += red[i];
  return t;
}

// Sum of squares of one piece, in every thread.
__device__ double piece_sum(const GradChunk& c, double* red) {
  const float s = c.bf16 ? square_sum(static_cast<const uint16_t*>(c.in), c.count)
                         : square_sum(static_cast<const float*>(c.in), c.count);
  const double t = block_sum_f64(static_cast<double>(warp_sum_f(s)) / 32., red);
  // Squares overflow beyond 1.8e19 and lose bits below 1e-19: take those pieces again in fp64.
  if (t < 1e38 && t > 1e-24) return t;
  const double w = c.bf16 ? square_sum_wide(static_cast<const uint16_t*>(c.in), c.count)
                          : square_sum_wide(static_cast<const float*>(c.in), c.count);
  return block_sum_f64(w, red);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const GradChunk* plan, int64_t chunks, float max_norm,
                                                             float* norm, ClipScratch* sc) {
  __shared__ double red[kThreads / 32];
  __shared__ bool last;
  double acc = 0.;
  for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) acc += piece_sum(plan[i], red);
  if (threadIdx.x == 0) {
    sc->part[blockIdx.x] = acc;
    __threadfence();
    last = atomicAdd(&sc->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0.;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) t += __ldcg(&sc->part[i]);
  t = block_sum_f64(t, red);
  if (threadIdx.x == 0) {
    const float nv = static_cast<float>(sqrt(t));
    *norm = nv;
    const float c = max_norm / (nv + 1e-6f);
    sc->coef = c > 1.f ? 1.f : c;  // NaN stays NaN
    sc->ticket = 0;
  }
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* in, T* out, int n, float c) {
  for (int i = threadIdx.x; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(in[i]) * c);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const GradChunk* plan, int64_t chunks,
                                                              const ClipScratch* sc) {
  const float c = sc->coef;
  for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const GradChunk p = plan[i];
    if (c == 1.f && p.in == p.out) continue;
    if (p.bf16)
      scale_piece(static_cast<const uint16_t*>(p.in), static_cast<uint16_t*>(p.out), p.count, c);
    else
      scale_piece(static_cast<const float*>(p.in), static_cast<float*>(p.out), p.count, c);
  }
}

}  // namespace

size_t grad_clip_scratch_bytes() { return sizeof(ClipScratch); }

cudaError_t launch_grad_clip(const GradChunk* plan, int64_t chunks, float max_norm, bool clip, float* norm, void* ws,
                             cudaStream_t s) {
  ClipScratch* sc = static_cast<ClipScratch*>(ws);
  cudaError_t e = cudaMemsetAsync(&sc->ticket, 0, sizeof(unsigned int), s);
  if (e != cudaSuccess) return e;
  const int grid = chunks < 1 ? 1 : static_cast<int>(chunks < kMaxBlocks ? chunks : kMaxBlocks);
  grad_norm_kernel<<<grid, kThreads, 0, s>>>(plan, chunks, max_norm, norm, sc);
  e = cudaGetLastError();
  if (e != cudaSuccess || !clip || chunks < 1) return e;
  grad_scale_kernel<<<grid, kThreads, 0, s>>>(plan, chunks, sc);
  return cudaGetLastError();
}

}  // namespace m2rnn
