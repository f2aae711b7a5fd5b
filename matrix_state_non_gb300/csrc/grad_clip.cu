// Global norm of many gradient tensors, and clipping by it:
//     norm = sqrt(sum over every tensor of x^2),
//     out  = x c,  c = min(1, max_norm / (norm + 1e-6)).
// A plan lists the tensors in pieces of at most kGradChunk elements; block b
// takes pieces b, b + grid, ...  Two passes over the data, both bound by HBM:
// the sums, then the scaling, which takes the pieces in the opposite order so
// that what the first pass left in L2 is read from there.
//
// A thread sums the squares of its up to 32 elements of a piece in fp32, then
// pieces, threads and blocks in fp64, all in a fixed order: results are
// bitwise reproducible.  Squares that leave the fp32 range are caught a piece
// at a time: next to x^2 the thread sums (x 2^90)^2, which serves where the
// first sum is so small that squares may have lost bits, and a sum that is
// not finite is taken again in fp64.
#include <cuda_runtime.h>

#include <cstdint>

#include "layer.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBlocks = 608;  // 4 per SM

struct ClipScratch {
  double part[kMaxBlocks];  // sums of squares of the first pass's blocks
};

template <typename T>
struct Vec {  // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  alignas(16) T e[kN];
};

// f(x) on the thread's elements of in[0, n): the vectors from the first
// 16-byte boundary on (kAhead loads in flight), then the ragged ends.
constexpr int kAhead = 4;

template <typename T, typename F>
__device__ __forceinline__ void for_elements(const T* in, int n, F f) {
  using V = Vec<T>;
  int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / static_cast<int>(sizeof(T));
  head = min(head, n);
  const int nv = (n - head) / V::kN, tail = head + nv * V::kN;
  const uint4* p = reinterpret_cast<const uint4*>(in + head);
  for (int i = threadIdx.x; i < nv; i += kAhead * kThreads) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u * kThreads < nv) r[u] = p[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + u * kThreads < nv) {
        V v;
        *reinterpret_cast<uint4*>(v.e) = r[u];
#pragma unroll
        for (int e = 0; e < V::kN; ++e) f(to_f32(v.e[e]));
      }
    }
  }
  if (static_cast<int>(threadIdx.x) < head) f(to_f32(in[threadIdx.x]));
  if (static_cast<int>(threadIdx.x) < n - tail) f(to_f32(in[tail + threadIdx.x]));
}

// The thread's share of a piece's sum of squares.
template <typename T>
__device__ __forceinline__ double square_sum(const T* in, int n) {
  constexpr float kUp = 0x1p90f;
  float s = 0.f, up = 0.f;
  for_elements(in, n, [&](float x) {
    s = fmaf(x, x, s);
    const float y = x * kUp;
    up = fmaf(y, y, up);
  });
  if (s < 0x1p-60f) return static_cast<double>(up) * 0x1p-180;  // every |x| < 2^-30
  if (s <= 3.4e38f) return s;
  double w = 0.;
  for_elements(in, n, [&](float x) { w += static_cast<double>(x) * x; });
  return w;
}

// Fixed-order block sum, in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += red[i];
  return t;
}

__global__ void __launch_bounds__(kThreads, 2) grad_sum_kernel(const GradChunk* plan, int64_t chunks, ClipScratch* sc) {
  __shared__ double red[kThreads / 32];
  double acc = 0.;
  for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const GradChunk c = plan[i];
    acc += c.bf16 ? square_sum(static_cast<const uint16_t*>(c.in), c.count)
                  : square_sum(static_cast<const float*>(c.in), c.count);
  }
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) sc->part[blockIdx.x] = acc;
}

// sqrt of the blocks' sums, in every thread of a block (each block of the
// second pass adds them up itself: no extra launch, no waiting).
__device__ __forceinline__ float total_norm(const ClipScratch* sc, int parts, double* red) {
  double t = 0.;
  for (int i = threadIdx.x; i < parts; i += kThreads) t += sc->part[i];
  return static_cast<float>(sqrt(block_sum(t, red)));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const ClipScratch* sc, int parts, float* norm) {
  __shared__ double red[kThreads / 32];
  const float t = total_norm(sc, parts, red);
  if (threadIdx.x == 0) *norm = t;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* in, T* out, int n, float c) {
  using V = Vec<T>;
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    for (int i = threadIdx.x; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(in[i]) * c);
    return;
  }
  int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / static_cast<int>(sizeof(T));
  head = min(head, n);
  const int nv = (n - head) / V::kN, tail = head + nv * V::kN;
  const uint4* p = reinterpret_cast<const uint4*>(in + head);
  uint4* o = reinterpret_cast<uint4*>(out + head);
  for (int i = threadIdx.x; i < nv; i += kAhead * kThreads) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u * kThreads < nv) r[u] = __ldcs(p + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + u * kThreads < nv) {
        V v, w;
        *reinterpret_cast<uint4*>(v.e) = r[u];
#pragma unroll
        for (int e = 0; e < V::kN; ++e) w.e[e] = from_f32<T>(to_f32(v.e[e]) * c);
        __stcs(o + i + u * kThreads, *reinterpret_cast<const uint4*>(w.e));
      }
    }
  }
  if (static_cast<int>(threadIdx.x) < head) out[threadIdx.x] = from_f32<T>(to_f32(in[threadIdx.x]) * c);
  if (static_cast<int>(threadIdx.x) < n - tail)
    out[tail + threadIdx.x] = from_f32<T>(to_f32(in[tail + threadIdx.x]) * c);
}

__global__ void __launch_bounds__(kThreads, 2) grad_scale_kernel(const GradChunk* plan, int64_t chunks,
                                                                 const ClipScratch* sc, int parts, float max_norm,
                                                                 float* norm) {
  __shared__ double red[kThreads / 32];
  const float t = total_norm(sc, parts, red);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = t;
  float c = max_norm / (t + 1e-6f);
  if (c > 1.f) c = 1.f;  // NaN stays NaN
  for (int64_t i = (chunks - 1 - blockIdx.x) / gridDim.x * gridDim.x + blockIdx.x; i >= 0; i -= gridDim.x) {
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
  const int grid = chunks < 1 ? 1 : static_cast<int>(chunks < kMaxBlocks ? chunks : kMaxBlocks);
  grad_sum_kernel<<<grid, kThreads, 0, s>>>(plan, chunks, sc);
  if (!clip || chunks < 1)
    grad_norm_kernel<<<1, kThreads, 0, s>>>(sc, grid, norm);
  else
    grad_scale_kernel<<<grid, kThreads, 0, s>>>(plan, chunks, sc, grid, max_norm, norm);
  return cudaGetLastError();
}

}  // namespace m2rnn
