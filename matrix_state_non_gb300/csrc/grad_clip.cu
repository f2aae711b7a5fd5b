// Global norm of many gradient tensors, and clipping by it:
//     norm = sqrt(sum over every tensor of x^2),
//     out  = x c,  c = min(1, max_norm / (norm + 1e-6)).
// A plan lists the tensors in pieces of at most kGradChunk elements; block b
// takes pieces b, b + grid, ..., its threads marching through a piece side by
// side (a piece per warp instead is 13 % slower on 1.6 GB: too many fronts in
// memory).  Two passes over the data, both bound by HBM: the sums, then the
// scaling, which takes the pieces from the back, so that what the first pass
// left in L2 is read from there.  1.65 GB of fp32 gradients (of a 410M model):
// 767 us, 6.4 TB/s over the three passes that the data makes; 32 MB of one
// layer's: 20 us (the second pass from L2; two launches).
//
// A thread sums the squares of its 32 elements of a piece in fp32, then pieces,
// threads, warps and blocks in fp64, all in a fixed order: results are bitwise
// reproducible.  (fp64 adds are few: the unit is slow here, and a whole block
// adding up in fp64 cost more than its share of the data.)  Squares that leave
// the fp32 range are caught a piece at a time: next to x^2 the thread sums
// (x 2^90)^2, which serves where the first sum is so small that squares may
// have lost bits, and a sum that is not finite is taken again in fp64.
#include <cuda_runtime.h>

#include <cstdint>

#include "layer.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kPerSm = 4;
constexpr int kBlocks = 152 * kPerSm;  // as many as run at once
constexpr int kAhead = 4;              // 16-byte loads in flight per thread

struct ClipScratch {
  double part[kBlocks];  // sums of squares of the first pass's blocks
};

template <typename T>
struct Vec {  // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  alignas(16) T e[kN];
};

// A piece: ragged ends around whole 16-byte vectors.
template <typename T>
struct Split {
  int head, vecs, tail;  // elements, vectors, first element behind them
  __device__ __forceinline__ Split(const T* in, int n) {
    head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / static_cast<int>(sizeof(T)));
    vecs = (n - head) / Vec<T>::kN;
    tail = head + vecs * Vec<T>::kN;
  }
};

// f(x) on the thread's elements of in[0, n).
template <typename T, typename F>
__device__ __forceinline__ void for_elements(const T* in, int n, F f) {
  const int id = threadIdx.x;
  const Split<T> s(in, n);
  const uint4* p = reinterpret_cast<const uint4*>(in + s.head);
  for (int i = id; i < s.vecs; i += kThreads * kAhead) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      r[u] = i + kThreads * u < s.vecs ? p[i + kThreads * u] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      Vec<T> v;
      *reinterpret_cast<uint4*>(v.e) = r[u];
#pragma unroll
      for (int e = 0; e < Vec<T>::kN; ++e) f(to_f32(v.e[e]));
    }
  }
  if (id < s.head) f(to_f32(in[id]));
  if (id < n - s.tail) f(to_f32(in[s.tail + id]));
}

// The thread's share of a piece's sum of squares.
template <typename T>
__device__ __forceinline__ double square_sum(const T* in, int n) {
  float s = 0.f, up = 0.f;
  for_elements(in, n, [&](float x) {
    s = fmaf(x, x, s);
    const float y = x * 0x1p90f;
    up = fmaf(y, y, up);
  });
  if (s < 0x1p-60f) return static_cast<double>(up) * 0x1p-180;  // every |x| < 2^-30
  if (s <= 3.4e38f) return s;
  double w = 0.;
  for_elements(in, n, [&](float x) { w += static_cast<double>(x) * x; });
  return w;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kThreads, kPerSm) grad_sum_kernel(const GradChunk* plan, int64_t pieces, ClipScratch* sc) {
  __shared__ double red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double acc = 0.;
  for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const GradChunk c = plan[i];
    acc += c.bf16 ? square_sum(static_cast<const uint16_t*>(c.in), c.count)
                  : square_sum(static_cast<const float*>(c.in), c.count);
  }
  let_next();
  acc = warp_sum(acc);
  if (lane == 0) red[warp] = acc;
  __syncthreads();
  if (warp == 0) {
    acc = warp_sum(lane < kWarps ? red[lane] : 0.);
    if (lane == 0) sc->part[blockIdx.x] = acc;
  }
}

// sqrt of the blocks' sums, in every lane of the calling warp (one of each
// block of the second pass: no extra launch, no waiting).
__device__ __forceinline__ float total_norm(const ClipScratch* sc, int parts, int lane) {
  double t[2] = {0., 0.};
  for (int i = lane, j = 0; i < parts; i += 32, j ^= 1) t[j] += sc->part[i];
  return static_cast<float>(sqrt(warp_sum(t[0] + t[1])));
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const ClipScratch* sc, int parts, float* norm) {
  wait_previous();
  const float t = total_norm(sc, parts, threadIdx.x);
  if (threadIdx.x == 0) *norm = t;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* in, T* out, int n, float c) {
  const int id = threadIdx.x;
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
#pragma unroll 8
    for (int i = id; i < n; i += kThreads) out[i] = from_f32<T>(to_f32(in[i]) * c);
    return;
  }
  const Split<T> s(in, n);
  const uint4* p = reinterpret_cast<const uint4*>(in + s.head);
  uint4* o = reinterpret_cast<uint4*>(out + s.head);
  for (int i = id; i < s.vecs; i += kThreads * kAhead) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + kThreads * u < s.vecs) r[u] = __ldcs(p + i + kThreads * u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + kThreads * u < s.vecs) {
        Vec<T> v, w;
        *reinterpret_cast<uint4*>(v.e) = r[u];
#pragma unroll
        for (int e = 0; e < Vec<T>::kN; ++e) w.e[e] = from_f32<T>(to_f32(v.e[e]) * c);
        __stcs(o + i + kThreads * u, *reinterpret_cast<const uint4*>(w.e));
      }
    }
  }
  if (id < s.head) out[id] = from_f32<T>(to_f32(in[id]) * c);
  if (id < n - s.tail) out[s.tail + id] = from_f32<T>(to_f32(in[s.tail + id]) * c);
}

__global__ void __launch_bounds__(kThreads, kPerSm) grad_scale_kernel(const GradChunk* plan, int64_t pieces,
                                                                 const ClipScratch* sc, int parts, float max_norm,
                                                                 float* norm) {
  __shared__ float coef;
  wait_previous();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const float t = total_norm(sc, parts, lane);
    if (lane == 0) {
      if (blockIdx.x == 0) *norm = t;
      const float c = max_norm / (t + 1e-6f);
      coef = c > 1.f ? 1.f : c;  // NaN stays NaN
    }
  }
  __syncthreads();
  const float c = coef;
  for (int64_t i = pieces - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
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
  const int grid = chunks < 1 ? 1 : static_cast<int>(chunks < kBlocks ? chunks : kBlocks);
  grad_sum_kernel<<<grid, kThreads, 0, s>>>(plan, chunks, sc);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (!clip || chunks < 1)
    e = launch_next(grad_norm_kernel, 1, 32, 0, s, sc, grid, norm);
  else
    e = launch_next(grad_scale_kernel, grid, kThreads, 0, s, plan, chunks, sc, grid, max_norm, norm);
  return e;
}

}  // namespace m2rnn
