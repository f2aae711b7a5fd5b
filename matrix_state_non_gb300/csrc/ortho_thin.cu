// The orthogonalised update (ortho.cu) of long matrices with one side of up to 64,
// the other above 256.  Every X of the iteration is a polynomial of A = X_0 X_0^T
// times X_0, and such polynomials commute, so that the steps need m x m matrices
// alone:
//     Q = a + b A + c A A,  R <- Q R,  A <- Q A Q,   X = R X_0.
// A is summed over blocks that share the long side, a block per matrix takes the
// steps, and blocks along the long side apply R.  All in fp32 on CUDA cores: the
// rounding noise of A grows 12-fold a step where A has nothing (2e4 in four steps),
// which 24 bits bear for five steps and no more: after each five, X is made and A
// taken anew.  Q stands on either side of A, as A is symmetric but for its noise: in
// A Q Q, the same without any, noise between what A has and what it has not grows
// 12-fold as well, not 2.4-fold, and left 1.4e-2 of a 64 x 513 matrix of ones (Q A Q:
// 6e-4, others of low rank 3e-4).
// 64 x 2000: 56 us, 38 of them the steps' eighteen products on one SM (90 by the
// launches of ortho.cu); 64 x 16384: 75 (355); 200 of 64 x 1024: 192 (260).
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"
#include "mma_common.cuh"

namespace m2rnn {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kSide = 64, kPitch = kSide + 4, kThreads = 256, kTogether = 5;  // steps between two sums
constexpr int kSquare = kSide * kSide;

// acc[i][j] += sum over kk < depth of l[kk][4 ty + i] r[kk][4 tx + j], rows of kPitch: l's transpose times r.
__device__ __forceinline__ void multiply(float (&acc)[4][4], const float* l, const float* r, int depth, int tx, int ty) {
#pragma unroll 8
  for (int kk = 0; kk < depth; ++kk) {
    const float4 a = *reinterpret_cast<const float4*>(l + kk * kPitch + 4 * ty), b = *reinterpret_cast<const float4*>(r + kk * kPitch + 4 * tx);
    const float x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}
__device__ __forceinline__ void put(float* to, const float (&v)[4][4], int tx, int ty) {
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(to + (4 * ty + i) * kPitch + 4 * tx) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
}

// Value (r, c) of X_0 (m x k) times f; tall: it lies as [k][m].
template <typename E>
__device__ __forceinline__ float value(const E* g, int r, int c, int m, int k, bool tall, Inverse f) {
  return r < m && c < k ? f.of(to_f32(g[tall ? static_cast<int64_t>(c) * m + r : static_cast<int64_t>(r) * k + c])) : 0.f;
}

__device__ __forceinline__ Inverse factor_of(const double* part, int parts, float eps, Inverse* shared) {
  if (threadIdx.x < 32) {
    double acc = 0.;
    for (int i = threadIdx.x; i < parts; i += 32) acc += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (threadIdx.x == 0) *shared = inverse_norm(acc, eps);
  }
  __syncthreads();
  return *shared;
}

// The sums over `per` columns (a multiple of 64) each: sums [n][pieces][64][64].
template <typename E>
__global__ void __launch_bounds__(kThreads) thin_gram_kernel(const E* g, const double* part, int parts, float eps, float* sums,
                                                             int m, int k, bool tall, int per, int pieces) {
  __shared__ __align__(16) float t[kSide * kPitch];  // [column][row]
  __shared__ Inverse shared;
  const int mat = blockIdx.x / pieces, piece = blockIdx.x - mat * pieces;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const E* p = g + static_cast<int64_t>(mat) * m * k;
  wait_previous();
  const Inverse f = part != nullptr ? factor_of(part + static_cast<int64_t>(mat) * parts, parts, eps, &shared) : Inverse{1.f, 1.f};
  float acc[4][4] = {};
  for (int c0 = piece * per; c0 < min(k, (piece + 1) * per); c0 += kSide) {
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < kSquare; i += kThreads) {
      const int fast = i % kSide, slow = i / kSide, r = tall ? fast : slow, c = tall ? slow : fast;
      t[c * kPitch + r] = value(p, r, c0 + c, m, k, tall, f);
    }
    __syncthreads();
    multiply(acc, t, t, kSide, tx, ty);
  }
  let_next();
  float* to = sums + static_cast<int64_t>(blockIdx.x) * kSquare + 4 * tx;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(to + (4 * ty + i) * kSide) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

// R of `steps` steps, transposed: [n][64][64].
__global__ void __launch_bounds__(kThreads) thin_steps_kernel(const float* sums, float* out, int m, int pieces, int steps) {
  extern __shared__ __align__(16) float s[];
  float *A = s, *Q = s + kSide * kPitch, *R = Q + kSide * kPitch, *T = R + kSide * kPitch;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  wait_previous();
  const float* from = sums + static_cast<int64_t>(blockIdx.x) * pieces * kSquare;
  float v[4][4] = {};
  for (int p = 0; p < pieces; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(from + p * kSquare + (4 * ty + i) * kSide + 4 * tx);
      v[i][0] += x.x, v[i][1] += x.y, v[i][2] += x.z, v[i][3] += x.w;
    }
  put(A, v, tx, ty);
  __syncthreads();
  const bool in = 4 * ty < m && 4 * tx < m;  // a warp's rows and columns that are not there stay 0
  for (int step = 0; step < steps; ++step) {
    float q[4][4] = {};
    if (in) multiply(q, A, A, m, tx, ty);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[i][j] = fmaf(kC, q[i][j], kB * A[(4 * ty + i) * kPitch + 4 * tx + j]) + (4 * ty + i == 4 * tx + j ? kA : 0.f);
    put(Q, q, tx, ty);
    if (step == 0) put(R, q, tx, ty);
    __syncthreads();
    float r[4][4] = {}, w[4][4] = {};
    if (step > 0 && in) multiply(r, Q, R, m, tx, ty);
    if (step < steps - 1 && in) multiply(w, A, Q, m, tx, ty);
    __syncthreads();
    if (step > 0) put(R, r, tx, ty);
    put(T, w, tx, ty);
    __syncthreads();
    if (step < steps - 1) {
      float x[4][4] = {};
      if (in) multiply(x, Q, T, m, tx, ty);
      put(A, x, tx, ty);  // (nobody reads A here)
    }
    __syncthreads();
  }
  let_next();
  for (int i = threadIdx.x; i < kSquare; i += kThreads)
    out[static_cast<int64_t>(blockIdx.x) * kSquare + i] = R[(i % kSide) * kPitch + i / kSide];
}

// X = R X_0, 64 columns to a block: to `x` [n][m][k] in fp32, or, where that is null, to `out` in bf16 as X_0 lies.
template <typename E>
__global__ void __launch_bounds__(kThreads) thin_apply_kernel(const E* g, const double* part, int parts, float eps, const float* R,
                                                              float* x, uint16_t* out, int m, int k, bool from_tall, bool tall,
                                                              int tiles) {
  __shared__ __align__(16) float t[kSide * kPitch], l[kSide * kPitch];
  __shared__ Inverse shared;
  const int mat = blockIdx.x / tiles, c0 = (blockIdx.x - mat * tiles) * kSide;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t base = static_cast<int64_t>(mat) * m * k;
  wait_previous();
  const Inverse f = part != nullptr ? factor_of(part + static_cast<int64_t>(mat) * parts, parts, eps, &shared) : Inverse{1.f, 1.f};
#pragma unroll 4
  for (int i = threadIdx.x; i < kSquare; i += kThreads) {
    const int fast = i % kSide, slow = i / kSide, r = from_tall ? fast : slow, c = from_tall ? slow : fast;
    t[r * kPitch + c] = value(g + base, r, c0 + c, m, k, from_tall, f);
    l[slow * kPitch + fast] = R[static_cast<int64_t>(mat) * kSquare + i];
  }
  __syncthreads();
  let_next();
  float v[4][4] = {};
  if (4 * ty < m) multiply(v, l, t, m, tx, ty);
  __syncthreads();
  put(l, v, tx, ty);  // (R has been used)
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < kSquare; i += kThreads) {
    const bool turned = x == nullptr && tall;
    const int fast = i % kSide, slow = i / kSide, r = turned ? fast : slow, c = turned ? slow : fast;
    if (r >= m || c0 + c >= k) continue;
    const float w = l[r * kPitch + c];
    const int64_t at = base + (turned ? static_cast<int64_t>(c0 + c) * m + r : static_cast<int64_t>(r) * k + c0 + c);
    if (x != nullptr)
      x[at] = w;
    else
      out[at] = from_f32<uint16_t>(w);
  }
}

struct Layout {
  double* part;
  float *sums, *R, *x;
  size_t bytes;
  int parts, per, pieces;
  Layout(void* ws, int64_t n, int64_t m, int64_t k) {
    parts = ortho_sum_parts(m * k);
    const int64_t tiles = (k + kSide - 1) / kSide;
    const int64_t of = tiles <= 128 ? 2 : (tiles + 63) / 64;  // tiles of a piece: at most 64 pieces
    per = static_cast<int>(of * kSide);
    pieces = static_cast<int>((tiles + of - 1) / of);
    uint8_t* at = static_cast<uint8_t*>(ws);
    bytes = 0;
    auto take = [&](int64_t size) {
      uint8_t* p = at + bytes;
      bytes += (size + 255) / 256 * 256;
      return p;
    };
    part = reinterpret_cast<double*>(take(n * parts * 8));
    sums = reinterpret_cast<float*>(take(n * pieces * kSquare * 4));
    R = reinterpret_cast<float*>(take(n * kSquare * 4));
    x = reinterpret_cast<float*>(take(n * m * k * 4));
  }
};

template <typename E>
cudaError_t run(const OrthoArgs& A, cudaStream_t s) {
  const bool tall = A.rows > A.cols;
  const int m = tall ? A.cols : A.rows, k = tall ? A.rows : A.cols;
  const Layout w(A.ws, A.n, m, k);
  constexpr int kSmem = 4 * kSide * kPitch * 4;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(thin_steps_kernel), kSmem, ready);
  if (e == cudaSuccess) e = launch_ortho_sum(A, w.parts, w.part, s);
  const int tiles = (k + kSide - 1) / kSide;
  const unsigned grams = static_cast<unsigned>(A.n * w.pieces), applies = static_cast<unsigned>(A.n * tiles);
  for (int done = 0; e == cudaSuccess && done < A.steps; done += kTogether) {
    const int steps = A.steps - done < kTogether ? A.steps - done : kTogether;
    float* x = done + steps < A.steps ? w.x : nullptr;
    e = done == 0 ? launch_next(thin_gram_kernel<E>, grams, kThreads, 0, s, static_cast<const E*>(A.g), w.part, w.parts, A.eps, w.sums,
                                m, k, tall, w.per, w.pieces)
                  : launch_next(thin_gram_kernel<float>, grams, kThreads, 0, s, w.x, nullptr, 0, 0.f, w.sums, m, k, false, w.per,
                                w.pieces);
    if (e != cudaSuccess) break;
    e = launch_next(thin_steps_kernel, static_cast<unsigned>(A.n), kThreads, kSmem, s, w.sums, w.R, m, w.pieces, steps);
    if (e != cudaSuccess) break;
    e = done == 0 ? launch_next(thin_apply_kernel<E>, applies, kThreads, 0, s, static_cast<const E*>(A.g), w.part, w.parts, A.eps,
                                w.R, x, A.out, m, k, tall, tall, tiles)
                  : launch_next(thin_apply_kernel<float>, applies, kThreads, 0, s, w.x, nullptr, 0, 0.f, w.R, x, A.out, m, k, false,
                                tall, tiles);
  }
  return e;
}

}  // namespace

bool ortho_thin(int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols, k = rows < cols ? cols : rows;
  return m <= kSide && k > 256;
}

size_t ortho_thin_scratch_bytes(int64_t n, int64_t rows, int64_t cols) {
  return Layout(nullptr, n, rows < cols ? rows : cols, rows < cols ? cols : rows).bytes;
}

cudaError_t launch_ortho_thin(const OrthoArgs& A, cudaStream_t s) { return A.bf16 ? run<uint16_t>(A, s) : run<float>(A, s); }

}  // namespace m2rnn
