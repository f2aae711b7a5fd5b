// Orthogonalised update: the singular values of a gradient's matrix are all
// brought near 1 by Newton-Schulz steps (as the Muon optimiser does),
//     X = G / (|G|_F + eps),
//     X <- a X + (b A + c A A) X,  A = X X^T,
// with a = 3.4445, b = -4.7750, c = 2.0315; the smaller side makes A (a tall G
// is transposed on the way in and out).  fp32 on CUDA cores, one product per
// launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"

namespace m2rnn {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kTile = 32;

// One block per matrix: 1 / (|G| + eps).
template <typename E>
__global__ void __launch_bounds__(1024) ortho_scale_kernel(const E* g, int64_t count, float eps, float* scale) {
  __shared__ double red[32];
  const E* p = g + blockIdx.x * count;
  double acc = 0.;
  for (int64_t i = threadIdx.x; i < count; i += 1024) {
    const double v = to_f32(p[i]);
    acc += v * v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 32; ++i) acc += red[i];
    scale[blockIdx.x] = static_cast<float>(1. / (sqrt(acc) + eps));
  }
}

// X [n][m][k] from G, transposed where G is tall.
template <typename E>
__global__ void __launch_bounds__(256) ortho_load_kernel(const E* g, const float* scale, float* x, int m, int k, bool tall) {
  const int64_t size = static_cast<int64_t>(m) * k, mat = blockIdx.y;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < size; i += gridDim.x * 256ll) {
    const int64_t r = i / k, c = i - r * k;
    x[mat * size + i] = to_f32(g[mat * size + (tall ? c * m + r : i)]) * scale[mat];
  }
}

__global__ void __launch_bounds__(256) ortho_store_kernel(const float* x, uint16_t* out, int m, int k, bool tall) {
  const int64_t size = static_cast<int64_t>(m) * k, mat = blockIdx.y;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < size; i += gridDim.x * 256ll) {
    const int64_t r = i / k, c = i - r * k;
    out[mat * size + (tall ? c * m + r : i)] = from_f32<uint16_t>(x[mat * size + i]);
  }
}

// D = p L R + q S for matrices of M x N, K inner; R given transposed (N x K) or not (K x N).
template <bool kTransposed>
__global__ void __launch_bounds__(kTile* kTile) ortho_product_kernel(const float* L, const float* R, const float* S, float* D,
                                                                     int M, int N, int K, float p, float q, int tiles_n) {
  __shared__ float l[kTile][kTile + 1], r[kTile][kTile + 1];
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const int64_t mat = blockIdx.y;
  const int m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  L += mat * M * static_cast<int64_t>(K);
  R += mat * N * static_cast<int64_t>(K);
  float acc = 0.f;
  for (int k0 = 0; k0 < K; k0 += kTile) {
    l[ty][tx] = m0 + ty < M && k0 + tx < K ? L[static_cast<int64_t>(m0 + ty) * K + k0 + tx] : 0.f;
    if (kTransposed)
      r[tx][ty] = n0 + ty < N && k0 + tx < K ? R[static_cast<int64_t>(n0 + ty) * K + k0 + tx] : 0.f;
    else
      r[ty][tx] = k0 + ty < K && n0 + tx < N ? R[static_cast<int64_t>(k0 + ty) * N + n0 + tx] : 0.f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTile; ++k) acc = fmaf(l[ty][k], r[k][tx], acc);
    __syncthreads();
  }
  if (m0 + ty < M && n0 + tx < N) {
    const int64_t i = mat * M * static_cast<int64_t>(N) + static_cast<int64_t>(m0 + ty) * N + n0 + tx;
    D[i] = p * acc + (S != nullptr ? q * S[i] : 0.f);
  }
}

}  // namespace

size_t ortho_scratch_bytes(int64_t n, int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols;
  return static_cast<size_t>(4 * (n + 3) / 16 * 16 + 16 + n * 8 * (rows * cols + m * m));
}

cudaError_t launch_orthogonalize(const OrthoArgs& A, cudaStream_t s) {
  const bool tall = A.rows > A.cols;
  const int m = tall ? A.cols : A.rows, k = tall ? A.rows : A.cols, n = static_cast<int>(A.n);
  const int64_t size = static_cast<int64_t>(m) * k, square = static_cast<int64_t>(m) * m;
  float* scale = static_cast<float*>(A.ws);
  float* x = scale + (n + 3) / 4 * 4 + 4;
  float *y = x + n * size, *gram = y + n * size, *poly = gram + n * square;
  const dim3 copy(static_cast<unsigned>(size / 256 < 1024 ? size / 256 + 1 : 1024), n);
  if (A.bf16) {
    ortho_scale_kernel<<<n, 1024, 0, s>>>(static_cast<const uint16_t*>(A.g), size, A.eps, scale);
    ortho_load_kernel<<<copy, 256, 0, s>>>(static_cast<const uint16_t*>(A.g), scale, x, m, k, tall);
  } else {
    ortho_scale_kernel<<<n, 1024, 0, s>>>(static_cast<const float*>(A.g), size, A.eps, scale);
    ortho_load_kernel<<<copy, 256, 0, s>>>(static_cast<const float*>(A.g), scale, x, m, k, tall);
  }
  const int tm = (m + kTile - 1) / kTile, tk = (k + kTile - 1) / kTile;
  for (int i = 0; i < A.steps; ++i) {
    ortho_product_kernel<true><<<dim3(tm * tm, n), kTile * kTile, 0, s>>>(x, x, nullptr, gram, m, m, k, 1.f, 0.f, tm);
    ortho_product_kernel<false><<<dim3(tm * tm, n), kTile * kTile, 0, s>>>(gram, gram, gram, poly, m, m, m, kC, kB, tm);
    ortho_product_kernel<false><<<dim3(tm * tk, n), kTile * kTile, 0, s>>>(poly, x, x, y, m, k, m, 1.f, kA, tk);
    float* t = x;
    x = y;
    y = t;
  }
  ortho_store_kernel<<<copy, 256, 0, s>>>(x, A.out, m, k, tall);
  return cudaGetLastError();
}

}  // namespace m2rnn
