// The orthogonalised update (ortho.cu) of small matrices, up to 64 x 256 or 256 x
// 64: a block per matrix, everything in shared memory from the norm to the last
// step, one launch.  The three products of a step run on warp MMA with fp16
// operands, scaled as in ortho.cu: A = X X^T and A A from one part of each, P X
// from two parts of each (three products), which leaves 1.0e-3 of the result at
// 64 x 64 of random entries (its rounding to bf16: 1.7e-3); all in two parts left
// 1e-5 for 1.8 times the matrix instructions, which bound a step.  Few rows (up to
// 32, kAll) average less over an entry's errors, 6e-3 at 3 x 5: there all products
// take both parts.  Eight warps: a
// quarter of the rows and half of the columns each.  Few operations are fp64,
// which is slow here (a root and a quotient per thread cost 10 us).  192 of 64 x 64:
// 20 us (a step: 1.5 us with one matrix on an SM, 2.6 with two); 600 of 64 x 256:
// 106 us, 239 by the kernels of ortho.cu; one of 33 x 128: 18 and 52.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"
#include "mma_common.cuh"

namespace m2rnn {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f, kScaleX = 0x1p14f;
constexpr int kRows = 64, kThreads = 256, kGroups = kThreads / 128, kSquare = kRows + 8;  // a row's pitch: 8 more, for the banks

// v0, v1 in two fp16 parts each.
__device__ __forceinline__ void split_pair(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2_f16(v0, v1);
  lo = pack2_f16(v0 - f16lo(hi), v1 - f16hi(hi));
}

// d += a b over 16 x (8 kTiles) x kDepth; a: rows of 16, b: [n][kDepth] (kTurned: [kDepth][n]); kParts: in two parts,
// `a_part` and `b_part` bytes apart (without what both lower parts make).
template <int kTiles, int kDepth, bool kTurned, bool kParts>
__device__ __forceinline__ void multiply(float (&d)[kTiles][4], uint32_t a, int a_pitch, uint32_t a_part, uint32_t b, int b_pitch,
                                         uint32_t b_part, int lane) {
  const uint32_t pa = a + ((lane & 15) * a_pitch + (lane >> 4) * 8) * 2;
  const uint32_t pb = kTurned ? b + ((lane & 15) * b_pitch + (lane >> 4) * 8) * 2
                              : b + (((lane & 7) + ((lane >> 4) << 3)) * b_pitch + ((lane >> 3) & 1) * 8) * 2;
#pragma unroll
  for (int k = 0; k < kDepth; k += 16) {
    uint32_t ah[4], al[4];
    ldmatrix_x4(ah, pa + k * 2);
    if (kParts) ldmatrix_x4(al, pa + a_part + k * 2);
#pragma unroll
    for (int t = 0; t < kTiles; t += 2) {
      uint32_t bh[4], bl[4];
      const uint32_t at = kTurned ? pb + (k * b_pitch + t * 8) * 2 : pb + (t * 8 * b_pitch + k) * 2;
      if constexpr (kTurned) {
        ldmatrix_x4_trans(bh, at);
        if (kParts) ldmatrix_x4_trans(bl, at + b_part);
      } else {
        ldmatrix_x4(bh, at);
        if (kParts) ldmatrix_x4(bl, at + b_part);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) mma_f16_16816(d[t + h], ah, bh[2 * h], bh[2 * h + 1]);
      if constexpr (kParts) {
#pragma unroll
        for (int h = 0; h < 2; ++h) mma_f16_16816(d[t + h], ah, bl[2 * h], bl[2 * h + 1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) mma_f16_16816(d[t + h], al, bh[2 * h], bh[2 * h + 1]);
      }
    }
  }
}

template <typename E, int kCols, bool kAll>
__global__ void __launch_bounds__(kThreads, kCols > 128 ? 2 : 3) ortho_small_kernel(const E* g, uint16_t* out, int m, int k,
                                                                                   bool tall, int steps, float eps,
                                                                                   StatusBlock* status) {
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int kPitch = kCols + 8;
  constexpr uint32_t kXPart = kRows * kPitch * 2, kSPart = kRows * kSquare * 2;
  __shared__ double red[kThreads / 32];
  __shared__ Inverse factor;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = lane & 3, row = 16 * (warp & 3) + (lane >> 2);
  const uint32_t x = smem_u32(raw), s = x + 2 * kXPart, p = s + (kAll ? 2 : 1) * kSPart;
  const int size = m * k, line = tall ? m : k;  // a line of G
  const int64_t at = static_cast<int64_t>(blockIdx.x) * size;

  if (blockIdx.x == 0 && threadIdx.x < sizeof(StatusBlock) / 4) reinterpret_cast<uint32_t*>(status)[threadIdx.x] = 0u;

  // ---- the norm; X ----
  float v[kCols * kRows / kThreads];
  float sum = 0.f, up = 0.f;
#pragma unroll
  for (int j = 0; j < kCols * kRows / kThreads; ++j) {
    const int i = threadIdx.x + kThreads * j;
    v[j] = i < size ? to_f32(g[at + i]) : 0.f;
  }
  for (uint32_t o = threadIdx.x * 16; o < 2 * kXPart; o += kThreads * 16) st_shared_f32x4(x + o, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll
  for (int j = 0; j < kCols * kRows / kThreads; ++j) {
    const float y = v[j] * 0x1p90f;
    sum = fmaf(v[j], v[j], sum);
    up = fmaf(y, y, up);
  }
  double acc = sum;  // squares that leave the fp32 range, as in ortho.cu
  if (sum < 0x1p-60f) acc = static_cast<double>(up) * 0x1p-180;
  if (!(sum <= 3.4e38f)) {
    acc = 0.;
#pragma unroll 1
    for (int i = threadIdx.x; i < size; i += kThreads) {
      const double w = to_f32(g[at + i]);
      acc += w * w;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) red[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) acc += red[w];
    factor = inverse_norm(acc, eps);
  }
  __syncthreads();
  const Inverse f = factor;
#pragma unroll
  for (int j = 0; j < kCols * kRows / kThreads; ++j) {
    const int i = threadIdx.x + kThreads * j, a = i / line, c = i - a * line;
    if (i < size) {
      const float w = f.of(v[j]) * kScaleX;
      const __half hi = __float2half_rn(w), lo = __float2half_rn(w - __half2float(hi));
      const uint32_t to = x + ((tall ? c : a) * kPitch + (tall ? a : c)) * 2;
      st_shared_u16(to, __half_as_ushort(hi));
      st_shared_u16(to + kXPart, __half_as_ushort(lo));
    }
  }
  __syncthreads();

  // ---- the steps ----
  const int c0 = kRows / kGroups * (warp >> 2);  // the warp's columns of A, P
  const int k0 = kCols / kGroups * (warp >> 2);  // and of X
  const uint32_t rows_x = x + 16 * (warp & 3) * kPitch * 2, rows_s = s + 16 * (warp & 3) * kSquare * 2,
                 rows_p = p + 16 * (warp & 3) * kSquare * 2;
  auto put = [&](uint32_t to, int pitch, uint32_t part, int r, int c, float v0, float v1) {
    uint32_t hi, lo;
    split_pair(v0, v1, hi, lo);
    st_shared_b32(to + (r * pitch + c) * 2, hi);
    st_shared_b32(to + (r * pitch + c) * 2 + part, lo);
  };
  for (int i = 0; i < steps; ++i) {
    constexpr int kSquares = kRows / kGroups / 8;
    float a[kSquares][4] = {};
    multiply<kSquares, kCols, false, kAll>(a, rows_x, kPitch, kXPart, x + c0 * kPitch * 2, kPitch, kXPart, lane);
#pragma unroll
    for (int t = 0; t < kSquares; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        a[t][e] *= 0x1p-14f;
        a[t][e + 1] *= 0x1p-14f;
        if constexpr (kAll) {
          put(s, kSquare, kSPart, row + 4 * e, c0 + 8 * t + 2 * q, a[t][e], a[t][e + 1]);
        } else {
          const uint32_t pair = pack2_f16(a[t][e], a[t][e + 1]);
          a[t][e] = f16lo(pair);  // the same A in both terms of P, whose errors then mostly cancel
          a[t][e + 1] = f16hi(pair);
          st_shared_b32(s + ((row + 4 * e) * kSquare + c0 + 8 * t + 2 * q) * 2, pair);
        }
      }
    __syncthreads();
    float b[kSquares][4] = {};
    multiply<kSquares, kRows, false, kAll>(b, rows_s, kSquare, kSPart, s + c0 * kSquare * 2, kSquare, kSPart, lane);
#pragma unroll
    for (int t = 0; t < kSquares; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        put(p, kSquare, kSPart, row + 4 * e, c0 + 8 * t + 2 * q, fmaf(kC * 0x1p-15f, b[t][e], kB * 0.5f * a[t][e]),
            fmaf(kC * 0x1p-15f, b[t][e + 1], kB * 0.5f * a[t][e + 1]));
    __syncthreads();
    constexpr int kTiles = kCols / kGroups / 8;
    float d[kTiles][4] = {};
    multiply<kTiles, kRows, true, true>(d, rows_p, kSquare, kSPart, x + k0 * 2, kPitch, kXPart, lane);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t from = x + ((row + 4 * e) * kPitch + k0 + 8 * t + 2 * q) * 2;
        const uint32_t hi = ld_shared_b32(from), lo = ld_shared_b32(from + kXPart);
        d[t][e] = fmaf(d[t][e], 0x1p-13f, kA * (f16lo(hi) + f16lo(lo)));
        d[t][e + 1] = fmaf(d[t][e + 1], 0x1p-13f, kA * (f16hi(hi) + f16hi(lo)));
      }
    __syncthreads();
    const bool last = i == steps - 1;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int r = row + 4 * e, c = k0 + 8 * t + 2 * q;
        if (last)  // the result takes X's upper part's place
          st_shared_b32(x + (r * kPitch + c) * 2, pack_bf16x2(d[t][e] * (1.f / kScaleX), d[t][e + 1] * (1.f / kScaleX)));
        else
          put(x, kPitch, kXPart, r, c, d[t][e], d[t][e + 1]);
      }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < size; i += kThreads) {
    const int a = i / line, c = i - a * line;
    out[at + i] = static_cast<uint16_t>(ld_shared_u16(x + ((tall ? c : a) * kPitch + (tall ? a : c)) * 2));
  }
}

template <typename E, int kCols, bool kAll>
cudaError_t launch_as(const OrthoArgs& A, int m, int k, cudaStream_t s) {
  constexpr int kSmem = 4 * kRows * (kCols + 8) + (kAll ? 8 : 6) * kRows * kSquare;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = ortho_small_kernel<E, kCols, kAll>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, ready);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(A.n), kThreads, kSmem, s>>>(static_cast<const E*>(A.g), A.out, m, k, A.rows > A.cols, A.steps,
                                                             A.eps, A.status);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch(const OrthoArgs& A, int m, int k, cudaStream_t s) {
  if (m <= 32)
    return k <= 64 ? launch_as<E, 64, true>(A, m, k, s) : k <= 128 ? launch_as<E, 128, true>(A, m, k, s) : launch_as<E, 256, true>(A, m, k, s);
  return k <= 64 ? launch_as<E, 64, false>(A, m, k, s) : k <= 128 ? launch_as<E, 128, false>(A, m, k, s) : launch_as<E, 256, false>(A, m, k, s);
}

}  // namespace

bool ortho_small(int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols, k = rows < cols ? cols : rows;
  return m <= kRows && k <= 256;
}

cudaError_t launch_ortho_small(const OrthoArgs& A, cudaStream_t s) {
  const int m = A.rows < A.cols ? A.rows : A.cols, k = A.rows < A.cols ? A.cols : A.rows;
  return A.bf16 ? launch<uint16_t>(A, m, k, s) : launch<float>(A, m, k, s);
}

}  // namespace m2rnn
