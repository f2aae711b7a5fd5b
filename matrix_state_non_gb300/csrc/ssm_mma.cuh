// Pieces of the tensor-core kernels of the selective state space scan: tiles
// in shared memory, the decays of a chunk of 64 steps, operands split into
// bf16 parts.
#pragma once

#include "gate.cuh"
#include "mma_common.cuh"
#include "ssm.cuh"

namespace m2rnn {

constexpr int kChunk = 64;  // steps of a chunk: four row blocks of 16

// A row-major bf16 tile; rows padded by 16 bytes, so that the eight rows of an
// ldmatrix fetch start on eight different 16-byte banks for every width.
template <int kCols>
struct Tile {
  static constexpr int kPitch = kCols * 2 + 16;  // bytes
  static constexpr int kBytes(int rows) { return rows * kPitch; }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Rows t0 .. t0 + 63 of one head into a tile: `width` columns of it are there,
// steps behind `len` and columns behind `width` become zero.  vec: rows on
// 16-byte boundaries and width a multiple of 8 (asynchronous copies);
// otherwise element by element.
template <int kCols, int kThreads>
__device__ __forceinline__ void load_tile(uint32_t tile, const uint16_t* p, int64_t stride, int width, int t0, int len,
                                          bool vec) {
  if (vec) {
    constexpr int kPer = kCols / 8;
#pragma unroll
    for (int i = 0; i < kChunk * kPer / kThreads; ++i) {
      const int e = i * kThreads + threadIdx.x, r = e / kPer, c = (e % kPer) * 8;
      const bool ok = t0 + r < len && c < width;
      cp_async_16(tile + r * Tile<kCols>::kPitch + c * 2, ok ? p + (t0 + r) * stride + c : p, ok);
    }
  } else {
#pragma unroll 4
    for (int e = threadIdx.x; e < kChunk * kCols; e += kThreads) {
      const int r = e / kCols, c = e % kCols;
      const uint16_t x = t0 + r < len && c < width ? p[(t0 + r) * stride + c] : uint16_t(0);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(tile + r * Tile<kCols>::kPitch + c * 2), "h"(x) : "memory");
    }
  }
}

// ldmatrix addresses within a tile, block (r0, c0) of 16 x 16 elements:
// in order (rows 0-7, cols 0-7), (rows 8-15, cols 0-7), (0-7, 8-15), (8-15, 8-15).
//  A (m = row, k = col): plain.   B (k = row, n = col): transposed, b0/b1 of
//  the n-tiles c0 and c0 + 8 in r[0], r[1] and r[2], r[3].
template <int kCols>
__device__ __forceinline__ uint32_t at_rows(uint32_t tile, int r0, int c0, int lane) {
  return tile + (r0 + (lane & 15)) * Tile<kCols>::kPitch + (c0 + (lane >> 4) * 8) * 2;
}
// In order (rows 0-7, cols 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15).
//  B (n = row, k = col): plain, b0/b1 of the n-tiles r0 and r0 + 8.
//  A (m = col, k = row): transposed.
template <int kCols>
__device__ __forceinline__ uint32_t at_cols(uint32_t tile, int r0, int c0, int lane) {
  return tile + (r0 + (lane & 7) + ((lane >> 4) << 3)) * Tile<kCols>::kPitch + (c0 + ((lane >> 3) & 1) * 8) * 2;
}

// A pair of fp32 values as three bf16 pairs whose sum is exact to 2^-24.
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  x -= bf16lo(hi);
  y -= bf16hi(hi);
  mid = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16lo(mid), y - bf16hi(mid));
}

// The decays of one chunk, in shared memory.  l_i is the sum of D A over the
// chunk's steps up to i; the factor exp(l_i - l_j) of row block ib and an
// earlier step j is row[i] col[ib][j] with the sum before the block as the
// reference, so a chunk takes a few hundred exponentials and not 64 x 64.
struct ChunkDecay {
  float hi[kChunk], lo[kChunk];  // l_i in two parts: differences of long sums keep their bits
  float D[kChunk];               // step sizes (0 behind the sequence's end)
  float first[kChunk];           // exp(l_i)
  float last[kChunk];            // exp(l_63 - l_i)
  float row[kChunk];             // exp(l_i - l_{16 ib - 1})
  float col[4][kChunk];          // exp(l_{16 ib - 1} - l_j) for j < 16 ib
  float tot;                     // exp(l_63)
};

__device__ __forceinline__ float exp_diff(float hi, float lo) { return ex2_fast(1.44269504f * hi + 1.44269504f * lo); }

// By one warp; lane i holds dt of steps t0 + 2 i, t0 + 2 i + 1 (already with
// the bias).  Sums in fp64: a chunk's sum reaches some hundreds and its
// differences have to be good to 1e-7.
__device__ __forceinline__ void chunk_decay(ChunkDecay& d, float x0, float x1, bool ok0, bool ok1, float A, int lane) {
  const float D0 = ok0 ? softplus_f(x0) : 0.f, D1 = ok1 ? softplus_f(x1) : 0.f;
  const double a0 = static_cast<double>(D0) * A, a1 = static_cast<double>(D1) * A;
  double l1 = a0 + a1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double p = __shfl_up_sync(0xffffffffu, l1, o);
    if (lane >= o) l1 += p;
  }
  double before = __shfl_up_sync(0xffffffffu, l1, 1);
  if (lane == 0) before = 0.;
  const double l0 = before + a0;
  const double end = __shfl_sync(0xffffffffu, l1, 31);
  const int i = 2 * lane;
  const float h0 = static_cast<float>(l0), h1 = static_cast<float>(l1);
  *reinterpret_cast<float2*>(&d.hi[i]) = make_float2(h0, h1);
  *reinterpret_cast<float2*>(&d.lo[i]) = make_float2(static_cast<float>(l0 - h0), static_cast<float>(l1 - h1));
  *reinterpret_cast<float2*>(&d.D[i]) = make_float2(D0, D1);
  *reinterpret_cast<float2*>(&d.first[i]) = make_float2(expf(h0), expf(h1));
  *reinterpret_cast<float2*>(&d.last[i]) =
      make_float2(expf(static_cast<float>(end - l0)), expf(static_cast<float>(end - l1)));
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
    const double ref = ib == 0 ? 0. : __shfl_sync(0xffffffffu, l1, 8 * ib - 1);
    if ((lane >> 3) == ib)
      *reinterpret_cast<float2*>(&d.row[i]) =
          make_float2(expf(static_cast<float>(l0 - ref)), expf(static_cast<float>(l1 - ref)));
    if ((lane >> 3) < ib)
      *reinterpret_cast<float2*>(&d.col[ib][i]) =
          make_float2(expf(static_cast<float>(ref - l0)), expf(static_cast<float>(ref - l1)));
  }
  if (lane == 0) d.tot = expf(static_cast<float>(end));
}

}  // namespace m2rnn
