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

// Whether a pair of bf16 values holds one that is not finite: bit 15 or 31 of the result, OR-ed over many.
constexpr uint32_t kNotFinite = 0x80008000u;
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return (x & 0x7F807F80u) + 0x00800080u; }

// Copies the 64 rows of a chunk of one head into a tile, chunk after chunk:
// `width` columns are there, steps behind `len` and columns behind `width`
// become zero.  vec: rows on 16-byte boundaries and width a multiple of 8
// (asynchronous copies); otherwise element by element.
template <int kCols, int kThreads>
struct TileLoader {
  static constexpr int kPer = kCols / 8, kStep = kThreads / kPer;  // 16-byte pieces of a row; rows apart
  const uint16_t* p;
  int64_t stride;
  int width;
  bool vec;

  __device__ __forceinline__ void load(uint32_t tile, int t0, int len) const {
    if (vec) {
      const int r = threadIdx.x / kPer, c = (threadIdx.x % kPer) * 8;
      const uint16_t* src = p + static_cast<int64_t>(t0 + r) * stride + c;
      const uint32_t dst = tile + r * Tile<kCols>::kPitch + c * 2;
      const int64_t step = kStep * stride;
      if (t0 + kChunk <= len && c < width) {
#pragma unroll
        for (int i = 0; i < kChunk / kStep; ++i, src += step)
          cp_async_16(dst + i * kStep * Tile<kCols>::kPitch, src, true);
      } else {
        const int live = c < width ? len - t0 - r : 0;
#pragma unroll
        for (int i = 0; i < kChunk / kStep; ++i, src += step) {
          const bool ok = i * kStep < live;
          cp_async_16(dst + i * kStep * Tile<kCols>::kPitch, ok ? src : p, ok);
        }
      }
    } else {
#pragma unroll 4
      for (int e = threadIdx.x; e < kChunk * kCols; e += kThreads) {
        const int r = e / kCols, c = e % kCols;
        const uint16_t x = t0 + r < len && c < width ? p[static_cast<int64_t>(t0 + r) * stride + c] : uint16_t(0);
        st_shared_u16(tile + r * Tile<kCols>::kPitch + c * 2, x);
      }
    }
  }

  // Whether one of the values that this thread has copied (and waited for) is not finite.
  __device__ __forceinline__ bool copied_not_finite(uint32_t tile) const {
    uint32_t any = 0u;
    if (vec) {
      const uint32_t at = tile + threadIdx.x / kPer * Tile<kCols>::kPitch + threadIdx.x % kPer * 16;
#pragma unroll
      for (int i = 0; i < kChunk / kStep; ++i) {
        const uint4 x = ld_shared_v4(at + i * kStep * Tile<kCols>::kPitch);
        any |= not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w);
      }
    } else {
#pragma unroll 4
      for (int e = threadIdx.x; e < kChunk * kCols; e += kThreads)
        any |= not_finite(ld_shared_u16(tile + e / kCols * Tile<kCols>::kPitch + e % kCols * 2));
    }
    return (any & kNotFinite) != 0u;
  }
};

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
  sub2(x, y, bf16lo(hi), bf16hi(hi));
  mid = pack_bf16x2(x, y);
  sub2(x, y, bf16lo(mid), bf16hi(mid));
  lo = pack_bf16x2(x, y);
}

// As two, whose sum is good to 2^-16.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  sub2(x, y, bf16lo(hi), bf16hi(hi));
  lo = pack_bf16x2(x, y);
}

// The same of two bf16 values times two weights, as three.
__device__ __forceinline__ void split3_weighted(uint32_t k, float w0, float w1, uint32_t& hi, uint32_t& mid,
                                                uint32_t& lo) {
  float x, y;
  mul2(x, y, bf16lo(k), bf16hi(k), w0, w1);
  split3(x, y, hi, mid, lo);
}

// The decays of one chunk.  l_i is the sum of D A over the chunk's steps up to
// i; the factor exp(l_i - l_j) of row block ib and a step j before the block is
// row[i] col[ib - 1][j] with the sum before the block as the reference, so a
// chunk takes a few hundred exponentials and not 64 x 64.  Made once per call
// for every (chain, chunk) and read by the chunk's blocks.
struct __align__(16) ChunkDecay {
  float first[kChunk];   // exp(l_i)
  float row[kChunk];     // exp(l_i - l before i's block)
  float rel[kChunk];     // l_i - l before i's block,
  float rel_lo[kChunk];  // and the part of it that rel leaves out: differences of long sums keep their bits
  float D[kChunk];       // step sizes, 0 behind the sequence's end
  float col[3][kChunk];  // exp(l before block ib - l_j) for j < 16 ib, ib = 1 .. 3 (else 0); the forward's times D_j
  float wD[kChunk];      // exp(l_63 - l_j) D_j, for the walks; the forward's outputs leave it out
};
constexpr int kChunkDecayCopied = 8 * kChunk * 4;
static_assert(kChunkDecayCopied == 2048 && sizeof(ChunkDecay) == kChunkDecayCopied + kChunk * 4,
              "128 copies of 16 bytes for the outputs");

// What the backward reads besides.
struct __align__(16) ChunkDecayGrad {
  ChunkDecay d;
  float last[kChunk];    // exp(l_63 - l_j)
  float sg[kChunk];      // sigmoid(dt + dt_bias)
};

// Decays of every (chain, chunk) into `out` (ChunkDecay, or ChunkDecayGrad for
// the backward), exp(l_63) into tot; clears the status block.
cudaError_t launch_ssm_decay(const SsmArgs& a, void* out, float* tot, int nc, bool grad, StatusBlock* status,
                             cudaStream_t s);

// exp(a) for a difference a of sums, by the hardware's 2^x.
__device__ __forceinline__ float exp_fast(float a) { return ex2_fast(1.44269504f * a); }

}  // namespace m2rnn
