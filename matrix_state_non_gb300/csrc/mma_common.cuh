// Helpers for the register-resident warp-MMA scan kernels (V = 64 value
// columns, 16 key rows per CTA): mma.sync m16n8k16 bf16 fragments, ldmatrix,
// movmatrix, the XOR-swizzled 16 x 64 bf16 operand tile in shared memory,
// and host-side TMA tensor-map construction.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace m2rnn {

// D (16 x 8, fp32) += A (16 x 16, bf16, row) * B (16 x 8, bf16, col).
// Fragment ownership, g = lane / 4, q = lane % 4:
//   A: a0 = A[g][2q..2q+1], a1 = A[g+8][2q..], a2 = A[g][2q+8..], a3 = A[g+8][2q+8..]
//   B: b0 = B[2q..2q+1][g], b1 = B[2q+8..2q+9][g]
//   C/D: c0 = D[g][2q], c1 = D[g][2q+1], c2 = D[g+8][2q], c3 = D[g+8][2q+1]
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A * B with a zero accumulator input.
__device__ __forceinline__ void mma_bf16_16816_zc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                  uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// D = A * B with a zero accumulator input, fp16 operands.
__device__ __forceinline__ void mma_f16_16816_zc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The same with fp16 operands (A and B both fp16).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x split into bf16 hi + lo (x - hi - lo is below 2^-16 |x|), as a bf16 pair
// {hi, lo} (hi in the low half).
__device__ __forceinline__ uint32_t bf16_hilo(float x) {
  const uint32_t hb = pack_bf16x2(x, 0.f) & 0xFFFFu;
  const float lo = x - __uint_as_float(hb << 16);
  return hb | (pack_bf16x2(lo, 0.f) << 16);
}

// Sum over the 32 lanes of x, in every lane, on the tensor core (no shuffles):
// with A = ones, a B fragment holding {hi, lo} of lane (g, q)'s x at rows 2q,
// 2q + 1 of column g sums the four lanes of group g (result s_n in column n);
// lane (g, q) then holds s_2q, s_2q+1, whose hi and lo parts form the B
// fragment of a second MMA that sums the eight groups.  Products with one are
// exact and the accumulation is fp32; the order is fixed.
__device__ __forceinline__ float warp_sum_mma(float x) {
  const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  mma_bf16_16816(d, ones, bf16_hilo(x), 0u);
  const uint32_t h0 = bf16_hilo(d[0]), h1 = bf16_hilo(d[1]);
  float e[4] = {0.f, 0.f, 0.f, 0.f};
  mma_bf16_16816(e, ones, (h0 & 0xFFFFu) | (h1 << 16), (h0 >> 16) | (h1 & 0xFFFF0000u));
  return e[0];
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Transpose of an 8 x 8 bf16 tile held one b32 (two elements) per thread.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A 16-row x 64-column bf16 tile, 128 bytes per row, 16-byte chunks XOR-
// swizzled by (row mod 8) so that ldmatrix row fetches hit distinct banks.
__device__ __forceinline__ uint32_t tile_off(int row, int col) {
  return static_cast<uint32_t>(row * 128 + ((((col >> 3) ^ (row & 7)) & 7) << 4) + (col & 7) * 2);
}

// Address thread `lane` hands to ldmatrix.x4 for the 16 x 16 sub-tile at
// column block kt (columns 16kt..16kt+15): matrices (rows 0-7, k 0-7),
// (rows 8-15, k 0-7), (rows 0-7, k 8-15), (rows 8-15, k 8-15).
__device__ __forceinline__ uint32_t ldsm_addr_a(uint32_t tile, int kt, int lane) {
  const int mi = lane >> 3, r = lane & 7;
  const int row = r + (mi & 1) * 8;
  const int col = 16 * kt + (mi >> 1) * 8;
  return tile + tile_off(row, col);
}

// Address for ldmatrix.x4.trans giving the B fragments (k = tile row, n =
// tile column) of two adjacent n-tiles 16nt2..16nt2+15: matrices
// (k 0-7, n 0-7), (k 8-15, n 0-7), (k 0-7, n 8-15), (k 8-15, n 8-15).
__device__ __forceinline__ uint32_t ldsm_addr_b_trans(uint32_t tile, int nt2, int lane) {
  const int mi = lane >> 3, r = lane & 7;
  const int row = r + (mi & 1) * 8;
  const int col = 16 * nt2 + (mi >> 1) * 8;
  return tile + tile_off(row, col);
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) { return pack_bf16x2(lo, hi); }

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void st_shared_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Explicit shared-space loads and stores for the step loops (the inputs sit
// in shared memory behind computed offsets; these keep every access a plain
// shared-memory instruction).
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_b32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_shared_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_shared_f32x2(uint32_t addr, float2 v) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_shared_f32x4(uint32_t addr, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Streaming (evict-first) 16-byte global store: data read back much later.
__device__ __forceinline__ void st_global_cs_v4(void* ptr, uint4 v) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(ptr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// fp16 pairs (IEEE binary16, round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16lo(uint32_t w) {
  float f;
  asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;\n}" : "=f"(f) : "r"(w));
  return f;
}
__device__ __forceinline__ float f16hi(uint32_t w) {
  float f;
  asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, h;\n}" : "=f"(f) : "r"(w));
  return f;
}

// fp16 pair -> two fp32 (lo in .x).
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w) { return make_float2(f16lo(w), f16hi(w)); }

// A pair of bf16 inputs re-encoded as fp16 (exact for magnitudes in fp16's
// normal range; |x| >= 65520 becomes infinite, see f16x2_finite).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) { return pack2_f16(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ bool f16x2_finite(uint32_t x) {
  return (x & 0x7C00u) != 0x7C00u && (x & 0x7C000000u) != 0x7C000000u;
}

// The recurrent state enters the state-transform MMAs as fp16 (|H| <= 1, 11
// significant bits) with W re-encoded as fp16: a bf16 state operand (8 bits)
// perturbs Z_t by ~2e-3 relative, and the backward chain can amplify that
// over thousands of steps; fp16 cuts it eightfold at no extra cost.

// The Z stash written by the V = 64 tcgen05 forward for the warp-MMA
// backward: for each (chain, row block of 16 rows) and step, 2 KB = 2 row runs
// x 64 columns x 8 fp16, the 16 bytes at (run c, column j) holding
// Z[8c .. 8c+7][j] (the forward's thread for that column and run writes them
// with one store).  One row block's steps are contiguous, so a chunk of steps
// is one bulk copy.
constexpr uint32_t kZStepBytes = 2048;

// Bounded wait without the CTA-wide abort flag: used by the compute warps,
// which then agree on the outcome through a flag read after a named barrier.
template <bool kClusterScope = false>
__device__ __forceinline__ bool mbar_wait_timed(uint32_t bar, uint32_t parity, StatusBlock* status,
                                                uint32_t where) {
  volatile int never = 0;
  return mbar_wait<kClusterScope>(bar, parity, &never, status, where);
}

// Host: 4-D bf16 / fp32 tensor map over [B][T][N][X] (X innermost), box
// {bx, 1, by, 1}, no swizzle, zero fill out of bounds.
bool make_tensor_map_btnx(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, int B,
                          int T, int N, int X, int bx, int by);

// Host: 4-D bf16 tensor map {X, heads, T, B} of rows `row_stride` elements
// apart (a column slice of a wider tensor), box {bx, 1, bt, 1} of 128-byte
// rows, 128-byte swizzle, zero fill out of bounds.
bool make_tensor_map_rows(CUtensorMap* m, const void* base, int X, int heads, int64_t row_stride, int T, int B, int bx,
                          int bt);

}  // namespace m2rnn
