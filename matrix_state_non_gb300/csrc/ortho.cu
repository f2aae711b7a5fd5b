// Orthogonalised update: the singular values of a gradient's matrix are all
// brought near 1 by Newton-Schulz steps (as the Muon optimiser does),
//     X = G / (|G|_F + eps),
//     X <- a X + (b A + c A A) X,  A = X X^T,
// with a = 3.4445, b = -4.7750, c = 2.0315; the smaller side makes A (a tall G
// is transposed on the way in and out).
//
// A step is three products on tcgen05, a launch each, over tiles of 128 rows of
// all matrices: A = X X^T and P = b A + c A A (symmetric: the tiles on and above
// the diagonal, written on both sides of it) and X' = a X + P X.
//
// Precision.  Operands are fp16 (11 bits, rounded to nearest) with fixed powers
// of two in front: the polynomial maps [0, 1.2025] into itself, so that no entry
// of X exceeds 1.2025, of A 1.4461, of P 2.81.  Matrices with a side of up to 64 are
// taken by ortho_small.cu and ortho_thin.cu.  X is kept in two fp16 parts (22
// bits) between steps: small singular values grow 480-fold in five steps, and
// the rounding noise of X in one part would grow with them (for a matrix of
// rank 1 the result would be 0.15 off; it is 3e-4).  Noise of A and P does not
// grow: P X stays in the row space of X.  What they leave is 1.0e-3 to 1.9e-3 of
// the result (1.3e-3 at 1024 x 1024 of random entries), the output's rounding to
// bf16 1.7e-3.  With X's lower part in P X as well (kLow) it is 1.0e-3 to
// 1.5e-3; matrices of fewer than 512 rows, where errors average least, get that.
// One part holds the first X where G is bf16, and, from 512 rows on, the last
// step's, whose noise grows once (a matrix of rank 1 comes out 1e-3 off for it).
// The three before it have a byte for the lower part there, 14 to 15 bits in all
// (another 9e-4 for rank 1): noise grows 3.44-fold a step where X has nothing, and
// with bytes before that seven steps left 1.8e-2 of a matrix of rank 1, eight 4e-2.
//
// 24 of 1024 x 4096 bf16, 5 steps: 1.51 to 1.60 ms (seven: 2.27), fp32 1.66; of 1.57, A 5 x 88 us (1.5 PFLOP/s, 3.2
// waves of tiles), P 5 x 34, X' 146 to 166 (15 TB/s between L2 and the SMs, 3.6 of
// HBM), the norm and the first X 100.  With two fp16 parts in all steps X' was 185,
// bound by HBM, and the whole 1.71 ms; with two but in the first and last 1.61.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"
#include "internal.h"
#include "ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 0x1p14f;  // X, A are stored times 2^14, P times 2^13

__host__ __device__ constexpr int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// ---------------------------------------------------------------------------
// The norm and the first X
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256, kSumParts = 64;  // blocks of a matrix, at most
constexpr int kSumCount = 16384;                  // values for a block, at least

// Eight values from p on (on 16 bytes).
__device__ __forceinline__ void load_8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The thread's share of a sum of squares over a block's piece, a multiple of 8
// values if `vec`.  Squares that leave the fp32 range are caught as in
// grad_clip.cu: next to x^2 it sums (x 2^90)^2, for where the first may have lost
// bits, and a sum that is not finite is taken again in fp64.
template <typename E>
__device__ double square_sum(const E* g, int64_t from, int64_t to, bool vec) {
  float s = 0.f, up = 0.f;
  auto add = [&](float x) {
    const float y = x * 0x1p90f;
    s = fmaf(x, x, s);
    up = fmaf(y, y, up);
  };
  if (vec) {
#pragma unroll 4
    for (int64_t i = from + 8 * threadIdx.x; i < to; i += 8 * kSumThreads) {
      float v[8];
      load_8(g + i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) add(v[e]);
    }
  } else {
#pragma unroll 8
    for (int64_t i = from + threadIdx.x; i < to; i += kSumThreads) add(to_f32(g[i]));
  }
  if (s < 0x1p-60f) return static_cast<double>(up) * 0x1p-180;
  if (s <= 3.4e38f) return s;
  double w = 0.;
  const int64_t step = vec ? 8 * kSumThreads : kSumThreads, run = vec ? 8 : 1;
  for (int64_t i = from + run * threadIdx.x; i < to; i += step)
    for (int64_t j = i; j < i + run; ++j) {
      const double x = to_f32(g[j]);
      w += x * x;
    }
  return w;
}

template <typename E>
__global__ void __launch_bounds__(kSumThreads) ortho_sum_kernel(const E* g, int64_t size, int parts, double* part,
                                                                StatusBlock* status) {
  if (blockIdx.x == 0 && threadIdx.x < sizeof(StatusBlock) / 4) reinterpret_cast<uint32_t*>(status)[threadIdx.x] = 0u;
  __shared__ double red[kSumThreads / 32];
  const int64_t mat = blockIdx.x / parts;
  const int p = static_cast<int>(blockIdx.x - mat * parts);
  const int64_t per = round_up((size + parts - 1) / parts, 8);
  double acc = square_sum(g + mat * size, p * per, min(size, (p + 1) * per), size % 8 == 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  let_next();
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSumThreads / 32; ++i) acc += red[i];
    part[blockIdx.x] = acc;
  }
}

// In every thread of a block: what the matrix's entries are multiplied with.
__device__ __forceinline__ Inverse first_factor(const double* part, int parts, float eps, Inverse* shared) {
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

union Eight {
  uint4 v;
  __half2 h[4];
};

__device__ __forceinline__ void split_8(const float (&v)[8], Eight& hi, Eight& lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi.h[e] = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
    lo.h[e] = __floats2half2_rn(v[2 * e] - __half2float(hi.h[e].x), v[2 * e + 1] - __half2float(hi.h[e].y));
  }
}

// What the first X is made with.  fp32: the factor, and X is in two parts.  bf16:
// the power of two below it, which leaves X in one part with all its digits; the
// rest, in [1, 2), is a factor of the first step (`rest`, for each matrix).
template <typename E>
__device__ __forceinline__ Inverse first_scale(Inverse f, float* rest) {
  if constexpr (sizeof(E) == 2) {
    int e = 0;
    const bool usual = f.factor > 0.f && f.factor <= 3.4e38f;
    const float r = usual ? 2.f * frexpf(f.factor, &e) : 1.f;
    if (threadIdx.x == 0 && rest != nullptr) *rest = r;
    if (usual) f.factor = ldexpf(1.f, e - 1);
  }
  return f;
}
__device__ __forceinline__ void store_first(float (&v)[8], Inverse f, __half* hi, __half* lo, int64_t at) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = f.of(v[e]) * kScaleX;
  Eight h, l;
  split_8(v, h, l);
  *reinterpret_cast<uint4*>(hi + at) = h.v;
  if (lo != nullptr) *reinterpret_cast<uint4*>(lo + at) = l.v;
}

// X [m][pitch] from G [m][k] (lo: null where one part is enough): eight values of a
// row to a thread, a block takes kLoadRun of its turns.
constexpr int kLoadRun = 4;
template <typename E>
__global__ void __launch_bounds__(256) ortho_load_kernel(const E* g, const double* part, int parts, float eps, __half* hi,
                                                         __half* lo, float* rest, int m, int k, int pitch, int blocks) {
  __shared__ Inverse shared;
  const int64_t mat = blockIdx.x / blocks;
  const int block = static_cast<int>(blockIdx.x - mat * blocks), per_row = pitch / 8;
  const E* p = g + mat * m * k;
  wait_previous();
  const Inverse f = first_scale<E>(first_factor(part + mat * parts, parts, eps, &shared), block == 0 ? rest + mat : nullptr);
  const int64_t size = static_cast<int64_t>(m) * per_row;
#pragma unroll
  for (int u = 0; u < kLoadRun; ++u) {
    const int64_t i = (static_cast<int64_t>(block) * kLoadRun + u) * 256 + threadIdx.x;
    if (i >= size) break;
    const int64_t r = i / per_row;
    const int c = static_cast<int>(i - r * per_row) * 8;
    float v[8];
    if (k % 8 == 0) {
      load_8(p + r * k + c, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < k ? to_f32(p[r * k + c + e]) : 0.f;
    }
    store_first(v, f, hi, lo, mat * m * pitch + i * 8);
  }
  let_next();
}

// The same from G [k][m] (tall), tiles of 64 x 64 through shared memory.
constexpr int kTurn = 64;
template <typename E>
__global__ void __launch_bounds__(256) ortho_load_tall_kernel(const E* g, const double* part, int parts, float eps, __half* hi,
                                                              __half* lo, float* rest, int m, int k, int pitch, int tiles_m,
                                                              int tiles) {
  __shared__ float t[kTurn][kTurn + 1];
  __shared__ Inverse shared;
  const int64_t mat = blockIdx.x / tiles;
  const int tile = static_cast<int>(blockIdx.x - mat * tiles);
  const int r0 = tile % tiles_m * kTurn, c0 = tile / tiles_m * kTurn;
  const E* p = g + mat * m * k;
#pragma unroll 8
  for (int i = threadIdx.x; i < kTurn * kTurn; i += 256) {
    const int r = i % kTurn, c = i / kTurn;
    t[r][c] = r0 + r < m && c0 + c < k ? to_f32(p[static_cast<int64_t>(c0 + c) * m + r0 + r]) : 0.f;
  }
  wait_previous();
  const Inverse f = first_scale<E>(first_factor(part + mat * parts, parts, eps, &shared), tile == 0 ? rest + mat : nullptr);
#pragma unroll
  for (int i = threadIdx.x; i < kTurn * kTurn / 8; i += 256) {
    const int r = i / (kTurn / 8), c = i % (kTurn / 8) * 8;
    if (r0 + r >= m || c0 + c >= pitch) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = t[r][c + e];
    store_first(v, f, hi, lo, (mat * m + r0 + r) * pitch + c0 + c);
  }
  let_next();
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
enum { kGram = 0, kPoly = 1, kUpdate = 2 };
// Lower parts: fp16; or the upper byte of an fp16 (2 bits of mantissa).
enum { kNone = 0, kBytes = 1, kHalf = 2 };

struct ProductArgs {
  uint16_t* last;  // kUpdate of the last step: the result in bf16, [m][k] or (tall) [k][m]
  const float* rest;  // [n], or null: X is that times what is stored
  StatusBlock* status;
  int m, k;   // X is m x k
  int inner;  // of the product
  int tiles_m, tiles_n, tiles;  // of one matrix; those that are computed
  int items;  // of all matrices
  bool tall;
  bool direct;  // last: rows that TMA cannot store (not on 16 bytes)
  int in_low, out_low;  // kUpdate: the lower parts of X and X', kNone, kBytes or kHalf
  int skip;  // test hook: stages of the first block that never fill, 0 or 1
};

// By TMA: the operands; `in`: kPoly: A; kUpdate: X, its lower part in_low; `out`: A, P or X' (out_low), or the result.
struct Operands {
  CUtensorMap left, right, right_low, in, in_low, out, out_low;
};

constexpr int kRows = 128, kDepth = 64;  // a tile's rows, the inner dimension of a stage
constexpr int kBoxRows = 32;            // of the right operand's loads, K-major
constexpr int kBlockBytes = 32 * 32 * 2;   // what an epilogue warp stores at once
__host__ __device__ constexpr int low_bytes(int low) { return low == kHalf ? kBlockBytes : low == kBytes ? kBlockBytes / 2 : 0; }
constexpr int kEpilogueWarps = 8, kFirstEpilogue = 2, kProductThreads = 32 * (kFirstEpilogue + kEpilogueWarps);

// kPair: two blocks of a cluster on two SMs share a tile of 256 rows, each with
// half of its rows, the accumulators of those, and half of its columns' operand.
template <int kMode, int kN, bool kLow, bool kPair>
struct Shape {
  static constexpr int kTileRows = kPair ? 2 * kRows : kRows, kOwnN = kPair ? kN / 2 : kN;
  static constexpr int kLeft = kRows * kDepth * 2, kRight = kOwnN * kDepth * 2;
  static constexpr int kStage = kLeft + kRight * (kLow ? 2 : 1);
  // An epilogue warp's ring of what it reads and writes: two 32 x 32 blocks a turn.
  static constexpr int kTurns = kMode == kGram ? 1 : kMode == kPoly || kLow ? 2 : 3, kTurn = 2 * kBlockBytes;
  static constexpr int kStages = kMode == kGram ? 6 : kMode == kPoly ? 5 : kLow ? 3 : 4;
  static constexpr int kOffRing = kStages * kStage;
  static constexpr int kOffBar = kOffRing + kEpilogueWarps * kTurns * kTurn;
  static constexpr int kSmem = kOffBar + 512 + 1024;  // 1024: alignment
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(2 * kN <= 512, "tensor memory");
};

struct Item {
  int mat, i, j;  // (a tile's row and column)
};
// Symmetric products: of row i the tiles with a column at or right of the diagonal.
template <int kMode, int kN, int kTileRows>
__device__ __forceinline__ Item item_at(const ProductArgs& A, int id) {
  Item t;
  t.mat = static_cast<unsigned>(id) / static_cast<unsigned>(A.tiles);
  int left = id - t.mat * A.tiles;
  if constexpr (kMode == kUpdate) {
    t.j = static_cast<unsigned>(left) / static_cast<unsigned>(A.tiles_m);
    t.i = left - t.j * A.tiles_m;  // neighbours share the columns of X
  } else {
    t.i = 0;
    int first = 0;
    while (left >= A.tiles_n - first) {
      left -= A.tiles_n - first;
      ++t.i;
      first = t.i * kTileRows / kN;
    }
    t.j = first + left;
  }
  return t;
}

// Tensor memory, products and their completion for one block or a pair (the pair's products are issued by its first
// block; both hear of their completion, on barriers at the same place).
template <bool kPair>
__device__ __forceinline__ void acquire_tmem(uint32_t slot) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  }
}
template <bool kPair>
__device__ __forceinline__ void release_tmem(uint32_t tmem) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  else
    tmem_dealloc(tmem, 512);
}
template <bool kPair>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc_mma_f16_ss(d, a, b, idesc, accumulate);
}
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}

// `bar` may be the other block's of a pair.
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t from, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(from), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// A thread's 16 of 32 bytes in a block of lower parts that are bytes (rows of 32 bytes, swizzled).
__device__ __forceinline__ uint32_t byte_line(uint32_t block, int lane, int half) {
  return block + kBlockBytes + lane * 32 + ((half ^ (lane >> 2 & 1)) << 4);
}

// A row's 32 columns of the result from the accumulators and what the turn's place holds: v.  f: what the stored X
// lacks.  Two values to an instruction where that can be: the epilogue's instructions are what is beside the products.
template <int kMode, int kIn>
__device__ __forceinline__ void combine_as(float (&v)[32], const uint32_t (&acc)[32], uint32_t block, int lane, float f) {
  const uint32_t line = block + lane * 64, swz = (lane >> 1) & 3;
  const float by = kMode == kGram ? 0x1p-14f * f * f : kMode == kPoly ? kC * 0x1p-15f : 0x1p-13f * f;
  const float a = kMode == kPoly ? kB * 0.5f : kA * f;
  uint32_t bytes[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    Eight h, l;
    if constexpr (kMode != kGram) h.v = ld_shared_v4(line + ((q ^ swz) << 4));
    if constexpr (kIn == kHalf) l.v = ld_shared_v4(line + kBlockBytes + ((q ^ swz) << 4));
    if constexpr (kIn == kBytes) {
      if (q % 2 == 0) {
        const uint4 u = ld_shared_v4(byte_line(block, lane, q / 2));
        bytes[0] = u.x, bytes[1] = u.y, bytes[2] = u.z, bytes[3] = u.w;
      }
      const uint32_t b0 = bytes[2 * (q % 2)], b1 = bytes[2 * (q % 2) + 1];
      l.v = make_uint4(__byte_perm(b0, 0u, 0x1404), __byte_perm(b0, 0u, 0x3424), __byte_perm(b1, 0u, 0x1404),
                       __byte_perm(b1, 0u, 0x3424));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float &v0 = v[8 * q + 2 * e], &v1 = v[8 * q + 2 * e + 1];
      mul2(v0, v1, __uint_as_float(acc[8 * q + 2 * e]), __uint_as_float(acc[8 * q + 2 * e + 1]), by, by);
      if constexpr (kMode != kGram) {
        const float2 x = __half22float2(h.h[e]);
        fma2(v0, v1, x.x, x.y, a, a);
      }
      if constexpr (kIn != kNone) {
        const float2 x = __half22float2(l.h[e]);
        fma2(v0, v1, x.x, x.y, a, a);
      }
    }
  }
}
template <int kMode>
__device__ __forceinline__ void combine(float (&v)[32], const uint32_t (&acc)[32], uint32_t block, int lane, float f, int low) {
  if (kMode == kUpdate && low == kBytes)
    combine_as<kMode, kBytes>(v, acc, block, lane, f);
  else if (kMode == kUpdate && low == kHalf)
    combine_as<kMode, kHalf>(v, acc, block, lane, f);
  else
    combine_as<kMode, kNone>(v, acc, block, lane, f);
}

// The warp's 32 x 32 block of the result from row r0 and column c0 on, to where it belongs: through the place `block`
// to TMA, which one lane commits; rows that TMA cannot store, directly.  kLast: in bf16.
template <int kMode, int kOut, bool kLast>
__device__ __forceinline__ void emit_as(const Operands& O, const ProductArgs& A, const float (&v)[32], uint32_t block, int r0,
                                        int c0, int mat, int lane) {
  const uint32_t line = block + lane * 64, swz = (lane >> 1) & 3;
  const bool mirror = (kMode != kUpdate && c0 != r0) || (kLast && A.tall);  // the diagonal's own blocks are whole
  uint32_t bytes[4];
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = v[8 * q + e] * (kLast ? 1.f / kScaleX : 1.f);
    Eight h;
    if constexpr (kLast) {
      h.v = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) h.h[e] = __floats2half2_rn(w[2 * e], w[2 * e + 1]);
    }
    st_shared_v4(line + ((q ^ swz) << 4), {h.v.x, h.v.y, h.v.z, h.v.w});
    if constexpr (kOut != kNone) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = __half22float2(h.h[e]);
        fma2(w[2 * e], w[2 * e + 1], x.x, x.y, -1.f, -1.f);
      }
    }
    if constexpr (kOut == kHalf) {
      Eight l;
#pragma unroll
      for (int e = 0; e < 4; ++e) l.h[e] = __floats2half2_rn(w[2 * e], w[2 * e + 1]);
      st_shared_v4(line + kBlockBytes + ((q ^ swz) << 4), {l.v.x, l.v.y, l.v.z, l.v.w});
    }
    if constexpr (kOut == kBytes) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(w[e], w[e + 1]), __NV_SATFINITE, __NV_E5M2);
        const uint32_t up = __nv_cvt_float2_to_fp8x2(make_float2(w[e + 2], w[e + 3]), __NV_SATFINITE, __NV_E5M2);
        bytes[2 * (q % 2) + e / 4] = lo | up << 16;
      }
      if (q % 2 == 1) st_shared_v4(byte_line(block, lane, q / 2), {bytes[0], bytes[1], bytes[2], bytes[3]});
    }
    if (mirror) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // row 8 q + e of the other side's block, column `lane`
        const int row = 8 * q + e;
        const uint32_t at = block + kBlockBytes + row * 64 + ((((lane >> 3) ^ (row >> 1)) & 3) << 4) + (lane & 7) * 2;
        const __half2 pair = h.h[e / 2];
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(__half_as_ushort(e % 2 == 0 ? pair.x : pair.y)) : "memory");
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (!(kLast && A.tall)) tma_store_3d(&O.out, block, c0, r0, mat);
    if (kOut != kNone) tma_store_3d(&O.out_low, block + kBlockBytes, c0, r0, mat);
    if (mirror) tma_store_3d(&O.out, block + kBlockBytes, r0, c0, mat);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
template <int kMode>
__device__ __forceinline__ void emit(const Operands& O, const ProductArgs& A, const float (&v)[32], uint32_t block, int r0, int c0,
                                     int mat, int lane) {
  if constexpr (kMode != kUpdate) {
    emit_as<kMode, kNone, false>(O, A, v, block, r0, c0, mat, lane);
  } else if (A.last == nullptr) {
    if (A.out_low == kBytes)
      emit_as<kMode, kBytes, false>(O, A, v, block, r0, c0, mat, lane);
    else if (A.out_low == kHalf)
      emit_as<kMode, kHalf, false>(O, A, v, block, r0, c0, mat, lane);
    else
      emit_as<kMode, kNone, false>(O, A, v, block, r0, c0, mat, lane);
  } else if (!A.direct) {
    emit_as<kMode, kNone, true>(O, A, v, block, r0, c0, mat, lane);
  } else {
    const int r = r0 + lane;
    const int64_t right = A.tall ? A.m : 1, down = A.tall ? 1 : A.k;
    uint16_t* to = A.last + (static_cast<int64_t>(mat) * A.m * A.k + r * down + c0 * right);
    if (r < A.m) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (c0 + e < A.k) to[e * right] = from_f32<uint16_t>(v[e] * (1.f / kScaleX));
    }
  }
}

// A wait that gives up leaves its block's tiles as they were.  The last step's blocks make that visible where nobody
// looks at the status: NaN in their tiles, if a wait of theirs (abort) or of any launch before theirs gave up.
template <int kMode>
__device__ __forceinline__ bool failed(const ProductArgs& A, int abort) {
  return kMode == kUpdate && A.last != nullptr && (abort != 0 || *const_cast<const volatile unsigned int*>(&A.status->code) != 0u);
}
__device__ __forceinline__ void spoil(const ProductArgs& A, int mat, int r, int c0, int width) {
  const int64_t right = A.tall ? A.m : 1, down = A.tall ? 1 : A.k;
  uint16_t* to = A.last + (static_cast<int64_t>(mat) * A.m * A.k + r * down);
  for (int c = c0; r < A.m && c < min(c0 + width, A.k); ++c) to[c * right] = 0x7fc0;
}

template <int kMode, int kN, bool kLow, bool kPair>
__global__ void __launch_bounds__(kProductThreads, 1)
    ortho_product_kernel(const __grid_constant__ Operands O, ProductArgs A) {
  using S = Shape<kMode, kN, kLow, kPair>;
  constexpr int kBlocks = kPair ? 2 : 1;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_u32(smem), bars = base + S::kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };         // [stages] TMA -> products
  auto empty = [&](int s) { return bars + 64 + 8 * s; };   // [stages] products -> TMA
  auto done = [&](int s) { return bars + 128 + 8 * s; };   // [2] products -> epilogue
  auto tfree = [&](int s) { return bars + 144 + 8 * s; };  // [2] epilogue -> products
  auto there = [&](int w, int s) { return bars + 192 + 8 * (w * S::kTurns + s); };  // [warps][turns] TMA -> epilogue
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffBar + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffBar + 164);
  static_assert(S::kStages <= 8, "barriers");
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / kBlocks, step = gridDim.x / kBlocks;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(done(s), 1);
      mbar_init(tfree(s), 32 * kEpilogueWarps * kBlocks);
    }
    for (int s = 0; s < kEpilogueWarps * S::kTurns; ++s) mbar_init(there(0, s), 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 1) acquire_tmem<kPair>(smem_u32(tmem_slot));
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (kPair)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_previous();
  const int depth = (A.inner + kDepth - 1) / kDepth;

  if (warp == 0) {
    // ---------------- loads ----------------
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");  // what earlier launches stored, before TMA reads it
      int d0 = first == 0 ? A.skip : 0, u = d0;  // stages filled
      bool ok = true;
      for (int id = first; ok && id < A.items; id += step) {
        const Item t = item_at<kMode, kN, S::kTileRows>(A, id);
        const int mat = t.mat;
        for (int d = d0; d < depth; ++d, ++u) {
          const int s = u % S::kStages;
          if (u >= S::kStages && !mbar_wait(empty(s), (u / S::kStages - 1) & 1, abort_flag, A.status, kWhereOrthoEmpty)) {
            ok = false;
            break;
          }
          const uint32_t to = base + s * S::kStage, bar = kPair ? mapa_shared(full(s), 0) : full(s);
          if (rank == 0) mbar_arrive_expect_tx(full(s), S::kStage * kBlocks);
          tma_load_3d<kPair>(to, &O.left, bar, d * kDepth, t.i * S::kTileRows + rank * kRows, mat);
          const int n0 = t.j * kN + rank * S::kOwnN;
          if constexpr (kMode == kUpdate) {  // 64 columns of 64 rows at a time
#pragma unroll
            for (int c = 0; c < S::kOwnN; c += 64) {
              tma_load_3d<kPair>(to + S::kLeft + c * kDepth * 2, &O.right, bar, n0 + c, d * kDepth, mat);
              if (kLow) tma_load_3d<kPair>(to + S::kLeft + S::kRight + c * kDepth * 2, &O.right_low, bar, n0 + c, d * kDepth, mat);
            }
          } else {
#pragma unroll
            for (int r = 0; r < S::kOwnN; r += kRows)
              tma_load_3d<kPair>(to + S::kLeft + r * kDepth * 2, &O.left, bar, d * kDepth, n0 + r, mat);
          }
        }
        d0 = 0;
      }
      if (!ok && rank == 0)  // the copies in flight land before the block ends (a pair's: before it has met)
        for (int x = max(0, u - S::kStages); x < u; ++x)
          mbar_wait_timed(full(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (rank == 0) {
    constexpr uint32_t kId = idesc_f16_f32(S::kTileRows, kN, false, kMode == kUpdate);
    int u = 0, n = 0;  // stages, tiles
    bool ok = true;
    for (int id = first; ok && id < A.items; id += step, ++n) {
      const int slot = n & 1;
      if (n >= 2 && !warp_wait(tfree(slot), ((n >> 1) - 1) & 1, abort_flag, A.status, kWhereOrthoFree)) break;
      tc_fence_after_sync();
      for (int d = 0; d < depth; ++d, ++u) {
        const int s = u % S::kStages;
        if (!warp_wait(full(s), (u / S::kStages) & 1, abort_flag, A.status, kWhereOrthoFull)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          tc_fence_after_sync();
          const uint32_t l = base + s * S::kStage, r = l + S::kLeft, tm = tmem + slot * kN;
#pragma unroll
          for (int kk = 0; kk < kDepth / 16; ++kk) {
            if constexpr (kMode == kUpdate) {
              multiply<kPair>(tm, desc_sw128(l + kk * 32), desc_sw128(r + kk * 2048, kDepth * 128), kId, d > 0 || kk > 0);
              if (kLow)
                multiply<kPair>(tm, desc_sw128(l + kk * 32), desc_sw128(r + S::kRight + kk * 2048, kDepth * 128), kId, 1);
            } else {
              multiply<kPair>(tm, desc_sw128(l + kk * 32), desc_sw128(r + kk * 32), kId, d > 0 || kk > 0);
            }
          }
          commit<kPair>(empty(s));
          if (d == depth - 1) commit<kPair>(done(slot));
        }
        __syncwarp();
      }
    }
    if (*abort_flag)  // the products in flight end before their memory is freed
      for (int x = max(0, u - S::kStages); x < u; ++x)
        mbar_wait_timed(empty(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
    }
  } else {
    // ---------------- epilogue: a thread has a row, its warp 32 columns at a time ----------------
    // What it reads comes by TMA, a turn or two ahead, and what it writes takes its place and goes by TMA: 64-byte
    // rows with their 16-byte pieces swizzled.
    const int me = warp - kFirstEpilogue, quarter = warp & 3, half = me >> 2;
    const int cols = kMode == kUpdate ? A.k : A.m;
    constexpr int kPerTile = kN / 64;  // turns of a tile
    const uint32_t ring = base + S::kOffRing + me * S::kTurns * S::kTurn;
    const int row = rank * kRows + quarter * 32, column = half * (kN / 2);  // in a tile
    // One lane reads ahead: the next block to read is number `next` of tile `coming`.
    int coming = first, next = 0, reads = 0;
    Item ahead = item_at<kMode, kN, S::kTileRows>(A, first);
    auto read = [&] {
      if (kMode == kGram || coming >= A.items) return;
      const int s = reads++ % S::kTurns;
      const int r0 = ahead.i * S::kTileRows + row, c0 = ahead.j * kN + column + 32 * next;
      const int low = kMode == kUpdate ? A.in_low : kNone;
      mbar_arrive_expect_tx(there(me, s), kBlockBytes + low_bytes(low));
      tma_load_3d<false>(ring + s * S::kTurn, &O.in, there(me, s), c0, r0, ahead.mat);
      if (low != kNone) tma_load_3d<false>(ring + s * S::kTurn + kBlockBytes, &O.in_low, there(me, s), c0, r0, ahead.mat);
      if (++next == kPerTile) {
        next = 0;
        coming += step;
        if (coming < A.items) ahead = item_at<kMode, kN, S::kTileRows>(A, coming);
      }
    };
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");
      for (int u = 0; u < S::kTurns - 1; ++u) read();
    }
    int u = 0, n = 0;
    bool ok = true;
    for (int id = first; ok && id < A.items; id += step, ++n) {
      const Item t = item_at<kMode, kN, S::kTileRows>(A, id);
      const int slot = n & 1, r0 = t.i * S::kTileRows + row;
      const float f = A.rest != nullptr ? A.rest[t.mat] : 1.f;
      ok = warp_wait(done(slot), (n >> 1) & 1, abort_flag, A.status, kWhereOrthoDone);
      tc_fence_after_sync();
      const uint32_t tm = tmem + slot * kN + half * (kN / 2) + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll 1
      for (int x = 0; ok && x < kPerTile; ++x, ++u) {
        const int c0 = t.j * kN + column + 32 * x, s = u % S::kTurns;
        const bool used = r0 < A.m && c0 < cols && (kMode == kUpdate || c0 >= r0);
        const uint32_t block = ring + s * S::kTurn;
        float v[32];
        if (kMode != kGram) {
          ok = warp_wait(there(me, s), (u / S::kTurns) & 1, abort_flag, A.status, kWhereOrthoIn);
          if (!ok) break;
        }
        if (used) {
          uint32_t acc[32];
          tmem_ld_32x32b<32>(tm + 32 * x, acc);
          tmem_ld_wait();
          tmem_ld_fence_regs(acc);
          combine<kMode>(v, acc, block, lane, f, A.in_low);
        }
        __syncwarp();
        if (lane == 0) {  // the turn before has left shared memory: its place is free
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          read();
        }
        if (used) emit<kMode>(O, A, v, block, r0, c0, t.mat, lane);
      }
      if (!ok) break;
      tc_fence_before_sync();
      if (rank == 0)
        mbar_arrive(tfree(slot));
      else
        mbar_arrive_cluster(mapa_shared(tfree(slot), 0));
    }
    if (lane == 0) {
      if (!ok && kMode != kGram)  // what is on its way lands before the block ends
        for (int x = u; x < reads; ++x) mbar_wait_timed(there(me, x % S::kTurns), (x / S::kTurns) & 1, nullptr, kWhereOrthoDrain);
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  }
  let_next();
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (kPair)
    cluster_sync_all();  // no block ends while the other's products read it or its epilogue signals to it
  else
    __syncthreads();
  if (warp == 1) release_tmem<kPair>(tmem);
  if (warp >= kFirstEpilogue && failed<kMode>(A, *abort_flag)) {
    const int quarter = warp & 3, half = (warp - kFirstEpilogue) >> 2;
    for (int id = first; id < A.items; id += step) {
      const Item t = item_at<kMode, kN, S::kTileRows>(A, id);
      spoil(A, t.mat, t.i * S::kTileRows + rank * kRows + quarter * 32 + lane, t.j * kN + half * (kN / 2), kN / 2);
    }
  }
}

// ---------------------------------------------------------------------------
// The same products where there are few tiles: a narrow tile (kN columns) to a
// block, so that there are enough of them, and nothing that a block does twice.
// The time is that of a launch behind another (2 us) and of a tile's operands on
// their way to one SM.  1024 x 1024, one matrix, 5 steps: 117 us; 2 of 1000 x 333:
// 100 us (163 and 140 by persistent blocks with tiles of 128 x 128; 131 and 113 with
// clusters of four that share a tile's inner dimension; 142 and 120 in one
// cooperative launch with barriers across the grid).
// ---------------------------------------------------------------------------
template <int kN, bool kLow>
struct NarrowShape {
  static constexpr int kLeft = kRows * kDepth * 2, kRight = kN * kDepth * 2, kStage = kLeft + kRight * (kLow ? 2 : 1);
  static constexpr int kStages = 196608 / kStage > 8 ? 8 : 196608 / kStage;
  // Once the products are done the stages hold the epilogue's blocks, kBlocks to a warp.
  static constexpr int kTurn = 2 * kBlockBytes, kBlocks = kN > 64 ? kN / 64 : 1;
  static constexpr int kOffBar = kStages * kStage, kSmem = kOffBar + 512 + 1024;
  static_assert(kStages <= 8 && kOffBar >= kEpilogueWarps * kBlocks * kTurn, "the stages' place");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int kMode, int kN, bool kLow>
__global__ void __launch_bounds__(kProductThreads, 1) ortho_narrow_kernel(const __grid_constant__ Operands O, ProductArgs A) {
  using S = NarrowShape<kN, kLow>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_u32(smem), bars = base + S::kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 64 + 8 * s; };
  const uint32_t done = bars + 128;
  auto there = [&](int w) { return bars + 192 + 8 * w; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffBar + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffBar + 164);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    for (int s = 0; s < kEpilogueWarps; ++s) mbar_init(there(s), 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 0 && lane == 1) {
    tma_prefetch_desc(&O.left);
    tma_prefetch_desc(&O.right);
    if (kLow) tma_prefetch_desc(&O.right_low);
    if (kMode != kGram) tma_prefetch_desc(&O.in);
    tma_prefetch_desc(&O.out);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kN);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncwarp();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const Item t = item_at<kMode, kN, kRows>(A, blockIdx.x);
  const int mat = t.mat, depth = (A.inner + kDepth - 1) / kDepth;
  // a warp's blocks: 32 rows, every second 32 of the columns
  const int me = warp - kFirstEpilogue, quarter = warp & 3, half = me >> 2;
  const int r0 = t.i * kRows + quarter * 32, blocks = (kN / 32 + 1 - half) / 2;
  auto column = [&](int x) { return 32 * (half + 2 * x); };  // in the tile
  const uint32_t ring = base + me * S::kBlocks * S::kTurn;
  wait_previous();

  if (warp == 0) {
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");
      bool ok = true;
      int u = blockIdx.x == 0 ? A.skip : 0;
      for (; u < depth; ++u) {
        const int s = u % S::kStages;
        if (u >= S::kStages && !mbar_wait(empty(s), (u / S::kStages - 1) & 1, abort_flag, A.status, kWhereOrthoEmpty)) {
          ok = false;
          break;
        }
        const uint32_t to = base + s * S::kStage, bar = full(s);
        mbar_arrive_expect_tx(bar, S::kStage);
        tma_load_3d<false>(to, &O.left, bar, u * kDepth, t.i * kRows, mat);
        if constexpr (kMode == kUpdate) {
#pragma unroll
          for (int c = 0; c < kN; c += 64) {
            tma_load_3d<false>(to + S::kLeft + c * kDepth * 2, &O.right, bar, t.j * kN + c, u * kDepth, mat);
            if (kLow) tma_load_3d<false>(to + S::kLeft + S::kRight + c * kDepth * 2, &O.right_low, bar, t.j * kN + c, u * kDepth, mat);
          }
        } else {
#pragma unroll
          for (int r = 0; r < kN; r += kBoxRows)
            tma_load_3d<false>(to + S::kLeft + r * kDepth * 2, &O.right, bar, u * kDepth, t.j * kN + r, mat);
        }
      }
      if (!ok)
        for (int x = max(0, u - S::kStages); x < u; ++x)
          mbar_wait_timed(full(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
    }
  } else if (warp == 1) {
    constexpr uint32_t kId = idesc_f16_f32(kRows, kN, false, kMode == kUpdate);
    int u = 0;
    for (; u < depth; ++u) {
      const int s = u % S::kStages;
      if (!warp_wait(full(s), (u / S::kStages) & 1, abort_flag, A.status, kWhereOrthoFull)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        const uint32_t l = base + s * S::kStage, r = l + S::kLeft;
#pragma unroll
        for (int kk = 0; kk < kDepth / 16; ++kk) {
          if constexpr (kMode == kUpdate) {
            tc_mma_f16_ss(tmem, desc_sw128(l + kk * 32), desc_sw128(r + kk * 2048, kDepth * 128), kId, u > 0 || kk > 0);
            if (kLow) tc_mma_f16_ss(tmem, desc_sw128(l + kk * 32), desc_sw128(r + S::kRight + kk * 2048, kDepth * 128), kId, 1);
          } else {
            tc_mma_f16_ss(tmem, desc_sw128(l + kk * 32), desc_sw128(r + kk * 32), kId, u > 0 || kk > 0);
          }
        }
        tc_commit(empty(s));
        if (u == depth - 1) tc_commit(done);
      }
      __syncwarp();
    }
    if (*abort_flag)
      for (int x = max(0, u - S::kStages); x < u; ++x)
        mbar_wait_timed(empty(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
  } else if (warp_wait(done, 0, abort_flag, A.status, kWhereOrthoDone) && blocks > 0) {
    // ---------------- epilogue, in the stages' place ----------------
    const int cols = kMode == kUpdate ? A.k : A.m;
    if (kMode != kGram) {
      if (lane == 0) {
        asm volatile("fence.proxy.async;" ::: "memory");
        const int low = kMode == kUpdate ? A.in_low : kNone;
        mbar_arrive_expect_tx(there(me), blocks * (kBlockBytes + low_bytes(low)));
        for (int x = 0; x < blocks; ++x) {
          const uint32_t to = ring + x * S::kTurn;
          tma_load_3d<false>(to, &O.in, there(me), t.j * kN + column(x), r0, mat);
          if (low != kNone) tma_load_3d<false>(to + kBlockBytes, &O.in_low, there(me), t.j * kN + column(x), r0, mat);
        }
      }
      if (!warp_wait(there(me), 0, abort_flag, A.status, kWhereOrthoIn) && lane == 0)
        mbar_wait_timed(there(me), 0, nullptr, kWhereOrthoDrain);  // what is on its way lands
    }
    tc_fence_after_sync();
    const float f = A.rest != nullptr ? A.rest[mat] : 1.f;
    for (int x = 0; x < blocks; ++x) {
      const int c = column(x), c0 = t.j * kN + c;
      const uint32_t block = ring + x * S::kTurn;
      if (r0 >= A.m || c0 >= cols || (kMode != kUpdate && c0 < r0)) continue;
      uint32_t acc[32];
      tmem_ld_32x32b<32>(tmem + c + (static_cast<uint32_t>(32 * quarter) << 16), acc);
      tmem_ld_wait();
      tmem_ld_fence_regs(acc);
      float v[32];
      combine<kMode>(v, acc, block, lane, f, A.in_low);
      emit<kMode>(O, A, v, block, r0, c0, mat, lane);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  let_next();
  tc_fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kN);
  if (warp >= kFirstEpilogue && failed<kMode>(A, *abort_flag))
    for (int x = 0; x < blocks; ++x) spoil(A, mat, r0 + lane, t.j * kN + column(x), 32);
}

// A stack of matrices [n][rows][pitch] as TMA sees it: boxes of `depth` rows of 64 columns for the products' operands
// (128-byte swizzle), of 32 x 32 for the epilogue (64-byte swizzle).
constexpr int kEpilogueBox = 0;
// Lower parts that are bytes: boxes of 32 x 32 (32-byte swizzle).
bool map_bytes(CUtensorMap* map, const void* p, int64_t n, int rows, int cols, int pitch) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
  const uint64_t strides[2] = {static_cast<uint64_t>(pitch), static_cast<uint64_t>(pitch) * rows};
  const uint32_t box[3] = {32, 32, 1};
  return make_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B);
}
bool map_matrix(CUtensorMap* map, const void* p, int64_t n, int rows, int cols, int pitch, int depth,
                CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
  const uint64_t strides[2] = {static_cast<uint64_t>(pitch) * 2, static_cast<uint64_t>(pitch) * 2 * rows};
  const bool small = depth == kEpilogueBox;
  const uint32_t box[3] = {small ? 32u : 64u, small ? 32u : static_cast<uint32_t>(depth), 1};
  return make_tensor_map(map, type, p, 3, dims, strides, box, small ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kMode, int kN, bool kLow, bool kPair>
cudaError_t product(const Operands& o, ProductArgs a, int64_t n, cudaStream_t s) {
  using S = Shape<kMode, kN, kLow, kPair>;
  constexpr int kBlocks = kPair ? 2 : 1;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = ortho_product_kernel<kMode, kN, kLow, kPair>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, ready);
  if (e != cudaSuccess) return e;
  a.tiles_m = (a.m + S::kTileRows - 1) / S::kTileRows;
  a.tiles_n = ((kMode == kUpdate ? a.k : a.m) + kN - 1) / kN;
  a.tiles = 0;
  for (int i = 0; i < a.tiles_m; ++i) a.tiles += a.tiles_n - (kMode == kUpdate ? 0 : i * S::kTileRows / kN);
  a.items = static_cast<int>(n * a.tiles);
  const int most = 152 / kBlocks;
  return launch_cluster(kernel, (a.items < most ? a.items : most) * kBlocks, kBlocks, kProductThreads, S::kSmem, true, s, o, a);
}

// The tiles of 128 x kN of n matrices.
template <int kMode, int kN>
ProductArgs small_tiles(ProductArgs a, int64_t n) {
  a.tiles_m = (a.m + kRows - 1) / kRows;
  a.tiles_n = ((kMode == kUpdate ? a.k : a.m) + kN - 1) / kN;
  a.tiles = 0;
  for (int i = 0; i < a.tiles_m; ++i) a.tiles += a.tiles_n - (kMode == kUpdate ? 0 : i * kRows / kN);
  a.items = static_cast<int>(n * a.tiles);
  return a;
}

template <int kMode, int kN, bool kLow>
cudaError_t narrow_product(const Operands& o, const ProductArgs& a, cudaStream_t s) {
  using S = NarrowShape<kN, kLow>;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = ortho_narrow_kernel<kMode, kN, kLow>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, ready);
  return e != cudaSuccess ? e : launch_next(kernel, static_cast<unsigned>(a.items), kProductThreads, S::kSmem, s, o, a);
}

// One product: by pairs of SMs (tiles of 256 x 256); where there are few tiles, by a block to each of the narrowest
// that do not exceed the SMs; else by persistent blocks.  X's lower part, if it has one, enters P X where m is below 512.
constexpr int kOnePart = 512;
template <int kMode>
cudaError_t run_product(const Operands& o, const ProductArgs& a, int64_t n, bool pair, cudaStream_t s) {
  if (pair) return product<kMode, 256, false, true>(o, a, n, s);
  if constexpr (kMode == kUpdate) {
    const ProductArgs t = small_tiles<kMode, 64>(a, n);
    if (a.m < kOnePart && a.in_low == kHalf) return t.items <= 152 ? narrow_product<kMode, 64, true>(o, t, s) : product<kMode, 128, true, false>(o, a, n, s);
    if (t.items <= 152) return narrow_product<kMode, 64, false>(o, t, s);
  } else {
    ProductArgs t = small_tiles<kMode, 32>(a, n);
    if (t.items <= 152) return narrow_product<kMode, 32, false>(o, t, s);
    t = small_tiles<kMode, 64>(a, n);
    if (t.items <= 152) return narrow_product<kMode, 64, false>(o, t, s);
  }
  const ProductArgs t = small_tiles<kMode, 128>(a, n);
  return t.items <= 152 ? narrow_product<kMode, 128, false>(o, t, s) : product<kMode, 128, false, false>(o, a, n, s);
}

struct Scratch {
  double* part;
  float* rest;
  __half *x[2], *low[2], *gram, *poly;
  size_t bytes;
  int pitch, square;  // of X, of A and P
  int parts;
  Scratch(void* ws, int64_t n, int64_t rows, int64_t cols) {
    const int64_t m = rows < cols ? rows : cols, k = rows < cols ? cols : rows;
    pitch = static_cast<int>(round_up(k, 8));
    square = static_cast<int>(round_up(m, 8));
    parts = ortho_sum_parts(m * k);
    uint8_t* at = static_cast<uint8_t*>(ws);
    bytes = 0;
    auto take = [&](int64_t size) {
      uint8_t* p = at + bytes;
      bytes += round_up(size, 256);
      return p;
    };
    part = reinterpret_cast<double*>(take(n * parts * 8));
    rest = reinterpret_cast<float*>(take(n * 4));
    for (int i = 0; i < 2; ++i) {
      x[i] = reinterpret_cast<__half*>(take(n * m * pitch * 2));
      low[i] = reinterpret_cast<__half*>(take(n * m * pitch * 2));
    }
    gram = reinterpret_cast<__half*>(take(n * m * square * 2));
    poly = reinterpret_cast<__half*>(take(n * m * square * 2));
  }
};

template <typename E>
cudaError_t load_first(const OrthoArgs& A, const Scratch& w, int m, int k, bool tall, cudaStream_t s) {
  const E* g = static_cast<const E*>(A.g);
  __half* low = sizeof(E) == 2 ? nullptr : w.low[0];
  const cudaError_t e = launch_ortho_sum(A, w.parts, w.part, s);
  if (e != cudaSuccess) return e;
  if (tall) {
    const int tiles_m = (m + kTurn - 1) / kTurn, tiles = tiles_m * ((k + kTurn - 1) / kTurn);
    return launch_next(ortho_load_tall_kernel<E>, static_cast<unsigned>(A.n * tiles), 256, 0, s, g, w.part, w.parts, A.eps,
                       w.x[0], low, w.rest, m, k, w.pitch, tiles_m, tiles);
  }
  const int64_t eights = static_cast<int64_t>(m) * (w.pitch / 8);
  const int blocks = static_cast<int>((eights + 256 * kLoadRun - 1) / (256 * kLoadRun));
  return launch_next(ortho_load_kernel<E>, static_cast<unsigned>(A.n * blocks), 256, 0, s, g, w.part, w.parts, A.eps, w.x[0],
                     low, w.rest, m, k, w.pitch, blocks);
}

}  // namespace

int ortho_sum_parts(int64_t size) {
  const int64_t want = (size + kSumCount - 1) / kSumCount;
  return static_cast<int>(want < kSumParts ? want : kSumParts);
}

cudaError_t launch_ortho_sum(const OrthoArgs& A, int parts, double* part, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(A.n * parts);
  const int64_t size = static_cast<int64_t>(A.rows) * A.cols;
  if (A.bf16)
    ortho_sum_kernel<uint16_t><<<grid, kSumThreads, 0, s>>>(static_cast<const uint16_t*>(A.g), size, parts, part, A.status);
  else
    ortho_sum_kernel<float><<<grid, kSumThreads, 0, s>>>(static_cast<const float*>(A.g), size, parts, part, A.status);
  return cudaGetLastError();
}

size_t ortho_scratch_bytes(int64_t n, int64_t rows, int64_t cols) {
  if (ortho_small(rows, cols)) return 0;
  return ortho_thin(rows, cols) ? ortho_thin_scratch_bytes(n, rows, cols) : Scratch(nullptr, n, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const OrthoArgs& A, cudaStream_t s) {
  if (ortho_small(A.rows, A.cols)) return launch_ortho_small(A, s);
  if (ortho_thin(A.rows, A.cols)) return launch_ortho_thin(A, s);
  const bool tall = A.rows > A.cols;
  const int m = tall ? A.cols : A.rows, k = tall ? A.rows : A.cols;
  const Scratch w(A.ws, A.n, A.rows, A.cols);
  cudaError_t e = A.bf16 ? load_first<uint16_t>(A, w, m, k, tall, s) : load_first<float>(A, w, m, k, tall, s);
  if (e != cudaSuccess) return e;
  // Pairs where there are tiles of 256 x 256 for all of them and few of their rows are empty or short of work: 16 of
  // 1024 x 1024 take 489 us by pairs and 518 without, 8 of 2048 x 2048 1198 and 1590, 24 of 512 x 4096 718 and 766;
  // but 60 of 512 x 512 394 and 355, 60 of 600 x 700 916 and 883.
  const int64_t edge = (m + 255) / 256;
  const bool pair = A.n * edge * (edge + 1) / 2 >= 76 && (m > 768 || (m >= 512 && k >= 4096));
  ProductArgs a{};
  a.status = A.status; a.m = m; a.k = k; a.tall = tall;
  a.direct = A.cols % 8 != 0;
  Operands to_gram[2], to_poly, to_x[2];
  CUtensorMap halves[2], bytes[2], result;  // X's lower part, the result, for the epilogue
  bool made = map_matrix(&to_poly.left, w.gram, A.n, m, m, w.square, kRows) &&
              map_matrix(&to_poly.in, w.gram, A.n, m, m, w.square, kEpilogueBox) &&
              map_matrix(&to_poly.out, w.poly, A.n, m, m, w.square, kEpilogueBox);
  made = made && map_matrix(&to_poly.right, w.gram, A.n, m, m, w.square, kBoxRows);
  to_poly.right_low = to_poly.right;
  to_poly.in_low = to_poly.out_low = to_poly.out;
  for (int i = 0; i < 2; ++i) {
    Operands &g = to_gram[i], &x = to_x[i];
    made = made && map_matrix(&g.left, w.x[i], A.n, m, k, w.pitch, kRows) && map_matrix(&x.left, w.poly, A.n, m, m, w.square, kRows) &&
           map_matrix(&x.right, w.x[i], A.n, m, k, w.pitch, kDepth) && map_matrix(&x.right_low, w.low[i], A.n, m, k, w.pitch, kDepth) &&
           map_matrix(&x.in, w.x[i], A.n, m, k, w.pitch, kEpilogueBox) &&
           map_matrix(&halves[i], w.low[i], A.n, m, k, w.pitch, kEpilogueBox) &&
           map_bytes(&bytes[i], w.low[i], A.n, m, k, static_cast<int>(round_up(k, 16)));
    made = made && map_matrix(&g.right, w.x[i], A.n, m, k, w.pitch, kBoxRows);
    g.right_low = g.right;
    g.out = g.out_low = g.in = g.in_low = to_poly.in;
  }
  for (int i = 0; i < 2; ++i) to_x[i].out = to_x[i ^ 1].in;
  if (!a.direct)
    made = made && map_matrix(&result, A.out, A.n, A.rows, A.cols, A.cols, kEpilogueBox, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
  if (!made) return cudaErrorInvalidValue;
  // The lower part of a step's X, by the steps still to come (its own among them), through which its noise grows: from
  // kOnePart rows on, where it is no operand, nothing serves in the last step and a byte in the three before it.
  auto low_part = [&](int step) {
    const int left = A.steps - step;
    if (step == 0) return A.bf16 ? kNone : kHalf;
    if (left < 1) return kNone;
    return m < kOnePart || left > 4 ? kHalf : left > 1 ? kBytes : kNone;
  };
  const int stall = option_test_stall_tile();
  for (int i = 0; i < A.steps && e == cudaSuccess; ++i) {
    const int at = i & 1;
    const bool last = i == A.steps - 1;
    a.inner = k;
    a.rest = i == 0 && A.bf16 ? w.rest : nullptr;
    a.in_low = low_part(i);
    a.out_low = low_part(i + 1);
    a.skip = stall == 3 * i;
    e = run_product<kGram>(to_gram[at], a, A.n, pair, s);
    if (e != cudaSuccess) break;
    a.inner = m;
    a.skip = stall == 3 * i + 1;
    e = run_product<kPoly>(to_poly, a, A.n, pair, s);
    if (e != cudaSuccess) break;
    a.last = last ? A.out : nullptr;
    Operands x = to_x[at];
    x.in_low = a.in_low == kBytes ? bytes[at] : halves[at];
    x.out_low = a.out_low == kBytes ? bytes[at ^ 1] : halves[at ^ 1];
    if (last && !a.direct) x.out = result;
    a.skip = stall == 3 * i + 2;
    e = run_product<kUpdate>(x, a, A.n, pair, s);
  }
  return e;
}

}  // namespace m2rnn
