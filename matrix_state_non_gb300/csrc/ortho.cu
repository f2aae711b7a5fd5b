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
// of X exceeds 1.2025, of A 1.4461, of P 2.81.  X is kept in two fp16 parts (22
// bits) between steps: small singular values grow 480-fold in five steps, and
// the rounding noise of X in one part would grow with them (for a matrix of
// rank 1 the result would be 0.15 off; it is 3e-4).  Noise of A and P does not
// grow: P X stays in the row space of X.  What they leave is 1.0e-3 to 1.9e-3 of
// the result (1.3e-3 at 1024 x 1024 of random entries), the output's rounding to
// bf16 1.7e-3.  With X's lower part in P X as well (kLow) it is 1.0e-3 to
// 1.5e-3, which matrices too small to fill the GPU get for nothing.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"
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

// The thread's share of a sum of squares over a block's piece.  Squares that
// leave the fp32 range are caught as in grad_clip.cu: next to x^2 it sums
// (x 2^90)^2, for where the first may have lost bits, and a sum that is not
// finite is taken again in fp64.
template <typename E>
__device__ double square_sum(const E* g, int64_t from, int64_t to) {
  float s = 0.f, up = 0.f;
#pragma unroll 8
  for (int64_t i = from + threadIdx.x; i < to; i += kSumThreads) {
    const float x = to_f32(g[i]), y = x * 0x1p90f;
    s = fmaf(x, x, s);
    up = fmaf(y, y, up);
  }
  if (s < 0x1p-60f) return static_cast<double>(up) * 0x1p-180;
  if (s <= 3.4e38f) return s;
  double w = 0.;
  for (int64_t i = from + threadIdx.x; i < to; i += kSumThreads) {
    const double x = to_f32(g[i]);
    w += x * x;
  }
  return w;
}

template <typename E>
__global__ void __launch_bounds__(kSumThreads) ortho_sum_kernel(const E* g, int64_t size, int parts, double* part) {
  __shared__ double red[kSumThreads / 32];
  const int64_t mat = blockIdx.x / parts;
  const int p = static_cast<int>(blockIdx.x - mat * parts);
  const int64_t per = (size + parts - 1) / parts;
  double acc = square_sum(g + mat * size, p * per, min(size, (p + 1) * per));
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

__device__ __forceinline__ void split_half(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// X [m][pitch] in two parts from G [rows][cols], a tile of 32 x 64 of X at a
// time; tall: G is [k][m] and goes through shared memory.
constexpr int kLoadRows = 32, kLoadCols = 64;
template <typename E>
__global__ void __launch_bounds__(256) ortho_load_kernel(const E* g, const double* part, int parts, float eps, __half* hi,
                                                         __half* lo, int m, int k, int pitch, bool tall, int tiles_m,
                                                         int tiles_k) {
  __shared__ float t[kLoadRows][kLoadCols + 1];
  __shared__ float factor;
  wait_previous();
  const int64_t tiles = static_cast<int64_t>(tiles_m) * tiles_k, mat = blockIdx.x / tiles;
  const int tile = static_cast<int>(blockIdx.x - mat * tiles);
  const int r0 = tile / tiles_k * kLoadRows, c0 = tile % tiles_k * kLoadCols;
  if (threadIdx.x < 32) {
    double acc = 0.;
    for (int i = threadIdx.x; i < parts; i += 32) acc += part[mat * parts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (threadIdx.x == 0) factor = static_cast<float>(1. / (sqrt(acc) + eps));
  }
  const E* p = g + mat * m * k;
  if (tall) {
    for (int i = threadIdx.x; i < kLoadRows * kLoadCols; i += 256) {
      const int r = i % kLoadRows, c = i / kLoadRows;
      t[r][c] = r0 + r < m && c0 + c < k ? to_f32(p[static_cast<int64_t>(c0 + c) * m + r0 + r]) : 0.f;
    }
  } else {
    for (int i = threadIdx.x; i < kLoadRows * kLoadCols; i += 256) {
      const int r = i / kLoadCols, c = i % kLoadCols;
      t[r][c] = r0 + r < m && c0 + c < k ? to_f32(p[static_cast<int64_t>(r0 + r) * k + c0 + c]) : 0.f;
    }
  }
  __syncthreads();
  let_next();
  for (int i = threadIdx.x; i < kLoadRows * kLoadCols / 2; i += 256) {
    const int r = i / (kLoadCols / 2), c = i % (kLoadCols / 2) * 2;
    if (r0 + r >= m || c0 + c >= pitch) continue;
    __half2 h, l;
    split_half(t[r][c] * factor * kScaleX, h.x, l.x);
    split_half(t[r][c + 1] * factor * kScaleX, h.y, l.y);
    const int64_t at = (mat * m + r0 + r) * pitch + c0 + c;
    *reinterpret_cast<__half2*>(hi + at) = h;
    *reinterpret_cast<__half2*>(lo + at) = l;
  }
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
enum { kGram = 0, kPoly = 1, kUpdate = 2 };

struct ProductArgs {
  const __half* in;      // kPoly: A; kUpdate: X's upper part
  const __half* in_low;  // kUpdate: X's lower part
  __half* out;           // A; P; X'
  __half* out_low;       // kUpdate
  uint16_t* last;        // kUpdate of the last step: the result in bf16, [m][k] or (tall) [k][m]
  StatusBlock* status;
  int m, k;              // X is m x k
  int pitch;             // of in, out
  int inner;             // of the product
  int tiles_m, tiles_n, tiles;  // of one matrix; those that are computed
  int64_t items;
  bool tall;
};

constexpr int kRows = 128, kDepth = 64;  // a tile's rows, the inner dimension of a stage
constexpr int kEpilogueWarps = 8, kFirstEpilogue = 2, kProductThreads = 32 * (kFirstEpilogue + kEpilogueWarps);

template <int kMode, int kN, bool kLow>
struct Shape {
  static constexpr int kLeft = kRows * kDepth * 2, kRight = kN * kDepth * 2;
  static constexpr int kStage = kLeft + kRight * (kLow ? 2 : 1);
  static constexpr int kStages = 196608 / kStage;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kSmem = kOffBar + 256 + 1024;  // 1024: alignment
};

struct Item {
  int64_t mat;
  int i, j;  // tile's row and column
};
// Symmetric products: of row i the tiles with a column at or right of the diagonal.
template <int kMode, int kN>
__device__ __forceinline__ Item item_at(const ProductArgs& A, int64_t id) {
  Item t;
  t.mat = id / A.tiles;
  int left = static_cast<int>(id - t.mat * A.tiles);
  if constexpr (kMode == kUpdate) {
    t.i = left % A.tiles_m;  // neighbours share the columns of X
    t.j = left / A.tiles_m;
  } else {
    t.i = 0;
    int first = 0;
    while (left >= A.tiles_n - first) {
      left -= A.tiles_n - first;
      ++t.i;
      first = t.i * kRows / kN;
    }
    t.j = first + left;
  }
  return t;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

union Eight {
  uint4 v;
  __half2 h[4];
};

template <int kMode, int kN, bool kLow>
__global__ void __launch_bounds__(kProductThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap left, const __grid_constant__ CUtensorMap right,
                         const __grid_constant__ CUtensorMap right_low, ProductArgs A) {
  using S = Shape<kMode, kN, kLow>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_u32(smem), bars = base + S::kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };         // [stages] TMA -> products
  auto empty = [&](int s) { return bars + 64 + 8 * s; };   // [stages] products -> TMA
  auto done = [&](int s) { return bars + 128 + 8 * s; };   // [2] products -> epilogue
  auto tfree = [&](int s) { return bars + 144 + 8 * s; };  // [2] epilogue -> products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffBar + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffBar + 164);
  static_assert(S::kStages <= 8, "barriers");
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(done(s), 1);
      mbar_init(tfree(s), 32 * kEpilogueWarps);
    }
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_previous();
  const int depth = (A.inner + kDepth - 1) / kDepth;

  if (warp == 0) {
    // ---------------- loads ----------------
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");  // what earlier launches stored, before TMA reads it
      int u = 0;  // stages filled
      bool ok = true;
      for (int64_t id = blockIdx.x; ok && id < A.items; id += gridDim.x) {
        const Item t = item_at<kMode, kN>(A, id);
        const int mat = static_cast<int>(t.mat);
        for (int d = 0; d < depth; ++d, ++u) {
          const int s = u % S::kStages;
          if (u >= S::kStages && !mbar_wait(empty(s), (u / S::kStages - 1) & 1, abort_flag, A.status, kWhereOrthoEmpty)) {
            ok = false;
            break;
          }
          const uint32_t to = base + s * S::kStage, bar = full(s);
          mbar_arrive_expect_tx(bar, S::kStage);
          tma_load_3d(to, &left, bar, d * kDepth, t.i * kRows, mat);
          if constexpr (kMode == kUpdate) {  // 64 columns of 64 rows at a time
#pragma unroll
            for (int c = 0; c < kN; c += 64) {
              tma_load_3d(to + S::kLeft + c * kDepth * 2, &right, bar, t.j * kN + c, d * kDepth, mat);
              if (kLow) tma_load_3d(to + S::kLeft + S::kRight + c * kDepth * 2, &right_low, bar, t.j * kN + c, d * kDepth, mat);
            }
          } else {
#pragma unroll
            for (int r = 0; r < kN; r += kRows)
              tma_load_3d(to + S::kLeft + r * kDepth * 2, &right, bar, d * kDepth, t.j * kN + r, mat);
          }
        }
      }
      if (!ok)  // the copies in flight land before the block ends
        for (int x = max(0, u - S::kStages); x < u; ++x)
          mbar_wait_timed(full(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    constexpr uint32_t kId = idesc_f16_f32(kRows, kN, false, kMode == kUpdate);
    int u = 0, n = 0;  // stages, tiles
    bool ok = true;
    for (int64_t id = blockIdx.x; ok && id < A.items; id += gridDim.x, ++n) {
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
              tc_mma_f16_ss(tm, desc_sw128(l + kk * 32), desc_sw128(r + kk * 2048, kDepth * 128), kId, d > 0 || kk > 0);
              if (kLow)
                tc_mma_f16_ss(tm, desc_sw128(l + kk * 32), desc_sw128(r + S::kRight + kk * 2048, kDepth * 128), kId, 1);
            } else {
              tc_mma_f16_ss(tm, desc_sw128(l + kk * 32), desc_sw128(r + kk * 32), kId, d > 0 || kk > 0);
            }
          }
          tc_commit(empty(s));
          if (d == depth - 1) tc_commit(done(slot));
        }
        __syncwarp();
      }
    }
    if (*abort_flag)  // the products in flight end before their memory is freed
      for (int x = max(0, u - S::kStages); x < u; ++x)
        mbar_wait_timed(empty(x % S::kStages), (x / S::kStages) & 1, nullptr, kWhereOrthoDrain);
  } else {
    // ---------------- epilogue: a thread has a row, its warp 32 columns at a time ----------------
    const int quarter = warp & 3, half = (warp - kFirstEpilogue) >> 2;
    int n = 0;
    for (int64_t id = blockIdx.x; id < A.items; id += gridDim.x, ++n) {
      const Item t = item_at<kMode, kN>(A, id);
      const int slot = n & 1;
      if (!warp_wait(done(slot), (n >> 1) & 1, abort_flag, A.status, kWhereOrthoDone)) break;
      tc_fence_after_sync();
      const int r0 = t.i * kRows + quarter * 32, r = r0 + lane;
      const uint32_t tm = tmem + slot * kN + (static_cast<uint32_t>(32 * quarter) << 16);
      const int cols = kMode == kUpdate ? A.k : A.m;
      const int64_t row = (t.mat * A.m + r) * A.pitch, turned = t.mat * A.m * static_cast<int64_t>(A.pitch);
#pragma unroll 1
      for (int x = half * (kN / 2); x < (half + 1) * (kN / 2); x += 32) {
        const int c0 = t.j * kN + x;
        if (r0 >= A.m || c0 >= cols || (kMode != kUpdate && c0 < r0)) continue;
        Eight up[4], low[4];
        if constexpr (kMode != kGram) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            up[q].v = low[q].v = make_uint4(0u, 0u, 0u, 0u);
            if (r < A.m && c0 + 8 * q < A.pitch) {
              up[q].v = *reinterpret_cast<const uint4*>(A.in + row + c0 + 8 * q);
              if (kMode == kUpdate) low[q].v = *reinterpret_cast<const uint4*>(A.in_low + row + c0 + 8 * q);
            }
          }
        }
        uint32_t acc[32];
        tmem_ld_32x32b<32>(tm + x, acc);
        tmem_ld_wait();
        tmem_ld_fence_regs(acc);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p = __uint_as_float(acc[e]);
          const __half2 u2 = up[e / 8].h[e % 8 / 2], l2 = low[e / 8].h[e % 8 / 2];
          const float u1 = __half2float(e % 2 == 0 ? u2.x : u2.y), l1 = __half2float(e % 2 == 0 ? l2.x : l2.y);
          if constexpr (kMode == kGram) v[e] = p * 0x1p-14f;
          if constexpr (kMode == kPoly) v[e] = fmaf(kC * 0x1p-15f, p, kB * 0.5f * u1);
          if constexpr (kMode == kUpdate) v[e] = fmaf(p, 0x1p-13f, kA * (u1 + l1));
        }
        if (kMode == kUpdate && A.last != nullptr) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= 1.f / kScaleX;
          if (A.tall) {
            uint16_t* to = A.last + (t.mat * A.k + c0) * A.m + r;
#pragma unroll
            for (int e = 0; e < 32; ++e, to += A.m)
              if (r < A.m && c0 + e < A.k) *to = from_f32<uint16_t>(v[e]);
          } else if (r < A.m) {
            uint16_t* to = A.last + (t.mat * A.m + r) * A.k + c0;
            if (A.k % 8 == 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (c0 + 8 * q < A.k)
                  *reinterpret_cast<uint4*>(to + 8 * q) =
                      make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                 pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c0 + e < A.k) to[e] = from_f32<uint16_t>(v[e]);
            }
          }
          continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = v[8 * q + 2 * e], b = v[8 * q + 2 * e + 1];
            up[q].h[e] = __floats2half2_rn(a, b);
            if constexpr (kMode == kUpdate)
              low[q].h[e] = __floats2half2_rn(a - __half2float(up[q].h[e].x), b - __half2float(up[q].h[e].y));
          }
          if (r < A.m && c0 + 8 * q < A.pitch) {
            *reinterpret_cast<uint4*>(A.out + row + c0 + 8 * q) = up[q].v;
            if (kMode == kUpdate) *reinterpret_cast<uint4*>(A.out_low + row + c0 + 8 * q) = low[q].v;
          }
        }
        if (kMode != kUpdate && c0 != r0 && r < A.m) {  // the other side of the diagonal (whose 32 x 32 blocks are whole)
          __half* to = A.out + turned + static_cast<int64_t>(c0) * A.pitch + r;
#pragma unroll
          for (int e = 0; e < 32; ++e, to += A.pitch)
            if (c0 + e < A.m) *to = e % 2 == 0 ? up[e / 8].h[e % 8 / 2].x : up[e / 8].h[e % 8 / 2].y;
        }
      }
      tc_fence_before_sync();
      mbar_arrive(tfree(slot));
    }
  }
  let_next();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Rows of a stack of matrices [n][rows][pitch], boxes of `depth` rows of 64 columns.
bool map_matrix(CUtensorMap* map, const __half* p, int64_t n, int rows, int cols, int pitch, int depth) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
  const uint64_t strides[2] = {static_cast<uint64_t>(pitch) * 2, static_cast<uint64_t>(pitch) * 2 * rows};
  const uint32_t box[3] = {64, static_cast<uint32_t>(depth), 1};
  return make_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, 3, dims, strides, box, true);
}

template <int kMode, int kN, bool kLow>
cudaError_t product(const CUtensorMap& l, const CUtensorMap& r, const CUtensorMap& low, ProductArgs a, int64_t n,
                    cudaStream_t s) {
  using S = Shape<kMode, kN, kLow>;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = ortho_product_kernel<kMode, kN, kLow>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, ready);
  if (e != cudaSuccess) return e;
  a.tiles_m = (a.m + kRows - 1) / kRows;
  a.tiles_n = ((kMode == kUpdate ? a.k : a.m) + kN - 1) / kN;
  a.tiles = 0;
  for (int i = 0; i < a.tiles_m; ++i) a.tiles += a.tiles_n - (kMode == kUpdate ? 0 : i * kRows / kN);
  a.items = n * a.tiles;
  return launch_next(kernel, static_cast<unsigned>(a.items < 152 ? a.items : 152), kProductThreads, S::kSmem, s, l, r, low, a);
}

struct Scratch {
  double* part;
  __half *x[2], *low[2], *gram, *poly;
  size_t bytes;
  int pitch, square;  // of X, of A and P
  int parts;
  Scratch(void* ws, int64_t n, int64_t rows, int64_t cols) {
    const int64_t m = rows < cols ? rows : cols, k = rows < cols ? cols : rows;
    pitch = static_cast<int>(round_up(k, 8));
    square = static_cast<int>(round_up(m, 8));
    const int64_t want = (m * k + kSumCount - 1) / kSumCount;
    parts = static_cast<int>(want < kSumParts ? want : kSumParts);
    uint8_t* at = static_cast<uint8_t*>(ws);
    bytes = 0;
    auto take = [&](int64_t size) {
      uint8_t* p = at + bytes;
      bytes += round_up(size, 256);
      return p;
    };
    part = reinterpret_cast<double*>(take(n * parts * 8));
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
  const int tiles_m = (m + kLoadRows - 1) / kLoadRows, tiles_k = (k + kLoadCols - 1) / kLoadCols;
  ortho_sum_kernel<E><<<static_cast<unsigned>(A.n * w.parts), kSumThreads, 0, s>>>(g, static_cast<int64_t>(m) * k, w.parts,
                                                                                   w.part);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(ortho_load_kernel<E>, static_cast<unsigned>(A.n * tiles_m * tiles_k), 256, 0, s, g, w.part, w.parts, A.eps,
                     w.x[0], w.low[0], m, k, w.pitch, tall, tiles_m, tiles_k);
}

}  // namespace

size_t ortho_scratch_bytes(int64_t n, int64_t rows, int64_t cols) { return Scratch(nullptr, n, rows, cols).bytes; }

cudaError_t launch_orthogonalize(const OrthoArgs& A, cudaStream_t s) {
  const bool tall = A.rows > A.cols;
  const int m = tall ? A.cols : A.rows, k = tall ? A.rows : A.cols;
  const Scratch w(A.ws, A.n, A.rows, A.cols);
  cudaError_t e = A.bf16 ? load_first<uint16_t>(A, w, m, k, tall, s) : load_first<float>(A, w, m, k, tall, s);
  CUtensorMap rows[2], cols[2], cols_low[2], gram, poly;
  for (int i = 0; i < 2; ++i)
    if (!map_matrix(&rows[i], w.x[i], A.n, m, k, w.pitch, kRows) || !map_matrix(&cols[i], w.x[i], A.n, m, k, w.pitch, kDepth) ||
        !map_matrix(&cols_low[i], w.low[i], A.n, m, k, w.pitch, kDepth))
      return cudaErrorInvalidValue;
  if (!map_matrix(&gram, w.gram, A.n, m, m, w.square, kRows) || !map_matrix(&poly, w.poly, A.n, m, m, w.square, kRows))
    return cudaErrorInvalidValue;
  ProductArgs a{};
  a.status = A.status; a.m = m; a.k = k; a.tall = tall;
  for (int i = 0; i < A.steps && e == cudaSuccess; ++i) {
    const int from = i & 1, to = from ^ 1;
    a.in = nullptr; a.out = w.gram; a.pitch = w.square; a.inner = k;
    e = product<kGram, 128, false>(rows[from], rows[from], rows[from], a, A.n, s);
    if (e != cudaSuccess) break;
    a.in = w.gram; a.out = w.poly; a.inner = m;
    e = product<kPoly, 128, false>(gram, gram, gram, a, A.n, s);
    if (e != cudaSuccess) break;
    a.in = w.x[from]; a.in_low = w.low[from]; a.out = w.x[to]; a.out_low = w.low[to]; a.pitch = w.pitch;
    a.last = i == A.steps - 1 ? A.out : nullptr;
    e = m < 512 ? product<kUpdate, 128, true>(poly, cols[from], cols_low[from], a, A.n, s)
                : product<kUpdate, 256, false>(poly, cols[from], cols_low[from], a, A.n, s);
  }
  return e;
}

}  // namespace m2rnn
