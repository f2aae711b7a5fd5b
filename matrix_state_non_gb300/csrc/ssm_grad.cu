// Backward of the selective state space scan on tensor cores (bf16 inputs; the
// mathematics in ssm.cu), in chunks of 64 steps, every chunk on its own:
//   1. decays of every chunk;
//   2. every chunk's sums sum_j last_j D_j k_j v_j^T and sum_i first_i q_i u_i^T;
//   3. a scan over the chunks turns them into the state S before each chunk and
//      the state gradient R behind it;
//   4. the chunk's gradients from q, k, v, u = dy, S and R;
//   5. sums over the chunks (dA, ddt_bias, dw_r) and over the heads that share
//      q and k.
// The gradients are fp32 and good to that: q, k, v and u are exact bf16
// operands, and whatever else enters a product (S, R, the decayed scores, the
// weighted rows) is split into three bf16 parts, whose products are summed
// from the smallest part up.
#include <cuda_runtime.h>

#include <cstdint>

#include "ssm_mma.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;  // four warps, 16 of the chunk's steps each

struct GradArgs {
  SsmArgs a;
  SsmGradOut o;
  const ChunkDecayGrad* decay;  // [B N][chunks]
  const float* tot;             // [B N][chunks]
  float* sums[2];               // [B N][chunks][K][V]: of S, of R
  uint16_t* planes[2];          // [B N][chunks][3][K][V]: S, R in three bf16 parts
  int nc;
  bool vq, vk, vv, vu;          // rows that asynchronous copies can take
};

template <int KP, int VS>
struct SumShape {
  static constexpr int kMw = KP >= 64 ? 4 : KP / 16, kNw = 4 / kMw;
  static constexpr int kMt = KP / 16 / kMw, kNt = VS / 8 / kNw;
  static_assert(kNt % 2 == 0, "value tiles are loaded in pairs");
  static constexpr int kK = Tile<KP>::kBytes(kChunk), kV = Tile<VS>::kBytes(kChunk), kBytes = kK + kV + kChunk * 4;
};

// Phase 2: block (S or R, value slice, chain, chunk); rows of the sum along K.
template <int KP, int VS>
__global__ void __launch_bounds__(kThreads) ssm_grad_sum_kernel(GradArgs W, int slices) {
  using Sh = SumShape<KP, VS>;
  extern __shared__ __align__(16) uint8_t smem[];
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int mw = warp % Sh::kMw, nw = warp / Sh::kMw;
  const bool rev = blockIdx.y >= static_cast<unsigned>(slices);
  const int v0 = (blockIdx.y - (rev ? slices : 0)) * VS, bn = blockIdx.x / W.nc, c = blockIdx.x - bn * W.nc;
  const int b = bn / A.N, n = bn - b * A.N, gq = n / (A.N / A.G), K = A.K, V = A.V, len = ssm_len(A, b), t0 = c * kChunk;
  const int width = min(VS, V - v0);
  const int64_t row = static_cast<int64_t>(b) * A.T;
  const uint32_t sK = smem_u32(smem), sV = sK + Sh::kK;
  const float* w = reinterpret_cast<const float*>(smem + Sh::kK + Sh::kV);
  const ChunkDecayGrad* d = W.decay + blockIdx.x;
  const TileLoader<KP, kThreads> lk =
      rev ? TileLoader<KP, kThreads>{static_cast<const uint16_t*>(A.q) + row * A.q_stride + static_cast<int64_t>(gq) * K,
                                     A.q_stride, K, W.vq}
          : TileLoader<KP, kThreads>{static_cast<const uint16_t*>(A.k) + row * A.k_stride + static_cast<int64_t>(gq) * K,
                                     A.k_stride, K, W.vk};
  const TileLoader<VS, kThreads> lv =
      rev ? TileLoader<VS, kThreads>{static_cast<const uint16_t*>(A.dy) + (row * A.N + n) * V + v0,
                                     static_cast<int64_t>(A.N) * V, width, W.vu}
          : TileLoader<VS, kThreads>{static_cast<const uint16_t*>(A.v) + row * A.v_stride + static_cast<int64_t>(n) * V + v0,
                                     A.v_stride, width, W.vv};
  if (tid < kChunk / 4) cp_async_16(sV + Sh::kV + tid * 16, (rev ? d->d.first : d->d.wD) + tid * 4, true);
  lk.load(sK, t0, len);
  lv.load(sV, t0, len);
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();
  // The small parts on their own: four adds, not twelve, at the sum's full size are truncated.
  float U[Sh::kMt][Sh::kNt][4] = {}, low[Sh::kMt][Sh::kNt][4] = {};
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    constexpr int kPairs = Sh::kNt / 2;
    uint32_t vf[kPairs][4];
#pragma unroll
    for (int np = 0; np < kPairs; ++np)
      ldmatrix_x4_trans(vf[np], at_rows<VS>(sV, 16 * jt, nw * Sh::kNt * 8 + 16 * np, lane));
    const int j = 16 * jt + 2 * q4;
    const float2 wa = *reinterpret_cast<const float2*>(&w[j]), wb = *reinterpret_cast<const float2*>(&w[j + 8]);
#pragma unroll
    for (int mt = 0; mt < Sh::kMt; ++mt) {
      uint32_t kf[4], p[3][4];
      ldmatrix_x4_trans(kf, at_cols<KP>(sK, 16 * jt, (mw * Sh::kMt + mt) * 16, lane));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float2 x = r < 2 ? wa : wb;
        split3_weighted(kf[r], x.x, x.y, p[2][r], p[1][r], p[0][r]);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int nt = 0; nt < Sh::kNt; ++nt)
          mma_bf16_16816(i < 2 ? low[mt][nt] : U[mt][nt], p[i], vf[nt / 2][2 * (nt & 1)], vf[nt / 2][2 * (nt & 1) + 1]);
    }
  }
  float* out = W.sums[rev] + static_cast<int64_t>(blockIdx.x) * K * V + v0;
#pragma unroll
  for (int mt = 0; mt < Sh::kMt; ++mt)
#pragma unroll
    for (int nt = 0; nt < Sh::kNt; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (mw * Sh::kMt + mt) * 16 + g + 8 * h, col = (nw * Sh::kNt + nt) * 8 + 2 * q4;
        if (r >= K || col >= width) continue;
        float* at = out + r * V + col;
        const float x = U[mt][nt][2 * h] + low[mt][nt][2 * h], y = U[mt][nt][2 * h + 1] + low[mt][nt][2 * h + 1];
        if (V % 2 == 0) {
          *reinterpret_cast<float2*>(at) = make_float2(x, y);
        } else {
          at[0] = x;
          if (col + 1 < width) at[1] = y;
        }
      }
}

// Phase 3: block (chain, 256 kVec elements of a state, S or R).
template <int kVec>
__global__ void __launch_bounds__(256) ssm_grad_scan_kernel(GradArgs W) {
  constexpr int kAhead = 4;
  const SsmArgs& A = W.a;
  const int KV = A.K * A.V, e = (blockIdx.y * 256 + threadIdx.x) * kVec;
  const bool rev = blockIdx.z == 1;
  const int64_t bn = blockIdx.x;
  if (e >= KV) return;
  const float* sums = W.sums[rev] + bn * W.nc * KV + e;
  uint16_t* planes = W.planes[rev] + bn * W.nc * 3 * KV + e;
  const float* tot = W.tot + bn * W.nc;
  const float* from = rev ? A.dH_T : A.H_0;
  float s[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) s[i] = from ? from[bn * KV + e + i] : 0.f;
  for (int i0 = 0; i0 < W.nc; i0 += kAhead) {
    float u[kAhead][kVec], a[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= W.nc) continue;
      const int c = rev ? W.nc - 1 - i0 - j : i0 + j;
      if constexpr (kVec == 4)
        *reinterpret_cast<float4*>(u[j]) = *reinterpret_cast<const float4*>(sums + static_cast<int64_t>(c) * KV);
      else
        u[j][0] = sums[static_cast<int64_t>(c) * KV];
      a[j] = tot[c];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= W.nc) continue;
      const int c = rev ? W.nc - 1 - i0 - j : i0 + j;
      uint16_t* out = planes + static_cast<int64_t>(c) * 3 * KV;
      if constexpr (kVec == 4) {
        uint32_t p[3][2];
        split3(s[0], s[1], p[0][0], p[1][0], p[2][0]);
        split3(s[2], s[3], p[0][1], p[1][1], p[2][1]);
#pragma unroll
        for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2*>(out + x * KV) = make_uint2(p[x][0], p[x][1]);
      } else {
        uint32_t p[3];
        split3(s[0], 0.f, p[0], p[1], p[2]);
#pragma unroll
        for (int x = 0; x < 3; ++x) out[x * KV] = static_cast<uint16_t>(p[x]);
      }
#pragma unroll
      for (int x = 0; x < kVec; ++x) s[x] = fmaf(a[j], s[x], u[j][x]);
    }
  }
  if (rev && A.dH_0 != nullptr) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) A.dH_0[bn * KV + e + i] = s[i];
  }
}

template <int KP, int VP>
struct GradShape {
  static constexpr int kQ = Tile<KP>::kBytes(kChunk), kV = Tile<VP>::kBytes(kChunk), kP = Tile<VP>::kBytes(KP);
  static constexpr int kTiles = 2 * kQ + 2 * kV + 3 * kP;
  static constexpr int kBytes = kTiles + static_cast<int>(sizeof(ChunkDecayGrad));
  static constexpr int kBlocks = kBytes > 115000 ? 1 : kBytes > 76000 || KP * VP > 4096 ? 2 : 3;
};

// A 16 x 16 block of scores times their factors, as three A operands.
__device__ __forceinline__ void split_scores(const float (&s)[2][4], uint32_t (&p)[3][4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    split3(s[h][0], s[h][1], p[2][2 * h], p[1][2 * h], p[0][2 * h]);
    split3(s[h][2], s[h][3], p[2][2 * h + 1], p[1][2 * h + 1], p[0][2 * h + 1]);
  }
}

// x += P f, P in three parts: the products are summed on their own, from the
// smallest part up, and added in fp32.  The tensor core truncates its adds;
// on the running sum itself that is a bias which dA and ddt_bias, differences
// of sums over all steps, cannot take.
__device__ __forceinline__ void add_split(float (&x)[4], const uint32_t (&p)[3][4], uint32_t f0, uint32_t f1) {
  float t[4];
  mma_bf16_16816_zc(t, p[0], f0, f1);
  mma_bf16_16816(t, p[1], f0, f1);
  mma_bf16_16816(t, p[2], f0, f1);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] += t[e];
}

// Phase 4: block (chain, chunk).  K padded to KP, V to VP.
template <int KP, int VP>
__global__ void __launch_bounds__(kThreads, GradShape<KP, VP>::kBlocks) ssm_grad_kernel(GradArgs W) {
  using Sh = GradShape<KP, VP>;
  constexpr int kKt = KP / 16, kVt = VP / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float qd[kChunk], ck[kChunk], ci[kChunk], red[4];
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int bn = blockIdx.x / W.nc, c = blockIdx.x - bn * W.nc, b = bn / A.N, n = bn - b * A.N, gq = n / (A.N / A.G);
  const int K = A.K, V = A.V, len = ssm_len(A, b), t0 = c * kChunk, rows = min(kChunk, A.T - t0);
  const int64_t row = static_cast<int64_t>(b) * A.T + t0, KV = static_cast<int64_t>(K) * V;
  const int64_t qk_stride = static_cast<int64_t>(W.o.qk_heads) * K, v_stride = static_cast<int64_t>(A.N) * V;
  float* dq = W.o.dq + row * qk_stride + static_cast<int64_t>(W.o.qk_heads == A.N ? n : gq) * K;
  float* dk = W.o.dk + row * qk_stride + static_cast<int64_t>(W.o.qk_heads == A.N ? n : gq) * K;
  float* dv = A.dv + row * v_stride + static_cast<int64_t>(n) * V;
  float* ddt = A.ddt + row * A.N + n;
  float* wr_part = W.o.wr_part ? W.o.wr_part + static_cast<int64_t>(blockIdx.x) * V : nullptr;
  if (t0 >= len) {  // behind the sequence's end
    for (int e = tid; e < rows * K; e += kThreads) {
      dq[(e / K) * qk_stride + e % K] = 0.f;
      dk[(e / K) * qk_stride + e % K] = 0.f;
    }
    for (int e = tid; e < rows * V; e += kThreads) dv[(e / V) * v_stride + e % V] = 0.f;
    for (int e = tid; e < rows; e += kThreads) ddt[static_cast<int64_t>(e) * A.N] = 0.f;
    if (wr_part)
      for (int e = tid; e < V; e += kThreads) wr_part[e] = 0.f;
    if (tid == 0) W.o.ab_part[blockIdx.x] = make_float2(0.f, 0.f);
    return;
  }
  const uint32_t sQ = smem_u32(smem), sK = sQ + Sh::kQ, sV = sK + Sh::kQ, sU = sV + Sh::kV, sP = sU + Sh::kV;
  const ChunkDecayGrad& dg = *reinterpret_cast<const ChunkDecayGrad*>(smem + Sh::kTiles);
  const ChunkDecay& d = dg.d;
  {
    const int64_t r0 = static_cast<int64_t>(b) * A.T;
    const TileLoader<KP, kThreads> lq{static_cast<const uint16_t*>(A.q) + r0 * A.q_stride + static_cast<int64_t>(gq) * K,
                                      A.q_stride, K, W.vq};
    const TileLoader<KP, kThreads> lk{static_cast<const uint16_t*>(A.k) + r0 * A.k_stride + static_cast<int64_t>(gq) * K,
                                      A.k_stride, K, W.vk};
    const TileLoader<VP, kThreads> lv{static_cast<const uint16_t*>(A.v) + r0 * A.v_stride + static_cast<int64_t>(n) * V,
                                      A.v_stride, V, W.vv};
    const TileLoader<VP, kThreads> lu{static_cast<const uint16_t*>(A.dy) + (r0 * A.N + n) * V, v_stride, V, W.vu};
    lu.load(sU, t0, len);
    lv.load(sV, t0, len);
    lk.load(sK, t0, len);
    lq.load(sQ, t0, len);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(W.decay + blockIdx.x);
    for (int e = tid; e < static_cast<int>(sizeof(ChunkDecayGrad)) / 16; e += kThreads)
      cp_async_16(sP + 3 * Sh::kP + e * 16, src + e * 16, true);
  }
  const uint16_t* gS = W.planes[0] + static_cast<int64_t>(blockIdx.x) * 3 * KV;
  const uint16_t* gR = W.planes[1] + static_cast<int64_t>(blockIdx.x) * 3 * KV;
  // Element pieces of the planes: 8 columns of a row, or single elements where rows are not whole pieces.
  const bool vec = V % 8 == 0;
  auto load_planes = [&](const uint16_t* src) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      if (vec) {
#pragma unroll 4
        for (int e = tid; e < KP * (VP / 8); e += kThreads) {
          const int r = e / (VP / 8), col = (e % (VP / 8)) * 8;
          const bool ok = r < K && col < V;
          cp_async_16(sP + p * Sh::kP + r * Tile<VP>::kPitch + col * 2, ok ? src + p * KV + r * V + col : src, ok);
        }
      } else {
        for (int e = tid; e < KP * VP; e += kThreads) {
          const int r = e / VP, col = e % VP;
          const uint16_t x = r < K && col < V ? src[p * KV + r * V + col] : uint16_t(0);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(sP + p * Sh::kP + r * Tile<VP>::kPitch + col * 2), "h"(x) : "memory");
        }
      }
    }
    cp_async_commit();
  };
  load_planes(gS);
  cp_async_wait<0>();
  __syncthreads();

  const int m0 = 16 * warp + g, m1 = m0 + 8;  // the warp's rows of every product
  // exp(l_i - l_j) for rows i of block bi > bj and columns j, or within a block (i >= j, else 0).
  auto diag = [&](int i, int j) {
    return i >= j ? exp_fast((d.rel[i] - d.rel[j]) + (dg.rel_lo[i] - dg.rel_lo[j])) : 0.f;
  };
  // Dot product of the warp's rows of a bf16 tile with accumulators, over the quad's lanes.
  auto row_dots = [&](uint32_t tile, const float (&x)[KP / 8][4], float* out) {
    float a = 0.f, e = 0.f;
#pragma unroll
    for (int nt = 0; nt < KP / 8; ++nt) {
      const uint32_t u0 = ld_shared_b32(tile + m0 * Tile<KP>::kPitch + (8 * nt + 2 * q4) * 2);
      const uint32_t u1 = ld_shared_b32(tile + m1 * Tile<KP>::kPitch + (8 * nt + 2 * q4) * 2);
      a = fmaf(bf16lo(u0), x[nt][0], fmaf(bf16hi(u0), x[nt][1], a));
      e = fmaf(bf16lo(u1), x[nt][2], fmaf(bf16hi(u1), x[nt][3], e));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    if (q4 == 0) {
      out[m0] = a;
      out[m1] = e;
    }
  };
  // Rows of an output: x f0 (row m0), x f1 (row m1); zero behind the sequence's end.
  auto store_rows = [&](float* out, int64_t stride, int width, const float (&x)[4], int nt, float f0, float f1) {
    const int col = 8 * nt + 2 * q4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = h ? m1 : m0;
      if (m >= rows || col >= width) continue;
      const bool ok = t0 + m < len;
      const float f = h ? f1 : f0, y0 = ok ? x[2 * h] * f : 0.f, y1 = ok ? x[2 * h + 1] * f : 0.f;
      float* at = out + m * stride + col;
      if (width % 2 == 0) {
        *reinterpret_cast<float2*>(at) = make_float2(y0, y1);
      } else {
        at[0] = y0;
        if (col + 1 < width) at[1] = y1;
      }
    }
  };

  {  // dq_i = first_i S u_i + sum_j E_ij D_j (u_i . v_j) k_j
    float x[KP / 8][4] = {};
    uint32_t uf[kVt][4];
#pragma unroll
    for (int vt = 0; vt < kVt; ++vt) ldmatrix_x4(uf[vt], at_rows<VP>(sU, 16 * warp, 16 * vt, lane));
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int vt = 0; vt < kVt; ++vt)
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
          uint32_t f[4];
          ldmatrix_x4(f, at_cols<VP>(sP + p * Sh::kP, 16 * kt, 16 * vt, lane));
          mma_bf16_16816(x[2 * kt], uf[vt], f[0], f[1]);
          mma_bf16_16816(x[2 * kt + 1], uf[vt], f[2], f[3]);
        }
    const float f0 = d.first[m0], f1 = d.first[m1], r0 = d.row[m0], r1 = d.row[m1];
#pragma unroll
    for (int nt = 0; nt < KP / 8; ++nt) {
      x[nt][0] *= f0;
      x[nt][1] *= f0;
      x[nt][2] *= f1;
      x[nt][3] *= f1;
    }
    // Not unrolled, here and below: four copies of the body do not fit the instruction cache.
#pragma unroll 1
    for (int jt = 0; jt <= warp; ++jt) {
      float s[2][4] = {};
#pragma unroll
      for (int vt = 0; vt < kVt; ++vt) {
        uint32_t f[4];
        ldmatrix_x4(f, at_cols<VP>(sV, 16 * jt, 16 * vt, lane));
        mma_bf16_16816(s[0], uf[vt], f[0], f[1]);
        mma_bf16_16816(s[1], uf[vt], f[2], f[3]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 16 * jt + 8 * h + 2 * q4 + e;
          const float Dj = d.D[j];
          if (jt < warp) {
            const float cf = d.col[warp - 1][j] * Dj;
            s[h][e] *= r0 * cf;
            s[h][2 + e] *= r1 * cf;
          } else {
            s[h][e] = j <= m0 ? s[h][e] * (diag(m0, j) * Dj) : 0.f;
            s[h][2 + e] = j <= m1 ? s[h][2 + e] * (diag(m1, j) * Dj) : 0.f;
          }
        }
      uint32_t p[3][4];
      split_scores(s, p);
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
        uint32_t f[4];
        ldmatrix_x4_trans(f, at_rows<KP>(sK, 16 * jt, 16 * kt, lane));
        add_split(x[2 * kt], p, f[0], f[1]);
        add_split(x[2 * kt + 1], p, f[2], f[3]);
      }
    }
    row_dots(sQ, x, qd);
#pragma unroll
    for (int nt = 0; nt < KP / 8; ++nt) store_rows(dq, qk_stride, K, x[nt], nt, 1.f, 1.f);
  }

  // dw_r's share: sum over the steps of u v.
  if (wr_part != nullptr) {
    for (int col = tid; col < V; col += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int j = 0; j < kChunk; ++j)
        s = fmaf(bf16_bits_to_f32(static_cast<uint16_t>(ld_shared_u16(sU + j * Tile<VP>::kPitch + col * 2))),
                 bf16_bits_to_f32(static_cast<uint16_t>(ld_shared_u16(sV + j * Tile<VP>::kPitch + col * 2))), s);
      wr_part[col] = s;
    }
  }

  __syncthreads();
  load_planes(gR);  // in S's place, behind the first half of dk

  const float l0 = dg.last[m0], l1 = dg.last[m1], D0 = d.D[m0], D1 = d.D[m1];
  // Rows j of the transposed scores: factors exp(l_i - l_j), columns i of block it.
  auto decay_columns = [&](int it, float (&s)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 16 * it + 8 * h + 2 * q4 + e;
        if (it > warp) {
          const float r = d.row[i];
          s[h][e] *= r * d.col[it - 1][m0];
          s[h][2 + e] *= r * d.col[it - 1][m1];
        } else {
          s[h][e] = i >= m0 ? s[h][e] * diag(i, m0) : 0.f;
          s[h][2 + e] = i >= m1 ? s[h][2 + e] * diag(i, m1) : 0.f;
        }
      }
  };

  {  // zk_j = last_j R v_j + sum_i E_ij (u_i . v_j) q_i
    float x[KP / 8][4] = {};
    uint32_t vf[kVt][4];
#pragma unroll
    for (int vt = 0; vt < kVt; ++vt) ldmatrix_x4(vf[vt], at_rows<VP>(sV, 16 * warp, 16 * vt, lane));
#pragma unroll 1
    for (int it = warp; it < 4; ++it) {
      float s[2][4] = {};
#pragma unroll
      for (int vt = 0; vt < kVt; ++vt) {
        uint32_t f[4];
        ldmatrix_x4(f, at_cols<VP>(sU, 16 * it, 16 * vt, lane));
        mma_bf16_16816(s[0], vf[vt], f[0], f[1]);
        mma_bf16_16816(s[1], vf[vt], f[2], f[3]);
      }
      decay_columns(it, s);
      uint32_t p[3][4];
      split_scores(s, p);
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
        uint32_t f[4];
        ldmatrix_x4_trans(f, at_rows<KP>(sQ, 16 * it, 16 * kt, lane));
        add_split(x[2 * kt], p, f[0], f[1]);
        add_split(x[2 * kt + 1], p, f[2], f[3]);
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    float z[KP / 8][4] = {};
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int vt = 0; vt < kVt; ++vt)
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
          uint32_t f[4];
          ldmatrix_x4(f, at_cols<VP>(sP + p * Sh::kP, 16 * kt, 16 * vt, lane));
          mma_bf16_16816(z[2 * kt], vf[vt], f[0], f[1]);
          mma_bf16_16816(z[2 * kt + 1], vf[vt], f[2], f[3]);
        }
    row_dots(sK, z, ci);  // times last_j below
#pragma unroll
    for (int nt = 0; nt < KP / 8; ++nt) {
      x[nt][0] = fmaf(l0, z[nt][0], x[nt][0]);
      x[nt][1] = fmaf(l0, z[nt][1], x[nt][1]);
      x[nt][2] = fmaf(l1, z[nt][2], x[nt][2]);
      x[nt][3] = fmaf(l1, z[nt][3], x[nt][3]);
    }
    row_dots(sK, x, ck);
#pragma unroll
    for (int nt = 0; nt < KP / 8; ++nt) store_rows(dk, qk_stride, K, x[nt], nt, D0, D1);
  }

  // <R, S>: the thread's pieces of S are loaded here and used behind dv, with
  // R from shared memory (the two larger parts of both: what the third adds to
  // a sum over K V elements is far below fp32).
  constexpr int kDot = KP * VP / 8 / kThreads < 4 ? KP * VP / 8 / kThreads : 4;
  uint4 s_hi[kDot], s_mid[kDot];
  if (vec) {
#pragma unroll
    for (int i = 0; i < kDot; ++i) {
      const int e = i * kThreads + tid, r = e / (VP / 8), col = (e % (VP / 8)) * 8;
      s_hi[i] = s_mid[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < K && col < V) {
        s_hi[i] = *reinterpret_cast<const uint4*>(gS + r * V + col);
        s_mid[i] = *reinterpret_cast<const uint4*>(gS + KV + r * V + col);
      }
    }
  }

  {  // zv_j = last_j R^T k_j + sum_i E_ij (q_i . k_j) u_i
    float x[VP / 8][4] = {};
    uint32_t kf[kKt][4];
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt) ldmatrix_x4(kf[kt], at_rows<KP>(sK, 16 * warp, 16 * kt, lane));
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int vt = 0; vt < kVt; ++vt) {
          uint32_t f[4];
          ldmatrix_x4_trans(f, at_rows<VP>(sP + p * Sh::kP, 16 * kt, 16 * vt, lane));
          mma_bf16_16816(x[2 * vt], kf[kt], f[0], f[1]);
          mma_bf16_16816(x[2 * vt + 1], kf[kt], f[2], f[3]);
        }
#pragma unroll
    for (int nt = 0; nt < VP / 8; ++nt) {
      x[nt][0] *= l0;
      x[nt][1] *= l0;
      x[nt][2] *= l1;
      x[nt][3] *= l1;
    }
#pragma unroll 1
    for (int it = warp; it < 4; ++it) {
      float s[2][4] = {};
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
        uint32_t f[4];
        ldmatrix_x4(f, at_cols<KP>(sQ, 16 * it, 16 * kt, lane));
        mma_bf16_16816(s[0], kf[kt], f[0], f[1]);
        mma_bf16_16816(s[1], kf[kt], f[2], f[3]);
      }
      decay_columns(it, s);
      uint32_t p[3][4];
      split_scores(s, p);
#pragma unroll
      for (int vt = 0; vt < kVt; ++vt) {
        uint32_t f[4];
        ldmatrix_x4_trans(f, at_rows<VP>(sU, 16 * it, 16 * vt, lane));
        add_split(x[2 * vt], p, f[0], f[1]);
        add_split(x[2 * vt + 1], p, f[2], f[3]);
      }
    }
    const uint16_t* wr = A.w_r ? static_cast<const uint16_t*>(A.w_r) + n * V : nullptr;
#pragma unroll
    for (int nt = 0; nt < VP / 8; ++nt) {
      const int col = 8 * nt + 2 * q4;
      x[nt][0] *= D0;
      x[nt][1] *= D0;
      x[nt][2] *= D1;
      x[nt][3] *= D1;
      if (wr != nullptr) {
        const float w0 = col < V ? to_f32(wr[col]) : 0.f, w1 = col + 1 < V ? to_f32(wr[col + 1]) : 0.f;
        const uint32_t u0 = ld_shared_b32(sU + m0 * Tile<VP>::kPitch + col * 2);
        const uint32_t u1 = ld_shared_b32(sU + m1 * Tile<VP>::kPitch + col * 2);
        x[nt][0] = fmaf(w0, bf16lo(u0), x[nt][0]);
        x[nt][1] = fmaf(w1, bf16hi(u0), x[nt][1]);
        x[nt][2] = fmaf(w0, bf16lo(u1), x[nt][2]);
        x[nt][3] = fmaf(w1, bf16hi(u1), x[nt][3]);
      }
      store_rows(dv, v_stride, V, x[nt], nt, 1.f, 1.f);
    }
  }
  float rs = 0.f;
  auto dot_piece = [&](const uint4& hi, const uint4& mid, int r, int col) {
    const uint4 b0 = ld_shared_v4(sP + r * Tile<VP>::kPitch + col * 2);
    const uint4 b1 = ld_shared_v4(sP + Sh::kP + r * Tile<VP>::kPitch + col * 2);
    const uint32_t x0[4] = {hi.x, hi.y, hi.z, hi.w}, x1[4] = {mid.x, mid.y, mid.z, mid.w};
    const uint32_t y0[4] = {b0.x, b0.y, b0.z, b0.w}, y1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rs = fmaf(bf16lo(x0[i]) + bf16lo(x1[i]), bf16lo(y0[i]) + bf16lo(y1[i]), rs);
      rs = fmaf(bf16hi(x0[i]) + bf16hi(x1[i]), bf16hi(y0[i]) + bf16hi(y1[i]), rs);
    }
  };
  if (vec) {
#pragma unroll
    for (int i = 0; i < kDot; ++i) {
      const int e = i * kThreads + tid;
      dot_piece(s_hi[i], s_mid[i], e / (VP / 8), (e % (VP / 8)) * 8);  // zeros where there is no S
    }
    for (int e = kDot * kThreads + tid; e < K * (VP / 8); e += kThreads) {
      const int r = e / (VP / 8), col = (e % (VP / 8)) * 8;
      if (col < V)
        dot_piece(*reinterpret_cast<const uint4*>(gS + r * V + col),
                  *reinterpret_cast<const uint4*>(gS + KV + r * V + col), r, col);
    }
  } else {
    for (int e = tid; e < K * V; e += kThreads) {
      const int r = e / V, col = e % V;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int p = 1; p >= 0; --p) {
        x += bf16_bits_to_f32(static_cast<uint16_t>(ld_shared_u16(sP + p * Sh::kP + r * Tile<VP>::kPitch + col * 2)));
        y += bf16_bits_to_f32(gS[p * KV + e]);
      }
      rs = fmaf(x, y, rs);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
  if (lane == 0) red[warp] = rs;
  __syncthreads();

  if (warp == 0) {  // two steps a lane
    const int i = 2 * lane;
    const float A_n = A.A[n];
    float s = d.wD[i] * ci[i] + d.wD[i + 1] * ci[i + 1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float end = fmaf(W.tot[blockIdx.x], (red[0] + red[1]) + (red[2] + red[3]), s);  // <R, S'>
    const float y0 = qd[i] - d.D[i] * ck[i], y1 = qd[i + 1] - d.D[i + 1] * ck[i + 1];
    float x = y0 + y1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float p = __shfl_down_sync(0xffffffffu, x, o);
      if (lane + o < 32) x += p;
    }
    const float next = __shfl_down_sync(0xffffffffu, x, 1), after = lane == 31 ? 0.f : next;
    const float g0 = x + end, g1 = y1 + after + end;
    const bool ok0 = t0 + i < len, ok1 = t0 + i + 1 < len;
    const float e0 = ok0 ? (ck[i] + A_n * g0) * dg.sg[i] : 0.f, e1 = ok1 ? (ck[i + 1] + A_n * g1) * dg.sg[i + 1] : 0.f;
    if (i < rows) ddt[static_cast<int64_t>(i) * A.N] = e0;
    if (i + 1 < rows) ddt[static_cast<int64_t>(i + 1) * A.N] = e1;
    float pa = (ok0 ? d.D[i] * g0 : 0.f) + (ok1 ? d.D[i + 1] * g1 : 0.f), pb = e0 + e1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      pa += __shfl_xor_sync(0xffffffffu, pa, o);
      pb += __shfl_xor_sync(0xffffffffu, pb, o);
    }
    if (lane == 0) W.o.ab_part[blockIdx.x] = make_float2(pa, pb);
  }
}

int padded(int64_t x) { return x <= 32 ? 32 : x <= 64 ? 64 : 128; }

struct Layout {
  size_t decay, tot, sums[2], planes[2], ab, wr, dq, dk, total;
};

Layout make_layout(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V) {
  Layout l{};
  l.total = sizeof(StatusBlock);
  auto take = [&](size_t bytes) {
    const size_t at = l.total;
    l.total += (bytes + 15) / 16 * 16;
    return at;
  };
  const size_t chunks = static_cast<size_t>(B) * N * ((T + kChunk - 1) / kChunk), KV = static_cast<size_t>(K) * V;
  l.decay = take(chunks * sizeof(ChunkDecayGrad));
  l.tot = take(chunks * 4);
  for (int i = 0; i < 2; ++i) {
    l.sums[i] = take(chunks * KV * 4);
    l.planes[i] = take(chunks * KV * 6);
  }
  l.ab = take(chunks * 8);
  l.wr = take(chunks * V * 4);
  if (G != N) {
    l.dq = take(static_cast<size_t>(B) * T * N * K * 4);
    l.dk = take(static_cast<size_t>(B) * T * N * K * 4);
  }
  return l;
}

template <int KP, int VP>
cudaError_t run(const GradArgs& w, cudaStream_t s) {
  constexpr int VS = VP < 64 ? VP : 64;
  using Sum = SumShape<KP, VS>;
  using Gr = GradShape<KP, VP>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_grad_kernel<KP, VP>), Gr::kBytes, done);
  if (e != cudaSuccess) return e;
  const SsmArgs& a = w.a;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.N * w.nc);
  const int slices = (a.V + VS - 1) / VS, KV = a.K * a.V;
  ssm_grad_sum_kernel<KP, VS><<<dim3(blocks, 2 * slices), kThreads, Sum::kBytes, s>>>(w, slices);
  if (KV % 4 == 0)
    ssm_grad_scan_kernel<4><<<dim3(a.B * a.N, (KV / 4 + 255) / 256, 2), 256, 0, s>>>(w);
  else
    ssm_grad_scan_kernel<1><<<dim3(a.B * a.N, (KV + 255) / 256, 2), 256, 0, s>>>(w);
  ssm_grad_kernel<KP, VP><<<blocks, kThreads, Gr::kBytes, s>>>(w);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_mma_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V) {
  return make_layout(B, T, N, G, K, V).total;
}

cudaError_t launch_ssm_mma_backward(const SsmArgs& a, cudaStream_t s) {
  const Layout l = make_layout(a.B, a.T, a.N, a.G, a.K, a.V);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  GradArgs w{};
  w.a = a;
  w.nc = (a.T + kChunk - 1) / kChunk;
  w.decay = reinterpret_cast<const ChunkDecayGrad*>(ws + l.decay);
  w.tot = reinterpret_cast<const float*>(ws + l.tot);
  for (int i = 0; i < 2; ++i) {
    w.sums[i] = reinterpret_cast<float*>(ws + l.sums[i]);
    w.planes[i] = reinterpret_cast<uint16_t*>(ws + l.planes[i]);
  }
  w.o = SsmGradOut{a.dq, a.dk, a.dw_r ? reinterpret_cast<float*>(ws + l.wr) : nullptr,
                   reinterpret_cast<float2*>(ws + l.ab), a.N};
  if (a.G != a.N) {
    w.o.dq = reinterpret_cast<float*>(ws + l.dq);
    w.o.dk = reinterpret_cast<float*>(ws + l.dk);
  }
  auto vec = [](const void* p, int64_t stride, int width) {
    return width % 8 == 0 && stride % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  w.vq = vec(a.q, a.q_stride, a.K);
  w.vk = vec(a.k, a.k_stride, a.K);
  w.vv = vec(a.v, a.v_stride, a.V);
  w.vu = vec(a.dy, static_cast<int64_t>(a.N) * a.V, a.V);
  cudaError_t e = launch_ssm_decay(a, ws + l.decay, reinterpret_cast<float*>(ws + l.tot), w.nc, true,
                                  reinterpret_cast<StatusBlock*>(ws), s);
  if (e != cudaSuccess) return e;
  const int kp = padded(a.K), vp = padded(a.V);
  e = cudaErrorInvalidValue;
#define M2RNN_SSM_CASE(KP, VP) \
  if (kp == KP && vp == VP) e = run<KP, VP>(w, s);
  M2RNN_SSM_CASE(32, 32)
  M2RNN_SSM_CASE(32, 64)
  M2RNN_SSM_CASE(32, 128)
  M2RNN_SSM_CASE(64, 32)
  M2RNN_SSM_CASE(64, 64)
  M2RNN_SSM_CASE(64, 128)
  M2RNN_SSM_CASE(128, 32)
  M2RNN_SSM_CASE(128, 64)
  M2RNN_SSM_CASE(128, 128)
#undef M2RNN_SSM_CASE
  if (e != cudaSuccess) return e;
  return launch_ssm_grad_sums(a, w.o, w.nc, s);
}

}  // namespace m2rnn
