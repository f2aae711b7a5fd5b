// Root-mean-square norm of the residual stream, with the branch's addition:
//     h = x + residual,  s = (sum_j h_j^2 / D + eps)^(-1/2),  y = w (*) h s,
// y in bf16, fp32, or e4m3 with a scale for each 128 values of a row; and its
// backward, with p = w (*) dy and r = sum_j p_j h_j per row:
//     dx = s p - r s^3 h / D + dh,   dw = sum over rows of dy (*) h s.
//
// Bound by HBM: a team of 1 to 16 warps has a row in registers, reads and
// writes it once, and goes from row to row with w in registers.  A lane holds
// groups of 8 neighbouring values (kVec: 16-byte accesses, where every row lies
// on 16 bytes), or values 32 apart; either way 128 values that share a scale are
// in one warp.  Sums run in a fixed order.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"

namespace m2rnn {
namespace {

__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over a team of kTeam warps (a block, where that is more than one).
template <int kTeam>
__device__ __forceinline__ float2 sum_team(float a, float b, float2 (&red)[2][kTeam], int turn) {
  a = sum_lanes(a);
  b = sum_lanes(b);
  if constexpr (kTeam == 1) return make_float2(a, b);
  float2* r = red[turn & 1];  // two in turn: one barrier is enough
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = r[0];
#pragma unroll
  for (int w = 1; w < kTeam; ++w) {
    t.x += r[w].x;
    t.y += r[w].y;
  }
  return t;
}

// A thread's share of a row of up to 256 kPer kTeam values: kPer groups of 8.
// Element e of group i is value at(i, e).
template <int kTeam, int kPer, bool kVec>
struct Share {
  int lane, warp;
  __device__ __forceinline__ Share() : lane(threadIdx.x & 31), warp(kTeam == 1 ? 0 : threadIdx.x >> 5) {}
  __device__ __forceinline__ int at(int i, int e) const {
    return kVec ? 8 * (lane + 32 * (warp * kPer + i)) + e : lane + 32 * (e + 8 * (warp * kPer + i));
  }
  // In flight: groups as they lie in memory.
  template <typename T>
  struct Raw {
    uint4 v[kPer][sizeof(T) / 2];
  };
  template <typename T>
  __device__ __forceinline__ void load(Raw<T>& r, const T* row, int D) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kVec) {
        const int j = at(i, 0);
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q)
          r.v[i][q] = j < D ? reinterpret_cast<const uint4*>(row + j)[q] : make_uint4(0u, 0u, 0u, 0u);
      } else {
        alignas(16) T e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = at(i, k) < D ? row[at(i, k)] : T(0);
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q) r.v[i][q] = reinterpret_cast<const uint4*>(e)[q];
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ float get(const Raw<T>& r, int i, int e) const {
    const uint4 u = r.v[i][e * sizeof(T) / 16];
    const uint32_t words[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(words[e % 4]);
    return __uint_as_float(e % 2 == 0 ? words[e / 2] << 16 : words[e / 2] & 0xffff0000u);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int i, const float (&v)[8], int D) const {
    if constexpr (kVec) {
      const int j = at(i, 0);
      if (j >= D) return;
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(row + j)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(row + j)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(row + j) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(i, e) < D) row[at(i, e)] = from_f32<T>(v[e]);
    }
  }
};

// Two values as e4m3, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

constexpr int kRowsPerBlock = 8;  // teams of one warp
template <int kTeam>
constexpr int kThreadsOf = kTeam == 1 ? 32 * kRowsPerBlock : 32 * kTeam;

template <typename X, typename H, int kTeam, int kPer, bool kVec>
__global__ void __launch_bounds__(kThreadsOf<kTeam>) residual_norm_kernel(NormRowsArgs A) {
  __shared__ float2 red[2][kTeam];
  using S = Share<kTeam, kPer, kVec>;
  const S me;
  const int D = A.D, blocks = (D + kScaleBlock - 1) / kScaleBlock;
  const int64_t teams = kTeam == 1 ? gridDim.x * static_cast<int64_t>(kRowsPerBlock) : gridDim.x;
  const int64_t team = kTeam == 1 ? blockIdx.x * static_cast<int64_t>(kRowsPerBlock) + (threadIdx.x >> 5) : blockIdx.x;
  typename S::template Raw<float> w;
  // w is allocated to 16 bytes; its end is guarded by value
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = me.at(i, 4 * q + k) < D ? A.w[me.at(i, 4 * q + k)] : 0.f;
      w.v[i][q] = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
    }
  int turn = 0;
  for (int64_t row = team; row < A.rows; row += teams, ++turn) {
    float h[kPer][8], ss = 0.f;
    {
      typename S::template Raw<X> x;
      me.load(x, static_cast<const X*>(A.x) + row * A.x_stride, D);
      if (A.residual != nullptr) {
        typename S::template Raw<H> r;
        me.load(r, static_cast<const H*>(A.residual) + row * D, D);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] = me.get(x, i, e) + me.get(r, i, e);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] = me.get(x, i, e);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
      if (A.h != nullptr) me.store(static_cast<H*>(A.h) + row * D, i, h[i], D);
    }
    const float s = rsqrtf(sum_team<kTeam>(ss, 0.f, red, turn).x / static_cast<float>(D) + A.eps);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * s * me.get(w, i, e);
      if (A.y_type == M2RNN_BF16) me.store(static_cast<uint16_t*>(A.y) + row * D, i, h[i], D);
      if (A.y_type == M2RNN_F32) me.store(static_cast<float*>(A.y) + row * D, i, h[i], D);
    }
    if (A.y_type != M2RNN_E4M3) continue;
    uint8_t* q = static_cast<uint8_t*>(A.y) + row * D;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kVec) {  // a scale's 128 values: 16 lanes of a group
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(h[i][e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float scale = fmaxf(most / 448.f, 0x1p-126f);
        const int j = me.at(i, 0);
        if (j < D) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = h[i][e] / scale;
          *reinterpret_cast<uint2*>(q + j) = make_uint2(e4m3_2(v[0], v[1]) | e4m3_2(v[2], v[3]) << 16,
                                                        e4m3_2(v[4], v[5]) | e4m3_2(v[6], v[7]) << 16);
          if (j % kScaleBlock == 0) A.scale[row * blocks + j / kScaleBlock] = scale;
        }
      } else {  // four values of each lane
#pragma unroll
        for (int half = 0; half < 8; half += 4) {
          float most = 0.f;
#pragma unroll
          for (int e = half; e < half + 4; ++e) most = fmaxf(most, fabsf(h[i][e]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          const float scale = fmaxf(most / 448.f, 0x1p-126f);
#pragma unroll
          for (int e = half; e < half + 4; ++e)
            if (me.at(i, e) < D) q[me.at(i, e)] = static_cast<uint8_t>(e4m3_2(h[i][e] / scale, 0.f));
          const int j = me.at(i, half) - me.lane;
          if (me.lane == 0 && j < D) A.scale[row * blocks + j / kScaleBlock] = scale;
        }
      }
    }
  }
}

template <typename H, typename G, int kTeam, int kPer, bool kVec>
__global__ void __launch_bounds__(kThreadsOf<kTeam>) residual_norm_backward_kernel(NormRowsArgs A) {
  __shared__ float2 red[2][kTeam];
  __shared__ float dws[kTeam == 1 ? kRowsPerBlock : 1][kTeam == 1 ? 256 * kPer : 1];
  using S = Share<kTeam, kPer, kVec>;
  const S me;
  const int D = A.D;
  const float inv = 1.f / static_cast<float>(D);
  const int64_t teams = kTeam == 1 ? gridDim.x * static_cast<int64_t>(kRowsPerBlock) : gridDim.x;
  const int64_t team = kTeam == 1 ? blockIdx.x * static_cast<int64_t>(kRowsPerBlock) + (threadIdx.x >> 5) : blockIdx.x;
  float w[kPer][8], dw[kPer][8];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = me.at(i, e) < D ? A.w[me.at(i, e)] : 0.f;
      dw[i][e] = 0.f;
    }
  int turn = 0;
  for (int64_t row = team; row < A.rows; row += teams, ++turn) {
    typename S::template Raw<H> h;
    typename S::template Raw<G> g;
    me.load(h, static_cast<const H*>(A.h) + row * D, D);
    me.load(g, static_cast<const G*>(A.dy) + row * D, D);
    float ss = 0.f, rr = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = me.get(h, i, e);
        ss = fmaf(v, v, ss);
        rr = fmaf(v, me.get(g, i, e) * w[i][e], rr);
      }
    const float2 t = sum_team<kTeam>(ss, rr, red, turn);
    const float s = rsqrtf(t.x * inv + A.eps), c = t.y * s * s * s * inv;
    const float* up = A.dh != nullptr ? A.dh + row * D : nullptr;
    float* out = A.dx + row * D;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = 0.f;
      if (up != nullptr) {
        if constexpr (kVec) {
          if (me.at(i, 0) < D) {
            const float4 a = *reinterpret_cast<const float4*>(up + me.at(i, 0)), b = *reinterpret_cast<const float4*>(up + me.at(i, 4));
            d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (me.at(i, e) < D) d[e] = up[me.at(i, e)];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = me.get(h, i, e), p = me.get(g, i, e);
        d[e] += s * (p * w[i][e]) - c * v;
        dw[i][e] = fmaf(p, v * s, dw[i][e]);
      }
      me.store(out, i, d, D);
    }
  }
  let_next();
  float* part = A.part + static_cast<int64_t>(blockIdx.x) * D;
  if constexpr (kTeam == 1) {  // the block's eight warps, in order
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dws[threadIdx.x >> 5][me.at(i, e)] = dw[i][e];
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += 32 * kRowsPerBlock) {
      float t = dws[0][j];
#pragma unroll
      for (int k = 1; k < kRowsPerBlock; ++k) t += dws[k][j];
      part[j] = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (me.at(i, e) < D) part[me.at(i, e)] = dw[i][e];
  }
}

// Warps to a row and groups of 8 per lane, by the width.
struct NormShape {
  int team, per;
};
NormShape norm_shape(int D) {
  if (D <= 256) return {1, 1};
  if (D <= 512) return {1, 2};
  if (D <= 1024) return {1, 4};
  if (D <= 2048) return {2, 4};
  if (D <= 4096) return {4, 4};
  if (D <= 8192) return {8, 4};
  return {16, 4};
}

constexpr int kSms = 152;

int forward_grid(int64_t rows, const NormShape& sh) {
  const int64_t blocks = sh.team == 1 ? (rows + kRowsPerBlock - 1) / kRowsPerBlock : rows;
  const int64_t most = sh.team == 1 ? 4 * kSms : kSms * (32 / sh.team);
  return static_cast<int>(blocks < most ? blocks : most);
}

template <typename X, typename H, bool kVec>
cudaError_t forward(const NormRowsArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.D);
  const int grid = forward_grid(a.rows, sh);
#define M2RNN_NORM_CASE(TEAM, PER)                                                          \
  if (sh.team == TEAM && sh.per == PER)                                                     \
  residual_norm_kernel<X, H, TEAM, PER, kVec><<<grid, kThreadsOf<TEAM>, 0, s>>>(a)
  M2RNN_NORM_CASE(1, 1);
  M2RNN_NORM_CASE(1, 2);
  M2RNN_NORM_CASE(1, 4);
  M2RNN_NORM_CASE(2, 4);
  M2RNN_NORM_CASE(4, 4);
  M2RNN_NORM_CASE(8, 4);
  M2RNN_NORM_CASE(16, 4);
#undef M2RNN_NORM_CASE
  return cudaGetLastError();
}

template <typename H, typename G, bool kVec>
cudaError_t backward(const NormRowsArgs& a, int grid, cudaStream_t s) {
  const NormShape sh = norm_shape(a.D);
#define M2RNN_NORM_CASE(TEAM, PER)                                                          \
  if (sh.team == TEAM && sh.per == PER)                                                     \
  residual_norm_backward_kernel<H, G, TEAM, PER, kVec><<<grid, kThreadsOf<TEAM>, 0, s>>>(a)
  M2RNN_NORM_CASE(1, 1);
  M2RNN_NORM_CASE(1, 2);
  M2RNN_NORM_CASE(1, 4);
  M2RNN_NORM_CASE(2, 4);
  M2RNN_NORM_CASE(4, 4);
  M2RNN_NORM_CASE(8, 4);
  M2RNN_NORM_CASE(16, 4);
#undef M2RNN_NORM_CASE
  return cudaGetLastError();
}

}  // namespace

int norm_rows_parts(int64_t rows, int64_t D) {
  const NormShape sh = norm_shape(static_cast<int>(D));
  const int64_t blocks = sh.team == 1 ? (rows + kRowsPerBlock - 1) / kRowsPerBlock : rows;
  const int64_t most = sh.team == 1 ? 2 * kSms : kSms * (16 / sh.team);
  return static_cast<int>(blocks < most ? blocks : most);
}

cudaError_t launch_residual_norm(const NormRowsArgs& a, cudaStream_t s) {
  // 16-byte accesses of x, residual, h and y, 8-byte ones of 8-bit y
  const bool vec = a.D % 8 == 0 && a.x_stride % (a.x_bf16 ? 8 : 4) == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0;
  if (a.x_bf16) {
    if (a.h_bf16) return vec ? forward<uint16_t, uint16_t, true>(a, s) : forward<uint16_t, uint16_t, false>(a, s);
    return vec ? forward<uint16_t, float, true>(a, s) : forward<uint16_t, float, false>(a, s);
  }
  if (a.h_bf16) return vec ? forward<float, uint16_t, true>(a, s) : forward<float, uint16_t, false>(a, s);
  return vec ? forward<float, float, true>(a, s) : forward<float, float, false>(a, s);
}

cudaError_t launch_residual_norm_backward(const NormRowsArgs& a, cudaStream_t s) {
  const int parts = norm_rows_parts(a.rows, a.D);
  const bool vec = a.D % 8 == 0;
  cudaError_t e;
  if (a.h_bf16) {
    if (a.dy_bf16)
      e = vec ? backward<uint16_t, uint16_t, true>(a, parts, s) : backward<uint16_t, uint16_t, false>(a, parts, s);
    else
      e = vec ? backward<uint16_t, float, true>(a, parts, s) : backward<uint16_t, float, false>(a, parts, s);
  } else {
    if (a.dy_bf16)
      e = vec ? backward<float, uint16_t, true>(a, parts, s) : backward<float, uint16_t, false>(a, parts, s);
    else
      e = vec ? backward<float, float, true>(a, parts, s) : backward<float, float, false>(a, parts, s);
  }
  return e != cudaSuccess ? e : launch_sum_parts(a.part, a.dw, nullptr, false, parts, a.D, s);
}

}  // namespace m2rnn
