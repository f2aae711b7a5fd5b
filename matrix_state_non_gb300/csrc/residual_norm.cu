// Root-mean-square norm of the residual stream, with the branch's addition:
//     h = x + residual,  s = (sum_j h_j^2 / D + eps)^(-1/2),  y = w (*) h s,
// y in bf16, fp32, or e4m3 with a scale for each 128 values of a row; and its
// backward, with p = w (*) dy and r = sum_j p_j h_j per row:
//     dx = s p - r s^3 h / D + dh,   dw = sum over rows of dy (*) h s.
//
// Bound by HBM: a team of 1 to 16 warps has a row in registers, reads and
// writes it once, and goes from row to row with w in registers, the next row's
// inputs on their way.  A lane holds groups of 8 neighbouring values (kVec:
// 16-byte accesses, where every row lies on 16 bytes), or values 32 apart; either
// way 128 values that share a scale are in one warp.  Sums run in a fixed order.
// 16384 x 1024 bf16, with the sum written back: 22.8 us, 5.9 TB/s; the backward
// with dh: 36.6 us, 5.5 TB/s, 4 of them the second launch's sums.  A warp to a row
// of 1024 with 32 values a lane was 26.9 and 65: too few loads in flight.
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

// Teams of kTeam warps: a block of eight warps has one or several, one of
// sixteen is a block.
template <int kTeam>
struct Team {
  static constexpr int kWarps = kTeam > 8 ? kTeam : 8, kTeams = kWarps / kTeam, kThreads = 32 * kWarps;
  float2 red[2][kWarps];
};

// The sums over a team, in every thread.
template <int kTeam>
__device__ __forceinline__ float2 sum_team(float a, float b, Team<kTeam>& t, int turn) {
  a = sum_lanes(a);
  b = sum_lanes(b);
  if constexpr (kTeam == 1) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, team = warp / kTeam;
  float2* r = t.red[turn & 1] + team * kTeam;  // two in turn: one barrier is enough
  if ((threadIdx.x & 31) == 0) r[warp - team * kTeam] = make_float2(a, b);
  if constexpr (Team<kTeam>::kTeams == 1)
    __syncthreads();
  else
    named_bar_sync(1 + team, 32 * kTeam);
  float2 s = r[0];
#pragma unroll
  for (int w = 1; w < kTeam; ++w) {
    s.x += r[w].x;
    s.y += r[w].y;
  }
  return s;
}

// A thread's share of a row of up to 256 kPer kTeam values: kPer groups of 8.
// Element e of group i is value at(i, e).
template <int kTeam, int kPer, bool kVec>
struct Share {
  int lane, warp;
  __device__ __forceinline__ Share() : lane(threadIdx.x & 31), warp((threadIdx.x >> 5) % kTeam) {}
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

// Blocks per SM: registers, by the groups of a lane.
template <int kTeam, int kPer>
constexpr int kBlocksPerSm = kTeam > 8 ? 1 : kPer == 1 ? 4 : kPer == 2 ? 3 : 2;
// Of the backward, for its registers and its grid alike: 4096 x 4096 bf16 with dh takes
// 43.9 us with two (4.6 TB/s), 53.8 with one, 57.6 where registers left one of two.
constexpr int backward_per_sm(int team, int per) { return per == 1 ? 3 : team == 8 ? 2 : 1; }

template <typename X, typename H, int kTeam, int kPer, bool kVec>
__global__ void __launch_bounds__(Team<kTeam>::kThreads, kBlocksPerSm<kTeam, kPer>) residual_norm_kernel(NormRowsArgs A) {
  __shared__ Team<kTeam> team;
  using S = Share<kTeam, kPer, kVec>;
  constexpr int kTeams = Team<kTeam>::kTeams;
  const S me;
  const int D = A.D, blocks = (D + kScaleBlock - 1) / kScaleBlock;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + (threadIdx.x >> 5) / kTeam;
  float w[kPer][8];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = me.at(i, e) < D ? A.w[me.at(i, e)] : 0.f;
  typename S::template Raw<X> x;
  typename S::template Raw<H> r;
  const bool added = A.residual != nullptr;
  auto load = [&](int64_t at) {
    me.load(x, static_cast<const X*>(A.x) + at * A.x_stride, D);
    if (added) me.load(r, static_cast<const H*>(A.residual) + at * D, D);
  };
  constexpr bool kAhead = kPer == 1;  // registers for the next row's inputs
  if (kAhead && row < A.rows) load(row);
  for (int turn = 0; row < A.rows; row += step, ++turn) {
    if (!kAhead) load(row);
    float h[kPer][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = me.get(x, i, e) + (added ? me.get(r, i, e) : 0.f);
    if (kAhead && row + step < A.rows) load(row + step);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
      if (A.h != nullptr) me.store(static_cast<H*>(A.h) + row * D, i, h[i], D);
    }
    const float s = rsqrtf(sum_team<kTeam>(ss, 0.f, team, turn).x / static_cast<float>(D) + A.eps);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * s * w[i][e];
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
__global__ void __launch_bounds__(Team<kTeam>::kThreads, backward_per_sm(kTeam, kPer)) residual_norm_backward_kernel(NormRowsArgs A) {
  __shared__ Team<kTeam> team;
  using S = Share<kTeam, kPer, kVec>;
  constexpr int kTeams = Team<kTeam>::kTeams, kWidth = 256 * kPer * kTeam;
  __shared__ float dws[kTeams > 1 ? kTeams : 1][kTeams > 1 ? kWidth : 1];
  const S me;
  const int D = A.D;
  const float inv = 1.f / static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  const int mine = (threadIdx.x >> 5) / kTeam;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + mine;
  float w[kPer][8], dw[kPer][8];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = me.at(i, e) < D ? A.w[me.at(i, e)] : 0.f;
      dw[i][e] = 0.f;
    }
  typename S::template Raw<H> nh;
  typename S::template Raw<G> ng;
  typename S::template Raw<float> nu;
  const bool added = A.dh != nullptr;
  auto load = [&](int64_t at) {
    me.load(nh, static_cast<const H*>(A.h) + at * D, D);
    me.load(ng, static_cast<const G*>(A.dy) + at * D, D);
    if (added) me.load(nu, A.dh + at * D, D);
  };
  constexpr bool kAhead = kPer == 1;
  if (kAhead && row < A.rows) load(row);
  for (int turn = 0; row < A.rows; row += step, ++turn) {
    if (!kAhead) load(row);
    const typename S::template Raw<H> h = nh;
    const typename S::template Raw<G> g = ng;
    const typename S::template Raw<float> up = nu;
    if (kAhead && row + step < A.rows) load(row + step);
    float ss = 0.f, rr = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = me.get(h, i, e);
        ss = fmaf(v, v, ss);
        rr = fmaf(v, me.get(g, i, e) * w[i][e], rr);
      }
    const float2 t = sum_team<kTeam>(ss, rr, team, turn);
    const float s = rsqrtf(t.x * inv + A.eps);
    const float c = t.y * s * (s * inv) * s;  // (in this order nothing overflows for small rows)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = me.get(h, i, e), p = me.get(g, i, e);
        d[e] = s * (p * w[i][e]) - c * v + (added ? me.get(up, i, e) : 0.f);
        dw[i][e] = fmaf(p, v * s, dw[i][e]);
      }
      me.store(A.dx + row * D, i, d, D);
    }
  }
  let_next();
  float* part = A.part + static_cast<int64_t>(blockIdx.x) * D;
  if constexpr (kTeams > 1) {  // the block's teams, in order
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dws[mine][me.at(i, e)] = dw[i][e];
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += Team<kTeam>::kThreads) {
      float t = dws[0][j];
#pragma unroll
      for (int k = 1; k < kTeams; ++k) t += dws[k][j];
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
NormShape norm_shape(int64_t D) {
  if (D <= 256) return {1, 1};
  if (D <= 512) return {2, 1};
  if (D <= 1024) return {4, 1};
  if (D <= 2048) return {8, 1};
  if (D <= 4096) return {8, 2};
  if (D <= 8192) return {16, 2};
  return {16, 4};
}

// As many blocks as run at once, or as there are rows for.
int norm_grid(int64_t rows, const NormShape& sh, int per_sm) {
  const int teams = sh.team >= 8 ? 1 : 8 / sh.team;
  const int64_t blocks = (rows + teams - 1) / teams, most = 152 * per_sm;
  return static_cast<int>(blocks < most ? blocks : most);
}

#define M2RNN_NORM_SHAPES(CASE) \
  CASE(1, 1) CASE(2, 1) CASE(4, 1) CASE(8, 1) CASE(8, 2) CASE(16, 2) CASE(16, 4)

template <typename X, typename H, bool kVec>
cudaError_t forward(const NormRowsArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.D);
#define M2RNN_NORM_CASE(TEAM, PER)                                                                       \
  if (sh.team == TEAM && sh.per == PER)                                                                  \
    residual_norm_kernel<X, H, TEAM, PER, kVec>                                                          \
        <<<norm_grid(a.rows, sh, kBlocksPerSm<TEAM, PER>), Team<TEAM>::kThreads, 0, s>>>(a);
  M2RNN_NORM_SHAPES(M2RNN_NORM_CASE)
#undef M2RNN_NORM_CASE
  return cudaGetLastError();
}

template <typename H, typename G, bool kVec>
cudaError_t backward(const NormRowsArgs& a, int grid, cudaStream_t s) {
  const NormShape sh = norm_shape(a.D);
#define M2RNN_NORM_CASE(TEAM, PER)      \
  if (sh.team == TEAM && sh.per == PER) \
    residual_norm_backward_kernel<H, G, TEAM, PER, kVec><<<grid, Team<TEAM>::kThreads, 0, s>>>(a);
  M2RNN_NORM_SHAPES(M2RNN_NORM_CASE)
#undef M2RNN_NORM_CASE
  return cudaGetLastError();
}

}  // namespace

int norm_rows_parts(int64_t rows, int64_t D) {
  const NormShape sh = norm_shape(D);
  return norm_grid(rows, sh, backward_per_sm(sh.team, sh.per));
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
