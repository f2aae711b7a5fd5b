// Selective state space scan, the linear sister of the library's recurrence
// on the same matrix state, per batch element b and head n:
//     D_t = softplus(dt_t + dt_bias),  a_t = exp(D_t A),
//     H_t = a_t H_{t-1} + D_t k_t v_t^T,   y_t = H_t^T q_t + w_r (*) v_t.
// It is affine in H, so the steps of a chunk can be taken together.  With
// l_i the sum of D A over the chunk's steps up to i, S the state before the
// chunk and E_ij = exp(l_i - l_j) for i >= j, else 0:
//     y_i = exp(l_i) S^T q_i + sum_j E_ij D_j (q_i . k_j) v_j + w_r (*) v_i,
//     S'  = exp(l_L) S + sum_j exp(l_L - l_j) D_j k_j v_j^T.
// Backward, u = dy, R the gradient of the state behind the chunk:
//     dq_i = exp(l_i) S u_i + sum_j E_ij D_j (u_i . v_j) k_j,
//     zk_j = exp(l_L - l_j) R v_j + sum_i E_ij (u_i . v_j) q_i,    dk = D zk,
//     zv_j = exp(l_L - l_j) R^T k_j + sum_i E_ij (q_i . k_j) u_i,  dv = D zv + w_r (*) u,
//     R'   = exp(l_L) R + sum_i exp(l_i) q_i u_i^T  (the gradient of S).
// The gradient g_t of log a_t is everything that crosses from before t to t
// and later.  With W_ij = E_ij D_j (u_i . v_j)(q_i . k_j), b_j = k_j . R v_j,
//     g_t = exp(l_L) <R, S> + sum_{j < t} exp(l_L - l_j) D_j b_j
//           + sum_{i >= t} exp(l_i) q_i . S u_i + sum_{j < t <= i} W_ij,
// the last sum as sum_{i >= t} (sum_{j < i} W_ij - sum_{j > i} W_ji): what lies
// on one side of t cancels exactly, because both sums are of the same W,
// rounded once, and are added up in two floats.  (The shorter q_i . dq_i -
// k_i . dk_i for what is summed over i loses up to ten times as much, and dA
// and ddt_bias, sums over all steps that mostly cancel, show it.)  And dD_t = k_t . zk_t + A g_t, ddt = dD sigmoid(dt + dt_bias), dA = sum D g.
//
// This file: the dispatch by type (ssm_f32.cu; ssm_mma.cu with ssm_tc.cu, and
// ssm_grad.cu, for bf16), the sums behind the chunks' gradients, and the one-token step.
#include <cuda_runtime.h>

#include <cstdint>

#include "gate.cuh"
#include "layer.cuh"
#include "ssm.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// dA, ddt_bias [N] and dw_r [N,V]: fixed-order sums of the partials over the
// chunks of every b, in one launch.  Block (n, 0): 512 threads take chunks i,
// i + 512, ... (fp64: both sums cancel); block (n, 1 + x): 16 warps take every
// sixteenth chunk of columns 32 x .., added in warp order.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) ssm_grad_sums_kernel(const float2* ab, const float* wr, float* dA,
                                                                    float* ddt_bias, float* dw_r, int B, int N, int nc,
                                                                    int V) {
  __shared__ double2 red[kSumThreads / 32];
  __shared__ float col[kSumThreads / 32][32];
  let_next();
  wait_previous();
  const int n = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5, chunks = B * nc;
  auto at = [&](int i) { return (static_cast<int64_t>(i / nc) * N + n) * nc + i % nc; };
  if (blockIdx.y == 0) {
    double2 s = make_double2(0., 0.);
    for (int i = threadIdx.x; i < chunks; i += kSumThreads) {
      const float2 p = ab[at(i)];
      s.x += p.x;
      s.y += p.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    if (lane == 0) red[w] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < kSumThreads / 32; ++i) {
      s.x += red[i].x;
      s.y += red[i].y;
    }
    dA[n] = static_cast<float>(s.x);
    if (ddt_bias != nullptr) ddt_bias[n] = static_cast<float>(s.y);
    return;
  }
  const int vv = (blockIdx.y - 1) * 32 + lane;
  float s = 0.f;
  if (vv < V) {
#pragma unroll 8
    for (int i = w; i < chunks; i += kSumThreads / 32) s += wr[at(i) * V + vv];
  }
  col[w][lane] = s;
  __syncthreads();
  if (w != 0 || vv >= V) return;
  for (int i = 1; i < kSumThreads / 32; ++i) s += col[i][lane];
  dw_r[static_cast<int64_t>(n) * V + vv] = s;
}

// dq, dk of the G shared heads: the per-head gradients summed in head order.
__global__ void __launch_bounds__(kThreads) ssm_sum_heads_kernel(const float* dqh, const float* dkh, float* dq,
                                                                 float* dk, int64_t n, int N, int G, int K) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  wait_previous();
  if (i >= n) return;
  const int kk = static_cast<int>(i % K), g = static_cast<int>((i / K) % G), r = N / G;
  const int64_t bt = i / (static_cast<int64_t>(K) * G), at = (bt * N + static_cast<int64_t>(g) * r) * K + kk;
  float a = 0.f, b = 0.f;
  for (int h = 0; h < r; ++h) {
    a += dqh[at + static_cast<int64_t>(h) * K];
    b += dkh[at + static_cast<int64_t>(h) * K];
  }
  dq[i] = a;
  dk[i] = b;
}

// One token.  Block (b, n) streams its state through registers once: thread
// (x, y) takes kVec columns of rows y, y + rows, ..., kAhead rows' loads in
// flight; y_t is summed over a thread's rows, then over the y in order.  Bound
// by HBM (8 bytes per state element) at large batches, by latency at small:
// 2048 states of 128 x 128 take 43.4 us (6.2 TB/s, 91 % of a plain copy's
// rate), 32 states of 64 x 64 2.9 us.
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 3) ssm_step_kernel(float* H, SsmArgs A) {
  constexpr int kAhead = kVec == 4 ? 8 : 4;
  __shared__ float red[kThreads * kVec], sk[128], sq[128];
  const int bn = blockIdx.x, b = bn / A.N, n = bn - b * A.N, g = n / (A.N / A.G), K = A.K, V = A.V;
  const int cols = V / kVec, rows = kThreads / cols, y = threadIdx.x / cols, x = threadIdx.x - y * cols;
  const float s = to_f32(static_cast<const T*>(A.dt)[b * A.dt_stride + n]) + (A.dt_bias ? A.dt_bias[n] : 0.f);
  const float An = A.A[n];
  float* h = H + static_cast<int64_t>(bn) * K * V + x * kVec;
  const bool own = y < rows;
  float st[kAhead][kVec];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = r0 + u * rows;
      if (!own || r >= K) continue;
      if constexpr (kVec == 4)
        *reinterpret_cast<float4*>(st[u]) = *reinterpret_cast<const float4*>(h + r * V);
      else
        st[u][0] = h[r * V];
    }
  };
  load(y);  // before anything waits
  float vx[kVec], acc[kVec];
  {
    const T* v = static_cast<const T*>(A.v) + b * A.v_stride + static_cast<int64_t>(n) * V + x * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      vx[e] = own ? to_f32(v[e]) : 0.f;
      acc[e] = 0.f;
    }
  }
  const float D = softplus_f(s), a = expf(D * An);
  if (threadIdx.x < K) {
    sk[threadIdx.x] = D * to_f32(static_cast<const T*>(A.k)[b * A.k_stride + static_cast<int64_t>(g) * K + threadIdx.x]);
    sq[threadIdx.x] = to_f32(static_cast<const T*>(A.q)[b * A.q_stride + static_cast<int64_t>(g) * K + threadIdx.x]);
  }
  __syncthreads();
  if (own) {
    for (int r0 = y; r0 < K; r0 += kAhead * rows) {
      if (r0 != y) load(r0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int r = r0 + u * rows;
        if (r >= K) continue;
        const float kd = sk[r], qr = sq[r];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          st[u][e] = fmaf(a, st[u][e], kd * vx[e]);
          acc[e] = fmaf(qr, st[u][e], acc[e]);
        }
        if constexpr (kVec == 4)
          *reinterpret_cast<float4*>(h + r * V) = *reinterpret_cast<const float4*>(st[u]);
        else
          h[r * V] = st[u][0];
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) red[y * V + x * kVec + e] = acc[e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < V; c += kThreads) {
    float t = 0.f;
    for (int r = 0; r < min(rows, K); ++r) t += red[r * V + c];
    if (A.w_r)
      t = fmaf(to_f32(static_cast<const T*>(A.w_r)[n * V + c]),
               to_f32(static_cast<const T*>(A.v)[b * A.v_stride + static_cast<int64_t>(n) * V + c]), t);
    static_cast<T*>(A.y)[static_cast<int64_t>(bn) * V + c] = from_f32<T>(t);
  }
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_ssm_grad_sums(const SsmArgs& a, const SsmGradOut& o, int nc, cudaStream_t s) {
  const cudaError_t e = launch_next(ssm_grad_sums_kernel, dim3(a.N, a.dw_r != nullptr ? 1 + (a.V + 31) / 32 : 1),
                                    kSumThreads, 0, s, o.ab_part, o.wr_part, a.dA, a.ddt_bias, a.dw_r, a.B, a.N, nc, a.V);
  if (e != cudaSuccess || a.G == a.N) return e;
  const int64_t n = static_cast<int64_t>(a.B) * a.T * a.G * a.K;
  return launch_next(ssm_sum_heads_kernel, static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s, o.dq,
                     o.dk, a.dq, a.dk, n, a.N, a.G, a.K);
}

size_t ssm_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, bool bf16) {
  return align256(bf16 ? ssm_mma_forward_scratch_bytes(B, T, N, K, V) : ssm_f32_forward_scratch_bytes(B, T, N, K, V));
}

size_t ssm_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V, bool bf16) {
  return align256(bf16 ? ssm_mma_backward_scratch_bytes(B, T, N, G, K, V)
                       : ssm_f32_backward_scratch_bytes(B, T, N, G, K, V));
}

cudaError_t launch_ssm_forward(const SsmArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_ssm_mma_forward(a, s) : launch_ssm_f32_forward(a, s);
}

cudaError_t launch_ssm_backward(const SsmArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_ssm_mma_backward(a, s) : launch_ssm_f32_backward(a, s);
}

cudaError_t launch_ssm_step(float* H, const SsmArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.B * a.N);
  if (a.bf16 && a.V % 4 == 0)
    ssm_step_kernel<uint16_t, 4><<<grid, kThreads, 0, s>>>(H, a);
  else if (a.bf16)
    ssm_step_kernel<uint16_t, 1><<<grid, kThreads, 0, s>>>(H, a);
  else if (a.V % 4 == 0)
    ssm_step_kernel<float, 4><<<grid, kThreads, 0, s>>>(H, a);
  else
    ssm_step_kernel<float, 1><<<grid, kThreads, 0, s>>>(H, a);
  return cudaGetLastError();
}

}  // namespace m2rnn
