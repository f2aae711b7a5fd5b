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
// and later; over the chunk it is a suffix sum,
//     g_t = <R, S'> + sum_{i >= t} (q_i . dq_i - k_i . dk_i),
// and dD_t = k_t . zk_t + A g_t, ddt = dD sigmoid(dt + dt_bias), dA = sum D g.
//
// This file: the kernels for every shape and type, on CUDA cores in fp32:
// chunk sums -> scan over the chunks -> outputs or gradients, each chunk on
// its own block; and the one-token step.
#include <cuda_runtime.h>

#include <cstdint>

#include "gate.cuh"
#include "layer.cuh"
#include "ssm.cuh"

namespace m2rnn {
namespace {

constexpr int kL = 32;  // steps per chunk: one per lane of the warp that prepares the decays
constexpr int kThreads = 256;

// The chunk's decays, in shared memory.
struct Decays {
  float D[kL];                // step sizes (0 behind the sequence's end)
  float sg[kL];               // sigmoid(dt + dt_bias)
  float hi[kL], lo[kL];       // l_i as hi + lo: differences of long sums keep their bits
  float first[kL], last[kL];  // exp(l_i), exp(l_L - l_i)
  float tot;                  // exp(l_L)
};

template <typename T>
__device__ void load_decays(const SsmArgs& A, int b, int n, int t0, int len, Decays& d) {
  const int i = threadIdx.x;
  if (i >= 32) return;
  const float An = A.A[n];
  float D = 0.f, sg = 0.f;
  if (t0 + i < len) {
    const float x = to_f32(static_cast<const T*>(A.dt)[(static_cast<int64_t>(b) * A.T + t0 + i) * A.dt_stride + n]) +
                    (A.dt_bias ? A.dt_bias[n] : 0.f);
    D = softplus_f(x);
    sg = 1.f / (1.f + expf(-x));
  }
  const double la = static_cast<double>(D) * An;
  double l = la;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double p = __shfl_up_sync(0xffffffffu, l, o);
    if (i >= o) l += p;
  }
  const double end = __shfl_sync(0xffffffffu, l, 31);
  d.D[i] = D;
  d.sg[i] = sg;
  d.hi[i] = static_cast<float>(l);
  d.lo[i] = static_cast<float>(l - d.hi[i]);
  d.first[i] = expf(static_cast<float>(l));
  d.last[i] = expf(static_cast<float>(end - l));
  if (i == 0) d.tot = expf(static_cast<float>(end));
}

__device__ __forceinline__ float decay(const Decays& d, int i, int j) {
  return expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
}

// Rows t0 .. t0 + kL - 1 of one head as fp32 (zero behind `len`), `ld` floats apart.
template <typename T>
__device__ void load_rows(const void* p, int64_t base, int64_t stride, int width, int t0, int len, float* dst, int ld) {
  const T* x = static_cast<const T*>(p) + base;
  for (int e = threadIdx.x; e < kL * width; e += kThreads) {
    const int i = e / width, j = e % width;
    dst[i * ld + j] = t0 + i < len ? to_f32(x[(t0 + i) * stride + j]) : 0.f;
  }
}

// blockIdx.y = 0: sum_j exp(l_L - l_j) D_j k_j v_j^T;  1: sum_i exp(l_i) q_i u_i^T, `other` floats behind.
template <typename T>
__global__ void __launch_bounds__(kThreads) ssm_chunk_sum_kernel(SsmArgs A, float* states, int64_t other, float* tot,
                                                                 int nc) {
  const bool rev = blockIdx.y == 1;
  extern __shared__ float sm[];
  __shared__ Decays dc;
  const int64_t id = blockIdx.x;
  const int c = static_cast<int>(id % nc), bn = static_cast<int>(id / nc), b = bn / A.N, n = bn % A.N;
  const int g = n / (A.N / A.G), len = ssm_len(A, b), t0 = c * kL, K = A.K, V = A.V;
  float *ra = sm, *rb = sm + kL * K;
  load_decays<T>(A, b, n, t0, len, dc);
  const int64_t row = static_cast<int64_t>(b) * A.T;
  if (rev) {
    load_rows<T>(A.q, row * A.q_stride + static_cast<int64_t>(g) * K, A.q_stride, K, t0, len, ra, K);
    load_rows<T>(A.dy, (row * A.N + n) * V, static_cast<int64_t>(A.N) * V, V, t0, len, rb, V);
  } else {
    load_rows<T>(A.k, row * A.k_stride + static_cast<int64_t>(g) * K, A.k_stride, K, t0, len, ra, K);
    load_rows<T>(A.v, row * A.v_stride + static_cast<int64_t>(n) * V, A.v_stride, V, t0, len, rb, V);
  }
  __syncthreads();
  float* out = states + (rev ? other : 0) + id * K * V;
  for (int e = threadIdx.x; e < K * V; e += kThreads) {
    const int kk = e / V, vv = e % V;
    float s = 0.f;
#pragma unroll 8
    for (int j = 0; j < kL; ++j) {
      const float w = rev ? dc.first[j] : dc.last[j] * dc.D[j];
      s = fmaf(ra[j * K + kk] * w, rb[j * V + vv], s);
    }
    out[e] = s;
  }
  if (!rev && threadIdx.x == 0) tot[id] = dc.tot;
}

// In place: chunk sums -> the state before each chunk (blockIdx.z = 1, for
// the sums `other` floats behind: the state gradient behind each chunk), and
// the state (gradient) at the other end.
__global__ void __launch_bounds__(kThreads) ssm_chunk_scan_kernel(float* states, int64_t other, const float* tot,
                                                                  const float* H_0, float* H_T, const float* dH_T,
                                                                  float* dH_0, int nc, int KV) {
  constexpr int kAhead = 8;  // chunks' loads in flight: the walk itself is one FMA a chunk
  const bool rev = blockIdx.z == 1;
  const int e = blockIdx.y * kThreads + threadIdx.x;
  const int64_t bn = blockIdx.x;
  if (e >= KV) return;
  const float* from = rev ? dH_T : H_0;
  float* to = rev ? dH_0 : H_T;
  float cur = from ? from[bn * KV + e] : 0.f;
  float* st = states + (rev ? other : 0) + bn * nc * KV + e;
  const float* tt = tot + bn * nc;
  for (int i = 0; i < nc; i += kAhead) {
    float u[kAhead], a[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= nc) continue;
      const int c = rev ? nc - 1 - i - j : i + j;
      u[j] = st[static_cast<int64_t>(c) * KV];
      a[j] = tt[c];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= nc) continue;
      const int c = rev ? nc - 1 - i - j : i + j;
      st[static_cast<int64_t>(c) * KV] = cur;
      cur = fmaf(a[j], cur, u[j]);
    }
  }
  if (to != nullptr) to[bn * KV + e] = cur;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ssm_chunk_out_kernel(SsmArgs A, const float* states, int nc) {
  extern __shared__ float sm[];
  __shared__ Decays dc;
  __shared__ float P[kL][kL + 1];
  const int64_t id = blockIdx.x;
  const int c = static_cast<int>(id % nc), bn = static_cast<int>(id / nc), b = bn / A.N, n = bn % A.N;
  const int g = n / (A.N / A.G), len = ssm_len(A, b), t0 = c * kL, K = A.K, V = A.V, ld = K + 1;
  float *sq = sm, *sk = sq + kL * ld, *sv = sk + kL * ld;
  const int64_t row = static_cast<int64_t>(b) * A.T;
  load_decays<T>(A, b, n, t0, len, dc);
  load_rows<T>(A.q, row * A.q_stride + static_cast<int64_t>(g) * K, A.q_stride, K, t0, len, sq, ld);
  load_rows<T>(A.k, row * A.k_stride + static_cast<int64_t>(g) * K, A.k_stride, K, t0, len, sk, ld);
  load_rows<T>(A.v, row * A.v_stride + static_cast<int64_t>(n) * V, A.v_stride, V, t0, len, sv, V);
  __syncthreads();
  for (int e = threadIdx.x; e < kL * kL; e += kThreads) {
    const int i = e / kL, j = e % kL;
    float s = 0.f;
    if (i >= j) {
      for (int x = 0; x < K; ++x) s = fmaf(sq[i * ld + x], sk[j * ld + x], s);
      s *= decay(dc, i, j) * dc.D[j];
    }
    P[i][j] = s;
  }
  __syncthreads();
  const float* S = states + id * K * V;
  T* y = static_cast<T*>(A.y);
  for (int e = threadIdx.x; e < kL * V; e += kThreads) {
    const int i = e / V, vv = e % V;
    if (t0 + i >= A.T) break;
    float r = 0.f;
    if (t0 + i < len) {
      for (int x = 0; x < K; ++x) r = fmaf(sq[i * ld + x], S[x * V + vv], r);
      r *= dc.first[i];
      for (int j = 0; j <= i; ++j) r = fmaf(P[i][j], sv[j * V + vv], r);
      if (A.w_r) r = fmaf(to_f32(static_cast<const T*>(A.w_r)[n * V + vv]), sv[i * V + vv], r);
    }
    y[((row + t0 + i) * A.N + n) * V + vv] = from_f32<T>(r);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ssm_chunk_grad_kernel(SsmArgs A, const float* states, const float* rstates,
                                                                  SsmGradOut o, int nc) {
  extern __shared__ float sm[];
  __shared__ Decays dc;
  __shared__ float P[kL][kL + 1], dP[kL][kL + 1], qd[kL], ck[kL], ci[kL], red[kThreads / 32];
  const int64_t id = blockIdx.x;
  const int c = static_cast<int>(id % nc), bn = static_cast<int>(id / nc), b = bn / A.N, n = bn % A.N;
  const int g = n / (A.N / A.G), len = ssm_len(A, b), t0 = c * kL, K = A.K, V = A.V, lk = K + 1, lv = V + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *sq = sm, *sk = sq + kL * lk, *sv = sk + kL * lk, *su = sv + kL * lv, *sS = su + kL * lv, *sX = sS + K * lv,
        *sY = sX + kL * lk;
  const int64_t row = static_cast<int64_t>(b) * A.T, KV = static_cast<int64_t>(K) * V;
  load_decays<T>(A, b, n, t0, len, dc);
  load_rows<T>(A.q, row * A.q_stride + static_cast<int64_t>(g) * K, A.q_stride, K, t0, len, sq, lk);
  load_rows<T>(A.k, row * A.k_stride + static_cast<int64_t>(g) * K, A.k_stride, K, t0, len, sk, lk);
  load_rows<T>(A.v, row * A.v_stride + static_cast<int64_t>(n) * V, A.v_stride, V, t0, len, sv, lv);
  load_rows<T>(A.dy, (row * A.N + n) * V, static_cast<int64_t>(A.N) * V, V, t0, len, su, lv);
  for (int e = tid; e < KV; e += kThreads) sS[(e / V) * lv + e % V] = states[id * KV + e];
  __syncthreads();
  for (int e = tid; e < kL * kL; e += kThreads) {
    const int i = e / kL, j = e % kL;
    float s = 0.f, d = 0.f;
    if (i >= j) {
      for (int x = 0; x < K; ++x) s = fmaf(sq[i * lk + x], sk[j * lk + x], s);
      for (int x = 0; x < V; ++x) d = fmaf(su[i * lv + x], sv[j * lv + x], d);
      const float E = decay(dc, i, j);
      s *= E;
      d *= E;
    }
    P[i][j] = s;
    dP[i][j] = d;
  }
  __syncthreads();
  for (int e = tid; e < kL * K; e += kThreads) {  // dq
    const int i = e / K, kk = e % K;
    float r = 0.f;
    for (int x = 0; x < V; ++x) r = fmaf(sS[kk * lv + x], su[i * lv + x], r);
    r *= dc.first[i];
    for (int j = 0; j <= i; ++j) r = fmaf(dP[i][j] * dc.D[j], sk[j * lk + kk], r);
    if (t0 + i >= len) r = 0.f;
    sX[i * lk + kk] = r;
    if (t0 + i < A.T) o.dq[((row + t0 + i) * o.qk_heads + (o.qk_heads == A.N ? n : g)) * K + kk] = r;
  }
  __syncthreads();
  for (int i = warp; i < kL; i += kThreads / 32) {
    float s = 0.f;
    for (int x = lane; x < K; x += 32) s = fmaf(sq[i * lk + x], sX[i * lk + x], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (lane == 0) qd[i] = s;
  }
  // R replaces S; <R, S> on the way.
  float rs = 0.f;
  for (int e = tid; e < KV; e += kThreads) {
    float& x = sS[(e / V) * lv + e % V];
    const float r = rstates[id * KV + e];
    rs = fmaf(r, x, rs);
    x = r;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, w);
  if (lane == 0) red[warp] = rs;
  __syncthreads();
  for (int e = tid; e < kL * K; e += kThreads) {  // dk
    const int j = e / K, kk = e % K;
    float r = 0.f;
    for (int x = 0; x < V; ++x) r = fmaf(sS[kk * lv + x], sv[j * lv + x], r);
    r *= dc.last[j];
    sY[j * lk + kk] = r;
    for (int i = j; i < kL; ++i) r = fmaf(dP[i][j], sq[i * lk + kk], r);
    sX[j * lk + kk] = r;
    if (t0 + j < A.T) o.dk[((row + t0 + j) * o.qk_heads + (o.qk_heads == A.N ? n : g)) * K + kk] =
        t0 + j < len ? dc.D[j] * r : 0.f;
  }
  for (int e = tid; e < kL * V; e += kThreads) {  // dv
    const int j = e / V, vv = e % V;
    float r = 0.f;
    for (int x = 0; x < K; ++x) r = fmaf(sk[j * lk + x], sS[x * lv + vv], r);
    r *= dc.last[j];
    for (int i = j; i < kL; ++i) r = fmaf(P[i][j], su[i * lv + vv], r);
    r *= dc.D[j];
    if (A.w_r) r = fmaf(to_f32(static_cast<const T*>(A.w_r)[n * V + vv]), su[j * lv + vv], r);
    if (t0 + j >= len) r = 0.f;
    if (t0 + j < A.T) A.dv[((row + t0 + j) * A.N + n) * V + vv] = r;
  }
  if (o.wr_part != nullptr)
    for (int vv = tid; vv < V; vv += kThreads) {
      float r = 0.f;
      for (int j = 0; j < kL; ++j) r = fmaf(su[j * lv + vv], sv[j * lv + vv], r);
      o.wr_part[id * V + vv] = r;
    }
  __syncthreads();
  for (int i = warp; i < kL; i += kThreads / 32) {
    float s = 0.f, s2 = 0.f;
    for (int x = lane; x < K; x += 32) {
      s = fmaf(sk[i * lk + x], sX[i * lk + x], s);
      s2 = fmaf(sk[i * lk + x], sY[i * lk + x], s2);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, w);
      s2 += __shfl_xor_sync(0xffffffffu, s2, w);
    }
    if (lane == 0) {
      ck[i] = s;
      ci[i] = s2;
    }
  }
  __syncthreads();
  if (warp == 0) {
    float r = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) r += red[w];
    const float D = dc.D[lane];
    float s = D * ci[lane];
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float end = fmaf(dc.tot, r, s);
    float x = qd[lane] - D * ck[lane];
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const float p = __shfl_down_sync(0xffffffffu, x, w);
      if (lane + w < 32) x += p;
    }
    const float gt = x + end;
    const bool live = t0 + lane < len;
    const float dd = live ? (ck[lane] + A.A[n] * gt) * dc.sg[lane] : 0.f;
    if (t0 + lane < A.T) A.ddt[(row + t0 + lane) * A.N + n] = dd;
    float pa = live ? D * gt : 0.f, pb = dd;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      pa += __shfl_xor_sync(0xffffffffu, pa, w);
      pb += __shfl_xor_sync(0xffffffffu, pb, w);
    }
    if (lane == 0) o.ab_part[id] = make_float2(pa, pb);
  }
}

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
// by HBM (8 bytes per state element) at large batches, by latency at small.
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

// Shared memory at K = V = 128.
constexpr int kMaxOut = sizeof(float) * kL * (2 * 129 + 128);
constexpr int kMaxGrad = sizeof(float) * (kL * (4 * 129 + 2 * 129) + 128 * 129);

template <typename T>
cudaError_t forward_simt(const SsmArgs& a, cudaStream_t s) {
  const int nc = (a.T + kL - 1) / kL, KV = a.K * a.V;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.N * nc;
  float* states = static_cast<float*>(a.ws);
  float* tot = states + blocks * KV;
  const size_t sm1 = sizeof(float) * kL * (a.K + a.V), sm2 = sizeof(float) * kL * (2 * (a.K + 1) + a.V);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_chunk_out_kernel<T>), kMaxOut, done);
  if (e != cudaSuccess) return e;
  ssm_chunk_sum_kernel<T><<<static_cast<unsigned>(blocks), kThreads, sm1, s>>>(a, states, 0, tot, nc);
  ssm_chunk_scan_kernel<<<dim3(a.B * a.N, (KV + kThreads - 1) / kThreads), kThreads, 0, s>>>(
      states, 0, tot, a.H_0, a.H_T, nullptr, nullptr, nc, KV);
  ssm_chunk_out_kernel<T><<<static_cast<unsigned>(blocks), kThreads, sm2, s>>>(a, states, nc);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_simt(const SsmArgs& a, cudaStream_t s) {
  const int nc = (a.T + kL - 1) / kL, KV = a.K * a.V;
  const int64_t blocks = static_cast<int64_t>(a.B) * a.N * nc, heads = static_cast<int64_t>(a.B) * a.T * a.N * a.K;
  float* states = static_cast<float*>(a.ws);
  float* rstates = states + blocks * KV;
  float2* ab = reinterpret_cast<float2*>(rstates + blocks * KV);
  float* tot = reinterpret_cast<float*>(ab + blocks);
  float* wr = tot + blocks;
  float* dqh = wr + blocks * a.V;
  float* dkh = dqh + heads;
  SsmGradOut o{a.dq, a.dk, a.dw_r ? wr : nullptr, ab, a.N};
  if (a.G != a.N) {
    o.dq = dqh;
    o.dk = dkh;
  }
  const size_t sm1 = sizeof(float) * kL * (a.K + a.V);
  const size_t sm2 = sizeof(float) * (kL * (4 * (a.K + 1) + 2 * (a.V + 1)) + a.K * (a.V + 1));
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_chunk_grad_kernel<T>), kMaxGrad, done);
  if (e != cudaSuccess) return e;
  ssm_chunk_sum_kernel<T><<<dim3(static_cast<unsigned>(blocks), 2), kThreads, sm1, s>>>(a, states, blocks * KV, tot, nc);
  ssm_chunk_scan_kernel<<<dim3(a.B * a.N, (KV + kThreads - 1) / kThreads, 2), kThreads, 0, s>>>(
      states, blocks * KV, tot, a.H_0, nullptr, a.dH_T, a.dH_0, nc, KV);
  ssm_chunk_grad_kernel<T><<<static_cast<unsigned>(blocks), kThreads, sm2, s>>>(a, states, rstates, o, nc);
  return launch_ssm_grad_sums(a, o, nc, s);
}

}  // namespace

cudaError_t launch_ssm_grad_sums(const SsmArgs& a, const SsmGradOut& o, int nc, cudaStream_t s) {
  ssm_grad_sums_kernel<<<dim3(a.N, a.dw_r != nullptr ? 1 + (a.V + 31) / 32 : 1), kSumThreads, 0, s>>>(
      o.ab_part, o.wr_part, a.dA, a.ddt_bias, a.dw_r, a.B, a.N, nc, a.V);
  if (a.G != a.N) {
    const int64_t n = static_cast<int64_t>(a.B) * a.T * a.G * a.K;
    ssm_sum_heads_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(
        o.dq, o.dk, a.dq, a.dk, n, a.N, a.G, a.K);
  }
  return cudaGetLastError();
}

size_t ssm_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, bool bf16) {
  if (bf16) return align256(ssm_mma_forward_scratch_bytes(B, T, N, K, V));
  const size_t blocks = static_cast<size_t>(B) * N * ((T + kL - 1) / kL);
  return align256(sizeof(float) * blocks * (static_cast<size_t>(K) * V + 1));
}

size_t ssm_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V, bool bf16) {
  if (bf16) return align256(ssm_mma_backward_scratch_bytes(B, T, N, G, K, V));
  const size_t blocks = static_cast<size_t>(B) * N * ((T + kL - 1) / kL);
  const size_t heads = G == N ? 0 : 2 * static_cast<size_t>(B) * T * N * K;
  return align256(sizeof(float) * (blocks * (2 * static_cast<size_t>(K) * V + 3 + V) + heads));
}

cudaError_t launch_ssm_forward(const SsmArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_ssm_mma_forward(a, s) : forward_simt<float>(a, s);
}

cudaError_t launch_ssm_backward(const SsmArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_ssm_mma_backward(a, s) : backward_simt<float>(a, s);
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
