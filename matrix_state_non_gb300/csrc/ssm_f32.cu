// Selective state space scan on fp32 inputs, on CUDA cores (the mathematics in
// ssm.cu): chunk sums -> scan over the chunks -> outputs or gradients, each
// chunk on its own block.  A chunk's products are small matrix products from
// shared memory, 4 x 4 results to a thread (a few at the edges fewer), eight
// 16-byte loads for 64 FMAs.  Chunks have 64 steps forward, where the states'
// traffic counts, and 32 backward, where shared memory holds twice as much.
// Bound by shared-memory loads and FMAs: B=4 heads=8 T=4096 64x64 forward
// 231 us (19 TFLOP/s of chunk products; one result to a thread took 821),
// T=2048 backward 403 us (685; the sums of W, see ssm.cu, are 8 of them).
#include <cuda_runtime.h>

#include <cstdint>

#include "gate.cuh"
#include "layer.cuh"
#include "ssm.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;
constexpr int kFwd = 64, kBwd = 32;  // steps per chunk

// Floats between the rows of a tile of `width` columns: a multiple of four
// whose quarter is odd, so that 16-byte loads down a column of rows start on
// eight different banks.
__host__ __device__ constexpr int pitch(int width) { return ((width + 3) / 4 | 1) * 4; }

// The chunk's decays, in shared memory.
template <int L>
struct Decays {
  float D[L];               // step sizes (0 behind the sequence's end)
  float sg[L];              // sigmoid(dt + dt_bias)
  float hi[L], lo[L];       // l_i as hi + lo: differences of long sums keep their bits
  float first[L], last[L];  // exp(l_i), exp(l_L - l_i)
  float tot;                // exp(l_L)
};

// By the first warp, L / 32 consecutive steps a lane.
template <int L>
__device__ void load_decays(const SsmArgs& A, int b, int n, int t0, int len, Decays<L>& d) {
  constexpr int kPer = L / 32;
  const int lane = threadIdx.x;
  if (lane >= 32) return;
  const float An = A.A[n], bias = A.dt_bias ? A.dt_bias[n] : 0.f;
  double l[kPer], sum = 0.;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = lane * kPer + e;
    float D = 0.f, sg = 0.f;
    if (t0 + i < len) {
      const float x = static_cast<const float*>(A.dt)[(static_cast<int64_t>(b) * A.T + t0 + i) * A.dt_stride + n] + bias;
      D = softplus_f(x);
      sg = 1.f / (1.f + expf(-x));
    }
    d.D[i] = D;
    d.sg[i] = sg;
    sum += log_decay<double>(D, An);
    l[e] = sum;
  }
  double up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double p = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += p;
  }
  const double end = __shfl_sync(0xffffffffu, up, 31);
  double before = __shfl_up_sync(0xffffffffu, up, 1);  // not up - sum: a NaN stays behind its step
  if (lane == 0) before = 0.;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = lane * kPer + e;
    const double x = before + l[e];
    d.hi[i] = static_cast<float>(x);
    d.lo[i] = static_cast<float>(x - d.hi[i]);
    d.first[i] = expf(static_cast<float>(x));
    d.last[i] = expf(static_cast<float>(end - x));
  }
  if (lane == 0) d.tot = expf(static_cast<float>(end));
}

template <int L>
__device__ __forceinline__ float decay(const Decays<L>& d, int i, int j) {
  return expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
}

// Rows of a head into a tile, zero behind `live` rows and in the padding.  True where the thread met a value that is
// not finite.
__device__ bool load_rows(const float* x, int64_t stride, int width, int rows, int live, float* dst) {
  const int ld = pitch(width);
  bool bad = false;
  for (int e = threadIdx.x; e < rows * ld; e += kThreads) {
    const int i = e / ld, j = e - i * ld;
    const float v = i < live && j < width ? x[i * stride + j] : 0.f;
    bad |= !isfinite(v);
    dst[e] = v;
  }
  return bad;
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void axpy4(float (&c)[4], float a, const float4& b) {
  fma2(c[0], c[1], a, a, b.x, b.y);
  fma2(c[2], c[3], a, a, b.z, b.w);
}

// Products of tiles, all in the layout of load_rows.  f(r, c, x) receives
// four results of row r, columns c .. c + 3 (rows < `rows`; columns padded to a
// multiple of four).  Threads take R x 4 blocks, rows `rows` / R apart.
//   kNN: x = sum_i A[r][i] B[i][c];  kNT: x = sum_i A[r][i] B[c][i];
//   kTN: x = sum_i A[i][r] B[i][c], R = 4 consecutive rows.
enum Form { kNN, kNT, kTN };

template <Form kForm, int R, typename F>
__device__ __forceinline__ void product_blocks(const float* A, int lda, const float* B, int ldb, int rows, int cols,
                                               int inner, F f) {
  const int rg = (rows + R - 1) / R, cg = (cols + 3) / 4;
  for (int it = threadIdx.x; it < rg * cg; it += kThreads) {
    const int r0 = it / cg, c0 = it - r0 * cg;
    float x[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
    if constexpr (kForm == kTN) {
      for (int i = 0; i < inner; ++i) {
        const float4 b = ld4(B + i * ldb + 4 * c0);
        if constexpr (R == 4) {
          const float4 a = ld4(A + i * lda + 4 * r0);
          axpy4(x[0], a.x, b);
          axpy4(x[1], a.y, b);
          axpy4(x[2], a.z, b);
          axpy4(x[3], a.w, b);
        }
      }
    } else {
      for (int i = 0; i < inner; i += 4) {
        float4 b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          b[e] = kForm == kNN ? ld4(B + (i + e) * ldb + 4 * c0) : ld4(B + min(c0 + e * cg, cols - 1) * ldb + i);
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const float4 a = ld4(A + (r0 + k * rg) * lda + i);
          if constexpr (kForm == kNN) {
            axpy4(x[k], a.x, b[0]);
            axpy4(x[k], a.y, b[1]);
            axpy4(x[k], a.z, b[2]);
            axpy4(x[k], a.w, b[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[k][e] = fmaf(a.w, b[e].w, fmaf(a.z, b[e].z, fmaf(a.y, b[e].y, fmaf(a.x, b[e].x, x[k][e]))));
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) f(kForm == kTN ? 4 * r0 + k : r0 + k * rg, c0, cg, x[k]);
  }
}

// Fewer rows to a thread where there are few columns, so that all threads work.
template <Form kForm, int kRows, typename F>
__device__ __forceinline__ void product(const float* A, int lda, const float* B, int ldb, int cols, int inner, F f) {
  const int cg = (cols + 3) / 4;
  if (kRows / 4 * cg >= kThreads)
    product_blocks<kForm, 4>(A, lda, B, ldb, kRows, cols, inner, f);
  else if (kRows / 2 * cg >= kThreads)
    product_blocks<kForm, 2>(A, lda, B, ldb, kRows, cols, inner, f);
  else
    product_blocks<kForm, 1>(A, lda, B, ldb, kRows, cols, inner, f);
}

// The columns of f's four results: consecutive for kNN, kTN; cg apart for kNT.
__device__ __forceinline__ int col_nn(int c0, int, int e) { return 4 * c0 + e; }
__device__ __forceinline__ int col_nt(int c0, int cg, int e) { return c0 + e * cg; }

struct Place {
  int b, n, g, c, t0, len, live;
  int64_t row;  // of the chunk's first step
};

template <int L>
__device__ __forceinline__ Place place(const SsmArgs& A, int nc) {
  Place p;
  const int bn = blockIdx.x / nc;
  p.c = blockIdx.x - bn * nc;
  p.b = bn / A.N;
  p.n = bn - p.b * A.N;
  p.g = p.n / (A.N / A.G);
  p.t0 = p.c * L;
  p.len = ssm_len(A, p.b);
  p.live = min(max(p.len - p.t0, 0), L);
  p.row = static_cast<int64_t>(p.b) * A.T + p.t0;
  return p;
}

__device__ __forceinline__ const float* q_rows(const SsmArgs& A, const Place& p) {
  return static_cast<const float*>(A.q) + p.row * A.q_stride + static_cast<int64_t>(p.g) * A.K;
}
__device__ __forceinline__ const float* k_rows(const SsmArgs& A, const Place& p) {
  return static_cast<const float*>(A.k) + p.row * A.k_stride + static_cast<int64_t>(p.g) * A.K;
}
__device__ __forceinline__ const float* v_rows(const SsmArgs& A, const Place& p) {
  return static_cast<const float*>(A.v) + p.row * A.v_stride + static_cast<int64_t>(p.n) * A.V;
}
__device__ __forceinline__ const float* u_rows(const SsmArgs& A, const Place& p) {
  return static_cast<const float*>(A.dy) + (p.row * A.N + p.n) * A.V;
}

// blockIdx.y = 0: sum_j exp(l_L - l_j) D_j k_j v_j^T;  1: sum_i exp(l_i) q_i u_i^T, `other` floats behind.
template <int L>
__global__ void __launch_bounds__(kThreads) ssm_chunk_sum_kernel(SsmArgs A, float* states, int64_t other, float* tot,
                                                                 int nc) {
  if (blockIdx.x == 0 && threadIdx.x < sizeof(StatusBlock) / 4) static_cast<unsigned*>(A.ws)[threadIdx.x] = 0u;
  extern __shared__ __align__(16) float sm[];
  __shared__ Decays<L> dc;
  const bool rev = blockIdx.y == 1;
  const Place p = place<L>(A, nc);
  const int K = A.K, V = A.V, lk = pitch(K), lv = pitch(V);
  float *ra = sm, *rb = sm + L * lk;
  load_decays<L>(A, p.b, p.n, p.t0, p.len, dc);
  load_rows(rev ? q_rows(A, p) : k_rows(A, p), rev ? A.q_stride : A.k_stride, K, L, p.live, ra);
  load_rows(rev ? u_rows(A, p) : v_rows(A, p), rev ? static_cast<int64_t>(A.N) * V : A.v_stride, V, L, p.live, rb);
  __syncthreads();
  for (int e = threadIdx.x; e < L * lk; e += kThreads) {
    const int j = e / lk;
    ra[e] *= rev ? dc.first[j] : dc.last[j] * dc.D[j];
  }
  __syncthreads();
  float* out = states + (rev ? other : 0) + static_cast<int64_t>(blockIdx.x) * K * V;
  product_blocks<kTN, 4>(ra, lk, rb, lv, K, V, L, [&](int r, int c0, int cg, const float (&x)[4]) {
    if (r >= K) return;
    if (V % 4 == 0) {
      *reinterpret_cast<float4*>(out + r * V + 4 * c0) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col_nn(c0, cg, e) < V) out[r * V + col_nn(c0, cg, e)] = x[e];
    }
  });
  if (!rev && threadIdx.x == 0) tot[blockIdx.x] = dc.tot;
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

// Scores f(i, j) x_i . y_j of a chunk; zero above the diagonal.
template <int L, typename F>
__device__ __forceinline__ void scores(const float* x, const float* y, int ld, int width, float* P, F f) {
  product<kNT, L>(x, ld, y, ld, L, width, [&](int i, int c0, int cg, const float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = col_nt(c0, cg, e);
      P[i * pitch(L) + j] = i >= j ? s[e] * f(i, j) : 0.f;
    }
  });
}

__global__ void __launch_bounds__(kThreads) ssm_chunk_out_kernel(SsmArgs A, const float* states, int nc) {
  constexpr int L = kFwd;
  extern __shared__ __align__(16) float sm[];
  __shared__ Decays<L> dc;
  __shared__ int s_from[128];  // the first step at which a value column is not finite
  const Place p = place<L>(A, nc);
  const int K = A.K, V = A.V, lk = pitch(K), lv = pitch(V);
  float *sq = sm, *sk = sq + L * lk, *sv = sk + L * lk, *P = sv + L * lv, *sS = P + L * pitch(L);
  float* y = static_cast<float*>(A.y) + (p.row * A.N + p.n) * V;
  const int64_t stride = static_cast<int64_t>(A.N) * V;
  if (p.live == 0) {
    for (int e = threadIdx.x; e < min(L, A.T - p.t0) * V; e += kThreads) y[(e / V) * stride + e % V] = 0.f;
    return;
  }
  load_decays<L>(A, p.b, p.n, p.t0, p.len, dc);
  load_rows(q_rows(A, p), A.q_stride, K, L, p.live, sq);
  load_rows(k_rows(A, p), A.k_stride, K, L, p.live, sk);
  const bool bad = load_rows(v_rows(A, p), A.v_stride, V, L, p.live, sv);
  load_rows(states + static_cast<int64_t>(blockIdx.x) * K * V, V, V, (K + 3) / 4 * 4, K, sS);
  // Values that are not finite make their column NaN from their step on; the product with the scores, in which a later
  // step's zero score would make NaN of them for the steps before, takes zeros in their place.
  const bool spoilt = __syncthreads_or(bad);
  if (spoilt) {
    for (int c = threadIdx.x; c < V; c += kThreads) {
      int from = L;
      for (int j = L - 1; j >= 0; --j) {
        if (isfinite(sv[j * lv + c])) continue;
        from = j;
        sv[j * lv + c] = 0.f;
      }
      s_from[c] = from;
    }
    __syncthreads();
  }
  scores<L>(sq, sk, lk, K, P, [&](int i, int j) { return decay(dc, i, j) * dc.D[j]; });
  __syncthreads();
  // The rows of y twice: q S, kept in the q tile's place by the same thread, then the scores times v.
  const float* wr = A.w_r ? static_cast<const float*>(A.w_r) + static_cast<int64_t>(p.n) * V : nullptr;
  float* O = sS + (K + 3) / 4 * 4 * lv;
  product<kNN, L>(sq, lk, sS, lv, V, (K + 3) / 4 * 4, [&](int i, int c0, int, const float (&x)[4]) {
    *reinterpret_cast<float4*>(O + i * lv + 4 * c0) =
        make_float4(x[0] * dc.first[i], x[1] * dc.first[i], x[2] * dc.first[i], x[3] * dc.first[i]);
  });
  product<kNN, L>(P, pitch(L), sv, lv, V, L, [&](int i, int c0, int cg, const float (&x)[4]) {
    if (p.t0 + i >= A.T) return;
    const float4 o = ld4(O + i * lv + 4 * c0), v = ld4(sv + i * lv + 4 * c0);
    const float oo[4] = {o.x, o.y, o.z, o.w}, vv[4] = {v.x, v.y, v.z, v.w};
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col_nn(c0, cg, e);
      r[e] = x[e] + oo[e];
      if (wr && c < V) r[e] = fmaf(wr[c], vv[e], r[e]);
      if (spoilt && c < V && i >= s_from[c]) r[e] = __int_as_float(0x7FFFFFFF);
      if (i >= p.live) r[e] = 0.f;
    }
    float* at = y + i * stride + 4 * c0;
    if (V % 4 == 0) {
      *reinterpret_cast<float4*>(at) = make_float4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * c0 + e < V) at[e] = r[e];
    }
  });
}

__global__ void __launch_bounds__(kThreads) ssm_chunk_grad_kernel(SsmArgs A, const float* states, const float* rstates,
                                                                  SsmGradOut o, int nc) {
  constexpr int L = kBwd, lp = pitch(L);
  extern __shared__ __align__(16) float sm[];
  __shared__ Decays<L> dc;
  __shared__ float sd[L], ck[L], ci[L], red[kThreads / 32];
  __shared__ Sum2 w_row[L], w_col[kThreads / 32][L];
  const Place p = place<L>(A, nc);
  const int K = A.K, V = A.V, lk = pitch(K), lv = pitch(V), K4 = (K + 3) / 4 * 4, V4 = (V + 3) / 4 * 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t KV = static_cast<int64_t>(K) * V, id = blockIdx.x;
  const int64_t qk_stride = static_cast<int64_t>(o.qk_heads) * K, v_stride = static_cast<int64_t>(A.N) * V;
  const int qk_head = o.qk_heads == A.N ? p.n : p.g, rows = min(L, A.T - p.t0);
  float* dq = o.dq + p.row * qk_stride + static_cast<int64_t>(qk_head) * K;
  float* dk = o.dk + p.row * qk_stride + static_cast<int64_t>(qk_head) * K;
  float* dv = A.dv + p.row * v_stride + static_cast<int64_t>(p.n) * V;
  float* ddt = A.ddt + p.row * A.N + p.n;
  float *sq = sm, *sk = sq + L * lk, *sv = sk + L * lk, *su = sv + L * lv, *P = su + L * lv, *dP = P + L * lp,
        *sX = dP + L * lp, *sY = sX + L * lk, *sS = sY + L * (lk > lv ? lk : lv);
  load_decays<L>(A, p.b, p.n, p.t0, p.len, dc);
  load_rows(q_rows(A, p), A.q_stride, K, L, p.live, sq);
  load_rows(k_rows(A, p), A.k_stride, K, L, p.live, sk);
  load_rows(v_rows(A, p), A.v_stride, V, L, p.live, sv);
  load_rows(u_rows(A, p), v_stride, V, L, p.live, su);
  load_rows(states + id * KV, V, V, K4, K, sS);
  __syncthreads();
  scores<L>(sq, sk, lk, K, P, [](int, int) { return 1.f; });
  scores<L>(su, sv, lv, V, dP, [&](int i, int j) { return decay(dc, i, j); });
  __syncthreads();
  {  // W's sums along rows and columns, a lane a column; P takes its decays.
    static_assert(L == 32, "a lane a column");
    Sum2 col;
    for (int i = warp; i < L; i += kThreads / 32) {
      float& x = P[i * lp + lane];
      const float w = lane < i ? x * dP[i * lp + lane] * dc.D[lane] : 0.f;
      Sum2 row;
      row.add(w);
      col.add(w);
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) row.add(row.across(m));
      if (lane == 0) w_row[i] = row;
      if (lane <= i) x *= decay(dc, i, lane);
    }
    w_col[warp][lane] = col;
  }
  auto row_dots = [&](const float* a, const float* b, float* out) {  // rows of two K-wide tiles
    for (int i = warp; i < L; i += kThreads / 32) {
      float s = 0.f;
      for (int x = lane; x < K; x += 32) s = fmaf(a[i * lk + x], b[i * lk + x], s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      if (lane == 0) out[i] = s;
    }
  };
  // dq_i = first_i S u_i + sum_j E_ij D_j (u_i . v_j) k_j
  product<kNT, L>(su, lv, sS, lv, K, V4, [&](int i, int c0, int cg, const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col_nt(c0, cg, e) < K) sX[i * lk + col_nt(c0, cg, e)] = x[e] * dc.first[i];
  });
  __syncthreads();
  row_dots(sq, sX, sd);
  for (int e = tid; e < L * lk; e += kThreads) sY[e] = sk[e] * dc.D[e / lk];
  __syncthreads();
  product<kNN, L>(dP, lp, sY, lk, K, L, [&](int i, int c0, int cg, const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col_nn(c0, cg, e);
      if (c >= K) continue;
      const float r = i < p.live ? x[e] + sX[i * lk + c] : 0.f;
      sX[i * lk + c] = r;
      if (i < rows) dq[i * qk_stride + c] = r;
    }
  });
  // R takes S's place; <R, S> on the way.
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
  if (o.wr_part != nullptr)
    for (int vv = tid; vv < V; vv += kThreads) {
      float r = 0.f;
      for (int j = 0; j < L; ++j) r = fmaf(su[j * lv + vv], sv[j * lv + vv], r);
      o.wr_part[id * V + vv] = r;
    }
  __syncthreads();
  // zk_j = last_j R v_j + sum_i E_ij (u_i . v_j) q_i
  product<kNT, L>(sv, lv, sS, lv, K, V4, [&](int j, int c0, int cg, const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col_nt(c0, cg, e) < K) sX[j * lk + col_nt(c0, cg, e)] = x[e] * dc.last[j];
  });
  __syncthreads();
  row_dots(sk, sX, ci);
  __syncthreads();
  product_blocks<kTN, 4>(dP, lp, sq, lk, L, K, L, [&](int j, int c0, int cg, const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col_nn(c0, cg, e);
      if (c >= K) continue;
      const float r = x[e] + sX[j * lk + c];
      sX[j * lk + c] = r;
      if (j < rows) dk[j * qk_stride + c] = j < p.live ? dc.D[j] * r : 0.f;
    }
  });
  __syncthreads();
  row_dots(sk, sX, ck);
  // zv_j = last_j R^T k_j + sum_i E_ij (q_i . k_j) u_i
  product<kNN, L>(sk, lk, sS, lv, V, K4, [&](int j, int c0, int, const float (&x)[4]) {
    *reinterpret_cast<float4*>(sY + j * lv + 4 * c0) =
        make_float4(x[0] * dc.last[j], x[1] * dc.last[j], x[2] * dc.last[j], x[3] * dc.last[j]);
  });
  __syncthreads();
  const float* wr = A.w_r ? static_cast<const float*>(A.w_r) + static_cast<int64_t>(p.n) * V : nullptr;
  product_blocks<kTN, 4>(P, lp, su, lv, L, V, L, [&](int j, int c0, int cg, const float (&x)[4]) {
    if (j >= rows) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col_nn(c0, cg, e);
      if (c >= V) continue;
      float r = dc.D[j] * (x[e] + sY[j * lv + c]);
      if (wr) r = fmaf(wr[c], su[j * lv + c], r);
      dv[j * v_stride + c] = j < p.live ? r : 0.f;
    }
  });
  __syncthreads();
  if (warp != 0) return;
  float r = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) r += red[w];
  const float D = dc.D[lane], from = D * ci[lane];
  Sum2 end, g;  // <R, S'>; g_t
  end.add(from);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) end.add(end.across(m));
  end.add(dc.tot * r);
  g.add(sd[lane]);
  g.add(w_row[lane]);
  for (int w = 0; w < kThreads / 32; ++w) g.subtract(w_col[w][lane]);
  g.add(-from);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) g.add(g.after(m));
  g.add(end);
  const float gt = g.value();
  const bool live = lane < p.live;
  const float dd = live ? (ck[lane] + A.A[p.n] * gt) * dc.sg[lane] : 0.f;
  if (lane < rows) ddt[static_cast<int64_t>(lane) * A.N] = dd;
  float pa = live ? D * gt : 0.f, pb = dd;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    pa += __shfl_xor_sync(0xffffffffu, pa, w);
    pb += __shfl_xor_sync(0xffffffffu, pb, w);
  }
  if (lane == 0) o.ab_part[id] = make_float2(pa, pb);
}

int sum_floats(int L, int K, int V) { return L * (pitch(K) + pitch(V)); }
int out_floats(int K, int V) {
  return kFwd * (2 * pitch(K) + 2 * pitch(V) + pitch(kFwd)) + (K + 3) / 4 * 4 * pitch(V);
}
int grad_floats(int K, int V) {
  const int lk = pitch(K), lv = pitch(V);
  return kBwd * (3 * lk + 2 * lv + 2 * pitch(kBwd) + (lk > lv ? lk : lv)) + (K + 3) / 4 * 4 * lv;
}

int64_t chunks_of(int64_t B, int64_t T, int64_t N, int L) { return B * N * ((T + L - 1) / L); }

}  // namespace

size_t ssm_f32_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  return sizeof(StatusBlock) + sizeof(float) * static_cast<size_t>(chunks_of(B, T, N, kFwd)) * (static_cast<size_t>(K) * V + 1);
}

size_t ssm_f32_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V) {
  const size_t heads = G == N ? 0 : 2 * static_cast<size_t>(B) * T * N * K;
  return sizeof(StatusBlock) + sizeof(float) * (static_cast<size_t>(chunks_of(B, T, N, kBwd)) * (2 * static_cast<size_t>(K) * V + 3 + V) + heads);
}

cudaError_t launch_ssm_f32_forward(const SsmArgs& a, cudaStream_t s) {
  const int nc = (a.T + kFwd - 1) / kFwd, KV = a.K * a.V;
  const int64_t blocks = chunks_of(a.B, a.T, a.N, kFwd);
  float* states = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + sizeof(StatusBlock));
  float* tot = states + blocks * KV;
  static std::atomic<uint64_t> sum{0}, out{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_chunk_sum_kernel<kFwd>), 4 * sum_floats(kFwd, 128, 128), sum);
  if (e == cudaSuccess)
    e = allow_smem(reinterpret_cast<const void*>(ssm_chunk_out_kernel), 4 * out_floats(128, 128), out);
  if (e != cudaSuccess) return e;
  ssm_chunk_sum_kernel<kFwd>
      <<<static_cast<unsigned>(blocks), kThreads, 4 * sum_floats(kFwd, a.K, a.V), s>>>(a, states, 0, tot, nc);
  ssm_chunk_scan_kernel<<<dim3(a.B * a.N, (KV + kThreads - 1) / kThreads), kThreads, 0, s>>>(
      states, 0, tot, a.H_0, a.H_T, nullptr, nullptr, nc, KV);
  ssm_chunk_out_kernel<<<static_cast<unsigned>(blocks), kThreads, 4 * out_floats(a.K, a.V), s>>>(a, states, nc);
  return cudaGetLastError();
}

cudaError_t launch_ssm_f32_backward(const SsmArgs& a, cudaStream_t s) {
  const int nc = (a.T + kBwd - 1) / kBwd, KV = a.K * a.V;
  const int64_t blocks = chunks_of(a.B, a.T, a.N, kBwd), heads = static_cast<int64_t>(a.B) * a.T * a.N * a.K;
  float* states = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + sizeof(StatusBlock));
  float* rstates = states + blocks * KV;
  float2* ab = reinterpret_cast<float2*>(rstates + blocks * KV);
  float* tot = reinterpret_cast<float*>(ab + blocks);
  float* wr = tot + blocks;
  float* dqh = wr + blocks * a.V;
  SsmGradOut o{a.dq, a.dk, a.dw_r ? wr : nullptr, ab, a.N};
  if (a.G != a.N) {
    o.dq = dqh;
    o.dk = dqh + heads;
  }
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_chunk_grad_kernel), 4 * grad_floats(128, 128), done);
  if (e != cudaSuccess) return e;
  ssm_chunk_sum_kernel<kBwd><<<dim3(static_cast<unsigned>(blocks), 2), kThreads, 4 * sum_floats(kBwd, a.K, a.V), s>>>(
      a, states, blocks * KV, tot, nc);
  ssm_chunk_scan_kernel<<<dim3(a.B * a.N, (KV + kThreads - 1) / kThreads, 2), kThreads, 0, s>>>(
      states, blocks * KV, tot, a.H_0, nullptr, a.dH_T, a.dH_0, nc, KV);
  ssm_chunk_grad_kernel<<<static_cast<unsigned>(blocks), kThreads, 4 * grad_floats(a.K, a.V), s>>>(a, states, rstates, o,
                                                                                               nc);
  return launch_ssm_grad_sums(a, o, nc, s);
}

}  // namespace m2rnn
