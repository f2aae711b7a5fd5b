// Short causal depthwise convolution with bias and SiLU, the layer that makes
// q, k and v from their projections ("M2RNN: Non-Linear RNNs with Matrix-
// Valued States for Scalable Language Modeling", Eq. 14-23 of the reading
// notes; width 4 there).  With xs = [x0 | x] along time (x0: the W - 1 inputs
// before the sequence, zero when not given), per channel c,
//     pre_t = b[c] + sum_w w[c][w] xs[t + w],   y_t = pre_t sigmoid(pre_t),
// and, with g_t = dy_t act'(pre_t) for t < length (0 behind it),
//     dxs[s] = sum_w w[c][w] g[s - w],  dw[c][w] = sum_{b,t} g_t xs[t + w],
//     db[c] = sum_{b,t} g_t.
#include <cuda_runtime.h>

#include <cstdint>

#include "layer.cuh"

namespace m2rnn {
namespace {

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// s = 1 / (1 + e^-x) by the hardware's 2^x and reciprocal, and tail = 1 - s.
// The rounding of the exponent -x log2 e counts x times: 2^-18 of the result at
// |x| = 80.  bf16 outputs are 2^9 times coarser; for fp32 the rounding and the
// rest of log2 e go into the power's first-order term, which leaves a few units
// at every x (the exact functions cost a quarter of the forward's time), and
// the tail of a large x is e^-x s, not what 1 - s leaves of it.
template <typename T>
__device__ __forceinline__ float sigmoid(float x, float* tail = nullptr) {
  if constexpr (sizeof(T) == 2) {
    const float s = sigmoid_fast(x);
    if (tail != nullptr) *tail = 1.f - s;
    return s;
  } else {
    constexpr float kHi = -1.44269504f, kLo = -1.44269504088896341 - static_cast<double>(kHi);  // -log2 e
    const float c = fminf(fmaxf(x, -88.f), 88.f);  // behind them s is 0 and 1, and nothing below leaves the fp32 range
    const float t = c * kHi, r = fmaf(c, kLo, fmaf(c, kHi, -t)), p = ex2_fast(t);
    const float e = fmaf(p, 0.693147181f * r, p), s = rcp_fast(1.f + e);
    if (tail != nullptr) *tail = x > 0.f ? e * s : 1.f - s;
    return s;
  }
}

// kVec consecutive elements of a row: one load or store of kVec elements
// (16 or 8 bytes on the vector paths).
template <typename T, int kVec>
struct Row {
  alignas(sizeof(T) * kVec) T e[kVec];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) * kVec == 16) {
      *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
    } else if constexpr (sizeof(T) * kVec == 8) {
      *reinterpret_cast<uint2*>(e) = __ldcs(reinterpret_cast<const uint2*>(p));
    } else if constexpr (sizeof(T) * kVec == 4) {
      *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
    } else {
      static_assert(kVec == 1, "vectors of 4, 8 or 16 bytes");
      e[0] = *p;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (sizeof(T) * kVec == 16) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    } else if constexpr (sizeof(T) * kVec == 8) {
      __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(e));
    } else if constexpr (sizeof(T) * kVec == 4) {
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(e);
    } else {
      *p = e[0];
    }
  }
  __device__ __forceinline__ void get(float (&f)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void set(const float (&f)[kVec]) {
    if constexpr (sizeof(T) == 2 && kVec % 2 == 0) {
      uint32_t* o = reinterpret_cast<uint32_t*>(e);
#pragma unroll
      for (int i = 0; i < kVec; i += 2) o[i / 2] = pack_bf16x2(f[i], f[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) e[i] = from_f32<T>(f[i]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = T(0);
  }
};

// One sequence's inputs at its channels: xs at x index s >= -(W - 1), zero
// where there is none.
template <typename T, int kVec>
struct Source {
  const T* x;
  const T* x0;  // null: zero
  int64_t stride;
  int C, W;
  __device__ __forceinline__ void at(int s, int len, Row<T, kVec>& r) const {
    if (s >= len || s < -(W - 1) || (s < 0 && x0 == nullptr))
      r.zero();
    else
      r.load(s >= 0 ? x + s * stride : x0 + static_cast<int64_t>(s + W - 1) * C);
  }
};

template <typename T, int kVec>
__device__ __forceinline__ Source<T, kVec> source(const ConvArgs& A, int b, int c) {
  return {static_cast<const T*>(A.x) + static_cast<int64_t>(b) * A.T * A.x_stride + c,
          A.x0 ? static_cast<const T*>(A.x0) + static_cast<int64_t>(b) * (A.W - 1) * A.C + c : nullptr, A.x_stride, A.C,
          A.W};
}

// The channels' weights.  They are consecutive and come as a few 16-byte loads
// where they fill them: 40 single loads per thread cost as much as the strip's
// own rows.
template <typename T, int kVec, int kW>
__device__ __forceinline__ void load_weights(const ConvArgs& A, int c, float (&w)[kW][kVec], float (&bias)[kVec]) {
  const T* p = static_cast<const T*>(A.w) + static_cast<int64_t>(c) * kW;
  constexpr int kPer = 16 / sizeof(T);
  if constexpr (kVec * kW % kPer == 0) {
#pragma unroll
    for (int i = 0; i < kVec * kW / kPer; ++i) {
      Row<T, kPer> r;
      r.load(p + i * kPer);
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[(i * kPer + e) % kW][(i * kPer + e) / kW] = to_f32(r.e[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j][i] = to_f32(p[i * kW + j]);
    }
  }
  Row<T, kVec> r;
  r.zero();
  if (A.bias != nullptr) r.load(static_cast<const T*>(A.bias) + c);
#pragma unroll
  for (int i = 0; i < kVec; ++i) bias[i] = to_f32(r.e[i]);
}

__device__ __forceinline__ int seq_len(const ConvArgs& A, int b) {
  return A.lengths ? min(max(A.lengths[b], 0), A.T) : A.T;
}

// Forward.  A thread takes kVec channels of a strip of `steps` steps (a
// multiple of kAhead) and keeps the last kW - 1 inputs in registers, so every
// input is loaded once but for the W - 1 rows before each strip; the next
// kAhead rows are in flight while it computes on the last.  kEdge: the strip
// may reach behind its sequence's end.  B=4 T=4096 C=1536 W=4 bf16, x a slice
// of a wider tensor: 21.5 us, 4.7 TB/s, 69 % of a plain copy's rate; fp32 41.2
// us, 72 %.  Neither DRAM (37 % busy over the launch) nor issue (48 %) is the
// limit but what a launch of one wave has in flight: 16 warps to an SM at 128
// registers, four rows each, and the wave's start and end (3 blocks per SM spill,
// strips of a fixed 64 steps leave SMs idle, 25 us).
constexpr int kFwdThreads = 256, kFwdBlocks = 2, kAhead = 4;

template <typename T, int kVec, int kW, bool kEdge>
__device__ __forceinline__ void forward_strip(const ConvArgs& A, const Source<T, kVec>& src, T* y, int c, int t0,
                                              int t1, int len) {
  float w[kW][kVec], bias[kVec], h[kW][kVec];
  Row<T, kVec> in[kAhead], next[kAhead];
  const T* px = src.x + t0 * src.stride;
  T* py = y + static_cast<int64_t>(t0) * A.C;
  auto load = [&](int t, Row<T, kVec>(&r)[kAhead]) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!kEdge || t + u < len)
        r[u].load(px + u * src.stride);
      else
        r[u].zero();
    }
    px += kAhead * src.stride;
  };
  load(t0, in);
#pragma unroll
  for (int j = 1; j < kW; ++j) {  // h[j] = xs at t - kW + j
    Row<T, kVec> r;
    src.at(t0 - kW + j, len, r);
    r.get(h[j]);
  }
  load_weights<T, kVec, kW>(A, c, w, bias);
  for (int t = t0; t < t1; t += kAhead) {
    if (t + kAhead < t1) load(t + kAhead, next);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float p[kVec];
      Row<T, kVec> out;
#pragma unroll
      for (int e = 0; e < kVec; ++e) p[e] = bias[e];
#pragma unroll
      for (int j = 0; j < kW - 1; ++j) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) h[j][e] = h[j + 1][e];
        fma_row<kVec>(p, w[j], h[j]);
      }
      in[u].get(h[kW - 1]);
      fma_row<kVec>(p, w[kW - 1], h[kW - 1]);
      if (A.silu) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) p[e] *= sigmoid<T>(p[e]);
      }
      out.set(p);
      if (kEdge && t + u >= len) out.zero();
      if (!kEdge || t + u < t1) out.store(py + static_cast<int64_t>(u) * A.C);
      in[u] = next[u];
    }
    py += static_cast<int64_t>(kAhead) * A.C;
  }
}

template <typename T, int kVec, int kW>
__global__ void __launch_bounds__(kFwdThreads, kFwdBlocks)
    conv_forward_kernel(ConvArgs A, int steps, int strips) {
  const int groups = A.C / kVec;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kFwdThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(A.B) * strips * groups) return;
  const int c = static_cast<int>(i % groups) * kVec;
  const int bs = static_cast<int>(i / groups), b = bs / strips, strip = bs % strips;
  const int len = seq_len(A, b), t0 = strip * steps, t1 = min(A.T, t0 + steps);
  const Source<T, kVec> src = source<T, kVec>(A, b, c);
  T* y = static_cast<T*>(A.y) + static_cast<int64_t>(b) * A.T * A.C + c;
  if (strip == 0 && A.x_T != nullptr) {
    for (int j = 0; j < A.W - 1; ++j) {
      Row<T, kVec> r;
      src.at(len + j - (A.W - 1), len, r);
      r.store(static_cast<T*>(A.x_T) + (static_cast<int64_t>(b) * (A.W - 1) + j) * A.C + c);
    }
  }
  if (t0 + steps <= len)
    forward_strip<T, kVec, kW, false>(A, src, y, c, t0, t1, len);
  else
    forward_strip<T, kVec, kW, true>(A, src, y, c, t0, t1, len);
}

// Backward.  A warp takes 32 kVec channels of a strip of `strip` steps (a
// multiple of kBwdAhead): it walks the steps with the last kW - 1 inputs and
// gradients g in registers, so that dxs comes out kW - 1 steps behind; the
// strip's last gradients are those of the kW - 1 steps behind it.  The block's
// warps are consecutive strips; their sums of dw, db are added in warp order
// through shared memory into one partial per block.  B=4 T=4096 C=1536 W=4 bf16
// (10 bytes an element) 49 us with the partials' sum, 5.2 TB/s, three quarters of
// a plain copy's rate; fp32 57 us, 78 %.  DRAM 57 % and issue 51 % busy over the
// launch: loads in flight and the instructions between them, in one wave.  Two
// channels a thread,
// whose products pair into one fp32 instruction; the next rows in flight while
// it computes (without, and a block more per SM, 54); strips as long as one
// wave of blocks wants them (a fixed 64 steps then took 59); gradients pass the
// caches by (2 us).
constexpr int kBwdWarps = 4, kBwdAhead = 4;

// Blocks to an SM, by the registers they take (fp32 at 6: 67 us for 57).
constexpr int backward_blocks(bool bf16, bool wide) { return wide ? 4 : bf16 ? 6 : 5; }

// Blocks of kBwdWarps strips along a sequence, and a strip's steps.
struct BwdCut {
  int blocks, strip;
};

BwdCut backward_cut(int64_t B, int64_t T, int64_t C, int per_sm) {
  const int64_t per_strip = B * ((C + 63) / 64), room = 152 * per_sm;
  int64_t blocks = room / per_strip < 1 ? 1 : room / per_strip;
  int64_t strip = (T + blocks * kBwdWarps - 1) / (blocks * kBwdWarps);
  strip = strip < 16 ? 16 : strip > 256 ? 256 : (strip + kBwdAhead - 1) / kBwdAhead * kBwdAhead;
  blocks = (T + strip * kBwdWarps - 1) / (strip * kBwdWarps);
  return {static_cast<int>(blocks), static_cast<int>(strip)};
}

// kEdge: the strip is its sequence's first or reaches its end.
template <typename T, int kVec, int kW, bool kEdge>
__device__ __forceinline__ void backward_strip(const ConvArgs& A, int b, int c, int t0, int t1, int strip, int len,
                                               float (&dw)[kW][kVec], float (&db)[kVec]) {
  const Source<T, kVec> src = source<T, kVec>(A, b, c);
  float w[kW][kVec], bias[kVec], h[kW][kVec], g[kW][kVec];
  const T* px = src.x + t0 * src.stride;
  const float* pu = A.dy + (static_cast<int64_t>(b) * A.T + t0) * A.C + c;
  float* pd = A.dx + (static_cast<int64_t>(b) * A.T + t0 - (kW - 1)) * A.C + c;
#pragma unroll
  for (int j = 1; j < kW; ++j) {
    Row<T, kVec> r;
    src.at(t0 - kW + j, len, r);
    r.get(h[j]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) g[j][e] = 0.f;  // gradients before the strip belong to the strip before
  }
  load_weights<T, kVec, kW>(A, c, w, bias);
  const int end = t0 + strip + kW - 1;  // g is wanted up to the last input's kW - 1 steps later
  const int lim = kEdge ? min(len, end) : end;
  Row<T, kVec> next_in[kBwdAhead];
  Row<float, kVec> next_up[kBwdAhead];
  auto load = [&](int t) {
#pragma unroll
    for (int u = 0; u < kBwdAhead; ++u) {
      if (t + u < lim) {
        next_in[u].load(px + u * src.stride);
        next_up[u].load(pu + static_cast<int64_t>(u) * A.C);
      } else {
        next_in[u].zero();
        next_up[u].zero();
      }
    }
    px += kBwdAhead * src.stride;
    pu += static_cast<int64_t>(kBwdAhead) * A.C;
  };
  load(t0);
  // One group of kBwdAhead steps, the next one's rows on their way; kMine: all of them belong to the strip.
  auto group = [&](int t, auto mine_tag) {
    constexpr bool kMine = decltype(mine_tag)::value;
    Row<T, kVec> in[kBwdAhead];
    Row<float, kVec> up[kBwdAhead];
#pragma unroll
    for (int u = 0; u < kBwdAhead; ++u) {
      in[u] = next_in[u];
      up[u] = next_up[u];
    }
    load(t + kBwdAhead);
#pragma unroll
    for (int u = 0; u < kBwdAhead; ++u) {
      float p[kVec], x[kVec], r[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        p[e] = bias[e];
        r[e] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < kW - 1; ++j) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          h[j][e] = h[j + 1][e];
          g[j][e] = g[j + 1][e];
        }
        fma_row<kVec>(p, w[j], h[j]);
      }
      in[u].get(h[kW - 1]);
      fma_row<kVec>(p, w[kW - 1], h[kW - 1]);
      up[u].get(x);
      if (A.silu) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          float tail;
          const float sg = sigmoid<T>(p[e], &tail);
          x[e] *= fmaf(p[e] * sg, tail, sg);
        }
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) g[kW - 1][e] = kEdge && t + u >= len ? 0.f : x[e];
      if (kMine || t + u < t1) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) db[e] += g[kW - 1][e];
#pragma unroll
        for (int j = 0; j < kW; ++j) fma_row<kVec>(dw[j], g[kW - 1], h[j]);
      }
      // x index s = t - (kW - 1) gets sum over j of g at s + j times w[kW - 1 - j].
#pragma unroll
      for (int j = 0; j < kW; ++j) fma_row<kVec>(r, g[j], w[kW - 1 - j]);
      const int s = t + u - (kW - 1);
      Row<float, kVec> out;
      out.set(r);
      if (!kEdge) {
        if (s >= t0 && (kMine || s < t1)) out.store(pd + static_cast<int64_t>(u) * A.C);
      } else if (s >= t0 ? s < t1 : t0 == 0 && s >= -(A.W - 1)) {
        if (A.dx_T != nullptr && s < len && s >= len - (A.W - 1)) {
          Row<float, kVec> last;
          last.load(A.dx_T + (static_cast<int64_t>(b) * (A.W - 1) + s - len + A.W - 1) * A.C + c);
#pragma unroll
          for (int e = 0; e < kVec; ++e) out.e[e] += last.e[e];
        }
        if (s >= 0)
          out.store(pd + static_cast<int64_t>(u) * A.C);
        else if (A.dx0 != nullptr)
          out.store(A.dx0 + (static_cast<int64_t>(b) * (A.W - 1) + s + A.W - 1) * A.C + c);
      }
    }
    pd += static_cast<int64_t>(kBwdAhead) * A.C;
  };
  int t = t0;
  if (!kEdge)
    for (; t < t0 + strip; t += kBwdAhead) group(t, Yes{});
  for (; t < end; t += kBwdAhead) group(t, No{});
}

template <typename T, int kVec, int kW>
__global__ void __launch_bounds__(32 * kBwdWarps, backward_blocks(sizeof(T) == 2, kW > 4))
    conv_backward_kernel(ConvArgs A, int blocks_c, int blocks_t, int strip) {
  __shared__ float red[kBwdWarps][kW + 1][32 * kVec];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bc = blockIdx.x % blocks_c, bt = blockIdx.x / blocks_c;
  const int b = bt / blocks_t, c = (bc * 32 + lane) * kVec;
  const int t0 = ((bt % blocks_t) * kBwdWarps + warp) * strip, t1 = min(A.T, t0 + strip);
  const int len = seq_len(A, b);
  float dw[kW][kVec], db[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < kW; ++j) dw[j][e] = 0.f;
  }
  if (c < A.C && t0 < A.T) {
    // The last kW steps of a sequence may take dx_T in.
    if (t0 > 0 && t0 + strip + kW - 1 <= len - kW)
      backward_strip<T, kVec, kW, false>(A, b, c, t0, t1, strip, len, dw, db);
    else
      backward_strip<T, kVec, kW, true>(A, b, c, t0, t1, strip, len, dw, db);
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
#pragma unroll
    for (int j = 0; j < kW; ++j) red[warp][j][lane * kVec + e] = dw[j][e];
    red[warp][kW][lane * kVec + e] = db[e];
  }
  __syncthreads();
  let_next();
  // Partials are [block of steps][kW taps, then the bias][C].
  for (int i = threadIdx.x; i < (kW + 1) * 32 * kVec; i += 32 * kBwdWarps) {
    const int j = i / (32 * kVec), x = i % (32 * kVec), cc = bc * 32 * kVec + x;
    if (cc >= A.C) continue;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kBwdWarps; ++v) s += red[v][j][x];
    A.part[(static_cast<int64_t>(bt) * (kW + 1) + j) * A.C + cc] = s;
  }
}

// Sum of the partials over the blocks of steps: block (32 channels, tap j),
// 8 warps taking every eighth partial, added in warp order.
__global__ void __launch_bounds__(256) conv_sum_parts_kernel(const float* part, float* dw, float* db, int parts, int C,
                                                             int W) {
  __shared__ float red[8][32];
  wait_previous();
  const int lane = threadIdx.x & 31, v = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
  float t = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int p = v; p < parts; p += 8) t += part[(static_cast<int64_t>(p) * (W + 1) + j) * C + c];
  }
  red[v][lane] = t;
  __syncthreads();
  if (v != 0 || c >= C) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += red[i][lane];
  if (j < W)
    dw[static_cast<int64_t>(c) * W + j] = t;
  else if (db != nullptr)
    db[c] = t;
}

// One token: a thread takes kVec channels of one sequence.  A latency: 32
// sequences of 1536 channels 2.1 us in a graph.
template <typename T, int kVec, int kW>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs A, T* state) {
  const int groups = A.C / kVec;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (i >= static_cast<int64_t>(A.B) * groups) return;
  const int c = static_cast<int>(i % groups) * kVec, b = static_cast<int>(i / groups);
  T* st = state + static_cast<int64_t>(b) * (kW - 1) * A.C + c;
  Row<T, kVec> r[kW], out;
  r[kW - 1].load(static_cast<const T*>(A.x) + b * A.x_stride + c);
#pragma unroll
  for (int j = 0; j < kW - 1; ++j) r[j].load(st + static_cast<int64_t>(j) * A.C);
  float w[kW][kVec], bias[kVec];
  load_weights<T, kVec, kW>(A, c, w, bias);
#pragma unroll
  for (int j = 1; j < kW; ++j) r[j].store(st + static_cast<int64_t>(j - 1) * A.C);
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    float p = bias[e];
#pragma unroll
    for (int j = 0; j < kW; ++j) p = fmaf(w[j][e], to_f32(r[j].e[e]), p);
    out.e[e] = from_f32<T>(A.silu ? p * sigmoid<T>(p) : p);
  }
  out.store(static_cast<T*>(A.y) + static_cast<int64_t>(b) * A.C + c);
}

// Rows that can be moved in vectors of v elements.
bool rows_of(const ConvArgs& a, int v) {
  const size_t bytes = (a.bf16 ? 2 : 4) * v;
  return a.C % v == 0 && a.x_stride % v == 0 && reinterpret_cast<uintptr_t>(a.x) % bytes == 0;
}

template <typename T, int kVec, int kW>
void forward(const ConvArgs& a, cudaStream_t s) {
  // Strips as short as it takes to fill every SM once (each strip loads W - 1 rows twice), at most 64 steps.
  const int64_t groups = a.C / kVec, room = 152ll * kFwdBlocks * kFwdThreads;
  int steps = static_cast<int>((static_cast<int64_t>(a.B) * a.T * groups + room - 1) / room);
  steps = steps > 64 ? 64 : (steps + kAhead - 1) / kAhead * kAhead;
  const int strips = (a.T + steps - 1) / steps;
  const int64_t n = static_cast<int64_t>(a.B) * strips * groups;
  conv_forward_kernel<T, kVec, kW>
      <<<static_cast<unsigned>((n + kFwdThreads - 1) / kFwdThreads), kFwdThreads, 0, s>>>(a, steps, strips);
}

template <typename T, int kVec, int kW>
void backward(const ConvArgs& a, cudaStream_t s) {
  const BwdCut cut = backward_cut(a.B, a.T, a.C, backward_blocks(a.bf16, a.W > 4));
  const int blocks_c = (a.C + 32 * kVec - 1) / (32 * kVec), blocks_t = cut.blocks;
  conv_backward_kernel<T, kVec, kW><<<static_cast<unsigned>(static_cast<int64_t>(blocks_c) * blocks_t * a.B),
                                      32 * kBwdWarps, 0, s>>>(a, blocks_c, blocks_t, cut.strip);
}

template <typename T, int kVec, int kW>
void step(const ConvArgs& a, void* state, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(a.B) * (a.C / kVec);
  conv_step_kernel<T, kVec, kW><<<static_cast<unsigned>((n + 127) / 128), 128, 0, s>>>(a, static_cast<T*>(state));
}

// Every width has its own kernels: taps that are not there would be products
// of zero with inputs outside the window, NaN where those are not finite.
// Widths above 4 with fewer channels a thread (8 taps of 8 channels spill).
#define M2RNN_CONV(CALL, T, VEC, VEC8, ...)                 \
  switch (a.W) {                                            \
    case 1: CALL<T, VEC, 1>(__VA_ARGS__); break;            \
    case 2: CALL<T, VEC, 2>(__VA_ARGS__); break;            \
    case 3: CALL<T, VEC, 3>(__VA_ARGS__); break;            \
    case 4: CALL<T, VEC, 4>(__VA_ARGS__); break;            \
    case 5: CALL<T, VEC8, 5>(__VA_ARGS__); break;           \
    case 6: CALL<T, VEC8, 6>(__VA_ARGS__); break;           \
    case 7: CALL<T, VEC8, 7>(__VA_ARGS__); break;           \
    case 8: CALL<T, VEC8, 8>(__VA_ARGS__); break;           \
    default: return cudaErrorInvalidValue;                  \
  }

}  // namespace

int conv_backward_parts(int64_t B, int64_t T, int64_t C) {
  int most = 0;
  for (int per_sm = 4; per_sm <= 6; ++per_sm) {
    const int blocks = backward_cut(B, T, C, per_sm).blocks;
    most = blocks > most ? blocks : most;
  }
  return static_cast<int>(B * most);
}

cudaError_t launch_conv_forward(const ConvArgs& a, cudaStream_t s) {
  if (a.bf16) {
    if (rows_of(a, 8)) {
      M2RNN_CONV(forward, uint16_t, 8, 4, a, s)
    } else {
      M2RNN_CONV(forward, uint16_t, 1, 1, a, s)
    }
  } else {
    if (rows_of(a, 4)) {
      M2RNN_CONV(forward, float, 4, 4, a, s)
    } else {
      M2RNN_CONV(forward, float, 1, 1, a, s)
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_conv_backward(const ConvArgs& a, cudaStream_t s) {
  if (a.bf16) {
    if (rows_of(a, 2)) {
      M2RNN_CONV(backward, uint16_t, 2, 1, a, s)
    } else {
      M2RNN_CONV(backward, uint16_t, 1, 1, a, s)
    }
  } else {
    if (rows_of(a, 2)) {
      M2RNN_CONV(backward, float, 2, 1, a, s)
    } else {
      M2RNN_CONV(backward, float, 1, 1, a, s)
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(conv_sum_parts_kernel, dim3((a.C + 31) / 32, a.W + 1), 256, 0, s, a.part, a.dw, a.db,
                     a.B * backward_cut(a.B, a.T, a.C, backward_blocks(a.bf16, a.W > 4)).blocks, a.C, a.W);
}

cudaError_t launch_conv_step(void* state, const ConvArgs& a, cudaStream_t s) {
  if (a.bf16) {
    if (rows_of(a, 8)) {
      M2RNN_CONV(step, uint16_t, 8, 4, a, state, s)
    } else {
      M2RNN_CONV(step, uint16_t, 1, 1, a, state, s)
    }
  } else {
    if (rows_of(a, 4)) {
      M2RNN_CONV(step, float, 4, 4, a, state, s)
    } else {
      M2RNN_CONV(step, float, 1, 1, a, state, s)
    }
  }
  return cudaGetLastError();
}

}  // namespace m2rnn
