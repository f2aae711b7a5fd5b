// Gated linear recurrence on a vector state, per batch element and channel,
// from H_0, with the gate of the matrix-state scans (gate.cuh):
//     f_t = exp(-alpha softplus(a_t + beta)),
//     h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t.
// Backward, with dh the gradient of h:
//     dh_t = dy_t + f_{t+1} dh_{t+1},   dx_t = (1 - f_t) dh_t,
//     g_t = dh_t f_t (h_{t-1} - x_t)  (= dL / d log f_t),
//     da_t = -alpha sigmoid(a_t + beta) g_t,
//     dalpha = -sum softplus(a_t + beta) g_t,  dbeta = sum da_t,
//     dH_0 = f_1 dh_1.
//
// Steps compose: a run of them takes a state h to F h + U.  A warp holds a
// segment of kL steps of 64 channels (two per lane) in registers, finds its F
// and U, and goes over it again once it knows the state before it, so that
// inputs are read and gates computed once.  The warps of a block hold a tile of
// consecutive segments, the blocks of a cluster consecutive tiles, and the
// cluster marches through the sequence in rounds: F and U of the warps go
// through shared memory, those of the blocks through the cluster's, and every
// thread composes what lies before it.  The next round's inputs are loaded
// before the exchange.  The backward marches the other way; the states before
// its segments are left by the forward's kernel, without y, in one launch
// before it.
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"

namespace m2rnn {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kChan = 64, kMaxCluster = 8;
static_assert(kWarps >= kMaxCluster, "a warp hands the block's total to each block of the cluster");

// ---------------------------------------------------------------------------
// Pairs of channels
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  fma2(c.x, c.y, a.x, a.y, b.x, b.y);
  return c;
}
__device__ __forceinline__ float2 mul_2(float2 a, float2 b) {
  float2 d;
  mul2(d.x, d.y, a.x, a.y, b.x, b.y);
  return d;
}
__device__ __forceinline__ float2 add_2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Two values of a row as they lie in memory: side by side (kPair, one load), or
// 32 channels apart.
template <typename E>
struct Raw2;
template <>
struct Raw2<uint16_t> {
  uint32_t v;
  __device__ __forceinline__ float2 f() const { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
};
template <>
struct Raw2<float> {
  float2 v;
  __device__ __forceinline__ float2 f() const { return v; }
};
// `other`: from the lane's first to its second channel (not kPair).
template <bool kPair>
__device__ __forceinline__ Raw2<uint16_t> load_2(const uint16_t* p, int other) {
  if constexpr (kPair) return {*reinterpret_cast<const uint32_t*>(p)};
  return {static_cast<uint32_t>(p[0]) | static_cast<uint32_t>(p[other]) << 16};
}
template <bool kPair>
__device__ __forceinline__ Raw2<float> load_2(const float* p, int other) {
  if constexpr (kPair) return {*reinterpret_cast<const float2*>(p)};
  return {make_float2(p[0], p[other])};
}
// kL rows from row t0 on; those at or behind `len` are zero.
template <bool kPair, int kL, typename E>
__device__ __forceinline__ void load_rows(Raw2<E> (&r)[kL], const E* p, int64_t stride, int other, int t0, int len) {
  p += t0 * stride;
  if (t0 + kL <= len) {
#pragma unroll
    for (int i = 0; i < kL; ++i, p += stride) r[i] = load_2<kPair>(p, other);
  } else {
#pragma unroll
    for (int i = 0; i < kL; ++i, p += stride) {
      r[i] = Raw2<E>{};
      if (t0 + i < len) r[i] = load_2<kPair>(p, other);
    }
  }
}
template <bool kPair>
__device__ __forceinline__ void store_2(uint16_t* p, float2 v, bool in0, bool in1) {
  if constexpr (kPair) {
    if (in0) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
  } else {
    if (in0) p[0] = from_f32<uint16_t>(v.x);
    if (in1) p[32] = from_f32<uint16_t>(v.y);
  }
}
template <bool kPair>
__device__ __forceinline__ void store_2(float* p, float2 v, bool in0, bool in1) {
  if constexpr (kPair) {
    if (in0) *reinterpret_cast<float2*>(p) = v;
  } else {
    if (in0) p[0] = v.x;
    if (in1) p[32] = v.y;
  }
}

// A lane's two channels: c and c + 1, or c and c + 32.  Lanes without a channel
// read the last one's (`from`, and `other` further on) and write nothing.
template <bool kPair>
struct Lane {
  int c, from, other;
  bool in0, in1;
  __device__ __forceinline__ Lane(int group, int C) {
    c = group * kChan + (threadIdx.x & 31) * (kPair ? 2 : 1);
    in0 = c < C;
    in1 = c + (kPair ? 1 : 32) < C;
    from = in0 ? c : C - (kPair ? 2 : 1);
    other = in1 ? (kPair ? 1 : 32) : 0;
  }
  __device__ __forceinline__ float2 get(const float* p) const {
    return p != nullptr ? make_float2(p[from], p[from + other]) : make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void put(float* p, float2 v) const {
    if (in0) p[c] = v.x;
    if (in1) p[c + (kPair ? 1 : 32)] = v.y;
  }
};

// ---------------------------------------------------------------------------
// The gate, for two channels
// ---------------------------------------------------------------------------
struct Gate2 {
  float2 f, e, soft, t;  // e = 1 - f; t = exp(-|z|)
};

// All to a few units of fp32.  softplus(z) = max(z, 0) + log(1 + t), t = exp(-|z|),
// and log(1 + t) = 2 atanh(v), v = t / (2 + t) <= 1/3: a polynomial in v^2 of
// degree 4 (minimax, 4e-9).  1 - f = u P(u), u = alpha softplus, for |u| <= 0.7
// (minimax, 3e-8), so that it keeps its digits where f is near 1, and f is what
// is left; beyond, f = 2^(-u log2 e).  kSmall: f keeps its digits where it is
// near 0 too, which only gradients show.
template <bool kSmall>
__device__ __forceinline__ Gate2 gate_of(float2 z, float2 alpha) {
  constexpr float kLog2e = 1.44269504f;
  Gate2 g;
  const float2 y = mul_2(z, two(kLog2e));
  g.t = make_float2(ex2_fast(-fabsf(y.x)), ex2_fast(-fabsf(y.y)));
  const float2 w = add_2(g.t, two(2.f));
  const float2 v = mul_2(g.t, make_float2(rcp_fast(w.x), rcp_fast(w.y)));
  const float2 s = mul_2(v, v);
  float2 p = fma_2(s, two(0.28178346157f), two(0.27960598469f));
  p = fma_2(s, p, two(0.40024909377f));
  p = fma_2(s, p, two(0.66666316986f));
  p = fma_2(s, p, two(2.f));
  g.soft = fma_2(v, p, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
  const float2 u = mul_2(alpha, g.soft);
  p = fma_2(u, two(0.00019840967f), two(-0.00141012867f));
  p = fma_2(u, p, two(0.00833449047f));
  p = fma_2(u, p, two(-0.04166151583f));
  p = fma_2(u, p, two(0.16666638851f));
  p = fma_2(u, p, two(-0.50000029802f));
  p = fma_2(u, p, two(1.f));
  const float2 e = mul_2(u, p), x = mul_2(u, two(-kLog2e));
  const float2 f = make_float2(ex2_fast(x.x), ex2_fast(x.y)), far = fma_2(f, two(-1.f), two(1.f));
  const bool near0 = fabsf(u.x) <= 0.7f, near1 = fabsf(u.y) <= 0.7f;
  g.e = make_float2(near0 ? e.x : far.x, near1 ? e.y : far.y);
  g.f = fma_2(g.e, two(-1.f), two(1.f));
  if constexpr (kSmall) g.f = make_float2(near0 ? g.f.x : f.x, near1 ? g.f.y : f.y);
  return g;
}

// ---------------------------------------------------------------------------
// The exchange
// ---------------------------------------------------------------------------
struct Exchange {
  float4 warp[2][kWarps][32];        // F, U of the block's segments
  float4 block[2][kMaxCluster][32];  // of the cluster's tiles
  alignas(8) uint64_t arrived[2];    // a phase for each second round: every tile's F and U are there
  int abort_flag;
};

__device__ __forceinline__ void open_exchange(Exchange& x, int blocks) {
  if (blocks == 1) return;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&x.arrived[0]), 1);
    mbar_init(smem_u32(&x.arrived[1]), 1);
    x.abort_flag = 0;
    fence_mbar_init_cluster();
  }
  cluster_sync_all();
}

// The state before the warp's segment, from `carry`, the state before the
// round; carry goes on to the next round.  Every thread of the cluster calls it.
// A block hands its F and U to every block of the cluster by stores that count
// on the receiver's mbarrier: a cluster barrier's release would wait for the
// outputs stored before it.  Buffers of two rounds serve: nobody sends for round
// i + 2 before it has what this block sent for round i + 1, after this block was
// done with round i; and nobody ends before all that is sent to it has come.  A
// wait that gives up (seconds) spoils the state with NaN.
__device__ __forceinline__ float2 state_before(Exchange& x, int round, float2 F, float2 U, float2& carry, int rank, int blocks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, buf = round & 1;
  x.warp[buf][warp][lane] = make_float4(F.x, F.y, U.x, U.y);
  __syncthreads();
  float2 pF = two(1.f), pU = two(0.f), tF = two(1.f), tU = two(0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      pF = tF;
      pU = tU;
    }
    const float4 s = x.warp[buf][w][lane];
    const float2 f = make_float2(s.x, s.y);
    tU = fma_2(f, tU, make_float2(s.z, s.w));
    tF = mul_2(f, tF);
  }
  float2 mine = carry;
  if (blocks == 1) {
    carry = fma_2(tF, carry, tU);
  } else {
    const uint32_t bar = smem_u32(&x.arrived[buf]);
    if (warp < blocks) {
      const uint32_t to = mapa_shared(smem_u32(&x.block[buf][rank][lane]), warp), at = mapa_shared(bar, warp);
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                   "f"(tF.x), "f"(tF.y), "f"(tU.x), "f"(tU.y), "r"(at)
                   : "memory");
    }
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, blocks * 32 * 16);
    if (!mbar_wait<true>(bar, (round >> 1) & 1, &x.abort_flag, nullptr, 0)) carry = two(__int_as_float(0x7fc00000));
    for (int r = 0; r < blocks; ++r) {
      if (r == rank) mine = carry;
      const float4 s = x.block[buf][r][lane];
      carry = fma_2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
    }
  }
  return fma_2(pF, mine, pU);
}

__device__ __forceinline__ int length_of(const LinearArgs& A, int b) {
  return A.lengths != nullptr ? min(max(A.lengths[b], 0), A.T) : A.T;
}

// ---------------------------------------------------------------------------
// Forward: y, H_T; or (kStates) the state before each kEvery steps
// ---------------------------------------------------------------------------
template <typename E, bool kPair, bool kStates, int kL, int kEvery>
__global__ void __launch_bounds__(kThreads, 2) linear_forward_kernel(LinearArgs A, float* states, int blocks, int groups) {
  __shared__ Exchange xch;
  constexpr int kTile = kWarps * kL;
  const int chain = blockIdx.x / blocks, rank = blockIdx.x - chain * blocks;
  const int b = chain / groups, group = chain - b * groups, warp = threadIdx.x >> 5;
  const Lane<kPair> me(group, A.C);
  const int len = length_of(A, b);
  const int64_t first = static_cast<int64_t>(b) * A.T;
  const E* px = static_cast<const E*>(A.x) + first * A.x_stride + me.from;
  const E* pa = static_cast<const E*>(A.a) + first * A.a_stride + me.from;
  E* py = static_cast<E*>(A.y) + first * A.C + me.c;
  const float2 alpha = me.get(A.alpha), beta = me.get(A.beta);
  float2 carry = me.get(A.H_0 != nullptr ? A.H_0 + static_cast<int64_t>(b) * A.C : nullptr);
  const int rounds = (len + kTile * blocks - 1) / (kTile * blocks);

  Raw2<E> ra[kL], rx[kL];
  auto load = [&](int t0) {
    load_rows<kPair>(ra, pa, A.a_stride, me.other, t0, len);
    load_rows<kPair>(rx, px, A.x_stride, me.other, t0, len);
  };
  open_exchange(xch, blocks);
  int t0 = rank * kTile + warp * kL;
  if (rounds > 0) load(t0);
  for (int it = 0; it < rounds; ++it) {
    float2 f[kL], in[kL], F = two(1.f), U = two(0.f);
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const Gate2 g = gate_of<false>(add_2(ra[i].f(), beta), alpha);
      f[i] = g.f;
      in[i] = mul_2(g.e, rx[i].f());
    }
    if (t0 + kL > len) {  // steps behind the end leave the state as it is
#pragma unroll
      for (int i = 0; i < kL; ++i)
        if (t0 + i >= len) {
          f[i] = two(1.f);
          in[i] = two(0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      U = fma_2(f[i], U, in[i]);
      F = mul_2(f[i], F);
    }
    const int now = t0;
    t0 += kTile * blocks;
    if (it + 1 < rounds) load(t0);
    float2 h = state_before(xch, it, F, U, carry, rank, blocks);
    if constexpr (kStates) {
      float* p = states + (static_cast<int64_t>(b) * ((A.T + kEvery - 1) / kEvery) + now / kEvery) * A.C;
#pragma unroll
      for (int i = 0; i < kL; ++i) {
        if (i % kEvery == 0 && now + i < len) me.put(p + static_cast<int64_t>(i / kEvery) * A.C, h);
        h = fma_2(f[i], h, in[i]);
      }
    } else {
      E* p = py + static_cast<int64_t>(now) * A.C;
      if (now + kL <= len) {
#pragma unroll
        for (int i = 0; i < kL; ++i, p += A.C) {
          h = fma_2(f[i], h, in[i]);
          store_2<kPair>(p, h, me.in0, me.in1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kL; ++i, p += A.C) {
          h = fma_2(f[i], h, in[i]);
          if (now + i < A.T) store_2<kPair>(p, now + i < len ? h : two(0.f), me.in0, me.in1);
        }
      }
    }
  }
  let_next();
  if constexpr (!kStates) {
    for (int t = rounds * kTile * blocks + rank * kWarps + warp; t < A.T; t += blocks * kWarps)
      store_2<kPair>(py + static_cast<int64_t>(t) * A.C, two(0.f), me.in0, me.in1);
    if (A.H_T != nullptr && rank == 0 && warp == 0) me.put(A.H_T + static_cast<int64_t>(b) * A.C, carry);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <typename E, bool kPair, int kL>
__global__ void __launch_bounds__(kThreads, 2) linear_backward_kernel(LinearArgs A, const float* states, float* part, int blocks,
                                                                      int groups) {
  __shared__ Exchange xch;
  constexpr int kTile = kWarps * kL;
  const int chain = blockIdx.x / blocks, rank = blockIdx.x - chain * blocks;
  const int b = chain / groups, group = chain - b * groups, warp = threadIdx.x >> 5;
  const Lane<kPair> me(group, A.C);
  const int len = length_of(A, b);
  const int64_t first = static_cast<int64_t>(b) * A.T;
  const E* px = static_cast<const E*>(A.x) + first * A.x_stride + me.from;
  const E* pa = static_cast<const E*>(A.a) + first * A.a_stride + me.from;
  const E* pd = static_cast<const E*>(A.dy) + first * A.C + me.from;
  float *pdx = A.dx + first * A.C + me.c, *pda = A.da + first * A.C + me.c;
  const float* ph = states + static_cast<int64_t>(b) * ((A.T + kL - 1) / kL) * A.C;
  const float2 alpha = me.get(A.alpha), beta = me.get(A.beta);
  const float2 minus_alpha = make_float2(-alpha.x, -alpha.y);
  float2 carry = me.get(A.dH_T != nullptr ? A.dH_T + static_cast<int64_t>(b) * A.C : nullptr);
  float2 sa = two(0.f), sb = two(0.f);
  const int tiles = (len + kTile - 1) / kTile, rounds = (tiles + blocks - 1) / blocks;

  // Rounds go from the end: block 0 has the last tile, warp 0 the last segment of it.
  int t0 = ((tiles - 1 - rank) * kWarps + kWarps - 1 - warp) * kL;
  Raw2<E> ra[kL], rx[kL], rd[kL];
  float2 hs = two(0.f);
  auto load = [&](int t0) {  // (before the sequence as behind it: zeros)
    const int from = t0 < 0 ? len : t0;
    load_rows<kPair>(ra, pa, A.a_stride, me.other, from, len);
    load_rows<kPair>(rx, px, A.x_stride, me.other, from, len);
    load_rows<kPair>(rd, pd, A.C, me.other, from, len);
  };
  auto load_state = [&](int t0) {
    if (t0 >= 0 && t0 < len) hs = me.get(ph + static_cast<int64_t>(t0 / kL) * A.C);
  };
  open_exchange(xch, blocks);
  if (rounds > 0) load(t0);
  wait_previous();
  if (rounds > 0) load_state(t0);
  for (int it = 0; it < rounds; ++it) {
    float2 f[kL], e[kL], ma[kL], ms[kL], dy[kL], F = two(1.f), U = two(0.f);
    float2 h = hs;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const float2 z = add_2(ra[i].f(), beta), x = rx[i].f();
      const Gate2 g = gate_of<true>(z, alpha);
      f[i] = g.f;
      e[i] = g.e;
      const float2 w = add_2(g.t, two(1.f));
      const float2 sig = make_float2((z.x >= 0.f ? 1.f : g.t.x) * rcp_fast(w.x), (z.y >= 0.f ? 1.f : g.t.y) * rcp_fast(w.y));
      const float2 away = mul_2(g.f, make_float2(h.x - x.x, h.y - x.y));
      ma[i] = mul_2(away, mul_2(minus_alpha, sig));
      ms[i] = mul_2(away, make_float2(-g.soft.x, -g.soft.y));
      h = fma_2(g.f, h, mul_2(g.e, x));
      dy[i] = rd[i].f();
    }
    if (t0 < 0 || t0 + kL > len) {  // steps that are not there hand the gradient on
#pragma unroll
      for (int i = 0; i < kL; ++i)
        if (t0 < 0 || t0 + i >= len) {
          f[i] = two(1.f);
          ma[i] = ms[i] = two(0.f);
        }
    }
#pragma unroll
    for (int i = kL - 1; i >= 0; --i) {
      U = mul_2(f[i], add_2(dy[i], U));
      F = mul_2(f[i], F);
    }
    const int now = t0;
    t0 -= kTile * blocks;
    if (it + 1 < rounds) {
      load(t0);
      load_state(t0);
    }
    float2 c = state_before(xch, it, F, U, carry, rank, blocks);
    if (now >= 0) {
#pragma unroll
      for (int i = kL - 1; i >= 0; --i) {
        const int t = now + i;
        const float2 d = add_2(dy[i], c);
        float2 dx = mul_2(e[i], d), da = mul_2(ma[i], d);
        sa = fma_2(ms[i], d, sa);
        sb = add_2(sb, da);
        c = mul_2(f[i], d);
        if (t >= len) dx = da = two(0.f);
        if (t < A.T) {
          store_2<kPair>(pdx + static_cast<int64_t>(t) * A.C, dx, me.in0, me.in1);
          store_2<kPair>(pda + static_cast<int64_t>(t) * A.C, da, me.in0, me.in1);
        }
      }
    }
  }
  let_next();
  for (int t = tiles * kTile + rank * kWarps + warp; t < A.T; t += blocks * kWarps) {
    store_2<kPair>(pdx + static_cast<int64_t>(t) * A.C, two(0.f), me.in0, me.in1);
    store_2<kPair>(pda + static_cast<int64_t>(t) * A.C, two(0.f), me.in0, me.in1);
  }
  if (A.dH_0 != nullptr && rank == 0 && warp == 0) me.put(A.dH_0 + static_cast<int64_t>(b) * A.C, carry);
  __syncthreads();
  xch.warp[0][warp][threadIdx.x & 31] = make_float4(sa.x, sa.y, sb.x, sb.y);
  __syncthreads();
  if (warp == 0) {
    float4 t = xch.warp[0][0][threadIdx.x];
    for (int w = 1; w < kWarps; ++w) {
      const float4 s = xch.warp[0][w][threadIdx.x];
      t.x += s.x;
      t.y += s.y;
      t.z += s.z;
      t.w += s.w;
    }
    float* p = part + (static_cast<int64_t>(b) * blocks + rank) * 2 * A.C;
    me.put(p, make_float2(t.x, t.y));
    me.put(p + A.C, make_float2(t.z, t.w));
  }
}

// ---------------------------------------------------------------------------
// One token
// ---------------------------------------------------------------------------
template <typename E, bool kPair>
__global__ void __launch_bounds__(128) linear_step_kernel(float* H, LinearArgs A, int groups) {
  const int64_t id = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int b = static_cast<int>(id / groups);
  if (b >= A.B) return;
  const Lane<kPair> me(static_cast<int>(id - static_cast<int64_t>(b) * groups), A.C);
  const Raw2<E> a = load_2<kPair>(static_cast<const E*>(A.a) + b * A.a_stride + me.from, me.other);
  const Raw2<E> x = load_2<kPair>(static_cast<const E*>(A.x) + b * A.x_stride + me.from, me.other);
  const int64_t at = static_cast<int64_t>(b) * A.C;
  const Gate2 g = gate_of<false>(add_2(a.f(), me.get(A.beta)), me.get(A.alpha));
  const float2 h = fma_2(g.f, me.get(H + at), mul_2(g.e, x.f()));
  me.put(H + at, h);
  store_2<kPair>(static_cast<E*>(A.y) + at + me.c, h, me.in0, me.in1);
}

// Sums over parts: eight warps of a block take every eighth part each of 32
// columns, then add up in order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* part, float* out, float* out2, int parts, int64_t D,
                                                        int64_t width) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  wait_previous();
  float t = 0.f;
  if (j < width) {
#pragma unroll 4
    for (int p = warp; p < parts; p += 8) t += part[p * width + j];
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp != 0 || j >= width) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) t += red[w][lane];
  if (j < D)
    out[j] = t;
  else if (out2 != nullptr)
    out2[j - D] = t;
}

constexpr int kEveryBf16 = 8, kEveryF32 = 4;  // steps of a segment of the backward

// Blocks to a cluster: more until two per SM are there, as long as each has a
// tile of its own.
int cluster_blocks(const LinearArgs& a, int tile) {
  const int64_t chains = static_cast<int64_t>(a.B) * ((a.C + kChan - 1) / kChan);
  int r = 1;
  while (r < kMaxCluster && chains * r < 2 * 152 - 64 && r * tile < a.T) r *= 2;
  return r;
}

template <typename... P, typename... V>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t grid, int blocks, bool behind, cudaStream_t s, V... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(kThreads);
  c.stream = s;
  c.attrs = at;
  c.numAttrs = behind ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// Whether rows can be read and written two channels at a time.
bool paired(const LinearArgs& a) {
  const uintptr_t two = a.bf16 ? 3 : 7;
  return a.C % 2 == 0 && a.x_stride % 2 == 0 && a.a_stride % 2 == 0 &&
         ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.a)) & two) == 0;
}

template <typename E, bool kPair, int kL, int kEvery>
cudaError_t forward(const LinearArgs& a, cudaStream_t s) {
  const int groups = (a.C + kChan - 1) / kChan, blocks = cluster_blocks(a, kWarps * kL);
  return launch_cluster(linear_forward_kernel<E, kPair, false, kL, kEvery>, static_cast<int64_t>(a.B) * groups * blocks,
                        blocks, false, s, a, nullptr, blocks, groups);
}

template <typename E, bool kPair, int kL, int kEvery>
cudaError_t backward(const LinearArgs& a, cudaStream_t s) {
  const int groups = (a.C + kChan - 1) / kChan;
  const int64_t chains = static_cast<int64_t>(a.B) * groups;
  float* part = static_cast<float*>(a.ws);
  float* states = part + static_cast<int64_t>(a.B) * kMaxCluster * 2 * a.C;
  const int before = cluster_blocks(a, kWarps * kL), blocks = cluster_blocks(a, kWarps * kEvery);
  cudaError_t e = launch_cluster(linear_forward_kernel<E, kPair, true, kL, kEvery>, chains * before, before, false, s, a,
                                 states, before, groups);
  if (e != cudaSuccess) return e;
  e = launch_cluster(linear_backward_kernel<E, kPair, kEvery>, chains * blocks, blocks, true, s, a, states, part, blocks,
                     groups);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(part, a.dalpha, a.dbeta, true, a.B * blocks, a.C, s);
}

}  // namespace

size_t linear_backward_scratch_bytes(int64_t B, int64_t T, int64_t C) {
  return static_cast<size_t>(B) * C * 4 * (2 * kMaxCluster + (T + kEveryF32 - 1) / kEveryF32);
}

cudaError_t launch_sum_parts(const float* part, float* out, float* out2, bool two, int parts, int64_t D, cudaStream_t s) {
  const int64_t width = two ? 2 * D : D;
  return launch_next(sum_parts_kernel, static_cast<unsigned>((width + 31) / 32), 256, 0, s, part, out, out2, parts, D, width);
}

cudaError_t launch_linear_forward(const LinearArgs& a, cudaStream_t s) {
  if (paired(a))
    return a.bf16 ? forward<uint16_t, true, 16, kEveryBf16>(a, s) : forward<float, true, 8, kEveryF32>(a, s);
  return a.bf16 ? forward<uint16_t, false, 16, kEveryBf16>(a, s) : forward<float, false, 8, kEveryF32>(a, s);
}

cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s) {
  if (paired(a))
    return a.bf16 ? backward<uint16_t, true, 16, kEveryBf16>(a, s) : backward<float, true, 8, kEveryF32>(a, s);
  return a.bf16 ? backward<uint16_t, false, 16, kEveryBf16>(a, s) : backward<float, false, 8, kEveryF32>(a, s);
}

cudaError_t launch_linear_step(float* H, const LinearArgs& a, cudaStream_t s) {
  const int groups = (a.C + kChan - 1) / kChan;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.B) * groups + 3) / 4);
  if (paired(a)) {
    if (a.bf16)
      linear_step_kernel<uint16_t, true><<<grid, 128, 0, s>>>(H, a, groups);
    else
      linear_step_kernel<float, true><<<grid, 128, 0, s>>>(H, a, groups);
  } else {
    if (a.bf16)
      linear_step_kernel<uint16_t, false><<<grid, 128, 0, s>>>(H, a, groups);
    else
      linear_step_kernel<float, false><<<grid, 128, 0, s>>>(H, a, groups);
  }
  return cudaGetLastError();
}

}  // namespace m2rnn
