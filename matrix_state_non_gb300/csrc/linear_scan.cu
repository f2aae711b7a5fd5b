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
// thread composes what lies before it.  Inputs come a few rounds ahead, by TMA
// into a ring of tiles in shared memory (kTma, where rows lie on 16 bytes), else
// a round ahead into registers.  The backward marches the other way; the states before
// its segments are left by the forward's kernel, without y, in one launch
// before it.
//
// Bound by no unit but by latency and load: 13 warps to an SM, of whose issue slots
// 54 % are used (the busier multiply-add pipe 45 %, DRAM 35 %), 256 blocks on 152
// SMs, and in each round an exchange of 0.9 us, partly behind the other block of an
// SM.  B=2 T=16384 C=1024 bf16: 58 us, 3.5 TB/s; backward B=4 T=4096: 27 + 53 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "around.cuh"
#include "cluster_fit.h"
#include "internal.h"
#include "mma_common.cuh"

namespace m2rnn {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kChan = 64;
static_assert(kWarps >= kMaxCluster, "a warp hands the block's total to each block of the cluster");

// ---------------------------------------------------------------------------
// Pairs of channels
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  fma2(c.x, c.y, a.x, a.y, b.x, b.y);
  return c;
}
__device__ __forceinline__ float2 fma_1(float2 a, float2 b, float2 c) {  // an instruction each
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
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

// A ring of tiles in shared memory: kN inputs of kRows steps of 64 channels, by
// TMA.  One thread fills, everybody waits.
template <typename E, int kN, int kRows>
struct Ring {
  static constexpr int kStages = 3, kTileBytes = kRows * kChan * static_cast<int>(sizeof(E));
  static constexpr int kBytes = kStages * kN * kTileBytes;
  uint8_t* tiles;  // on 128 bytes
  uint64_t* full;  // [kStages]
  __device__ __forceinline__ const E* row(int stage, int input, int r) const {
    return reinterpret_cast<const E*>(tiles + (stage * kN + input) * kTileBytes) + r * kChan + 2 * (threadIdx.x & 31);
  }
  __device__ __forceinline__ void fill(int stage, const CUtensorMap* const (&maps)[kN], int c, int t, int b) const {
    const uint32_t bar = smem_u32(full + stage);
    mbar_arrive_expect_tx(bar, kN * kTileBytes);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
              smem_u32(tiles + (stage * kN + i) * kTileBytes)),
          "l"(reinterpret_cast<uint64_t>(maps[i])), "r"(bar), "r"(c), "r"(t), "r"(b)
          : "memory");
  }
};
// A block that gave up waits for what is still on its way to its ring, of
// `fills` tiles in all.
template <typename Tiles>
__device__ __forceinline__ void drain(uint64_t* full, int fills) {
  for (int i = max(0, fills - Tiles::kStages); i < fills; ++i)
    mbar_wait_timed(smem_u32(full + i % Tiles::kStages), (i / Tiles::kStages) & 1, nullptr, 0);
}
template <int kN>
struct Maps {
  CUtensorMap m[kN];
};

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
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f, kMost = 0x1.fffffep127f;

struct Gate2 {
  float2 f, e, soft, t;  // e = 1 - f; soft = softplus(z) log2 e; t = exp(-|z|)
};

// All to a few units of fp32, from y = z log2 e.  With t = 2^-|y|,
//     softplus(z) log2 e = max(y, 0) + log2(1 + t),
// and log2(1 + t) = 2 log2 e atanh(v), v = t / (2 + t) <= 1/3: a polynomial in v^2
// of degree 4 (minimax, 4e-9).  f = 2^-w, w = alpha softplus(z) log2 e; 1 - f is
// w P(w) for |w| <= 0.7 (minimax, 8e-8), so that it keeps its digits where f is
// near 1, and f is what is left; beyond, f is the hardware's power, whose digits a
// state shows that decays far below what it was, and 1 - f what is left.
// kGradient: softplus stops at fp32's largest value, so that no 0 times infinity
// is a gradient where y overflows (it does for a of the type's largest value).
// Without that, only alpha = 0 would meet it: there shut() takes y to -infinity,
// where f is 1, too.  (The bound took the forward from 57.8 to 59.3 us; 1 - e for
// 1 - w P in pairs, 58.0 to 62.4.)
// Multiply-adds are most of the instructions.  Two channels to an instruction take two
// cycles of one of the two pipes, so some (here and in the scan itself) are left
// single for the other: B=2 T=16384 C=1024 bf16 takes 57 us so, 62 with all in
// pairs, 65 with none.  log2(1 + t) by a polynomial in t, one reciprocal less and
// three multiply-adds more, is 7 % slower.
__device__ __forceinline__ float2 shut(float2 beta, float2 alpha) {
  return make_float2(alpha.x == 0.f ? -INFINITY : beta.x, alpha.y == 0.f ? -INFINITY : beta.y);
}
template <bool kGradient>
__device__ __forceinline__ Gate2 gate_of(float2 y, float2 alpha) {
  Gate2 g;
  g.t = make_float2(ex2_fast(-fabsf(y.x)), ex2_fast(-fabsf(y.y)));
  const float2 d = add_2(g.t, two(2.f));
  const float2 v = mul_2(g.t, make_float2(rcp_fast(d.x), rcp_fast(d.y)));
  const float2 s = mul_2(v, v);
  float2 p = fma_2(s, two(0.40652760863f), two(0.40338617563f));
  p = fma_2(s, p, two(0.57743740082f));
  p = fma_2(s, p, two(0.96179163456f));
  p = fma_2(s, p, two(2.88539004326f));
  float2 above = make_float2(fmaxf(y.x, 0.f), fmaxf(y.y, 0.f));
  if constexpr (kGradient) above = make_float2(fminf(above.x, kMost), fminf(above.y, kMost));
  g.soft = fma_2(v, p, above);
  const float2 w = mul_2(alpha, g.soft);
  p = fma_2(w, two(-0.00015403463f), two(0.00134455867f));
  p = fma_2(w, p, two(-0.00961854495f));
  p = fma_1(w, p, two(0.05550206453f));
  p = fma_1(w, p, two(-0.24022643268f));
  p = fma_1(w, p, two(0.69314724207f));
  const float2 e = make_float2(w.x * p.x, w.y * p.y);
  const float2 f = make_float2(ex2_fast(-w.x), ex2_fast(-w.y)), far = fma_2(f, two(-1.f), two(1.f));
  const bool near0 = fabsf(w.x) <= 0.7f, near1 = fabsf(w.y) <= 0.7f;
  g.e = make_float2(near0 ? e.x : far.x, near1 ? e.y : far.y);
  const float2 rest = make_float2(fmaf(-w.x, p.x, 1.f), fmaf(-w.y, p.y, 1.f));
  g.f = make_float2(near0 ? rest.x : f.x, near1 ? rest.y : f.y);
  return g;
}

// ---------------------------------------------------------------------------
// The exchange
// ---------------------------------------------------------------------------
struct Exchange {
  float4 warp[2][kWarps][32];        // F, U of the block's segments
  float4 block[2][kMaxCluster][32];  // of the cluster's tiles
  alignas(8) uint64_t arrived[2];    // a phase for each second round: every tile's F and U are there
  alignas(8) uint64_t full[3];       // the ring's
  int abort_flag;                    // a wait of the block gave up
  int fills, rounds;                 // the ring's tiles that thread 0 asked for, the rounds
  int failed, armed;                 // the round whose exchange thread 0 gave up (-1: none), and whether it had arrived
  __device__ __forceinline__ bool alive() const { return *const_cast<const volatile int*>(&abort_flag) == 0; }
};

__device__ __forceinline__ void open_exchange(Exchange& x, int rounds, int blocks) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&x.arrived[i]), 1);
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&x.full[i]), 1);
    x.abort_flag = x.fills = x.armed = 0;
    x.rounds = rounds;
    x.failed = -1;
    fence_mbar_init_cluster();
  }
  if (blocks > 1)
    cluster_sync_all();
  else
    __syncthreads();
}

constexpr float kSpoilt = __builtin_nanf("");
constexpr int kRoundBytes = 32 * 16;  // of a block's F and U

// The state before the warp's segment, from `carry`, the state before the
// round; carry goes on to the next round.  Every thread of the cluster calls it.
// A block hands its F and U to every block of the cluster by stores that count
// on the receiver's mbarrier: a cluster barrier's release would wait for the
// outputs stored before it.  Buffers of two rounds serve: nobody sends for round
// i + 2 before it has what this block sent for round i + 1, after this block was
// done with round i; and nobody ends before all that is sent to it has come.
// A wait that gives up (seconds) spoils the state with NaN, and the block neither
// waits, arrives nor sends any more: the others of its cluster, which miss what
// it would have sent, give up in their turn, and nobody sends for a round that
// the receiver has not got to (which would count in the wrong phase).
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
    const bool alive = x.alive();
    if (alive && warp < blocks) {
      const uint32_t to = mapa_shared(smem_u32(&x.block[buf][rank][lane]), warp), at = mapa_shared(bar, warp);
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                   "f"(tF.x), "f"(tF.y), "f"(tU.x), "f"(tU.y), "r"(at)
                   : "memory");
    }
    if (alive && threadIdx.x == 0) mbar_arrive_expect_tx(bar, blocks * kRoundBytes);
    if (!alive || !mbar_wait<true>(bar, (round >> 1) & 1, &x.abort_flag, nullptr, 0)) {
      carry = two(kSpoilt);
      if (threadIdx.x == 0 && x.failed < 0) {
        x.failed = round;
        x.armed = alive;
      }
    }
    for (int r = 0; r < blocks; ++r) {
      if (r == rank) mine = carry;
      const float4 s = x.block[buf][r][lane];
      carry = fma_2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
    }
  }
  return fma_2(pF, mine, pU);
}

// Behind its rounds a block says that it sends no more, and it ends when all of
// its cluster have said so: one that gave up may be far ahead of the others.
// Without release: there is nothing to be seen but that.
__device__ __forceinline__ void done_sending(int blocks) {
  __syncwarp();
  if (blocks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
// The last that a block does.  If it gave up, what is still on its way to it lands
// first: tiles of the ring, and what the others sent for rounds that it did not
// take part in (its thread 0 does, here; not inlined, for registers).
template <typename Tiles>
__device__ __noinline__ void land(Exchange& x, int blocks) {
  drain<Tiles>(x.full, x.fills);
#pragma unroll 1
  for (int r = x.failed; r >= 0 && r < x.rounds; ++r) {
    const uint32_t bar = smem_u32(&x.arrived[r & 1]);
    if (r > x.failed || !x.armed) mbar_arrive_expect_tx(bar, blocks * kRoundBytes);
    if (!mbar_wait_timed<true>(bar, (r >> 1) & 1, nullptr, 0)) break;
  }
}
template <typename Tiles>
__device__ __forceinline__ void leave(Exchange& x, int blocks) {
  __syncwarp();
  if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0 && !x.alive()) land<Tiles>(x, blocks);
}

__device__ __forceinline__ uint8_t* align_smem(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 127) & ~static_cast<uintptr_t>(127));
}

__device__ __forceinline__ int length_of(const LinearArgs& A, int b) {
  return A.lengths != nullptr ? min(max(A.lengths[b], 0), A.T) : A.T;
}

// ---------------------------------------------------------------------------
// Forward: y, H_T; or (kStates) the state before each kEvery steps
// ---------------------------------------------------------------------------
template <typename E, bool kPair, bool kTma, bool kStates, int kL, int kEvery>
__global__ void __launch_bounds__(kThreads, 2) linear_forward_kernel(LinearArgs A, float* states, int blocks, int groups, int stall,
                                                                     const __grid_constant__ Maps<2> maps) {
  __shared__ Exchange xch;
  extern __shared__ uint8_t raw[];
  constexpr int kTile = kWarps * kL;
  const int chain = blockIdx.x / blocks, rank = blockIdx.x - chain * blocks;
  const int b = chain / groups, group = chain - b * groups, warp = threadIdx.x >> 5;
  const Lane<kPair> me(group, A.C);
  const int len = length_of(A, b);
  const int64_t first = static_cast<int64_t>(b) * A.T;
  const E* px = static_cast<const E*>(A.x) + first * A.x_stride + me.from;
  const E* pa = static_cast<const E*>(A.a) + first * A.a_stride + me.from;
  E* py = static_cast<E*>(A.y) + first * A.C + me.c;
  const float2 alpha = me.get(A.alpha), beta = shut(mul_2(me.get(A.beta), two(kLog2e)), alpha);
  float2 carry = me.get(A.H_0 != nullptr ? A.H_0 + static_cast<int64_t>(b) * A.C : nullptr);
  const int rounds = (len + kTile * blocks - 1) / (kTile * blocks);

  using Tiles = Ring<E, 2, kTile>;
  const Tiles ring{align_smem(raw), xch.full};
  const CUtensorMap* const from[2] = {&maps.m[0], &maps.m[1]};
  Raw2<E> ra[kTma ? 1 : kL], rx[kTma ? 1 : kL];
  open_exchange(xch, rounds, blocks);
  int t0 = rank * kTile + warp * kL;
  auto load = [&](int round) {  // the tile of a round, if it has steps
    if constexpr (kTma) {
      const int t = (round * blocks + rank) * kTile;
      if (threadIdx.x == 0 && t < len && xch.alive()) {
        xch.fills = round + 1;
        if (round != stall || blockIdx.x != 0) ring.fill(round % Tiles::kStages, from, group * kChan, t, b);
      }
    } else if (round < rounds) {
      load_rows<kPair>(ra, pa, A.a_stride, me.other, (round * blocks + rank) * kTile + warp * kL, len);
      load_rows<kPair>(rx, px, A.x_stride, me.other, (round * blocks + rank) * kTile + warp * kL, len);
    }
  };
  for (int i = 0; i < (kTma ? Tiles::kStages : 1); ++i) load(i);
  for (int it = 0; it < rounds; ++it) {
    const int stage = it % Tiles::kStages;
    if (kTma && (it * blocks + rank) * kTile < len &&
        !mbar_wait(smem_u32(ring.full + stage), (it / Tiles::kStages) & 1, &xch.abort_flag, nullptr, 0))
      carry = two(kSpoilt);
    float2 f[kL], in[kL], F = two(1.f), U = two(0.f);
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const Raw2<E> a = kTma ? load_2<true>(ring.row(stage, 0, warp * kL + i), 0) : ra[kTma ? 0 : i];
      const Raw2<E> x = kTma ? load_2<true>(ring.row(stage, 1, warp * kL + i), 0) : rx[kTma ? 0 : i];
      const Gate2 g = gate_of<false>(fma_2(a.f(), two(kLog2e), beta), alpha);
      f[i] = g.f;
      in[i] = mul_2(g.e, x.f());
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
      U = fma_1(f[i], U, in[i]);
      F = make_float2(f[i].x * F.x, f[i].y * F.y);
    }
    const int now = t0;
    t0 += kTile * blocks;
    if (!kTma) load(it + 1);
    float2 h = state_before(xch, it, F, U, carry, rank, blocks);
    if (kTma) load(it + Tiles::kStages);  // the block is done with this round's tile
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
          h = fma_1(f[i], h, in[i]);
          store_2<kPair>(p, h, me.in0, me.in1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kL; ++i, p += A.C) {
          h = fma_1(f[i], h, in[i]);
          if (now + i < A.T) store_2<kPair>(p, now + i < len ? h : two(0.f), me.in0, me.in1);
        }
      }
    }
  }
  done_sending(blocks);
  let_next();
  if constexpr (!kStates) {
    for (int t = rounds * kTile * blocks + rank * kWarps + warp; t < A.T; t += blocks * kWarps)
      store_2<kPair>(py + static_cast<int64_t>(t) * A.C, two(0.f), me.in0, me.in1);
    if (A.H_T != nullptr && rank == 0 && warp == 0) me.put(A.H_T + static_cast<int64_t>(b) * A.C, carry);
  }
  leave<Tiles>(xch, blocks);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <typename E, bool kPair, bool kTma, int kL>
__global__ void __launch_bounds__(kThreads, 2) linear_backward_kernel(LinearArgs A, const float* states, float* part, int blocks,
                                                                      int groups, int stall, const __grid_constant__ Maps<3> maps) {
  __shared__ Exchange xch;
  extern __shared__ uint8_t raw[];
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
  const float2 alpha = me.get(A.alpha), beta = mul_2(me.get(A.beta), two(kLog2e));
  const float2 minus_alpha = make_float2(-alpha.x, -alpha.y);
  float2 carry = me.get(A.dH_T != nullptr ? A.dH_T + static_cast<int64_t>(b) * A.C : nullptr);
  float2 sa = two(0.f), sb = two(0.f);
  const int tiles = (len + kTile - 1) / kTile, rounds = (tiles + blocks - 1) / blocks;

  // Rounds go from the end: block 0 has the last tile, warp 0 the last segment of it.
  int t0 = ((tiles - 1 - rank) * kWarps + kWarps - 1 - warp) * kL;
  using Tiles = Ring<E, 3, kTile>;
  const Tiles ring{align_smem(raw), xch.full};
  const CUtensorMap* const from[3] = {&maps.m[0], &maps.m[1], &maps.m[2]};
  Raw2<E> ra[kTma ? 1 : kL], rx[kTma ? 1 : kL], rd[kTma ? 1 : kL];
  float2 hs = two(0.f);
  auto load = [&](int round) {  // the tile of a round; before the sequence as behind it: zeros
    const int tile = tiles - 1 - (round * blocks + rank);
    if constexpr (kTma) {
      if (threadIdx.x == 0 && tile >= 0 && xch.alive()) {
        xch.fills = round + 1;
        if (round != stall || blockIdx.x != 0) ring.fill(round % Tiles::kStages, from, group * kChan, tile * kTile, b);
      }
    } else if (round < rounds) {
      const int t = tile < 0 ? len : tile * kTile + (kWarps - 1 - warp) * kL;
      load_rows<kPair>(ra, pa, A.a_stride, me.other, t, len);
      load_rows<kPair>(rx, px, A.x_stride, me.other, t, len);
      load_rows<kPair>(rd, pd, A.C, me.other, t, len);
    }
  };
  auto load_state = [&](int t0) {
    if (t0 >= 0 && t0 < len) hs = me.get(ph + static_cast<int64_t>(t0 / kL) * A.C);
  };
  open_exchange(xch, rounds, blocks);
  for (int i = 0; i < (kTma ? Tiles::kStages : 1); ++i) load(i);
  wait_previous();
  if (rounds > 0) load_state(t0);
  for (int it = 0; it < rounds; ++it) {
    const int stage = it % Tiles::kStages, r0 = (kWarps - 1 - warp) * kL;
    if (kTma && tiles - 1 - (it * blocks + rank) >= 0 &&
        !mbar_wait(smem_u32(ring.full + stage), (it / Tiles::kStages) & 1, &xch.abort_flag, nullptr, 0))
      carry = two(kSpoilt);
    float2 f[kL], e[kL], ma[kL], ms[kL], dy[kL], F = two(1.f), U = two(0.f);
    float2 h = hs;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const Raw2<E> qa = kTma ? load_2<true>(ring.row(stage, 0, r0 + i), 0) : ra[kTma ? 0 : i];
      const Raw2<E> qx = kTma ? load_2<true>(ring.row(stage, 1, r0 + i), 0) : rx[kTma ? 0 : i];
      const Raw2<E> qd = kTma ? load_2<true>(ring.row(stage, 2, r0 + i), 0) : rd[kTma ? 0 : i];
      const float2 y = fma_2(qa.f(), two(kLog2e), beta), x = qx.f();
      const Gate2 g = gate_of<true>(y, alpha);
      f[i] = g.f;
      e[i] = g.e;
      const float2 w = add_2(g.t, two(1.f));
      const float2 sig = make_float2((y.x >= 0.f ? 1.f : g.t.x) * rcp_fast(w.x), (y.y >= 0.f ? 1.f : g.t.y) * rcp_fast(w.y));
      const float2 away = mul_2(g.f, make_float2(h.x - x.x, h.y - x.y));
      ma[i] = mul_2(away, mul_2(minus_alpha, sig));
      ms[i] = mul_2(away, make_float2(-g.soft.x, -g.soft.y));
      h = fma_2(g.f, h, mul_2(g.e, x));
      dy[i] = qd.f();
    }
    if (t0 < 0 || t0 + kL > len) {  // steps that are not there hand the gradient on
#pragma unroll
      for (int i = 0; i < kL; ++i)
        if (t0 < 0 || t0 + i >= len) {
          f[i] = two(1.f);
          ma[i] = ms[i] = dy[i] = two(0.f);
        }
    }
#pragma unroll
    for (int i = kL - 1; i >= 0; --i) {
      U = mul_2(f[i], add_2(dy[i], U));
      F = mul_2(f[i], F);
    }
    const int now = t0;
    t0 -= kTile * blocks;
    if (!kTma) load(it + 1);
    if (it + 1 < rounds) load_state(t0);
    float2 c = state_before(xch, it, F, U, carry, rank, blocks);
    if (kTma) load(it + Tiles::kStages);
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
  if (kTma && xch.abort_flag) drain<Tiles>(xch.full, xch.fills);  // (registers: not in leave alone)
  done_sending(blocks);
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
    me.put(p, make_float2(t.x * kLn2, t.y * kLn2));  // (softplus in units of log2)
    me.put(p + A.C, make_float2(t.z, t.w));
  }
  leave<Tiles>(xch, blocks);
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
  const float2 alpha = me.get(A.alpha);
  const Gate2 g = gate_of<false>(mul_2(add_2(a.f(), shut(me.get(A.beta), alpha)), two(kLog2e)), alpha);
  const float2 h = fma_2(g.f, me.get(H + at), mul_2(g.e, x.f()));
  me.put(H + at, h);
  store_2<kPair>(static_cast<E*>(A.y) + at + me.c, h, me.in0, me.in1);
}

// Sums over parts: a block has 8 columns, its threads take parts in turn, then
// add up as a tree.
constexpr int kSumThreads = 1024, kSumCols = 8, kSumRows = kSumThreads / kSumCols;
__global__ void __launch_bounds__(kSumThreads) sum_parts_kernel(const float* part, float* out, float* out2, int parts,
                                                                int64_t D, int64_t width) {
  __shared__ float red[kSumRows][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kSumCols + col;
  wait_previous();
  float t = 0.f;
  if (j < width) {
#pragma unroll 4
    for (int p = row; p < parts; p += kSumRows) t += part[p * width + j];
  }
  red[row][col] = t;
  __syncthreads();
  if (warp >= kSumCols) return;
  float v = 0.f;
#pragma unroll
  for (int r = 0; r < kSumRows; r += 32) v += red[r + lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kSumCols + warp;
  if (lane == 0 && k < D) out[k] = v;
  if (lane == 0 && k >= D && k < width && out2 != nullptr) out2[k - D] = v;
}

constexpr int kEveryBf16 = 8, kEveryF32 = 4;  // steps of a segment of the backward

// Clusters of `size` blocks of the kernel that the current device, `device`, runs at
// once (if it does not say: as many as two blocks to an SM would be).
template <typename... P>
int clusters_at_once(void (*kernel)(P...), int smem, int device, int size, ClusterFit& fit) {
  return fit.get(device, size, 304 / size, [&] {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = size;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(size);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.attrs = &at;
    c.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return 0;
  });
}

// Blocks to a cluster, each with a tile at least: the shortest of the waves of all
// clusters (152, 97, 74, 58, 46, 38, 36 of 2 to 8 blocks run at once, two blocks to
// an SM).  A block of r takes 1 / r of the steps, and 0.06 for the exchange, which
// grows with r; a last wave with one block to an SM takes 0.64.  44 chains of
// T=4096 bf16 take 22.0 us so, 26.3 with the power of two that first makes 240
// blocks, 90 take 38.8 and 42.7; 100 take 43.8 with 4 and 52.6 with 2 or 3.  With
// more than 152 clusters the waves overlap: 2 where that is shorter (200: 79.6 us,
// 90.9 with 1; 230: 96.8 and 91.3; more than 2 lose a third at T=512).
template <typename... P>
int cluster_blocks(void (*kernel)(P...), int smem, const LinearArgs& a, int tile, ClusterFit& fit) {
  const int64_t chains = static_cast<int64_t>(a.B) * ((a.C + kChan - 1) / kChan);
  const int tiles = (a.T + tile - 1) / tile;
  if (chains > 152) return chains <= 216 && tiles > 1 ? 2 : 1;
  int best = 1, device = -1;
  if (tiles > 1 && cudaGetDevice(&device) != cudaSuccess) (void)cudaGetLastError();
  float least = 1.06f;
  for (int r = 2; r <= kMaxCluster && r <= tiles; ++r) {
    const int at_once = clusters_at_once(kernel, smem, device, r, fit), left = static_cast<int>(chains) % at_once;
    const bool half = 2 * left <= at_once && chains > at_once;
    const float waves = static_cast<float>(chains / at_once) + (left == 0 ? 0.f : half ? 0.64f : 1.f);
    const float time = waves * (1.f / static_cast<float>(r) + 0.06f);
    if (time < least) {
      best = r;
      least = time;
    }
  }
  return best;
}

// How rows can be read: value by value, two channels at a time, or (on 16 bytes)
// by TMA, which took B=2 T=16384 C=1024 bf16 from 79 to 67 us.
enum class Access { kSingle, kPair, kTma };
Access access_of(const LinearArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.a);
  const int e = a.bf16 ? 2 : 4;
  auto all = [&](int bytes) {
    return a.C * e % bytes == 0 && a.x_stride * e % bytes == 0 && a.a_stride * e % bytes == 0 && at % bytes == 0;
  };
  return all(16) ? Access::kTma : all(2 * e) ? Access::kPair : Access::kSingle;
}

// Tiles of `rows` steps of 64 channels of [B,T,C].
bool map_rows(CUtensorMap* m, const LinearArgs& a, const void* p, int64_t stride, int rows) {
  const uint64_t e = a.bf16 ? 2 : 4;
  const uint64_t dims[3] = {static_cast<uint64_t>(a.C), static_cast<uint64_t>(a.T), static_cast<uint64_t>(a.B)};
  const uint64_t strides[2] = {stride * e, stride * e * a.T};
  const uint32_t box[3] = {kChan, static_cast<uint32_t>(rows), 1};
  return make_tensor_map(m, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p, 3, dims, strides,
                         box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <typename E, bool kPair, bool kTma, bool kStates, int kL, int kEvery>
cudaError_t forward(const LinearArgs& a, float* states, cudaStream_t s) {
  constexpr int kTile = kWarps * kL, kSmem = kTma ? Ring<E, 2, kTile>::kBytes + 128 : 0;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = linear_forward_kernel<E, kPair, kTma, kStates, kL, kEvery>;
  Maps<2> maps{};
  if constexpr (kTma) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, ready);
    if (e != cudaSuccess) return e;
    if (!map_rows(&maps.m[0], a, a.a, a.a_stride, kTile) || !map_rows(&maps.m[1], a, a.x, a.x_stride, kTile))
      return cudaErrorInvalidValue;
  }
  static ClusterFit fit;
  const int groups = (a.C + kChan - 1) / kChan, blocks = cluster_blocks(kernel, kSmem, a, kTile, fit);
  return launch_cluster(kernel, static_cast<int64_t>(a.B) * groups * blocks, blocks, kThreads, kSmem, false, s, a, states, blocks, groups,
                        option_test_stall_tile(), maps);
}

template <typename E, bool kPair, bool kTma, int kL, int kEvery>
cudaError_t backward(const LinearArgs& a, cudaStream_t s) {
  constexpr int kTile = kWarps * kEvery, kSmem = kTma ? Ring<E, 3, kTile>::kBytes + 128 : 0;
  float* part = static_cast<float*>(a.ws);
  float* states = part + static_cast<int64_t>(a.B) * kMaxCluster * 2 * a.C;
  cudaError_t e = forward<E, kPair, kTma, true, kL, kEvery>(a, states, s);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};
  const auto kernel = linear_backward_kernel<E, kPair, kTma, kEvery>;
  Maps<3> maps{};
  if constexpr (kTma) {
    e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, ready);
    if (e != cudaSuccess) return e;
    if (!map_rows(&maps.m[0], a, a.a, a.a_stride, kTile) || !map_rows(&maps.m[1], a, a.x, a.x_stride, kTile) ||
        !map_rows(&maps.m[2], a, a.dy, a.C, kTile))
      return cudaErrorInvalidValue;
  }
  static ClusterFit fit;
  const int groups = (a.C + kChan - 1) / kChan, blocks = cluster_blocks(kernel, kSmem, a, kTile, fit);
  e = launch_cluster(kernel, static_cast<int64_t>(a.B) * groups * blocks, blocks, kThreads, kSmem, true, s, a, states, part, blocks, groups,
                     option_test_stall_tile(), maps);
  if (e != cudaSuccess) return e;
  return launch_sum_parts(part, a.dalpha, a.dbeta, true, a.B * blocks, a.C, s);
}

}  // namespace

size_t linear_backward_scratch_bytes(int64_t B, int64_t T, int64_t C) {
  return static_cast<size_t>(B) * C * 4 * (2 * kMaxCluster + (T + kEveryF32 - 1) / kEveryF32);
}

cudaError_t launch_sum_parts(const float* part, float* out, float* out2, bool two, int parts, int64_t D, cudaStream_t s) {
  const int64_t width = two ? 2 * D : D;
  return launch_next(sum_parts_kernel, static_cast<unsigned>((width + kSumCols - 1) / kSumCols), kSumThreads, 0, s, part, out, out2, parts, D, width);
}

// Steps of a segment: 16 in bf16, 8 in fp32 (registers); of the backward's, kEvery.
cudaError_t launch_linear_forward(const LinearArgs& a, cudaStream_t s) {
  switch (access_of(a)) {
    case Access::kTma:
      return a.bf16 ? forward<uint16_t, true, true, false, 16, kEveryBf16>(a, nullptr, s)
                    : forward<float, true, true, false, 8, kEveryF32>(a, nullptr, s);
    case Access::kPair:
      return a.bf16 ? forward<uint16_t, true, false, false, 16, kEveryBf16>(a, nullptr, s)
                    : forward<float, true, false, false, 8, kEveryF32>(a, nullptr, s);
    default:
      return a.bf16 ? forward<uint16_t, false, false, false, 16, kEveryBf16>(a, nullptr, s)
                    : forward<float, false, false, false, 8, kEveryF32>(a, nullptr, s);
  }
}

cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s) {
  switch (access_of(a)) {
    case Access::kTma:
      return a.bf16 ? backward<uint16_t, true, true, 16, kEveryBf16>(a, s) : backward<float, true, true, 8, kEveryF32>(a, s);
    case Access::kPair:
      return a.bf16 ? backward<uint16_t, true, false, 16, kEveryBf16>(a, s) : backward<float, true, false, 8, kEveryF32>(a, s);
    default:
      return a.bf16 ? backward<uint16_t, false, false, 16, kEveryBf16>(a, s)
                    : backward<float, false, false, 8, kEveryF32>(a, s);
  }
}

cudaError_t launch_linear_step(float* H, const LinearArgs& a, cudaStream_t s) {
  const int groups = (a.C + kChan - 1) / kChan;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.B) * groups + 3) / 4);
  if (access_of(a) != Access::kSingle) {
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
