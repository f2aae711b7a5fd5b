// Forward of the selective state space scan on tensor cores (bf16 inputs; the
// mathematics in ssm.cu), in chunks of 64 steps.  A sequence is cut into
// segments of chunks, enough of them to fill the GPU:
//   1. decays of every chunk;
//   2. a block per (head, value slice, segment) walks the segment's chunks
//      with the state in its warps' accumulators, from zero (the first segment
//      from H_0), and leaves the state before each chunk, in fp32;
//   3. a scan over the segments: the state before each, and H_T;
//   4. a block per (head, value slice, chunk), all independent: the outputs
//        y_i = first_i (S + (decay since the segment's start) S0)^T q_i
//              + sum_j P_ij v_j + w_r (*) v_i,
//      S the segment's own state before the chunk, S0 the state before the
//      segment, P the decayed scores.
// 64 x 64 states with tiles enough take phases 2 and 4 on tcgen05, 128 steps at
// a time (ssm_tc_walk.cu, ssm_tc.cu).
// y is the fp32 result rounded once: the joined state and P enter their
// products as two bf16 parts each, good to 2^-16, 1/256 of y's own rounding
// (one part each made y's error a fifth larger than its rounding, for 24 us less
// at B=2 heads=16 T=16384 64x64 on tcgen05, 96 and 120), and differences of
// sums of log decays keep their low parts.  The states themselves stay good to
// fp32: k_j exp(l_63 - l_j) D_j is split into three bf16 parts (v is exact),
// their products are summed from the smallest part up, and the chunk's sum is
// added to the state by an fp32 FMA, so that the tensor core's truncating adds
// never see the running state.
//
// B=4 heads=16 T=4096 64x64, shared q and k: 88 us (65 with tcgen05).  B=8
// heads=16 T=4096 128x128: 609 us, of which decays 7, walk 234, outputs 368:
// the walk is bound by the latency of its MMAs and of the operand split (8
// warps to an SM, by registers), the outputs by the states that they read (537
// MB in all) with as few warps, by shared memory.
//
// The state is held transposed, V rows by K columns: an accumulator fragment
// of it, packed to bf16, is as it stands the B operand of Q S, so states go
// from the walk to the outputs as fragments, without a transposition.
#include <cuda_runtime.h>

#include <cstdint>

#include "ssm_mma.cuh"
#include "ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;  // four warps

// One warp per (chain, chunk), two steps a lane; a block takes the same chunk
// of eight heads, whose dt lie side by side.  Sums run within a block of 16
// steps first and only from there over the blocks, each from its own end: no
// two long sums are ever subtracted, so fp32 is enough.
template <bool kGrad>
__global__ void __launch_bounds__(256) ssm_decay_kernel(SsmArgs A, void* out, float* tot, int nc,
                                                        StatusBlock* status) {
  if (blockIdx.x == 0 && threadIdx.x < sizeof(StatusBlock) / 4) reinterpret_cast<unsigned*>(status)[threadIdx.x] = 0u;
  const int lane = threadIdx.x & 31, heads = (A.N + 7) / 8, own = lane >> 3;
  const unsigned bc = blockIdx.x / heads;
  const int n = (blockIdx.x - bc * heads) * 8 + (threadIdx.x >> 5), b = bc / nc, c = bc - b * nc;
  if (n >= A.N) return;
  const int64_t id = (static_cast<int64_t>(b) * A.N + n) * nc + c;
  const int len = ssm_len(A, b), t = c * kChunk + 2 * lane;
  const uint16_t* p = static_cast<const uint16_t*>(A.dt) + (static_cast<int64_t>(b) * A.T + t) * A.dt_stride + n;
  const float bias = A.dt_bias ? A.dt_bias[n] : 0.f, An = A.A[n];
  const float x0 = t < len ? to_f32(p[0]) + bias : 0.f, x1 = t + 1 < len ? to_f32(p[A.dt_stride]) + bias : 0.f;
  const float D0 = t < len ? softplus_f(x0) : 0.f, D1 = t + 1 < len ? softplus_f(x1) : 0.f;
  const float a0 = log_decay(D0, An), a1 = log_decay(D1, An);
  // Within the block of 16 steps: the sum up to a step, and the sum behind it.
  float up = a0 + a1, down = up, low = two_sum_low(a0, a1, up);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, up, o, 8), y = __shfl_down_sync(0xffffffffu, down, o, 8);
    const float z = __shfl_up_sync(0xffffffffu, low, o, 8);
    if ((lane & 7) >= o) {
      const float s = up + x;
      low += z + two_sum_low(up, x, s);
      up = s;
    }
    if ((lane & 7) + o < 8) down += y;
  }
  float before = __shfl_up_sync(0xffffffffu, up, 1, 8), behind = __shfl_down_sync(0xffffffffu, down, 1, 8);
  float before_low = __shfl_up_sync(0xffffffffu, low, 1, 8);
  if ((lane & 7) == 0) before = before_low = 0.f;
  if ((lane & 7) == 7) behind = 0.f;
  const float r0 = before + a0, r1 = up, s0 = behind + a1, s1 = behind;
  float T[4];  // the blocks' sums
#pragma unroll
  for (int i = 0; i < 4; ++i) T[i] = __shfl_sync(0xffffffffu, up, 8 * i + 7);
  const float base = own == 0 ? 0.f : own == 1 ? T[0] : own == 2 ? T[0] + T[1] : T[0] + T[1] + T[2];
  const float rest = own == 3 ? 0.f : own == 2 ? T[3] : own == 1 ? T[3] + T[2] : T[3] + T[2] + T[1];
  let_next();
  ChunkDecay& d = kGrad ? static_cast<ChunkDecayGrad*>(out)[id].d : static_cast<ChunkDecay*>(out)[id];
  const int i = 2 * lane;
  auto put = [&](float* at, float x, float y) { *reinterpret_cast<float2*>(at + i) = make_float2(x, y); };
  const float e0 = expf(s0 + rest), e1 = expf(s1 + rest);
  put(d.D, D0, D1);
  put(d.rel, r0, r1);
  put(d.rel_lo, before_low + two_sum_low(before, a0, r0), low);
  put(d.row, expf(r0), expf(r1));
  put(d.first, expf(base + r0), expf(base + r1));
  put(d.wD, e0 * D0, e1 * D1);
#pragma unroll
  for (int ib = 1; ib < 4; ++ib) {
    // From the end of the step's block to the start of block ib.
    float mid = 0.f;
#pragma unroll
    for (int x = 1; x < ib; ++x) mid += own < x ? T[x] : 0.f;
    const bool past = own < ib;
    put(d.col[ib - 1], past ? expf(s0 + mid) * (kGrad ? 1.f : D0) : 0.f, past ? expf(s1 + mid) * (kGrad ? 1.f : D1) : 0.f);
  }
  if (kGrad) {
    ChunkDecayGrad& dg = static_cast<ChunkDecayGrad*>(out)[id];
    put(dg.last, e0, e1);
    put(dg.sg, 1.f / (1.f + expf(-x0)), 1.f / (1.f + expf(-x1)));
  }
  if (lane == 0) tot[id] = expf(T[0] + T[1] + T[2] + T[3]);
}

struct ScanArgs {
  SsmArgs a;
  const ChunkDecay* decay;  // [B N][chunks]
  const float* tot;         // [B N][chunks]: exp(l_63)
  float* since;             // [B N][chunks]: decay from the segment's start to the chunk's
  float4* local;            // [B N][slices][chunks][2 x fragments]: a segment's own state before each chunk
  float4* sums;             // [B N][slices][segs][2 x fragments]: the state each segment leaves
  float* seg_tot;           // [B N][segs]
  float4* start;            // [B N][slices][segs][2 x fragments]: the state before each segment (kTile, for the tiles
                            // of ssm_tc.cu: in the order of tc_piece_at)
  int nc, segs, per_seg, slices;
  bool vq, vk, vv;          // rows that asynchronous copies can take
};

// A fragment: 16 state rows kt by 16 value columns vt, 32 lanes of 8 values
// (k, v) = (16 kt + 8 b + 2 (lane % 4) + e, 16 vt + 8 h + lane / 4), in order
// h, b, e: as bf16 pairs the B operands of value tiles 2 vt and 2 vt + 1.  In
// fp32 two float4 (h), in one bf16 part a uint4.
template <int KP, int VS>
struct Frag {
  static constexpr int kVt = VS / 16, kCount = (KP / 16) * kVt * 32;  // per state of a slice
  static __device__ __forceinline__ int at(int kt, int vt, int lane) { return (kt * kVt + vt) * 32 + lane; }
};

template <int KP, int VS>
struct WalkShape {
  static constexpr int kNw = KP >= 64 ? 4 : KP / 16, kMw = 4 / kNw;  // warps along K (16 columns and more), V
  static constexpr int kKt = KP / 16 / kNw;                          // a warp's 16-column tiles
  static constexpr int kVt = VS / 16 >= kMw ? VS / 16 / kMw : 1;     // and its 16-row tiles
  static constexpr int kK = Tile<KP>::kBytes(kChunk), kV = Tile<VS>::kBytes(kChunk), kStage = kK + kV + kChunk * 4;
  static constexpr int kBytes = 2 * kStage;
  static constexpr int kBlocks = KP * VS > 4096 ? 2 : 3;  // per SM (registers)
};

// Phase 2.
template <int KP, int VS>
__global__ void __launch_bounds__(kThreads, WalkShape<KP, VS>::kBlocks) ssm_walk_kernel(ScanArgs W) {
  using Sh = WalkShape<KP, VS>;
  using Fr = Frag<KP, VS>;
  extern __shared__ __align__(16) uint8_t smem[];
  wait_previous();
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int nw = warp % Sh::kNw, mw = warp / Sh::kNw;
  const bool busy = mw * Sh::kVt < VS / 16;
  const unsigned head = blockIdx.x / W.segs;  // (chain, slice)
  const int seg = blockIdx.x - head * W.segs, bn = head / W.slices, slice = head - bn * W.slices;
  const int b = bn / A.N, n = bn % A.N, gq = n / (A.N / A.G), K = A.K, V = A.V, v0 = slice * VS;
  const int len = ssm_len(A, b), width = min(VS, V - v0);
  const int c0 = seg * W.per_seg, c1 = min(W.nc, c0 + W.per_seg);
  const int live = min(c1, (len + kChunk - 1) / kChunk);  // chunks with steps in them

  const uint32_t base = smem_u32(smem);
  const int64_t row = static_cast<int64_t>(b) * A.T;
  const TileLoader<KP, kThreads> lk{static_cast<const uint16_t*>(A.k) + row * A.k_stride + static_cast<int64_t>(gq) * K,
                                    A.k_stride, K, W.vk};
  const TileLoader<VS, kThreads> lv{
      static_cast<const uint16_t*>(A.v) + row * A.v_stride + static_cast<int64_t>(n) * V + v0, A.v_stride, width, W.vv};
  const ChunkDecay* pd = W.decay + static_cast<int64_t>(bn) * W.nc;
  const float* ptot = W.tot + static_cast<int64_t>(bn) * W.nc;
  auto load_chunk = [&](int c) {
    const uint32_t st = base + (c & 1) * Sh::kStage;
    lk.load(st, c * kChunk, len);
    lv.load(st + Sh::kK, c * kChunk, len);
    if (tid < kChunk / 4) cp_async_16(st + Sh::kK + Sh::kV + tid * 16, pd[c].wD + tid * 4, true);
    cp_async_commit();
  };

  // The state, transposed: rows (value columns) 16 (mw kVt + vt) + g (+ 8), columns (state
  // rows) 16 (nw kKt + kt) + 8 b + 2 q4 (+ 1).
  float S[Sh::kVt][Sh::kKt][2][4];
  auto each = [&](auto f) {
#pragma unroll
    for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
      for (int kt = 0; kt < Sh::kKt; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 16 * (mw * Sh::kVt + vt) + g + 8 * (e >> 1);
            const int k = 16 * (nw * Sh::kKt + kt) + 8 * h + 2 * q4 + (e & 1);
            f(S[vt][kt][h][e], k, v, busy && k < K && v < width);
          }
  };
  const float* from = seg == 0 && A.H_0 ? A.H_0 + static_cast<int64_t>(bn) * K * V : nullptr;
  each([&](float& s, int k, int v, bool ok) { s = from != nullptr && ok ? from[k * V + v0 + v] : 0.f; });

  float tot = 0.f, decay = 1.f;  // of a chunk; since the segment's start
  float4* local = W.local + (static_cast<int64_t>(head) * W.nc + c0) * (2 * Fr::kCount);
  if (c0 < live) {
    load_chunk(c0);
    tot = ptot[c0];
  }
  for (int c = c0; c < live; ++c) {
    cp_async_wait<0>();
    __syncthreads();
    const float tot_c = tot;
    if (c + 1 < live) {
      load_chunk(c + 1);
      tot = ptot[c + 1];
    }
    if (slice == 0 && tid == 0) W.since[static_cast<int64_t>(bn) * W.nc + c] = decay;
    decay *= tot_c;
    const int stage = (c & 1) * Sh::kStage;
    const uint32_t sK = base + stage, sV = sK + Sh::kK;
    const float* wD = reinterpret_cast<const float*>(smem + stage + Sh::kK + Sh::kV);
    if (busy) {
#pragma unroll
      for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
        for (int kt = 0; kt < Sh::kKt; ++kt) {
          const auto& s = S[vt][kt];
          float4* to = local + 2 * Fr::at(nw * Sh::kKt + kt, mw * Sh::kVt + vt, lane);
          to[0] = make_float4(s[0][0], s[0][1], s[1][0], s[1][1]);
          to[1] = make_float4(s[0][2], s[0][3], s[1][2], s[1][3]);
        }
      local += 2 * Fr::kCount;
      float U[Sh::kVt][Sh::kKt][2][4] = {};
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        uint32_t vf[Sh::kVt][4];
#pragma unroll
        for (int vt = 0; vt < Sh::kVt; ++vt)
          ldmatrix_x4_trans(vf[vt], at_cols<VS>(sV, 16 * jt, 16 * (mw * Sh::kVt + vt), lane));
        const int j = 16 * jt + 2 * q4;
        const float2 wa = *reinterpret_cast<const float2*>(&wD[j]), wb = *reinterpret_cast<const float2*>(&wD[j + 8]);
#pragma unroll
        for (int kt = 0; kt < Sh::kKt; ++kt) {
          uint32_t kf[4], hi[4], mid[4], lo[4];
          ldmatrix_x4_trans(kf, at_rows<KP>(sK, 16 * jt, 16 * (nw * Sh::kKt + kt), lane));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 w = r & 1 ? wb : wa;
            split3_weighted(kf[r], w.x, w.y, hi[r], mid[r], lo[r]);
          }
#pragma unroll
          for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16_16816(U[vt][kt][h], vf[vt], lo[2 * h], lo[2 * h + 1]);
#pragma unroll
          for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16_16816(U[vt][kt][h], vf[vt], mid[2 * h], mid[2 * h + 1]);
#pragma unroll
          for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_bf16_16816(U[vt][kt][h], vf[vt], hi[2 * h], hi[2 * h + 1]);
        }
      }
#pragma unroll
      for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
        for (int kt = 0; kt < Sh::kKt; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[vt][kt][h][e] = fmaf(tot_c, S[vt][kt][h][e], U[vt][kt][h][e]);
    }
  }
  let_next();
  if (W.segs == 1) {
    if (A.H_T != nullptr)
      each([&](float& s, int k, int v, bool ok) {
        if (ok) A.H_T[static_cast<int64_t>(bn) * K * V + k * V + v0 + v] = s;
      });
    return;
  }
  if (busy) {
    float4* to = W.sums + ((static_cast<int64_t>(bn) * W.slices + slice) * W.segs + seg) * (2 * Fr::kCount);
#pragma unroll
    for (int vt = 0; vt < Sh::kVt; ++vt)
#pragma unroll
      for (int kt = 0; kt < Sh::kKt; ++kt) {
        const auto& s = S[vt][kt];
        const int at = Fr::at(nw * Sh::kKt + kt, mw * Sh::kVt + vt, lane);
        to[2 * at] = make_float4(s[0][0], s[0][1], s[1][0], s[1][1]);
        to[2 * at + 1] = make_float4(s[0][2], s[0][3], s[1][2], s[1][3]);
      }
  }
  if (tid == 0 && slice == 0) W.seg_tot[static_cast<int64_t>(bn) * W.segs + seg] = decay;
}

// Phase 3: block (chain and slice, 256 halves of fragments); thread (fragment, h).
template <int KP, int VS, bool kTile>
__global__ void __launch_bounds__(256) ssm_segment_scan_kernel(ScanArgs W) {
  using Fr = Frag<KP, VS>;
  constexpr int kAhead = 8, kN = 2 * Fr::kCount;
  if (kTile) let_next();  // a persistent kernel, which has barriers and tensor memory to set up meanwhile
  wait_previous();
  const SsmArgs& A = W.a;
  const int e = blockIdx.y * 256 + threadIdx.x;
  if (e >= kN) return;
  const int64_t bn = blockIdx.x / W.slices;
  const int slice = blockIdx.x % W.slices;
  const int lane = (e >> 1) & 31, tile = e >> 6, vt = tile % Fr::kVt, kt = tile / Fr::kVt;
  const int v = 16 * vt + 8 * (e & 1) + (lane >> 2), k = 16 * kt + 2 * (lane & 3);  // (and k + 1, k + 8, k + 9)
  const float4* sums = W.sums + static_cast<int64_t>(blockIdx.x) * W.segs * kN + e;
  float4* start = W.start + static_cast<int64_t>(blockIdx.x) * W.segs * kN;
  const float* tot = W.seg_tot + bn * W.segs;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < W.segs; i += kAhead) {
    float4 u[kAhead];
    float a[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= W.segs) continue;
      u[j] = sums[static_cast<int64_t>(i + j) * kN];
      a[j] = tot[i + j];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= W.segs) continue;
      if constexpr (kTile) {
        float* out = reinterpret_cast<float*>(start + static_cast<int64_t>(i + j) * kN);
        *reinterpret_cast<float2*>(out + 4 * tc_piece_at(k, v) + (k & 3)) = make_float2(s.x, s.y);
        *reinterpret_cast<float2*>(out + 4 * tc_piece_at(k + 8, v) + (k & 3)) = make_float2(s.z, s.w);
      } else {
        start[static_cast<int64_t>(i + j) * kN + e] = s;
      }
      s = make_float4(fmaf(a[j], s.x, u[j].x), fmaf(a[j], s.y, u[j].y), fmaf(a[j], s.z, u[j].z),
                      fmaf(a[j], s.w, u[j].w));
    }
  }
  if (!kTile) let_next();
  if (A.H_T == nullptr || slice * VS + v >= A.V) return;
  float* H = A.H_T + bn * A.K * A.V + slice * VS + v;
  const float x[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int kk = k + 8 * (r >> 1) + (r & 1);
    if (kk < A.K) H[kk * A.V] = x[r];
  }
}

template <int KP, int VS>
struct OutShape {
  static constexpr int kQ = Tile<KP>::kBytes(kChunk), kV = Tile<VS>::kBytes(kChunk), kS = Frag<KP, VS>::kCount * 16;
  static constexpr int kBytes = 2 * kQ + kV + kChunkDecayCopied + 2 * kS + VS * 4;
  static constexpr int kBlocks = KP * VS > 4096 ? 2 : 4;
};

// Phase 4.
template <int KP, int VS>
__global__ void __launch_bounds__(kThreads, OutShape<KP, VS>::kBlocks) ssm_out_kernel(ScanArgs W) {
  using Sh = OutShape<KP, VS>;
  using Fr = Frag<KP, VS>;
  static_assert(VS <= KP, "outputs pass through the q tile");
  constexpr int kKt = KP / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_from[VS];  // the first step at which a value column is not finite
  wait_previous();
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const unsigned head = blockIdx.x / W.nc;  // (chain, slice)
  const int c = blockIdx.x - head * W.nc, bn = head / W.slices, slice = head - bn * W.slices;
  const int b = bn / A.N, n = bn % A.N, gq = n / (A.N / A.G), K = A.K, V = A.V, v0 = slice * VS;
  const int len = ssm_len(A, b), width = min(VS, V - v0), t0 = c * kChunk, seg = c / W.per_seg;
  const int64_t row = static_cast<int64_t>(b) * A.T;
  uint16_t* y = static_cast<uint16_t*>(A.y) + ((row + t0) * A.N + n) * V + v0;
  const int64_t y_stride = static_cast<int64_t>(A.N) * V;
  if (t0 >= len) {  // behind the sequence's end
    for (int e = tid; e < min(kChunk, A.T - t0) * width; e += kThreads) y[(e / width) * y_stride + e % width] = 0;
    return;
  }
  const uint32_t sQ = smem_u32(smem), sK = sQ + Sh::kQ, sV = sK + Sh::kQ, sD = sV + Sh::kV;
  const ChunkDecay& d = *reinterpret_cast<const ChunkDecay*>(smem + 2 * Sh::kQ + Sh::kV);  // without wD
  uint4* fS = reinterpret_cast<uint4*>(smem + 2 * Sh::kQ + Sh::kV + kChunkDecayCopied);  // hi, then lo
  float* s_wr = reinterpret_cast<float*>(smem + 2 * Sh::kQ + Sh::kV + kChunkDecayCopied + 2 * Sh::kS);
  const TileLoader<KP, kThreads> lq{static_cast<const uint16_t*>(A.q) + row * A.q_stride + static_cast<int64_t>(gq) * K,
                                    A.q_stride, K, W.vq};
  const TileLoader<KP, kThreads> lk{static_cast<const uint16_t*>(A.k) + row * A.k_stride + static_cast<int64_t>(gq) * K,
                                    A.k_stride, K, W.vk};
  const TileLoader<VS, kThreads> lv{
      static_cast<const uint16_t*>(A.v) + row * A.v_stride + static_cast<int64_t>(n) * V + v0, A.v_stride, width, W.vv};
  const bool more = seg > 0;  // a state before the segment
  lq.load(sQ, t0, len);
  lk.load(sK, t0, len);
  const int64_t at = static_cast<int64_t>(bn) * W.nc + c;
  static_assert(kChunkDecayCopied == 16 * kThreads, "a copy a thread");
  cp_async_16(sD + tid * 16, reinterpret_cast<const uint8_t*>(W.decay + at) + tid * 16, true);
  lv.load(sV, t0, len);
  cp_async_commit();
  {  // The state before the chunk, joined and in two parts.
    const float4* l = W.local + ((static_cast<int64_t>(bn) * W.slices + slice) * W.nc + c) * (2 * Fr::kCount);
    const float4* s = W.start + ((static_cast<int64_t>(bn) * W.slices + slice) * W.segs + seg) * (2 * Fr::kCount);
    const float since = more ? W.since[at] : 0.f;
    auto part = [&](const float4& own, const float4& before, uint32_t* hi, uint32_t* lo) {
      split2(fmaf(since, before.x, own.x), fmaf(since, before.y, own.y), hi[0], lo[0]);
      split2(fmaf(since, before.z, own.z), fmaf(since, before.w, own.w), hi[1], lo[1]);
    };
    constexpr int kPer = (Fr::kCount + kThreads - 1) / kThreads, kMost = Sh::kBlocks == 2 ? 8 : 4,
                  kBatch = kPer < kMost ? kPer : kMost;
#pragma unroll
    for (int i0 = 0; i0 < kPer; i0 += kBatch) {
      float4 own[kBatch][2], before[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = (i0 + i) * kThreads + tid;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          own[i][h] = before[i][h] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e >= Fr::kCount) continue;
          own[i][h] = l[2 * e + h];
          if (more) before[i][h] = s[2 * e + h];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = (i0 + i) * kThreads + tid;
        if (e >= Fr::kCount) continue;
        uint32_t hi[4], lo[4];
        part(own[i][0], before[i][0], hi, lo);
        part(own[i][1], before[i][1], hi + 2, lo + 2);
        fS[e] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        fS[Fr::kCount + e] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  for (int e = tid; e < VS; e += kThreads)
    s_wr[e] = A.w_r != nullptr && e < width ? to_f32(static_cast<const uint16_t*>(A.w_r)[n * V + v0 + e]) : 0.f;
  cp_async_wait<0>();
  // Values that are not finite make their column NaN from their step on; the products, in which a later step's zero
  // score would make NaN of them for the steps before, take zeros in their place.
  const bool spoilt = __syncthreads_or(lv.copied_not_finite(sV));
  if (spoilt) {
    for (int col = tid; col < VS; col += kThreads) {
      int from = kChunk;
      for (int j = kChunk - 1; j >= 0; --j) {
        const uint32_t at = sV + j * Tile<VS>::kPitch + col * 2;
        if ((not_finite(ld_shared_u16(at)) & kNotFinite) == 0u) continue;
        from = j;
        st_shared_u16(at, 0);
      }
      s_from[col] = from;
    }
    __syncthreads();
  }

  uint32_t qf[kKt][4];
#pragma unroll
  for (int kt = 0; kt < kKt; ++kt) ldmatrix_x4(qf[kt], at_rows<KP>(sQ, 16 * warp, 16 * kt, lane));
  const int i0 = 16 * warp + g, i1 = i0 + 8;
  // The state's part, from its small part up.
  float O[VS / 8][4] = {};
#pragma unroll
  for (int part = 1; part >= 0; --part)
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
      for (int vt = 0; vt < VS / 16; ++vt) {
        const uint4 s = fS[part * Fr::kCount + Fr::at(kt, vt, lane)];
        mma_bf16_16816(O[2 * vt], qf[kt], s.x, s.y);
        mma_bf16_16816(O[2 * vt + 1], qf[kt], s.z, s.w);
      }
  const float e0 = d.first[i0], e1 = d.first[i1];
#pragma unroll
  for (int nt = 0; nt < VS / 8; ++nt) {
    O[nt][0] *= e0;
    O[nt][1] *= e0;
    O[nt][2] *= e1;
    O[nt][3] *= e1;
  }
  // Blocks of 16 steps: scores, their decays, in two parts times v.
  const float r0 = d.row[i0], r1 = d.row[i1], l0 = d.rel[i0], l1 = d.rel[i1], m0 = d.rel_lo[i0], m1 = d.rel_lo[i1];
#pragma unroll 1
  for (int jt = 0; jt <= warp; ++jt) {
    float s[2][4] = {};
#pragma unroll
    for (int kt = 0; kt < kKt; ++kt) {
      uint32_t kf[4];
      ldmatrix_x4(kf, at_cols<KP>(sK, 16 * jt, 16 * kt, lane));
      mma_bf16_16816(s[0], qf[kt], kf[0], kf[1]);
      mma_bf16_16816(s[1], qf[kt], kf[2], kf[3]);
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 16 * jt + 8 * h + 2 * q4;
      if (jt < warp) {
        const float2 cf = *reinterpret_cast<const float2*>(&d.col[warp - 1][j]);
        split2(s[h][0] * (r0 * cf.x), s[h][1] * (r0 * cf.y), hi[2 * h], lo[2 * h]);
        split2(s[h][2] * (r1 * cf.x), s[h][3] * (r1 * cf.y), hi[2 * h + 1], lo[2 * h + 1]);
      } else {
        const float2 D = *reinterpret_cast<const float2*>(&d.D[j]);
        const float2 lj = *reinterpret_cast<const float2*>(&d.rel[j]), mj = *reinterpret_cast<const float2*>(&d.rel_lo[j]);
        const float p0 = j <= i0 ? s[h][0] * (exp_fast((l0 - lj.x) + (m0 - mj.x)) * D.x) : 0.f;
        const float p1 = j + 1 <= i0 ? s[h][1] * (exp_fast((l0 - lj.y) + (m0 - mj.y)) * D.y) : 0.f;
        const float p2 = j <= i1 ? s[h][2] * (exp_fast((l1 - lj.x) + (m1 - mj.x)) * D.x) : 0.f;
        const float p3 = j + 1 <= i1 ? s[h][3] * (exp_fast((l1 - lj.y) + (m1 - mj.y)) * D.y) : 0.f;
        split2(p0, p1, hi[2 * h], lo[2 * h]);
        split2(p2, p3, hi[2 * h + 1], lo[2 * h + 1]);
      }
    }
#pragma unroll
    for (int vt = 0; vt < VS / 16; ++vt) {
      uint32_t vf[4];
      ldmatrix_x4_trans(vf, at_rows<VS>(sV, 16 * jt, 16 * vt, lane));
      mma_bf16_16816(O[2 * vt], lo, vf[0], vf[1]);
      mma_bf16_16816(O[2 * vt + 1], lo, vf[2], vf[3]);
      mma_bf16_16816(O[2 * vt], hi, vf[0], vf[1]);
      mma_bf16_16816(O[2 * vt + 1], hi, vf[2], vf[3]);
    }
  }
  // y = O + w_r v, rounded to bf16, by way of the warp's own rows of the q tile.
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 16 * warp + g + 8 * h;
#pragma unroll
    for (int nt = 0; nt < VS / 8; ++nt) {
      const int col = 8 * nt + 2 * q4;
      const uint32_t vv = ld_shared_b32(sV + i * Tile<VS>::kPitch + col * 2);
      const float2 wr = *reinterpret_cast<const float2*>(&s_wr[col]);
      float y0 = fmaf(wr.x, bf16lo(vv), O[nt][2 * h]), y1 = fmaf(wr.y, bf16hi(vv), O[nt][2 * h + 1]);
      if (spoilt) {
        if (i >= s_from[col]) y0 = __int_as_float(0x7FFFFFFF);
        if (i >= s_from[col + 1]) y1 = __int_as_float(0x7FFFFFFF);
      }
      st_shared_b32(sQ + i * Tile<KP>::kPitch + col * 2, pack_bf16x2(y0, y1));
    }
  }
  __syncwarp();
  constexpr int kPer = VS / 8;  // 16-byte pieces of a row
#pragma unroll
  for (int e = lane; e < 16 * kPer; e += 32) {
    const int i = 16 * warp + e / kPer, col = (e % kPer) * 8, t = t0 + i;
    if (t >= A.T || col >= width) continue;
    const uint4 r = t < len ? ld_shared_v4(sQ + i * Tile<KP>::kPitch + col * 2) : make_uint4(0u, 0u, 0u, 0u);
    uint16_t* yr = y + i * y_stride + col;
    if (V % 8 == 0) {
      *reinterpret_cast<uint4*>(yr) = r;
    } else {
      const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (col + u < width) yr[u] = static_cast<uint16_t>(x[u / 2] >> (16 * (u & 1)));
    }
  }
}

// The tcgen05 walk and outputs are built for 64 x 64 states, have one block per SM and want two tiles for each of
// them.  Measured, a whole call with them / with the walk and the outputs of this file, us: 64 tiles 14.4 / 13.9,
// 128 tiles 19.9 / 17.4, 256 20.8 / 19.8, 512 26.4 / 32.5, 1024 35.8 / 52.7, 2048 65 / 88.
constexpr int64_t kMinTiles = 2 * 152;

int padded_rows(int64_t K) { return K <= 32 ? 32 : K <= 64 ? 64 : 128; }
int slice_cols(int64_t K, int64_t V) { return V <= 16 ? 16 : V <= 32 || K <= 32 ? 32 : 64; }

struct Plan {
  int kp, vs, slices, segs, per_seg, nc;
  bool tile;  // walk and outputs on tcgen05 (ssm_tc_walk.cu, ssm_tc.cu)
};

// Segments: as many as the GPU holds walking blocks at once.
Plan make_plan(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  Plan p{};
  p.kp = padded_rows(K);
  p.vs = slice_cols(K, V);
  p.slices = static_cast<int>((V + p.vs - 1) / p.vs);
  p.nc = static_cast<int>((T + kChunk - 1) / kChunk);
  const int64_t chains = B * N * p.slices;
  p.tile = p.kp == kTcK && p.vs == kTcV && chains * ((p.nc + 1) / 2) >= kMinTiles;
  const int unit = p.tile ? 2 : 1;
  if (p.tile) p.nc = (p.nc + 1) / 2 * 2;
  const int64_t room = 152 * (p.tile ? 1 : p.kp * p.vs > 4096 ? 2 : 3);
  int64_t segs = room / chains;
  segs = segs < 1 ? 1 : segs > p.nc / unit ? p.nc / unit : segs;
  p.per_seg = static_cast<int>((p.nc / unit + segs - 1) / segs) * unit;
  p.segs = (p.nc + p.per_seg - 1) / p.per_seg;
  return p;
}

// Scratch, in bytes, each on a 16-byte boundary; the status block first.
struct Layout {
  size_t decay, tot, since, local, sums, seg_tot, start, total;
};

Layout make_layout(const Plan& p, int64_t chains) {
  Layout l{};
  l.total = sizeof(StatusBlock);
  auto take = [&](size_t bytes) {
    const size_t at = l.total;
    l.total += (bytes + 15) / 16 * 16;
    return at;
  };
  const size_t state = static_cast<size_t>(p.kp) * p.vs, chunks = static_cast<size_t>(chains) * p.nc,
               segs = static_cast<size_t>(chains) * p.segs;
  l.decay = take(chunks * sizeof(ChunkDecay));  // (the tiles' decays and states are smaller; rows that they
  // cannot take fall back on the larger)
  l.tot = take(chunks * 4);
  l.since = take(chunks * 4);
  l.local = take(chunks * p.slices * state * 4);
  if (p.segs > 1) {
    l.sums = take(segs * p.slices * state * 4);
    l.seg_tot = take(segs * 4);
    l.start = take(segs * p.slices * state * 4);
  }
  return l;
}

template <int KP, int VS, bool kTile>
cudaError_t join_segments(const ScanArgs& w, int64_t heads, cudaStream_t s) {
  if (w.segs == 1) return cudaSuccess;
  return launch_next(ssm_segment_scan_kernel<KP, VS, kTile>,
                     dim3(static_cast<unsigned>(heads), (2 * Frag<KP, VS>::kCount + 255) / 256), 256, 0, s, w);
}

template <int KP, int VS>
cudaError_t run(const ScanArgs& w, int64_t chains, cudaStream_t s) {
  using Walk = WalkShape<KP, VS>;
  using Out = OutShape<KP, VS>;
  const int64_t heads = chains * w.slices;
  static std::atomic<uint64_t> done_walk{0}, done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_walk_kernel<KP, VS>), Walk::kBytes, done_walk);
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(ssm_out_kernel<KP, VS>), Out::kBytes, done);
  if (e == cudaSuccess)
    e = launch_next(ssm_walk_kernel<KP, VS>, static_cast<unsigned>(heads * w.segs), kThreads, Walk::kBytes, s, w);
  if (e == cudaSuccess) e = join_segments<KP, VS, false>(w, heads, s);
  if (e != cudaSuccess) return e;
  return launch_next(ssm_out_kernel<KP, VS>, static_cast<unsigned>(heads * w.nc), kThreads, Out::kBytes, s, w);
}

}  // namespace

cudaError_t launch_ssm_decay(const SsmArgs& a, void* out, float* tot, int nc, bool grad, StatusBlock* status,
                             cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.B) * nc * ((a.N + 7) / 8));
  if (grad)
    ssm_decay_kernel<true><<<blocks, 256, 0, s>>>(a, out, tot, nc, status);
  else
    ssm_decay_kernel<false><<<blocks, 256, 0, s>>>(a, out, tot, nc, status);
  return cudaGetLastError();
}

size_t ssm_mma_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  return make_layout(make_plan(B, T, N, K, V), B * N).total;
}

cudaError_t launch_ssm_mma_forward(const SsmArgs& a, cudaStream_t s) {
  const Plan p = make_plan(a.B, a.T, a.N, a.K, a.V);
  const int64_t chains = static_cast<int64_t>(a.B) * a.N;
  const Layout l = make_layout(p, chains);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  StatusBlock* status = reinterpret_cast<StatusBlock*>(ws);
  auto vec = [](const void* p, int64_t stride, int width) {
    return width % 8 == 0 && stride % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  ScanArgs w{};
  w.a = a;
  w.tot = reinterpret_cast<float*>(ws + l.tot);
  w.since = reinterpret_cast<float*>(ws + l.since);
  w.local = reinterpret_cast<float4*>(ws + l.local);
  w.sums = reinterpret_cast<float4*>(ws + l.sums);
  w.seg_tot = reinterpret_cast<float*>(ws + l.seg_tot);
  w.start = reinterpret_cast<float4*>(ws + l.start);
  w.nc = p.nc;
  w.segs = p.segs;
  w.per_seg = p.per_seg;
  w.slices = p.slices;
  w.vq = vec(a.q, a.q_stride, a.K);
  w.vk = vec(a.k, a.k_stride, a.K);
  w.vv = vec(a.v, a.v_stride, a.V);
  float* tot = reinterpret_cast<float*>(ws + l.tot);
  // TMA takes strides below 2^40 bytes.
  const int64_t widest = a.q_stride > a.k_stride ? (a.q_stride > a.v_stride ? a.q_stride : a.v_stride)
                                                 : (a.k_stride > a.v_stride ? a.k_stride : a.v_stride);
  if (p.tile && w.vq && w.vk && w.vv && widest * a.T < (int64_t{1} << 39)) {
    TileDecay* decay = reinterpret_cast<TileDecay*>(ws + l.decay);
    cudaError_t e = launch_ssm_tile_decay(a, decay, tot, p.nc, status, s);
    if (e == cudaSuccess)
      e = launch_ssm_tc_walk(TcWalkArgs{a, decay, tot, w.local, w.sums, w.seg_tot, status, p.nc, p.nc / 2, p.segs,
                                        p.per_seg, p.slices}, s);
    if (e == cudaSuccess) e = join_segments<kTcK, kTcV, true>(w, chains * w.slices, s);
    if (e != cudaSuccess) return e;
    return launch_ssm_tc_out(TcOutArgs{a, decay, w.local, w.start, status, p.nc, p.nc / 2, p.segs,
                                       p.per_seg, p.slices}, s);
  }
  ChunkDecay* decay = reinterpret_cast<ChunkDecay*>(ws + l.decay);
  w.decay = decay;
  const cudaError_t e = launch_ssm_decay(a, decay, tot, p.nc, false, status, s);
  if (e != cudaSuccess) return e;
#define M2RNN_SSM_CASE(KP, VS) \
  if (p.kp == KP && p.vs == VS) return run<KP, VS>(w, chains, s);
  M2RNN_SSM_CASE(32, 16)
  M2RNN_SSM_CASE(32, 32)
  M2RNN_SSM_CASE(64, 16)
  M2RNN_SSM_CASE(64, 32)
  M2RNN_SSM_CASE(64, 64)
  M2RNN_SSM_CASE(128, 16)
  M2RNN_SSM_CASE(128, 32)
  M2RNN_SSM_CASE(128, 64)
#undef M2RNN_SSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace m2rnn
