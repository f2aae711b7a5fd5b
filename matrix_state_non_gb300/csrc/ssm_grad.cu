// Backward of the selective state space scan on tensor cores (bf16 inputs; the
// mathematics in ssm.cu), in chunks of 64 steps, every chunk on its own:
//   1. decays of every chunk;
//   2. the state S before each chunk and the state gradient R behind it: a
//      sequence is cut into segments, enough of them to fill the GPU, and a
//      block walks a segment's chunks with the state in its warps' accumulators,
//      adding sum_j last_j D_j k_j v_j^T (for R, from the last chunk to the
//      first, sum_i first_i q_i u_i^T);
//   3. a scan over the segments: what each of them is handed;
//   4. the chunk's gradients from q, k, v, u = dy, S and R, all chunks at once;
//   5. sums over the chunks (dA, ddt_bias, dw_r) and over the heads that share
//      q and k.
// The gradients are fp32 and good to that: q, k, v and u are exact bf16
// operands, and whatever else enters a product (S, R, the decayed scores, the
// weighted rows) is split into three bf16 parts, whose products are summed
// from the smallest part up.
//
// B=4 heads=8 T=4096 64x64: 172 us, of which decays 4, walk 32, segments 5,
// gradients 123, sums 5.  The gradients' kernel is bound by latency: 12 warps
// to an SM (168 registers, 67 KB a block), the tensor pipe 24 % and HBM 22 %
// busy, one instruction in three cycles issued; larger batches of loads or
// rolled loops change nothing.  The sums of W (ssm.cu) are 9 us of it.  Sums of
// single chunks and a scan over all of them in the walk's place, with the
// states' three parts in memory, cost 14 us more.
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
  // Of S and of R (walked from the sequence's end):
  float* local[2];  // [B N][chunks][K][V]: what the segment's own steps put into S before a chunk, R behind it
  float* since[2];  // [B N][chunks]: the decay between there and the segment's start (R: end)
  float* ends[2];   // [B N][segs][K][V]: what a segment hands on
  float* start[2];  // [B N][segs][K][V]: what it is handed
  float* seg_tot;   // [B N][segs]
  int nc, segs, per_seg;
  bool vq, vk, vv, vu;  // rows that asynchronous copies can take
};

template <int KP, int VS>
struct WalkShape {
  static constexpr int kMw = KP >= 64 ? 4 : KP / 16, kNw = 4 / kMw;
  static constexpr int kMt = KP / 16 / kMw, kNt = VS / 8 / kNw;
  static_assert(kNt % 2 == 0, "value tiles are loaded in pairs");
  static constexpr int kK = Tile<KP>::kBytes(kChunk), kV = Tile<VS>::kBytes(kChunk), kStage = kK + kV + kChunk * 4;
  static constexpr int kBytes = 2 * kStage;
  static constexpr int kBlocks = KP * VS > 4096 ? 2 : 3;  // per SM (registers)
};

// Phase 2: block (chain and segment, S or R and value slice); the state's rows along K.
template <int KP, int VS>
__global__ void __launch_bounds__(kThreads, WalkShape<KP, VS>::kBlocks) ssm_grad_walk_kernel(GradArgs W, int slices) {
  using Sh = WalkShape<KP, VS>;
  extern __shared__ __align__(16) uint8_t smem[];
  wait_previous();
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int mw = warp % Sh::kMw, nw = warp / Sh::kMw;
  const bool rev = blockIdx.y >= static_cast<unsigned>(slices);
  const int slice = blockIdx.y - (rev ? slices : 0), v0 = slice * VS;
  const int bn = blockIdx.x / W.segs, seg = blockIdx.x - bn * W.segs;
  const int b = bn / A.N, n = bn - b * A.N, gq = n / (A.N / A.G), K = A.K, V = A.V, len = ssm_len(A, b);
  const int width = min(VS, V - v0);
  const int c0 = seg * W.per_seg, live = min(min(W.nc, c0 + W.per_seg), (len + kChunk - 1) / kChunk);
  const int64_t row = static_cast<int64_t>(b) * A.T, KV = static_cast<int64_t>(K) * V;
  const uint32_t base = smem_u32(smem);
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
  const ChunkDecayGrad* pd = W.decay + static_cast<int64_t>(bn) * W.nc;
  const float* ptot = W.tot + static_cast<int64_t>(bn) * W.nc;
  auto load_chunk = [&](int c, int stage) {
    const uint32_t st = base + stage * Sh::kStage;
    lk.load(st, c * kChunk, len);
    lv.load(st + Sh::kK, c * kChunk, len);
    if (tid < kChunk / 4) cp_async_16(st + Sh::kK + Sh::kV + tid * 16, (rev ? pd[c].d.first : pd[c].d.wD) + tid * 4, true);
    cp_async_commit();
  };
  float S[Sh::kMt][Sh::kNt][4];
  // Pairs of columns of the accumulators: f(row, column, x, y).
  auto each = [&](auto f) {
#pragma unroll
    for (int mt = 0; mt < Sh::kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < Sh::kNt; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (mw * Sh::kMt + mt) * 16 + g + 8 * h, col = (nw * Sh::kNt + nt) * 8 + 2 * q4;
          f(r, col, S[mt][nt][2 * h], S[mt][nt][2 * h + 1]);
        }
  };
  auto store = [&](float* state) {
    each([&](int r, int col, float& x, float& y) {
      if (r >= K || col >= width) return;
      float* at = state + r * V + v0 + col;
      if (V % 2 == 0) {
        *reinterpret_cast<float2*>(at) = make_float2(x, y);
      } else {
        at[0] = x;
        if (col + 1 < width) at[1] = y;
      }
    });
  };
  const float* given = seg == (rev ? W.segs - 1 : 0) ? (rev ? A.dH_T : A.H_0) : nullptr;
  each([&](int r, int col, float& x, float& y) {
    const float* at = given + bn * KV + r * V + v0 + col;
    x = given != nullptr && r < K && col < width ? at[0] : 0.f;
    y = given != nullptr && r < K && col + 1 < width ? at[1] : 0.f;
  });

  const int step = rev ? -1 : 1, count = live - c0;
  int c = rev ? live - 1 : c0;
  float tot = 0.f, decay = 1.f;  // of a chunk; of the chunks so far
  if (count > 0) {
    load_chunk(c, 0);
    tot = ptot[c];
  }
  for (int i = 0; i < count; ++i, c += step) {
    cp_async_wait<0>();
    __syncthreads();
    const float tot_c = tot;
    if (i + 1 < count) {
      load_chunk(c + step, (i + 1) & 1);
      tot = ptot[c + step];
    }
    const int64_t id = static_cast<int64_t>(bn) * W.nc + c;
    if (slice == 0 && tid == 0) W.since[rev][id] = decay;
    decay *= tot_c;
    store(W.local[rev] + id * KV);
    const int stage = (i & 1) * Sh::kStage;
    const uint32_t sK = base + stage, sV = sK + Sh::kK;
    const float* w = reinterpret_cast<const float*>(smem + stage + Sh::kK + Sh::kV);
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
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int nt = 0; nt < Sh::kNt; ++nt)
            mma_bf16_16816(part < 2 ? low[mt][nt] : U[mt][nt], p[part], vf[nt / 2][2 * (nt & 1)],
                           vf[nt / 2][2 * (nt & 1) + 1]);
      }
    }
#pragma unroll
    for (int mt = 0; mt < Sh::kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < Sh::kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[mt][nt][e] = fmaf(tot_c, S[mt][nt][e], U[mt][nt][e] + low[mt][nt][e]);
  }
  let_next();
  if (W.segs > 1) {
    store(W.ends[rev] + (static_cast<int64_t>(bn) * W.segs + seg) * KV);
    if (!rev && slice == 0 && tid == 0) W.seg_tot[static_cast<int64_t>(bn) * W.segs + seg] = decay;
  } else if (rev && A.dH_0 != nullptr) {
    store(A.dH_0 + bn * KV);
  }
}

// Phase 3: block (chain, 256 elements of a state, S or R).
__global__ void __launch_bounds__(256) ssm_grad_segments_kernel(GradArgs W) {
  constexpr int kAhead = 8;
  let_next();
  wait_previous();
  const SsmArgs& A = W.a;
  const int64_t KV = static_cast<int64_t>(A.K) * A.V, bn = blockIdx.x;
  const int e = blockIdx.y * 256 + threadIdx.x;
  const bool rev = blockIdx.z == 1;
  if (e >= KV) return;
  const float* ends = W.ends[rev] + bn * W.segs * KV + e;
  float* start = W.start[rev] + bn * W.segs * KV + e;
  const float* tot = W.seg_tot + bn * W.segs;
  float s = 0.f;
  for (int i0 = 0; i0 < W.segs; i0 += kAhead) {
    float u[kAhead], a[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= W.segs) continue;
      const int c = rev ? W.segs - 1 - i0 - j : i0 + j;
      u[j] = ends[c * KV];
      a[j] = tot[c];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= W.segs) continue;
      start[(rev ? W.segs - 1 - i0 - j : i0 + j) * KV] = s;
      s = fmaf(a[j], s, u[j]);
    }
  }
  if (rev && A.dH_0 != nullptr) A.dH_0[bn * KV + e] = s;
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
// smallest part up, and added in fp32.  The tensor core truncates its adds,
// which on the running sum itself is a bias (dq 1.9e-7 of the float64 value
// instead of 1.3e-7); the eight chains of three also hide each other's
// latency better than one of twelve, so it costs no time.
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
  __shared__ float sd[kChunk], ck[kChunk], ci[kChunk], red[4];
  __shared__ Sum2 w_row[kChunk], w_col[4][kChunk];  // sums of W; w_col of each warp's rows
  let_next();
  wait_previous();
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
  cp_async_commit();
  // S and R, four columns of a row at a time: the segment's own and, behind the segment that S (R) comes into first,
  // what the segment was handed.
  constexpr int kPieces = KP * VP / 4 / kThreads, kBatch = kPieces < 4 ? kPieces : 4;
  const int seg = c / W.per_seg;
  struct State {
    const float *own, *start;
    float since;
  };
  const int64_t at_seg = (static_cast<int64_t>(bn) * W.segs + seg) * KV;
  const State gS{W.local[0] + blockIdx.x * KV, seg > 0 ? W.start[0] + at_seg : nullptr, W.since[0][blockIdx.x]};
  const State gR{W.local[1] + blockIdx.x * KV, seg < W.segs - 1 ? W.start[1] + at_seg : nullptr, W.since[1][blockIdx.x]};
  auto piece_row = [&](int i) { return (i * kThreads + tid) / (VP / 4); };
  auto piece_col = [&](int i) { return (i * kThreads + tid) % (VP / 4) * 4; };
  auto fetch = [&](const float* p, int i) {
    const int r = piece_row(i), col = piece_col(i);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p == nullptr || r >= K || col >= V) return x;
    const float* at = p + r * V + col;
    if (V % 4 == 0) return *reinterpret_cast<const float4*>(at);
    x.x = at[0];
    if (col + 1 < V) x.y = at[1];
    if (col + 2 < V) x.z = at[2];
    if (col + 3 < V) x.w = at[3];
    return x;
  };
  auto joined = [](const float4& own, const float4& start, float since) {
    return make_float4(fmaf(since, start.x, own.x), fmaf(since, start.y, own.y), fmaf(since, start.z, own.z),
                       fmaf(since, start.w, own.w));
  };
  auto put = [&](const float4& x, int i) {  // as three bf16 parts
    uint32_t p[3][2];
    split3(x.x, x.y, p[0][0], p[1][0], p[2][0]);
    split3(x.z, x.w, p[0][1], p[1][1], p[2][1]);
    const uint32_t at = sP + piece_row(i) * Tile<VP>::kPitch + piece_col(i) * 2;
#pragma unroll
    for (int part = 0; part < 3; ++part)
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + part * Sh::kP), "r"(p[part][0]), "r"(p[part][1])
                   : "memory");
  };
#pragma unroll 1
  for (int i0 = 0; i0 < kPieces; i0 += kBatch) {
    float4 own[kBatch], start[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) own[i] = fetch(gS.own, i0 + i);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) start[i] = fetch(gS.start, i0 + i);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) put(joined(own[i], start[i], gS.since), i0 + i);
  }
  cp_async_wait<0>();
  __syncthreads();

  const int m0 = 16 * warp + g, m1 = m0 + 8;  // the warp's rows of every product
  // exp(l_i - l_j) for rows i of block bi > bj and columns j, or within a block (i >= j, else 0).
  auto diag = [&](int i, int j) {
    return i >= j ? exp_fast((d.rel[i] - d.rel[j]) + (d.rel_lo[i] - d.rel_lo[j])) : 0.f;
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

  // Sums of a 16 x 16 block of W along its columns, over the eight lanes that share them: at each of the first two
  // steps a lane keeps half of its columns and passes the others on.
  auto add_columns = [&](const float (&w)[2][4], int jt) {
    Sum2 c[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c[h][e].add(w[h][e]);
        c[h][e].add(w[h][2 + e]);
      }
    const bool up = g & 4, odd = g & 2;
    Sum2 half[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      half[e] = up ? c[1][e] : c[0][e];
      half[e].add((up ? c[0][e] : c[1][e]).across(16));
    }
    Sum2 one = odd ? half[1] : half[0];
    one.add((odd ? half[0] : half[1]).across(8));
    one.add(one.across(4));
    if ((g & 1) == 0) w_col[warp][16 * jt + 8 * up + 2 * q4 + odd] = one;
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
    row_dots(sQ, x, sd);
    Sum2 row0, row1;
    // Not unrolled, here and below: four copies of the body do not fit the instruction cache.
#pragma unroll 1
    for (int jt = 0; jt <= warp; ++jt) {
      float s[2][4] = {}, w[2][4] = {};
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
        uint32_t qf[4], f[4];
        ldmatrix_x4(qf, at_rows<KP>(sQ, 16 * warp, 16 * kt, lane));
        ldmatrix_x4(f, at_cols<KP>(sK, 16 * jt, 16 * kt, lane));
        mma_bf16_16816(w[0], qf, f[0], f[1]);
        mma_bf16_16816(w[1], qf, f[2], f[3]);
      }
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
          w[h][e] = jt < warp || j < m0 ? s[h][e] * w[h][e] : 0.f;
          w[h][2 + e] = jt < warp || j < m1 ? s[h][2 + e] * w[h][2 + e] : 0.f;
          row0.add(w[h][e]);
          row1.add(w[h][2 + e]);
        }
      add_columns(w, jt);
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
    row0.add(row0.across(1));
    row1.add(row1.across(1));
    row0.add(row0.across(2));
    row1.add(row1.across(2));
    if (q4 == 0) {
      w_row[m0] = row0;
      w_row[m1] = row1;
    }
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

  // R's first pieces, behind the first half of dk.
  constexpr int kHold = kPieces < 8 ? kPieces : 8, kDot = kHold < 4 ? kHold : 4;
  float4 held[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) held[i] = fetch(gR.own, i);

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

  float rs = 0.f;  // <R, S>
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
    __syncthreads();  // S has been read
    auto place = [&](const float4& own, const float4& start, const float4& s_own, const float4& s_start, int i) {
      const float4 r = joined(own, start, gR.since), s = joined(s_own, s_start, gS.since);
      rs = fmaf(r.x, s.x, fmaf(r.y, s.y, fmaf(r.z, s.z, fmaf(r.w, s.w, rs))));
      put(r, i);
    };
#pragma unroll
    for (int i0 = 0; i0 < kHold; i0 += kDot) {
      float4 start[kDot], s_own[kDot], s_start[kDot];
#pragma unroll
      for (int i = 0; i < kDot; ++i) {
        start[i] = fetch(gR.start, i0 + i);
        s_own[i] = fetch(gS.own, i0 + i);
        s_start[i] = fetch(gS.start, i0 + i);
      }
#pragma unroll
      for (int i = 0; i < kDot; ++i) place(held[i0 + i], start[i], s_own[i], s_start[i], i0 + i);
    }
#pragma unroll 2
    for (int i = kHold; i < kPieces; ++i)
      place(fetch(gR.own, i), fetch(gR.start, i), fetch(gS.own, i), fetch(gS.start, i), i);
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
  if (lane == 0) red[warp] = rs;
  __syncthreads();

  if (warp == 0) {  // two steps a lane
    const int i = 2 * lane;
    const float A_n = A.A[n];
    const float from0 = d.wD[i] * ci[i], from1 = d.wD[i + 1] * ci[i + 1];
    Sum2 end;  // <R, S'>
    end.add(from0);
    end.add(from1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) end.add(end.across(o));
    end.add(W.tot[blockIdx.x] * ((red[0] + red[1]) + (red[2] + red[3])));
    auto term = [&](int at, float from) {
      Sum2 y;
      y.add(sd[at]);
      y.add(w_row[at]);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x >= at / 16) y.subtract(w_col[x][at]);
      y.add(-from);
      return y;
    };
    const Sum2 y1 = term(i + 1, from1);
    Sum2 x = term(i, from0);
    x.add(y1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) x.add(x.after(o));
    Sum2 x1 = x.after(1);
    x1.add(y1);
    x.add(end);
    x1.add(end);
    const float g0 = x.value(), g1 = x1.value();
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

int slice_cols(int vp) { return vp < 64 ? vp : 64; }

struct Plan {
  int kp, vp, slices, nc, segs, per_seg;
};

// Segments: as many as the GPU holds walking blocks at once, half of them for S.
Plan make_plan(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  Plan p{};
  p.kp = padded(K);
  p.vp = p.kp > 32 && V <= 16 ? 16 : padded(V);
  const int vs = slice_cols(p.vp);
  p.slices = static_cast<int>((V + vs - 1) / vs);
  p.nc = static_cast<int>((T + kChunk - 1) / kChunk);
  const int64_t room = 152 * (p.kp * vs > 4096 ? 2 : 3) / (2 * B * N * p.slices);
  const int64_t segs = room < 1 ? 1 : room > p.nc ? p.nc : room;
  p.per_seg = static_cast<int>((p.nc + segs - 1) / segs);
  p.segs = (p.nc + p.per_seg - 1) / p.per_seg;
  return p;
}

struct Layout {
  size_t decay, tot, local[2], since[2], ends[2], start[2], seg_tot, ab, wr, dq, dk, total;
};

Layout make_layout(const Plan& p, int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V) {
  Layout l{};
  l.total = sizeof(StatusBlock);
  auto take = [&](size_t bytes) {
    const size_t at = l.total;
    l.total += (bytes + 15) / 16 * 16;
    return at;
  };
  const size_t chains = static_cast<size_t>(B) * N, chunks = chains * p.nc, KV = static_cast<size_t>(K) * V;
  l.decay = take(chunks * sizeof(ChunkDecayGrad));
  l.tot = take(chunks * 4);
  for (int i = 0; i < 2; ++i) {
    l.local[i] = take(chunks * KV * 4);
    l.since[i] = take(chunks * 4);
    if (p.segs == 1) continue;
    l.ends[i] = take(chains * p.segs * KV * 4);
    l.start[i] = take(chains * p.segs * KV * 4);
  }
  if (p.segs > 1) l.seg_tot = take(chains * p.segs * 4);
  l.ab = take(chunks * 8);
  l.wr = take(chunks * V * 4);
  if (G != N) {
    l.dq = take(static_cast<size_t>(B) * T * N * K * 4);
    l.dk = take(static_cast<size_t>(B) * T * N * K * 4);
  }
  return l;
}

template <int KP, int VP>
cudaError_t run(const GradArgs& w, int slices, cudaStream_t s) {
  constexpr int VS = VP < 64 ? VP : 64;
  using Walk = WalkShape<KP, VS>;
  using Gr = GradShape<KP, VP>;
  static std::atomic<uint64_t> done{0}, done_walk{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_grad_kernel<KP, VP>), Gr::kBytes, done);
  if (e == cudaSuccess)
    e = allow_smem(reinterpret_cast<const void*>(ssm_grad_walk_kernel<KP, VS>), Walk::kBytes, done_walk);
  if (e != cudaSuccess) return e;
  const SsmArgs& a = w.a;
  const unsigned chains = static_cast<unsigned>(a.B) * a.N, blocks = chains * w.nc;
  e = launch_next(ssm_grad_walk_kernel<KP, VS>, dim3(chains * w.segs, 2 * slices), kThreads, Walk::kBytes, s, w, slices);
  if (e == cudaSuccess && w.segs > 1)
    e = launch_next(ssm_grad_segments_kernel, dim3(chains, (a.K * a.V + 255) / 256, 2), 256, 0, s, w);
  if (e != cudaSuccess) return e;
  return launch_next(ssm_grad_kernel<KP, VP>, blocks, kThreads, Gr::kBytes, s, w);
}

}  // namespace

size_t ssm_mma_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V) {
  return make_layout(make_plan(B, T, N, K, V), B, T, N, G, K, V).total;
}

cudaError_t launch_ssm_mma_backward(const SsmArgs& a, cudaStream_t s) {
  const Plan p = make_plan(a.B, a.T, a.N, a.K, a.V);
  const Layout l = make_layout(p, a.B, a.T, a.N, a.G, a.K, a.V);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  GradArgs w{};
  w.a = a;
  w.nc = p.nc;
  w.segs = p.segs;
  w.per_seg = p.per_seg;
  w.decay = reinterpret_cast<const ChunkDecayGrad*>(ws + l.decay);
  w.tot = reinterpret_cast<const float*>(ws + l.tot);
  for (int i = 0; i < 2; ++i) {
    w.local[i] = reinterpret_cast<float*>(ws + l.local[i]);
    w.since[i] = reinterpret_cast<float*>(ws + l.since[i]);
    w.ends[i] = reinterpret_cast<float*>(ws + l.ends[i]);
    w.start[i] = reinterpret_cast<float*>(ws + l.start[i]);
  }
  w.seg_tot = reinterpret_cast<float*>(ws + l.seg_tot);
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
  e = cudaErrorInvalidValue;
#define M2RNN_SSM_CASE(KP, VP) \
  if (p.kp == KP && p.vp == VP) e = run<KP, VP>(w, p.slices, s);
  M2RNN_SSM_CASE(32, 32)
  M2RNN_SSM_CASE(32, 64)
  M2RNN_SSM_CASE(32, 128)
  M2RNN_SSM_CASE(64, 16)
  M2RNN_SSM_CASE(64, 32)
  M2RNN_SSM_CASE(64, 64)
  M2RNN_SSM_CASE(64, 128)
  M2RNN_SSM_CASE(128, 16)
  M2RNN_SSM_CASE(128, 32)
  M2RNN_SSM_CASE(128, 64)
  M2RNN_SSM_CASE(128, 128)
#undef M2RNN_SSM_CASE
  if (e != cudaSuccess) return e;
  return launch_ssm_grad_sums(a, w.o, w.nc, s);
}

}  // namespace m2rnn
