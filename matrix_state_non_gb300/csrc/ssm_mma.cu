// Forward of the selective state space scan on tensor cores (bf16 inputs; the
// mathematics in ssm.cu).  A sequence is cut into segments, enough of them to
// fill the GPU; a block walks the chunks (64 steps) of one segment of one
// head, on up to 64 value columns, with the state in the accumulators of its
// warps:
//   1. every segment but the last: the state its own steps leave, from zero;
//   2. a scan over the segments gives the state before each;
//   3. every segment again from there, with the outputs.
// With one segment (enough heads) only 3 runs.  Per chunk a warp holds 16 of
// the 64 steps as rows of Q K^T, the outputs and Q S, and a quarter of the
// state's rows:
//   y = diag(first) Q S + (Q K^T (*) decays) V     S, decayed scores: one bf16
//   S = tot S + K^T diag(last D) V                 rounding each, as y has
// The state has to stay good to fp32: the rows of K^T diag(last D) are split
// into three bf16 parts (K, V themselves are exact), their products summed
// from the smallest part up, and the chunk's sum added to the state by an
// fp32 FMA, so that the tensor core's truncating adds never see the state.
#include <cuda_runtime.h>

#include <cstdint>

#include "ssm_mma.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 128;  // four warps

struct WalkArgs {
  SsmArgs a;
  const float* start;  // [B N][segs][K][V]: the state before each segment; null: H_0 (one segment)
  float* sums;         // phase 1: [B N][segs][K][V]
  float* tot;          // phase 1: [B N][segs]
  int segs, per_seg;   // segments, chunks in each
  int slices;          // of the value columns
  bool vq, vk, vv;     // rows that asynchronous copies can take
};

template <int KP, int VS, bool kOut>
struct WalkSmem {
  static constexpr int kQ = kOut ? Tile<KP>::kBytes(kChunk) : 0, kK = Tile<KP>::kBytes(kChunk),
                       kV = Tile<VS>::kBytes(kChunk), kStage = kQ + kK + kV;
  static constexpr int kS = kOut ? Tile<VS>::kBytes(KP) : 0;
  static constexpr int kDecay = (sizeof(ChunkDecay) + 15) / 16 * 16;
  static constexpr int kBytes = 2 * kStage + 2 * kS + 2 * kDecay;
};

// kOut false: phase 1.  KP: K padded to 32, 64 or 128; VS: columns of a slice.
template <int KP, int VS, bool kOut>
__global__ void __launch_bounds__(kThreads, KP * VS > 4096 ? 2 : 3) ssm_walk_kernel(WalkArgs W) {
  using Sm = WalkSmem<KP, VS, kOut>;
  constexpr int kKt = KP / 16;                                  // k-steps over the state's rows
  constexpr int kMw = KP >= 64 ? 4 : KP / 16, kNw = 4 / kMw;    // warps along the state's rows, columns
  constexpr int kMt = KP / 16 / kMw, kNt = VS / 8 / kNw;        // a warp's 16-row, 8-column tiles of the state
  static_assert(kNt >= 1, "slice too narrow for the warps");
  extern __shared__ __align__(16) uint8_t smem[];
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int mw = warp % kMw, nw = warp / kMw;
  int64_t id = blockIdx.x;
  const int seg = static_cast<int>(id % W.segs);
  id /= W.segs;
  const int slice = static_cast<int>(id % W.slices), bn = static_cast<int>(id / W.slices);
  const int b = bn / A.N, n = bn % A.N, gq = n / (A.N / A.G), K = A.K, V = A.V, v0 = slice * VS;
  if (!kOut && seg == W.segs - 1) return;
  const int len = ssm_len(A, b), width = min(VS, V - v0);
  const int c0 = seg * W.per_seg, c1 = min((A.T + kChunk - 1) / kChunk, c0 + W.per_seg);
  const int live = min(c1, (len + kChunk - 1) / kChunk);  // chunks with steps in them

  const uint32_t base = smem_u32(smem), sS = base + 2 * Sm::kStage;
  ChunkDecay* dec = reinterpret_cast<ChunkDecay*>(smem + 2 * Sm::kStage + 2 * Sm::kS);
  auto decay_of = [&](int c) -> ChunkDecay& {
    return *reinterpret_cast<ChunkDecay*>(reinterpret_cast<uint8_t*>(dec) + (c & 1) * Sm::kDecay);
  };
  const int64_t row = static_cast<int64_t>(b) * A.T;
  const uint16_t* pq = static_cast<const uint16_t*>(A.q) + row * A.q_stride + static_cast<int64_t>(gq) * K;
  const uint16_t* pk = static_cast<const uint16_t*>(A.k) + row * A.k_stride + static_cast<int64_t>(gq) * K;
  const uint16_t* pv = static_cast<const uint16_t*>(A.v) + row * A.v_stride + static_cast<int64_t>(n) * V + v0;
  const uint16_t* pt = static_cast<const uint16_t*>(A.dt) + row * A.dt_stride + n;
  const float An = A.A[n], bias = A.dt_bias ? A.dt_bias[n] : 0.f;
  auto load_chunk = [&](int c) {
    const uint32_t st = base + (c & 1) * Sm::kStage;
    if (kOut) load_tile<KP, kThreads>(st, pq, A.q_stride, K, c * kChunk, len, W.vq);
    load_tile<KP, kThreads>(st + Sm::kQ, pk, A.k_stride, K, c * kChunk, len, W.vk);
    load_tile<VS, kThreads>(st + Sm::kQ + Sm::kK, pv, A.v_stride, width, c * kChunk, len, W.vv);
    cp_async_commit();
  };
  // dt of a chunk, two steps a lane of warp 0 (whose row block has the fewest scores).
  float x0 = 0.f, x1 = 0.f;
  auto load_dt = [&](int c) {
    const int t = c * kChunk + 2 * lane;
    if (t < len) x0 = to_f32(pt[t * A.dt_stride]) + bias;
    if (t + 1 < len) x1 = to_f32(pt[(t + 1) * A.dt_stride]) + bias;
  };
  auto make_decay = [&](int c) {
    const int t = c * kChunk + 2 * lane;
    chunk_decay(decay_of(c), x0, x1, t < len, t + 1 < len, An, lane);
  };

  // The state: rows (mw kMt + mt) 16 + g (+ 8), columns (nw kNt + nt) 8 + 2 q4 (+ 1).
  float S[kMt][kNt][4];
  const float* from = kOut ? (W.start ? W.start + (static_cast<int64_t>(bn) * W.segs + seg) * K * V
                                      : (A.H_0 ? A.H_0 + static_cast<int64_t>(bn) * K * V : nullptr))
                           : nullptr;
  auto each_state = [&](auto f) {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = (mw * kMt + mt) * 16 + g + (e >> 1) * 8, c = (nw * kNt + nt) * 8 + 2 * q4 + (e & 1);
          f(S[mt][nt][e], r, c, r < K && c < width);
        }
  };
  each_state([&](float& s, int r, int c, bool ok) { s = from != nullptr && ok ? from[r * V + v0 + c] : 0.f; });
  auto store_operand = [&](int c) {  // the state before chunk c as bf16
    const uint32_t t = sS + (c & 1) * Sm::kS;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        const uint32_t at = t + ((mw * kMt + mt) * 16 + g) * Tile<VS>::kPitch + ((nw * kNt + nt) * 8 + 2 * q4) * 2;
        st_shared_b32(at, pack_bf16x2(S[mt][nt][0], S[mt][nt][1]));
        st_shared_b32(at + 8 * Tile<VS>::kPitch, pack_bf16x2(S[mt][nt][2], S[mt][nt][3]));
      }
  };

  float decay = 1.f;  // over the whole segment
  if (c0 < live) {
    load_chunk(c0);
    if (warp == 0) {
      load_dt(c0);
      make_decay(c0);
    }
    if (kOut) store_operand(c0);
  }
  for (int c = c0; c < live; ++c) {
    cp_async_wait<0>();
    __syncthreads();
    if (c + 1 < live) {
      load_chunk(c + 1);
      if (warp == 0) load_dt(c + 1);
    }
    const uint32_t sQ = base + (c & 1) * Sm::kStage, sK = sQ + Sm::kQ, sV = sK + Sm::kK;
    const ChunkDecay& d = decay_of(c);

    uint32_t P[4][4];    // decayed scores as A operands, per 16 steps j
    float O[VS / 8][4];  // outputs of the warp's rows
    if (kOut) {
      uint32_t qf[kKt][4];
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) ldmatrix_x4(qf[kt], at_rows<KP>(sQ, 16 * warp, 16 * kt, lane));
      const int i0 = 16 * warp + g, i1 = i0 + 8;
      const float r0 = d.row[i0], r1 = d.row[i1];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > warp) continue;
        float s[2][4] = {};
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
          uint32_t kf[4];
          ldmatrix_x4(kf, at_cols<KP>(sK, 16 * jt, 16 * kt, lane));
          mma_bf16_16816(s[0], qf[kt], kf[0], kf[1]);
          mma_bf16_16816(s[1], qf[kt], kf[2], kf[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = 16 * jt + 8 * h + 2 * q4;
          const float2 D = *reinterpret_cast<const float2*>(&d.D[j]);
          if (jt < warp) {
            const float2 cf = *reinterpret_cast<const float2*>(&d.col[warp][j]);
            const float f0 = cf.x * D.x, f1 = cf.y * D.y;
            P[jt][2 * h] = pack_bf16x2(s[h][0] * (r0 * f0), s[h][1] * (r0 * f1));
            P[jt][2 * h + 1] = pack_bf16x2(s[h][2] * (r1 * f0), s[h][3] * (r1 * f1));
          } else {
            const float2 hj = *reinterpret_cast<const float2*>(&d.hi[j]);
            const float2 lj = *reinterpret_cast<const float2*>(&d.lo[j]);
            const float h0 = d.hi[i0], l0 = d.lo[i0], h1 = d.hi[i1], l1 = d.lo[i1];
            const float p0 = j <= i0 ? s[h][0] * (exp_diff(h0 - hj.x, l0 - lj.x) * D.x) : 0.f;
            const float p1 = j + 1 <= i0 ? s[h][1] * (exp_diff(h0 - hj.y, l0 - lj.y) * D.y) : 0.f;
            const float p2 = j <= i1 ? s[h][2] * (exp_diff(h1 - hj.x, l1 - lj.x) * D.x) : 0.f;
            const float p3 = j + 1 <= i1 ? s[h][3] * (exp_diff(h1 - hj.y, l1 - lj.y) * D.y) : 0.f;
            P[jt][2 * h] = pack_bf16x2(p0, p1);
            P[jt][2 * h + 1] = pack_bf16x2(p2, p3);
          }
        }
      }
      // Q S
      const uint32_t st = sS + (c & 1) * Sm::kS;
#pragma unroll
      for (int nt = 0; nt < VS / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[nt][e] = 0.f;
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int np = 0; np < VS / 16; ++np) {
          uint32_t sf[4];
          ldmatrix_x4_trans(sf, at_rows<VS>(st, 16 * kt, 16 * np, lane));
          mma_bf16_16816(O[2 * np], qf[kt], sf[0], sf[1]);
          mma_bf16_16816(O[2 * np + 1], qf[kt], sf[2], sf[3]);
        }
      const float e0 = d.first[i0], e1 = d.first[i1];
#pragma unroll
      for (int nt = 0; nt < VS / 8; ++nt) {
        O[nt][0] *= e0;
        O[nt][1] *= e0;
        O[nt][2] *= e1;
        O[nt][3] *= e1;
      }
    }

    // The scores times V, and the chunk's own state.
    float U[kMt][kNt][4];
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[mt][nt][e] = 0.f;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      uint32_t vf[VS / 16][4];
#pragma unroll
      for (int np = 0; np < VS / 16; ++np) ldmatrix_x4_trans(vf[np], at_rows<VS>(sV, 16 * jt, 16 * np, lane));
      if (kOut && jt <= warp) {
#pragma unroll
        for (int np = 0; np < VS / 16; ++np) {
          mma_bf16_16816(O[2 * np], P[jt], vf[np][0], vf[np][1]);
          mma_bf16_16816(O[2 * np + 1], P[jt], vf[np][2], vf[np][3]);
        }
      }
      const int j = 16 * jt + 2 * q4;
      const float2 wa = *reinterpret_cast<const float2*>(&d.last[j]), wb = *reinterpret_cast<const float2*>(&d.last[j + 8]);
      const float2 Da = *reinterpret_cast<const float2*>(&d.D[j]), Db = *reinterpret_cast<const float2*>(&d.D[j + 8]);
      const float w0 = wa.x * Da.x, w1 = wa.y * Da.y, w2 = wb.x * Db.x, w3 = wb.y * Db.y;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        uint32_t kf[4], hi[4], mid[4], lo[4];
        ldmatrix_x4_trans(kf, at_cols<KP>(sK, 16 * jt, (mw * kMt + mt) * 16, lane));
#pragma unroll
        for (int r = 0; r < 4; ++r)
          split3(bf16lo(kf[r]) * (r < 2 ? w0 : w2), bf16hi(kf[r]) * (r < 2 ? w1 : w3), hi[r], mid[r], lo[r]);
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          constexpr int kHalf = kNw == 1 ? 0 : kNt;  // the second column half's first tile
          const int o = nt + kHalf;
          const uint32_t b0 = kNw == 1 || nw == 0 ? vf[nt / 2][2 * (nt & 1)] : vf[o / 2][2 * (o & 1)];
          const uint32_t b1 = kNw == 1 || nw == 0 ? vf[nt / 2][2 * (nt & 1) + 1] : vf[o / 2][2 * (o & 1) + 1];
          mma_bf16_16816(U[mt][nt], lo, b0, b1);
          mma_bf16_16816(U[mt][nt], mid, b0, b1);
          mma_bf16_16816(U[mt][nt], hi, b0, b1);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[mt][nt][e] = fmaf(d.tot, S[mt][nt][e], U[mt][nt][e]);
    if (!kOut) decay *= d.tot;

    if (c + 1 < live) {
      if (kOut) store_operand(c + 1);
      if (warp == 0) make_decay(c + 1);
    }
    if (kOut) {
      // y = O + w_r v, rounded to bf16
      uint16_t* y = static_cast<uint16_t*>(A.y);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 16 * warp + g + 8 * h, t = c * kChunk + i;
        if (t >= A.T) continue;
        uint16_t* yr = y + ((row + t) * A.N + n) * V + v0;
#pragma unroll
        for (int nt = 0; nt < VS / 8; ++nt) {
          const int col = 8 * nt + 2 * q4;
          float a0 = O[nt][2 * h], a1 = O[nt][2 * h + 1];
          if (A.w_r != nullptr) {
            const uint32_t vv = ld_shared_b32(sV + i * Tile<VS>::kPitch + col * 2);
            const uint16_t* wr = static_cast<const uint16_t*>(A.w_r) + n * V + v0;
            if (col < width) a0 = fmaf(to_f32(wr[col]), bf16lo(vv), a0);
            if (col + 1 < width) a1 = fmaf(to_f32(wr[col + 1]), bf16hi(vv), a1);
          }
          uint32_t r = pack_bf16x2(a0, a1);
          if (t >= len) r = 0u;
          if (W.vv) {  // width a multiple of 8
            if (col < width) *reinterpret_cast<uint32_t*>(yr + col) = r;
          } else {
            if (col < width) yr[col] = static_cast<uint16_t>(r);
            if (col + 1 < width) yr[col + 1] = static_cast<uint16_t>(r >> 16);
          }
        }
      }
    }
  }
  if (kOut) {
    // Chunks behind the sequence's end: zero outputs.
    uint16_t* y = static_cast<uint16_t*>(A.y);
    const int t0 = max(c0, live) * kChunk, t1 = min(A.T, c1 * kChunk);
    for (int e = tid; e < (t1 - t0) * width; e += kThreads)
      y[((row + t0 + e / width) * A.N + n) * V + v0 + e % width] = 0;
    if (A.H_T != nullptr && seg == W.segs - 1)
      each_state([&](float& s, int r, int c, bool ok) {
        if (ok) A.H_T[static_cast<int64_t>(bn) * K * V + r * V + v0 + c] = s;
      });
  } else {
    float* to = W.sums + (static_cast<int64_t>(bn) * W.segs + seg) * K * V;
    each_state([&](float& s, int r, int c, bool ok) {
      if (ok) to[r * V + v0 + c] = s;
    });
    if (tid == 0 && slice == 0) W.tot[static_cast<int64_t>(bn) * W.segs + seg] = decay;
  }
}

int padded_rows(int K) { return K <= 32 ? 32 : K <= 64 ? 64 : 128; }
int slice_cols(int V) { return V <= 16 ? 16 : V <= 32 ? 32 : 64; }

struct Plan {
  int slices, segs, per_seg;
};

// Segments: as many as the GPU holds blocks at once, where that is two or
// more per head; a single one costs no first phase.
Plan make_plan(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  Plan p{};
  const int vs = slice_cols(static_cast<int>(V));
  p.slices = static_cast<int>((V + vs - 1) / vs);
  const int64_t chains = B * N * p.slices, room = 152 * (padded_rows(static_cast<int>(K)) * vs > 4096 ? 2 : 3);
  const int64_t nc = (T + kChunk - 1) / kChunk;
  int64_t segs = room / chains;
  segs = segs < 1 ? 1 : segs > nc ? nc : segs;
  p.per_seg = static_cast<int>((nc + segs - 1) / segs);
  p.segs = static_cast<int>((nc + p.per_seg - 1) / p.per_seg);
  return p;
}

template <int KP, int VS>
cudaError_t run(const WalkArgs& w, int64_t chains, cudaStream_t s) {
  using Out = WalkSmem<KP, VS, true>;
  using Sum = WalkSmem<KP, VS, false>;
  cudaError_t e = cudaFuncSetAttribute(ssm_walk_kernel<KP, VS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Out::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(ssm_walk_kernel<KP, VS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sum::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(chains * w.slices * w.segs);
  if (w.segs > 1) {
    ssm_walk_kernel<KP, VS, false><<<grid, kThreads, Sum::kBytes, s>>>(w);
    e = launch_ssm_piece_scan(w.sums, w.tot, w.a.H_0, nullptr, w.segs, w.a.K * w.a.V, chains, false, s);
    if (e != cudaSuccess) return e;
  }
  ssm_walk_kernel<KP, VS, true><<<grid, kThreads, Out::kBytes, s>>>(w);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_mma_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V) {
  const Plan p = make_plan(B, T, N, K, V);
  if (p.segs == 1) return 16;
  return sizeof(float) * static_cast<size_t>(B) * N * p.segs * (static_cast<size_t>(K) * V + 1);
}

cudaError_t launch_ssm_mma_forward(const SsmArgs& a, cudaStream_t s) {
  const Plan p = make_plan(a.B, a.T, a.N, a.K, a.V);
  const int64_t chains = static_cast<int64_t>(a.B) * a.N;
  WalkArgs w{};
  w.a = a;
  w.segs = p.segs;
  w.per_seg = p.per_seg;
  w.slices = p.slices;
  if (p.segs > 1) {
    w.sums = static_cast<float*>(a.ws);
    w.tot = w.sums + chains * p.segs * a.K * a.V;
    w.start = w.sums;
  }
  auto vec = [](const void* p, int64_t stride, int width) {
    return width % 8 == 0 && stride % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  w.vq = vec(a.q, a.q_stride, a.K);
  w.vk = vec(a.k, a.k_stride, a.K);
  w.vv = vec(a.v, a.v_stride, a.V);
  const int kp = padded_rows(a.K), vs = slice_cols(a.V);
#define M2RNN_SSM_CASE(KP, VS) \
  if (kp == KP && vs == VS) return run<KP, VS>(w, chains, s);
  M2RNN_SSM_CASE(32, 16)
  M2RNN_SSM_CASE(32, 32)
  M2RNN_SSM_CASE(32, 64)
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
