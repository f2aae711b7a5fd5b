// The walk over a segment's states (phase 2 of ssm_mma.cu) on the 5th-generation
// tensor cores, in tiles of 128 steps, for up to 64 state rows and value columns:
//     S' = tot S + sum_j (w_j k_j) v_j^T,  w_j = exp(l_end - l_j) D_j,
// held transposed: D = v^T (w k) has value columns as rows and state rows as
// columns, so a thread of the accumulator's 64 lanes has a value column's whole
// row and leaves it in fp32, 16 bytes at a time, side by side with its neighbours.
// v is exact in bf16; w k is split into three bf16 parts, side by side one
// operand of 192 columns with an accumulator each, so that eight truncating
// adds see a sum's full size.  The state itself is fp32 in registers.
// B=2 heads=16 T=16384 64x64, shared q and k: 38 us (46 on mma.sync).  A tile takes 1900 cycles, in which the products (64 KB of
// operands) and the split (48 KB written) share the bandwidth of shared memory:
// k through shared memory as well, 24 products of 64 columns in the place of 8,
// or two groups of split warps on tiles in turn are 4 to 7 us slower each.
// One persistent block per SM takes (head, value slice, segment) after another:
//   warps 13-15  producers: v by TMA (128-byte swizzle) into a ring of three
//                stages; a sequence's last tile row by row, with zeros behind
//                its end;
//   warps 4-11   split: k and the weights come straight to registers, a tile
//                ahead, their three parts go to the stage, swizzled like v;
//   warp 12      issues the eight products (M = 64, N = 192) of a tile into one
//                of two tensor-memory slots;
//   warps 0-3    the state: leave it before the tile, add the tile's sum.
#include <cuda_runtime.h>

#include <cstdint>

#include "ssm_tc.cuh"

namespace m2rnn {
namespace {

constexpr int kState = 128, kSplit = 256, kMmaWarp = 12, kProd = 96, kThreads = kState + kSplit + 32 + kProd;
constexpr int kStages = 3;
constexpr int kOffK = kOp, kStage = 4 * kOp;  // v, the three parts of w k
constexpr int kOffBar = kStages * kStage;
constexpr int kSmem = kOffBar + 256 + 1024;  // 1024: alignment
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kSlot = 3 * kTcK;  // tensor-memory columns: an accumulator for each part

// Item `id`: a (chain, slice) head's segment and its tiles with steps in them.
struct WalkPlace {
  int b, n, gq, slice, v0, width, len, seg, t0, t1;
  int64_t chain, head;
};

__device__ __forceinline__ WalkPlace walk_place(const TcWalkArgs& W, unsigned id) {
  const SsmArgs& A = W.a;
  WalkPlace p;
  const unsigned head = id / W.segs, bn = head / W.slices;
  p.seg = id - head * W.segs;
  p.slice = head - bn * W.slices;
  p.head = head;
  p.chain = bn;
  p.b = bn / A.N;
  p.n = bn - p.b * A.N;
  p.gq = p.n / (A.N / A.G);
  p.v0 = p.slice * kTcV;
  p.width = min(kTcV, A.V - p.v0);
  p.len = ssm_len(A, p.b);
  p.t0 = p.seg * (W.per_seg / 2);
  p.t1 = min(min(W.nt, p.t0 + W.per_seg / 2), (p.len + kTile - 1) / kTile);
  return p;
}

__global__ void __launch_bounds__(kThreads, 1)
    ssm_tc_walk_kernel(const __grid_constant__ CUtensorMap map_v, TcWalkArgs W, unsigned items) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem), bars = base + kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };        // [3] producers -> products
  auto split = [&](int s) { return bars + 24 + 8 * s; };  // [3] split -> products
  auto empty = [&](int s) { return bars + 48 + 8 * s; };  // [3] products -> producers, split
  auto done = [&](int s) { return bars + 72 + 8 * s; };   // [2] products -> state
  auto tfree = [&](int s) { return bars + 88 + 8 * s; };  // [2] state -> products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 128);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 132);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), kProd);
      mbar_init(split(s), kSplit);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(done(s), 1);
      mbar_init(tfree(s), kState);
    }
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_previous();

  if (warp > kMmaWarp) {
    // ---------------- producers ----------------
    const int p = tid - kState - kSplit - 32;
    if (p == 0) tma_prefetch_desc(&map_v);
    int u = 0;  // tiles of this block
    bool ok = true;
    for (unsigned id = blockIdx.x; ok && id < items; id += gridDim.x) {
      const WalkPlace at = walk_place(W, id);
      for (int tt = at.t0; tt < at.t1; ++tt, ++u) {
        const int s = u % kStages, t0 = tt * kTile;
        if (u >= kStages && !warp_wait(empty(s), (u / kStages - 1) & 1, abort_flag, W.status, kWhereWalkEmpty)) {
          ok = false;
          break;
        }
        const uint32_t st = base + s * kStage, bar = full(s);
        if (t0 + kTile <= at.len) {
          if (p == 0) {
            mbar_expect_tx(bar, kOp);
            tma_load_4d(st, &map_v, bar, at.v0, at.n, t0, at.b);
          }
        } else {
          const int piece = p & 7;
          const uint16_t* src = static_cast<const uint16_t*>(A.v) + (static_cast<int64_t>(at.b) * A.T + t0) * A.v_stride +
                                static_cast<int64_t>(at.n) * A.V + at.v0;
          for (int r = p >> 3; r < kTile; r += kProd / 8) {
            const bool in = piece * 8 < at.width && t0 + r < at.len;
            cp_async_16(st + piece_at(r, piece), in ? src + r * A.v_stride + piece * 8 : src, in);
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
        }
        mbar_arrive(bar);
      }
    }
    if (!ok)  // the copies in flight land before the block ends
      for (int x = max(0, u - kStages); x < u; ++x)
        mbar_wait_timed(full(x % kStages), (x / kStages) & 1, nullptr, kWhereWalkDrain);
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    constexpr uint32_t kId = idesc_bf16_f32(64, 3 * kTcK, true, true);
    int u = 0;
    bool ok = true;
    for (unsigned id = blockIdx.x; ok && id < items; id += gridDim.x) {
      const WalkPlace at = walk_place(W, id);
      for (int tt = at.t0; tt < at.t1; ++tt, ++u) {
        const int s = u % kStages, slot = u & 1;
        ok = warp_wait(full(s), (u / kStages) & 1, abort_flag, W.status, kWhereWalkFull) &&
             (u < 2 || warp_wait(tfree(slot), ((u >> 1) - 1) & 1, abort_flag, W.status, kWhereWalkFree)) &&
             warp_wait(split(s), (u / kStages) & 1, abort_flag, W.status, kWhereWalkSplit);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after_sync();
          const uint32_t tm = tmem + slot * kSlot, st = base + s * kStage;
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_f16_ss(tm, desc_sw128(st + kk * 2048), desc_sw128(st + kOffK + kk * 2048, kOp), kId, kk > 0);
          tc_commit(done(slot));
          tc_commit(empty(s));
        }
        __syncwarp();
      }
    }
    if (!ok)  // the products in flight end before their memory is freed
      for (int x = max(0, u - 2); x < u; ++x) mbar_wait_timed(done(x & 1), (x >> 1) & 1, nullptr, kWhereWalkDrain);
  } else if (warp >= kState / 32) {
    // ---------------- split ----------------
    const int q = tid - kState, piece = q & 7;
    constexpr int kRows = kTile * 8 / kSplit;  // rows (q >> 3) + 32 i
    uint4 k[kRows];
    float w[kRows], behind;  // (the second chunk's decay, for the first's steps)
    unsigned id = blockIdx.x;
    int left = 0, t0 = 0, len = 0;  // tiles of the item; steps
    const uint16_t* pk = nullptr;
    const float *pw = nullptr, *pt = nullptr;
    const bool col = piece * 8 < A.K;
    auto open = [&] {
      const WalkPlace at = walk_place(W, id);
      left = at.t1 - at.t0;
      t0 = at.t0 * kTile + (q >> 3);
      len = at.len;
      pk = static_cast<const uint16_t*>(A.k) + (static_cast<int64_t>(at.b) * A.T + t0) * A.k_stride +
           static_cast<int64_t>(at.gq) * A.K + piece * 8;
      pw = W.decay[at.chain * W.nc + 2 * at.t0].wD + (q >> 3);
      pt = W.tot + at.chain * W.nc + 2 * at.t0 + 1;
    };
    auto find = [&] {  // the next tile, if there is one
      while (id < items && left <= 0) {
        id += gridDim.x;
        if (id < items) open();
      }
      return id < items;
    };
    const int64_t row = (kSplit / 8) * A.k_stride;
    auto load = [&] {
      const uint16_t* p = pk;
#pragma unroll
      for (int i = 0; i < kRows; ++i, p += row) {
        k[i] = make_uint4(0u, 0u, 0u, 0u);
        if (col && t0 + i * (kSplit / 8) < len) k[i] = __ldg(reinterpret_cast<const uint4*>(p));
        w[i] = pw[i * (kSplit / 8) + (i < kRows / 2 ? 0 : static_cast<int>(sizeof(TileDecay) / 4) - kChunk)];
      }
      behind = *pt;
      pk = p;
      pw += 2 * sizeof(TileDecay) / 4;
      pt += 2;
      t0 += kTile;
      --left;
    };
    if (id < items) open();
    bool there = find();
    if (there) load();
    for (int u = 0; there; ++u) {
      const int s = u % kStages;
      uint4 now[kRows];
      float x[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        now[i] = k[i];
        x[i] = i < kRows / 2 ? w[i] * behind : w[i];
      }
      there = find();
      if (there) load();
      if (u >= kStages && !warp_wait(empty(s), (u / kStages - 1) & 1, abort_flag, W.status, kWhereWalkEmpty)) break;
      const uint32_t sk = base + s * kStage + kOffK;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint32_t to = sk + piece_at(i * (kSplit / 8) + (q >> 3), piece);
        const uint32_t in[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
        uint32_t p[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split3_weighted(in[e], x[i], x[i], p[0][e], p[1][e], p[2][e]);
#pragma unroll
        for (int part = 0; part < 3; ++part)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + part * kOp), "r"(p[part][0]),
                       "r"(p[part][1]), "r"(p[part][2]), "r"(p[part][3])
                       : "memory");
      }
      fence_proxy_async_smem();
      mbar_arrive(split(s));
    }
  } else {
    // ---------------- the state: lanes 0-15 of warp w, value columns 16 w .. ----------------
    const int v = 16 * warp + (lane & 15);
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const bool own = lane < 16;
    int u = 0;
    bool ok = true;
    for (unsigned id = blockIdx.x; ok && id < items; id += gridDim.x) {
      const WalkPlace at = walk_place(W, id);
      const bool in = own && v < at.width;
      const int64_t state = at.chain * A.K * A.V + at.v0 + v;
      float S[kTcK];
#pragma unroll
      for (int k = 0; k < kTcK; ++k)
        S[k] = at.seg == 0 && A.H_0 != nullptr && in && k < A.K ? A.H_0[state + static_cast<int64_t>(k) * A.V] : 0.f;
      float decay = 1.f;  // since the segment's start
      float4* to = W.local + (at.head * W.nt + at.t0) * kTcState + tc_piece_at(0, v);
      for (int tt = at.t0; tt < at.t1; ++tt, ++u, to += kTcState) {
        const int slot = u & 1;
        const float* tot = W.tot + at.chain * W.nc + 2 * tt;
        const float t = tot[0] * tot[1];
        if (at.slice == 0 && tid == 0) W.decay[at.chain * W.nc + 2 * tt].T[2] = decay;
        decay *= t;
        if (own) {
#pragma unroll
          for (int k = 0; k < kTcK; k += 4) to[tc_piece_at(k, 0)] = make_float4(S[k], S[k + 1], S[k + 2], S[k + 3]);
        }
        ok = warp_wait(done(slot), (u >> 1) & 1, abort_flag, W.status, kWhereWalkDone);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t tm = tmem + slot * kSlot + lanes;
#pragma unroll
        for (int k = 0; k < kTcK; k += 16) {
          uint32_t x[16], y[16], z[16];
          tmem_ld_32x32b<16>(tm + k, x);
          tmem_ld_32x32b<16>(tm + kTcK + k, y);
          tmem_ld_32x32b<16>(tm + 2 * kTcK + k, z);
          tmem_ld_wait();
          tmem_ld_fence_regs(x);
          tmem_ld_fence_regs(y);
          tmem_ld_fence_regs(z);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            S[k + e] = fmaf(t, S[k + e], __uint_as_float(x[e]) + (__uint_as_float(y[e]) + __uint_as_float(z[e])));
        }
        tc_fence_before_sync();
        mbar_arrive(tfree(slot));
      }
      if (!ok) break;
      if (W.segs == 1) {
        if (A.H_T != nullptr && in) {
#pragma unroll
          for (int k = 0; k < kTcK; ++k)
            if (k < A.K) A.H_T[state + static_cast<int64_t>(k) * A.V] = S[k];
        }
        continue;
      }
      if (own) {
        float4* sums = W.sums + (at.head * W.segs + at.seg) * (kTcK * kTcV / 4);
#pragma unroll
        for (int kt = 0; kt < kTcK / 16; ++kt)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sums[2 * ((kt * (kTcV / 16) + (v >> 4)) * 32 + (v & 7) * 4 + q) + ((v >> 3) & 1)] = make_float4(
                S[16 * kt + 2 * q], S[16 * kt + 2 * q + 1], S[16 * kt + 2 * q + 8], S[16 * kt + 2 * q + 9]);
      }
      if (tid == 0 && at.slice == 0) W.seg_tot[at.chain * W.segs + at.seg] = decay;
    }
  }
  let_next();
  cp_async_wait<0>();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_ssm_tc_walk(const TcWalkArgs& w, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_tc_walk_kernel), kSmem, ready);
  if (e != cudaSuccess) return e;
  const SsmArgs& a = w.a;
  CUtensorMap v;
  if (!make_tensor_map_rows(&v, a.v, a.V, a.N, a.v_stride, a.T, a.B, kTcV, kTile))
    return cudaErrorInvalidValue;
  const unsigned items = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.N * w.slices * w.segs);
  return launch_next(ssm_tc_walk_kernel, items < 152 ? items : 152, kThreads, kSmem, s, v, w, items);
}

}  // namespace m2rnn
