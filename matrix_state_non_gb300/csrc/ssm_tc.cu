// Outputs of the selective state space scan on the 5th-generation tensor
// cores, for tiles of 128 steps of one head and up to 64 state rows and value
// columns (the mathematics in ssm.cu, the phases in ssm_mma.cu):
//     y_i = first_i (S + since S0)^T q_i + sum_j P_ij v_j + w_r (*) v_i,
//     P_ij = exp(l_i - l_j) D_j (q_i . k_j) for j <= i.
// One persistent block per SM:
//   warps 9-11  producers: q, k, v by TMA (128-byte swizzle), the decays by bulk
//               copies, into a ring of three stages; a sequence's last tile row by
//               row, with zeros behind its end; the state, S and S0 joined in fp32,
//               by way of registers as two bf16 operands;
//   warp 8      issues the products: Q K^T and Q times the state's two parts
//               (M = 128) into one of two tensor-memory slots, then P V, with P's
//               two parts taken from tensor memory;
//   warps 0-3, 4-7  take the slots in turn, a thread a row: decay the scores,
//               split P into two bf16 parts and write them back; then y.
// P's large part takes its place in the scores' first half and P V the second,
// so with the state's product and P's small part a slot is 256 columns and two
// tiles are in work at once.  The factor of row i and an
// earlier block of 32 steps is one exponential per row and block times a
// tabled factor per step, so a tile takes some 40 exponentials a row, not 128.
//
// B=2 heads=16 T=16384 64x64, shared q and k: 73 us (whole scan 120), 412 MB
// through L2; without the states' 134 MB, which go through L2 in fp32, and
// their split it would be 57.  (Operands in one bf16 part each, rounded by the
// walk: 52 us, and y's error a fifth above its rounding.)  y by a TMA store: no
// gain, left out.
#include <cuda_runtime.h>

#include <cstdint>

#include "gate.cuh"
#include "ssm_tc.cuh"

namespace m2rnn {
namespace {

// One warp per (chain, chunk), two steps a lane, eight heads a block.
__global__ void __launch_bounds__(256) ssm_tile_decay_kernel(SsmArgs A, TileDecay* out, float* tot, int nc,
                                                             StatusBlock* status) {
  let_next();
  if (blockIdx.x == 0 && threadIdx.x < sizeof(StatusBlock) / 4) reinterpret_cast<unsigned*>(status)[threadIdx.x] = 0u;
  const int lane = threadIdx.x & 31, heads = (A.N + 7) / 8, own = lane >> 4, in = lane & 15;
  const unsigned bc = blockIdx.x / heads;
  const int n = (blockIdx.x - bc * heads) * 8 + (threadIdx.x >> 5), b = bc / nc, c = bc - b * nc;
  if (n >= A.N) return;
  const int64_t id = (static_cast<int64_t>(b) * A.N + n) * nc + c;
  const int len = ssm_len(A, b), t = c * kChunk + 2 * lane;
  const uint16_t* p = static_cast<const uint16_t*>(A.dt) + (static_cast<int64_t>(b) * A.T + t) * A.dt_stride + n;
  const float bias = A.dt_bias ? A.dt_bias[n] : 0.f, An = A.A[n];
  const float D0 = t < len ? softplus_f(to_f32(p[0]) + bias) : 0.f;
  const float D1 = t + 1 < len ? softplus_f(to_f32(p[A.dt_stride]) + bias) : 0.f;
  const float a0 = log_decay(D0, An), a1 = log_decay(D1, An);
  // Within the block of 32 steps: the sum up to a step, and the sum behind it.
  float up = a0 + a1, down = up, low = two_sum_low(a0, a1, up);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, up, o, 16), y = __shfl_down_sync(0xffffffffu, down, o, 16);
    const float z = __shfl_up_sync(0xffffffffu, low, o, 16);
    if (in >= o) {
      const float s = up + x;
      low += z + two_sum_low(up, x, s);
      up = s;
    }
    if (in + o < 16) down += y;
  }
  float before = __shfl_up_sync(0xffffffffu, up, 1, 16), behind = __shfl_down_sync(0xffffffffu, down, 1, 16);
  float before_low = __shfl_up_sync(0xffffffffu, low, 1, 16);
  if (in == 0) before = before_low = 0.f;
  if (in == 15) behind = 0.f;
  const float s0 = behind + a1, s1 = behind;
  const float T0 = __shfl_sync(0xffffffffu, up, 15), T1 = __shfl_sync(0xffffffffu, up, 31);
  const float rest = own == 0 ? T1 : 0.f;
  TileDecay& d = out[id];
  const int i = 2 * lane;
  auto put = [&](float* at, float x, float y) { *reinterpret_cast<float2*>(at + i) = make_float2(x, y); };
  const float r0 = before + a0;
  put(d.rel, r0, up);
  put(d.lo, before_low + two_sum_low(before, a0, r0), low);
  put(d.cf, expf(s0) * D0, expf(s1) * D1);
  put(d.D, D0, D1);
  put(d.wD, expf(s0 + rest) * D0, expf(s1 + rest) * D1);
  if (lane == 0) {
    *reinterpret_cast<float4*>(d.T) = make_float4(T0, T1, 0.f, 0.f);
    tot[id] = expf(T0 + T1);
  }
}

constexpr int kEpi = 256, kMmaWarp = 8, kProd = 96, kThreads = kEpi + 32 + kProd;  // 12 warps: 168 registers
constexpr int kStages = 3;

// Shared memory of a stage.  Q, K, V: 128 rows of 128 bytes, 16-byte pieces
// XOR-swizzled by (row mod 8), 1 KB aligned, as TMA writes and the products'
// descriptors read them; the states as tc_state_at orders them.
constexpr int kOffK = kOp, kOffV = 2 * kOp, kOffS = 3 * kOp, kOffSLo = kOffS + kTcStateBytes,
              kOffD = kOffSLo + kTcStateBytes, kOffWr = kOffD + 2 * kTileDecayCopied,
              kStage = (kOffWr + kTcV * 2 + 1023) / 1024 * 1024;
constexpr int kOffBar = kStages * kStage;  // barriers, then the tensor-memory address and the abort flag
constexpr int kSmem = kOffBar + 256 + 1024;  // 1024: alignment
constexpr int kYPitch = kTcV * 2 + 16;  // y rows on their way out, over Q and K
static_assert(kTile * kYPitch <= 2 * kOp, "y fits over Q and K");
static_assert(kSmem <= 227 * 1024, "shared memory");

// Tensor-memory columns of a slot.
constexpr uint32_t kColP = 0, kColPV = 64, kColS = 128, kColPLo = 192, kSlot = 256;

// The tiles of a block in order: tile tt of (chain, slice) `head`, every gridDim.x-th of them, heads side by side.
// Stepping and `live` go without divisions where there are no lengths: the warps ask for every tile of the block.
struct TileWalk {
  const TcOutArgs& W;
  unsigned id, tt, head, heads, tiles, rows, rest;
  __device__ __forceinline__ TileWalk(const TcOutArgs& w, unsigned heads, unsigned tiles)
      : W(w), id(blockIdx.x), heads(heads), tiles(tiles) {
    tt = id / heads;
    head = id - tt * heads;
    rows = gridDim.x / heads;
    rest = gridDim.x - rows * heads;
  }
  __device__ __forceinline__ bool there() const { return id < tiles; }
  __device__ __forceinline__ void next() {
    id += gridDim.x;
    tt += rows;
    head += rest;
    if (head >= heads) {
      head -= heads;
      ++tt;
    }
  }
  __device__ __forceinline__ bool live() const {  // steps of the sequence in it
    const int len = W.a.lengths ? ssm_len(W.a, head / (W.slices * W.a.N)) : W.a.T;
    return static_cast<int>(tt) * kTile < len;
  }
};

struct TilePlace {
  int b, n, gq, v0, width, len, t0, seg;
  int64_t chain, head;
};

__device__ __forceinline__ TilePlace tile_place(const TileWalk& at) {
  const TcOutArgs& W = at.W;
  const SsmArgs& A = W.a;
  TilePlace p;
  const unsigned bn = W.slices == 1 ? at.head : at.head / W.slices, slice = at.head - bn * W.slices;
  p.head = at.head;
  p.chain = bn;
  p.b = bn / A.N;
  p.n = bn - p.b * A.N;
  p.gq = A.G == 1 ? 0 : p.n / (A.N / A.G);
  p.v0 = slice * kTcV;
  p.width = min(kTcV, A.V - p.v0);
  p.len = ssm_len(A, p.b);
  p.t0 = at.tt * kTile;
  p.seg = 2 * static_cast<int>(at.tt) / W.per_seg;
  return p;
}

// A value of v that is not finite times the zero scores of the steps before it is NaN: those rows of P V are summed
// again, over their own steps alone, column by column.  For the rows of one warp (row i of the tile at yr, its
// tensor-memory lanes at tm), whose y has been staged; rows that are not finite by themselves come out as they were.
// (A tile whose state is not finite already is not summed again: nothing would come of it.)
__device__ __noinline__ void mend_columns(uint32_t st, uint32_t yr, uint32_t tm, int w, int i, bool in, float first) {
  for (int c = 0; c < kTcV; ++c) {
    bool hit = in && (not_finite(ld_shared_u16(yr + 2 * c)) & kNotFinite) != 0u;
    if (!__any_sync(0xffffffffu, hit)) continue;
    uint32_t s[2];
    tmem_ld_32x32b<2>(tm + kColS + (c & ~1), s);
    tmem_ld_wait();
    tmem_ld_fence_regs(s);
    auto v = [&](int j) { return bf16_bits_to_f32(ld_shared_u16(st + kOffV + piece_at(j, c >> 3) + (c & 7) * 2)); };
    float y = fmaf(bf16_bits_to_f32(ld_shared_u16(st + kOffWr + c * 2)), v(i), first * __uint_as_float(s[c & 1]));
    hit = hit && isfinite(y);
    if (!__any_sync(0xffffffffu, hit)) continue;
    for (int jb = 0; jb <= w; ++jb) {
      uint32_t hi[16], lo[16];
      tmem_ld_32x32b<16>(tm + kColP + 16 * jb, hi);
      tmem_ld_32x32b<16>(tm + kColPLo + 16 * jb, lo);
      tmem_ld_wait();
      tmem_ld_fence_regs(hi);
      tmem_ld_fence_regs(lo);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int j = 32 * jb + 2 * x;
        if (j <= i) y = fmaf(bf16lo(hi[x]) + bf16lo(lo[x]), v(j), y);
        if (j + 1 <= i) y = fmaf(bf16hi(hi[x]) + bf16hi(lo[x]), v(j + 1), y);
      }
    }
    if (hit) st_shared_u16(yr + 2 * c, static_cast<uint16_t>(pack_bf16x2(y, 0.f) & 0xFFFFu));
  }
}

__device__ __forceinline__ uint64_t desc_state(uint32_t addr) { return smem_desc_noswizzle(addr, kTcV * 16, 128); }

__global__ void __launch_bounds__(kThreads, 1) 
    ssm_tc_out_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, TcOutArgs W, unsigned heads, unsigned tiles) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const SsmArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem), bars = base + kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };               // [3] producers -> products, outputs
  auto empty = [&](int s) { return bars + 24 + 8 * s; };         // [3] outputs -> producers
  auto scores = [&](int s) { return bars + 48 + 8 * s; };        // [2] products -> outputs
  auto pready = [&](int s) { return bars + 64 + 8 * s; };        // [2] outputs -> products
  auto ofull = [&](int s) { return bars + 80 + 8 * s; };         // [2] products -> outputs
  auto tfree = [&](int s) { return bars + 96 + 8 * s; };         // [2] outputs -> products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 128);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 132);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), kProd);
      mbar_init(empty(s), kEpi / 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(scores(s), 1);
      mbar_init(pready(s), kEpi / 2);
      mbar_init(ofull(s), 1);
      mbar_init(tfree(s), kEpi / 2);
    }
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (tid < kTcV / 2)  // w_r where there is none
    for (int s = 0; s < kStages; ++s) reinterpret_cast<uint32_t*>(smem + s * kStage + kOffWr)[tid] = 0u;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_previous();

  if (warp > kMmaWarp) {
    // ---------------- producers ----------------
    const int p = tid - kEpi - 32;
    if (p == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
    }
    int u = 0;  // live tiles of this block
    bool ok = true;
    for (TileWalk at(W, heads, tiles); at.there(); at.next()) {
      if (!at.live()) continue;
      const TilePlace t = tile_place(at);
      const int s = u % kStages;
      // The state before the tile, eight state rows of a value column at a time: on its way before the stage is free.
      constexpr int kPieces = kTcState / 2, kPer = (kPieces + kProd - 1) / kProd;
      float4 own[kPer][2], before[kPer][2];
      const float4* l = W.local + (t.head * W.nt + t.t0 / kTile) * kTcState;
      const float4* z = W.start + (t.head * W.segs + t.seg) * kTcState;
      const TileDecay* d = W.decay + t.chain * W.nc + t.t0 / kChunk;
      const float since = t.seg > 0 ? d->T[2] : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = p + i * kProd, x = tc_piece_at(e / kTcV * 8, e % kTcV);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          own[i][h] = before[i][h] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e >= kPieces) continue;
          own[i][h] = l[x + h * kTcV];
          if (t.seg > 0) before[i][h] = z[x + h * kTcV];
        }
      }
      if (u >= kStages && !warp_wait(empty(s), (u / kStages - 1) & 1, abort_flag, W.status, kWhereOutEmpty)) {
        ok = false;
        break;
      }
      const uint32_t st = base + s * kStage, bar = full(s);
      const bool whole = t.t0 + kTile <= t.len;
      if (p == 0) {
        const uint32_t wr_bytes = A.w_r != nullptr ? 2 * t.width : 0;
        mbar_expect_tx(bar, 2 * kTileDecayCopied + wr_bytes + (whole ? 3 * kOp : 0));
        if (whole) {
          tma_load_4d(st, &map_q, bar, 0, t.gq, t.t0, t.b);
          tma_load_4d(st + kOffK, &map_k, bar, 0, t.gq, t.t0, t.b);
          tma_load_4d(st + kOffV, &map_v, bar, t.v0, t.n, t.t0, t.b);
        }
        bulk_load(st + kOffD, d, kTileDecayCopied, bar);
        bulk_load(st + kOffD + kTileDecayCopied, d + 1, kTileDecayCopied, bar);
        if (wr_bytes != 0)
          bulk_load(st + kOffWr, static_cast<const uint16_t*>(A.w_r) + t.n * A.V + t.v0, wr_bytes, bar);
      }
      if (!whole) {
        // A warp an operand; rows r, r + 4, ..., the eight pieces of a row side by side.
        const int op = warp - kMmaWarp - 1, piece = lane & 7;
        const int64_t row = static_cast<int64_t>(t.b) * A.T + t.t0;
        const int64_t stride = op == 0 ? A.q_stride : op == 1 ? A.k_stride : A.v_stride;
        const uint16_t* src =
            op == 0   ? static_cast<const uint16_t*>(A.q) + row * stride + static_cast<int64_t>(t.gq) * A.K
            : op == 1 ? static_cast<const uint16_t*>(A.k) + row * stride + static_cast<int64_t>(t.gq) * A.K
                      : static_cast<const uint16_t*>(A.v) + row * stride + static_cast<int64_t>(t.n) * A.V + t.v0;
        const bool col = piece * 8 < (op == 2 ? t.width : A.K);
#pragma unroll 4
        for (int r = lane >> 3; r < kTile; r += 4) {
          const bool in = col && t.t0 + r < t.len;
          cp_async_16(st + op * kOp + piece_at(r, piece), in ? src + r * stride + piece * 8 : src, in);
        }
        cp_async_commit();
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = p + i * kProd;
        if (e >= kPieces) continue;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 &a = own[i][h], &b = before[i][h];
          split2(fmaf(since, b.x, a.x), fmaf(since, b.y, a.y), hi[2 * h], lo[2 * h]);
          split2(fmaf(since, b.z, a.z), fmaf(since, b.w, a.w), hi[2 * h + 1], lo[2 * h + 1]);
        }
        const uint32_t to = st + kOffS + tc_state_at(e / kTcV * 8, e % kTcV);
        st_shared_v4(to, hi);
        st_shared_v4(to + kTcStateBytes, lo);
      }
      if (!whole) cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(bar);
      ++u;
    }
    if (!ok)  // the copies in flight land before the block ends
      for (int x = max(0, u - kStages); x < u; ++x)
        mbar_wait_timed(full(x % kStages), (x / kStages) & 1, nullptr, kWhereOutDrain);
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    constexpr uint32_t kIdQK = idesc_bf16_f32(128, kTile, false, false), kIdS = idesc_bf16_f32(128, kTcV, false, false),
                       kIdPV = idesc_bf16_f32(128, kTcV, false, true);
    // Live tiles in order: `s` is the next whose scores are issued (its segment's place known), `o` the next
    // for P V.  Whichever has its operands is issued; neither waits behind the other.
    int s = 0, o = 0;
    TileWalk at(W, heads, tiles);
    auto find = [&] {  // the next live tile
      while (at.there() && !at.live()) at.next();
    };
    find();
    uint64_t since = global_timer_ns();
    for (uint32_t spins = 0; at.there() || o < s;) {
      bool moved = false;
      if (o < s && __all_sync(0xffffffffu, mbar_test_wait(pready(o & 1), (o >> 1) & 1))) {
        if (elect_one()) {
          tc_fence_after_sync();
          const uint32_t tm = tmem + (o & 1) * kSlot, sv = base + (o % kStages) * kStage + kOffV;
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_f16_ts(tm + kColPV, tm + kColPLo + 8 * kk, desc_sw128(sv + kk * 2048), kIdPV, kk > 0);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_f16_ts(tm + kColPV, tm + kColP + 8 * kk, desc_sw128(sv + kk * 2048), kIdPV, true);
          tc_commit(ofull(o & 1));
        }
        __syncwarp();
        ++o;
        moved = true;
      }
      if (at.there() && s - o < 2 && __all_sync(0xffffffffu, mbar_test_wait(full(s % kStages), (s / kStages) & 1)) &&
          (s < 2 || __all_sync(0xffffffffu, mbar_test_wait(tfree(s & 1), ((s >> 1) - 1) & 1)))) {
        if (elect_one()) {
          tc_fence_after_sync();
          const uint32_t tm = tmem + (s & 1) * kSlot, sq = base + (s % kStages) * kStage;
#pragma unroll
          for (int kk = 0; kk < kTcK / 16; ++kk)
            tc_mma_f16_ss(tm, desc_sw128(sq + kk * 32), desc_sw128(sq + kOffK + kk * 32), kIdQK, kk > 0);
#pragma unroll
          for (int kk = 0; kk < kTcK / 16; ++kk)
            tc_mma_f16_ss(tm + kColS, desc_sw128(sq + kk * 32), desc_state(sq + kOffSLo + kk * 2 * kTcV * 16), kIdS,
                          kk > 0);
#pragma unroll
          for (int kk = 0; kk < kTcK / 16; ++kk)
            tc_mma_f16_ss(tm + kColS, desc_sw128(sq + kk * 32), desc_state(sq + kOffS + kk * 2 * kTcV * 16), kIdS,
                          true);
          tc_commit(scores(s & 1));
        }
        __syncwarp();
        ++s;
        at.next();
        find();
        moved = true;
      }
      if (moved) {
        spins = 0;
        since = global_timer_ns();
      } else if ((++spins & 255u) == 0u) {  // bounded, as every wait
        bool stop = *abort_flag != 0;
        if (!stop && global_timer_ns() - since > kWaitLimitNs) {
          if (lane == 0) report_device_error(W.status, kStatusTimeout, kWhereOutP);
          *abort_flag = 1;
          stop = true;
        }
        if (__any_sync(0xffffffffu, stop)) break;
      }
    }
    if (at.there() || o < s) {  // given up: the products in flight end before their memory is freed
      for (int x = max(0, s - 2); x < s; ++x) mbar_wait_timed(scores(x & 1), (x >> 1) & 1, nullptr, kWhereOutDrain);
      for (int x = max(0, o - 2); x < o; ++x) mbar_wait_timed(ofull(x & 1), (x >> 1) & 1, nullptr, kWhereOutDrain);
    }
  } else {
    // ---------------- outputs: thread = row of the tile ----------------
    const int group = warp >> 2, w = warp & 3, i = 32 * w + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    int u = 0;
    for (TileWalk at(W, heads, tiles); at.there(); at.next()) {
      const bool live = at.live();
      const int v = u;
      u += live;
      if (live ? (v & 1) != group : group != 0) continue;
      const TilePlace t = tile_place(at);
      uint16_t* y = static_cast<uint16_t*>(A.y) + ((static_cast<int64_t>(t.b) * A.T + t.t0) * A.N + t.n) * A.V + t.v0;
      const int64_t stride = static_cast<int64_t>(A.N) * A.V;
      const int rows = min(kTile, A.T - t.t0);
      if (!live) {  // behind the sequence's end
        for (int e = tid; e < rows * (t.width / 8); e += kEpi / 2) {
          const int per = t.width / 8;
          *reinterpret_cast<uint4*>(y + (e / per) * stride + (e % per) * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const int s = v % kStages, slot = v & 1;
      const uint32_t tm = tmem + slot * kSlot + lanes, st = base + s * kStage;
      const uint8_t* stp = smem + s * kStage;
      // The stage (decays, v) and then the scores.
      if (!warp_wait(full(s), (v / kStages) & 1, abort_flag, W.status, kWhereOutFull)) break;
      const float* dec = reinterpret_cast<const float*>(stp + kOffD);
      constexpr int kHalf = kTileDecayCopied / 4;
      auto decays = [&](int block) { return dec + (block >> 1) * kHalf + (block & 1) * 32; };  // rel; cf 64, D 128, lo 192 behind
      const float rel = decays(w)[lane], low = decays(w)[3 * kChunk + lane];
      float T[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) T[x] = dec[(x >> 1) * kHalf + 4 * kChunk + (x & 1)];
      if (!warp_wait(scores(slot), (v >> 1) & 1, abort_flag, W.status, kWhereOutScores)) break;
      tc_fence_after_sync();
      // Blocks of 32 steps before the warp's own, the next block's scores on their way.  (A loop, not unrolled: the
      // warps are in different phases, and their code has to fit the instruction cache together.)
      uint32_t sc[32];
      tmem_ld_32x32b<32>(tm, sc);
      float mid = w < 2 ? 0.f : w == 2 ? T[1] : T[1] + T[2];  // the blocks between
#pragma unroll 1
      for (int jb = 0; jb < w; ++jb) {
        const float4* f = reinterpret_cast<const float4*>(decays(jb) + kChunk);
        const float rf = exp_fast(rel + mid);
        mid = jb == 0 && w == 3 ? T[2] : 0.f;
        uint32_t hi[16], lo[16];
        tmem_ld_wait();
        tmem_ld_fence_regs(sc);
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 c = f[x / 4];
          float a, b, d, e;
          mul2(a, b, c.x, c.y, rf, rf);
          mul2(d, e, c.z, c.w, rf, rf);
          mul2(a, b, a, b, __uint_as_float(sc[x]), __uint_as_float(sc[x + 1]));
          mul2(d, e, d, e, __uint_as_float(sc[x + 2]), __uint_as_float(sc[x + 3]));
          split2(a, b, hi[x / 2], lo[x / 2]);
          split2(d, e, hi[x / 2 + 1], lo[x / 2 + 1]);
        }
        tmem_ld_32x32b<32>(tm + 32 * (jb + 1), sc);
        tmem_st_32x32b_x16(tm + kColP + 16 * jb, hi);
        tmem_st_32x32b_x16(tm + kColPLo + 16 * jb, lo);
      }
      {
        const float4* dr = reinterpret_cast<const float4*>(decays(w));
        uint32_t hi[16], lo[16];
        tmem_ld_wait();
        tmem_ld_fence_regs(sc);
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 r = dr[x / 4], D = dr[(2 * kChunk + x) / 4], m = dr[(3 * kChunk + x) / 4];
          const float a = x <= lane ? __uint_as_float(sc[x]) * (exp_fast((rel - r.x) + (low - m.x)) * D.x) : 0.f;
          const float b = x + 1 <= lane ? __uint_as_float(sc[x + 1]) * (exp_fast((rel - r.y) + (low - m.y)) * D.y) : 0.f;
          const float c = x + 2 <= lane ? __uint_as_float(sc[x + 2]) * (exp_fast((rel - r.z) + (low - m.z)) * D.z) : 0.f;
          const float e = x + 3 <= lane ? __uint_as_float(sc[x + 3]) * (exp_fast((rel - r.w) + (low - m.w)) * D.w) : 0.f;
          split2(a, b, hi[x / 2], lo[x / 2]);
          split2(c, e, hi[x / 2 + 1], lo[x / 2 + 1]);
        }
        tmem_st_32x32b_x16(tm + kColP + 16 * w, hi);
        tmem_st_32x32b_x16(tm + kColPLo + 16 * w, lo);
#pragma unroll
        for (int x = 0; x < 16; ++x) hi[x] = 0u;
#pragma unroll 1
        for (int jb = w + 1; jb < 4; ++jb) {
          tmem_st_32x32b_x16(tm + kColP + 16 * jb, hi);
          tmem_st_32x32b_x16(tm + kColPLo + 16 * jb, hi);
        }
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(pready(slot));
      // Meanwhile the states' part and w_r v.
      float out[kTcV];
      float first = rel;
#pragma unroll
      for (int x = 0; x < 3; ++x) first += x < w ? T[x] : 0.f;
      first = exp_fast(first);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[32];
        tmem_ld_32x32b<32>(tm + kColS + 32 * h, a);
        tmem_ld_wait();
        tmem_ld_fence_regs(a);
#pragma unroll
        for (int x = 0; x < 32; x += 2)
          mul2(out[32 * h + x], out[32 * h + x + 1], __uint_as_float(a[x]), __uint_as_float(a[x + 1]), first, first);
      }
#pragma unroll
      for (int c = 0; c < kTcV / 8; ++c) {
        const uint4 vv = ld_shared_v4(st + kOffV + piece_at(i, c)), ww = ld_shared_v4(st + kOffWr + c * 16);
        const uint32_t x[4] = {vv.x, vv.y, vv.z, vv.w}, z[4] = {ww.x, ww.y, ww.z, ww.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          fma2(out[8 * c + 2 * e], out[8 * c + 2 * e + 1], bf16lo(x[e]), bf16hi(x[e]), bf16lo(z[e]), bf16hi(z[e]));
      }
      if (!warp_wait(ofull(slot), (v >> 1) & 1, abort_flag, W.status, kWhereOutDone)) break;
      tc_fence_after_sync();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[32];
        tmem_ld_32x32b<32>(tm + kColPV + 32 * h, a);
        tmem_ld_wait();
        tmem_ld_fence_regs(a);
#pragma unroll
        for (int x = 0; x < 32; ++x) out[32 * h + x] += __uint_as_float(a[x]);
      }
      const bool in = t.t0 + i < t.len;
      float zero[2] = {0.f, 0.f};  // NaN where one of the row's values is not finite
#pragma unroll
      for (int x = 0; x < kTcV; x += 2) fma2(zero[0], zero[1], out[x], out[x + 1], 0.f, 0.f);
      const bool spoilt = __any_sync(0xffffffffu, in && !(zero[0] + zero[1] == 0.f));
      if (!spoilt) {
        tc_fence_before_sync();
        mbar_arrive(tfree(slot));
      }
      // Rows to shared memory (over Q and K, which the products are done with), then out in whole lines.
      const uint32_t yr = st + i * kYPitch;
#pragma unroll
      for (int c = 0; c < kTcV / 8; ++c) {
        const uint32_t x0 = pack_bf16x2(out[8 * c], out[8 * c + 1]), x1 = pack_bf16x2(out[8 * c + 2], out[8 * c + 3]),
                       x2 = pack_bf16x2(out[8 * c + 4], out[8 * c + 5]), x3 = pack_bf16x2(out[8 * c + 6], out[8 * c + 7]);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(yr + 16 * c), "r"(in ? x0 : 0u), "r"(in ? x1 : 0u),
                     "r"(in ? x2 : 0u), "r"(in ? x3 : 0u)
                     : "memory");
      }
      if (spoilt) {
        mend_columns(st, yr, tm, w, i, in, first);
        tc_fence_before_sync();
        mbar_arrive(tfree(slot));
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = 32 * w + 4 * e + (lane >> 3), c = (lane & 7) * 8;
        if (r < rows && c < t.width)
          *reinterpret_cast<uint4*>(y + r * stride + c) = ld_shared_v4(st + r * kYPitch + c * 2);
      }
      fence_proxy_async_smem();  // TMA writes there next
      mbar_arrive(empty(s));
    }
  }
  cp_async_wait<0>();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_ssm_tile_decay(const SsmArgs& a, TileDecay* out, float* tot, int nc, StatusBlock* status,
                                  cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.B) * nc * ((a.N + 7) / 8));
  ssm_tile_decay_kernel<<<blocks, 256, 0, s>>>(a, out, tot, nc, status);
  return cudaGetLastError();
}

cudaError_t launch_ssm_tc_out(const TcOutArgs& w, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_tc_out_kernel), kSmem, done);
  if (e != cudaSuccess) return e;
  const SsmArgs& a = w.a;
  CUtensorMap q, k, v;
  if (!make_tensor_map_rows(&q, a.q, a.K, a.G, a.q_stride, a.T, a.B, kTcK, kTile) ||
      !make_tensor_map_rows(&k, a.k, a.K, a.G, a.k_stride, a.T, a.B, kTcK, kTile) ||
      !make_tensor_map_rows(&v, a.v, a.V, a.N, a.v_stride, a.T, a.B, kTcV, kTile))
    return cudaErrorInvalidValue;
  const unsigned heads = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.N * w.slices);
  const unsigned tiles = heads * static_cast<unsigned>(w.nt);
  return launch_next(ssm_tc_out_kernel, tiles < 152 ? tiles : 152, kThreads, kSmem, s, q, k, v, w, heads, tiles);
}

}  // namespace m2rnn
