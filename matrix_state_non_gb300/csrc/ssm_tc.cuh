// The outputs of the selective state space scan on tcgen05 (ssm_tc.cu), in
// tiles of 128 steps: two chunks, one state.
#pragma once

#include "mma_common.cuh"
#include "ssm_mma.cuh"

namespace m2rnn {

// The decays of one chunk (64 steps) for the tiles: sums run within blocks of
// 32 steps, the rows of one warp's share of a tile.
struct __align__(16) TileDecay {
  float rel[kChunk];   // l_i - l before i's block,
  float cf[kChunk];    // exp(l at the end of j's block - l_j) D_j
  float D[kChunk];     // step sizes, 0 behind the sequence's end
  float lo[kChunk];    // the part of the sum that rel leaves out
  float T[4];          // the two blocks' sums; the decay from the segment's start to the chunk's (the walk's); padding
  float wD[kChunk];    // exp(l_63 - l_j) D_j, for the walk; not copied by the tiles
};
static_assert(sizeof(TileDecay) <= sizeof(ChunkDecay), "they share a scratch area");
constexpr int kTileDecayCopied = (4 * kChunk + 4) * 4;  // bytes of it a tile reads

constexpr int kTcK = 64, kTcV = 64;            // padded widths it is built for
constexpr int kTile = 2 * kChunk;               // steps
constexpr int kOp = kTile * 128;                // bytes of an operand of 128 rows of 64 columns
constexpr int kTcState = kTcK * kTcV / 4;       // a state in fp32: float4
constexpr int kTcStateBytes = kTcK * kTcV * 2;  // one bf16 part of it as the B operand of Q S

struct TcOutArgs {
  SsmArgs a;
  const TileDecay* decay;   // [B N][chunks]
  const float4* local;      // [B N][slices][tiles][kTcState]: the segment's own state before each tile
  const float4* start;      // [B N][slices][segs][kTcState]: the state before each segment
  StatusBlock* status;
  int nc, nt, segs, per_seg, slices;  // chunks (even), tiles, segments, chunks in each (even)
};

// A state in memory: float4 (k / 4, v) of four state rows of a value column.
__host__ __device__ constexpr int tc_piece_at(int k, int v) { return (k / 4) * kTcV + v; }

// Byte of state element (k, v) in an operand: core matrices of 8 value
// columns by 8 state rows, state rows contiguous.
__host__ __device__ constexpr int tc_state_at(int k, int v) {
  return (k / 8) * (kTcV * 16) + (v / 8) * 128 + (v % 8) * 16 + (k % 8) * 2;
}

// A bounded wait of a whole warp: all lanes go on, or all give up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, StatusBlock* status,
                                          uint32_t where) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, where));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
               : "memory");
}

// Descriptor of a 128-byte swizzled operand: 8-row groups 1 KB apart; an operand wider than 64 columns goes on in
// another such tile, `next` bytes behind.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t next = 16) {
  return smem_desc_noswizzle(addr, next, 1024) | (static_cast<uint64_t>(2) << 61);
}
// Byte of 16-byte piece c of row r in a swizzled operand.
__device__ __forceinline__ uint32_t piece_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

struct TcWalkArgs {
  SsmArgs a;
  TileDecay* decay;    // [B N][chunks]; the walk writes T[2] of every second
  const float* tot;    // [B N][chunks]: a chunk's whole decay
  float4* local;       // [B N][slices][tiles][kTcState], in the order of tc_piece_at
  float4* sums;        // [B N][slices][segs][1024]: the state each segment leaves, in the order of Frag (ssm_mma.cu)
  float* seg_tot;      // [B N][segs]
  StatusBlock* status;
  int nc, nt, segs, per_seg, slices;
};

cudaError_t launch_ssm_tc_walk(const TcWalkArgs& w, cudaStream_t s);
cudaError_t launch_ssm_tile_decay(const SsmArgs& a, TileDecay* out, float* tot, int nc, StatusBlock* status,
                                  cudaStream_t s);
cudaError_t launch_ssm_tc_out(const TcOutArgs& w, cudaStream_t s);

}  // namespace m2rnn
