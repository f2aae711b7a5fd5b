// Shared by the selective state space scan's kernel files.
#pragma once

#include "layer.cuh"

namespace m2rnn {

// Where a chunk's gradients go: dq, dk [B,T,qk_heads,K] (qk_heads = N: per
// value head, summed over shared heads afterwards where G < N), per-chunk
// partials of dw_r [chunks][V] (or null) and of (dA, ddt_bias) [chunks].
struct SsmGradOut {
  float* dq;
  float* dk;
  float* wr_part;
  float2* ab_part;
  int qk_heads;
};

}  // namespace m2rnn
