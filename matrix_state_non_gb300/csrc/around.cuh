// Shared by the operators around the scans' layer: the residual norm, the gated
// linear recurrence and the orthogonalised update.  Argument blocks that the
// C-ABI layer fills, and the launchers.
#pragma once

#include "layer.cuh"

namespace m2rnn {

// A tiled tensor map of up to 5 dimensions, innermost first (strides in bytes,
// from the second dimension on); what lies outside reads as zero.
bool make_tensor_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int rank, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle);

// A launch in clusters of `blocks` blocks; behind: as launch_next.
template <typename... P, typename... V>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t grid, int blocks, int threads, int smem, bool behind, cudaStream_t s,
                           V... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = at;
  c.numAttrs = behind ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// out[j] = sum over p of part[p][j], in a fixed order; with `two`, rows are 2 D
// wide and columns from D on are out2's (which may be null).
cudaError_t launch_sum_parts(const float* part, float* out, float* out2, bool two, int parts, int64_t D,
                             cudaStream_t s);

// ---------------------------------------------------------------------------
// Residual norm
// ---------------------------------------------------------------------------
constexpr int kNormMaxWidth = 16384;
constexpr int kScaleBlock = 128;  // values of a row that share a scale

struct NormRowsArgs {
  const void* x;         // [rows, D], rows x_stride elements apart
  const void* residual;  // [rows, D] or null
  const float* w;        // [D]
  void* h;               // [rows, D]: forward: out or null; backward: in
  void* y;               // [rows, D]
  float* scale;          // [rows, ceil(D / 128)], for e4m3
  const void* dy;        // backward: [rows, D]
  const float* dh;       // backward: [rows, D] or null
  float* dx;             // backward: [rows, D]
  float* dw;             // backward: [D]
  float* part;           // backward: [parts][D]
  int64_t rows, x_stride;
  int D;
  float eps;
  bool x_bf16, h_bf16, dy_bf16;
  int y_type;
};

int norm_rows_parts(int64_t rows, int64_t D);
cudaError_t launch_residual_norm(const NormRowsArgs& a, cudaStream_t s);
cudaError_t launch_residual_norm_backward(const NormRowsArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Gated linear recurrence
// ---------------------------------------------------------------------------
struct LinearArgs {
  const void* x;       // [B,T,C], rows x_stride elements apart
  const void* a;       // [B,T,C], rows a_stride elements apart
  const float* alpha;  // [C]
  const float* beta;   // [C] or null
  const float* H_0;    // [B,C] or null
  const int* lengths;  // [B] or null
  void* y;             // forward: [B,T,C]
  float* H_T;          // forward: [B,C] or null
  const void* dy;      // backward: [B,T,C]
  const float* dH_T;   // backward: [B,C] or null
  float* dx;           // backward: [B,T,C]
  float* da;           // backward: [B,T,C]
  float* dalpha;       // backward: [C]
  float* dbeta;        // backward: [C] or null
  float* dH_0;         // backward: [B,C] or null
  void* ws;            // backward
  int64_t x_stride, a_stride;
  int B, T, C;
  bool bf16;
};

size_t linear_backward_scratch_bytes(int64_t B, int64_t T, int64_t C);
cudaError_t launch_linear_forward(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s);
// One token: H [B,C] in place; a.x, a.a, a.y [B,C].
cudaError_t launch_linear_step(float* H, const LinearArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Orthogonalised update
// ---------------------------------------------------------------------------
constexpr int kOrthoMaxDim = 16384, kOrthoMaxSteps = 32;

struct OrthoArgs {
  const void* g;  // [n, rows, cols]
  uint16_t* out;  // [n, rows, cols] bf16
  void* ws;       // scratch behind the status block
  StatusBlock* status;
  int64_t n;
  int rows, cols, steps;
  float eps;
  bool bf16;
};

// 1 / (sqrt(sum) + eps) as a power of two times a factor: fp32 holds neither a norm beyond its largest value nor the
// inverse of one below 2^-128, so the power takes 64 binary places of those.
struct Inverse {
  float power, factor;
  __device__ __forceinline__ float of(float v) const { return v * power * factor; }
};
// With few fp64 operations (slow here): the root of the sum times an even power of two.
__device__ __forceinline__ Inverse inverse_norm(double sum, float eps) {
  float root = static_cast<float>(sum);  // 0, an infinity or NaN
  int half = sum == 0. ? -1000 : 0;
  if (sum > 0. && sum < 1.7e308) {
    half = ((__double2hiint(sum) >> 20) - 1023) >> 1;
    root = sqrtf(static_cast<float>(sum * __hiloint2double((1023 - 2 * half) << 20, 0)));  // in [1, 2)
  }
  const int by = half > 100 ? -64 : half < -100 && eps < 0x1p-100f ? 64 : 0;
  return {ldexpf(1.f, by), 1.f / (scalbnf(root, half + by) + ldexpf(eps, by))};
}

size_t ortho_scratch_bytes(int64_t n, int64_t rows, int64_t cols);
cudaError_t launch_orthogonalize(const OrthoArgs& a, cudaStream_t s);
// Matrices that a block has in shared memory (no scratch).
bool ortho_small(int64_t rows, int64_t cols);
cudaError_t launch_ortho_small(const OrthoArgs& a, cudaStream_t s);
// Long matrices with a side of up to 64.
bool ortho_thin(int64_t rows, int64_t cols);
size_t ortho_thin_scratch_bytes(int64_t n, int64_t rows, int64_t cols);
cudaError_t launch_ortho_thin(const OrthoArgs& a, cudaStream_t s);
// Clears the status block and sums the squares of every matrix: part [n][parts].
int ortho_sum_parts(int64_t size);
cudaError_t launch_ortho_sum(const OrthoArgs& a, int parts, double* part, cudaStream_t s);

}  // namespace m2rnn
