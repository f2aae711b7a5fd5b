// Shared by the hybrid layer's kernels (short convolution, selective state
// space scan, gradient clipping): element access in the input type, the
// argument blocks that the C-ABI layer fills, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/m2rnn.h"
#include "ptx.cuh"

namespace m2rnn {

// Element type tags: bf16 as raw bits, fp32 as float.
__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float x) {
  return static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
}

// Allows `kernel` its dynamic shared memory, once per GPU: `done` is a static
// of the caller, a bit for each device.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches of one call that follow one another: when every block of a kernel
// has called let_next (or ended), the next one's blocks come to the SMs, where
// wait_previous holds them until its end and its writes (before they touch
// anything that an earlier launch of the call writes).  Mostly called behind a
// kernel's main loop: earlier, blocks that only wait cost a small call 1 to 2
// us of the 2 to 4 that this saves.  The first launch of a call is an ordinary
// one, so that inputs are there before any of them starts.
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... V>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, V... args) {
  cudaLaunchAttribute behind{};
  behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t at{};
  at.gridDim = grid;
  at.blockDim = dim3(threads);
  at.dynamicSmemBytes = smem;
  at.stream = s;
  at.attrs = &behind;
  at.numAttrs = 1;
  return cudaLaunchKernelEx(&at, kernel, static_cast<P>(args)...);
}

// 2^x and 1 / x by the hardware's approximations (a few units of fp32).
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.f + ex2_fast(-1.44269504f * x)); }

// Two fp32 fused multiply-adds in one instruction.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 d, {%0, %1};\n\t"
      "fma.rn.f32x2 d, a, b, d;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// Two fp32 products, two differences in one instruction.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void sub2(float& d0, float& d1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "sub.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(b0), "f"(b1));
}
// What the rounding of s = a + b left out, exactly (two-sum).
__device__ __forceinline__ float two_sum_low(float a, float b, float s) {
  const float w = s - a;
  return (a - (s - w)) + (b - w);
}
// d += a * b over kN elements, in pairs.
template <int kN>
__device__ __forceinline__ void fma_row(float (&d)[kN], const float (&a)[kN], const float (&b)[kN]) {
#pragma unroll
  for (int i = 0; i + 1 < kN; i += 2) fma2(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
  if constexpr (kN % 2 == 1) d[kN - 1] = fmaf(a[kN - 1], b[kN - 1], d[kN - 1]);
}

// ---------------------------------------------------------------------------
// Short causal convolution
// ---------------------------------------------------------------------------
constexpr int kConvMaxWidth = 8;

struct ConvArgs {
  const void* x;       // [B,T,C], rows x_stride elements apart
  const void* w;       // [C,W]
  const void* bias;    // [C] or null
  const void* x0;      // [B,W-1,C] or null (zero)
  const int* lengths;  // [B] or null (all T)
  void* y;             // forward: [B,T,C]
  void* x_T;           // forward: [B,W-1,C] or null
  const float* dy;     // backward: [B,T,C]
  const float* dx_T;   // backward: [B,W-1,C] or null
  float* dx;           // backward: [B,T,C]
  float* dw;           // backward: [C,W]
  float* db;           // backward: [C] or null
  float* dx0;          // backward: [B,W-1,C] or null
  float* part;         // backward: [parts][W+1][C]
  int64_t x_stride;
  int B, T, C, W;
  bool silu, bf16;
};

int conv_backward_parts(int64_t B, int64_t T, int64_t C);  // the most that any type and width takes
cudaError_t launch_conv_forward(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_backward(const ConvArgs& a, cudaStream_t s);
// One token: state [B,W-1,C] in place; a.x, a.y [B,C].
cudaError_t launch_conv_step(void* state, const ConvArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Selective state space scan
// ---------------------------------------------------------------------------
struct SsmArgs {
  const void* q;         // [B,T,G,K], tokens q_stride elements apart
  const void* k;         // [B,T,G,K]
  const void* v;         // [B,T,N,V]
  const void* dt;        // [B,T,N]
  const float* A;        // [N]
  const float* dt_bias;  // [N] or null
  const void* w_r;       // [N,V] or null
  const float* H_0;      // [B,N,K,V] or null
  const int* lengths;    // [B] or null
  void* y;               // forward: [B,T,N,V] in the input type
  float* H_T;            // forward: [B,N,K,V] or null
  const void* dy;        // backward: [B,T,N,V] in the input type
  const float* dH_T;     // backward: or null
  float* dq;             // backward: [B,T,G,K]
  float* dk;
  float* dv;             // [B,T,N,V]
  float* ddt;            // [B,T,N]
  float* dA;             // [N]
  float* ddt_bias;       // [N] or null
  float* dw_r;           // [N,V] or null
  float* dH_0;           // [B,N,K,V] or null
  void* ws;              // scratch behind the status block
  int64_t q_stride, k_stride, v_stride, dt_stride;
  int B, T, N, G, K, V;
  bool bf16;
};

size_t ssm_forward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t V, bool bf16);
size_t ssm_backward_scratch_bytes(int64_t B, int64_t T, int64_t N, int64_t G, int64_t K, int64_t V, bool bf16);
cudaError_t launch_ssm_forward(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_ssm_backward(const SsmArgs& a, cudaStream_t s);
// One token: H [B,N,K,V] in place; q, k [B,G,K], v, y [B,N,V], dt [B,N]
// (strides between sequences in the *_stride fields; T is ignored).
cudaError_t launch_ssm_step(float* H, const SsmArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------
// One piece of one tensor, the unit of work of a block.
struct GradChunk {
  const void* in;
  void* out;
  int32_t count;  // elements
  int32_t bf16;
  int64_t pad;
};
static_assert(sizeof(GradChunk) == 32, "plan entries are 32 bytes");

constexpr int kGradChunk = 8192;  // elements of a piece

size_t grad_clip_scratch_bytes();
// clip false: only the norm.
cudaError_t launch_grad_clip(const GradChunk* plan, int64_t chunks, float max_norm, bool clip, float* norm, void* ws,
                             cudaStream_t s);

}  // namespace m2rnn
