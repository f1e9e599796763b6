// block.cuh — argument blocks and device helpers of what stands around a mixer: the
// matrix product with its epilogue, and the norms with gate and residual scale.
#pragma once

#include <cuda_fp16.h>

#include "layers.cuh"

namespace dr {

// y = act(x W + bias) + residual; M rows, K -> N channels.  W[k, n] stands at k w_s + n, or
// (w_t) at n w_s + k.
struct LinearArgs {
  const void* x;
  const void* w;
  const void* bias;
  const void* res;
  void* y;
  void* slope;                 // act'(x W + bias), fp16 (bf16 types) or fp32; may be null
  int M, K, N, act, w_t;
  long long x_s, w_s, r_s;
  // backward
  const void* d_y;             // [M,N]
  void* dx;
  void* dw;
  void* db;
};

// h' = h + scale f(gate) n(branch);  y = n(h')
struct BlockNormArgs {
  const void* h;
  const void* branch;
  const void* gate;
  const float* scale;
  const float* post_w;
  const float* pre_w;
  void* h_out;
  void* y;
  int M, D, gate_act, post_norm;
  float eps, inv_d;
  long long h_s, b_s, g_s;
  // backward
  const void* d_h;
  const void* d_y;
  void* dh;
  void* db;
  void* dg;
  float* part;                 // [blocks][2][D]: of scale and post_w, of pre_w
};

// A call's kernels after its first may be launched while the one before still runs, and wait for
// its end themselves, behind their own start: bf16 M1003 K1511 N2051 behind its copies 29 us
// instead of 33, norms' training M2731 D1111 52 instead of 62.  Each one waits, be it as its
// last act, so that the end of a call's last kernel is the end of all of them.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// after: a kernel of the same call stands before this one in the stream
template <typename... P, typename... A>
cudaError_t launch_in_call(bool after, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                           unsigned cluster, A&&... args) {
  cudaLaunchAttribute at[2] = {};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st, cfg.attrs = at;
  if (cluster) {
    cudaLaunchAttribute& a = at[cfg.numAttrs++];
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = cluster, a.val.clusterDim.y = a.val.clusterDim.z = 1;
  }
  if (after) {
    cudaLaunchAttribute& a = at[cfg.numAttrs++];
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();   // it is returned here, not by the next call
  return e;
}

// f(x) and f'(x).  The products with 1 - s take x as it is at a border behind which they are 0 to
// fp32: they stay 0 instead of 0 times infinity.  Of a sigmoid s of x itself that is above 30,
// where s is 1, and below -88, where s is 0 (it is cut below fp32's normal values, from -87.3 on;
// at -60 it is 8.8e-27 and counts).  Gelu's sigmoid is one of a cube, and 0 or 1 behind +-30.
template <int ACT> __device__ __forceinline__ float act_of(float x) {
  if constexpr (ACT == DR_ACT_RELU) return x > 0.f ? x : x == x ? 0.f : x;
  if constexpr (ACT == DR_ACT_SILU) return x * sigmoid_f(x);
  if constexpr (ACT == DR_ACT_SIGMOID) return sigmoid_f(x);
  if constexpr (ACT == DR_ACT_GELU_TANH) {
    const float c = fminf(fmaxf(x, -30.f), 30.f);
    const float s = sigmoid_f(c * fmaf(0.07135481283f, c * c, 1.595769122f));   // 0.5 + 0.5 tanh(u) = sigmoid(2 u)
    return x * s;
  }
  return x;
}

template <int ACT> __device__ __forceinline__ float act_of(float x, float& slope) {
  const float c = fminf(fmaxf(x, ACT == DR_ACT_SILU ? -88.f : -30.f), 30.f);
  if constexpr (ACT == DR_ACT_RELU) {
    slope = x > 0.f ? 1.f : 0.f;
    return x > 0.f ? x : x == x ? 0.f : x;
  }
  if constexpr (ACT == DR_ACT_SILU) {
    const float s = sigmoid_f(x);
    slope = s * fmaf(c, 1.f - s, 1.f);
    return x * s;
  }
  if constexpr (ACT == DR_ACT_SIGMOID) {
    const float s = sigmoid_f(x);
    slope = s * (1.f - s);
    return s;
  }
  if constexpr (ACT == DR_ACT_GELU_TANH) {
    const float cc = c * c;
    const float s = sigmoid_f(c * fmaf(0.07135481283f, cc, 1.595769122f));
    slope = fmaf(c * s * (1.f - s), fmaf(0.21406443849f, cc, 1.595769122f), s);
    slope = x == x ? slope : x;
    return x * s;
  }
  slope = 1.f;
  return x;
}

}  // namespace dr
