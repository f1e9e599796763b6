// linear_simt.cu — the matrix product with its epilogue on the CUDA cores, and the gradient
// at the product that both of its backward products start from.
#include "block.cuh"

namespace dr {
namespace {

// C[m,n] = sum_k A(m,k) B(k,n), then the epilogue.  Element strides on either side, so that
// the forward product and both gradients are one kernel.
struct Gemm {
  const void* A;
  const void* B;
  void* C;
  const void* bias;
  const void* res;
  void* slope;
  int M, N, K;
  long long a_m, a_k, b_k, b_n, c_m, r_m;
  int act;
};

constexpr int kT = 64, kK = 16;

template <typename T, typename S>
__global__ void __launch_bounds__(256) gemm_simt_kernel(Gemm g) {
  __shared__ float sa[kK][kT + 4], sb[kK][kT + 4];
  const long long tiles_n = (g.N + kT - 1) / kT;
  const int m0 = static_cast<int>(blockIdx.x / tiles_n) * kT, n0 = static_cast<int>(blockIdx.x % tiles_n) * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const T* A = static_cast<const T*>(g.A);
  const T* B = static_cast<const T*>(g.B);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kK) {
    for (int e = threadIdx.x; e < kT * kK; e += 256) {
      int m, k;   // neighbours in memory to neighbouring threads
      if (g.a_k == 1) k = e % kK, m = e / kK;
      else m = e % kT, k = e / kT;
      sa[k][m] = m0 + m < g.M && k0 + k < g.K ? to_f(A[(m0 + m) * g.a_m + (k0 + k) * g.a_k]) : 0.f;
      int n;
      if (g.b_k == 1) k = e % kK, n = e / kK;
      else n = e % kT, k = e / kT;
      sb[k][n] = n0 + n < g.N && k0 + k < g.K ? to_f(B[(k0 + k) * g.b_k + (n0 + n) * g.b_n]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sa[k][ty * 4 + i], y[i] = sb[k][tx * 4 + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    if (m >= g.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= g.N) break;
      float v = acc[i][j], s = 1.f;
      if (g.bias) v += to_f(static_cast<const T*>(g.bias)[n]);
      switch (g.act) {
        case DR_ACT_RELU: v = act_of<DR_ACT_RELU>(v, s); break;
        case DR_ACT_SILU: v = act_of<DR_ACT_SILU>(v, s); break;
        case DR_ACT_GELU_TANH: v = act_of<DR_ACT_GELU_TANH>(v, s); break;
        case DR_ACT_SIGMOID: v = act_of<DR_ACT_SIGMOID>(v, s); break;
        default: break;
      }
      if (g.slope) static_cast<S*>(g.slope)[(long long)m * g.N + n] = static_cast<S>(s);
      if (g.res) v += to_f(static_cast<const T*>(g.res)[m * g.r_m + n]);
      static_cast<T*>(g.C)[m * g.c_m + n] = from_f<T>(v);
    }
  }
}

cudaError_t gemm(const Gemm& g, int dtype, cudaStream_t st) {
  const long long tiles = ((g.M + kT - 1LL) / kT) * ((g.N + kT - 1LL) / kT);
  if (dtype == DR_FP32) gemm_simt_kernel<float, float><<<static_cast<unsigned>(tiles), 256, 0, st>>>(g);
  else gemm_simt_kernel<__nv_bfloat16, __half><<<static_cast<unsigned>(tiles), 256, 0, st>>>(g);
  return cudaGetLastError();
}

// d = d_y * slope [M,N] and its columns' sums: a block takes kRows rows of 32 columns, and the
// parts [row blocks][N] are joined in order.
constexpr int kRows = 64;

template <typename T, typename S>
__global__ void __launch_bounds__(256) slope_kernel(const T* d_y, const S* slope, T* d, float* part, long long M, int N) {
  __shared__ float buf[8][32];
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, n = blockIdx.y * 32 + lane;
  float s = 0.f;
  for (int i = g; i < kRows; i += 8) {
    const long long m = (long long)blockIdx.x * kRows + i;
    if (m >= M || n >= N) break;
    float v = to_f(d_y[m * N + n]);
    if (slope) v *= static_cast<float>(slope[m * N + n]);
    if (d) d[m * N + n] = from_f<T>(v);
    s += v;
  }
  if (!part) return;
  buf[g][lane] = s;
  __syncthreads();
  if (g == 0 && n < N) {
    for (int i = 1; i < 8; ++i) s += buf[i][lane];
    part[(long long)blockIdx.x * N + n] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) join_bias_kernel(const float* part, int blocks, int N, T* db) {
  __shared__ float buf[8][32];
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, n = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (n < N)
    for (int b = g; b < blocks; b += 8) s += part[(long long)b * N + n];
  buf[g][lane] = s;
  __syncthreads();
  if (g == 0 && n < N) {
    for (int i = 1; i < 8; ++i) s += buf[i][lane];
    db[n] = from_f<T>(s);
  }
}

}  // namespace

cudaError_t launch_linear_fwd_simt(const LinearArgs& a, int dtype, cudaStream_t st) {
  Gemm g{a.x, a.w, a.y, a.bias, a.res, a.slope, a.M, a.N, a.K, a.x_s, 1, a.w_t ? 1 : a.w_s, a.w_t ? a.w_s : 1, a.N, a.r_s, a.act};
  return gemm(g, dtype, st);
}

// dx and dw from d [M,N]
cudaError_t launch_linear_bwd_simt(const LinearArgs& a, const void* d, int dtype, cudaStream_t st) {
  const long long w_k = a.w_t ? 1 : a.w_s, w_n = a.w_t ? a.w_s : 1;
  cudaError_t e = cudaSuccess;
  if (a.dx)
    e = gemm(Gemm{d, a.w, a.dx, nullptr, nullptr, nullptr, a.M, a.K, a.N, a.N, 1, w_n, w_k, a.K, 0, DR_ACT_NONE}, dtype, st);
  if (a.dw && e == cudaSuccess)
    e = a.w_t ? gemm(Gemm{d, a.x, a.dw, nullptr, nullptr, nullptr, a.N, a.K, a.M, 1, a.N, a.x_s, 1, a.K, 0, DR_ACT_NONE}, dtype, st)
              : gemm(Gemm{a.x, d, a.dw, nullptr, nullptr, nullptr, a.K, a.N, a.M, 1, a.x_s, a.N, 1, a.N, 0, DR_ACT_NONE}, dtype, st);
  return e;
}

// d = d_y * slope [M,N] (null: not kept) and the bias's gradient (null: not wanted), over
// part [linear_slope_blocks(M)][N]
int linear_slope_blocks(int M) { return static_cast<int>((M + (long long)kRows - 1) / kRows); }

cudaError_t launch_linear_slope(const LinearArgs& a, int dtype, void* d, float* part, cudaStream_t st) {
  const int blocks = linear_slope_blocks(a.M);
  const dim3 grid(blocks, (a.N + 31) / 32);
  if (dtype == DR_FP32)
    slope_kernel<float, float><<<grid, 256, 0, st>>>(static_cast<const float*>(a.d_y), static_cast<const float*>(a.slope),
                                                     static_cast<float*>(d), part, a.M, a.N);
  else
    slope_kernel<__nv_bfloat16, __half><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(a.d_y),
                                                              static_cast<const __half*>(a.slope),
                                                              static_cast<__nv_bfloat16*>(d), part, a.M, a.N);
  if (a.db) {
    if (dtype == DR_FP32) join_bias_kernel<<<(a.N + 31) / 32, 256, 0, st>>>(part, blocks, a.N, static_cast<float*>(a.db));
    else join_bias_kernel<<<(a.N + 31) / 32, 256, 0, st>>>(part, blocks, a.N, static_cast<__nv_bfloat16*>(a.db));
  }
  return cudaGetLastError();
}

}  // namespace dr
