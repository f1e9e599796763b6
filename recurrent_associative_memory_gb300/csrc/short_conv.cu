// short_conv.cu — short causal convolution, one filter of K taps per channel, with
// bias and SiLU: forward, backward, one token.
//
// Bandwidth-bound: 2 K multiply-adds per value read and written.  A thread owns 8
// neighbouring channels (one 16-byte access of bf16) and walks a run of kRun tokens
// with the last K - 1 inputs in registers, so a value is read once plus K - 1 of
// every kRun at the runs' borders.
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 32;          // tokens a thread walks
constexpr int kLanes = 32;        // channel groups of 8 per CTA (backward)
constexpr int kRows = kThreads / kLanes;

// input t of the sequence, t >= -(K - 1): of the state before the first token
template <int K, typename T, bool VEC>
__device__ __forceinline__ void load_in(const ConvArgs& a, int b, int t, int c, int n, float (&f)[8]) {
  if (t >= 0)
    load8<T, VEC>(static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + c, n, f);
  else
    load8<T, VEC>(static_cast<const T*>(a.s0) + ((long long)b * (K - 1) + t + K - 1) * a.D + c,
                  a.s0 ? n : 0, f);
}

template <int K>
__device__ __forceinline__ void load_filter(const ConvArgs& a, int c, int n, float (&w)[K][8],
                                            float (&bias)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = a.bias && i < n ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = i < n ? a.w[(long long)(c + i) * K + j] : 0.f;
  }
}

template <int K, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  const int groups = (a.D + 7) / 8, runs = (a.T + kRun - 1) / kRun;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c = 8 * (e % groups);
  const long long r = e / groups;
  if (r >= (long long)a.B * runs) return;
  const int b = r / runs, t0 = (r % runs) * kRun, n = min(8, a.D - c);
  const int len = real_len(a.lens, b, a.T);
  float w[K][8], bias[8], x[K][8];
  load_filter<K>(a, c, n, w, bias);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) load_in<K, T, VEC>(a, b, t0 - (K - 1) + j, c, n, x[j]);
  T* y = static_cast<T*>(a.y) + ((long long)b * a.T + t0) * a.D + c;
#pragma unroll 4
  for (int i = 0; i < kRun; ++i) {
    const int t = t0 + i;
    if (t >= a.T) break;
    load_in<K, T, VEC>(a, b, t, c, n, x[K - 1]);
    float u[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      u[v] = bias[v];
#pragma unroll
      for (int j = 0; j < K; ++j) u[v] += w[j][v] * x[j][v];
      if (a.silu) u[v] *= sigmoid_f(u[v]);
      if (t >= len) u[v] = 0.f;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) x[j][v] = x[j + 1][v];
    }
    store8<T, VEC>(y + (long long)i * a.D, n, u);
  }
}

// the last K - 1 inputs of each sequence; backward: its gradient for the initial state
template <int K, typename T>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(ConvArgs a) {
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (e >= (long long)a.B * (K - 1) * a.D) return;
  const int c = e % a.D, j = (e / a.D) % (K - 1), b = e / a.D / (K - 1);
  const int t = real_len(a.lens, b, a.T) - (K - 1) + j;
  T v = from_f<T>(0.f);
  if (t >= 0)
    v = static_cast<const T*>(a.x)[b * a.x_sb + t * a.x_st + c];
  else if (a.s0)
    v = static_cast<const T*>(a.s0)[((long long)b * (K - 1) + t + K - 1) * a.D + c];
  static_cast<T*>(a.s1)[e] = v;
}

// Backward.  With du = dy (silu'(u)):  dx_t = sum_j w_j du_{t+K-1-j} (+ d_final),
// d weight_j = sum_t du_t x_{t-K+1+j}.  A thread walks tokens t0 .. t0 + kRun + K - 2,
// forming du_t on the way (its last K - 1 tokens only for dx), and owns dx of
// t0 .. t0 + kRun - 1 and the weights' sums over its own tokens.  The first run also
// owns dx of the initial state (t < 0).  A CTA is 32 channel groups x 8 runs; the
// runs' sums meet in shared memory and leave as one part per CTA.
template <int K, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvArgs a) {
  __shared__ float s_sum[kRows][K + 1][kLanes * 8 + 8];
  const int cgs = (a.D + 8 * kLanes - 1) / (8 * kLanes);
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int c = (blockIdx.x % cgs) * 8 * kLanes + 8 * lane, n = min(8, a.D - c);
  const int blocks = (a.T + kRun * kRows - 1) / (kRun * kRows);
  const int part = blockIdx.x / cgs, b = part / blocks, t0 = (part % blocks) * kRun * kRows + row * kRun;
  const int len = real_len(a.lens, b, a.T);
  float dw[K + 1][8];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int v = 0; v < 8; ++v) dw[j][v] = 0.f;
  if (n > 0 && t0 < a.T) {
    float w[K][8], bias[8], x[K][8], du[K][8];
    load_filter<K>(a, c, n, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_in<K, T, VEC>(a, b, t0 - (K - 1) + j, c, n, x[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int v = 0; v < 8; ++v) du[j][v] = 0.f;
    const int first = t0 == 0 ? -(K - 1) : t0, last = min(t0 + kRun, a.T);   // own dx rows
    const T* gy = static_cast<const T*>(a.d_y) + (long long)b * a.T * a.D + c;
#pragma unroll 2
    for (int t = t0; t < last + K - 1; ++t) {
      if (t < a.T) {
        load_in<K, T, VEC>(a, b, t, c, n, x[K - 1]);
        float g[8];
        load8<T, VEC>(gy + (long long)t * a.D, t < len ? n : 0, g);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          if (a.silu) {
            float u = bias[v];
#pragma unroll
            for (int j = 0; j < K; ++j) u += w[j][v] * x[j][v];
            const float s = sigmoid_f(u);
            g[v] *= s * (1.f + u * (1.f - s));
          }
          du[K - 1][v] = g[v];
          if (t < last) {
            dw[K][v] += g[v];
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][v] += g[v] * x[j][v];
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) du[K - 1][v] = 0.f;
      }
      // du[j] holds du_{t-K+1+j}: row t-K+1 is complete
      const int r = t - (K - 1);
      if (r >= first) {
        float o[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          o[v] = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) o[v] += w[K - 1 - j][v] * du[j][v];
        }
        const int f = r - (len - (K - 1));   // its place in the final state
        if (a.d_s1 && f >= 0 && f < K - 1) {
          float g[8];
          load8<T, VEC>(static_cast<const T*>(a.d_s1) + ((long long)b * (K - 1) + f) * a.D + c, n, g);
#pragma unroll
          for (int v = 0; v < 8; ++v) o[v] += g[v];
        }
        if (r >= 0)
          store8<T, VEC>(static_cast<T*>(a.dx) + ((long long)b * a.T + r) * a.D + c, n, o);
        else if (a.d_s0)
          store8<T, VEC>(static_cast<T*>(a.d_s0) + ((long long)b * (K - 1) + r + K - 1) * a.D + c, n, o);
      }
#pragma unroll
      for (int v = 0; v < 8; ++v) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) x[j][v] = x[j + 1][v], du[j][v] = du[j + 1][v];
      }
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int v = 0; v < 8; ++v) s_sum[row][j][8 * lane + v] = dw[j][v];
  __syncthreads();
  for (int e = threadIdx.x; e < (K + 1) * 8 * kLanes; e += kThreads) {
    const int j = e / (8 * kLanes), i = e % (8 * kLanes), ch = (blockIdx.x % cgs) * 8 * kLanes + i;
    if (ch >= a.D) continue;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) s += s_sum[r][j][i];
    a.part[((long long)part * (K + 1) + j) * a.D + ch] = s;
  }
}

// the parts' sums, in their order: 8 threads per value, each every eighth part
template <int K>
__global__ void __launch_bounds__(kThreads) conv_sum_kernel(ConvArgs a, int parts, float* dw, float* db) {
  __shared__ float s[8][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + x;
  float v = 0.f;
  if (e < (K + 1) * a.D)
    for (int p = y; p < parts; p += 8) v += a.part[(long long)p * (K + 1) * a.D + e];
  s[y][x] = v;
  __syncthreads();
  if (y || e >= (K + 1) * a.D) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += s[i][x];
  const int j = e / a.D, c = e % a.D;
  if (j < K)
    dw[(long long)c * K + j] = v;
  else if (db)
    db[c] = v;
}

template <int K, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a) {
  const int groups = (a.D + 7) / 8;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c = 8 * (e % groups), n = min(8, a.D - c);
  const int b = e / groups;
  if (b >= a.B) return;
  float w[K][8], bias[8], x[K][8], u[8];
#pragma unroll
  for (int j = 0; j < K; ++j) load_in<K, T, VEC>(a, b, j - (K - 1), c, n, x[j]);
  load_filter<K>(a, c, n, w, bias);
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    u[v] = bias[v];
#pragma unroll
    for (int j = 0; j < K; ++j) u[v] += w[j][v] * x[j][v];
    if (a.silu) u[v] *= sigmoid_f(u[v]);
  }
  store8<T, VEC>(static_cast<T*>(a.y) + (long long)b * a.D + c, n, u);
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    store8<T, VEC>(static_cast<T*>(a.s1) + ((long long)b * (K - 1) + j) * a.D + c, n, x[j + 1]);
}

unsigned blocks(long long n) { return static_cast<unsigned>((n + kThreads - 1) / kThreads); }

int bwd_parts(const ConvArgs& a) { return a.B * ((a.T + kRun * kRows - 1) / (kRun * kRows)); }

template <int K, typename T, bool VEC>
cudaError_t fwd(const ConvArgs& a, cudaStream_t st) {
  conv_fwd_kernel<K, T, VEC><<<blocks((long long)a.B * ((a.T + kRun - 1) / kRun) * ((a.D + 7) / 8)), kThreads,
                               0, st>>>(a);
  if (a.s1) conv_state_kernel<K, T><<<blocks((long long)a.B * (K - 1) * a.D), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int K, typename T, bool VEC>
cudaError_t bwd(const ConvArgs& a, float* dw, float* db, cudaStream_t st) {
  const int parts = bwd_parts(a), cgs = (a.D + 8 * kLanes - 1) / (8 * kLanes);
  conv_bwd_kernel<K, T, VEC><<<static_cast<unsigned>((long long)parts * cgs), kThreads, 0, st>>>(a);
  conv_sum_kernel<K><<<(a.D * (K + 1) + 31) / 32, kThreads, 0, st>>>(a, parts, dw, db);
  return cudaGetLastError();
}

template <int K, typename T, bool VEC>
cudaError_t step(const ConvArgs& a, cudaStream_t st) {
  conv_step_kernel<K, T, VEC><<<blocks((long long)a.B * ((a.D + 7) / 8)), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool vec_ok(const ConvArgs& a, int dtype) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int v = dtype == DR_FP32 ? 4 : 8;
  return a.D % 8 == 0 && a.x_st % v == 0 && a.x_sb % v == 0 && al(a.x) && al(a.s0) && al(a.y) &&
         al(a.s1) && al(a.d_y) && al(a.d_s1) && al(a.dx) && al(a.d_s0);
}

}  // namespace

// 16-byte accesses where every row starts on 16 bytes, single values otherwise.
#define DR_CONV_CASE(K_, CALL)                                                          \
  case K_:                                                                              \
    if (dtype == DR_FP32)                                                               \
      return vec_ok(a, dtype) ? CALL(K_, float, true) : CALL(K_, float, false);         \
    return vec_ok(a, dtype) ? CALL(K_, __nv_bfloat16, true) : CALL(K_, __nv_bfloat16, false);
#define DR_CONV_DISPATCH(CALL) \
  switch (a.K) {               \
    DR_CONV_CASE(2, CALL)      \
    DR_CONV_CASE(3, CALL)      \
    DR_CONV_CASE(4, CALL)      \
  }                            \
  return cudaErrorInvalidValue;

cudaError_t launch_conv_fwd(const ConvArgs& a, int dtype, cudaStream_t st) {
#define DR_CALL(K_, T_, V_) (fwd<K_, T_, V_>(a, st))
  DR_CONV_DISPATCH(DR_CALL)
#undef DR_CALL
}

cudaError_t launch_conv_bwd(const ConvArgs& a, int dtype, float* dw, float* db, cudaStream_t st) {
#define DR_CALL(K_, T_, V_) (bwd<K_, T_, V_>(a, dw, db, st))
  DR_CONV_DISPATCH(DR_CALL)
#undef DR_CALL
}

cudaError_t launch_conv_step(const ConvArgs& a, int dtype, cudaStream_t st) {
#define DR_CALL(K_, T_, V_) (step<K_, T_, V_>(a, st))
  DR_CONV_DISPATCH(DR_CALL)
#undef DR_CALL
}

size_t conv_bwd_part_floats(const ConvArgs& a) { return (size_t)bwd_parts(a) * (a.K + 1) * a.D; }

}  // namespace dr
