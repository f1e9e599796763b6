// linear_rows.cu — the matrix product for up to 8 rows in fp32, on the CUDA cores.
//
// So few rows are bound by the weights, which the tensor cores would need as pieces first: three
// times their bytes written and read again.  Here they go straight from memory through
// registers, four at a time, M multiply-adds each.  The sum over k is cut over the CTAs of a
// cluster, each of which holds its rows of x in shared memory; a CTA's warps, then the CTAs, add
// their parts up in order.
//   W [K,N]: a CTA takes 128 columns, a lane 4 of them, warp w the k with k mod 8 = w
//   W [N,K]: a CTA takes 32 columns, a warp 4 of them, a lane 4 of every 128 k
// K4096 N16384 (268 MB): one row 45 us, 5.9 TB/s, 8 rows 76 us, bound by its multiply-adds and
// their reads of x.
#include "linear_tc.cuh"

namespace dr {
namespace {

using lin::Epilogue;

constexpr int kWarps = 8, kThreads = 32 * kWarps;

struct Rows {
  const float* x;
  const float* w;
  long long x_s, w_s;
  int K, split;
};

__device__ __forceinline__ float4 load4(const float* p, int n) {   // n: how many there are
  if (n >= 4) return *reinterpret_cast<const float4*>(p);
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, 0.f);
}
__device__ __forceinline__ void fma4(float (&a)[4], float x, const float4& w) {
  a[0] = fmaf(x, w.x, a[0]), a[1] = fmaf(x, w.y, a[1]), a[2] = fmaf(x, w.z, a[2]), a[3] = fmaf(x, w.w, a[3]);
}

// MT: rows, W_T: the weight's order.  C's columns of a CTA: 128, or 32 where W_T.
template <int MT, bool W_T>
__global__ void __launch_bounds__(kThreads) linear_rows_kernel(Rows a, Epilogue e) {
  constexpr int NC = W_T ? 32 : 128;
  constexpr int kTile = 512;   // k that x is held for at once
  __shared__ __align__(16) float xs[MT][kTile];
  __shared__ float part[W_T ? 1 : kWarps][MT][NC];   // [0]: the CTA's, in the end
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = blockIdx.x % a.split, n0 = blockIdx.x / a.split * NC;
  // multiples of 128 k, so that no 4 of them are cut
  const int blocks = (a.K + 127) / 128;
  const int k0 = static_cast<int>((long long)blocks * rank / a.split) * 128;
  const int k1 = min(a.K, static_cast<int>((long long)blocks * (rank + 1) / a.split) * 128);
  float acc[MT][4] = {};
  for (int kt = k0; kt < k1; kt += kTile) {
    const int kn = min(kTile, k1 - kt);
    __syncthreads();
    for (int i = threadIdx.x; i < MT * kTile; i += kThreads) {
      const int m = i / kTile, k = i % kTile;
      xs[m][k] = m < e.M && k < kn ? a.x[m * a.x_s + kt + k] : 0.f;
    }
    __syncthreads();
    if constexpr (W_T) {   // acc[m][c]: column n0 + 4 warp + c
      const int n = n0 + 4 * warp;
      for (int k = 4 * lane; k < kn; k += 128) {
        float4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = n + c < e.N ? load4(a.w + (n + c) * a.w_s + kt + k, kn - k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float4 x = *reinterpret_cast<const float4*>(&xs[m][k]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[m][c] = fmaf(x.x, w[c].x, fmaf(x.y, w[c].y, fmaf(x.z, w[c].z, fmaf(x.w, w[c].w, acc[m][c]))));
        }
      }
    } else {               // acc[m][c]: column n0 + 4 lane + c
      const int n = n0 + 4 * lane, left = e.N - n;
      constexpr int U = 8;   // loads on their way
      for (int k = warp; k < kn; k += kWarps * U) {
        float4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          w[u] = k + kWarps * u < kn ? load4(a.w + (kt + k + kWarps * u) * a.w_s + n, left) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int m = 0; m < MT; ++m) fma4(acc[m], xs[m][(k + kWarps * u) % kTile], w[u]);
      }
    }
  }
  if constexpr (W_T) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float s = warp_sum(acc[m][c]);
        if (lane == 0) part[0][m][4 * warp + c] = s;
      }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) part[warp][m][4 * lane + c] = acc[m][c];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * NC; i += kThreads) {
      const int m = i / NC, c = i % NC;
      float s = part[0][m][c];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += part[w][m][c];
      part[0][m][c] = s;
    }
  }
  lin::cluster_sync();   // every part is there
  for (int i = rank * kThreads + threadIdx.x; i < MT * NC; i += a.split * kThreads) {
    const int m = i / NC, c = i % NC, n = n0 + c;
    if (m >= e.M || n >= e.N) continue;
    float v = 0.f;
    const uint32_t at = lin::smem_u32(&part[0][m][c]);
    for (int r = 0; r < a.split; ++r) {
      float u;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(lin::map_rank(at, r)) : "memory");
      v += u;
    }
    float x[1] = {v + (e.bias ? static_cast<const float*>(e.bias)[n] : 0.f)}, s[1];
    lin::act_all(e.act, e.slope != nullptr, x, s);
    const long long to = m * (long long)e.N + n;
    if (e.slope) static_cast<float*>(e.slope)[to] = s[0];
    if (e.res) x[0] += static_cast<const float*>(e.res)[m * e.r_m + n];
    static_cast<float*>(e.C)[to] = x[0];
  }
  lin::cluster_sync();   // nobody reads this CTA's part any more
}

template <int MT, bool W_T> cudaError_t go(const Rows& a, const Epilogue& e, long long tiles, cudaStream_t st) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.split, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, linear_rows_kernel<MT, W_T>, a, e);
  if (err != cudaSuccess) cudaGetLastError();   // it is returned here, not by the next call
  return err;
}

}  // namespace

// Up to 8 rows whose weight has rows on 16 bytes.  us, with 4 of events, here and as pieces:
//   K2048 N2048   1 row 12, 8 rows 16; 16 rows 25, as [N,K] 39;  pieces 22.5 for any of them
//   K4096 N16384  1 row 45, 8 rows 76; 16 rows 125, as [N,K] 268;  pieces 176
//   K8192 N1024   8 rows 33; 16 rows 52, as [N,K] 59;  pieces 43
// So 16 rows would gain for a wide weight as [K,N] (125 for 176) and lose for narrower ones and as
// [N,K]: 8 is where every size and order gains.
bool linear_rows_supported(const LinearArgs& a, int dtype) {
  return dtype == DR_FP32 && a.M <= 8 && a.w_s % 4 == 0 && a.w_s >= 0;
}

cudaError_t launch_linear_rows(const LinearArgs& a, int sms, cudaStream_t st) {
  const long long tiles = (a.N + (a.w_t ? 31LL : 127LL)) / (a.w_t ? 32 : 128);
  // enough CTAs for two to an SM, each with 128 k at least
  int split = 1;
  while (split < 8 && tiles * split < 2LL * sms && 128LL * 2 * split <= a.K) split *= 2;
  const Rows r{static_cast<const float*>(a.x), static_cast<const float*>(a.w), a.x_s, a.w_s, a.K, split};
  const Epilogue e{a.y, a.bias, a.res, a.slope, a.M, a.N, a.act, lin::kFirst, a.r_s};
  auto order = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    return a.w_t ? go<MT, true>(r, e, tiles, st) : go<MT, false>(r, e, tiles, st);
  };
  if (a.M == 1) return order(std::integral_constant<int, 1>{});
  if (a.M <= 4) return order(std::integral_constant<int, 4>{});
  return order(std::integral_constant<int, 8>{});
}

}  // namespace dr
