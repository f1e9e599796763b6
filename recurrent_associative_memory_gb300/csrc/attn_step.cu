// attn_step.cu — window attention for one token per sequence over the ring cache,
// and the ring's layout from a prompt.
//
// Position p lives in slot p (p < n_sink) or n_sink + (p - n_sink) mod window, so
// what position p sees is exactly the slots 0 .. min(p, n_sink + window - 1): no
// masks, and no slot that was never written is read.  Bandwidth-bound: both caches
// are read once, 4 d bytes (bf16) per slot for 4 G d multiply-adds.
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ long long slot_of(int p, int n_sink, int window) {
  return p < n_sink ? p : n_sink + (p - n_sink) % window;
}

// One CTA per (sequence, key/value head, block of GB query heads, piece of the
// slots).  D / 8 lanes hold a slot's row, 8 channels each, so a warp takes 256 / D
// slots at once, with a running maximum and sum of its own.
template <int D, int GB, typename T>
__global__ void __launch_bounds__(kThreads) attn_step_simt_kernel(AttnStepArgs a) {
  constexpr int LK = D / 8, KPW = 32 / LK, U = 4;
  __shared__ float s_o[kWarps][GB][D], s_m[kWarps][GB], s_l[kWarps][GB];
  const int nb = (a.G + GB - 1) / GB;
  const int piece = blockIdx.x % a.n_piece;
  const int gb = (blockIdx.x / a.n_piece) % nb;
  const int hk = (blockIdx.x / a.n_piece / nb) % a.Hkv, b = blockIdx.x / a.n_piece / nb / a.Hkv;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sub = lane / LK, c0 = 8 * (lane % LK);
  const int h0 = hk * a.G + gb * GB, nh = min(GB, a.G - gb * GB);
  const int pos = a.pos[b];
  const int C = a.n_sink + a.window;
  const int n = pos < 0 ? 0 : min(pos, C - 1) + 1;
  const int per = (n + a.n_piece - 1) / a.n_piece;
  const int begin = min(n, piece * per), end = min(n, begin + per);

  T* kc = static_cast<T*>(a.kc) + ((long long)b * a.Hkv + hk) * C * D;
  T* vc = static_cast<T*>(a.vc) + ((long long)b * a.Hkv + hk) * C * D;
  if (n > 0) {   // the new token, written by the CTAs that read its slot
    const long long s = slot_of(pos, a.n_sink, a.window);
    if (s >= begin && s < end && threadIdx.x < D) {
      kc[s * D + threadIdx.x] = static_cast<const T*>(a.k)[((long long)b * a.Hkv + hk) * D + threadIdx.x];
      vc[s * D + threadIdx.x] = static_cast<const T*>(a.v)[((long long)b * a.Hkv + hk) * D + threadIdx.x];
    }
  }
  __syncthreads();

  float q[GB][8], o[GB][8], m[GB], l[GB];
#pragma unroll
  for (int g = 0; g < GB; ++g) {
    load8<T, true>(static_cast<const T*>(a.q) + ((long long)b * a.H + h0 + g) * D + c0, g < nh ? 8 : 0, q[g]);
#pragma unroll
    for (int c = 0; c < 8; ++c) q[g][c] *= a.scale * 1.4426950408889634f, o[g][c] = 0.f;
    m[g] = -INFINITY, l[g] = 0.f;
  }
  for (int j0 = begin + warp * KPW * U; j0 < end; j0 += kWarps * KPW * U) {
    float kf[U][8], s[U][GB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * KPW + sub;
      load8<T, true>(kc + (long long)j * D + c0, j < end ? 8 : 0, kf[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) x += q[g][c] * kf[u][c];
#pragma unroll
        for (int w = LK / 2; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        s[u][g] = j0 + u * KPW + sub < end ? x : -INFINITY;
      }
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      float mx = m[g];
#pragma unroll
      for (int u = 0; u < U; ++u) mx = fmaxf(mx, s[u][g]);
      const float at = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(m[g] - at);
      m[g] = mx;
      l[g] *= f;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[g][c] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u][g] = ex2(s[u][g] - at);
        l[g] += s[u][g];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * KPW + sub;
      float vf[8];
      load8<T, true>(vc + (long long)j * D + c0, j < end ? 8 : 0, vf);
#pragma unroll
      for (int g = 0; g < GB; ++g)
#pragma unroll
        for (int c = 0; c < 8; ++c) o[g][c] += s[u][g] * vf[c];
    }
  }
  // join the warp's KPW parts, then the warps'
#pragma unroll
  for (int g = 0; g < GB; ++g) {
#pragma unroll
    for (int w = 16; w >= LK; w >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[g], w);
      const float mx = fmaxf(m[g], mo), at = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(m[g] - at), fo = ex2(mo - at);
      l[g] = l[g] * f + __shfl_xor_sync(0xffffffffu, l[g], w) * fo;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[g][c] = o[g][c] * f + __shfl_xor_sync(0xffffffffu, o[g][c], w) * fo;
      m[g] = mx;
    }
    if (sub == 0) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_o[warp][g][c0 + c] = o[g][c];
      if (c0 == 0) s_m[warp][g] = m[g], s_l[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nh * D; e += kThreads) {
    const int g = e / D, c = e % D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][g]);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][g] - at);
      sum += s_l[w][g] * f;
      acc += s_o[w][g][c] * f;
    }
    const long long row = (long long)b * a.H + h0 + g;
    if (a.n_piece == 1) {
      static_cast<T*>(a.out)[row * D + c] = from_f<T>(sum != 0.f ? acc / sum : 0.f);
    } else {
      float* p = a.part + (row * a.n_piece + piece) * (D + 2);
      p[c] = acc;
      if (c == 0) p[D] = mx, p[D + 1] = sum;
    }
  }
}

// out = sum over the pieces of o exp2(m - max) / sum of l exp2(m - max)
template <int D, typename T>
__global__ void __launch_bounds__(D) attn_step_join_kernel(AttnStepArgs a) {
  const float* p = a.part + (long long)blockIdx.x * a.n_piece * (D + 2);
  float mx = -INFINITY;
  for (int i = 0; i < a.n_piece; ++i) mx = fmaxf(mx, p[i * (D + 2) + D]);
  const float at = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, acc = 0.f;
  for (int i = 0; i < a.n_piece; ++i) {
    const float f = ex2(p[i * (D + 2) + D] - at);
    sum += p[i * (D + 2) + D + 1] * f;
    acc += p[i * (D + 2) + threadIdx.x] * f;
  }
  static_cast<T*>(a.out)[(long long)blockIdx.x * D + threadIdx.x] = from_f<T>(sum != 0.f ? acc / sum : 0.f);
}

template <int D, int GB, typename T>
cudaError_t step(const AttnStepArgs& a, cudaStream_t st) {
  const long long grid = (long long)a.B * a.Hkv * ((a.G + GB - 1) / GB) * a.n_piece;
  attn_step_simt_kernel<D, GB, T><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.n_piece == 1) return e;
  attn_step_join_kernel<D, T><<<static_cast<unsigned>(a.B * a.H), D, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D, typename T>
cudaError_t step_heads(const AttnStepArgs& a, cudaStream_t st) {
  if (a.G == 1) return step<D, 1, T>(a, st);
  if (a.G == 2) return step<D, 2, T>(a, st);
  return step<D, 4, T>(a, st);
}

// Each block copies 8-channel pieces of one slot row per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_fill_kernel(AttnArgs a, T* kc, T* vc) {
  const int C = a.n_sink + a.window, per = a.d / 8;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = e / per;   // [B,Hkv,C]
  if (row >= (long long)a.B * a.Hkv * C) return;
  const int slot = row % C, hk = (row / C) % a.Hkv, b = row / C / a.Hkv, c = 8 * (e % per);
  const int len = real_len(a.lens, b, a.S);
  int p = slot;                   // the last position before len that lives in this slot
  if (slot >= a.n_sink) {
    const int r = slot - a.n_sink, last = len - 1 - a.n_sink;   // ring index of the last token
    if (last < r) return;
    p = a.n_sink + r + (last - r) / a.window * a.window;
  }
  if (p >= len) return;
  float f[8];
  load8<T, true>(static_cast<const T*>(a.k) + b * a.k_sb + p * a.k_st + hk * a.k_sh + c, 8, f);
  store8<T, true>(kc + row * a.d + c, 8, f);
  load8<T, true>(static_cast<const T*>(a.v) + b * a.v_sb + p * a.v_st + hk * a.v_sh + c, 8, f);
  store8<T, true>(vc + row * a.d + c, 8, f);
}

}  // namespace

// Pieces along the slots: as many as fill two CTAs on every SM, of 128 slots at least.
int attn_step_pieces(const AttnStepArgs& a, int sms) {
  const long long rows = (long long)a.B * a.Hkv * ((a.G + 3) / 4);
  const long long most = ((long long)a.n_sink + a.window + 127) / 128;
  const long long want = 2LL * sms / rows;
  return static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
}

cudaError_t launch_attn_step(const AttnStepArgs& a, int dtype, cudaStream_t st) {
  if (dtype == DR_FP32) return a.d == 64 ? step_heads<64, float>(a, st) : step_heads<128, float>(a, st);
  return a.d == 64 ? step_heads<64, __nv_bfloat16>(a, st) : step_heads<128, __nv_bfloat16>(a, st);
}

cudaError_t launch_cache_fill(const AttnArgs& a, int dtype, void* kc, void* vc, cudaStream_t st) {
  const long long n = (long long)a.B * a.Hkv * (a.n_sink + a.window) * (a.d / 8);
  const unsigned grid = static_cast<unsigned>((n + kThreads - 1) / kThreads);
  if (dtype == DR_FP32)
    cache_fill_kernel<float><<<grid, kThreads, 0, st>>>(a, static_cast<float*>(kc), static_cast<float*>(vc));
  else
    cache_fill_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(
        a, static_cast<__nv_bfloat16*>(kc), static_cast<__nv_bfloat16*>(vc));
  return cudaGetLastError();
}

}  // namespace dr
