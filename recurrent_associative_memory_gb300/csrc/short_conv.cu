// short_conv.cu — short causal convolution, one filter of K taps per channel, with
// bias and SiLU: forward, backward, one token.
//
// Bandwidth-bound: 2 K multiply-adds per value read and written.  A thread owns CH = 2
// neighbouring channels (a warp's row is 128 bytes of bf16) and walks a run of kRun
// tokens with the last K - 1 inputs in registers; kAhead tokens are loaded, as they are,
// while the kAhead before them are computed, so that enough bytes are under way.
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 64;          // tokens a thread walks
constexpr int kAhead = 16;        // tokens whose loads go together (backward: half)
constexpr int kLanes = 32;        // threads along the channels of a CTA (backward)
constexpr int kRows = kThreads / kLanes;

// CH neighbouring channels as they lie in memory
template <typename T, int CH> struct alignas(sizeof(T) * CH) Raw { T v[CH]; };
template <typename T, int CH>
__device__ __forceinline__ Raw<T, CH> raw_ch(const T* p) {
  if constexpr (CH == 2 && sizeof(T) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return *reinterpret_cast<const Raw<T, CH>*>(&u);
  } else if constexpr (CH == 2) {
    const float2 u = *reinterpret_cast<const float2*>(p);
    return {u.x, u.y};
  } else {
    return {*p};
  }
}

// CH neighbouring channels: one access (CH = 2) or a single value (CH = 1)
template <typename T, int CH>
__device__ __forceinline__ void load_ch(const T* p, bool in, float (&f)[CH]) {
  if constexpr (CH == 1) {
    f[0] = in ? to_f<T>(*p) : 0.f;
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t v = in ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xFFFF0000u);
  } else {
    const float2 v = in ? *reinterpret_cast<const float2*>(p) : make_float2(0.f, 0.f);
    f[0] = v.x, f[1] = v.y;
  }
}
template <typename T, int CH>
__device__ __forceinline__ void store_ch(T* p, const float (&f)[CH]) {
  if constexpr (CH == 1) {
    *p = from_f<T>(f[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
  } else {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  }
}

// input t of the sequence, t >= -(K - 1): of the state before the first token
template <int K, typename T, int CH>
__device__ __forceinline__ void load_in(const ConvArgs& a, int b, int t, int c, bool in, float (&f)[CH]) {
  if (t >= 0)
    load_ch<T, CH>(static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + c, in, f);
  else
    load_ch<T, CH>(static_cast<const T*>(a.s0) + ((long long)b * (K - 1) + t + K - 1) * a.D + c, in && a.s0, f);
}

template <int K, int CH>
__device__ __forceinline__ void load_filter(const ConvArgs& a, int c, float (&w)[K][CH], float (&bias)[CH]) {
#pragma unroll
  for (int v = 0; v < CH; ++v) {
    bias[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][v] = a.w[(long long)(c + v) * K + j];
  }
}

// u of the token whose input is x[K - 1]
template <int K, int CH>
__device__ __forceinline__ float filtered(const float (&w)[K][CH], const float (&bias)[CH],
                                          const float (&x)[K][CH], int v) {
  float u = bias[v];
#pragma unroll
  for (int j = 0; j < K; ++j) u += w[j][v] * x[j][v];
  return u;
}

template <int K, typename T, int CH>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  const int groups = a.D / CH, runs = (a.T + kRun - 1) / kRun;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c = CH * (e % groups);
  const long long r = e / groups;
  if (r >= (long long)a.B * runs) return;
  const int b = r / runs, t0 = (r % runs) * kRun, last = min(t0 + kRun, a.T);
  const int len = real_len(a.lens, b, a.T), state0 = len - (K - 1);
  float w[K][CH], bias[CH], x[K][CH];
  load_filter<K, CH>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int t = t0 - (K - 1) + j;
    load_in<K, T, CH>(a, b, t, c, true, x[j]);
    if (a.s1 && t < 0 && t >= state0)   // a short sequence keeps some of its initial state
      store_ch<T, CH>(static_cast<T*>(a.s1) + ((long long)b * (K - 1) + t - state0) * a.D + c, x[j]);
  }
  const T* xp = static_cast<const T*>(a.x) + b * a.x_sb + t0 * a.x_st + c;
  T* y = static_cast<T*>(a.y) + ((long long)b * a.T + t0) * a.D + c;
  Raw<T, CH> next[kAhead];
  auto fetch = [&](int tb) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (tb + i < last) next[i] = raw_ch<T, CH>(xp);
      xp += a.x_st;
    }
  };
  fetch(t0);
  for (int tb = t0; tb < last; tb += kAhead) {
    Raw<T, CH> now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
    if (tb + kAhead < last) fetch(tb + kAhead);
    const bool plain = tb + kAhead <= min(last, len) && (!a.s1 || tb + kAhead <= state0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = tb + i;
      if (!plain && t >= last) break;
      float u[CH];
#pragma unroll
      for (int v = 0; v < CH; ++v) {
        x[K - 1][v] = to_f<T>(now[i].v[v]);
        u[v] = filtered<K, CH>(w, bias, x, v);
        if (a.silu) u[v] *= sigmoid_f(u[v]);
        if (!plain && t >= len) u[v] = 0.f;
      }
      store_ch<T, CH>(y, u);
      y += a.D;
      if (!plain && a.s1 && t >= state0 && t < len)
        store_ch<T, CH>(static_cast<T*>(a.s1) + ((long long)b * (K - 1) + t - state0) * a.D + c, x[K - 1]);
#pragma unroll
      for (int v = 0; v < CH; ++v)
#pragma unroll
        for (int j = 0; j < K - 1; ++j) x[j][v] = x[j + 1][v];
    }
  }
}

// Backward.  With du = dy (silu'(u)):  dx_t = sum_j w_j du_{t+K-1-j} (+ d_final),
// d weight_j = sum_t du_t x_{t-K+1+j}.  A thread walks tokens t0 .. t0 + kRun + K - 2,
// forming du_t on the way (its last K - 1 tokens only for dx), and owns dx of
// t0 .. t0 + kRun - 1 and the weights' sums over its own tokens.  The first run also
// owns dx of the initial state (t < 0).  A CTA is 32 threads along the channels x 8
// runs; the runs' sums meet in shared memory and leave as one part per CTA.
template <int K, typename T, int CH>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvArgs a) {
  __shared__ float s_sum[kRows][K + 1][kLanes * CH];
  const int cgs = (a.D + CH * kLanes - 1) / (CH * kLanes);
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int c0 = (blockIdx.x % cgs) * CH * kLanes, c = c0 + CH * lane;
  const int blocks = (a.T + kRun * kRows - 1) / (kRun * kRows);
  const int part = blockIdx.x / cgs, b = part / blocks, t0 = (part % blocks) * kRun * kRows + row * kRun;
  const int len = real_len(a.lens, b, a.T);
  float dw[K + 1][CH];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int v = 0; v < CH; ++v) dw[j][v] = 0.f;
  if (c < a.D && t0 < a.T) {
    float w[K][CH], bias[CH], x[K][CH], du[K][CH];
    load_filter<K, CH>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      load_in<K, T, CH>(a, b, t0 - (K - 1) + j, c, true, x[j]);
#pragma unroll
      for (int v = 0; v < CH; ++v) du[j][v] = 0.f;
    }
    const int first = t0 == 0 ? -(K - 1) : t0, last = min(t0 + kRun, a.T);   // own dx rows
    constexpr int A = kAhead / 2;
    const T* xp = static_cast<const T*>(a.x) + b * a.x_sb + t0 * a.x_st + c;
    const T* gp = static_cast<const T*>(a.d_y) + ((long long)b * a.T + t0) * a.D + c;
    T* dx = static_cast<T*>(a.dx) + ((long long)b * a.T + t0 - (K - 1)) * a.D + c;   // of the row that is complete
    const int loads = min(len, last + K - 1);   // du is 0 from len on
    Raw<T, CH> xn[A], gn[A];
    auto fetch = [&](int tb) {
#pragma unroll
      for (int i = 0; i < A; ++i) {
        if (tb + i < loads) xn[i] = raw_ch<T, CH>(xp), gn[i] = raw_ch<T, CH>(gp);
        xp += a.x_st, gp += a.D;
      }
    };
    fetch(t0);
    for (int tb = t0; tb < last + K - 1; tb += A) {
      Raw<T, CH> xr[A], gr[A];
#pragma unroll
      for (int i = 0; i < A; ++i) xr[i] = xn[i], gr[i] = gn[i];
      if (tb + A < last + K - 1) fetch(tb + A);
      // every token real, within the run, behind its first rows, before the final state's
      const bool plain = tb + A <= min(last, len) && tb - (K - 1) >= t0 && (!a.d_s1 || tb + A <= len - (K - 1));
#pragma unroll
      for (int i = 0; i < A; ++i) {
        const int t = tb + i;
        if (!plain && t >= last + K - 1) break;
#pragma unroll
        for (int v = 0; v < CH; ++v) {
          const bool in = plain || t < loads;
          x[K - 1][v] = in ? to_f<T>(xr[i].v[v]) : 0.f;
          float g = in ? to_f<T>(gr[i].v[v]) : 0.f;
          if (a.silu) {
            const float u = filtered<K, CH>(w, bias, x, v), s = sigmoid_f(u);
            g *= s * (1.f + u * (1.f - s));
          }
          du[K - 1][v] = g;
          if (plain || t < last) {
            dw[K][v] += g;
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][v] += g * x[j][v];
          }
        }
        // du[j] holds du_{t-K+1+j}: row t-K+1 is complete
        const int r = t - (K - 1);
        if (plain || r >= first) {
          float o[CH];
#pragma unroll
          for (int v = 0; v < CH; ++v) {
            o[v] = 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) o[v] += w[K - 1 - j][v] * du[j][v];
          }
          const int f = r - (len - (K - 1));   // its place in the final state
          if (!plain && a.d_s1 && f >= 0 && f < K - 1) {
            float g[CH];
            load_ch<T, CH>(static_cast<const T*>(a.d_s1) + ((long long)b * (K - 1) + f) * a.D + c, true, g);
#pragma unroll
            for (int v = 0; v < CH; ++v) o[v] += g[v];
          }
          if (plain || r >= 0)
            store_ch<T, CH>(dx, o);
          else if (a.d_s0)
            store_ch<T, CH>(static_cast<T*>(a.d_s0) + ((long long)b * (K - 1) + r + K - 1) * a.D + c, o);
        }
        dx += a.D;
#pragma unroll
        for (int v = 0; v < CH; ++v)
#pragma unroll
          for (int j = 0; j < K - 1; ++j) x[j][v] = x[j + 1][v], du[j][v] = du[j + 1][v];
      }
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int v = 0; v < CH; ++v) s_sum[row][j][CH * lane + v] = dw[j][v];
  __syncthreads();
  for (int e = threadIdx.x; e < (K + 1) * CH * kLanes; e += kThreads) {
    const int j = e / (CH * kLanes), i = e % (CH * kLanes);
    if (c0 + i >= a.D) continue;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) s += s_sum[r][j][i];
    a.part[((long long)part * (K + 1) + j) * a.D + c0 + i] = s;
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

template <int K, typename T, int CH>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a) {
  const int groups = a.D / CH;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c = CH * (e % groups);
  const int b = e / groups;
  if (b >= a.B) return;
  float w[K][CH], bias[CH], x[K][CH], u[CH];
#pragma unroll
  for (int j = 0; j < K; ++j) load_in<K, T, CH>(a, b, j - (K - 1), c, true, x[j]);
  load_filter<K, CH>(a, c, w, bias);
#pragma unroll
  for (int v = 0; v < CH; ++v) {
    u[v] = filtered<K, CH>(w, bias, x, v);
    if (a.silu) u[v] *= sigmoid_f(u[v]);
  }
  store_ch<T, CH>(static_cast<T*>(a.y) + (long long)b * a.D + c, u);
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    store_ch<T, CH>(static_cast<T*>(a.s1) + ((long long)b * (K - 1) + j) * a.D + c, x[j + 1]);
}

unsigned blocks(long long n) { return static_cast<unsigned>((n + kThreads - 1) / kThreads); }

int bwd_parts(const ConvArgs& a) { return a.B * ((a.T + kRun * kRows - 1) / (kRun * kRows)); }

template <int K, typename T, int CH>
cudaError_t fwd(const ConvArgs& a, cudaStream_t st) {
  const long long n = (long long)a.B * ((a.T + kRun - 1) / kRun) * (a.D / CH);
  conv_fwd_kernel<K, T, CH><<<blocks(n), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int K, typename T, int CH>
cudaError_t bwd(const ConvArgs& a, float* dw, float* db, cudaStream_t st) {
  const int parts = bwd_parts(a), cgs = (a.D + CH * kLanes - 1) / (CH * kLanes);
  conv_bwd_kernel<K, T, CH><<<static_cast<unsigned>((long long)parts * cgs), kThreads, 0, st>>>(a);
  conv_sum_kernel<K><<<(a.D * (K + 1) + 31) / 32, kThreads, 0, st>>>(a, parts, dw, db);
  return cudaGetLastError();
}

template <int K, typename T, int CH>
cudaError_t step(const ConvArgs& a, cudaStream_t st) {
  conv_step_kernel<K, T, CH><<<blocks((long long)a.B * (a.D / CH)), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// Two channels per thread where every row starts on a pair.
bool pairs_ok(const ConvArgs& a, int dtype) {
  const uintptr_t mask = dtype == DR_FP32 ? 7 : 3;
  auto al = [&](const void* p) { return (reinterpret_cast<uintptr_t>(p) & mask) == 0; };
  return a.D % 2 == 0 && a.x_st % 2 == 0 && a.x_sb % 2 == 0 && al(a.x) && al(a.s0) && al(a.y) && al(a.s1) &&
         al(a.d_y) && al(a.d_s1) && al(a.dx) && al(a.d_s0);
}

}  // namespace

#define DR_CONV_CASE(K_, CALL)                                                    \
  case K_:                                                                        \
    if (dtype == DR_FP32)                                                         \
      return pairs_ok(a, dtype) ? CALL(K_, float, 2) : CALL(K_, float, 1);        \
    return pairs_ok(a, dtype) ? CALL(K_, __nv_bfloat16, 2) : CALL(K_, __nv_bfloat16, 1);
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
