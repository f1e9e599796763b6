// short_conv.cu — short causal convolution, one filter of K taps per channel, with
// bias and SiLU: forward, backward, one token.
//
// 2 K multiply-adds and two calls of the special units per value read and written: the
// bytes' 20 us and the instructions' 22 are about the same.  A thread owns CH = 2
// neighbouring channels (a warp's row is 128 bytes of bf16) and walks a run of kRun
// tokens with the last K - 1 inputs in registers; kAhead tokens are loaded, as they are,
// while the kAhead before them are computed, so that enough bytes are under way.
// Sums are fp32; outputs are rounded once.
//   B8 T2048 D2048 K4 bf16: forward 28 us (4.7 TB/s), backward 53 us (3.8 TB/s) and 4 of sums;
//   runs of 32 or 128 tokens cost 8 to 12 us more, 4 or 16 tokens ahead 18 to 60.  The run is as
//   long for few tokens: B1 D2048 forward and backward 12 and 18 us at T1024, 12 and 16 at T96.
#include <type_traits>

#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 64;          // tokens a thread walks
constexpr int kAhead = 8;         // tokens whose loads go together
constexpr int kLanes = 32;        // threads along the channels of a CTA (backward)
constexpr int kRows = kThreads / kLanes;

// CH neighbouring channels as they lie in memory: one access (CH = 2) or a single value
// (CH = 1).  In registers they are a pair of fp32, the second 0 where CH = 1.
template <typename T, int CH> struct Raw;
template <> struct Raw<__nv_bfloat16, 2> { uint32_t v; };
template <> struct Raw<__nv_bfloat16, 1> { uint16_t v; };
template <> struct Raw<float, 2> { f2 v; };
template <> struct Raw<float, 1> { float v; };

template <typename T, int CH>
__device__ __forceinline__ Raw<T, CH> raw_ch(const T* p) { return *reinterpret_cast<const Raw<T, CH>*>(p); }

__device__ __forceinline__ f2 pair_of(Raw<__nv_bfloat16, 2> r) {
  return pack2(__uint_as_float(r.v << 16), __uint_as_float(r.v & 0xFFFF0000u));
}
__device__ __forceinline__ f2 pair_of(Raw<__nv_bfloat16, 1> r) {
  return pack2(__uint_as_float((uint32_t)r.v << 16), 0.f);
}
__device__ __forceinline__ f2 pair_of(Raw<float, 2> r) { return r.v; }
__device__ __forceinline__ f2 pair_of(Raw<float, 1> r) { return pack2(r.v, 0.f); }

template <typename T, int CH>
__device__ __forceinline__ f2 load_ch(const T* p, bool in) {
  return in ? pair_of(raw_ch<T, CH>(p)) : 0ull;
}
template <typename T, int CH>
__device__ __forceinline__ void store_ch(T* p, f2 v) {
  float x, y;
  unpack2(v, x, y);
  if constexpr (CH == 1)
    *p = from_f<T>(x);
  else if constexpr (sizeof(T) == 2)
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
  else
    *reinterpret_cast<f2*>(p) = v;
}

// input t of the sequence, t >= -(K - 1): of the state before the first token
template <int K, typename T, int CH>
__device__ __forceinline__ f2 load_in(const ConvArgs& a, int b, int t, int c) {
  return t >= 0 ? load_ch<T, CH>(static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + c, true)
                : load_ch<T, CH>(static_cast<const T*>(a.s0) + ((long long)b * (K - 1) + t + K - 1) * a.D + c,
                                 a.s0 != nullptr);
}

template <int K, int CH>
__device__ __forceinline__ void load_filter(const ConvArgs& a, int c, f2 (&w)[K], f2& bias) {
  bias = pack2(a.bias ? a.bias[c] : 0.f, a.bias && CH == 2 ? a.bias[c + 1] : 0.f);
#pragma unroll
  for (int j = 0; j < K; ++j)
    w[j] = pack2(a.w[(long long)c * K + j], CH == 2 ? a.w[(long long)(c + 1) * K + j] : 0.f);
}

// u of the token whose input is x[K - 1]
template <int K>
__device__ __forceinline__ f2 filtered(const f2 (&w)[K], f2 bias, const f2 (&x)[K]) {
  f2 u = bias;
#pragma unroll
  for (int j = 0; j < K; ++j) u = fma2(w[j], x[j], u);
  return u;
}
__device__ __forceinline__ f2 sigmoid2(f2 u) {
  float x, y;
  unpack2(u, x, y);
  return pack2(sigmoid_f(x), sigmoid_f(y));
}

template <int K, typename T, int CH>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) conv_fwd_kernel(ConvArgs a) {
  const int groups = a.D / CH, runs = (a.T + kRun - 1) / kRun;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  long long r, rb;
  const int c = CH * div_mod(e, groups, r);
  const int t0 = div_mod(r, runs, rb) * kRun, last = min(t0 + kRun, a.T);
  if (rb >= a.B) return;
  const int b = rb;
  const int len = real_len(a.lens, b, a.T);
  f2 w[K], bias, x[K];
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
  load_filter<K, CH>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    x[j] = load_in<K, T, CH>(a, b, t0 - (K - 1) + j, c);
  }
  for (int tb = t0; tb < last; tb += kAhead) {
    Raw<T, CH> now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
    if (tb + kAhead < last) fetch(tb + kAhead);
    auto walk = [&](auto is_plain) {
      constexpr bool plain = decltype(is_plain)::value;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = tb + i;
        if (!plain && t >= last) break;
        x[K - 1] = pair_of(now[i]);
        f2 u = filtered<K>(w, bias, x);
        if (a.silu) u = mul2(u, sigmoid2(u));
        if (!plain && t >= len) u = 0;
        store_ch<T, CH>(y, u);
        y += a.D;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) x[j] = x[j + 1];
      }
    };
    if (tb + kAhead <= min(last, len))   // every token real
      walk(std::true_type());
    else
      walk(std::false_type());
  }
  // The final state, by the thread that alone reads the initial one: they may be one buffer.
  // Row j of it is input len - (K - 1) + j, in a short sequence a row of the initial state at
  // or behind j.
  if (t0 == 0 && a.s1) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      store_ch<T, CH>(static_cast<T*>(a.s1) + ((long long)b * (K - 1) + j) * a.D + c,
                      load_in<K, T, CH>(a, b, len - (K - 1) + j, c));
  }
}

// Backward.  With du = dy (silu'(u)):  dx_t = sum_j w_j du_{t+K-1-j} (+ d_final),
// d weight_j = sum_t du_t x_{t-K+1+j}.  A thread walks tokens t0 .. t0 + kRun + K - 2,
// forming du_t on the way (its last K - 1 tokens only for dx), and owns dx of
// t0 .. t0 + kRun - 1 and the weights' sums over its own tokens.  The first run also
// owns dx of the initial state (t < 0).  A CTA is 32 threads along the channels x 8
// runs; the runs' sums meet in shared memory and leave as one part per CTA.
template <int K, typename T, int CH>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(ConvArgs a) {
  __shared__ f2 s_sum[kRows][K + 1][kLanes];
  const int cgs = (a.D + CH * kLanes - 1) / (CH * kLanes);
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  const int c0 = (blockIdx.x % cgs) * CH * kLanes, c = c0 + CH * lane;
  const int blocks = (a.T + kRun * kRows - 1) / (kRun * kRows);
  const int part = blockIdx.x / cgs, b = part / blocks, t0 = (part % blocks) * kRun * kRows + row * kRun;
  const int len = real_len(a.lens, b, a.T);
  const f2 one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
  f2 dw[K + 1];
#pragma unroll
  for (int j = 0; j <= K; ++j) dw[j] = 0;
  if (c < a.D && t0 < a.T) {
    f2 w[K], bias, x[K], du[K];
    const int first = t0 == 0 ? -(K - 1) : t0, last = min(t0 + kRun, a.T);   // own dx rows
    const T* xp = static_cast<const T*>(a.x) + b * a.x_sb + t0 * a.x_st + c;
    const T* gp = static_cast<const T*>(a.d_y) + ((long long)b * a.T + t0) * a.D + c;
    T* dx = static_cast<T*>(a.dx) + ((long long)b * a.T + t0 - (K - 1)) * a.D + c;   // of the row that is complete
    const int loads = min(len, last + K - 1);   // du is 0 from len on
    Raw<T, CH> xn[kAhead], gn[kAhead];
    auto fetch = [&](int tb) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (tb + i < loads) xn[i] = raw_ch<T, CH>(xp), gn[i] = raw_ch<T, CH>(gp);
        xp += a.x_st, gp += a.D;
      }
    };
    fetch(t0);
    load_filter<K, CH>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = t0 - (K - 1) + j;   // nothing from behind the end: 0 times it may be NaN
      x[j] = t < len ? load_in<K, T, CH>(a, b, t, c) : 0ull;
      du[j] = 0;
    }
    for (int tb = t0; tb < last + K - 1; tb += kAhead) {
      Raw<T, CH> xr[kAhead], gr[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) xr[i] = xn[i], gr[i] = gn[i];
      if (tb + kAhead < last + K - 1) fetch(tb + kAhead);
      auto walk = [&](auto is_plain) {
        constexpr bool plain = decltype(is_plain)::value;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int t = tb + i;
          if (!plain && t >= last + K - 1) break;
          const bool in = plain || t < loads;
          x[K - 1] = in ? pair_of(xr[i]) : 0ull;
          f2 g = in ? pair_of(gr[i]) : 0ull;
          if (a.silu) {   // silu'(u) = s (1 + u (1 - s))
            const f2 u = filtered<K>(w, bias, x), s = sigmoid2(u);
            g = mul2(g, mul2(s, fma2(u, fma2(s, minus, one), one)));
          }
          du[K - 1] = g;
          if (plain || t < last) {
            dw[K] = add2(dw[K], g);
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j] = fma2(g, x[j], dw[j]);
          }
          // du[j] holds du_{t-K+1+j}: row t-K+1 is complete
          const int r = t - (K - 1);
          if (plain || r >= first) {
            f2 o = mul2(w[K - 1], du[0]);
#pragma unroll
            for (int j = 1; j < K; ++j) o = fma2(w[K - 1 - j], du[j], o);
            const int f = r - (len - (K - 1));   // its place in the final state
            if (!plain && a.d_s1 && f >= 0 && f < K - 1)
              o = add2(o, load_ch<T, CH>(static_cast<const T*>(a.d_s1) + ((long long)b * (K - 1) + f) * a.D + c, true));
            if (plain || r >= 0)
              store_ch<T, CH>(dx, o);
            else if (a.d_s0)
              store_ch<T, CH>(static_cast<T*>(a.d_s0) + ((long long)b * (K - 1) + r + K - 1) * a.D + c, o);
          }
          dx += a.D;
#pragma unroll
          for (int j = 0; j < K - 1; ++j) x[j] = x[j + 1], du[j] = du[j + 1];
        }
      };
      // every token real, within the run, behind its first rows, before the final state's
      if (tb + kAhead <= min(last, len) && tb - (K - 1) >= t0 && (!a.d_s1 || tb + kAhead <= len - (K - 1)))
        walk(std::true_type());
      else
        walk(std::false_type());
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j) s_sum[row][j][lane] = dw[j];
  __syncthreads();
  for (int e = threadIdx.x; e < (K + 1) * kLanes; e += kThreads) {
    const int j = e / kLanes, i = e % kLanes;
    if (c0 + CH * i >= a.D) continue;
    f2 s = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) s = add2(s, s_sum[r][j][i]);
    store_ch<float, CH>(a.part + ((long long)part * (K + 1) + j) * a.D + c0 + CH * i, s);
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
  long long b;
  const int c = CH * div_mod(e, groups, b);
  if (b >= a.B) return;
  f2 w[K], bias, x[K];
#pragma unroll
  for (int j = 0; j < K; ++j) x[j] = load_in<K, T, CH>(a, b, j - (K - 1), c);
  load_filter<K, CH>(a, c, w, bias);
  f2 u = filtered<K>(w, bias, x);
  if (a.silu) u = mul2(u, sigmoid2(u));
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
