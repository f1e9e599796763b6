// selective_scan.cu — selective state space scan: forward, backward, one token.
//
//   h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] B_t[n] x_t[c]
//   y_t[c]   = sum_n C_t[n] h_t[c,n] + D[c] x_t[c],  gated by z sigmoid(z)
//
// Per (token, channel, state): one exponential, two products, two multiply-adds;
// the issue slots and the exponential units bound it, not the bytes.  N / 4
// neighbouring lanes own a pair of channels, four states of each in registers as
// packed pairs (one instruction for two products), and walk the tokens; B_t and C_t are
// the same for all channels of a group and come from shared memory as broadcast reads,
// once for both channels.  The lanes' parts of y are summed for N / 4 tokens at once by
// exchanging halves (N / 4 - 1 shuffles for N / 4 tokens).
//
// Few rows and many tokens are cut into pieces along the tokens: over a piece the
// state is h_end = exp(A sum dt) h_start + (end from zero), so a first pass takes
// every piece's end from zero and its sum of dt, a scan joins them, and the second
// pass starts every piece from its true state.
//   B1 T8192 D2048 N16 bf16: 168 us, 62 + 8 + 98; the exponentials of a pass alone take 29,
//   the second pass issues an instruction in 65 % of its cycles.
//
// Backward, with dy the gradient behind the gate and g_t that of h_t:
//   g_t = C_t dy_t + exp(dt_{t+1} A) g_{t+1}
//   dC_t[n] = sum_c dy h,  dB_t[n] = sum_c g dt x,  dx = dt sum_n g B + D dy
//   d dt = sum_n g exp(dt A) h_{t-1} A + x sum_n g B,  dA = sum_t g exp(dt A) h_{t-1} dt
// in pieces of kPiece tokens: a first pass takes every piece's end state from zero and
// the gradient that it hands to its start, a scan joins both, and the second pass
// recomputes a few tokens' states at a time in registers and walks them backwards.
// The sums over channels leave as one part per channel tile and are added in a fixed
// order: no atomics.
//   B4 T2048 D2048 N16 bf16: 460 us, 110 + 24 + 297 (71 % of the issue slots) + 27 of sums.
// Everything between loads and stores is fp32; outputs are rounded once.
#include <algorithm>

#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 32;    // tokens of a backward piece
constexpr int kEndsPerSM = 8;  // CTAs of the backward's first pass
constexpr int kTile = 16;     // tokens in shared memory at a time (forward)
constexpr int kSub = 8;       // tokens whose states are in registers (backward)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int N> struct Shape {
  static constexpr int LPC = N / 4;               // lanes per pair of channels
  static constexpr int CPC = 2 * kThreads / LPC;  // channels per CTA
  static constexpr int CW = 32 / LPC;             // pairs of channels per warp
  static constexpr int HP = CPC / 2;              // pairs of channels per CTA
  static constexpr int WC = 2 * CW;               // channels per warp
  static constexpr int ROWS = kThreads / HP;      // tokens that the CTA loads at a time (backward)
};

// log(1 + e^v) = max(v, 0) + log1p(e), e = exp(-|v|).  log1p(e) / e over [0, 1] is a polynomial of
// degree 8, fitted to the least largest relative error by reweighted least squares (3e-8; in
// fp32 arithmetic 1.7e-7).  fp32 takes the type's exponential, bf16 the approximate one, whose
// exponent is |v| 2^-24 off.  (A base-2 logarithm of 1 + e in its place is 2^-18.5 off at e =
// 1/16, 1.2e-6 of dA.)
template <typename T>
__device__ __forceinline__ float softplus_f(float v) {
  const float e = sizeof(T) == 4 ? expf(-fabsf(v)) : ex2(-fabsf(v) * kLog2e);
  float p = 0.0052326913f;
  p = fmaf(e, p, -0.0295052268f);
  p = fmaf(e, p, 0.078225933f);
  p = fmaf(e, p, -0.136632442f);
  p = fmaf(e, p, 0.191060066f);
  p = fmaf(e, p, -0.24842982f);
  p = fmaf(e, p, 0.333190978f);
  p = fmaf(e, p, -0.499994934f);
  p = fmaf(e, p, 0.99999994f);
  return fmaf(e, p, fmaxf(v, 0.f));
}

// Two neighbouring channels as loaded.  A thread's pair of channels follows its
// neighbour's: whole 128-byte rows in global memory, and 16 bytes a lane in shared memory
// without a conflict of banks (8 channels a thread cost a third of the time there).
template <typename T> struct alignas(2 * sizeof(T)) Raw2 { T v[2]; };

template <typename T>
__device__ __forceinline__ void widen2(float (&f)[2], const T* p) {
  const Raw2<T> r = *reinterpret_cast<const Raw2<T>*>(p);
  f[0] = to_f<T>(r.v[0]), f[1] = to_f<T>(r.v[1]);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store2(T* p, int n, const float (&f)[2]) {
  Raw2<T> r;
  r.v[0] = from_f<T>(f[0]), r.v[1] = from_f<T>(f[1]);
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<Raw2<T>*>(p) = r;
  } else {
    if (n > 0) p[0] = r.v[0];
    if (n > 1) p[1] = r.v[1];
  }
}

// ROWS rows from t0 on of WIDTH neighbouring values, src at row 0, into shared memory by
// `THREADS` threads: in 16-byte pieces, or as wide as a row, that go on in the background;
// zeros in place of rows from t_real on and of values from n on.
template <typename T, bool VEC, int WIDTH, int ROWS = kTile, int THREADS = 32>
__device__ __forceinline__ void fetch_rows(T* dst, const T* src, long long stride, int t0, int t_real, int n, int tid) {
  if constexpr (VEC) {
    constexpr int ROW = WIDTH * sizeof(T), CB = ROW < 16 ? ROW : 16, PER = ROW / CB, ALL = ROWS * PER;
#pragma unroll
    for (int e0 = 0; e0 < ALL; e0 += THREADS) {
      const int e = e0 + tid, t = t0 + e / PER, k = e % PER * (CB / (int)sizeof(T));
      const bool in = t < t_real && k < n;
      if (ALL % THREADS == 0 || e < ALL)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + e * CB),
                     "l"(in ? src + t * stride + k : src), "n"(CB), "r"(in ? CB : 0)
                     : "memory");
    }
  } else {
    for (int e = tid; e < ROWS * WIDTH; e += THREADS) {
      const int t = t0 + e / WIDTH, k = e % WIDTH;
      dst[e] = t < t_real && k < n ? src[t * stride + k] : from_f<T>(0.f);
    }
  }
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ROWS rows of N values to fp32
template <int N, typename T, int ROWS = kTile, int THREADS = 32>
__device__ __forceinline__ void widen_rows(float* dst, const T* src, int tid) {
#pragma unroll
  for (int e = 4 * tid; e < ROWS * N; e += 4 * THREADS) {
    float4 f;
    if constexpr (sizeof(T) == 2) {
      const uint2 r = *reinterpret_cast<const uint2*>(src + e);
      f = make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                      __uint_as_float(r.y & 0xffff0000u));
    } else {
      f = *reinterpret_cast<const float4*>(src + e);
    }
    *reinterpret_cast<float4*>(dst + e) = f;
  }
}

// Sum over L lanes, STRIDE apart, of M values each: halves are exchanged as long as a
// lane holds more than one.  Lane position p ends with the values p M/L .. (M >= L),
// or with value p / (L/M).
template <int M, int L, int STRIDE>
__device__ __forceinline__ void lane_sums(float (&v)[M], int lane) {
  int m = M;
#pragma unroll
  for (int w = L / 2; w >= 1; w >>= 1) {
    if (m > 1) {
      const int half = m / 2;
      const bool up = lane & (w * STRIDE);
#pragma unroll
      for (int i = 0; i < M / 2; ++i) {
        if (i >= half) break;
        const float send = up ? v[i] : v[i + half];
        const float keep = up ? v[i + half] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w * STRIDE);
      }
      m = half;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], w * STRIDE);
    }
  }
}

// Which channels a CTA owns: tile `i` of the tiles of CPC channels, none across a group.
struct ChannelTile {
  int g, c0, n;
  __device__ __forceinline__ ChannelTile(const ScanArgs& a, int cpc, int i) {
    const int dg = a.D / a.G, per = (dg + cpc - 1) / cpc;
    g = i / per;
    const int k = i % per * cpc;
    c0 = g * dg + k;
    n = min(cpc, dg - k);
  }
};

// Four states of one channel: two register pairs.
struct Four { f2 a, b; };
__device__ __forceinline__ Four load4(const float* p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  return {v.x, v.y};
}
__device__ __forceinline__ void store4(float* p, const Four& v) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v.a, v.b);
}
__device__ __forceinline__ Four both(f2 x) { return {x, x}; }
__device__ __forceinline__ Four mul(const Four& x, const Four& y) { return {mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ Four mul(const Four& x, f2 y) { return {mul2(x.a, y), mul2(x.b, y)}; }
__device__ __forceinline__ Four fma(const Four& x, const Four& y, const Four& z) {
  return {fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)};
}
__device__ __forceinline__ Four fma(const Four& x, f2 y, const Four& z) {
  return {fma2(x.a, y, z.a), fma2(x.b, y, z.b)};
}
__device__ __forceinline__ Four exp2_4(const Four& x) { return {ex2_2(x.a), ex2_2(x.b)}; }
// exp2 of the rates times the time step.  A state goes through the product of thousands of
// decays, and ex2.approx rounds low: by 1e-8 to 3e-8 on average for exponents of -0.4 to -0.005,
// 2e-6 of a state after 100 tokens.  kUp in the exponent, where the multiply-add takes it for
// nothing, leaves 1e-8 either way (7e-7); exp2(kUp) is 1, so that dt = 0 keeps a state as it is.
constexpr float kUp = 2e-8f;
__device__ __forceinline__ Four decay(const Four& A2, f2 dt) { return exp2_4(fma(A2, dt, both(pack2(kUp, kUp)))); }
// sum over the four of x y
__device__ __forceinline__ float dot(const Four& x, const Four& y) { return sum2(fma2(x.a, y.a, mul2(x.b, y.b))); }

// dt, dt x of a pair of neighbouring channels, each value twice
struct Steps { f2 dt[2], dx[2]; };
__device__ __forceinline__ Steps load_steps(const float2* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  return {{pack2(v.x, v.x), pack2(v.z, v.z)}, {pack2(v.y, v.y), pack2(v.w, v.w)}};
}

// A log2(e) of this lane's four states of its two channels
template <int N>
__device__ __forceinline__ void load_rates(const ScanArgs& a, int c, int n, int part, Four (&A2)[2]) {
  const f2 k = pack2(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    A2[i] = i < n ? mul(load4(a.A + (long long)(c + i) * N + 4 * part), k) : both(0);
}

__device__ __forceinline__ float bias_of(const ScanArgs& a, int c) { return a.bias ? a.bias[c] : 0.f; }

// ------------------------------------------------------------------ forward

// One warp's shared memory: (dt, dt x), B and for outputs C and y in fp32; two tiles as
// loaded: x, dt, B and for outputs z and C.
template <int N, typename T, bool FULL> struct FwdTile {
  static constexpr int WC = Shape<N>::WC;
  static constexpr int kRaw = kTile * (FULL ? 3 * WC + 2 * N : 2 * WC + N);   // values of a tile as loaded
  static constexpr int kBytes = 4 * kTile * (FULL ? 3 * WC + 2 * N : 2 * WC + N) + 2 * kRaw * (int)sizeof(T);
};

// FULL: outputs from the state at the piece's start; otherwise the piece's end from
// zero and its sum of dt.  The warps share nothing and never wait for each other: with one
// tile for the CTA, its barriers and conflicts of banks cost 166 us instead of 105
// (B4 T2048 D2048 N16).
template <int N, typename T, bool VEC, bool FULL>
__global__ void __launch_bounds__(kThreads, FULL ? (N == 64 ? 3 : N == 32 ? 4 : 5) : (N == 64 ? 4 : N == 32 ? 5 : 6)) scan_fwd_kernel(ScanArgs a) {
  using S = Shape<N>;
  using W = FwdTile<N, T, FULL>;
  constexpr int CPC = S::CPC, LPC = S::LPC, WC = S::WC, TT = kTile;
  constexpr int NP = TT / LPC;   // tokens of a tile per lane
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = tid % LPC, ch = 2 * (tid / LPC);
  float2* s_u = reinterpret_cast<float2*>(reinterpret_cast<char*>(sm) + warp * W::kBytes);   // [TT][WC]
  float* s_B = reinterpret_cast<float*>(s_u + TT * WC);                                    // [TT][N]
  float* s_C = s_B + TT * N;
  float* s_y = s_C + (FULL ? TT * N : 0);                                                  // [TT][WC]
  T* raw = reinterpret_cast<T*>(s_y + (FULL ? TT * WC : 0));
  const int tiles = gridDim.x / (a.B * a.n_piece);
  const ChannelTile ct(a, CPC, blockIdx.x % tiles);
  const int piece = (blockIdx.x / tiles) % a.n_piece, b = blockIdx.x / tiles / a.n_piece;
  const int t_begin = piece * a.piece, t_end = min(a.T, t_begin + a.piece);
  const int len = real_len(a.lens, b, a.T), t_real = min(len, t_end);
  const int c = ct.c0 + ch, real = ct.n - ch;   // channels of the pair that exist: real > 0, > 1
  const int wc = ct.c0 + warp * WC, wn = ct.n - warp * WC;   // the warp's channels
  if (wn <= 0) return;

  Four A2[2], h[2] = {both(0), both(0)};
  float sum[2] = {0.f, 0.f};
  load_rates<N>(a, c, real, part, A2);
  if (FULL) {
    const float* from = a.n_piece > 1 ? a.hs + ((long long)b * a.n_piece + piece) * a.D * N
                                      : (a.h0 ? a.h0 + (long long)b * a.D * N : nullptr);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (from && i < real) h[i] = load4(from + (long long)(c + i) * N + 4 * part);
  }
  // between the tile as loaded and the walk a lane has tokens vt + i LPC, channels vc, vc + 1
  const int vt = lane / S::CW, vc = 2 * (lane % S::CW), n = wn - vc;
  float bias[2], skip[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bias[i] = i < n ? bias_of(a, wc + vc + i) : 0.f;
    skip[i] = i < n && a.Dskip ? a.Dskip[wc + vc + i] : 0.f;
  }
  auto fetch = [&](T* r, int t0) {
    fetch_rows<T, VEC, WC>(r, static_cast<const T*>(a.x) + b * a.x_sb + wc, a.x_st, t0, t_real, wn, lane);
    fetch_rows<T, VEC, WC>(r + TT * WC, static_cast<const T*>(a.dt) + b * a.dt_sb + wc, a.dt_st, t0, t_real, wn, lane);
    fetch_rows<T, VEC, N>(r + 2 * TT * WC, static_cast<const T*>(a.Bm) + b * a.B_sb + ct.g * N, a.B_st, t0, t_real, N,
                          lane);
    if (FULL) {
      fetch_rows<T, VEC, N>(r + TT * (2 * WC + N), static_cast<const T*>(a.Cm) + b * a.C_sb + ct.g * N, a.C_st, t0,
                            t_real, N, lane);
      if (a.z)
        fetch_rows<T, VEC, WC>(r + TT * (2 * WC + 2 * N), static_cast<const T*>(a.z) + b * a.z_sb + wc, a.z_st, t0,
                               t_real, wn, lane);
    }
  };
  fetch(raw, t_begin);
  T* now = raw;
  T* next = raw + W::kRaw;
  for (int t0 = t_begin; t0 < t_end; t0 += TT) {
    fetched();
    __syncwarp();
    if (t0 + TT < t_end) fetch(next, t0 + TT);
    const Raw2<T>* x_in = reinterpret_cast<const Raw2<T>*>(now + vt * WC + vc);   // a lane's: 16 pairs apart
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int t = vt + i * LPC, k = t0 + t < t_real ? n : 0;
      const Raw2<T> xr = x_in[i * 32], dr = x_in[i * 32 + TT * S::CW];
      float d[2], u[2];   // nothing of a token that is not there: its state stays as it is
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        d[j] = to_f<T>(dr.v[j]) + bias[j];
        if (a.softplus) d[j] = softplus_f<T>(d[j]);
        d[j] = j < k ? d[j] : 0.f;
        u[j] = d[j] * to_f<T>(xr.v[j]);
      }
      *reinterpret_cast<float4*>(s_u + t * WC + vc) = make_float4(d[0], u[0], d[1], u[1]);
    }
    widen_rows<N>(s_B, now + 2 * TT * WC, lane);
    if (FULL) widen_rows<N>(s_C, now + TT * (2 * WC + N), lane);
    __syncwarp();
#pragma unroll 1
    for (int g = 0; g < TT; g += LPC) {
      float y[2][LPC];
#pragma unroll
      for (int k = 0; k < LPC; ++k) {
        const Steps u = load_steps(s_u + (g + k) * WC + 2 * (lane / LPC));
        const Four B = load4(s_B + (g + k) * N + 4 * part);
        Four C = B;
        if (FULL) C = load4(s_C + (g + k) * N + 4 * part);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          h[i] = fma(decay(A2[i], u.dt[i]), h[i], mul(B, u.dx[i]));
          if (FULL) {
            y[i][k] = dot(C, h[i]);
          } else {
            float d, same;
            unpack2(u.dt[i], d, same);
            sum[i] += d;
          }
        }
      }
      if (FULL) {
        lane_sums<LPC, LPC, 1>(y[0], lane);
        lane_sums<LPC, LPC, 1>(y[1], lane);
        *reinterpret_cast<float2*>(s_y + (g + part) * WC + 2 * (lane / LPC)) = make_float2(y[0][0], y[1][0]);
      }
    }
    __syncwarp();
    if (FULL) {
      const Raw2<T>* z_in = reinterpret_cast<const Raw2<T>*>(now + TT * (2 * WC + 2 * N) + vt * WC + vc);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int t = t0 + vt + i * LPC;
        if (t >= t_end) break;
        const float2 y = *reinterpret_cast<const float2*>(s_y + (vt + i * LPC) * WC + vc);
        const Raw2<T> xr = x_in[i * 32];
        float o[2] = {y.x, y.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          o[j] += skip[j] * to_f<T>(xr.v[j]);
          if (a.z) {
            const float z = to_f<T>(z_in[i * 32].v[j]);
            o[j] *= z * sigmoid_f(z);
          }
          if (t >= len) o[j] = 0.f;
        }
        store2<T, VEC>(static_cast<T*>(a.y) + ((long long)b * a.T + t) * a.D + wc + vc, n, o);
      }
    }
    T* const was = now;
    now = next, next = was;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= real) break;
    const long long row = ((long long)b * a.n_piece + piece) * a.D + c + i;
    if (!FULL) {
      store4(a.hs + row * N + 4 * part, h[i]);
      if (part == 0) a.sum_dt[row] = sum[i];
    } else if (a.hT && piece == a.n_piece - 1) {
      store4(a.hT + ((long long)b * a.D + c + i) * N + 4 * part, h[i]);
    }
  }
}

// Joins the pieces: hs becomes the state at each piece's start; for the backward, whose
// blocks are twice as many, es the gradient at each piece's end, and the gradient of the
// initial state.  One thread per state; the next kBatch pieces are loaded ahead of the chain
// that goes through these.
__global__ void __launch_bounds__(kThreads) scan_join_kernel(ScanArgs a) {
  constexpr int kBatch = 8;
  const long long per = (long long)a.D * a.N, all = a.B * per;
  const unsigned half = static_cast<unsigned>((all + kThreads - 1) / kThreads);
  const bool back = blockIdx.x >= half;
  const long long e = (long long)(back ? blockIdx.x - half : blockIdx.x) * kThreads + threadIdx.x;
  if (e >= all) return;
  const long long b = e / per, cn = e % per, c = cn / a.N, first = b * a.n_piece + (back ? a.n_piece - 1 : 0);
  const float A2 = a.A[cn] * kLog2e;
  const long long ds = back ? -per : per, dd = back ? -a.D : a.D;
  float* s = (back ? a.es : a.hs) + first * per + cn;
  const float* in = s;
  const float* sd = a.sum_dt + first * a.D + c;
  const float* from = back ? a.d_hT : a.h0;
  float h = from ? from[e] : 0.f;
  float end[2][kBatch], d[2][kBatch];
  int left = a.n_piece;   // to load
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k < left) end[i][k] = *in, d[i][k] = *sd;
      in += ds, sd += dd;
    }
    left -= kBatch;
  };
  auto chain = [&](int i, int n) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k >= n) break;
      *s = h;
      s += ds;
      h = ex2(A2 * d[i][k]) * h + end[i][k];
    }
  };
  load(0);
  for (int n = a.n_piece; n > 0; n -= 2 * kBatch) {
    load(1);
    chain(0, n);
    load(0);
    chain(1, n - kBatch);
  }
  if (back && a.g.d_init_state) a.g.d_init_state[e] = h;
}

// ------------------------------------------------------------------ backward

// dt, dt x and dy behind the gate of a lane's pair of channels
template <typename T>
__device__ __forceinline__ void widen_steps(const ScanArgs& a, const T* x_in, const T* d_in, const T* g_in, const T* z_in,
                                            const float (&bias)[2], int n, float2* u, float* dy) {
  float x[2], d[2], g[2], z[2];
  widen2(x, x_in), widen2(d, d_in), widen2(g, g_in);
  if (a.z) widen2(z, z_in);
#pragma unroll
  for (int k = 0; k < 2; ++k) {   // nothing of a token that is not there
    d[k] += bias[k];
    if (a.softplus) d[k] = softplus_f<T>(d[k]);
    d[k] = k < n ? d[k] : 0.f;
    x[k] *= d[k];
    if (a.z) g[k] *= z[k] * sigmoid_f(z[k]);
  }
  *reinterpret_cast<float4*>(u) = make_float4(d[0], x[0], d[1], x[1]);
  *reinterpret_cast<float2*>(dy) = make_float2(g[0], g[1]);
}

// Where channel c of token t is in an array of [kPiece][CPC]: the rows turn, so that the lanes
// of a channel pair, which write neighbouring tokens, meet in no bank.
template <int N> __device__ __forceinline__ int turned(int t, int c) {
  return t * Shape<N>::CPC + ((c + t * Shape<N>::CW) & (Shape<N>::CPC - 1));
}

__device__ __forceinline__ void load_dy(const float* p, f2 (&dy)[2]) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  dy[0] = pack2(v.x, v.x), dy[1] = pack2(v.y, v.y);
}

// One warp's shared memory: (dt, dt x), dy, B and C in fp32; two tiles as loaded: x, dt, dy,
// z, B, C.
template <int N, typename T> struct EndsTile {
  static constexpr int WC = Shape<N>::WC;
  static constexpr int kRaw = kTile * (4 * WC + 2 * N);
  static constexpr int kBytes = 4 * kTile * (3 * WC + 2 * N) + 2 * kRaw * (int)sizeof(T);
};

// Of `span` pieces one after the other: the end state from zero, the gradient that reaches
// the piece's start, its sum of dt.  The warps never wait for each other.
template <int N, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) scan_bwd_ends_kernel(ScanArgs a) {
  using S = Shape<N>;
  using W = EndsTile<N, T>;
  constexpr int CPC = S::CPC, LPC = S::LPC, WC = S::WC, TT = kTile;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = tid % LPC, ch = 2 * (tid / LPC);
  float2* s_u = reinterpret_cast<float2*>(reinterpret_cast<char*>(sm) + warp * W::kBytes);
  float* s_dy = reinterpret_cast<float*>(s_u + TT * WC);
  float* s_B = s_dy + TT * WC;
  float* s_C = s_B + TT * N;
  T* now = reinterpret_cast<T*>(s_C + TT * N);
  T* next = now + W::kRaw;
  const int n_span = (a.n_piece + a.span - 1) / a.span, tiles = gridDim.x / (a.B * n_span);
  const ChannelTile ct(a, CPC, blockIdx.x % tiles);
  const int p0 = (blockIdx.x / tiles) % n_span * a.span, b = blockIdx.x / tiles / n_span;
  const int t_end = min(a.n_piece, p0 + a.span) * kPiece, t_real = real_len(a.lens, b, a.T);
  const int c = ct.c0 + ch, real = ct.n - ch;
  const int wc = ct.c0 + warp * WC, wn = ct.n - warp * WC;   // the warp's channels
  if (wn <= 0) return;
  const f2 one = pack2(1.f, 1.f);
  Four A2[2], h[2] = {both(0), both(0)}, e[2] = {both(0), both(0)}, cp[2] = {both(one), both(one)};
  float sum[2] = {0.f, 0.f};
  load_rates<N>(a, c, real, part, A2);
  const int vt = lane / S::CW, vc = 2 * (lane % S::CW), n = wn - vc;
  float bias[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) bias[i] = i < n ? bias_of(a, wc + vc + i) : 0.f;
  auto fetch = [&](T* r, int t0) {
    fetch_rows<T, VEC, WC>(r, static_cast<const T*>(a.x) + b * a.x_sb + wc, a.x_st, t0, t_real, wn, lane);
    fetch_rows<T, VEC, WC>(r + TT * WC, static_cast<const T*>(a.dt) + b * a.dt_sb + wc, a.dt_st, t0, t_real, wn, lane);
    fetch_rows<T, VEC, WC>(r + 2 * TT * WC, static_cast<const T*>(a.d_y) + (long long)b * a.T * a.D + wc, a.D, t0, t_real,
                           wn, lane);
    if (a.z)
      fetch_rows<T, VEC, WC>(r + 3 * TT * WC, static_cast<const T*>(a.z) + b * a.z_sb + wc, a.z_st, t0, t_real, wn, lane);
    fetch_rows<T, VEC, N>(r + 4 * TT * WC, static_cast<const T*>(a.Bm) + b * a.B_sb + ct.g * N, a.B_st, t0, t_real, N,
                          lane);
    fetch_rows<T, VEC, N>(r + TT * (4 * WC + N), static_cast<const T*>(a.Cm) + b * a.C_sb + ct.g * N, a.C_st, t0, t_real,
                          N, lane);
  };
  fetch(now, p0 * kPiece);
  for (int t0 = p0 * kPiece; t0 < t_end; t0 += TT) {
    fetched();
    __syncwarp();
    if (t0 + TT < t_end) fetch(next, t0 + TT);
#pragma unroll
    for (int i = 0; i < TT / LPC; ++i) {
      const int t = vt + i * LPC, at = t * WC + vc;
      widen_steps<T>(a, now + at, now + TT * WC + at, now + 2 * TT * WC + at, now + 3 * TT * WC + at, bias,
                     t0 + t < t_real ? n : 0, s_u + at, s_dy + at);
    }
    widen_rows<N>(s_B, now + 4 * TT * WC, lane);
    widen_rows<N>(s_C, now + TT * (4 * WC + N), lane);
    __syncwarp();
#pragma unroll 4
    for (int t = 0; t < TT; ++t) {
      const Steps u = load_steps(s_u + t * WC + 2 * (lane / LPC));
      f2 dy[2];
      load_dy(s_dy + t * WC + 2 * (lane / LPC), dy);
      const Four B = load4(s_B + t * N + 4 * part), C = load4(s_C + t * N + 4 * part);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Four x = decay(A2[i], u.dt[i]);
        h[i] = fma(x, h[i], mul(B, u.dx[i]));
        cp[i] = mul(cp[i], x);
        e[i] = fma(cp[i], mul(C, dy[i]), e[i]);
        float d, same;
        unpack2(u.dt[i], d, same);
        sum[i] += d;
      }
    }
    __syncwarp();
    T* const was = now;
    now = next, next = was;
    if ((t0 + TT) % kPiece) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long row = ((long long)b * a.n_piece + t0 / kPiece) * a.D + c + i;
      if (i < real) {
        store4(a.hs + row * N + 4 * part, h[i]);
        store4(a.es + row * N + 4 * part, e[i]);
        if (part == 0) a.sum_dt[row] = sum[i];
      }
      h[i] = both(0), e[i] = both(0), cp[i] = both(one), sum[i] = 0.f;
    }
  }
}

// A piece's x, dt, dy and z as loaded lie where its states are put later, and come a second
// time for the gradients of the inputs when the states have been read; B and C as loaded lie
// where the sums are put.
template <int N, typename T> constexpr int bwd_smem() {
  using S = Shape<N>;
  const int states = 4 * 8 * kThreads * (kPiece / kSub), raw = 4 * kPiece * S::CPC * (int)sizeof(T);
  return 4 * (kPiece * (4 * S::CPC + 2 * N) + kWarps * kSub * 2 * N) + (raw > states ? raw : states);
}

template <int N, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) scan_bwd_kernel(ScanArgs a) {
  using S = Shape<N>;
  constexpr int CPC = S::CPC, LPC = S::LPC, CW = S::CW;
  constexpr int TG = LPC < kSub ? LPC : kSub;   // tokens whose sums over a channel's lanes go together
  extern __shared__ __align__(16) float sm[];
  float2* s_u = reinterpret_cast<float2*>(sm);         // (dt, dt x), then (dt, sum_n g B)
  float* s_dy = sm + 2 * kPiece * CPC;                 // dy, then sum_n g a h A
  float* s_B = s_dy + kPiece * CPC;
  float* s_C = s_B + kPiece * N;
  float* s_y = s_C + kPiece * N;                       // sum_n C h
  float* s_bc = s_y + kPiece * CPC;                    // [warp][kSub][2N] sums over a warp's channels
  float* s_h = s_bc + kWarps * kSub * 2 * N;           // states at the sub-tiles' starts
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = tid % LPC, ch = 2 * (tid / LPC);
  const int tiles = gridDim.x / (a.B * a.n_piece);
  const int tile = blockIdx.x % tiles;
  const ChannelTile ct(a, CPC, tile);
  const int piece = (blockIdx.x / tiles) % a.n_piece, b = blockIdx.x / tiles / a.n_piece;
  const int t0 = piece * kPiece, len = real_len(a.lens, b, a.T);
  const int c = ct.c0 + ch, real = ct.n - ch;
  const long long row = ((long long)b * a.n_piece + piece) * a.D + c;
  Four A2[2], h[2] = {both(0), both(0)}, gc[2] = {both(0), both(0)}, dA[2] = {both(0), both(0)};
  load_rates<N>(a, c, real, part, A2);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (i < real) {
      h[i] = load4(a.hs + (row + i) * N + 4 * part);
      gc[i] = load4(a.es + (row + i) * N + 4 * part);
    }
  T* raw = reinterpret_cast<T*>(s_h);
  auto fetch = [&] {
    constexpr int ALL = kPiece * CPC;
    auto rows = [&](int i, const void* p, long long sb, long long st) {
      fetch_rows<T, VEC, CPC, kPiece, kThreads>(raw + i * ALL, static_cast<const T*>(p) + b * sb + ct.c0, st, t0, len, ct.n,
                                                tid);
    };
    rows(0, a.x, a.x_sb, a.x_st);
    rows(1, a.dt, a.dt_sb, a.dt_st);
    rows(2, a.d_y, (long long)a.T * a.D, a.D);
    if (a.z) rows(3, a.z, a.z_sb, a.z_st);
  };
  fetch();
  T* raw_B = reinterpret_cast<T*>(s_y);
  T* raw_C = raw_B + kPiece * N;
  fetch_rows<T, VEC, N, kPiece, kThreads>(raw_B, static_cast<const T*>(a.Bm) + b * a.B_sb + ct.g * N, a.B_st, t0, len, N,
                                          tid);
  fetch_rows<T, VEC, N, kPiece, kThreads>(raw_C, static_cast<const T*>(a.Cm) + b * a.C_sb + ct.g * N, a.C_st, t0, len, N,
                                          tid);
  // between the piece as loaded and the walk a thread has every ROWS-th token, channels vc, vc + 1
  const int vc = 2 * (tid % S::HP), n = ct.n - vc;
  float bias[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) bias[k] = k < n ? bias_of(a, ct.c0 + vc + k) : 0.f;
  fetched();
  __syncthreads();
#pragma unroll 4
  for (int vt = tid / S::HP; vt < kPiece; vt += S::ROWS) {
    const int at = vt * CPC + vc;
    constexpr int ALL = kPiece * CPC;
    widen_steps<T>(a, raw + at, raw + ALL + at, raw + 2 * ALL + at, raw + 3 * ALL + at, bias, t0 + vt < len ? n : 0,
                   s_u + at, s_dy + at);
  }
  widen_rows<N, T, kPiece, kThreads>(s_B, raw_B, tid);
  widen_rows<N, T, kPiece, kThreads>(s_C, raw_C, tid);
  __syncthreads();
  // the state at each sub-tile's start
  float* own = s_h + 4 * tid;   // [sub][channel][thread][4]
  for (int s = 0; s < kPiece / kSub; ++s) {
    store4(own + (2 * s) * 4 * kThreads, h[0]);
    store4(own + (2 * s + 1) * 4 * kThreads, h[1]);
    if (s == kPiece / kSub - 1) break;
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      const int t = s * kSub + k;
      const Steps u = load_steps(s_u + t * CPC + ch);
      const Four B = load4(s_B + t * N + 4 * part);
#pragma unroll
      for (int i = 0; i < 2; ++i) h[i] = fma(decay(A2[i], u.dt[i]), h[i], mul(B, u.dx[i]));
    }
  }
#pragma unroll 1
  for (int s = kPiece / kSub - 1; s >= 0; --s) {
    Four hh[kSub + 1][2];   // hh[k]: the state before token k
#pragma unroll
    for (int i = 0; i < 2; ++i) hh[0][i] = load4(own + (2 * s + i) * 4 * kThreads);
#pragma unroll
    for (int g = 0; g < kSub; g += TG) {
      float y[2][TG];
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const int t = s * kSub + g + k;
        const Steps u = load_steps(s_u + t * CPC + ch);
        const Four B = load4(s_B + t * N + 4 * part), C = load4(s_C + t * N + 4 * part);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          hh[g + k + 1][i] = fma(decay(A2[i], u.dt[i]), hh[g + k][i], mul(B, u.dx[i]));
          y[i][k] = dot(C, hh[g + k + 1][i]);
        }
      }
      if (a.z) {
        lane_sums<TG, LPC, 1>(y[0], lane);
        lane_sums<TG, LPC, 1>(y[1], lane);
        *reinterpret_cast<float2*>(s_y + turned<N>(s * kSub + g + part * TG / LPC, ch)) =
            make_float2(y[0][0], y[1][0]);
      }
    }
    __syncthreads();   // the last sub-tile's s_bc has been read, and at s = 0 every state of s_h
    if (s == 0) fetch();
#pragma unroll
    for (int g = kSub - TG; g >= 0; g -= TG) {
      float q[2][2 * TG];   // token k: sum g B, sum e A
#pragma unroll
      for (int k = TG - 1; k >= 0; --k) {
        const int t = s * kSub + g + k;
        const Steps u = load_steps(s_u + t * CPC + ch);
        f2 dy[2];
        load_dy(s_dy + t * CPC + ch, dy);
        const Four B = load4(s_B + t * N + 4 * part), C = load4(s_C + t * N + 4 * part);
        Four sB = both(0), sC = both(0);   // dB and dC of this lane's channels
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Four gi = fma(C, dy[i], gc[i]);
          q[i][2 * k] = dot(gi, B);
          sB = i ? fma(gi, u.dx[i], sB) : mul(gi, u.dx[i]);
          sC = i ? fma(hh[g + k + 1][i], dy[i], sC) : mul(hh[g + k + 1][i], dy[i]);
          gc[i] = mul(gi, decay(A2[i], u.dt[i]));
          const Four e = mul(gc[i], hh[g + k][i]);
          q[i][2 * k + 1] = dot(e, A2[i]);
          dA[i] = fma(e, u.dt[i], dA[i]);
        }
        float v[8];
        unpack2(sB.a, v[0], v[1]), unpack2(sB.b, v[2], v[3]);
        unpack2(sC.a, v[4], v[5]), unpack2(sC.b, v[6], v[7]);
        lane_sums<8, CW, LPC>(v, lane);
        float* bc = s_bc + (warp * kSub + g + k) * 2 * N + 4 * part;
        constexpr int PER = 8 / CW > 0 ? 8 / CW : 1;   // values a lane ends with
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int idx = CW <= 8 ? (lane / LPC) * PER + i : (lane / LPC) / (CW / 8);
          bc[(idx / 4) * N + idx % 4] = v[i];
        }
      }
      constexpr int PER = 2 * TG / LPC;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lane_sums<2 * TG, LPC, 1>(q[i], lane);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int idx = part * PER + k, at = (s * kSub + g + idx / 2) * CPC + ch + i;
          if (idx % 2 == 0)
            s_u[at].y = q[i][k];
          else
            s_dy[at] = q[i][k] * kLn2;   // A2 carries log2(e)
        }
      }
    }
    __syncthreads();
    for (int e = tid; e < kSub * 2 * N; e += kThreads) {
      const int t = t0 + s * kSub + e / (2 * N);
      if (t >= a.T) break;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s_bc[w * kSub * 2 * N + e];
      a.part_bc[(((long long)tile * a.B + b) * a.T + t) * 2 * N + e % (2 * N)] = v;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (i < real) store4(a.hs + (row + i) * N + 4 * part, dA[i]);
  // dx, ddt, dz of two channels per thread and token; the sums over the piece for dD and d bias
  float sd[2] = {}, sb[2] = {}, skip[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) skip[k] = k < n && a.Dskip ? a.Dskip[ct.c0 + vc + k] : 0.f;
  fetched();
  __syncthreads();
#pragma unroll 4
  for (int vt = tid / S::HP; vt < kPiece; vt += S::ROWS) {
    const int t = t0 + vt;
    if (t >= a.T || n <= 0) break;
    const int nr = t < len ? n : 0;
    float x[2], d[2], gy[2], z[2], dx[2], ddt[2], dz[2];
    constexpr int ALL = kPiece * CPC;
    const T* in = raw + vt * CPC + vc;
    widen2(x, in), widen2(d, in + ALL), widen2(gy, in + 2 * ALL);
    if (a.z) widen2(z, in + 3 * ALL);
    const float4 u4 = *reinterpret_cast<const float4*>(s_u + vt * CPC + vc);   // dt, sum g B
    const float2 e2 = *reinterpret_cast<const float2*>(s_dy + vt * CPC + vc);
    float2 y2 = make_float2(0.f, 0.f);
    if (a.z) y2 = *reinterpret_cast<const float2*>(s_y + turned<N>(vt, vc));
    const float dt[2] = {u4.x, u4.z}, gB[2] = {u4.y, u4.w}, eA[2] = {e2.x, e2.y}, y[2] = {y2.x, y2.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool ok = k < nr;
      float dy = gy[k];
      if (a.z) {
        const float sg = sigmoid_f(z[k]);
        dz[k] = ok ? gy[k] * (y[k] + skip[k] * x[k]) * sg * (1.f + z[k] * (1.f - sg)) : 0.f;
        dy *= z[k] * sg;
      }
      dx[k] = ok ? gB[k] * dt[k] + skip[k] * dy : 0.f;
      ddt[k] = ok ? eA[k] + gB[k] * x[k] : 0.f;
      if (a.softplus && ok) ddt[k] *= sigmoid_f(d[k] + bias[k]);
      sd[k] += ok ? dy * x[k] : 0.f;
      sb[k] += ddt[k];
    }
    const long long o = ((long long)b * a.T + t) * a.D + ct.c0 + vc;
    store2<T, VEC>(static_cast<T*>(a.g.dx) + o, n, dx);
    store2<T, VEC>(static_cast<T*>(a.g.ddt) + o, n, ddt);
    if (a.z) store2<T, VEC>(static_cast<T*>(a.g.dz) + o, n, dz);
  }
  __syncthreads();
  constexpr int R = S::ROWS;   // rows of partial sums, over the piece's buffers
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    sm[(tid / S::HP) * CPC + vc + k] = sd[k];
    sm[(R + tid / S::HP) * CPC + vc + k] = sb[k];
  }
  __syncthreads();
  for (int e = tid; e < 2 * CPC; e += kThreads) {
    const int k = e % CPC;
    if (k >= ct.n) continue;
    float v = 0.f;
    for (int r = 0; r < R; ++r) v += sm[((e / CPC) * R + r) * CPC + k];
    a.part_d[(((long long)b * a.n_piece + piece) * 2 + e / CPC) * a.D + ct.c0 + k] = v;
  }
}

// out[col] = sum of `rows` rows of `cols` values, kRowThreads threads per column
constexpr int kRowThreads = 16;
__global__ void __launch_bounds__(32 * kRowThreads) column_sum_kernel(const float* in, long long rows, long long cols,
                                                              long long split, float* o0, float* o1) {
  __shared__ float s[kRowThreads][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const long long col = (long long)blockIdx.x * 32 + x;
  float v = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (long long r = y; r < rows; r += kRowThreads) v += in[r * cols + col];
  }
  s[y][x] = v;
  __syncthreads();
  if (y || col >= cols) return;
#pragma unroll
  for (int i = 1; i < kRowThreads; ++i) v += s[i][x];
  if (col < split) {
    if (o0) o0[col] = v;
  } else if (o1) {
    o1[col - split] = v;
  }
}

// dB, dC [B,T,G,N] from the channel tiles' parts
template <typename T>
__global__ void __launch_bounds__(kThreads) scan_bc_kernel(ScanArgs a, int tiles) {
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;   // [B T][G][2N]
  const long long bt_n = (long long)a.B * a.T;
  if (e >= bt_n * a.G * 2 * a.N) return;
  long long q, bt;
  const int k = div_mod(e, 2 * a.N, q), g = div_mod(q, a.G, bt);
  const int per = tiles / a.G;
  float v = 0.f;
  const float* in = a.part_bc + ((long long)g * per * bt_n + bt) * 2 * a.N + k;
  const long long step = bt_n * 2 * a.N;
#pragma unroll 16
  for (int i = 0; i < per; ++i) v += in[i * step];
  T* o = static_cast<T*>(k < a.N ? a.g.dB : a.g.dC);
  o[(bt * a.G + g) * a.N + k % a.N] = from_f<T>(v);
}

// ------------------------------------------------------------------ one token

// Four states per lane as above; the state is read once and written once.  A thread owns
// one channel of kStepSeqs sequences, whose rates it reads once; all loads are issued before
// the first is used.
//   B256 D4096 N16 bf16 (143 MB): 32.8 us, 4.4 TB/s; two sequences 36.9, eight 59 us, the rates
//   read for every sequence 36.1.  64 % of the issue slots are taken (DRAM 41 %): each of a
//   channel's N / 4 lanes forms its time step and its gate.  Fewer rows were not tuned for:
//   B64 D4096 14 us, B16 D2048 8, B1 D2048 6.
constexpr int kStepSeqs = 4;

template <int N, typename T>
__global__ void __launch_bounds__(kThreads, 8) scan_step_kernel(ScanArgs a) {
  constexpr int LPC = N / 4, CPC = kThreads / LPC;
  __shared__ __align__(16) float s_bc[kStepSeqs][2 * N];
  const int blocks = (a.B + kStepSeqs - 1) / kStepSeqs, tiles = gridDim.x / blocks;
  const int b0 = blockIdx.x / tiles * kStepSeqs;
  const ChannelTile ct(a, CPC, blockIdx.x % tiles);
  const int tid = threadIdx.x, part = tid % LPC, k = tid / LPC, c = ct.c0 + k;
  const bool mine = k < ct.n;
  Four h[kStepSeqs];
  float x[kStepSeqs], dt[kStepSeqs], z[kStepSeqs];
#pragma unroll
  for (int r = 0; r < kStepSeqs; ++r) {
    const long long b = b0 + r;
    const bool real = mine && b < a.B;
    h[r] = real ? load4(a.h0 + (b * a.D + c) * N + 4 * part) : both(0);
    x[r] = real ? to_f<T>(static_cast<const T*>(a.x)[b * a.x_sb + c]) : 0.f;
    dt[r] = real ? to_f<T>(static_cast<const T*>(a.dt)[b * a.dt_sb + c]) : 0.f;
    z[r] = real && a.z ? to_f<T>(static_cast<const T*>(a.z)[b * a.z_sb + c]) : 0.f;
  }
  const f2 k2 = pack2(kLog2e, kLog2e);
  const Four A2 = mine ? mul(load4(a.A + (long long)c * N + 4 * part), k2) : both(0);
  const float bias = mine ? bias_of(a, c) : 0.f, skip = mine && a.Dskip ? a.Dskip[c] : 0.f;
  for (int e = tid; e < kStepSeqs * 2 * N; e += kThreads) {
    const int r = e / (2 * N), n = e % N;
    const long long b = min(b0 + r, a.B - 1);
    s_bc[r][e % (2 * N)] = to_f<T>(e % (2 * N) < N ? static_cast<const T*>(a.Bm)[b * a.B_sb + ct.g * N + n]
                                                   : static_cast<const T*>(a.Cm)[b * a.C_sb + ct.g * N + n]);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kStepSeqs; ++r) {
    const long long b = b0 + r;
    const Four B = load4(s_bc[r] + 4 * part), C = load4(s_bc[r] + N + 4 * part);
    float d = dt[r] + bias;
    if (a.softplus) d = softplus_f<T>(d);
    const float dx = d * x[r];
    h[r] = fma(decay(A2, pack2(d, d)), h[r], mul(B, pack2(dx, dx)));
    float y = dot(C, h[r]);
#pragma unroll
    for (int w = LPC / 2; w >= 1; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
    if (!mine || b >= a.B) continue;
    store4(a.hT + (b * a.D + c) * N + 4 * part, h[r]);
    if (part) continue;
    y += skip * x[r];
    if (a.z) y *= z[r] * sigmoid_f(z[r]);
    static_cast<T*>(a.y)[b * a.D + c] = from_f<T>(y);
  }
}

// ------------------------------------------------------------------ host side

unsigned blocks(long long n) { return static_cast<unsigned>((n + kThreads - 1) / kThreads); }

int tiles_of(int D, int G, int N) {
  const int cpc = 2 * kThreads / (N / 4);
  return G * ((D / G + cpc - 1) / cpc);
}

template <typename K>
cudaError_t launch(K kernel, long long grid, int smem, const ScanArgs& a, cudaStream_t st) {
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int N, typename T, bool VEC>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st) {
  const long long grid = (long long)tiles_of(a.D, a.G, N) * a.B * a.n_piece;
  cudaError_t e = cudaSuccess;
  if (a.n_piece > 1) {
    e = launch(scan_fwd_kernel<N, T, VEC, false>, grid, kWarps * FwdTile<N, T, false>::kBytes, a, st);
    if (e == cudaSuccess) e = launch(scan_join_kernel, blocks((long long)a.B * a.D * N), 0, a, st);
  }
  return e == cudaSuccess ? launch(scan_fwd_kernel<N, T, VEC, true>, grid, kWarps * FwdTile<N, T, true>::kBytes, a, st) : e;
}

template <int N, typename T, bool VEC>
cudaError_t bwd(ScanArgs a, int sms, cudaStream_t st) {
  const int tiles = tiles_of(a.D, a.G, N);
  const long long grid = (long long)tiles * a.B * a.n_piece;
  // a warp walks several pieces where there are many: its loads then go ahead from piece to
  // piece (one piece per warp 170 us, several 110; 4, 8 or 16 CTAs per SM make no difference)
  a.span = static_cast<int>(std::max(1LL, std::min<long long>(8, grid / (kEndsPerSM * sms))));
  cudaError_t e = launch(scan_bwd_ends_kernel<N, T, VEC>, (long long)tiles * a.B * ((a.n_piece + a.span - 1) / a.span),
                         kWarps * EndsTile<N, T>::kBytes, a, st);
  if (e == cudaSuccess) e = launch(scan_join_kernel, 2LL * blocks((long long)a.B * a.D * N), 0, a, st);
  if (e == cudaSuccess) e = launch(scan_bwd_kernel<N, T, VEC>, grid, bwd_smem<N, T>(), a, st);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.n_piece, cols = (long long)a.D * N;
  column_sum_kernel<<<static_cast<unsigned>((cols + 31) / 32), 32 * kRowThreads, 0, st>>>(a.hs, rows, cols, cols,
                                                                                   a.g.dA, nullptr);
  column_sum_kernel<<<(2 * a.D + 31) / 32, 32 * kRowThreads, 0, st>>>(a.part_d, rows, 2LL * a.D, a.D, a.g.dDskip,
                                                              a.g.ddt_bias);
  scan_bc_kernel<T><<<blocks((long long)a.B * a.T * a.G * 2 * N), kThreads, 0, st>>>(a, tiles);
  return cudaGetLastError();
}

template <int N, typename T>
cudaError_t step(const ScanArgs& a, cudaStream_t st) {
  constexpr int cpc = kThreads / (N / 4);
  const long long tiles = (long long)a.G * ((a.D / a.G + cpc - 1) / cpc);
  return launch(scan_step_kernel<N, T>, tiles * ((a.B + kStepSeqs - 1) / kStepSeqs), 0, a, st);
}

bool vec_ok(const ScanArgs& a, int dtype) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const long long v = dtype == DR_FP32 ? 4 : 8;
  return (a.D / a.G) % 8 == 0 &&
         (a.x_sb | a.x_st | a.dt_sb | a.dt_st | a.B_sb | a.B_st | a.C_sb | a.C_st) % v == 0 &&
         (!a.z || (a.z_sb | a.z_st) % v == 0) && al(a.x) && al(a.dt) && al(a.z) && al(a.Bm) && al(a.Cm) && al(a.y) &&
         al(a.d_y) && al(a.g.dx) && al(a.g.ddt) && al(a.g.dz);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

// Wide accesses where every row starts on 16 bytes, single values otherwise.
#define DR_SCAN_CASE(N_, CALL)                                                    \
  case N_:                                                                        \
    if (dtype == DR_FP32)                                                         \
      return vec_ok(a, dtype) ? CALL(N_, float, true) : CALL(N_, float, false);   \
    return vec_ok(a, dtype) ? CALL(N_, __nv_bfloat16, true) : CALL(N_, __nv_bfloat16, false);
#define DR_SCAN_DISPATCH(CALL) \
  switch (a.N) {               \
    DR_SCAN_CASE(8, CALL)      \
    DR_SCAN_CASE(16, CALL)     \
    DR_SCAN_CASE(32, CALL)     \
    DR_SCAN_CASE(64, CALL)     \
  }                            \
  return cudaErrorInvalidValue;

// Pieces along the tokens, each token walked twice, where rows (channel tiles x sequences)
// alone are fewer than 4/3 of the SMs: then for twelve CTAs per SM, of 64 tokens at least.
// D 2048, N 16, in pieces / in one pass: B1 T8192 160 / 901 us, B4 T2048 164 / 229,
// B6 (192 rows on 152 SMs) 248 / 284, B8 (256 rows) 321 / 284, B1 T512 21 / 58.
void scan_fwd_pieces(const ScanArgs& a, int sms, int* n_piece, int* piece) {
  const long long rows = (long long)tiles_of(a.D, a.G, a.N) * a.B;
  const int tile = 32;   // of tokens; pieces are whole tiles
  long long n = 12LL * sms / rows;
  const long long most = (a.T + 2 * tile - 1) / (2 * tile);
  if (n > most) n = most;
  *n_piece = 1, *piece = a.T;
  if (3 * rows > 4LL * sms || n < 3) return;
  const long long len = ((a.T + n - 1) / n + tile - 1) / tile * tile;
  *piece = static_cast<int>(len);
  *n_piece = static_cast<int>((a.T + len - 1) / len);
}

size_t scan_fwd_workspace(const ScanArgs& a, int sms) {
  int n, len;
  scan_fwd_pieces(a, sms, &n, &len);
  if (n == 1) return 0;
  const size_t rows = (size_t)a.B * n * a.D;
  return align256(4 * rows * a.N) + align256(4 * rows);
}

cudaError_t launch_scan_fwd(ScanArgs a, int dtype, int sms, void* workspace, cudaStream_t st) {
  a.n_piece = 1, a.piece = a.T;
  if (workspace) {
    scan_fwd_pieces(a, sms, &a.n_piece, &a.piece);
    char* p = static_cast<char*>(workspace);
    a.hs = reinterpret_cast<float*>(p);
    a.sum_dt = reinterpret_cast<float*>(p + align256((size_t)4 * a.B * a.n_piece * a.D * a.N));
  }
#define DR_CALL(N_, T_, V_) (fwd<N_, T_, V_>(a, st))
  DR_SCAN_DISPATCH(DR_CALL)
#undef DR_CALL
}

size_t scan_bwd_workspace(const ScanArgs& a) {
  const size_t rows = (size_t)a.B * ((a.T + kPiece - 1) / kPiece) * a.D;
  return 2 * align256(4 * rows * a.N) + align256(4 * rows) + align256(8 * rows) +
         align256((size_t)8 * tiles_of(a.D, a.G, a.N) * a.B * a.T * a.N);
}

cudaError_t launch_scan_bwd(ScanArgs a, int dtype, int sms, void* workspace, cudaStream_t st) {
  a.piece = kPiece;
  a.n_piece = (a.T + kPiece - 1) / kPiece;
  const size_t rows = (size_t)a.B * a.n_piece * a.D;
  char* p = static_cast<char*>(workspace);
  auto take = [&](size_t bytes) {
    float* f = reinterpret_cast<float*>(p);
    p += align256(bytes);
    return f;
  };
  a.hs = take(4 * rows * a.N);
  a.es = take(4 * rows * a.N);
  a.sum_dt = take(4 * rows);
  a.part_d = take(8 * rows);
  a.part_bc = take(0);
#define DR_CALL(N_, T_, V_) (bwd<N_, T_, V_>(a, sms, st))
  DR_SCAN_DISPATCH(DR_CALL)
#undef DR_CALL
}

cudaError_t launch_scan_step(const ScanArgs& a, int dtype, cudaStream_t st) {
#define DR_STEP(N_) \
  case N_: return dtype == DR_FP32 ? step<N_, float>(a, st) : step<N_, __nv_bfloat16>(a, st);
  switch (a.N) { DR_STEP(8) DR_STEP(16) DR_STEP(32) DR_STEP(64) }
#undef DR_STEP
  return cudaErrorInvalidValue;
}

}  // namespace dr
