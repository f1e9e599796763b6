// selective_scan.cu — selective state space scan: forward, backward, one token.
//
//   h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] B_t[n] x_t[c]
//   y_t[c]   = sum_n C_t[n] h_t[c,n] + D[c] x_t[c],  gated by z sigmoid(z)
//
// Per (token, channel, state): one exponential, two products, two multiply-adds;
// the exponential units and the issue slots bound it, not the bytes.  N / 4
// neighbouring lanes own a channel, four states each in registers, and walk the
// tokens; B_t and C_t are the same for all channels of a group and come from shared
// memory as broadcast reads.  The lanes' parts of y are summed for N / 4 tokens at
// once by exchanging halves (N / 4 - 1 shuffles for N / 4 tokens).
//
// Few rows and many tokens are cut into pieces along the tokens: over a piece the
// state is h_end = exp(A sum dt) h_start + (end from zero), so a first pass takes
// every piece's end from zero and its sum of dt, a scan joins them, and the second
// pass starts every piece from its true state.
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
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;     // tokens in shared memory at a time (forward)
constexpr int kPiece = 64;    // tokens of a backward piece
constexpr int kSub = 8;       // tokens whose states are in registers (backward)
constexpr float kLog2e = 1.4426950408889634f;

template <int N> struct Shape {
  static constexpr int LPC = N / 4;            // lanes per channel
  static constexpr int CPC = kThreads / LPC;   // channels per CTA
  static constexpr int CW = 32 / LPC;          // channels per warp
};

__device__ __forceinline__ float softplus_f(float v) { return v > 20.f ? v : log1pf(__expf(v)); }

// 8 neighbouring values as loaded
template <typename T> struct alignas(16) Raw8 { T v[8]; };

template <typename T, bool VEC>
__device__ __forceinline__ void fetch8(Raw8<T>& r, const T* p, int n) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(r.v)[i] =
          n > 0 ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < n ? p[i] : from_f<T>(0.f);
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

template <int N>
__device__ __forceinline__ void load_rates(const ScanArgs& a, int c, bool real, int part, float (&A)[4]) {
  const float4 v = real ? *reinterpret_cast<const float4*>(a.A + (long long)c * N + 4 * part)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  A[0] = v.x, A[1] = v.y, A[2] = v.z, A[3] = v.w;
}

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}

// ------------------------------------------------------------------ forward

// FULL: outputs from the state at the piece's start; otherwise the piece's end from
// zero and its sum of dt.
template <int N, typename T, bool VEC, bool FULL>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanArgs a) {
  using S = Shape<N>;
  constexpr int CPC = S::CPC, LPC = S::LPC;
  constexpr int NV = (kTile * CPC / 8 + kThreads - 1) / kThreads;   // 8-value loads per thread
  __shared__ float2 s_u[kTile][CPC];                                // dt, dt x
  __shared__ float s_y[FULL ? kTile : 1][CPC];
  __shared__ __align__(16) float s_B[kTile][N], s_C[kTile][N];
  const int tid = threadIdx.x, lane = tid % 32, part = tid % LPC, ch = tid / LPC;
  const int tiles = gridDim.x / (a.B * a.n_piece);
  const ChannelTile ct(a, CPC, blockIdx.x % tiles);
  const int piece = (blockIdx.x / tiles) % a.n_piece, b = blockIdx.x / tiles / a.n_piece;
  const int t_begin = piece * a.piece, t_end = min(a.T, t_begin + a.piece);
  const int len = real_len(a.lens, b, a.T);
  const bool real = ch < ct.n;
  const int c = ct.c0 + ch;

  float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  load_rates<N>(a, c, real, part, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
  if (FULL && real) {
    if (a.n_piece > 1)
      load4(a.hs + (((long long)b * a.n_piece + piece) * a.D + c) * N + 4 * part, h);
    else if (a.h0)
      load4(a.h0 + ((long long)b * a.D + c) * N + 4 * part, h);
  }

  // this thread's loads of a tile: token vt, channels vc .. vc + 7 of the tile
  Raw8<T> rx[NV], rd[NV], rz[NV];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * kThreads, vt = v / (CPC / 8), vc = 8 * (v % (CPC / 8));
      const int t = t0 + vt, n = vt < kTile && t < t_end ? ct.n - vc : 0;
      fetch8<T, VEC>(rx[i], static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + ct.c0 + vc, n);
      fetch8<T, VEC>(rd[i], static_cast<const T*>(a.dt) + b * a.dt_sb + t * a.dt_st + ct.c0 + vc, n);
      if (FULL && a.z)
        fetch8<T, VEC>(rz[i], static_cast<const T*>(a.z) + b * a.z_sb + t * a.z_st + ct.c0 + vc, n);
    }
  };
  fetch(t_begin);
  for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
    Raw8<T> cx[NV], cz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * kThreads, vt = v / (CPC / 8), vc = 8 * (v % (CPC / 8));
      if (vt >= kTile) break;
      const bool in = t0 + vt < min(len, t_end);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool ok = in && vc + k < ct.n;
        float d = ok ? to_f<T>(rd[i].v[k]) + (a.bias ? a.bias[ct.c0 + vc + k] : 0.f) : 0.f;
        if (a.softplus) d = softplus_f(d);
        if (!ok) d = 0.f;
        s_u[vt][vc + k] = make_float2(d, ok ? d * to_f<T>(rx[i].v[k]) : 0.f);
      }
      cx[i] = rx[i], cz[i] = rz[i];
    }
    for (int e = tid; e < kTile * N; e += kThreads) {
      const int t = t0 + e / N, n = e % N;
      const bool in = t < t_end;
      s_B[e / N][n] = in ? to_f<T>(static_cast<const T*>(a.Bm)[b * a.B_sb + t * a.B_st + ct.g * N + n]) : 0.f;
      if (FULL)
        s_C[e / N][n] = in ? to_f<T>(static_cast<const T*>(a.Cm)[b * a.C_sb + t * a.C_st + ct.g * N + n]) : 0.f;
    }
    __syncthreads();
    if (t0 + kTile < t_end) fetch(t0 + kTile);
#pragma unroll 1
    for (int g = 0; g < kTile; g += LPC) {
      float y[LPC];
#pragma unroll
      for (int k = 0; k < LPC; ++k) {
        const float2 u = s_u[g + k][ch];
        float B[4], C[4];
        load4(&s_B[g + k][4 * part], B);
        if (FULL) load4(&s_C[g + k][4 * part], C);
        if (!FULL) sum += u.x;
        y[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = ex2(u.x * A2[i]) * h[i] + u.y * B[i];
          if (FULL) y[k] += C[i] * h[i];
        }
      }
      if (FULL) {
        lane_sums<LPC, LPC, 1>(y, lane);
        s_y[g + part][ch] = y[0];
      }
    }
    __syncthreads();
    if (FULL) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * kThreads, vt = v / (CPC / 8), vc = 8 * (v % (CPC / 8));
        const int t = t0 + vt;
        if (vt >= kTile || t >= t_end || vc >= ct.n) break;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool ok = t < len && vc + k < ct.n;
          o[k] = ok ? s_y[vt][vc + k] + (a.Dskip ? a.Dskip[ct.c0 + vc + k] * to_f<T>(cx[i].v[k]) : 0.f) : 0.f;
          if (a.z && ok) {
            const float z = to_f<T>(cz[i].v[k]);
            o[k] *= z * sigmoid_f(z);
          }
        }
        store8<T, VEC>(static_cast<T*>(a.y) + ((long long)b * a.T + t) * a.D + ct.c0 + vc, ct.n - vc, o);
      }
    }
  }
  if (!real) return;
  const float4 hv = make_float4(h[0], h[1], h[2], h[3]);
  if (!FULL) {
    const long long row = ((long long)b * a.n_piece + piece) * a.D + c;
    *reinterpret_cast<float4*>(a.hs + row * N + 4 * part) = hv;
    if (part == 0) a.sum_dt[row] = sum;
  } else if (a.hT && piece == a.n_piece - 1) {
    *reinterpret_cast<float4*>(a.hT + ((long long)b * a.D + c) * N + 4 * part) = hv;
  }
}

// Joins the pieces: hs becomes the state at each piece's start; BWD: es the gradient
// at each piece's end, and the gradient of the initial state.
template <bool BWD>
__global__ void __launch_bounds__(kThreads) scan_join_kernel(ScanArgs a) {
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x, per = (long long)a.D * a.N;
  if (e >= a.B * per) return;
  const long long b = e / per, cn = e % per, c = cn / a.N;
  const float A2 = a.A[cn] * kLog2e;
  float h = a.h0 ? a.h0[e] : 0.f;
#pragma unroll 4
  for (int p = 0; p < a.n_piece; ++p) {
    const long long row = b * a.n_piece + p;
    float* s = a.hs + row * per + cn;
    const float end = *s;
    *s = h;
    h = ex2(A2 * a.sum_dt[row * a.D + c]) * h + end;
  }
  if (!BWD) return;
  float g = a.d_hT ? a.d_hT[e] : 0.f;
#pragma unroll 4
  for (int p = a.n_piece - 1; p >= 0; --p) {
    const long long row = b * a.n_piece + p;
    float* s = a.es + row * per + cn;
    const float start = *s;
    *s = g;
    g = ex2(A2 * a.sum_dt[row * a.D + c]) * g + start;
  }
  if (a.g.d_init_state) a.g.d_init_state[e] = g;
}

// ------------------------------------------------------------------ backward

// One piece's tokens in shared memory: (dt, dt x), dy behind the gate, B and C.
template <int N, typename T, bool VEC>
__device__ __forceinline__ void load_piece(const ScanArgs& a, const ChannelTile& ct, int b, int t0, int len,
                                           float2* s_u, float* s_dy, float* s_B, float* s_C) {
  constexpr int CPC = Shape<N>::CPC;
  const int tid = threadIdx.x;
  for (int v = tid; v < kPiece * CPC / 8; v += kThreads) {
    const int vt = v / (CPC / 8), vc = 8 * (v % (CPC / 8)), t = t0 + vt;
    const int n = t < len ? ct.n - vc : 0;
    Raw8<T> rx, rd, rg, rz;
    fetch8<T, VEC>(rx, static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + ct.c0 + vc, n);
    fetch8<T, VEC>(rd, static_cast<const T*>(a.dt) + b * a.dt_sb + t * a.dt_st + ct.c0 + vc, n);
    fetch8<T, VEC>(rg, static_cast<const T*>(a.d_y) + ((long long)b * a.T + t) * a.D + ct.c0 + vc, n);
    if (a.z) fetch8<T, VEC>(rz, static_cast<const T*>(a.z) + b * a.z_sb + t * a.z_st + ct.c0 + vc, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool ok = k < n;
      float d = ok ? to_f<T>(rd.v[k]) + (a.bias ? a.bias[ct.c0 + vc + k] : 0.f) : 0.f;
      if (a.softplus) d = softplus_f(d);
      if (!ok) d = 0.f;
      s_u[vt * CPC + vc + k] = make_float2(d, ok ? d * to_f<T>(rx.v[k]) : 0.f);
      float g = ok ? to_f<T>(rg.v[k]) : 0.f;
      if (a.z && ok) {
        const float z = to_f<T>(rz.v[k]);
        g *= z * sigmoid_f(z);
      }
      s_dy[vt * CPC + vc + k] = g;
    }
  }
  for (int e = tid; e < kPiece * N; e += kThreads) {
    const int t = t0 + e / N, n = e % N;
    const bool in = t < len;
    s_B[e] = in ? to_f<T>(static_cast<const T*>(a.Bm)[b * a.B_sb + t * a.B_st + ct.g * N + n]) : 0.f;
    s_C[e] = in ? to_f<T>(static_cast<const T*>(a.Cm)[b * a.C_sb + t * a.C_st + ct.g * N + n]) : 0.f;
  }
}

template <int N> constexpr int piece_floats() {   // of load_piece
  return kPiece * (3 * Shape<N>::CPC + 2 * N);
}

// A piece's end state from zero, the gradient that reaches its start, its sum of dt.
template <int N, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_bwd_ends_kernel(ScanArgs a) {
  using S = Shape<N>;
  constexpr int CPC = S::CPC, LPC = S::LPC;
  extern __shared__ __align__(16) float sm[];
  float2* s_u = reinterpret_cast<float2*>(sm);
  float* s_dy = sm + 2 * kPiece * CPC;
  float* s_B = s_dy + kPiece * CPC;
  float* s_C = s_B + kPiece * N;
  const int tid = threadIdx.x, part = tid % LPC, ch = tid / LPC;
  const int tiles = gridDim.x / (a.B * a.n_piece);
  const ChannelTile ct(a, CPC, blockIdx.x % tiles);
  const int piece = (blockIdx.x / tiles) % a.n_piece, b = blockIdx.x / tiles / a.n_piece;
  const int c = ct.c0 + ch;
  float A2[4], h[4] = {}, e[4] = {}, cp[4] = {1.f, 1.f, 1.f, 1.f}, sum = 0.f;
  load_rates<N>(a, c, ch < ct.n, part, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
  load_piece<N, T, VEC>(a, ct, b, piece * kPiece, real_len(a.lens, b, a.T), s_u, s_dy, s_B, s_C);
  __syncthreads();
#pragma unroll 4
  for (int t = 0; t < kPiece; ++t) {
    const float2 u = s_u[t * CPC + ch];
    const float dy = s_dy[t * CPC + ch];
    float B[4], C[4];
    load4(s_B + t * N + 4 * part, B);
    load4(s_C + t * N + 4 * part, C);
    sum += u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = ex2(u.x * A2[i]);
      h[i] = x * h[i] + u.y * B[i];
      cp[i] *= x;
      e[i] += cp[i] * (C[i] * dy);
    }
  }
  if (ch >= ct.n) return;
  const long long row = ((long long)b * a.n_piece + piece) * a.D + c;
  *reinterpret_cast<float4*>(a.hs + row * N + 4 * part) = make_float4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<float4*>(a.es + row * N + 4 * part) = make_float4(e[0], e[1], e[2], e[3]);
  if (part == 0) a.sum_dt[row] = sum;
}

template <int N> constexpr int bwd_smem() {
  using S = Shape<N>;
  return 4 * (piece_floats<N>() + kPiece * S::CPC + kWarps * kSub * 2 * N + 4 * kThreads * (kPiece / kSub));
}

template <int N, typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanArgs a) {
  using S = Shape<N>;
  constexpr int CPC = S::CPC, LPC = S::LPC, CW = S::CW;
  constexpr int TG = LPC < kSub ? LPC : kSub;   // tokens whose sums over a channel's lanes go together
  extern __shared__ __align__(16) float sm[];
  float2* s_u = reinterpret_cast<float2*>(sm);         // (dt, dt x), then (sum g B, sum e A)
  float* s_dy = sm + 2 * kPiece * CPC;
  float* s_B = s_dy + kPiece * CPC;
  float* s_C = s_B + kPiece * N;
  float* s_y = s_C + kPiece * N;                       // sum_n C h
  float* s_bc = s_y + kPiece * CPC;                    // [warp][kSub][2N] sums over a warp's channels
  float4* s_h = reinterpret_cast<float4*>(s_bc + kWarps * kSub * 2 * N);   // states at the sub-tiles' starts
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = tid % LPC, ch = tid / LPC;
  const int tiles = gridDim.x / (a.B * a.n_piece);
  const int tile = blockIdx.x % tiles;
  const ChannelTile ct(a, CPC, tile);
  const int piece = (blockIdx.x / tiles) % a.n_piece, b = blockIdx.x / tiles / a.n_piece;
  const int t0 = piece * kPiece, len = real_len(a.lens, b, a.T);
  const int c = ct.c0 + ch;
  const bool real = ch < ct.n;
  const long long row = ((long long)b * a.n_piece + piece) * a.D + c;
  float A[4], A2[4], h[4] = {}, gc[4] = {}, dA[4] = {};
  load_rates<N>(a, c, real, part, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = A[i] * kLog2e;
  if (real) {
    load4(a.hs + row * N + 4 * part, h);
    load4(a.es + row * N + 4 * part, gc);
  }
  load_piece<N, T, VEC>(a, ct, b, t0, len, s_u, s_dy, s_B, s_C);
  __syncthreads();
  // the state at each sub-tile's start
  for (int s = 0; s < kPiece / kSub; ++s) {
    s_h[s * kThreads + tid] = make_float4(h[0], h[1], h[2], h[3]);
    if (s == kPiece / kSub - 1) break;
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      const int t = s * kSub + k;
      const float2 u = s_u[t * CPC + ch];
      float B[4];
      load4(s_B + t * N + 4 * part, B);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = ex2(u.x * A2[i]) * h[i] + u.y * B[i];
    }
  }
  for (int s = kPiece / kSub - 1; s >= 0; --s) {
    float hh[kSub + 1][4];   // hh[k]: the state before token k
    const float4 hv = s_h[s * kThreads + tid];
    hh[0][0] = hv.x, hh[0][1] = hv.y, hh[0][2] = hv.z, hh[0][3] = hv.w;
#pragma unroll
    for (int g = 0; g < kSub; g += TG) {
      float y[TG];
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const int t = s * kSub + g + k;
        const float2 u = s_u[t * CPC + ch];
        float B[4], C[4];
        load4(s_B + t * N + 4 * part, B);
        load4(s_C + t * N + 4 * part, C);
        y[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hh[g + k + 1][i] = ex2(u.x * A2[i]) * hh[g + k][i] + u.y * B[i];
          y[k] += C[i] * hh[g + k + 1][i];
        }
      }
      lane_sums<TG, LPC, 1>(y, lane);
      s_y[(s * kSub + g + part * TG / LPC) * CPC + ch] = y[0];
    }
    __syncthreads();   // the last sub-tile's s_bc has been read
#pragma unroll
    for (int g = kSub - TG; g >= 0; g -= TG) {
      float q[2 * TG];   // token k: sum g B, sum e A
#pragma unroll
      for (int k = TG - 1; k >= 0; --k) {
        const int t = s * kSub + g + k;
        const float2 u = s_u[t * CPC + ch];
        const float dy = s_dy[t * CPC + ch];
        float B[4], C[4], v[8];
        load4(s_B + t * N + 4 * part, B);
        load4(s_C + t * N + 4 * part, C);
        q[2 * k] = q[2 * k + 1] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gi = gc[i] + C[i] * dy;
          q[2 * k] += gi * B[i];
          v[i] = gi * u.y;
          v[4 + i] = hh[g + k + 1][i] * dy;
          gc[i] = gi * ex2(u.x * A2[i]);
          const float e = gc[i] * hh[g + k][i];
          q[2 * k + 1] += e * A[i];
          dA[i] += e * u.x;
        }
        lane_sums<8, CW, LPC>(v, lane);
        float* bc = s_bc + (warp * kSub + g + k) * 2 * N + 4 * part;
        constexpr int PER = 8 / CW > 0 ? 8 / CW : 1;   // values a lane ends with
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int idx = CW <= 8 ? (lane / LPC) * PER + i : (lane / LPC) / (CW / 8);
          bc[(idx / 4) * N + idx % 4] = v[i];
        }
      }
      lane_sums<2 * TG, LPC, 1>(q, lane);
      constexpr int PER = 2 * TG / LPC;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int idx = part * PER + i;
        reinterpret_cast<float*>(s_u + (s * kSub + g + idx / 2) * CPC + ch)[idx % 2] = q[i];
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
  if (real)
    *reinterpret_cast<float4*>(a.hs + row * N + 4 * part) = make_float4(dA[0], dA[1], dA[2], dA[3]);
  // dx, ddt, dz of 8 channels per thread and token; the sums over the piece for dD and d bias
  float sd[8] = {}, sb[8] = {};
  const int vc = 8 * (tid % (CPC / 8)), n = ct.n - vc;
  for (int vt = tid / (CPC / 8); vt < kPiece; vt += kThreads / (CPC / 8)) {
    const int t = t0 + vt;
    if (t >= a.T || n <= 0) break;
    const int nr = t < len ? n : 0;
    float x[8], d[8], gy[8], z[8], dx[8], ddt[8], dz[8];
    load8<T, VEC>(static_cast<const T*>(a.x) + b * a.x_sb + t * a.x_st + ct.c0 + vc, nr, x);
    load8<T, VEC>(static_cast<const T*>(a.dt) + b * a.dt_sb + t * a.dt_st + ct.c0 + vc, nr, d);
    load8<T, VEC>(static_cast<const T*>(a.d_y) + ((long long)b * a.T + t) * a.D + ct.c0 + vc, nr, gy);
    if (a.z) load8<T, VEC>(static_cast<const T*>(a.z) + b * a.z_sb + t * a.z_st + ct.c0 + vc, nr, z);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool ok = k < nr;
      const float2 q = s_u[vt * CPC + vc + k];
      const float skip = ok && a.Dskip ? a.Dskip[ct.c0 + vc + k] : 0.f;
      const float raw = d[k] + (ok && a.bias ? a.bias[ct.c0 + vc + k] : 0.f);
      const float dt = a.softplus ? softplus_f(raw) : raw;
      float dy = gy[k];
      if (a.z) {
        const float sg = sigmoid_f(z[k]), y = s_y[vt * CPC + vc + k] + skip * x[k];
        dz[k] = ok ? gy[k] * y * sg * (1.f + z[k] * (1.f - sg)) : 0.f;
        dy *= z[k] * sg;
      }
      dx[k] = ok ? q.x * dt + skip * dy : 0.f;
      ddt[k] = ok ? (q.y + q.x * x[k]) * (a.softplus ? sigmoid_f(raw) : 1.f) : 0.f;
      sd[k] += ok ? dy * x[k] : 0.f;
      sb[k] += ddt[k];
    }
    const long long o = ((long long)b * a.T + t) * a.D + ct.c0 + vc;
    store8<T, VEC>(static_cast<T*>(a.g.dx) + o, n, dx);
    store8<T, VEC>(static_cast<T*>(a.g.ddt) + o, n, ddt);
    if (a.z) store8<T, VEC>(static_cast<T*>(a.g.dz) + o, n, dz);
  }
  __syncthreads();
  constexpr int R = kThreads / (CPC / 8);   // rows of partial sums, over the piece's buffers
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    sm[(tid / (CPC / 8)) * CPC + vc + k] = sd[k];
    sm[(R + tid / (CPC / 8)) * CPC + vc + k] = sb[k];
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

// out[col] = sum of `rows` rows of `cols` values, 8 threads per column
__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float* in, long long rows, long long cols,
                                                              long long split, float* o0, float* o1) {
  __shared__ float s[8][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const long long col = (long long)blockIdx.x * 32 + x;
  float v = 0.f;
  if (col < cols)
    for (long long r = y; r < rows; r += 8) v += in[r * cols + col];
  s[y][x] = v;
  __syncthreads();
  if (y || col >= cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += s[i][x];
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
  const int k = e % (2 * a.N), g = (e / (2 * a.N)) % a.G;
  const long long bt = e / (2 * a.N) / a.G;
  const int per = tiles / a.G;
  float v = 0.f;
  for (int i = 0; i < per; ++i) v += a.part_bc[((g * per + i) * bt_n + bt) * 2 * a.N + k];
  T* o = static_cast<T*>(k < a.N ? a.g.dB : a.g.dC);
  o[(bt * a.G + g) * a.N + k % a.N] = from_f<T>(v);
}

// ------------------------------------------------------------------ one token

// Four states per lane as above; the state is read once and written once.
template <int N, typename T>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  constexpr int LPC = N / 4;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;   // [B][D][LPC]
  const bool real = e < (long long)a.B * a.D * LPC;
  const long long bc = (real ? e : 0) / LPC;
  const int part = e % LPC, c = bc % a.D, b = bc / a.D, g = c / (a.D / a.G);
  float h[4], A[4];
  load4(a.h0 + bc * N + 4 * part, h);
  load4(a.A + (long long)c * N + 4 * part, A);
  const T* Bp = static_cast<const T*>(a.Bm) + b * a.B_sb + g * N + 4 * part;
  const T* Cp = static_cast<const T*>(a.Cm) + b * a.C_sb + g * N + 4 * part;
  const float x = to_f<T>(static_cast<const T*>(a.x)[b * a.x_sb + c]);
  float dt = to_f<T>(static_cast<const T*>(a.dt)[b * a.dt_sb + c]) + (a.bias ? a.bias[c] : 0.f);
  if (a.softplus) dt = softplus_f(dt);
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = ex2(dt * A[i] * kLog2e) * h[i] + dt * x * to_f<T>(Bp[i]);
    y += to_f<T>(Cp[i]) * h[i];
  }
#pragma unroll
  for (int w = LPC / 2; w >= 1; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
  if (!real) return;
  *reinterpret_cast<float4*>(a.hT + bc * N + 4 * part) = make_float4(h[0], h[1], h[2], h[3]);
  if (part) return;
  if (a.Dskip) y += a.Dskip[c] * x;
  if (a.z) {
    const float z = to_f<T>(static_cast<const T*>(a.z)[b * a.z_sb + c]);
    y *= z * sigmoid_f(z);
  }
  static_cast<T*>(a.y)[bc] = from_f<T>(y);
}

// ------------------------------------------------------------------ host side

unsigned blocks(long long n) { return static_cast<unsigned>((n + kThreads - 1) / kThreads); }

int tiles_of(int D, int G, int N) {
  const int cpc = kThreads / (N / 4);
  return G * ((D / G + cpc - 1) / cpc);
}

template <int N, typename T, bool VEC>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((long long)tiles_of(a.D, a.G, N) * a.B * a.n_piece);
  if (a.n_piece > 1) {
    scan_fwd_kernel<N, T, VEC, false><<<grid, kThreads, 0, st>>>(a);
    scan_join_kernel<false><<<blocks((long long)a.B * a.D * N), kThreads, 0, st>>>(a);
  }
  scan_fwd_kernel<N, T, VEC, true><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int N, typename T, bool VEC>
cudaError_t bwd(const ScanArgs& a, cudaStream_t st) {
  const int tiles = tiles_of(a.D, a.G, N);
  const unsigned grid = static_cast<unsigned>((long long)tiles * a.B * a.n_piece);
  constexpr int smem_ends = 4 * piece_floats<N>(), smem = bwd_smem<N>();
  cudaError_t e = cudaFuncSetAttribute(scan_bwd_ends_kernel<N, T, VEC>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem_ends);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(scan_bwd_kernel<N, T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  scan_bwd_ends_kernel<N, T, VEC><<<grid, kThreads, smem_ends, st>>>(a);
  scan_join_kernel<true><<<blocks((long long)a.B * a.D * N), kThreads, 0, st>>>(a);
  scan_bwd_kernel<N, T, VEC><<<grid, kThreads, smem, st>>>(a);
  const long long rows = (long long)a.B * a.n_piece, cols = (long long)a.D * N;
  column_sum_kernel<<<static_cast<unsigned>((cols + 31) / 32), kThreads, 0, st>>>(a.hs, rows, cols, cols,
                                                                                   a.g.dA, nullptr);
  column_sum_kernel<<<(2 * a.D + 31) / 32, kThreads, 0, st>>>(a.part_d, rows, 2LL * a.D, a.D, a.g.dDskip,
                                                              a.g.ddt_bias);
  scan_bc_kernel<T><<<blocks((long long)a.B * a.T * a.G * 2 * N), kThreads, 0, st>>>(a, tiles);
  return cudaGetLastError();
}

template <int N, typename T>
cudaError_t step(const ScanArgs& a, cudaStream_t st) {
  scan_step_kernel<N, T><<<blocks((long long)a.B * a.D * (N / 4)), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool vec_ok(const ScanArgs& a, int dtype) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int v = dtype == DR_FP32 ? 4 : 8;
  return (a.D / a.G) % 8 == 0 && a.x_sb % v == 0 && a.x_st % v == 0 && a.dt_sb % v == 0 && a.dt_st % v == 0 &&
         (!a.z || (a.z_sb % v == 0 && a.z_st % v == 0)) && al(a.x) && al(a.dt) && al(a.z) && al(a.y) &&
         al(a.d_y) && al(a.g.dx) && al(a.g.ddt) && al(a.g.dz);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

// 16-byte accesses where every row starts on 16 bytes, single values otherwise.
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

// Pieces along the tokens: where the rows give fewer than half the SMs a CTA.
void scan_fwd_pieces(const ScanArgs& a, int sms, int* n_piece, int* piece) {
  const long long rows = (long long)tiles_of(a.D, a.G, a.N) * a.B;
  long long n = 2LL * sms / rows;
  const long long most = (a.T + 2 * kTile - 1) / (2 * kTile);
  if (n > most) n = most;
  *n_piece = 1, *piece = a.T;
  if (n < 4) return;
  const long long len = ((a.T + n - 1) / n + kTile - 1) / kTile * kTile;
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

cudaError_t launch_scan_bwd(ScanArgs a, int dtype, void* workspace, cudaStream_t st) {
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
#define DR_CALL(N_, T_, V_) (bwd<N_, T_, V_>(a, st))
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
