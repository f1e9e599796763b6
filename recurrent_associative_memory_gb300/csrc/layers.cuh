// layers.cuh — argument blocks and device helpers of the layers next to the
// recurrence: window attention, short convolution, selective scan.
#pragma once

#include "dr_common.cuh"

namespace dr {

// ------------------------------------------------------------------ window attention

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int* lens;
  int B, T, S, H, Hkv, d, G;   // G = H / Hkv query heads per key/value head
  int window, n_sink, q_start; // window clamped to q_start + T
  int reach;                   // keys up to the last query's position: min(S, q_start + T)
  float scale;
  long long q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  // backward
  const void* d_out;
  void* dq;
  void* dk;
  void* dv;
  float* delta;                // fp32: [B,H,T] rowsum(dO * O); bf16: -delta [B,H,Tp]
  float* nlse2;                // bf16: -lse log2(e) [B,H,Tp], -infinity for rows that see nothing
  int Tp;                      // T rounded up to 64
  // bf16: the query rows from far_first on see nothing of key tile 0 but its sinks; their
  // part of the sinks' gradients is cut into n_far pieces of far_rows rows, which leave
  // [B,Hkv,1 + n_far][dk, dv][n_sink][d] (piece 0: from the rows before)
  int far_first, far_rows, n_far;
  float* sink_part;
};

__device__ __forceinline__ int real_len(const int* lens, int b, int n) {
  return lens ? max(0, min(lens[b], n)) : n;
}

__device__ __forceinline__ bool attn_sees(int p, int j, int len, int window, int n_sink) {
  return j <= p && j < len && (p - j < window || j < n_sink);
}

// The key tiles that the positions p0 .. p1 can see: those that hold a sink, then
// those of the window, each tile once.
struct KeyTiles {
  int n_first, w_begin, n;
  __device__ __forceinline__ KeyTiles(int p0, int p1, int len, int window, int n_sink, int tile) {
    const int hi = min(p1, len - 1);
    const int lo = max(0, p0 - window + 1);
    w_begin = lo / tile;
    const int n_win = hi >= lo ? hi / tile + 1 - w_begin : 0;
    const int sinks = max(0, min(n_sink, hi + 1));
    n_first = (sinks + tile - 1) / tile;
    if (n_win > 0) n_first = min(n_first, w_begin);
    n = n_first + n_win;
  }
  __device__ __forceinline__ int operator[](int i) const {
    return i < n_first ? i : w_begin + i - n_first;
  }
};

// The query rows that can see a key of j0 .. j1 (j1 inclusive): [begin, end).
struct QueryRows {
  int begin, end;
  __device__ __forceinline__ QueryRows(int j0, int j1, int len, int window, int n_sink, int q_start,
                                       int T) {
    begin = max(0, j0 - q_start);
    const long long last = j0 < n_sink ? (long long)T - 1
                                       : min((long long)T - 1, (long long)j1 + window - 1 - q_start);
    end = j0 < len ? static_cast<int>(last) + 1 : 0;
    if (end < begin) end = begin;
  }
};

// One token over the ring cache.
struct AttnStepArgs {
  const void* q;
  const void* k;
  const void* v;
  void* kc;
  void* vc;
  const int* pos;
  void* out;
  float* part;                 // o [B,H,pieces][d], then (m, l) [B,H,pieces]
  int B, H, Hkv, G, d, window, n_sink, n_piece;
  float scale;
};

// ------------------------------------------------------------------ convolution and scan

struct ConvArgs {
  const void* x;
  const float* w;
  const float* bias;
  const void* s0;
  void* y;
  void* s1;
  const int* lens;
  int B, T, D, K, silu;
  long long x_sb, x_st;
  // backward
  const void* d_y;
  const void* d_s1;
  void* dx;
  void* d_s0;
  float* part;
};

struct ScanArgs {
  const void* x;
  const void* dt;
  const void* Bm;
  const void* Cm;
  const void* z;
  const float* h0;
  void* y;
  float* hT;
  const int* lens;
  const float* A;
  const float* Dskip;
  const float* bias;
  int B, T, D, N, G, softplus;
  long long x_sb, x_st, dt_sb, dt_st, z_sb, z_st, B_sb, B_st, C_sb, C_st;
  // pieces along the tokens: number and length, the state at each piece's start
  // (first: at its end, from zero) and the sum of its time steps
  int n_piece, piece;
  int span;                    // pieces that a warp of the backward's first pass walks
  float* hs;
  float* sum_dt;
  // backward
  const void* d_y;
  const float* d_hT;
  dr_scan_grads g;
  float* es;                   // the state's gradient at each piece's end
  float* part_bc;              // [channel tiles][B][T][2N]
  float* part_d;               // [B][pieces][2][D]: of Dskip and dt_bias
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// q = e / d, returns e mod d (e >= 0): short where it fits, a long division takes a hundred
// instructions
__device__ __forceinline__ int div_mod(long long e, int d, long long& q) {
  if (e >> 31 == 0) {
    const uint32_t u = static_cast<uint32_t>(e), r = u / static_cast<uint32_t>(d);
    q = r;
    return static_cast<int>(u - r * static_cast<uint32_t>(d));
  }
  q = e / d;
  return static_cast<int>(e - q * d);
}

// Two fp32 values in one register pair, and the arithmetic that takes both at once.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ float sum2(f2 v) {
  float x, y;
  unpack2(v, x, y);
  return x + y;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
  float x, y;
  unpack2(v, x, y);
  return pack2(ex2(x), ex2(y));
}

__device__ __forceinline__ float sigmoid_f(float x) {   // far below zero: 1 / infinity = 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x * -1.4426950408889634f)));
  return r;
}

// 8 consecutive values, 16-byte aligned, to fp32; zeros where n <= 0
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[8]) {
  if (n <= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
  } else if constexpr (sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

}  // namespace dr
