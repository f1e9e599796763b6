// attn_simt.cu — window attention with sinks on fp32 CUDA cores: forward, dQ, and
// dK / dV.  Every product is an fp32 multiply-add, so the fp32 type keeps its full
// precision.
//
// One CTA of 256 threads owns 64 query rows of a head (dK / dV: 64 keys of a
// key/value head) and walks the 64-wide tiles of the other axis that it can see.
// Thread (ty, tx) of a 16 x 16 grid holds the products of rows ty + 16 i and
// columns tx + 16 j (i, j < 4); tiles in shared memory have a row pitch of d + 4
// floats, so the 16-byte reads of eight neighbouring rows meet eight different
// groups of banks.
//   forward: the running maximum m and sum l of a row (shared by its 16 threads),
//     o <- o exp(m - m') + P V;  lse = m + log l
//   dQ: P = exp(s - lse), dS = P (dO V^T - delta), dQ += dS K
//   dK, dV over the query heads of the group: dV += P^T dO, dK += dS^T Q
// The reads of shared memory bound it: 8 of 16 bytes for 64 multiply-adds of a thread (6 for
// 32 at 32 rows).  fp32, B4 H8 T1024 d64, window 257: forward 115 us, 17 TFLOP/s, backward 459;
// B2 T4096 H16 over 4 d128, window 512: 1215 and 7270.
// bf16 with strides that no tensor map holds comes here too (everything fp32 but the
// operands as loaded and the outputs): the second forward, keys expanded over the batch, takes
// 1190 us where the tensor cores take 57.
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kT = 64;        // tile: rows and columns
constexpr int kThreads = 256;

template <int D> constexpr int pitch() { return D + 4; }
constexpr int kPP = kT + 4;   // row pitch of the P / dS tile

// rows [r0, r0 + ROWS) of a strided [*, D] matrix to shared memory as fp32; rows at or past
// n read as zero.  fetch() loads them, put() stores them: what lies between hides the way.
template <int D, typename T, int ROWS = kT> struct Tile {
  static constexpr int NC = ROWS * D / 8 / kThreads;   // 8 values at a time
  static_assert(NC * kThreads * 8 == ROWS * D, "whole rounds of loads");
  const int tid = threadIdx.x % kThreads;
  float f[NC][8];
  __device__ __forceinline__ void fetch(const T* src, long long st, int r0, int n) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int e = tid + i * kThreads, r = r0 + e / (D / 8);
      load8<T>(src + (long long)r * st + 8 * (e % (D / 8)), r < n ? 8 : 0, f[i]);
    }
  }
  __device__ __forceinline__ void put(float* dst) const {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int e = tid + i * kThreads;
      float* p = dst + e / (D / 8) * pitch<D>() + 8 * (e % (D / 8));
      *reinterpret_cast<float4*>(p) = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
    }
  }
};
template <int D, typename T, int ROWS = kT>
__device__ __forceinline__ void load_tile(float* dst, const T* src, long long st, int r0, int n) {
  Tile<D, T, ROWS> t;
  t.fetch(src, st, r0, n);
  t.put(dst);
}

// s[i][j] = sum_c a[ty + 16 i][c] b[tx + 16 j][c]
template <int D, int RI>
__device__ __forceinline__ void product_abt(float (&s)[RI][4], const float* a, const float* b, int ty,
                                            int tx) {
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[RI], y[4];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty + 16 * i) * pitch<D>() + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * pitch<D>() + c);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
  }
}

// o[i][..] += sum_r p[ty + 16 i][r] b[r][columns of tx]; the columns of tx are
// 4 tx + 64 m (m < D / 64)
template <int D, int RI>
__device__ __forceinline__ void product_pb(float (&o)[RI][D / 16], const float* p, const float* b, int ty,
                                           int tx) {
#pragma unroll 2
  for (int r0 = 0; r0 < kT; r0 += 4) {
    float w[RI][4];
#pragma unroll
    for (int i = 0; i < RI; ++i)
      *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(p + (ty + 16 * i) * kPP + r0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int m = 0; m < D / 64; ++m) {
        const float4 y = *reinterpret_cast<const float4*>(b + (r0 + r) * pitch<D>() + 4 * tx + 64 * m);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          o[i][4 * m] += w[i][r] * y.x;
          o[i][4 * m + 1] += w[i][r] * y.y;
          o[i][4 * m + 2] += w[i][r] * y.z;
          o[i][4 * m + 3] += w[i][r] * y.w;
        }
      }
  }
}

// o[i][..] = o[i][..] f[i] + that sum.  Sums go over thousands of terms (a key's over G heads x
// the rows that see it); one after the other, n terms leave an error of about sqrt(n / 6) units,
// 1e-6 at n = 1640.  A tile's 64 by themselves first: 3e-7, in the same time.
template <int D, int RI>
__device__ __forceinline__ void add_product_pb(float (&o)[RI][D / 16], const float (&f)[RI], const float* p,
                                               const float* b, int ty, int tx) {
  float t[RI][D / 16] = {};
  product_pb<D, RI>(t, p, b, ty, tx);
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = o[i][c] * f[i] + t[i][c];
}

template <int D, typename T, int RI>
__device__ __forceinline__ void store_rows(T* dst, long long st, int r0, int n,
                                           const float (&o)[RI][D / 16], const float (&f)[RI], int ty,
                                           int tx) {
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = r0 + ty + 16 * i;
    if (r >= n) continue;
#pragma unroll
    for (int m = 0; m < D / 64; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[(long long)r * st + 4 * tx + 64 * m + e] = from_f<T>(o[i][4 * m + e] * f[i]);
  }
}

__device__ __forceinline__ float row_max(float v) {   // over the 16 threads of a row
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 16 RI query rows; the next tile's keys and values are on their way while this one's are used.
// KS groups of 256 threads take every KS-th tile of keys each, with their own m, l and o, and
// join them at the end: more warps where the rows leave one CTA per SM.
template <int D, typename T, int RI, int KS>
__global__ void __launch_bounds__(KS * kThreads) attn_fwd_simt_kernel(AttnArgs a) {
  constexpr int kRows = 16 * RI;
  extern __shared__ float sm[];
  float* sQ = sm;
  const int group = threadIdx.x / kThreads;
  float* sK = sQ + kRows * pitch<D>() + group * (2 * kT * pitch<D>() + kRows * kPP);
  float* sV = sK + kT * pitch<D>();
  float* sP = sV + kT * pitch<D>();
  auto group_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory"); };
  const int n_tile = (a.T + kRows - 1) / kRows;
  const int i0 = (blockIdx.x % n_tile) * kRows;
  const int h = (blockIdx.x / n_tile) % a.H, b = blockIdx.x / n_tile / a.H;
  const int ty = threadIdx.x % kThreads / 16, tx = threadIdx.x % 16;
  const int len = real_len(a.lens, b, a.reach);
  const T* kp = static_cast<const T*>(a.k) + b * a.k_sb + (h / a.G) * a.k_sh;
  const T* vp = static_cast<const T*>(a.v) + b * a.v_sb + (h / a.G) * a.v_sh;
  const KeyTiles tiles(a.q_start + i0, a.q_start + min(i0 + kRows, a.T) - 1, len, a.window, a.n_sink, kT);
  Tile<D, T> k, v;
  if (group < tiles.n) {
    k.fetch(kp, a.k_st, tiles[group] * kT, len);
    v.fetch(vp, a.v_st, tiles[group] * kT, len);
  }
  if (group == 0) load_tile<D, T, kRows>(sQ, static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh, a.q_st, i0, a.T);
  __syncthreads();
  float o[RI][D / 16] = {}, m[RI], l[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) m[i] = -INFINITY, l[i] = 0.f;
  const float s2 = a.scale * 1.4426950408889634f;   // logits in base 2
  for (int n = group; n < tiles.n; n += KS) {
    const int j0 = tiles[n] * kT;
    group_sync();
    k.put(sK);
    v.put(sV);
    group_sync();
    if (n + KS < tiles.n) {
      k.fetch(kp, a.k_st, tiles[n + KS] * kT, len);
      v.fetch(vp, a.v_st, tiles[n + KS] * kT, len);
    }
    float s[RI][4], f[RI];
    product_abt<D, RI>(s, sQ, sK, ty, tx);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int p = a.q_start + i0 + ty + 16 * i;
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = attn_sees(p, j0 + tx + 16 * j, len, a.window, a.n_sink) ? s[i][j] * s2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = row_max(mx);
      const float at = mx == -INFINITY ? 0.f : mx;   // a row that has seen nothing yet
      f[i] = ex2(m[i] - at);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] - at);
        sum += s[i][j];
        sP[(ty + 16 * i) * kPP + tx + 16 * j] = s[i][j];
      }
      l[i] = l[i] * f[i] + row_sum(sum);
      m[i] = mx;
    }
    __syncwarp();   // a row's 16 threads are in one warp
    add_product_pb<D, RI>(o, f, sP, sV, ty, tx);
  }
  if constexpr (KS == 2) {
    constexpr int V = RI * (D / 16 + 2);
    float* other = sm + kRows * pitch<D>() + (threadIdx.x % kThreads);   // [V][kThreads], over the first group's tiles
    static_assert(V * kThreads <= 2 * kT * pitch<D>(), "the second group's results fit");
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        other[(2 * i) * kThreads] = m[i], other[(2 * i + 1) * kThreads] = l[i];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) other[(2 * RI + i * (D / 16) + c) * kThreads] = o[i][c];
      }
    }
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const float m1 = other[(2 * i) * kThreads], mx = fmaxf(m[i], m1), at = mx == -INFINITY ? 0.f : mx;
      const float f0 = ex2(m[i] - at), f1 = ex2(m1 - at);
      l[i] = l[i] * f0 + other[(2 * i + 1) * kThreads] * f1;
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        o[i][c] = o[i][c] * f0 + other[(2 * RI + i * (D / 16) + c) * kThreads] * f1;
    }
  }
  float f[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    f[i] = l[i] != 0.f ? 1.f / l[i] : 0.f;
    const int r = i0 + ty + 16 * i;
    if (a.lse && tx == 0 && r < a.T)
      a.lse[((long long)b * a.H + h) * a.T + r] =
          l[i] != 0.f ? m[i] * 0.6931471805599453f + logf(l[i]) : -INFINITY;
  }
  store_rows<D, T, RI>(static_cast<T*>(a.out) + ((long long)b * a.T * a.H + h) * D, (long long)a.H * D, i0,
                       a.T, o, f, ty, tx);
}

// delta = rowsum(dO * O), one warp per row
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(AttnArgs a) {
  const long long row = (long long)blockIdx.x * 8 + threadIdx.x / 32;   // [B,T,H]
  const int lane = threadIdx.x % 32;
  if (row >= (long long)a.B * a.T * a.H) return;
  const T* o = static_cast<const T*>(a.out) + row * D;
  const T* g = static_cast<const T*>(a.d_out) + row * D;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s += to_f<T>(o[lane + 32 * c]) * to_f<T>(g[lane + 32 * c]);
  s = warp_sum(s);
  const int h = row % a.H;
  const long long bt = row / a.H;
  if (lane == 0) a.delta[(bt / a.T * a.H + h) * a.T + bt % a.T] = s;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) attn_dq_simt_kernel(AttnArgs a) {
  extern __shared__ float sm[];
  float* sQ = sm;
  float* sK = sQ + kT * pitch<D>();
  float* sV = sK + kT * pitch<D>();
  float* sO = sV + kT * pitch<D>();
  float* sP = sO + kT * pitch<D>();
  const int n_tile = (a.T + kT - 1) / kT;
  const int i0 = (blockIdx.x % n_tile) * kT;
  const int h = (blockIdx.x / n_tile) % a.H, b = blockIdx.x / n_tile / a.H;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int len = real_len(a.lens, b, a.reach);
  const T* kp = static_cast<const T*>(a.k) + b * a.k_sb + (h / a.G) * a.k_sh;
  const T* vp = static_cast<const T*>(a.v) + b * a.v_sb + (h / a.G) * a.v_sh;
  const long long out0 = ((long long)b * a.T * a.H + h) * D, out_st = (long long)a.H * D;
  load_tile<D, T>(sQ, static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh, a.q_st, i0, a.T);
  load_tile<D, T>(sO, static_cast<const T*>(a.d_out) + out0, out_st, i0, a.T);
  const KeyTiles tiles(a.q_start + i0, a.q_start + min(i0 + kT, a.T) - 1, len, a.window, a.n_sink, kT);
  float o[4][D / 16] = {}, lse[4], delta[4];
  const float one[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = min(i0 + ty + 16 * i, a.T - 1);
    lse[i] = a.lse[((long long)b * a.H + h) * a.T + r];
    delta[i] = a.delta[((long long)b * a.H + h) * a.T + r];
  }
  for (int n = 0; n < tiles.n; ++n) {
    const int j0 = tiles[n] * kT;
    __syncthreads();
    load_tile<D, T>(sK, kp, a.k_st, j0, len);
    load_tile<D, T>(sV, vp, a.v_st, j0, len);
    __syncthreads();
    float s[4][4], g[4][4];
    product_abt<D, 4>(s, sQ, sK, ty, tx);
    product_abt<D, 4>(g, sO, sV, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = a.q_start + i0 + ty + 16 * i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool sees = attn_sees(p, j0 + tx + 16 * j, len, a.window, a.n_sink);
        sP[(ty + 16 * i) * kPP + tx + 16 * j] =
            sees ? __expf(s[i][j] * a.scale - lse[i]) * (g[i][j] - delta[i]) : 0.f;
      }
    }
    __syncwarp();
    add_product_pb<D, 4>(o, one, sP, sK, ty, tx);
  }
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<D, T, 4>(static_cast<T*>(a.dq) + out0, out_st, i0, a.T, o, f, ty, tx);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) attn_dkv_simt_kernel(AttnArgs a) {
  extern __shared__ float sm[];
  float* sK = sm;
  float* sV = sK + kT * pitch<D>();
  float* sQ = sV + kT * pitch<D>();
  float* sO = sQ + kT * pitch<D>();
  float* sP = sO + kT * pitch<D>();   // [key][query]
  float* sL = sP + kT * kPP;          // the query tile's lse and delta
  const int n_tile = (a.S + kT - 1) / kT;
  const int j0 = (blockIdx.x % n_tile) * kT;
  const int hk = (blockIdx.x / n_tile) % a.Hkv, b = blockIdx.x / n_tile / a.Hkv;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int len = real_len(a.lens, b, a.reach);
  load_tile<D, T>(sK, static_cast<const T*>(a.k) + b * a.k_sb + hk * a.k_sh, a.k_st, j0, len);
  load_tile<D, T>(sV, static_cast<const T*>(a.v) + b * a.v_sb + hk * a.v_sh, a.v_st, j0, len);
  const QueryRows rows(j0, min(j0 + kT, a.S) - 1, len, a.window, a.n_sink, a.q_start, a.T);
  float dk[4][D / 16] = {}, dv[4][D / 16] = {};
  const float one[4] = {1.f, 1.f, 1.f, 1.f};
  for (int g = 0; g < a.G; ++g) {
    const int h = hk * a.G + g;
    const T* qp = static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh;
    const T* op = static_cast<const T*>(a.d_out) + ((long long)b * a.T * a.H + h) * D;
    for (int i0 = rows.begin / kT * kT; i0 < rows.end; i0 += kT) {
      __syncthreads();
      load_tile<D, T>(sQ, qp, a.q_st, i0, a.T);
      load_tile<D, T>(sO, op, (long long)a.H * D, i0, a.T);
      if (threadIdx.x < kT) {
        const int r = min(i0 + (int)threadIdx.x, a.T - 1);
        sL[threadIdx.x] = a.lse[((long long)b * a.H + h) * a.T + r];
        sL[kT + threadIdx.x] = a.delta[((long long)b * a.H + h) * a.T + r];
      }
      __syncthreads();
      float s[4][4], t[4][4];
      product_abt<D, 4>(s, sK, sQ, ty, tx);   // [key][query]
      product_abt<D, 4>(t, sV, sO, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = i0 + tx + 16 * j;
          const bool sees = r < a.T && attn_sees(a.q_start + r, j0 + ty + 16 * i, len, a.window, a.n_sink);
          s[i][j] = sees ? __expf(s[i][j] * a.scale - sL[tx + 16 * j]) : 0.f;
          sP[(ty + 16 * i) * kPP + tx + 16 * j] = s[i][j];
        }
      __syncwarp();
      add_product_pb<D, 4>(dv, one, sP, sO, ty, tx);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sP[(ty + 16 * i) * kPP + tx + 16 * j] =
              s[i][j] != 0.f ? s[i][j] * (t[i][j] - sL[kT + tx + 16 * j]) : 0.f;
      __syncwarp();
      add_product_pb<D, 4>(dk, one, sP, sQ, ty, tx);
    }
  }
  const long long o0 = ((long long)b * a.S * a.Hkv + hk) * D, st = (long long)a.Hkv * D;
  const float fk[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<D, T, 4>(static_cast<T*>(a.dk) + o0, st, j0, a.S, dk, fk, ty, tx);
  store_rows<D, T, 4>(static_cast<T*>(a.dv) + o0, st, j0, a.S, dv, one, ty, tx);
}

template <typename K>
cudaError_t launch(K kernel, long long grid, int threads, int smem, const AttnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(grid), threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D, typename T>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
  const int tile = kT * pitch<D>() * 4, p = kT * kPP * 4;
  const long long rows = (long long)a.B * a.T * a.H;
  attn_delta_kernel<D, T><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch(attn_dq_simt_kernel<D, T>, (long long)a.B * a.H * ((a.T + kT - 1) / kT), kThreads, 4 * tile + p, a, st);
  if (e != cudaSuccess) return e;
  return launch(attn_dkv_simt_kernel<D, T>, (long long)a.B * a.Hkv * ((a.S + kT - 1) / kT),
                kThreads, 4 * tile + p + 2 * kT * 4, a, st);
}

template <int D, typename T, int RI, int KS>
cudaError_t fwd_rows(const AttnArgs& a, cudaStream_t st) {
  return launch(attn_fwd_simt_kernel<D, T, RI, KS>, (long long)a.B * a.H * ((a.T + 16 * RI - 1) / (16 * RI)), KS * kThreads,
                (16 * RI * pitch<D>() + KS * (2 * kT * pitch<D>() + 16 * RI * kPP)) * 4, a, st);
}

// 64 rows per CTA reuse a tile of keys most; where those leave SMs without one, 32 rows, and
// at d 64, where the registers allow it, two groups of threads over the tiles of keys.  fp32,
// 32 rows / 64: B2 H6 T333 d64, window 257 (72 CTAs of 64) 23 / 33 us, B1 at d128 (36) 42 / 57,
// B4 H8 T1024 (512) 141 / 108, B8 H16 T1024, window 512 (2048) 737 / 543.
template <int D, typename T>
cudaError_t fwd(const AttnArgs& a, int sms, cudaStream_t st) {
  const bool few = (long long)a.B * a.H * ((a.T + 63) / 64) < sms;
  return few ? fwd_rows<D, T, 2, D == 64 ? 2 : 1>(a, st) : fwd_rows<D, T, 4, 1>(a, st);
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const AttnArgs& a, int dtype, int sms, cudaStream_t st) {
  if (dtype == DR_FP32) return a.d == 64 ? fwd<64, float>(a, sms, st) : fwd<128, float>(a, sms, st);
  return a.d == 64 ? fwd<64, __nv_bfloat16>(a, sms, st) : fwd<128, __nv_bfloat16>(a, sms, st);
}

cudaError_t launch_attn_bwd_simt(const AttnArgs& a, int dtype, cudaStream_t st) {
  if (dtype == DR_FP32) return a.d == 64 ? bwd<64, float>(a, st) : bwd<128, float>(a, st);
  return a.d == 64 ? bwd<64, __nv_bfloat16>(a, st) : bwd<128, __nv_bfloat16>(a, st);
}

}  // namespace dr
