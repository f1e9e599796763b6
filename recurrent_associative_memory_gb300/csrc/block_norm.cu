// block_norm.cu — the norms before and after a block, with its gate and residual scale.
//
//   u  = branch, or branch * rstd(branch) * post_w        rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   h' = h + scale f(gate) u
//   y  = h' * rstd(h') * pre_w
//
// A block of threads takes one row (short rows: a warp takes several), keeps it in registers
// between its sums, and reads and writes every value once.  The norm takes h' as it was
// summed, before its rounding to the stream's type, and the backward pass sums it again from
// the same inputs, so nothing but h', y and the gradients is ever rounded.
//
// Backward, with t = dy pre_w, n = h' rstd:
//   dh' = d_h + rstd (t - n mean(t n))      dpre_w  = sum over rows of dy n
//   du  = dh' scale f(gate)                 dscale  = sum of dh' f(gate) u
//   dgate = dh' scale u f'(gate)            dpost_w = sum of du v,  v = branch rstd(branch)
//   dbranch = rstd(branch) (du post_w - v mean(du post_w v))
// A thread keeps its columns over all of its block's rows, so the weights' sums stay in
// registers; the blocks leave one partial sum each, which a second kernel joins in order.
#include "block.cuh"

namespace dr {
namespace {

constexpr int kE = 8;            // columns per thread
constexpr int kMaxThreads = 1024;

template <typename T, int VEC> __device__ __forceinline__ void load_row(const T* p, int D, int tpr, int t, float (&f)[kE]) {
  if constexpr (VEC == 8) {
    load8(p + 8 * t, 8 * t < D ? 1 : 0, f);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = e * tpr + t;
      f[e] = c < D ? to_f(p[c]) : 0.f;
    }
  }
}

template <typename T, int VEC> __device__ __forceinline__ void store_row(T* p, int D, int tpr, int t, const float (&f)[kE]) {
  if constexpr (VEC == 8) {
    if (8 * t < D) store8(p + 8 * t, f);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = e * tpr + t;
      if (c < D) p[c] = from_f<T>(f[e]);
    }
  }
}

// N sums over the threads of a row at once, the same in each of them.  Rows of up to 32
// threads stay within a warp; a wider one has its block to itself and goes through shared
// memory, two buffers in turn so that one barrier does: whoever writes a buffer again has
// passed the other one's barrier, which everyone reached after reading the first.
template <int N> __device__ __forceinline__ void row_sums(float (&v)[N], int tpr, float (&bufs)[2][64], int& turn) {
  static_assert(N <= 2, "");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  if (tpr <= 32) return;
  float* buf = bufs[turn];
  turn ^= 1;
  const int warps = tpr / 32, warp = threadIdx.x / 32;
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += buf[i * 32 + w];
    v[i] = s;
  }
}

template <bool SLOPE> __device__ __forceinline__ void gate_of(int act, const float (&z)[kE], float (&f)[kE], float (&s)[kE]) {
  auto each = [&](auto one) {
#pragma unroll
    for (int e = 0; e < kE; ++e) one(e);
  };
  switch (act) {
    case DR_ACT_RELU: each([&](int e) { f[e] = SLOPE ? act_of<DR_ACT_RELU>(z[e], s[e]) : act_of<DR_ACT_RELU>(z[e]); }); break;
    case DR_ACT_SILU: each([&](int e) { f[e] = SLOPE ? act_of<DR_ACT_SILU>(z[e], s[e]) : act_of<DR_ACT_SILU>(z[e]); }); break;
    case DR_ACT_GELU_TANH:
      each([&](int e) { f[e] = SLOPE ? act_of<DR_ACT_GELU_TANH>(z[e], s[e]) : act_of<DR_ACT_GELU_TANH>(z[e]); });
      break;
    case DR_ACT_SIGMOID:
      each([&](int e) { f[e] = SLOPE ? act_of<DR_ACT_SIGMOID>(z[e], s[e]) : act_of<DR_ACT_SIGMOID>(z[e]); });
      break;
    default: each([&](int e) { f[e] = z[e], s[e] = 1.f; });
  }
}

template <typename TA, typename TH, int VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_fwd_kernel(BlockNormArgs a, int tpr) {
  __shared__ float buf[2][64];
  int turn = 0;
  const int t = threadIdx.x % tpr, D = a.D;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.M;   // of a whole row; the others take part in the sums
  const long long r = live ? row : 0;
  float h[kE], w[kE];
  load_row<TH, VEC>(static_cast<const TH*>(a.h) + r * a.h_s, D, tpr, t, h);
  if (a.branch) {
    float u[kE], f[kE], z[kE];
    load_row<TA, VEC>(static_cast<const TA*>(a.branch) + r * a.b_s, D, tpr, t, u);
    if (a.gate) {
      load_row<TA, VEC>(static_cast<const TA*>(a.gate) + r * a.g_s, D, tpr, t, z);
      gate_of<false>(a.gate_act, z, f, w);
    }
    if (a.post_norm) {
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < kE; ++e) s[0] = fmaf(u[e], u[e], s[0]);
      row_sums(s, tpr, buf, turn);
      const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      if (a.post_w) {
        load_row<float, VEC>(a.post_w, D, tpr, t, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) u[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) u[e] *= rstd;
    }
    if (a.gate) {
#pragma unroll
      for (int e = 0; e < kE; ++e) u[e] *= f[e];
    }
    if (a.scale) {
      load_row<float, VEC>(a.scale, D, tpr, t, w);
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] = fmaf(w[e], u[e], h[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] += u[e];
    }
    if (live && a.h_out) store_row<TH, VEC>(static_cast<TH*>(a.h_out) + r * D, D, tpr, t, h);
  }
  if (!a.y) return;
  float s[1] = {0.f};
#pragma unroll
  for (int e = 0; e < kE; ++e) s[0] = fmaf(h[e], h[e], s[0]);
  row_sums(s, tpr, buf, turn);
  const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
  for (int e = 0; e < kE; ++e) h[e] *= rstd;
  if (a.pre_w) {
    load_row<float, VEC>(a.pre_w, D, tpr, t, w);
#pragma unroll
    for (int e = 0; e < kE; ++e) h[e] *= w[e];
  }
  if (live) store_row<TA, VEC>(static_cast<TA*>(a.y) + r * D, D, tpr, t, h);
}

template <typename TA, typename TH, int VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_bwd_kernel(BlockNormArgs a, int tpr) {
  __shared__ float buf[2][64];
  int turn = 0;
  const int t = threadIdx.x % tpr, D = a.D, rows = blockDim.x / tpr, slot = threadIdx.x / tpr;
  float sum_s[kE] = {}, sum_q[kE] = {}, sum_p[kE] = {};   // of scale, post_w, pre_w
  for (long long r0 = (long long)blockIdx.x * rows; r0 < a.M; r0 += (long long)gridDim.x * rows) {
    const bool live = r0 + slot < a.M;
    const long long r = live ? r0 + slot : 0;
    float h[kE], u[kE], v[kE], f[kE], fs[kE], w[kE], g[kE];
    float rstd_b = 1.f;
    load_row<TH, VEC>(static_cast<const TH*>(a.h) + r * a.h_s, D, tpr, t, h);
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = 1.f, fs[e] = 0.f, u[e] = v[e] = 0.f;
    if (a.branch) {   // h' again; u the branch's norm with its weight, v without it
      load_row<TA, VEC>(static_cast<const TA*>(a.branch) + r * a.b_s, D, tpr, t, v);
      if (a.gate) {
        float z[kE];
        load_row<TA, VEC>(static_cast<const TA*>(a.gate) + r * a.g_s, D, tpr, t, z);
        gate_of<true>(a.gate_act, z, f, fs);
      }
      if (a.post_norm) {
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < kE; ++e) s[0] = fmaf(v[e], v[e], s[0]);
        row_sums(s, tpr, buf, turn);
        rstd_b = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] *= rstd_b;
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) u[e] = v[e];
      if (a.post_w) {
        load_row<float, VEC>(a.post_w, D, tpr, t, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) u[e] *= w[e];
      }
      if (a.scale) load_row<float, VEC>(a.scale, D, tpr, t, w);
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] = fmaf(a.scale ? w[e] * f[e] : f[e], u[e], h[e]);
    }
    if (a.d_h) {
      load_row<TH, VEC>(static_cast<const TH*>(a.d_h) + r * D, D, tpr, t, g);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) g[e] = 0.f;
    }
    if (a.d_y) {
      float dy[kE], s[2] = {0.f, 0.f};
      load_row<TA, VEC>(static_cast<const TA*>(a.d_y) + r * D, D, tpr, t, dy);
      if (a.pre_w) {
        load_row<float, VEC>(a.pre_w, D, tpr, t, w);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) w[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        s[0] = fmaf(h[e], h[e], s[0]);
        s[1] = fmaf(dy[e] * w[e], h[e], s[1]);
      }
      row_sums(s, tpr, buf, turn);
      const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      const float k = s[1] * a.inv_d * rstd * rstd * rstd;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        if (live) sum_p[e] = fmaf(dy[e], h[e] * rstd, sum_p[e]);
        g[e] = fmaf(dy[e] * w[e], rstd, fmaf(-k, h[e], g[e]));
      }
    }
    if (live && a.dh) store_row<TH, VEC>(static_cast<TH*>(a.dh) + r * D, D, tpr, t, g);
    if (!a.branch) continue;
    if (a.scale) {
      load_row<float, VEC>(a.scale, D, tpr, t, w);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] = 1.f;
    }
    float dg[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if (live) sum_s[e] = fmaf(g[e] * f[e], u[e], sum_s[e]);
      dg[e] = g[e] * w[e] * u[e] * fs[e];
      g[e] *= w[e] * f[e];   // du from here on
      if (live) sum_q[e] = fmaf(g[e], v[e], sum_q[e]);
    }
    if (live && a.dg) store_row<TA, VEC>(static_cast<TA*>(a.dg) + r * D, D, tpr, t, dg);
    if (a.post_norm) {
      if (a.post_w) {
        load_row<float, VEC>(a.post_w, D, tpr, t, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) g[e] *= w[e];
      }
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < kE; ++e) s[0] = fmaf(g[e], v[e], s[0]);
      row_sums(s, tpr, buf, turn);
      const float k = s[0] * a.inv_d;
#pragma unroll
      for (int e = 0; e < kE; ++e) g[e] = rstd_b * fmaf(-k, v[e], g[e]);
    }
    if (live && a.db) store_row<TA, VEC>(static_cast<TA*>(a.db) + r * D, D, tpr, t, g);
  }
  if (!a.part) return;
  // rows of a warp first, then one after another over the slots of the block
  extern __shared__ float slots[];   // [warps][3][D] where a warp or more rows share the block
  float* part = a.part + (long long)blockIdx.x * 3 * D;
  auto each = [&](auto use) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = VEC == 8 ? 8 * t + e : e * tpr + t;
      if (c < D) use(e, c);
    }
  };
  if (rows == 1) {
    each([&](int e, int c) { part[c] = sum_s[e], part[D + c] = sum_q[e], part[2 * D + c] = sum_p[e]; });
    return;
  }
  each([&](int e, int c) {
    float* p = slots + (long long)slot * 3 * D;
    p[c] = sum_s[e], p[D + c] = sum_q[e], p[2 * D + c] = sum_p[e];
  });
  __syncthreads();
  for (int c = threadIdx.x; c < 3 * D; c += blockDim.x) {
    float s = 0.f;
    for (int i = 0; i < rows; ++i) s += slots[i * 3 * D + c];
    part[c] = s;
  }
}

// out[c] = sum over the blocks of part[block][which][c]: 8 groups of threads over the blocks,
// joined in order
__global__ void __launch_bounds__(256) join_parts_kernel(const float* part, int blocks, int D, float* o0, float* o1, float* o2) {
  __shared__ float buf[8][32];
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, which = blockIdx.y;
  float* out = which == 0 ? o0 : which == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D)
    for (int b = g; b < blocks; b += 8) s += part[((long long)b * 3 + which) * D + c];
  buf[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < D) {
    for (int i = 1; i < 8; ++i) s += buf[i][lane];
    out[c] = s;
  }
}

// threads per row: a power of two up to 32, whole warps from there on, which have their block
// to themselves
int threads_of(int D) {
  const int n = (D + kE - 1) / kE;
  if (n > 32) return (n + 31) / 32 * 32;
  int t = 1;
  while (t < n) t *= 2;
  return t;
}
int rows_of(int tpr) { return tpr <= 32 ? 128 / tpr : 1; }

bool vectors(const BlockNormArgs& a, int es_a, int es_h) {
  auto ok = [](const void* p, long long s, int es) { return !p || ((reinterpret_cast<uintptr_t>(p) | (s * es)) & 15) == 0; };
  return a.D % 8 == 0 && ok(a.h, a.h_s, es_h) && ok(a.branch, a.b_s, es_a) && ok(a.gate, a.g_s, es_a) &&
         ok(a.h_out, 0, es_h) && ok(a.y, 0, es_a) && ok(a.scale, 0, 4) && ok(a.post_w, 0, 4) && ok(a.pre_w, 0, 4) &&
         ok(a.d_h, 0, es_h) && ok(a.d_y, 0, es_a) && ok(a.dh, 0, es_h) && ok(a.db, 0, es_a) && ok(a.dg, 0, es_a);
}

template <typename F> void by_type(int dtype, int h_dtype, bool vec, F&& go) {
  auto types = [&](auto v) {
    if (dtype == DR_FP32) go(float{}, float{}, v);
    else if (h_dtype == DR_FP32) go(__nv_bfloat16{}, float{}, v);
    else go(__nv_bfloat16{}, __nv_bfloat16{}, v);
  };
  if (vec) types(std::integral_constant<int, 8>{});
  else types(std::integral_constant<int, 1>{});
}

}  // namespace

int block_norm_bwd_blocks(const BlockNormArgs& a, int sms) {
  const int tpr = threads_of(a.D), rows = rows_of(tpr);
  const long long most = (a.M + rows - 1LL) / rows;
  return static_cast<int>(most < 2LL * sms ? most : 2LL * sms);
}

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, int dtype, int h_dtype, cudaStream_t st) {
  const int tpr = threads_of(a.D), rows = rows_of(tpr);
  const unsigned grid = static_cast<unsigned>((a.M + (long long)rows - 1) / rows);
  by_type(dtype, h_dtype, vectors(a, dtype == DR_FP32 ? 4 : 2, h_dtype == DR_FP32 ? 4 : 2), [&](auto ta, auto th, auto v) {
    block_norm_fwd_kernel<decltype(ta), decltype(th), decltype(v)::value><<<grid, rows * tpr, 0, st>>>(a, tpr);
  });
  return cudaGetLastError();
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, float* d_scale, float* d_post,
                                  float* d_pre, cudaStream_t st) {
  const int tpr = threads_of(a.D), rows = rows_of(tpr);
  const int grid = block_norm_bwd_blocks(a, sms);
  const size_t smem = rows > 1 && a.part ? sizeof(float) * rows * 3 * a.D : 0;
  by_type(dtype, h_dtype, vectors(a, dtype == DR_FP32 ? 4 : 2, h_dtype == DR_FP32 ? 4 : 2), [&](auto ta, auto th, auto v) {
    block_norm_bwd_kernel<decltype(ta), decltype(th), decltype(v)::value><<<grid, rows * tpr, smem, st>>>(a, tpr);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  join_parts_kernel<<<dim3((a.D + 31) / 32, 3), 256, 0, st>>>(a.part, grid, a.D, d_scale, d_post, d_pre);
  return cudaGetLastError();
}

}  // namespace dr
