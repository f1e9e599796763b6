// attn_step.cu — window attention for one token per sequence over the ring cache,
// and the ring's layout from a prompt.
//
// Position p lives in slot p (p < n_sink) or n_sink + (p - n_sink) mod window, so
// what position p sees is exactly the slots 0 .. min(p, n_sink + window - 1): no
// masks, and no slot that was never written is read.  Bandwidth-bound: both caches
// are read once, 4 d bytes (bf16) per slot for 4 G d multiply-adds.
//   bf16  the heads of a group are the rows of warp-level m16n8k16 products (a row of the
//         tensor cores' 128 would be one in 16 or 32 used): about 8 instructions per slot
//         where multiply-adds on the CUDA cores take 96 at G = 4
//   fp32  CUDA cores
// Long caches of few sequences are cut into pieces of the slots, joined by a second launch.
//   bf16, d 128, 16 heads over 4: B256, 1028 slots at most, ragged (272 MB) 62 us, 4.4 TB/s, all full (539 MB)
//   105 us, 5.1 TB/s;
//   B1, 32772 slots (67 MB, which the L2 holds) 15 us on the GPU, 11 + 3 of the join.
//   fp32: B256, all full (1078 MB) 252 us, 4.3 TB/s; B1, 32772 slots (134 MB, cold) 53 us.
// Scores, sums and O are fp32; P is rounded to bf16 as an operand, its sum l is not; the
// outputs once.
#include "layers.cuh"

namespace dr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ long long slot_of(int p, int n_sink, int window) {
  return p < n_sink ? p : n_sink + (p - n_sink) % window;
}

// The parts: o [B,H,pieces][D], then (m, l) [B,H,pieces].
template <int D>
__device__ __forceinline__ float2* part_ml(const AttnStepArgs& a) {
  return reinterpret_cast<float2*>(a.part + (long long)a.B * a.H * a.n_piece * D);
}
template <int D>
__device__ __forceinline__ void put_part(const AttnStepArgs& a, long long row, int piece, int c, float o, float m,
                                         float l) {
  a.part[(row * a.n_piece + piece) * D + c] = o;
  if (c == 0) part_ml<D>(a)[row * a.n_piece + piece] = make_float2(m, l);
}

// One CTA per (sequence, key/value head, block of GB query heads, piece of the
// slots).  D / 8 lanes hold a slot's row, 8 channels each, so a warp takes 256 / D
// slots at once, with a running maximum and sum of its own.
template <int D, int GB, typename T>
__global__ void __launch_bounds__(kThreads) attn_step_simt_kernel(AttnStepArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");   // the join waits for this grid's end
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
    load8<T>(static_cast<const T*>(a.q) + ((long long)b * a.H + h0 + g) * D + c0, g < nh ? 8 : 0, q[g]);
#pragma unroll
    for (int c = 0; c < 8; ++c) q[g][c] *= a.scale * 1.4426950408889634f, o[g][c] = 0.f;
    m[g] = -INFINITY, l[g] = 0.f;
  }
  for (int j0 = begin + warp * KPW * U; j0 < end; j0 += kWarps * KPW * U) {
    float kf[U][8], s[U][GB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * KPW + sub;
      load8<T>(kc + (long long)j * D + c0, j < end ? 8 : 0, kf[u]);
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
      load8<T>(vc + (long long)j * D + c0, j < end ? 8 : 0, vf);
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
      put_part<D>(a, row, piece, c, acc, mx, sum);
    }
  }
}

// ------------------------------------------------------------------ bf16

// A piece of a cache row.  ONCE: it leaves no copy in L1, where nothing reads it again.
template <bool ONCE>
__device__ __forceinline__ uint4 cache16(const __nv_bfloat16* p) {
  if constexpr (!ONCE) return *reinterpret_cast<const uint4*>(p);
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");   // behind the barrier after which the new token's row is there
  return r;
}

constexpr int kMmaThreads = 128;
constexpr int kMmaWarps = kMmaThreads / 32;

// d (16 x 8) += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma16816(float& d0, float& d1, float& d2, float& d3, uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d0), "+f"(d1), "+f"(d2), "+f"(d3)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One CTA per (sequence, key/value head, block of 8 R query heads, piece of the slots);
// a warp takes 16 slots at a time.  With lane = 4 g + t, a fragment's row or column is g
// and its pairs along the summed axis belong to t.  That axis may be numbered freely as
// long as both operands agree, so every operand comes straight from memory in 16-byte
// pieces:
//   S = Q K^T    lane (g, t) holds channels 32 s + 8 t .. + 7 of slot g and of head g
//   O += P V     P is S's own accumulator; lane (g, t) holds channels 64 f + 8 g .. + 7 of
//                the slots 2t, 2t+1, 2t+8, 2t+9, and product e of a block takes channel e
//                of each lane's 8
// R = 1: the rows 8 .. 15 are not there and share two registers that stay 0.
template <int D, int R, bool ONCE>
__global__ void __launch_bounds__(kMmaThreads, R == 1 ? 3 : 2) attn_step_mma_kernel(AttnStepArgs a) {
  using T = __nv_bfloat16;
  constexpr int HB = 8 * R, KS = D / 32, VF = D / 64;
  __shared__ float s_o[kMmaWarps][HB][D], s_m[kMmaWarps][HB], s_l[kMmaWarps][HB];
  asm volatile("griddepcontrol.launch_dependents;");   // the join waits for this grid's end
  const int nb = (a.G + HB - 1) / HB;
  const int piece = blockIdx.x % a.n_piece, hb = (blockIdx.x / a.n_piece) % nb;
  const int hk = (blockIdx.x / a.n_piece / nb) % a.Hkv, b = blockIdx.x / a.n_piece / nb / a.Hkv;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int h0 = hk * a.G + hb * HB, nh = min(HB, a.G - hb * HB);
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
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 q[R][KS];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int s = 0; s < KS; ++s)
      q[r][s] = g + 8 * r < nh ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                                 ((long long)b * a.H + h0 + g + 8 * r) * D + 32 * s +
                                                                 8 * t)
                               : zero;
  __syncthreads();

  float o[R][VF][8][2], m[R], l[R], z0 = 0.f, z1 = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int f = 0; f < VF; ++f)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[r][f][e][0] = o[r][f][e][1] = 0.f;
  }
  const float c2 = a.scale * 1.4426950408889634f;
  uint4 k[2][KS];
  auto load_k = [&](int j0) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int j = j0 + 8 * u + g;
        k[u][s] = j < end ? cache16<ONCE>(kc + (long long)j * D + 32 * s + 8 * t) : zero;
      }
  };
  load_k(begin + 16 * warp);
  for (int j0 = begin + 16 * warp; j0 < end; j0 += 16 * kMmaWarps) {
    uint4 v[VF][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int f = 0; f < VF; ++f) {
        const int j = j0 + 2 * t + (u & 1) + 8 * (u >> 1);
        v[f][u] = j < end ? cache16<ONCE>(vc + (long long)j * D + 64 * f + 8 * g) : zero;
      }
    float s[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const uint4 q1 = R == 2 ? q[R - 1][i] : zero;
        mma16816(s[u][0], s[u][1], s[u][2], s[u][3], q[0][i].x, q1.x, q[0][i].y, q1.y, k[u][i].x, k[u][i].y);
        mma16816(s[u][0], s[u][1], s[u][2], s[u][3], q[0][i].z, q1.z, q[0][i].w, q1.w, k[u][i].z, k[u][i].w);
      }
    }
    load_k(j0 + 16 * kMmaWarps);   // on their way while this block's softmax and P V run
    uint32_t p[2][2] = {{0u, 0u}, {0u, 0u}};   // [slots 0-7, 8-15][heads 0-7, 8-15]
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[4], top = m[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = j0 + 8 * (e >> 1) + 2 * t + (e & 1) < end ? s[e >> 1][2 * r + (e & 1)] * c2 : -INFINITY;
        top = fmaxf(top, x[e]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (__any_sync(0xffffffffu, top > m[r])) {
        const float f = top == -INFINITY ? 1.f : ex2(m[r] - top);
        m[r] = top;
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < VF; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[r][i][e][0] *= f, o[r][i][e][1] *= f;
      }
      const float at = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ex2(x[e] - at);
        l[r] += x[e];
      }
      p[0][r] = pack_bf16(x[0], x[1]), p[1][r] = pack_bf16(x[2], x[3]);
    }
#pragma unroll
    for (int f = 0; f < VF; ++f)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
        const uint32_t* v0 = &v[f][0].x + e / 2;
        const uint32_t b0 = __byte_perm(v0[0], v0[4], sel), b1 = __byte_perm(v0[8], v0[12], sel);
        mma16816(o[0][f][e][0], o[0][f][e][1], R == 2 ? o[R - 1][f][e][0] : z0, R == 2 ? o[R - 1][f][e][1] : z1,
                 p[0][0], p[0][1], p[1][0], p[1][1], b0, b1);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t == 0) s_m[warp][g + 8 * r] = m[r], s_l[warp][g + 8 * r] = l[r];
#pragma unroll
    for (int f = 0; f < VF; ++f)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<float4*>(&s_o[warp][g + 8 * r][64 * f + 8 * (2 * t + x) + e]) = make_float4(
              o[r][f][e][x], o[r][f][e + 1][x], o[r][f][e + 2][x], o[r][f][e + 3][x]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nh * D; e += kMmaThreads) {
    const int h = e / D, c = e % D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kMmaWarps; ++w) mx = fmaxf(mx, s_m[w][h]);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kMmaWarps; ++w) {
      const float f = ex2(s_m[w][h] - at);
      sum += s_l[w][h] * f;
      acc += s_o[w][h][c] * f;
    }
    const long long row = (long long)b * a.H + h0 + h;
    if (a.n_piece == 1) {
      static_cast<T*>(a.out)[row * D + c] = __float2bfloat16_rn(sum != 0.f ? acc / sum : 0.f);
    } else {
      put_part<D>(a, row, piece, c, acc, mx, sum);
    }
  }
}

// out = sum over the pieces of o exp2(m - max) / sum of l exp2(m - max).  The warps take
// the pieces in turn, D / 32 channels per lane.
constexpr int kJoinWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_step_join_kernel(AttnStepArgs a) {
  constexpr int PER = D / 32;
  __shared__ float s_o[kJoinWarps][D], s_l[kJoinWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float2* ml = part_ml<D>(a) + (long long)blockIdx.x * a.n_piece;
  const float* o = a.part + (long long)blockIdx.x * a.n_piece * D + lane;
  float mx = -INFINITY;   // every warp forms it for itself
  for (int i = lane; i < a.n_piece; i += 32) mx = fmaxf(mx, ml[i].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  const float at = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, acc[PER] = {};
#pragma unroll 4
  for (int i = warp; i < a.n_piece; i += kJoinWarps) {
    const float2 p = ml[i];
    const float f = ex2(p.x - at);
    sum += p.y * f;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] += o[(long long)i * D + 32 * c] * f;
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) s_o[warp][lane + 32 * c] = acc[c];
  if (lane == 0) s_l[warp] = sum;
  __syncthreads();
  if (threadIdx.x >= D) return;
  float l = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += s_l[w], x += s_o[w][threadIdx.x];
  static_cast<T*>(a.out)[(long long)blockIdx.x * D + threadIdx.x] = from_f<T>(l != 0.f ? x / l : 0.f);
}

// The join may be launched while the pieces still run; it waits for them itself.
template <int D, typename T>
cudaError_t join(const AttnStepArgs& a, cudaStream_t st) {
  if (a.n_piece == 1) return cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.H));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, attn_step_join_kernel<D, T>, a) : e;
}

template <int D, int GB>
cudaError_t step(const AttnStepArgs& a, cudaStream_t st) {
  const long long grid = (long long)a.B * a.Hkv * ((a.G + GB - 1) / GB) * a.n_piece;
  attn_step_simt_kernel<D, GB, float><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
  return join<D, float>(a, st);
}

template <int D>
cudaError_t step_fp32(const AttnStepArgs& a, cudaStream_t st) {
  if (a.G == 1) return step<D, 1>(a, st);
  if (a.G == 2) return step<D, 2>(a, st);
  return step<D, 4>(a, st);
}

// Whole sequences to a CTA fill the SMs several times over, and their rows need no place in L1:
// B256, 1028 slots at most, 62 us instead of 67; in pieces (B1, 32772 slots) 19 instead of 15.
template <int D, int R>
cudaError_t step_mma(const AttnStepArgs& a, cudaStream_t st) {
  const long long grid = (long long)a.B * a.Hkv * ((a.G + 8 * R - 1) / (8 * R)) * a.n_piece;
  if (a.n_piece == 1)
    attn_step_mma_kernel<D, R, true><<<static_cast<unsigned>(grid), kMmaThreads, 0, st>>>(a);
  else
    attn_step_mma_kernel<D, R, false><<<static_cast<unsigned>(grid), kMmaThreads, 0, st>>>(a);
  return join<D, __nv_bfloat16>(a, st);
}

template <int D>
cudaError_t step_bf16(const AttnStepArgs& a, cudaStream_t st) {
  return a.G <= 8 ? step_mma<D, 1>(a, st) : step_mma<D, 2>(a, st);
}

// Each block copies 8-channel pieces of one slot row per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_fill_kernel(AttnArgs a, T* kc, T* vc) {
  const int C = a.n_sink + a.window, per = a.d / 8;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  long long row, bh, rb;   // row [B,Hkv,C]
  const int c = 8 * div_mod(e, per, row), slot = div_mod(row, C, bh), hk = div_mod(bh, a.Hkv, rb);
  if (rb >= a.B) return;
  const int b = rb;
  const int len = real_len(a.lens, b, a.S);
  int p = slot;                   // the last position before len that lives in this slot
  if (slot >= a.n_sink) {
    const int r = slot - a.n_sink, last = len - 1 - a.n_sink;   // ring index of the last token
    if (last < r) return;
    p = a.n_sink + r + (last - r) / a.window * a.window;
  }
  if (p >= len) return;
  float f[8];
  load8<T>(static_cast<const T*>(a.k) + b * a.k_sb + p * a.k_st + hk * a.k_sh + c, 8, f);
  store8<T>(kc + row * a.d + c, f);
  load8<T>(static_cast<const T*>(a.v) + b * a.v_sb + p * a.v_st + hk * a.v_sh + c, 8, f);
  store8<T>(vc + row * a.d + c, f);
}

}  // namespace

// Pieces along the slots: as many as fill three CTAs on every SM, of 128 slots at least.
// bf16, d 128, 16 heads over 4, for one / three / six CTAs per SM / without pieces:
// B1 32772 slots 16.1 / 14.8 / 20.9 / 467 us, B4 4100 slots 11.4 / 10.9 / 13.0 / 49,
// B16 1028 slots 11.8 / 10.1 / 13.0 / 15.7; B256 is one piece either way.
int attn_step_pieces(const AttnStepArgs& a, int dtype, int sms) {
  const int heads = dtype == DR_FP32 ? 4 : (a.G <= 8 ? 8 : 16);   // of one CTA
  const long long rows = (long long)a.B * a.Hkv * ((a.G + heads - 1) / heads);
  const long long most = ((long long)a.n_sink + a.window + 127) / 128;
  const long long want = 3LL * sms / rows;
  return static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
}

cudaError_t launch_attn_step(const AttnStepArgs& a, int dtype, cudaStream_t st) {
  if (dtype == DR_FP32) return a.d == 64 ? step_fp32<64>(a, st) : step_fp32<128>(a, st);
  return a.d == 64 ? step_bf16<64>(a, st) : step_bf16<128>(a, st);
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
