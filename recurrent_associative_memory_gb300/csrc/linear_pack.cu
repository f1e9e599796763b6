// linear_pack.cu — operands of the tensor-core products that memory does not hold as they
// need them, and the gradient at the product.
//
// An fp32 value becomes three bf16 ones, x = p0 + p1 + p2 with p0 = bf16(x), p1 = bf16(x - p0),
// p2 = bf16(x - p0 - p1): 24 bits, so that six products of pieces keep an fp32 product's
// precision at a sixth of the bf16 rate, five times what the CUDA cores do.  bf16 rows whose
// stride no tensor map takes are copied to one that it does.
// The gradient at the product, d = d_y * slope, is formed once for both backward products, in
// the same layout, and the bias's gradient is summed from it in fp32 on the way (bf16 M8192 N8192
// 66 us, 6.1 TB/s).
//
// bf16 rounds d to its type, as a gradient that is handed from one bf16 operator to the next is:
// dx and dW are 2.4e-3 off (relative, over all of M8192 K2048 N8192), 1.7e-3 if d were exact.  A
// second piece of d would give that and double both products, 162 us each of the call's 516.  The
// slope is fp16: at most 2^-11 off where it counts, next to d's 2^-8.  Its steps of 2^-24 at the
// bottom leave slopes below 7.6e-6 (a sigmoid's from |x| = 11.8 on, SiLU's from x = -14.4) fewer
// bits than bf16 has and those below 3e-8 none: at most 2^-25 |d_y| of d.
#include "linear_tc.cuh"

namespace dr {
namespace {

constexpr int kRows = 64;    // of a block's tile, by 256 columns

template <typename T, bool VEC> __device__ __forceinline__ void read8(const T* p, int n, float (&f)[8]) {
  if constexpr (VEC) {
    load8(p, n, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
template <bool VEC> __device__ __forceinline__ void read8(const __half* p, int n, float (&f)[8]) {
  if constexpr (VEC) {
    const uint4 u = n > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(h[i]);
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? __half2float(p[i]) : 0.f;
  }
}

// The pieces of 8 values, to dst, dst + piece, ...
template <typename T> __device__ __forceinline__ void write_pieces(__nv_bfloat16* dst, long long piece, float (&f)[8]) {
#pragma unroll
  for (int p = 0; p < (sizeof(T) == 4 ? 3 : 1); ++p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = tc::pack_bf16(f[2 * i], f[2 * i + 1]);
      f[2 * i] -= __uint_as_float(w[i] << 16);
      f[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint4*>(dst + p * piece) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// rows x cols, columns contiguous -> pieces with rows of `pitch`; two matrices at once, the
// blocks shared out by their sizes
template <typename T, bool VEC>
__device__ __forceinline__ void pack_one(const PackJob& j, long long i, long long step) {
  const long long per = j.pitch / 8, n = j.rows * per;
  for (; i < n; i += step) {
    long long r;
    const int c = 8 * div_mod(i, static_cast<int>(per), r);
    float f[8];
    read8<T, VEC>(static_cast<const T*>(j.src) + r * j.stride + c, j.cols - c, f);
    write_pieces<T>(static_cast<__nv_bfloat16*>(j.dst) + r * j.pitch + c, j.piece, f);
  }
}
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(PackJob a, PackJob b, int blocks_a) {
  let_next_start();
  const bool first = static_cast<int>(blockIdx.x) < blocks_a;
  const PackJob& j = first ? a : b;
  const long long at = (long long)(blockIdx.x - (first ? 0 : blocks_a)) * 256 + threadIdx.x;
  const long long step = (long long)(first ? blocks_a : gridDim.x - blocks_a) * 256;
  if (j.cols % 8 == 0 && j.stride % (16 / (int)sizeof(T)) == 0) pack_one<T, true>(j, at, step);
  else pack_one<T, false>(j, at, step);
  wait_for_last();   // nothing here reads what that one writes, but whoever waits for this waits for both
}

// d = d_y * slope [M,N] in pieces with rows of `pitch` (dst null: not kept), and the columns'
// sums of each block's rows, part [row blocks][N] (null: not wanted).  A warp takes 256 columns
// of a row, 8 warps the rows in turns.
template <typename T, typename S, bool VEC>
__global__ void __launch_bounds__(256) slope_kernel(const T* d_y, const S* slope, __nv_bfloat16* dst, int pitch,
                                                    long long piece, float* part, int M, int N) {
  let_next_start();
  __shared__ float buf[8][256];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, col_blocks = (N + 255) / 256;
  const int c = blockIdx.x % col_blocks * 256 + lane * 8;
  const long long rb = blockIdx.x / col_blocks;
  float sum[8] = {};
  if (c < N) {
#pragma unroll 4
    for (int i = warp; i < kRows; i += 8) {
      const long long m = rb * kRows + i;
      if (m >= M) break;
      float f[8], s[8];
      read8<T, VEC>(d_y + m * N + c, N - c, f);
      if (slope) {
        if constexpr (sizeof(S) == 2) read8<VEC>(slope + m * N + c, N - c, s);
        else read8<S, VEC>(slope + m * N + c, N - c, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], s[j]);   // the same d, kept or only summed
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      if (dst) write_pieces<T>(dst + m * pitch + c, piece, f);
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) buf[warp][j * 32 + lane] = sum[j];
  __syncthreads();
  const int j = threadIdx.x / 32, n = blockIdx.x % col_blocks * 256 + lane * 8 + j;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += buf[w][j * 32 + lane];
  if (n < N) part[rb * N + n] = s;
}

// db = the sums over the row blocks, 32 groups of threads over them
template <typename T>
__global__ void __launch_bounds__(1024) join_bias_kernel(const float* part, int blocks, int N, T* db) {
  __shared__ float buf[32][33];
  let_next_start();
  wait_for_last();
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, n = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (n < N)
    for (int b = g; b < blocks; b += 32) s += part[(long long)b * N + n];
  buf[g][lane] = s;
  __syncthreads();
  s = warp_sum(buf[lane][g]);   // a warp per column now
  const int m = blockIdx.x * 32 + g;
  if (lane == 0 && m < N) db[m] = from_f<T>(s);
}

}  // namespace

// One or two (b.src null: one) copies in one launch.
cudaError_t launch_linear_pack(const PackJob& a, const PackJob& b, int dtype, int sms, bool after, cudaStream_t st) {
  auto blocks = [&](const PackJob& j) {
    const long long n = j.src ? ((long long)j.rows * (j.pitch / 8) + 255) / 256 : 0;
    return static_cast<int>(min(n, 16LL * sms));
  };
  const int na = blocks(a), nb = blocks(b);
  return launch_in_call(after, dtype == DR_FP32 ? pack_kernel<float> : pack_kernel<__nv_bfloat16>, na + nb, 256, 0, st, 0, a,
                        b, na);
}

int linear_slope_blocks(int M) { return static_cast<int>((M + (long long)kRows - 1) / kRows); }

// d into dst (or not, null) and the bias's gradient over part (or not, null)
cudaError_t launch_linear_slope(const LinearArgs& a, int dtype, void* dst, int pitch, long long piece, float* part,
                                cudaStream_t st) {
  const int blocks = linear_slope_blocks(a.M);
  const unsigned grid = static_cast<unsigned>(blocks * ((a.N + 255LL) / 256));
  const bool vec = a.N % 8 == 0;
  auto* d = static_cast<__nv_bfloat16*>(dst);
  auto go = [&](auto* kernel, auto t, auto s) {
    using T = decltype(t);
    cudaError_t e = launch_in_call(false, kernel, grid, 256, 0, st, 0, static_cast<const T*>(a.d_y),
                                   static_cast<const decltype(s)*>(a.slope), d, pitch, piece, part, a.M, a.N);
    if (e != cudaSuccess || !part) return e;
    return launch_in_call(true, join_bias_kernel<T>, (a.N + 31) / 32, 1024, 0, st, 0, part, blocks, a.N, static_cast<T*>(a.db));
  };
  if (dtype == DR_FP32) return go(vec ? slope_kernel<float, float, true> : slope_kernel<float, float, false>, 0.f, 0.f);
  using B = __nv_bfloat16;
  return go(vec ? slope_kernel<B, __half, true> : slope_kernel<B, __half, false>, B{}, __half{});
}

}  // namespace dr
