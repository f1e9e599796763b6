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
// Backward, with t = dy pre_w, n = h' rstd(h'), v = branch rstd(branch), c = scale post_w:
//   dh' = d_h + rstd (t - n mean(t n))        dpre_w  = sum over rows of dy n
//   q   = dh' f(gate) c                       S = sum of dh' f(gate) v
//   dgate = dh' c v f'(gate)                  dscale = post_w S,  dpost_w = scale S
//   dbranch = rstd(branch) (q - v mean(q v))
// A thread keeps its columns over all of its block's rows, so the two sums stay in registers;
// the blocks leave one partial sum each, which a second kernel joins in order.
#include <type_traits>

#include "block.cuh"
#include "umma.cuh"

namespace dr {
namespace {

constexpr int kMaxStages = 8;

// A thread's E columns of a row: groups of 8 neighbours where rows start on 16 bytes, else one
// of every tpr so that a warp's accesses stay next to each other.
template <int VEC, int E> struct Columns {
  int D, tpr, t;
  __device__ __forceinline__ int at(int e) const { return VEC == 8 ? (e / 8 * tpr + t) * 8 + e % 8 : e * tpr + t; }
};

// Rows come into shared memory by background copies of the whole 16-byte units inside them;
// the few values before the first and after the last unit are read where they are.
struct RowCopy {
  uintptr_t p, lo;   // the row, its first whole unit
  uint32_t bytes;    // of whole units
  __device__ __forceinline__ RowCopy(const void* base, long long row, long long stride, int D, int es) {
    p = reinterpret_cast<uintptr_t>(base) + row * stride * es;
    lo = (p + 15) & ~uintptr_t(15);
    const uintptr_t hi = (p + static_cast<uint32_t>(D) * es) & ~uintptr_t(15);
    bytes = hi > lo ? static_cast<uint32_t>(hi - lo) : 0u;
  }
};

// A thread's values of row `row`, from its copy at `at` in shared memory (WIDE), or from memory.
template <typename T, bool WIDE, int VEC, int E>
__device__ __forceinline__ void row_values(const void* base, long long row, long long stride, uint32_t at,
                                           const Columns<VEC, E>& c, f2 (&r)[E / 2]) {
  float f[E];
  if constexpr (VEC == 8) {
#pragma unroll
    for (int g = 0; g < E; g += 8) {
      const int n = c.at(g);
      if (n >= c.D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[g + e] = 0.f;
        continue;
      }
      uint32_t w[2 * sizeof(T)];
#pragma unroll
      for (int i = 0; i < 2 * (int)sizeof(T); i += 4) {
        if constexpr (WIDE) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                       : "r"(at + n * (int)sizeof(T) + 4 * i)
                       : "memory");
        } else {
          const uint4 u = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + row * stride + n)[i / 4];
          w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 2) f[g + e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        else f[g + e] = __uint_as_float(w[e]);
      }
    }
  } else {
    const RowCopy rc(base, row, stride, c.D, sizeof(T));
    const uint32_t head = static_cast<uint32_t>(rc.lo - rc.p);   // bytes before the first unit
#pragma unroll
    for (int e = 0; e < E; ++e) {
      f[e] = 0.f;
      if (c.at(e) >= c.D) continue;
      const uint32_t b = c.at(e) * (uint32_t)sizeof(T), in = b - head;   // below the first unit: huge
      if (WIDE && in < rc.bytes) {
        if constexpr (sizeof(T) == 2) {
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at + in) : "memory");
          f[e] = __uint_as_float(static_cast<uint32_t>(v) << 16);
        } else {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[e]) : "r"(at + in) : "memory");
        }
      } else {
        f[e] = to_f(*reinterpret_cast<const T*>(rc.p + b));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) r[i] = pack2(f[2 * i], f[2 * i + 1]);
}

// Values in pairs: two fp32 operations per instruction, as instructions are what bounds these
// kernels next to memory.
__device__ __forceinline__ f2 both(float x) { return pack2(x, x); }
template <int P> __device__ __forceinline__ void fill(f2 (&r)[P], float x) {
#pragma unroll
  for (int i = 0; i < P; ++i) r[i] = both(x);
}
template <int P> __device__ __forceinline__ float dot(const f2 (&x)[P], const f2 (&y)[P]) {
  f2 a = mul2(x[0], y[0]), b = mul2(x[1], y[1]);
#pragma unroll
  for (int i = 2; i < P; i += 2) a = fma2(x[i], y[i], a), b = fma2(x[i + 1], y[i + 1], b);
  return sum2(add2(a, b));
}
template <int P, typename F> __device__ __forceinline__ void pairs(F&& f) {
#pragma unroll
  for (int i = 0; i < P; ++i) f(i);
}

template <int VEC, int E> __device__ __forceinline__ void load_vector(const float* p, const Columns<VEC, E>& c, f2 (&r)[E / 2]) {
  float f[E];
  if constexpr (VEC == 8) {
#pragma unroll
    for (int g = 0; g < E; g += 8)
      load8(p + c.at(g), c.at(g) < c.D ? 1 : 0, reinterpret_cast<float(&)[8]>(f[g]));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = c.at(e) < c.D ? p[c.at(e)] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) r[i] = pack2(f[2 * i], f[2 * i + 1]);
}

template <typename T, int VEC, int E>
__device__ __forceinline__ void store_row(T* p, const Columns<VEC, E>& c, const f2 (&r)[E / 2]) {
  float f[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) unpack2(r[i], f[2 * i], f[2 * i + 1]);
  if constexpr (VEC == 8) {
#pragma unroll
    for (int g = 0; g < E; g += 8)
      if (c.at(g) < c.D) store8(p + c.at(g), reinterpret_cast<float(&)[8]>(f[g]));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c.at(e) < c.D) p[c.at(e)] = from_f<T>(f[e]);
  }
}

// The rows of a block.  WIDE: one at a time, through a ring of `stages` of them in shared
// memory.  Tensor i of a row is copied by warp i, once the block has passed a barrier behind
// the reads of the row whose place it takes: the first one of the next row.  (To issue a copy
// takes a few hundred cycles: one thread for all of them holds the block up, M16384 D4096
// forward 156 us instead of XXX; a warp of its own costs the others 32 registers each.)
// Otherwise straight from memory.
template <int N> struct Ring {
  uint64_t* full;
  uint32_t at, stage_bytes;   // shared memory of stage 0; from stage to stage
  int stages;
  const void* base[N];
  long long stride[N];
  uint32_t off[N];            // of the tensors in a stage
  int es[N];
  int stage;
  uint32_t parity;
  bool lost;

  // One thread of a warp: that warp's tensor of a row.
  __device__ __forceinline__ void issue(int warp, long long row, int s, int D) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i != warp || !base[i]) continue;
      const RowCopy r(base[i], row, stride[i], D, es[i]);
      umma::mbar_expect_tx(full + s, r.bytes);
      if (r.bytes)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         at + s * stage_bytes + off[i]),
                     "l"(r.lo), "r"(r.bytes), "r"(umma::smem_u32(full + s))
                     : "memory");
    }
  }
  // Bounded; after one that gave up none waits any more, and what comes out means nothing.
  __device__ __forceinline__ void wait() {
    if (lost || umma::mbar_wait(full + stage, parity, 2000000000ull)) return;
    lost = true;
    set_status(DR_ERR_TIMEOUT);
  }
  __device__ __forceinline__ void next() {
    if (++stage == stages) stage = 0, parity ^= 1;
  }
  // Behind the first barrier of `row`: the place of the row before goes to the one `stages`
  // further on.
  __device__ __forceinline__ void refill(long long row, long long first, long long step, int M, int D) {
    const long long to = row + (stages - 1) * step;
    if (threadIdx.x < 32 * N && threadIdx.x % 32 == 0 && row > first && to < M)
      issue(threadIdx.x / 32, to, stage == 0 ? stages - 1 : stage - 1, D);
  }
  // No copy may be in flight when the block ends; only after a wait that gave up there can be.
  __device__ __forceinline__ void drain() {
    if (!lost) return;
    for (int i = 0; i < stages; ++i) {
      umma::mbar_wait(full + stage, parity, 500000000ull);
      next();
    }
  }
  template <typename T, bool WIDE, int VEC, int E>
  __device__ __forceinline__ void get(int i, long long row, const Columns<VEC, E>& c, f2 (&r)[E / 2]) const {
    row_values<T, WIDE>(base[i], row, stride[i], at + stage * stage_bytes + off[i], c, r);
  }
};

// N sums over the threads of a row at once, the same in each of them.  Rows of up to 32
// threads stay within a warp; a wider one has its block to itself and goes through shared
// memory, two buffers in turn so that one barrier does: whoever writes a buffer again has
// passed the other one's barrier, which everyone reached after reading the first.
template <bool WIDE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr, float (&bufs)[2][64], int& turn) {
  static_assert(N <= 2, "");
  auto over_lanes = [&](int most) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (WIDE || o < most) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
  };
  over_lanes(tpr);
  if constexpr (WIDE) {
    float* buf = bufs[turn];
    turn ^= 1;
    const int lane = threadIdx.x % 32;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i * 32 + threadIdx.x / 32] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane * 32 < tpr ? buf[i * 32 + lane] : 0.f;
    over_lanes(32);
  }
}

__device__ __forceinline__ f2 sigmoid2(f2 x) {
  float a, b;
  unpack2(add2(ex2_2(mul2(x, both(-1.4426950408889634f))), both(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack2(a, b);
}

// f(z), and f'(z) where SLOPE: s (1 - s) of a sigmoid s, s + z s (1 - s) of z s.
template <bool SLOPE, int P> __device__ __forceinline__ void gate_of(int act, const f2 (&z)[P], f2 (&f)[P], f2 (&d)[P]) {
  auto scalar = [&](auto code) {
    pairs<P>([&](int i) {
      float x[2], s[2];
      unpack2(z[i], x[0], x[1]);
      x[0] = act_of<decltype(code)::value>(x[0], s[0]), x[1] = act_of<decltype(code)::value>(x[1], s[1]);
      f[i] = pack2(x[0], x[1]);
      if constexpr (SLOPE) d[i] = pack2(s[0], s[1]);
    });
  };
  if (act == DR_ACT_SILU) {
    pairs<P>([&](int i) {
      const f2 s = sigmoid2(z[i]);
      f[i] = mul2(z[i], s);
      if constexpr (SLOPE) d[i] = add2(s, fma2(f[i], mul2(s, both(-1.f)), f[i]));
    });
  } else if (act == DR_ACT_SIGMOID) {
    pairs<P>([&](int i) {
      f[i] = sigmoid2(z[i]);
      if constexpr (SLOPE) d[i] = fma2(f[i], mul2(f[i], both(-1.f)), f[i]);
    });
  } else if (act == DR_ACT_RELU) {
    scalar(std::integral_constant<int, DR_ACT_RELU>{});
  } else if (act == DR_ACT_GELU_TANH) {
    scalar(std::integral_constant<int, DR_ACT_GELU_TANH>{});
  } else {
    scalar(std::integral_constant<int, DR_ACT_NONE>{});
  }
}

// How a launch lays the rows' copies out.
struct RingLayout {
  int stages;
  uint32_t stage_bytes;
};

constexpr int kNarrow = 128;   // threads of a block whose rows are up to 32 threads each

template <int N, int VEC, int E>
__device__ __forceinline__ void start(Ring<N>& ring, uint64_t (&bars)[kMaxStages], const RingLayout& l,
                                      const Columns<VEC, E>& c, long long row, long long step, int M) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  ring.full = bars;
  ring.at = umma::smem_u32(dynamic);
  ring.stage_bytes = l.stage_bytes;
  ring.stages = l.stages;
  ring.stage = 0, ring.parity = 0, ring.lost = false;
  uint32_t at = 0;
  int there = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ring.off[i] = at;
    if (ring.base[i]) at += (c.D * ring.es[i] + 15) / 16 * 16, ++there;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < l.stages; ++i) umma::mbar_init(ring.full + i, there);
    umma::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0)
    for (int i = 0; i < l.stages && row + i * step < M; ++i) ring.issue(threadIdx.x / 32, row + i * step, i, c.D);
}

// THREADS: kNarrow, or the largest block that the kernel is built for; BLOCKS of them on an SM.
template <typename TA, typename TH, int VEC, int E, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_norm_fwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  constexpr bool WIDE = THREADS != kNarrow;
  constexpr int P = E / 2;
  using Row = f2[P];
  __shared__ float buf[2][64];
  __shared__ uint64_t bars[kMaxStages];
  int turn = 0;
  const Columns<VEC, E> c{a.D, tpr, WIDE ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % tpr};
  const int rows = WIDE ? 1 : kNarrow / tpr;
  const long long step = (long long)gridDim.x * rows, first = (long long)blockIdx.x * rows;
  Ring<3> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s;
  ring.es[0] = sizeof(TH), ring.es[1] = ring.es[2] = sizeof(TA);
  if (WIDE) start(ring, bars, l, c, first, step, a.M);
  Row ws, wy;   // scale post_w; pre_w
  fill(ws, 1.f), fill(wy, 1.f);
  if (a.pre_w) load_vector(a.pre_w, c, wy);
  if (a.scale) load_vector(a.scale, c, ws);
  if (a.post_w) {
    Row w;
    load_vector(a.post_w, c, w);
    pairs<P>([&](int i) { ws[i] = mul2(ws[i], w[i]); });
  }
  long long row = first + (WIDE ? 0 : threadIdx.x / tpr);
  // rows of other slots of the same warp may end earlier: those go on with zeros
  for (long long r0 = first; r0 < a.M; r0 += step, row += step) {
    const bool live = WIDE || row < a.M;
    Row h, u, f;
    if (!WIDE) fill(h, 0.f), fill(u, 0.f), fill(f, 0.f);
    if (WIDE) ring.wait();
    if (live) {
      if (a.branch) ring.template get<TA, WIDE>(1, row, c, u);
      ring.template get<TH, WIDE>(0, row, c, h);
      if (a.gate) {
        Row z, none;
        ring.template get<TA, WIDE>(2, row, c, z);
        gate_of<false>(a.gate_act, z, f, none);
      }
    }
    if (a.branch) {
      float rstd = 1.f;
      if (a.post_norm) {
        float s[1] = {dot(u, u)};
        row_sums<WIDE>(s, tpr, buf, turn);
        rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      }
      if (a.gate) pairs<P>([&](int i) { u[i] = mul2(u[i], f[i]); });
      pairs<P>([&](int i) { h[i] = fma2(mul2(u[i], both(rstd)), ws[i], h[i]); });
      if (live) store_row(static_cast<TH*>(a.h_out) + row * a.D, c, h);
    }
    if (a.y) {
      float s[1] = {dot(h, h)};
      row_sums<WIDE>(s, tpr, buf, turn);
      const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      if (WIDE) ring.refill(row, first, step, a.M, a.D);
      pairs<P>([&](int i) { h[i] = mul2(h[i], mul2(both(rstd), wy[i])); });
      if (live) store_row(static_cast<TA*>(a.y) + row * a.D, c, h);
    } else if (WIDE) {
      __syncthreads();
      ring.refill(row, first, step, a.M, a.D);
    }
    if (WIDE) ring.next();
  }
  if (WIDE) ring.drain();
}

template <typename TA, typename TH, int VEC, int E, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_norm_bwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  constexpr bool WIDE = THREADS != kNarrow;
  constexpr int P = E / 2;
  using Row = f2[P];
  __shared__ float buf[2][64];
  __shared__ uint64_t bars[kMaxStages];
  int turn = 0;
  const Columns<VEC, E> c{a.D, tpr, WIDE ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % tpr};
  const int D = a.D, rows = WIDE ? 1 : kNarrow / tpr, slot = WIDE ? 0 : threadIdx.x / tpr;
  const long long step = (long long)gridDim.x * rows, first = (long long)blockIdx.x * rows;
  Ring<5> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate, ring.base[3] = a.d_y, ring.base[4] = a.d_h;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s, ring.stride[3] = ring.stride[4] = D;
  ring.es[0] = ring.es[4] = sizeof(TH), ring.es[1] = ring.es[2] = ring.es[3] = sizeof(TA);
  if (WIDE) start(ring, bars, l, c, first, step, a.M);
  Row sum_s, sum_p, ws, wy;   // S, the sum of dpre_w; scale post_w, pre_w
  fill(sum_s, 0.f), fill(sum_p, 0.f), fill(ws, 1.f), fill(wy, 1.f);
  if (a.pre_w) load_vector(a.pre_w, c, wy);
  if (a.scale) load_vector(a.scale, c, ws);
  if (a.post_w) {
    Row w;
    load_vector(a.post_w, c, w);
    pairs<P>([&](int i) { ws[i] = mul2(ws[i], w[i]); });
  }
  long long row = first + slot;
  for (long long r0 = first; r0 < a.M; r0 += step, row += step) {
    const bool live = WIDE || row < a.M;
    // a row that is none: zeros, so that it adds nothing to any sum
    Row h, v, f, vs, g;   // vs: v f'(gate)
    float rstd_b = 1.f;
    if (!WIDE) fill(h, 0.f), fill(v, 0.f);
    if (WIDE) ring.wait();
    if (live) ring.template get<TH, WIDE>(0, row, c, h);
    if (a.branch) {   // h' again
      if (live) ring.template get<TA, WIDE>(1, row, c, v);
      if (a.post_norm) {
        float s[1] = {dot(v, v)};
        row_sums<WIDE>(s, tpr, buf, turn);
        rstd_b = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
        pairs<P>([&](int i) { v[i] = mul2(v[i], both(rstd_b)); });
      }
      fill(f, 1.f), fill(vs, 0.f);
      if (a.gate && live) {
        Row z;
        ring.template get<TA, WIDE>(2, row, c, z);
        gate_of<true>(a.gate_act, z, f, vs);
        pairs<P>([&](int i) { vs[i] = mul2(vs[i], v[i]); });
      }
      pairs<P>([&](int i) { h[i] = fma2(mul2(f[i], v[i]), ws[i], h[i]); });
    }
    if (a.d_y) {
      Row dy, t;
      if (!WIDE) fill(dy, 0.f);
      if (live) ring.template get<TA, WIDE>(3, row, c, dy);
      pairs<P>([&](int i) { t[i] = mul2(dy[i], wy[i]); });
      float s[2] = {dot(h, h), dot(t, h)};
      row_sums<WIDE>(s, tpr, buf, turn);
      const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      const f2 k = both(-s[1] * a.inv_d * rstd * rstd), r2 = both(rstd);
      pairs<P>([&](int i) {
        h[i] = mul2(h[i], r2);
        sum_p[i] = fma2(dy[i], h[i], sum_p[i]);
        t[i] = fma2(t[i], r2, mul2(k, h[i]));
      });
      if (a.d_h) {
        if (!WIDE) fill(g, 0.f);
        if (live) ring.template get<TH, WIDE>(4, row, c, g);
        pairs<P>([&](int i) { g[i] = add2(g[i], t[i]); });
      } else {
        pairs<P>([&](int i) { g[i] = t[i]; });
      }
    } else {
      if (!WIDE) fill(g, 0.f);
      if (live) ring.template get<TH, WIDE>(4, row, c, g);
      if (WIDE) __syncthreads();
    }
    if (WIDE) ring.refill(row, first, step, a.M, D), ring.next();
    if (live && a.dh) store_row(static_cast<TH*>(a.dh) + row * D, c, g);
    if (!a.branch) continue;
    pairs<P>([&](int i) {
      const f2 x = mul2(g[i], ws[i]);
      sum_s[i] = fma2(g[i], mul2(f[i], v[i]), sum_s[i]);
      vs[i] = mul2(x, vs[i]);
      g[i] = mul2(x, f[i]);   // q from here on
    });
    if (live && a.dg) store_row(static_cast<TA*>(a.dg) + row * D, c, vs);
    if (a.post_norm) {
      float s[1] = {dot(g, v)};
      row_sums<WIDE>(s, tpr, buf, turn);
      const f2 k = both(-s[0] * a.inv_d * rstd_b), r2 = both(rstd_b);
      pairs<P>([&](int i) { g[i] = fma2(k, v[i], mul2(r2, g[i])); });
    }
    if (live && a.db) store_row(static_cast<TA*>(a.db) + row * D, c, g);
  }
  if (WIDE) ring.drain();
  if (!a.part) return;
  float ss[E], sp[E];
  pairs<P>([&](int i) {
    unpack2(sum_s[i], ss[2 * i], ss[2 * i + 1]);
    unpack2(sum_p[i], sp[2 * i], sp[2 * i + 1]);
  });
  float* part = a.part + (long long)blockIdx.x * 2 * D;
  auto each = [&](float* to) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int n = c.at(e);
      if (n < D) to[n] = ss[e], to[D + n] = sp[e];
    }
  };
  if constexpr (WIDE) {
    each(part);
  } else {   // the block's rows, one after another
    extern __shared__ __align__(16) uint8_t dynamic[];   // [rows][2][D]
    float* slots = reinterpret_cast<float*>(dynamic);
    each(slots + slot * 2 * D);
    __syncthreads();
    for (int n = threadIdx.x; n < 2 * D; n += kNarrow) {
      float s = 0.f;
      for (int i = 0; i < rows; ++i) s += slots[i * 2 * D + n];
      part[n] = s;
    }
  }
}

// The sums over the blocks of part[block][which][D], 8 groups of threads over the blocks, joined
// in order: which 0 is S, of dscale and dpost_w, 1 is dpre_w.
__global__ void __launch_bounds__(256) join_parts_kernel(const float* part, int blocks, int D, const float* scale,
                                                         const float* post_w, float* d_scale, float* d_post, float* d_pre) {
  __shared__ float buf[8][32];
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, which = blockIdx.y;
  if (which == 0 ? !d_scale && !d_post : !d_pre) return;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D)
    for (int b = g; b < blocks; b += 8) s += part[((long long)b * 2 + which) * D + c];
  buf[g][lane] = s;
  __syncthreads();
  if (g != 0 || c >= D) return;
  for (int i = 1; i < 8; ++i) s += buf[i][lane];
  if (which == 1) {
    d_pre[c] = s;
    return;
  }
  if (d_scale) d_scale[c] = post_w ? s * post_w[c] : s;
  if (d_post) d_post[c] = scale ? s * scale[c] : s;
}

bool vectors(const BlockNormArgs& a, int es_a, int es_h) {
  auto ok = [](const void* p, long long s, int es) { return !p || ((reinterpret_cast<uintptr_t>(p) | (s * es)) & 15) == 0; };
  return a.D % 8 == 0 && ok(a.h, a.h_s, es_h) && ok(a.branch, a.b_s, es_a) && ok(a.gate, a.g_s, es_a) &&
         ok(a.h_out, 0, es_h) && ok(a.y, 0, es_a) && ok(a.scale, 0, 4) && ok(a.post_w, 0, 4) && ok(a.pre_w, 0, 4) &&
         ok(a.d_h, 0, es_h) && ok(a.d_y, 0, es_a) && ok(a.dh, 0, es_h) && ok(a.db, 0, es_a) && ok(a.dg, 0, es_a);
}

template <int N> using Int = std::integral_constant<int, N>;

template <typename F> void by_type(int dtype, int h_dtype, bool vec, F&& go) {
  auto types = [&](auto v) {
    if (dtype == DR_FP32) go(float{}, float{}, v);
    else if (h_dtype == DR_FP32) go(__nv_bfloat16{}, float{}, v);
    else go(__nv_bfloat16{}, __nv_bfloat16{}, v);
  };
  if (vec) types(Int<8>{});
  else types(Int<1>{});
}

// A launch: blocks that stay on every SM, and the rows on their way in what each of them has of
// its shared memory.
struct Plan {
  int tpr, threads, grid;
  RingLayout ring;
  size_t smem;
  Plan(const BlockNormArgs& a, int sms, int e, int blocks, int row_bytes, bool sums) {
    const int n = (a.D + e - 1) / e;
    int rows = 1;
    smem = 0;
    if (n <= 32) {
      for (tpr = 4; tpr < n; tpr *= 2) {}
      rows = kNarrow / tpr, threads = kNarrow;
      if (sums) smem = sizeof(float) * rows * 2 * a.D;
    } else {
      tpr = threads = (n + 31) / 32 * 32;
      if (threads < 32 * 5) threads = tpr = 32 * 5;   // a warp for each tensor's copies
    }
    const long long most = (a.M + rows - 1LL) / rows, there = (long long)sms * blocks;
    grid = static_cast<int>(most < there ? most : there);
    ring.stage_bytes = row_bytes, ring.stages = 1;
    if (n > 32) {
      const long long fit = ((224 * 1024) / blocks - 2048) / row_bytes, need = (most + grid - 1) / (grid ? grid : 1);
      ring.stages = static_cast<int>(fit < kMaxStages ? fit : kMaxStages);
      if (ring.stages > need) ring.stages = static_cast<int>(need);
      if (ring.stages < 1) ring.stages = 1;
      smem = (size_t)ring.stages * row_bytes;
    }
  }
};

int row_bytes(const BlockNormArgs& a, int es_a, int es_h) {
  auto of = [&](const void* p, int es) { return p ? (a.D * es + 15) / 16 * 16 : 0; };
  return of(a.h, es_h) + of(a.branch, es_a) + of(a.gate, es_a) + of(a.d_y, es_a) + of(a.d_h, es_h);
}

template <typename K> cudaError_t launch(K* kernel, const Plan& p, const BlockNormArgs& a, cudaStream_t st) {
  if (p.smem > 40 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e != cudaSuccess) return e;
  }
  kernel<<<p.grid, p.threads, p.smem, st>>>(a, p.ring, p.tpr);
  return cudaGetLastError();
}

// Columns per thread, the largest block and the blocks on an SM, by the row's length.
template <typename F> void fwd_shape(int D, F&& go) {
  if (D <= 256) go(Int<8>{}, Int<kNarrow>{}, Int<8>{});
  else if (D <= 2048) go(Int<8>{}, Int<256>{}, Int<4>{});
  else if (D <= 4096) go(Int<16>{}, Int<256>{}, Int<2>{});
  else go(Int<16>{}, Int<512>{}, Int<1>{});
}
template <typename F> void bwd_shape(int D, F&& go) {
  if (D <= 256) go(Int<8>{}, Int<kNarrow>{}, Int<4>{});
  else if (D <= 2048) go(Int<8>{}, Int<256>{}, Int<2>{});
  else if (D <= 4096) go(Int<8>{}, Int<512>{}, Int<1>{});
  else go(Int<16>{}, Int<512>{}, Int<1>{});
}

}  // namespace

int block_norm_bwd_blocks(const BlockNormArgs& a, int sms) {
  int n = 0;
  bwd_shape(a.D, [&](auto e, auto, auto blocks) { n = Plan(a, sms, e, blocks, 16, false).grid; });
  return n;
}

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2;
  cudaError_t err = cudaSuccess;
  by_type(dtype, h_dtype, vectors(a, es_a, es_h), [&](auto ta, auto th, auto v) {
    fwd_shape(a.D, [&](auto e, auto threads, auto blocks) {
      err = launch(block_norm_fwd_kernel<decltype(ta), decltype(th), decltype(v)::value, decltype(e)::value,
                                         decltype(threads)::value, decltype(blocks)::value>,
                   Plan(a, sms, e, blocks, row_bytes(a, es_a, es_h), false), a, st);
    });
  });
  return err;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, float* d_scale, float* d_post,
                                  float* d_pre, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2;
  cudaError_t err = cudaSuccess;
  int grid = 0;
  by_type(dtype, h_dtype, vectors(a, es_a, es_h), [&](auto ta, auto th, auto v) {
    bwd_shape(a.D, [&](auto e, auto threads, auto blocks) {
      const Plan p(a, sms, e, blocks, row_bytes(a, es_a, es_h), a.part != nullptr);
      grid = p.grid;
      err = launch(block_norm_bwd_kernel<decltype(ta), decltype(th), decltype(v)::value, decltype(e)::value,
                                         decltype(threads)::value, decltype(blocks)::value>,
                   p, a, st);
    });
  });
  if (err != cudaSuccess || !a.part) return err;
  join_parts_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, st>>>(a.part, grid, a.D, a.scale, a.post_w, d_scale, d_post, d_pre);
  return cudaGetLastError();
}

}  // namespace dr
