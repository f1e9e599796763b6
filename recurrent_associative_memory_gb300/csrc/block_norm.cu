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
//
// bf16 with every part: forward M16384 D4096 104 us, 6.4 TB/s, memory bounds it; backward M8192
// D4096 125 us, 4.3 TB/s: latency, with 16 warps on an SM as the registers allow.  Issue slots are
// 48 % busy and no pipe above 32 % (fma; alu 26, lsu 14, xu 9); of the 8.4 cycles that a warp has
// per instruction 2.2 wait for shared memory, shuffles and exponentials, 1.8 for the instruction
// before, 0.5 at a barrier and 0.4 for memory.
#include <type_traits>

#include "block_norm_rows.cuh"
#include "umma.cuh"

namespace dr {
namespace {

using namespace norm_rows;

// 8 of a thread's values of row `row`, from e on, from its copy at `at` in shared memory (RING), or from memory.
template <typename T, bool RING, int ORDER, int E>
__device__ __forceinline__ void row_values(const void* base, long long row, long long stride, uint32_t at, int M,
                                           const Columns<ORDER, E>& c, int e0, f2 (&r)[4]) {
  float f[8];
  const T* p = static_cast<const T*>(base) + row * stride;
  const int n = c.at(e0);
  if constexpr (ORDER == kApart) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c.in(c.at(e0 + e)) ? to_f(p[c.at(e0 + e)]) : 0.f;
  } else if (RING && ORDER == kOdd ? row == M - 1 && !c.whole(e0, n) : !c.whole(e0, n)) {
    // a ring's copy does not hold a group of the tensor's last row that is not whole
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = ORDER != kEven && c.in(n + e) ? to_f(p[n + e]) : 0.f;
  } else {
    uint32_t w[2 * sizeof(T)];
    // a thread without columns reads those of the row's first group, and no bit of it stays
    const int from = ORDER == kOdd && n >= c.D ? 0 : n + c.phase();
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); i += 4) {
      if constexpr (RING) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                     : "r"(at + from * (int)sizeof(T) + 4 * i)
                     : "memory");
      } else {
        const uint4 u = reinterpret_cast<const uint4*>(p + n)[i / 4];
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t x;
      if constexpr (sizeof(T) == 2) x = e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16;
      else x = w[e];
      // what is copied along of the neighbouring rows may be anything
      if (RING && ORDER == kOdd) x &= static_cast<uint32_t>(static_cast<int32_t>(c.valid << (31 - e0 - e)) >> 31);
      f[e] = __uint_as_float(x);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2(f[2 * i], f[2 * i + 1]);
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

// The same 8 of a vector over the channels, on any address.
template <int ORDER, int E>
__device__ __forceinline__ void load_vector(const float* p, const Columns<ORDER, E>& c, int e0, f2 (&r)[4]) {
  float f[8];
  if (ORDER != kApart && c.whole(e0, c.at(e0)) && (reinterpret_cast<uintptr_t>(p + c.at(e0)) & 15) == 0) {
    load8(p + c.at(e0), 1, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c.in(c.at(e0 + e)) ? p[c.at(e0 + e)] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2(f[2 * i], f[2 * i + 1]);
}

template <typename T, int ORDER, int E>
__device__ __forceinline__ void store_group(T* p, const Columns<ORDER, E>& c, int e0, const f2 (&r)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(r[i], f[2 * i], f[2 * i + 1]);
  const int n = c.at(e0);
  if (ORDER != kApart && c.whole(e0, n)) {
    store8(p + n, f);
  } else if (ORDER == kOdd) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c.valid >> (e0 + e) & 1u) p[n + e] = from_f<T>(f[e]);
  } else if (ORDER == kApart) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c.in(c.at(e0 + e))) p[c.at(e0 + e)] = from_f<T>(f[e]);
  }
}

// All E of them.
template <int ORDER, int E> __device__ __forceinline__ void load_vector(const float* p, const Columns<ORDER, E>& c, f2 (&r)[E / 2]) {
#pragma unroll
  for (int g = 0; g < E; g += 8) load_vector(p, c, g, reinterpret_cast<f2(&)[4]>(r[g / 2]));
}
template <typename T, int ORDER, int E>
__device__ __forceinline__ void store_row(T* p, const Columns<ORDER, E>& c, const f2 (&r)[E / 2]) {
#pragma unroll
  for (int g = 0; g < E; g += 8) store_group(p, c, g, reinterpret_cast<const f2(&)[4]>(r[g / 2]));
}

// The rows of a block.  RING: one at a time, through a ring of `stages` of them in shared
// memory.  Tensor i of a row is copied by a thread of warp i (blocks of fewer warps: by a second
// one of a warp), once the block has passed a barrier behind the reads of the row whose place it
// takes: the first one of the next row.  (What a copy costs its warp, the others wait for: issued
// by one thread for all tensors M16384 D4096 forward took 156 us instead of 103, and with the
// addresses formed for each row M8192 D4096 backward 143 instead of 137.  A warp of its own
// would cost the others their registers.)  Otherwise straight from memory.
template <int N> struct Ring {
  uint64_t* full;
  uint32_t at, stage_bytes;   // shared memory of stage 0; from stage to stage
  int stages;
  const void* base[N];
  long long stride[N];
  uint32_t off[N];            // of the tensors in a stage
  int es[N], M;
  int stage;
  uint32_t parity;
  bool lost;
  // this thread's tensor: where its next copy comes from, and the one after it; its place in a
  // stage; the bytes of a row, and of the tensor's last one
  uintptr_t from;
  long long from_step;
  uint32_t to, bytes, last_bytes;
  bool mine;

  // This thread's tensor of `row`, the rows in their order.
  __device__ __forceinline__ void issue(long long row, int s) {
    const uint32_t n = row == M - 1 ? last_bytes : bytes;
    umma::mbar_expect_tx(full + s, n);
    if (n)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       to + s * stage_bytes),
                   "l"(from), "r"(n), "r"(umma::smem_u32(full + s))
                   : "memory");
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
  __device__ __forceinline__ void refill(long long row, long long first, long long step) {
    const long long next = row + (stages - 1) * step;
    if (mine && row > first && next < M) {
      issue(next, stage == 0 ? stages - 1 : stage - 1);
      from += from_step;
    }
  }
  // No copy may be in flight when the block ends; only after a wait that gave up there can be.
  __device__ __forceinline__ void drain() {
    if (!lost) return;
    for (int i = 0; i < stages; ++i) {
      umma::mbar_wait(full + stage, parity, 500000000ull);
      next();
    }
  }
  template <typename T, bool RING, int ORDER, int E>
  __device__ __forceinline__ void get(int i, long long row, const Columns<ORDER, E>& c, int e0, f2 (&r)[4]) const {
    row_values<T, RING>(base[i], row, stride[i], at + stage * stage_bytes + off[i], M, c, e0, r);
  }
  template <typename T, bool RING, int ORDER, int E>
  __device__ __forceinline__ void get(int i, long long row, const Columns<ORDER, E>& c, f2 (&r)[E / 2]) const {
#pragma unroll
    for (int g = 0; g < E; g += 8) get<T, RING>(i, row, c, g, reinterpret_cast<f2(&)[4]>(r[g / 2]));
  }
};

__device__ __forceinline__ void clear(float (&bufs)[2][32]) {   // the parts of warps that a block has not
  for (int i = threadIdx.x; i < 64; i += blockDim.x) bufs[i / 32][i % 32] = 0.f;
  __syncthreads();
}

// One or two sums over the threads of a row at once, the same in each of them.  Rows of up to
// 32 threads stay within a warp; a wider one has its block to itself and goes through shared
// memory, two buffers in turn so that one barrier does: whoever writes a buffer again has
// passed the other one's barrier, which everyone reached after reading the first.
// Two sums share the shuffles: after the first each half of a warp has one of them.  One sum's
// parts every thread adds up for itself, 16 values at the same addresses for all: shorter than
// four more shuffles (bf16 M32768 D1024 70 + 126 -> 66 + 122 us, M2731 D1111 35 -> 33), two
// sums' were not (M65536 D300 153 us, so 162).
template <bool WIDE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr, float (&bufs)[2][32], int& turn) {
  static_assert(N <= 2, "");
  if constexpr (!WIDE) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < tpr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
  } else {
    float* buf = bufs[turn];
    turn ^= 1;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool up = lane & 16;
    auto half = [&](float x) {   // over the 16 lanes
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      return x;
    };
    float x;
    if constexpr (N == 2) x = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    else x = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
    x = half(x);
    if (lane % 16 == 0 && (N == 2 || !up)) buf[(up ? 16 : 0) + warp] = x;
    __syncthreads();
    if constexpr (N == 1) {
      f2 q[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 u = reinterpret_cast<const float4*>(buf)[i];
        q[2 * i] = pack2(u.x, u.y), q[2 * i + 1] = pack2(u.z, u.w);
      }
#pragma unroll
      for (int n = 4; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) q[i] = add2(q[i], q[i + n]);
      unpack2(q[0], v[0], x);
      v[0] += x;
    } else {   // 16 warps at most: a sum's parts are one half's
      x = half((lane & 15) * 32 < tpr ? buf[lane] : 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, 16 * i);
    }
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

template <int N, int ORDER, int E>
__device__ __forceinline__ void start(Ring<N>& ring, uint64_t (&bars)[kMaxStages], const RingLayout& l,
                                      const Columns<ORDER, E>& c, long long row, long long step, int M) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  ring.full = bars;
  ring.at = umma::smem_u32(dynamic);
  ring.stage_bytes = l.stage_bytes;
  ring.stages = l.stages;
  ring.M = M;
  ring.stage = 0, ring.parity = 0, ring.lost = false;
  uint32_t at = 0;
  int there = 0;
  ring.mine = false;
  ring.from = 0, ring.from_step = 0, ring.to = ring.bytes = ring.last_bytes = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ring.off[i] = at;
    if (!ring.base[i]) continue;
    if (static_cast<int>(threadIdx.x / 32 + threadIdx.x % 32 * (c.tpr / 32)) == i) {
      const RowCopy usual(ring.base[i], row, ring.stride[i], c.D, c.phase(), ring.es[i], -1);
      ring.mine = true;
      ring.from = usual.lo, ring.from_step = step * ring.stride[i] * ring.es[i];
      ring.to = ring.at + at;
      ring.bytes = usual.bytes;
      ring.last_bytes = RowCopy(ring.base[i], M - 1, ring.stride[i], c.D, c.phase(), ring.es[i], M).bytes;
    }
    at += copy_bytes(c.D, ring.es[i]), ++there;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < l.stages; ++i) umma::mbar_init(ring.full + i, there);
    umma::fence_mbar_init();
  }
  __syncthreads();
  if (ring.mine)
    for (int i = 0; i < l.stages && row + i * step < M; ++i) {
      ring.issue(row + i * step, i);
      ring.from += ring.from_step;
    }
}

// THREADS: kNarrow, or the largest block that the kernel is built for; BLOCKS of them on an SM.
template <typename TA, typename TH, int ORDER, int E, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_norm_fwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  constexpr bool WIDE = THREADS != kNarrow, RING = WIDE && ORDER != kApart;
  // fp32 rows fill the ring with two of them: the next copies begin as soon as they can, behind the
  // first of two sums (M4096 D4096 66 -> 59 us); bf16 ones, four and more, only waited for their
  // issue there (M8192 D4096 59 -> 61)
  constexpr bool EARLY = RING && sizeof(TA) == 4;
  constexpr int P = E / 2;
  using Row = f2[P];
  __shared__ __align__(16) float buf[2][32];
  if (WIDE) clear(buf);
  __shared__ uint64_t bars[kMaxStages];
  int turn = 0;
  const int rows = WIDE ? 1 : kNarrow / tpr, slot = WIDE ? 0 : threadIdx.x / tpr;
  const long long step = (long long)gridDim.x * rows, first = (long long)blockIdx.x * rows;
  const Columns<ORDER, E> c(a.D, tpr, static_cast<int>(threadIdx.x) - slot * tpr, phase_of(first + slot, a.D));
  Ring<3> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s;
  ring.es[0] = sizeof(TH), ring.es[1] = ring.es[2] = sizeof(TA);
  if (RING) start(ring, bars, l, c, first, step, a.M);
  Row ws, wy;   // scale post_w; pre_w
  fill(ws, 1.f), fill(wy, 1.f);
  if (a.pre_w) load_vector(a.pre_w, c, wy);
  if (a.scale) load_vector(a.scale, c, ws);
  if (a.post_w) {
    Row w;
    load_vector(a.post_w, c, w);
    pairs<P>([&](int i) { ws[i] = mul2(ws[i], w[i]); });
  }
  long long row = first + slot;
  // rows of other slots of the same warp may end earlier: those go on with zeros
  for (long long r0 = first; r0 < a.M; r0 += step, row += step) {
    const bool live = WIDE || row < a.M;
    Row h, u, f;
    if (!WIDE) fill(h, 0.f), fill(u, 0.f), fill(f, 0.f);
    if (RING) ring.wait();
    if (live) {
      if (a.branch) ring.template get<TA, RING>(1, row, c, u);
      ring.template get<TH, RING>(0, row, c, h);
      if (a.gate) {
        Row z, none;
        ring.template get<TA, RING>(2, row, c, z);
        gate_of<false>(a.gate_act, z, f, none);
      }
    }
    if (a.branch) {
      float rstd = 1.f;
      if (a.post_norm) {
        float s[1] = {dot(u, u)};
        row_sums<WIDE>(s, tpr, buf, turn);
        if (EARLY) ring.refill(row, first, step);
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
      if (RING && !(EARLY && a.branch && a.post_norm)) ring.refill(row, first, step);
      pairs<P>([&](int i) { h[i] = mul2(h[i], mul2(both(rstd), wy[i])); });
      if (live) store_row(static_cast<TA*>(a.y) + row * a.D, c, h);
    } else if (RING && !(EARLY && a.branch && a.post_norm)) {
      __syncthreads();
      ring.refill(row, first, step);
    }
    if (RING) ring.next();
  }
  if (RING) ring.drain();
}

template <typename TA, typename TH, int ORDER, int E, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_norm_bwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  constexpr bool WIDE = THREADS != kNarrow, RING = WIDE && ORDER != kApart && ring_holds<TH, E>();
  constexpr bool AGAIN = RING && E > 8;   // the branch is read twice, not kept (182 -> 168 us)
  constexpr int P = E / 2;
  using Row = f2[P];
  __shared__ __align__(16) float buf[2][32];
  if (WIDE) clear(buf);
  __shared__ uint64_t bars[kMaxStages];
  let_next_start();
  int turn = 0;
  const int D = a.D, rows = WIDE ? 1 : kNarrow / tpr, slot = WIDE ? 0 : threadIdx.x / tpr;
  const long long step = (long long)gridDim.x * rows, first = (long long)blockIdx.x * rows;
  const Columns<ORDER, E> c(D, tpr, static_cast<int>(threadIdx.x) - slot * tpr, phase_of(first + slot, D));
  Ring<5> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate, ring.base[3] = a.d_y, ring.base[4] = a.d_h;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s, ring.stride[3] = ring.stride[4] = D;
  ring.es[0] = ring.es[4] = sizeof(TH), ring.es[1] = ring.es[2] = ring.es[3] = sizeof(TA);
  if (RING) start(ring, bars, l, c, first, step, a.M);
  Row sum_s, sum_p;   // S, the sum of dpre_w
  Row ws_r, wy_r;     // scale post_w, pre_w
  fill(sum_s, 0.f), fill(sum_p, 0.f), fill(ws_r, 1.f), fill(wy_r, 1.f);
  if (a.pre_w) load_vector(a.pre_w, c, wy_r);
  if (a.scale) load_vector(a.scale, c, ws_r);
  if (a.post_w) {
    Row w;
    load_vector(a.post_w, c, w);
    pairs<P>([&](int i) { ws_r[i] = mul2(ws_r[i], w[i]); });
  }
  // 16 columns' weights would be spilled: they stay in shared memory behind the ring, where each
  // thread reads its own (bf16 M4096 D8192 217 -> 182 us, M2048 with an fp32 stream 150 -> 129)
  extern __shared__ __align__(16) uint8_t dynamic[];
  f2* own = reinterpret_cast<f2*>(dynamic + (RING ? l.stages * l.stage_bytes : 0)) + threadIdx.x;
  if (E > 8)
    pairs<P>([&](int i) { own[i * blockDim.x] = ws_r[i], own[(P + i) * blockDim.x] = wy_r[i]; });
  auto ws = [&](int i) { return E > 8 ? own[i * blockDim.x] : ws_r[i]; };
  auto wy = [&](int i) { return E > 8 ? own[(P + i) * blockDim.x] : wy_r[i]; };
  long long row = first + slot;
  for (long long r0 = first; r0 < a.M; r0 += step, row += step) {
    const bool live = WIDE || row < a.M;
    // a row that is none: zeros, and norms of 0 (1 / sqrt(0 + eps) is none where eps is 0), so that
    // it adds nothing to any sum
    Row h, v, f, vs, g;   // vs: v f'(gate); AGAIN: f'(gate) until v is there again
    float rstd_b = 1.f;
    if (!WIDE) fill(h, 0.f), fill(v, 0.f);
    if (RING) ring.wait();
    if (live) ring.template get<TH, RING>(0, row, c, h);
    if (a.branch) {   // h' again
      if (live) ring.template get<TA, RING>(1, row, c, v);
      if (a.post_norm) {
        float s[1] = {dot(v, v)};
        row_sums<WIDE>(s, tpr, buf, turn);
        if (RING) ring.refill(row, first, step);
        rstd_b = live ? rsqrtf(fmaf(s[0], a.inv_d, a.eps)) : 0.f;
        pairs<P>([&](int i) { v[i] = mul2(v[i], both(rstd_b)); });
      }
      if (a.gate) {
        Row z;
        if (!WIDE) fill(z, 0.f);
        if (live) ring.template get<TA, RING>(2, row, c, z);
        gate_of<true>(a.gate_act, z, f, vs);
        if (!AGAIN) pairs<P>([&](int i) { vs[i] = mul2(vs[i], v[i]); });
      } else {
        fill(f, 1.f);
      }
      pairs<P>([&](int i) { h[i] = fma2(mul2(f[i], v[i]), ws(i), h[i]); });
    }
    if (a.d_y) {
      Row dy, t;
      if (!WIDE) fill(dy, 0.f);
      if (live) ring.template get<TA, RING>(3, row, c, dy);
      pairs<P>([&](int i) { t[i] = mul2(dy[i], wy(i)); });
      float s[2] = {dot(h, h), dot(t, h)};
      row_sums<WIDE>(s, tpr, buf, turn);
      const float rstd = live ? rsqrtf(fmaf(s[0], a.inv_d, a.eps)) : 0.f;
      const f2 k = both(-s[1] * a.inv_d * rstd * rstd), r2 = both(rstd);
      pairs<P>([&](int i) {
        h[i] = mul2(h[i], r2);
        sum_p[i] = fma2(dy[i], h[i], sum_p[i]);
        t[i] = fma2(t[i], r2, mul2(k, h[i]));
      });
      if (a.d_h) {
        if (!WIDE) fill(g, 0.f);
        if (live) ring.template get<TH, RING>(4, row, c, g);
        pairs<P>([&](int i) { g[i] = add2(g[i], t[i]); });
      } else {
        pairs<P>([&](int i) { g[i] = t[i]; });
      }
    } else {
      if (!WIDE) fill(g, 0.f);
      if (live) ring.template get<TH, RING>(4, row, c, g);
      if (RING) __syncthreads();
    }
    if (RING && !(a.branch && a.post_norm)) ring.refill(row, first, step);
    if (RING && !AGAIN) ring.next();
    if (live && a.dh) store_row(static_cast<TH*>(a.dh) + row * D, c, g);
    if (!a.branch) {
      if (RING && AGAIN) ring.next();
      continue;
    }
    if (AGAIN) {
      ring.template get<TA, RING>(1, row, c, v);
      if (a.post_norm) pairs<P>([&](int i) { v[i] = mul2(v[i], both(rstd_b)); });
      if (a.gate) pairs<P>([&](int i) { vs[i] = mul2(vs[i], v[i]); });
    }
    pairs<P>([&](int i) {
      const f2 x = mul2(g[i], ws(i));
      sum_s[i] = fma2(g[i], mul2(f[i], v[i]), sum_s[i]);
      if (a.gate) vs[i] = mul2(x, vs[i]);
      g[i] = mul2(x, f[i]);   // q from here on
    });
    if (live && a.dg) store_row(static_cast<TA*>(a.dg) + row * D, c, vs);
    if (a.post_norm) {
      float s[1] = {dot(g, v)};
      row_sums<WIDE>(s, tpr, buf, turn);
      const f2 k = both(-s[0] * a.inv_d * rstd_b), r2 = both(rstd_b);
      pairs<P>([&](int i) { g[i] = fma2(k, v[i], mul2(r2, g[i])); });
    }
    if (RING && AGAIN) ring.next();
    if (live && a.db) store_row(static_cast<TA*>(a.db) + row * D, c, g);
  }
  if (RING) ring.drain();
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
      if (c.in(n)) to[n] = ss[e], to[D + n] = sp[e];
    }
  };
  if constexpr (WIDE) {
    each(part);
  } else {   // the block's rows, one after another
    float* slots = reinterpret_cast<float*>(dynamic);   // [rows][2][D]
    each(slots + slot * 2 * D);
    __syncthreads();
    for (int n = threadIdx.x; n < 2 * D; n += kNarrow) {
      float s = 0.f;
      for (int i = 0; i < rows; ++i) s += slots[i * 2 * D + n];
      part[n] = s;
    }
  }
}

// The sums over the blocks of part[block][which][D], 32 groups of threads over the blocks, joined
// in order: which 0 is S, of dscale and dpost_w, 1 is dpre_w.
__global__ void __launch_bounds__(1024) join_parts_kernel(const float* part, int blocks, int D, const float* scale,
                                                          const float* post_w, float* d_scale, float* d_post, float* d_pre) {
  __shared__ float buf[32][33];
  wait_for_last();
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32, which = blockIdx.y;
  if (which == 0 ? !d_scale && !d_post : !d_pre) return;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D)
    for (int b = g; b < blocks; b += 32) s += part[((long long)b * 2 + which) * D + c];
  buf[g][lane] = s;
  __syncthreads();
  s = buf[lane][g];   // a warp per column now
  s = warp_sum(s);
  const int n = blockIdx.x * 32 + g;
  if (lane != 0 || n >= D) return;
  if (which == 1) {
    d_pre[n] = s;
    return;
  }
  if (d_scale) d_scale[n] = post_w ? s * post_w[n] : s;
  if (d_post) d_post[n] = scale ? s * scale[n] : s;
}

template <typename F> void by_type(int dtype, int h_dtype, int order, F&& go) {
  auto types = [&](auto v) {
    if (dtype == DR_FP32) go(float{}, float{}, v);
    else if (h_dtype == DR_FP32) go(__nv_bfloat16{}, float{}, v);
    else go(__nv_bfloat16{}, __nv_bfloat16{}, v);
  };
  if (order == kEven) types(Int<kEven>{});
  else if (order == kOdd) types(Int<kOdd>{});
  else types(Int<kApart>{});
}

template <typename K> cudaError_t launch(K* kernel, const Plan& p, const BlockNormArgs& a, cudaStream_t st) {
  if (p.smem > 40 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
  }
  kernel<<<p.grid, p.threads, p.smem, st>>>(a, p.ring, p.tpr);
  return cudaGetLastError();
}

}  // namespace

// the most that any order of the columns takes
int block_norm_bwd_blocks(const BlockNormArgs& a, int sms) {
  int n = 0;
  for (int order : {kEven, kOdd, kApart})
    bwd_shape(a.D, order, [&](auto e, auto threads, auto blocks) {
      const int g = Plan(a, sms, order, e, threads * blocks, false, 16, false).grid;
      n = n > g ? n : g;
    });
  return n;
}

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2, order = order_of(a);
  cudaError_t err = cudaSuccess;
  by_type(dtype, h_dtype, order, [&](auto ta, auto th, auto o) {
    fwd_shape(a.D, order, [&](auto e, auto threads, auto blocks) {
      err = launch(block_norm_fwd_kernel<decltype(ta), decltype(th), decltype(o)::value, decltype(e)::value,
                                         decltype(threads)::value, decltype(blocks)::value>,
                   Plan(a, sms, order, e, threads * blocks, true, row_bytes(a, es_a, es_h), false), a, st);
    });
  });
  return err;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, float* d_scale, float* d_post,
                                  float* d_pre, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2, order = order_of(a);
  cudaError_t err = cudaSuccess;
  int grid = 0;
  by_type(dtype, h_dtype, order, [&](auto ta, auto th, auto o) {
    bwd_shape(a.D, order, [&](auto e, auto threads, auto blocks) {
      const Plan p(a, sms, order, e, threads * blocks, ring_holds<decltype(th), decltype(e)::value>(),
                   row_bytes(a, es_a, es_h), a.part != nullptr, bwd_own(e));
      grid = p.grid;
      err = launch(block_norm_bwd_kernel<decltype(ta), decltype(th), decltype(o)::value, decltype(e)::value,
                                         decltype(threads)::value, decltype(blocks)::value>,
                   p, a, st);
    });
  });
  if (err != cudaSuccess || !a.part) return err;
  return launch_in_call(true, join_parts_kernel, dim3((a.D + 31) / 32, 2), 1024, 0, st, 0, a.part, grid, a.D, a.scale, a.post_w,
                        d_scale, d_post, d_pre);
}

}  // namespace dr
