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
#include <type_traits>

#include "block.cuh"
#include "umma.cuh"

namespace dr {
namespace {

constexpr int kE = 8;            // columns per thread
constexpr int kMaxStages = 8;

// A thread's columns of a row: 8 neighbours where rows start on 16 bytes, else one of every
// tpr so that a warp's accesses stay next to each other.
template <int VEC> struct Columns {
  int D, tpr, t;
  __device__ __forceinline__ int at(int e) const { return VEC == 8 ? 8 * t + e : e * tpr + t; }
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

// A thread's values of a row whose copy stands at `at` in shared memory.
template <typename T, int VEC>
__device__ __forceinline__ void row_values(const RowCopy& r, uint32_t at, const Columns<VEC>& c, float (&f)[kE]) {
  if constexpr (VEC == 8) {
    if (8 * c.t >= c.D) {
#pragma unroll
      for (int e = 0; e < kE; ++e) f[e] = 0.f;
      return;
    }
    uint32_t w[2 * sizeof(T)];
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); i += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(at + 8 * c.t * (int)sizeof(T) + 4 * i)
                   : "memory");
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if constexpr (sizeof(T) == 2) f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
      else f[e] = __uint_as_float(w[e]);
    }
  } else {
    const uint32_t head = static_cast<uint32_t>(r.lo - r.p);   // bytes before the first unit
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      f[e] = 0.f;
      if (c.at(e) >= c.D) continue;
      const uint32_t b = c.at(e) * (uint32_t)sizeof(T), in = b - head;   // below the row's start: huge
      if (in < r.bytes) {
        if constexpr (sizeof(T) == 2) {
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at + in) : "memory");
          f[e] = __uint_as_float(static_cast<uint32_t>(v) << 16);
        } else {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[e]) : "r"(at + in) : "memory");
        }
      } else {
        f[e] = to_f(*reinterpret_cast<const T*>(r.p + b));
      }
    }
  }
}

template <int VEC> __device__ __forceinline__ void load_vector(const float* p, const Columns<VEC>& c, float (&f)[kE]) {
  if constexpr (VEC == 8) {
    load8(p + 8 * c.t, 8 * c.t < c.D ? 1 : 0, f);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = c.at(e) < c.D ? p[c.at(e)] : 0.f;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const Columns<VEC>& c, const float (&f)[kE]) {
  if constexpr (VEC == 8) {
    if (8 * c.t < c.D) store8(p + 8 * c.t, f);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (c.at(e) < c.D) p[c.at(e)] = from_f<T>(f[e]);
  }
}

// The ring of rows of a row slot: its first thread issues a row's copies, counted on the
// slot's barrier of that stage, `stages` rows ahead of the one that is worked on.
template <int N> struct Ring {
  uint64_t* bar;            // [stages], of this slot
  uint32_t at, stage_bytes; // shared memory of stage 0 of this slot; from stage to stage
  int stages;
  const void* base[N];
  long long stride[N];
  uint32_t off[N];          // of the tensors in a stage
  int es[N];
  bool lost;

  __device__ __forceinline__ void issue(long long row, int stage, int D) {
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (base[i]) bytes += RowCopy(base[i], row, stride[i], D, es[i]).bytes;
    umma::mbar_expect_tx(bar + stage, bytes);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!base[i]) continue;
      const RowCopy r(base[i], row, stride[i], D, es[i]);
      if (r.bytes)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                at + stage * stage_bytes + off[i]),
            "l"(r.lo), "r"(r.bytes), "r"(umma::smem_u32(bar + stage))
            : "memory");
    }
  }
  // Bounded; after one that gave up none waits any more, and what comes out means nothing.
  __device__ __forceinline__ void wait(int stage, uint32_t parity) {
    if (lost || umma::mbar_wait(bar + stage, parity, 2000000000ull)) return;
    lost = true;
    set_status(DR_ERR_TIMEOUT);
  }
  template <typename T, int VEC>
  __device__ __forceinline__ void get(int i, long long row, int stage, const Columns<VEC>& c, float (&f)[kE]) const {
    row_values<T>(RowCopy(base[i], row, stride[i], c.D, sizeof(T)), at + stage * stage_bytes + off[i], c, f);
  }
};

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

// How a launch lays the rows' copies out.
struct RingLayout {
  int stages;
  uint32_t slot_bytes;   // of all tensors of a row
};

// Sets a slot's ring up and starts its first rows.
template <int N, int VEC>
__device__ __forceinline__ void start(Ring<N>& ring, uint64_t (&bars)[32 * kMaxStages], const RingLayout& l, const Columns<VEC>& c,
                                      int rows, int slot, long long row, long long step, int M) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  ring.bar = bars + slot * l.stages;
  ring.at = umma::smem_u32(dynamic) + slot * l.slot_bytes;
  ring.stage_bytes = rows * l.slot_bytes;
  ring.stages = l.stages;
  ring.lost = false;
  uint32_t at = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ring.off[i] = at;
    if (ring.base[i]) at += (c.D * ring.es[i] + 15) / 16 * 16;
  }
  if (c.t == 0) {
    for (int i = 0; i < l.stages; ++i) umma::mbar_init(ring.bar + i, 1);
    umma::fence_mbar_init();
    for (int i = 0; i < l.stages && row + i * step < M; ++i) ring.issue(row + i * step, i, c.D);
  }
  __syncthreads();
}

// A row has been read by all of its threads: its place goes to the row `stages` further on.
template <int N, int VEC>
__device__ __forceinline__ void next(Ring<N>& ring, const Columns<VEC>& c, long long row, long long step, int M, int& stage,
                                     uint32_t& parity) {
  if (c.tpr > 32) __syncthreads();
  else __syncwarp();
  if (c.t == 0 && row + ring.stages * step < M) ring.issue(row + ring.stages * step, stage, c.D);
  if (++stage == ring.stages) stage = 0, parity ^= 1;
}

// No copy may be in flight when the block ends; only after a wait that gave up there can be.
template <int N, int VEC>
__device__ __forceinline__ void drain(Ring<N>& ring, const Columns<VEC>& c, long long row, long long step, int M, int stage,
                                      uint32_t parity) {
  if (!ring.lost || c.t != 0) return;
  for (int i = 0; i < ring.stages && row + i * step < M; ++i) {
    umma::mbar_wait(ring.bar + stage, parity, 2000000000ull);
    if (++stage == ring.stages) stage = 0, parity ^= 1;
  }
}

// Threads on an SM, by the registers that they need: 64 forward, 128 backward and where the
// columns of a thread are not neighbours.
constexpr int fwd_threads(int vec, int size) { return vec == 8 || size > 512 ? 1024 : 512; }
constexpr int bwd_threads(int size) { return size > 512 ? 1024 : 512; }

// THREADS: the largest block that the kernel is built for.
template <typename TA, typename TH, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, fwd_threads(VEC, THREADS) / THREADS)
    block_norm_fwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  __shared__ float buf[2][64];
  __shared__ uint64_t bars[32 * kMaxStages];
  int turn = 0, stage = 0;
  uint32_t parity = 0;
  const Columns<VEC> c{a.D, tpr, static_cast<int>(threadIdx.x) % tpr};
  const int rows = blockDim.x / tpr, slot = threadIdx.x / tpr;
  const long long step = (long long)gridDim.x * rows;
  long long row = (long long)blockIdx.x * rows + slot;
  Ring<3> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s;
  ring.es[0] = sizeof(TH), ring.es[1] = ring.es[2] = sizeof(TA);
  start(ring, bars, l, c, rows, slot, row, step, a.M);
  float ws[kE], wy[kE];   // scale post_w; pre_w
#pragma unroll
  for (int e = 0; e < kE; ++e) ws[e] = wy[e] = 1.f;
  if (a.pre_w) load_vector(a.pre_w, c, wy);
  if (a.scale) load_vector(a.scale, c, ws);
  if (a.post_w) {
    float w[kE];
    load_vector(a.post_w, c, w);
#pragma unroll
    for (int e = 0; e < kE; ++e) ws[e] *= w[e];
  }
  // rows of other slots of the same warp may end earlier: those go on with zeros
  for (long long r0 = (long long)blockIdx.x * rows; r0 < a.M; r0 += step, row += step) {
    const bool live = row < a.M;
    float h[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) h[e] = 0.f;
    if (live) {
      ring.wait(stage, parity);
      ring.template get<TH>(0, row, stage, c, h);
    }
    if (a.branch) {
      float u[kE];
#pragma unroll
      for (int e = 0; e < kE; ++e) u[e] = 0.f;
      if (live) ring.template get<TA>(1, row, stage, c, u);
      float rstd = 1.f;
      if (a.post_norm) {
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < kE; ++e) s[0] = fmaf(u[e], u[e], s[0]);
        row_sums(s, tpr, buf, turn);
        rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      }
      if (a.gate && live) {
        float z[kE], f[kE], none[kE];
        ring.template get<TA>(2, row, stage, c, z);
        gate_of<false>(a.gate_act, z, f, none);
#pragma unroll
        for (int e = 0; e < kE; ++e) u[e] *= f[e];
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] = fmaf(u[e] * rstd, ws[e], h[e]);
    }
    next(ring, c, row, step, a.M, stage, parity);
    if (live && a.branch) store_row(static_cast<TH*>(a.h_out) + row * a.D, c, h);
    if (a.y) {
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < kE; ++e) s[0] = fmaf(h[e], h[e], s[0]);
      row_sums(s, tpr, buf, turn);
      const float rstd = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] *= rstd * wy[e];
      if (live) store_row(static_cast<TA*>(a.y) + row * a.D, c, h);
    }
  }
  drain(ring, c, row, step, a.M, stage, parity);
}

template <typename TA, typename TH, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, bwd_threads(THREADS) / THREADS)
    block_norm_bwd_kernel(BlockNormArgs a, RingLayout l, int tpr) {
  __shared__ float buf[2][64];
  __shared__ uint64_t bars[32 * kMaxStages];
  int turn = 0, stage = 0;
  uint32_t parity = 0;
  const Columns<VEC> c{a.D, tpr, static_cast<int>(threadIdx.x) % tpr};
  const int D = a.D, rows = blockDim.x / tpr, slot = threadIdx.x / tpr;
  const long long step = (long long)gridDim.x * rows;
  long long row = (long long)blockIdx.x * rows + slot;
  Ring<5> ring;
  ring.base[0] = a.h, ring.base[1] = a.branch, ring.base[2] = a.gate, ring.base[3] = a.d_y, ring.base[4] = a.d_h;
  ring.stride[0] = a.h_s, ring.stride[1] = a.b_s, ring.stride[2] = a.g_s, ring.stride[3] = ring.stride[4] = D;
  ring.es[0] = ring.es[4] = sizeof(TH), ring.es[1] = ring.es[2] = ring.es[3] = sizeof(TA);
  start(ring, bars, l, c, rows, slot, row, step, a.M);
  float sum_s[kE] = {}, sum_q[kE] = {}, sum_p[kE] = {};   // of scale, post_w, pre_w
  for (long long r0 = (long long)blockIdx.x * rows; r0 < a.M; r0 += step, row += step) {
    const bool live = row < a.M;
    // a row that is none: zeros, so that it adds nothing to any sum
    float h[kE], u[kE], v[kE], f[kE], fs[kE], w[kE], g[kE];
    float rstd_b = 1.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) h[e] = u[e] = v[e] = g[e] = fs[e] = 0.f, f[e] = 1.f;
    if (live) {
      ring.wait(stage, parity);
      ring.template get<TH>(0, row, stage, c, h);
    }
    if (a.branch) {   // h' again; u the branch's norm with its weight, v without it
      if (live) ring.template get<TA>(1, row, stage, c, v);
      if (a.gate && live) {
        float z[kE];
        ring.template get<TA>(2, row, stage, c, z);
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
        load_vector(a.post_w, c, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) u[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] = 1.f;
      if (a.scale) load_vector(a.scale, c, w);
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] = fmaf(w[e] * f[e], u[e], h[e]);
    }
    if (a.d_h && live) ring.template get<TH>(4, row, stage, c, g);
    if (a.d_y) {
      float dy[kE], s[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < kE; ++e) dy[e] = 0.f, w[e] = 1.f;
      if (live) ring.template get<TA>(3, row, stage, c, dy);
      if (a.pre_w) load_vector(a.pre_w, c, w);
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
        sum_p[e] = fmaf(dy[e], h[e] * rstd, sum_p[e]);
        g[e] = fmaf(dy[e] * w[e], rstd, fmaf(-k, h[e], g[e]));
      }
    }
    next(ring, c, row, step, a.M, stage, parity);
    if (live && a.dh) store_row(static_cast<TH*>(a.dh) + row * D, c, g);
    if (!a.branch) continue;
#pragma unroll
    for (int e = 0; e < kE; ++e) w[e] = 1.f;
    if (a.scale) load_vector(a.scale, c, w);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      sum_s[e] = fmaf(g[e] * f[e], u[e], sum_s[e]);
      fs[e] *= g[e] * w[e] * u[e];
      g[e] *= w[e] * f[e];   // du from here on
      sum_q[e] = fmaf(g[e], v[e], sum_q[e]);
    }
    if (live && a.dg) store_row(static_cast<TA*>(a.dg) + row * D, c, fs);
    if (a.post_norm) {
      if (a.post_w) {
        load_vector(a.post_w, c, w);
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
    if (live && a.db) store_row(static_cast<TA*>(a.db) + row * D, c, g);
  }
  drain(ring, c, row, step, a.M, stage, parity);
  if (!a.part) return;
  // rows of a warp first, then one after another over the slots of the block
  extern __shared__ __align__(16) uint8_t dynamic[];   // the ring's place: [rows][3][D]
  float* slots = reinterpret_cast<float*>(dynamic);
  float* part = a.part + (long long)blockIdx.x * 3 * D;
  auto each = [&](auto use) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if (c.at(e) < D) use(e, c.at(e));
    }
  };
  if (rows == 1) {
    each([&](int e, int n) { part[n] = sum_s[e], part[D + n] = sum_q[e], part[2 * D + n] = sum_p[e]; });
    return;
  }
  __syncthreads();
  each([&](int e, int n) {
    float* p = slots + (long long)slot * 3 * D;
    p[n] = sum_s[e], p[D + n] = sum_q[e], p[2 * D + n] = sum_p[e];
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

// threads per row: a power of two from 4 to 32, whole warps from there on, which have their
// block to themselves
int threads_of(int D) {
  const int n = (D + kE - 1) / kE;
  if (n > 32) return (n + 31) / 32 * 32;
  int t = 4;
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

template <int N> using Int = std::integral_constant<int, N>;

// types, width of an access and largest block of a call
template <typename F> void by_type(int dtype, int h_dtype, bool vec, int threads, F&& go) {
  auto size = [&](auto ta, auto th, auto v) {
    if (threads <= 256) go(ta, th, v, Int<256>{});
    else if (threads <= 512) go(ta, th, v, Int<512>{});
    else go(ta, th, v, Int<1024>{});
  };
  auto types = [&](auto v) {
    if (dtype == DR_FP32) size(float{}, float{}, v);
    else if (h_dtype == DR_FP32) size(__nv_bfloat16{}, float{}, v);
    else size(__nv_bfloat16{}, __nv_bfloat16{}, v);
  };
  if (vec) types(Int<8>{});
  else types(Int<1>{});
}

// A launch: blocks that stay on every SM, and the rows on their way in what
// each of them has of its shared memory.
struct Plan {
  int tpr, threads, grid;
  RingLayout ring;
  size_t smem;
  Plan(const BlockNormArgs& a, int sms, bool bwd, int vec, int row_bytes, bool sums) {
    tpr = threads_of(a.D);
    const int rows = rows_of(tpr);
    threads = tpr * rows;
    const int size = threads <= 256 ? 256 : threads <= 512 ? 512 : 1024;
    const int blocks = (bwd ? bwd_threads(size) : fwd_threads(vec, size)) / size;
    const long long most = (a.M + rows - 1LL) / rows;
    grid = static_cast<int>(most < (long long)sms * blocks ? most : (long long)sms * blocks);
    ring.slot_bytes = row_bytes;
    const long long stage = (long long)rows * row_bytes, there = (224 * 1024) / blocks - 4096;
    ring.stages = static_cast<int>(there / stage < kMaxStages ? there / stage : kMaxStages);
    if (ring.stages < 1) ring.stages = 1;
    const long long steps = (most + grid - 1) / (grid ? grid : 1);
    if (ring.stages > steps && steps > 0) ring.stages = static_cast<int>(steps);
    smem = ring.stages * stage;
    const size_t parts = sums && rows > 1 ? sizeof(float) * rows * 3 * a.D : 0;
    if (smem < parts) smem = parts;
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

}  // namespace

int block_norm_bwd_blocks(const BlockNormArgs& a, int sms) { return Plan(a, sms, true, 8, 16, false).grid; }

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2;
  const bool vec = vectors(a, es_a, es_h);
  const Plan p(a, sms, false, vec ? 8 : 1, row_bytes(a, es_a, es_h), false);
  cudaError_t e = cudaSuccess;
  by_type(dtype, h_dtype, vec, p.threads, [&](auto ta, auto th, auto v, auto n) {
    e = launch(block_norm_fwd_kernel<decltype(ta), decltype(th), decltype(v)::value, decltype(n)::value>, p, a, st);
  });
  return e;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, float* d_scale, float* d_post,
                                  float* d_pre, cudaStream_t st) {
  const int es_a = dtype == DR_FP32 ? 4 : 2, es_h = h_dtype == DR_FP32 ? 4 : 2;
  const Plan p(a, sms, true, 8, row_bytes(a, es_a, es_h), a.part != nullptr);
  cudaError_t e = cudaSuccess;
  by_type(dtype, h_dtype, vectors(a, es_a, es_h), p.threads, [&](auto ta, auto th, auto v, auto n) {
    e = launch(block_norm_bwd_kernel<decltype(ta), decltype(th), decltype(v)::value, decltype(n)::value>, p, a, st);
  });
  if (e != cudaSuccess || !a.part) return e;
  join_parts_kernel<<<dim3((a.D + 31) / 32, 3), 256, 0, st>>>(a.part, p.grid, a.D, d_scale, d_post, d_pre);
  return cudaGetLastError();
}

}  // namespace dr
