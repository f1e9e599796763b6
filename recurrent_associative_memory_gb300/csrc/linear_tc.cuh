// linear_tc.cuh — what the tcgen05 matrix-product kernels share: operands and their tensor
// maps, instructions over a pair of CTAs, and the epilogue.
//
// C[m,n] = sum_k A[m,k] B[n,k].  Either operand is stored with k contiguous (K-major) or with
// its rows contiguous (MN-major: the weight of a forward product, both operands of a weight's
// gradient); the tensor cores take both, so nothing is ever transposed in memory.
#pragma once

#include "attn_tc.cuh"
#include "block.cuh"

namespace dr {

// A copy of a matrix, its columns contiguous, with rows of `pitch` (fp32: three of them,
// `piece` apart).
struct PackJob {
  const void* src;
  void* dst;
  long long stride, piece;
  int rows, cols, pitch;
};

namespace lin {

using namespace umma;
using attn::elect_one;
using attn::tmem_ld32;
using attn::uniform;
using attn::wait_phase;

constexpr int kBK = 64;     // k of a stage: 128 bytes, the swizzle's width

// One operand: rows x k, bf16.  Rows (K-major) or steps of k (MN-major) are `stride` apart.
// An fp32 operand comes as three of them, `piece` apart, whose sum it is: bf16(x), bf16 of
// what that leaves, and again.
struct Operand {
  const void* p;
  int rows, k;
  long long stride;
  bool mn;
  long long piece = 0;   // 0: bf16
};

// Where a product stands in its call: first, behind the kernel whose results it reads, or behind
// a product whose results it does not read: it begins on the SMs that the last tiles of that one
// leave, and waits for it before it ends (all gradients of bf16 M8192 K2048 N8192: 256 tiles on
// 76 pairs twice; with the launches above the call's 560 us became 515).
enum Place { kFirst, kAfter, kBeside };

struct Epilogue {
  void* C;
  const void* bias;
  const void* res;
  void* slope;
  int M, N, act;
  Place place;
  long long r_m;       // C and the slope have rows of N
  int vec;             // 16 columns at once by 32-byte accesses: N is a multiple of 16, every row of C, res
                       // and slope starts on 32 bytes
};

inline bool make_operand_map(CUtensorMap* m, const Operand& o, int box_rows) {
  tc::EncodeTiledFn enc = tc::get_encode();
  if (!enc) return false;
  const cuuint64_t inner = o.mn ? o.rows : o.k, outer = o.mn ? o.k : o.rows;
  cuuint64_t dims[3] = {inner, outer, o.piece ? 3u : 1u};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(outer > 1 ? 2 * o.stride : (2 * inner + 15) / 16 * 16),
                           static_cast<cuuint64_t>(o.piece ? 2 * o.piece : 16)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(o.mn ? kBK : box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- a pair of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of the same place in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// "These columns of TMEM have been read", to either CTA of the pair: between tcgen05.wait::ld
// with its fence there and the fence behind the wait here nothing but tensor memory is handed
// over, so neither side needs an order of its other memory accesses.  (As a release over the
// cluster, an arrival takes 1450 cycles: M4096 K4096 N4096 in fp32, where a tile has 64 sums,
// 700 us instead of 485.)
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 255) == 0) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > attn::kWaitNs) return false;
    }
  }
}

// For an accumulator of n_k stages: the longest sums take seconds.
__device__ __forceinline__ bool wait_sum(uint64_t* bar, uint32_t parity, int n_k) {
  for (int i = 0; i <= n_k >> 20; ++i)
    if (wait_phase(bar, parity)) return true;
  return false;
}

// A box into this CTA's shared memory, its bytes counted on a barrier of either CTA.
__device__ __forceinline__ void pair_load(void* dst, const void* tmap, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void load_box(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Arrive on `bar`, in the CTAs of the mask, once every MMA issued so far has completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t ranks = 3) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(ranks)
      : "memory");
}

// ---------------------------------------------------------------- stages

// A stage holds 64 k of both operands.  bf16: the n_k stages of a tile in turns, one
// accumulator.  fp32: three stages per 64 k, the pieces 2, 1 and 0 of both operands, and six
// products of them, the smallest first (piece 1 is about 2^-8 of piece 0, piece 2 2^-16; what
// is left out is below 2^-25 of a term).  Their sum leaves TMEM after every 64 k and is added
// up in registers: the tensor cores cut each addition to the accumulator's 24 bits, which
// over thousands of k comes to 1e-5.
template <bool FP32> struct Walk {
  int n_k;
  __device__ __forceinline__ int sums() const { return FP32 ? n_k : 1; }      // accumulators per tile
  __device__ __forceinline__ int stages() const { return FP32 ? 3 * n_k : n_k; }
  __device__ __forceinline__ void at(int i, int& k, int& piece) const {
    if constexpr (FP32) k = i / 3, piece = 2 - (i - 3 * k);
    else k = i, piece = 0;
  }
};

// The products of one accumulator: full(stage) waits for a stage, mma(stage of A, stage of B,
// first of all) issues one product, free(stage) gives a stage back.  n counts stages.
template <bool FP32, int NS, typename Full, typename Mma, typename Free>
__device__ __forceinline__ bool products(int n_k, uint32_t& n, Full&& full, Mma&& mma, Free&& free) {
  if constexpr (FP32) {
    const uint32_t s2 = n % NS, s1 = (n + 1) % NS, s0 = (n + 2) % NS;
    for (int i = 0; i < 3; ++i)
      if (!full((n + i) % NS, ((n + i) / NS) & 1)) return false;
    mma(s0, s2, true);
    mma(s2, s0, false);
    free(s2);
    mma(s1, s1, false);
    mma(s0, s1, false);
    mma(s1, s0, false);
    free(s1);
    mma(s0, s0, false);
    free(s0);
    n += 3;
  } else {
    for (int i = 0; i < n_k; ++i, ++n) {
      const uint32_t s = n % NS;
      if (!full(s, (n / NS) & 1)) return false;
      mma(s, s, i == 0);
      free(s);
    }
  }
  return true;
}

// ---------------------------------------------------------------- epilogue

// 32 bytes at once
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* v) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}

// Brings the 128 bytes around p to L2: where a residual is read after the products, its rows
// come from memory meanwhile (M1003 K1511 N2051: 21.8 us instead of 22.9; where the next tile's
// products hide those loads it costs more than it gives, M8192 K4096 N4096 156 instead of 149).
__device__ __forceinline__ void to_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// f over n values, with their slopes or without
template <int N> __device__ __forceinline__ void act_all(int act, bool want, float (&v)[N], float (&s)[N]) {
  auto with = [&](auto code) {
    constexpr int A = decltype(code)::value;
    if (want) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_of<A>(v[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_of<A>(v[i]);
    }
  };
  switch (act) {
    case DR_ACT_RELU: with(std::integral_constant<int, DR_ACT_RELU>{}); break;
    case DR_ACT_SILU: with(std::integral_constant<int, DR_ACT_SILU>{}); break;
    case DR_ACT_GELU_TANH: with(std::integral_constant<int, DR_ACT_GELU_TANH>{}); break;
    case DR_ACT_SIGMOID: with(std::integral_constant<int, DR_ACT_SIGMOID>{}); break;
    default:   // x itself, and a slope of 1
      if (want) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 1.f;
      }
  }
}

// 16 values of a row, 32-byte aligned, to and from memory
template <typename T> __device__ __forceinline__ void put16(T* p, const float* v) {
  uint32_t w[8];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = tc::pack_bf16(v[2 * i], v[2 * i + 1]);
      }
    }
    store32(p, w);
  } else {
    store32(p, reinterpret_cast<const uint32_t*>(v));
    store32(p + 8, reinterpret_cast<const uint32_t*>(v) + 8);
  }
}
template <typename T> struct Raw16 {   // 16 values as they are held
  uint32_t w[sizeof(T) * 4];
  __device__ __forceinline__ void load(const T* p) {
    load32(p, w);
    if constexpr (sizeof(T) == 4) load32(p + 8, w + 8);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

}  // namespace lin
}  // namespace dr
