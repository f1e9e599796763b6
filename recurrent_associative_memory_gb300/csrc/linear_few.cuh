// linear_few.cuh — the matrix product on tcgen05 where C is small: few rows (single tokens, a
// short prompt), or few tiles.
//
// The roles are turned round: 128 columns n of C are the MMA's 128 rows, the rows m of C its
// N = TN columns, so that a handful of tokens wastes no tensor-core row and a weight tile is
// read once.  The sum over k is cut over the S CTAs of a cluster, each of which leaves its
// part of C in its shared memory; they add them up in the ranks' order, each for its share of
// the rows, so the result does not depend on which CTA is first.
//   warps 0-7  the accumulator to shared memory, then the sums and the epilogue, a row per warp
//   warp 8     TMA, 4 to 11 stages of 64 k
//   warp 9     the MMAs
// Weights are what bounds it, 16 KB of each stage, so an SM keeps 200 KB of them under way: bf16
// M64 K4096 N16384 29 us, 4.7 TB/s with the start and the end of its one wave; M1 K2048 N2048 8.6.
#pragma once

#include <type_traits>

#include "linear_tc.cuh"

namespace dr {
namespace lin {

constexpr int kFewThreads = 320, kFewWarps = 8, kFewLoadWarp = 8, kFewMmaWarp = 9;

template <int TN> struct FewSmem {
  static constexpr int kN = 128 * kBK * 2, kM = TN * kBK * 2, kStage = kN + kM;
  static constexpr int kStages = 200 * 1024 / kStage;
  static constexpr int kBytes = kStages * kStage + 1024;
  static_assert(kStages >= 4, "fp32 takes three of them at once");
  static_assert(TN * 128 * 4 <= kStages * kStage, "the parts of C take the stages' place");
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

struct FewGrid {
  int tiles_m, split;   // tiles of rows; CTAs over k
};

__device__ __forceinline__ float4 load_peer(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 4 neighbouring values; `whole`: at once, else those below n
template <typename T> __device__ __forceinline__ void get4(const T* p, bool whole, int n, float (&v)[4]) {
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
  } else if constexpr (sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  }
}
template <typename T> __device__ __forceinline__ void put4(T* p, bool whole, int n, const float (&v)[4]) {
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = static_cast<T>(v[i]);
  } else if constexpr (std::is_same<T, __half>::value) {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// N_MN, M_MN: the operands of C's columns and rows are MN-major
template <int TN, bool N_MN, bool M_MN, typename T, bool FULL>
__global__ void __launch_bounds__(kFewThreads, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmN, const __grid_constant__ CUtensorMap tmM, Epilogue e,
                      FewGrid g, int n_k) {
  static_assert(!M_MN || TN % 64 == 0, "a swizzled row of an MN-major operand is 64 of its rows");
  using L = FewSmem<TN>;
  using S = typename std::conditional<sizeof(T) == 2, __half, float>::type;
  constexpr bool FP32 = sizeof(T) == 4;
  constexpr int NS = L::kStages;
  constexpr int kCols = FP32 ? TN : 0;                                          // to the second accumulator
  constexpr int kAll = FP32 ? 2 * TN : TN;
  constexpr int kTmem = kAll <= 32 ? 32 : kAll <= 64 ? 64 : kAll <= 128 ? 128 : kAll <= 256 ? 256 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t b_full[NS], b_empty[NS], b_acc[2], b_free[2], b_end;
  __shared__ uint32_t s_tmem;
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
  const int m0 = tile % g.tiles_m * TN, n0 = tile / g.tiles_m * 128;
  const int k0 = static_cast<int>((long long)n_k * rank / g.split);
  const Walk<FP32> walk{static_cast<int>((long long)n_k * (rank + 1) / g.split) - k0};

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&b_acc[i], 1), mbar_init(&b_free[i], kFewWarps);
    mbar_init(&b_end, 1);
    fence_mbar_init();
  }
  if (warp == kFewMmaWarp) tmem_alloc(&s_tmem, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (e.place != kBeside) wait_for_last(), let_next_start();
  const uint32_t tmem = uniform(s_tmem);
  auto wait = [&](uint64_t* bar, uint32_t parity, int sum = 0) {
    const bool ok = wait_sum(bar, parity, sum);
    if (!ok) set_status(DR_ERR_TIMEOUT);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  float* part = reinterpret_cast<float*>(sm);   // [TN][128]

  if (warp < kFewWarps) {   // ---------------------------------------------- accumulators
    constexpr int H = TN / 2, C = H % 32 == 0 ? 32 : H % 16 == 0 ? 16 : 8;   // columns of a warp, and at once
    const int c0 = warp / 4 * H, row = warp % 4 * 32 + lane;
    const uint32_t at = tmem + c0 + (static_cast<uint32_t>(warp % 4 * 32) << 16);
    float acc[FP32 ? H : C];
    bool ok = true;
    if (FULL && e.res) {   // the rows that this warp finishes
      const int c = n0 + lane * (128 / (int)sizeof(T));
      if (lane < (int)sizeof(T) && c < e.N)
        for (int p = rank * kFewWarps + warp; p < TN && m0 + p < e.M; p += g.split * kFewWarps)
          to_l2(static_cast<const T*>(e.res) + (m0 + p) * e.r_m + c);
    }
    auto load = [&](uint32_t from, float* v) {
      if constexpr (C == 32) tmem_ld32(from, reinterpret_cast<uint32_t*>(v));
      else if constexpr (C == 16) tmem_ld16(from, reinterpret_cast<float(&)[16]>(*v));
      else tmem_ld8(from, reinterpret_cast<uint32_t*>(v));
      tmem_ld_wait();
    };
    auto keep = [&](int c, const float* v) {
#pragma unroll
      for (int i = 0; i < C; ++i) part[(c0 + c + i) * 128 + row] = v[i];
    };
    for (int i = 0; i < walk.sums() && ok; ++i) {
      if (!(ok = wait(&b_acc[i & 1], (i / 2) & 1, FP32 ? 0 : n_k))) break;
      tc_fence_after();
      if constexpr (FP32) {
#pragma unroll
        for (int c = 0; c < H; c += C) {
          float v[C];
          load(at + (i & 1) * kCols + c, v);
#pragma unroll
          for (int x = 0; x < C; ++x) acc[c + x] = i ? acc[c + x] + v[x] : v[x];
        }
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(&b_free[i & 1]);
      } else {
        for (int c = 0; c < H; c += C) {
          load(at + c, acc);
          keep(c, acc);
        }
        tc_fence_before();
      }
    }
    if constexpr (FP32) {
      // the last products are done, so nothing reads or fills a stage any more
      if (ok) {
#pragma unroll
        for (int c = 0; c < H; c += C) keep(c, acc + c);
      }
    }
  } else if (warp == kFewLoadWarp) {   // ---------------------------------------------- loads
    uint32_t n = 0;
    bool ok = true;
    for (int i = 0; i < walk.stages(); ++i, ++n) {
      int k, piece;
      walk.at(i, k, piece);
      const uint32_t s = n % NS;
      if (n >= NS && !(ok = wait(&b_empty[s], (n / NS - 1) & 1))) break;
      if (elect_one()) {
        uint8_t* pn = sm + s * L::kStage;
        uint8_t* pm = pn + L::kN;
        const int kc = (k0 + k) * kBK;
        mbar_expect_tx(&b_full[s], L::kStage);
        if constexpr (N_MN) {
#pragma unroll
          for (int h = 0; h < 2; ++h) load_box(pn + h * 8192, &tmN, &b_full[s], n0 + 64 * h, kc, piece);
        } else {
          load_box(pn, &tmN, &b_full[s], kc, n0, piece);
        }
        if constexpr (M_MN) {
#pragma unroll
          for (int h = 0; h < TN / 64; ++h) load_box(pm + h * 8192, &tmM, &b_full[s], m0 + 64 * h, kc, piece);
        } else {
          load_box(pm, &tmM, &b_full[s], kc, m0, piece);
        }
      }
      __syncwarp();
    }
    if (!ok)   // no copy may be in flight when the CTA ends
      for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i) wait_phase(&b_full[i % NS], (i / NS) & 1);
  } else {   // ------------------------------------------------------------------------ MMAs
    constexpr uint32_t ID = idesc_bf16(128, TN, N_MN, M_MN);
    const uint32_t a0 = smem_u32(sm), b0 = a0 + L::kN;
    const uint64_t da = desc_sw128(a0, N_MN ? 8192 : 0, 1024), db = desc_sw128(b0, M_MN ? 8192 : 0, 1024);
    uint32_t n = 0;
    bool ok = true;
    for (int i = 0; i < walk.sums() && ok; ++i) {
      const int buf = i & 1;
      if (FP32 && i >= 2 && !(ok = wait(&b_free[buf], (i / 2 - 1) & 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * kCols;
      auto full = [&](uint32_t s, uint32_t parity) {
        const bool there = wait(&b_full[s], parity);
        tc_fence_after();
        return there;
      };
      auto mma = [&](uint32_t sa, uint32_t sb, bool first) {
        const uint64_t a = da + ((sa * L::kStage) >> 4), b = db + ((sb * L::kStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            mma_bf16(d, a + j * (N_MN ? 128 : 2), b + j * (M_MN ? 128 : 2), ID, !first || j > 0);
        }
        __syncwarp();
      };
      auto free = [&](uint32_t s) {
        if (elect_one()) mma_commit(&b_empty[s]);
        __syncwarp();
      };
      ok = products<FP32, NS>(walk.n_k, n, full, mma, free);
      if (ok && elect_one()) mma_commit(&b_acc[buf]);
      __syncwarp();
    }
    if (elect_one()) mma_commit(&b_end);   // no MMA may be under way when the CTA ends
    __syncwarp();
    wait_phase(&b_end, 0);
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();   // every part is there
  tc_fence_after();
  if (warp == kFewMmaWarp) tmem_dealloc(tmem, kTmem);
  const int n = n0 + lane * 4, left = e.N - n;
  if (warp < kFewWarps && left > 0) {   // ----------------------------- sums and epilogue
    const bool whole = e.vec && left >= 4;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (FULL && e.bias) get4(static_cast<const T*>(e.bias) + n, false, left, bias);
    const uint32_t mine = smem_u32(part) + lane * 16;
    constexpr int B = TN / kFewWarps < 4 ? TN / kFewWarps : 4;   // rows at once: their loads are under way together
    const int rows = min(TN, e.M - m0);
    for (int p = rank * kFewWarps + warp; p < rows; p += B * g.split * kFewWarps) {
      float x[B][4], r[B][4];
      int ml[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        ml[b] = min(p + b * g.split * kFewWarps, rows - 1);   // behind the last row: that one again, not stored
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][i] = bias[i];
        if (FULL && e.res) get4(static_cast<const T*>(e.res) + (m0 + ml[b]) * e.r_m + n, whole, left, r[b]);
      }
      for (int c = 0; c < g.split; ++c) {
        const uint32_t from = map_rank(mine, c);
        float4 u[B];
#pragma unroll
        for (int b = 0; b < B; ++b) u[b] = load_peer(from + ml[b] * 512);
#pragma unroll
        for (int b = 0; b < B; ++b) x[b][0] += u[b].x, x[b][1] += u[b].y, x[b][2] += u[b].z, x[b][3] += u[b].w;
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (p + b * g.split * kFewWarps >= rows) break;
        const long long at = (m0 + ml[b]) * (long long)e.N + n;
        if constexpr (FULL) {
          float s[4];
          act_all(e.act, e.slope != nullptr, x[b], s);
          if (e.slope) put4(static_cast<S*>(e.slope) + at, whole, left, s);
          if (e.res) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[b][i] += r[b][i];
          }
        }
        put4(static_cast<T*>(e.C) + at, whole, left, x[b]);
      }
    }
  }
  __syncwarp();
  cluster_sync();   // nobody reads this CTA's part any more
  if (e.place == kBeside) wait_for_last();   // whoever waits for this kernel waits for that one too
}

template <int TN, bool N_MN, bool M_MN, typename T, bool FULL>
cudaError_t few(const Operand& M, const Operand& N, Epilogue e, int split, cudaStream_t st) {
  CUtensorMap tn, tm;
  if (!make_operand_map(&tn, N, 128) || !make_operand_map(&tm, M, TN)) return cudaErrorInvalidValue;
  auto* kernel = linear_few_kernel<TN, N_MN, M_MN, T, FULL>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<TN>::kBytes);
  if (err != cudaSuccess) return err;
  const FewGrid g{(M.rows + TN - 1) / TN, split};
  e.vec = e.N % 4 == 0 && (!e.res || e.r_m % 4 == 0);   // four columns at once
  return launch_in_call(e.place != kFirst, kernel, dim3(static_cast<unsigned>(g.tiles_m * ((N.rows + 127LL) / 128) * split)),
                        kFewThreads, FewSmem<TN>::kBytes, st, split, tn, tm, e, g, (N.k + kBK - 1) / kBK);
}

template <typename T, int TN>
cudaError_t few_by_order(const Operand& M, const Operand& N, const Epilogue& e, bool full, int split, cudaStream_t st) {
  if (full) return N.mn ? few<TN, true, false, T, true>(M, N, e, split, st) : few<TN, false, false, T, true>(M, N, e, split, st);
  if constexpr (TN % 64 == 0) {
    if (M.mn) return few<TN, true, true, T, false>(M, N, e, split, st);
  }
  return N.mn ? few<TN, true, false, T, false>(M, N, e, split, st) : few<TN, false, false, T, false>(M, N, e, split, st);
}

template <typename T>
cudaError_t few_by_tile(int tn, const Operand& M, const Operand& N, const Epilogue& e, bool full, int split, cudaStream_t st) {
  switch (tn) {
    case 16: return few_by_order<T, 16>(M, N, e, full, split, st);
    case 32: return few_by_order<T, 32>(M, N, e, full, split, st);
    case 64: return few_by_order<T, 64>(M, N, e, full, split, st);
    case 96: return few_by_order<T, 96>(M, N, e, full, split, st);
    case 128: return few_by_order<T, 128>(M, N, e, full, split, st);
    case 160: return few_by_order<T, 160>(M, N, e, full, split, st);
    case 192: return few_by_order<T, 192>(M, N, e, full, split, st);
    default: break;
  }
  if constexpr (sizeof(T) == 2) return few_by_order<T, 256>(M, N, e, full, split, st);
  return cudaErrorInvalidValue;   // 128 sums per thread take more registers than it has
}

}  // namespace lin
}  // namespace dr
