// linear_few.cuh — the matrix product on tcgen05 where C is small: few rows (single tokens, a
// short prompt), or few tiles.
//
// The roles are turned round: 128 columns n of C are the MMA's 128 rows, the rows m of C its
// N = TN columns, so that a handful of tokens wastes no tensor-core row and a weight tile is
// read once.  The sum over k is cut over the S CTAs of a cluster, each of which leaves its
// part of C in its shared memory; they add them up in the ranks' order, each for its share of
// the rows, so the result does not depend on which CTA is first.
//   warps 0-3  the accumulator to shared memory, then the sums and the epilogue
//   warp 4     TMA, 3 to 6 stages of 64 k
//   warp 5     the MMAs
// About 100 KB of shared memory: two CTAs per SM, so that one's loads cover the other's start
// and end.  Weights are what bounds it: every stage is 16 KB of them.
#pragma once

#include <type_traits>

#include "linear_tc.cuh"

namespace dr {
namespace lin {

constexpr int kFewThreads = 192, kFewLoadWarp = 4, kFewMmaWarp = 5;

template <int TN> struct FewSmem {
  static constexpr int kN = 128 * kBK * 2, kM = TN * kBK * 2, kStage = kN + kM;
  static constexpr int kStages = TN == 16 ? 6 : TN == 32 ? 5 : TN == 64 ? 4 : 3;
  static constexpr int kBytes = kStages * kStage + 1024;
  static_assert(TN * 128 * 4 <= kStages * kStage, "the parts of C take the stages' place");
};

struct FewGrid {
  int tiles_m, split;   // tiles of rows; CTAs over k
};

__device__ __forceinline__ float2 load_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// N_MN, M_MN: the operands of C's columns and rows are MN-major
template <int TN, bool N_MN, bool M_MN, typename T, bool FULL>
__global__ void __launch_bounds__(kFewThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmN, const __grid_constant__ CUtensorMap tmM, Epilogue e,
                      FewGrid g, int n_k) {
  static_assert(!M_MN || TN >= 64, "a swizzled row of an MN-major operand is 64 of its rows");
  using L = FewSmem<TN>;
  using S = typename std::conditional<sizeof(T) == 2, __half, float>::type;
  constexpr bool FP32 = sizeof(T) == 4;
  constexpr int NS = L::kStages, kCols = TN < 32 ? 32 : TN;   // TMEM columns of an accumulator
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t b_full[NS], b_empty[NS], b_acc[2], b_free[2], b_end;
  __shared__ uint32_t s_tmem;
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
  const int m0 = tile % g.tiles_m * TN, n0 = tile / g.tiles_m * 128;
  const int k0 = static_cast<int>((long long)n_k * rank / g.split);
  const Stages<FP32> stages{static_cast<int>((long long)n_k * (rank + 1) / g.split) - k0};
  const int n_chunk = stages.chunks();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&b_acc[i], 1), mbar_init(&b_free[i], 4);
    mbar_init(&b_end, 1);
    fence_mbar_init();
  }
  if (warp == kFewMmaWarp) tmem_alloc(&s_tmem, (FP32 ? 2 : 1) * kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    bool ok = wait_phase(bar, parity);
    if (!ok) set_status(DR_ERR_TIMEOUT);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  float* part = reinterpret_cast<float*>(sm);   // [TN][128]

  if (warp < 4) {   // ------------------------------------------------------ accumulators
    const uint32_t at = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    constexpr int C = TN < 32 ? TN : 32;
    float acc[FP32 ? TN : C];
    bool ok = true;
    auto load = [&](uint32_t from, float* v) {
      if constexpr (C == 32) {
        tmem_ld32(from, reinterpret_cast<uint32_t*>(v));
      } else {
        float w[16];
        tmem_ld16(from, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = w[i];
      }
      tmem_ld_wait();
    };
    auto keep = [&](int c, const float* v) {
#pragma unroll
      for (int i = 0; i < C; ++i) part[(c + i) * 128 + warp * 32 + lane] = v[i];
    };
    for (int i = 0; i < n_chunk && ok; ++i) {
      if (!(ok = wait(&b_acc[i & 1], (i / 2) & 1))) break;
      tc_fence_after();
      if constexpr (FP32) {
#pragma unroll
        for (int c = 0; c < TN; c += C) {
          float v[C];
          load(at + (i & 1) * kCols + c, v);
#pragma unroll
          for (int x = 0; x < C; ++x) acc[c + x] = i ? acc[c + x] + v[x] : v[x];
        }
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(&b_free[i & 1]);
      } else {
        for (int c = 0; c < TN; c += C) {
          load(at + c, acc);
          keep(c, acc);
        }
        tc_fence_before();
      }
    }
    if constexpr (FP32) {
      // the last chunk's products are done, so nothing reads or fills a stage any more
      if (ok) {
#pragma unroll
        for (int c = 0; c < TN; c += C) keep(c, acc + c);
      }
    }
  } else if (warp == kFewLoadWarp) {   // ---------------------------------------------- loads
    uint32_t n = 0;
    bool ok = true;
    for (int i = 0, chunk = 0; chunk < n_chunk; ++n) {
      int k, pm, pn;
      stages.at(chunk, i, k, pm, pn);
      if (++i == stages.of(chunk)) i = 0, ++chunk;
      const uint32_t s = n % NS;
      if (n >= NS && !(ok = wait(&b_empty[s], (n / NS - 1) & 1))) break;
      if (elect_one()) {
        uint8_t* pn_ = sm + s * L::kStage;
        uint8_t* pm_ = pn_ + L::kN;
        const int kc = (k0 + k) * kBK;
        mbar_expect_tx(&b_full[s], L::kStage);
        if constexpr (N_MN) {
#pragma unroll
          for (int h = 0; h < 2; ++h) load_box(pn_ + h * 8192, &tmN, &b_full[s], n0 + 64 * h, kc, pn);
        } else {
          load_box(pn_, &tmN, &b_full[s], kc, n0, pn);
        }
        if constexpr (M_MN) {
#pragma unroll
          for (int h = 0; h < TN / 64; ++h) load_box(pm_ + h * 8192, &tmM, &b_full[s], m0 + 64 * h, kc, pm);
        } else {
          load_box(pm_, &tmM, &b_full[s], kc, m0, pm);
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
    for (int chunk = 0; chunk < n_chunk && ok; ++chunk) {
      const int buf = chunk & 1, n_stage = stages.of(chunk);
      if (FP32 && chunk >= 2 && !(ok = wait(&b_free[buf], (chunk / 2 - 1) & 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * kCols;
      for (int i = 0; i < n_stage; ++i, ++n) {
        const uint32_t s = n % NS;
        if (!(ok = wait(&b_full[s], (n / NS) & 1))) break;
        tc_fence_after();
        const uint32_t at = (s * L::kStage) >> 4;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            mma_bf16(d, da + at + j * (N_MN ? 128 : 2), db + at + j * (M_MN ? 128 : 2), ID, i > 0 || j > 0);
          mma_commit(&b_empty[s]);
        }
        __syncwarp();
      }
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
  if (warp == kFewMmaWarp) tmem_dealloc(tmem, (FP32 ? 2 : 1) * kCols);
  if (warp < 4) {   // ------------------------------------------------- sums and epilogue
    const int nl = threadIdx.x % 64 * 2, n = n0 + nl;
    const bool two = e.vec && n + 1 < e.N;
    float bias[2] = {0.f, 0.f};
    if constexpr (FULL) {
      if (e.bias) {
        if (n < e.N) bias[0] = to_f(static_cast<const T*>(e.bias)[n]);
        if (n + 1 < e.N) bias[1] = to_f(static_cast<const T*>(e.bias)[n + 1]);
      }
    }
    const uint32_t mine = smem_u32(part) + nl * 4;
#pragma unroll 2
    for (int p = rank; p < TN / 2; p += g.split) {   // pairs of rows, in turns over the CTAs
      const int ml = 2 * p + threadIdx.x / 64, m = m0 + ml;
      if (m >= e.M || n >= e.N) continue;
      float2 v = make_float2(0.f, 0.f);
      for (int r = 0; r < g.split; ++r) {
        const float2 u = load_peer2(map_rank(mine + ml * 512, r));
        v.x += u.x, v.y += u.y;
      }
      float x[2] = {v.x + bias[0], v.y + bias[1]}, s[2];
      const long long at = m * (long long)e.N + n;
      T* C = static_cast<T*>(e.C) + at;
      if constexpr (FULL) {
        act_all(e.act, e.slope != nullptr, x, s);
        if (e.slope) {
          S* q = static_cast<S*>(e.slope) + at;
          if (two) {
            if constexpr (FP32) *reinterpret_cast<float2*>(q) = make_float2(s[0], s[1]);
            else *reinterpret_cast<__half2*>(q) = __floats2half2_rn(s[0], s[1]);
          } else {
            q[0] = static_cast<S>(s[0]);
            if (n + 1 < e.N) q[1] = static_cast<S>(s[1]);
          }
        }
        if (e.res) {
          const T* q = static_cast<const T*>(e.res) + m * e.r_m + n;
          x[0] += to_f(q[0]);
          if (n + 1 < e.N) x[1] += to_f(q[1]);
        }
      }
      if (two) {
        if constexpr (FP32) *reinterpret_cast<float2*>(C) = make_float2(x[0], x[1]);
        else *reinterpret_cast<uint32_t*>(C) = tc::pack_bf16(x[0], x[1]);
      } else {
        C[0] = from_f<T>(x[0]);
        if (n + 1 < e.N) C[1] = from_f<T>(x[1]);
      }
    }
  }
  __syncwarp();
  cluster_sync();   // nobody reads this CTA's part any more
}

template <int TN, bool N_MN, bool M_MN, typename T, bool FULL>
cudaError_t few(const Operand& M, const Operand& N, Epilogue e, int split, cudaStream_t st) {
  CUtensorMap tn, tm;
  if (!make_operand_map(&tn, N, 128) || !make_operand_map(&tm, M, TN)) return cudaErrorInvalidValue;
  auto* kernel = linear_few_kernel<TN, N_MN, M_MN, T, FULL>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<TN>::kBytes);
  if (err != cudaSuccess) return err;
  const FewGrid g{(M.rows + TN - 1) / TN, split};
  e.vec = e.N % 2 == 0;   // pairs of columns at once
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(g.tiles_m * ((N.rows + 127LL) / 128) * split));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = FewSmem<TN>::kBytes;
  cfg.stream = st;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tn, tm, e, g, (N.k + kBK - 1) / kBK);
}

template <int TN, typename T>
cudaError_t few_by_order(const Operand& M, const Operand& N, const Epilogue& e, bool full, int split, cudaStream_t st) {
  if (full) return N.mn ? few<TN, true, false, T, true>(M, N, e, split, st) : few<TN, false, false, T, true>(M, N, e, split, st);
  if constexpr (TN >= 64) {
    if (M.mn) return few<TN, true, true, T, false>(M, N, e, split, st);
  }
  return N.mn ? few<TN, true, false, T, false>(M, N, e, split, st) : few<TN, false, false, T, false>(M, N, e, split, st);
}

template <typename T>
cudaError_t few_by_tile(int tn, const Operand& M, const Operand& N, const Epilogue& e, bool full, int split, cudaStream_t st) {
  switch (tn) {
    case 16: return few_by_order<16, T>(M, N, e, full, split, st);
    case 32: return few_by_order<32, T>(M, N, e, full, split, st);
    case 64: return few_by_order<64, T>(M, N, e, full, split, st);
    default: break;
  }
  if constexpr (sizeof(T) == 2) return few_by_order<128, T>(M, N, e, full, split, st);
  return cudaErrorInvalidValue;   // 128 sums per thread do not fit an fp32 kernel's registers
}

}  // namespace lin
}  // namespace dr
