// linear_pair.cu — the matrix product on tcgen05, tiles of 256 rows by BN columns over a pair
// of CTAs.
//
// Each CTA of a pair holds 128 rows of A and half of B's columns; one MMA of the pair
// multiplies 256 x BN x 16 from both shared memories, so that a stage of 64 k moves
// (128 + BN / 2) x 128 bytes into each SM for 512 (BN = 256) cycles of products: 64 bytes a
// cycle, where one CTA by itself would need 96.  Accumulators take all of TMEM, two buffers of
// 256 columns or four of 128: while the epilogue reads one, the products go on in the next.
// (fp32, whose epilogue takes no more sums of 64 k while it stores a tile: M2048 K1024 N4096 with
// all gradients 269 us with two buffers, 264 with four.)
//   warps 0-7  epilogue: rows 32 (w mod 4) .. of the CTA's 128, a thread per row, and half of
//              the columns each
//   warp 8     TMA: this CTA's part of each stage, counted on the first CTA's barrier
//   warp 9     the MMAs, in the first CTA of the pair
// The pairs stay: one per two SMs walks the tiles, eight tiles of rows at a time, so that
// neighbours in time share columns of B and rows of A in L2.
// bf16 M8192 K4096 N4096 with a residual: 148 us, 1860 TFLOP/s, the tensor cores 85 % busy; on
// end, at the power limit, 172 us.  fp32 (three pieces, six products, sums in registers) M4096
// K4096 N4096: 469 us, 293 TFLOP/s; BN is 128 there, as a warp's 128 columns of 256 spill (800 us).
// Ten warps are three on a partition, so each has 168 registers, the two that load and issue too;
// fp32 with the whole epilogue spills 208 bytes of them at that (the gradients' products none).
#include <type_traits>

#include "linear_tc.cuh"

namespace dr {
namespace {

using namespace lin;

constexpr int kThreads = 320, kEpilogueWarps = 8, kLoadWarp = 8, kMmaWarp = 9;
constexpr int kGroup = 8;   // tiles of rows that are walked together

template <int BN> struct Smem {
  static constexpr int kA = 128 * kBK * 2, kB = BN / 2 * kBK * 2, kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int oBias = kStages * kStage;                  // fp32, each epilogue warp's [BN / 2]
  static constexpr int oTurn = oBias + kEpilogueWarps * BN / 2 * 4;   // and [32][17]: rows to columns
  static constexpr int kBytes = oTurn + kEpilogueWarps * 32 * 17 * 4 + 1024;
};

struct Tiles {
  int m, n;   // numbers of tiles
  __device__ __forceinline__ void at(int t, int& tm, int& tn) const {
    const int per = kGroup * n, g = t / per, r = t - g * per, size = min(kGroup, m - g * kGroup);
    tn = r / size;
    tm = g * kGroup + r - tn * size;
  }
};

// T: the type of C, bias and residual; FULL: with bias, activation, residual, slope
template <int BN, bool A_MN, bool B_MN, typename T, bool FULL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Epilogue e,
                       Tiles tiles, int n_k) {
  using L = Smem<BN>;
  using S = typename std::conditional<sizeof(T) == 2, __half, float>::type;
  constexpr int NS = L::kStages, NB = 512 / BN;
  constexpr bool FP32 = sizeof(T) == 4;
  const Walk<FP32> walk{n_k};
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t b_full[NS], b_empty[NS], b_acc[NB], b_free[NB], b_end;
  __shared__ uint32_t s_tmem;
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
    for (int i = 0; i < NB; ++i) mbar_init(&b_acc[i], 1), mbar_init(&b_free[i], 2 * kEpilogueWarps);
    mbar_init(&b_end, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) pair_tmem_alloc(&s_tmem, NB * BN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (e.place != kBeside) wait_for_last(), let_next_start();
  const uint32_t tmem = uniform(s_tmem);
  const int n_tile = tiles.m * tiles.n, first = blockIdx.x / 2, step = gridDim.x / 2;

  auto give_up = [&] {
    set_status(DR_ERR_TIMEOUT);
    return false;
  };
  auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return all(wait_phase(bar, parity) || give_up()); };

  if (warp < kEpilogueWarps) {   // ------------------------------------------------ epilogue
    constexpr int NC = BN / 2;   // columns of this warp
    const int part = warp / 4, row0 = warp % 4 * 32;
    float* turn = reinterpret_cast<float*>(sm + L::oTurn) + warp * 32 * 17;
    int it = 0;   // accumulators gone by
    bool ok = true;
    for (int t = first; t < n_tile && ok; t += step) {
      int tm, tn;
      tiles.at(t, tm, tn);
      const int n0 = tn * BN + part * NC;
      const int m0 = tm * 256 + rank * 128 + row0, m = m0 + lane;
      float* bias = reinterpret_cast<float*>(sm + L::oBias) + warp * NC;   // a warp's own: no barrier to be left at
      if constexpr (FULL) {
        __syncwarp();   // every lane has read the last tile's: those without a row get here first
        for (int c = lane; c < NC; c += 32)
          bias[c] = e.bias && n0 + c < e.N ? to_f(static_cast<const T*>(e.bias)[n0 + c]) : 0.f;
        __syncwarp();
      }
      const bool live = m < e.M;
      const T* res = FULL && e.res && live ? static_cast<const T*>(e.res) + m * e.r_m + n0 : nullptr;
      T* C = static_cast<T*>(e.C) + (long long)m * e.N + n0;
      S* slope = FULL && e.slope ? static_cast<S*>(e.slope) + (long long)m * e.N + n0 : nullptr;
      if (res && !e.vec)
        for (int c = 0; c < NC && n0 + c < e.N; c += 128 / (int)sizeof(T)) to_l2(res + c);
      Raw16<T> r[2];
      auto ahead = [&](int c) {   // the residual of columns c .. c + 31
        if (!FULL || FP32 || !res || !e.vec) return;   // fp32: its sums have the registers
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 16 * h < NC && n0 + c + 16 * h < e.N) r[h].load(res + c + 16 * h);
      };
      ahead(0);
      auto emit = [&](int c, const float* v) {   // columns c .. c + 31
        if (e.vec) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[16], s[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = v[16 * h + i];
            if constexpr (FULL) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 b = *reinterpret_cast<const float4*>(bias + c + 16 * h + i);
                x[i] += b.x, x[i + 1] += b.y, x[i + 2] += b.z, x[i + 3] += b.w;
              }
              act_all(e.act, slope != nullptr, x, s);
              if (res) {
                if (FP32 && n0 + c + 16 * h < e.N) r[h].load(res + c + 16 * h);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] += r[h][i];
              }
            }
            if (live && n0 + c + 16 * h < e.N) {
              put16(C + c + 16 * h, x);
              if (FULL && slope) put16(slope + c + 16 * h, s);
            }
          }
          ahead(c + 32);
        } else {   // rows on any address: a lane takes a column, and rows are stored one by one
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = c + 16 * h + lane % 16, n = n0 + at;
            const bool in = n < e.N;
            const float b = FULL && in ? bias[at] : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) turn[lane * 17 + i] = v[16 * h + i];
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; ++q) {   // 8 rows at once, so that their loads are
              float x[8], s[8], r[8];
              const int m1 = m0 + 16 * q + lane / 16;
              auto there = [&](int i) { return in && m1 + 2 * i < e.M; };
              if (FULL && e.res) {
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = there(i) ? to_f(static_cast<const T*>(e.res)[(m1 + 2 * i) * e.r_m + n]) : 0.f;
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = turn[(16 * q + lane / 16 + 2 * i) * 17 + lane % 16] + b;
              if constexpr (FULL) {
                act_all(e.act, e.slope != nullptr, x, s);
                if (e.slope) {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (there(i)) static_cast<S*>(e.slope)[(m1 + 2 * i) * (long long)e.N + n] = static_cast<S>(s[i]);
                }
                if (e.res) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) x[i] += r[i];
                }
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (there(i)) static_cast<T*>(e.C)[(m1 + 2 * i) * (long long)e.N + n] = from_f<T>(x[i]);
            }
            __syncwarp();
          }
        }
      };
      const uint32_t lanes = static_cast<uint32_t>(row0) << 16;
      auto release = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (elect_one()) arrive_remote(map_rank(smem_u32(&b_free[buf]), 0));
      };
      if constexpr (FP32) {
        float acc[NC];
        for (int i = 0; i < n_k && ok; ++i, ++it) {
          const int buf = it % NB;
          if (!(ok = wait(&b_acc[buf], (it / NB) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NC; c += 32) {
            float v[32];
            tmem_ld32(tmem + buf * BN + part * NC + c + lanes, reinterpret_cast<uint32_t*>(v));
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) acc[c + x] = i ? acc[c + x] + v[x] : v[x];
          }
          release(buf);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < NC; c += 32)
          if (n0 + c < e.N) emit(c, acc + c);
      } else {
        const int buf = it % NB;
        if (!(ok = all(wait_sum(&b_acc[buf], (it / NB) & 1, n_k) || give_up()))) break;
        tc_fence_after();
        for (int c = 0; c < NC && n0 + c < e.N; c += 32) {
          float v[32];
          tmem_ld32(tmem + buf * BN + part * NC + c + lanes, reinterpret_cast<uint32_t*>(v));
          tmem_ld_wait();
          emit(c, v);
        }
        release(buf);
        ++it;
      }
    }
  } else if (warp == kLoadWarp) {   // --------------------------------------------- loads
    uint32_t n = 0;
    bool ok = true;
    for (int t = first; t < n_tile && ok; t += step) {
      int tm, tn;
      tiles.at(t, tm, tn);
      const int m0 = tm * 256 + rank * 128, n0 = tn * BN + rank * (BN / 2);
      for (int i = 0; i < walk.stages(); ++i, ++n) {
        int k, piece;
        walk.at(i, k, piece);
        const uint32_t s = n % NS;
        if (n >= NS && !(ok = wait(&b_empty[s], (n / NS - 1) & 1))) break;
        if (elect_one()) {
          uint8_t* a = sm + s * L::kStage;
          uint8_t* b = a + L::kA;
          const uint32_t bar = map_rank(smem_u32(&b_full[s]), 0);
          if (rank == 0) mbar_expect_tx(&b_full[s], 2 * L::kStage);
          if constexpr (A_MN) {
#pragma unroll
            for (int h = 0; h < 2; ++h) pair_load(a + h * 8192, &tmA, bar, m0 + 64 * h, k * kBK, piece);
          } else {
            pair_load(a, &tmA, bar, k * kBK, m0, piece);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int h = 0; h < BN / 128; ++h) pair_load(b + h * 8192, &tmB, bar, n0 + 64 * h, k * kBK, piece);
          } else {
            pair_load(b, &tmB, bar, k * kBK, n0, piece);
          }
        }
        __syncwarp();
      }
    }
    // no copy may be in flight when the pair ends, nor the MMAs' word that a stage is free: the
    // first CTA's barriers count both's copies, each CTA's own the MMAs'
    const uint32_t last = n > NS ? n - NS : 0;
    if (rank == 0)
      for (uint32_t i = last; i < n; ++i) wait_phase(&b_full[i % NS], (i / NS) & 1);
    if (ok)
      for (uint32_t i = last; i < n; ++i) wait_phase(&b_empty[i % NS], (i / NS) & 1);
  } else if (rank == 0) {   // ------------------------------------------------------ MMAs
    constexpr uint32_t ID = idesc_bf16(256, BN, A_MN, B_MN);
    const uint32_t a0 = smem_u32(sm), b0 = a0 + L::kA;
    const uint64_t da = desc_sw128(a0, A_MN ? 8192 : 0, 1024), db = desc_sw128(b0, B_MN ? 8192 : 0, 1024);
    uint32_t n = 0;
    int it = 0;
    bool ok = true;
    for (int t = first; t < n_tile && ok; t += step) {
      for (int i = 0; i < walk.sums() && ok; ++i, ++it) {
        const int buf = it % NB;
        if (it >= NB && !(ok = all(wait_cluster(&b_free[buf], (it / NB - 1) & 1) || give_up()))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
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
              pair_mma(d, a + j * (A_MN ? 128 : 2), b + j * (B_MN ? 128 : 2), ID, !first || j > 0);
          }
          __syncwarp();
        };
        auto free = [&](uint32_t s) {
          if (elect_one()) pair_commit(&b_empty[s]);
          __syncwarp();
        };
        ok = products<FP32, NS>(n_k, n, full, mma, free);
        if (ok && elect_one()) pair_commit(&b_acc[buf]);
        __syncwarp();
      }
    }
    if (elect_one()) pair_commit(&b_end, 1);   // no MMA may be under way when the pair ends
    __syncwarp();
    wait_phase(&b_end, 0);
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();   // nothing of this CTA is read or counted on any more
  tc_fence_after();
  if (warp == kMmaWarp) pair_tmem_dealloc(tmem, NB * BN);
  if (e.place == kBeside) wait_for_last();   // whoever waits for this kernel waits for that one too
}

template <int BN, bool A_MN, bool B_MN, typename T, bool FULL>
cudaError_t go(const Operand& A, const Operand& B, const Epilogue& e, int sms, cudaStream_t st) {
  CUtensorMap a, b;
  if (!make_operand_map(&a, A, 128) || !make_operand_map(&b, B, BN / 2)) return cudaErrorInvalidValue;
  auto* kernel = linear_pair_kernel<BN, A_MN, B_MN, T, FULL>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<BN>::kBytes);
  if (err != cudaSuccess) return err;
  const Tiles t{(A.rows + 255) / 256, (B.rows + BN - 1) / BN};
  const int pairs = static_cast<int>(min((long long)t.m * t.n, sms / 2LL));
  return launch_in_call(e.place != kFirst, kernel, 2 * pairs, kThreads, Smem<BN>::kBytes, st, 0, a, b, e, t,
                        (A.k + kBK - 1) / kBK);
}

template <typename T, int BN>
cudaError_t by_order(const Operand& A, const Operand& B, const Epilogue& e, bool full, int sms, cudaStream_t st) {
  if (full) return B.mn ? go<BN, false, true, T, true>(A, B, e, sms, st) : go<BN, false, false, T, true>(A, B, e, sms, st);
  if (A.mn) return go<BN, true, true, T, false>(A, B, e, sms, st);
  return B.mn ? go<BN, false, true, T, false>(A, B, e, sms, st) : go<BN, false, false, T, false>(A, B, e, sms, st);
}

}  // namespace

// `full`: a forward product, A K-major; otherwise C alone, and A MN-major only if B is too.
// bn: columns of a tile, 128 or 256 (fp32: 128, as a tile's sums stay in registers)
cudaError_t launch_linear_pair(int bn, const lin::Operand& A, const lin::Operand& B, const lin::Epilogue& e, bool full,
                               int sms, cudaStream_t st) {
  if (A.piece) return by_order<float, 128>(A, B, e, full, sms, st);
  return bn == 128 ? by_order<__nv_bfloat16, 128>(A, B, e, full, sms, st)
                   : by_order<__nv_bfloat16, 256>(A, B, e, full, sms, st);
}

}  // namespace dr
