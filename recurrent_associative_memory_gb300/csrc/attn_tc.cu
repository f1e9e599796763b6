// attn_tc.cu — window attention with sinks, forward, bf16 on tcgen05.
//
// One CTA owns 256 query rows of a head, two tiles of 128, and walks the 128-key tiles
// that they can see.  Per tile w and key tile n:
//   S_w = Q_w K_n^T      M = N = 128, K = d     (operands in shared memory, S in TMEM)
//   P_w = exp2(S c - m)  one thread per row; bf16, written over S in TMEM
//   O_w += P_w V_n       M = 128, N = d, K = 128 keys  (A = P from TMEM)
// The two tiles take turns: while the four softmax warps of one work, the tensor cores run
// the other's P V and next S.  S and P V of a tile wait for each other, so a step is the
// longer of four products (2048 cycles at d = 128) and the softmax's latency plus two.
// To keep that latency short, a tile's exponentials take a reference m from the tiles
// before it: any m is right as long as nothing overflows (the final division takes it out).
// m is set 2^8 above a row's maximum, so that P stays at most 1 and P V within what the sum of
// |v| allows; where a maximum passes m (or m is not set: the first tile), the tile is taken
// again.  P V of the first 64 keys starts while the second 64 are still exponentials.  Raising
// m rescales O; S of tile n is issued behind P V of tile n - 1, so a thread that has S may
// touch O.
// The CTAs stay: one per SM walks the work items, and the next item's Q, K and V are on their
// way while the last one's softmax and stores run.
//   warps 0-3, 4-7  softmax and epilogue of the tiles 0 and 1
//   warp 8          TMA: K and V tiles, two slots each (d = 64: four)
//   warps 9, 10     the MMAs of the tiles 0 and 1: a warp walks its loop together and one
//                   lane issues.  (Issued under a branch on the lane, an MMA takes 51
//                   cycles instead of 14, its descriptors going through vector registers;
//                   one warp for both tiles spends 2300 cycles of a step on its waits.)
//                   They issue P V and the next S of their tile in turns: interleaved, both
//                   tiles would finish together and their softmax would run at the same time.
// d 128, 16 heads over 4, window 2048, B1 T16384: 215 us, 1200 TFLOP/s; window 1024, B2 T4096
// with lengths from half to all of it 58 to 70 us as they fall, 50 GFLOP of visible pairs on
// average, 750 TFLOP/s.  The softmax's instructions and the waits between it and
// the products bound it: a step takes about 3200 cycles.
// Rounding: P to bf16 (the sum l takes it in fp32), O once at the end.
// The tile that holds lens[b] has its V rows from there on zeroed in shared memory, as
// 0 times whatever stands there may be NaN; scores are masked by selection.
#include <type_traits>

#include "attn_tc.cuh"

namespace dr {
namespace {

using namespace attn;

constexpr int kThreads = 384;   // three warpgroups; the third has an idle warp
// registers per thread after the split: 2 x 208 + 88 = 3 x 168, what the launch takes
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * kLaunchRegs, "a larger sum would wait for ever");
constexpr int kLoadWarp = 8, kMmaWarp = 9;   // and the one after it
constexpr float kAbove = 8.f;   // what m is set above a row's maximum, in base 2

template <int D> struct Smem {
  static constexpr int kTile = kM * D * 2;                  // bytes of 128 rows
  static constexpr int kSlots = D == 64 ? 4 : 2;
  static constexpr int oQ = 0, oK = 2 * kTile, oV = oK + kSlots * kTile, kBytes = oV + kSlots * kTile + 1024;
};

// One work item: 256 query rows of a head.  Heads of a group are neighbours: they read the
// same K and V.
struct Item {
  int h, i0, b, hk, len;
  TileSet set0, set1;
  KeyTiles tiles;
  __device__ __forceinline__ Item(const AttnArgs& a, int n_block, uint32_t it)
      : h(it % a.H),
        i0(it / a.H % n_block * 2 * kM),
        b(it / a.H / n_block),
        hk(h / a.G),
        len(uniform(real_len(a.lens, b, a.reach))),
        set0(a, i0, len),
        set1(a, i0 + kM, len),
        tiles(a.q_start + i0, a.q_start + min(i0 + 2 * kM, a.T) - 1, len, a.window, a.n_sink, kM) {}
  // a tile outside every row's window is there for its sinks only: of up to 32 (the smallest
  // tile of keys) the product and softmax of 32 keys do (60 us instead of 68 for B2 T4096
  // above, 214 instead of 221 for T16384)
  __device__ __forceinline__ bool sinks_only(const AttnArgs& a, int tile) const {
    return tile < tiles.n_first && a.n_sink - tile * kM <= 32;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, AttnArgs a) {
  using L = Smem<D>;
  constexpr int NS = L::kSlots;
  constexpr uint32_t ID_S = idesc_bf16(128, 128, 0, 0), ID_S32 = idesc_bf16(128, 32, 0, 0);
  constexpr uint32_t ID_O = idesc_bf16(128, D, 0, 1);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // full and empty: Q, the K and V slots; S; P of the first and of the other 64 keys; O
  __shared__ uint64_t b_qf, b_qe, b_kf[NS], b_ke[NS], b_vf[NS], b_ve[NS], b_fix, b_s[2], b_pa[2], b_pb[2], b_o[2],
      b_end[2], b_turn[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;

  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
  const int n_block = (a.T + 2 * kM - 1) / (2 * kM);
  const uint32_t n_item = a.B * a.H * n_block;   // a grid's worth: below 2^31

  if (tid == 0) {
    mbar_init(&b_qf, 1), mbar_init(&b_qe, 2), mbar_init(&b_fix, 1);
    for (int i = 0; i < NS; ++i)
      mbar_init(&b_kf[i], 1), mbar_init(&b_ke[i], 2), mbar_init(&b_vf[i], 1), mbar_init(&b_ve[i], 2);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&b_s[w], 1), mbar_init(&b_pa[w], 128), mbar_init(&b_pb[w], 128), mbar_init(&b_o[w], 1);
      mbar_init(&b_end[w], 1), mbar_init(&b_turn[w], 1);
    }
    fence_mbar_init();
    mbar_arrive(&b_turn[0]);   // tile 0 goes first
    s_abort = 0;
  }
  if (warp == kMmaWarp) tmem_alloc(&s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s_tmem);

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (wait_phase(bar, parity)) return true;
    s_abort = 1;
    set_status(DR_ERR_TIMEOUT);
    return false;
  };
  // of a whole warp: what follows is collective
  auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  if (warp < 8) {   // ---------------------------------------------------------- softmax
    more_registers<kSoftmaxRegs>();
    const int w = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + w * 128 + lanes, tO = tmem + 256 + w * D + lanes;
    const float c2 = a.scale * 1.4426950408889634f;
    uint32_t ns = 0, no = 0;   // phases of S and O that have gone by
    bool ok = true;

    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const Item x(a, n_block, it);
      const int i = x.i0 + w * kM + row, p = a.q_start + i;
      const int p0 = a.q_start + x.i0 + w * kM, p1 = p0 + kM - 1;
      float m = -INFINITY, l = 0.f;   // m in base 2
      bool any = false;

      auto rescale = [&](float f) {   // l and O, of all rows of the warp
        l *= f;
        if (!any) return;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(tO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tmem_st16(tO + c, reinterpret_cast<uint32_t*>(o));
        }
        tmem_st_wait();   // a second call loads what this one stored
      };

      auto one_tile = [&](auto cols, int j0) {   // cols.value keys from j0
        constexpr int NC = decltype(cols)::value, NA = NC < 64 ? NC : 64;
        const bool whole = j0 + NC - 1 <= p0 && j0 + NC <= x.len && p1 - j0 < a.window;
        float s[NC];
        uint32_t pk[NA / 2];
        f2 sum[2], aa;
        const f2 cc = pack2(c2, c2);
        auto exponentials = [&](int c0) {   // of NA columns
#pragma unroll
          for (int c = 0; c < NA; c += 2) {
            const f2 e = ex2_2(dr::fma2(pack2(s[c0 + c], s[c0 + c + 1]), cc, aa));
            sum[c / 2 % 2] = add2(sum[c / 2 % 2], e);
            float u, v;
            unpack2(e, u, v);
            pk[c / 2] = tc::pack_bf16(u, v);
          }
        };
        for (;;) {
#pragma unroll
          for (int c = 0; c < NC; c += 32) tmem_ld32(tS + c, reinterpret_cast<uint32_t*>(s) + c);
          tmem_ld_wait();
          if (!whole) {
            const RowMask mask(a, p, j0, x.len);
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 32) {
              const uint32_t word = mask.word(c0);
#pragma unroll
              for (int c = 0; c < 32; ++c) s[c0 + c] = word & (1u << c) ? s[c0 + c] : -INFINITY;
            }
          }
          const float at = m == -INFINITY ? 0.f : -m;   // a row that has seen nothing so far
          aa = pack2(at, at);
          sum[0] = sum[1] = 0;
          exponentials(0);
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c + 8 <= NC; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
          const float top = c2 * max3(max3(mx[0], mx[1], mx[2]), mx[3],
                                      max3(max3(s[NC - 4], s[NC - 3], s[NC - 2]), s[NC - 1], -INFINITY));
          const bool far = top > m;   // true too where nothing was summed so far
          if (!__any_sync(0xffffffffu, far)) break;
          rescale(far && m != -INFINITY ? ex2(m - (top + kAbove)) : 1.f);
          if (far) m = top + kAbove;
        }
#pragma unroll
        for (int c = 0; c < NA / 2; c += 16) tmem_st16(tS + c, pk + c);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&b_pa[w]);
        if constexpr (NC > NA) {
          exponentials(NA);
#pragma unroll
          for (int c = 0; c < NA / 2; c += 16) tmem_st16(tS + NA / 2 + c, pk + c);
          tmem_st_wait();
          tc_fence_before();
        }
        mbar_arrive(&b_pb[w]);
        l += sum2(add2(sum[0], sum[1]));
      };

      const TileSet& set = w ? x.set1 : x.set0;
      for (int n = 0; n < x.tiles.n && ok; ++n) {
        const int tile = x.tiles[n];
        if (!set.has(tile)) continue;
        if (!(ok = all_wait(&b_s[w], ns++ & 1))) break;
        tc_fence_after();
        if (x.sinks_only(a, tile))
          one_tile(std::integral_constant<int, 32>{}, tile * kM);
        else
          one_tile(std::integral_constant<int, 128>{}, tile * kM);
        any = true;
      }
      if (any && ok) {
        ok = all_wait(&b_o[w], no++ & 1);
        tc_fence_after();
      }
      if (ok && x.i0 + w * kM < a.T) {
        const float f = l != 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (((long long)x.b * a.T + i) * a.H + x.h) * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          if (any) {
            tmem_ld32(tO + c, v);
            tmem_ld_wait();
          }
          if (i < a.T) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 u;
              uint32_t* q = &u.x;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                q[k] = any ? tc::pack_bf16(__uint_as_float(v[e + 2 * k]) * f, __uint_as_float(v[e + 2 * k + 1]) * f)
                           : 0u;
              *reinterpret_cast<uint4*>(o + c + e) = u;
            }
          }
        }
        if (a.lse && i < a.T)
          a.lse[((long long)x.b * a.H + x.h) * a.T + i] =
              l != 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
      }
      tc_fence_before();   // O has been read before the P that lets the next item's P V go
    }
  } else {
    fewer_registers<kOtherRegs>();
  }
  if (warp == kLoadWarp) {   // ----------------------------------------------------- loads
    uint32_t nk = 0, nv = 0, nq = 0, n_fix = 0;   // loads issued so far
    bool ok = true;
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const Item x(a, n_block, it);
      const int fix_tile = x.len < a.S && x.len % kM ? x.len / kM : -1;   // its V rows from len on become 0
      for (int n = 0; n < x.tiles.n; ++n) {
        const int tile = x.tiles[n], ks = nk % NS, vs = nv % NS;
        if (nk >= NS && !(ok = all_wait(&b_ke[ks], (nk / NS - 1) & 1))) break;
        if (lane == 0) {
          mbar_expect_tx(&b_kf[ks], L::kTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sm + L::oK + ks * L::kTile + c * kM * 128, &tmK, &b_kf[ks], 64 * c, x.hk, tile * kM, x.b);
        }
        ++nk;
        if (n == 0) {
          if (nq > 0 && !(ok = all_wait(&b_qe, (nq - 1) & 1))) break;
          if (lane == 0) {
            mbar_expect_tx(&b_qf, 2 * L::kTile);
            for (int w = 0; w < 2; ++w)
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sm + L::oQ + w * L::kTile + c * kM * 128, &tmQ, &b_qf, 64 * c, x.h, x.i0 + w * kM, x.b);
          }
          ++nq;
        }
        if (nv >= NS && !(ok = all_wait(&b_ve[vs], (nv / NS - 1) & 1))) break;
        uint8_t* v = sm + L::oV + vs * L::kTile;
        uint64_t* full = tile == fix_tile ? &b_fix : &b_vf[vs];
        if (lane == 0) {
          mbar_expect_tx(full, L::kTile);
          for (int c = 0; c < D / 64; ++c) tma_load_4d(v + c * kM * 128, &tmV, full, 64 * c, x.hk, tile * kM, x.b);
        }
        if (tile == fix_tile) {
          if (!(ok = all_wait(&b_fix, n_fix & 1))) break;
          ++n_fix;
          const int r0 = x.len % kM;   // rows are 128 bytes in each block of 64 channels
          for (int e = lane; e < (kM - r0) * 8 * (D / 64); e += 32) {
            const int c = e / ((kM - r0) * 8), y = e % ((kM - r0) * 8);
            reinterpret_cast<uint4*>(v + c * kM * 128 + r0 * 128)[y] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_vf[vs]);
        }
        ++nv;
      }
    }
    if (!ok || s_abort) {   // no copy may be in flight when the CTA ends
      if (nq > 0) wait_phase(&b_qf, (nq - 1) & 1);
      for (uint32_t n = nk > NS ? nk - NS : 0; n < nk; ++n) wait_phase(&b_kf[n % NS], (n / NS) & 1);
      for (uint32_t n = nv > NS ? nv - NS : 0; n < nv; ++n) wait_phase(&b_vf[n % NS], (n / NS) & 1);
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {   // --------------------------- MMAs
    const int w = warp - kMmaWarp;
    const uint64_t q = desc_kmajor(smem_u32(sm + L::oQ + w * L::kTile)), k0 = desc_kmajor(smem_u32(sm + L::oK));
    const uint64_t v0 = desc_mnmajor<kM>(smem_u32(sm + L::oV));
    const uint32_t o = tmem + 256 + w * D, s = tmem + w * 128;
    uint32_t nt = 0, nq = 0, np = 0, turn = 0;   // key tiles, items, P tiles and turns gone by
    bool ok = true;
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const Item x(a, n_block, it);
      if (x.tiles.n == 0) continue;
      const TileSet& set = w ? x.set1 : x.set0;
      if (!(ok = all_wait(&b_qf, nq++ & 1))) break;
      bool pend = false, first = true;           // is P V of the tile before still to come?
      for (int n = 0; n <= x.tiles.n; ++n, ++nt) {
        // tile n is number nt of the CTA; the one before it has the slot of nt - 1
        const uint32_t ks = nt % NS, vs = (nt + NS - 1) % NS;
        if (n < x.tiles.n && !(ok = all_wait(&b_kf[ks], (nt / NS) & 1))) break;
        const bool small = pend && x.sinks_only(a, x.tiles[n - 1]);
        const uint64_t v = v0 + vs * (L::kTile >> 4);
        if (pend) {
          if (!(ok = all_wait(&b_pa[w], np & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            mma_bf16_ta(o, s, v, ID_O, !first);
            mma_bf16_ta(o, s + 8, v + step_mnmajor(1), ID_O, true);
            if (!small) {
              mma_bf16_ta(o, s + 16, v + step_mnmajor(2), ID_O, true);
              mma_bf16_ta(o, s + 24, v + step_mnmajor(3), ID_O, true);
            }
          }
          if (!(ok = all_wait(&b_pb[w], np & 1))) break;
          ++np;
        }
        if (!(ok = all_wait(&b_turn[w], turn++ & 1))) break;
        tc_fence_after();
        if (pend && !small && elect_one()) {
#pragma unroll
          for (int k = 4; k < kM / 16; ++k) mma_bf16_ta(o, s + 8 * k, v + step_mnmajor(k), ID_O, true);
        }
        if (pend) first = false;
        if (n > 0 && elect_one()) mma_commit(&b_ve[vs]);
        pend = n < x.tiles.n && set.has(x.tiles[n]);
        if (pend) {
          const uint32_t id = x.sinks_only(a, x.tiles[n]) ? ID_S32 : ID_S;
          const uint64_t k = k0 + ks * (L::kTile >> 4);
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < D / 16; ++e) mma_bf16(s, q + step_kmajor<kM>(e), k + step_kmajor<kM>(e), id, e > 0);
            mma_commit(&b_s[w]);
          }
        }
        if (elect_one()) {
          mbar_arrive(&b_turn[w ^ 1]);
          if (n < x.tiles.n) mma_commit(&b_ke[ks]);
          if (n == x.tiles.n - 1) mma_commit(&b_qe);
          if (n == x.tiles.n && !first) mma_commit(&b_o[w]);   // a tile without keys has no O
        }
        if (n == x.tiles.n) break;
        if (!(ok = all_wait(&b_vf[ks], (nt / NS) & 1))) break;   // for the next step
      }
    }
    __syncwarp();
    if (elect_one()) mma_commit(&b_end[w]);      // no MMA may be under way when the CTA ends
    wait_phase(&b_end[w], 0);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t fwd(const AttnArgs& a, int sms, cudaStream_t st) {
  CUtensorMap q, k, v;
  if (!make_map(&q, a.q, a.B, a.T, a.H, D, a.q_sb, a.q_st, a.q_sh) ||
      !make_map(&k, a.k, a.B, a.S, a.Hkv, D, a.k_sb, a.k_st, a.k_sh) ||
      !make_map(&v, a.v, a.B, a.S, a.Hkv, D, a.v_sb, a.v_st, a.v_sh))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attn_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.B * a.H * ((a.T + 2 * kM - 1) / (2 * kM));
  attn_fwd_tc_kernel<D><<<static_cast<unsigned>(items < sms ? items : sms), kThreads, Smem<D>::kBytes, st>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace

// bf16 with strides that a tensor map can hold
bool attn_tc_supported(const AttnArgs& a, int dtype) {
  return dtype == DR_BF16 && map_strides_ok(a.B, a.T, a.H, a.q_sb, a.q_st, a.q_sh) &&
         map_strides_ok(a.B, a.S, a.Hkv, a.k_sb, a.k_st, a.k_sh) &&
         map_strides_ok(a.B, a.S, a.Hkv, a.v_sb, a.v_st, a.v_sh);
}

cudaError_t attn_fwd_tc_status(int* word, cudaStream_t st) { return take_status(word, st); }

cudaError_t launch_attn_fwd_tc(const AttnArgs& a, int sms, cudaStream_t st) {
  return a.d == 64 ? fwd<64>(a, sms, st) : fwd<128>(a, sms, st);
}

}  // namespace dr
