// attn_bwd_tc.cu — window attention with sinks, backward, bf16 on tcgen05.
//
//   P = exp(s - lse);  dV = P^T dO;  dS = P * (dO V^T - delta);  dQ = c dS K;  dK = c dS^T Q
// with delta = rowsum(dO * O), in three launches and a fourth for the sinks:
//   rows   -lse log2(e) and -delta of every query row, padded to whole tiles of 64 (rows
//          that see nothing get -infinity, which makes their P zero by itself)
//   dK/dV  a CTA owns 128 keys of a key/value head and walks the 64-row query tiles of
//          the group's heads that see them:  S^T = K Q^T and dP^T = V dO^T into TMEM, two
//          threads per key form P^T and dS^T in bf16 in their place, and from there they
//          are the A operands of  dV += P^T dO,  dK += dS^T Q  (Q and dO rows as the k axis)
//   dQ     a CTA owns 128 query rows and walks 64-key tiles: S, dP, dS in place,
//          dQ += dS K
// S and dP are formed twice (7 products instead of 5): the alternative, one kernel that
// adds its dQ parts to memory, would depend on the order of atomics.  Two TMEM slots let
// the softmax warpgroup of one tile work while the tensor cores run the other's products.
// The sinks' keys are seen by every later row: rows that see nothing else of key tile 0
// are cut into pieces of their own, whose sums are joined in a fixed order at the end (one CTA
// walking all of them: 510 us for the training step below instead of 268).
// d 128, 16 heads over 4, window 512, B2 T4096 (forward 57 us before it): rows 17 us, dK/dV
// 107, dQ 87, sinks 6.  A step of 64 rows takes about 2000 cycles for products of 1536 (dK/dV)
// or 1280 (dQ): the chain S -> softmax -> sums of a slot, and two slots only half hide it.
// Rounding: P to bf16 as an operand.  dS as two bf16, itself and what its rounding left, in
// products of their own (16 us of the 200): P (dP - delta) cancels, delta is taken from a
// rounded O, and one bf16 on top left dQ and dK 1.6 times as far off as their own rounding
// does, where this leaves 1.15 times.  The gradients are rounded once at the end.
#include <limits.h>

#include "attn_tc.cuh"

namespace dr {
namespace {

using namespace attn;

// 16 softmax warps, 8 per TMEM slot: two threads per row, 32 columns each, as a slot's turn
// is their latency plus its products; then the load warp, two MMA warps and an idle one
constexpr int kThreads = 640;
constexpr int kLoadWarp = 16, kMmaWarp = 17;   // and the one after it
constexpr int kHalf = 32;
// registers per thread of the dK/dV kernel: 4 x 104 + 64 = 5 x 96, what the launch takes
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 104, kOtherRegs = 64;
static_assert(4 * kSoftmaxRegs + kOtherRegs == 5 * kLaunchRegs, "a larger sum would wait for ever");
constexpr int kN = 64;         // rows of a tile on the walked axis

// dK/dV: few long items, four stages.  dQ: many short ones, so the next item's own tiles are
// loaded behind this one (their load takes 5000 cycles, as long as four steps), three stages.
template <int D, bool KV> struct Smem {
  static constexpr int kStages = KV ? 4 : 3, kOwns = KV ? 1 : 2;
  static constexpr int kOwn = kM * D * 2, kTile = kN * D * 2;
  static constexpr int oX = 0, oY = kOwn, kOwnStride = 2 * kOwn;
  static constexpr int oA = kOwns * kOwnStride, oB = oA + kStages * kTile;
  static constexpr int oVec = oB + kStages * kTile, kBytes = oVec + (KV ? kStages * 2 * kN * 4 : 0) + 1024;
};
constexpr int kMostStages = 4;

// Column of k-step k of P or dS: each thread leaves its 32 values, packed in 16 columns,
// over the first of the 32 that it read, so the two threads of a row need no barrier.
__host__ __device__ constexpr uint32_t half_col(int k) { return (k >> 1) * kHalf + (k & 1) * 8; }

// A thread's 32 values of dS as bf16 and, in the other 16 columns, what that rounding left.
__device__ __forceinline__ void put_split(uint32_t to, const float (&g)[kHalf]) {
#pragma unroll
  for (int h = 0; h < kHalf / 2; h += 8) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = g[2 * (h + k)], y = g[2 * (h + k) + 1];
      hi[k] = tc::pack_bf16(x, y);
      lo[k] = tc::pack_bf16(x - __uint_as_float(hi[k] << 16), y - __uint_as_float(hi[k] & 0xffff0000u));
    }
    tmem_st8(to + h, hi);
    tmem_st8(to + kHalf / 2 + h, lo);
  }
}

__device__ __forceinline__ bool bounded(uint64_t* bar, uint32_t parity) {
  if (wait_phase(bar, parity)) return true;
  set_status(DR_ERR_TIMEOUT);
  return false;
}

// ------------------------------------------------------------------ the rows' numbers

// D / 8 lanes per row, kRowsAhead rows whose loads go together.
constexpr int kRowsAhead = 4;

template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(AttnArgs a) {
  constexpr int LK = D / 8, G = 256 / LK;
  const int c = 8 * (threadIdx.x % LK);
  // a block's first row by one long division, its others by short ones
  const long long all = (long long)a.B * a.Tp * a.H, e0 = (long long)blockIdx.x * (G * kRowsAhead);
  const long long bt0 = e0 / a.H;
  const int h0 = static_cast<int>(e0 - bt0 * a.H), b0 = static_cast<int>(bt0 / a.Tp),
            t0 = static_cast<int>(bt0 - (long long)b0 * a.Tp);
  uint4 o[kRowsAhead], g[kRowsAhead];
  int t[kRowsAhead];
  long long bh[kRowsAhead];
#pragma unroll
  for (int r = 0; r < kRowsAhead; ++r) {
    const int x = threadIdx.x / LK + r * G;
    const uint32_t hh = h0 + x, tt = t0 + hh / a.H, h = hh % a.H;
    t[r] = tt % a.Tp;
    const int b = b0 + tt / a.Tp;
    bh[r] = (long long)b * a.H + h;
    const bool in = e0 + x < all && t[r] < a.T;
    if (e0 + x >= all) t[r] = -1;
    const long long at = (((long long)b * a.T + t[r]) * a.H + h) * D + c;
    o[r] = in ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.out) + at) : make_uint4(0, 0, 0, 0);
    g[r] = in ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d_out) + at) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < kRowsAhead; ++r) {
    float x[8], y[8], s = 0.f;
    tc::unpack8(o[r], x);
    tc::unpack8(g[r], y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * y[i];
#pragma unroll
    for (int w = LK / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (c || t[r] < 0) continue;
    const float lse = t[r] < a.T ? a.lse[bh[r] * a.T + t[r]] : -INFINITY;
    a.nlse2[bh[r] * a.Tp + t[r]] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
    a.delta[bh[r] * a.Tp + t[r]] = -s;
  }
}

// ------------------------------------------------------------------ the shared pipeline

// One CTA per SM walks its work items, an item's steps one after another; steps and items
// are numbered through, so that the next item's loads and first products run behind the last
// one's softmax and stores.  X, Y: the own tiles (dK/dV: K, V; dQ: Q, dO), A, B: the walked
// ones (Q, dO; K, V).  Per step: slot S = X A^T, slot dP = Y B^T; then, from what the softmax
// warps left in their place, acc0 += [S] B (dK/dV only) and acc1 += [dP] A.
struct Pipe {
  uint64_t own_full[2], own_empty[2], full[kMostStages], empty[kMostStages], fix, s[2], p[2], free[2], acc_full, acc_empty, end[2];
  uint32_t tmem;
};

__device__ __forceinline__ void pipe_init(Pipe& q, int tid, int warp) {
  if (tid == 0) {
    for (int i = 0; i < kMostStages; ++i) mbar_init(&q.full[i], 1), mbar_init(&q.empty[i], 1);
    mbar_init(&q.fix, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&q.own_full[i], 1), mbar_init(&q.own_empty[i], 1), mbar_init(&q.s[i], 1), mbar_init(&q.p[i], 256), mbar_init(&q.free[i], 1), mbar_init(&q.end[i], 1);
    mbar_init(&q.acc_full, 1), mbar_init(&q.acc_empty, 512);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&q.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity) {   // of a whole warp
  return __all_sync(0xffffffffu, bounded(bar, parity)) != 0;
}

// Where a warp stands: items (with steps) and steps gone by.
struct Walk { uint32_t items, steps; };

// The MMA warps' parts of an item of n steps: one issues S and dP, the other the products
// into the accumulators (in order, so that sums keep their order).  A wait costs either of
// them 200 to 300 cycles even where nothing is waited for, in which the queue of issued
// products runs dry; two warps cover each other's.  A warp walks together and one lane
// issues, so that the descriptors stay in uniform registers.  TMEM: slot i at 128 i (S, then
// 64 columns on dP), accumulators at 256 and 256 + D.  KV: the dK/dV products, else dQ's.
template <int D, bool KV>
__device__ __forceinline__ bool scores_item(Pipe& q, uint8_t* sm, uint32_t tm, Walk& at, int n) {
  using L = Smem<D, KV>;
  constexpr uint32_t kStages = L::kStages, ID_S = idesc_bf16(kM, kN, 0, 0);
  const uint32_t own = at.items % L::kOwns;
  const uint64_t x = desc_kmajor(smem_u32(sm + L::oX + own * L::kOwnStride));
  const uint64_t y = desc_kmajor(smem_u32(sm + L::oY + own * L::kOwnStride));
  const uint32_t A = smem_u32(sm + L::oA), B = smem_u32(sm + L::oB);
  if (!all_wait(&q.own_full[own], (at.items / L::kOwns) & 1)) return false;
  for (int i = 0; i < n; ++i, ++at.steps) {
    const uint32_t gi = at.steps, slot = gi & 1, st = gi % kStages, s = tm + 128 * slot;
    if (!all_wait(&q.full[st], (gi / kStages) & 1)) return false;
    if (gi >= 2 && !all_wait(&q.free[slot], ((gi >> 1) - 1) & 1)) return false;
    tc_fence_after();   // the slot's columns have been read and its operands used
    const uint64_t dA = desc_kmajor(A + st * L::kTile), dB = desc_kmajor(B + st * L::kTile);
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) mma_bf16(s, x + step_kmajor<kM>(k), dA + step_kmajor<kN>(k), ID_S, k > 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) mma_bf16(s + 64, y + step_kmajor<kM>(k), dB + step_kmajor<kN>(k), ID_S, k > 0);
      mma_commit(&q.s[slot]);
      if (i == n - 1) mma_commit(&q.own_empty[own]);
    }
  }
  at.items += 1;
  return true;
}

template <int D, bool KV>
__device__ __forceinline__ bool sums_item(Pipe& q, uint8_t* sm, uint32_t tm, Walk& at, int n) {
  using L = Smem<D, KV>;
  constexpr uint32_t kStages = L::kStages, ID_ACC = idesc_bf16(kM, D, 0, 1);
  const uint32_t A = smem_u32(sm + L::oA), B = smem_u32(sm + L::oB);
  if (at.items > 0 && !all_wait(&q.acc_empty, (at.items - 1) & 1)) return false;
  for (int j = 0; j < n; ++j, ++at.steps) {
    const uint32_t gj = at.steps, slot = gj & 1, st = gj % kStages, p = tm + 128 * slot;
    if (!all_wait(&q.p[slot], (gj >> 1) & 1)) return false;
    tc_fence_after();
    const uint64_t dA = desc_mnmajor<kN>(A + st * L::kTile), dB = desc_mnmajor<kN>(B + st * L::kTile);
    if (elect_one()) {
      if (KV) {
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          mma_bf16_ta(tm + 256, p + half_col(k), dB + step_mnmajor(k), ID_ACC, j > 0 || k > 0);
      }
#pragma unroll
      for (int k = 0; k < kN / 16; ++k)
        mma_bf16_ta(tm + 256 + D, p + 64 + half_col(k), dA + step_mnmajor(k), ID_ACC, j > 0 || k > 0);
#pragma unroll
      for (int k = 0; k < kN / 16; ++k)
        mma_bf16_ta(tm + 256 + D, p + 64 + kHalf / 2 + half_col(k), dA + step_mnmajor(k), ID_ACC, true);
      mma_commit(&q.free[slot]);
      mma_commit(&q.empty[st]);
      if (j == n - 1) mma_commit(&q.acc_full);
    }
  }
  at.items += 1;
  return true;
}

// An MMA warp's end: no MMA may be under way when the CTA ends.
__device__ __forceinline__ void mma_end(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mma_commit(bar);
  wait_phase(bar, 0);
  tc_fence_before();
}

// The load warp's end: no copy may be in flight when the CTA ends.
template <class L>
__device__ __forceinline__ void load_end(Pipe& q, const Walk& at) {
  for (uint32_t i = at.items > L::kOwns ? at.items - L::kOwns : 0; i < at.items; ++i)
    wait_phase(&q.own_full[i % L::kOwns], (i / L::kOwns) & 1);
  for (uint32_t i = at.steps > L::kStages ? at.steps - L::kStages : 0; i < at.steps; ++i)
    wait_phase(&q.full[i % L::kStages], (i / L::kStages) & 1);
}

// Loads the own tiles of the load warp's next item: 128 rows from `row` of two tensors.
template <class L, int D>
__device__ __forceinline__ bool load_own(Pipe& q, uint8_t* sm, Walk& at, int lane, const CUtensorMap& X,
                                         const CUtensorMap& Y, int h, int row, int b) {
  const uint32_t own = at.items % L::kOwns;
  if (at.items >= L::kOwns && !all_wait(&q.own_empty[own], (at.items / L::kOwns - 1) & 1)) return false;
  if (lane == 0) {
    uint8_t* to = sm + own * L::kOwnStride;
    mbar_expect_tx(&q.own_full[own], 2 * L::kOwn);
    for (int c = 0; c < D / 64; ++c) {
      tma_load_4d(to + L::oX + c * kM * 128, &X, &q.own_full[own], 64 * c, h, row, b);
      tma_load_4d(to + L::oY + c * kM * 128, &Y, &q.own_full[own], 64 * c, h, row, b);
    }
  }
  ++at.items;
  return true;
}

// 128 lanes' rows of N accumulator columns -> bf16 rows (or fp32 parts)
template <int N>
__device__ __forceinline__ void store_acc(uint32_t tacc, bool any, float f, __nv_bfloat16* o, float* part) {
#pragma unroll
  for (int c = 0; c < N; c += 16) {
    float v[16];
    if (any) {
      tmem_ld16(tacc + c, v);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
    }
    if (part) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(part + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else if (o) {
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = v[e + k] * f;
        *reinterpret_cast<uint4*>(o + c + e) = tc::pack8(x);
      }
    }
  }
}

// ------------------------------------------------------------------ dK, dV

// One work item: 128 keys of a key/value head and the query rows that see them, or one piece
// of the rows that see only the sinks (first: they are as long as the others or longer).
struct KeyItem {
  int hk, b, j0, len, i_begin, per, n, piece;   // steps: `per` tiles of kN rows from i_begin, for each head
  bool far;
  __device__ __forceinline__ KeyItem(const AttnArgs& a, uint32_t it) {
    hk = it % a.Hkv, b = it / a.Hkv % a.B;
    const int item = it / a.Hkv / a.B;
    far = item < a.n_far;
    piece = far ? 1 + item : 0;
    j0 = far ? 0 : (item - a.n_far) * kM;
    len = uniform(real_len(a.lens, b, a.reach));
    int i_end;   // i_begin is a multiple of kN
    if (far) {
      i_begin = a.far_first + item * a.far_rows;
      i_end = len > 0 ? min(a.T, i_begin + a.far_rows) : i_begin;
    } else {
      const QueryRows r(j0, min(j0 + kM, a.S) - 1, len, a.window, a.n_sink, a.q_start, a.T);
      i_begin = r.begin / kN * kN;
      i_end = j0 == 0 && a.n_far ? min(r.end, a.far_first) : r.end;
    }
    per = i_end > i_begin ? (i_end - i_begin + kN - 1) / kN : 0;
    n = per * a.G;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       AttnArgs a) {
  using L = Smem<D, true>;
  constexpr uint32_t kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Pipe q;
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
  const uint32_t n_item = ((a.S + kM - 1) / kM + a.n_far) * a.B * a.Hkv;   // a grid's worth: below 2^31
  pipe_init(q, tid, warp);
  const uint32_t tmem = uniform(q.tmem);
  Walk at = {0, 0};
  bool ok = true;

  if (warp < 16) {   // two threads per key; the slots' warps take the steps in turn
    more_registers<kSoftmaxRegs>();
    const int w = warp / 8, half = warp / 4 % 2, row = (warp % 4) * 32 + lane, c0 = kHalf * half;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + 128 * w + lanes;
    const float c2 = a.scale * 1.4426950408889634f;
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      int n, per, first, j0, len;
      {
        const KeyItem x(a, it);
        n = x.n, per = x.per, first = a.q_start + x.i_begin, j0 = x.j0, len = x.len;
      }
      const int j = j0 + row;
      for (int i = (w - at.steps) & 1; i < n; i += 2) {
        const uint32_t gi = at.steps + i, st = gi % kStages;
        if (!(ok = all_wait(&q.s[w], (gi >> 1) & 1))) break;
        // this stage's numbers (with its tiles)
        if (!(ok = all_wait(&q.full[st], (gi / kStages) & 1))) break;
        tc_fence_after();
        const uint32_t nl = smem_u32(sm + L::oVec + st * 2 * kN * 4) + 4 * c0, nd = nl + kN * 4;
        const int p0 = first + (i % per) * kN;
        const bool whole = p0 >= j0 + kM - 1 && j0 + kM <= len &&
                           (p0 + kN - 1 - j0 < a.window || j0 + kM <= a.n_sink);
        // the rows of this half that see this key, as bits
        const uint32_t word =
            j < len ? bits_below(j < a.n_sink ? 32 : j + a.window - p0 - c0) & ~bits_below(j - p0 - c0) : 0u;
        float s[kHalf], g[kHalf];
        uint32_t pk[kHalf / 2];
        tmem_ld32(tS + c0, reinterpret_cast<uint32_t*>(s));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kHalf; c += 4) {
          const float4 l4 = lds128(nl + 4 * c);
          fma2v(s[c], s[c + 1], c2, l4.x, l4.y);
          fma2v(s[c + 2], s[c + 3], c2, l4.z, l4.w);
        }
#pragma unroll
        for (int c = 0; c < kHalf; ++c) s[c] = ex2(s[c]);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < kHalf; ++c) s[c] = word & (1u << c) ? s[c] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < kHalf; c += 2) pk[c / 2] = tc::pack_bf16(s[c], s[c + 1]);
        tmem_ld32(tS + 64 + c0, reinterpret_cast<uint32_t*>(g));
        tmem_st16(tS + c0, pk);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kHalf; c += 4) {
          const float4 d4 = lds128(nd + 4 * c);
          add_mul2(g[c], g[c + 1], d4.x, d4.y, s[c], s[c + 1]);
          add_mul2(g[c + 2], g[c + 3], d4.z, d4.w, s[c + 2], s[c + 3]);
        }
        if (!whole) {   // what a key past the end holds may be NaN
#pragma unroll
          for (int c = 0; c < kHalf; ++c) g[c] = word & (1u << c) ? g[c] : 0.f;
        }
        put_split(tS + 64 + c0, g);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&q.p[w]);
      }
      if (!ok || (n > 0 && !(ok = all_wait(&q.acc_full, at.items & 1)))) break;
      tc_fence_after();
      const KeyItem x(a, it);   // again: not carried through the steps
      // slot 0's warps: dV, slot 1's: dK, half of the channels each
      const long long o = (((long long)x.b * a.S + j) * a.Hkv + x.hk) * D + half * (D / 2);
      const bool part = a.n_far && x.j0 == 0 && j < a.n_sink;
      float* p = part ? a.sink_part + (((((long long)x.b * a.Hkv + x.hk) * (1 + a.n_far) + x.piece) * 2 + (1 - w)) *
                                           a.n_sink + j) * D + half * (D / 2)
                      : nullptr;
      store_acc<D / 2>(tmem + 256 + w * D + half * (D / 2) + lanes, x.n > 0, w ? a.scale : 1.f,
                       j < a.S && !part && !x.far ? static_cast<__nv_bfloat16*>(w ? a.dk : a.dv) + o : nullptr, p);
      tc_fence_before();
      if (x.n > 0) mbar_arrive(&q.acc_empty);
      at.steps += x.n, at.items += x.n > 0;
    }
  } else {
    fewer_registers<kOtherRegs>();
  }
  if (warp == kLoadWarp) {   // the whole warp walks, one lane issues
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const KeyItem x(a, it);
      for (int i = 0; i < x.n; ++i) {
        const uint32_t gi = at.steps, st = gi % kStages;
        const int h = x.hk * a.G + i / x.per, i0 = x.i_begin + (i % x.per) * kN;
        if (gi >= kStages && !(ok = all_wait(&q.empty[st], (gi / kStages - 1) & 1))) break;
        if (lane == 0) {
          mbar_expect_tx(&q.full[st], 2 * L::kTile + 2 * kN * 4);
          for (int c = 0; c < D / 64; ++c) {
            tma_load_4d(sm + L::oA + st * L::kTile + c * kN * 128, &tmQ, &q.full[st], 64 * c, h, i0, x.b);
            tma_load_4d(sm + L::oB + st * L::kTile + c * kN * 128, &tmO, &q.full[st], 64 * c, h, i0, x.b);
          }
          const long long row = ((long long)x.b * a.H + h) * a.Tp + i0;
          bulk_load(sm + L::oVec + st * 2 * kN * 4, a.nlse2 + row, kN * 4, &q.full[st]);
          bulk_load(sm + L::oVec + st * 2 * kN * 4 + kN * 4, a.delta + row, kN * 4, &q.full[st]);
        }
        ++at.steps;
        if (i == 0) {
          if (!(ok = load_own<L, D>(q, sm, at, lane, tmK, tmV, x.hk, x.j0, x.b))) break;
        }
      }
    }
    load_end<L>(q, at);
  } else if (warp == kMmaWarp) {
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const KeyItem x(a, it);
      if (x.n > 0) ok = scores_item<D, true>(q, sm, tmem, at, x.n);
    }
    mma_end(&q.end[0]);
  } else if (warp == kMmaWarp + 1) {
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const KeyItem x(a, it);
      if (x.n > 0) ok = sums_item<D, true>(q, sm, tmem, at, x.n);
    }
    mma_end(&q.end[1]);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The sinks' gradients: their pieces in order.
template <int D>
__global__ void __launch_bounds__(D) attn_sink_join_kernel(AttnArgs a) {
  const int j = blockIdx.x % a.n_sink, x = blockIdx.x / a.n_sink % 2;   // x = 0: dk, 1: dv
  const long long bh = blockIdx.x / a.n_sink / 2;
  if (j >= a.S) return;
  const float* p = a.sink_part + (bh * (1 + a.n_far) * 2 + x) * a.n_sink * D + j * D + threadIdx.x;
  float s = 0.f;
  for (int i = 0; i <= a.n_far; ++i) s += p[(long long)i * 2 * a.n_sink * D];
  const long long b = bh / a.Hkv, hk = bh % a.Hkv;
  const long long o = ((b * a.S + j) * a.Hkv + hk) * D + threadIdx.x;
  static_cast<__nv_bfloat16*>(x ? a.dv : a.dk)[o] = __float2bfloat16_rn(x ? s : s * a.scale);
}

// ------------------------------------------------------------------ dQ

// One work item: 128 query rows of a head; steps: the tiles of kN keys that they see.
struct RowItem {
  int h, i0, b, hk, len;
  KeyTiles tiles;
  __device__ __forceinline__ RowItem(const AttnArgs& a, int n_block, uint32_t it)
      : h(it % a.H),
        i0(it / a.H % n_block * kM),
        b(it / a.H / n_block),
        hk(h / a.G),
        len(uniform(real_len(a.lens, b, a.reach))),
        tiles(a.q_start + i0, a.q_start + min(i0 + kM, a.T) - 1, len, a.window, a.n_sink, kN) {}
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      AttnArgs a) {
  using L = Smem<D, false>;
  constexpr uint32_t kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Pipe q;
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
  const int n_block = (a.T + kM - 1) / kM;
  const uint32_t n_item = a.B * a.H * n_block;   // a grid's worth: below 2^31
  pipe_init(q, tid, warp);
  const uint32_t tmem = uniform(q.tmem);
  Walk at = {0, 0};
  bool ok = true;

  if (warp < 16) {   // two threads per query row; the slots' warps take the steps in turn
    const int w = warp / 8, row = (warp % 4) * 32 + lane, c0 = kHalf * (warp / 4 % 2);
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + 128 * w + lanes;
    const float c2 = a.scale * 1.4426950408889634f;
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const RowItem x(a, n_block, it);
      const int n = x.tiles.n, i = x.i0 + row, p = a.q_start + i, p0 = a.q_start + x.i0;
      float nl = -INFINITY, nd = 0.f;
      if (i < a.T) {
        const long long r = ((long long)x.b * a.H + x.h) * a.Tp + i;
        nl = a.nlse2[r], nd = a.delta[r];
      }
      for (int k = (w - at.steps) & 1; k < n; k += 2) {
        const int t0 = x.tiles[k] * kN;
        if (!(ok = all_wait(&q.s[w], ((at.steps + k) >> 1) & 1))) break;
        tc_fence_after();
        const bool whole = t0 + kN - 1 <= p0 && t0 + kN <= x.len && p0 + kM - 1 - t0 < a.window;
        const uint32_t word = RowMask(a, p, t0, x.len).word(c0);
        float s[kHalf], g[kHalf];
        uint32_t pk[kHalf / 2];
        tmem_ld32(tS + c0, reinterpret_cast<uint32_t*>(s));
        tmem_ld32(tS + 64 + c0, reinterpret_cast<uint32_t*>(g));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kHalf; c += 2) {
          fma2(s[c], s[c + 1], c2, nl);
          s[c] = ex2(s[c]), s[c + 1] = ex2(s[c + 1]);
          add_mul2(g[c], g[c + 1], nd, nd, s[c], s[c + 1]);
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < kHalf; ++c) g[c] = word & (1u << c) ? g[c] : 0.f;
        }
        put_split(tS + 64 + c0, g);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&q.p[w]);
      }
      if (!ok || (n > 0 && !(ok = all_wait(&q.acc_full, at.items & 1)))) break;
      tc_fence_after();
      const int o = warp / 4 * (D / 4);   // a quarter of the channels each
      store_acc<D / 4>(tmem + 256 + D + o + lanes, n > 0, a.scale,
                       i < a.T ? static_cast<__nv_bfloat16*>(a.dq) + (((long long)x.b * a.T + i) * a.H + x.h) * D + o
                               : nullptr,
                       nullptr);
      tc_fence_before();
      if (n > 0) mbar_arrive(&q.acc_empty);
      at.steps += n, at.items += n > 0;
    }
  } else if (warp == kLoadWarp) {
    uint32_t n_fix = 0;
    bool ahead = false;   // has this item's Q and dO been loaded with the last one?
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const RowItem x(a, n_block, it);
      const int fix_tile = x.len < a.S && x.len % kN ? x.len / kN : -1;   // its K rows from len on become 0
      for (int k = 0; k < x.tiles.n; ++k) {
        const uint32_t gi = at.steps, st = gi % kStages;
        const int t0 = x.tiles[k] * kN;
        if (gi >= kStages && !(ok = all_wait(&q.empty[st], (gi / kStages - 1) & 1))) break;
        uint64_t* full = x.tiles[k] == fix_tile ? &q.fix : &q.full[st];
        if (lane == 0) {
          mbar_expect_tx(full, 2 * L::kTile);
          for (int c = 0; c < D / 64; ++c) {
            tma_load_4d(sm + L::oA + st * L::kTile + c * kN * 128, &tmK, full, 64 * c, x.hk, t0, x.b);
            tma_load_4d(sm + L::oB + st * L::kTile + c * kN * 128, &tmV, full, 64 * c, x.hk, t0, x.b);
          }
        }
        if (k == 0 && !ahead && !(ok = load_own<L, D>(q, sm, at, lane, tmQ, tmO, x.h, x.i0, x.b))) break;
        if (k == min(2, x.tiles.n - 1)) {
          ahead = false;
          if (it + gridDim.x < n_item) {
            const RowItem y(a, n_block, it + gridDim.x);
            ahead = y.tiles.n > 0;
            if (ahead && !(ok = load_own<L, D>(q, sm, at, lane, tmQ, tmO, y.h, y.i0, y.b))) break;
          }
        }
        if (full == &q.fix) {
          if (!(ok = all_wait(&q.fix, n_fix & 1))) break;
          ++n_fix;
          const int r0 = x.len % kN;
          for (int e = lane; e < (kN - r0) * 8 * (D / 64); e += 32) {
            const int c = e / ((kN - r0) * 8), y = e % ((kN - r0) * 8);
            reinterpret_cast<uint4*>(sm + L::oA + st * L::kTile + c * kN * 128 + r0 * 128)[y] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q.full[st]);
        }
        ++at.steps;
      }
    }
    load_end<L>(q, at);
  } else if (warp == kMmaWarp) {
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const RowItem x(a, n_block, it);
      if (x.tiles.n > 0) ok = scores_item<D, false>(q, sm, tmem, at, x.tiles.n);
    }
    mma_end(&q.end[0]);
  } else if (warp == kMmaWarp + 1) {
    for (uint32_t it = blockIdx.x; it < n_item && ok; it += gridDim.x) {
      const RowItem x(a, n_block, it);
      if (x.tiles.n > 0) ok = sums_item<D, false>(q, sm, tmem, at, x.tiles.n);
    }
    mma_end(&q.end[1]);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host side

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// How the query rows that see only the sinks of key tile 0 are cut: pieces about as long
// as what any other key tile is seen by.
void cut_far(AttnArgs& a) {
  a.Tp = (a.T + kN - 1) / kN * kN;
  a.n_far = 0, a.far_first = a.Tp, a.far_rows = kN;
  if (a.n_sink == 0) return;
  const long long first = ((long long)kM - 1 + a.window - a.q_start + kN - 1) / kN * kN;
  if (first >= a.T) return;
  a.far_first = first > 0 ? static_cast<int>(first) : 0;
  const long long rows = ((long long)a.window + kM + kN - 1) / kN * kN;
  a.far_rows = static_cast<int>(rows < 512 ? 512 : rows);
  a.n_far = (a.T - a.far_first + a.far_rows - 1) / a.far_rows;
}

template <int D>
cudaError_t bwd(const AttnArgs& a, int sms, cudaStream_t st) {
  using KeySmem = Smem<D, true>;
  using RowSmem = Smem<D, false>;
  constexpr int LK = D / 8;
  const long long rows = (long long)a.B * a.Tp * a.H;
  const long long per = 256 / LK * kRowsAhead;
  attn_rows_kernel<D><<<static_cast<unsigned>((rows + per - 1) / per), 256, 0, st>>>(a);
  const long long o_st = (long long)a.H * D, o_sb = o_st * a.T;
  CUtensorMap q, o, k, v;
  auto maps = [&](int q_rows, int k_rows) {
    return make_map(&q, a.q, a.B, a.T, a.H, D, a.q_sb, a.q_st, a.q_sh, q_rows) &&
           make_map(&o, a.d_out, a.B, a.T, a.H, D, o_sb, o_st, D, q_rows) &&
           make_map(&k, a.k, a.B, a.S, a.Hkv, D, a.k_sb, a.k_st, a.k_sh, k_rows) &&
           make_map(&v, a.v, a.B, a.S, a.Hkv, D, a.v_sb, a.v_st, a.v_sh, k_rows);
  };
  cudaError_t e = cudaFuncSetAttribute(attn_dkv_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, KeySmem::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_dq_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowSmem::kBytes);
  if (e != cudaSuccess) return e;
  if (!maps(kN, kM)) return cudaErrorInvalidValue;
  auto grid = [&](long long items) { return static_cast<unsigned>(items < sms ? items : sms); };
  const long long key_items = ((long long)(a.S + kM - 1) / kM + a.n_far) * a.B * a.Hkv;
  attn_dkv_tc_kernel<D><<<grid(key_items), kThreads, KeySmem::kBytes, st>>>(q, o, k, v, a);
  if (!maps(kM, kN)) return cudaErrorInvalidValue;
  const long long row_items = (long long)a.B * a.H * ((a.T + kM - 1) / kM);
  attn_dq_tc_kernel<D><<<grid(row_items), kThreads, RowSmem::kBytes, st>>>(q, o, k, v, a);
  if (a.n_far) attn_sink_join_kernel<D><<<static_cast<unsigned>((long long)a.B * a.Hkv * 2 * a.n_sink), D, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_bwd_tc_status(int* word, cudaStream_t st) { return take_status(word, st); }

size_t attn_bwd_tc_workspace(const AttnArgs& in) {
  AttnArgs a = in;
  cut_far(a);
  const size_t rows = align256(static_cast<size_t>(a.B) * a.H * a.Tp * 4);
  return 2 * rows +
         (a.n_far ? align256(static_cast<size_t>(a.B) * a.Hkv * (1 + a.n_far) * 2 * a.n_sink * a.d * 4) : 0);
}

cudaError_t launch_attn_bwd_tc(AttnArgs a, int sms, void* workspace, cudaStream_t st) {
  cut_far(a);
  const size_t rows = align256(static_cast<size_t>(a.B) * a.H * a.Tp * 4);
  char* p = static_cast<char*>(workspace);
  a.nlse2 = reinterpret_cast<float*>(p);
  a.delta = reinterpret_cast<float*>(p + rows);
  a.sink_part = reinterpret_cast<float*>(p + 2 * rows);
  return a.d == 64 ? bwd<64>(a, sms, st) : bwd<128>(a, sms, st);
}

}  // namespace dr
