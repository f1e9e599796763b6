// block_norm_rows.cuh — how the norms around a block share a row out over threads and bring it
// into shared memory: the columns of a thread, the bytes of a copy, the blocks of a launch.
// Host code too, so that its addresses can be checked for every row length without a GPU.
#pragma once

#include <type_traits>

#include "block.cuh"

namespace dr {
namespace norm_rows {

constexpr int kMaxStages = 8;
constexpr int kMaxRow = 8192;     // 512 threads of 16 columns

// How a thread's E columns stand.
//   kEven  groups of 8 neighbours; the row's length is a multiple of 8
//   kOdd   groups of 8, cut where the row's values stand at multiples of 8 of the tensor.  In a
//          row of odd length that is `phase` columns before its start, and the first and the
//          last group are not whole.  A block's rows are a multiple of 8 apart, so the phase
//          and with it a thread's columns are the same in all of them.
//   kApart one column of every tpr, for rows that do not stand so
enum { kEven, kOdd, kApart };
template <int ORDER, int E> struct Columns {
  int D, tpr, t, phase_;
  uint32_t valid;   // kOdd: which of its columns are the row's, a bit for each
  __host__ __device__ __forceinline__ Columns(int D_, int tpr_, int t_, int phase)
      : D(D_), tpr(tpr_), t(t_), phase_(phase), valid(0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (ORDER == kOdd && in(at(e))) valid |= 1u << e;
  }
  __host__ __device__ __forceinline__ int phase() const { return ORDER == kOdd ? phase_ : 0; }
  __host__ __device__ __forceinline__ int at(int e) const {
    return ORDER == kApart ? e * tpr + t : (e / 8 * tpr + t) * 8 + e % 8 - phase();
  }
  __host__ __device__ __forceinline__ bool in(int n) const { return (ORDER != kOdd || n >= 0) && n < D; }
  // of the group from column e0 on, which is column n of the row
  __host__ __device__ __forceinline__ bool whole(int e0, int n) const {
    return ORDER == kEven ? n < D : (valid >> e0 & 255u) == 255u;
  }
};

// Rows come into shared memory by background copies, from their first group on.  What a group
// holds of the neighbouring rows is copied along; behind the tensor's last row nothing is, only
// the whole 16 bytes before its end.
struct RowCopy {
  uintptr_t lo;
  uint32_t bytes;
  __host__ __device__ __forceinline__ RowCopy(const void* base, long long row, long long stride, int D, int phase, int es,
                                              int M) {
    lo = reinterpret_cast<uintptr_t>(base) + (row * stride - phase) * es;
    const uint32_t all = static_cast<uint32_t>(phase + D) * es;
    bytes = row == M - 1 ? all & ~15u : (all + 8 * es - 1) / (8 * es) * (8 * es);
  }
};
// what a row's copy takes of shared memory
__host__ __device__ __forceinline__ int copy_bytes(int D, int es) { return (D % 8 ? D / 8 + 2 : D / 8) * 8 * es; }

// How a launch lays the rows' copies out.
struct RingLayout {
  int stages;
  uint32_t stage_bytes;
};

constexpr int kNarrow = 128;   // threads of a block whose rows are up to 32 threads each

__host__ __device__ __forceinline__ int phase_of(long long row, int D) { return static_cast<int>(row * D & 7); }

// Two rows of all five tensors have to fit an SM's shared memory.  With fp32 among them, rows of
// more than 4096 columns (16 per thread) would not: those are read from memory.
template <typename TH, int E> __host__ __device__ constexpr bool ring_holds() { return sizeof(TH) == 2 || E == 8; }

template <int N> using Int = std::integral_constant<int, N>;

// Do all rows start at multiples of 8 values of tensors on 16 bytes, or all equally far from
// one?  (Contiguous tensors of any row length do.)
inline int order_of(const BlockNormArgs& a) {
  auto ok = [&](const void* p, long long s) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (a.M == 1 || ((s - a.D) % 8 == 0 && (s >= a.D || a.D % 8 == 0))));
  };
  const bool groups = ok(a.h, a.h_s) && ok(a.branch, a.b_s) && ok(a.gate, a.g_s) && ok(a.h_out, a.D) && ok(a.y, a.D) &&
                      ok(a.d_h, a.D) && ok(a.d_y, a.D) && ok(a.dh, a.D) && ok(a.db, a.D) && ok(a.dg, a.D);
  return !groups || (a.D % 8 && a.D + 7 > kMaxRow) ? kApart : a.D % 8 ? kOdd : kEven;
}

// A launch: blocks that stay on every SM, in the place of `place` threads, and the rows on their
// way in what each of them has of its shared memory, two at least (a row's place goes to the
// next but one while the next is worked on): so much there is at every length.
constexpr int kShared = 227 * 1024 - 512;   // of an SM, for what a launch asks for

struct Plan {
  int tpr, threads, grid;
  RingLayout ring;
  size_t smem;
  Plan(const BlockNormArgs& a, int sms, int order, int e, int place, bool with_ring, int row_bytes, bool sums, int own = 0) {
    const int n = (a.D + (order == kOdd ? 7 : 0) + e - 1) / e;   // with the most that a phase adds
    int rows = 1;
    if (n <= 32) {
      for (tpr = 4; tpr < n; tpr *= 2) {}
      rows = kNarrow / tpr, threads = kNarrow;
    } else {
      tpr = threads = (n + 31) / 32 * 32;
    }
    with_ring = with_ring && n > 32 && order != kApart;
    const int blocks = place / threads;
    auto fit = [&] { return (blocks > 1 ? kShared / blocks - 2048 : kShared - own * threads) / row_bytes; };
    const long long most = (a.M + rows - 1LL) / rows, there = (long long)sms * blocks;
    grid = static_cast<int>(most < there ? most : there);
    if (order == kOdd && grid < most) grid = grid / 8 * 8;   // a block's rows have one phase
    ring.stage_bytes = row_bytes, ring.stages = 0;
    smem = sums && n <= 32 ? sizeof(float) * rows * 2 * a.D : 0;   // the block's rows' sums
    if (with_ring && grid) {
      const long long need = (most + grid - 1) / grid;
      ring.stages = fit() < kMaxStages ? fit() : kMaxStages;
      if (ring.stages > need) ring.stages = static_cast<int>(need);
      smem = (size_t)ring.stages * row_bytes;
    }
    smem += own * threads;
  }
};

inline int row_bytes(const BlockNormArgs& a, int es_a, int es_h) {
  auto of = [&](const void* p, int es) { return p ? copy_bytes(a.D, es) : 0; };
  return of(a.h, es_h) + of(a.branch, es_a) + of(a.gate, es_a) + of(a.d_y, es_a) + of(a.d_h, es_h);
}

// Columns per thread, the largest block and how many of them an SM's registers hold, by the
// row's length.
template <typename F> void fwd_shape(int D, int order, F&& go) {
  D += order == kOdd ? 7 : 0;
  if (D <= 256) go(Int<8>{}, Int<kNarrow>{}, Int<8>{});
  else if (D <= 2048) go(Int<8>{}, Int<256>{}, Int<3>{});
  else if (D <= 4096) go(Int<16>{}, Int<256>{}, Int<2>{});
  else go(Int<16>{}, Int<512>{}, Int<1>{});
}
template <typename F> void bwd_shape(int D, int order, F&& go) {
  D += order == kOdd ? 7 : 0;
  if (D <= 256) go(Int<8>{}, Int<kNarrow>{}, Int<4>{});
  else if (D <= 2048) go(Int<8>{}, Int<256>{}, Int<2>{});
  else if (D <= 4096) go(Int<8>{}, Int<512>{}, Int<1>{});
  else go(Int<16>{}, Int<512>{}, Int<1>{});
}

// Bytes of shared memory that a thread of the backward keeps its weights in.
constexpr int bwd_own(int e) { return e > 8 ? 2 * 4 * e : 0; }

}  // namespace norm_rows
}  // namespace dr
