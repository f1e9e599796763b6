// Host program: the addresses that the norms around a block form, for every row length from 1 to
// 8192 values, both directions, all types and every phase of odd rows.  Prints "ok" or what is wrong.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "block_norm_rows.cuh"

using namespace dr;
using namespace dr::norm_rows;

#define CHECK(x)                                                                                           \
  do {                                                                                                     \
    if (!(x)) printf("line %d: %s: D %d M %d order %d E %d es %d phase %d\n", __LINE__, #x, D, M, ORDER, E, es, phase), exit(1); \
  } while (0)

// One tensor's rows, `es` bytes a value, as the threads of a row read them from their copies.
template <int ORDER, int E> void rows(int D, int tpr, int es, bool ring, int M) {
  std::vector<char> seen(D);
  for (int first = 0; first < (ORDER == kOdd ? 8 : 1); ++first) {
    const int phase = phase_of(first, D);
    const long long at[] = {first, first + 8, M - 1 - (M - 1 - first) % 8};   // rows of one block
    for (long long row : at) CHECK(phase_of(row, D) == phase);
    const char* base = reinterpret_cast<const char*>(uintptr_t(1) << 40);
    const uintptr_t end = reinterpret_cast<uintptr_t>(base) + (uintptr_t)M * D * es;
    if (ring) {
      for (long long row : at) {
        const RowCopy r(base, row, D, D, phase, es, M);
        CHECK(r.lo % 16 == 0 && r.bytes % 16 == 0 && r.lo >= reinterpret_cast<uintptr_t>(base) && r.lo + r.bytes <= end);
        CHECK((int)r.bytes <= copy_bytes(D, es));
      }
      CHECK(copy_bytes(D, es) % 16 == 0);
    }
    const int usual = RowCopy(base, first, D, D, phase, es, M).bytes / es;
    const int last = RowCopy(base, M - 1, D, D, phase_of(M - 1, D), es, M).bytes / es;
    const bool is_last = phase == phase_of(M - 1, D);
    std::fill(seen.begin(), seen.end(), 0);
    for (int t = 0; t < tpr; ++t) {
      const Columns<ORDER, E> c(D, tpr, t, phase);
      for (int e0 = 0; e0 < E; e0 += 8) {
        const int n = c.at(e0);
        for (int e = 0; e < 8; ++e) {
          if (!c.in(c.at(e0 + e))) continue;
          CHECK(!seen[c.at(e0 + e)]);
          seen[c.at(e0 + e)] = 1;
        }
        if (ORDER == kApart) continue;
        if (c.whole(e0, n)) {   // 8 neighbours at once, on 8 of the tensor
          CHECK(n >= 0 && n + 8 <= D && (n + c.phase()) % 8 == 0);
          if (ring && is_last) CHECK(n + c.phase() + 8 <= last);
        }
        if (ring && (ORDER == kOdd || c.whole(e0, n))) {   // what is read of a copy, masked or not
          const int from = ORDER == kOdd && n >= D ? 0 : n + c.phase();
          CHECK(from >= 0 && from + 8 <= usual);
        }
      }
    }
    for (int n = 0; n < D; ++n) CHECK(seen[n]);
  }
}

template <int ORDER, int E>
void plans(const BlockNormArgs& args, int threads, int blocks, bool with_ring, int es_a, int es_h, int own) {
  const int D = args.D, es = es_h;
  BlockNormArgs a = args;
  for (int M : {1, 2, 151, 153, 1000, 100000, 1 << 30}) {
    const int phase = -1;
    a.M = M;
    const int bytes = row_bytes(a, es_a, es_h);
    const Plan p(a, 152, ORDER, E, threads * blocks, with_ring, bytes, own > 0, own);
    const bool wide = threads != kNarrow, ring = wide && with_ring && ORDER != kApart;
    const int in_row = D + (ORDER == kOdd ? 7 : 0);
    CHECK(p.threads <= threads && p.grid >= 1 && p.tpr * E >= in_row && (wide ? p.tpr == p.threads : p.tpr <= 32));
    CHECK(ring == (p.ring.stages > 0));
    const int rows = wide ? 1 : kNarrow / p.tpr;
    const long long per_block = ((long long)M + (long long)p.grid * rows - 1) / ((long long)p.grid * rows);
    if (ORDER == kOdd && per_block > 1) CHECK(p.grid * rows % 8 == 0);
    const int on_sm = (p.grid + 151) / 152;
    if (ring) {
      CHECK(p.ring.stages <= kMaxStages && (p.ring.stages >= 2 || per_block == 1));
      CHECK(p.smem >= (size_t)p.ring.stages * bytes + (size_t)own * p.threads && bytes % 16 == 0);
      CHECK((p.smem + 1024) * on_sm <= 228 * 1024);
    }
    CHECK(p.smem <= (size_t)kShared);
  }
}

template <int ORDER> void length(int D) {
  BlockNormArgs a{};
  a.D = D;
  a.h = a.branch = a.gate = &a;
  for (bool bwd : {false, true}) {
    if (bwd) a.d_y = a.d_h = &a;
    auto go = [&](auto e, auto threads, auto blocks) {
      constexpr int E = decltype(e)::value;
      auto types = [&](int es_a, int es_h, bool with_ring) {
        plans<ORDER, E>(a, threads, blocks, with_ring, es_a, es_h, bwd ? bwd_own(E) : 0);
        if (es_a != es_h) return;   // a tensor's rows are those of either type
        a.M = 4096;
        const Plan p(a, 152, ORDER, E, threads * blocks, with_ring, row_bytes(a, es_a, es_h), false, 0);
        rows<ORDER, E>(D, p.tpr, es_a, p.ring.stages > 0, D / 2 % 2 ? 4093 : 4096);   // the tensor ends on 8 values or elsewhere
      };
      types(2, 2, !bwd || ring_holds<__nv_bfloat16, E>());
      types(2, 4, !bwd || ring_holds<float, E>());
      types(4, 4, !bwd || ring_holds<float, E>());
    };
    if (bwd) bwd_shape(D, ORDER, go);
    else fwd_shape(D, ORDER, go);
  }
}

int main() {
  for (int D = 1; D <= kMaxRow; ++D) {
    BlockNormArgs a{};
    a.M = 4096, a.D = D, a.h_s = a.b_s = a.g_s = D;
    const int order = order_of(a);
    if (order == kEven) length<kEven>(D);
    else if (order == kOdd) length<kOdd>(D);
    if (order == kApart || D % 512 == 1 || D < 300) length<kApart>(D);
  }
  printf("ok\n");
  return 0;
}
