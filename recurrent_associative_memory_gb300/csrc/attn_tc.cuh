// attn_tc.cuh — what the tcgen05 window-attention kernels share: TMEM loads and stores,
// the MMA with its A operand in TMEM, packed fp32 arithmetic, tile masks, tensor maps.
// Their translation units are compiled as whole programs: with relocatable device code the
// compiler ignores setmaxnreg, and a row of 128 scores does not fit the registers that an
// even split leaves (428 bytes of spills per thread instead of none).
#pragma once

#include "layers.cuh"
#include "tc_common.cuh"

namespace dr {
namespace attn {

using namespace umma;

constexpr uint64_t kWaitNs = 2000000000ull;   // a wait gives up after this long
constexpr int kM = 128;                       // rows of a tile, on either axis

// Bounded wait.  The global timer is only read every 256 polls: sixteen warps that read it
// at every poll slow the one that issues the MMAs.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255) == 0) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitNs) return false;
    }
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The same value in every lane, known as such to the compiler: an MMA's descriptors, built
// from such values under uniform control flow, stay in uniform registers, where the
// instruction wants them.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// D(tmem) (+)= A(tmem) * B(smem desc): row r of A in lane r, two bf16 per column
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// 32 lanes x 32 consecutive columns (lane = thread)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21,"
      " %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (x0, x1) * m + a on a pair of fp32 at once
__device__ __forceinline__ void fma2(float& x0, float& x1, float m, float a) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(m), "f"(a));
}

// (x0, x1) * m + (a0, a1) and (x0 + a0, x1 + a1) * (y0, y1), a pair of fp32 at once
__device__ __forceinline__ void fma2v(float& x0, float& x1, float m, float a0, float a1) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %4};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(m), "f"(a0), "f"(a1));
}
__device__ __forceinline__ void add_mul2(float& x0, float& x1, float a0, float a1, float y0, float y1) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 z, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, z;\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1), "f"(y0), "f"(y1));
}

// The key tiles of kM keys that a tile of query rows can see, as a set.
struct TileSet {
  int n_first, w_begin, w_end;
  __device__ __forceinline__ TileSet(const AttnArgs& a, int i0, int len) {
    const KeyTiles t(a.q_start + i0, a.q_start + min(i0 + kM, a.T) - 1, len, a.window, a.n_sink, kM);
    n_first = t.n_first, w_begin = t.w_begin, w_end = t.w_begin + t.n - t.n_first;
    if (i0 >= a.T) n_first = w_end = 0;
  }
  __device__ __forceinline__ bool has(int tile) const {
    return tile < n_first || (tile >= w_begin && tile < w_end);
  }
};

// 16 bytes of shared memory by their 32-bit address: behind the rounding of the dynamic
// array's start the compiler no longer knows the space and would load generically.
__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");   // behind the wait for the copy that wrote them
  return v;
}

// The bits below `n` of a word.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }

// Which columns of a tile of keys from j0 a row at position p sees: [lo, hi], and those below
// `sink` that are at most hi; 32 columns from c0 as the bits of a word.  (Compared one by one
// they become branches: 2700 cycles for 32 columns, a word and its bits' tests 70.)
struct RowMask {
  int lo, hi, sink;
  __device__ __forceinline__ RowMask(const AttnArgs& a, int p, int j0, int len) {
    lo = p - a.window + 1 - j0;
    hi = min(p, len - 1) - j0;
    sink = a.n_sink - j0;
  }
  __device__ __forceinline__ uint32_t word(int c0) const {
    return bits_below(hi + 1 - c0) & (~bits_below(lo - c0) | bits_below(sink - c0));
  }
};

// Operands in shared memory: a descriptor at the tile's start, plus a constant per k-step of
// 16.  One thread issues every MMA, so what it computes for each is on the critical path.
//   K-major: ROWS rows in blocks of 64 columns;  MN-major: the ROWS rows are the k axis
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t base) { return desc_sw128(base, 0, 1024); }
template <int ROWS> __host__ __device__ constexpr uint32_t step_kmajor(int k) {
  return ((k >> 2) * (ROWS * 128) + (k & 3) * 32) >> 4;
}
template <int ROWS> __device__ __forceinline__ uint64_t desc_mnmajor(uint32_t base) {
  return desc_sw128(base, ROWS * 128, 1024);
}
__host__ __device__ constexpr uint32_t step_mnmajor(int k) { return (k * 2048) >> 4; }

// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <uint32_t REGS> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <uint32_t REGS> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// ------------------------------------------------------------------ host side

// Enqueues the read and the clearing of this translation unit's status word.
static inline cudaError_t take_status(int* word, cudaStream_t st) {
  static const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
}

// [B, rows, heads, d] bf16 with strides in elements; box of 64 channels x box_rows rows
inline bool make_map(CUtensorMap* m, const void* ptr, int B, int rows, int heads, int d, long long sb,
                     long long st, long long sh, int box_rows = kM) {
  tc::EncodeTiledFn enc = tc::get_encode();
  if (!enc) return false;
  auto bytes = [](int n, long long s) { return static_cast<cuuint64_t>(n > 1 ? 2 * s : 16); };
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)B};
  cuuint64_t strides[3] = {bytes(heads, sh), bytes(rows, st), bytes(B, sb)};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a tensor map takes positive strides below 2^40 bytes
inline bool map_strides_ok(int B, int rows, int heads, long long sb, long long st, long long sh) {
  auto ok = [](int n, long long s) { return n == 1 || (s > 0 && s < (1LL << 39)); };
  return ok(B, sb) && ok(rows, st) && ok(heads, sh);
}

}  // namespace attn
}  // namespace dr
