// linear.cu — host side of the matrix product: which kernels a call takes, and its workspace.
#include "linear_tc.cuh"

namespace dr {

cudaError_t launch_linear_pack(const PackJob& a, const PackJob& b, int dtype, int sms, bool after, cudaStream_t st);
int linear_slope_blocks(int M);
cudaError_t launch_linear_slope(const LinearArgs& a, int dtype, void* dst, int pitch, long long piece, float* part,
                                cudaStream_t st);
cudaError_t launch_linear_pair(int bn, const lin::Operand& A, const lin::Operand& B, const lin::Epilogue& e, bool full,
                               int sms, cudaStream_t st);
cudaError_t launch_linear_few_bf16(int tn, const lin::Operand& M, const lin::Operand& N, const lin::Epilogue& e, bool full,
                                   int split, cudaStream_t st);
cudaError_t launch_linear_few_fp32(int tn, const lin::Operand& M, const lin::Operand& N, const lin::Epilogue& e, bool full,
                                   int split, cudaStream_t st);
bool linear_rows_supported(const LinearArgs& a, int dtype);
cudaError_t launch_linear_rows(const LinearArgs& a, int sms, cudaStream_t st);

namespace {

using lin::Epilogue;
using lin::Operand;
using lin::Place;

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

template <typename... P> bool on32(const P*... p) { return (((reinterpret_cast<uintptr_t>(p) | ...)) & 31) == 0; }

// A matrix as a tensor map has to find it: in place, or as a copy in the workspace (fp32: its
// pieces).
struct Packed {
  bool copy;
  int rows, cols, pitch;
  long long stride, piece;
  size_t bytes;
  Packed(int dtype, int rows_, int cols_, long long s) : rows(rows_), cols(cols_), stride(s) {
    copy = dtype == DR_FP32 || (rows > 1 && (s <= 0 || s % 8 || s >= (1LL << 38)));
    pitch = (cols + 7) / 8 * 8;
    piece = dtype == DR_FP32 ? (long long)rows * pitch : 0;
    bytes = copy ? round256((size_t)rows * pitch * (dtype == DR_FP32 ? 6 : 2)) : 0;
  }
  PackJob job(const void*& p, void* to) {   // p: where it is to be found from then on
    const PackJob j{p, to, stride, piece, rows, cols, pitch};
    p = to, stride = pitch;
    return j;
  }
  // k along the columns, or along the rows
  Operand k_cols(const void* p) const { return {p, rows, cols, stride, false, piece}; }
  Operand k_rows(const void* p) const { return {p, cols, rows, stride, true, piece}; }
};

Packed pack_x(const LinearArgs& a, int dtype) { return {dtype, a.M, a.K, a.x_s}; }
// The copies that one or both of two matrices need.
cudaError_t make(Packed* a, const void** pa, void* to_a, Packed* b, const void** pb, void* to_b, int dtype, int sms,
                 Place& place, cudaStream_t st) {
  PackJob j[2]{};
  int n = 0;
  if (a && a->copy) j[n++] = a->job(*pa, to_a);
  if (b && b->copy) j[n++] = b->job(*pb, to_b);
  if (!n) return cudaSuccess;
  const bool after = place != lin::kFirst;
  place = lin::kAfter;
  return launch_linear_pack(j[0], j[1], dtype, sms, after, st);
}

Packed pack_w(const LinearArgs& a, int dtype) { return {dtype, a.w_t ? a.N : a.K, a.w_t ? a.K : a.N, a.w_s}; }

// Cycles of one 64-k step of a tile of m x n in an SM that holds `rows` rows of operands for it:
// its products, or what shared memory takes in (128 bytes a row at 64 a cycle from L2, and as
// it writes 128 a cycle) and gives to the tensor cores.  fp32 takes six products of three
// pieces.
long long step_cycles(bool fp32, int m, int n, int rows) {
  const long long mma = (long long)m * n / 64;
  return fp32 ? (6 * mma > 9LL * rows ? 6 * mma : 9LL * rows) : mma > 2LL * rows ? mma : 2LL * rows;
}

// C[m,n] = sum over k of A[m,k] B[n,k], and its epilogue where `full`.
// Which kernel: the one whose busiest SM needs the fewest cycles for its tiles, or for the
// operands out of memory (3500 bytes a cycle; a quarter of the shorter of the two does not
// overlap), and for what a kernel costs besides: start, first loads and the last epilogue.
// Clusters of several CTAs leave SMs unused (a GPC's number of SMs is no multiple of theirs; eight
// of 200 KB hardly find their place), and a second wave of the small kernel waits for the first.
// Both sides, bf16, us with 4 us of events: M512 K4096 N4096 pairs of 256 x 128 23.5, of 256 x 256
// 30.7, small 26.6; M128 22.5, 30, and small, 128 rows cut in four, 16.4; M64 N16384 36.8, 34.1,
// small, 64 rows, 28.7, cut in two 34.8.
// Its constants are fitted, so it misses here and there.  With every offer timed, in graphs of 24
// calls, at 85 sizes (M 1 to 1024, K512 N512 to K4096 N16384 and K8192 N2048; fp32 M 16 to 1024),
// the choice is within 10 % of the best at 76; elsewhere it mostly cuts K too often: bf16 M64 K512
// N1536 32 rows cut in four 6.2 us, 16 in two 4.9; M512 K512 N512 64 in four 6.7, 32 in two 5.4;
// M512 K2048 N2048 256 in four 12.3, pairs of 256 x 128 9.9; fp32 M300 K512 N1536 13.6, 64 in two
// 10.9.
cudaError_t product(const Operand& A, const Operand& B, Epilogue e, bool full, int dtype, int sms, cudaStream_t st) {
  const bool fp32 = dtype == DR_FP32;
  const int es = fp32 ? 4 : 2;
  const long long n_k = ceil_div(A.k, lin::kBK);
  const long long memory = ((long long)A.rows + B.rows) * A.k * (fp32 ? 6 : 2) / 3500;
  long long best = 0;
  int bn = 0, tn = 0, split = 1;
  auto offer = [&](long long work, long long fixed, int bn_, int tn_, int split_) {
    const long long cost = (work > memory ? work + memory / 4 : memory + work / 4) + fixed;
    if (!best || cost < best) best = cost, bn = bn_, tn = tn_, split = split_;
  };
  for (int b = fp32 ? 128 : 256; b >= 128; b /= 2)
    offer(ceil_div(ceil_div(A.rows, 256) * ceil_div(B.rows, b), sms / 2) * n_k * step_cycles(fp32, 128, b, 128 + b / 2),
          b == 256 ? 17000 : 11500, b, 0, 1);
  const long long n_tiles = ceil_div(B.rows, 128);
  for (int t : {16, 32, 64, 96, 128, 160, 192, 256}) {
    if ((A.mn && t % 64) || (fp32 && t > 192)) continue;
    const long long tiles = n_tiles * ceil_div(A.rows, t);
    if (tiles > 4LL * sms) continue;
    for (int s = 1; s <= 6 && s <= n_k; ++s) {
      const long long waves = ceil_div(tiles * s, s > 1 ? sms * 27 / 32 : sms);
      offer(waves * ceil_div(n_k, s) * step_cycles(fp32, 128, t, 128 + t), 10500 + 12 * t + (waves - 1) * 14000, 0, t, s);
    }
  }
  if (tn) return (fp32 ? launch_linear_few_fp32 : launch_linear_few_bf16)(tn, A, B, e, full, split, st);
  e.vec = e.N % 16 == 0 && on32(e.C, e.res) && on32(e.slope) && (!e.res || e.r_m * es % 32 == 0);
  return launch_linear_pair(bn, A, B, e, full, sms, st);
}

struct BwdPlan {
  Packed x, w;
  bool keep_d;
  int pitch;                           // of d
  long long piece;
  size_t o_x, o_w, o_d, o_part, bytes;
  BwdPlan(const LinearArgs& a, int dtype, bool act) : x(pack_x(a, dtype)), w(pack_w(a, dtype)) {
    const bool fp32 = dtype == DR_FP32;
    pitch = (a.N + 7) / 8 * 8;
    keep_d = act || fp32 || (a.N % 8 != 0 && a.M > 1);
    piece = fp32 ? (long long)a.M * pitch : 0;
    o_x = 0, o_w = x.bytes, o_d = o_w + w.bytes;
    o_part = o_d + (keep_d ? round256((size_t)a.M * pitch * (fp32 ? 6 : 2)) : 0);
    bytes = o_part + round256((size_t)linear_slope_blocks(a.M) * a.N * 4);
  }
};

}  // namespace

size_t linear_fwd_workspace(const LinearArgs& a, int dtype) {
  return linear_rows_supported(a, dtype) ? 0 : pack_x(a, dtype).bytes + pack_w(a, dtype).bytes;
}

cudaError_t launch_linear_fwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st) {
  if (linear_rows_supported(a, dtype)) return launch_linear_rows(a, sms, st);
  char* ws = static_cast<char*>(workspace);
  Packed px = pack_x(a, dtype), pw = pack_w(a, dtype);
  const void *x = a.x, *w = a.w;
  Place place = lin::kFirst;
  cudaError_t e = make(&px, &x, ws, &pw, &w, ws + px.bytes, dtype, sms, place, st);
  if (e != cudaSuccess) return e;
  return product(px.k_cols(x), a.w_t ? pw.k_cols(w) : pw.k_rows(w),
                 Epilogue{a.y, a.bias, a.res, a.slope, a.M, a.N, a.act, place, a.r_s}, true, dtype, sms, st);
}

size_t linear_bwd_workspace(const LinearArgs& a, int dtype, bool act) { return BwdPlan(a, dtype, act).bytes; }

cudaError_t launch_linear_bwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st) {
  BwdPlan p(a, dtype, a.slope != nullptr);
  char* ws = static_cast<char*>(workspace);
  const bool keep = p.keep_d && (a.dx || a.dw);
  cudaError_t e = cudaSuccess;
  Place place = lin::kFirst;
  if (keep || a.db)
    place = lin::kAfter, e = launch_linear_slope(a, dtype, keep ? ws + p.o_d : nullptr, p.pitch, p.piece,
                            a.db ? reinterpret_cast<float*>(ws + p.o_part) : nullptr, st);
  const void* d = keep ? ws + p.o_d : a.d_y;
  const Operand rows{d, a.M, a.N, keep ? p.pitch : a.N, false, p.piece};   // k along the channels out
  const Operand cols{d, a.N, a.M, keep ? p.pitch : a.N, true, p.piece};    // k along the tokens
  const void *x = a.x, *w = a.w;
  if (e == cudaSuccess)
    e = make(a.dw ? &p.x : nullptr, &x, ws + p.o_x, a.dx ? &p.w : nullptr, &w, ws + p.o_w, dtype, sms, place, st);
  if (a.dx && e == cudaSuccess)   // dx[m,k] = sum over n of d[m,n] W[k,n]
    e = product(rows, a.w_t ? p.w.k_rows(w) : p.w.k_cols(w), Epilogue{a.dx, nullptr, nullptr, nullptr, a.M, a.K, 0, place}, false,
                dtype, sms, st);
  if (a.dw && e == cudaSuccess)   // dw[k,n] = sum over m of x[m,k] d[m,n], in W's order
    e = product(a.w_t ? cols : p.x.k_rows(x), a.w_t ? p.x.k_rows(x) : cols,
                Epilogue{a.dw, nullptr, nullptr, nullptr, a.w_t ? a.N : a.K, a.w_t ? a.K : a.N, 0, a.dx ? lin::kBeside : place},
                false, dtype, sms, st);
  return e;
}

}  // namespace dr
