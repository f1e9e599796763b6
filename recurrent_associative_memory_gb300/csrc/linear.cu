// linear.cu — host side of the matrix product: which kernels a call takes, and its workspace.
#include "linear_tc.cuh"

namespace dr {

cudaError_t launch_linear_fwd_simt(const LinearArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_linear_bwd_simt(const LinearArgs& a, const void* d, int dtype, cudaStream_t st);
int linear_slope_blocks(int M);
cudaError_t launch_linear_slope(const LinearArgs& a, int dtype, void* d, float* part, cudaStream_t st);
cudaError_t launch_linear_pair(const lin::Operand& A, const lin::Operand& B, const lin::Epilogue& e, bool full, int sms,
                               cudaStream_t st);

namespace {

using lin::Epilogue;
using lin::Operand;

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

template <typename... P> bool on32(const P*... p) { return (((reinterpret_cast<uintptr_t>(p) | ...)) & 31) == 0; }

// x and W of a product y = x W
Operand rows_of(const void* p, int rows, int k, long long s) { return {p, rows, k, s, false}; }
Operand weight_of(const LinearArgs& a) { return {a.w, a.N, a.K, a.w_s, !a.w_t}; }

struct BwdPlan {
  size_t d, part, bytes;   // offsets: d_y * slope, the bias's parts
};

BwdPlan bwd_plan(const LinearArgs& a, int dtype, bool act) {
  BwdPlan p{};
  p.d = 0;
  p.part = act ? round256((size_t)a.M * a.N * (dtype == DR_FP32 ? 4 : 2)) : 0;
  p.bytes = p.part + round256((size_t)linear_slope_blocks(a.M) * a.N * 4);
  return p;
}

}  // namespace

size_t linear_fwd_workspace(const LinearArgs& a, int dtype) { return 0; }

cudaError_t launch_linear_fwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st) {
  const Operand x = rows_of(a.x, a.M, a.K, a.x_s), w = weight_of(a);
  if (dtype == DR_BF16 && operand_ok(x) && operand_ok(w)) {
    Epilogue e{a.y, a.bias, a.res, a.slope, a.M, a.N, a.act, a.r_s, 0};
    e.vec = a.N % 16 == 0 && on32(a.y, a.slope, a.res) && (!a.res || a.r_s % 16 == 0);
    return launch_linear_pair(x, w, e, true, sms, st);
  }
  return launch_linear_fwd_simt(a, dtype, st);
}

size_t linear_bwd_workspace(const LinearArgs& a, int dtype, bool act) { return bwd_plan(a, dtype, act).bytes; }

cudaError_t launch_linear_bwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st) {
  const BwdPlan p = bwd_plan(a, dtype, a.slope != nullptr);
  char* ws = static_cast<char*>(workspace);
  const void* d = a.d_y;
  cudaError_t e = cudaSuccess;
  if (a.slope || a.db) {
    e = launch_linear_slope(a, dtype, a.slope ? ws + p.d : nullptr, a.db ? reinterpret_cast<float*>(ws + p.part) : nullptr, st);
    if (e != cudaSuccess) return e;
    if (a.slope) d = ws + p.d;
  }
  const bool tc = dtype == DR_BF16 && operand_ok(rows_of(a.x, a.M, a.K, a.x_s)) && operand_ok(weight_of(a)) && a.N % 8 == 0;
  if (!tc) return launch_linear_bwd_simt(a, d, dtype, st);
  if (a.dx) {   // dx[m,k] = sum over n of d[m,n] W[k,n]
    const Operand W{a.w, a.K, a.N, a.w_s, a.w_t != 0};
    e = launch_linear_pair(rows_of(d, a.M, a.N, a.N), W, Epilogue{a.dx, nullptr, nullptr, nullptr, a.M, a.K, 0, 0,
                           a.K % 16 == 0 && on32(a.dx)}, false, sms, st);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {   // dw[k,n] = sum over m of x[m,k] d[m,n]
    const Operand X{a.x, a.K, a.M, a.x_s, true}, D{d, a.N, a.M, a.N, true};
    const int rows = a.w_t ? a.N : a.K, cols = a.w_t ? a.K : a.N;
    e = launch_linear_pair(a.w_t ? D : X, a.w_t ? X : D, Epilogue{a.dw, nullptr, nullptr, nullptr, rows, cols, 0, 0,
                           cols % 16 == 0 && on32(a.dw)}, false, sms, st);
  }
  return e;
}

}  // namespace dr
