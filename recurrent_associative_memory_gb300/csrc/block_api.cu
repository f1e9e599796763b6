// block_api.cu — the extern "C" entry points of what stands around a mixer: argument
// checks, path selection and launches.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "block.cuh"

namespace dr {

size_t linear_fwd_workspace(const LinearArgs& a, int dtype);
cudaError_t launch_linear_fwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st);
size_t linear_bwd_workspace(const LinearArgs& a, int dtype, bool act);
cudaError_t launch_linear_bwd(const LinearArgs& a, int dtype, int sms, void* workspace, cudaStream_t st);
int block_norm_bwd_blocks(const BlockNormArgs& a, int sms);
cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, cudaStream_t st);
cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, int dtype, int h_dtype, int sms, float* d_scale, float* d_post,
                                  float* d_pre, cudaStream_t st);

namespace {

constexpr long long kMaxElements = 1LL << 40;   // of one tensor
constexpr int kMaxChannels = 1 << 24;           // of a matrix product
constexpr int kMaxRows = INT_MAX - 511;         // and its rows: the last tile, of 256 at most, counts in an int too
constexpr int kMaxRow = 8192;                   // channels of a norm
constexpr long long kMaxBlocks = 0x7fffffffLL;  // of one launch

template <typename... P> bool aligned(unsigned n, const P*... p) {
  return (((reinterpret_cast<uintptr_t>(p) | ...)) & (n - 1)) == 0;
}
unsigned bytes_of(int dtype) { return dtype == DR_FP32 ? 4 : 2; }
bool dtype_ok(int t) { return t == DR_FP32 || t == DR_BF16; }
bool act_ok(int t) { return t >= DR_ACT_NONE && t <= DR_ACT_SIGMOID; }
// is p one of the others?
template <typename... P> bool among(const void* p, const P*... q) { return p && ((p == static_cast<const void*>(q)) || ...); }
cudaStream_t stream_of(dr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
int status_of(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

int check_linear(const dr_linear* a) {
  if (!dtype_ok(a->dtype)) return DR_ERR_DTYPE;
  if (!act_ok(a->act)) return DR_ERR_ARG;
  if (a->M < 1 || a->K < 1 || a->N < 1 || a->M > kMaxRows || a->K > kMaxChannels || a->N > kMaxChannels) return DR_ERR_SHAPE;
  if (a->M >= kMaxElements / a->K || a->M >= kMaxElements / a->N || (long long)a->K * a->N >= kMaxElements) return DR_ERR_SHAPE;
  // blocks of the launches: tiles of 64 by 64
  const long long m = (a->M + 63LL) / 64, k = (a->K + 63LL) / 64, n = (a->N + 63LL) / 64;
  if (m * n > kMaxBlocks || m * k > kMaxBlocks || k * n > kMaxBlocks) return DR_ERR_SHAPE;
  return DR_OK;
}

LinearArgs linear_args(const dr_linear* a) {
  LinearArgs r{};
  r.M = a->M, r.K = a->K, r.N = a->N, r.act = a->act, r.w_t = a->w_transposed ? 1 : 0;
  r.x_s = a->x_s, r.w_s = a->w_s, r.r_s = a->r_s;
  return r;
}

int check_block_norm(const dr_block_norm* a) {
  if (!dtype_ok(a->dtype) || !dtype_ok(a->h_dtype) || (a->dtype == DR_FP32 && a->h_dtype == DR_BF16)) return DR_ERR_DTYPE;
  if (!act_ok(a->gate_act) || !isfinite(a->eps) || a->eps < 0.f) return DR_ERR_ARG;
  if (a->M < 1 || a->D < 1 || a->D > kMaxRow || a->M >= kMaxElements / a->D) return DR_ERR_SHAPE;
  return DR_OK;
}

// No gradient in the buffer of another one or of an input.  A row's dh may go over its d_h or h,
// its dbranch over its branch and its dgate over its gate: whoever stores a value has read what
// stood there, and nobody else reads it.
bool norm_grads_apart(const dr_block_norm* a, const void* h, const void* branch, const void* gate, const float* scale,
                      const float* post_weight, const float* pre_weight, const void* d_h, const void* d_y,
                      const dr_block_norm_grads* g) {
  auto rows = [&](const void* grad, const void* of, long long stride) {   // of's rows where they are not grad's
    return grad && grad == of && a->M > 1 && stride != a->D;
  };
  if (rows(g->dh, h, a->h_s) || rows(g->dbranch, branch, a->b_s) || rows(g->dgate, gate, a->g_s)) return false;
  const void* const grads[] = {g->dh, g->dbranch, g->dgate, g->dscale, g->dpost_weight, g->dpre_weight};
  for (int i = 0; i < 6; ++i) {
    const void* p = grads[i];
    for (int j = i + 1; j < 6; ++j)
      if (p && p == grads[j]) return false;
    if (among(p, scale, post_weight, pre_weight, d_y)) return false;
    if ((i != 0 && among(p, h, d_h)) || (i != 1 && among(p, branch)) || (i != 2 && among(p, gate))) return false;
  }
  return true;
}

BlockNormArgs block_norm_args(const dr_block_norm* a) {
  BlockNormArgs r{};
  r.M = a->M, r.D = a->D, r.gate_act = a->gate_act, r.post_norm = a->post_norm ? 1 : 0;
  r.eps = a->eps, r.inv_d = 1.f / static_cast<float>(a->D);
  r.h_s = a->h_s, r.b_s = a->b_s, r.g_s = a->g_s;
  return r;
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" {

size_t dr_linear_fwd_workspace_bytes(const dr_linear* a) {
  if (!a || check_linear(a) != DR_OK) return 0;
  return linear_fwd_workspace(linear_args(a), a->dtype);
}

int dr_linear_fwd(const dr_linear* a, const void* x, const void* weight, const void* bias, const void* residual, void* y,
                  void* slope, void* workspace, size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !x || !weight || !y) return DR_ERR_NULL;
  int st = check_linear(a);
  if (st != DR_OK) return st;
  if (!aligned(16, x, weight, residual, y, slope) || !aligned(bytes_of(a->dtype), bias)) return DR_ERR_ALIGN;
  const size_t need = dr_linear_fwd_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need)) return DR_ERR_WORKSPACE;
  if (!aligned(256, workspace)) return DR_ERR_ALIGN;
  // a tile's rows are read by other tiles too; a residual's value only where it is added
  if (among(y, x, weight, bias) || among(slope, x, weight, bias, residual, y) ||
      (y == residual && a->M > 1 && a->r_s != a->N))
    return DR_ERR_ARG;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  LinearArgs r = linear_args(a);
  r.x = x, r.w = weight, r.bias = bias, r.res = residual, r.y = y, r.slope = slope;
  return status_of(launch_linear_fwd(r, a->dtype, sms, workspace, stream_of(stream)));
}

size_t dr_linear_bwd_workspace_bytes(const dr_linear* a) {
  if (!a || check_linear(a) != DR_OK) return 0;
  return linear_bwd_workspace(linear_args(a), a->dtype, a->act != DR_ACT_NONE);
}

int dr_linear_bwd(const dr_linear* a, const void* x, const void* weight, const void* d_y, const void* slope, void* dx,
                  void* d_weight, void* d_bias, void* workspace, size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !d_y || (!dx && !d_weight && !d_bias) || (dx && !weight) || (d_weight && !x)) return DR_ERR_NULL;
  if (a->act != DR_ACT_NONE && !slope) return DR_ERR_NULL;
  int st = check_linear(a);
  if (st != DR_OK) return st;
  if (!aligned(16, x, weight, d_y, slope, dx, d_weight) || !aligned(bytes_of(a->dtype), d_bias)) return DR_ERR_ALIGN;
  const size_t need = dr_linear_bwd_workspace_bytes(a);
  if (need && (!workspace || workspace_bytes < need)) return DR_ERR_WORKSPACE;
  if (!aligned(256, workspace)) return DR_ERR_ALIGN;
  if (among(dx, x, weight, d_y, slope, d_weight, d_bias) || among(d_weight, x, weight, d_y, slope, d_bias) ||
      among(d_bias, x, weight, d_y, slope))
    return DR_ERR_ARG;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  LinearArgs r = linear_args(a);
  r.x = x, r.w = weight, r.d_y = d_y, r.slope = a->act != DR_ACT_NONE ? const_cast<void*>(slope) : nullptr;
  r.dx = dx, r.dw = d_weight, r.db = d_bias;
  return status_of(launch_linear_bwd(r, a->dtype, sms, workspace, stream_of(stream)));
}

int dr_block_norm_fwd(const dr_block_norm* a, const void* h, const void* branch, const void* gate, const float* scale,
                      const float* post_weight, const float* pre_weight, void* h_out, void* y, dr_stream_t stream) {
  if (!a || !h || (!h_out && !y) || (branch && !h_out)) return DR_ERR_NULL;
  int st = check_block_norm(a);
  if (st != DR_OK) return st;
  if (!branch && (gate || scale || h_out || a->post_norm)) return DR_ERR_ARG;
  if ((post_weight && !a->post_norm) || (pre_weight && !y)) return DR_ERR_ARG;
  if (among(y, h, branch, gate, scale, post_weight, pre_weight, h_out) ||
      among(h_out, branch, gate, scale, post_weight, pre_weight) || (h_out == h && a->M > 1 && a->h_s != a->D))
    return DR_ERR_ARG;
  if (!aligned(bytes_of(a->dtype), branch, gate, y) || !aligned(bytes_of(a->h_dtype), h, h_out) ||
      !aligned(4, scale, post_weight, pre_weight))
    return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  BlockNormArgs r = block_norm_args(a);
  r.h = h, r.branch = branch, r.gate = gate, r.scale = scale, r.post_w = post_weight, r.pre_w = pre_weight;
  r.h_out = h_out, r.y = y;
  return status_of(launch_block_norm_fwd(r, a->dtype, a->h_dtype, sms, stream_of(stream)));
}

size_t dr_block_norm_bwd_workspace_bytes(const dr_block_norm* a) {
  if (!a || check_block_norm(a) != DR_OK) return 0;
  return (static_cast<size_t>(block_norm_bwd_blocks(block_norm_args(a), sm_count())) * 2 * a->D * 4 + 255) & ~size_t(255);
}

int dr_block_norm_bwd(const dr_block_norm* a, const void* h, const void* branch, const void* gate, const float* scale,
                      const float* post_weight, const float* pre_weight, const void* d_h, const void* d_y,
                      const dr_block_norm_grads* g, void* workspace, size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !g || !h || (!d_h && !d_y)) return DR_ERR_NULL;
  int st = check_block_norm(a);
  if (st != DR_OK) return st;
  if (!branch && (gate || scale || a->post_norm || g->dbranch)) return DR_ERR_ARG;
  if ((post_weight && !a->post_norm) || (g->dgate && !gate) || (g->dscale && !scale) || (g->dpost_weight && !post_weight) ||
      (g->dpre_weight && (!pre_weight || !d_y)))
    return DR_ERR_ARG;
  if (!aligned(bytes_of(a->dtype), branch, gate, d_y, g->dbranch, g->dgate) || !aligned(bytes_of(a->h_dtype), h, d_h, g->dh) ||
      !aligned(4, scale, post_weight, pre_weight, g->dscale, g->dpost_weight, g->dpre_weight))
    return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  if (!norm_grads_apart(a, h, branch, gate, scale, post_weight, pre_weight, d_h, d_y, g)) return DR_ERR_ARG;
  BlockNormArgs r = block_norm_args(a);
  if (g->dscale || g->dpost_weight || g->dpre_weight) {
    if (!workspace || workspace_bytes < dr_block_norm_bwd_workspace_bytes(a)) return DR_ERR_WORKSPACE;
    if (!aligned(256, workspace)) return DR_ERR_ALIGN;
    r.part = static_cast<float*>(workspace);
  }
  r.h = h, r.branch = branch, r.gate = gate, r.scale = scale, r.post_w = post_weight, r.pre_w = pre_weight;
  r.d_h = d_h, r.d_y = d_y, r.dh = g->dh, r.db = g->dbranch, r.dg = g->dgate;
  return status_of(launch_block_norm_bwd(r, a->dtype, a->h_dtype, sms, g->dscale, g->dpost_weight, g->dpre_weight,
                                         stream_of(stream)));
}

}  // extern "C"
