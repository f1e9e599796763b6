// layers_api.cu — the extern "C" entry points of the layers next to the recurrence:
// argument checks, path selection and launches.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "layers.cuh"

namespace dr {

cudaError_t launch_attn_fwd_simt(const AttnArgs& a, int dtype, int sms, cudaStream_t st);
cudaError_t launch_attn_bwd_simt(const AttnArgs& a, int dtype, cudaStream_t st);
bool attn_tc_supported(const AttnArgs& a, int dtype);
cudaError_t launch_attn_fwd_tc(const AttnArgs& a, int sms, cudaStream_t st);
size_t attn_bwd_tc_workspace(const AttnArgs& a);
cudaError_t launch_attn_bwd_tc(AttnArgs a, int sms, void* workspace, cudaStream_t st);
int attn_step_pieces(const AttnStepArgs& a, int dtype, int sms);
cudaError_t launch_attn_step(const AttnStepArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_cache_fill(const AttnArgs& a, int dtype, void* kc, void* vc, cudaStream_t st);
cudaError_t launch_conv_fwd(const ConvArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvArgs& a, int dtype, float* dw, float* db, cudaStream_t st);
cudaError_t launch_conv_step(const ConvArgs& a, int dtype, cudaStream_t st);
size_t conv_bwd_part_floats(const ConvArgs& a);
size_t scan_fwd_workspace(const ScanArgs& a, int sms);
cudaError_t launch_scan_fwd(ScanArgs a, int dtype, int sms, void* workspace, cudaStream_t st);
size_t scan_bwd_workspace(const ScanArgs& a);
cudaError_t launch_scan_bwd(ScanArgs a, int dtype, int sms, void* workspace, cudaStream_t st);
cudaError_t launch_scan_step(const ScanArgs& a, int dtype, cudaStream_t st);

namespace {

constexpr long long kMaxElements = 1LL << 40;   // of one tensor
constexpr int kMaxPositions = 1 << 30;          // position + window stays an int
constexpr long long kMaxBlocks = 0x7fffffffLL;  // of one launch

template <typename... P> bool aligned16(const P*... p) {
  return (((reinterpret_cast<uintptr_t>(p) | ...)) & 15u) == 0;
}
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool dtype_ok(int t) { return t == DR_FP32 || t == DR_BF16; }
// values in 16 bytes
int vec_of(int dtype) { return dtype == DR_FP32 ? 4 : 8; }
cudaStream_t stream_of(dr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
int status_of(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }

// SMs of the current device; 0 where there is none, and no launch is cut for it
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// What every window-attention call shares; T, S and the strides are checked apart.
int check_heads(const dr_attn* a) {
  if (!dtype_ok(a->dtype)) return DR_ERR_DTYPE;
  if (a->B < 1 || a->H < 1 || a->Hkv < 1 || a->H % a->Hkv || (a->d != 64 && a->d != 128)) return DR_ERR_SHAPE;
  if (a->window < 1 || a->n_sink < 0 || a->n_sink > 128) return DR_ERR_ARG;
  if (!isfinite(a->scale) || a->scale < 0.f) return DR_ERR_ARG;
  return DR_OK;
}

bool strides_ok(const dr_attn* a, bool with_q) {
  const int v = vec_of(a->dtype);
  const long long s[] = {a->k_sb, a->k_st, a->k_sh, a->v_sb, a->v_st, a->v_sh, a->q_sb, a->q_st, a->q_sh};
  for (int i = 0; i < (with_q ? 9 : 6); ++i)
    if (s[i] % v) return false;
  return true;
}

int check_attn(const dr_attn* a) {
  int st = check_heads(a);
  if (st != DR_OK) return st;
  if (a->T < 1 || a->S < 1 || a->S > kMaxPositions) return DR_ERR_SHAPE;
  if (a->q_start < 0 || (long long)a->q_start + a->T > kMaxPositions) return DR_ERR_ARG;
  const long long rows = (long long)a->B * a->T * a->H, keys = (long long)a->B * a->S * a->Hkv;
  if (rows >= kMaxElements / a->d || keys >= kMaxElements / a->d) return DR_ERR_SHAPE;
  // blocks of the launches: a query tile of 64 rows, a warp per row, a tile of 64 keys
  if ((long long)a->B * a->H * ((a->T + 63LL) / 64) > kMaxBlocks || rows / 8 >= kMaxBlocks ||
      (long long)a->B * a->Hkv * ((a->S + 63LL) / 64) > kMaxBlocks)
    return DR_ERR_SHAPE;
  return DR_OK;
}

AttnArgs attn_args(const dr_attn* a) {
  AttnArgs r{};
  r.lens = a->lens;
  r.B = a->B, r.T = a->T, r.S = a->S, r.H = a->H, r.Hkv = a->Hkv, r.d = a->d, r.G = a->H / a->Hkv;
  r.n_sink = a->n_sink, r.q_start = a->q_start;
  // positions reach q_start + T - 1: a wider window sees the same keys
  r.window = a->window < a->q_start + a->T ? a->window : a->q_start + a->T;
  // and keys from there on are nobody's: whatever they hold, no kernel multiplies by it
  r.reach = a->S < a->q_start + a->T ? a->S : a->q_start + a->T;
  r.scale = a->scale > 0.f ? a->scale : 1.f / sqrtf(static_cast<float>(a->d));
  r.q_sb = a->q_sb, r.q_st = a->q_st, r.q_sh = a->q_sh;
  r.k_sb = a->k_sb, r.k_st = a->k_st, r.k_sh = a->k_sh;
  r.v_sb = a->v_sb, r.v_st = a->v_st, r.v_sh = a->v_sh;
  return r;
}

size_t attn_bwd_workspace(const dr_attn* a) {
  const AttnArgs r = attn_args(a);
  if (attn_tc_supported(r, a->dtype)) return attn_bwd_tc_workspace(r);
  return (static_cast<size_t>(a->B) * a->H * a->T * 4 + 255) & ~size_t(255);
}

int check_step(const dr_attn* a, AttnStepArgs* s) {
  int st = check_heads(a);
  if (st != DR_OK) return st;
  const long long C = (long long)a->n_sink + a->window;
  if (C > INT_MAX || (long long)a->B * a->Hkv >= kMaxElements / C / a->d ||
      (long long)a->B * a->H > kMaxBlocks / 4)
    return DR_ERR_SHAPE;
  s->B = a->B, s->H = a->H, s->Hkv = a->Hkv, s->G = a->H / a->Hkv, s->d = a->d;
  s->window = a->window, s->n_sink = a->n_sink, s->n_piece = 1;
  s->scale = a->scale > 0.f ? a->scale : 1.f / sqrtf(static_cast<float>(a->d));
  return DR_OK;
}

size_t step_workspace(const AttnStepArgs& s, int pieces) {
  return pieces > 1 ? static_cast<size_t>(s.B) * s.H * pieces * (s.d + 2) * 4 : 0;
}

int check_conv(const dr_conv* a) {
  if (!dtype_ok(a->dtype)) return DR_ERR_DTYPE;
  if (a->B < 1 || a->T < 1 || a->D < 1 || a->K < 2 || a->K > 4) return DR_ERR_SHAPE;
  if ((long long)a->B * a->T >= kMaxElements / a->D || a->D > INT_MAX / 8) return DR_ERR_SHAPE;
  return DR_OK;
}

ConvArgs conv_args(const dr_conv* a, const void* x, const float* w, const float* bias, const void* s0) {
  ConvArgs r{};
  r.x = x, r.w = w, r.bias = bias, r.s0 = s0, r.lens = a->lens;
  r.B = a->B, r.T = a->T, r.D = a->D, r.K = a->K, r.silu = a->silu ? 1 : 0;
  r.x_sb = a->x_sb, r.x_st = a->x_st;
  return r;
}

int check_scan(const dr_scan* a) {
  if (!dtype_ok(a->dtype)) return DR_ERR_DTYPE;
  if (a->B < 1 || a->T < 1 || a->D < 1 || a->G < 1 || a->D % a->G) return DR_ERR_SHAPE;
  if (a->N != 8 && a->N != 16 && a->N != 32 && a->N != 64) return DR_ERR_SHAPE;
  if ((long long)a->B * a->T >= kMaxElements / 2 / a->D / a->N || a->D > INT_MAX / 64) return DR_ERR_SHAPE;
  if (!a->A) return DR_ERR_NULL;
  if (!aligned16(a->A)) return DR_ERR_ALIGN;
  return DR_OK;
}

ScanArgs scan_args(const dr_scan* a, const void* x, const void* dt, const void* Bm, const void* Cm,
                   const void* z, const float* h0) {
  ScanArgs r{};
  r.x = x, r.dt = dt, r.Bm = Bm, r.Cm = Cm, r.z = z, r.h0 = h0;
  r.lens = a->lens, r.A = a->A, r.Dskip = a->Dskip, r.bias = a->dt_bias;
  r.B = a->B, r.T = a->T, r.D = a->D, r.N = a->N, r.G = a->G, r.softplus = a->softplus ? 1 : 0;
  r.x_sb = a->x_sb, r.x_st = a->x_st, r.dt_sb = a->dt_sb, r.dt_st = a->dt_st;
  r.z_sb = a->z_sb, r.z_st = a->z_st, r.B_sb = a->B_sb, r.B_st = a->B_st, r.C_sb = a->C_sb, r.C_st = a->C_st;
  return r;
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" {

void dr_attn_init(dr_attn* a) {
  if (!a) return;
  *a = dr_attn{};
  a->dtype = DR_BF16;
  a->window = INT_MAX;
}

int dr_window_attn_fwd(const dr_attn* a, const void* q, const void* k, const void* v, void* out, float* lse,
                       dr_stream_t stream) {
  if (!a || !q || !k || !v || !out) return DR_ERR_NULL;
  int st = check_attn(a);
  if (st != DR_OK) return st;
  if (!aligned16(q, k, v, out) || !strides_ok(a, true)) return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  AttnArgs r = attn_args(a);
  r.q = q, r.k = k, r.v = v, r.out = out, r.lse = lse;
  if (attn_tc_supported(r, a->dtype)) return status_of(launch_attn_fwd_tc(r, sms, stream_of(stream)));
  return status_of(launch_attn_fwd_simt(r, a->dtype, sms, stream_of(stream)));
}

size_t dr_window_attn_bwd_workspace_bytes(const dr_attn* a) {
  if (!a || check_attn(a) != DR_OK) return 0;
  return attn_bwd_workspace(a);
}

int dr_window_attn_bwd(const dr_attn* a, const void* q, const void* k, const void* v, const void* out,
                       const float* lse, const void* d_out, void* dq, void* dk, void* dv, void* workspace,
                       size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !q || !k || !v || !out || !lse || !d_out || !dq || !dk || !dv) return DR_ERR_NULL;
  int st = check_attn(a);
  if (st != DR_OK) return st;
  if (!aligned16(q, k, v, out, d_out, dq, dk, dv) || !strides_ok(a, true)) return DR_ERR_ALIGN;
  if (!workspace || workspace_bytes < attn_bwd_workspace(a)) return DR_ERR_WORKSPACE;
  if (!aligned256(workspace)) return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  AttnArgs r = attn_args(a);
  r.q = q, r.k = k, r.v = v, r.out = const_cast<void*>(out), r.lse = const_cast<float*>(lse);
  r.d_out = d_out, r.dq = dq, r.dk = dk, r.dv = dv;
  if (attn_tc_supported(r, a->dtype)) return status_of(launch_attn_bwd_tc(r, sms, workspace, stream_of(stream)));
  r.delta = static_cast<float*>(workspace);
  return status_of(launch_attn_bwd_simt(r, a->dtype, stream_of(stream)));
}

size_t dr_window_attn_step_workspace_bytes(const dr_attn* a) {
  AttnStepArgs s{};
  if (!a || check_step(a, &s) != DR_OK) return 0;
  return step_workspace(s, attn_step_pieces(s, a->dtype, sm_count()));
}

int dr_window_attn_step(const dr_attn* a, const void* q, const void* k, const void* v, void* k_cache,
                        void* v_cache, const int* pos, void* out, void* workspace, size_t workspace_bytes,
                        dr_stream_t stream) {
  if (!a || !q || !k || !v || !k_cache || !v_cache || !pos || !out) return DR_ERR_NULL;
  AttnStepArgs s{};
  int st = check_step(a, &s);
  if (st != DR_OK) return st;
  if (!aligned16(q, k, v, k_cache, v_cache, out)) return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  if (workspace) {
    s.n_piece = attn_step_pieces(s, a->dtype, sms);
    if (workspace_bytes < step_workspace(s, s.n_piece)) return DR_ERR_WORKSPACE;
    if (!aligned256(workspace)) return DR_ERR_ALIGN;
  }
  s.q = q, s.k = k, s.v = v, s.kc = k_cache, s.vc = v_cache, s.pos = pos, s.out = out;
  s.part = static_cast<float*>(workspace);
  return status_of(launch_attn_step(s, a->dtype, stream_of(stream)));
}

int dr_window_cache_fill(const dr_attn* a, const void* k, const void* v, void* k_cache, void* v_cache,
                         dr_stream_t stream) {
  if (!a || !k || !v || !k_cache || !v_cache) return DR_ERR_NULL;
  AttnStepArgs s{};
  int st = check_step(a, &s);
  if (st != DR_OK) return st;
  if (a->S < 1 || (long long)a->B * a->S * a->Hkv >= kMaxElements / a->d ||
      (long long)a->B * a->Hkv * ((long long)a->n_sink + a->window) / 32 >= kMaxBlocks / a->d * 8)
    return DR_ERR_SHAPE;
  if (!aligned16(k, v, k_cache, v_cache) || !strides_ok(a, false)) return DR_ERR_ALIGN;
  AttnArgs r = attn_args(a);
  r.k = k, r.v = v, r.window = a->window;
  return status_of(launch_cache_fill(r, a->dtype, k_cache, v_cache, stream_of(stream)));
}

int dr_short_conv_fwd(const dr_conv* a, const void* x, const float* weight, const float* bias,
                      const void* init_state, void* y, void* final_state, dr_stream_t stream) {
  if (!a || !x || !weight || !y) return DR_ERR_NULL;
  int st = check_conv(a);
  if (st != DR_OK) return st;
  ConvArgs r = conv_args(a, x, weight, bias, init_state);
  r.y = y, r.s1 = final_state;
  return status_of(launch_conv_fwd(r, a->dtype, stream_of(stream)));
}

size_t dr_short_conv_bwd_workspace_bytes(const dr_conv* a) {
  if (!a || check_conv(a) != DR_OK) return 0;
  return 4 * conv_bwd_part_floats(conv_args(a, nullptr, nullptr, nullptr, nullptr));
}

int dr_short_conv_bwd(const dr_conv* a, const void* x, const float* weight, const float* bias,
                      const void* init_state, const void* d_y, const void* d_final_state, void* dx,
                      float* d_weight, float* d_bias, void* d_init_state, void* workspace,
                      size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !x || !weight || !d_y || !dx || !d_weight) return DR_ERR_NULL;
  int st = check_conv(a);
  if (st != DR_OK) return st;
  // the first tokens' threads write the one, the last tokens' read the other
  if (d_init_state && d_init_state == d_final_state) return DR_ERR_ARG;
  ConvArgs r = conv_args(a, x, weight, bias, init_state);
  if (!workspace || workspace_bytes < 4 * conv_bwd_part_floats(r)) return DR_ERR_WORKSPACE;
  if (!aligned256(workspace)) return DR_ERR_ALIGN;
  r.d_y = d_y, r.d_s1 = d_final_state, r.dx = dx, r.d_s0 = d_init_state;
  r.part = static_cast<float*>(workspace);
  return status_of(launch_conv_bwd(r, a->dtype, d_weight, d_bias, stream_of(stream)));
}

int dr_short_conv_step(const dr_conv* a, const void* x, const float* weight, const float* bias,
                       const void* state, void* state_out, void* y, dr_stream_t stream) {
  if (!a || !x || !weight || !state || !state_out || !y) return DR_ERR_NULL;
  dr_conv one = *a;
  one.T = 1, one.x_st = 0, one.lens = nullptr;
  int st = check_conv(&one);
  if (st != DR_OK) return st;
  ConvArgs r = conv_args(&one, x, weight, bias, state);
  r.y = y, r.s1 = state_out;
  return status_of(launch_conv_step(r, a->dtype, stream_of(stream)));
}

size_t dr_selective_scan_fwd_workspace_bytes(const dr_scan* a) {
  if (!a || check_scan(a) != DR_OK) return 0;
  return scan_fwd_workspace(scan_args(a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), sm_count());
}

int dr_selective_scan_fwd(const dr_scan* a, const void* x, const void* dt, const void* Bm, const void* Cm,
                          const void* z, const float* init_state, void* y, float* final_state, void* workspace,
                          size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !x || !dt || !Bm || !Cm || !y) return DR_ERR_NULL;
  int st = check_scan(a);
  if (st != DR_OK) return st;
  if (!aligned16(init_state, final_state)) return DR_ERR_ALIGN;
  ScanArgs r = scan_args(a, x, dt, Bm, Cm, z, init_state);
  r.y = y, r.hT = final_state;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  if (workspace) {
    const size_t need = scan_fwd_workspace(r, sms);
    if (workspace_bytes < need) return DR_ERR_WORKSPACE;
    if (!aligned256(workspace)) return DR_ERR_ALIGN;
    if (!need) workspace = nullptr;
  }
  return status_of(launch_scan_fwd(r, a->dtype, sms, workspace, stream_of(stream)));
}

size_t dr_selective_scan_bwd_workspace_bytes(const dr_scan* a) {
  if (!a || check_scan(a) != DR_OK) return 0;
  return scan_bwd_workspace(scan_args(a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr));
}

int dr_selective_scan_bwd(const dr_scan* a, const void* x, const void* dt, const void* Bm, const void* Cm,
                          const void* z, const float* init_state, const void* d_y, const float* d_final_state,
                          const dr_scan_grads* g, void* workspace, size_t workspace_bytes, dr_stream_t stream) {
  if (!a || !x || !dt || !Bm || !Cm || !d_y || !g || !g->dx || !g->ddt || !g->dB || !g->dC || !g->dA ||
      (z && !g->dz))
    return DR_ERR_NULL;
  int st = check_scan(a);
  if (st != DR_OK) return st;
  ScanArgs r = scan_args(a, x, dt, Bm, Cm, z, init_state);
  if (!workspace || workspace_bytes < scan_bwd_workspace(r)) return DR_ERR_WORKSPACE;
  if (!aligned256(workspace)) return DR_ERR_ALIGN;
  const int sms = sm_count();
  if (!sms) return DR_ERR_CUDA;
  r.d_y = d_y, r.d_hT = d_final_state, r.g = *g;
  if (!z) r.g.dz = nullptr;
  return status_of(launch_scan_bwd(r, a->dtype, sms, workspace, stream_of(stream)));
}

int dr_selective_scan_step(const dr_scan* a, const void* x, const void* dt, const void* Bm, const void* Cm,
                           const void* z, const float* state, float* state_out, void* y, dr_stream_t stream) {
  if (!a || !x || !dt || !Bm || !Cm || !state || !state_out || !y) return DR_ERR_NULL;
  dr_scan one = *a;
  one.T = 1, one.lens = nullptr;
  int st = check_scan(&one);
  if (st != DR_OK) return st;
  if (!aligned16(state, state_out)) return DR_ERR_ALIGN;
  ScanArgs r = scan_args(&one, x, dt, Bm, Cm, z, state);
  r.y = y, r.hT = state_out;
  return status_of(launch_scan_step(r, a->dtype, stream_of(stream)));
}

}  // extern "C"
