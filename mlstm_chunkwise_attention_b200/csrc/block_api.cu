// C ABI of the operators around the recurrence: argument checks, the choice of
// 16-byte or element accesses, workspace layouts and launches.  Declared in
// include/mlstm_block.h, which states the operations, layouts and errors.
#include "mlstm_block.h"

#include "block.h"

namespace {

using mlstm::Rows;
using mlstm::cuda_result;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t elem_size(int dtype) { return dtype == MLSTM_BF16 ? 2 : 4; }
bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3) != 0; }
bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a != nullptr && b != nullptr && x < y + bytes && y < x + bytes;
}

// A strided tensor with the strides of dimensions of size 1 taken as 0 (they are never used).
Rows rows_of(const mlstm_rows_t* r, int B, int T, int G) {
  Rows o;
  if (r == nullptr) return o;
  o.p = r->data;
  o.sb = B > 1 ? r->batch : 0;
  o.st = T > 1 ? r->token : 0;
  o.sh = G > 1 ? r->head : 0;
  return o;
}
bool bad_rows(const Rows& r, int dtype) {
  return r.p == nullptr || ((uintptr_t)r.p & (elem_size(dtype) - 1)) != 0;
}
// Whether every vector of eight at a multiple of eight channels is 16-byte aligned.
bool aligned(const Rows& r, int dtype) {
  const long long per = 16 / (long long)elem_size(dtype);
  return !off16(r.p) && r.sb % per == 0 && r.st % per == 0 && r.sh % per == 0;
}

// Errors in order: nonsense first, then what the kernels do not cover.
int check_common(int B, int T, int dtype) {
  if (B < 0 || T < 0) return MLSTM_ERR_INVALID;
  if (dtype != MLSTM_BF16 && dtype != MLSTM_FP32) return MLSTM_ERR_INVALID;
  if ((long long)B * T >= (1LL << 30)) return MLSTM_ERR_UNSUPPORTED;
  return MLSTM_OK;
}
int check_channels(int B, int T, int NH, int d) {
  if (NH <= 0 || d <= 0) return MLSTM_ERR_INVALID;
  const long long D = (long long)NH * d;
  if (D > (1 << 24) || B * D >= (1LL << 31) || B * D * T >= (1LL << 40)) return MLSTM_ERR_UNSUPPORTED;
  return MLSTM_OK;
}
int check_conv(int B, int T, int NH, int d, int W, int dtype) {
  int st = check_common(B, T, dtype);
  if (st == MLSTM_OK) st = check_channels(B, T, NH, d);
  if (st != MLSTM_OK) return st;
  if (W <= 0) return MLSTM_ERR_INVALID;
  return W >= 2 && W <= 4 ? MLSTM_OK : MLSTM_ERR_UNSUPPORTED;
}
int check_scan(int B, int T, int D, int G, int N, int dtype) {
  int st = check_common(B, T, dtype);
  if (st == MLSTM_OK) st = check_channels(B, T, 1, D);
  if (st != MLSTM_OK) return st;
  if (G <= 0 || N <= 0 || D % G != 0) return MLSTM_ERR_INVALID;
  if (N > 64 || (long long)B * T * G >= (1LL << 31)) return MLSTM_ERR_UNSUPPORTED;
  return MLSTM_OK;
}
int check_norm(int B, int T, int NH, int d, int scope, int dtype) {
  int st = check_common(B, T, dtype);
  if (st == MLSTM_OK) st = check_channels(B, T, NH, d);
  if (st != MLSTM_OK) return st;
  if (scope != MLSTM_SCOPE_TOKEN && scope != MLSTM_SCOPE_SEQUENCE) return MLSTM_ERR_INVALID;
  if (scope == MLSTM_SCOPE_TOKEN) return d > 512 ? MLSTM_ERR_UNSUPPORTED : MLSTM_OK;
  if ((long long)B * T == 0) return MLSTM_OK;
  return (long long)B * NH >= (1 << 28) || mlstm::norm_sequence_items(B, T, NH, d) >= (1LL << 31)
             ? MLSTM_ERR_UNSUPPORTED
             : MLSTM_OK;
}

int pending_error(const char* where) { return cuda_result(cudaPeekAtLastError(), where); }

// dst = src, or zeros without one.
int fill(void* dst, const void* src, size_t bytes, void* stream, const char* where) {
  if (dst == nullptr || bytes == 0) return MLSTM_OK;
  return cuda_result(src != nullptr ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice,
                                                      (cudaStream_t)stream)
                                    : cudaMemsetAsync(dst, 0, bytes, (cudaStream_t)stream),
                     where);
}

struct ScanWorkspace {
  mlstm::ScanSegments cut;
  size_t seg_state, seg_sum, turn, bc, a, d, total;
};
// The forward's workspace holds what the segments need alone (nothing for a whole sequence).
ScanWorkspace scan_workspace(int B, int T, int D, int G, int N, bool backward) {
  ScanWorkspace w = {};
  if ((long long)B * T == 0) return w;
  w.cut = backward ? mlstm::scan_bwd_segments(B, T, D, G, N) : mlstm::scan_fwd_segments(B, T, D, G, N);
  size_t rows = 0;
  if (w.cut.count > 1) rows = (size_t)(w.cut.in_turn ? 1 : w.cut.count) * B * D;
  w.seg_sum = align256(rows * mlstm::scan_pad(N) * 4);
  w.turn = align256(w.seg_sum + (w.cut.in_turn ? 0 : rows * 4));
  w.bc = align256(w.turn + (w.cut.in_turn ? ((size_t)w.cut.tiles + mlstm::kTurnTiles) * 4 : 0));
  w.total = w.bc;
  if (backward) {
    const mlstm::ScanBwdSizes z = mlstm::scan_bwd_sizes(B, T, D, G, N);
    w.a = align256(w.bc + z.part_bc * 4);
    w.d = align256(w.a + z.part_a * 4);
    w.total = align256(w.d + z.part_d * 4);
  }
  return w;
}
int use_segments(mlstm::ScanArgs* a, char* ws, const ScanWorkspace& w, void* stream) {
  a->seg_len = w.cut.len;
  a->segs = w.cut.count;
  a->in_turn = w.cut.in_turn;
  a->seg_state = (float*)(ws + w.seg_state);
  a->seg_sum = (float*)(ws + w.seg_sum);
  a->turn = (unsigned int*)(ws + w.turn);
  if (!a->in_turn) return MLSTM_OK;
  return fill(a->turn, nullptr, ((size_t)w.cut.tiles + mlstm::kTurnTiles) * 4, stream, "scan turns");
}

// The inputs of a scan call; T is that of the call (1 for a step).
int scan_inputs(const mlstm_scan_t* p, int T, mlstm::ScanArgs* a) {
  a->B = p->B; a->T = T; a->D = p->D; a->G = p->G; a->N = p->N;
  a->softplus = p->softplus; a->dtype = p->dtype;
  a->x = rows_of(&p->x, p->B, T, 1);
  a->dt = rows_of(&p->dt, p->B, T, 1);
  a->z = rows_of(&p->z, p->B, T, 1);
  a->b = rows_of(&p->b, p->B, T, p->G);
  a->c = rows_of(&p->c, p->B, T, p->G);
  a->A = p->a; a->skip = p->skip; a->dt_bias = p->dt_bias;
  a->state_in = p->state_in;
  if (bad_rows(a->x, p->dtype) || bad_rows(a->dt, p->dtype) || bad_rows(a->b, p->dtype) ||
      bad_rows(a->c, p->dtype) || (a->z.p != nullptr && bad_rows(a->z, p->dtype)))
    return MLSTM_ERR_INVALID;
  if (p->a == nullptr || off4(p->a) || off4(p->skip) || off4(p->dt_bias) || off16(p->state_in))
    return MLSTM_ERR_INVALID;
  a->wide = (p->D / p->G) % 8 == 0 && aligned(a->x, p->dtype) && aligned(a->dt, p->dtype) &&
            (a->z.p == nullptr || aligned(a->z, p->dtype));
  a->wide_bc = aligned(a->b, p->dtype) && aligned(a->c, p->dtype);
  return MLSTM_OK;
}

int check_act(int act, bool sigmoid) {
  return act == MLSTM_ACT_NONE || act == MLSTM_ACT_SILU || (sigmoid && act == MLSTM_ACT_SIGMOID)
             ? MLSTM_OK
             : MLSTM_ERR_INVALID;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// causal convolution
// ---------------------------------------------------------------------------

int mlstm_conv_fwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                   const void* state_in, const mlstm_rows_t* y, void* state_out, int B, int T,
                   int NH, int d, int W, int act, int dtype, void* stream) {
  int st = check_conv(B, T, NH, d, W, dtype);
  if (st == MLSTM_OK) st = check_act(act, false);
  if (st != MLSTM_OK) return st;
  const size_t es = elem_size(dtype), state = (size_t)B * (W - 1) * NH * d * es;
  if (((uintptr_t)state_in | (uintptr_t)state_out) & (es - 1)) return MLSTM_ERR_INVALID;
  if (overlap(state_in, state_out, state)) return MLSTM_ERR_INVALID;
  if (B == 0) return MLSTM_OK;
  if (T == 0) return fill(state_out, state_in, state, stream, "conv state");
  mlstm::ConvArgs a = {};
  a.x = rows_of(x, B, T, 1);
  a.y = rows_of(y, B, T, NH);
  if (bad_rows(a.x, dtype) || bad_rows(a.y, dtype) || weight == nullptr || off4(weight) || off4(bias))
    return MLSTM_ERR_INVALID;
  a.w = weight; a.bias = bias; a.state_in = state_in; a.state_out = state_out;
  a.B = B; a.T = T; a.NH = NH; a.d = d; a.W = W; a.act = act; a.dtype = dtype;
  a.wide = d % 8 == 0 && aligned(a.x, dtype) && aligned(a.y, dtype) && !off16(state_in) &&
           !off16(state_out) && !off16(weight);
  if ((st = pending_error("before mlstm_conv_fwd")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_conv_fwd(a, (cudaStream_t)stream), "conv_fwd");
}

size_t mlstm_conv_bwd_workspace_size(int B, int T, int NH, int d, int W, int dtype) {
  if (check_conv(B, T, NH, d, W, dtype) != MLSTM_OK) return 0;
  return (size_t)mlstm::conv_bwd_rows(B, T, NH * d) * (W + 1) * NH * d * 4;
}

int mlstm_conv_bwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                   const void* state_in, const mlstm_rows_t* dy, const void* dstate_out,
                   const mlstm_rows_t* dx, float* dweight, float* dbias, void* dstate_in,
                   void* workspace, size_t workspace_bytes, int B, int T, int NH, int d, int W,
                   int act, int dtype, void* stream) {
  int st = check_conv(B, T, NH, d, W, dtype);
  if (st == MLSTM_OK) st = check_act(act, false);
  if (st != MLSTM_OK) return st;
  const size_t es = elem_size(dtype), D = (size_t)NH * d, state = (size_t)B * (W - 1) * D * es;
  if (((uintptr_t)state_in | (uintptr_t)dstate_out | (uintptr_t)dstate_in) & (es - 1))
    return MLSTM_ERR_INVALID;
  if (overlap(dstate_out, dstate_in, state) || overlap(state_in, dstate_in, state))
    return MLSTM_ERR_INVALID;
  if (dweight == nullptr || off4(dweight) || off4(dbias)) return MLSTM_ERR_INVALID;
  if (B == 0 || T == 0) {
    if ((st = fill(dweight, nullptr, D * W * 4, stream, "conv dweight")) != MLSTM_OK) return st;
    if ((st = fill(dbias, nullptr, D * 4, stream, "conv dbias")) != MLSTM_OK) return st;
    return fill(dstate_in, dstate_out, state, stream, "conv dstate");
  }
  mlstm::ConvArgs a = {};
  a.x = rows_of(x, B, T, 1);
  a.y = rows_of(dy, B, T, NH);
  a.dx = rows_of(dx, B, T, 1);
  if (bad_rows(a.x, dtype) || bad_rows(a.y, dtype) || bad_rows(a.dx, dtype) || weight == nullptr ||
      off4(weight) || off4(bias) || off16(workspace))
    return MLSTM_ERR_INVALID;
  if (workspace == nullptr || workspace_bytes < mlstm_conv_bwd_workspace_size(B, T, NH, d, W, dtype))
    return MLSTM_ERR_WORKSPACE;
  a.w = weight; a.bias = bias; a.state_in = state_in; a.dstate_out = dstate_out;
  a.dstate_in = dstate_in; a.dw = dweight; a.dbias = dbias; a.partial = (float*)workspace;
  a.B = B; a.T = T; a.NH = NH; a.d = d; a.W = W; a.act = act; a.dtype = dtype;
  a.wide = d % 8 == 0 && aligned(a.x, dtype) && aligned(a.y, dtype) && aligned(a.dx, dtype) &&
           !off16(state_in) && !off16(dstate_out) && !off16(dstate_in) && !off16(weight);
  if ((st = pending_error("before mlstm_conv_bwd")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_conv_bwd(a, (cudaStream_t)stream), "conv_bwd");
}

int mlstm_conv_step(const mlstm_rows_t* x, const float* weight, const float* bias,
                    const void* state_in, const mlstm_rows_t* y, void* state_out, int B, int NH,
                    int d, int W, int act, int dtype, void* stream) {
  int st = check_conv(B, 1, NH, d, W, dtype);
  if (st == MLSTM_OK) st = check_act(act, false);
  if (st != MLSTM_OK) return st;
  if (B == 0) return MLSTM_OK;
  const size_t es = elem_size(dtype), state = (size_t)B * (W - 1) * NH * d * es;
  mlstm::ConvArgs a = {};
  a.x = rows_of(x, B, 1, 1);
  a.y = rows_of(y, B, 1, NH);
  if (bad_rows(a.x, dtype) || bad_rows(a.y, dtype) || weight == nullptr || off4(weight) ||
      off4(bias) || state_in == nullptr || state_out == nullptr ||
      (((uintptr_t)state_in | (uintptr_t)state_out) & (es - 1)) != 0 ||
      (state_in != state_out && overlap(state_in, state_out, state)))
    return MLSTM_ERR_INVALID;
  a.w = weight; a.bias = bias; a.state_in = state_in; a.state_out = state_out;
  a.B = B; a.T = 1; a.NH = NH; a.d = d; a.W = W; a.act = act; a.dtype = dtype;
  a.wide = d % 8 == 0 && aligned(a.x, dtype) && aligned(a.y, dtype) && !off16(state_in) &&
           !off16(state_out) && !off16(weight);
  if ((st = pending_error("before mlstm_conv_step")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_conv_step(a, (cudaStream_t)stream), "conv_step");
}

// ---------------------------------------------------------------------------
// selective scan
// ---------------------------------------------------------------------------

size_t mlstm_scan_saved_size(int B, int T, int D, int G, int N, int dtype) {
  if (check_scan(B, T, D, G, N, dtype) != MLSTM_OK) return 0;
  const size_t NC = ((size_t)T + mlstm::kScanEvery - 1) / mlstm::kScanEvery;
  return (size_t)B * NC * D * mlstm::scan_pad(N) * 4;
}

size_t mlstm_scan_fwd_workspace_size(int B, int T, int D, int G, int N, int dtype) {
  if (check_scan(B, T, D, G, N, dtype) != MLSTM_OK) return 0;
  return scan_workspace(B, T, D, G, N, false).total;
}

int mlstm_scan_fwd(const mlstm_scan_t* p, const mlstm_rows_t* y, void* saved, float* state_out,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (p == nullptr) return MLSTM_ERR_INVALID;
  int st = check_scan(p->B, p->T, p->D, p->G, p->N, p->dtype);
  if (st != MLSTM_OK) return st;
  const size_t state = (size_t)p->B * p->D * p->N * 4;
  if (off16(p->state_in) || off16(state_out) || off16(saved) || overlap(p->state_in, state_out, state))
    return MLSTM_ERR_INVALID;
  if (p->B == 0) return MLSTM_OK;
  if (p->T == 0) return fill(state_out, p->state_in, state, stream, "scan state");
  mlstm::ScanArgs a = {};
  if ((st = scan_inputs(p, p->T, &a)) != MLSTM_OK) return st;
  a.y = rows_of(y, p->B, p->T, 1);
  if (bad_rows(a.y, p->dtype)) return MLSTM_ERR_INVALID;
  a.wide = a.wide && aligned(a.y, p->dtype);
  const ScanWorkspace w = scan_workspace(p->B, p->T, p->D, p->G, p->N, false);
  if (off16(workspace)) return MLSTM_ERR_INVALID;
  if (w.total > 0 && (workspace == nullptr || workspace_bytes < w.total)) return MLSTM_ERR_WORKSPACE;
  a.state_out = state_out;
  a.saved = (float*)saved;
  if ((st = pending_error("before mlstm_scan_fwd")) != MLSTM_OK) return st;
  if ((st = use_segments(&a, (char*)workspace, w, stream)) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_scan_fwd(a, (cudaStream_t)stream), "scan_fwd");
}

int mlstm_scan_step(const mlstm_scan_t* p, const mlstm_rows_t* y, float* state_out, void* stream) {
  if (p == nullptr) return MLSTM_ERR_INVALID;
  int st = check_scan(p->B, 1, p->D, p->G, p->N, p->dtype);
  if (st != MLSTM_OK) return st;
  if (p->B == 0) return MLSTM_OK;
  const size_t state = (size_t)p->B * p->D * p->N * 4;
  mlstm::ScanArgs a = {};
  if ((st = scan_inputs(p, 1, &a)) != MLSTM_OK) return st;
  a.y = rows_of(y, p->B, 1, 1);
  if (bad_rows(a.y, p->dtype) || p->state_in == nullptr || state_out == nullptr || off16(state_out) ||
      (p->state_in != state_out && overlap(p->state_in, state_out, state)))
    return MLSTM_ERR_INVALID;
  a.state_out = state_out;
  if ((st = pending_error("before mlstm_scan_step")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_scan_step(a, (cudaStream_t)stream), "scan_step");
}

size_t mlstm_scan_bwd_workspace_size(int B, int T, int D, int G, int N, int dtype) {
  if (check_scan(B, T, D, G, N, dtype) != MLSTM_OK) return 0;
  return scan_workspace(B, T, D, G, N, true).total;
}

int mlstm_scan_bwd(const mlstm_scan_t* p, const mlstm_rows_t* dy, const void* saved,
                   const float* dstate_out, const mlstm_scan_grads_t* grads, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (p == nullptr || grads == nullptr) return MLSTM_ERR_INVALID;
  int st = check_scan(p->B, p->T, p->D, p->G, p->N, p->dtype);
  if (st != MLSTM_OK) return st;
  const int B = p->B, T = p->T, D = p->D, dt = p->dtype;
  const size_t state = (size_t)B * D * p->N * 4;
  if (off16(dstate_out) || off16(grads->dstate_in) || overlap(dstate_out, grads->dstate_in, state) ||
      overlap(p->state_in, grads->dstate_in, state))
    return MLSTM_ERR_INVALID;
  if (grads->da == nullptr || off4(grads->da) || off4(grads->dskip) || off4(grads->ddt_bias))
    return MLSTM_ERR_INVALID;
  if (B == 0 || T == 0) {
    if ((st = fill(grads->da, nullptr, (size_t)D * p->N * 4, stream, "scan da")) != MLSTM_OK) return st;
    if ((st = fill(grads->dskip, nullptr, (size_t)D * 4, stream, "scan dskip")) != MLSTM_OK) return st;
    if ((st = fill(grads->ddt_bias, nullptr, (size_t)D * 4, stream, "scan ddt_bias")) != MLSTM_OK)
      return st;
    return fill(grads->dstate_in, dstate_out, state, stream, "scan dstate");
  }
  mlstm::ScanArgs a = {};
  if ((st = scan_inputs(p, T, &a)) != MLSTM_OK) return st;
  a.y = rows_of(dy, B, T, 1);
  a.dx = rows_of(&grads->dx, B, T, 1);
  a.ddt = rows_of(&grads->ddt, B, T, 1);
  a.dz = rows_of(&grads->dz, B, T, 1);
  a.db = rows_of(&grads->db, B, T, p->G);
  a.dc = rows_of(&grads->dc, B, T, p->G);
  const bool gate = a.z.p != nullptr;
  if (bad_rows(a.y, dt) || bad_rows(a.dx, dt) || bad_rows(a.ddt, dt) || bad_rows(a.db, dt) ||
      bad_rows(a.dc, dt) || (gate && bad_rows(a.dz, dt)) || saved == nullptr || off16(saved) ||
      off16(workspace))
    return MLSTM_ERR_INVALID;
  const ScanWorkspace w = scan_workspace(B, T, D, p->G, p->N, true);
  if (workspace == nullptr || workspace_bytes < w.total) return MLSTM_ERR_WORKSPACE;
  a.wide = a.wide && aligned(a.y, dt) && aligned(a.dx, dt) && aligned(a.ddt, dt) &&
           (!gate || aligned(a.dz, dt));
  a.saved = (float*)saved;
  a.dstate_out = dstate_out;
  a.dA = grads->da; a.dskip = grads->dskip; a.ddt_bias = grads->ddt_bias;
  a.dstate_in = grads->dstate_in;
  char* ws = (char*)workspace;
  a.part_bc = (float*)(ws + w.bc);
  a.part_a = (float*)(ws + w.a);
  a.part_d = (float*)(ws + w.d);
  if ((st = pending_error("before mlstm_scan_bwd")) != MLSTM_OK) return st;
  if ((st = use_segments(&a, ws, w, stream)) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_scan_bwd(a, (cudaStream_t)stream), "scan_bwd");
}

// ---------------------------------------------------------------------------
// group norm
// ---------------------------------------------------------------------------

size_t mlstm_group_norm_stats_size(int B, int T, int NH, int d, int scope) {
  if (check_norm(B, T, NH, d, scope, MLSTM_FP32) != MLSTM_OK) return 0;
  return (size_t)B * (scope == MLSTM_SCOPE_TOKEN ? T : 1) * NH * 2 * 4;
}

size_t mlstm_group_norm_workspace_size(int B, int T, int NH, int d, int scope, int dtype,
                                       int backward) {
  if (check_norm(B, T, NH, d, scope, dtype) != MLSTM_OK || (long long)B * T == 0) return 0;
  return mlstm::norm_workspace(B, T, NH, d, scope, dtype, backward != 0);
}

int mlstm_group_norm_fwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                         const mlstm_rows_t* gate, const mlstm_rows_t* y, float* stats,
                         void* workspace, size_t workspace_bytes, int B, int T, int NH, int d,
                         int scope, int act, float eps, int dtype, void* stream) {
  int st = check_norm(B, T, NH, d, scope, dtype);
  if (st == MLSTM_OK) st = check_act(act, true);
  if (st != MLSTM_OK) return st;
  if (!(eps > 0.f)) return MLSTM_ERR_INVALID;
  if ((long long)B * T == 0) return MLSTM_OK;
  mlstm::NormArgs a = {};
  a.x = rows_of(x, B, T, NH);
  a.y = rows_of(y, B, T, NH);
  a.gate = rows_of(gate, B, T, NH);
  const bool gated = a.gate.p != nullptr;
  if (bad_rows(a.x, dtype) || bad_rows(a.y, dtype) || (gated && bad_rows(a.gate, dtype)) ||
      off4(weight) || off4(bias) || ((uintptr_t)stats & 7) != 0 || off16(workspace))
    return MLSTM_ERR_INVALID;
  const size_t need = mlstm::norm_workspace(B, T, NH, d, scope, dtype, false);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
  a.w = weight; a.bias = bias; a.stats = stats; a.ws = (float*)workspace;
  a.B = B; a.T = T; a.NH = NH; a.d = d; a.scope = scope; a.act = act; a.dtype = dtype; a.eps = eps;
  a.wide = d % 8 == 0 && aligned(a.x, dtype) && aligned(a.y, dtype) &&
           (!gated || aligned(a.gate, dtype)) && !off16(weight) && !off16(bias);
  if ((st = pending_error("before mlstm_group_norm_fwd")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_norm_fwd(a, (cudaStream_t)stream), "group_norm_fwd");
}

int mlstm_group_norm_bwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                         const mlstm_rows_t* gate, const mlstm_rows_t* dy, const float* stats,
                         const mlstm_rows_t* dx, const mlstm_rows_t* dgate, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, int B, int T,
                         int NH, int d, int scope, int act, int dtype, void* stream) {
  int st = check_norm(B, T, NH, d, scope, dtype);
  if (st == MLSTM_OK) st = check_act(act, true);
  if (st != MLSTM_OK) return st;
  if (off4(dweight) || off4(dbias)) return MLSTM_ERR_INVALID;
  if ((long long)B * T == 0) {
    if ((st = fill(dweight, nullptr, (size_t)NH * d * 4, stream, "norm dweight")) != MLSTM_OK) return st;
    return fill(dbias, nullptr, (size_t)NH * d * 4, stream, "norm dbias");
  }
  mlstm::NormArgs a = {};
  a.x = rows_of(x, B, T, NH);
  a.y = rows_of(dy, B, T, NH);
  a.gate = rows_of(gate, B, T, NH);
  a.dx = rows_of(dx, B, T, NH);
  a.dgate = rows_of(dgate, B, T, NH);
  const bool gated = a.gate.p != nullptr;
  if (bad_rows(a.x, dtype) || bad_rows(a.y, dtype) || bad_rows(a.dx, dtype) ||
      (gated && (bad_rows(a.gate, dtype) || bad_rows(a.dgate, dtype))) || stats == nullptr ||
      ((uintptr_t)stats & 7) != 0 || off4(weight) || off4(bias) || off16(workspace))
    return MLSTM_ERR_INVALID;
  const size_t need = mlstm::norm_workspace(B, T, NH, d, scope, dtype, true);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
  a.w = weight; a.bias = bias; a.stats = (float*)stats; a.dw = dweight; a.dbias = dbias;
  a.ws = (float*)workspace;
  a.B = B; a.T = T; a.NH = NH; a.d = d; a.scope = scope; a.act = act; a.dtype = dtype;
  a.wide = d % 8 == 0 && aligned(a.x, dtype) && aligned(a.y, dtype) && aligned(a.dx, dtype) &&
           (!gated || (aligned(a.gate, dtype) && aligned(a.dgate, dtype))) && !off16(weight) &&
           !off16(bias);
  if ((st = pending_error("before mlstm_group_norm_bwd")) != MLSTM_OK) return st;
  return cuda_result(mlstm::launch_norm_bwd(a, (cudaStream_t)stream), "group_norm_bwd");
}

int mlstm_block_selftest_timeout(int family, void* workspace, size_t workspace_bytes, void* stream) {
  if (family < MLSTM_WAITS_SCAN_FWD || family > MLSTM_WAITS_NORM || off4(workspace)) return MLSTM_ERR_INVALID;
  if (workspace == nullptr || workspace_bytes < 8) return MLSTM_ERR_WORKSPACE;
  int st = pending_error("before mlstm_block_selftest_timeout");
  if (st == MLSTM_OK) st = fill(workspace, nullptr, 8, stream, "selftest words");
  if (st != MLSTM_OK) return st;
  auto launch = family == MLSTM_WAITS_SCAN_FWD   ? mlstm::launch_scan_fwd_selftest
                : family == MLSTM_WAITS_SCAN_BWD ? mlstm::launch_scan_bwd_selftest
                                                 : mlstm::launch_norm_selftest;
  return cuda_result(launch((unsigned int*)workspace, (cudaStream_t)stream), "block selftest_timeout");
}

}  // extern "C"
