// C-ABI layer of the row operators: argument checks, then the launchers. The
// declarations and their contracts are in include/logmel.h.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <new>
#include <vector>

#include "logmel.h"
#include "logmel_plan.h"
#include "logmel_rows_launch.h"

namespace {

int64_t type_size(int32_t type) {
  switch (type) {
    case LOGMEL_F32: return 4;
    case LOGMEL_F16:
    case LOGMEL_BF16: return 2;
    default: return 0;
  }
}

// Bytes a call touches: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Span {
  uintptr_t p;
  int64_t rows, width, pitch;
  uintptr_t end() const { return p + (uintptr_t)((rows - 1) * pitch + width); }
};

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  if (a.end() <= b.p || b.end() <= a.p) return false;
  // column slices of one buffer: the rows interleave and never meet
  if (a.pitch == b.pitch && a.rows > 1 && b.rows > 1) {
    const int64_t d = (int64_t)((a.p > b.p ? a.p - b.p : b.p - a.p) % (uintptr_t)a.pitch);
    const int64_t lo = a.p > b.p ? b.width : a.width;   // of the one that starts first
    const int64_t hi = a.p > b.p ? a.width : b.width;
    if (d >= lo && d + hi <= a.pitch) return false;
  }
  return true;
}

// Collects a call's operands and its first fault.
class Operands {
 public:
  Operands(int32_t type, int64_t rows, int64_t channels)
      : size_(type_size(type)), rows_(rows), channels_(channels) {
    if (rows < 0 || channels < 1) {
      fault(LOGMEL_ERR_INVALID_ARGUMENT);
    } else if (!size_) {
      fault(LOGMEL_ERR_UNSUPPORTED);
    } else if (channels > INT64_MAX / 8) {
      fault(LOGMEL_ERR_INPUT_TOO_LONG);
    }
  }

  void row(const void* p, int64_t stride, bool output, bool required) {
    row(p, stride, output, required, channels_);
  }

  // a row operand of a width of its own
  void row(const void* p, int64_t stride, bool output, bool required, int64_t channels) {
    if (status_) return;
    if (!p) {
      if (required && rows_) fault(LOGMEL_ERR_INVALID_ARGUMENT);
      return;
    }
    if ((uintptr_t)p % (uintptr_t)size_ || stride < channels)
      return fault(LOGMEL_ERR_INVALID_ARGUMENT);
    if (rows_ && stride > INT64_MAX / 8 / rows_) return fault(LOGMEL_ERR_INPUT_TOO_LONG);
    add({(uintptr_t)p, rows_, channels * size_, stride * size_}, output);
  }

  // n rows of `channels` fp32; except: the one operand that this output may
  // be as well (as `at` returned it), none by default
  void floats(const float* p, int64_t n, bool output, int except = -1) {
    floats(p, n, channels_, output, except);
  }

  // n rows of `width` fp32
  void floats(const float* p, int64_t n, int64_t width, bool output, int except) {
    if (status_ || !p) return;
    if ((uintptr_t)p % 4) return fault(LOGMEL_ERR_INVALID_ARGUMENT);
    if (n && width > INT64_MAX / 8 / n) return fault(LOGMEL_ERR_INPUT_TOO_LONG);
    add({(uintptr_t)p, n, width * 4, width * 4}, output, except);
  }

  // the operand at p that was added last; -1 if it is another or none
  int at(const void* p) const {
    return n_ && p && span_[n_ - 1].p == (uintptr_t)p ? n_ - 1 : -1;
  }

  void bytes(const void* p, int64_t n, bool output) {
    if (!status_ && p) add({(uintptr_t)p, 1, n, n}, output);
  }

  void fault(int status) {
    if (!status_) status_ = status;
  }

  int status() const { return status_; }

 private:
  void add(const Span& s, bool output, int except = -1) {
    for (int i = 0; i < n_; ++i)
      if ((output || out_[i]) && !(i == except && s.p == span_[i].p) && overlap(span_[i], s))
        return fault(LOGMEL_ERR_INVALID_ARGUMENT);
    span_[n_] = s;
    out_[n_++] = output;
  }

  int64_t size_, rows_, channels_;
  int status_ = LOGMEL_OK;
  Span span_[16];
  bool out_[16];
  int n_ = 0;
};

Operands scan_operands(const logmel_scan_input& in) {
  Operands o(in.type, in.rows, in.channels);
  if (in.n_seq < 0 || in.max_frames < 0 || (!in.d_seq_offsets && in.n_seq) ||
      (uintptr_t)in.d_seq_offsets % 8)
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (in.n_seq > INT64_MAX / 16 || in.channels > LOGMEL_SCAN_MAX_CHANNELS)
    o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  o.row(in.d_x, in.x_stride, false, in.n_seq > 0);
  o.row(in.d_gate, in.gate_stride, false, in.n_seq > 0);
  if (!o.status()) o.bytes(in.d_seq_offsets, (in.n_seq + 1) * 8, false);
  o.floats(in.d_bias, 1, false);
  o.floats(in.d_state, in.n_seq, false);
  return o;
}

void workspace_operand(Operands& o, const void* ws, int64_t bytes, int64_t need) {
  if (o.status() || need == 0) return;
  if (!ws || bytes < need || (uintptr_t)ws % 16) return o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  o.bytes(ws, need, true);
}

int64_t checkpoint_rows(int64_t rows) {
  return rows / LOGMEL_SCAN_CHECKPOINT + (rows % LOGMEL_SCAN_CHECKPOINT != 0);
}

// The offsets read back (one synchronisation), for LOGMEL_VALIDATE=1.
// Input: that of an operator along sequences.
template <typename Input>
int validate_offsets(const Input& in, hipStream_t st) {
  if (!env_validate() || in.n_seq == 0) return LOGMEL_OK;
  std::vector<int64_t> off;
  try {
    off.resize((size_t)in.n_seq + 1);
  } catch (const std::exception&) {
    return LOGMEL_ERR_OUT_OF_MEMORY;
  }
  if (hipMemcpyAsync(off.data(), in.d_seq_offsets, off.size() * 8, hipMemcpyDeviceToHost, st) !=
          hipSuccess ||
      hipStreamSynchronize(st) != hipSuccess)
    return LOGMEL_ERR_DEVICE;
  if (off[0] != 0 || off.back() > in.rows) return LOGMEL_ERR_INVALID_ARGUMENT;
  for (size_t i = 0; i + 1 < off.size(); ++i)
    if (off[i + 1] < off[i] || (in.max_frames && off[i + 1] - off[i] > in.max_frames))
      return LOGMEL_ERR_INVALID_ARGUMENT;
  return LOGMEL_OK;
}

int cus_of(const logmel_plan* plan) { return plan->resident_waves / 4; }

Operands norm_operands(const logmel_norm_input& in) {
  Operands o(in.type, in.rows, in.channels);
  if (!o.status() && in.channels > LOGMEL_NORM_MAX_CHANNELS) o.fault(LOGMEL_ERR_UNSUPPORTED);
  if (!std::isfinite(in.eps) || in.eps < 0.0f) o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (!in.d_h && (in.d_gate || in.d_w_post || in.d_scale)) o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  o.row(in.d_res, in.res_stride, false, true);
  o.row(in.d_h, in.h_stride, false, false);
  o.row(in.d_gate, in.gate_stride, false, false);
  o.floats(in.d_w_post, 1, false);
  o.floats(in.d_scale, 1, false);
  o.floats(in.d_w_pre, 1, false);
  return o;
}

// The checks of a call along sequences that do not depend on its operands.
template <typename Input>
void sequences(Operands& o, const Input& in) {
  if (in.n_seq < 0 || in.max_frames < 0 || (!in.d_seq_offsets && in.n_seq) ||
      (uintptr_t)in.d_seq_offsets % 8)
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (in.n_seq > INT64_MAX / 16) o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  if (!o.status()) o.bytes(in.d_seq_offsets, (in.n_seq + 1) * 8, false);
}

// Heads that fit the kernels' indexes; their product with a head's width and
// state does not overflow.
constexpr int64_t kMostHeads = 1 << 20;

Operands attention_operands(const logmel_attention_input& in) {
  Operands o(in.type, in.rows, in.heads);
  if (in.qk_heads < 1 || in.head_dk < 1 || in.head_dv < 1)
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (!o.status() && in.heads > kMostHeads) o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  if (!o.status() && (in.heads % in.qk_heads || !std::isfinite(in.scale)))
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (!o.status() && (in.head_dk > LOGMEL_ATTENTION_MAX_HEAD_DIM ||
                      in.head_dv > LOGMEL_ATTENTION_MAX_HEAD_DIM))
    o.fault(LOGMEL_ERR_UNSUPPORTED);
  sequences(o, in);
  const bool some = in.n_seq > 0;
  if (some && !in.d_log_decay) o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  o.row(in.d_q, in.q_stride, false, some, in.qk_heads * in.head_dk);
  o.row(in.d_k, in.k_stride, false, some, in.qk_heads * in.head_dk);
  o.row(in.d_v, in.v_stride, false, some, in.heads * in.head_dv);
  o.floats(in.d_log_decay, 1, false);
  // the workspace's count too, for any way of splitting
  if (!o.status() && in.rows && in.heads * in.head_dk > INT64_MAX / 64 / in.rows)
    o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  if (!o.status() && some && in.heads * in.head_dk * in.head_dv > INT64_MAX / 8 / in.n_seq)
    o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  return o;
}

int64_t head_state(const logmel_attention_input& in) {
  return in.heads * in.head_dk * in.head_dv;
}

Operands group_operands(const logmel_group_norm_input& in) {
  Operands o(in.type, in.rows, in.channels);
  if (!o.status() && in.channels > LOGMEL_NORM_MAX_CHANNELS) o.fault(LOGMEL_ERR_UNSUPPORTED);
  if (!std::isfinite(in.eps) || in.eps < 0.0f || in.groups < 1)
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (!o.status() && in.channels % in.groups) o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  if (in.activation != LOGMEL_ACT_NONE && in.activation != LOGMEL_ACT_SILU)
    o.fault(LOGMEL_ERR_UNSUPPORTED);
  if (!in.d_seq_offsets && in.max_frames) o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  sequences(o, in);
  o.row(in.d_x, in.x_stride, false, !in.d_seq_offsets || in.n_seq > 0);
  o.row(in.d_gate, in.gate_stride, false, false);
  o.floats(in.d_weight, 1, false);
  o.floats(in.d_bias, 1, false);
  // the workspace's count, for rows by themselves
  if (!o.status() && in.rows > INT64_MAX / 64 / in.channels) o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  // and over sequences
  if (!o.status() && in.n_seq > INT64_MAX / 64 / in.groups) o.fault(LOGMEL_ERR_INPUT_TOO_LONG);
  return o;
}

// Whether a call of the group norm has anything to do.
bool empty(const logmel_group_norm_input& in) {
  return in.d_seq_offsets ? in.n_seq == 0 : in.rows == 0;
}

}  // namespace

extern "C" {

int64_t logmel_gated_scan_checkpoint_rows(int64_t rows) {
  return rows < 0 ? -1 : checkpoint_rows(rows);
}

int64_t logmel_gated_scan_workspace(const logmel_plan* plan, const logmel_scan_input* in,
                                    int backward) {
  if (!plan || !in || scan_operands(*in).status()) return -1;
  return logmel_scan_workspace(*in, backward != 0, cus_of(plan));
}

int logmel_gated_scan(const logmel_plan* plan, const logmel_scan_input* in, void* d_h,
                      int64_t h_stride, float* d_state_out, float* d_checkpoints,
                      void* d_workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = scan_operands(*in);
  if (o.status()) return o.status();
  const int state = o.at(in->d_state);   // the last operand of scan_operands
  const int64_t need = logmel_scan_workspace(*in, 0, cus_of(plan));
  o.row(d_h, h_stride, true, in->n_seq > 0);
  o.floats(d_state_out, in->n_seq, true, state);   // may be the state, and no other operand
  o.floats(d_checkpoints, checkpoint_rows(in->rows), true);
  workspace_operand(o, d_workspace, workspace_bytes, need);
  if (o.status()) return o.status();
  if (in->n_seq == 0) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_scan(*in, d_h, h_stride, d_state_out, d_checkpoints, d_workspace,
                            cus_of(plan), st) == hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int logmel_gated_scan_backward(const logmel_plan* plan, const logmel_scan_input* in,
                               const float* d_checkpoints, const logmel_scan_grad* grad,
                               void* d_workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in || !grad) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = scan_operands(*in);
  if (o.status()) return o.status();
  const int64_t need = logmel_scan_workspace(*in, 1, cus_of(plan));
  if (!d_checkpoints && in->rows && in->n_seq) return LOGMEL_ERR_INVALID_ARGUMENT;
  // the sums of a bias that is not there have no place in the workspace
  if (grad->d_dbias && !in->d_bias) return LOGMEL_ERR_INVALID_ARGUMENT;
  o.floats(d_checkpoints, checkpoint_rows(in->rows), false);
  o.row(grad->d_dh, grad->dh_stride, false, in->n_seq > 0);
  o.floats(grad->d_dstate_out, in->n_seq, false);
  o.row(grad->d_dx, grad->dx_stride, true, in->n_seq > 0);
  o.row(grad->d_dgate, grad->dgate_stride, true, in->n_seq > 0);
  o.floats(grad->d_dbias, 1, true);
  o.floats(grad->d_dstate, in->n_seq, true);
  workspace_operand(o, d_workspace, workspace_bytes, need);
  if (o.status()) return o.status();
  if (in->n_seq == 0 && !grad->d_dbias) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_scan_backward(*in, d_checkpoints, *grad, d_workspace, cus_of(plan), st) ==
                 hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int logmel_block_norm(const logmel_plan* plan, const logmel_norm_input* in, void* d_y,
                      int64_t y_stride, void* d_z, int64_t z_stride, void* hip_stream) {
  if (!plan || !in) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = norm_operands(*in);
  if (in->rows > 0 && ((!d_y && !d_z) || (d_y && !in->d_h)))
    o.fault(LOGMEL_ERR_INVALID_ARGUMENT);
  o.row(d_y, y_stride, true, false);
  o.row(d_z, z_stride, true, false);
  if (o.status()) return o.status();
  if (in->rows == 0) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  return logmel_launch_norm(*in, d_y, y_stride, d_z, z_stride, cus_of(plan),
                            static_cast<hipStream_t>(hip_stream)) == hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int64_t logmel_block_norm_workspace(const logmel_plan* plan, const logmel_norm_input* in) {
  if (!plan || !in || norm_operands(*in).status()) return -1;
  return logmel_norm_workspace(*in, cus_of(plan));
}

int logmel_block_norm_backward(const logmel_plan* plan, const logmel_norm_input* in,
                               const logmel_norm_grad* grad, void* d_workspace,
                               int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in || !grad) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = norm_operands(*in);
  if (o.status()) return o.status();
  const bool rows = in->rows > 0;
  if ((rows && !grad->d_dy && !grad->d_dz) || (rows && in->d_h && !grad->d_dh) ||
      (!in->d_h && grad->d_dh) || (rows && in->d_gate && !grad->d_dgate) ||
      (!in->d_gate && grad->d_dgate) || (!in->d_h && (grad->d_dw_post || grad->d_dscale)) ||
      (rows && !grad->d_dz && grad->d_dw_pre))
    return LOGMEL_ERR_INVALID_ARGUMENT;
  o.row(grad->d_dy, grad->dy_stride, false, false);
  o.row(grad->d_dz, grad->dz_stride, false, false);
  o.row(grad->d_dres, grad->dres_stride, true, true);
  o.row(grad->d_dh, grad->dh_stride, true, false);
  o.row(grad->d_dgate, grad->dgate_stride, true, false);
  o.floats(grad->d_dw_post, 1, true);
  o.floats(grad->d_dscale, 1, true);
  o.floats(grad->d_dw_pre, 1, true);
  workspace_operand(o, d_workspace, workspace_bytes, logmel_norm_workspace(*in, cus_of(plan)));
  if (o.status()) return o.status();
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  return logmel_launch_norm_backward(*in, *grad, d_workspace, cus_of(plan),
                                     static_cast<hipStream_t>(hip_stream)) == hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int64_t logmel_linear_attention_workspace(const logmel_plan* plan,
                                          const logmel_attention_input* in, int backward) {
  if (!plan || !in || attention_operands(*in).status()) return -1;
  return logmel_attention_workspace(*in, backward != 0, cus_of(plan));
}

int logmel_linear_attention(const logmel_plan* plan, const logmel_attention_input* in, void* d_o,
                            int64_t o_stride, float* d_state_out, void* d_workspace,
                            int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = attention_operands(*in);
  if (o.status()) return o.status();
  o.floats(in->d_state, in->n_seq, head_state(*in), false, -1);
  if (o.status()) return o.status();
  const int state = o.at(in->d_state);
  const int64_t need = logmel_attention_workspace(*in, 0, cus_of(plan));
  o.row(d_o, o_stride, true, in->n_seq > 0, in->heads * in->head_dv);
  o.floats(d_state_out, in->n_seq, head_state(*in), true, state);
  workspace_operand(o, d_workspace, workspace_bytes, need);
  if (o.status()) return o.status();
  if (in->n_seq == 0) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_attention(*in, d_o, o_stride, d_state_out, d_workspace, cus_of(plan), st) ==
                 hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int logmel_linear_attention_backward(const logmel_plan* plan, const logmel_attention_input* in,
                                     const logmel_attention_grad* grad, void* d_workspace,
                                     int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in || !grad) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = attention_operands(*in);
  if (o.status()) return o.status();
  o.floats(in->d_state, in->n_seq, head_state(*in), false, -1);
  if (o.status()) return o.status();
  const int64_t need = logmel_attention_workspace(*in, 1, cus_of(plan));
  const bool some = in->n_seq > 0;
  const int64_t qk = in->qk_heads * in->head_dk, vw = in->heads * in->head_dv;
  o.row(grad->d_do, grad->do_stride, false, some, vw);
  o.floats(grad->d_dstate_out, in->n_seq, head_state(*in), false, -1);
  o.row(grad->d_dq, grad->dq_stride, true, some, qk);
  o.row(grad->d_dk, grad->dk_stride, true, some, qk);
  o.row(grad->d_dv, grad->dv_stride, true, some, vw);
  o.floats(grad->d_dstate, in->n_seq, head_state(*in), true, -1);
  workspace_operand(o, d_workspace, workspace_bytes, need);
  if (o.status()) return o.status();
  if (!some) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_attention_backward(*in, *grad, d_workspace, cus_of(plan), st) == hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int64_t logmel_group_norm_workspace(const logmel_plan* plan, const logmel_group_norm_input* in,
                                    int backward) {
  if (!plan || !in || group_operands(*in).status()) return -1;
  return logmel_group_workspace(*in, backward != 0, cus_of(plan));
}

int logmel_group_norm(const logmel_plan* plan, const logmel_group_norm_input* in, void* d_y,
                      int64_t y_stride, float* d_stats, void* d_workspace,
                      int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = group_operands(*in);
  if (o.status()) return o.status();
  if (d_stats && !in->d_seq_offsets) return LOGMEL_ERR_INVALID_ARGUMENT;
  o.row(d_y, y_stride, true, !empty(*in));
  o.floats(d_stats, in->n_seq, in->groups * 2, true, -1);
  workspace_operand(o, d_workspace, workspace_bytes,
                    logmel_group_workspace(*in, 0, cus_of(plan)));
  if (o.status()) return o.status();
  if (empty(*in)) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_group(*in, d_y, y_stride, d_stats, d_workspace, cus_of(plan), st) ==
                 hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

int logmel_group_norm_backward(const logmel_plan* plan, const logmel_group_norm_input* in,
                               const float* d_stats, const logmel_group_norm_grad* grad,
                               void* d_workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!plan || !in || !grad) return LOGMEL_ERR_INVALID_ARGUMENT;
  Operands o = group_operands(*in);
  if (o.status()) return o.status();
  const bool some = !empty(*in);
  if ((d_stats && !in->d_seq_offsets) || (some && in->d_seq_offsets && !d_stats) ||
      (some && in->rows && in->d_gate && !grad->d_dgate) || (!in->d_gate && grad->d_dgate) ||
      (!in->d_weight && grad->d_dweight) || (!in->d_bias && grad->d_dbias))
    return LOGMEL_ERR_INVALID_ARGUMENT;
  o.floats(d_stats, in->n_seq, in->groups * 2, false, -1);
  o.row(grad->d_dy, grad->dy_stride, false, some);
  o.row(grad->d_dx, grad->dx_stride, true, some);
  o.row(grad->d_dgate, grad->dgate_stride, true, false);
  o.floats(grad->d_dweight, 1, true);
  o.floats(grad->d_dbias, 1, true);
  workspace_operand(o, d_workspace, workspace_bytes,
                    logmel_group_workspace(*in, 1, cus_of(plan)));
  if (o.status()) return o.status();
  if (!some && !grad->d_dweight && !grad->d_dbias) return LOGMEL_OK;
  DeviceGuard g(plan->cfg.device);
  if (!g.ok) return LOGMEL_ERR_DEVICE;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  const int v = validate_offsets(*in, st);
  if (v != LOGMEL_OK) return v;
  return logmel_launch_group_backward(*in, d_stats, *grad, d_workspace, cus_of(plan), st) ==
                 hipSuccess
             ? LOGMEL_OK
             : LOGMEL_ERR_DEVICE;
}

}  // extern "C"
