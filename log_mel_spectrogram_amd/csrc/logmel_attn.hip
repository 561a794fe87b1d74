// Linear attention with a decay for each head, and its gradient (gfx950). Per
// sequence and head, with lambda = e^log_decay,
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t.
// The gradient is the same operator three times. With T_t = lambda T_{t+1} +
// scale q_t do_t^T, from the last row to the first,
//   dq_t = scale do_t S_t^T,   dk_t = v_t T_t^T,   dv_t = k_t T_t,
// so that every kernel here works on a job: operands a, b and c, a state W of
// b times c, a direction, and
//   W = lambda W + gamma b_t c_t^T,   o_t = beta a_t W.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "logmel_rows.h"
#include "logmel_rows_launch.h"

namespace logmel {
namespace {

// One pass of the operator. Head h of an operand is columns (h / share) * width
// on: a and b are da wide, c and o dc.
template <typename T>
struct AttnJob {
  int64_t rows, n_seq;
  const int64_t* off;
  int heads, da, dc;
  const T* a;
  int64_t as;
  const T* b;
  int64_t bs;
  const T* c;
  int64_t cs;
  int share_a, share_b, share_c;
  T* o;             // rows of heads * dc, rounded; or
  float* of;        // the same as fp32, dense, where heads are summed afterwards
  int64_t os;
  const float* log_decay;
  const float* state;   // [n_seq][heads][da][dc], or [dc][da] where transposed; or null
  float* state_out;
  bool transposed;
  bool back;            // from each sequence's last row to its first
  float beta, gamma;
};

// Rows [from, to) of sequence i, inside the operands whatever the offsets hold.
struct Run {
  int64_t from, to;
};
template <typename T>
__device__ __forceinline__ Run run_of(const AttnJob<T>& p, int64_t i) {
  int64_t from = p.off[i], to = p.off[i + 1];
  from = from < 0 ? 0 : from;
  to = to > p.rows ? p.rows : to;
  return {from, to};
}

// ------------------------------------------------------- row after row
//
// A workgroup holds the 64 columns of a sequence's and head's state that one
// slab of c makes: lane (ag, cg) of 16 x 16 holds four columns of every
// sixteenth row. 16 rows at a time are laid out in LDS, worked one after the
// other, and their products with the state joined at the end. Right for any
// length; the form for single rows and short pushes, whose time is that of
// reading and writing the states.
constexpr int kStepRows = 16;
constexpr int kSlab = 64;

template <typename T, int DA>
__global__ __launch_bounds__(256) void logmel_attn_rows_kernel(AttnJob<T> p, int slabs,
                                                               int64_t items) {
  constexpr int kU = DA / 16;
  __shared__ float sa[kStepRows][DA], sb[kStepRows][DA];
  __shared__ __attribute__((aligned(16))) float sc[kStepRows][kSlab];
  __shared__ __attribute__((aligned(16))) float part[kStepRows][4][kSlab];
  const int tid = threadIdx.x, cg = tid & 15, ag = tid >> 4;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int slab = (int)(item % slabs);
    const int h = (int)(item / slabs % p.heads);
    const int64_t seq = item / slabs / p.heads;
    const Run run = run_of(p, seq);
    const int c0 = slab * kSlab;
    const float lambda = __expf(p.log_decay[h]);
    const float* in = p.state ? p.state + (seq * p.heads + h) * p.da * p.dc : nullptr;
    float* out = p.state_out ? p.state_out + (seq * p.heads + h) * p.da * p.dc : nullptr;
    auto at = [&](int a, int c) {
      return p.transposed ? (int64_t)c * p.da + a : (int64_t)a * p.dc + c;
    };
    float w[kU][4];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = ag + 16 * u, c = c0 + 4 * cg + j;
        w[u][j] = in && a < p.da && c < p.dc ? in[at(a, c)] : 0.0f;
      }
    const int64_t n = run.to > run.from ? run.to - run.from : 0;
    for (int64_t t0 = 0; t0 < n; t0 += kStepRows) {
      const int held = (int)(n - t0 < kStepRows ? n - t0 : kStepRows);
      auto row = [&](int t) { return p.back ? run.to - 1 - t0 - t : run.from + t0 + t; };
      __syncthreads();   // the rows before are read to the end
      for (int i = tid; i < kStepRows * DA; i += 256) {
        const int t = i / DA, d = i % DA;
        const bool on = t < held && d < p.da;
        sa[t][d] = on ? (float)p.a[row(t) * p.as + h / p.share_a * p.da + d] : 0.0f;
        sb[t][d] = on ? (float)p.b[row(t) * p.bs + h / p.share_b * p.da + d] * p.gamma : 0.0f;
      }
      for (int i = tid; i < kStepRows * kSlab; i += 256) {
        const int t = i / kSlab, d = i % kSlab;
        const bool on = t < held && c0 + d < p.dc;
        sc[t][d] = on ? (float)p.c[row(t) * p.cs + h / p.share_c * p.dc + c0 + d] : 0.0f;
      }
      __syncthreads();
      for (int t = 0; t < held; ++t) {
        const float keep = p.back && t0 + t == 0 ? 1.0f : lambda;
        const float4 c = *reinterpret_cast<const float4*>(&sc[t][4 * cg]);
        float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float a = sa[t][ag + 16 * u], b = sb[t][ag + 16 * u];
          const float cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[u][j] = __builtin_fmaf(keep, w[u][j], b * cv[j]);
            o[j] = __builtin_fmaf(a, w[u][j], o[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j] += __shfl_xor(o[j], 16);
          o[j] += __shfl_xor(o[j], 32);
        }
        if ((tid & 63) < 16)
          *reinterpret_cast<float4*>(&part[t][tid >> 6][4 * cg]) =
              make_float4(o[0], o[1], o[2], o[3]);
      }
      __syncthreads();
      for (int i = tid; i < held * kSlab; i += 256) {
        const int t = i / kSlab, d = i % kSlab;
        if (c0 + d >= p.dc) continue;
        const float v =
            p.beta * ((part[t][0][d] + part[t][1][d]) + (part[t][2][d] + part[t][3][d]));
        const int64_t to = row(t) * p.os + (int64_t)h * p.dc + c0 + d;
        if (p.of)
          p.of[to] = v;
        else
          p.o[to] = (T)v;
      }
    }
    if (!out) continue;
    const float last = p.back && n > 0 ? lambda : 1.0f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = ag + 16 * u, c = c0 + 4 * cg + j;
        if (a < p.da && c < p.dc) out[at(a, c)] = last * w[u][j];
      }
  }
}

// out[r][g width + d] = sum over the `share` heads of group g, in their order:
// the gradient of an operand that several heads share.
template <typename T>
__global__ __launch_bounds__(256) void logmel_attn_share_kernel(const float* part, int64_t rows,
                                                                int groups, int share, int width,
                                                                const int64_t* off, int64_t n_seq,
                                                                T* out, int64_t stride) {
  const int64_t last = off[n_seq] < rows ? off[n_seq] : rows;
  const int64_t n = last * groups * width;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int d = (int)(i % width), g = (int)(i / width % groups);
    const int64_t r = i / width / groups;
    const float* v = part + (r * groups + g) * share * width + d;
    float s = v[0];
    for (int j = 1; j < share; ++j) s += v[j * width];
    out[r * stride + (int64_t)g * width + d] = (T)s;
  }
}

template <typename T>
hipError_t launch_job(const AttnJob<T>& p, hipStream_t stream) {
  const int slabs = (p.dc + kSlab - 1) / kSlab;
  const int64_t items = p.n_seq * p.heads * slabs;
  const unsigned grid = (unsigned)(items < (1 << 22) ? items : 1 << 22);
  if (p.da <= 64)
    logmel_attn_rows_kernel<T, 64><<<grid, 256, 0, stream>>>(p, slabs, items);
  else
    logmel_attn_rows_kernel<T, 128><<<grid, 256, 0, stream>>>(p, slabs, items);
  return hipGetLastError();
}

template <typename T>
AttnJob<T> job_of(const logmel_attention_input& in) {
  AttnJob<T> p{};
  p.rows = in.rows;
  p.n_seq = in.n_seq;
  p.off = in.d_seq_offsets;
  p.heads = (int)in.heads;
  p.share_a = p.share_b = p.share_c = 1;
  p.log_decay = in.d_log_decay;
  return p;
}

template <typename T>
hipError_t launch_attention(const logmel_attention_input& in, void* o, int64_t o_stride,
                            float* state_out, void* ws, int cus, hipStream_t stream) {
  AttnJob<T> p = job_of<T>(in);
  p.da = (int)in.head_dk;
  p.dc = (int)in.head_dv;
  p.a = static_cast<const T*>(in.d_q);
  p.as = in.q_stride;
  p.b = static_cast<const T*>(in.d_k);
  p.bs = in.k_stride;
  p.c = static_cast<const T*>(in.d_v);
  p.cs = in.v_stride;
  p.share_a = p.share_b = (int)(in.heads / in.qk_heads);
  p.o = static_cast<T*>(o);
  p.os = o_stride;
  p.state = in.d_state;
  p.state_out = state_out;
  p.beta = in.scale;
  p.gamma = 1.0f;
  return launch_job(p, stream);
}

template <typename T>
hipError_t launch_attention_backward(const logmel_attention_input& in,
                                     const logmel_attention_grad& g, void* ws, int cus,
                                     hipStream_t stream) {
  const int share = (int)(in.heads / in.qk_heads);
  const T* q = static_cast<const T*>(in.d_q);
  const T* k = static_cast<const T*>(in.d_k);
  const T* v = static_cast<const T*>(in.d_v);
  const T* d = static_cast<const T*>(g.d_do);
  const int dk = (int)in.head_dk, dv = (int)in.head_dv;
  float* part = share > 1 ? static_cast<float*>(ws) : nullptr;
  // a gradient of q or k: its own rows, or each head's first and then their sums
  auto shared = [&](AttnJob<T>& p, void* out, int64_t stride) {
    p.o = static_cast<T*>(out);
    p.of = part;
    p.os = part ? in.heads * dk : stride;
    hipError_t e = launch_job(p, stream);
    if (e != hipSuccess || !part) return e;
    const int64_t n = in.rows * in.qk_heads * dk;
    const int64_t blocks = (n + 255) / 256;
    if (n)
      logmel_attn_share_kernel<T><<<(unsigned)(blocks < cus * 8 ? blocks : cus * 8), 256, 0, stream>>>(
          part, in.rows, (int)in.qk_heads, share, dk, in.d_seq_offsets, in.n_seq,
          static_cast<T*>(out), stride);
    return hipGetLastError();
  };
  AttnJob<T> p = job_of<T>(in);   // dq
  p.a = d, p.as = g.do_stride;
  p.b = v, p.bs = in.v_stride;
  p.c = k, p.cs = in.k_stride;
  p.share_c = share;
  p.da = dv, p.dc = dk;
  p.state = in.d_state;
  p.transposed = true;
  p.beta = in.scale, p.gamma = 1.0f;
  hipError_t e = shared(p, g.d_dq, g.dq_stride);
  if (e != hipSuccess) return e;
  p.back = true;                  // dk
  p.a = v, p.as = in.v_stride;
  p.b = d, p.bs = g.do_stride;
  p.c = q, p.cs = in.q_stride;
  p.state = g.d_dstate_out;
  p.beta = 1.0f, p.gamma = in.scale;
  e = shared(p, g.d_dk, g.dk_stride);
  if (e != hipSuccess) return e;
  p.a = k, p.as = in.k_stride;    // dv, and the initial state's gradient
  p.b = q, p.bs = in.q_stride;
  p.c = d, p.cs = g.do_stride;
  p.share_a = p.share_b = share;
  p.share_c = 1;
  p.da = dk, p.dc = dv;
  p.transposed = false;
  p.state_out = g.d_dstate;
  p.of = nullptr;
  p.o = static_cast<T*>(g.d_dv);
  p.os = g.dv_stride;
  return launch_job(p, stream);
}

}  // namespace
}  // namespace logmel

int64_t logmel_attention_workspace(const logmel_attention_input& in, int backward, int cus) {
  return backward && in.heads > in.qk_heads ? in.rows * in.heads * in.head_dk * 4 : 0;
}

hipError_t logmel_launch_attention(const logmel_attention_input& in, void* o, int64_t o_stride,
                                   float* state_out, void* ws, int cus, hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_attention<decltype(zero)>(in, o, o_stride, state_out, ws, cus, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}

hipError_t logmel_launch_attention_backward(const logmel_attention_input& in,
                                            const logmel_attention_grad& grad, void* ws, int cus,
                                            hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_attention_backward<decltype(zero)>(in, grad, ws, cus, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}
