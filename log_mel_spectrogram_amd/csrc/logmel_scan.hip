// The gated scan over packed sequences and its gradient (gfx950):
//   a = sigmoid(gate + bias), u = 1 - a;  h_t = a_t h_{t-1} + u_t x_t.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "logmel_rows.h"
#include "logmel_rows_launch.h"

namespace logmel {

constexpr int64_t kCk = LOGMEL_SCAN_CHECKPOINT;

template <typename T>
struct ScanArgs {
  int64_t rows, channels, n_seq;
  const int64_t* off;
  const T* x;
  int64_t xs;
  const T* g;
  int64_t gs;
  const float* bias;
  const float* state;
  T* h;
  int64_t hs;
  float* state_out;
  float* ck;
};

template <typename T>
struct ScanGradArgs {
  const T* dh;
  int64_t dhs;
  const float* dstate_out;
  T* dx;
  int64_t dxs;
  T* dg;
  int64_t dgs;
  float* dbias_part;   // [n_seq][channels]
  float* dstate;
};

// A lane's first channel: V channels per lane, the last lane of an odd width
// shifted back so that its pair stays inside the row (both lanes then hold
// that channel and write the same value).
template <int V>
__device__ __forceinline__ int64_t lane_channel(int64_t lane, int64_t channels) {
  const int64_t c = lane * V;
  return c + V > channels ? channels - V : c;
}

__device__ __forceinline__ void seq_range(const int64_t* off, int64_t j, int64_t rows, int64_t& s,
                                          int64_t& e) {
  s = off[j];
  e = off[j + 1];
  s = s < 0 ? 0 : s;
  e = e > rows ? rows : e;
}

// One lane per sequence and channel group, row after row.
template <typename T, int V>
__global__ void logmel_scan_serial_kernel(ScanArgs<T> p) {
  const int64_t groups = (p.channels + V - 1) / V;
  const int64_t total = p.n_seq * groups;
  for (int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; id < total;
       id += (int64_t)gridDim.x * blockDim.x) {
    const int64_t j = id / groups;
    const int64_t c = lane_channel<V>(id % groups, p.channels);
    int64_t s, e;
    seq_range(p.off, j, p.rows, s, e);
    float h[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = p.state ? p.state[j * p.channels + c + v] : 0.0f;
      b[v] = p.bias ? p.bias[c + v] : 0.0f;
    }
    for (int64_t t = s; t < e; ++t) {
      if (p.ck && t % kCk == 0 && t > s) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.ck[t / kCk * p.channels + c + v] = h[v];
      }
      const auto x = row_load<T, V>(p.x + t * p.xs + c);
      const auto g = row_load<T, V>(p.g + t * p.gs + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, u;
        gate_pair<T>((float)g.v[v] + b[v], a, u);
        h[v] = __builtin_fmaf(a, h[v], u * (float)x.v[v]);
      }
      row_store<T, V>(p.h + t * p.hs + c, h);
    }
    if (p.state_out) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.state_out[j * p.channels + c + v] = h[v];
    }
  }
}

// One wavefront per sequence and 64 channels, a block of kCk rows after the
// other from the last: the states before each of its rows into LDS, then the
// rows backwards.
template <typename T>
__global__ __launch_bounds__(64) void logmel_scan_backward_serial_kernel(ScanArgs<T> p,
                                                                         ScanGradArgs<T> q) {
  __shared__ float prev[kCk][64];
  const int lane = threadIdx.x;
  const int64_t slabs = (p.channels + 63) / 64;
  for (int64_t id = blockIdx.x; id < p.n_seq * slabs; id += gridDim.x) {
    const int64_t j = id / slabs;
    const int64_t c = id % slabs * 64 + lane;
    if (c >= p.channels) continue;
    int64_t s, e;
    seq_range(p.off, j, p.rows, s, e);
    const int64_t at = j * p.channels + c;
    const float b = p.bias ? p.bias[c] : 0.0f;
    float carry = q.dstate_out ? q.dstate_out[at] : 0.0f;   // a_{t+1} D_{t+1}
    float db = 0.0f;
    for (int64_t k = e > s ? (e - 1) / kCk : -1; k >= 0 && (k + 1) * kCk > s; --k) {
      const int64_t r0 = k * kCk < s ? s : k * kCk;
      const int64_t r1 = (k + 1) * kCk < e ? (k + 1) * kCk : e;
      float h = r0 > s ? p.ck[k * p.channels + c] : (p.state ? p.state[at] : 0.0f);
      for (int64_t t = r0; t < r1; ++t) {
        prev[t - r0][lane] = h;
        float a, u;
        gate_pair<T>((float)p.g[t * p.gs + c] + b, a, u);
        h = __builtin_fmaf(a, h, u * (float)p.x[t * p.xs + c]);
      }
      for (int64_t t = r1 - 1; t >= r0; --t) {
        float a, u;
        gate_pair<T>((float)p.g[t * p.gs + c] + b, a, u);
        const float d = (float)q.dh[t * q.dhs + c] + carry;
        const float dg = a * u * (prev[t - r0][lane] - (float)p.x[t * p.xs + c]) * d;
        q.dx[t * q.dxs + c] = (T)(u * d);
        q.dg[t * q.dgs + c] = (T)dg;
        db += dg;
        carry = a * d;
      }
    }
    if (q.dbias_part) q.dbias_part[at] = db;
    if (q.dstate) q.dstate[at] = carry;
  }
}

// 64 channels per workgroup; each of its 4 wavefronts sums every fourth part,
// and the four sums are added in order.
__global__ __launch_bounds__(256) void logmel_part_sum_kernel(const float* part, int64_t parts,
                                                              int64_t stride, int64_t channels,
                                                              float* out) {
  __shared__ float sums[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < channels)
    for (int64_t g = wave; g < parts; g += 4) s += part[g * stride + c];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < channels)
    out[c] = sums[0][lane] + sums[1][lane] + sums[2][lane] + sums[3][lane];
}

template <typename T>
ScanArgs<T> scan_args(const logmel_scan_input& in) {
  ScanArgs<T> p{};
  p.rows = in.rows;
  p.channels = in.channels;
  p.n_seq = in.n_seq;
  p.off = in.d_seq_offsets;
  p.x = static_cast<const T*>(in.d_x);
  p.xs = in.x_stride;
  p.g = static_cast<const T*>(in.d_gate);
  p.gs = in.gate_stride;
  p.bias = in.d_bias;
  p.state = in.d_state;
  return p;
}

unsigned grid_of(int64_t blocks) {
  constexpr int64_t kMost = 1 << 20;
  return (unsigned)(blocks < 1 ? 1 : blocks > kMost ? kMost : blocks);
}

template <typename T>
hipError_t launch_scan(const logmel_scan_input& in, void* h, int64_t h_stride, float* state_out,
                       float* checkpoints, void*, int, hipStream_t stream) {
  ScanArgs<T> p = scan_args<T>(in);
  p.h = static_cast<T*>(h);
  p.hs = h_stride;
  p.state_out = state_out;
  p.ck = checkpoints;
  const int64_t lanes = in.n_seq * ((in.channels + 1) / 2);
  if (in.channels == 1)
    logmel_scan_serial_kernel<T, 1><<<grid_of((in.n_seq + 255) / 256), 256, 0, stream>>>(p);
  else
    logmel_scan_serial_kernel<T, 2><<<grid_of((lanes + 255) / 256), 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan_backward(const logmel_scan_input& in, const float* checkpoints,
                                const logmel_scan_grad& grad, void* ws, int,
                                hipStream_t stream) {
  ScanArgs<T> p = scan_args<T>(in);
  p.ck = const_cast<float*>(checkpoints);
  ScanGradArgs<T> q{};
  q.dh = static_cast<const T*>(grad.d_dh);
  q.dhs = grad.dh_stride;
  q.dstate_out = grad.d_dstate_out;
  q.dx = static_cast<T*>(grad.d_dx);
  q.dxs = grad.dx_stride;
  q.dg = static_cast<T*>(grad.d_dgate);
  q.dgs = grad.dgate_stride;
  q.dbias_part = grad.d_dbias ? static_cast<float*>(ws) : nullptr;
  q.dstate = grad.d_dstate;
  logmel_scan_backward_serial_kernel<T>
      <<<grid_of(in.n_seq * ((in.channels + 63) / 64)), 64, 0, stream>>>(p, q);
  if (grad.d_dbias)
    return logmel_launch_part_sum(q.dbias_part, in.n_seq, in.channels, in.channels, grad.d_dbias,
                                  stream);
  return hipGetLastError();
}

}  // namespace logmel

hipError_t logmel_launch_part_sum(const float* part, int64_t parts, int64_t stride,
                                  int64_t channels, float* out, hipStream_t stream) {
  logmel::logmel_part_sum_kernel<<<(unsigned)((channels + 63) / 64), 256, 0, stream>>>(
      part, parts, stride, channels, out);
  return hipGetLastError();
}

int64_t logmel_scan_workspace(const logmel_scan_input& in, int backward, int) {
  return backward ? in.n_seq * in.channels * 4 : 0;
}

hipError_t logmel_launch_scan(const logmel_scan_input& in, void* h, int64_t h_stride,
                              float* state_out, float* checkpoints, void* ws, int cus,
                              hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_scan<decltype(zero)>(in, h, h_stride, state_out, checkpoints, ws, cus,
                                               stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}

hipError_t logmel_launch_scan_backward(const logmel_scan_input& in, const float* checkpoints,
                                       const logmel_scan_grad& grad, void* ws, int cus,
                                       hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_scan_backward<decltype(zero)>(in, checkpoints, grad, ws, cus, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}
