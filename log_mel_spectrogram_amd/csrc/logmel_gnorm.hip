// The group norm with an activation, channels last, and its gradient (gfx950):
//   n = (x - mean) / sqrt(var + eps) * weight + bias,  y = act(n) * silu(gate),
// mean and var over a group's channels of one row, or of all rows of a sequence.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "logmel_rows.h"
#include "logmel_rows_launch.h"

namespace logmel {
namespace {

template <typename T>
struct GroupArgs {
  int64_t rows, n_seq;
  const int64_t* off;   // null: every row by itself
  int channels, groups, width;
  const T* x;
  int64_t xs;
  const T* gate;
  int64_t gs;
  const float* weight;
  const float* bias;
  int silu;
  float eps;
  T* y;
  int64_t ys;
  float* stats;          // [units][groups][2]: mean, 1 / sqrt(var + eps)
  // the gradient's
  const T* dy;
  int64_t dys;
  T* dx;
  int64_t dxs;
  T* dgate;
  int64_t dgs;
  float* sums;           // [units][groups][2]: means of dn w and dn w xh
  float* part;           // [parts][2][channels]
};

// A unit is what a mean is taken over: a row, or a sequence.
template <typename T>
__device__ __forceinline__ void unit_rows(const GroupArgs<T>& p, int64_t u, int64_t& from,
                                          int64_t& to) {
  if (!p.off) {
    from = u, to = u + 1;
    return;
  }
  from = p.off[u], to = p.off[u + 1];
  from = from < 0 ? 0 : from;
  to = to > p.rows ? p.rows : to;
}

template <typename T>
__device__ __forceinline__ int64_t unit_of(const GroupArgs<T>& p, int64_t row) {
  if (!p.off) return row;
  int64_t lo = 0, hi = p.n_seq;   // the last sequence that starts at or before row
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (p.off[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int N>
__device__ __forceinline__ double block_sum(double v, double (&slots)[N]) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) s += slots[i];
  return s;
}

// What one value gives and takes.
template <typename T>
struct Value {
  float xh, n, act, slope, gated, gate_slope;
  __device__ Value(const GroupArgs<T>& p, int64_t r, int c, float mean, float root) {
    xh = ((float)p.x[r * p.xs + c] - mean) * root;
    n = xh * (p.weight ? p.weight[c] : 1.0f) + (p.bias ? p.bias[c] : 0.0f);
    act = n, slope = 1.0f, gated = 1.0f, gate_slope = 0.0f;
    if (p.silu) {
      const float s = Gate<float>::sigmoid(n);
      act = n * s;
      slope = s * (1.0f + n * (1.0f - s));
    }
    if (p.gate) {
      const float g = (float)p.gate[r * p.gs + c];
      const float s = Gate<T>::sigmoid(g);
      gated = g * s;
      gate_slope = s * (1.0f + g * (1.0f - s));
    }
  }
};

template <typename T>
__global__ __launch_bounds__(256) void logmel_group_stats_kernel(GroupArgs<T> p, int64_t items) {
  __shared__ double slots[4];
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int g = (int)(item % p.groups);
    int64_t from, to;
    unit_rows(p, item / p.groups, from, to);
    const int64_t n = to > from ? (to - from) * p.width : 0;
    const double inv = n ? 1.0 / (double)n : 0.0;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256)
      s += (double)(float)p.x[(from + i / p.width) * p.xs + g * p.width + i % p.width];
    const double mean = block_sum(s, slots) * inv;
    s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
      const double d =
          (double)(float)p.x[(from + i / p.width) * p.xs + g * p.width + i % p.width] - mean;
      s += d * d;
    }
    const double var = block_sum(s, slots) * inv;
    if (threadIdx.x == 0) {
      p.stats[item * 2] = (float)mean;
      p.stats[item * 2 + 1] = (float)(1.0 / sqrt(var + (double)p.eps));
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logmel_group_apply_kernel(GroupArgs<T> p) {
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    if (p.off && r >= p.off[p.n_seq]) break;
    const int64_t u = unit_of(p, r);
    for (int c = threadIdx.x; c < p.channels; c += 256) {
      const float* st = p.stats + (u * p.groups + c / p.width) * 2;
      const Value<T> v(p, r, c, st[0], st[1]);
      p.y[r * p.ys + c] = (T)(v.act * v.gated);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logmel_group_sums_kernel(GroupArgs<T> p, int64_t items) {
  __shared__ double slots[4];
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int g = (int)(item % p.groups);
    int64_t from, to;
    unit_rows(p, item / p.groups, from, to);
    const int64_t n = to > from ? (to - from) * p.width : 0;
    const double inv = n ? 1.0 / (double)n : 0.0;
    double s1 = 0.0, s2 = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
      const int64_t r = from + i / p.width;
      const int c = g * p.width + (int)(i % p.width);
      const Value<T> v(p, r, c, p.stats[item * 2], p.stats[item * 2 + 1]);
      const float q = (float)p.dy[r * p.dys + c] * v.gated * v.slope *
                      (p.weight ? p.weight[c] : 1.0f);
      s1 += (double)q;
      s2 += (double)(q * v.xh);
    }
    s1 = block_sum(s1, slots) * inv;
    s2 = block_sum(s2, slots) * inv;
    if (threadIdx.x == 0) {
      p.sums[item * 2] = (float)s1;
      p.sums[item * 2 + 1] = (float)s2;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logmel_group_dx_kernel(GroupArgs<T> p) {
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    if (p.off && r >= p.off[p.n_seq]) break;
    const int64_t u = unit_of(p, r);
    for (int c = threadIdx.x; c < p.channels; c += 256) {
      const int64_t at = (u * p.groups + c / p.width) * 2;
      const float root = p.stats[at + 1];
      const Value<T> v(p, r, c, p.stats[at], root);
      const float dy = (float)p.dy[r * p.dys + c];
      const float q = dy * v.gated * v.slope * (p.weight ? p.weight[c] : 1.0f);
      p.dx[r * p.dxs + c] = (T)(root * (q - p.sums[at] - v.xh * p.sums[at + 1]));
      if (p.dgate) p.dgate[r * p.dgs + c] = (T)(dy * v.act * v.gate_slope);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logmel_group_params_kernel(GroupArgs<T> p,
                                                                  int64_t part_rows) {
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t from = blockIdx.x * part_rows;
  int64_t to = from + part_rows < p.rows ? from + part_rows : p.rows;
  if (p.off && to > p.off[p.n_seq]) to = p.off[p.n_seq];
  double s1 = 0.0, s2 = 0.0;
  for (int64_t r = from; r < to; ++r) {
    const float* st = p.stats + (unit_of(p, r) * p.groups + c / p.width) * 2;
    const Value<T> v(p, r, c, st[0], st[1]);
    const float dn = (float)p.dy[r * p.dys + c] * v.gated * v.slope;
    s1 += (double)(dn * v.xh);
    s2 += (double)dn;
  }
  p.part[(blockIdx.x * 2 + 0) * (int64_t)p.channels + c] = (float)s1;
  p.part[(blockIdx.x * 2 + 1) * (int64_t)p.channels + c] = (float)s2;
}

template <typename T>
GroupArgs<T> group_args(const logmel_group_norm_input& in) {
  GroupArgs<T> p{};
  p.rows = in.rows;
  p.n_seq = in.n_seq;
  p.off = in.d_seq_offsets;
  p.channels = (int)in.channels;
  p.groups = (int)in.groups;
  p.width = (int)(in.channels / in.groups);
  p.x = static_cast<const T*>(in.d_x);
  p.xs = in.x_stride;
  p.gate = static_cast<const T*>(in.d_gate);
  p.gs = in.gate_stride;
  p.weight = in.d_weight;
  p.bias = in.d_bias;
  p.silu = in.activation == LOGMEL_ACT_SILU;
  p.eps = in.eps;
  return p;
}

constexpr int64_t kPartRows = 512;

int64_t units_of(const logmel_group_norm_input& in) {
  return in.d_seq_offsets ? in.n_seq : in.rows;
}
int64_t parts_of(const logmel_group_norm_input& in) { return (in.rows + kPartRows - 1) / kPartRows; }
unsigned grid_of(int64_t n) { return (unsigned)(n < (1 << 22) ? n : 1 << 22); }

template <typename T>
hipError_t launch_group(const logmel_group_norm_input& in, void* y, int64_t y_stride, float* stats,
                        void* ws, hipStream_t stream) {
  GroupArgs<T> p = group_args<T>(in);
  p.y = static_cast<T*>(y);
  p.ys = y_stride;
  p.stats = stats ? stats : static_cast<float*>(ws);
  const int64_t items = units_of(in) * in.groups;
  if (items) logmel_group_stats_kernel<T><<<grid_of(items), 256, 0, stream>>>(p, items);
  if (in.rows) logmel_group_apply_kernel<T><<<grid_of(in.rows), 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_group_backward(const logmel_group_norm_input& in, const float* stats,
                                 const logmel_group_norm_grad& g, void* ws, hipStream_t stream) {
  GroupArgs<T> p = group_args<T>(in);
  const int64_t items = units_of(in) * in.groups;
  p.sums = static_cast<float*>(ws);
  p.part = p.sums + items * 2;
  p.stats = stats ? const_cast<float*>(stats) : p.part + parts_of(in) * 2 * in.channels;
  p.dy = static_cast<const T*>(g.d_dy);
  p.dys = g.dy_stride;
  p.dx = static_cast<T*>(g.d_dx);
  p.dxs = g.dx_stride;
  p.dgate = static_cast<T*>(g.d_dgate);
  p.dgs = g.dgate_stride;
  if (items && !stats) logmel_group_stats_kernel<T><<<grid_of(items), 256, 0, stream>>>(p, items);
  if (items) logmel_group_sums_kernel<T><<<grid_of(items), 256, 0, stream>>>(p, items);
  if (in.rows && items) logmel_group_dx_kernel<T><<<grid_of(in.rows), 256, 0, stream>>>(p);
  if (g.d_dweight || g.d_dbias) {
    const int64_t parts = items ? parts_of(in) : 0;
    if (parts)
      logmel_group_params_kernel<T><<<dim3((unsigned)parts, (unsigned)((in.channels + 255) / 256)),
                                      256, 0, stream>>>(p, kPartRows);
    const PartSums out[3] = {
        {g.d_dweight, 0, nullptr}, {g.d_dbias, 1, nullptr}, {nullptr, 0, nullptr}};
    return logmel_launch_part_sums(p.part, parts, 2, in.channels, out, stream);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace logmel

int64_t logmel_group_workspace(const logmel_group_norm_input& in, int backward, int cus) {
  using namespace logmel;
  const int64_t items = units_of(in) * in.groups;
  if (!backward) return items * 8;
  return items * 16 + parts_of(in) * 2 * in.channels * 4;
}

hipError_t logmel_launch_group(const logmel_group_norm_input& in, void* y, int64_t y_stride,
                               float* stats, void* ws, int cus, hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_group<decltype(zero)>(in, y, y_stride, stats, ws, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}

hipError_t logmel_launch_group_backward(const logmel_group_norm_input& in, const float* stats,
                                        const logmel_group_norm_grad& grad, void* ws, int cus,
                                        hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_group_backward<decltype(zero)>(in, stats, grad, ws, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}
