// The block norm and its gradient (gfx950):
//   t = h / rms(h) * w_post * silu(gate), y = res + scale * t,
//   z = y / rms(y) * w_pre.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "logmel_rows.h"
#include "logmel_rows_launch.h"

namespace logmel {

template <typename T>
struct NormArgs {
  int64_t rows, channels;
  const T* res;
  int64_t ress;
  const T* h;
  int64_t hs;
  const T* o;
  int64_t os;
  const float* w_post;
  const float* scale;
  const float* w_pre;
  float eps;
};

template <typename T>
struct NormGradArgs {
  const T* dy;
  int64_t dys;
  const T* dz;
  int64_t dzs;
  T* dres;
  int64_t dress;
  T* dh;
  int64_t dhs;
  T* dgate;
  int64_t dgates;
  double* part;   // [workgroups][3][channels]: dw_post, dscale, dw_pre
};

// Sum over the workgroup's 4 wavefronts, in every lane.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float sums[4];
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// The factors of channel c of row r; r1 = 1 / rms(h).
template <typename T>
struct Cell {
  float h, n, act, slope, s, t, y;
  __device__ Cell(const NormArgs<T>& p, int64_t r, int64_t c, float r1) {
    y = (float)p.res[r * p.ress + c];
    if (!p.h) return;
    h = (float)p.h[r * p.hs + c];
    n = h * r1 * (p.w_post ? p.w_post[c] : 1.0f);
    act = 1.0f;
    if (p.o) {
      const float o = (float)p.o[r * p.os + c];
      float a, u;
      Gate<T>::pair(o, 0.0f, a, u);
      act = o * a;
      slope = a * __builtin_fmaf(o, u, 1.0f);
    }
    s = p.scale ? p.scale[c] : 1.0f;
    t = n * act;
    y = __builtin_fmaf(s, t, y);
  }
};

// One workgroup per row, a pass over the row for each sum it needs.
template <typename T>
__global__ __launch_bounds__(256) void logmel_norm_simple_kernel(NormArgs<T> p, T* y, int64_t ys,
                                                                 T* z, int64_t zs) {
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    float r1 = 0.0f;
    if (p.h) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
        const float h = (float)p.h[r * p.hs + c];
        s = __builtin_fmaf(h, h, s);
      }
      r1 = 1.0f / __builtin_sqrtf(block_sum(s) / (float)p.channels + p.eps);
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
      const Cell<T> k(p, r, c, r1);
      s = __builtin_fmaf(k.y, k.y, s);
      if (y) y[r * ys + c] = (T)k.y;
    }
    if (!z) continue;
    const float r2 = 1.0f / __builtin_sqrtf(block_sum(s) / (float)p.channels + p.eps);
    for (int64_t c = threadIdx.x; c < p.channels; c += 256)
      z[r * zs + c] = (T)(Cell<T>(p, r, c, r1).y * r2 * (p.w_pre ? p.w_pre[c] : 1.0f));
  }
}

template <typename T>
__global__ __launch_bounds__(256) void logmel_norm_backward_simple_kernel(NormArgs<T> p,
                                                                          NormGradArgs<T> q) {
  double* part = q.part + (int64_t)blockIdx.x * 3 * p.channels;
  for (int64_t c = threadIdx.x; c < p.channels; c += 256)
    part[c] = part[p.channels + c] = part[2 * p.channels + c] = 0.0;
  const float inv = 1.0f / (float)p.channels;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    float r1 = 0.0f;
    if (p.h) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
        const float h = (float)p.h[r * p.hs + c];
        s = __builtin_fmaf(h, h, s);
      }
      r1 = 1.0f / __builtin_sqrtf(block_sum(s) * inv + p.eps);
    }
    float r2 = 0.0f, m2 = 0.0f;
    auto weighted = [&](int64_t c) {
      return q.dz ? (float)q.dz[r * q.dzs + c] * (p.w_pre ? p.w_pre[c] : 1.0f) : 0.0f;
    };
    if (q.dz) {
      float s = 0.0f, m = 0.0f;
      for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
        const float y = Cell<T>(p, r, c, r1).y;
        s = __builtin_fmaf(y, y, s);
        m = __builtin_fmaf(weighted(c), y, m);
      }
      r2 = 1.0f / __builtin_sqrtf(block_sum(s) * inv + p.eps);
      m2 = block_sum(m) * inv;
    }
    auto total = [&](int64_t c, float y) {
      float d = q.dy ? (float)q.dy[r * q.dys + c] : 0.0f;
      if (q.dz) d += r2 * (weighted(c) - y * (r2 * r2 * m2));
      return d;
    };
    float m = 0.0f;
    for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
      const Cell<T> k(p, r, c, r1);
      const float d = total(c, k.y);
      if (p.h)
        m = __builtin_fmaf(d * k.s * k.act * (p.w_post ? p.w_post[c] : 1.0f), k.h, m);
    }
    const float m1 = p.h ? block_sum(m) * inv : 0.0f;
    for (int64_t c = threadIdx.x; c < p.channels; c += 256) {
      const Cell<T> k(p, r, c, r1);
      const float d = total(c, k.y);
      q.dres[r * q.dress + c] = (T)d;
      if (p.h) {
        const float ds = d * k.s;
        const float qa = ds * k.act;
        if (p.o) q.dgate[r * q.dgates + c] = (T)(ds * k.n * k.slope);
        const float w = qa * (p.w_post ? p.w_post[c] : 1.0f);
        q.dh[r * q.dhs + c] = (T)(r1 * (w - k.h * (r1 * r1 * m1)));
        part[c] += qa * k.h * r1;
        part[p.channels + c] += d * k.t;
      }
      if (q.dz) part[2 * p.channels + c] += (float)q.dz[r * q.dzs + c] * k.y * r2;
    }
  }
}

template <typename T>
NormArgs<T> norm_args(const logmel_norm_input& in) {
  return {in.rows,
          in.channels,
          static_cast<const T*>(in.d_res),
          in.res_stride,
          static_cast<const T*>(in.d_h),
          in.h_stride,
          static_cast<const T*>(in.d_gate),
          in.gate_stride,
          in.d_w_post,
          in.d_scale,
          in.d_w_pre,
          in.eps};
}

int64_t norm_parts(int64_t rows, int cus) { return rows < 4 * cus ? rows : 4 * cus; }

template <typename T>
hipError_t launch_norm(const logmel_norm_input& in, void* y, int64_t ys, void* z, int64_t zs,
                       hipStream_t stream) {
  const unsigned grid = (unsigned)(in.rows < (1 << 20) ? in.rows : 1 << 20);
  logmel_norm_simple_kernel<T><<<grid, 256, 0, stream>>>(norm_args<T>(in), static_cast<T*>(y), ys,
                                                         static_cast<T*>(z), zs);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_backward(const logmel_norm_input& in, const logmel_norm_grad& g, void* ws,
                                int cus, hipStream_t stream) {
  NormGradArgs<T> q{static_cast<const T*>(g.d_dy),
                    g.dy_stride,
                    static_cast<const T*>(g.d_dz),
                    g.dz_stride,
                    static_cast<T*>(g.d_dres),
                    g.dres_stride,
                    static_cast<T*>(g.d_dh),
                    g.dh_stride,
                    static_cast<T*>(g.d_dgate),
                    g.dgate_stride,
                    static_cast<double*>(ws)};
  const int64_t parts = norm_parts(in.rows, cus);
  if (parts)
    logmel_norm_backward_simple_kernel<T>
        <<<(unsigned)parts, 256, 0, stream>>>(norm_args<T>(in), q);
  float* outs[3] = {g.d_dw_post, g.d_dscale, g.d_dw_pre};
  for (int i = 0; i < 3; ++i)
    if (outs[i]) {
      const hipError_t e = logmel_launch_part_sum(q.part + i * in.channels, parts,
                                                  3 * in.channels, in.channels, outs[i], stream);
      if (e != hipSuccess) return e;
    }
  return hipGetLastError();
}

}  // namespace logmel

int64_t logmel_norm_workspace(const logmel_norm_input& in, int cus) {
  return logmel::norm_parts(in.rows, cus) * 3 * in.channels * 8;
}

hipError_t logmel_launch_norm(const logmel_norm_input& in, void* y, int64_t y_stride, void* z,
                              int64_t z_stride, int, hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_norm<decltype(zero)>(in, y, y_stride, z, z_stride, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}

hipError_t logmel_launch_norm_backward(const logmel_norm_input& in, const logmel_norm_grad& grad,
                                       void* ws, int cus, hipStream_t stream) {
  auto go = [&](auto zero) {
    return logmel::launch_norm_backward<decltype(zero)>(in, grad, ws, cus, stream);
  };
  if (in.type == LOGMEL_F32) return go(0.0f);
  if (in.type == LOGMEL_F16) return go((logmel::f16_t)0.0f);
  return go((logmel::bf16_t)0.0f);
}
