// The block norm and its gradient (gfx950):
//   t = h / rms(h) * w_post * silu(gate), y = res + scale * t,
//   z = y / rms(y) * w_pre.
//
// A row is held by kLanes lanes, 16 bytes of it per lane and vector, kVecs
// vectors per lane, from its one read to its writes; the sums over it are
// formed in registers (and across wavefronts, where a row takes more than
// one, through LDS). The grid is resident and walks the rows, so a lane reads
// its channels' parameters once, and the next rows' values are on their way
// while a row is worked.
//
// Bound by memory: 64 x 2998 x 512 bf16 with gate and both outputs 188 us
// (5.2 TB/s, the rate of a copy, traffic 1.00 x the bytes), 191,872 x 128 42 us,
// 2998 x 4096 fp32 46 us. Small calls cost their launch: 4096 x 128 fp16 2.9 us
// on the device, one row 2.4 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "logmel_rows.h"
#include "logmel_rows_launch.h"

namespace logmel {

template <typename T>
struct NormArgs {
  int64_t rows;
  int channels;
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
struct NormOut {
  T* y;
  int64_t ys;
  T* z;
  int64_t zs;
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
  float* part;   // [workgroups][2][channels]: sums of G n act and of dz y / rms(y); or null
};

// What stands between res and y.
enum Parts { kNone, kNorm, kGated };

// Wavefronts per SIMD that the kernels leave room for: the gradient holds eight
// values of five operands per lane within the 128 registers of four.
constexpr int front_waves(int lanes) { return lanes > 256 ? 4 : 5; }
constexpr int kBackWaves = 4;

// Rows of a lane that are summed in fp32: 16 equal terms are off by 9 roundings
// at most, as many as a row's own arithmetic, whatever the number of rows.
constexpr int kHeld = 16;

template <int kLanes>
constexpr int kThreads = kLanes > 256 ? kLanes : 256;

// Sums over a row's lanes, up to two at once. Rows of several wavefronts meet
// in LDS: one barrier per sum, on two slots in turn (a slot is written again
// only after the barrier of the other, which comes after its last read).
template <int kLanes>
struct RowSum {
  static constexpr bool kShared = kLanes > 64;
  static constexpr int kWaves = kThreads<kLanes> / 64;
  float (*slots)[2][kWaves];
  int turn = 0;

  __device__ void operator()(float& a, float& b, bool two) {
    a = lane_sum<kLanes>(a);
    if (two) b = lane_sum<kLanes>(b);
    if constexpr (kShared) {
      const int wave = threadIdx.x >> 6;
      constexpr int kPer = kLanes / 64;
      const int w0 = wave / kPer * kPer;
      if ((threadIdx.x & 63) == 0) {
        slots[turn][0][wave] = a;
        if (two) slots[turn][1][wave] = b;
      }
      __syncthreads();
      a = b = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        a += slots[turn][0][w0 + i];
        if (two) b += slots[turn][1][w0 + i];
      }
      turn ^= 1;
    }
  }
  __device__ void operator()(float& a) {
    float b = 0.0f;
    (*this)(a, b, false);
  }
};

// The channels a lane holds: vector j is c[j] .. c[j] + V - 1. The last vector
// of a width that V does not divide is shifted back to end with the row, so
// that it is read and written whole: its first values are another lane's too,
// who writes the same, and only the sums leave them out. Lanes past the row's
// end hold nothing. Rows narrower than 16 bytes take V = 1, in kernels of their
// own: value by value in a branch beside the wide loads they cost every
// gradient registers and waits (191,872 x 128 bf16 with its call 136 us, 126
// without the branch; 3000 x 5000 fp32 255 and 211).
template <int kLanes, int kVecs, int V>
struct Channels {
  int C;
  int c[kVecs], skip[kVecs];
  bool on[kVecs];

  __device__ explicit Channels(int channels) : C(channels) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int first = (j * kLanes + (int)(threadIdx.x & (kLanes - 1))) * V;
      on[j] = first < C;
      c[j] = first + V <= C ? first : C - V;
      skip[j] = first - c[j];
    }
  }
  // Where channel c counts: in which lane, and as which of its values.
  __device__ __forceinline__ void place(int c, int& lane, int& value) const {
    const int vec = c / V;
    const int from = vec * V + V <= C ? vec * V : C - V;
    lane = vec % kLanes;
    value = vec / kLanes * V + c - from;
  }
  // Whether value i of vector j counts in this lane's sums.
  __device__ __forceinline__ bool counts(int j, int i) const {
    return on[j] && i >= skip[j];
  }
};

// A lane's vectors of one row operand, 0 where it holds nothing.
template <typename T, int kLanes, int kVecs, int V>
struct RowPiece {
  using Ch = Channels<kLanes, kVecs, V>;
  Packed<T, V> v[kVecs];

  __device__ __forceinline__ void load(const T* row, const Ch& k, bool on) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      v[j] = Packed<T, V>{};
      if (on && k.on[j]) v[j] = row_load<T, V>(row + k.c[j]);
    }
  }

  __device__ __forceinline__ float at(int j, int i) const { return (float)v[j].v[i]; }

  __device__ __forceinline__ void unpack_anew() {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) repack(v[j]);
    }
  }
};

template <typename T, int kLanes, int kVecs, int V>
__device__ __forceinline__ void piece_store(T* row, const Channels<kLanes, kVecs, V>& k,
                                            const float (&x)[kVecs][V]) {
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (k.on[j]) row_store<T, V>(row + k.c[j], x[j]);
}

// A lane's channels of a parameter, 1 where it is absent.
template <int kLanes, int kVecs, int V>
__device__ __forceinline__ void load_params(float (&r)[kVecs][V], const float* p,
                                            const Channels<kLanes, kVecs, V>& k) {
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[j][i] = 1.0f;
    if (!p || !k.on[j]) continue;
    const auto v = row_load<float, V>(p + k.c[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) r[j][i] = v.v[i];
  }
}

// w_post scale, the two factors of t that do not depend on the row.
template <typename T, int kLanes, int kVecs, int V>
__device__ __forceinline__ void load_block_params(float (&r)[kVecs][V], const NormArgs<T>& p,
                                                  const Channels<kLanes, kVecs, V>& k) {
  float s[kVecs][V];
  load_params(r, p.w_post, k);
  load_params(s, p.scale, k);
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) r[j][i] *= s[j][i];
}

// The workgroup's row of this lane, 0 on; one for the whole wavefront, and so
// in a scalar register, where a row takes a wavefront or more.
template <int kLanes>
__device__ __forceinline__ int group_of() {
  const int g = threadIdx.x / kLanes;
  return kLanes >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

template <typename T, int kParts, int kLanes, int kVecs, int V>
__global__ __launch_bounds__(kThreads<kLanes>, front_waves(kLanes)) void logmel_norm_kernel(NormArgs<T> p,
                                                                         NormOut<T> out) {
  using P = RowPiece<T, kLanes, kVecs, V>;
  constexpr int kRows = kThreads<kLanes> / kLanes;
  __shared__ float slots[2][2][kThreads<kLanes> / 64];
  RowSum<kLanes> sum{slots};
  const typename P::Ch k(p.channels);
  const float inv = 1.0f / (float)p.channels;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + group_of<kLanes>();
  P res, h, o;
  auto load = [&](int64_t row) {
    const bool on = row < p.rows;
    res.load(p.res + row * p.ress, k, on);
    if constexpr (kParts != kNone) h.load(p.h + row * p.hs, k, on);
    if constexpr (kParts == kGated) o.load(p.o + row * p.os, k, on);
  };
  load(r);   // on its way before the parameters are waited for
  float w1[kVecs][V], w2[kVecs][V];
  if constexpr (kParts != kNone) load_block_params(w1, p, k);
  load_params(w2, p.w_pre, k);
  // the workgroup's rows together: barriers are met by all of it
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += step, r += step) {
    float y[kVecs][V], t[kVecs][V];
    float s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[j][i] = res.at(j, i);
        if constexpr (kParts != kNone) {
          const float x = h.at(j, i);
          s1 = k.counts(j, i) ? __builtin_fmaf(x, x, s1) : s1;
          t[j][i] = x * w1[j][i];
        }
        if constexpr (kParts == kGated) t[j][i] *= o.at(j, i) * Gate<T>::sigmoid(o.at(j, i));
      }
    if (first + step < p.rows) load(r + step);
    if constexpr (kParts != kNone) {
      sum(s1);
      const float r1 = inv_root(__builtin_fmaf(s1, inv, p.eps));
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) y[j][i] = __builtin_fmaf(t[j][i], r1, y[j][i]);
      if (out.y && r < p.rows) piece_store(out.y + r * out.ys, k, y);
    }
    if (out.z) {
      float s2 = 0.0f;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          s2 = k.counts(j, i) ? __builtin_fmaf(y[j][i], y[j][i], s2) : s2;
      sum(s2);
      const float r2 = inv_root(__builtin_fmaf(s2, inv, p.eps));
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) y[j][i] *= r2 * w2[j][i];
      if (r < p.rows) piece_store(out.z + r * out.zs, k, y);
    }
  }
}

// The gradient. Per row, with n = h / rms(h), w = w_post scale, q = dz w_pre
// and G = dy + r2 (q - y r2^2 mean(q y)):
//   dres = G;  e = G act w;  dh = r1 (e - h r1^2 mean(e h));
//   dgate = G n w slope;  dw_post = scale sum(G n act), dscale = w_post of the
//   same sum;  dw_pre = sum(dz y r2).
// Without dz G is dy, and res is not read.
// Three sums over the row one after the other. The two sums over the lane's
// rows stay in its registers for kHeld rows, then go to fp64 places of its own
// in LDS; at the end the workgroup's rows are added there and each workgroup
// writes one part. Eight values per lane keep all of it within 128 registers,
// so that 16 wavefronts a compute unit have their rows in flight. 64 x 2998 x
// 512 bf16: 302 us (5.2 TB/s, traffic 1.00 x); with 40 values spilled to memory
// it took 896. 2998 x 4096 fp32 82 us. fp32 rows of more than 4096 channels hold
// 8 values a lane in 1024 lanes and spill 20 (3000 x 5000 with its call 198 us,
// 3.9 TB/s).
template <typename T, int kParts, bool kDz, int kLanes, int kVecs, int V>
__global__ __launch_bounds__(kThreads<kLanes>, kBackWaves) void logmel_norm_backward_kernel(
    NormArgs<T> p, NormGradArgs<T> q) {
  using P = RowPiece<T, kLanes, kVecs, V>;
  constexpr int kRows = kThreads<kLanes> / kLanes;
  __shared__ float slots[2][2][kThreads<kLanes> / 64];
  __shared__ double sums[2][kVecs * V][kThreads<kLanes>];
  RowSum<kLanes> sum{slots};
  const typename P::Ch k(p.channels);
  const float inv = 1.0f / (float)p.channels;
  float w1[kVecs][V], w2[kVecs][V];
  float a1[kVecs][V], a2[kVecs][V];
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) a1[j][i] = a2[j][i] = 0.0f;
  if (q.part) {
#pragma unroll
    for (int n = 0; n < kVecs * V; ++n) sums[0][n][threadIdx.x] = sums[1][n][threadIdx.x] = 0.0;
  }
  // the rows since the last time out of the registers, into the lane's places
  auto flush = [&] {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (kParts != kNone) sums[0][j * V + i][threadIdx.x] += (double)a1[j][i];
        if constexpr (kDz) sums[1][j * V + i][threadIdx.x] += (double)a2[j][i];
        a1[j][i] = a2[j][i] = 0.0f;
      }
  };
  int held = 0;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + group_of<kLanes>();
  if constexpr (kParts != kNone) load_block_params(w1, p, k);
  if constexpr (kDz) load_params(w2, p.w_pre, k);
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += step, r += step) {
    P res, h, o, dy, dz;
    const bool on = r < p.rows;
    if constexpr (kParts != kNone) h.load(p.h + r * p.hs, k, on);
    if constexpr (kDz) res.load(p.res + r * p.ress, k, on);
    if constexpr (kParts == kGated) o.load(p.o + r * p.os, k, on);
    if constexpr (kDz) dz.load(q.dz + r * q.dzs, k, on);
    dy.load(q.dy + r * q.dys, k, on && q.dy);
    float r1 = 0.0f;
    float y[kVecs][V], sig[kVecs][V];   // sig: sigmoid(gate)
    if constexpr (kParts != kNone) {
      float s1 = 0.0f;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          s1 = k.counts(j, i) ? __builtin_fmaf(h.at(j, i), h.at(j, i), s1) : s1;
      sum(s1);
      // without a row 0, which leaves the sums over rows as they are: the
      // root of a mean square and eps of 0 would not
      r1 = on ? inv_root(__builtin_fmaf(s1, inv, p.eps)) : 0.0f;
      h.unpack_anew();
    }
    // silu(gate), formed again wherever it is needed
    auto act = [&](int j, int i) { return kParts == kGated ? o.at(j, i) * sig[j][i] : 1.0f; };
    float s2 = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (kParts == kGated) sig[j][i] = Gate<T>::sigmoid(o.at(j, i));
        if constexpr (kDz) {
          y[j][i] = res.at(j, i);
          if constexpr (kParts != kNone)
            y[j][i] = __builtin_fmaf(h.at(j, i) * r1, w1[j][i] * act(j, i), y[j][i]);
          const float yc = k.counts(j, i) ? y[j][i] : 0.0f;
          s2 = __builtin_fmaf(yc, y[j][i], s2);
          m2 = __builtin_fmaf(dz.at(j, i) * w2[j][i], yc, m2);
        }
      }
    float r2 = 0.0f, k2 = 0.0f;
    if constexpr (kDz) {
      sum(s2, m2, true);
      r2 = on ? inv_root(__builtin_fmaf(s2, inv, p.eps)) : 0.0f;
      k2 = r2 * (r2 * (m2 * inv));   // r2 alone squared overflows for tiny rows
      dz.unpack_anew();
    }
    if constexpr (kParts != kNone) h.unpack_anew();
    if constexpr (kParts == kGated) o.unpack_anew();
    float m1 = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // y holds G from here on
        if constexpr (kDz) {
          const float z = dz.at(j, i);
          a2[j][i] = __builtin_fmaf(z * r2, y[j][i], a2[j][i]);
          y[j][i] =
              __builtin_fmaf(r2, __builtin_fmaf(-k2, y[j][i], z * w2[j][i]), dy.at(j, i));
        } else {
          y[j][i] = dy.at(j, i);
        }
        if constexpr (kParts != kNone)
          m1 = k.counts(j, i)
                   ? __builtin_fmaf(y[j][i] * (w1[j][i] * act(j, i)), h.at(j, i), m1)
                   : m1;
      }
    if (on) piece_store(q.dres + r * q.dress, k, y);
    if constexpr (kParts != kNone) {
      sum(m1);
      h.unpack_anew();
      o.unpack_anew();
      const float k1 = r1 * (r1 * (m1 * inv));
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = h.at(j, i);
          const float n = x * r1;
          const float silu = act(j, i);
          a1[j][i] = __builtin_fmaf(y[j][i] * silu, n, a1[j][i]);
          const float gw = y[j][i] * w1[j][i];
          if constexpr (kParts == kGated) {
            const float s = sig[j][i];   // the slope of silu: s (1 + gate (1 - s))
            sig[j][i] = gw * n * (s * __builtin_fmaf(o.at(j, i), 1.0f - s, 1.0f));
          }
          y[j][i] = r1 * __builtin_fmaf(-k1, x, gw * silu);
        }
      if (on) {
        piece_store(q.dh + r * q.dhs, k, y);
        if constexpr (kParts == kGated)
          piece_store(q.dgate + r * q.dgates, k, sig);
      }
    }
    if (q.part && ++held == kHeld) {
      flush();
      held = 0;
    }
  }
  if (!q.part) return;
  flush();
  __syncthreads();
  for (int c = threadIdx.x; c < k.C; c += kThreads<kLanes>) {
    int lane, value;
    k.place(c, lane, value);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which == 0 ? kParts == kNone : !kDz) continue;
      double s = 0.0;
      for (int g = 0; g < kRows; ++g) s += sums[which][value][g * kLanes + lane];
      q.part[((int64_t)blockIdx.x * 2 + which) * k.C + c] = (float)s;
    }
  }
}

template <typename T>
NormArgs<T> norm_args(const logmel_norm_input& in) {
  return {in.rows,
          (int)in.channels,
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

// The lanes a row takes: the fewest, in powers of two from 16, that hold it
// with one vector each (8192 fp32 channels: 1024 lanes with two), and the
// values of a vector.
struct NormShape {
  int lanes, vecs, values;
};

NormShape norm_shape(const logmel_norm_input& in) {
  const int v = in.type == LOGMEL_F32 ? 4 : 8;
  const int64_t vecs = (in.channels + v - 1) / v;
  NormShape s{16, 1, in.channels < v ? 1 : v};
  while (s.lanes < vecs && s.lanes < 1024) s.lanes *= 2;
  if (s.lanes < vecs) s.vecs = 2;
  return s;
}

// Workgroups: as many as are resident at once (the kernels' bounds on their
// registers), or one pass over the rows. Fewer leave rows waiting for memory,
// more a last round of workgroups that runs alone: 64 x 2998 x 512 bf16 with 3,
// 4, 5, 6 and 8 wavefronts per SIMD 243, 201, 191, 195 and 234 us.
int64_t norm_grid(const logmel_norm_input& in, int cus, bool backward) {
  const int lanes = norm_shape(in).lanes;
  const int threads = lanes > 256 ? lanes : 256;
  const int waves = backward ? kBackWaves : front_waves(lanes);
  const int64_t all = (in.rows + threads / lanes - 1) / (threads / lanes);
  const int64_t most = (int64_t)cus * waves * 256 / threads;
  return all < most ? all : most;
}

// f(type, parts, lanes, vecs, values) as compile-time constants.
template <typename F>
void norm_dispatch(const logmel_norm_input& in, F&& f) {
  const NormShape s = norm_shape(in);
  auto shape = [&](auto zero, auto parts) {
    using std::integral_constant;
    integral_constant<int, 1> one;
    integral_constant<int, 16 / (int)sizeof(zero)> v;
    if (s.values == 1) return f(zero, parts, integral_constant<int, 16>{}, one, one);
    if constexpr (sizeof(zero) == 4)
      if (s.vecs == 2)
        return f(zero, parts, integral_constant<int, 1024>{}, integral_constant<int, 2>{}, v);
    switch (s.lanes) {
      case 16: return f(zero, parts, integral_constant<int, 16>{}, one, v);
      case 32: return f(zero, parts, integral_constant<int, 32>{}, one, v);
      case 64: return f(zero, parts, integral_constant<int, 64>{}, one, v);
      case 128: return f(zero, parts, integral_constant<int, 128>{}, one, v);
      case 256: return f(zero, parts, integral_constant<int, 256>{}, one, v);
      case 512: return f(zero, parts, integral_constant<int, 512>{}, one, v);
      default: return f(zero, parts, integral_constant<int, 1024>{}, one, v);
    }
  };
  auto parts = [&](auto zero) {
    if (!in.d_h) return shape(zero, std::integral_constant<int, kNone>{});
    if (!in.d_gate) return shape(zero, std::integral_constant<int, kNorm>{});
    return shape(zero, std::integral_constant<int, kGated>{});
  };
  if (in.type == LOGMEL_F32)
    parts(0.0f);
  else if (in.type == LOGMEL_F16)
    parts((f16_t)0.0f);
  else
    parts((bf16_t)0.0f);
}


}  // namespace logmel

int64_t logmel_norm_workspace(const logmel_norm_input& in, int cus) {
  return logmel::norm_grid(in, cus, true) * 2 * in.channels * 4;
}

hipError_t logmel_launch_norm(const logmel_norm_input& in, void* y, int64_t y_stride, void* z,
                              int64_t z_stride, int cus, hipStream_t stream) {
  using namespace logmel;
  norm_dispatch(in, [&](auto zero, auto parts, auto lanes, auto vecs, auto values) {
    using T = decltype(zero);
    const NormOut<T> out{static_cast<T*>(y), y_stride, static_cast<T*>(z), z_stride};
    logmel_norm_kernel<T, parts.value, lanes.value, vecs.value, values.value>
        <<<(unsigned)norm_grid(in, cus, false), kThreads<lanes.value>, 0, stream>>>(
            norm_args<T>(in), out);
  });
  return hipGetLastError();
}

hipError_t logmel_launch_norm_backward(const logmel_norm_input& in, const logmel_norm_grad& g,
                                       void* ws, int cus, hipStream_t stream) {
  using namespace logmel;
  const int64_t grid = norm_grid(in, cus, true);
  const PartSums sums[3] = {{g.d_dw_post, 0, in.d_scale},
                            {g.d_dscale, 0, in.d_w_post},
                            {g.d_dw_pre, 1, nullptr}};
  const bool params = g.d_dw_post || g.d_dscale || g.d_dw_pre;
  float* part = params ? static_cast<float*>(ws) : nullptr;
  if (grid)
    norm_dispatch(in, [&](auto zero, auto parts, auto lanes, auto vecs, auto values) {
      using T = decltype(zero);
      const NormGradArgs<T> q{static_cast<const T*>(g.d_dy),
                              g.dy_stride,
                              static_cast<const T*>(g.d_dz),
                              g.dz_stride,
                              static_cast<T*>(g.d_dres),
                              g.dres_stride,
                              static_cast<T*>(g.d_dh),
                              g.dh_stride,
                              static_cast<T*>(g.d_dgate),
                              g.dgate_stride,
                              part};
      auto go = [&](auto has_dz) {
        logmel_norm_backward_kernel<T, parts.value, has_dz.value, lanes.value, vecs.value,
                                    values.value>
            <<<(unsigned)grid, kThreads<lanes.value>, 0, stream>>>(norm_args<T>(in), q);
      };
      g.d_dz ? go(std::true_type{}) : go(std::false_type{});
    });
  if (params) return logmel_launch_part_sums(part, grid, 2, in.channels, sums, stream);
  return hipGetLastError();
}
