// The group norm with an activation, channels last, and its gradient (gfx950):
//   n = (x - mean) / sqrt(var + eps) * weight + bias,  y = act(n) * silu(gate),
// mean and var over a group's channels of one row, or of all rows of a sequence.
//
// Row by row, a group is held by kLanes lanes from its one read to its writes,
// as the block norm's rows are. Over sequences the rows are cut into parts,
// whatever sequences they hold: a first kernel sums each part's pieces of
// sequences, one wavefront per sequence and group joins the pieces of those that
// lie in several parts, and a last kernel reads the rows again.
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
  float* stats;         // [n_seq][groups][2]: mean, 1 / sqrt(var + eps)
  // the gradient's
  const T* dy;
  int64_t dys;
  T* dx;
  int64_t dxs;
  T* dgate;
  int64_t dgs;
  float* sums;          // [n_seq][groups][2]: means of dn w and dn w xh
  float* part;          // [parts][2][channels]: sums of dn xh and dn; or null
  // over sequences
  double* pieces;       // [parts][2][groups][2]: of the sequence that enters a part, of the one
                        // that starts in it and leaves it
  double* wide;         // [parts][2][channels]: `part` while its pieces are added, of groups
                        // of more vectors than a workgroup has lanes
  int64_t part_rows;
};

// n of a centred value, and what follows from it. T: whose sigmoid. Over sequences
// 2-byte rows take theirs, as their gates do (64 x 2998 x 32 x 16 bf16 with gradient
// 355 us, 364 with that of fp32); rows by themselves wait for memory and take that
// of fp32.
template <typename T>
struct Act {
  float act, slope;
  template <bool kSlope>
  static __device__ __forceinline__ Act of(float n, int silu) {
    Act a{n, 1.0f};
    if (silu) {
      const float s = Gate<T>::sigmoid(n);
      a.act = n * s;
      if (kSlope) a.slope = s * __builtin_fmaf(n, 1.0f - s, 1.0f);
    }
    return a;
  }
};

// ------------------------------------------------------------ row by row
//
// Memory bounds both directions: 64 x 2998 x 8 x 64 bf16 with its gate 116 us (589 MB,
// 5.1 TB/s) and the gradient 187 us (982 MB, 5.2 TB/s).

template <int kLanes>
constexpr int kThreads = kLanes > 256 ? kLanes : 256;
constexpr int kHeld = 16;   // rows of a lane that are summed in fp32

// Sums over a group's lanes, one or two at once; groups of several wavefronts
// meet in LDS, on two slots in turn (a slot is written again only after the
// barrier of the other, which comes after its last read).
template <int kLanes>
struct GroupSum {
  static constexpr int kWaves = kThreads<kLanes> / 64;
  float (*slots)[2][kWaves];
  int turn = 0;

  template <bool kTwo>
  __device__ __forceinline__ void operator()(float& a, float& b) {
    constexpr int kIn = kLanes < 64 ? kLanes : 64;
    a = lane_sum<kIn>(a);
    if (kTwo) b = lane_sum<kIn>(b);
    if constexpr (kLanes > 64) {
      const int wave = threadIdx.x >> 6;
      constexpr int kPer = kLanes / 64;
      const int w0 = wave / kPer * kPer;
      if ((threadIdx.x & 63) == 0) {
        slots[turn][0][wave] = a;
        if (kTwo) slots[turn][1][wave] = b;
      }
      __syncthreads();
      a = 0.0f;
      if (kTwo) b = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        a += slots[turn][0][w0 + i];
        if (kTwo) b += slots[turn][1][w0 + i];
      }
      turn ^= 1;
    }
  }
  __device__ __forceinline__ void one(float& a) {
    float b = 0.0f;
    this->template operator()<false>(a, b);
  }
  __device__ __forceinline__ void two(float& a, float& b) { this->template operator()<true>(a, b); }
};

// Where this lane works: its group, the rows of the workgroup's step it takes,
// and the channels it holds of each: vector j is columns c[j] on, of which the
// first skip[j] are the vector's before (the last vector of a width that V does
// not divide is shifted back to end with the group).
template <int kLanes, int kVecs, int V>
struct Cell {
  int group, row, per;   // per: rows of a workgroup at a time
  int64_t base;          // the group's first column
  int c[kVecs], skip[kVecs];
  bool on, has[kVecs];

  __device__ Cell(int groups, int width) {
    constexpr int kCells = kThreads<kLanes> / kLanes;
    int cell = threadIdx.x / kLanes;
    if (kLanes >= 64) cell = __builtin_amdgcn_readfirstlane(cell);
    if (groups <= kCells) {
      per = kCells / groups;
      row = cell / groups;
      group = cell - row * groups;
      on = row < per;
    } else {
      per = 1;
      row = 0;
      group = blockIdx.y * kCells + cell;
      on = group < groups;
    }
    if (!on) group = 0;
    base = (int64_t)group * width;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int first = (j * kLanes + (int)(threadIdx.x & (kLanes - 1))) * V;
      has[j] = on && first < width;
      c[j] = first + V <= width ? first : width - V;
      skip[j] = first - c[j];
    }
  }
  __device__ __forceinline__ bool counts(int j, int i) const { return has[j] && i >= skip[j]; }
};

template <typename T, int kLanes, int kVecs, int V>
struct Piece {
  using C = Cell<kLanes, kVecs, V>;
  Packed<T, V> v[kVecs];
  __device__ __forceinline__ void load(const T* row, const C& k, bool on) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      v[j] = Packed<T, V>{};
      if (on && k.has[j]) v[j] = row_load<T, V>(row + k.base + k.c[j]);
    }
  }
  __device__ __forceinline__ float at(int j, int i) const { return (float)v[j].v[i]; }
};

template <typename T, int kLanes, int kVecs, int V>
__device__ __forceinline__ void piece_store(T* row, const Cell<kLanes, kVecs, V>& k,
                                            const float (&x)[kVecs][V]) {
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (k.has[j]) row_store<T, V>(row + k.base + k.c[j], x[j]);
}

template <int kLanes, int kVecs, int V>
__device__ __forceinline__ void load_params(float (&r)[kVecs][V], const float* p, float absent,
                                            const Cell<kLanes, kVecs, V>& k) {
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[j][i] = absent;
    if (!p || !k.has[j]) continue;
    const auto v = row_load<float, V>(p + k.base + k.c[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) r[j][i] = v.v[i];
  }
}

// x becomes x - mean, and the result 1 / sqrt(var + eps): the sum; then, of what
// is left, the sum, which holds what the first one rounded away (a mean may be
// large against what is left), and the sum of squares.
template <int kLanes, int kVecs, int V>
__device__ __forceinline__ float centre(float (&x)[kVecs][V], const Cell<kLanes, kVecs, V>& k,
                                        GroupSum<kLanes>& sum, float inv, float eps) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) s += k.counts(j, i) ? x[j][i] : 0.0f;
  sum.one(s);
  const float mean = s * inv;
  float q = 0.0f, rest = 0.0f;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[j][i] -= mean;
      if (k.counts(j, i)) {
        rest += x[j][i];
        q = __builtin_fmaf(x[j][i], x[j][i], q);
      }
    }
  sum.two(q, rest);
  rest *= inv;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) x[j][i] -= rest;
  const float var = __builtin_fmaf(q, inv, -rest * rest);
  return inv_root((var < 0.0f ? 0.0f : var) + eps);
}

template <typename T, bool kGate, int kLanes, int kVecs, int V>
__global__ __launch_bounds__(kThreads<kLanes>) void logmel_group_rows_kernel(GroupArgs<T> p) {
  using P = Piece<T, kLanes, kVecs, V>;
  __shared__ float slots[2][2][kThreads<kLanes> / 64];
  GroupSum<kLanes> sum{slots};
  const typename P::C k(p.groups, p.width);
  const float inv = 1.0f / (float)p.width;
  const int64_t step = (int64_t)gridDim.x * k.per;
  int64_t r = (int64_t)blockIdx.x * k.per + k.row;
  P x, o;
  auto load = [&](int64_t row) {
    x.load(p.x + row * p.xs, k, row < p.rows);
    if constexpr (kGate) o.load(p.gate + row * p.gs, k, row < p.rows);
  };
  load(r);   // on its way before the parameters are waited for
  float w[kVecs][V], b[kVecs][V];
  load_params(w, p.weight, 1.0f, k);
  load_params(b, p.bias, 0.0f, k);
  // the workgroup's rows together: barriers are met by all of it
  for (int64_t first = (int64_t)blockIdx.x * k.per; first < p.rows; first += step, r += step) {
    float y[kVecs][V], gated[kVecs][V];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[j][i] = x.at(j, i);
        if constexpr (kGate) gated[j][i] = o.at(j, i) * Gate<T>::sigmoid(o.at(j, i));
      }
    if (first + step < p.rows) load(r + step);
    const float root = centre(y, k, sum, inv, p.eps);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = __builtin_fmaf(y[j][i] * root, w[j][i], b[j][i]);
        y[j][i] = Act<float>::of<false>(n, p.silu).act;
        if constexpr (kGate) y[j][i] *= gated[j][i];
      }
    if (k.on && r < p.rows) piece_store(p.y + r * p.ys, k, y);
  }
}

// The gradient, with dn = dy silu(gate) act'(n) and q = dn w:
//   dx = root (q - mean(q) - xh mean(q xh)),  dgate = dy act silu'(gate),
//   dweight = sum dn xh,  dbias = sum dn.
// The sums over rows stay in a lane's registers for kHeld rows, then go to fp64
// places of its own in LDS; at the end each workgroup writes one part.
template <typename T, bool kGate, int kLanes, int kVecs, int V>
__global__ __launch_bounds__(kThreads<kLanes>, 4) void logmel_group_rows_back_kernel(
    GroupArgs<T> p) {
  using P = Piece<T, kLanes, kVecs, V>;
  constexpr int kAll = kThreads<kLanes>;
  __shared__ float slots[2][2][kAll / 64];
  __shared__ double sums[2][kVecs * V][kAll];
  GroupSum<kLanes> sum{slots};
  const typename P::C k(p.groups, p.width);
  const float inv = 1.0f / (float)p.width;
  const int64_t step = (int64_t)gridDim.x * k.per;
  int64_t r = (int64_t)blockIdx.x * k.per + k.row;
  float w[kVecs][V], b[kVecs][V], a1[kVecs][V], a2[kVecs][V];
  load_params(w, p.weight, 1.0f, k);
  load_params(b, p.bias, 0.0f, k);
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) a1[j][i] = a2[j][i] = 0.0f;
  if (p.part)
#pragma unroll
    for (int n = 0; n < kVecs * V; ++n) sums[0][n][threadIdx.x] = sums[1][n][threadIdx.x] = 0.0;
  auto flush = [&] {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sums[0][j * V + i][threadIdx.x] += (double)a1[j][i];
        sums[1][j * V + i][threadIdx.x] += (double)a2[j][i];
        a1[j][i] = a2[j][i] = 0.0f;
      }
  };
  int held = 0;
  for (int64_t first = (int64_t)blockIdx.x * k.per; first < p.rows; first += step, r += step) {
    const bool on = k.on && r < p.rows;
    P x, o, d;
    x.load(p.x + r * p.xs, k, on);
    if constexpr (kGate) o.load(p.gate + r * p.gs, k, on);
    d.load(p.dy + r * p.dys, k, on);
    float h[kVecs][V], q[kVecs][V], dg[kVecs][V];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) h[j][i] = x.at(j, i);
    float root = centre(h, k, sum, inv, p.eps);
    root = on ? root : 0.0f;   // without a row nothing is added below
    float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[j][i] *= root;
        const float n = __builtin_fmaf(h[j][i], w[j][i], b[j][i]);
        const Act<float> a = Act<float>::of<true>(n, p.silu);
        float dn = d.at(j, i) * a.slope;
        if constexpr (kGate) {
          const float g = o.at(j, i), s = Gate<T>::sigmoid(g);
          dg[j][i] = d.at(j, i) * a.act * (s * __builtin_fmaf(g, 1.0f - s, 1.0f));
          dn *= g * s;
        }
        a1[j][i] = __builtin_fmaf(dn, h[j][i], a1[j][i]);
        a2[j][i] += dn;
        q[j][i] = dn * w[j][i];
        if (k.counts(j, i)) {
          m1 += q[j][i];
          m2 = __builtin_fmaf(q[j][i], h[j][i], m2);
        }
      }
    if constexpr (kGate)
      if (on) piece_store(p.dgate + r * p.dgs, k, dg);
    sum.two(m1, m2);
    m1 *= inv, m2 *= inv;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) q[j][i] = root * __builtin_fmaf(-h[j][i], m2, q[j][i] - m1);
    if (on) piece_store(p.dx + r * p.dxs, k, q);
    if (p.part && ++held == kHeld) {
      flush();
      held = 0;
    }
  }
  if (!p.part) return;
  flush();
  __syncthreads();
  // the workgroup's groups, channel by channel, over its rows
  constexpr int kCells = kAll / kLanes;
  const bool whole = p.groups <= kCells;
  const int g0 = whole ? 0 : blockIdx.y * kCells;
  const int ng = whole ? p.groups : p.groups - g0 < kCells ? p.groups - g0 : kCells;
  for (int c = threadIdx.x; c < ng * p.width; c += kAll) {
    const int g = c / p.width, at = c - g * p.width, vec = at / V;
    const int from = vec * V + V <= p.width ? vec * V : p.width - V;
    const int lane = vec % kLanes, value = vec / kLanes * V + at - from;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      double s = 0.0;
      for (int row = 0; row < k.per; ++row)
        s += sums[which][value][(row * (whole ? p.groups : 0) + g) * kLanes + lane];
      p.part[((int64_t)blockIdx.x * 2 + which) * p.channels + (int64_t)g0 * p.width + c] =
          (float)s;
    }
  }
}

// ---------------------------------------------------------- over sequences
//
// x is read twice forward, x and dy twice for the gradient: a clip's rows do not fit
// one workgroup's registers. Of 64 x 2998 x 32 x 16 bf16 (196 MB an operand) the
// passes that write are bound by memory (69 us, 5.7 TB/s; with the gradient 107 us, 5.5),
// the sums of the gradient by the activation's slope (110 us, 3.6 TB/s), the
// statistics by neither alone (55 us, 3.6 TB/s: more rows on their way, more or
// smaller parts changed nothing).

// How many of off[0 .. n] are at or before row: 64 probes a step, the whole
// wavefront together.
__device__ __forceinline__ int64_t starts_to(const int64_t* off, int64_t n, int64_t row) {
  int64_t lo = 0, hi = n + 1;   // the answer is in [lo, hi]
  while (hi > lo) {
    const int64_t gap = (hi - lo + 63) / 64;
    const int64_t at = lo + gap * ((threadIdx.x & 63) + 1) - 1;
    const bool yes = at < hi && off[at] <= row;
    const int64_t k = __popcll(__ballot(yes));
    lo += k * gap;
    hi = lo + gap - 1 < hi ? lo + gap - 1 : hi;
  }
  return lo;
}

constexpr int kWork = 256;

// The channels of a workgroup over sequences: whole groups, as vectors of V
// channels that lie in one group; as many rows side by side as there is room.
template <int V>
struct Columns {
  int vg;        // vectors of a group
  int groups;    // of this workgroup, from g0 on
  int g0, vecs, lanes;
  __device__ Columns(int all, int width) {
    vg = width / V;
    int most = kWork / vg;
    most = most < 1 ? 1 : most;
    const int sets = (all + most - 1) / most;
    most = (all + sets - 1) / sets;   // even ones
    g0 = blockIdx.y * most;
    groups = all - g0 < most ? all - g0 : most;
    groups = groups < 0 ? 0 : groups;
    vecs = groups * vg;
    lanes = vecs ? kWork / vecs : 1;
    lanes = lanes < 1 ? 1 : lanes;
  }
};

int group_sets(int groups, int width, int v) {
  const int most = kWork / (width / v) < 1 ? 1 : kWork / (width / v);
  return (groups + most - 1) / most;
}

// The sequence that the workgroup's part begins in or before.
template <typename T>
__device__ __forceinline__ int64_t first_piece(const GroupArgs<T>& p) {
  const int64_t i = starts_to(p.off, p.n_seq, (int64_t)blockIdx.x * p.part_rows) - 1;
  return i < 0 ? 0 : i;
}

// Calls f(sequence, from, to, starts, ends) for each piece of a sequence in the
// workgroup's part, from sequence i on.
template <typename T, typename F>
__device__ __forceinline__ void for_pieces(const GroupArgs<T>& p, int64_t i, F&& f) {
  const int64_t r0 = (int64_t)blockIdx.x * p.part_rows;
  int64_t r1 = r0 + p.part_rows;
  r1 = r1 < p.rows ? r1 : p.rows;
  int64_t from = i < p.n_seq ? p.off[i] : r1;
  for (; i < p.n_seq && from < r1; ++i) {
    const int64_t to = p.off[i + 1];
    const int64_t a = from > r0 ? from : r0, b = to < r1 ? to : r1;
    if (a < b) f(i, a, b, from >= r0, to <= r1);
    from = to;
  }
}

// Two sums of fp64 over each group's values, as thread g < groups receives them.
template <int V>
__device__ __forceinline__ void group_sums(const Columns<V>& k, double (&red)[kWork][2], double& a,
                                           double& b) {
  const int tid = threadIdx.x;
  red[tid][0] = a;
  red[tid][1] = b;
  __syncthreads();
  // up to 16 threads a group take every so many-th, then one theirs
  const int room = k.groups ? kWork / k.groups : 1, per = room < 16 ? room : 16;
  const int across = k.vecs <= kWork ? k.vg : kWork;
  a = b = 0.0;
  if (tid < k.groups * per)
    for (int e = tid % per; e < k.lanes * across; e += per) {
      const int t = e / across * k.vecs + tid / per * k.vg + e % across;
      a += red[t][0];
      b += red[t][1];
    }
  __syncthreads();
  red[tid][0] = a;
  red[tid][1] = b;
  __syncthreads();
  a = b = 0.0;
  if (tid < k.groups)
    for (int j = 0; j < per; ++j) {
      a += red[tid * per + j][0];
      b += red[tid * per + j][1];
    }
  __syncthreads();
}

// Weight and bias of V channels from c on, 1 and 0 where they are absent.
template <typename T, int V>
__device__ __forceinline__ void affine_at(const GroupArgs<T>& p, int64_t c, float (&w)[V],
                                          float (&b)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) w[j] = 1.0f, b[j] = 0.0f;
  if (p.weight) {
    const auto t = row_load<float, V>(p.weight + c);
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = t.v[j];
  }
  if (p.bias) {
    const auto t = row_load<float, V>(p.bias + c);
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = t.v[j];
  }
}

constexpr int kBatch = 8;   // rows of a lane on their way at a time

// f(row, whole) for a lane's rows first, first + step, .. below to, kN at a time:
// whole (a compile-time constant): all of them are there.
template <int kN, typename F>
__device__ __forceinline__ void in_batches(int64_t first, int64_t to, int step, F&& f) {
  int64_t r = first;
  for (; r + (kN - 1) * step < to; r += kN * step) f(r, std::true_type{});
  if (r < to) f(r, std::false_type{});
}

// Each piece's sum and sum of squares: a lane's kBatch rows at a time are
// centred on their mean, summed again (what the mean's rounding left) and squared
// in fp32, and taken to moments about 0 in fp64, which keep the digits that the
// subtraction of the squared mean takes.
template <typename T, int V>
__global__ __launch_bounds__(kWork) void logmel_group_stats_kernel(GroupArgs<T> p) {
  __shared__ double red[kWork][2];
  const Columns<V> k(p.groups, p.width);
  const int64_t i0 = first_piece(p);
  const int vec = threadIdx.x % (k.vecs < kWork && k.vecs ? k.vecs : kWork);
  const int lane = k.vecs < kWork && k.vecs ? threadIdx.x / k.vecs : 0;
  for_pieces(p, i0, [&](int64_t i, int64_t from, int64_t to, bool starts, bool ends) {
    double s = 0.0, ss = 0.0;
    if (lane < k.lanes)
      for (int v = vec; v < k.vecs; v += kWork) {
        const T* x = p.x + ((int64_t)k.g0 * p.width + (int64_t)v * V);
        in_batches<kBatch>(from + lane, to, k.lanes, [&](int64_t r, auto whole) {
          Packed<T, V> q[kBatch];
          const T* xr = x + r * p.xs;
          int n = 0;
#pragma unroll
          for (int m = 0; m < kBatch; ++m) {
            const bool on = whole || r + m * k.lanes < to;
            q[m] = row_load<T, V>(xr + (on ? m * k.lanes * p.xs : 0));
            n += on;
          }
          float sum = 0.0f;
#pragma unroll
          for (int m = 0; m < kBatch; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j) sum += m < n ? (float)q[m].v[j] : 0.0f;
          const float mean = sum / (float)(n * V);
          float sq = 0.0f, rest = 0.0f;
#pragma unroll
          for (int m = 0; m < kBatch; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float d = (float)q[m].v[j] - mean;
              rest = m < n ? rest + d : rest;
              sq = m < n ? __builtin_fmaf(d, d, sq) : sq;
            }
          const double all = (double)(n * V) * (double)mean;
          s += all + (double)rest;
          ss += (double)sq + (all + 2.0 * (double)rest) * (double)mean;
        });
      }
    group_sums(k, red, s, ss);
    if ((int)threadIdx.x < k.groups) {
      const int g = k.g0 + threadIdx.x;
      if (starts && ends) {
        const double inv = 1.0 / ((double)(to - from) * p.width);
        const double mean = s * inv;
        double var = ss * inv - mean * mean;
        var = var < 0.0 ? 0.0 : var;
        float* st = p.stats + (i * p.groups + g) * 2;
        st[0] = (float)mean;
        st[1] = (float)(1.0 / sqrt(var + (double)p.eps));
      } else {
        double* d = p.pieces + (((int64_t)blockIdx.x * 2 + starts) * p.groups + g) * 2;
        d[0] = s;
        d[1] = ss;
      }
    }
  });
}

// What the pieces of a sequence in several parts come to, one wavefront for
// each and group: its statistics, or (kBack) the means of its gradient's sums.
// An empty sequence has the statistics of nothing.
template <typename T, bool kBack>
__global__ __launch_bounds__(256) void logmel_group_join_kernel(GroupArgs<T> p) {
  const int lane = threadIdx.x & 63;
  const int64_t all = p.n_seq * p.groups;
  for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < all;
       item += (int64_t)gridDim.x * 4) {
    const int64_t i = item / p.groups;
    const int g = (int)(item - i * p.groups);
    int64_t from = p.off[i], to = p.off[i + 1];
    from = from < 0 ? 0 : from;
    to = to > p.rows ? p.rows : to;
    const int64_t first = from / p.part_rows, last = (to - 1) / p.part_rows;
    if (from < to && first == last) continue;
    double a = 0.0, b = 0.0;
    if (from < to)
      for (int64_t k = first + lane; k <= last; k += 64) {
        const double* d = p.pieces + ((k * 2 + (k == first)) * p.groups + g) * 2;
        a += d[0];
        b += d[1];
      }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      a += __shfl_xor(a, d);
      b += __shfl_xor(b, d);
    }
    if (lane) continue;
    const double inv = from < to ? 1.0 / ((double)(to - from) * p.width) : 0.0;
    if constexpr (kBack) {
      p.sums[item * 2] = (float)(a * inv);
      p.sums[item * 2 + 1] = (float)(b * inv);
    } else {
      const double mean = a * inv;
      double var = b * inv - mean * mean;
      var = var < 0.0 ? 0.0 : var;
      p.stats[item * 2] = (float)mean;
      p.stats[item * 2 + 1] = (float)(1.0 / sqrt(var + (double)p.eps));
    }
  }
}

template <typename T, bool kGate, int V>
__global__ __launch_bounds__(kWork) void logmel_group_apply_kernel(GroupArgs<T> p) {
  constexpr int kRows = 4;
  const Columns<V> k(p.groups, p.width);
  const int64_t i0 = first_piece(p);
  const int vec = threadIdx.x % (k.vecs < kWork && k.vecs ? k.vecs : kWork);
  const int lane = k.vecs < kWork && k.vecs ? threadIdx.x / k.vecs : 0;
  if (lane >= k.lanes) return;
  for (int v = vec; v < k.vecs; v += kWork) {
    const int64_t c = (int64_t)k.g0 * p.width + (int64_t)v * V;
    const int g = k.g0 + v / k.vg;
    float w[V], b[V];
    affine_at(p, c, w, b);
    for_pieces(p, i0, [&](int64_t i, int64_t from, int64_t to, bool, bool) {
      const float mean = p.stats[(i * p.groups + g) * 2];
      const float root = p.stats[(i * p.groups + g) * 2 + 1];
      in_batches<kRows>(from + lane, to, k.lanes, [&](int64_t r, auto whole) {
        Packed<T, V> x[kRows], o[kRows];
        const T* xr = p.x + r * p.xs + c;
        const T* gr = kGate ? p.gate + r * p.gs + c : nullptr;
        T* yr = p.y + r * p.ys + c;
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
          const int64_t by = whole || r + m * k.lanes < to ? m * k.lanes : 0;
          x[m] = row_load<T, V>(xr + by * p.xs);
          if constexpr (kGate) o[m] = row_load<T, V>(gr + by * p.gs);
        }
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
          if (!whole && r + m * k.lanes >= to) break;
          float y[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float xh = ((float)x[m].v[j] - mean) * root;
            y[j] = Act<T>::template of<false>(__builtin_fmaf(xh, w[j], b[j]), p.silu).act;
            if constexpr (kGate) {
              const float gt = (float)o[m].v[j];
              y[j] *= gt * Gate<T>::sigmoid(gt);
            }
          }
          row_store(yr + m * k.lanes * p.ys, y);
        }
      });
    });
  }
}

// What a value gives the gradient.
template <typename T, bool kGate>
struct Back {
  float xh, dn, dgate;
  __device__ __forceinline__ Back(float x, float o, float dy, float mean, float root, float w,
                                  float b, int silu) {
    xh = (x - mean) * root;
    const Act<T> a = Act<T>::template of<true>(__builtin_fmaf(xh, w, b), silu);
    dn = dy * a.slope;
    dgate = 0.0f;
    if constexpr (kGate) {
      const float s = Gate<T>::sigmoid(o);
      dgate = dy * a.act * (s * __builtin_fmaf(o, 1.0f - s, 1.0f));
      dn *= o * s;
    }
  }
};

// Each part's sums of dn xh and dn, channel by channel, and weighted those of
// its pieces' groups. A lane's rows are summed in fp32 four at a time, then in
// fp64. kWide: of groups of more vectors than a workgroup has lanes, which go through
// theirs 256 at a time; the sums over a part's pieces, which may be as many as its
// rows, are in memory, unless one piece is the whole part.
template <typename T, bool kGate, int V, bool kWide>
__global__ __launch_bounds__(kWork) void logmel_group_back_sums_kernel(GroupArgs<T> p) {
  constexpr int kRows = 4;
  __shared__ double red[kWork][2];
  const Columns<V> k(p.groups, p.width);
  const int64_t i0 = first_piece(p);
  const int vec = threadIdx.x % (k.vecs < kWork && k.vecs ? k.vecs : kWork);
  const int lane = k.vecs < kWork && k.vecs ? threadIdx.x / k.vecs : 0;
  const int rounds = kWide ? (k.vecs + kWork - 1) / kWork : 1;
  double p1[V], p2[V];   // over the part, if not wide
  bool some = false, alone = false;   // pieces before; one that is the whole part
#pragma unroll
  for (int j = 0; j < V; ++j) p1[j] = p2[j] = 0.0;
  auto part_at = [&](int which, int v) {
    return p.part + (((int64_t)blockIdx.x * 2 + which) * p.channels +
                     (int64_t)k.g0 * p.width + (int64_t)v * V);
  };
  auto wide_at = [&](int which, int v) {
    return p.wide + (((int64_t)blockIdx.x * 2 + which) * p.channels +
                     (int64_t)k.g0 * p.width + (int64_t)v * V);
  };
  for_pieces(p, i0, [&](int64_t i, int64_t from, int64_t to, bool starts, bool ends) {
    double s1 = 0.0, s2 = 0.0;
    if (kWide)
      alone = to - from == p.part_rows || (from == (int64_t)blockIdx.x * p.part_rows && to == p.rows);
    for (int round = 0; round < rounds; ++round) {
      const int v = vec + round * kWork;
      if (lane >= k.lanes || v >= k.vecs) continue;
      const int64_t c = (int64_t)k.g0 * p.width + (int64_t)v * V;
      const int g = k.g0 + v / k.vg;
      const float mean = p.stats[(i * p.groups + g) * 2];
      const float root = p.stats[(i * p.groups + g) * 2 + 1];
      float w[V], b[V];
      affine_at(p, c, w, b);
      double d1[V], d2[V];
#pragma unroll
      for (int j = 0; j < V; ++j) d1[j] = d2[j] = 0.0;
      in_batches<kRows>(from + lane, to, k.lanes, [&](int64_t r, auto whole) {
        Packed<T, V> x[kRows], o[kRows], d[kRows];
        const T* xr = p.x + r * p.xs + c;
        const T* dr = p.dy + r * p.dys + c;
        const T* gr = kGate ? p.gate + r * p.gs + c : nullptr;
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
          const int64_t by = whole || r + m * k.lanes < to ? m * k.lanes : 0;
          x[m] = row_load<T, V>(xr + by * p.xs);
          d[m] = row_load<T, V>(dr + by * p.dys);
          if constexpr (kGate) o[m] = row_load<T, V>(gr + by * p.gs);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float a1 = 0.0f, a2 = 0.0f;
#pragma unroll
          for (int m = 0; m < kRows; ++m) {
            const Back<T, kGate> t((float)x[m].v[j], kGate ? (float)o[m].v[j] : 0.0f,
                                   (float)d[m].v[j], mean, root, w[j], b[j], p.silu);
            const bool on = whole || r + m * k.lanes < to;
            a1 = on ? __builtin_fmaf(t.dn, t.xh, a1) : a1;
            a2 = on ? a2 + t.dn : a2;
          }
          d1[j] += (double)a1;
          d2[j] += (double)a2;
        }
      });
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s1 += (double)w[j] * d2[j];   // of q
        s2 += (double)w[j] * d1[j];   // of q xh
        if (!kWide) {
          p1[j] += d1[j];
          p2[j] += d2[j];
        } else if (p.part && alone) {
          part_at(0, v)[j] = (float)d1[j];
          part_at(1, v)[j] = (float)d2[j];
        } else if (p.part) {
          wide_at(0, v)[j] = some ? wide_at(0, v)[j] + d1[j] : d1[j];
          wide_at(1, v)[j] = some ? wide_at(1, v)[j] + d2[j] : d2[j];
        }
      }
    }
    some = true;
    group_sums(k, red, s1, s2);
    if ((int)threadIdx.x < k.groups) {
      const int g = k.g0 + threadIdx.x;
      if (starts && ends) {
        const double inv = 1.0 / ((double)(to - from) * p.width);
        float* st = p.sums + (i * p.groups + g) * 2;
        st[0] = (float)(s1 * inv);
        st[1] = (float)(s2 * inv);
      } else {
        double* d = p.pieces + (((int64_t)blockIdx.x * 2 + starts) * p.groups + g) * 2;
        d[0] = s1;
        d[1] = s2;
      }
    }
  });
  if (!p.part) return;
  if constexpr (kWide) {
    for (int v = vec; v < k.vecs && !alone; v += kWork)
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int j = 0; j < V; ++j)
          part_at(which, v)[j] = some ? (float)wide_at(which, v)[j] : 0.0f;
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    __syncthreads();
    red[threadIdx.x][0] = p1[j];
    red[threadIdx.x][1] = p2[j];
    __syncthreads();
    if ((int)threadIdx.x >= k.vecs) continue;
    double a = 0.0, b = 0.0;
    for (int l = 0; l < k.lanes; ++l) {
      a += red[l * k.vecs + threadIdx.x][0];
      b += red[l * k.vecs + threadIdx.x][1];
    }
    part_at(0, threadIdx.x)[j] = (float)a;
    part_at(1, threadIdx.x)[j] = (float)b;
  }
}

template <typename T, bool kGate, int V>
__global__ __launch_bounds__(kWork) void logmel_group_dx_kernel(GroupArgs<T> p) {
  constexpr int kRows = 4;
  const Columns<V> k(p.groups, p.width);
  const int64_t i0 = first_piece(p);
  const int vec = threadIdx.x % (k.vecs < kWork && k.vecs ? k.vecs : kWork);
  const int lane = k.vecs < kWork && k.vecs ? threadIdx.x / k.vecs : 0;
  if (lane >= k.lanes) return;
  for (int v = vec; v < k.vecs; v += kWork) {
    const int64_t c = (int64_t)k.g0 * p.width + (int64_t)v * V;
    const int g = k.g0 + v / k.vg;
    float w[V], b[V];
    affine_at(p, c, w, b);
    for_pieces(p, i0, [&](int64_t i, int64_t from, int64_t to, bool, bool) {
      const int64_t at = (i * p.groups + g) * 2;
      const float mean = p.stats[at], root = p.stats[at + 1];
      const float m1 = p.sums[at], m2 = p.sums[at + 1];
      in_batches<kRows>(from + lane, to, k.lanes, [&](int64_t r, auto whole) {
        Packed<T, V> x[kRows], o[kRows], d[kRows];
        const T* xr = p.x + r * p.xs + c;
        const T* dr = p.dy + r * p.dys + c;
        const T* gr = kGate ? p.gate + r * p.gs + c : nullptr;
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
          const int64_t by = whole || r + m * k.lanes < to ? m * k.lanes : 0;
          x[m] = row_load<T, V>(xr + by * p.xs);
          d[m] = row_load<T, V>(dr + by * p.dys);
          if constexpr (kGate) o[m] = row_load<T, V>(gr + by * p.gs);
        }
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
          if (!whole && r + m * k.lanes >= to) break;
          float dx[V], dg[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const Back<T, kGate> t((float)x[m].v[j], kGate ? (float)o[m].v[j] : 0.0f,
                                   (float)d[m].v[j], mean, root, w[j], b[j], p.silu);
            dx[j] = root * __builtin_fmaf(-t.xh, m2, __builtin_fmaf(t.dn, w[j], -m1));
            dg[j] = t.dgate;
          }
          row_store(p.dx + r * p.dxs + c + m * k.lanes * p.dxs, dx);
          if constexpr (kGate) row_store(p.dgate + r * p.dgs + c + m * k.lanes * p.dgs, dg);
        }
      });
    });
  }
}

// -------------------------------------------------------------- the host's

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

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// The lanes that a group of one row takes: the fewest, in powers of two, that
// hold it with one vector each; groups narrower than a vector go value by value.
struct RowShape {
  int lanes, vecs, values;
};
RowShape row_shape(const logmel_group_norm_input& in) {
  const int width = (int)(in.channels / in.groups);
  const int v = in.type == LOGMEL_F32 ? 4 : 8;
  RowShape s{1, 1, width < v ? 1 : v};
  const int vecs = (width + s.values - 1) / s.values;
  while (s.lanes < vecs && s.lanes < 64) s.lanes *= 2;
  if (s.lanes < vecs) s.lanes = vecs <= 256 ? 256 : 1024;
  if (s.lanes < vecs) s.vecs = 2;
  return s;
}

// Workgroups: as many as are resident at once, or one pass over the rows.
dim3 row_grid(const logmel_group_norm_input& in, int cus, bool backward) {
  const RowShape s = row_shape(in);
  const int threads = s.lanes > 256 ? s.lanes : 256, cells = threads / s.lanes;
  const int64_t sets = in.groups <= cells ? 1 : ceil_div(in.groups, cells);
  const int64_t per = in.groups <= cells ? cells / in.groups : 1;
  const int64_t all = ceil_div(in.rows, per);
  int64_t most = (int64_t)cus * (backward ? 4 : 6) * 256 / threads / sets;
  most = most < 1 ? 1 : most;
  return dim3((unsigned)(all < most ? all : most), (unsigned)sets);
}

// f(type, gate, lanes, vecs, values) as compile-time constants.
template <typename F>
void row_dispatch(const logmel_group_norm_input& in, F&& f) {
  using std::integral_constant;
  const RowShape s = row_shape(in);
  auto shape = [&](auto zero, auto gate) {
    integral_constant<int, 1> one;
    integral_constant<int, 16 / (int)sizeof(zero)> v;
    auto lanes = [&](auto n, auto vecs, auto values) { f(zero, gate, n, vecs, values); };
    if (s.values == 1) {
      switch (s.lanes) {
        case 1: return lanes(one, one, one);
        case 2: return lanes(integral_constant<int, 2>{}, one, one);
        case 4: return lanes(integral_constant<int, 4>{}, one, one);
        default: return lanes(integral_constant<int, 8>{}, one, one);
      }
    }
    if constexpr (sizeof(zero) == 4)
      if (s.vecs == 2)
        return lanes(integral_constant<int, 1024>{}, integral_constant<int, 2>{}, v);
    switch (s.lanes) {
      case 1: return lanes(one, one, v);
      case 2: return lanes(integral_constant<int, 2>{}, one, v);
      case 4: return lanes(integral_constant<int, 4>{}, one, v);
      case 8: return lanes(integral_constant<int, 8>{}, one, v);
      case 16: return lanes(integral_constant<int, 16>{}, one, v);
      case 32: return lanes(integral_constant<int, 32>{}, one, v);
      case 64: return lanes(integral_constant<int, 64>{}, one, v);
      case 256: return lanes(integral_constant<int, 256>{}, one, v);
      default: return lanes(integral_constant<int, 1024>{}, one, v);
    }
  };
  auto gate = [&](auto zero) {
    in.d_gate ? shape(zero, std::true_type{}) : shape(zero, std::false_type{});
  };
  if (in.type == LOGMEL_F32)
    gate(0.0f);
  else if (in.type == LOGMEL_F16)
    gate((f16_t)0.0f);
  else
    gate((bf16_t)0.0f);
}

// Over sequences: vectors of 16 bytes where they divide a group, else single
// values; parts enough to fill the card four times, of 64 rows at least.
int seq_values(const logmel_group_norm_input& in) {
  const int v = in.type == LOGMEL_F32 ? 4 : 8;
  return in.channels / in.groups % v ? 1 : v;
}
bool seq_wide(const logmel_group_norm_input& in) {
  return in.channels / in.groups / seq_values(in) > kWork;
}
int64_t part_rows_of(const logmel_group_norm_input& in, int cus) {
  const int64_t sets =
      group_sets((int)in.groups, (int)(in.channels / in.groups), seq_values(in));
  const int64_t rows = ceil_div(in.rows * sets, (int64_t)cus * 4);
  return rows < 64 ? 64 : rows;
}

// Where a call over sequences has what in its workspace: pieces first, then in this
// order.
struct SeqSpace {
  int64_t parts, pieces, stats, wide, part, bytes;
};
SeqSpace seq_space(const logmel_group_norm_input& in, bool backward, int cus) {
  SeqSpace s{};
  s.parts = ceil_div(in.rows, part_rows_of(in, cus));
  s.pieces = s.parts * in.groups * 32;
  s.stats = in.n_seq * in.groups * 8;   // forward: statistics nobody asked for; backward: sums
  s.wide = backward && seq_wide(in) ? s.parts * in.channels * 16 : 0;
  s.part = backward ? s.parts * in.channels * 8 : 0;
  s.bytes = s.pieces + s.stats + s.wide + s.part;
  return s;
}

template <typename F>
void seq_dispatch(const logmel_group_norm_input& in, F&& f) {
  using std::integral_constant;
  auto values = [&](auto zero, auto gate) {
    if (seq_values(in) == 1)
      f(zero, gate, integral_constant<int, 1>{});
    else
      f(zero, gate, integral_constant<int, 16 / (int)sizeof(zero)>{});
  };
  auto gate = [&](auto zero) {
    in.d_gate ? values(zero, std::true_type{}) : values(zero, std::false_type{});
  };
  if (in.type == LOGMEL_F32)
    gate(0.0f);
  else if (in.type == LOGMEL_F16)
    gate((f16_t)0.0f);
  else
    gate((bf16_t)0.0f);
}

unsigned join_grid(const logmel_group_norm_input& in) {
  const int64_t n = ceil_div(in.n_seq * in.groups, 4);
  return (unsigned)(n < (1 << 20) ? n : 1 << 20);
}

}  // namespace
}  // namespace logmel

int64_t logmel_group_workspace(const logmel_group_norm_input& in, int backward, int cus) {
  using namespace logmel;
  if (in.d_seq_offsets) return in.n_seq ? seq_space(in, backward, cus).bytes : 0;
  return backward ? row_grid(in, cus, true).x * 2 * in.channels * 4 : 0;
}

hipError_t logmel_launch_group(const logmel_group_norm_input& in, void* y, int64_t y_stride,
                               float* stats, void* ws, int cus, hipStream_t stream) {
  using namespace logmel;
  if (!in.d_seq_offsets) {
    row_dispatch(in, [&](auto zero, auto gate, auto lanes, auto vecs, auto values) {
      using T = decltype(zero);
      GroupArgs<T> p = group_args<T>(in);
      p.y = static_cast<T*>(y);
      p.ys = y_stride;
      logmel_group_rows_kernel<T, gate.value, lanes.value, vecs.value, values.value>
          <<<row_grid(in, cus, false), kThreads<lanes.value>, 0, stream>>>(p);
    });
    return hipGetLastError();
  }
  const SeqSpace s = seq_space(in, false, cus);
  seq_dispatch(in, [&](auto zero, auto gate, auto values) {
    using T = decltype(zero);
    GroupArgs<T> p = group_args<T>(in);
    p.y = static_cast<T*>(y);
    p.ys = y_stride;
    p.pieces = static_cast<double*>(ws);
    p.stats = stats ? stats : reinterpret_cast<float*>(static_cast<char*>(ws) + s.pieces);
    p.part_rows = part_rows_of(in, cus);
    const dim3 grid((unsigned)s.parts, (unsigned)group_sets(p.groups, p.width, values.value));
    if (s.parts) logmel_group_stats_kernel<T, values.value><<<grid, kWork, 0, stream>>>(p);
    logmel_group_join_kernel<T, false><<<join_grid(in), 256, 0, stream>>>(p);
    if (s.parts)
      logmel_group_apply_kernel<T, gate.value, values.value><<<grid, kWork, 0, stream>>>(p);
  });
  return hipGetLastError();
}

hipError_t logmel_launch_group_backward(const logmel_group_norm_input& in, const float* stats,
                                        const logmel_group_norm_grad& g, void* ws, int cus,
                                        hipStream_t stream) {
  using namespace logmel;
  const bool params = g.d_dweight || g.d_dbias;
  auto fill = [&](auto& p) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p.x)>>;
    p.stats = const_cast<float*>(stats);
    p.dy = static_cast<const T*>(g.d_dy);
    p.dys = g.dy_stride;
    p.dx = static_cast<T*>(g.d_dx);
    p.dxs = g.dx_stride;
    p.dgate = static_cast<T*>(g.d_dgate);
    p.dgs = g.dgate_stride;
  };
  float* part = nullptr;
  int64_t parts = 0;
  if (!in.d_seq_offsets) {
    part = static_cast<float*>(ws);
    const dim3 grid = row_grid(in, cus, true);
    parts = grid.x;
    if (parts)
      row_dispatch(in, [&](auto zero, auto gate, auto lanes, auto vecs, auto values) {
        using T = decltype(zero);
        GroupArgs<T> p = group_args<T>(in);
        fill(p);
        p.part = params ? part : nullptr;
        logmel_group_rows_back_kernel<T, gate.value, lanes.value, vecs.value, values.value>
            <<<grid, kThreads<lanes.value>, 0, stream>>>(p);
      });
  } else if (in.n_seq) {
    const SeqSpace s = seq_space(in, true, cus);
    char* at = static_cast<char*>(ws);
    part = reinterpret_cast<float*>(at + s.pieces + s.stats + s.wide);
    parts = s.parts;
    if (parts)
      seq_dispatch(in, [&](auto zero, auto gate, auto values) {
        using T = decltype(zero);
        GroupArgs<T> p = group_args<T>(in);
        fill(p);
        p.pieces = reinterpret_cast<double*>(at);
        p.sums = reinterpret_cast<float*>(at + s.pieces);
        p.part = params ? part : nullptr;
        p.wide = reinterpret_cast<double*>(at + s.pieces + s.stats);
        p.part_rows = part_rows_of(in, cus);
        const dim3 grid((unsigned)s.parts, (unsigned)group_sets(p.groups, p.width, values.value));
        if (seq_wide(in))
          logmel_group_back_sums_kernel<T, gate.value, values.value, true>
              <<<grid, kWork, 0, stream>>>(p);
        else
          logmel_group_back_sums_kernel<T, gate.value, values.value, false>
              <<<grid, kWork, 0, stream>>>(p);
        logmel_group_join_kernel<T, true><<<join_grid(in), 256, 0, stream>>>(p);
        logmel_group_dx_kernel<T, gate.value, values.value><<<grid, kWork, 0, stream>>>(p);
      });
  }
  if (params) {
    const PartSums out[3] = {
        {g.d_dweight, 0, nullptr}, {g.d_dbias, 1, nullptr}, {nullptr, 0, nullptr}};
    return logmel_launch_part_sums(part, parts, 2, in.channels, out, stream);
  }
  return hipGetLastError();
}
