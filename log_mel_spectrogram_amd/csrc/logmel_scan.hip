// The gated scan over packed sequences and its gradient (gfx950):
//   a = sigmoid(gate + bias), u = 1 - a;  h_t = a_t h_{t-1} + u_t x_t.
//
// A step is an affine map of the state, h -> a h + b, and affine maps compose:
// the map of a run of rows is (product of the a, the run's recurrence from
// zero). So rows can be worked side by side and joined afterwards, and where
// there are enough sequences nothing need be joined at all. Three ways, chosen
// by scan_split: a lane per sequence, a workgroup per sequence, or parts of
// the rows whatever sequences they hold.
//
// Bytes bound it: 3 values per row and channel (5 in the gradient) against
// some 18 instructions (36), which at full rate take about half the time of
// the 2-byte rows' bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

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
  double* dbias_part;   // [work items][channels], or null
  float* dbias;         // where there is one work item, its sums themselves; or null
  float* dstate;
};

__device__ __forceinline__ void seq_range(const int64_t* off, int64_t j, int64_t rows, int64_t& s,
                                          int64_t& e) {
  s = off[j];
  e = off[j + 1];
  s = s < 0 ? 0 : s;
  e = e > rows ? rows : e;
}

// One lane per sequence and V channels (V divides the width: no channel has
// two lanes, of which one could write a state in place that the other has yet
// to read), row after row. With 131,072 lanes or more bound by memory (4000
// sequences of 50 rows x 512 bf16: 123 us, 5.0 TB/s; 512 of 128 rows 44 us, 4.6
// TB/s, of fp32 82 us, 4.9 TB/s), below by the latency of a batch of rows; the
// push of 512 x 8 rows takes 7 us on the device. 2-byte rows take two channels
// per lane (2000 x 100 x 128 bf16 35 us, one channel 39); fp32 rows one, as two
// with a batch in flight spill (65 against 106 us).
template <typename T, int V>
__global__ void logmel_scan_lanes_kernel(ScanArgs<T> p) {
  const int64_t groups = p.channels / V;
  const int64_t total = p.n_seq * groups;
  for (int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; id < total;
       id += (int64_t)gridDim.x * blockDim.x) {
    const int64_t j = id / groups;
    const int64_t c = id % groups * V;
    int64_t s, e;
    seq_range(p.off, j, p.rows, s, e);
    float h[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = p.state ? p.state[j * p.channels + c + v] : 0.0f;
      b[v] = Gate<T>::bias_of(p.bias ? p.bias[c + v] : 0.0f);
    }
    // rows in batches, the next one on its way while one is worked
    constexpr int kBatch = 8;
    Packed<T, V> x[kBatch], g[kBatch];
    auto load = [&](int64_t t0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (t0 + i < e) {
          x[i] = row_load<T, V>(p.x + (t0 + i) * p.xs + c);
          g[i] = row_load<T, V>(p.g + (t0 + i) * p.gs + c);
        }
    };
    load(s);
    for (int64_t t0 = s; t0 < e; t0 += kBatch) {
      float a[kBatch][V], ux[kBatch][V];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float u;
          Gate<T>::pair((float)g[i].v[v], b[v], a[i][v], u);
          ux[i][v] = u * (float)x[i].v[v];
        }
      load(t0 + kBatch);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t t = t0 + i;
        if (t >= e) break;
        if (p.ck && t % kCk == 0 && t > s) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.ck[t / kCk * p.channels + c + v] = h[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(a[i][v], h[v], ux[i][v]);
        row_store<T, V>(p.h + t * p.hs + c, h);
      }
    }
    if (p.state_out) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.state_out[j * p.channels + c + v] = h[v];
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: a workgroup of 8 wavefronts walks a range of rows, kCk rows at a
// time, for 64 V channels; wavefront w holds rows 16 w .. 16 w + 15 of a tile,
// V channels per lane.
// ---------------------------------------------------------------------------

constexpr int kWaves = 8;
constexpr int kRun = (int)kCk / kWaves;   // rows per wavefront and tile

// What a run of rows does to the state before it, h -> A h + B, per channel.
// A < 0 marks a run in which a sequence starts: h -> B, whatever h holds (a
// product with 0 would let another sequence's NaN through).
template <int V>
struct Affine {
  float a[V], b[V];
};

constexpr float kCut = -1.0f;

__device__ __forceinline__ float apply(float a, float b, float h) {
  return a < 0.0f ? b : __builtin_fmaf(a, h, b);
}

// The sequence a row belongs to: the last j with off[j] <= row, and its rows.
struct Cursor {
  int64_t j, s, e;
};

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

__device__ __forceinline__ void cursor_read(const int64_t* off, int64_t rows, Cursor& k) {
  int64_t s, e;
  seq_range(off, k.j, rows, s, e);
  k.s = uniform64(s);
  k.e = uniform64(e);
}

// All 64 lanes look at once; every round leaves at most a 64th of the range.
__device__ __forceinline__ Cursor cursor_find(const int64_t* off, int64_t n, int64_t rows,
                                              int64_t row) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t i = lo + lane * step;
    const int under = __popcll(__ballot(i < hi && off[i] <= row));
    lo += under ? (under - 1) * step : 0;
    hi = lo + step < hi ? lo + step : hi;
  }
  Cursor k;
  k.j = uniform64(lo);
  cursor_read(off, rows, k);
  return k;
}

// f(j) for the sequences without rows among a worker's share: sequences
// [64 i, 64 i + 64) for worker i, and so on in steps of all workers.
template <int V, typename F>
__device__ __forceinline__ void for_empty(const int64_t* off, int64_t n, int64_t rows,
                                          int64_t worker, int64_t workers, F&& f) {
  const int lane = threadIdx.x & 63;
  for (int64_t j0 = worker * 64; j0 < n; j0 += workers * 64) {
    bool empty = false;
    if (j0 + lane < n) {
      int64_t s, e;
      seq_range(off, j0 + lane, rows, s, e);
      empty = s >= e;
    }
    for (uint64_t m = __ballot(empty); m; m &= m - 1) f(j0 + (__ffsll((long long)m) - 1));
  }
}

// The offset of the next row, as a new value to the compiler.
__device__ __forceinline__ int64_t next_row(int64_t at, int64_t stride) {
  at += stride;
  asm("" : "+s"(at));
  return at;
}

template <typename T, int V>
__device__ __forceinline__ void load_run(Packed<T, V> (&r)[kRun], const T* base, int64_t stride,
                                         uint32_t c, int64_t w0, int64_t lo, int64_t hi) {
  // a running scalar offset: 16 multiples of the stride kept over the tiles
  // would not fit the scalar registers
  int64_t at = w0 * stride;
  if (lo <= w0 && w0 + kRun <= hi) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      r[i] = row_load<T, V>(base + at + c);
      at = next_row(at, stride);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      r[i] = Packed<T, V>{};
      if (w0 + i >= lo && w0 + i < hi) r[i] = row_load<T, V>(base + at + c);
      at = next_row(at, stride);
    }
  }
}

template <int V>
__device__ __forceinline__ void load_floats(float (&r)[V], const float* p, int64_t row,
                                            int64_t channels, uint32_t c) {
#pragma unroll
  for (int v = 0; v < V; ++v) r[v] = p ? p[row * channels + c + v] : 0.0f;
}

template <typename T, int V>
__device__ __forceinline__ void load_bias(float (&r)[V], const float* bias, int64_t c0,
                                          uint32_t c) {
  load_floats<V>(r, bias ? bias + c0 : nullptr, 0, 0, c);
#pragma unroll
  for (int v = 0; v < V; ++v) r[v] = Gate<T>::bias_of(r[v]);
}

template <int V>
__device__ __forceinline__ void store_floats(float* p, int64_t row, int64_t channels, uint32_t c,
                                             const float (&r)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) p[row * channels + c + v] = r[v];
}

// The workgroup's channels: a uniform first one, and each lane's offset from
// it. The last lanes of a ragged slab hold the row's last V channels again
// and write the same values; with two channels per lane and one channel over
// the slabs, the last slab holds one of the slab before as well.
template <int V>
__device__ __forceinline__ uint32_t lane_offset(int64_t slab, int64_t channels, int64_t& base) {
  base = slab * 64 * V;
  if (base + V > channels) base = channels - V;
  const int64_t most = channels - V - base;
  const int64_t c = (threadIdx.x & 63) * V;
  return (uint32_t)(c < most ? c : most);
}

// A workgroup's item and slab. Workgroups go to the 8 dies in turn; by_die,
// the slabs of one item are 8 apart, so that the ends of unaligned row pieces,
// which two slabs share, meet in one die's L2 (24 x 2917 x 257 fp16 55 us, 70
// with the slabs side by side).
struct Place {
  int64_t item, slab;
};

__device__ __forceinline__ Place place_of(int64_t slabs, bool by_die) {
  const int64_t b = blockIdx.x;
  if (by_die) return {b / (8 * slabs) * 8 + b % 8, b / 8 % slabs};
  return {b / slabs, b % slabs};
}

struct PartArgs {
  bool by_die;
  int64_t part_rows;   // a multiple of kCk
  int64_t parts;
  float* a;            // [parts][channels]: the part's Affine out of its first or last row
  float* b;
  float* state;        // [parts][channels]: the initial state of the sequence that leaves the part
};

// Rows of part k that belong to a sequence.
template <typename T>
__device__ __forceinline__ void part_range(const ScanArgs<T>& p, const PartArgs& q, int64_t k,
                                           int64_t& r0, int64_t& r1) {
  const int64_t last = p.off[p.n_seq];
  const int64_t end = uniform64(last < p.rows ? last : p.rows);
  r0 = k * q.part_rows;
  r1 = r0 + q.part_rows < end ? r0 + q.part_rows : end;
}

// Folds the Affine of `count` runs, the i-th at f(i), onto nothing: the
// composition of all of them in order.
template <int V, typename F>
__device__ __forceinline__ Affine<V> compose(int64_t count, F&& f) {
  Affine<V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    r.a[v] = 1.0f;
    r.b[v] = 0.0f;
  }
#pragma unroll 4
  for (int64_t i = 0; i < count; ++i) {
    const Affine<V> n = f(i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      r.b[v] = apply(n.a[v], n.b[v], r.b[v]);
      r.a[v] = n.a[v] < 0.0f ? kCut : n.a[v] * r.a[v];
    }
  }
  return r;
}

template <int V>
struct WaveTotals {
  Affine<V> t[kWaves][64];
};

// The composition over the workgroup of what each wavefront holds for its
// share of `count` runs (wavefront w: runs [w per, (w + 1) per)).
template <int V, typename F>
__device__ __forceinline__ Affine<V> compose_by_waves(WaveTotals<V>& lds, int64_t count, F&& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = (count + kWaves - 1) / kWaves;
  const int64_t i0 = wave * per < count ? wave * per : count;
  const int64_t i1 = i0 + per < count ? i0 + per : count;
  lds.t[wave][lane] = compose<V>(i1 - i0, [&](int64_t i) { return f(i0 + i); });
  __syncthreads();
  return compose<V>(kWaves, [&](int64_t w) { return lds.t[w][lane]; });
}

// Before the tiles of parts: what each part does to the state of a sequence
// that runs on past its end. Only the rows of that sequence count, so a part
// whose last row ends a sequence has nothing to do. One sequence of 521,998 x
// 128 fp32: 120 us, 4.4 TB/s over x and gate. Reading them a second time is
// the price of few long sequences (5 values instead of 3): a single pass would
// have to wait in the kernel for the parts before, hop by hop between dies.
// Taking the two kernels in turn over pieces that fit the 256 MB cache was
// slower at every size (284 us with 140 MB, 262 without pieces).
template <typename T, int V>
__global__ __launch_bounds__(512) void logmel_scan_parts_kernel(ScanArgs<T> p, PartArgs q) {
  __shared__ WaveTotals<V> lds;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slabs = (p.channels + 64 * V - 1) / (64 * V);
  const Place at_grid = place_of(slabs, q.by_die);
  // from the last part down: the tiles start with the first, whose rows are
  // then the latest read
  const int64_t k = q.parts - 1 - at_grid.item;
  if (k < 0) return;
  int64_t c0;
  const uint32_t c = lane_offset<V>(at_grid.slab, p.channels, c0);
  int64_t r0, r1;
  part_range(p, q, k, r0, r1);
  if (r1 <= r0) return;
  const Cursor at = cursor_find(p.off, p.n_seq, p.rows, r1 - 1);
  if (at.e <= r1) return;
  const bool starts = at.s >= r0;
  const int64_t lo = starts ? at.s : r0;
  const int64_t per = ((r1 - lo + kWaves - 1) / kWaves + kRun - 1) / kRun * kRun;
  const int64_t w0 = lo + wave * per, w1 = w0 + per < r1 ? w0 + per : r1;
  float bias[V], h0[V];
  load_bias<T, V>(bias, p.bias, c0, c);
  if (starts) load_floats<V>(h0, p.state ? p.state + c0 : nullptr, at.j, p.channels, c);
  float A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    B[v] = 0.0f;
    if (starts && wave == 0) B[v] = h0[v];
  }
  Packed<T, V> x[kRun], g[kRun];
  if (w0 < w1) {
    load_run<T, V>(x, p.x + c0, p.xs, c, w0, w0, w1);
    load_run<T, V>(g, p.g + c0, p.gs, c, w0, w0, w1);
  }
  for (int64_t t = w0; t < w1; t += kRun) {
    float a[kRun][V], b[kRun][V];
    const bool whole = t + kRun <= w1;
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u;
        Gate<T>::pair((float)g[i].v[v], bias[v], a[i][v], u);
        b[i][v] = u * (float)x[i].v[v];
      }
    if (t + kRun < w1) {
      load_run<T, V>(x, p.x + c0, p.xs, c, t + kRun, w0, w1);
      load_run<T, V>(g, p.g + c0, p.gs, c, t + kRun, w0, w1);
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (!whole && t + i >= w1) break;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        B[v] = __builtin_fmaf(a[i][v], B[v], b[i][v]);
        A[v] *= a[i][v];
      }
    }
  }
  Affine<V> mine;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mine.a[v] = starts && wave == 0 ? kCut : A[v];
    mine.b[v] = B[v];
  }
  lds.t[wave][threadIdx.x & 63] = mine;
  __syncthreads();
  if (wave == 0) {
    const Affine<V> all =
        compose<V>(kWaves, [&](int64_t w) { return lds.t[w][threadIdx.x & 63]; });
    store_floats<V>(q.a + c0, k, p.channels, c, all.a);
    store_floats<V>(q.b + c0, k, p.channels, c, all.b);
    if (starts) store_floats<V>(q.state + c0, k, p.channels, c, h0);
  }
}

// The tiles. kParts: a work item is a part of the rows, entered with the state
// the parts before it leave (q.a null: there is one part); otherwise it is one
// sequence. Each tile is read once, ahead of its use: its local recurrence
// from zero (H) and the product of its gates (P) stay in registers while the
// wavefronts exchange their runs' Affine through LDS, then h = P carry + H.
// One barrier a tile, on two buffers in turn; the next tile's loads pass it in
// flight. 16 rows a wavefront: 64 registers of P and H for two channels. By
// sequences 64 x 2998 x 512 bf16 takes 125 us (4.7 TB/s; traffic 1.00 x the
// bytes), fp32 231 us (5.1 TB/s); in parts 521,998 x 128 fp32 140 us after the
// 120 of the parts' maps.
template <typename T, int V, bool kParts, bool kEarly>
__global__ __launch_bounds__(512, kEarly ? 2 : 4) void logmel_scan_tiles_kernel(
    ScanArgs<T> p, PartArgs q) {
  __shared__ WaveTotals<V> lds[2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slabs = (p.channels + 64 * V - 1) / (64 * V);
  const Place at_grid = place_of(slabs, q.by_die);
  const int64_t item = at_grid.item;
  if (item >= (kParts ? q.parts : p.n_seq)) return;
  int64_t c0;
  const uint32_t c = lane_offset<V>(at_grid.slab, p.channels, c0);
  const float* state = p.state ? p.state + c0 : nullptr;
  float bias[V], carry[V];
  load_bias<T, V>(bias, p.bias, c0, c);
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.0f;
  int64_t r0, r1;
  Cursor at;
  Cursor out;   // the sequence that runs on past r1, where a part's last one does
  out.j = -1;
  if constexpr (kParts) {
    if (wave == 0 && p.state_out)
      for_empty<V>(p.off, p.n_seq, p.rows, item, q.parts, [&](int64_t j) {
        float h[V];
        load_floats<V>(h, state, j, p.channels, c);
        store_floats<V>(p.state_out + c0, j, p.channels, c, h);
      });
    part_range(p, q, item, r0, r1);
    if (r1 <= r0) return;
    at = cursor_find(p.off, p.n_seq, p.rows, r0);
    if (q.a) {
      const Cursor end = cursor_find(p.off, p.n_seq, p.rows, r1 - 1);
      if (end.e > r1) out = end;
      if (at.s < r0) {
        const int64_t k0 = at.s / q.part_rows;
        const Affine<V> in = compose_by_waves<V>(lds[1], item - k0, [&](int64_t i) {
          Affine<V> n;
          load_floats<V>(n.a, q.a + c0, k0 + i, p.channels, c);
          load_floats<V>(n.b, q.b + c0, k0 + i, p.channels, c);
          return n;
        });
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = in.b[v];
      }
    }
  } else {
    at.j = item;
    cursor_read(p.off, p.rows, at);
    r0 = at.s;
    r1 = at.e;
    if (r0 >= r1) {
      if (wave == 0 && p.state_out) {
        load_floats<V>(carry, state, item, p.channels, c);
        store_floats<V>(p.state_out + c0, item, p.channels, c, carry);
      }
      return;
    }
  }
  int64_t tile = r0 / kCk * kCk;
  struct Raw {
    Packed<T, V> x[kRun], g[kRun];
  };
  auto load = [&](Raw& raw, int64_t first) {
    load_run<T, V>(raw.x, p.x + c0, p.xs, c, first + wave * kRun, r0, r1);
    load_run<T, V>(raw.g, p.g + c0, p.gs, c, first + wave * kRun, r0, r1);
  };
  auto one_tile = [&](Raw& raw, Raw& ahead, int buf) {
    auto& x = raw.x;
    auto& g = raw.g;
    const int64_t next = tile + kCk;
    if (kEarly && next < r1) load(ahead, next);
    const int64_t w0 = tile + wave * kRun;
    if (p.ck && wave == 0 && (tile > r0 || (kParts && at.s < r0)))
      store_floats<V>(p.ck + c0, tile / kCk, p.channels, c, carry);
    // the wavefront's rows that belong to a sequence here
    const int64_t lo = w0 < r0 ? r0 : w0, hi = w0 + kRun < r1 ? w0 + kRun : r1;
    if (kParts && lo < hi && lo >= at.e) at = cursor_find(p.off, p.n_seq, p.rows, lo);
    const Cursor first = at;
    const bool plain = w0 > at.s && w0 + kRun < at.e && w0 >= r0 && w0 + kRun <= r1;
    float P[kRun][V], H[kRun][V];
    float A[V], B[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = 1.0f;
      B[v] = 0.0f;
    }
    auto step = [&](int i, auto may_cut) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, u;
        Gate<T>::pair((float)g[i].v[v], bias[v], a, u);
        B[v] = __builtin_fmaf(a, B[v], u * (float)x[i].v[v]);
        A[v] = may_cut && A[v] < 0.0f ? A[v] : A[v] * a;
        P[i][v] = A[v];
        H[i][v] = B[v];
      }
    };
    if (plain) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) step(i, std::false_type{});
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t t = w0 + i;
        if (t >= lo && t < hi) {
          if (kParts)
            while (t >= at.e && at.j + 1 < p.n_seq) {
              ++at.j;
              cursor_read(p.off, p.rows, at);
            }
          if (t == at.s) {
            float h0[V];
            if (at.j == out.j)
              load_floats<V>(h0, q.state + c0, item, p.channels, c);
            else
              load_floats<V>(h0, state, at.j, p.channels, c);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              A[v] = kCut;
              B[v] = h0[v];
            }
          }
          step(i, std::true_type{});
        }
      }
    }
    Affine<V> mine;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      mine.a[v] = A[v];
      mine.b[v] = B[v];
    }
    lds[buf].t[wave][lane] = mine;
    if (!kEarly && next < r1) load(raw, next);
    __syncthreads();
    float in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) {
#pragma unroll
        for (int v = 0; v < V; ++v) in[v] = carry[v];
      }
      const Affine<V> n = lds[buf].t[w][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = apply(n.a[v], n.b[v], carry[v]);
    }
    T* const out_h = p.h + c0;
    int64_t out_at = w0 * p.hs;
    if (plain) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(P[i][v], in[v], H[i][v]);
        row_store<T, V>(out_h + out_at + c, h);
        out_at = next_row(out_at, p.hs);
      }
    } else {
      Cursor k = first;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t t = w0 + i;
        if (t >= lo && t < hi) {
          if (kParts)
            while (t >= k.e && k.j + 1 < p.n_seq) {
              ++k.j;
              cursor_read(p.off, p.rows, k);
            }
          float h[V];
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = apply(P[i][v], H[i][v], in[v]);
          row_store<T, V>(out_h + t * p.hs + c, h);
          if (t + 1 == k.e && p.state_out)
            store_floats<V>(p.state_out + c0, k.j, p.channels, c, h);
        }
      }
    }
    tile = next;
  };
  Raw even, odd;
  load(even, tile);
  for (;;) {
    one_tile(even, odd, 0);
    if (tile >= r1) break;
    if constexpr (kEarly)
      one_tile(odd, even, 1);
    else
      one_tile(even, even, 1);
    if (tile >= r1) break;
  }
}

// ---------------------------------------------------------------------------
// The gradient. With E_t = a_t D_t, what row t hands to the row before it,
//   D_t = dh_t + E_{t+1},  E_t = a_t (dh_t + E_{t+1}),
// an affine recurrence over the rows backwards, which ends at a sequence's
// last row (E after it is dstate_out). h_{t-1} is formed anew from the
// checkpoint before the tile, by the same recurrence as in the forward call:
// reading the rounded h instead would cost as many bytes as reading x does,
// and lose the digits that h_{t-1} - x cancels. 64 x 2998 x 512 bf16: 220 us on
// the device (4.5 TB/s; traffic 1.00 x), fp32 383 us (5.1 TB/s): two
// wavefronts per SIMD, whose instructions take half of that time for 2-byte
// rows. Loading a tile ahead as well does not fit the registers (358 us).
// ---------------------------------------------------------------------------

// Before the tiles of parts: what each part does to the E of a sequence that
// entered the part before its first row.
template <typename T, int V>
__global__ __launch_bounds__(512) void logmel_scan_back_parts_kernel(ScanArgs<T> p,
                                                                     ScanGradArgs<T> d,
                                                                     PartArgs q) {
  __shared__ WaveTotals<V> lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slabs = (p.channels + 64 * V - 1) / (64 * V);
  const Place at_grid = place_of(slabs, q.by_die);
  const int64_t k = at_grid.item;
  if (k >= q.parts) return;
  int64_t c0;
  const uint32_t c = lane_offset<V>(at_grid.slab, p.channels, c0);
  int64_t r0, r1;
  part_range(p, q, k, r0, r1);
  if (r1 <= r0) return;
  const Cursor at = cursor_find(p.off, p.n_seq, p.rows, r0);
  if (at.s >= r0) return;
  const bool ends = at.e <= r1;
  const int64_t hi = ends ? at.e : r1;
  const int64_t per = ((hi - r0 + kWaves - 1) / kWaves + kRun - 1) / kRun * kRun;
  const int64_t w0 = r0 + wave * per, w1 = w0 + per < hi ? w0 + per : hi;
  const bool last = ends && w0 < hi && w1 == hi;   // the wavefront with the sequence's last row
  float bias[V];
  load_bias<T, V>(bias, p.bias, c0, c);
  Affine<V> mine;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mine.a[v] = 1.0f;
    mine.b[v] = 0.0f;
  }
  if (last)
    load_floats<V>(mine.b, d.dstate_out ? d.dstate_out + c0 : nullptr, at.j, p.channels, c);
  // rows from the wavefront's last run down
  Packed<T, V> dh[kRun], g[kRun];
  int64_t t = w0 < w1 ? w0 + (w1 - 1 - w0) / kRun * kRun : w0 - kRun;
  if (t >= w0) {
    load_run<T, V>(dh, d.dh + c0, d.dhs, c, t, w0, w1);
    load_run<T, V>(g, p.g + c0, p.gs, c, t, w0, w1);
  }
  for (; t >= w0; t -= kRun) {
    float a[kRun][V], b[kRun][V];
    const bool whole = t + kRun <= w1;
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u;
        Gate<T>::pair((float)g[i].v[v], bias[v], a[i][v], u);
        b[i][v] = (float)dh[i].v[v];
      }
    if (t - kRun >= w0) {
      load_run<T, V>(dh, d.dh + c0, d.dhs, c, t - kRun, w0, w1);
      load_run<T, V>(g, p.g + c0, p.gs, c, t - kRun, w0, w1);
    }
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
      if (whole || t + i < w1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          mine.b[v] = a[i][v] * (b[i][v] + mine.b[v]);
          mine.a[v] *= a[i][v];
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) mine.a[v] = last ? kCut : mine.a[v];
  lds.t[wave][lane] = mine;
  __syncthreads();
  if (wave == 0) {
    const Affine<V> all = compose<V>(kWaves, [&](int64_t w) { return lds.t[kWaves - 1 - w][lane]; });
    store_floats<V>(q.a + c0, k, p.channels, c, all.a);
    store_floats<V>(q.b + c0, k, p.channels, c, all.b);
  }
}

// The tiles, from a work item's last to its first.
template <typename T, int V, bool kParts>
__global__ __launch_bounds__(512, 2) void logmel_scan_back_tiles_kernel(ScanArgs<T> p,
                                                                        ScanGradArgs<T> d,
                                                                        PartArgs q) {
  __shared__ WaveTotals<V> fwd[2], rev[2];
  __shared__ double sums[kWaves][64][V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slabs = (p.channels + 64 * V - 1) / (64 * V);
  const Place at_grid = place_of(slabs, q.by_die);
  const int64_t item = at_grid.item;
  if (item >= (kParts ? q.parts : p.n_seq)) return;
  int64_t c0;
  const uint32_t c = lane_offset<V>(at_grid.slab, p.channels, c0);
  const float* state = p.state ? p.state + c0 : nullptr;
  const float* dstate_out = d.dstate_out ? d.dstate_out + c0 : nullptr;
  float* dstate = d.dstate ? d.dstate + c0 : nullptr;
  float bias[V], carry[V];
  double db[V];
  load_bias<T, V>(bias, p.bias, c0, c);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    carry[v] = 0.0f;
    db[v] = 0.0;
  }
  int64_t r0, r1;
  Cursor at;
  if constexpr (kParts) {
    if (wave == 0 && dstate)
      for_empty<V>(p.off, p.n_seq, p.rows, item, q.parts, [&](int64_t j) {
        float e[V];
        load_floats<V>(e, dstate_out, j, p.channels, c);
        store_floats<V>(dstate, j, p.channels, c, e);
      });
    part_range(p, q, item, r0, r1);
    if (r0 < r1) {
      at = cursor_find(p.off, p.n_seq, p.rows, r1 - 1);
      if (q.a && at.e > r1) {
        const int64_t k1 = (at.e - 1) / q.part_rows;
        const Affine<V> in = compose_by_waves<V>(fwd[1], k1 - item, [&](int64_t i) {
          Affine<V> n;
          load_floats<V>(n.a, q.a + c0, k1 - i, p.channels, c);
          load_floats<V>(n.b, q.b + c0, k1 - i, p.channels, c);
          return n;
        });
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = in.b[v];
      }
    }
  } else {
    at.j = item;
    cursor_read(p.off, p.rows, at);
    r0 = at.s;
    r1 = at.e;
    if (r0 >= r1 && wave == 0 && dstate) {
      load_floats<V>(carry, dstate_out, item, p.channels, c);
      store_floats<V>(dstate, item, p.channels, c, carry);
    }
  }
  struct Raw {
    Packed<T, V> x[kRun], g[kRun], dh[kRun];
    float ck[V];
  };
  auto load = [&](Raw& raw, int64_t first) {
    const int64_t w0 = first + wave * kRun;
    load_floats<V>(raw.ck, p.ck + c0, first / kCk, p.channels, c);
    load_run<T, V>(raw.x, p.x + c0, p.xs, c, w0, r0, r1);
    load_run<T, V>(raw.g, p.g + c0, p.gs, c, w0, r0, r1);
    load_run<T, V>(raw.dh, d.dh + c0, d.dhs, c, w0, r0, r1);
  };
  int64_t tile = (r1 - 1) / kCk * kCk;
  auto one_tile = [&](Raw& raw, int buf) {
    const int64_t w0 = tile + wave * kRun;
    const int64_t next = tile - kCk;
    const bool more = next + kCk > r0;
    const int64_t lo = w0 < r0 ? r0 : w0, hi = w0 + kRun < r1 ? w0 + kRun : r1;
    if (kParts && lo < hi && (lo < at.s || lo >= at.e))
      at = cursor_find(p.off, p.n_seq, p.rows, lo);
    const bool plain = w0 > at.s && w0 + kRun < at.e && w0 >= r0 && w0 + kRun <= r1;
    float a[kRun][V], u[kRun][V];
    Affine<V> f, e;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f.a[v] = e.a[v] = 1.0f;
      f.b[v] = e.b[v] = 0.0f;
    }
    auto onward = [&](Cursor& k, int64_t t) {
      if (kParts)
        while (t >= k.e && k.j + 1 < p.n_seq) {
          ++k.j;
          cursor_read(p.off, p.rows, k);
        }
    };
    auto backward = [&](Cursor& k, int64_t t) {
      if (kParts)
        while (t < k.s && k.j > 0) {
          --k.j;
          cursor_read(p.off, p.rows, k);
        }
    };
    Cursor k = at;
    if (plain) {
#pragma unroll
      for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Gate<T>::pair((float)raw.g[i].v[v], bias[v], a[i][v], u[i][v]);
          f.b[v] = __builtin_fmaf(a[i][v], f.b[v], u[i][v] * (float)raw.x[i].v[v]);
          f.a[v] *= a[i][v];
        }
      // the product of the gates is the same both ways
#pragma unroll
      for (int v = 0; v < V; ++v) e.a[v] = f.a[v];
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          e.b[v] = a[i][v] * ((float)raw.dh[i].v[v] + e.b[v]);
    } else {
      // rows that are not the item's change nothing: a = 1, u = 0
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t t = w0 + i;
        const bool in = t >= lo && t < hi;
        if (in) {
          onward(k, t);
          if (t == k.s) {
            load_floats<V>(f.b, state, k.j, p.channels, c);
#pragma unroll
            for (int v = 0; v < V; ++v) f.a[v] = kCut;
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Gate<T>::pair((float)raw.g[i].v[v], bias[v], a[i][v], u[i][v]);
          a[i][v] = in ? a[i][v] : 1.0f;
          u[i][v] = in ? u[i][v] : 0.0f;
          f.b[v] = __builtin_fmaf(a[i][v], f.b[v], u[i][v] * (float)raw.x[i].v[v]);
          f.a[v] = f.a[v] < 0.0f ? f.a[v] : f.a[v] * a[i][v];
        }
      }
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        const int64_t t = w0 + i;
        if (t >= lo && t < hi) {
          backward(k, t);
          if (t + 1 == k.e) {
            load_floats<V>(e.b, dstate_out, k.j, p.channels, c);
#pragma unroll
            for (int v = 0; v < V; ++v) e.a[v] = kCut;
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          e.b[v] = a[i][v] * ((float)raw.dh[i].v[v] + e.b[v]);
          e.a[v] = e.a[v] < 0.0f ? e.a[v] : e.a[v] * a[i][v];
        }
      }
    }
    fwd[buf].t[wave][lane] = f;
    rev[buf].t[wave][lane] = e;
    __syncthreads();
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        repack(raw.x[i]);
        repack(raw.dh[i]);
      }
    }
    float h[V], E[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = raw.ck[v];
      E[v] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w)
      if (w < wave) {
        const Affine<V> n = fwd[buf].t[w][lane];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(n.a[v], n.b[v], h[v]);
      }
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w) {
      if (w == wave) {
#pragma unroll
        for (int v = 0; v < V; ++v) E[v] = carry[v];
      }
      const Affine<V> n = rev[buf].t[w][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = apply(n.a[v], n.b[v], carry[v]);
    }
    float prev[kRun][V], part[V];
#pragma unroll
    for (int v = 0; v < V; ++v) part[v] = 0.0f;
    int64_t dx_at = (w0 + kRun - 1) * d.dxs, dg_at = (w0 + kRun - 1) * d.dgs;
    auto forward_row = [&](int i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = (float)raw.x[i].v[v];
        prev[i][v] = h[v] - x;
        h[v] = __builtin_fmaf(a[i][v], h[v], u[i][v] * x);
      }
    };
    auto backward_row = [&](int i) {
      float dx[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float D = (float)raw.dh[i].v[v] + E[v];
        E[v] = a[i][v] * D;
        dx[v] = u[i][v] * D;
        dg[v] = prev[i][v] * (u[i][v] * E[v]);
        part[v] += dg[v];
      }
      row_store<T, V>(d.dx + c0 + dx_at + c, dx);
      row_store<T, V>(d.dg + c0 + dg_at + c, dg);
    };
    auto row_up = [&] {
      dx_at = next_row(dx_at, -d.dxs);
      dg_at = next_row(dg_at, -d.dgs);
    };
    if (plain) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) forward_row(i);
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        backward_row(i);
        row_up();
      }
    } else {
      k = at;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t t = w0 + i;
        if (t >= lo && t < hi) {
          onward(k, t);
          if (t == k.s) load_floats<V>(h, state, k.j, p.channels, c);
          forward_row(i);
        }
      }
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        const int64_t t = w0 + i;
        if (t >= lo && t < hi) {
          backward(k, t);
          if (t + 1 == k.e) load_floats<V>(E, dstate_out, k.j, p.channels, c);
          backward_row(i);
          if (t == k.s && dstate) store_floats<V>(dstate, k.j, p.channels, c, E);
        }
        row_up();
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) db[v] += (double)part[v];
    if (more) load(raw, next);
    tile = next;
  };
  if (r0 < r1) {
    Raw raw;
    load(raw, tile);
    for (int buf = 0; tile + kCk > r0; buf ^= 1) one_tile(raw, buf);
  }
  if (!d.dbias_part && !d.dbias) return;
#pragma unroll
  for (int v = 0; v < V; ++v) sums[wave][lane][v] = db[v];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      double s = 0.0;
      for (int w = 0; w < kWaves; ++w) s += sums[w][lane][v];
      if (d.dbias)
        d.dbias[c0 + c + v] = (float)s;
      else
        d.dbias_part[item * p.channels + c0 + c + v] = s;
    }
  }
}

// Sums over work items: 32 channels per workgroup, 32 lanes a channel, each
// taking every 32nd part; the 32 sums are added in order. Up to three sums in
// one launch, one per blockIdx.y.
struct SumOut {
  PartSums s[3];
};

template <typename T>
__global__ __launch_bounds__(1024) void logmel_part_sum_kernel(const T* part, int64_t parts,
                                                               int64_t stride, int64_t channels,
                                                               SumOut o) {
  __shared__ double sums[32][33];
  const PartSums k = o.s[blockIdx.y];
  if (!k.out) return;
  part += k.which * channels;
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  double s = 0.0;
  if (c < channels) {
#pragma unroll 8
    for (int64_t g = row; g < parts; g += 32) s += (double)part[g * stride + c];
  }
  sums[row][lane] = s;
  __syncthreads();
  if (row == 0 && c < channels) {
    double t = sums[0][lane];
    for (int w = 1; w < 32; ++w) t += sums[w][lane];
    k.out[c] = (float)(k.factor ? t * (double)k.factor[c] : t);
  }
}

hipError_t launch_part_sum(const double* part, int64_t parts, int64_t channels, float* out,
                           hipStream_t stream) {
  logmel_part_sum_kernel<<<(unsigned)((channels + 31) / 32), 1024, 0, stream>>>(
      part, parts, channels, channels, SumOut{{{out, 0, nullptr}}});
  return hipGetLastError();
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

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// Whether a die each for 8 items in turn leaves none of them much behind.
bool by_die(int64_t items) { return ceil_div(items, 8) * 8 <= items + items / 8; }

unsigned grid_for(int64_t items, int64_t slabs) {
  return (unsigned)((by_die(items) ? ceil_div(items, 8) * 8 : items) * slabs);
}

// How a call's rows are split over workgroups.
struct Split {
  enum How { kLanes, kSequences, kParts } how;
  int pairs;          // channels per lane
  int64_t slabs;      // of 64 pairs channels
  int64_t part_rows, parts;
};

// Which way is the fastest follows from the sizes and a few times measured on
// this card, in us:
//  - once: each value read or written once, 4.6 TB/s over the bytes (3 values
//    of the type per row and channel, 5 in the gradient);
//  - a row of a lane that walks a sequence alone: 0.2;
//  - a tile: 3 for a workgroup on an idle card, whose longest sequence sets
//    the least time of a split by sequences (6 in the gradient); 5 where the
//    compute units are full, with one workgroup of two channels per lane or
//    two of one channel per lane each (7 to 8.5 and 6 in the gradient, one
//    workgroup a compute unit in either), and 3 (4) to start. A sequence of L
//    rows touches (L + 127) / 128 tiles on average;
//  - in parts, the first kernel reads two values per row and channel again of
//    each sequence that runs on past its part, and costs a launch, 8; a tile
//    with a sequence's end in it takes up to 1.4 times as long, and for 2-byte
//    rows the lanes past a width's end cost what the others do.
// Measured, the way taken first: 512 sequences of 128 rows x 512 bf16 one lane
// each 44, by sequences 59, in parts 75; 64 of them by sequences 10, one lane
// each 27; 64 x 2998 x 512 by sequences 126, in parts 183; 64 x 2998 x 128 in
// parts 60, by sequences 67; 8 x 2998 x 512 in parts 32, by sequences 61.
// Gradient: 64 x 2998 x 512 by sequences 228, in parts 258; 2000 x 100 x 100
// fp32 in parts 130, by sequences 215; 64 x 2998 x 128 in parts 90, by
// sequences 149.
// Two channels per lane halve the memory instructions (64 x 2998 x 512 bf16
// 126 against 140 with one, fp32 231 against 250), but need workgroups for
// most compute units (64 x 2998 x 128: 99 against 75) and most of their lanes.
// In parts, whose first kernel only reads, one channel per lane is the faster
// (64 x 2998 x 512 183 against 210); in the gradient's, whose tiles hold twice
// the registers, two and as many parts as compute units (64 x 2998 x 128 bf16
// 89 against 108 with one and twice the parts, 6 x 9000 x 1024 fp16 182 against
// 223).
Split scan_split(const logmel_scan_input& in, int cus, bool backward) {
  Split s{};
  const int64_t longest = in.max_frames ? in.max_frames : in.rows;
  const int64_t rows = in.rows < 1 ? 1 : in.rows;
  const double mean = (double)rows / (double)(in.n_seq < 1 ? 1 : in.n_seq);
  const double units = backward ? 5.0 : 3.0;
  const double size = in.type == LOGMEL_F32 ? 4.0 : 2.0;
  const double once = units * size * (double)rows * (double)in.channels / 4.6e6;

  // by sequences
  const int64_t pair_slabs = ceil_div(in.channels, 128);
  const int64_t over = in.channels % 128;
  // the gradient may share a channel over the slabs between two workgroups;
  // in a call, one could write the state in place that the other has yet to
  // read
  const bool pairs = in.channels > 1 && (over == 0 || over > 64 || (backward && pair_slabs > 2)) &&
                     in.n_seq >= ceil_div(3 * cus, 4 * pair_slabs);
  const int64_t slabs = ceil_div(in.channels, pairs ? 128 : 64);
  // a launch takes less than 2^32 threads: 2^23 workgroups, of which by_die
  // may add an eighth
  const bool too_many = in.n_seq > (int64_t(1) << 22) / slabs;
  const int64_t groups = too_many ? 0 : in.n_seq * slabs;
  const int64_t slots = !backward && !pairs ? 2 * cus : cus;
  const double tile = backward ? (!pairs ? 6.0 : groups <= cus ? 7.0 : 8.5)
                               : !pairs && groups <= cus ? 3.0 : 5.0;
  const double start = backward ? 4.0 : 3.0;
  const double full = (double)ceil_div(groups, slots) * ((mean + 127.0) / 128.0 * tile + start);
  const double alone = (backward ? 6.0 : 3.0) * (double)ceil_div(longest, kCk);
  double by_sequences = once > alone ? once : alone;
  if (full > by_sequences) by_sequences = full;
  if (too_many) by_sequences = HUGE_VAL;

  // in parts
  const int part_pairs = backward && in.channels > 1 ? 2 : 1;
  const int64_t part_slabs = ceil_div(in.channels, 64 * part_pairs);
  // as many as the compute units hold, of every die
  int64_t want = (backward ? 1 : 2) * cus / part_slabs;
  want = want >= 8 ? want / 8 * 8 : want < 1 ? 1 : want;
  const int64_t part_rows = ceil_div(ceil_div(rows, kCk), want) * kCk;
  const int64_t parts = ceil_div(rows, part_rows);
  const double again = mean >= 2.0 * part_rows ? 1.0 : mean / (2.0 * part_rows);
  const double lanes =
      size == 2.0 ? (double)(part_slabs * 64 * part_pairs) / (double)in.channels : 1.0;
  double in_parts = once * lanes * (1.0 + again * 2.0 / units) *
                    (1.0 + 0.4 * (mean > 128.0 ? 128.0 / mean : 1.0));
  const double walk = (backward ? 6.0 : 3.0) * (double)(part_rows / kCk);
  if (walk > in_parts) in_parts = walk;
  if (parts > 1) in_parts += 8.0;

  // one lane each
  const double rowwise = 0.2 * (double)longest;
  const double in_lanes = rowwise > once ? rowwise : once;

  if (!backward && in_lanes <= by_sequences && in_lanes <= in_parts) {
    s.how = Split::kLanes;
    s.pairs = in.channels % 2 || size == 4.0 ? 1 : 2;
  } else if (by_sequences <= in_parts) {
    s.how = Split::kSequences;
    s.pairs = pairs ? 2 : 1;
    s.slabs = slabs;
  } else {
    s.how = Split::kParts;
    s.pairs = part_pairs;
    s.slabs = part_slabs;
    s.part_rows = part_rows;
    s.parts = parts;
  }
  return s;
}

template <typename T, int V>
void launch_scan_lanes(const ScanArgs<T>& p, hipStream_t stream) {
  const int64_t lanes = p.n_seq * (p.channels / V);
  logmel_scan_lanes_kernel<T, V><<<grid_of(ceil_div(lanes, 256)), 256, 0, stream>>>(p);
}

template <typename T>
hipError_t launch_scan(const logmel_scan_input& in, void* h, int64_t h_stride, float* state_out,
                       float* checkpoints, void* ws, int cus, hipStream_t stream) {
  ScanArgs<T> p = scan_args<T>(in);
  p.h = static_cast<T*>(h);
  p.hs = h_stride;
  p.state_out = state_out;
  p.ck = checkpoints;
  const Split s = scan_split(in, cus, false);
  PartArgs q{};
  if (s.how == Split::kLanes) {
    if constexpr (sizeof(T) == 2) {
      if (s.pairs == 2)
        launch_scan_lanes<T, 2>(p, stream);
      else
        launch_scan_lanes<T, 1>(p, stream);
    } else {
      launch_scan_lanes<T, 1>(p, stream);
    }
  } else if (s.how == Split::kSequences) {
    const unsigned grid = grid_for(in.n_seq, s.slabs);
    q.by_die = by_die(in.n_seq);
    if (s.pairs == 2)
      logmel_scan_tiles_kernel<T, 2, false, true><<<grid, 512, 0, stream>>>(p, q);
    else
      logmel_scan_tiles_kernel<T, 1, false, false><<<grid, 512, 0, stream>>>(p, q);
  } else {
    const unsigned grid = grid_for(s.parts, s.slabs);
    q.by_die = by_die(s.parts);
    q.part_rows = s.part_rows;
    q.parts = s.parts;
    if (s.parts > 1) {
      q.a = static_cast<float*>(ws);
      q.b = q.a + s.parts * in.channels;
      q.state = q.b + s.parts * in.channels;
      logmel_scan_parts_kernel<T, 1><<<grid, 512, 0, stream>>>(p, q);
    }
    logmel_scan_tiles_kernel<T, 1, true, false><<<grid, 512, 0, stream>>>(p, q);
  }
  return hipGetLastError();
}

// Where a gradient's workspace holds what, in bytes from its start: the sums
// of dgate (doubles, first), then the parts' Affine.
struct BackSpace {
  int64_t items, sums, affine, bytes;
};

BackSpace back_space(const logmel_scan_input& in, const Split& s) {
  BackSpace b;
  b.items = s.how == Split::kParts ? s.parts : in.n_seq;
  b.sums = in.d_bias && b.items > 1 ? b.items * in.channels * 8 : 0;
  b.affine = s.how == Split::kParts && s.parts > 1 ? 2 * s.parts * in.channels * 4 : 0;
  b.bytes = b.sums + b.affine;
  return b;
}

template <typename T>
hipError_t launch_scan_backward(const logmel_scan_input& in, const float* checkpoints,
                                const logmel_scan_grad& grad, void* ws, int cus,
                                hipStream_t stream) {
  ScanArgs<T> p = scan_args<T>(in);
  p.ck = const_cast<float*>(checkpoints);
  const Split s = scan_split(in, cus, true);
  const BackSpace b = back_space(in, s);
  if (in.n_seq == 0)   // no offsets to read; the sum over no rows
    return launch_part_sum(nullptr, 0, in.channels, grad.d_dbias, stream);
  ScanGradArgs<T> d{};
  d.dh = static_cast<const T*>(grad.d_dh);
  d.dhs = grad.dh_stride;
  d.dstate_out = grad.d_dstate_out;
  d.dx = static_cast<T*>(grad.d_dx);
  d.dxs = grad.dx_stride;
  d.dg = static_cast<T*>(grad.d_dgate);
  d.dgs = grad.dgate_stride;
  if (b.items == 1)
    d.dbias = grad.d_dbias;
  else if (grad.d_dbias)
    d.dbias_part = static_cast<double*>(ws);
  d.dstate = grad.d_dstate;
  PartArgs q{};
  if (s.how == Split::kSequences) {
    const unsigned grid = grid_for(in.n_seq, s.slabs);
    q.by_die = by_die(in.n_seq);
    if (s.pairs == 2)
      logmel_scan_back_tiles_kernel<T, 2, false><<<grid, 512, 0, stream>>>(p, d, q);
    else
      logmel_scan_back_tiles_kernel<T, 1, false><<<grid, 512, 0, stream>>>(p, d, q);
  } else {
    const unsigned grid = grid_for(s.parts, s.slabs);
    q.by_die = by_die(s.parts);
    q.part_rows = s.part_rows;
    q.parts = s.parts;
    if (s.parts > 1) {
      q.a = reinterpret_cast<float*>(static_cast<char*>(ws) + b.sums);
      q.b = q.a + s.parts * in.channels;
      if (s.pairs == 2)
        logmel_scan_back_parts_kernel<T, 2><<<grid, 512, 0, stream>>>(p, d, q);
      else
        logmel_scan_back_parts_kernel<T, 1><<<grid, 512, 0, stream>>>(p, d, q);
    }
    if (s.pairs == 2)
      logmel_scan_back_tiles_kernel<T, 2, true><<<grid, 512, 0, stream>>>(p, d, q);
    else
      logmel_scan_back_tiles_kernel<T, 1, true><<<grid, 512, 0, stream>>>(p, d, q);
  }
  if (d.dbias_part)
    return launch_part_sum(d.dbias_part, b.items, in.channels, grad.d_dbias, stream);
  return hipGetLastError();
}

}  // namespace logmel

hipError_t logmel_launch_part_sums(const float* part, int64_t parts, int sums, int64_t channels,
                                   const PartSums out[3], hipStream_t stream) {
  logmel::logmel_part_sum_kernel<<<dim3((unsigned)((channels + 31) / 32), 3), 1024, 0, stream>>>(
      part, parts, sums * channels, channels, logmel::SumOut{{out[0], out[1], out[2]}});
  return hipGetLastError();
}

int64_t logmel_scan_workspace(const logmel_scan_input& in, int backward, int cus) {
  const logmel::Split s = logmel::scan_split(in, cus, backward);
  if (backward) return logmel::back_space(in, s).bytes;
  return s.how == logmel::Split::kParts && s.parts > 1 ? 3 * s.parts * in.channels * 4 : 0;
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
