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

#include <initializer_list>
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

// lambda^n as a sum of two fp32: a state decays through many chunks by the same
// factor, whose own rounding would grow with them.
struct Decay {
  float hi, lo;
};
__device__ __forceinline__ Decay decay_of(float g, float n) {
  if (n == 0.0f) return {1.0f, 0.0f};
  const float e = expm1f(g * n);
  if (!(e > -0.5f)) return {expf(g * n), 0.0f};
  const float hi = 1.0f + e;
  return {hi, e - (hi - 1.0f)};
}
__device__ __forceinline__ float decayed(Decay d, float x) {
  return __builtin_fmaf(d.lo, x, d.hi * x);
}

// ------------------------------------------------------- row after row
//
// A workgroup holds the 64 columns of a sequence's and head's state that one
// slab of c makes: lane (ag, cg) of 16 x 16 holds four columns of every
// sixteenth row. Eight rows at a time are laid out in LDS, worked one after the
// other, and their products with the state joined at the end. Right for any
// length; the form for single rows and short pushes, whose time is that of
// reading and writing the states (512 x 8 x 8 x 64 bf16, 134 MB of states: 43 us).
constexpr int kStepRows = 8;
constexpr int kSlab = 64;
// Rows of the longest sequence that this form is taken for: 64 sequences x 16 x 8 x 64
// bf16 15.1 us, 17.5 in chunks, x 24 19.1 and 18.7, x 48 32 and 20; 512 sequences x 16
// 63 and 117, x 32 102 and 119, x 48 145 and 122 (fp32 within a tenth).
constexpr int kShort = 16;

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
    const float* in = p.state ? p.state + (seq * p.heads + h) * p.da * p.dc : nullptr;
    float* out = p.state_out ? p.state_out + (seq * p.heads + h) * p.da * p.dc : nullptr;
    const int c = c0 + 4 * cg;
    auto at = [&](int a, int j) { return p.transposed ? (c + j) * p.da + a : a * p.dc + c + j; };
    const bool whole = !p.transposed && c + 4 <= p.dc;   // four neighbours in memory
    float w[kU][4];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int a = ag + 16 * u;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[u][j] = 0.0f;
      if (!in || a >= p.da) continue;
      if (whole) {
        const auto v = row_load<float, 4>(in + at(a, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[u][j] = v.v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < p.dc) w[u][j] = in[at(a, j)];
      }
    }
    const Decay lambda = decay_of(p.log_decay[h], 1.0f);
    const int64_t n = run.to > run.from ? run.to - run.from : 0;
    for (int64_t t0 = 0; t0 < n; t0 += kStepRows) {
      const int held = (int)(n - t0 < kStepRows ? n - t0 : kStepRows);
      auto row = [&](int t) { return p.back ? run.to - 1 - t0 - t : run.from + t0 + t; };
      // the rows before are read to the end: the barrier before their outputs
      for (int i = tid; i < held * DA; i += 256) {
        const int t = i / DA, d = i % DA;
        const bool on = d < p.da;
        sa[t][d] = on ? (float)p.a[row(t) * p.as + h / p.share_a * p.da + d] : 0.0f;
        sb[t][d] = on ? (float)p.b[row(t) * p.bs + h / p.share_b * p.da + d] * p.gamma : 0.0f;
      }
      for (int i = tid; i < held * kSlab; i += 256) {
        const int t = i / kSlab, d = i % kSlab;
        const bool on = c0 + d < p.dc;
        sc[t][d] = on ? (float)p.c[row(t) * p.cs + h / p.share_c * p.dc + c0 + d] : 0.0f;
      }
      __syncthreads();
      for (int t = 0; t < held; ++t) {
        const Decay keep = p.back && t0 + t == 0 ? Decay{1.0f, 0.0f} : lambda;
        const float4 cv4 = *reinterpret_cast<const float4*>(&sc[t][4 * cg]);
        const float cv[4] = {cv4.x, cv4.y, cv4.z, cv4.w};
        float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float a = sa[t][ag + 16 * u], b = sb[t][ag + 16 * u];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[u][j] = __builtin_fmaf(b, cv[j], decayed(keep, w[u][j]));
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
    const Decay last = p.back && n > 0 ? lambda : Decay{1.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int a = ag + 16 * u;
      if (a >= p.da) continue;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = decayed(last, w[u][j]);
      if (whole) {
        row_store(out + at(a, 0), x);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < p.dc) out[at(a, j)] = x[j];
      }
    }
  }
}

// ------------------------------------------------------- chunk after chunk
//
// With a chunk of n rows and E = lambda W before it, the state as its first
// row meets it,
//   o_i = beta (gamma sum_{j<=i} lambda^(i-j) (a_i . b_j) c_j + lambda^i a_i E)
//   E'  = lambda^n E + gamma sum_j lambda^(n-j) b_j c_j^T,
// four products on the matrix cores. A workgroup walks the chunks of a sequence's
// rows; half of its wavefronts hold the state, 16 columns each in their
// accumulators, and the other half form the scores, a few blocks of 16 x 16 each,
// which they exchange through LDS. The scores come out of the matrix cores
// with a row i per lane and four neighbouring j in its registers, the state with
// a column per lane and four neighbouring rows: both are fed back as operands
// just so, as the order of the summed index is free, if rows of b are taken in
// the order that `place` gives.
//
// The operands are bf16 pieces: a bf16 row one, an fp16 row two (exactly), an
// fp32 row three (exactly). What the products make is cut into pieces too, by
// rounding, with the rest to the next: scores and the state that meets a in two
// for 2-byte rows, which leave 2^-18 of each where the output keeps 2^-9 or
// 2^-12; three for fp32 rows and for the weighted rows that enter the state,
// which is fp32 for every type. Products of pieces whose places sum to the
// count are left out: 2^-18 or 2^-26 of the whole as well.
//
// bf16 rounds the largest fp32 values to infinity. The state is held at half its
// size, which keeps it and the rows that enter it below that at no cost; the pieces of
// fp32 rows and of their scores are held below it one by one (`cut`). Scores of 2-byte
// rows are not: a result of fp32 may be lost where one is within 2^-9 of overflow.
//
// Causality is exact, for NaN and infinities too: a score above the diagonal is
// left out by a select, and a chunk with a value of b or c that is not finite
// is cut short before its row, which starts a chunk of its own.

// The same value to a reader, to the compiler a new one: addresses and
// conditions formed from it are formed where they are used, not held in
// registers through the walk.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

template <typename T>
struct Pieces;
template <>
struct Pieces<bf16_t> {
  static constexpr int kIn = 1, kMid = 2, kState = 3;
};
template <>
struct Pieces<f16_t> {
  static constexpr int kIn = 2, kMid = 2, kState = 3;
};
template <>
struct Pieces<float> {
  static constexpr int kIn = 3, kMid = 3, kState = 3;
};

using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float low(uint32_t v) { return __builtin_bit_cast(float, v << 16); }
__device__ __forceinline__ float high(uint32_t v) {
  return __builtin_bit_cast(float, v & 0xffff0000u);
}

// M values as N pieces each, packed in pairs; x keeps the rest. kLarge: values from
// 0x1.ffp127 on, which bf16 rounds to infinity, are there too: their first piece is
// bf16's largest, with which three pieces hold them exactly as well.
template <bool kLarge, int N, int M>
__device__ __forceinline__ void cut(float (&x)[M], uint32_t (&piece)[N][M / 2]) {
  static_assert(!kLarge || N > 1);
  auto held = [](float v) { return __builtin_amdgcn_fmed3f(v, -0x1.fep127f, 0x1.fep127f); };
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      piece[n][i] = kLarge && n == 0 ? pack(held(x[2 * i]), held(x[2 * i + 1]))
                                     : pack(x[2 * i], x[2 * i + 1]);
      if (n + 1 < N) {
        x[2 * i] -= low(piece[n][i]);
        x[2 * i + 1] -= high(piece[n][i]);
      }
    }
}

__device__ __forceinline__ bf16x8 frag(const uint32_t (&w)[4]) {
  return __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
}
__device__ __forceinline__ bf16x8 frag(const uint16_t* tile, uint32_t at) {
  return __builtin_bit_cast(
      bf16x8, *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(tile) + at));
}

// acc += sum over the pairs of pieces whose places sum to less than the count.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const bf16x8 (&a)[NA], const bf16x8 (&b)[NB]) {
  constexpr int kMost = NA > NB ? NA : NB;
#pragma unroll
  for (int s = kMost - 1; s >= 0; --s)   // the smallest first
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], acc, 0, 0, 0);
}

// Where the block of four rows (columns) 4 i .. 4 i + 3 stands in a tile whose
// 16-blocks are read as operands of results that are operands again.
__device__ __forceinline__ int place(int i) {
  return 32 * (i >> 3) + 16 * (i & 1) + 4 * ((i >> 1) & 3);
}

// Where a tile of rows of kUnits 16-byte units holds unit u of row r: the units
// of a 128-byte line change places with the row, so that eight lanes that read
// one unit of neighbouring rows, and sixteen that write half units, along rows
// or across them (kAcross), meet 32 different banks each.
template <int kUnits, bool kAcross>
__device__ __forceinline__ int unit_at(int r, int u) {
  if constexpr (kUnits >= 8) {
    const int h = kAcross ? ((r ^ (r >> 3)) & 7) ^ ((r >> 4) & 2)
                          : (r & 7) ^ ((r >> 3) & 1) ^ ((r >> 2) & 4);
    return r * kUnits + (u ^ h);
  } else {
    const int line = r >> 1;
    const int h = (((line ^ (line >> 2)) & 1) | (line & 2) | ((line >> 1) & 4)) ^
                  (6 * ((line >> 4) & 1));
    return line * 8 + ((((r & 1) << 2) | u) ^ h);
  }
}

// The same in bytes for unit u + 4 s of row r + 16 i, r below 16 and u below 4,
// from that of r and u.
template <int kUnits, bool kAcross>
__device__ __forceinline__ uint32_t operand_at(uint32_t at, int i, int s) {
  const uint32_t turn = kUnits >= 8 ? (kAcross ? (2 * (i & 1)) ^ (6 * ((i >> 1) & 1)) : 4 * (i & 1))
                                    : (4 * (i & 1)) ^ (6 * ((i >> 1) & 1));
  return (at ^ (16 * (turn ^ (uint32_t)(4 * s)))) + (uint32_t)i * (kUnits * 256);
}

// The same in bytes for the first of four rows r0 .. r0 + 3 (r0 a multiple of 4)
// and half a unit, and from there for the others: the places differ by bits of
// the row alone.
template <int kUnits, bool kAcross>
__device__ __forceinline__ uint32_t half_at(int r0, int half) {
  return 16 * unit_at<kUnits, kAcross>(r0, half >> 1) + 8 * (half & 1);
}
template <int kUnits>
__device__ __forceinline__ uint32_t half_below(uint32_t at, int r) {
  return kUnits >= 8 ? (at ^ (16 * r)) + r * kUnits * 16
                     : (at ^ (16 * (((r & 1) << 2) | (r >> 1)))) + (r >> 1) * 128;
}

// A buffer resource of `bytes` bytes at p: reads behind them give 0, writes
// there are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

// A tile's place in memory and LDS.
template <typename T>
struct TileAt {
  const T* base;      // its lowest row
  uint32_t pitch;     // bytes between rows
  int width;          // channels there are
  uint16_t* rows;     // where it goes, along rows and along columns
  uint16_t* cols;
};

// kTiles (one or two) tiles of kRows rows and kWidth channels in registers, on
// their way from memory to LDS, in blocks of four rows by 16 bytes: up to eight
// blocks side by side in a wavefront, so that memory is read 128 bytes at a time
// and LDS is written, along rows and along columns, without bank conflicts. Each
// block is a thread's, each wavefront's blocks are of one tile; kThreads bring
// them, a number that divides the workgroup's. Of two tiles the first goes to LDS
// along its rows, the second along both; one goes along its columns. kSkip: the
// first of two is not wanted, nor the second's rows.
template <typename T, int kRows, int kWidth, int kThreads, int kTiles, bool kSkip>
struct Tiles {
  static constexpr int kIn = Pieces<T>::kIn;
  // fp16 rows, which are cut into pieces on the way, go by 8 bytes: more threads
  // take part (70,001 x 6 x 40 x 71 with gradient 1,114 us, 1,183 by 16); bf16 rows,
  // which are stored as they are, by 16 (64 x 2998 x 8 x 64 259 us, 271 by 8)
  static constexpr int kCols = std::is_same_v<T, f16_t> ? 4 : 16 / (int)sizeof(T);
  static constexpr int kDwords = kCols * (int)sizeof(T) / 4;   // of a block's row
  using Row = std::conditional_t<kDwords == 4, u32x4, u32x2>;
  static constexpr int kWide = kWidth / kCols, kBlocks = kRows / 4 * kWide;   // of a tile
  static constexpr int kIts = (kTiles * kBlocks + kThreads - 1) / kThreads;
  static_assert(kBlocks % 64 == 0);

  // The first block of this wavefront: kTiles * kBlocks and more where it has none.
  static __device__ __forceinline__ int first(int it) {
    return (int)(__builtin_amdgcn_readfirstlane(threadIdx.x) % kThreads & ~63) + kThreads * it;
  }
  static __device__ __forceinline__ bool second(int it) {
    if (kTiles == 1) return false;
    return kBlocks % kThreads == 0 ? it >= kBlocks / kThreads : first(it) >= kBlocks;
  }
  static __device__ __forceinline__ bool on(int it) {
    return (kTiles * kBlocks % kThreads == 0 || first(it) < kTiles * kBlocks) &&
           !(kSkip && !second(it));
  }
  static __device__ __forceinline__ void at(int tid, int it, int& rb, int& cb) {
    constexpr int kSide = kWide < 8 ? kWide : 8, kDown = 64 / kSide;
    const int i = (tid % kThreads + kThreads * it) % kBlocks, rest = i >> 6;
    cb = i % kSide + kSide * (rest % (kWide / kSide));
    rb = (i & 63) / kSide + kDown * (rest / (kWide / kSide));
  }

  // Where this lane's blocks lie: in memory from the tile's lowest row on (from
  // its first row upwards, from its last row downwards), and in LDS. Blocks do not
  // pass the row's end (of 2-byte values a word that does would be 0 at the
  // buffer's): the last ones are shifted back.
  struct Places {
    uint32_t from[kIts], row[kIts], col[kIts], col2[kIts];
    __device__ __forceinline__ Places(const TileAt<T>& x, const TileAt<T>& y, bool up,
                                      bool placed_second) {
#pragma unroll
      for (int it = 0; it < kIts; ++it) {
        int rb, cb;
        at(threadIdx.x, it, rb, cb);
        const TileAt<T>& t = second(it) ? y : x;
        const bool placed = second(it) && placed_second;
        const uint32_t down = (uint32_t)(4 * rb) * t.pitch;
        const int c = kCols * cb > t.width - kCols ? t.width - kCols : kCols * cb;
        from[it] = (up ? down : 0u - down) + (uint32_t)c * (uint32_t)sizeof(T);
        row[it] = kCols == 8
                      ? 16 * unit_at<kWidth / 8, false>(placed ? place(rb) : 4 * rb, cb)
                      : half_at<kWidth / 8, false>(placed ? place(rb) : 4 * rb, cb);
        // columns four at a time: the block's first four, and the others
        const int c4 = kCols / 4 * cb;
        col[it] = half_at<kRows / 8, true>(placed ? place(c4) : 4 * c4, rb);
        col2[it] = half_at<kRows / 8, true>(placed ? place(c4 + 1) : 4 * c4 + 4, rb);
      }
    }
  };

  Row v[kIts][4];

  // up: whether the lowest row is the first; held: the rows there are, which may
  // be none. Rows from held on lie behind the buffer (or, their offsets being
  // negative, far behind it) and are 0; `settle` sees to the channels.
  __device__ __forceinline__ void load(const Places& k, const TileAt<T>& x, const TileAt<T>& y,
                                       bool up, int held) {
#pragma unroll
    for (int it = 0; it < kIts; ++it) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[it][r] = Row{};
      if (!on(it)) continue;
      const T* base = second(it) ? y.base : x.base;
      const uint32_t pitch = second(it) ? y.pitch : x.pitch;
      const int width = second(it) ? y.width : x.width;
      const uint32_t row = (uint32_t)width * (uint32_t)sizeof(T);
      const auto buffer = buffer_of(base, held > 0 ? (uint32_t)(held - 1) * pitch + row : 0u);
      uint32_t to = k.from[it] + (up ? 0u : (uint32_t)(held - 1) * pitch);
      const uint32_t step = up ? pitch : 0u - pitch;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kDwords == 4)
          v[it][r] = __builtin_amdgcn_raw_buffer_load_b128(buffer, to, 0, 0);
        else
          v[it][r] = __builtin_amdgcn_raw_buffer_load_b64(buffer, to, 0, 0);
        to += step;
      }
    }
  }

  // 0 in channels from the width on, and the last ones where they belong.
  __device__ __forceinline__ void settle(int width) {
    const int tid = fresh(threadIdx.x);
#pragma unroll
    for (int it = 0; it < kIts; ++it) {
      int rb, cb;
      at(tid, it, rb, cb);
      const int left = width - kCols * cb;   // channels of the block that there are
      const int by = left >= kCols || left <= 0 ? 0 : kCols - left;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kDwords == 2) {
          const uint64_t x = left > 0 ? __builtin_bit_cast(uint64_t, v[it][r]) >> (16 * by) : 0;
          v[it][r] = __builtin_bit_cast(Row, x);
          continue;
        }
        Row x = v[it][r];
        constexpr int kHalf = sizeof(T) == 2, kN = kDwords;   // words are two values
        if constexpr (kHalf) {
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            const uint32_t next = j + 1 < kN ? x[(j + 1) % kN] : 0u;
            x[j] = by & 1 ? __builtin_amdgcn_alignbit(next, x[j], 16) : x[j];
          }
        }
#pragma unroll
        for (int j = 0; j < kN; ++j)
          x[j] = by >> kHalf & 1 ? (j + 1 < kN ? x[(j + 1) % kN] : 0u) : x[j];
#pragma unroll
        for (int j = 0; j < kN; ++j)
          x[j] = by >> kHalf & 2 ? (j + 2 < kN ? x[(j + 2) % kN] : 0u) : x[j];
        if (left <= 0) x = Row{};
        v[it][r] = x;
      }
    }
  }

  // Whether a value of the tile `which` is not finite: the largest of the words
  // without signs is.
  __device__ __forceinline__ bool any_bad(bool which) const {
    bool bad = false;
#pragma unroll
    for (int it = 0; it < kIts; ++it) {
      if (second(it) != which) continue;
      if constexpr (sizeof(T) == 2) {
        using u16x2 = __attribute__((ext_vector_type(2))) uint16_t;
        constexpr uint16_t kInf = std::is_same_v<T, bf16_t> ? 0x7f80 : 0x7c00;
        u16x2 m = {0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < kDwords; ++j)
            m = __builtin_elementwise_max(
                m, __builtin_bit_cast(u16x2, (uint32_t)(v[it][r][j] & 0x7fff7fffu)));
        bad |= m[0] >= kInf || m[1] >= kInf;
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < kDwords; ++j) {
            const uint32_t w = v[it][r][j] & 0x7fffffffu;
            m = m > w ? m : w;
          }
        bad |= m >= 0x7f800000u;
      }
    }
    return bad;
  }

  // The first row of it with a value that is not finite, or kRows.
  __device__ __forceinline__ int first_bad(bool which) const {
    const int tid = fresh(threadIdx.x);
    int found = kRows;
#pragma unroll
    for (int it = 0; it < kIts; ++it) {
      if (second(it) != which || !on(it)) continue;
      int rb, cb;
      at(tid, it, rb, cb);
#pragma unroll
      for (int r = 3; r >= 0; --r) {
        const auto x = __builtin_bit_cast(Packed<T, kCols>, v[it][r]);
        bool bad = false;
#pragma unroll
        for (int j = 0; j < kCols; ++j) bad |= !__builtin_isfinite((float)x.v[j]);
        found = bad && 4 * rb + r < found ? 4 * rb + r : found;
      }
    }
    return found;
  }

  // Into LDS: rows [kIn][kRows][kWidth] and columns [kIn][kWidth][kRows],
  // whichever there are.
  __device__ __forceinline__ void store(const Places& k, const TileAt<T>& x,
                                        const TileAt<T>& y) const {
    constexpr int kBytes = kRows * kWidth * 2;   // of a piece's tile
    constexpr int kWords = kCols / 2;
#pragma unroll
    for (int it = 0; it < kIts; ++it) {
      if (!on(it)) continue;
      uint32_t w[4][kIn][kWords];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kIn == 1) {
#pragma unroll
          for (int j = 0; j < kWords; ++j) w[r][0][j] = v[it][r][j];
        } else {
          const auto z = __builtin_bit_cast(Packed<T, kCols>, v[it][r]);
          float f[kCols];
#pragma unroll
          for (int j = 0; j < kCols; ++j) f[j] = (float)z.v[j];
          cut<sizeof(T) == 4, kIn, kCols>(f, w[r]);
        }
      }
      uint16_t* rows = second(it) ? y.rows : x.rows;
      uint16_t* cols = kTiles == 2 ? y.cols : x.cols;
      if (kTiles == 2 && !kSkip) {
        const uint32_t row = fresh(k.row[it]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          char* to = reinterpret_cast<char*>(rows) + half_below<kWidth / 8>(row, r);
#pragma unroll
          for (int n = 0; n < kIn; ++n) {
            if constexpr (kCols == 8)
              *reinterpret_cast<u32x4*>(to + n * kBytes) =
                  u32x4{w[r][n][0], w[r][n][1], w[r][n][2], w[r][n][3]};
            else
              *reinterpret_cast<u32x2*>(to + n * kBytes) = u32x2{w[r][n][0], w[r][n][1]};
          }
        }
      }
      if (kTiles == 1 || second(it)) {
        const uint32_t col = fresh(k.col[it]), col2 = fresh(k.col2[it]);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          char* to =
              reinterpret_cast<char*>(cols) + half_below<kRows / 8>(c < 4 ? col : col2, c & 3);
          const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
          for (int n = 0; n < kIn; ++n)
            *reinterpret_cast<u32x2*>(to + n * kBytes) =
                u32x2{__builtin_amdgcn_perm(w[1][n][c / 2], w[0][n][c / 2], sel),
                      __builtin_amdgcn_perm(w[3][n][c / 2], w[2][n][c / 2], sel)};
        }
      }
    }
  }
};

// How the rows are split: a workgroup per sequence (parts 0), or parts of
// part_rows packed rows each, whatever sequences they hold. Between parts b and
// b + 1 stands state b of `between`, as the next row of the sequence there meets
// it; kept: the initial state of the sequence that starts in part b and leaves
// it, as its first row meets it, where state_out may overwrite it. Both at the size at
// which the chunks hold them.
struct Walk {
  int64_t part_rows, parts;
  float* between;
  float* kept;
  int* through;   // of each such place: 0 no sequence lies across it, 1 one does, 2 the one that
                  // lies across the place before (behind it, backwards) too
  int64_t items;
};

// Rows of a chunk of most C, of the `left` that there are: none where left is
// below 0, as far below as offsets that decrease make it.
template <int C>
__host__ __device__ constexpr int held_of(int64_t left) {
  return (int)(left < 0 ? 0 : left < C ? left : C);
}
static_assert(held_of<64>(-((int64_t)1 << 32) + 5) == 0 && held_of<64>(-((int64_t)1 << 40)) == 0);
static_assert(held_of<64>(0) == 0 && held_of<64>(5) == 5 && held_of<64>(64) == 64 &&
              held_of<64>(((int64_t)1 << 32) + 5) == 64);

// The first offset at or behind row: n_seq + 1 if there is none.
template <typename T>
__device__ __forceinline__ int64_t first_from(const AttnJob<T>& p, int64_t row) {
  int64_t lo = 0, hi = p.n_seq + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (p.off[mid] < row)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}
// The sequence that holds rows on both sides of `row`: -1 if there is none.
template <typename T>
__device__ __forceinline__ int64_t across(const AttnJob<T>& p, int64_t row) {
  const int64_t i = first_from(p, row);
  return i > 0 && i <= p.n_seq && p.off[i] > row ? i - 1 : -1;
}

template <typename T, int DA, int kWide, int C, bool kOut>
struct ChunkLds {
  static constexpr int kIn = Pieces<T>::kIn, kMid = Pieces<T>::kMid;
  static constexpr int kScores = C == 64 ? 6 : 2;
  uint16_t bt[kIn][DA * C];      // columns as `place` has them
  uint16_t ct[kIn][kWide * C];
  float weight[kWide / 16][C];   // of a chunk's rows as they enter the state, a copy per wavefront
  uint16_t a[kIn][kOut ? C * DA : 8];
  uint16_t b[kIn][kOut ? C * DA : 8];   // rows as `place` has them
  uint16_t p[kMid][kOut ? kScores : 1][kOut ? 64 : 1][8];
  float from_state[kOut ? kWide / 16 : 1][C / 16][kOut ? 64 : 1][4];
  int bad;
};

// Rows of a chunk: 64 where a compute unit's LDS holds 16 wavefronts' tiles so
// (two workgroups of four columns' wavefronts, one of eight), else 32. Where only
// the state is formed that is always so.
template <typename T, int DA, int kWaves, bool kOut>
constexpr int kChunk =
    sizeof(ChunkLds<T, DA, 16 * kWaves, 64, kOut>) <= (kWaves == 4 ? 80 : 160) * 1024 ? 64 : 32;

// Wavefronts that a SIMD holds at a time as LDS has it, four at most.
template <typename T, int DA, int kWaves, bool kOut>
constexpr int kHeld = [] {
  const int lds = (int)sizeof(ChunkLds<T, DA, 16 * kWaves, kChunk<T, DA, kWaves, kOut>, kOut>);
  const int held = 160 * 1024 / lds * 2 * kWaves / 4;
  return held < 4 ? held : 4;
}();

// A workgroup is kWaves wavefronts that see to the scores and kWaves that hold
// the state, 16 columns of it each; a wavefront alone waits for half of its time,
// for LDS and for the other wavefronts. (64 x 2998 x 8 x 64 bf16, 786 MB: 218 us,
// 3.6 TB/s; the vector units are busy for 45 % of the cycles, the matrix cores for
// 21 %.) Of a chunk
//   the first bring a and b, form the scores, and join them with c and with what
//   comes from the state to the output's rows;
//   the second bring c, multiply the state with a, and take b and c into it.
// Two barriers: the tiles are written; the scores and the state's part are
// written and the tiles read.
template <typename T, int DA, int kWaves, bool kOut>
__global__ __launch_bounds__(128 * kWaves, (kHeld<T, DA, kWaves, kOut>)) void
logmel_attn_chunk_kernel(AttnJob<T> p, Walk walk) {
  constexpr int kThreads = 64 * kWaves, kWide = 16 * kWaves;   // of each half
  constexpr int kIn = Pieces<T>::kIn, kMid = Pieces<T>::kMid, kState = Pieces<T>::kState;
  constexpr int C = kChunk<T, DA, kWaves, kOut>;
  constexpr int kI = C / 16, kT = C / 32, kS = DA / 32, kU = DA / 16;
  // of the scores' half (a is not brought where only the state is wanted), and of
  // the state's
  using TilesAB = Tiles<T, C, DA, kThreads, 2, !kOut>;
  using TileC = Tiles<T, C, kWide, kThreads, 1, false>;
  __shared__ __attribute__((aligned(16))) ChunkLds<T, DA, kWide, C, kOut> lds;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % kWaves;
  const bool of_scores = __builtin_amdgcn_readfirstlane(tid >> 6) < kWaves;
  const int64_t cells = (int64_t)p.da * p.dc;
  if constexpr (kOut) {
    if (tid == 0) lds.bad = C;
    __syncthreads();   // before another wavefront marks a row in it
  }

  // A lane's operand: unit 4 s + g of row 16 i + n of a tile of rows, or of columns
  const uint32_t row_base = 16 * unit_at<DA / 8, false>(n, g);
  const uint32_t col_base = 16 * unit_at<C / 8, true>(n, g);
  // The memory instructions in flight are as many on every usual way through a
  // loop, so that a wait leaves the ones behind it alone; the rare way ends with a
  // wait for all.
  auto wait_all = [] { __builtin_amdgcn_s_waitcnt(0x0f70); };

  // Rows [lo, hi) of one sequence, chunk by chunk: both halves of the workgroup
  // go through this, each with its own parts. bring(row, held): the chunk whose
  // lowest row is `row` on its way (held rows; none: nothing); put(): into LDS;
  // bad(): the first row brought with a value that is not finite, or C; work(row,
  // held, end): between the barriers; after(row, held): behind them.
  auto chunks = [&](int64_t lo, int64_t hi, auto bring, auto put, auto bad, auto work,
                    auto after) __attribute__((always_inline)) {
    const int64_t rows = hi - lo;
    auto lowest = [&](int64_t at, int held) {
      return held <= 0 ? lo : p.back ? hi - at - held : lo + at;
    };
    auto held_at = [&](int64_t at) { return held_of<C>(rows - at); };   // 0 behind the last
    bring(lowest(0, held_at(0)), held_at(0));
    for (int64_t at = 0; at < rows;) {
      int held = held_at(at);
      for (bool cut_short = false;;) {
        put();
        if constexpr (kOut)
          if (!cut_short) {
            const int first = bad();
            if (first < C) atomicMin(&lds.bad, first);
          }
        __syncthreads();
        if constexpr (!kOut) break;
        const int first = lds.bad;
        if (cut_short || first == C) break;   // for the whole workgroup
        cut_short = true;
        held = first > 0 ? first : 1;
        bring(lowest(at, held), held);
        wait_all();
        __syncthreads();
        if (tid == 0) lds.bad = C;
      }
      const int64_t next = at + held;
      const int64_t row = lowest(at, held);
      bring(lowest(next, held_at(next)), held_at(next));
      work(held, next == rows);
      __syncthreads();
      after(row, held);
      at = next;
    }
  };

  for (int64_t item = blockIdx.x; item < walk.items; item += gridDim.x) {
    const int h = (int)(item % p.heads);
    const int64_t which = item / p.heads;   // sequence or part
    const float decay = p.log_decay[h];
    const float log2 = decay * 1.44269504088896340736f;
    auto power = [&](int i) { return i > 0 ? __builtin_amdgcn_exp2f(log2 * (float)i) : 1.0f; };
    const int wide = p.dc;               // columns of c and of the output
    const bool works = 16 * wave < wide;   // has some of them

    // f(sequence, from, to, starts, ends): the sequences of this workgroup's rows,
    // in order: its own, or those of its part from the one that enters it on.
    const int64_t r0 = which * walk.part_rows;
    const int64_t r1 = walk.parts == 0 || r0 + walk.part_rows > p.rows ? p.rows
                                                                       : r0 + walk.part_rows;
    auto within = [&](int64_t r) { return r < r0 ? r0 : r > r1 ? r1 : r; };
    auto each = [&](auto f) __attribute__((always_inline)) {
      if constexpr (!kOut) {
        // the one across the part's end (its start, backwards), whose state leaves it
        const int64_t i = across(p, p.back ? r0 : r1), place = p.back ? which - 1 : which;
        if (place < 0 || place >= walk.parts - 1) return;
        const int64_t from = i < 0 ? 0 : p.off[i], to = i < 0 ? 0 : p.off[i + 1];
        const bool starts = from >= r0, ends = to <= r1;
        if (tid == 0 && h == 0) walk.through[place] = i < 0 ? 0 : (p.back ? ends : starts) ? 1 : 2;
        if (i >= 0) f(i, within(from), within(to), starts, ends);
      } else {
        int64_t i = which;
        bool enters = false;
        if (walk.parts) {
          i = first_from(p, r0);
          enters = which > 0 && i > 0 && i <= p.n_seq && p.off[i] > r0;
          i -= enters;
        }
        const bool end = walk.parts == 0 || which == walk.parts - 1;
        do {
          if (i >= p.n_seq || !(enters || end || p.off[i] < r1)) break;
          const int64_t lo = enters ? r0 : within(p.off[i]);
          f(i, lo, within(p.off[i + 1]), !enters, end || p.off[i + 1] <= r1);
          enters = false;
          ++i;
        } while (walk.parts);
      }
    };

    if (of_scores) {
      const T* pa = p.a + (int64_t)(h / p.share_a) * p.da;
      const T* pb = p.b + (int64_t)(h / p.share_b) * p.da;
      const uint32_t sa = (uint32_t)(p.as * sizeof(T)), sb = (uint32_t)(p.bs * sizeof(T));
      TileAt<T> a{pa, sa, p.da, lds.a[0], nullptr};
      TileAt<T> b{pb, sb, p.da, lds.b[0], lds.bt[0]};
      const typename TilesAB::Places places(a, b, !p.back, true);
      // this lane's weights of the scores: block (rows 16 bi, columns 32 t and half);
      // of eight wavefronts the first four take the blocks on the diagonal
      constexpr int kMine = C == 64 ? 3 : 1;
      const int half = wave & 1, pair = (wave >> 1) & 1;
      auto mine = [&](int m) { return kWaves == 4 || (m == 1) == (wave >= 4); };
      float ws[kMine][4];
      // where row j of b is at or before row i of a in the blocks on the diagonal (the
      // first and the third): from this register on
      const int after = 8 * g + 4 * half - (16 * pair + n);
      if constexpr (kOut) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int bi = m ? 2 + pair : pair, t = m == 2;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int age = 16 * bi + n - (32 * t + 8 * g + 4 * half + r);
            ws[m][r] = p.beta * p.gamma * power(age);
          }
        }
      }
      TilesAB tiles;
      bf16x8 fc[kT][kIn];

      auto bring = [&](int64_t row, int held) __attribute__((always_inline)) {
        a.base = pa + row * p.as;
        b.base = pb + row * p.bs;
        tiles.load(places, a, b, !p.back, held);
      };
      auto put = [&]() __attribute__((always_inline)) {
        if (p.da < DA) tiles.settle(p.da);
        tiles.store(places, a, b);
      };
      auto bad = [&]() __attribute__((always_inline)) {
        return __any(tiles.any_bad(true)) ? tiles.first_bad(true) : C;
      };
      auto scores = [&](int, bool) __attribute__((always_inline)) {
        if constexpr (kOut) {
          const uint32_t at_row = fresh(row_base), at_col = fresh(col_base);
          // transposed: block (t, half) of 16 rows of b by rows 16 bi of a
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            if (!mine(m)) continue;
            const int bi = m ? 2 + pair : pair, t = m == 2;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < kS; ++s) {
              if (s && 32 * s >= p.da) break;
              bf16x8 fb[kIn], fa[kIn];
#pragma unroll
              for (int k = 0; k < kIn; ++k) {
                fb[k] = frag(lds.b[k], operand_at<DA / 8, false>(at_row, 2 * t + half, s));
                fa[k] = frag(lds.a[k], operand_at<DA / 8, false>(at_row, bi, s));
              }
              mma(acc, fb, fa);
            }
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[r] = ws[m][r] * acc[r];
              if (m != 1) x[r] = after + r <= 0 ? x[r] : 0.0f;
            }
            uint32_t piece[kMid][2];
            cut<sizeof(T) == 4, kMid, 4>(x, piece);
            const int f = bi < 2 ? bi : 2 * bi - 2 + t;
#pragma unroll
            for (int k = 0; k < kMid; ++k)
              *reinterpret_cast<u32x2*>(&lds.p[k][f][lane][4 * half]) =
                  u32x2{piece[k][0], piece[k][1]};
          }
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int k = 0; k < kIn; ++k)
              fc[t][k] = frag(lds.ct[k], operand_at<C / 8, true>(at_col, wave, t));
        }
      };
      auto output = [&](int64_t row, int held) __attribute__((always_inline)) {
        if constexpr (kOut) {
          f32x4 o[kI];
#pragma unroll
          for (int i = 0; i < kI; ++i) {
            o[i] = *reinterpret_cast<const f32x4*>(lds.from_state[wave][i][lane]);
#pragma unroll
            for (int t = 0; t <= i / 2; ++t) {
              bf16x8 fp[kMid];
              const int f = i < 2 ? i : 2 * i - 2 + t;
#pragma unroll
              for (int k = 0; k < kMid; ++k) fp[k] = frag(lds.p[k][f][lane], 0);
              mma(o[i], fc[t], fp);
            }
          }
          // rows i of the output: four channels of a row per lane where there are
          // four, else behind the buffer
          const int64_t to = row * p.os + (int64_t)h * p.dc;
          const uint32_t size = p.of ? 4 : (uint32_t)sizeof(T), pitch = (uint32_t)p.os * size;
          const auto buffer = buffer_of(p.of ? static_cast<const void*>(p.of + to) : p.o + to,
                                        (uint32_t)(held - 1) * pitch + (uint32_t)wide * size);
          constexpr uint32_t kNowhere = 0u - 16u;
          const int c = 16 * wave + 4 * g;
          const uint32_t side = (uint32_t)c * size;
          auto at_row = [&](int i) __attribute__((always_inline)) {
            const int r = 16 * i + n;
            return (uint32_t)(p.back ? held - 1 - r : r) * pitch + side;
          };
          const bool quad = c + 4 <= wide;
#pragma unroll
          for (int i = 0; i < kI; ++i) {
            const uint32_t at = quad ? at_row(i) : kNowhere;
            if (p.of || sizeof(T) == 4) {
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[i]), buffer, at,
                                                     0, 0);
            } else if constexpr (sizeof(T) == 2) {
              Packed<T, 4> y;
#pragma unroll
              for (int j = 0; j < 4; ++j) y.v[j] = (T)o[i][j];
              __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, y), buffer, at, 0, 0);
            }
          }
          if ((wide & 3) && works && 16 * wave + 16 > wide) {   // up to three at the end
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const bool on = !quad && c + j < wide && 16 * i + n < held;
                const uint32_t at = on ? at_row(i) + j * size : kNowhere;
                const float y = o[i][j];
                if (p.of || sizeof(T) == 4)
                  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, y), buffer,
                                                        at, 0, 0);
                else if constexpr (sizeof(T) == 2)
                  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)y),
                                                        buffer, at, 0, 0);
              }
          }
        }
      };
      each([&](int64_t, int64_t lo, int64_t hi, bool, bool) __attribute__((always_inline)) {
        chunks(lo, hi, bring, put, bad, scores, output);
      });
    } else {
      const T* pc = p.c + (int64_t)(h / p.share_c) * p.dc;
      const uint32_t sc = (uint32_t)(p.cs * sizeof(T));
      TileAt<T> c{pc, sc, wide, nullptr, lds.ct[0]};
      const typename TileC::Places places(c, c, !p.back, false);
      // the state's part that is held: half of it (a scale that would pass fp32 when
      // doubled takes all of it)
      const float part = __builtin_fabsf(p.beta) < 1e38f ? 0.5f : 1.0f, whole_of = 1.0f / part;
      float enter[kI];
      if constexpr (kOut) {
#pragma unroll
        for (int i = 0; i < kI; ++i) enter[i] = p.beta * whole_of * power(16 * i + n);
      }
      // of the rows that enter the state, `left` rows before the next chunk's first
      Decay whole;
      int left = -1;
      auto weigh = [&](int to) __attribute__((always_inline)) {
        if (to == left) return;
        left = to;
        whole = decay_of(decay, (float)to);
        if (lane < C)
          lds.weight[wave][lane] = lane <= to ? p.gamma * (part * power(to - lane)) : 0.0f;
      };

      f32x4 w[kU];
      // f(u, r, cell of the state) for this lane's values w[u][r] that are cells
      auto cells_of = [&](auto f) __attribute__((always_inline)) {
        const int c = fresh(16 * wave + n), a0 = fresh(8 * g);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int a = a0 + 32 * (u >> 1) + 4 * (u & 1) + r;
            if (a < p.da && c < p.dc) f(u, r, p.transposed ? c * p.da + a : a * p.dc + c);
          }
      };
      auto load_state = [&](const float* s, Decay d) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) w[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (s)
          cells_of([&](int u, int r, int i) __attribute__((always_inline)) {
            w[u][r] = decayed(d, s[i]);
          });
      };
      auto store_state = [&](float* s, float by) __attribute__((always_inline)) {
        cells_of([&](int u, int r, int i) __attribute__((always_inline)) { s[i] = w[u][r] * by; });
      };
      TileC tc;
      bool undecayed = false;   // the state behind the segment's last row is wanted so

      auto bring = [&](int64_t row, int held) __attribute__((always_inline)) {
        c.base = pc + row * p.cs;
        tc.load(places, c, c, !p.back, held);
      };
      auto put = [&]() __attribute__((always_inline)) {
        if (wide < kWide) tc.settle(wide);
        tc.store(places, c, c);
      };
      auto bad = [&]() __attribute__((always_inline)) {
        return __any(tc.any_bad(false)) ? tc.first_bad(false) : C;
      };
      auto update = [&](int held, bool end) __attribute__((always_inline)) {
        if (!works) return;
        const uint32_t at_row = fresh(row_base), at_col = fresh(col_base);
        if constexpr (kOut) {
          f32x4 o[kI];
#pragma unroll
          for (int i = 0; i < kI; ++i) o[i] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < kS; ++s) {
            if (s && 32 * s >= p.da) break;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = w[2 * s + e / 4][e & 3];
            uint32_t piece[kMid][4];
            cut<false, kMid, 8>(x, piece);
            bf16x8 fw[kMid];
#pragma unroll
            for (int k = 0; k < kMid; ++k) fw[k] = frag(piece[k]);
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              bf16x8 fa[kIn];
#pragma unroll
              for (int k = 0; k < kIn; ++k)
                fa[k] = frag(lds.a[k], operand_at<DA / 8, false>(at_row, i, s));
              mma(o[i], fw, fa);
            }
          }
#pragma unroll
          for (int i = 0; i < kI; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) o[i][r] *= enter[i];
            *reinterpret_cast<f32x4*>(lds.from_state[wave][i][lane]) = o[i];
          }
        }
        weigh(undecayed && end ? held - 1 : held);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) w[u][r] = decayed(whole, w[u][r]);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          bf16x8 fc[kIn];
#pragma unroll
          for (int k = 0; k < kIn; ++k)
            fc[k] = frag(lds.ct[k], operand_at<C / 8, true>(at_col, wave, t));
          const f32x4* weights =
              reinterpret_cast<const f32x4*>(&lds.weight[wave][32 * t + 8 * g]);
          const f32x4 w0 = weights[0], w1 = weights[1];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = 0.0f;
#pragma unroll
            for (int k = kIn - 1; k >= 0; --k) x[e] += (float)fc[k][e];
            x[e] *= e < 4 ? w0[e & 3] : w1[e & 3];
          }
          uint32_t piece[kState][4];
          cut<false, kState, 8>(x, piece);
          bf16x8 fw[kState];
#pragma unroll
          for (int k = 0; k < kState; ++k) fw[k] = frag(piece[k]);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            bf16x8 fb[kIn];
#pragma unroll
            for (int k = 0; k < kIn; ++k)
              fb[k] = frag(lds.bt[k], operand_at<C / 8, true>(at_col, u, t));
            mma(w[u], fb, fw);
          }
        }
      };
      // of a sequence's own initial state, before its first row and undecayed
      const Decay lambda = decay_of(decay, 1.0f);
      const Decay first = {part * lambda.hi, part * lambda.lo}, last = {part, 0.0f};
      each([&](int64_t i, int64_t lo, int64_t hi, bool starts, bool ends)
               __attribute__((always_inline)) {
        const int64_t of_seq = (i * p.heads + h) * cells;
        const float* in = p.state ? p.state + of_seq : nullptr;
        float* out = p.state_out ? p.state_out + of_seq : nullptr;
        if (kOut && lo >= hi) {   // an empty sequence
          if (starts && ends && out)
            cells_of([&](int, int, int i) __attribute__((always_inline)) {
              out[i] = in ? in[i] : 0.0f;
            });
          return;
        }
        // the state before the first row worked: the sequence's own, as its first row
        // meets it, or that of the place between two parts
        auto slot = [&](float* s, int64_t at) { return s + (at * p.heads + h) * cells; };
        const bool own = p.back ? ends : starts;
        const bool put_by = kOut && starts && !ends && walk.kept;
        const float* from = own ? (put_by ? slot(walk.kept, which) : in)
                            : kOut ? slot(walk.between, p.back ? which : which - 1)
                                   : nullptr;
        load_state(from, !own || put_by ? Decay{1.0f, 0.0f} : p.back ? last : first);
        if (!kOut && own && walk.kept) store_state(slot(walk.kept, which), 1.0f);
        undecayed = kOut && !p.back && ends;
        chunks(lo, hi, bring, put, bad, update, [](int64_t, int) {});
        if constexpr (!kOut)
          store_state(slot(walk.between, p.back ? which - 1 : which), 1.0f);
        else if ((p.back ? starts : ends) && out)
          store_state(out, whole_of);
      });
    }
  }
}

// The states between the parts, from those that each part makes: in order (from
// the last, backwards), the state that enters a part decays through it where
// its sequence does not end in it. A lane per cell; up to kRun places in a row are
// a wavefront's, read at once: 16 wavefronts go through theirs from 0, join what
// leaves them, and go through theirs again from what enters (254 places of 2 x 64 x
// 64 cells 12.5 us, 62 one after the other by one wavefront).
template <typename T>
__global__ __launch_bounds__(1024) void logmel_attn_between_kernel(AttnJob<T> p, Walk walk) {
  constexpr int kWaves = 16, kRun = 16;
  __shared__ float left[kWaves][64];
  __shared__ int goes[kWaves];   // whether what enters a wavefront's places leaves them
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t cells = (int64_t)p.da * p.dc, all = cells * p.heads;
  const int64_t x0 = (int64_t)blockIdx.x * 64 + lane, x = x0 < all ? x0 : all - 1;
  const int64_t count = walk.parts - 1;
  const int run = count >= kWaves * kRun ? kRun : (int)((count + kWaves - 1) / kWaves);
  const float decay = p.log_decay[x / cells];
  const Decay whole = decay_of(decay, (float)walk.part_rows);
  const Decay through = decay_of(decay, (float)(walk.part_rows * run));
  float enters = 0.0f;   // the state before place k0
  for (int64_t k0 = 0; k0 < count; k0 += kWaves * run) {
    float u[kRun];
    int how[kRun];   // 0 as well where there is no place
    auto place = [&](int m) {
      const int64_t k = k0 + wave * run + m;
      return p.back ? count - 1 - k : k;
    };
#pragma unroll
    for (int m = 0; m < kRun; ++m) {
      const bool on = m < run && k0 + wave * run + m < count;
      how[m] = on ? walk.through[place(m)] : 0;
      u[m] = on ? walk.between[place(m) * all + x] : 0.0f;
    }
    auto go = [&](float e, auto f) {
#pragma unroll
      for (int m = 0; m < kRun; ++m) {
        if (how[m] == 0) continue;   // what its place holds is not used
        e = how[m] == 2 ? u[m] + decayed(whole, e) : u[m];
        f(m, e);
      }
      return e;
    };
    bool kept = true;
#pragma unroll
    for (int m = 0; m < kRun; ++m) kept = kept && (m >= run || how[m] == 2);
    left[wave][lane] = go(0.0f, [](int, float) {});
    if (lane == 0) goes[wave] = kept;
    __syncthreads();
    float e = enters;
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) go(e, [&](int m, float y) {
        if (x0 < all) walk.between[place(m) * all + x] = y;
      });
      e = goes[w] ? left[w][lane] + decayed(through, e) : left[w][lane];
    }
    enters = e;
    __syncthreads();   // for the next places
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

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// How a call's rows are split over workgroups.
struct AttnSplit {
  enum How { kRows, kSequences, kParts } how;
  int64_t part_rows, parts;
};

// dc: the narrowest c of the jobs that share the split; widest: the longest row
// stride.
//
// The times are counted in chunks that one workgroup works one after the other. Both
// ways measured, us of n sequences of 2998 rows, 8 heads x 64 (bf16; fp32), parts and a
// workgroup per sequence:
//   n = 8     92, 158   (121, 278)
//   n = 16   122, 157   (195, 279)
//   n = 24   161, 159   (266, 280)
//   n = 32   197, 160   (331, 283)
//   n = 48   265, 211   (476, 408)
// of which parts are taken to n = 32, a fifth too long at its end. One sequence of 8
// heads: 384 rows bf16 50, 28 (taken), 1024 rows 53 (taken), 58; fp32 384 rows 51
// (taken), 43, 512 rows 52 (taken), 55.
AttnSplit split_of(const logmel_attention_input& in, int64_t dc, int64_t widest, int cus) {
  AttnSplit s{AttnSplit::kSequences, 0, 0};
  const int64_t longest =
      in.max_frames && in.max_frames < in.rows ? in.max_frames : in.rows;
  // a chunk's rows are addressed by 32 bits from its lowest one, in blocks of so
  // many values
  const int64_t block = in.type == LOGMEL_BF16 ? 8 : 4;
  if (longest <= kShort || widest >= (int64_t)1 << 22 || in.head_dk < block ||
      in.head_dv < block) {
    s.how = AttnSplit::kRows;
    return s;
  }
  const int64_t chunk = in.type == LOGMEL_BF16 ? 64 : 32;   // the output's at most widths
  const int64_t lanes = in.heads;   // workgroups side by side
  // those that are resident: of four columns' wavefronts two on a compute unit, of
  // eight one (70,001 x 6 x 40 x 71 fp16 287 us with one part for each, 336 with two
  // parts that take turns)
  const int64_t slots = (dc > 64 ? 1 : 2) * (int64_t)cus;
  // times in chunks one after the other
  const int64_t by_seq = ceil_div(longest, chunk);
  const int64_t seq_all = ceil_div(in.rows, chunk) * lanes / slots;
  const double seq_time = (double)(by_seq > seq_all ? by_seq : seq_all);
  const int64_t most = slots / lanes;   // parts in one round of workgroups
  int64_t rows = ceil_div(ceil_div(in.rows, most < 1 ? 1 : most), chunk) * chunk;
  rows = rows < 4 * chunk ? 4 * chunk : rows;
  const int64_t parts = ceil_div(in.rows, rows);
  // the states between parts are formed in a pass of their own, counted as half of the
  // output's (0.38 of it for 521,998 x 2 x 64 fp32), and joined by a launch, counted
  // as four chunks
  const double part_time =
      1.5 * (double)(rows / chunk) * (double)ceil_div(parts * lanes, slots) + 4.0;
  if (parts > 1 && part_time < seq_time) {
    s.how = AttnSplit::kParts;
    s.part_rows = rows;
    s.parts = parts;
  }
  return s;
}

// Where the parts of a call have what in its workspace, in floats: the states
// between them (of one job at a time), their `through`, the initial states kept.
struct PartSpace {
  int64_t between, through, kept;
  PartSpace(const AttnSplit& s, const logmel_attention_input& in, bool keep)
      : between(0), through(0), kept(0) {
    if (s.how != AttnSplit::kParts) return;
    const int64_t state = in.heads * in.head_dk * in.head_dv;
    between = (s.parts - 1) * state;
    through = s.parts;
    kept = keep ? s.parts * state : 0;
  }
  int64_t all() const { return between + through + kept; }
};

template <typename T, int DA, int kWaves>
hipError_t launch_chunks(const AttnJob<T>& p, const AttnSplit& s, Walk k, bool between,
                         hipStream_t stream) {
  // of up to 1024 threads, of which a launch takes fewer than 2^32
  auto grid = [](int64_t items) { return (unsigned)(items < (1 << 20) ? items : 1 << 20); };
  if (s.how == AttnSplit::kParts) {
    k.part_rows = s.part_rows;
    k.parts = s.parts;
    k.items = s.parts * p.heads;
    if (between) {
      logmel_attn_chunk_kernel<T, DA, kWaves, false>
          <<<grid(k.items), 128 * kWaves, 0, stream>>>(p, k);
      logmel_attn_between_kernel<T>
          <<<(unsigned)ceil_div((int64_t)p.heads * p.da * p.dc, 64), 1024, 0, stream>>>(p, k);
    }
  } else {
    k.items = p.n_seq * p.heads;
  }
  logmel_attn_chunk_kernel<T, DA, kWaves, true>
      <<<grid(k.items), 128 * kWaves, 0, stream>>>(p, k);
  return hipGetLastError();
}

// One job. between: whether the states between its parts are yet to be formed.
template <typename T>
hipError_t launch_job(const AttnJob<T>& p, const AttnSplit& s, const PartSpace& space, float* ws,
                      bool between, hipStream_t stream) {
  if (s.how == AttnSplit::kRows) {
    const int slabs = (p.dc + kSlab - 1) / kSlab;
    const int64_t items = p.n_seq * p.heads * slabs;
    const unsigned grid = (unsigned)(items < (1 << 22) ? items : 1 << 22);
    if (p.da <= 64)
      logmel_attn_rows_kernel<T, 64><<<grid, 256, 0, stream>>>(p, slabs, items);
    else
      logmel_attn_rows_kernel<T, 128><<<grid, 256, 0, stream>>>(p, slabs, items);
    return hipGetLastError();
  }
  Walk k{};
  k.between = ws;
  k.through = reinterpret_cast<int*>(ws + space.between);
  k.kept = space.kept ? ws + space.between + space.through : nullptr;
  auto go = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    if (p.da <= 32) return launch_chunks<T, 32, W>(p, s, k, between, stream);
    if (p.da <= 64) return launch_chunks<T, 64, W>(p, s, k, between, stream);
    return launch_chunks<T, 128, W>(p, s, k, between, stream);
  };
  return p.dc <= 64 ? go(std::integral_constant<int, 4>{}) : go(std::integral_constant<int, 8>{});
}

int64_t longest_of(std::initializer_list<int64_t> strides) {
  int64_t most = 0;
  for (int64_t s : strides) most = s > most ? s : most;
  return most;
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
  const AttnSplit s = split_of(
      in, p.dc, longest_of({in.q_stride, in.k_stride, in.v_stride, o_stride}), cus);
  const PartSpace space(s, in, state_out && state_out == in.d_state);
  return launch_job(p, s, space, static_cast<float*>(ws), true, stream);
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
  const int64_t widest =
      longest_of({in.q_stride, in.k_stride, in.v_stride, g.do_stride, g.dq_stride, g.dk_stride,
                  g.dv_stride, share > 1 ? in.heads * dk : 0});
  const AttnSplit of_q = split_of(in, dk, widest, cus);
  const AttnSplit of_kv = split_of(in, dk < dv ? dk : dv, widest, cus);   // they share the states
  // the shared heads' parts first, then the splits'
  float* part = share > 1 ? static_cast<float*>(ws) : nullptr;
  float* between = static_cast<float*>(ws) + (part ? in.rows * in.heads * dk : 0);
  // a gradient of q or k: its own rows, or each head's first and then their sums
  auto shared = [&](AttnJob<T>& p, const AttnSplit& s, void* out, int64_t stride) {
    p.o = static_cast<T*>(out);
    p.of = part;
    p.os = part ? in.heads * dk : stride;
    hipError_t e = launch_job(p, s, PartSpace(s, in, false), between, true, stream);
    if (e != hipSuccess || !part) return e;
    const int64_t n = in.rows * in.qk_heads * dk;
    const int64_t blocks = (n + 255) / 256;
    if (n)
      logmel_attn_share_kernel<T>
          <<<(unsigned)(blocks < cus * 8 ? blocks : cus * 8), 256, 0, stream>>>(
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
  hipError_t e = shared(p, of_q, g.d_dq, g.dq_stride);
  if (e != hipSuccess) return e;
  p.back = true;                  // dk
  p.a = v, p.as = in.v_stride;
  p.b = d, p.bs = g.do_stride;
  p.c = q, p.cs = in.q_stride;
  p.state = g.d_dstate_out;
  p.beta = 1.0f, p.gamma = in.scale;
  e = shared(p, of_kv, g.d_dk, g.dk_stride);
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
  // its states are those of dk
  return launch_job(p, of_kv, PartSpace(of_kv, in, false), between, false, stream);
}

}  // namespace
}  // namespace logmel

int64_t logmel_attention_workspace(const logmel_attention_input& in, int backward, int cus) {
  using namespace logmel;
  if (!in.n_seq) return 0;
  const int64_t dk = in.head_dk, dv = in.head_dv;
  auto parts = [&](int64_t dc) {
    return PartSpace(split_of(in, dc, 0, cus), in, !backward && in.d_state).all();
  };
  if (!backward) return parts(dv) * 4;
  const int64_t share = in.heads > in.qk_heads ? in.rows * in.heads * dk : 0;
  const int64_t of_q = parts(dk), of_kv = parts(dk < dv ? dk : dv);
  return (share + (of_q > of_kv ? of_q : of_kv)) * 4;
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
