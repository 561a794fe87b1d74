// Device helpers of the row operators (gated scan, block norm): row operands
// in fp32, fp16 or bf16, read and written as fp32 values, V neighbouring
// channels per lane.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace logmel {

using bf16_t = __bf16;
using f16_t = _Float16;

// V values at p, of any element alignment: the hardware's global accesses
// need no more than their dword (for two 2-byte values: no) alignment.
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Packed {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Packed<T, V> row_load(const T* p) {
  Packed<T, V> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void row_store(T* p, const float (&x)[V]) {
  Packed<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = (T)x[i];   // to nearest even, once
  __builtin_memcpy(p, &r, sizeof(r));
}

// sigmoid(g) and sigmoid(-g), each to full relative precision: e = e^-|g| is
// at most 1, so neither is formed as 1 minus the other. A NaN gives two NaN.
// fp32 rows correct e for the rounding of |g| log2(e) (|g| 2^-24 relative in
// e, ten ulps at |g| = 10); 2-byte rows, whose own rounding is 2^-11 or 2^-8,
// do without those four instructions.
template <typename T>
__device__ __forceinline__ void gate_pair(float g, float& a, float& u) {
  constexpr float kLog2e = 1.44269504088896340736f;
  const float x = -__builtin_fabsf(g);
  const float t = x * kLog2e;
  float e = __builtin_amdgcn_exp2f(t);
  if constexpr (sizeof(T) == 4) {
    constexpr float kLn2 = 0.693147180559945309417f;
    constexpr float kLog2eRest = (float)(1.44269504088896340735992468 - (double)kLog2e);
    const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
    // e is 0 from x = -inf on down: rest is NaN at -inf
    e = e == 0.0f ? e : __builtin_fmaf(e, rest * kLn2, e);
  }
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float s = e * r;
  a = g >= 0.0f ? r : s;
  u = g >= 0.0f ? s : r;
}

}  // namespace logmel
