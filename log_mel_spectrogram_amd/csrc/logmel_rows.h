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

// The same values to a reader, to the compiler new ones: what is unpacked from
// them afterwards is unpacked anew (an instruction per 2-byte value) instead
// of being held as floats, in up to twice the registers, since its last use.
template <typename T, int V>
__device__ __forceinline__ void repack(Packed<T, V>& p) {
  if constexpr (sizeof(p) % 4 == 0) {
    struct Words {
      uint32_t w[sizeof(p) / 4];
    };
    Words x = __builtin_bit_cast(Words, p);
#pragma unroll
    for (size_t i = 0; i < sizeof(p) / 4; ++i) asm("" : "+v"(x.w[i]));
    p = __builtin_bit_cast(Packed<T, V>, x);
  } else {
    static_assert(sizeof(p) == 2);
    uint16_t x = __builtin_bit_cast(uint16_t, p);
    asm("" : "+v"(x));
    p = __builtin_bit_cast(Packed<T, V>, x);
  }
}

template <typename T, int V>
__device__ __forceinline__ void row_store(T* p, const float (&x)[V]) {
  Packed<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = (T)x[i];   // to nearest even, once
  __builtin_memcpy(p, &r, sizeof(r));
}

// sigmoid(g + bias) and sigmoid(-(g + bias)), each to full relative precision:
// with e = e^-(g + bias) they are r = 1 / (1 + e) and e r, and neither is
// formed as 1 minus the other. The exponent is kept below 2^126 so that e is
// finite and r is not flushed: from g + bias = -87 on down r would stay at
// 1e-38, which of a state near fp32's largest value leaves ones, so there a is
// 0, in 2-byte rows too: their states are fp32, and the caller's (two
// instructions: 1 to 2 % of a 2-byte call's time).
// minimum and maximum are those that return a NaN operand, so a NaN gate gives
// two NaN. Six instructions of a 2-byte row beside the two transcendentals,
// which take as long: the recurrence reads 4 bytes per value and is held up by
// instructions as much as by memory (see the tiles).
// 2-byte rows take the bias into the exponent's multiply-add (nb = -bias
// log2(e)): e is off by (|g + bias| + |bias|) 2^-24 relative. fp32 rows add
// first and correct e for the rounding of the product (|g| 2^-24 in e, ten
// ulps at |g| = 10).
template <typename T>
struct Gate {
  static constexpr float kLog2e = 1.44269504088896340736f;
  static constexpr float kClosed = 5e37f;   // the largest e there is is 6.0e37
  static __device__ __forceinline__ float bias_of(float bias) {
    return sizeof(T) == 4 ? bias : -bias * kLog2e;
  }
  static __device__ __forceinline__ void pair(float g, float b, float& a, float& u) {
    float e;
    if constexpr (sizeof(T) == 4) {
      constexpr float kLn2 = 0.693147180559945309417f;
      constexpr float kRest = (float)(1.44269504088896340735992468 - (double)kLog2e);
      float x = __builtin_elementwise_maximum(g + b, -87.0f);
      x = __builtin_elementwise_minimum(x, 110.0f);   // e is 0 from 88 on
      const float t = x * -kLog2e;
      const float rest = __builtin_fmaf(x, -kRest, __builtin_fmaf(x, -kLog2e, -t));
      e = __builtin_amdgcn_exp2f(t);
      e = __builtin_fmaf(e, rest * kLn2, e);
    } else {
      e = __builtin_amdgcn_exp2f(
          __builtin_elementwise_minimum(__builtin_fmaf(g, -kLog2e, b), 125.5f));
    }
    a = __builtin_amdgcn_rcpf(1.0f + e);
    u = e * a;
    a = e > kClosed ? 0.0f : a;
  }
  // a alone, of a gate without a bias: nothing needs e finite for 2-byte rows.
  static __device__ __forceinline__ float sigmoid(float g) {
    float a, u;
    if constexpr (sizeof(T) == 4)
      pair(g, 0.0f, a, u);
    else
      a = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -kLog2e));
    return a;
  }
};

}  // namespace logmel
