// Helpers of the kernels that walk rows of activations: eight consecutive values per lane as 16- or
// 32-byte loads and stores of any alignment, sums and maxima over the lanes of a row, and the rounding
// to 8-bit integers.
#pragma once
#include "common.hpp"

namespace wr {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Global memory takes 16-byte accesses at any address; the types' alignment says so to the compiler.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// Eight consecutive values of a row as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {  // bf16 bit patterns
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_any*>(p); }
  __device__ __forceinline__ void load_part(const uint16_t* p, int cnt) {
    v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cnt) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
  }
};
template <>
struct Raw8<float> {
  u32x4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = *reinterpret_cast<const u32x4_any*>(p);
    hi = *reinterpret_cast<const u32x4_any*>(p + 4);
  }
  __device__ __forceinline__ void load_part(const float* p, int cnt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = e < cnt ? __float_as_uint(p[e]) : 0u;
      hi[e] = e + 4 < cnt ? __float_as_uint(p[e + 4]) : 0u;
    }
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(e < 4 ? lo[e & 3] : hi[e & 3]); }
};

// The eight values at column c of a row of n (zeros past its end).
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* row, int c, int n) {
  if (c + 8 <= n) {
    r.load(row + c);
  } else {
    r.load_part(row + c, n - c);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ void store8(uint16_t* row, int c, int n, const float (&f)[8]) {
  const u32x4 v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  if (c + 8 <= n) {
    *reinterpret_cast<u32x4_any*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ void store8(float* row, int c, int n, const float (&f)[8]) {
  if (c + 8 <= n) {
    const u32x4 lo = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    const u32x4 hi = {__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
    *reinterpret_cast<u32x4_any*>(row + c) = lo;
    *reinterpret_cast<u32x4_any*>(row + c + 4) = hi;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = f[e];
  }
}

// ---------------------------------------------------------------- reductions over the lanes of a row
struct AddF32 {
  static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct MaxU32 {
  static __device__ __forceinline__ uint32_t op(uint32_t a, uint32_t b) { return a > b ? a : b; }
};

template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Over aligned groups of LANES (a power of two, 8..64) lanes; every lane gets the result, formed in
// the same order on each.  Up to 16 lanes the partners come by DPP inside a row of 16, then by shuffles.
template <typename OP, int LANES, typename T>
__device__ __forceinline__ T lanes_reduce(T v) {
  v = OP::op(v, dpp<0xB1>(v));   // lane ^ 1
  v = OP::op(v, dpp<0x4E>(v));   // lane ^ 2
  v = OP::op(v, dpp<0x141>(v));  // the other four of eight
  if constexpr (LANES >= 16) v = OP::op(v, dpp<0x140>(v));  // the other eight of sixteen
  if constexpr (LANES >= 32) v = OP::op(v, __shfl_xor(v, 16));
  if constexpr (LANES >= 64) v = OP::op(v, __shfl_xor(v, 32));
  return v;
}

// The lanes that share a row: LANES of a wave, or (LANES == 0) the whole workgroup of up to 16 waves.
// `side` alternates between two LDS buffers, so one barrier per reduction is enough: a buffer is
// written again only after the next reduction's barrier, by which every wave has read it.
template <int LANES>
struct RowGroup {
  static constexpr int kMaxWaves = 16;
  uint32_t (*lds)[3][kMaxWaves];
  int side = 0;

  template <typename OP, int K, typename T>
  __device__ __forceinline__ void reduce(T (&v)[K]) {
    if constexpr (LANES > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = lanes_reduce<OP, LANES>(v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = lanes_reduce<OP, 64>(v[k]);
      const int waves = blockDim.x >> 6;
      if (waves > 1) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int k = 0; k < K; ++k) lds[side][k][threadIdx.x >> 6] = __builtin_bit_cast(uint32_t, v[k]);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
          v[k] = __builtin_bit_cast(T, lds[side][k][0]);
          for (int w = 1; w < waves; ++w) v[k] = OP::op(v[k], __builtin_bit_cast(T, lds[side][k][w]));
        }
        side ^= 1;
      }
    }
  }
  __device__ __forceinline__ float sum(float v) {
    float a[1] = {v};
    reduce<AddF32>(a);
    return a[0];
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    uint32_t a[1] = {v};
    reduce<MaxU32>(a);
    return a[0];
  }
};

// ---------------------------------------------------------------- 8-bit integers
// One row's rounding q = rint(127 v / m), m = max |v|, from the bits of m.  As integers the bit
// patterns of |v| order NaN > infinity > finite, so a row with either has m_bits >= 0x7f800000.  The
// quotient is the correctly rounded one of fl(127 v) and m, but divides only near a tie:
// fl(127 v) * fl(1 / m) is within 1.5 units in the last place of it (below 127: 1.2e-5), so a value
// further than 4e-5 from a half rounds the same way.  A division of every value instead takes twelve more
// instructions for each.
// Very large and very small rows are scaled by a power of two first (exact where it matters: what
// falls below the fp32 range there rounds to code 0 either way).
struct RowCoder {
  float m, inv, pre;
  bool live;
  float scale;
  __device__ __forceinline__ explicit RowCoder(uint32_t m_bits) {
    const float top = __uint_as_float(m_bits);
    scale = m_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : top / 127.0f;
    live = m_bits != 0u && m_bits < 0x7f800000u;
    pre = top > 0x1p100f ? 0x1p-30f : top < 0x1p-80f ? 0x1p70f : 1.0f;
    m = live ? top * pre : 1.0f;
    inv = 1.0f / m;
  }
  // Eight codes as bytes, the first in the lowest.
  __device__ __forceinline__ u32x2_any codes(const float (&v)[8]) const {
    float p[8], t[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = live ? v[e] * pre * 127.0f : 0.0f;
      t[e] = p[e] * inv;
      near |= fabsf(__builtin_amdgcn_fractf(t[e]) - 0.5f) < 4e-5f;
    }
    if (near)
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = p[e] / m;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= ((uint32_t)(int)rintf(t[e]) & 0xffu) << (8 * (e & 3));
    return u32x2_any{w[0], w[1]};
  }
};

__device__ __forceinline__ void store_codes(int8_t* row, int c, int n, const u32x2_any& v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u32x2_any*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (int8_t)(v[e >> 2] >> (8 * (e & 3)));
  }
}

}  // namespace wr
