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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Eight values of a row as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {  // bf16 bit patterns
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_any*>(p); }
  __device__ __forceinline__ void fill(float f) {
    const uint32_t h = f32_to_bf16_bits(f) * 0x10001u;
    v = u32x4{h, h, h, h};
  }
  __device__ __forceinline__ void set(int e, uint16_t h) {
    v[e >> 1] = e & 1 ? (v[e >> 1] & 0xffffu) | (uint32_t)h << 16 : (v[e >> 1] & 0xffff0000u) | h;
  }
  __device__ __forceinline__ void round(const float (&f)[8]) {  // to nearest even
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = pack_bf16(f[2 * d], f[2 * d + 1]);
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<u32x4_any*>(p) = v; }
  __device__ __forceinline__ uint16_t at(int e) const { return (uint16_t)(v[e >> 1] >> (16 * (e & 1))); }
  __device__ __forceinline__ void mask(int keep) {  // zeros where bit e of keep is clear
#pragma unroll
    for (int d = 0; d < 4; ++d)
      v[d] &= (uint32_t)(__builtin_amdgcn_sbfe(keep, 2 * d, 1) & 0xffff) | (uint32_t)__builtin_amdgcn_sbfe(keep, 2 * d + 1, 1) << 16;
  }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
  }
};
template <>
struct Raw8<float> {
  u32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const u32x4_any*>(p);
    v[1] = *reinterpret_cast<const u32x4_any*>(p + 4);
  }
  __device__ __forceinline__ void fill(float f) {
    const uint32_t h = __float_as_uint(f);
    v[0] = v[1] = u32x4{h, h, h, h};
  }
  __device__ __forceinline__ void set(int e, float f) { v[e >> 2][e & 3] = __float_as_uint(f); }
  __device__ __forceinline__ void round(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) set(e, f[e]);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<u32x4_any*>(p) = v[0];
    *reinterpret_cast<u32x4_any*>(p + 4) = v[1];
  }
  __device__ __forceinline__ void mask(int keep) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] &= (uint32_t)__builtin_amdgcn_sbfe(keep, e, 1);
  }
  __device__ __forceinline__ float at(int e) const { return get(e); }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(v[e >> 2][e & 3]); }
};

// ---------------------------------------------------------------- which values a thread owns
// A row of n values lies on LANES lanes of a wave, or (LANES == 0) on a whole workgroup; a thread owns CH
// chunks of eight columns.  So that every access is one full vector inside the row, the chunk that would
// pass the row's end starts at n - 8 instead: it holds up to seven values of its neighbour as well, which
// count in sums only where they are owned (`keep`) and are otherwise treated like the thread's own, so that both
// store the same results there.  Lanes beyond the row load the last chunk, own nothing and store nothing.
// LANES == 8 is for rows of fewer than eight values: the first lane of eight holds them all, one by one.
template <int CH, int LANES>
struct RowMap {
  uint32_t col[CH];
  int keep[CH];
  int n;
  bool ragged;  // some lane of this wave does not own all it holds (uniform)
  __device__ __forceinline__ RowMap(int lane, int cstep, int n_) : n(n_) {
    bool part = false;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if constexpr (LANES == 8) {
        col[k] = 0;
        keep[k] = lane == 0 ? (1 << n) - 1 : 0;
      } else {
        col[k] = c < n - 8 ? c : n - 8;
        keep[k] = c < n ? (0xff << (c - (int)col[k])) & 0xff : 0;
      }
      part |= keep[k] != 0xff;
    }
    ragged = __builtin_amdgcn_ballot_w64(part) != 0;
  }
  // Where chunk k of a row starts: a uniform pointer plus a 32-bit offset of the lane, which needs no 64-bit
  // address registers.
  template <typename T>
  __device__ __forceinline__ T* at(T* row, int k) const {
    using C = typename std::conditional<std::is_const<T>::value, const char, char>::type;
    return reinterpret_cast<T*>(reinterpret_cast<C*>(row) + (uint32_t)(col[k] * sizeof(T)));
  }
  template <typename T>
  __device__ __forceinline__ void load(Raw8<T>& r, const T* row, int k) const {
    if constexpr (LANES == 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.set(e, row[e < n ? e : n - 1]);
    } else {
      r.load(at(row, k));
    }
  }
  // keep[k] for the rare paths, unknown to the compiler before them: it would else form every mask and
  // condition ahead of the row loop and hold them in registers.
  __device__ __forceinline__ int bits(int k) const {
    int b = keep[k];
    asm volatile("" : "+v"(b));
    return b;
  }
  // Zeros in the place of what chunk k holds but does not own.
  __device__ __forceinline__ void own(float (&v)[8], int k) const {
    if (ragged) {
      const int b = bits(k);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(__float_as_uint(v[e]) & (uint32_t)__builtin_amdgcn_sbfe(b, e, 1));
    }
  }
  template <typename T>
  __device__ __forceinline__ void own(Raw8<T>& r, int k) const {
    if (ragged) r.mask(bits(k));
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int k, const Raw8<T>& r) const {
    if (keep[k] == 0) return;
    if constexpr (LANES == 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) row[e] = r.at(e);
    } else {
      r.store(at(row, k));
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int k, const float (&f)[8]) const {
    Raw8<T> r;
    r.round(f);
    store(row, k, r);
  }
  __device__ __forceinline__ void store(int8_t* row, int k, const u32x2_any& v) const {
    if (keep[k] == 0) return;
    if constexpr (LANES == 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) row[e] = (int8_t)(v[e >> 2] >> (8 * (e & 3)));
    } else {
      *reinterpret_cast<u32x2_any*>(at(row, k)) = v;
    }
  }
  // Only what the chunk owns: for rows of which each thread has zeros in its neighbours' places (the gradient, whose
  // registers hold no more), and for values that are read, changed and stored.
  template <typename T>
  __device__ __forceinline__ void store_own(T* row, int k, const Raw8<T>& r) const {
    if (keep[k] == 0xff) {
      r.store(at(row, k));
    } else if (keep[k]) {
      const int b = bits(k);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (b >> e & 1) at(row, k)[e] = r.at(e);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store_own(T* row, int k, const float (&f)[8]) const {
    Raw8<T> r;
    r.round(f);
    store_own(row, k, r);
  }
};

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
// the same order on each.  The partners come by DPP inside a row of 16 lanes, then by swapping rows
// and halves of the wave (a swap of a register with itself leaves one half in each result).
template <typename OP, int LANES, typename T>
__device__ __forceinline__ T lanes_reduce(T v) {
  v = OP::op(v, dpp<0xB1>(v));   // lane ^ 1
  v = OP::op(v, dpp<0x4E>(v));   // lane ^ 2
  v = OP::op(v, dpp<0x141>(v));  // the other four of eight
  if constexpr (LANES >= 16) v = OP::op(v, dpp<0x140>(v));  // the other eight of sixteen
  if constexpr (LANES >= 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = OP::op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  if constexpr (LANES >= 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = OP::op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
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
      const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = lanes_reduce<OP, 64>(v[k]);
      if (waves > 1) {
        if (lane == 0)
#pragma unroll
          for (int k = 0; k < K; ++k) lds[side][k][threadIdx.x >> 6] = __builtin_bit_cast(uint32_t, v[k]);
        // LDS only: loads of a later row may stay in flight across the barrier
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        // every 16 lanes add the waves' values in the same order (0 is neutral for both operations)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const uint32_t u = lds[side][k][lane & 15];
          v[k] = lanes_reduce<OP, 16>(__builtin_bit_cast(T, (lane & 15) < waves ? u : 0u));
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

}  // namespace wr
