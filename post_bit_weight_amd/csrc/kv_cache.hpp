// The paged cache of keys and values in 4 bits: where everything in a page lies, and what a call's sequences are.
#pragma once
#include "rowops.hpp"

namespace wr {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int64_t kMostThreads = 4294967295;  // of a launch, in x

// What keys and values saturate at: the largest code's value, off + 15 scale with both rounded to fp16, stays in
// fp16's range (off is off by 16 at most, scale by 4: 65024 + 16 + 60 < 65504).
constexpr float kKvMost = 65024.0f;

// Places in a page, in bytes, for heads of DIM values in groups of GROUP.
template <int DIM, int GROUP>
struct KvLayout {
  static constexpr int kGroups = DIM / GROUP;
  static constexpr int kTileBytes = 16 * DIM / 2;  // the codes of 16 tokens
  int page_tokens;
  __host__ __device__ __forceinline__ int codes() const { return page_tokens * (DIM / 2); }
  __host__ __device__ __forceinline__ int metas() const { return page_tokens * (4 * kGroups); }
  __host__ __device__ __forceinline__ int head_bytes() const { return 2 * (codes() + metas()); }
  __device__ __forceinline__ int v_codes() const { return codes(); }
  __device__ __forceinline__ int k_meta() const { return 2 * codes(); }
  __device__ __forceinline__ int v_meta() const { return 2 * codes() + metas(); }
  // Among the values' fp16 numbers: the scale of a token; its offset is two behind it.
  __device__ __forceinline__ int v_scale(int first, int token) const {
    return 2 * (first + (token & ~3)) + 4 * (token & 1) + (token >> 1 & 1);
  }
};

// What a kernel gets of wr_kv_cache and wr_kv_seqs.
struct KvArgs {
  uint8_t* pages;
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* table;
  int64_t ldt;
  int64_t rows;
  int32_t count;         // pages (clamped to what an int32 page number reaches)
  int32_t heads, page_shift;  // page_tokens = 1 << page_shift
  int32_t n, most_new, most_tokens;  // most_tokens at most width * page_tokens
};

struct KvSeq {
  int row, fresh, length;  // first row, rows, positions; fresh = -1: left out
};

// Every bound that a kernel relies on: rows in 0 .. rows - 1, positions in the table.
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int i) {
  const int b = a.starts[i], e = a.starts[i + 1], length = a.lengths[i];
  const bool ok = b >= 0 && e >= b && e <= a.rows && e - b <= a.most_new && length >= 0 && length <= a.most_tokens;
  return KvSeq{b, ok ? e - b : -1, length};
}

// Calls f(dim, group) with both as compile-time constants; false for a form that is not there.
template <typename F>
bool kv_form(int dim, int group, F&& f) {
  using std::integral_constant;
  auto with = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (group == 32) return f(d, integral_constant<int, 32>{}), true;
    if (group == 64) return f(d, integral_constant<int, 64>{}), true;
    if constexpr (D >= 128)
      if (group == 128) return f(d, integral_constant<int, 128>{}), true;
    return false;
  };
  if (dim == 64) return with(integral_constant<int, 64>{});
  if (dim == 128) return with(integral_constant<int, 128>{});
  if (dim == 256) return with(integral_constant<int, 256>{});
  return false;
}

KvArgs kv_args(const wr_kv_cache& c, const wr_kv_seqs& s, int64_t rows);

}  // namespace wr
