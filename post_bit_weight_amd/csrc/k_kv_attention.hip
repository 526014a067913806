// Attention over the 4-bit cache.
//
// A value s c + o (code c, scale s and offset o of its group) becomes an fp16 number, rounded once, on its way to
// the matrix cores: the code OR-ed into the mantissa of 1024 is the fp16 number 1024 + c, less 1024 is c, and one packed
// fused multiply-add makes two values.  All of that is exact up to the one rounding (2^-11 relative; s and o are fp16,
// so that small values are exact multiples of 2^-24, and the cache holds nothing beyond fp16's range), an eighth of what bf16 would lose.
// Queries are scaled by a power of two each, which the scores give back, and fit fp16 exactly.  Weights are kept
// as 2^15 times what they are relative to the row's largest: fp16 then holds those down to 2^-39 of it.
// The scores come out transposed (a lane holds four tokens of one query), which is the layout in which the second product
// takes its weights: nothing crosses lanes but the maximum.
#include "kv_cache.hpp"

namespace wr {

namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr int kPaged = 1024;  // tokens whose pages a wave holds: one of 64 tiles of 16 a lane

constexpr float kLift = 15.0f;   // log2 of what a row's largest weight is held as

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma16x16x32_f16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {  // round to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}
// The values of the codes in bits 0..3 and 16..19, with a scale and an offset for each.
__device__ __forceinline__ uint32_t two_values(uint32_t w, f16x2 scale, f16x2 off) {
  const f16x2 lifted = __builtin_bit_cast(f16x2, (w & 0x000f000fu) | 0x64006400u);
  const f16x2 c = lifted - f16x2{(_Float16)1024.0f, (_Float16)1024.0f};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, scale, off));
}
__device__ __forceinline__ f16x2 low_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(b, a, 0x05040100u));
}
__device__ __forceinline__ f16x2 high_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(b, a, 0x07060302u));
}

struct AttentionArgs {
  KvArgs kv;
  const uint16_t* q;
  uint16_t* out;
  float* part;   // unnormalised outputs of the chunks: (row, head, chunk, dim)
  f32x2* stats;  // their maximum (of log2 weights) and sum: (row, head, chunk)
  int64_t ldq, ldo;
  int heads, share;  // query heads, and how many of them share a head of the cache
  float scale;       // times log2(e)
  int window;
  bool causal;
  int chunk, splits;  // tokens a workgroup takes, chunks of a row at most
};

// The positions that queries first .. last of a sequence see: lo .. hi - 1.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span seen(const AttentionArgs& a, const KvSeq& s, int first, int last) {
  const int64_t p0 = (int64_t)s.length - s.fresh + first, p1 = (int64_t)s.length - s.fresh + last;
  int64_t hi = a.causal ? p1 + 1 : a.window ? p1 + a.window : s.length;
  if (hi > s.length) hi = s.length;
  int64_t lo = a.window ? p0 - a.window + 1 : 0;
  if (lo < 0) lo = 0;
  if (hi < lo) hi = lo;
  return Span{(int)lo, (int)hi};
}

// The queries of a tile of rows (query, head of the share), numbered query first.
struct RowTile {
  int first, last;
};
__device__ __forceinline__ RowTile row_tile(const AttentionArgs& a, const KvSeq& s, int tile, int rows) {
  const uint32_t m0 = tile * rows, m1 = min(m0 + rows, (uint32_t)(s.fresh * a.share)) - 1;
  return RowTile{(int)(m0 / (uint32_t)a.share), (int)(m1 / (uint32_t)a.share)};
}

// ---------------------------------------------------------------- few rows: 16 NT of them against one chunk
template <int DIM, int GROUP, int NT>
__global__ __launch_bounds__(256) void attend_rows_kernel(AttentionArgs a, int tiles) {
  constexpr int SL = DIM / 32;      // slices of 32 dims: dwords a lane loads of a tile
  constexpr int NG = DIM / GROUP;
  constexpr int WAVES = 4;
  __shared__ __attribute__((aligned(16))) float sums[16 * NT][DIM + 4];
  __shared__ float tops[WAVES][16 * NT], dens[WAVES][16 * NT];

  uint32_t block = blockIdx.x;
  const int head = block % (uint32_t)a.kv.heads;
  block /= (uint32_t)a.kv.heads;
  const int tile = block % (uint32_t)tiles;
  block /= (uint32_t)tiles;
  const int split = block % (uint32_t)a.splits;
  const int seq = block / (uint32_t)a.splits;

  const KvSeq s = kv_seq(a.kv, seq);
  if (s.fresh <= 0 || tile * 16 * NT >= s.fresh * a.share) return;
  const RowTile rt = row_tile(a, s, tile, 16 * NT);
  const Span all = seen(a, s, rt.first, rt.last);
  const int begin = (all.lo & ~15) + split * a.chunk;
  const int end = min(all.hi, begin + a.chunk);
  if (split > 0 && begin >= end) return;  // the first chunk of rows that see nothing writes their zeros

  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int col = lane % 16, g = lane / 16;

  // queries, as fp16 times 2^-e each; unit: what turns a product into log2 of a weight
  u32x4 qr[NT][SL];
  float unit[NT];
  Span mine[NT];
  const Span first = seen(a, s, rt.first, rt.first), last = seen(a, s, rt.last, rt.last);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t m = tile * 16 * NT + 16 * n + col;
    const bool live = m < (uint32_t)(s.fresh * a.share);
    const int j = m / (uint32_t)a.share, h = head * a.share + m % (uint32_t)a.share;
    mine[n] = live ? seen(a, s, j, j) : Span{0, 0};
    const uint16_t* qp = a.q + (int64_t)(s.row + (live ? j : 0)) * a.ldq + (int64_t)(live ? h : 0) * DIM + 8 * g;
    Raw8<uint16_t> x[SL];
    float big = 0.0f;
#pragma unroll
    for (int sl = 0; sl < SL; ++sl) {
      x[sl].load(qp + 32 * sl);
#pragma unroll
      for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[sl].get(e)));
    }
    big = fmaxf(big, __shfl_xor(big, 16));
    big = fmaxf(big, __shfl_xor(big, 32));
    // 2^e <= big < 2^(e + 1), within what has a reciprocal in fp32
    const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -120), 120);
    const float down = live ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.0f;
    unit[n] = a.scale * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int sl = 0; sl < SL; ++sl)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // codes i and 4 + i of a dword go together
        qr[n][sl][i] = live ? pack_f16(x[sl].get(i) * down, x[sl].get(4 + i) * down) : 0u;
  }

  f32x4 acc[NT][2][SL];  // [half][m]: dims half * DIM / 2 + 16 m + 4 g + r
  float top[NT], den[NT];
  const f32x4 zero{0, 0, 0, 0};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    top[n] = kLowest;
    den[n] = 0.0f;
#pragma unroll
    for (int m = 0; m < SL; ++m) acc[n][0][m] = acc[n][1][m] = zero;
  }

  const KvLayout<DIM, GROUP> at{1 << a.kv.page_shift};
  const int64_t page_bytes = (int64_t)a.kv.heads * at.head_bytes();
  const uint8_t* cache = a.kv.pages + (int64_t)head * at.head_bytes();
  const int32_t* table = a.kv.table + (int64_t)seq * a.kv.ldt;
  int pages = -1;

  for (int t0 = begin + 32 * wave; t0 < end; t0 += 32 * WAVES) {
    const int nth0 = (t0 - begin) % kPaged / 16;
    if (nth0 < 2 * WAVES) {
      const int t = t0 + 16 * (lane - nth0);
      pages = t < end ? table[t >> a.kv.page_shift] : -1;
    }
    uint32_t kc[2][SL], vc[2][SL];
    uint32_t km[2][NG];
    u32x4 vm[2][NG];
    bool there[2];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      const int t = t0 + 16 * tt;
      int page = __builtin_amdgcn_readlane(pages, nth0 + tt);
      there[tt] = t < end && page >= 0 && page < a.kv.count;
      if (!there[tt]) page = 0;
      const int in_page = t & (at.page_tokens - 1);
      const uint8_t* base = cache + page * page_bytes;
      const uint8_t* kp = base + in_page * (DIM / 2) + col * (DIM / 2) + g * (DIM / 8);
      const uint8_t* vp = base + at.v_codes() + in_page * (DIM / 2) + lane * (DIM / 8);
      __builtin_memcpy(kc[tt], __builtin_assume_aligned(kp, DIM / 8 < 16 ? DIM / 8 : 16), SL * 4);
      __builtin_memcpy(vc[tt], __builtin_assume_aligned(vp, DIM / 8 < 16 ? DIM / 8 : 16), SL * 4);
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        km[tt][k] = *reinterpret_cast<const uint32_t*>(base + at.k_meta() + (k * at.page_tokens + in_page + col) * 4);
        vm[tt][k] = *reinterpret_cast<const u32x4*>(base + at.v_meta() + (k * at.page_tokens + in_page + 4 * g) * 4);
      }
    }
    // every row sees all of these 32 tokens
    const bool whole = there[0] && there[1] && t0 + 32 <= min(first.hi, last.hi) && t0 >= max(first.lo, last.lo);

    f32x4 score[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) score[n][0] = score[n][1] = zero;
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        const uint32_t meta = km[tt][sl * 32 / GROUP], w = kc[tt][sl];
        const f16x2 sc = low_halves(meta, meta), of = high_halves(meta, meta);
        const u32x4 keys{two_values(w, sc, of), two_values(w >> 4, sc, of), two_values(w >> 8, sc, of), two_values(w >> 12, sc, of)};
#pragma unroll
        for (int n = 0; n < NT; ++n) score[n][tt] = mfma16x16x32_f16(keys, qr[n][sl], score[n][tt]);
      }

    u32x4 weights[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[2][4];
      float high = kLowest;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[tt][i] = score[n][tt][i] * unit[n];
          if (!whole) {
            const int t = t0 + 16 * tt + 4 * g + i;
            if (!(there[tt] && t >= mine[n].lo && t < mine[n].hi)) p[tt][i] = -INFINITY;
          }
          high = fmaxf(high, p[tt][i]);
        }
      high = fmaxf(high, __shfl_xor(high, 16));
      high = fmaxf(high, __shfl_xor(high, 32));
      if (__builtin_amdgcn_ballot_w64(high > top[n]) != 0) {
        const float now = fmaxf(high, top[n]);
        const float keep = exp2_fast(top[n] - now);
        top[n] = now;
        den[n] *= keep;
#pragma unroll
        for (int m = 0; m < SL; ++m) {
          acc[n][0][m] *= keep;
          acc[n][1][m] *= keep;
        }
      }
      const float less = top[n] - kLift;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[tt][i] = exp2_fast(p[tt][i] - less);
          den[n] += p[tt][i];
        }
      weights[n] = u32x4{pack_f16(p[0][0], p[0][2]), pack_f16(p[0][1], p[0][3]), pack_f16(p[1][0], p[1][2]),
                         pack_f16(p[1][1], p[1][3])};
    }
    if (!whole) {
      // A token that a row does not see may hold NaNs or anything, which its weight of 0 would not hide: what no row
      // sees becomes 0, and a NaN goes to the rows that see it by itself.
      int poison[NT] = {};
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 16 * tt + 4 * g + i;
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            if (!(there[tt] && t >= all.lo && t < all.hi)) vm[tt][k][i] = 0;
            if ((vm[tt][k][i] & 0x7fffu) <= 0x7c00u) continue;
            vm[tt][k][i] = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (t >= mine[n].lo && t < mine[n].hi) poison[n] |= 1 << k;
          }
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (__builtin_amdgcn_ballot_w64(poison[n] != 0) == 0) continue;
        poison[n] |= __shfl_xor(poison[n], 16);
        poison[n] |= __shfl_xor(poison[n], 32);
#pragma unroll
        for (int m = 0; m < SL; ++m)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            if (poison[n] >> ((half * (DIM / 2) + 16 * m) / GROUP) & 1)
              acc[n][half][m] = f32x4{NAN, NAN, NAN, NAN};
      }
    }
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      f16x2 sc[2][2], of[2][2];  // tokens 0 and 2, 1 and 3
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sc[tt][i] = low_halves(vm[tt][k][i], vm[tt][k][i + 2]);
          of[tt][i] = high_halves(vm[tt][k][i], vm[tt][k][i + 2]);
        }
#pragma unroll
      for (int m = 0; m < SL; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if ((half * (DIM / 2) + 16 * m) / GROUP != k) continue;
          const int sh = 4 * half;
          const u32x4 values{two_values(vc[0][m] >> sh, sc[0][0], of[0][0]), two_values(vc[0][m] >> (8 + sh), sc[0][1], of[0][1]),
                             two_values(vc[1][m] >> sh, sc[1][0], of[1][0]), two_values(vc[1][m] >> (8 + sh), sc[1][1], of[1][1])};
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n][half][m] = mfma16x16x32_f16(values, weights[n], acc[n][half][m]);
        }
    }
  }

  // the waves' parts: one maximum, then the sums in the waves' order
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    den[n] += __shfl_xor(den[n], 16);
    den[n] += __shfl_xor(den[n], 32);
    if (g == 0) {
      tops[wave][16 * n + col] = top[n];
      dens[wave][16 * n + col] = den[n];
    }
  }
  __syncthreads();
  float keep[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float now = kLowest;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) now = fmaxf(now, tops[w][16 * n + col]);
    keep[n] = exp2_fast(top[n] - now);
  }
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (wave == w) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < SL; ++m)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            f32x4* dst = reinterpret_cast<f32x4*>(&sums[16 * n + col][half * (DIM / 2) + 16 * m + 4 * g]);
            const f32x4 v = acc[n][half][m] * keep[n];
            *dst = w ? *dst + v : v;
          }
    }
    __syncthreads();
  }
  for (int u = threadIdx.x; u < 16 * NT * (DIM / 4); u += 256) {
    const int r = u / (DIM / 4), d = u % (DIM / 4) * 4;
    const uint32_t m = tile * 16 * NT + r;
    if (m >= (uint32_t)(s.fresh * a.share)) break;
    const int64_t row = s.row + m / (uint32_t)a.share;
    const int h = head * a.share + m % (uint32_t)a.share;
    float now = kLowest, total = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) now = fmaxf(now, tops[w][r]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) total += dens[w][r] * exp2_fast(tops[w][r] - now);
    const f32x4 v = *reinterpret_cast<const f32x4*>(&sums[r][d]);
    if (a.splits == 1) {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      u32x2_any o;
      o[0] = pack_bf16(v[0] * inv, v[1] * inv);
      o[1] = pack_bf16(v[2] * inv, v[3] * inv);
      *reinterpret_cast<u32x2_any*>(a.out + row * a.ldo + (int64_t)h * DIM + d) = o;
    } else {
      const int64_t slot = (row * a.heads + h) * a.splits + split;
      *reinterpret_cast<f32x4*>(a.part + slot * DIM + d) = v;
      if (d == 0) a.stats[slot] = f32x2{now, total};
    }
  }
}

// The chunks' parts of a row, added in the chunks' order: a wave a row and head.
template <int DIM>
__global__ __launch_bounds__(256) void attend_join_kernel(AttentionArgs a, int tile_rows) {
  constexpr int PER = DIM / kWave;
  const int lane = threadIdx.x % kWave;
  const uint32_t unit = blockIdx.x * 4 + threadIdx.x / kWave;
  const int h = unit % (uint32_t)a.heads;
  const uint32_t rest = unit / (uint32_t)a.heads;
  const int j = rest % (uint32_t)a.kv.most_new;
  const int seq = rest / (uint32_t)a.kv.most_new;
  if (seq >= a.kv.n) return;
  const KvSeq s = kv_seq(a.kv, seq);
  if (j >= s.fresh) return;
  const int m = j * a.share + h % a.share;
  const RowTile rt = row_tile(a, s, m / tile_rows, tile_rows);
  const Span all = seen(a, s, rt.first, rt.last);
  const int parts = min(a.splits, max(1, (all.hi - (all.lo & ~15) + a.chunk - 1) / a.chunk));
  const int64_t slot = ((int64_t)(s.row + j) * a.heads + h) * a.splits;
  float top = kLowest;
  for (int c = lane; c < parts; c += kWave) top = fmaxf(top, a.stats[slot + c].x);
  for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  float sum[PER], total = 0.0f;
#pragma unroll
  for (int e = 0; e < PER; ++e) sum[e] = 0.0f;
#pragma unroll 4
  for (int c = 0; c < parts; ++c) {
    const f32x2 st = a.stats[slot + c];
    const float keep = exp2_fast(st.x - top);
    total = fmaf(st.y, keep, total);
#pragma unroll
    for (int e = 0; e < PER; ++e) sum[e] = fmaf(a.part[(slot + c) * DIM + e * kWave + lane], keep, sum[e]);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* o = a.out + (int64_t)(s.row + j) * a.ldo + (int64_t)h * DIM;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e * kWave + lane] = (uint16_t)f32_to_bf16_bits(sum[e] * inv);
}

struct Plan {
  int chunk, splits;
  int64_t tiles;  // row tiles of a sequence and head
};

constexpr int kTileRows = 16;
constexpr int kWanted = 2048;  // workgroups: eight for every compute unit

Plan plan_of(const wr_kv_cache& c, const wr_kv_seqs& s, int heads, int flags, int window) {
  const int share = heads / c.heads;
  Plan p;
  p.tiles = ((int64_t)s.most_new * share + kTileRows - 1) / kTileRows;
  // positions that a tile's rows can see, from a multiple of 16
  const int64_t queries = std::min<int64_t>(s.most_new, (kTileRows + share - 2) / share + 1);
  int64_t span = std::min<int64_t>(s.most_tokens, (int64_t)s.width * c.page_tokens);
  if (window > 0) span = std::min(span, (int64_t)window * (flags & WR_ATTENTION_CAUSAL ? 1 : 2) + queries + 15);
  const int64_t groups = std::max<int64_t>(1, s.n * p.tiles * c.heads);
  const int64_t most_splits = std::max<int64_t>(1, kWanted / groups);
  int64_t chunk = std::max<int64_t>(128, (span + most_splits - 1) / most_splits);
  chunk = (chunk + 127) / 128 * 128;
  p.chunk = (int)std::min<int64_t>(chunk, 1 << 30);
  p.splits = (int)std::max<int64_t>(1, (span + chunk - 1) / chunk);
  return p;
}

}  // namespace

}  // namespace wr

using namespace wr;

// The chunks are split off only up to kWanted workgroups, each with kTileRows rows at most.
size_t wr_kv_attention_ws_bytes(int64_t rows, int64_t n, int32_t dim) {
  const int64_t parts = kWanted * std::min<int64_t>(kTileRows, rows * (n / dim));
  return (size_t)parts * (dim + 2) * sizeof(float);
}

int wr_kv_attention_impl(wr_ctx* ctx, const wr_kv_cache& c, const wr_kv_seqs& s, const void* q, int64_t ldq, int64_t rows,
                         int32_t heads, float scale, int flags, int32_t window, void* out, int64_t ldo) {
  const Plan p = plan_of(c, s, heads, flags, window);
  const int64_t blocks = (int64_t)s.n * p.splits * p.tiles * c.heads;
  const int64_t joins = ((int64_t)s.n * s.most_new * heads + 3) / 4;
  if (blocks > 1 << 30 || joins > 1 << 29) return WR_EUNSUPPORTED;
  if (p.splits > 1 && ctx->ws_bytes < (size_t)rows * heads * p.splits * (c.dim + 2) * sizeof(float)) return WR_EWORKSPACE;
  AttentionArgs a;
  a.kv = kv_args(c, s, rows);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.part = static_cast<float*>(ctx->ws);
  a.stats = reinterpret_cast<f32x2*>(a.part + (size_t)rows * heads * p.splits * c.dim);
  a.ldq = ldq;
  a.ldo = ldo;
  a.heads = heads;
  a.share = heads / c.heads;
  a.scale = scale * 1.4426950408889634f;
  a.window = window;
  a.causal = flags & WR_ATTENTION_CAUSAL;
  a.chunk = p.chunk;
  a.splits = p.splits;
  const bool there = kv_form(c.dim, c.group, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    hipLaunchKernelGGL((attend_rows_kernel<D, G, 1>), dim3((uint32_t)blocks), dim3(256), 0, ctx->stream, a, (int)p.tiles);
    if (p.splits > 1)
      hipLaunchKernelGGL(attend_join_kernel<D>, dim3((uint32_t)joins), dim3(256), 0, ctx->stream, a, kTileRows);
  });
  if (!there) return WR_EUNSUPPORTED;
  WR_CHECK_LAUNCH();
  return WR_OK;
}
