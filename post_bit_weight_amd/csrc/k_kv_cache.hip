// Writing rows of keys and values into the 4-bit cache and reading them back.
//
// Both stream: a value is 2 or 4 bytes on the row side and half a byte (plus 4 bytes a group) in the cache, so the
// bound is memory.  A workgroup takes 16 consecutive positions of one head that start at a multiple of 16, which is a
// tile of the values' layout: it alone writes the tile's dwords, and no two workgroups share a byte.  16384 tokens of eight heads of
// 128 in bf16 are written in 27 us (88 MB, 3.3 TB/s: vector instructions issue for 19 of them) and read in 18 (4.8 TB/s).
#include "kv_cache.hpp"

namespace wr {

namespace {

constexpr int kThreads = 256;

// One of the 16-token tiles that a sequence's rows touch, for one head.
struct Tile {
  int row0;        // row of the tile's first position (below the first row for positions that are not rows)
  int from, to;    // tokens of the tile that are rows
  int page;        // outside 0 .. count - 1: absent
  int at;          // the tile's first token in its page
};

// Blocks take `per` heads of a tile, so that many of them share the latency of finding it; they are numbered heads fastest, then tile,
// then sequence.
struct Work {
  int tiles, per;  // tiles of a sequence, heads of a block
};
__device__ __forceinline__ bool tile_of(const KvArgs& a, const Work& w, uint32_t block, int& head, Tile& t) {
  const uint32_t parts = (a.heads + w.per - 1) / (uint32_t)w.per, rest = block / parts;
  head = (block - rest * parts) * w.per;
  const int i = rest / (uint32_t)w.tiles, nth = rest - (uint32_t)i * w.tiles;
  const KvSeq s = kv_seq(a, i);
  if (s.fresh <= 0) return false;
  const int first = s.length - s.fresh;             // position of the first row; below 0 where rows have none
  const int tile = (first >= 0 ? first / 16 : -((15 - first) / 16)) + nth;  // floor
  const int p0 = 16 * tile;
  if (p0 >= s.length) return false;
  t.row0 = s.row + p0 - first;
  t.from = max(first - p0, 0);
  t.to = min(s.length - p0, 16);
  t.page = -1;
  if (tile >= 0) {  // a whole tile is on one side of position 0
    t.page = a.table[(int64_t)i * a.ldt + (p0 >> a.page_shift)];
    t.at = p0 & ((1 << a.page_shift) - 1);
  }
  return true;
}

// The value of the lane that differs in the bit STEP (1, 2, 4 or 8) of a row of 16; for 4 and 8 some lane of the other half, which is the
// same where the lanes of each half agree already.
template <int STEP>
__device__ __forceinline__ float across(float v) {
  constexpr int ctrl = STEP == 1 ? 0xb1 : STEP == 2 ? 0x4e : STEP == 4 ? 0x141 : 0x140;  // quad_perm, half mirror, mirror
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), ctrl, 0xf, 0xf, true));
}

// The codes of a lane's eight values and the scale and offset of the LANES lanes that share a group.
template <int LANES, typename T>
__device__ __forceinline__ void group_codes(const Raw8<T>& raw, uint32_t& codes, uint32_t& meta) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = raw.get(e);
  auto least = [](float a, float b) { return __builtin_elementwise_minimum(a, b); };  // NaN where there is one
  auto most = [](float a, float b) { return __builtin_elementwise_maximum(a, b); };
  float lo = least(least(x[0], x[1]), x[2]), hi = most(most(x[0], x[1]), x[2]);
#pragma unroll
  for (int e = 3; e < 7; e += 2) {
    lo = least(least(lo, x[e]), x[e + 1]);
    hi = most(most(hi, x[e]), x[e + 1]);
  }
  lo = least(lo, x[7]);
  hi = most(hi, x[7]);
  static_for<0, LANES == 4 ? 2 : LANES == 8 ? 3 : 4>([&](auto n) {
    constexpr int step = 1 << decltype(n)::value;
    lo = least(lo, across<step>(lo));
    hi = most(hi, across<step>(hi));
  });
  const bool finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
  if (__builtin_amdgcn_ballot_w64(lo < -kKvMost || hi > kKvMost)) {
    asm volatile("");
    lo = fminf(fmaxf(lo, -kKvMost), kKvMost);
    hi = fminf(fmaxf(hi, -kKvMost), kKvMost);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -kKvMost), kKvMost);
  }
  // Quotients correctly rounded, by Markstein's theorem: with y the correctly rounded reciprocal of the divisor, q = d y and the
  // exact rest r = d - q divisor, q + r y rounds to the quotient.  One Newton step makes y out of a reciprocal that is
  // off by up to two units in the last place, for every divisor of eleven bits.
  auto quotient = [](float d, float divisor, float y) {
    const float q = d * y;
    return fmaf(fmaf(-q, divisor, d), y, q);
  };
  const uint16_t off_bits = __builtin_bit_cast(uint16_t, (_Float16)lo);
  const float off = f16_bits_to_f32(off_bits);
  float step = quotient(hi - off, 15.0f, 1.0f / 15.0f);
  asm("" : "+v"(step));  // rounded to fp32 first: an instruction that rounds the last product and sum straight to fp16 differs at ties
  const uint16_t scale_bits = __builtin_bit_cast(uint16_t, (_Float16)step);
  const float scale = f16_bits_to_f32(scale_bits);
  meta = finite ? scale_bits | (uint32_t)off_bits << 16 : 0x7e007e00u;
  const bool some = finite && scale > 0.0f;
  const float divisor = some ? scale : 1.0f, y0 = __builtin_amdgcn_rcpf(divisor);
  const float y = fmaf(fmaf(-divisor, y0, 1.0f), y0, y0);
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = rintf(__builtin_amdgcn_fmed3f(quotient(x[e] - off, divisor, y), 0.0f, 15.0f));
  }
  const uint32_t low = (uint32_t)fmaf(4096.0f, c[3], fmaf(256.0f, c[2], fmaf(16.0f, c[1], c[0])));
  const uint32_t high = (uint32_t)fmaf(4096.0f, c[7], fmaf(256.0f, c[6], fmaf(16.0f, c[5], c[4])));
  codes = some ? low | high << 16 : 0u;
}

template <int DIM, int GROUP, typename T>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvArgs a, Work work, const T* __restrict__ k, int64_t ldk,
                                                            const T* __restrict__ v, int64_t ldv) {
  constexpr int UNITS = DIM / 8;  // of eight values a token
  __shared__ uint32_t vcodes[2][16][UNITS + 1];
  constexpr int ITERS = 2 * 16 * UNITS / kThreads;  // a wave has units of either k or v
  Tile t;
  int head;
  if (!tile_of(a, work, blockIdx.x, head, t)) return;
  const int end = min(head + work.per, a.heads);
  Raw8<T> x[ITERS];
  bool live[ITERS];
  auto load = [&](int h) {
#pragma unroll
    for (int n = 0; n < ITERS; ++n) {
      const int u = threadIdx.x + n * kThreads;
      const bool values = u >= 16 * UNITS;
      const int token = u / UNITS % 16, c = u % UNITS;
      const T* src = values ? v : k;
      live[n] = src && token >= t.from && token < t.to;
      if (live[n]) x[n].load(src + (int64_t)(t.row0 + token) * (values ? ldv : ldk) + h * DIM + 8 * c);
    }
  };
  load(head);
  if (t.page < 0 || t.page >= a.count) return;
  const KvLayout<DIM, GROUP> at{1 << a.page_shift};
  uint8_t* base = a.pages + (int64_t)t.page * ((int64_t)a.heads * at.head_bytes()) + (int64_t)head * at.head_bytes();
  for (int which = 0; head < end; ++head, which ^= 1, base += at.head_bytes()) {
    uint32_t codes[ITERS], meta[ITERS];
#pragma unroll
    for (int n = 0; n < ITERS; ++n) {
      codes[n] = meta[n] = 0;
      if (__builtin_amdgcn_ballot_w64(live[n])) group_codes<GROUP / 8>(x[n], codes[n], meta[n]);
    }
    if (head + 1 < end) load(head + 1);  // on its way while these are stored
#pragma unroll
    for (int n = 0; n < ITERS; ++n) {
      if (!live[n]) continue;
      const int u = threadIdx.x + n * kThreads;
      const bool values = u >= 16 * UNITS;
      const int token = u / UNITS % 16, c = u % UNITS, in_page = t.at + token;
      if (values)
        vcodes[which][token][c] = codes[n];
      else
        *reinterpret_cast<uint32_t*>(base + in_page * (DIM / 2) + (c % 4) * (DIM / 8) + (c / 4) * 4) = codes[n];
      if (c % (GROUP / 8) == 0) {
        const int first = (c / (GROUP / 8)) * at.page_tokens;
        if (values) {
          uint16_t* m = reinterpret_cast<uint16_t*>(base + at.v_meta()) + at.v_scale(first, in_page);
          m[0] = (uint16_t)meta[n];
          m[2] = (uint16_t)(meta[n] >> 16);
        } else {
          *reinterpret_cast<uint32_t*>(base + at.k_meta() + (first + in_page) * 4) = meta[n];
        }
      }
    }
    if (!v) continue;
    __syncthreads();
    uint8_t* tile = base + at.v_codes() + t.at * (DIM / 2);
    for (int w = threadIdx.x; w < 2 * DIM; w += kThreads) {  // the tile's dwords
      const int m = w % (DIM / 32), l = w / (DIM / 32) % 16, g = w / (DIM / 2);
      const int d = 16 * m + l;
      uint32_t word = 0;
      int there = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = 4 * g + i;
        if (token >= t.from && token < t.to) {
          const uint32_t lo = vcodes[which][token][d / 8] >> (4 * (d % 8)) & 15u;
          const uint32_t hi = vcodes[which][token][(DIM / 2 + d) / 8] >> (4 * (d % 8)) & 15u;
          word |= (lo | hi << 4) << (8 * i);
          there |= 1 << i;
        }
      }
      if (there == 15) {
        *reinterpret_cast<uint32_t*>(tile + 4 * w) = word;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (there >> i & 1) tile[4 * w + i] = (uint8_t)(word >> (8 * i));
      }
    }
  }
}

template <int DIM, int GROUP, typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvArgs a, Work work, T* __restrict__ k, int64_t ldk,
                                                           T* __restrict__ v, int64_t ldv) {
  constexpr int UNITS = DIM / 8;
  __shared__ uint32_t vtile[2][2 * DIM];
  Tile t;
  int head;
  if (!tile_of(a, work, blockIdx.x, head, t)) return;
  const int end = min(head + work.per, a.heads);
  const bool there = t.page >= 0 && t.page < a.count;
  const KvLayout<DIM, GROUP> at{1 << a.page_shift};
  const uint8_t* base = a.pages + (int64_t)(there ? t.page : 0) * ((int64_t)a.heads * at.head_bytes()) + (int64_t)head * at.head_bytes();
  for (int which = 0; head < end; ++head, which ^= 1, base += at.head_bytes()) {
    if (v) {
      const uint8_t* tile = base + at.v_codes() + t.at * (DIM / 2);
      if (there)
        for (int w = threadIdx.x; w < 2 * DIM; w += kThreads) vtile[which][w] = *reinterpret_cast<const uint32_t*>(tile + 4 * w);
      __syncthreads();
    }
    for (int u = threadIdx.x; u < 2 * 16 * UNITS; u += kThreads) {
      const bool values = u >= 16 * UNITS;
      const int token = u / UNITS % 16, c = u % UNITS;
      T* dst = values ? v : k;
      if (!dst || token < t.from || token >= t.to) continue;
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (there) {
        const int in_page = t.at + token;
        const int first = (c / (GROUP / 8)) * at.page_tokens;
        const uint16_t* m = values ? reinterpret_cast<const uint16_t*>(base + at.v_meta()) + at.v_scale(first, in_page)
                                   : reinterpret_cast<const uint16_t*>(base + at.k_meta()) + 2 * (first + in_page);
        const float scale = f16_bits_to_f32(m[0]), off = f16_bits_to_f32(m[values ? 2 : 1]);
        uint32_t codes;
        if (values) {
          codes = 0;
          const int cc = c % (UNITS / 2), shift = 8 * (token % 4) + (c >= UNITS / 2 ? 4 : 0);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = 8 * cc + e;
            codes |= (vtile[which][((token / 4) * 16 + d % 16) * (DIM / 32) + d / 16] >> shift & 15u) << (4 * e);
          }
        } else {
          codes = *reinterpret_cast<const uint32_t*>(base + in_page * (DIM / 2) + (c % 4) * (DIM / 8) + (c / 4) * 4);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf((float)(codes >> (4 * e) & 15u), scale, off);  // the product is exact
      }
      Raw8<T> r;
      r.round(f);
      r.store(dst + (int64_t)(t.row0 + token) * (values ? ldv : ldk) + head * DIM + 8 * c);
    }
  }
}

}  // namespace

KvArgs kv_args(const wr_kv_cache& c, const wr_kv_seqs& s, int64_t rows) {
  KvArgs a;
  a.pages = static_cast<uint8_t*>(c.pages);
  a.starts = s.starts;
  a.lengths = s.lengths;
  a.table = s.table;
  a.ldt = s.ldt;
  a.rows = rows;
  a.count = (int32_t)std::min<int64_t>(c.count, 2147483647);
  a.heads = c.heads;
  a.page_shift = __builtin_ctz((unsigned)c.page_tokens);
  a.n = s.n;
  a.most_new = s.most_new;
  a.most_tokens = (int32_t)std::min<int64_t>(s.most_tokens, (int64_t)s.width * c.page_tokens);
  return a;
}

}  // namespace wr

using namespace wr;

// Tiles that most_new consecutive positions can touch.
static int64_t tiles_of(const wr_kv_seqs& s) { return ((int64_t)s.most_new + 14) / 16 + 1; }

int64_t wr_kv_blocks(const wr_kv_cache& c, const wr_kv_seqs& s) { return (int64_t)c.heads * s.n * tiles_of(s); }

// One head a block until the card is full eight times over, then as many as leave it that.  False: more blocks than a launch has.
static bool work_of(wr_ctx* ctx, const wr_kv_cache& c, const wr_kv_seqs& s, dim3& grid, Work& work) {
  const int64_t full = 8 * (int64_t)ctx->num_cu, tiles = s.n * tiles_of(s);
  const int per = (int)std::min<int64_t>(c.heads, std::max<int64_t>(1, c.heads * tiles / full));
  const int64_t blocks = tiles * ((c.heads + per - 1) / per);
  grid = dim3((uint32_t)blocks);
  work = Work{(int)tiles_of(s), per};
  return blocks <= kMostThreads / kThreads;
}

int wr_kv_write_impl(wr_ctx* ctx, const wr_kv_cache& c, const wr_kv_seqs& s, const void* k, int64_t ldk, const void* v,
                     int64_t ldv, int dtype, int64_t rows) {
  const KvArgs a = kv_args(c, s, rows);
  dim3 grid;
  Work work;
  if (!work_of(ctx, c, s, grid, work)) return WR_EUNSUPPORTED;
  const bool there = kv_form(c.dim, c.group, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    if (dtype == WR_BF16)
      hipLaunchKernelGGL((kv_write_kernel<D, G, uint16_t>), grid, dim3(kThreads), 0, ctx->stream, a, work,
                         static_cast<const uint16_t*>(k), ldk, static_cast<const uint16_t*>(v), ldv);
    else
      hipLaunchKernelGGL((kv_write_kernel<D, G, float>), grid, dim3(kThreads), 0, ctx->stream, a, work,
                         static_cast<const float*>(k), ldk, static_cast<const float*>(v), ldv);
  });
  if (!there) return WR_EUNSUPPORTED;
  WR_CHECK_LAUNCH();
  return WR_OK;
}

int wr_kv_read_impl(wr_ctx* ctx, const wr_kv_cache& c, const wr_kv_seqs& s, void* k, int64_t ldk, void* v, int64_t ldv,
                    int dtype, int64_t rows) {
  const KvArgs a = kv_args(c, s, rows);
  dim3 grid;
  Work work;
  if (!work_of(ctx, c, s, grid, work)) return WR_EUNSUPPORTED;
  const bool there = kv_form(c.dim, c.group, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    if (dtype == WR_BF16)
      hipLaunchKernelGGL((kv_read_kernel<D, G, uint16_t>), grid, dim3(kThreads), 0, ctx->stream, a, work,
                         static_cast<uint16_t*>(k), ldk, static_cast<uint16_t*>(v), ldv);
    else
      hipLaunchKernelGGL((kv_read_kernel<D, G, float>), grid, dim3(kThreads), 0, ctx->stream, a, work,
                         static_cast<float*>(k), ldk, static_cast<float*>(v), ldv);
  });
  if (!there) return WR_EUNSUPPORTED;
  WR_CHECK_LAUNCH();
  return WR_OK;
}
