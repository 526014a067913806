// Attention over the 4-bit cache for many rows: prompts and chunks of prompts.
//
// A workgroup of four waves takes 128 RT rows (query, head of the share) of a sequence and head of the cache, a wave 32 RT
// of them.  The workgroup turns the codes of a tile of tokens into fp16 values in LDS once, in the order in which the
// matrix cores take them, while it works on the tile before; every wave reads all of them.  Per 32 x 32 scores a wave
// reads 8 KB of keys and as much of values for each 32 tokens (128 dims): with RT = 1 that alone would keep LDS as busy
// as the matrix cores, so RT is 2 where registers allow.  Three tiles lie in LDS, so that one barrier a tile is enough.
// Scores are formed for the next 32 tokens while the weights of the present ones are: both are in one stretch of
// code, and the matrix cores have something to do beside the exponentials.
#include "kv_attention.hpp"

namespace wr {

namespace {

__device__ __forceinline__ f32x16 mfma32x32x16_f16(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ float max_of_two(float v) {  // lanes that differ in bit 5
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// The token of accumulator register v of half h in 32 scores, and the dim of an output likewise.
__device__ __forceinline__ int at_reg(int v, int h) { return 8 * (v >> 2) + 4 * h + (v & 3); }

template <int DIM, int GROUP>
struct Tile {
  static constexpr int TOKENS = DIM == 256 ? 32 : 64;
  static constexpr int SL = DIM / 32;
  // keys: [block of 32][step of 16 dims][half][token]; values: [16 tokens][32 dims][half][dim], 16 bytes each
  u32x4 keys[TOKENS / 32][DIM / 16][2][32];
  u32x4 values[TOKENS / 16][DIM / 32][2][32];
  int bad[4];  // a wave has met a NaN among the values
};

template <int DIM, int GROUP, int RT>
__global__ __launch_bounds__(256, 1) void attend_many_kernel(AttentionArgs a, uint32_t tiles) {
  using T = Tile<DIM, GROUP>;
  constexpr int TOKENS = T::TOKENS, NB = TOKENS / 32, KS = DIM / 16, SL = DIM / 32, ROWS = 128 * RT;
  constexpr int XT = DIM / 32;                 // tiles of 32 dims
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* buf = reinterpret_cast<T*>(lds);

  uint32_t block = blockIdx.x;
  const int head = block % (uint32_t)a.kv.heads;
  block /= (uint32_t)a.kv.heads;
  const int seq = block % (uint32_t)a.kv.n;
  block /= (uint32_t)a.kv.n;
  const int split = block % (uint32_t)a.splits;
  const int tile = tiles - 1 - block / (uint32_t)a.splits;  // those that see most first

  const KvSeq s = kv_seq(a.kv, seq);
  if (s.fresh <= 0 || tile * ROWS >= s.fresh * a.share) return;
  const RowTile rt = row_tile(a, s, tile, ROWS);
  const Span all = seen(a, s, rt.first, rt.last);
  const int begin = (all.lo & ~15) + split * a.chunk;
  const int end = min(all.hi, begin + a.chunk);
  if (split > 0 && begin >= end) return;  // the first chunk of rows that see nothing writes their zeros

  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane % 32, h = lane / 32;
  const KvLayout<DIM, GROUP> at{1 << a.kv.page_shift};
  const int64_t page_bytes = (int64_t)a.kv.heads * at.head_bytes();
  const uint8_t* cache = a.kv.pages + (int64_t)head * at.head_bytes();
  const int32_t* table = a.kv.table + (int64_t)seq * a.kv.ldt;
  const Unpack unpack;

  // ---- codes of a tile on their way from memory to LDS
  // keys: a thread has part g (DIM / 8 bytes) of a token; values: 2 M dims m .. of the quads h and 2 + h of 16 tokens
  constexpr int KT = TOKENS * 4 / 256 > 0 ? 256 : TOKENS * 4;  // threads with keys
  constexpr int VM = SL * TOKENS / 16 * 2 * 16 / 256;           // neighbouring m a thread takes
  static_assert(KT == TOKENS * 4 && VM * 256 == SL * TOKENS * 2, "a thread has one unit of keys and one of values");
  const int k_token = threadIdx.x % TOKENS, k_part = threadIdx.x / TOKENS;
  const int v_l = threadIdx.x % 16, v_h = threadIdx.x / 16 % 2, v_m = threadIdx.x / 32 % (SL / VM) * VM,
            v_16 = threadIdx.x / 32 / (SL / VM);
  struct Raw {
    uint32_t k[SL], km[DIM / GROUP], v[2][VM];
    u32x4 vm[2][2];  // quad; low or high half of the dims
    int there;       // bit i: tokens 16 i .. of the tile are in the cache
  } raw;
  auto pages_of = [&](int t0) {  // lane i: the page of 16 tokens i
    const int t = t0 + 16 * (lane % (TOKENS / 16));
    return t >= 0 && t < end ? table[t >> a.kv.page_shift] : -1;
  };
  auto load = [&](int t0, int pages) {
    raw.there = 0;
    const uint8_t* base[TOKENS / 16];
#pragma unroll
    for (int i = 0; i < TOKENS / 16; ++i) {
      const int page = __builtin_amdgcn_readlane(pages, i);
      const bool ok = page >= 0 && page < a.kv.count;
      raw.there |= ok << i;
      base[i] = cache + (ok ? page : 0) * page_bytes;
    }
    auto pick = [&](int i) {
      const uint8_t* p = base[0];
#pragma unroll
      for (int j = 1; j < TOKENS / 16; ++j) p = i == j ? base[j] : p;
      return p;
    };
    if (KT == 256 || k_part < 4) {
      const uint8_t* p = pick(k_token / 16);
      const int in_page = (t0 + k_token) & (at.page_tokens - 1);
      __builtin_memcpy(raw.k, __builtin_assume_aligned(p + in_page * (DIM / 2) + k_part * (DIM / 8), 8), DIM / 8);
#pragma unroll
      for (int k = 0; k < DIM / GROUP; ++k)
        raw.km[k] = *reinterpret_cast<const uint32_t*>(p + at.k_meta() + (k * at.page_tokens + in_page) * 4);
    }
    const uint8_t* p = pick(v_16);
    const int in_page = (t0 + 16 * v_16) & (at.page_tokens - 1);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int g = v_h + 2 * q;
      const uint8_t* c = p + at.v_codes() + in_page * (DIM / 2) + ((g * 16 + v_l) * SL + v_m) * 4;
      __builtin_memcpy(raw.v[q], __builtin_assume_aligned(c, 4 * VM), 4 * VM);
#pragma unroll
      for (int half = 0; half < 2; ++half)
        raw.vm[q][half] = *reinterpret_cast<const u32x4*>(
            p + at.v_meta() + (((half * (DIM / 2) + 16 * v_m) / GROUP) * at.page_tokens + in_page + 4 * g) * 4);
    }
  };
  auto store = [&](T& to) {
    if (KT == 256 || k_part < 4) {
      const bool ok = raw.there >> (k_token / 16) & 1;
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        const f16x2 both = __builtin_bit_cast(f16x2, ok ? raw.km[sl * 32 / GROUP] : 0u), sc = both.xx, of = both.yy;
        const uint32_t w = raw.k[sl];
        to.keys[k_token / 32][2 * sl + k_part / 2][k_part % 2][k_token % 32] =
            u32x4{unpack.two<0>(w, sc, of), unpack.two<4>(w, sc, of), unpack.two<0>(w >> 8, sc, of), unpack.two<4>(w >> 8, sc, of)};
      }
    }
    bool nan = false;
    f16x2 sc[2][2][2], of[2][2][2];  // [quad][half][0: tokens 0 and 2, 1: tokens 1 and 3]
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const bool ok = raw.there >> v_16 & 1;
          f16x2 x = __builtin_bit_cast(f16x2, ok ? raw.vm[q][half][2 * o] : 0u);
          f16x2 y = __builtin_bit_cast(f16x2, ok ? raw.vm[q][half][2 * o + 1] : 0u);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (x[e] != x[e]) {  // its rows get their NaN by themselves (0 times NaN would reach the others)
              nan = true;
              x[e] = y[e] = (_Float16)0.0f;
            }
          sc[q][half][o] = x;
          of[q][half][o] = y;
        }
#pragma unroll
    for (int i = 0; i < VM; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        u32x4 out;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const uint32_t w = o ? raw.v[q][i] >> 8 : raw.v[q][i];
            out[2 * q + o] = half ? unpack.two<4>(w, sc[q][half][o], of[q][half][o]) : unpack.two<0>(w, sc[q][half][o], of[q][half][o]);
          }
        const int d = half * (DIM / 2) + 16 * (v_m + i) + v_l;
        to.values[v_16][d / 32][v_h][d % 32] = out;
      }
    const bool any = __builtin_amdgcn_ballot_w64(nan) != 0;
    if (lane == 0) to.bad[wave] = any;
  };

  // ---- the wave's rows
  u32x4 q[RT][KS];
  float unit[RT];
  Span mine[RT];
  int every_lo = 0, every_hi = 2147483647;  // seen by every row of the wave
  int64_t out_row[RT];
  int out_head[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const uint32_t m = tile * ROWS + (wave * RT + r) * 32 + col;
    const bool live = m < (uint32_t)(s.fresh * a.share);
    const int j = m / (uint32_t)a.share, hd = head * a.share + m % (uint32_t)a.share;
    mine[r] = live ? seen(a, s, j, j) : Span{0, 2147483647};
    out_row[r] = live ? s.row + j : -1;
    out_head[r] = hd;
    const uint16_t* qp = a.q + (int64_t)(s.row + (live ? j : 0)) * a.ldq + (int64_t)(live ? hd : 0) * DIM;
    Raw8<uint16_t> x[SL][2];
    float big = 0.0f;
#pragma unroll
    for (int sl = 0; sl < SL; ++sl)
#pragma unroll
      for (int o = 0; o < 2; ++o) {  // step 2 sl + o of 16 dims: parts 2 o + h of the slice
        x[sl][o].load(qp + 32 * sl + 8 * (2 * o + h));
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[sl][o].get(e)));
      }
    big = max_of_two(big);
    const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -120), 120);
    const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), a.scale);
    unit[r] = fabsf(a.scale) * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int sl = 0; sl < SL; ++sl)
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[r][2 * sl + o][i] = live ? pack_f16(x[sl][o].get(i) * down, x[sl][o].get(4 + i) * down) : 0u;
  }
  {
    const uint32_t m0 = tile * ROWS + wave * RT * 32, most = s.fresh * a.share;
    if (m0 < most) {
      const int j0 = m0 / (uint32_t)a.share, j1 = min(m0 + RT * 32, most) - 1;
      every_hi = seen(a, s, j0, j0).hi;
      every_lo = seen(a, s, j1 / (uint32_t)a.share, j1 / (uint32_t)a.share).lo;
    }
  }
  f32x16 acc[RT][XT];
  float top[RT], den[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    top[r] = kLowest;
    den[r] = 0.0f;
#pragma unroll
    for (int x = 0; x < XT; ++x) acc[r][x] = f32x16{};
  }

  f32x16 score[RT];
  auto scores = [&](const T& from, int b, f32x16 (&sc)[RT]) {
#pragma unroll
    for (int r = 0; r < RT; ++r) sc[r] = f32x16{};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const u32x4 k = from.keys[b][ks][h][col];
#pragma unroll
      for (int r = 0; r < RT; ++r) sc[r] = mfma32x32x16_f16(k, q[r][ks], sc[r]);
    }
  };

  int pages = pages_of(begin);
  load(begin, pages);
  pages = pages_of(begin + TOKENS);
  int there = raw.there;
  store(buf[0]);
  load(begin + TOKENS, pages);
  pages = pages_of(begin + 2 * TOKENS);
  __syncthreads();
  scores(buf[0], 0, score);
  int which = 0;
  for (int t0 = begin; t0 < end; t0 += TOKENS) {
    const int next = which == 2 ? 0 : which + 1;
    const T& now = buf[which];
    int there_next = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int tb = t0 + 32 * b;
      const bool whole = (there >> (2 * b) & 3) == 3 && tb + 32 <= every_hi && tb >= every_lo;
      float less[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (!whole) {
          asm volatile("");
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int t = tb + at_reg(v, h);
            if (!((there >> (2 * b + v / 8) & 1) && t >= mine[r].lo && t < mine[r].hi)) score[r][v] = -INFINITY;
          }
        }
        float high = score[r][0];
#pragma unroll
        for (int v = 1; v < 16; ++v) high = fmaxf(high, score[r][v]);
        high = max_of_two(high);
        high = high == -INFINITY ? kLowest : high * unit[r];
        if (__builtin_amdgcn_ballot_w64(high > top[r]) != 0) {
          const float t = fmaxf(high, top[r]);
          const float keep = exp2_fast(top[r] - t);
          top[r] = t;
          den[r] *= keep;
#pragma unroll
          for (int x = 0; x < XT; ++x) acc[r][x] *= keep;
        }
        less[r] = top[r] - kLift;
      }
      if (b == 0) {
        there_next = raw.there;
        store(buf[next]);
        load(t0 + 2 * TOKENS, pages);
        pages = pages_of(t0 + 3 * TOKENS);
      }
      if (b == NB - 1) __syncthreads();
      f32x16 ahead[RT];
      scores(b == NB - 1 ? buf[next] : now, b == NB - 1 ? 0 : b + 1, ahead);
      u32x4 w[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          score[r][v] = exp2_fast(fmaf(score[r][v], unit[r], -less[r]));
        }
        if (!whole) {
          asm volatile("");
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int t = tb + at_reg(v, h);
            if (!((there >> (2 * b + v / 8) & 1) && t >= mine[r].lo && t < mine[r].hi)) score[r][v] = 0.0f;
          }
        }
#pragma unroll
        for (int v = 0; v < 16; ++v) den[r] += score[r][v];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[r][j] = u32x4{pack_f16(score[r][8 * j], score[r][8 * j + 2]), pack_f16(score[r][8 * j + 1], score[r][8 * j + 3]),
                          pack_f16(score[r][8 * j + 4], score[r][8 * j + 6]), pack_f16(score[r][8 * j + 5], score[r][8 * j + 7])};
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < XT; ++x) {
          const u32x4 v = now.values[2 * b + j][x][h][col];
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][x] = mfma32x32x16_f16(v, w[r][j], acc[r][x]);
        }
#pragma unroll
      for (int r = 0; r < RT; ++r) score[r] = ahead[r];
    }
    if (now.bad[0] | now.bad[1] | now.bad[2] | now.bad[3]) {  // NaNs go to the rows that see them, group by group
      for (int t = t0; t < min(t0 + TOKENS, end); ++t) {
        const int page = table[t >> a.kv.page_shift];
        if (page < 0 || page >= a.kv.count) continue;
        const uint8_t* p = cache + page * page_bytes;
#pragma unroll
        for (int k = 0; k < DIM / GROUP; ++k) {
          const uint16_t scale = reinterpret_cast<const uint16_t*>(p + at.v_meta())[at.v_scale(k * at.page_tokens, t & (at.page_tokens - 1))];
          if ((scale & 0x7fffu) <= 0x7c00u) continue;
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (t >= mine[r].lo && t < mine[r].hi)
#pragma unroll
              for (int x = 0; x < XT; ++x)
                if (x * 32 / GROUP == k)
#pragma unroll
                  for (int v = 0; v < 16; ++v) acc[r][x][v] = NAN;
        }
      }
    }
    there = there_next;
    which = next;
  }

#pragma unroll
  for (int r = 0; r < RT; ++r) {
    den[r] += __shfl_xor(den[r], 32);
    if (out_row[r] < 0) continue;
    const float inv = den[r] == 0.0f ? 0.0f : 1.0f / den[r];
    const int64_t slot = (out_row[r] * a.heads + out_head[r]) * a.splits + split;
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 32 * x + 8 * i + 4 * h;
        f32x4 v{acc[r][x][4 * i], acc[r][x][4 * i + 1], acc[r][x][4 * i + 2], acc[r][x][4 * i + 3]};
        if (a.splits == 1) {
          u32x2_any o;
          o[0] = pack_bf16(v[0] * inv, v[1] * inv);
          o[1] = pack_bf16(v[2] * inv, v[3] * inv);
          *reinterpret_cast<u32x2_any*>(a.out + out_row[r] * a.ldo + (int64_t)out_head[r] * DIM + d) = o;
        } else {
          *reinterpret_cast<f32x4*>(a.part + slot * DIM + d) = v;
        }
      }
    if (a.splits > 1 && h == 0) a.stats[slot] = f32x2{top[r], den[r]};
  }
}

// The chunks' parts of a row and head, in the chunks' order: a wave each.
template <int DIM>
__global__ __launch_bounds__(256) void attend_chunks_kernel(AttentionArgs a, int tile_rows) {
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
  const RowTile rt = row_tile(a, s, (j * a.share + h % a.share) / tile_rows, tile_rows);
  const Span all = seen(a, s, rt.first, rt.last);
  const int parts = min(a.splits, max(1, (all.hi - (all.lo & ~15) + a.chunk - 1) / a.chunk));
  const int64_t slot = ((int64_t)(s.row + j) * a.heads + h) * a.splits;
  float top = kLowest, total = 0.0f, sum[PER];
  for (int c = lane; c < parts; c += kWave) top = fmaxf(top, a.stats[slot + c].x);
  for (int x = 1; x < kWave; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
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

constexpr int kWanted = 512;  // workgroups, two for every compute unit, below which the positions are split as well
constexpr int most_rows_of(int dim) { return dim == 256 ? 128 : 256; }

}  // namespace

}  // namespace wr

using namespace wr;

// rows * heads * splits stays below kWanted workgroups' rows.
size_t wr_kv_many_ws_bytes(int64_t rows, int64_t n, int32_t dim) {
  return (size_t)std::min<int64_t>(rows * (n / dim), most_rows_of(dim)) * kWanted * (dim + 2) * sizeof(float);
}

int wr_kv_many_impl(wr_ctx* ctx, const wr_kv_cache& c, const wr_kv_seqs& s, AttentionArgs a, int flags) {
  const int64_t most = (int64_t)s.most_new * a.share;
  const int rows = most <= 128 ? 128 : most_rows_of(c.dim);
  const int64_t tiles = (most + rows - 1) / rows;
  // positions that a tile's rows can see, from a multiple of 16
  int64_t span = a.kv.most_tokens;
  const int64_t queries = std::min<int64_t>(s.most_new, (rows + a.share - 2) / a.share + 1);
  if (a.window > 0) span = std::min(span, (int64_t)a.window * (flags & WR_ATTENTION_CAUSAL ? 1 : 2) + queries + 15);
  const int64_t groups = std::max<int64_t>(1, s.n * tiles * c.heads);
  const int64_t splits = std::max<int64_t>(1, std::min((span + 511) / 512, kWanted / groups));
  a.chunk = (int)std::min<int64_t>(((span + splits - 1) / splits + 127) / 128 * 128, 1 << 30);
  a.splits = (int)std::max<int64_t>(1, (span + a.chunk - 1) / a.chunk);
  const int64_t blocks = groups * a.splits, joins = ((int64_t)s.n * s.most_new * a.heads + 3) / 4;
  if (blocks > 1 << 30 || (a.splits > 1 && joins > 1 << 28)) return WR_EUNSUPPORTED;
  if (a.splits > 1 && ctx->ws_bytes < (size_t)a.kv.rows * a.heads * a.splits * (c.dim + 2) * sizeof(float)) return WR_EWORKSPACE;
  a.stats = reinterpret_cast<f32x2*>(a.part + (size_t)a.kv.rows * a.heads * a.splits * c.dim);
  bool limits = true;
  const bool there = kv_form(c.dim, c.group, [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, G = decltype(g)::value;
    constexpr int bytes = 3 * sizeof(Tile<D, G>);
    auto go = [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      limits = lds_limit(reinterpret_cast<const void*>(&attend_many_kernel<D, G, RT>), bytes);
      if (limits) hipLaunchKernelGGL((attend_many_kernel<D, G, RT>), dim3((uint32_t)blocks), dim3(256), bytes, ctx->stream, a, (uint32_t)tiles);
    };
    if (rows == 128) go(std::integral_constant<int, 1>{});
    else if constexpr (D < 256) go(std::integral_constant<int, 2>{});
    if (limits && a.splits > 1)
      hipLaunchKernelGGL(attend_chunks_kernel<D>, dim3((uint32_t)joins), dim3(256), 0, ctx->stream, a, rows);
  });
  if (!there) return WR_EUNSUPPORTED;
  if (!limits) return WR_EHIP;
  WR_CHECK_LAUNCH();
  return WR_OK;
}
