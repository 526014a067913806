// Tokens times weights in 8-bit integers: y[t][r] = xs[t] ws[r] sum_j x[t][j] w[r][j] + bias[r], and
// silu(gate) * up of two halves of the weights' rows.
//
// Both operands have the summed index contiguous, which is what a matrix-core operand wants: lane l of a 16x16x64
// int8 MFMA holds 16 consecutive bytes of row l % 16, of a 32x32x32 one of row l % 32.  The sums are exact in
// int32, so neither their order nor any split of them changes the result.  Two kernels: small products cut the
// sum over a workgroup's waves (matmul_i8_stream_kernel), large ones share operand tiles among them
// (matmul_i8_big_kernel).
#include "rowops.hpp"

namespace wr {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

struct I8Args {
  const int8_t* x;
  int64_t ldx;
  const float* xs;
  int batch;
  const int8_t* w;
  int64_t ldw;
  const float* ws;
  int rows, n;
  const float* bias;
  void* y;
  int64_t ldy;
};

// Sixteen bytes at column c of a row of n >= 16 bytes, zeros past its end: one load inside the row, shifted down.
__device__ __forceinline__ u32x4 load16(const int8_t* row, int c, int n) {
  const int at = std::min(c, n - 16), d = c - at;
  const u32x4 v = *reinterpret_cast<const u32x4_any*>(row + at);
  const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  const int sh = 8 * (d & 7);
  const uint64_t low = sh ? lo >> sh | hi << (64 - sh) : lo, high = hi >> sh;
  const uint64_t a = d < 8 ? low : d < 16 ? high : 0, b = d < 8 ? high : 0;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
}

__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

__device__ __forceinline__ void put4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<u32x2_any*>(p) = u32x2_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ __forceinline__ void put4(float* p, const float (&v)[4]) {
  *reinterpret_cast<u32x4_any*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}

// v / (1 + exp(-v)) by the hardware's base-2 exponential and reciprocal (one unit in the last place each); rounding -v
// log2(e) is worth |v| 2^-24 in exp(-v), which changes the result by less than a rounding of v itself does.
__device__ __forceinline__ float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

// Scales and stores four consecutive outputs o .. o + 3 of token t from their sums (with GLU also the up rows').
template <typename TY, bool GLU>
__device__ __forceinline__ void store_outputs(const I8Args& a, int outs, int t, int o, const i32x4& sum, const i32x4& up,
                                              float xs, const f32x4& ws, const f32x4& wu, const f32x4& bs, const f32x4& bu) {
  float z[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    z[e] = fmaf((float)sum[e] * xs, ws[e], bs[e]);
    if constexpr (GLU) z[e] = silu(z[e]) * fmaf((float)up[e] * xs, wu[e], bu[e]);
  }
  if (t >= a.batch || o >= outs) return;
  TY* p = (TY*)a.y + t * a.ldy + o;
  if (o + 4 <= outs) {
    put4(p, z);
  } else {
    for (int e = 0; e < outs - o; ++e) put(p + e, z[e]);
  }
}
// Four values at o .. o + 3 of a vector of `outs` (the last one again past its end; zeros without a vector).
__device__ __forceinline__ f32x4 load_outputs(const float* v, int outs, int o) {
  if (!v) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (o + 4 <= outs) return __builtin_bit_cast(f32x4, (u32x4)*reinterpret_cast<const u32x4_any*>(v + o));
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = v[std::min(o + e, outs - 1)];
  return r;
}

// The end of a workgroup whose NW waves hold int32 sums over shares of the summed index: adds them in LDS, scales and
// stores.  Register v of lane l holds weight row 4 (l / 16) + v and token l % 16 of a 16 x 16 block; a token's
// four quads of outputs lie in an order that spreads the tokens over the banks.
template <typename TY, bool GLU, int RF, int NT, int NW>
__device__ __forceinline__ void add_and_store(const I8Args& a, const i32x4 (&acc)[RF][NT], int32_t (*red)[RF * NT][256],
                                              int o0, int t0) {
  constexpr int OF = GLU ? RF / 2 : RF, OQ = 4 * OF, T = 64 * NW, kIter = (OF * NT * 64 + T - 1) / T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, outs = GLU ? a.rows / 2 : a.rows;
  // a thread's outputs are the same for all its tokens
  const int oq = threadIdx.x % OQ, o = o0 + 4 * oq;
  const f32x4 ws = load_outputs(a.ws, outs, o), bs = load_outputs(a.bias, outs, o);
  f32x4 wu = {}, bu = {};
  if constexpr (GLU) {
    wu = load_outputs(a.ws + outs, outs, o);
    bu = load_outputs(a.bias ? a.bias + outs : nullptr, outs, o);
  }
  float xs[kIter];
#pragma unroll
  for (int k = 0; k < kIter; ++k) xs[k] = a.xs[std::min(t0 + (int)(threadIdx.x + k * T) / OQ, a.batch - 1)];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = lane & 15, quad = (lane >> 4) ^ (tok >> 1 & 3);
      *reinterpret_cast<i32x4*>(&red[wave][f * NT + t][16 * tok + 4 * quad]) = acc[f][t];
    }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kIter; ++k) {
    const int i = threadIdx.x + k * T, ti = i / OQ;
    if (OF * NT * 64 % T != 0 && i >= OF * NT * 64) break;
    const int blk = (oq >> 2) * NT + (ti >> 4), tok = ti & 15, e = 16 * tok + 4 * ((oq & 3) ^ (tok >> 1 & 3));
    i32x4 sum = {}, up = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      sum += *reinterpret_cast<const i32x4*>(&red[w][blk][e]);
      if constexpr (GLU) up += *reinterpret_cast<const i32x4*>(&red[w][OF * NT + blk][e]);
    }
    store_outputs<TY, GLU>(a, outs, t0 + ti, o, sum, up, xs[k], ws, wu, bs, bu);
  }
}

// Rows of fewer than 16 bytes, or 8 MiB apart or more: a thread for each output.
template <typename TY, bool GLU>
__global__ __launch_bounds__(256) void matmul_i8_short_kernel(const I8Args a) {
  const int outs = GLU ? a.rows / 2 : a.rows;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < (int64_t)a.batch * outs; i += gridDim.x * (int64_t)256) {
    const int t = (int)(i / outs), o = (int)(i % outs);
    auto z = [&](int r) {
      int sum = 0;
      for (int j = 0; j < a.n; ++j) sum += (int)a.x[t * a.ldx + j] * (int)a.w[r * a.ldw + j];
      return fmaf((float)sum * a.xs[t], a.ws[r], a.bias ? a.bias[r] : 0.0f);
    };
    put((TY*)a.y + t * a.ldy + o, GLU ? silu(z(o)) * z(outs + o) : z(o));
  }
}

// ---- LDS DMA.  Sixteen-byte chunk c of row r of a slice lies at chunk c ^ swizzle(r), so that the sixteen rows an
// operand read touches at once lie on different banks (two rows of 128 bytes fill the banks once).
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ int swizzle(int row) { return row >> 1 & 7; }
// Wave-wide LDS DMA: lane l copies the 16 bytes at base + off to LDS byte m0 + 16 l.  In assembly so that the compiler
// does not wait for it before every LDS read; vm_wait awaits it.  The M0 write needs one wait state before the DMA.
// Global addresses may have any alignment, as for every other load (rows of odd strides come this way too).
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2" ::"v"(off), "s"(m0), "s"(base) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void vm_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Small products.  A workgroup owns RF x 16 weight rows (with GLU half of them gate rows and half the same outputs' up
// rows) by NT x 16 tokens, and its NW waves cut the sum into contiguous ranges of 128-byte slices: few tokens or
// few outputs still occupy the chip, and a byte is read from LDS once.  Each wave streams its range through a ring
// of NS slots of its own, eight rows of 128 bytes (whole cache lines) per copy instruction; the waves share nothing
// before their sums are added at the end, so the loop has no barrier.  The copies go to LDS directly, NS slices ahead
// and without registers.  Rows and tokens past the end repeat the last one and are not stored.
//
// Bound by the weights' bytes and, with so few of them, by latency: one token 9728 -> 2560 (25 MB) 6.2 us, 4.0 TB/s; 48
// tokens 2560 -> 4096 5.2 us; 777 tokens 2531 -> 1023 with odd strides 12.9 us.  Loading the operands straight into
// registers, without LDS, took twice as long: 16 rows a load, each a quarter of a cache line.
template <typename TY, bool GLU, int RF, int NT, int NW, int NS>
__global__ __launch_bounds__(64 * NW) void matmul_i8_stream_kernel(const I8Args a) {
  constexpr int F = RF + NT, OF = GLU ? RF / 2 : RF;  // blocks of 16 rows; of 16 outputs
  constexpr int kSlot = F * 16 * 128;
  extern __shared__ __attribute__((aligned(1024))) char i8_lds[];
  lds_char* const lds = (lds_char*)i8_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int outs = GLU ? a.rows / 2 : a.rows;
  const int o0 = blockIdx.x * 16 * OF, t0 = blockIdx.y * 16 * NT;
  lds_char* const ring = lds + wave * NS * kSlot;
  const uint32_t ring_at = (uint32_t)(uintptr_t)ring;

  // Copies: instruction i (of 2 F) fills rows 8 i .. + 7 of a slot, lane l the place l % 8 of its row l / 8: the chunk at
  // column `col` of a slice.  The row starts `off` bytes after `base`, which is the same for all lanes.
  const int8_t* base[2 * F];
  uint32_t off[2 * F];
  int col[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) col[h] = 16 * ((lane & 7) ^ swizzle(8 * h + (lane >> 3)));
#pragma unroll
  for (int i = 0; i < 2 * F; ++i) {
    const int f = i >> 1, r = 8 * (i & 1) + (lane >> 3);
    base[i] = f < RF ? a.w + o0 * a.ldw + (int64_t)(f / OF * outs) * a.ldw : a.x + t0 * a.ldx;
    off[i] = f < RF ? (uint32_t)std::min(16 * (f % OF) + r, outs - 1 - o0) * (uint32_t)a.ldw
                    : (uint32_t)std::min(16 * (f - RF) + r, a.batch - 1 - t0) * (uint32_t)a.ldx;
  }
  const int slices = (a.n + 127) / 128, s0 = slices * wave / NW, s1 = slices * (wave + 1) / NW;
  const int whole = std::min(s1, a.n / 128);  // slices from here on pass n
  auto issue = [&](int s, int slot) {
    if (s < whole) {
      const uint32_t at = __builtin_amdgcn_readfirstlane(ring_at + slot * kSlot);
#pragma unroll
      for (int i = 0; i < 2 * F; ++i) lds_dma16(base[i] + 128 * s, off[i] + col[i & 1], at + 1024 * i);
    } else {  // through registers, with zeros past n
#pragma unroll
      for (int i = 0; i < 2 * F; ++i)
        *(__attribute__((address_space(3))) u32x4*)(ring + slot * kSlot + 1024 * i + 16 * lane) = load16(base[i] + off[i], 128 * s + col[i & 1], a.n);
    }
  };
  const int r = lane & 15;
  uint32_t rd[2];  // where this lane reads in a block, for either half of a slice
#pragma unroll
  for (int u = 0; u < 2; ++u) rd[u] = r * 128 + (((4 * u + (lane >> 4)) ^ swizzle(r)) << 4);

  i32x4 acc[RF][NT] = {};
#pragma unroll
  for (int p = 0; p < NS; ++p)
    if (s0 + p < s1) issue(s0 + p, p);
  int slot = 0;
  for (int s = s0; s < s1; ++s) {
    // slice s has landed once only the copies of later slices are outstanding
    if (s + NS <= whole) vm_wait<(NS - 1) * 2 * F>();
    else vm_wait<0>();
    const lds_char* st = ring + slot * kSlot;
    i32x4 fr[2][F];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int f = 0; f < F; ++f) fr[u][f] = *(const __attribute__((address_space(3))) i32x4*)(st + f * 2048 + rd[u]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the slot may be filled again
    __builtin_amdgcn_sched_barrier(0);
    if (s + NS < s1) issue(s + NS, slot);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int f = 0; f < RF; ++f) acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fr[u][f], fr[u][RF + t], acc[f][t], 0, 0, 0);
    slot = slot == NS - 1 ? 0 : slot + 1;
  }
  __syncthreads();  // the sums go where the rings were
  add_and_store<TY, GLU, RF, NT, NW>(a, acc, reinterpret_cast<int32_t(*)[RF * NT][256]>(i8_lds), o0, t0);
}

// Large products: WI x WJ waves share a tile of 32 FI WI tokens x 32 FJ WJ weight rows, each with 32 FI x 32 FJ of it
// in registers (32x32x32 MFMAs).  Slices of 128 bytes of the tile's rows are copied into a ring of NS slots by LDS
// DMA, NS slices ahead; the operands of the next 32 bytes are read while the present ones are multiplied.  Chunk c
// of row r lies at chunk c ^ swizzle(r), without which half of the LDS cycles were bank conflicts.  KG such groups of
// waves, each with a ring of its own, take every KG-th slice of the same tile; their sums meet in LDS at the end.
//
// 16384 tokens 4096 -> 2560 take 149 us (2309 TOPS), 8192 tokens 2560 -> 2 x 9728 with SwiGLU 374 us (2184 TOPS), timed in
// turn with a library's product of the same sizes without scales (168 and 414 us).  By the counters no unit is full: the matrix cores
// are busy for 53 % of the cycles (at 1.9 GHz), LDS reads for 25 %, HBM gives 1.4 to 1.8 TB/s; the waves, two a SIMD, wait for 35 %
// of theirs.  Short sums are bound by the outputs: 8192 tokens 256 -> 4096 25 us, 2.7 TB/s.  Slower: copies issued
// between the MFMAs, five slots of 64 bytes, eight waves for 128 x 128, raised wave priority.
template <typename TY, bool GLU, int FI, int FJ, int WI, int WJ, int NS, bool LATE, int KG>
__global__ __launch_bounds__(64 * WI * WJ * KG, 1) void matmul_i8_big_kernel(const I8Args a, int tiles_t, int tiles_o) {
  constexpr int NW = WI * WJ, TM = 32 * FI * WI, TN = 32 * FJ * WJ;
  constexpr int BK = 128, CPR = BK / 16, RPI = 64 / CPR;  // bytes of a slice, chunks per row, rows per copy instruction
  constexpr int kSlot = (TM + TN) * BK;
  constexpr int kCopies = (TM + TN) / RPI / NW;      // copy instructions per wave and slice
  constexpr int KS = BK / 32;                        // MFMA steps per slice
  constexpr int kOuts = GLU ? TN / 2 : TN;
  static_assert((TM + TN) % (RPI * NW) == 0 && KS % 2 == 0 && NW * RPI % 16 == 0 && (!GLU || FJ % 2 == 0), "tile shape");
  extern __shared__ __attribute__((aligned(1024))) char i8_lds[];
  const int lane = threadIdx.x & 63, wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = KG > 1 ? wave_of_all / NW : 0, wave = KG > 1 ? wave_of_all % NW : wave_of_all;
  lds_char* const lds = (lds_char*)i8_lds + group * NS * kSlot;
  const uint32_t lds_at = (uint32_t)(uintptr_t)lds;
  const int wi = wave / WJ, wj = wave % WJ;
  const int outs = GLU ? a.rows / 2 : a.rows;

  // Workgroup b runs on XCD b % 8: each XCD takes a contiguous range of the tiles, in bands of eight token tiles
  // by all output tiles, so that the workgroups it runs at once share operand rows in its L2.
  int ti, oi;
  {
    const int tiles = tiles_t * tiles_o, q = tiles / 8, rem = tiles % 8, x = blockIdx.x % 8, at = blockIdx.x / 8;
    if (at >= q + (x < rem ? 1 : 0)) return;  // the grid is rounded up to a multiple of 8
    const int t = x * q + std::min(x, rem) + at, band = t / (8 * tiles_o), r = t - band * 8 * tiles_o;
    const int height = std::min(8, tiles_t - 8 * band);
    ti = 8 * band + r % height;
    oi = r / height;
  }
  const int t0 = ti * TM, o0 = oi * kOuts;

  // Copies: instruction k = i NW + wave of a slice fills rows k RPI .. of the slot (TN weight rows, then TM tokens),
  // lane l the place l % CPR of its row l / CPR.  With GLU the weight rows are 32 gate rows, the same outputs' 32 up
  // rows, and so on.
  const int crow = lane / CPR;
  const int8_t* base[kCopies];  // the same for all lanes
  uint32_t off[kCopies];
  // the same for every i: NW RPI rows are a multiple of the rows after which the swizzle repeats
  const int col = 16 * ((lane % CPR) ^ swizzle(wave * RPI + crow));
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r0 = (i * NW + wave) * RPI, r = r0 + crow;
    const int64_t up = GLU ? (int64_t)((r0 >> 5 & 1) * outs) * a.ldw : 0;
    base[i] = r0 >= TN ? a.x + t0 * a.ldx : a.w + o0 * a.ldw + up;
    off[i] = r >= TN ? (uint32_t)std::min(r - TN, a.batch - 1 - t0) * (uint32_t)a.ldx
                     : (uint32_t)std::min(GLU ? (r >> 6) * 32 + (r & 31) : r, outs - 1 - o0) * (uint32_t)a.ldw;
  }
  // This group's slices are KG s + group; those from `whole` on pass n, or lie beyond it (zeros).
  const int slices = (a.n + BK * KG - 1) / (BK * KG), whole = (a.n / BK + KG - 1 - group) / KG;
  auto issue = [&](int s, int slot) {
    if (s < whole) {
      const uint32_t at = __builtin_amdgcn_readfirstlane(lds_at + slot * kSlot + wave * 1024);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) lds_dma16(base[i] + BK * (KG * s + group), off[i] + col, at + i * NW * 1024);
    } else {  // through registers, with zeros past n
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        // The accumulators leave few registers: no full addresses kept for this one slice, three loads in flight.
        uint32_t from = off[i];
        asm volatile("" : "+v"(from));
        *(__attribute__((address_space(3))) u32x4*)(lds + slot * kSlot + (i * NW + wave) * 1024 + 16 * lane) = load16(base[i] + from, BK * (KG * s + group) + col, a.n);
        if (i % 3 == 2) asm volatile("" ::: "memory");
      }
    }
  };

  uint32_t rd[KS];  // this lane's place in a block of 32 rows for each MFMA step of a slice
#pragma unroll
  for (int u = 0; u < KS; ++u) rd[u] = (lane & 31) * BK + (((2 * u + (lane >> 5)) ^ swizzle(lane & 31)) << 4);
  i32x4 fw[2][FJ], fx[2][FI];
  auto read = [&](int slot, int u, int set) {
    const lds_char* st = lds + slot * kSlot + rd[u];
#pragma unroll
    for (int j = 0; j < FJ; ++j) fw[set][j] = *(const __attribute__((address_space(3))) i32x4*)(st + (wj * FJ + j) * 32 * BK);
#pragma unroll
    for (int i = 0; i < FI; ++i) fx[set][i] = *(const __attribute__((address_space(3))) i32x4*)(st + (TN + (wi * FI + i) * 32) * BK);
  };
  i32x16 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[i][j] = i32x16{};
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][j], fx[set][i], acc[i][j], 0, 0, 0);
  };

  // The tile's scales and biases, in registers until LDS has room for them.
  static_assert(TN <= 64 * NW && TM <= 64 * NW, "a thread loads one scale");
  const int r = threadIdx.x, own_t = std::min(t0 + r, a.batch - 1);
  const int own_r = std::min(o0 + (GLU ? (r >> 6) * 32 + (r & 31) : r), outs - 1) + (GLU ? (r >> 5 & 1) * outs : 0);
  const float own_xs = a.xs[own_t], own_ws = a.ws[own_r], own_bias = a.bias ? a.bias[own_r] : 0.0f;
#pragma unroll
  for (int p = 0; p < NS; ++p)
    if (p < slices) issue(p, p);
  if (whole >= NS) vm_wait<kCopies*(NS - 1)>();
  else vm_wait<0>();
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  read(0, 0, 0);
  int slot = 0;
  for (int s = 0; s < slices; ++s) {
    const int next = slot == NS - 1 ? 0 : slot + 1;
#pragma unroll
    for (int u = 0; u < KS; ++u) {
      if (u + 1 < KS) {
        read(slot, u + 1, (u + 1) & 1);
        multiply(u & 1);
      } else {
        if (s + 1 < slices) {
          // slice s + 1 has landed once only the copies of slices s + 2 .. s + NS - 1 are outstanding
          if (s + NS <= whole) vm_wait<kCopies*(NS - 2)>();
          else vm_wait<0>();
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          // every wave has read all of slice s: its slot is free.  With one workgroup on a CU the copies wait
          // until the matrix cores have work; with two, the other one's products cover them.
          if (!LATE && s + NS < slices) issue(s + NS, slot);
          read(next, 0, 0);
        }
        multiply(u & 1);
        if (LATE && s + NS < slices) issue(s + NS, slot);
      }
    }
    slot = next;
  }

  // Register v of lane l holds weight row acc_row(v, l) and token l % 32 of a 32 x 32 block: four consecutive outputs of 32
  // tokens at a time.  Stored like that a wave would write pieces of 16 bytes; each wave instead turns 32 tokens'
  // outputs in LDS (rows padded by 16 bytes, which spreads them over the banks) and stores whole rows.
  constexpr int WO = GLU ? 16 * FJ : 32 * FJ;               // outputs of a wave
  constexpr int RB = WO * (int)sizeof(TY), LS = RB + 16;    // bytes of a token's outputs, and in LDS
  constexpr int LPR = RB / 16, kPer = 16 / (int)sizeof(TY);  // lanes that store a row, outputs of one of them
  constexpr int kShared = NW * 32 * LS + 4 * (TM + 2 * TN), kAcc = KG > 1 ? NW * FI * FJ * 4096 : 0;
  static_assert(kShared % 16 == 0 && kShared + kAcc <= KG * NS * kSlot, "outputs, scales and sums take the rings' place");
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // no wave reads the ring any more
  lds_char* const turn = (lds_char*)i8_lds + wave * 32 * LS;
  typedef __attribute__((address_space(3))) float lds_float;
  lds_float* const ws_lds = (lds_float*)((lds_char*)i8_lds + NW * 32 * LS);
  lds_float* const bias_lds = ws_lds + TN;
  lds_float* const xs_lds = bias_lds + TN;
  if (r < TN) {
    ws_lds[r] = own_ws;
    bias_lds[r] = own_bias;
  }
  if (r < TM) xs_lds[r] = own_xs;
  // The second group hands its sums to the first, which stores.
  auto sum_at = [&](int f, int q) {
    return (__attribute__((address_space(3))) i32x4*)((lds_char*)i8_lds + kShared + ((wave * FI * FJ + f) * 4 + q) * 1024 + 16 * lane);
  };
  if (KG > 1 && group)
#pragma unroll
    for (int f = 0; f < FI * FJ; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x16& v = acc[f / FJ][f % FJ];
        *sum_at(f, q) = i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (KG > 1) {
    if (group) return;
#pragma unroll
    for (int f = 0; f < FI * FJ; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x4 v = *sum_at(f, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[f / FJ][f % FJ][4 * q + e] += v[e];
      }
  }
  const int ow = o0 + wj * WO;
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    const int tw = t0 + (wi * FI + i) * 32;
    const float xs = xs_lds[(wi * FI + i) * 32 + (lane & 31)];
#pragma unroll
    for (int j = 0; j < FJ; j += GLU ? 2 : 1)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        auto scale4 = [&](const lds_float* v, int j) {
          return *(const __attribute__((address_space(3))) f32x4*)(v + (wj * FJ + j) * 32 + 8 * q + 4 * (lane >> 5));
        };
        const f32x4 ws = scale4(ws_lds, j), bs = scale4(bias_lds, j);
        f32x4 wu = {}, bu = {};
        if constexpr (GLU) {
          wu = scale4(ws_lds, j + 1);
          bu = scale4(bias_lds, j + 1);
        }
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[e] = fmaf((float)acc[i][j][4 * q + e] * xs, ws[e], bs[e]);
          if constexpr (GLU) z[e] = silu(z[e]) * fmaf((float)acc[i][j + 1][4 * q + e] * xs, wu[e], bu[e]);
        }
        lds_char* const to = turn + (lane & 31) * LS + ((GLU ? j / 2 : j) * 32 + 8 * q + 4 * (lane >> 5)) * (int)sizeof(TY);
        if constexpr (sizeof(TY) == 2)
          *(__attribute__((address_space(3))) u32x2*)to = u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
        else
          *(__attribute__((address_space(3))) f32x4*)to = f32x4{z[0], z[1], z[2], z[3]};
      }
#pragma unroll
    for (int k = 0; k < LPR / 2; ++k) {
      const int row = (k * 64 + lane) / LPR, at = (k * 64 + lane) % LPR, t = tw + row, o = ow + at * kPer;
      const u32x4 v = *(const __attribute__((address_space(3))) u32x4*)(turn + row * LS + 16 * at);
      if (t >= a.batch || o >= outs) continue;
      TY* p = (TY*)a.y + t * a.ldy + o;
      if (o + kPer <= outs) {
        *reinterpret_cast<u32x4_any*>(p) = v;
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (o + e < outs) {
            if constexpr (sizeof(TY) == 2) p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            else p[e] = __uint_as_float(v[e]);
          }
      }
    }
  }
}

}  // namespace wr

using namespace wr;

template <typename TY, bool GLU, int RF, int NT, int NW, int NS>
static int stream_launch(wr_ctx* ctx, const I8Args& a) {
  constexpr int OF = GLU ? RF / 2 : RF;
  constexpr int lds = NW * std::max(NS * (RF + NT) * 2048, RF * NT * 1024);
  static_assert(lds <= 160 * 1024, "LDS");
  const int outs = GLU ? a.rows / 2 : a.rows;
  const dim3 grid((outs + 16 * OF - 1) / (16 * OF), (a.batch + 16 * NT - 1) / (16 * NT));
  auto* kernel = matmul_i8_stream_kernel<TY, GLU, RF, NT, NW, NS>;
  if (!lds_limit((const void*)kernel, lds)) return WR_EHIP;
  hipLaunchKernelGGL(kernel, grid, dim3(64 * NW), lds, ctx->stream, a);
  return WR_OK;
}

template <typename TY, bool GLU, int FI, int FJ, int WI, int WJ, int NS, bool LATE, int KG = 1>
static int big_launch(wr_ctx* ctx, const I8Args& a) {
  constexpr int TM = 32 * FI * WI, TN = 32 * FJ * WJ, kOuts = GLU ? TN / 2 : TN;
  constexpr int lds = KG * NS * (TM + TN) * 128;
  static_assert(lds <= 160 * 1024, "LDS");
  const int outs = GLU ? a.rows / 2 : a.rows;
  const int tt = (a.batch + TM - 1) / TM, to = (outs + kOuts - 1) / kOuts;
  auto* kernel = matmul_i8_big_kernel<TY, GLU, FI, FJ, WI, WJ, NS, LATE, KG>;
  if (!lds_limit((const void*)kernel, lds)) return WR_EHIP;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((tt * to + 7) / 8 * 8)), dim3(64 * WI * WJ * KG), lds, ctx->stream, a, tt, to);
  return WR_OK;
}

template <typename TY, bool GLU>
static int matmul_launch(wr_ctx* ctx, const I8Args& a) {
  if (a.n < 16 || std::max(a.ldx, a.ldw) >= 1 << 23) {  // a tile's rows, up to 320, are at 32-bit offsets from its first
    const int64_t all = (int64_t)a.batch * (GLU ? a.rows / 2 : a.rows);
    hipLaunchKernelGGL((matmul_i8_short_kernel<TY, GLU>), dim3((unsigned)std::min<int64_t>((all + 255) / 256, 1 << 20)),
                       dim3(256), 0, ctx->stream, a);
    return WR_OK;
  }
  constexpr int R = GLU ? 2 : 1;
  const int64_t cu = ctx->num_cu;
  auto tiles = [&](int64_t rows, int64_t tokens) { return ((a.rows + rows - 1) / rows) * ((a.batch + tokens - 1) / tokens); };
  // The smallest tile whose workgroups run all at once (the time of a small product is its latency), measured at
  // n = 2560 and 9728, 4096 and 2560 outputs: 1 token 3.8 and 6.2 us on 16 x 16 (a floor of 2.0 and 4.8 at a copy's
  // rate; 7.0 and 13.7 on 64 x 64), 64 tokens 5.2 and 9.7 on 32 x 32 (7.3 and 12.4 on 16 x 16, 8.2 and 16.5 on
  // 64 x 64), 256 tokens 8.8 and 16.8 on 64 x 64 (15.0 and 24.9 on 32 x 32).
  if (a.batch <= 16 && tiles(16 * R, 16) <= 2 * cu) return stream_launch<TY, GLU, R, 1, 8, 2>(ctx, a);
  if (tiles(16 * R, 32) <= cu) return stream_launch<TY, GLU, R, 2, 8, 2>(ctx, a);
  if (tiles(32, 32) <= cu) return stream_launch<TY, GLU, 2, 2, 8, 2>(ctx, a);
  if (tiles(64, 32) <= cu) return stream_launch<TY, GLU, 4, 2, 4, 3>(ctx, a);
  if (a.batch <= 16) return stream_launch<TY, GLU, R, 1, 8, 2>(ctx, a);
  if (tiles(32, 64) <= cu) return stream_launch<TY, GLU, 2, 4, 4, 2>(ctx, a);
  if (tiles(64, 64) <= cu) return stream_launch<TY, GLU, 4, 4, 4, 2>(ctx, a);
  // From here on shared tiles: a second round of 64 x 64 takes 51 us for 770 tokens 9664 -> 1672, one of 64 x 128 35.
  // With one workgroup a CU, two groups of waves cut the sum: 512 tokens 9728 -> 2560 26.4 us against 33.7, 512 tokens
  // 4096 -> 2 x 2048 14.5 against 18.3, 64 tokens 2560 -> 2 x 9728 11.8 against 12.8; with two, one covers the other's waits.
  if (tiles(128, 64) <= cu) return big_launch<TY, GLU, 1, 2, 2, 2, 3, false, 2>(ctx, a);
  if (tiles(128, 64) <= 2 * cu) return big_launch<TY, GLU, 1, 2, 2, 2, 3, false>(ctx, a);
  // Shared tiles: the least number of rounds over the CUs times the time of one round, measured in hundredths of that of
  // 256 x 256 (n = 2560: 44 us, 4096: 62): the larger tile wins by the bytes it reads from LDS, the other by
  // a last round that is nearly empty.  8192 tokens 2560 -> 2 x 9728: 497, 461, 436 and 401 us in this order; 16384
  // tokens 4096 -> 2560: 196, 193, 187, 205 and 160; 4096 tokens 9728 -> 2560: 134, 107, 117, 131 and 128.
  struct Tile {
    int64_t tokens, rows, per_cu, time;
  };
  constexpr Tile kTiles[5] = {{128, 128, 2, 62}, {192, 256, 1, 77}, {256, 256, 1, 100}, {320, 256, 1, 116}, {256, 320, 1, 123}};
  constexpr int kWide = !GLU && sizeof(TY) == 2 ? 5 : 4;  // the last one's gate and up blocks would not pair, nor its fp32 outputs fit LDS
  int best = 0;
  int64_t least = INT64_MAX;
  for (int i = 0; i < kWide; ++i) {
    const int64_t at_once = kTiles[i].per_cu * cu, t = (tiles(kTiles[i].rows, kTiles[i].tokens) + at_once - 1) / at_once * kTiles[i].time;
    if (t < least) best = i, least = t;
  }
  switch (best) {
    case 0: return big_launch<TY, GLU, 2, 2, 2, 2, 2, false>(ctx, a);
    case 1: return big_launch<TY, GLU, 3, 2, 2, 4, 2, true>(ctx, a);
    case 2: return big_launch<TY, GLU, 4, 2, 2, 4, 2, true>(ctx, a);
    case 3: return big_launch<TY, GLU, 5, 2, 2, 4, 2, true>(ctx, a);
  }
  if constexpr (kWide == 5) return big_launch<TY, GLU, 2, 5, 4, 2, 2, true>(ctx, a);
  return WR_EINVAL;
}

int wr_matmul_i8_impl(wr_ctx* ctx, const int8_t* x, int64_t ldx, const float* x_scales, int64_t batch, const int8_t* w,
                      int64_t ldw, const float* w_scales, int64_t rows, int64_t n, const float* bias, bool glu, void* y,
                      int y_dtype, int64_t ldy) {
  if (batch == 1) ldx = 0;  // a single row's stride is not used
  if (rows == 1) ldw = 0;
  if (n == 0) {  // nothing is read
    x = w = nullptr;
    ldx = ldw = 0;
  }
  // tokens per launch: at most 32768 rows of the grid (of 16 tokens or more each), and tiles within 32 bits
  const int64_t slice = std::min<int64_t>((int64_t)1 << 19, std::max<int64_t>(256, ((int64_t)1 << 36) / rows));
  for (int64_t t0 = 0; t0 < batch; t0 += slice) {
    const I8Args a{x + t0 * ldx, ldx, x_scales + t0, (int)std::min(slice, batch - t0), w, ldw, w_scales, (int)rows,
                   (int)n, bias, (char*)y + t0 * ldy * (y_dtype == WR_BF16 ? 2 : 4), ldy};
    int rc;
    if (y_dtype == WR_BF16) rc = glu ? matmul_launch<uint16_t, true>(ctx, a) : matmul_launch<uint16_t, false>(ctx, a);
    else rc = glu ? matmul_launch<float, true>(ctx, a) : matmul_launch<float, false>(ctx, a);
    if (rc != WR_OK) return rc;
    WR_CHECK_LAUNCH();
  }
  return WR_OK;
}
