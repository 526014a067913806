// The norms before and after a block with the gate and the residual scale between them, and the
// quantization of activation rows to 8-bit integers.
//
//   u = w_post b / rms(b),  x' = rscale x + bscale g u,  y = w_pre x' / rms(x'),  q = rint(127 y / max|y|)
//
// Every value of a row stays in registers from its one load to its stores: the two sums of squares and
// the maximum are reductions over the lanes that share the row.  Rows of up to 512 values take 16, 32 or
// 64 lanes of a wave (no barrier); wider rows take a workgroup of up to 1024 threads with one or two
// chunks of eight values per thread.
//
// Bound by memory.  16384 x 2560 bf16 with both norms, gate and residual (335 MB) take 64 us and 131072 x 128 bf16 with
// one norm (67 MB) 13 us, both at the 5.2 TB/s of a large copy; 1013 x 9727 fp32 (158 MB) 41 us, 3.9 TB/s: two rows a
// workgroup, and nothing hides the first one's loads; one token 3.3 us, a launch's latency.
#include "rowops.hpp"

namespace wr {

struct NormArgs {
  int rows, n;
  const void* branch;
  int64_t ldb;
  const void* w_post;
  const void* gate;
  int64_t ldg;
  int gate_rows;
  float bscale;
  const void* resid;
  int64_t ldr;
  float rscale;
  const void* w_pre;
  float eps;
  void* resid_out;
  int64_t ldo;
  void* y;
  int64_t ldy;
  int8_t* q;
  int64_t ldq;
  float* q_scales;
  float* stats;
};

// This thread's place in its row, first row, row step and column step.
template <int LANES>
struct RowWalk {
  int lane, first, step, cstep;
  __device__ __forceinline__ RowWalk() {
    if constexpr (LANES > 0) {
      const int per = blockDim.x / LANES;
      lane = threadIdx.x % LANES;
      first = blockIdx.x * per + threadIdx.x / LANES;
      step = gridDim.x * per;
      cstep = 8 * LANES;
    } else {
      lane = threadIdx.x;
      first = blockIdx.x;
      step = gridDim.x;
      cstep = 8 * blockDim.x;
    }
  }
};

// Inputs that are absent take a value that leaves the formula as it is (weights and gate 1, branch and
// residual 0), so that the row's arithmetic has no branches.
template <typename TB, typename TR, typename TW, int CH, int LANES, int MAXT>
__global__ __launch_bounds__(MAXT) void block_norm_kernel(const NormArgs a) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  RowGroup<LANES> grp{red};
  const RowWalk<LANES> walk;
  const int n = a.n;
  const RowMap<CH, LANES> map(walk.lane, walk.cstep, n);
  const float inv_n = 1.0f / (float)n;

  Raw8<TW> wp[CH], wq[CH];
  Raw8<TB> b[CH], g[CH];
  Raw8<TR> x[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    wp[k].fill(1.0f);
    wq[k].fill(1.0f);
    b[k].fill(0.0f);
    g[k].fill(1.0f);
    x[k].fill(0.0f);
    if (a.w_post) map.load(wp[k], (const TW*)a.w_post, k);
    if (a.w_pre) map.load(wq[k], (const TW*)a.w_pre, k);
  }
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if (a.branch) map.load(b[k], (const TB*)a.branch + row * a.ldb, k);
      if (a.resid) map.load(x[k], (const TR*)a.resid + row * a.ldr, k);
      if (a.gate) map.load(g[k], (const TB*)a.gate + (a.gate_rows ? (uint32_t)row / (uint32_t)a.gate_rows : 0u) * a.ldg, k);
    }
  };
  if (walk.first < a.rows) load_row(walk.first);
  for (int64_t row = walk.first; row < a.rows; row += walk.step) {
    float v[CH][8];
    float r1 = 1.0f, r2 = 1.0f;
    if (a.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = b[k].get(e);
        map.own(t, k);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(t[e], t[e], ss);
      }
      r1 = 1.0f / sqrtf(grp.sum(ss) * inv_n + a.eps);
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = b[k].get(e) * r1 * wp[k].get(e) * g[k].get(e) * a.bscale;
        v[k][e] = t[e] = fmaf(a.rscale, x[k].get(e), u);
      }
      map.own(t, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(t[e], t[e], ss);
    }
    // Where resid_out is resid, x' is stored once all waves have read x.  The reduction for the pre norm waits for that; the
    // one for the post norm waits for b alone, so without a pre norm every wave awaits its loads and meets the others.
    if (LANES == 0 && !a.w_pre && a.resid_out == a.resid) asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    // the next row's loads are in flight during the rest of this one
    if (row + walk.step < a.rows) load_row(row + walk.step);
    if (a.w_pre) r2 = 1.0f / sqrtf(grp.sum(ss) * inv_n + a.eps);
    if (a.resid_out)
#pragma unroll
      for (int k = 0; k < CH; ++k) map.store((TR*)a.resid_out + row * a.ldo, k, v[k]);
    if (a.w_pre) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * r2 * wq[k].get(e);
        if (a.y) map.store((TB*)a.y + row * a.ldy, k, v[k]);
      }
      if (a.q) {
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = MaxU32::op(top, __float_as_uint(v[k][e]) & 0x7fffffffu);
        const RowCoder code(grp.max(top));
#pragma unroll
        for (int k = 0; k < CH; ++k) map.store(a.q + row * a.ldq, k, code.codes(v[k]));
        if (walk.lane == 0) a.q_scales[row] = code.scale;
      }
    }
    if (a.stats && walk.lane == 0) {
      a.stats[2 * row] = r1;
      a.stats[2 * row + 1] = r2;
    }
  }
}

// One pass: the row's maximum, its scale max / 127, and the codes from the values still in registers.  Bound by memory (3
// bytes a bf16 value): 16384 x 4096 take 40 us, 5.0 TB/s.
template <typename T, int CH, int LANES, int MAXT>
__global__ __launch_bounds__(MAXT) void quant_rows_kernel(const T* __restrict__ x, int64_t ldx, int rows, int n,
                                                          int8_t* __restrict__ q, int64_t ldq,
                                                          float* __restrict__ scales) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  RowGroup<LANES> grp{red};
  const RowWalk<LANES> walk;
  const RowMap<CH, LANES> map(walk.lane, walk.cstep, n);
  Raw8<T> r[CH];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < CH; ++k) map.load(r[k], x + row * ldx, k);
  };
  if (walk.first < rows) load_row(walk.first);
  for (int64_t row = walk.first; row < rows; row += walk.step) {
    float v[CH][8];
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] = r[k].get(e);
        top = MaxU32::op(top, __float_as_uint(v[k][e]) & 0x7fffffffu);
      }
    }
    if (row + walk.step < rows) load_row(row + walk.step);
    const RowCoder code(grp.max(top));
#pragma unroll
    for (int k = 0; k < CH; ++k) map.store(q + row * ldq, k, code.codes(v[k]));
    if (walk.lane == 0) scales[row] = code.scale;
  }
}

// Rows wider than the registers of a workgroup: two passes over the row, the second from the caches.  2000 x 20000 bf16
// take 33 us (3.7 TB/s), 4096 x 32768 101 us (4.0 TB/s).
template <typename T>
__global__ __launch_bounds__(512) void quant_rows_wide_kernel(const T* __restrict__ x, int64_t ldx, int rows, int64_t n,
                                                              int8_t* __restrict__ q, int64_t ldq,
                                                              float* __restrict__ scales) {
  __shared__ uint32_t red[2][3][RowGroup<0>::kMaxWaves];
  RowGroup<0> grp{red};
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* from = x + row * ldx;
    uint32_t top = 0u;
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * 512) {
      Raw8<T> r;
      r.load(from + std::min(c, n - 8));  // a value read twice does not change the maximum
#pragma unroll
      for (int e = 0; e < 8; ++e) top = MaxU32::op(top, __float_as_uint(r.get(e)) & 0x7fffffffu);
    }
    const RowCoder code(grp.max(top));
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * 512) {
      const int64_t at = std::min(c, n - 8);  // nor does a code written twice
      Raw8<T> r;
      r.load(from + at);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = r.get(e);
      *reinterpret_cast<u32x2_any*>(q + row * ldq + at) = code.codes(v);
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
  }
}

}  // namespace wr

using namespace wr;

template <int N>
using Int = std::integral_constant<int, N>;

// Calls launch(chunks, lanes, most threads, threads, workgroups) -- the first three integral constants -- for rows
// of n values.  Workgroups walk the rows with the next row's loads in flight, so there are only as many as
// `per_cu` threads a CU make.
template <int LANES, int CH, typename F>
static void wave_rows(int num_cu, int per_cu, int64_t rows, F&& launch) {
  const int64_t per = 256 / LANES;
  launch(Int<CH>{}, Int<LANES>{}, Int<256>{}, 256, (int)std::min<int64_t>((int64_t)num_cu * (per_cu / 256), (rows + per - 1) / per));
}
template <int CH, int MAXT, typename F>
static void group_rows(int num_cu, int per_cu, int64_t rows, int64_t n, F&& launch) {
  const int threads = ((int)((n + 7) / 8 + CH - 1) / CH + 63) / 64 * 64;
  launch(Int<CH>{}, Int<0>{}, Int<MAXT>{}, threads, (int)std::min<int64_t>((int64_t)num_cu * std::max(1, per_cu / threads), rows));
}
// Norm: 16384 x 2560 bf16 with 1280 threads a CU takes 64 us, with 768, 1600 and 2048 it takes 75, 70 and 70 (at
// 5.2 TB/s a copy of as many bytes takes 65).
template <typename F>
static void norm_shape(int num_cu, int64_t rows, int64_t n, F&& launch) {
  if (n < 8) wave_rows<8, 1>(num_cu, 1024, rows, launch);
  else if (n <= 128) wave_rows<16, 1>(num_cu, 1024, rows, launch);
  else if (n <= 256) wave_rows<32, 1>(num_cu, 1024, rows, launch);
  else if (n <= 512) wave_rows<64, 1>(num_cu, 1024, rows, launch);
  else if (n <= 4096) group_rows<1, 512>(num_cu, 1280, rows, n, launch);
  else if (n <= 8192) group_rows<1, 1024>(num_cu, 1280, rows, n, launch);
  else if (n <= 12288) group_rows<2, 768>(num_cu, 1280, rows, n, launch);
  else group_rows<2, 1024>(num_cu, 1280, rows, n, launch);
}
// Quantizer: with one input and one byte out per value, a thread needs more chunks in flight: 16384 x 4096 bf16
// takes 40 us with four chunks and 1024 threads a CU, 72 with one chunk and 2048 (a copy of as many bytes: 39).
// A few rows are a matter of latency, and take the most threads.
template <typename F>
static void quant_shape(int num_cu, int64_t rows, int64_t n, F&& launch) {
  if (n < 8) wave_rows<8, 1>(num_cu, 2048, rows, launch);
  else if (n <= 128) wave_rows<16, 1>(num_cu, 2048, rows, launch);
  else if (n <= 256) wave_rows<32, 1>(num_cu, 2048, rows, launch);
  else if (n <= 512) wave_rows<64, 1>(num_cu, 2048, rows, launch);
  else if (n <= 8192 && rows <= num_cu) group_rows<1, 1024>(num_cu, 1024, rows, n, launch);
  else if (rows <= num_cu) group_rows<2, 1024>(num_cu, 1024, rows, n, launch);
  else if (n <= 1024) wave_rows<64, 2>(num_cu, 1024, rows, launch);
  else if (n <= 2048) wave_rows<64, 4>(num_cu, 1024, rows, launch);
  else group_rows<4, 512>(num_cu, 1024, rows, n, launch);
}

template <typename TB, typename TR, typename TW>
static int norm_launch(wr_ctx* ctx, const NormArgs& a) {
  norm_shape(ctx->num_cu, a.rows, a.n, [&](auto ch, auto lanes, auto most, int threads, int grid) {
    hipLaunchKernelGGL((block_norm_kernel<TB, TR, TW, decltype(ch)::value, decltype(lanes)::value, decltype(most)::value>),
                       dim3(grid), dim3(threads), 0, ctx->stream, a);
  });
  WR_CHECK_LAUNCH();
  return WR_OK;
}

int wr_block_norm_impl(wr_ctx* ctx, int64_t rows, int64_t n, const void* branch, int b_dtype, int64_t ldb,
                       const void* w_post, const void* gate, int64_t ldg, int64_t gate_rows, float branch_scale,
                       const void* resid, int r_dtype, int64_t ldr, float resid_scale, const void* w_pre, int w_dtype,
                       float eps, void* resid_out, int64_t ldo, void* y, int64_t ldy, int8_t* q, int64_t ldq,
                       float* q_scales, float* stats) {
  const NormArgs a{(int)rows, (int)n, branch, ldb,       w_post, gate, ldg, gate_rows >= rows ? 0 : (int)gate_rows,
                   branch_scale, resid, ldr, resid_scale, w_pre, eps, resid_out, ldo,
                   y,     ldy,  q,     ldq,       q_scales, stats};
  const int key = (b_dtype == WR_BF16 ? 4 : 0) + (r_dtype == WR_BF16 ? 2 : 0) + (w_dtype == WR_BF16 ? 1 : 0);
  switch (key) {
    case 0: return norm_launch<float, float, float>(ctx, a);
    case 1: return norm_launch<float, float, uint16_t>(ctx, a);
    case 2: return norm_launch<float, uint16_t, float>(ctx, a);
    case 3: return norm_launch<float, uint16_t, uint16_t>(ctx, a);
    case 4: return norm_launch<uint16_t, float, float>(ctx, a);
    case 5: return norm_launch<uint16_t, float, uint16_t>(ctx, a);
    case 6: return norm_launch<uint16_t, uint16_t, float>(ctx, a);
    default: return norm_launch<uint16_t, uint16_t, uint16_t>(ctx, a);
  }
}

template <typename T>
static int quant_launch(wr_ctx* ctx, const T* x, int64_t rows, int64_t n, int64_t ldx, int8_t* q, int64_t ldq,
                        float* scales) {
  if (n > 16384) {
    hipLaunchKernelGGL(quant_rows_wide_kernel<T>, dim3((int)std::min<int64_t>(rows, 1 << 20)), dim3(512), 0,
                       ctx->stream, x, ldx, (int)rows, n, q, ldq, scales);
  } else {
    quant_shape(ctx->num_cu, rows, n, [&](auto ch, auto lanes, auto most, int threads, int grid) {
      hipLaunchKernelGGL((quant_rows_kernel<T, decltype(ch)::value, decltype(lanes)::value, decltype(most)::value>),
                         dim3(grid), dim3(threads), 0, ctx->stream, x, ldx, (int)rows, (int)n, q, ldq, scales);
    });
  }
  WR_CHECK_LAUNCH();
  return WR_OK;
}

int wr_quant_rows_i8_impl(wr_ctx* ctx, const void* x, int x_dtype, int64_t rows, int64_t n, int64_t ldx, int8_t* q,
                          int64_t ldq, float* scales) {
  if (x_dtype == WR_BF16) return quant_launch(ctx, (const uint16_t*)x, rows, n, ldx, q, ldq, scales);
  return quant_launch(ctx, (const float*)x, rows, n, ldx, q, ldq, scales);
}
