// The norms before and after a block with the gate and the residual scale between them, and the
// quantization of activation rows to 8-bit integers.
//
//   u = w_post b / rms(b),  x' = rscale x + bscale g u,  y = w_pre x' / rms(x'),  q = rint(127 y / max|y|)
//
// Every value of a row stays in registers from its one load to its stores: the two sums of squares and
// the maximum are reductions over the lanes that share the row.  Rows of up to 512 values take 16, 32 or
// 64 lanes of a wave (no barrier); wider rows take a workgroup of up to 512 threads with one, two or four
// chunks of eight values per thread.
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

template <int LANES>
__device__ __forceinline__ int row_lane() {
  return LANES > 0 ? threadIdx.x % (LANES > 0 ? LANES : 1) : threadIdx.x;
}
// First row, step and column step of this thread's row group.
template <int LANES>
__device__ __forceinline__ void row_walk(int& first, int& step, int& cstep) {
  if constexpr (LANES > 0) {
    const int per = blockDim.x / LANES;
    first = blockIdx.x * per + threadIdx.x / LANES;
    step = gridDim.x * per;
    cstep = 8 * LANES;
  } else {
    first = blockIdx.x;
    step = gridDim.x;
    cstep = 8 * blockDim.x;
  }
}

template <typename TB, typename TR, typename TW, int CH, int LANES>
__global__ __launch_bounds__(LANES > 0 ? 256 : 512) void block_norm_kernel(const NormArgs a) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  RowGroup<LANES> grp{red};
  int first, step, cstep;
  row_walk<LANES>(first, step, cstep);
  const int lane = row_lane<LANES>(), n = a.n;
  const float inv_n = 1.0f / (float)n;
  for (int64_t row = first; row < a.rows; row += step) {
    Raw8<TB> b[CH], g[CH];
    Raw8<TR> x[CH];
    Raw8<TW> wp[CH], wq[CH];
    const TB* brow = (const TB*)a.branch + row * a.ldb;
    const TR* xrow = (const TR*)a.resid + row * a.ldr;
    const TB* grow = (const TB*)a.gate + (a.gate_rows ? (uint32_t)row / (uint32_t)a.gate_rows : 0u) * a.ldg;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c < n) {
        if (a.branch) load8(b[k], brow, c, n);
        if (a.resid) load8(x[k], xrow, c, n);
        if (a.w_post) load8(wp[k], (const TW*)a.w_post, c, n);
        if (a.gate) load8(g[k], grow, c, n);
        if (a.w_pre) load8(wq[k], (const TW*)a.w_pre, c, n);
      }
    }
    float r1 = 1.0f, r2 = 1.0f;
    if (a.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < CH; ++k)
        if (8 * lane + k * cstep < n)
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(b[k].get(e), b[k].get(e), ss);
      r1 = 1.0f / sqrtf(grp.sum(ss) * inv_n + a.eps);
    }
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c >= n) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float u = 0.0f;
        if (a.branch) {
          u = b[k].get(e);
          if (a.w_post) u = u * r1 * wp[k].get(e);
          if (a.gate) u *= g[k].get(e);
          u *= a.bscale;
        }
        v[k][e] = a.resid ? fmaf(a.rscale, x[k].get(e), u) : u;
        ss = fmaf(v[k][e], v[k][e], ss);
      }
      if (a.resid_out) store8((TR*)a.resid_out + row * a.ldo, c, n, v[k]);
    }
    if (a.w_pre) {
      r2 = 1.0f / sqrtf(grp.sum(ss) * inv_n + a.eps);
      uint32_t top = 0u;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = 8 * lane + k * cstep;
        if (c >= n) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[k][e] = v[k][e] * r2 * wq[k].get(e);
          if (c + e < n) top = MaxU32::op(top, __float_as_uint(v[k][e]) & 0x7fffffffu);
        }
        if (a.y) store8((TB*)a.y + row * a.ldy, c, n, v[k]);
      }
      if (a.q) {
        const RowCoder code(grp.max(top));
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int c = 8 * lane + k * cstep;
          if (c < n) store_codes(a.q + row * a.ldq, c, n, code.codes(v[k]));
        }
        if (lane == 0) a.q_scales[row] = code.scale;
      }
    }
    if (a.stats && lane == 0) {
      a.stats[2 * row] = r1;
      a.stats[2 * row + 1] = r2;
    }
  }
}

template <typename T, int CH, int LANES>
__global__ __launch_bounds__(LANES > 0 ? 256 : 512) void quant_rows_kernel(const T* __restrict__ x, int64_t ldx,
                                                                           int rows, int n, int8_t* __restrict__ q,
                                                                           int64_t ldq, float* __restrict__ scales) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  RowGroup<LANES> grp{red};
  int first, step, cstep;
  row_walk<LANES>(first, step, cstep);
  const int lane = row_lane<LANES>();
  for (int64_t row = first; row < rows; row += step) {
    Raw8<T> r[CH];
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c < n) {
        load8(r[k], x + row * ldx, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = MaxU32::op(top, __float_as_uint(r[k].get(e)) & 0x7fffffffu);
      }
    }
    const RowCoder code(grp.max(top));
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c < n) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r[k].get(e);
        store_codes(q + row * ldq, c, n, code.codes(v));
      }
    }
    if (lane == 0) scales[row] = code.scale;
  }
}

// Rows wider than the registers of a workgroup: two passes over the row, the second from the caches.
template <typename T>
__global__ __launch_bounds__(512) void quant_rows_wide_kernel(const T* __restrict__ x, int64_t ldx, int rows, int64_t n,
                                                              int8_t* __restrict__ q, int64_t ldq,
                                                              float* __restrict__ scales) {
  __shared__ uint32_t red[2][3][RowGroup<0>::kMaxWaves];
  RowGroup<0> grp{red};
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    uint32_t top = 0u;
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * 512) {
      Raw8<T> r;
      load8(r, x + row * ldx + c, 0, (int)std::min<int64_t>(n - c, 8));
#pragma unroll
      for (int e = 0; e < 8; ++e) top = MaxU32::op(top, __float_as_uint(r.get(e)) & 0x7fffffffu);
    }
    const RowCoder code(grp.max(top));
    for (int64_t c = 8 * threadIdx.x; c < n; c += 8 * 512) {
      Raw8<T> r;
      const int cnt = (int)std::min<int64_t>(n - c, 8);
      load8(r, x + row * ldx + c, 0, cnt);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = r.get(e);
      store_codes(q + row * ldq + c, 0, cnt, code.codes(v));
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
  }
}

}  // namespace wr

using namespace wr;

// Lanes per row, chunks per thread and threads for rows of n values (n <= 16384): `launch` gets them as
// integral constants (chunks, lanes) and the number of threads and workgroups.
template <typename F>
static void row_shape(int64_t rows, int64_t n, F&& launch) {
  const int64_t most = (int64_t)1 << 20;  // workgroups; each walks further rows beyond that
  const int chunks = (int)((n + 7) / 8);
  auto lanes = [&](auto l) {
    const int64_t per = 256 / decltype(l)::value;
    launch(std::integral_constant<int, 1>{}, l, 256, (int)std::min(most, (rows + per - 1) / per));
  };
  auto wide = [&](auto ch) {
    const int threads = ((chunks + decltype(ch)::value - 1) / decltype(ch)::value + 63) / 64 * 64;
    launch(ch, std::integral_constant<int, 0>{}, threads, (int)std::min(most, rows));
  };
  if (n <= 128) lanes(std::integral_constant<int, 16>{});
  else if (n <= 256) lanes(std::integral_constant<int, 32>{});
  else if (n <= 512) lanes(std::integral_constant<int, 64>{});
  else if (n <= 4096) wide(std::integral_constant<int, 1>{});
  else if (n <= 8192) wide(std::integral_constant<int, 2>{});
  else wide(std::integral_constant<int, 4>{});
}

template <typename TB, typename TR, typename TW>
static int norm_launch(wr_ctx* ctx, const NormArgs& a) {
  row_shape(a.rows, a.n, [&](auto ch, auto lanes, int threads, int grid) {
    hipLaunchKernelGGL((block_norm_kernel<TB, TR, TW, decltype(ch)::value, decltype(lanes)::value>), dim3(grid),
                       dim3(threads), 0, ctx->stream, a);
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
    row_shape(rows, n, [&](auto ch, auto lanes, int threads, int grid) {
      hipLaunchKernelGGL((quant_rows_kernel<T, decltype(ch)::value, decltype(lanes)::value>), dim3(grid),
                         dim3(threads), 0, ctx->stream, x, ldx, (int)rows, (int)n, q, ldq, scales);
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
