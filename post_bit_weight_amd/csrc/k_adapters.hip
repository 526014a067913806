// Low-rank adapters of many requests beside a shared projection: y = base + s B (A x).
#include "rowops.hpp"

namespace wr {

namespace {

constexpr int kThreads = 256;

struct AdapterArgs {
  const int32_t* starts;
  const int32_t* ids;
  const int32_t* ranks;
  const float* scales;
  const uint16_t* A;
  const uint16_t* B;
  float* t;        // rows x rank
  int64_t rows, n, outs, most;
  int64_t ldx, ldb, ldy;
  int32_t adapters, rank, n_seqs;
};

struct Request {
  int64_t row, count;  // count 0: nothing to do
  int adapter, rank;   // adapter -1: none
};

__device__ __forceinline__ Request request_of(const AdapterArgs& a, int i) {
  const int64_t b = a.starts[i], e = a.starts[i + 1];
  const bool ok = b >= 0 && e >= b && e <= a.rows && e - b <= a.most;
  int id = a.ids[i];
  if (id < 0 || id >= a.adapters) id = -1;
  int rank = a.rank;
  if (id >= 0 && a.ranks) rank = min(max(a.ranks[id], 0), a.rank);
  return Request{b, ok ? e - b : 0, id, id >= 0 ? rank : 0};
}

template <typename T>
__device__ __forceinline__ float value(T v) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_f32(v);
  else return v;
}

// t = A x: a workgroup a row.
template <typename X>
__global__ __launch_bounds__(kThreads) void adapters_in_kernel(AdapterArgs a, const X* __restrict__ x) {
  const Request q = request_of(a, blockIdx.y);
  if (q.adapter < 0) return;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int64_t j = blockIdx.x; j < q.count; j += gridDim.x) {
    const X* xr = x + (q.row + j) * a.ldx;
    for (int r = wave; r < q.rank; r += kThreads / kWave) {
      const uint16_t* ar = a.A + ((int64_t)q.adapter * a.rank + r) * a.n;
      float sum = 0.0f;
      for (int64_t c = lane; c < a.n; c += kWave) sum = fmaf(bf16_bits_to_f32(ar[c]), value(xr[c]), sum);
      for (int m = 1; m < kWave; m <<= 1) sum += __shfl_xor(sum, m);
      if (lane == 0) a.t[(q.row + j) * a.rank + r] = sum;
    }
  }
}

// y = base + s B t: a workgroup a row.
template <typename Y>
__global__ __launch_bounds__(kThreads) void adapters_out_kernel(AdapterArgs a, const Y* base, Y* y) {
  const Request q = request_of(a, blockIdx.y);
  const float s = q.adapter >= 0 ? a.scales[q.adapter] : 0.0f;
  for (int64_t j = blockIdx.x; j < q.count; j += gridDim.x) {
    const int64_t row = q.row + j;
    for (int64_t o = threadIdx.x; o < a.outs; o += kThreads) {
      float sum = 0.0f;
      if (q.adapter >= 0) {
        const uint16_t* br = a.B + ((int64_t)q.adapter * a.outs + o) * a.rank;
        for (int r = 0; r < q.rank; ++r) sum = fmaf(bf16_bits_to_f32(br[r]), a.t[row * a.rank + r], sum);
        sum *= s;
      }
      if (base) sum += value(base[row * a.ldb + o]);
      if constexpr (sizeof(Y) == 2) y[row * a.ldy + o] = (Y)f32_to_bf16_bits(sum);
      else y[row * a.ldy + o] = sum;
    }
  }
}

}  // namespace

}  // namespace wr

using namespace wr;

size_t wr_adapters_ws_bytes(int64_t rows, int64_t n, int32_t rank) {
  (void)n;
  return (size_t)rows * rank * sizeof(float);
}

int wr_adapters_impl(wr_ctx* ctx, const void* x, int x_dtype, int64_t rows, int64_t n, int64_t ldx, const void* A,
                     const void* B, int32_t adapters, int32_t rank, int64_t outs, const float* scales,
                     const int32_t* ranks, const int32_t* starts, const int32_t* ids, int32_t n_seqs, int64_t most,
                     const void* base, int64_t ldb, void* y, int y_dtype, int64_t ldy) {
  const AdapterArgs a{starts, ids, ranks, scales, static_cast<const uint16_t*>(A), static_cast<const uint16_t*>(B),
                      static_cast<float*>(ctx->ws), rows, n, outs, most, ldx, ldb, ldy, adapters, rank, n_seqs};
  if (ctx->ws_bytes < wr_adapters_ws_bytes(rows, n, rank)) return WR_EWORKSPACE;
  const dim3 grid((uint32_t)std::min<int64_t>(std::max<int64_t>(std::min(most, rows), 1), 4096), (uint32_t)n_seqs);
  if (adapters > 0 && rank > 0) {
    if (x_dtype == WR_BF16)
      hipLaunchKernelGGL(adapters_in_kernel<uint16_t>, grid, dim3(kThreads), 0, ctx->stream, a, static_cast<const uint16_t*>(x));
    else
      hipLaunchKernelGGL(adapters_in_kernel<float>, grid, dim3(kThreads), 0, ctx->stream, a, static_cast<const float*>(x));
    WR_CHECK_LAUNCH();
  }
  if (y_dtype == WR_BF16)
    hipLaunchKernelGGL(adapters_out_kernel<uint16_t>, grid, dim3(kThreads), 0, ctx->stream, a,
                       static_cast<const uint16_t*>(base), static_cast<uint16_t*>(y));
  else
    hipLaunchKernelGGL(adapters_out_kernel<float>, grid, dim3(kThreads), 0, ctx->stream, a, static_cast<const float*>(base),
                       static_cast<float*>(y));
  WR_CHECK_LAUNCH();
  return WR_OK;
}
