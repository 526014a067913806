// Tokens times weights in 8-bit integers: y[t][r] = xs[t] ws[r] sum_j x[t][j] w[r][j] + bias[r], and
// silu(gate) * up of two halves of the weights' rows.
//
// Both operands have the summed index contiguous, which is what a matrix-core operand wants: lane l of
// a 32x32x32 int8 MFMA holds 16 consecutive bytes of row l % 32.  The sums are exact in int32, so their
// order and any split of them change nothing.
#include "rowops.hpp"

namespace wr {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
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

// Sixteen bytes at column c of a row of n bytes, zeros past its end.
__device__ __forceinline__ u32x4 load16(const int8_t* row, int c, int n) {
  if (c + 16 <= n) return *reinterpret_cast<const u32x4_any*>(row + c);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (c + e < n) v[e >> 2] |= (uint32_t)(uint8_t)row[c + e] << (8 * (e & 3));
  return v;
}

__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// 128 tokens x 128 weight rows per workgroup, four waves of 64 x 64, 64 bytes of the sum per step.  With
// GLU the tile's weight rows are 64 gate rows and the 64 up rows of the same outputs, alternating by 32,
// so that a lane holds both sums of an output.
constexpr int T8 = 128, T8_K = 64, T8_LD = T8_K + 16;

template <typename TY, bool GLU>
__global__ __launch_bounds__(256) void matmul_i8_tile_kernel(const I8Args a) {
  __shared__ __attribute__((aligned(16))) int8_t lx[T8 * T8_LD], lw[T8 * T8_LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wi = wave >> 1, wj = wave & 1;
  const int outs = GLU ? a.rows / 2 : a.rows;
  constexpr int kOuts = GLU ? T8 / 2 : T8;
  const int t0 = blockIdx.y * T8, o0 = blockIdx.x * kOuts;
  // the weight row of tile row i, or -1
  auto weight_row = [&](int i) {
    if constexpr (GLU) {
      const int o = o0 + (i >> 6) * 32 + (i & 31);
      return o < outs ? o + ((i >> 5) & 1) * outs : -1;
    } else {
      return o0 + i < outs ? o0 + i : -1;
    }
  };
  i32x16 acc[2][2] = {};
  for (int k0 = 0; k0 < a.n; k0 += T8_K) {
    u32x4 vx[2], vw[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = (tid >> 2) + 64 * u, c = k0 + 16 * (tid & 3), wr_ = weight_row(i);
      vx[u] = t0 + i < a.batch ? load16(a.x + (t0 + i) * a.ldx, c, a.n) : u32x4{0u, 0u, 0u, 0u};
      vw[u] = wr_ >= 0 ? load16(a.w + wr_ * a.ldw, c, a.n) : u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = ((tid >> 2) + 64 * u) * T8_LD + 16 * (tid & 3);
      *reinterpret_cast<u32x4*>(lx + at) = vx[u];
      *reinterpret_cast<u32x4*>(lw + at) = vw[u];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < T8_K; k += 32) {
      i32x4 fx[2], fw[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = (32 * u + (lane & 31)) * T8_LD + k + 16 * (lane >> 5);
        fx[u] = *reinterpret_cast<const i32x4*>(lx + 64 * wi * T8_LD + at);
        fw[u] = *reinterpret_cast<const i32x4*>(lw + 64 * wj * T8_LD + at);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fx[i], fw[j], acc[i][j], 0, 0, 0);
    }
  }
  TY* y = (TY*)a.y;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int t = t0 + 64 * wi + 32 * i + acc_row(v, lane);
      if (t >= a.batch) continue;
      const float xs = a.xs[t];
      if constexpr (GLU) {
        const int o = o0 + 32 * wj + (lane & 31);
        if (o < outs) {
          float g = (float)acc[i][0][v] * xs * a.ws[o], u = (float)acc[i][1][v] * xs * a.ws[outs + o];
          if (a.bias) {
            g += a.bias[o];
            u += a.bias[outs + o];
          }
          put(y + t * a.ldy + o, silu(g) * u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int o = o0 + 64 * wj + 32 * j + (lane & 31);
          if (o < outs) {
            const float z = (float)acc[i][j][v] * xs * a.ws[o];
            put(y + t * a.ldy + o, a.bias ? z + a.bias[o] : z);
          }
        }
      }
    }
}

}  // namespace wr

using namespace wr;

int wr_matmul_i8_impl(wr_ctx* ctx, const int8_t* x, int64_t ldx, const float* x_scales, int64_t batch, const int8_t* w,
                      int64_t ldw, const float* w_scales, int64_t rows, int64_t n, const float* bias, bool glu, void* y,
                      int y_dtype, int64_t ldy) {
  const int64_t outs = glu ? rows / 2 : rows, per = glu ? T8 / 2 : T8;
  const int64_t slice = (int64_t)T8 * 32768;  // tokens per launch (grid.y)
  for (int64_t t0 = 0; t0 < batch; t0 += slice) {
    const I8Args a{x + t0 * ldx, ldx, x_scales + t0, (int)std::min(slice, batch - t0), w, ldw, w_scales, (int)rows,
                   (int)n, bias, (char*)y + t0 * ldy * (y_dtype == WR_BF16 ? 2 : 4), ldy};
    const dim3 grid((unsigned)((outs + per - 1) / per), (unsigned)((a.batch + T8 - 1) / T8));
    if (y_dtype == WR_BF16 && glu) hipLaunchKernelGGL((matmul_i8_tile_kernel<uint16_t, true>), grid, dim3(256), 0, ctx->stream, a);
    else if (y_dtype == WR_BF16) hipLaunchKernelGGL((matmul_i8_tile_kernel<uint16_t, false>), grid, dim3(256), 0, ctx->stream, a);
    else if (glu) hipLaunchKernelGGL((matmul_i8_tile_kernel<float, true>), grid, dim3(256), 0, ctx->stream, a);
    else hipLaunchKernelGGL((matmul_i8_tile_kernel<float, false>), grid, dim3(256), 0, ctx->stream, a);
    WR_CHECK_LAUNCH();
  }
  return WR_OK;
}
