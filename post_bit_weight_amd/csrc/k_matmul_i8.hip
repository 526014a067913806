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

// Few tokens (up to 64): the weights are read once, straight from memory into matrix-core operands, and
// everything else is hidden behind that.  A workgroup owns 16 outputs (with GLU or RF = 2, 32 weight rows) for
// all tokens; its NW waves cut the sum into contiguous ranges of 64-byte steps, so that a wave has
// many rows' loads in flight at once, and add their int32 sums in LDS.  A 16x16x64 MFMA takes 64
// bytes of 16 weight rows (lane l: row l % 16, bytes 16 (l / 16) .. + 15) against 16 tokens; tokens
// past the batch repeat its last one and are not stored.
template <typename TY, bool GLU, int RF, int NT, int NW, int U>
__global__ __launch_bounds__(64 * NW) void matmul_i8_few_kernel(const I8Args a) {
  __shared__ int32_t red[NW][RF * NT][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int outs = GLU ? a.rows / 2 : a.rows;
  const int o0 = blockIdx.x * (GLU ? 16 : 16 * RF), t0 = blockIdx.y * 16 * NT;
  const int r = lane & 15, kb = 16 * (lane >> 4);
  const int8_t* wrow[RF];
  const int8_t* xrow[NT];
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int o = GLU ? std::min(o0 + r, outs - 1) + f * outs : std::min(o0 + 16 * f + r, outs - 1);
    wrow[f] = a.w + o * a.ldw;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = a.x + std::min(t0 + 16 * t + r, a.batch - 1) * a.ldx;

  i32x4 acc[RF][NT] = {};
  const int steps = a.n / 64, s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
  for (int s = s0; s < s1; s += U) {
    i32x4 fw[U][RF], fx[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 64 * std::min(s + u, s1 - 1) + kb;
#pragma unroll
      for (int f = 0; f < RF; ++f) fw[u][f] = __builtin_bit_cast(i32x4, (u32x4)*reinterpret_cast<const u32x4_any*>(wrow[f] + c));
#pragma unroll
      for (int t = 0; t < NT; ++t) fx[u][t] = __builtin_bit_cast(i32x4, (u32x4)*reinterpret_cast<const u32x4_any*>(xrow[t] + c));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool past = s + u >= s1;  // a step past the range was read again and counts nothing
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const i32x4 x = past ? i32x4{0, 0, 0, 0} : fx[u][t];
#pragma unroll
        for (int f = 0; f < RF; ++f) acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][f], x, acc[f][t], 0, 0, 0);
      }
    }
  }
  if (a.n % 64 != 0 && wave == NW - 1) {
    const int c = 64 * steps + kb;
    i32x4 fw[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) fw[f] = __builtin_bit_cast(i32x4, load16(wrow[f], c, a.n));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const i32x4 x = __builtin_bit_cast(i32x4, load16(xrow[t], c, a.n));
#pragma unroll
      for (int f = 0; f < RF; ++f) acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[f], x, acc[f][t], 0, 0, 0);
    }
  }
  // Register v of lane l holds weight row 4 (l / 16) + v and token l % 16 of a 16 x 16 block.
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][f * NT + t][16 * (lane & 15) + 4 * (lane >> 4) + v] = acc[f][t][v];
  __syncthreads();
  TY* y = (TY*)a.y;
  constexpr int kBlocks = GLU ? NT : RF * NT;  // blocks of 16 outputs x 16 tokens to store
  for (int i = threadIdx.x; i < kBlocks * 256; i += 64 * NW) {
    const int blk = i >> 8, e = i & 255, f = blk / NT, t = t0 + 16 * (blk % NT) + (e >> 4), o = o0 + 16 * f + (e & 15);
    if (t >= a.batch || o >= outs) continue;
    int32_t sum = 0, up = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      sum += red[w][blk][e];
      if constexpr (GLU) up += red[w][NT + blk][e];
    }
    const float xs = a.xs[t];
    float z = (float)sum * xs * a.ws[o];
    if (a.bias) z += a.bias[o];
    if constexpr (GLU) {
      float u = (float)up * xs * a.ws[outs + o];
      if (a.bias) u += a.bias[outs + o];
      z = silu(z) * u;
    }
    put(y + t * a.ldy + o, z);
  }
}

}  // namespace wr

using namespace wr;

template <typename TY, bool GLU, int NT>
static void few_launch(wr_ctx* ctx, const I8Args& a) {
  const int outs = GLU ? a.rows / 2 : a.rows;
  constexpr int RF = GLU ? 2 : 1;
  const dim3 grid((outs + 15) / 16, (a.batch + 16 * NT - 1) / (16 * NT));
  constexpr int U = NT == 1 ? 8 : 4;
  if (a.n >= 4096) {
    constexpr int NW = NT <= 2 ? 16 : 8;
    hipLaunchKernelGGL((matmul_i8_few_kernel<TY, GLU, RF, NT, NW, U>), grid, dim3(64 * NW), 0, ctx->stream, a);
  } else {
    hipLaunchKernelGGL((matmul_i8_few_kernel<TY, GLU, RF, NT, 8, U>), grid, dim3(512), 0, ctx->stream, a);
  }
}

int wr_matmul_i8_impl(wr_ctx* ctx, const int8_t* x, int64_t ldx, const float* x_scales, int64_t batch, const int8_t* w,
                      int64_t ldw, const float* w_scales, int64_t rows, int64_t n, const float* bias, bool glu, void* y,
                      int y_dtype, int64_t ldy) {
  const int64_t outs = glu ? rows / 2 : rows, per = glu ? T8 / 2 : T8;
  const int64_t slice = (int64_t)T8 * 32768;  // tokens per launch (grid.y)
  for (int64_t t0 = 0; t0 < batch; t0 += slice) {
    const I8Args a{x + t0 * ldx, ldx, x_scales + t0, (int)std::min(slice, batch - t0), w, ldw, w_scales, (int)rows,
                   (int)n, bias, (char*)y + t0 * ldy * (y_dtype == WR_BF16 ? 2 : 4), ldy};
    if (a.batch <= 64) {
      auto few = [&](auto ty, auto g) {
        using TY = decltype(ty);
        constexpr bool kGlu = decltype(g)::value;
        if (a.batch <= 16) few_launch<TY, kGlu, 1>(ctx, a);
        else if (a.batch <= 32) few_launch<TY, kGlu, 2>(ctx, a);
        else few_launch<TY, kGlu, 4>(ctx, a);
      };
      if (y_dtype == WR_BF16 && glu) few(uint16_t{}, std::true_type{});
      else if (y_dtype == WR_BF16) few(uint16_t{}, std::false_type{});
      else if (glu) few(float{}, std::true_type{});
      else few(float{}, std::false_type{});
      WR_CHECK_LAUNCH();
      continue;
    }
    const dim3 grid((unsigned)((outs + per - 1) / per), (unsigned)((a.batch + T8 - 1) / T8));
    if (y_dtype == WR_BF16 && glu) hipLaunchKernelGGL((matmul_i8_tile_kernel<uint16_t, true>), grid, dim3(256), 0, ctx->stream, a);
    else if (y_dtype == WR_BF16) hipLaunchKernelGGL((matmul_i8_tile_kernel<uint16_t, false>), grid, dim3(256), 0, ctx->stream, a);
    else if (glu) hipLaunchKernelGGL((matmul_i8_tile_kernel<float, true>), grid, dim3(256), 0, ctx->stream, a);
    else hipLaunchKernelGGL((matmul_i8_tile_kernel<float, false>), grid, dim3(256), 0, ctx->stream, a);
    WR_CHECK_LAUNCH();
  }
  return WR_OK;
}
