// Rotary positions with several axes.
//
// Every value is read and written once, so the bound is memory.  A row's angles serve all of its heads: a workgroup
// forms the cosines and sines of its rows once, in LDS, and then streams the rows.  The angle is an fp64 product of
// position and frequency that is reduced to a part of a turn in fp64 (fp32 would leave position 40960 an error of
// 2^-9 radians); the part goes through sincospi in fp32.
#include "rowops.hpp"

namespace wr {

namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 512;  // dim <= 1024

struct RotaryArgs {
  int64_t ldx, ldy, ldp;
  const int32_t* positions;
  const int32_t* axis_of;
  const double* freqs;
  int64_t rows;
  int heads, dim, pairs, axes;
  bool interleaved, inverse, in_place;
};

// The row's turns into LDS: cos in turn[.].x, sin in turn[.].y; a pair that does not turn has (1, 0).
__device__ __forceinline__ void row_turns(const RotaryArgs& a, int64_t row, f32x2* turn, int first, int step) {
  for (int i = first; i < a.pairs; i += step) {
    const int axis = a.axis_of ? a.axis_of[i] : 0;
    f32x2 t{1.0f, 0.0f};
    if (axis >= 0 && axis < a.axes) {
      const double turns = (double)a.positions[axis * a.ldp + row] * a.freqs[i] * 0.15915494309189533577;  // 1 / 2 pi
      const float part = (float)(2.0 * (turns - rint(turns)));
      float s, c;
      sincospif(part, &s, &c);
      t = f32x2{c, a.inverse ? -s : s};
    }
    turn[i] = t;
  }
}

// One value or pair at a time, for any pairs and dim.
template <typename T>
__global__ __launch_bounds__(kThreads) void rotary_any_kernel(RotaryArgs a, const T* x, T* y) {
  __shared__ f32x2 turn[kPairs];
  auto get = [](T v) {
    if constexpr (sizeof(T) == 2) return bf16_bits_to_f32(v);
    else return v;
  };
  auto put = [](float f) {
    if constexpr (sizeof(T) == 2) return (T)f32_to_bf16_bits(f);
    else return f;
  };
  const int units = a.dim - a.pairs;  // pairs, then the values behind them
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    __syncthreads();
    row_turns(a, row, turn, threadIdx.x, kThreads);
    __syncthreads();
    const T* xr = x + row * a.ldx;
    T* yr = y + row * a.ldy;
    for (int64_t u = threadIdx.x; u < (int64_t)a.heads * units; u += kThreads) {
      const int64_t h = u / units * a.dim;
      const int i = (int)(u % units);
      if (i < a.pairs) {
        const int64_t p = h + (a.interleaved ? 2 * i : i), q = h + (a.interleaved ? 2 * i + 1 : a.pairs + i);
        const float v0 = get(xr[p]), v1 = get(xr[q]);
        const f32x2 t = turn[i];
        yr[p] = put(v0 * t.x - v1 * t.y);
        yr[q] = put(v0 * t.y + v1 * t.x);
      } else if (!a.in_place) {
        yr[h + a.pairs + i] = xr[h + a.pairs + i];
      }
    }
  }
}

}  // namespace

}  // namespace wr

using namespace wr;

template <typename T>
static void rotary_launch(wr_ctx* ctx, const RotaryArgs& a, const void* x, void* y) {
  const uint32_t blocks = (uint32_t)std::min<int64_t>(a.rows, 1 << 20);
  hipLaunchKernelGGL(rotary_any_kernel<T>, dim3(blocks), dim3(kThreads), 0, ctx->stream, a, static_cast<const T*>(x),
                     static_cast<T*>(y));
}

int wr_rotary_impl(wr_ctx* ctx, const void* x, int dtype, int64_t rows, int32_t heads, int32_t dim, int64_t ldx,
                   int32_t pairs, const int32_t* positions, int32_t axes, int64_t ldp, const int32_t* axis_of,
                   const double* freqs, int flags, void* y, int64_t ldy) {
  const RotaryArgs a{ldx,   ldy,  ldp, positions, axis_of, freqs,
                     rows,  heads, dim, pairs,     axes,    (flags & WR_ROTARY_INTERLEAVED) != 0,
                     (flags & WR_ROTARY_INVERSE) != 0, x == y};
  if (dtype == WR_BF16)
    rotary_launch<uint16_t>(ctx, a, x, y);
  else
    rotary_launch<float>(ctx, a, x, y);
  WR_CHECK_LAUNCH();
  return WR_OK;
}
