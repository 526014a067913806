// Gradient of the block norm (see k_norm.hip): u = w_post bn, x' = rscale x + bscale g u,
// y = w_pre xn with bn = b / rms(b), xn = x' / rms(x').
//
// With d = dy w_pre and c = bscale g w_post bn (the derivative's direction along bn), the gradient of x' is
// dx' = dres + r2 (d - xn m1), m1 = mean(d xn), and that of b needs mean(c dx') =
// mean(c (dres + r2 d)) - r2 m1 mean(c xn): three sums over the row that do not wait for one another, so
// one reduction per row.  The row's values stay in registers; x' is formed again from b and x.
//
// The parameters' gradients are sums over tokens.  A unit (the lanes that share a row) walks consecutive
// tokens with its columns' sums in registers and writes them once; a second kernel adds the units in
// index order.  Nothing is added with atomics, so the result does not depend on timing.
#include "rowops.hpp"

namespace wr {

// How the tokens are cut: `units` ranges of at most `span` tokens.  Gate rows of at most `span` tokens lie
// whole inside a unit (`segs` == 0: the unit writes their gradient itself); longer ones are cut into
// `segs` units each, whose partial sums a second kernel adds.
struct BwdPlan {
  int64_t units, span, gate_rows, gates, segs, blocks;
  int lanes, threads, chunks;
};

constexpr int64_t kBwdBlocks = 1024;  // four workgroups for each of 256 CUs

static BwdPlan bwd_plan(int64_t rows, int64_t n, int64_t gate_rows) {
  BwdPlan p;
  const int64_t per8 = (n + 7) / 8;
  p.lanes = n <= 128 ? 16 : n <= 256 ? 32 : n <= 512 ? 64 : 0;
  p.chunks = n <= 4096 ? 1 : n <= 8192 ? 2 : 4;
  p.threads = p.lanes ? 256 : (int)(((per8 + p.chunks - 1) / p.chunks + 63) / 64 * 64);
  const int64_t per = p.lanes ? 256 / p.lanes : 1;  // units per workgroup
  p.span = std::max<int64_t>(1, (rows + kBwdBlocks * per - 1) / (kBwdBlocks * per));
  p.gate_rows = gate_rows == 0 || gate_rows >= rows ? rows : gate_rows;
  p.gates = (rows + p.gate_rows - 1) / p.gate_rows;
  if (p.gate_rows <= p.span) {
    p.span = p.span / p.gate_rows * p.gate_rows;
    p.segs = 0;
    p.units = (rows + p.span - 1) / p.span;
  } else {
    p.segs = (p.gate_rows + p.span - 1) / p.span;
    p.span = (p.gate_rows + p.segs - 1) / p.segs;
    p.units = p.gates * p.segs;
  }
  p.blocks = (p.units + per - 1) / per;
  return p;
}

struct BwdArgs {
  int rows, n, span, segs, gate_rows;
  int64_t units;
  const void* branch;
  int64_t ldb;
  const void* w_post;
  const void* gate;
  int64_t ldg;
  float bscale;
  const void* resid;
  int64_t ldr;
  float rscale;
  const void* w_pre;
  const float* stats;
  const void* dy;
  int64_t lddy;
  const void* dres;
  int64_t lddo;
  void* db;
  int64_t lddb;
  void* dx;
  int64_t lddr;
  float* part_post;  // blocks x n, or null
  float* part_pre;   // blocks x n, or null
  float* part_gate;  // units x n (segs > 0), or null
  float* dgate;      // gates x n (segs == 0), or null
};

template <typename TB, typename TR, typename TW, int CH, int LANES>
__global__ __launch_bounds__(LANES > 0 ? 256 : 512) void block_norm_bwd_kernel(const BwdArgs a) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  __shared__ float comb[LANES > 0 ? 8 * 256 : 1];
  RowGroup<LANES> grp{red};
  const int lane = LANES > 0 ? threadIdx.x % (LANES > 0 ? LANES : 1) : threadIdx.x;
  const int cstep = LANES > 0 ? 8 * LANES : 8 * blockDim.x;
  const int64_t unit = LANES > 0 ? (int64_t)blockIdx.x * (256 / (LANES > 0 ? LANES : 1)) + threadIdx.x / (LANES > 0 ? LANES : 1)
                                 : (int64_t)blockIdx.x;
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  int64_t r0, r1;
  int64_t gidx;
  if (a.segs) {
    gidx = unit / a.segs;
    r0 = gidx * a.gate_rows + unit % a.segs * a.span;
    r1 = std::min<int64_t>(std::min<int64_t>(r0 + a.span, (gidx + 1) * a.gate_rows), a.rows);
  } else {
    r0 = unit * a.span;
    r1 = std::min<int64_t>(r0 + a.span, a.rows);
    gidx = r0 / a.gate_rows;
  }
  int64_t gend = (gidx + 1) * a.gate_rows;

  float s_pre[CH][8], s_post[CH][8], s_gate[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) s_pre[k][e] = s_post[k][e] = s_gate[k][e] = 0.0f;

  for (int64_t row = r0; row < r1; ++row) {
    Raw8<TB> b[CH], g[CH], dy[CH];
    Raw8<TR> x[CH], dr[CH];
    Raw8<TW> wp[CH], wq[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c < n) {
        if (a.branch) load8(b[k], (const TB*)a.branch + row * a.ldb, c, n);
        if (a.resid) load8(x[k], (const TR*)a.resid + row * a.ldr, c, n);
        if (a.dy) load8(dy[k], (const TB*)a.dy + row * a.lddy, c, n);
        if (a.dres) load8(dr[k], (const TR*)a.dres + row * a.lddo, c, n);
        if (a.gate) load8(g[k], (const TB*)a.gate + gidx * a.ldg, c, n);
        if (a.w_post) load8(wp[k], (const TW*)a.w_post, c, n);
        if (a.dy) load8(wq[k], (const TW*)a.w_pre, c, n);
      }
    }
    const float ib = a.w_post ? a.stats[2 * row] : 1.0f, ix = a.dy ? a.stats[2 * row + 1] : 0.0f;
    float bn[CH][8], xn[CH][8], t[CH][8], cg[CH][8];  // t: dres + r2 d;  cg: bscale g
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c >= n) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bn[k][e] = a.branch ? b[k].get(e) * ib : 0.0f;
        cg[k][e] = a.gate ? a.bscale * g[k].get(e) : a.bscale;
        const float cw = a.w_post ? cg[k][e] * wp[k].get(e) : cg[k][e];  // derivative of x' by bn
        const float xo = a.resid ? fmaf(a.rscale, x[k].get(e), cw * bn[k][e]) : cw * bn[k][e];
        xn[k][e] = xo * ix;
        const float d = a.dy ? dy[k].get(e) : 0.0f;
        s_pre[k][e] = fmaf(d, xn[k][e], s_pre[k][e]);
        const float dw = a.dy ? d * wq[k].get(e) : 0.0f;
        t[k][e] = fmaf(ix, dw, a.dres ? dr[k].get(e) : 0.0f);
        sums[0] = fmaf(dw, xn[k][e], sums[0]);
        sums[1] = fmaf(cw * bn[k][e], t[k][e], sums[1]);
        sums[2] = fmaf(cw * bn[k][e], xn[k][e], sums[2]);
      }
    }
    grp.template reduce<AddF32>(sums);
    const float m1 = sums[0] * inv_n * ix;           // r2 mean(d xn)
    const float m2 = (sums[1] - m1 * sums[2]) * inv_n;  // mean(c dx')
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c >= n) continue;
      float dxo[8], out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dxo[e] = fmaf(-m1, xn[k][e], t[k][e]);
        out[e] = a.rscale * dxo[e];
      }
      if (a.dx) store8((TR*)a.dx + row * a.lddr, c, n, out);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = a.w_post ? wp[k].get(e) : 1.0f;
        const float du = cg[k][e] * dxo[e];
        s_post[k][e] = fmaf(du, bn[k][e], s_post[k][e]);
        s_gate[k][e] = fmaf(a.bscale * dxo[e], w * bn[k][e], s_gate[k][e]);
        out[e] = a.w_post ? ib * fmaf(-m2, bn[k][e], du * w) : du;
      }
      if (a.db) store8((TB*)a.db + row * a.lddb, c, n, out);
    }
    if (a.segs == 0 && (row + 1 == gend || row + 1 == r1)) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = 8 * lane + k * cstep;
        if (a.dgate && c < n) store8(a.dgate + gidx * n, c, n, s_gate[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s_gate[k][e] = 0.0f;
      }
      ++gidx;
      gend += a.gate_rows;
    }
  }

  if (a.part_gate && unit < a.units) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c < n) store8(a.part_gate + unit * n, c, n, s_gate[k]);
    }
  }
  if constexpr (LANES > 0) {
    // the workgroup's units, added in order; a unit past the last one holds zeros
    constexpr int per = 256 / (LANES > 0 ? LANES : 1), width = 8 * LANES;
    auto combine = [&](const float (&s)[8], float* part) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) comb[threadIdx.x * 8 + e] = s[e];
      __syncthreads();
      for (int c = threadIdx.x; c < n; c += 256) {
        float sum = 0.0f;
        for (int u = 0; u < per; ++u) sum += comb[u * width + c];
        part[(int64_t)blockIdx.x * n + c] = sum;
      }
    };
    if (a.part_pre) combine(s_pre[0], a.part_pre);
    if (a.part_post) combine(s_post[0], a.part_post);
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * lane + k * cstep;
      if (c >= n) continue;
      if (a.part_pre) store8(a.part_pre + (int64_t)blockIdx.x * n, c, n, s_pre[k]);
      if (a.part_post) store8(a.part_post + (int64_t)blockIdx.x * n, c, n, s_post[k]);
    }
  }
}

// out[g][c] = sum over p < count of part[g * count + p][c], p in order within 32 strided shares, the shares
// in order.  blockIdx.x: 32 columns; blockIdx.y: output row.
constexpr int CS_COLS = 32, CS_SHARES = 32;
__global__ __launch_bounds__(CS_COLS* CS_SHARES) void column_sum_kernel(const float* __restrict__ part, int64_t count,
                                                                        int n, float* __restrict__ out) {
  __shared__ float red[CS_SHARES][CS_COLS + 1];
  const int cx = threadIdx.x % CS_COLS, sh = threadIdx.x / CS_COLS, c = blockIdx.x * CS_COLS + cx;
  const int64_t first = blockIdx.y * count;
  float s = 0.0f;
  if (c < n) {
    const float* p = part + first * n + c;
    int64_t i = sh;
    for (; i + 3 * CS_SHARES < count; i += 4 * CS_SHARES) {
      const float v0 = p[i * n], v1 = p[(i + CS_SHARES) * n], v2 = p[(i + 2 * CS_SHARES) * n],
                  v3 = p[(i + 3 * CS_SHARES) * n];
      s += v0;
      s += v1;
      s += v2;
      s += v3;
    }
    for (; i < count; i += CS_SHARES) s += p[i * n];
  }
  red[sh][cx] = s;
  __syncthreads();
  if (sh == 0 && c < n) {
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < CS_SHARES; ++k) total += red[k][cx];
    out[blockIdx.y * (int64_t)n + c] = total;
  }
}

}  // namespace wr

using namespace wr;

static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

size_t wr_norm_bwd_ws_bytes(int64_t rows, int64_t n, int64_t gate_rows) {
  if (rows <= 0) return 256;
  const BwdPlan p = bwd_plan(rows, n, gate_rows);
  return 2 * round256((size_t)p.blocks * n * 4) + (p.segs ? round256((size_t)p.units * n * 4) : 0);
}

template <typename TB, typename TR, typename TW>
static void bwd_launch(wr_ctx* ctx, const BwdPlan& p, const BwdArgs& a) {
  auto go = [&](auto ch, auto lanes) {
    hipLaunchKernelGGL((block_norm_bwd_kernel<TB, TR, TW, decltype(ch)::value, decltype(lanes)::value>),
                       dim3((unsigned)p.blocks), dim3(p.threads), 0, ctx->stream, a);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 0> group;
  if (p.lanes == 16) go(one, std::integral_constant<int, 16>{});
  else if (p.lanes == 32) go(one, std::integral_constant<int, 32>{});
  else if (p.lanes == 64) go(one, std::integral_constant<int, 64>{});
  else if (p.chunks == 1) go(one, group);
  else if (p.chunks == 2) go(std::integral_constant<int, 2>{}, group);
  else go(std::integral_constant<int, 4>{}, group);
}

int wr_block_norm_backward_impl(wr_ctx* ctx, int64_t rows, int64_t n, const void* branch, int b_dtype, int64_t ldb,
                                const void* w_post, const void* gate, int64_t ldg, int64_t gate_rows,
                                float branch_scale, const void* resid, int r_dtype, int64_t ldr, float resid_scale,
                                const void* w_pre, int w_dtype, const float* stats, const void* dy, int64_t lddy,
                                const void* dresid_out, int64_t lddo, void* dbranch, int64_t lddb, void* dresid,
                                int64_t lddr, float* dw_post, float* dgate, float* dw_pre) {
  const unsigned cols = (unsigned)((n + CS_COLS - 1) / CS_COLS);
  auto sum = [&](const float* from, int64_t count, int64_t groups, float* to) {
    for (int64_t g0 = 0; g0 < groups; g0 += 65535) {
      const unsigned gs = (unsigned)std::min<int64_t>(65535, groups - g0);
      hipLaunchKernelGGL(column_sum_kernel, dim3(cols, gs), dim3(CS_COLS * CS_SHARES), 0, ctx->stream,
                         from + g0 * count * n, count, (int)n, to + g0 * n);
    }
  };
  if (rows == 0) {  // sums over no tokens
    if (dw_post) sum(nullptr, 0, 1, dw_post);
    if (dw_pre) sum(nullptr, 0, 1, dw_pre);
    if (dgate && gate_rows == 0) sum(nullptr, 0, 1, dgate);
    WR_CHECK_LAUNCH();
    return WR_OK;
  }
  if (ctx->ws_bytes < wr_norm_bwd_ws_bytes(rows, n, gate_rows) || !ctx->ws) return WR_EWORKSPACE;
  const BwdPlan p = bwd_plan(rows, n, gate_rows);
  char* ws = (char*)ctx->ws;
  const size_t part = round256((size_t)p.blocks * n * 4);
  BwdArgs a{};
  a.rows = (int)rows;
  a.n = (int)n;
  a.span = (int)p.span;
  a.segs = (int)p.segs;
  a.gate_rows = (int)p.gate_rows;
  a.units = p.units;
  a.branch = branch;
  a.ldb = ldb;
  a.w_post = w_post;
  a.gate = gate;
  a.ldg = ldg;
  a.bscale = branch_scale;
  a.resid = resid;
  a.ldr = ldr;
  a.rscale = resid_scale;
  a.w_pre = w_pre;
  a.stats = stats;
  a.dy = dy;
  a.lddy = lddy;
  a.dres = dresid_out;
  a.lddo = lddo;
  a.db = dbranch;
  a.lddb = lddb;
  a.dx = dresid;
  a.lddr = lddr;
  a.part_post = dw_post ? (float*)ws : nullptr;
  a.part_pre = dw_pre ? (float*)(ws + part) : nullptr;
  a.part_gate = dgate && p.segs ? (float*)(ws + 2 * part) : nullptr;
  a.dgate = p.segs ? nullptr : dgate;
  const int key = (b_dtype == WR_BF16 ? 4 : 0) + (r_dtype == WR_BF16 ? 2 : 0) + (w_dtype == WR_BF16 ? 1 : 0);
  switch (key) {
    case 0: bwd_launch<float, float, float>(ctx, p, a); break;
    case 1: bwd_launch<float, float, uint16_t>(ctx, p, a); break;
    case 2: bwd_launch<float, uint16_t, float>(ctx, p, a); break;
    case 3: bwd_launch<float, uint16_t, uint16_t>(ctx, p, a); break;
    case 4: bwd_launch<uint16_t, float, float>(ctx, p, a); break;
    case 5: bwd_launch<uint16_t, float, uint16_t>(ctx, p, a); break;
    case 6: bwd_launch<uint16_t, uint16_t, float>(ctx, p, a); break;
    default: bwd_launch<uint16_t, uint16_t, uint16_t>(ctx, p, a); break;
  }
  WR_CHECK_LAUNCH();
  if (dw_post) sum(a.part_post, p.blocks, 1, dw_post);
  if (dw_pre) sum(a.part_pre, p.blocks, 1, dw_pre);
  if (a.part_gate) sum(a.part_gate, p.segs, p.gates, dgate);
  WR_CHECK_LAUNCH();
  return WR_OK;
}
