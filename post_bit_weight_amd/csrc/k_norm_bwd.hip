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
//
// Bound by memory: it reads b, x, dy, dres and writes db, dx once.  8192 x 2560 bf16 (252 MB) take 50 us, 5.0 TB/s, and
// the sums over its 512 units (16 MB) 4.8 us; 2000 x 5120 fp32 (246 MB) 50 us.  Rows of more than 8192 bf16 values leave
// no registers for the next row's loads: 2100 x 9728 bf16 (245 MB) 118 us, 2.1 TB/s.
#include "rowops.hpp"

namespace wr {

// How the tokens are cut: `units` ranges of at most `span` tokens.  Gate rows of at most `span` tokens lie
// whole inside a unit (`segs` == 0: the unit writes their gradient itself); longer ones are cut into
// `segs` units each, whose partial sums a second kernel adds.
struct BwdPlan {
  int64_t units, span, gate_rows, gates, segs, blocks;
  int lanes, threads, chunks;
  bool wide;
};

static BwdPlan bwd_plan(int64_t rows, int64_t n, int64_t gate_rows, bool fp32) {
  BwdPlan p;
  const int64_t per8 = (n + 7) / 8;
  p.lanes = n < 8 ? 8 : n <= 128 ? 16 : n <= 256 ? 32 : n <= 512 ? 64 : 0;
  // A workgroup of up to 512 threads holds rows of up to 4096 values with one chunk each, and of up to 8192 with two if
  // nothing is fp32.  With the parameters' sums in LDS 1024 threads hold 8192 values in any type and 768 hold 12288
  // in bf16.  Wider rows are walked (`wide`).
  p.wide = n > (fp32 ? 8192 : 12288);
  p.chunks = p.wide ? 2 : n <= 4096 || (fp32 && n <= 8192) ? 1 : 2;
  p.threads = p.lanes ? 256 : (int)(((per8 + p.chunks - 1) / p.chunks + 63) / 64 * 64);
  // Two workgroups for each of 256 CUs, one where a workgroup fills the registers: more of them write more
  // partial sums and hide nothing that the next row's loads do not.  The number is fixed, not the context's: the
  // workspace's size is asked for without a context, and has to be that of the launch.
  const int64_t most = n > 4096 ? 256 : 512;
  const int64_t per = p.lanes ? 256 / p.lanes : 1;  // units per workgroup
  p.span = std::max<int64_t>(1, (rows + most * per - 1) / (most * per));
  if (rows <= 4) p.span = rows;  // one workgroup, whose sums are the result: no second launch
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
  bool one_gate;
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
  float* part_gate;  // units x n (segs > 0), blocks x n for a single gate row, or null
  float* dgate;      // gates x n (segs == 0), or null
};

// One value's share of a row: bn, x' without the residual (along), xn, dres + r2 d (t) and bscale g (cg).  Without dy
// nothing depends on x': xn is 0 then, and not x' times 0, which an infinity in x' would turn to NaN.
struct NormTerms {
  float bn, along, xn, t, cg;
  NormTerms() = default;
  __device__ __forceinline__ NormTerms(const BwdArgs& a, float ib, float ix, float b, float g, float x, float dy,
                                       float dr, float wp, float wq) {
    bn = b * ib;
    cg = a.bscale * g;
    along = cg * wp * bn;
    xn = a.dy ? fmaf(a.rscale, x, along) * ix : 0.0f;
    t = fmaf(ix, dy * wq, dr);
  }
  // Adds the value's terms to the row's three sums.
  __device__ __forceinline__ void add(float (&sums)[3], float dy, float wq) const {
    sums[0] = fmaf(dy * wq, xn, sums[0]);
    sums[1] = fmaf(along, t, sums[1]);
    sums[2] = fmaf(along, xn, sums[2]);
  }
};
// r2 mean(d xn) and mean(c dx') of a row from its sums.
__device__ __forceinline__ void row_means(const float (&sums)[3], float inv_n, float ix, float& m1, float& m2) {
  m1 = sums[0] * inv_n * ix;
  m2 = (sums[1] - m1 * sums[2]) * inv_n;
}
// The tokens of a unit and its first gate row.
__device__ __forceinline__ void unit_range(const BwdArgs& a, int64_t unit, int64_t& r0, int64_t& r1, int64_t& gidx) {
  const uint32_t u = (uint32_t)unit;  // units fit 32 bits, and 64-bit divisions take long
  if (a.segs) {
    gidx = u / (uint32_t)a.segs;
    r0 = gidx * a.gate_rows + (int64_t)(u % (uint32_t)a.segs) * a.span;
    r1 = std::min<int64_t>(std::min<int64_t>(r0 + a.span, (gidx + 1) * a.gate_rows), a.rows);
  } else {
    r0 = unit * a.span;
    r1 = std::min<int64_t>(r0 + a.span, a.rows);
    gidx = (uint32_t)r0 / (uint32_t)a.gate_rows;  // a unit past the last one walks no rows
  }
}

// Absent inputs take a value that leaves the formula as it is, so that the row's arithmetic has no branches.
// MAXT: most threads.  SUMS_LDS: the parameters' sums are in LDS (each thread's own, two float4 per chunk and sum), for
// rows whose workgroup leaves too few registers to each thread: 2000 x 5120 fp32 98 -> 50 us, 1400 x 8000 fp32 99 -> 62,
// 2100 x 9728 bf16 141 -> 118 (before on the walked rows below); with the sums in registers the rows of up to 4096
// values are as fast and need no LDS pass.
template <typename TB, typename TR, typename TW, int CH, int LANES, int MAXT, bool SUMS_LDS>
__global__ __launch_bounds__(MAXT) void block_norm_bwd_kernel(const BwdArgs a) {
  __shared__ uint32_t red[2][3][RowGroup<LANES>::kMaxWaves];
  constexpr int kPer = LANES > 0 ? 256 / (LANES > 0 ? LANES : 1) : 1;  // units per workgroup
  constexpr int kWidth = 8 * LANES;
  __shared__ float comb[LANES > 0 ? 8 * 256 : 1];
  RowGroup<LANES> grp{red};
  const int lane = LANES > 0 ? threadIdx.x % (LANES > 0 ? LANES : 1) : threadIdx.x;
  const int64_t unit = (int64_t)blockIdx.x * kPer + (LANES > 0 ? threadIdx.x / (LANES > 0 ? LANES : 1) : 0);
  const int n = a.n;
  const RowMap<CH, LANES> map(lane, LANES > 0 ? kWidth : 8 * blockDim.x, n);
  const float inv_n = 1.0f / (float)n;
  // The next row's loads are in flight during a row, where the registers hold both.
  constexpr bool kAhead = !SUMS_LDS || (CH == 1 && MAXT <= 768);
  int64_t r0, r1, gidx;
  unit_range(a, unit, r0, r1, gidx);
  int64_t gend = (gidx + 1) * a.gate_rows;

  Raw8<TW> wp[CH], wq[CH];
  Raw8<TB> b[CH], g[CH], dy[CH];
  Raw8<TR> x[CH], dr[CH];
  Raw8<TR> odx[CH];  // the previous row's results, not yet stored
  Raw8<TB> odb[CH];
  enum { PRE, POST, GATE };
  constexpr int RC = SUMS_LDS ? 1 : CH;
  float held[3][RC][8];
  extern __shared__ __attribute__((aligned(16))) f32x4 sums_lds[];
  auto sum_at = [&](int which, int k, int h) -> f32x4& { return sums_lds[((which * CH + k) * 2 + h) * blockDim.x + threadIdx.x]; };
  auto get_sum = [&](int which, int k, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = SUMS_LDS ? sum_at(which, k, e >> 2)[e & 3] : held[which][SUMS_LDS ? 0 : k][e];
  };
  auto set_sum = [&](int which, int k, const float (&v)[8]) {
    if constexpr (SUMS_LDS) {
      sum_at(which, k, 0) = f32x4{v[0], v[1], v[2], v[3]};
      sum_at(which, k, 1) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) held[which][k][e] = v[e];
    }
  };
  const float zeros[8] = {};
#pragma unroll
  for (int k = 0; k < CH; ++k) {
#pragma unroll
    for (int w = 0; w < 3; ++w) set_sum(w, k, zeros);
    wp[k].fill(1.0f);
    wq[k].fill(1.0f);
    b[k].fill(0.0f);
    g[k].fill(1.0f);
    dy[k].fill(0.0f);
    x[k].fill(0.0f);
    dr[k].fill(0.0f);
    if (a.w_post) map.load(wp[k], (const TW*)a.w_post, k);
    if (a.dy) map.load(wq[k], (const TW*)a.w_pre, k);
  }
  float ib = 1.0f, ix = 0.0f;
  auto load_row = [&](int64_t row, int64_t gate_row) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if (a.branch) map.load(b[k], (const TB*)a.branch + row * a.ldb, k);
      if (a.resid) map.load(x[k], (const TR*)a.resid + row * a.ldr, k);
      if (a.dy) map.load(dy[k], (const TB*)a.dy + row * a.lddy, k);
      if (a.dres) map.load(dr[k], (const TR*)a.dres + row * a.lddo, k);
      if (a.gate) map.load(g[k], (const TB*)a.gate + gate_row * a.ldg, k);
    }
    if (a.w_post) ib = a.stats[2 * row];
    if (a.dy) ix = a.stats[2 * row + 1];
  };
  // A row's results are stored during the next row, before the loads of the one after it: the wait for
  // those loads, which cannot pass older accesses, then waits for no store made late in the same row.
  auto store_row = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if (a.dx) map.store_own((TR*)a.dx + row * a.lddr, k, odx[k]);
      if (a.db) map.store_own((TB*)a.db + row * a.lddb, k, odb[k]);
    }
  };
  if (kAhead && r0 < r1) load_row(r0, gidx);
  for (int64_t row = r0; row < r1; ++row) {
    if (!kAhead) load_row(row, gidx);
    const float jb = ib, jx = ix;
    NormTerms kept[CH][8];
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      map.own(b[k], k);
      map.own(x[k], k);
      map.own(dy[k], k);
      map.own(dr[k], k);
      float pre[8];
      get_sum(PRE, k, pre);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = dy[k].get(e), w = wq[k].get(e);
        const NormTerms m(a, jb, jx, b[k].get(e), g[k].get(e), x[k].get(e), d, dr[k].get(e), wp[k].get(e), w);
        pre[e] = fmaf(d, m.xn, pre[e]);
        m.add(sums, d, w);
        kept[k][e] = m;
      }
      set_sum(PRE, k, pre);
    }
    const int64_t here = gidx;
    if (a.segs == 0 && row + 1 == gend) {
      ++gidx;
      gend += a.gate_rows;
    }
    const bool last = row + 1 == r1;
    if (kAhead && row > r0) store_row(row - 1);
    if (kAhead && !last) load_row(row + 1, gidx);  // in flight during the rest of this row
    grp.template reduce<AddF32>(sums);
    float m1, m2;
    row_means(sums, inv_n, jx, m1, m2);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float dx_f[8], db_f[8], post[8], gate[8];
      get_sum(POST, k, post);
      get_sum(GATE, k, gate);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const NormTerms m = kept[k][e];
        const float w = wp[k].get(e), dxo = fmaf(-m1, m.xn, m.t), du = m.cg * dxo;
        dx_f[e] = a.rscale * dxo;
        post[e] = fmaf(du, m.bn, post[e]);
        gate[e] = fmaf(a.bscale * dxo, w * m.bn, gate[e]);
        db_f[e] = a.w_post ? jb * fmaf(-m2, m.bn, du * w) : du;
      }
      set_sum(POST, k, post);
      set_sum(GATE, k, gate);
      odx[k].round(dx_f);
      odb[k].round(db_f);
    }
    if (!kAhead) store_row(row);
    if (a.dgate && (last || gidx != here)) {  // a gate row's last token
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float gate[8];
        get_sum(GATE, k, gate);
        map.store_own(a.dgate + here * n, k, gate);
        set_sum(GATE, k, zeros);
      }
    }
  }
  if (kAhead && r0 < r1) store_row(r1 - 1);
  auto write_sum = [&](int which, float* part) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float v[8];
      get_sum(which, k, v);
      map.store_own(part, k, v);
    }
  };
  if (a.part_gate && !(LANES > 0 && a.one_gate) && unit < a.units) write_sum(GATE, a.part_gate + unit * n);
  if constexpr (LANES > 0) {
    // the workgroup's units, added in order; a unit past the last one holds zeros
    auto combine = [&](int which, float* part) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (map.keep[0] >> e & 1) comb[threadIdx.x / LANES * kWidth + map.col[0] + e] = held[which][0][e];
      __syncthreads();
      for (int c = threadIdx.x; c < n; c += 256) {
        float sum = 0.0f;
        for (int u = 0; u < kPer; ++u) sum += comb[u * kWidth + c];
        part[(int64_t)blockIdx.x * n + c] = sum;
      }
    };
    if (a.part_pre) combine(PRE, a.part_pre);
    if (a.part_post) combine(POST, a.part_post);
    if (a.part_gate && a.one_gate) combine(GATE, a.part_gate);
  } else {
    if (a.part_pre) write_sum(PRE, a.part_pre + (int64_t)blockIdx.x * n);
    if (a.part_post) write_sum(POST, a.part_post + (int64_t)blockIdx.x * n);
  }
}

// Rows too wide for a workgroup's registers: the row is walked in chunks of eight columns per thread twice, once for
// its three sums and once, read again from the caches, for the results; the parameters' sums stay in the
// unit's own partials (read and written by the thread that owns the columns), which the caches hold too.  1100 x
// 9728 fp32 (257 MB) take 113 us, 2.3 TB/s: the second read and the partials' traffic come on top of the row's own bytes.
template <typename TB, typename TR, typename TW>
__global__ __launch_bounds__(1024) void block_norm_bwd_wide_kernel(const BwdArgs a) {
  __shared__ uint32_t red[2][3][RowGroup<0>::kMaxWaves];
  RowGroup<0> grp{red};
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  const int64_t unit = blockIdx.x;
  int64_t r0, r1, gidx;
  unit_range(a, unit, r0, r1, gidx);
  int64_t gend = (gidx + 1) * a.gate_rows;
  float* const post = a.part_post ? a.part_post + unit * n : nullptr;
  float* const pre = a.part_pre ? a.part_pre + unit * n : nullptr;
  const float zeros[8] = {};

  Raw8<TW> wp, wq;
  Raw8<TB> b, g, dy;
  Raw8<TR> x, dr;
  wp.fill(1.0f);
  wq.fill(1.0f);
  b.fill(0.0f);
  g.fill(1.0f);
  dy.fill(0.0f);
  x.fill(0.0f);
  dr.fill(0.0f);
  // adds v to the columns' running sums, which start at the first token
  auto accumulate = [&](const RowMap<1, 0>& map, float* sum, bool first, const float (&v)[8]) {
    float out[8];
    Raw8<float> old;
    if (!first) map.load(old, sum, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = first ? v[e] : old.get(e) + v[e];
    map.store_own(sum, 0, out);
  };
  for (int64_t row = r0; row < r1; ++row) {
    const float ib = a.w_post ? a.stats[2 * row] : 1.0f, ix = a.dy ? a.stats[2 * row + 1] : 0.0f;
    auto load_chunk = [&](const RowMap<1, 0>& map) {
      if (a.w_post) map.load(wp, (const TW*)a.w_post, 0);
      if (a.dy) map.load(wq, (const TW*)a.w_pre, 0);
      if (a.branch) map.load(b, (const TB*)a.branch + row * a.ldb, 0);
      if (a.resid) map.load(x, (const TR*)a.resid + row * a.ldr, 0);
      if (a.dy) map.load(dy, (const TB*)a.dy + row * a.lddy, 0);
      if (a.dres) map.load(dr, (const TR*)a.dres + row * a.lddo, 0);
      if (a.gate) map.load(g, (const TB*)a.gate + gidx * a.ldg, 0);
      map.own(b, 0);
      map.own(x, 0);
      map.own(dy, 0);
      map.own(dr, 0);
    };
    float sums[3] = {0.0f, 0.0f, 0.0f};
    for (int c = 0; c < n; c += 8 * blockDim.x) {
      const RowMap<1, 0> map(threadIdx.x + c / 8, 0, n);
      load_chunk(map);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = dy.get(e), w = wq.get(e);
        NormTerms(a, ib, ix, b.get(e), g.get(e), x.get(e), d, dr.get(e), wp.get(e), w).add(sums, d, w);
      }
    }
    grp.template reduce<AddF32>(sums);
    float m1, m2;
    row_means(sums, inv_n, ix, m1, m2);
    const bool gate_first = row == r0 || row + a.gate_rows == gend;
    for (int c = 0; c < n; c += 8 * blockDim.x) {
      const RowMap<1, 0> map(threadIdx.x + c / 8, 0, n);
      load_chunk(map);
      float dx_f[8], db_f[8], v_pre[8], v_post[8], v_gate[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = dy.get(e), w = wp.get(e);
        const NormTerms m(a, ib, ix, b.get(e), g.get(e), x.get(e), d, dr.get(e), w, wq.get(e));
        const float dxo = fmaf(-m1, m.xn, m.t), du = m.cg * dxo;
        dx_f[e] = a.rscale * dxo;
        v_pre[e] = d * m.xn;
        v_post[e] = du * m.bn;
        v_gate[e] = a.bscale * dxo * (w * m.bn);
        db_f[e] = a.w_post ? ib * fmaf(-m2, m.bn, du * w) : du;
      }
      if (a.dx) map.store_own((TR*)a.dx + row * a.lddr, 0, dx_f);
      if (a.db) map.store_own((TB*)a.db + row * a.lddb, 0, db_f);
      if (pre) accumulate(map, pre, row == r0, v_pre);
      if (post) accumulate(map, post, row == r0, v_post);
      if (a.dgate) accumulate(map, a.dgate + gidx * n, gate_first, v_gate);
      if (a.part_gate) accumulate(map, a.part_gate + unit * n, row == r0, v_gate);
    }
    if (a.segs == 0 && row + 1 == gend) {
      ++gidx;
      gend += a.gate_rows;
    }
  }
  if (r0 >= r1)  // no tokens: its partials are zero
    for (int c = 0; c < n; c += 8 * blockDim.x) {
      const RowMap<1, 0> map(threadIdx.x + c / 8, 0, n);
      if (pre) map.store_own(pre, 0, zeros);
      if (post) map.store_own(post, 0, zeros);
      if (a.part_gate) map.store_own(a.part_gate + unit * n, 0, zeros);
    }
}

// Up to three sums over partials in one launch: out[g][c] = sum over p < count of part[g * count + p][c], p in
// order within SHARES strided shares, the shares in order.  blockIdx.x: COLS columns; blockIdx.y: output row, the
// sums' rows one after the other.
struct ColumnSums {
  struct One {
    const float* part;
    float* out;
    int64_t count, groups;
  } s[3];
  int n;
};
template <int COLS, int SHARES>
__global__ __launch_bounds__(COLS* SHARES) void column_sum_kernel(const ColumnSums a) {
  __shared__ float red[SHARES][COLS + 1];
  const int cx = threadIdx.x % COLS, sh = threadIdx.x / COLS, c = blockIdx.x * COLS + cx, n = a.n;
  for (int64_t row = blockIdx.y;; row += gridDim.y) {
    int64_t g = row;
    int k = 0;
    while (k < 3 && g >= a.s[k].groups) g -= a.s[k++].groups;
    if (k == 3) return;
    const int64_t count = a.s[k].count;
    float s = 0.0f;
    if (c < n) {
      const float* p = a.s[k].part + g * count * n + c;
      for (int64_t i = sh; i < count; i += 8 * SHARES) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = i + u * SHARES < count ? p[(i + u * SHARES) * n] : 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
      }
    }
    if constexpr (SHARES > 1) {
      red[sh][cx] = s;
      __syncthreads();
      for (int half = SHARES / 2; half > 0; half >>= 1) {
        if (sh < half) red[sh][cx] += red[sh + half][cx];
        __syncthreads();
      }
      s = red[0][cx];
      __syncthreads();
    }
    if (sh == 0 && c < n) a.s[k].out[g * n + c] = s;
  }
}

}  // namespace wr

using namespace wr;

template <int N>
using Int = std::integral_constant<int, N>;

static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

size_t wr_norm_bwd_ws_bytes(int64_t rows, int64_t n, int64_t gate_rows) {
  if (rows <= 0) return 256;
  size_t most = 0;  // the larger of what the types need
  for (const bool fp32 : {false, true}) {
    const BwdPlan p = bwd_plan(rows, n, gate_rows, fp32);
    most = std::max(most, 2 * round256((size_t)p.blocks * n * 4) + (p.segs ? round256((size_t)p.units * n * 4) : 0));
  }
  return most;
}

template <typename TB, typename TR, typename TW>
static int bwd_launch(wr_ctx* ctx, const BwdPlan& p, const BwdArgs& a) {
  auto go = [&](auto ch, auto lanes, auto most, auto in_lds) {
    constexpr int kCh = decltype(ch)::value;
    constexpr bool kLds = decltype(in_lds)::value;
    auto* kernel = block_norm_bwd_kernel<TB, TR, TW, kCh, decltype(lanes)::value, decltype(most)::value, kLds>;
    const int lds = kLds ? 3 * kCh * 32 * p.threads : 0;
    if (kLds && !lds_limit((const void*)kernel, 3 * kCh * 32 * decltype(most)::value)) return WR_EHIP;
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks), dim3(p.threads), lds, ctx->stream, a);
    return WR_OK;
  };
  const std::false_type regs;
  const std::true_type in_lds;
  constexpr bool kHalf = sizeof(TB) + sizeof(TR) == 4;
  if (p.lanes == 8) return go(Int<1>{}, Int<8>{}, Int<256>{}, regs);
  if (p.lanes == 16) return go(Int<1>{}, Int<16>{}, Int<256>{}, regs);
  if (p.lanes == 32) return go(Int<1>{}, Int<32>{}, Int<256>{}, regs);
  if (p.lanes == 64) return go(Int<1>{}, Int<64>{}, Int<256>{}, regs);
  if (p.wide) {
    hipLaunchKernelGGL((block_norm_bwd_wide_kernel<TB, TR, TW>), dim3((unsigned)p.blocks), dim3(p.threads), 0, ctx->stream, a);
    return WR_OK;
  }
  if (a.n <= 4096) return go(Int<1>{}, Int<0>{}, Int<512>{}, regs);
  if constexpr (kHalf) {
    if (a.n <= 8192) return go(Int<2>{}, Int<0>{}, Int<512>{}, regs);
    return go(Int<2>{}, Int<0>{}, Int<768>{}, in_lds);
  } else {
    if (a.n <= 6144) return go(Int<1>{}, Int<0>{}, Int<768>{}, in_lds);
    return go(Int<1>{}, Int<0>{}, Int<1024>{}, in_lds);
  }
}

int wr_block_norm_backward_impl(wr_ctx* ctx, int64_t rows, int64_t n, const void* branch, int b_dtype, int64_t ldb,
                                const void* w_post, const void* gate, int64_t ldg, int64_t gate_rows,
                                float branch_scale, const void* resid, int r_dtype, int64_t ldr, float resid_scale,
                                const void* w_pre, int w_dtype, const float* stats, const void* dy, int64_t lddy,
                                const void* dresid_out, int64_t lddo, void* dbranch, int64_t lddb, void* dresid,
                                int64_t lddr, float* dw_post, float* dgate, float* dw_pre) {
  auto add_up = [&](const ColumnSums& c, auto cols, auto shares) {
    const int64_t outs = c.s[0].groups + c.s[1].groups + c.s[2].groups;
    if (outs == 0) return;
    constexpr int kCols = decltype(cols)::value, kShares = decltype(shares)::value;
    const dim3 grid((unsigned)((n + kCols - 1) / kCols), (unsigned)std::min<int64_t>(outs, 65535));
    hipLaunchKernelGGL((column_sum_kernel<kCols, kShares>), grid, dim3(kCols * kShares), 0, ctx->stream, c);
  };
  if (rows == 0) {  // sums over no tokens
    add_up({{{nullptr, dw_post, 0, dw_post ? 1 : 0}, {nullptr, dw_pre, 0, dw_pre ? 1 : 0},
             {nullptr, dgate, 0, dgate && gate_rows == 0 ? 1 : 0}}, (int)n}, Int<256>{}, Int<1>{});
    WR_CHECK_LAUNCH();
    return WR_OK;
  }
  if (ctx->ws_bytes < wr_norm_bwd_ws_bytes(rows, n, gate_rows) || !ctx->ws) return WR_EWORKSPACE;
  const BwdPlan p = bwd_plan(rows, n, gate_rows, b_dtype == WR_F32 || r_dtype == WR_F32);
  char* ws = (char*)ctx->ws;
  const size_t part = round256((size_t)p.blocks * n * 4);
  BwdArgs a{};
  a.rows = (int)rows;
  a.n = (int)n;
  a.span = (int)p.span;
  a.segs = (int)p.segs;
  a.gate_rows = (int)p.gate_rows;
  a.one_gate = p.gates == 1;
  a.units = p.units;
  a.branch = branch;
  a.ldb = ldb;
  a.w_post = w_post;
  a.gate = gate;
  a.ldg = ldg;
  a.bscale = branch_scale;
  a.resid = dy ? resid : nullptr;  // read for xn alone
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
  if (p.blocks == 1) {
    a.part_post = dw_post;
    a.part_pre = dw_pre;
  }
  a.part_gate = dgate && p.segs ? (float*)(ws + 2 * part) : nullptr;
  a.dgate = p.segs ? nullptr : dgate;
  if (p.blocks == 1 && a.one_gate && a.part_gate) a.part_gate = dgate;
  const int key = (b_dtype == WR_BF16 ? 4 : 0) + (r_dtype == WR_BF16 ? 2 : 0) + (w_dtype == WR_BF16 ? 1 : 0);
  int rc;
  switch (key) {
    case 0: rc = bwd_launch<float, float, float>(ctx, p, a); break;
    case 1: rc = bwd_launch<float, float, uint16_t>(ctx, p, a); break;
    case 2: rc = bwd_launch<float, uint16_t, float>(ctx, p, a); break;
    case 3: rc = bwd_launch<float, uint16_t, uint16_t>(ctx, p, a); break;
    case 4: rc = bwd_launch<uint16_t, float, float>(ctx, p, a); break;
    case 5: rc = bwd_launch<uint16_t, float, uint16_t>(ctx, p, a); break;
    case 6: rc = bwd_launch<uint16_t, uint16_t, float>(ctx, p, a); break;
    default: rc = bwd_launch<uint16_t, uint16_t, uint16_t>(ctx, p, a); break;
  }
  if (rc != WR_OK) return rc;
  WR_CHECK_LAUNCH();
  // Many short sums (gate rows of a few units) take a thread for each column; the others share a column's
  // partials among threads, with narrower workgroups where there are few columns.
  const ColumnSums::One none{nullptr, nullptr, 0, 0};
  const int64_t shares = p.gates == 1 ? p.blocks : p.segs;
  const ColumnSums::One gates{a.part_gate, dgate, shares, a.part_gate && a.part_gate != dgate ? p.gates : 0};
  const bool sum = p.blocks > 1;
  const bool apart = shares <= 32;
  if (apart) add_up({{gates, none, none}, (int)n}, Int<256>{}, Int<1>{});
  const ColumnSums sums{{{a.part_post, dw_post, p.blocks, sum && dw_post ? 1 : 0}, {a.part_pre, dw_pre, p.blocks, sum && dw_pre ? 1 : 0},
                         apart ? none : gates}, (int)n};
  if (n >= 1024) add_up(sums, Int<32>{}, Int<32>{});
  else add_up(sums, Int<8>{}, Int<128>{});
  WR_CHECK_LAUNCH();
  return WR_OK;
}
