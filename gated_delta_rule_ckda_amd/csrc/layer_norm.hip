// Layer norm of rows of d elements, with the residual add before it:
//
//   h = r + x                         (x itself without r)
//   n = (h - mean h) rstd w + b       rstd = 1 / sqrt(mean (h - mean h)^2 + eps)
//
// n is formed from h before its rounding.  The row is centred twice: a mean far
// above the spread is off by several 2^-24 of itself, which the centred row would keep
// as a shift (a row of 77777.7 gave n = 0.9).  What the centred row's own mean is,
// summed beside its squares, is taken out of both, so such a mean costs no
// digits, and no further round of sums (gradients of 32768 rows of 2048: 110 us
// before, 112 now).  Backwards, with c = (h - mean h) rstd and m = dn w,
//
//   dw = sum_rows dn c,  db = sum_rows dn
//   dx = dh + rstd (m - mean m - c mean(m c))
//
// Bound by HBM: every activation is read and written once.  TPR threads hold a
// row, EPL elements each, weights and sums over rows in registers; workgroups walk
// over rows and load a row ahead.  Rows of odd widths move an element at a time:
// with the row ahead that is faster in bf16 than wide accesses at odd addresses
// (32768 rows with a residual, of 2001 in bf16: 119 us against 148; of 1001 in float32:
// 105 and 101).  Measured, 32768 rows of 2048 with a residual: bf16 99 us (5.4
// TB/s), gradients 112 (4.8); float32 195 (5.5), gradients 206 (5.2).  524288 rows of
// 128 in bf16: 60 us (4.5).  Gradients past 8192 elements have 128 registers a thread
// and keep 96 bytes a lane in scratch in float32, 208 at odd widths of either type
// (4096 rows of 16384 with a residual: bf16 136 us, float32 251; of 16383: 361
// and 418); odd widths from 4097 to 8192 run one wave a SIMD.
#include "row_ops.h"

namespace ckda {
namespace {

// The mean square about the mean, from a mean square and what is left of the mean:
// a row of one value may leave less than nothing.  NaN stays.
__device__ __forceinline__ float centred_square(float square, float left) {
  const float v = __builtin_fmaf(-left, left, square);
  return v < 0.f ? 0.f : v;
}

template <class IO, bool ALIGNED, int EPL, int NT>
__global__ __launch_bounds__(NT) void layer_norm_kernel(LayerNormArgs a, int tpr) {
  constexpr int VEC = ALIGNED ? 16 / sizeof(typename IO::storage) : 1, K = EPL / VEC;
  constexpr bool kAhead = NT == 256;  // more threads leave no registers for it
  using X = Chans<IO, VEC, ALIGNED>;
  __shared__ float red[4 * (NT / 64)];
  int half = 0;
  const int t = threadIdx.x, lane = t & (tpr - 1);
  const int rpb = NT / tpr;  // rows a workgroup and step
  float w[EPL], b[EPL];
  bool ok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + tpr * k) * VEC;
    ok[k] = c < a.d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[k * VEC + e] = a.w && c + e < a.d ? a.w[c + e] : 1.f;
      b[k * VEC + e] = a.b && c + e < a.d ? a.b[c + e] : 0.f;
    }
  }
  // whether an element is one of the row's
  const auto in = [&](int k, int e) { return ALIGNED ? ok[k] : (lane + tpr * k) * VEC + e < a.d; };
  const float inv_d = 1.f / a.d;
  typename X::V nx[K], nr[K];
  const auto load = [&](int64_t r0) {
    const int64_t row = r0 + t / tpr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = row * a.d + (lane + tpr * k) * VEC;
      nx[k] = typename X::V{};
      nr[k] = nx[k];
      if (row < a.rows && ok[k]) {
        nx[k] = X::load(a.x, i, a.d - (lane + tpr * k) * VEC);
        if (a.r) nr[k] = X::load(a.r, i, a.d - (lane + tpr * k) * VEC);
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
  if (kAhead) load(static_cast<int64_t>(blockIdx.x) * rpb);
  // every thread of a workgroup takes the same number of steps (barriers)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + t / tpr;
    const bool live = row < a.rows;
    if (!kAhead) load(r0);
    typename X::V vx[K], vr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      vx[k] = nx[k];
      vr[k] = nr[k];
    }
    if (kAhead) load(r0 + step);  // a row ahead, while this one's sums go around
    float h[EPL], s1[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        h[j] = X::get(vx[k], e) + (a.r ? X::get(vr[k], e) : 0.f);
        s1[0] += h[j];
      }
    if (a.h && live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(a.h, row * a.d + (lane + tpr * k) * VEC, a.d - (lane + tpr * k) * VEC, h + k * VEC);
    }
    row_sum<1, NT>(s1, tpr, red, half);
    const float mean = s1[0] * inv_d;
    float s[2] = {0.f, 0.f};  // of (h - mean)^2 and h - mean
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        h[j] = in(k, e) ? h[j] - mean : 0.f;
        s[0] += h[j] * h[j];
        s[1] += h[j];
      }
    row_sum<2, NT>(s, tpr, red, half);
    const float left = s[1] * inv_d;
    const float rstd = 1.f / sqrtf(centred_square(s[0] * inv_d, left) + a.eps);
#pragma unroll
    for (int j = 0; j < EPL; ++j) h[j] = __builtin_fmaf(h[j], rstd, -left * rstd) * w[j] + b[j];
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(a.n, row * a.d + (lane + tpr * k) * VEC, a.d - (lane + tpr * k) * VEC, h + k * VEC);
    }
  }
}

// Gradients; each workgroup leaves its rows' sums for dw and db in
// part[workgroup][2][d].
template <class IO, bool ALIGNED, int EPL, int NT>
__global__ __launch_bounds__(NT) void layer_norm_bwd_kernel(LayerNormArgs a, LayerNormGrads g, int tpr) {
  constexpr int VEC = ALIGNED ? 16 / sizeof(typename IO::storage) : 1, K = EPL / VEC;
  constexpr bool kAhead = NT == 256;  // more threads leave no registers for it
  using X = Chans<IO, VEC, ALIGNED>;
  __shared__ float red[2 * 4 * (NT / 64)];
  extern __shared__ float cols[];  // [rows a step][d] for rows of less than a workgroup
  int half = 0;
  const int t = threadIdx.x, lane = t & (tpr - 1);
  const int rpb = NT / tpr;
  float w[EPL], dw[EPL], db[EPL];
  bool ok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + tpr * k) * VEC;
    ok[k] = c < a.d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[k * VEC + e] = c + e < a.d ? (a.w ? a.w[c + e] : 1.f) : 0.f;
      dw[k * VEC + e] = db[k * VEC + e] = 0.f;
    }
  }
  // whether an element is one of the row's
  const auto in = [&](int k, int e) { return ALIGNED ? ok[k] : (lane + tpr * k) * VEC + e < a.d; };
  const float inv_d = 1.f / a.d;
  typename X::V nx[K], nn[K], nh[K];
  const auto load = [&](int64_t r0) {
    const int64_t row = r0 + t / tpr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = row * a.d + (lane + tpr * k) * VEC;
      nx[k] = typename X::V{};
      nn[k] = nh[k] = nx[k];
      if (row < a.rows && ok[k]) {
        nx[k] = X::load(a.x, i, a.d - (lane + tpr * k) * VEC);
        nn[k] = X::load(g.dn, i, a.d - (lane + tpr * k) * VEC);
        if (g.dh) nh[k] = X::load(g.dh, i, a.d - (lane + tpr * k) * VEC);
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
  if (kAhead) load(static_cast<int64_t>(blockIdx.x) * rpb);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + t / tpr;
    const bool live = row < a.rows;
    if (!kAhead) load(r0);
    typename X::V vx[K], vn[K], vh[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      vx[k] = nx[k];
      vn[k] = nn[k];
      vh[k] = nh[k];
    }
    if (kAhead) load(r0 + step);
    float h[EPL], s1[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[k * VEC + e] = X::get(vx[k], e);
        s1[0] += h[k * VEC + e];
      }
    row_sum<1, NT, 4>(s1, tpr, red, half);
    const float mean = s1[0] * inv_d;
    float s[4] = {0.f, 0.f, 0.f, 0.f};  // of (h - mean)^2, m, m (h - mean), h - mean
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        h[j] = in(k, e) ? h[j] - mean : 0.f;
        const float m = X::get(vn[k], e) * w[j];
        s[0] += h[j] * h[j];
        s[1] += m;
        s[2] += m * h[j];
        s[3] += h[j];
      }
    row_sum<4, NT, 4>(s, tpr, red, half);
    const float left = s[3] * inv_d, mm = s[1] * inv_d;
    // with eps = 0 a thread without a row would add inf * 0 to its sums over rows
    const float rstd = live ? 1.f / sqrtf(centred_square(s[0] * inv_d, left) + a.eps) : 0.f;
    const float mc = (s[2] * inv_d - left * mm) * rstd;
    float dx[EPL];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        const float c = __builtin_fmaf(h[j], rstd, -left * rstd), dn = X::get(vn[k], e);
        dw[j] += dn * c;
        db[j] += dn;
        dx[j] = rstd * (dn * w[j] - mm - c * mc);
        if (g.dh) dx[j] += X::get(vh[k], e);
      }
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(g.dx, row * a.d + (lane + tpr * k) * VEC, a.d - (lane + tpr * k) * VEC, dx + k * VEC);
    }
  }
  // sums over the rows of this workgroup, row groups in order
  float* out = g.part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (!(q == 0 ? g.dw : g.db)) continue;
    const float* sum = q == 0 ? dw : db;
    if (rpb == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k])
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (in(k, e)) out[q * a.d + (lane + tpr * k) * VEC + e] = sum[k * VEC + e];
    } else {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k])
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (in(k, e)) cols[(t / tpr) * a.d + (lane + tpr * k) * VEC + e] = sum[k * VEC + e];
      __syncthreads();
      for (int c = t; c < a.d; c += NT) {
        float v = 0.f;
        for (int j = 0; j < rpb; ++j) v += cols[j * a.d + c];
        out[q * a.d + c] = v;
      }
    }
  }
}

// out[c] = sum over workgroups of part[.][q][c]: 32 columns a workgroup, its
// 32 groups of lanes taking every 32nd workgroup's; their sums are added in order.
__global__ __launch_bounds__(1024) void layer_norm_cols_kernel(const float* part, int parts, int d, float* dw,
                                                               float* db) {
  __shared__ float red[32][33];
  const int q = blockIdx.y, l = threadIdx.x & 31, c = blockIdx.x * 32 + l, grp = threadIdx.x >> 5;
  float* out = q == 0 ? dw : db;
  if (!out) return;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int p = grp; p < parts; p += 32) v += part[(static_cast<int64_t>(p) * 2 + q) * d + c];
  }
  red[grp][l] = v;
  __syncthreads();
  if (grp == 0 && c < d) {
    for (int i = 1; i < 32; ++i) v += red[i][l];
    out[c] = v;
  }
}

// How rows of d elements are held: EPL elements a thread, TPR threads.
struct Shape {
  int epl, tpr, nt;
};
Shape shape_of(int d) {
  Shape s;
  s.nt = d > 8192 ? 1024 : 256;
  s.epl = d <= 2048 ? 8 : (d <= 4096 || d > 8192 ? 16 : 32);
  s.tpr = 4;
  while (s.tpr * s.epl < d) s.tpr *= 2;
  return s;
}

int64_t grid_of(int64_t rows, const Shape& s, int64_t most) {
  const int64_t steps = (rows + s.nt / s.tpr - 1) / (s.nt / s.tpr);
  return steps < most ? steps : most;
}

// Workgroups: as many as the 256 CUs hold at once, each walking over rows.  Rows
// within a wave need no barrier, and twice as many keep more loads in flight
// (524288 rows of 128 in bf16: 59 us with 2048, 65 with 1024; 32768 rows of 2048
// with a residual: 112 with 2048, 99 with 1024).
int64_t fwd_groups(const Shape& s) { return s.tpr <= 64 ? 2048 : 1024; }
int64_t bwd_groups(const Shape& s) { return s.nt == 1024 ? 256 : (s.epl == 8 ? 1024 : 512); }

template <class IO, bool ALIGNED, int EPL, int NT>
launch_result launch_one(const LayerNormArgs& a, const LayerNormGrads* g, const Shape& s, hipStream_t st) {
  if (!g) {
    hipLaunchKernelGGL((layer_norm_kernel<IO, ALIGNED, EPL, NT>),
                       dim3(static_cast<unsigned>(grid_of(a.rows, s, fwd_groups(s)))), dim3(NT), 0, st, a, s.tpr);
    return hipGetLastError();
  }
  const int64_t grid = grid_of(a.rows, s, bwd_groups(s));
  const int rpb = NT / s.tpr;
  const size_t lds = rpb > 1 ? static_cast<size_t>(rpb) * a.d * 4 : 0;
  hipLaunchKernelGGL((layer_norm_bwd_kernel<IO, ALIGNED, EPL, NT>), dim3(static_cast<unsigned>(grid)), dim3(NT), lds,
                     st, a, *g, s.tpr);
  const launch_result e = hipGetLastError();
  if (e != hipSuccess || (!g->dw && !g->db)) return e;
  hipLaunchKernelGGL(layer_norm_cols_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, st, g->part,
                     static_cast<int>(grid), a.d, g->dw, g->db);
  return hipGetLastError();
}

template <class IO, bool ALIGNED>
launch_result launch_shape(const LayerNormArgs& a, const LayerNormGrads* g, const Shape& s, hipStream_t st) {
  if (s.nt == 1024) return launch_one<IO, ALIGNED, 16, 1024>(a, g, s, st);
  if (s.epl == 8) return launch_one<IO, ALIGNED, 8, 256>(a, g, s, st);
  if (s.epl == 16) return launch_one<IO, ALIGNED, 16, 256>(a, g, s, st);
  return launch_one<IO, ALIGNED, 32, 256>(a, g, s, st);
}

template <class IO>
launch_result launch_io(const LayerNormArgs& a, const LayerNormGrads* g, hipStream_t st) {
  const Shape s = shape_of(a.d);
  if (a.d % (16 / sizeof(typename IO::storage)) == 0) return launch_shape<IO, true>(a, g, s, st);
  return launch_shape<IO, false>(a, g, s, st);
}

launch_result launch(const LayerNormArgs& a, const LayerNormGrads* g, int32_t io_dtype, hipStream_t st) {
  return io_dtype == CKDA_DTYPE_BF16 ? launch_io<io_bf16>(a, g, st) : launch_io<io_f32>(a, g, st);
}

}  // namespace

size_t layer_norm_bwd_workspace(int64_t rows, int32_t d) {
  const Shape s = shape_of(d);
  return static_cast<size_t>(grid_of(rows, s, bwd_groups(s))) * 2 * d * 4;
}

launch_result launch_layer_norm(const LayerNormArgs& a, int32_t io_dtype, hipStream_t s) {
  return launch(a, nullptr, io_dtype, s);
}

launch_result launch_layer_norm_bwd(const LayerNormArgs& a, LayerNormGrads g, int32_t io_dtype, void* ws,
                                    hipStream_t s) {
  g.part = static_cast<float*>(ws);
  return launch(a, &g, io_dtype, s);
}

}  // namespace ckda
