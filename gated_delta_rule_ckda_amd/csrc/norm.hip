// The norms around a block, fused with its gate and residual scale.  A row at
// a time, in float32:
//
//   u = y rsqrt(mean y^2 + eps) w      (y itself without w)
//   v = u act(g)                       (u without g)
//   h = x + s v                        (s v without x, s = 1 without s)
//   n = h rsqrt(mean h^2 + eps) w2     (not written without w2)
//
// n is formed from h before its rounding.  Backwards, given dh and dn,
//
//   dw2 = sum_rows dn h~,  c = dn w2,  D = dh + r2 (c - h~ mean(c h~)),  h~ = h r2
//   dx = D,  ds = sum_rows D v,  dv = s D
//   dg = dv u act'(g),  du = dv act(g)
//   dw = sum_rows du y~,  c = du w,  dy = r1 (c - y~ mean(c y~)),        y~ = y r1
//
// Both are bound by HBM: every activation is read once and written once, and
// everything between stays in registers.  TPR threads hold a row, EPL elements
// each in vectors of VEC; a workgroup keeps its columns' weights in registers
// and walks over rows, so weights are read once a workgroup and the sums over
// rows are a thread's own until its last row.  8 elements a thread keep three
// workgroups of gradients a CU (146 registers); more only where a row is too
// long for 256 threads.  Measured in bf16: 524288 rows of 128 with a gate 72 us
// (5.6 TB/s), gradients of 32768 rows of 2048 with all parts 206 us (5.2 TB/s;
// a copy of 2 GB runs at 5.0).
#include "row_ops.h"

namespace ckda {
namespace {

enum { kActNone = 0, kActSigmoid = 1, kActSilu = 2 };

template <class IO, int VEC, int EPL, int NT>
__global__ __launch_bounds__(NT) void norm_fwd_kernel(NormArgs a, int tpr) {
  constexpr int K = EPL / VEC;
  using X = Vec<IO, VEC>;
  __shared__ float red[4 * (NT / 64)];
  int half = 0;
  const int t = threadIdx.x, lane = t & (tpr - 1);
  const int rpb = NT / tpr;  // rows a workgroup and step
  float w[EPL], s[EPL], w2[EPL];
  bool ok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + tpr * k) * VEC;
    ok[k] = c < a.d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[k * VEC + e] = a.w && ok[k] ? a.w[c + e] : 1.f;
      s[k * VEC + e] = a.s && ok[k] ? a.s[c + e] : 1.f;
      w2[k * VEC + e] = a.w2 && ok[k] ? a.w2[c + e] : 1.f;
    }
  }
  const float inv_d = 1.f / a.d;
  // every thread of a workgroup takes the same number of steps (barriers)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t row = r0 + t / tpr;
    const bool live = row < a.rows;
    typename X::V vy[K], vg[K], vx[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = row * a.d + (lane + tpr * k) * VEC;
      vy[k] = typename X::V{};
      vg[k] = vx[k] = vy[k];
      if (live && ok[k]) {
        vy[k] = X::load(a.y, i);
        if (a.g) vg[k] = X::load(a.g, i);
        if (a.x) vx[k] = X::load(a.x, i);
      }
    }
    float h[EPL];
    float ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[k * VEC + e] = X::get(vy[k], e);
        ss[0] += h[k * VEC + e] * h[k * VEC + e];
      }
    float r1 = 1.f;
    if (a.w) {
      row_sum<1, NT>(ss, tpr, red, half);
      r1 = 1.f / sqrtf(ss[0] * inv_d + a.eps);
    }
    ss[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        float u = h[j] * r1 * w[j];
        if (a.g) {
          const float g = X::get(vg[k], e), p = sigmoid_of<IO>(g);
          u *= a.act == kActSilu ? (p == 0.f ? 0.f : g * p) : p;
        }
        u *= s[j];
        h[j] = a.x ? X::get(vx[k], e) + u : u;
        if (!ok[k]) h[j] = 0.f;
        ss[0] += h[j] * h[j];
      }
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(a.h, row * a.d + (lane + tpr * k) * VEC, h + k * VEC);
    }
    if (a.w2) {
      row_sum<1, NT>(ss, tpr, red, half);
      const float r2 = 1.f / sqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < EPL; ++j) h[j] = h[j] * r2 * w2[j];
      if (live) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (ok[k]) X::store(a.n, row * a.d + (lane + tpr * k) * VEC, h + k * VEC);
      }
    }
  }
}

// Gradients; each workgroup leaves its rows' sums for dw, ds, dw2 in
// part[workgroup][3][d].
template <class IO, int VEC, int EPL, int NT>
__global__ __launch_bounds__(NT, (EPL == 8 ? 3 : 1)) void norm_bwd_kernel(NormArgs a, NormGrads g, int tpr) {
  constexpr int K = EPL / VEC;
  using X = Vec<IO, VEC>;
  __shared__ float red[4 * (NT / 64)];
  extern __shared__ float cols[];  // [rows a step][d] for rows of less than a workgroup
  int half = 0;
  const int t = threadIdx.x, lane = t & (tpr - 1);
  const int rpb = NT / tpr;
  float w[EPL], s[EPL], w2[EPL], dw[EPL], ds[EPL], dw2[EPL];
  bool ok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + tpr * k) * VEC;
    ok[k] = c < a.d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int j = k * VEC + e;
      w[j] = a.w && ok[k] ? a.w[c + e] : 1.f;
      s[j] = a.s && ok[k] ? a.s[c + e] : 1.f;
      w2[j] = a.w2 && ok[k] ? a.w2[c + e] : 0.f;
      dw[j] = ds[j] = dw2[j] = 0.f;
    }
  }
  const float inv_d = 1.f / a.d;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t row = r0 + t / tpr;
    const bool live = row < a.rows;
    typename X::V vy[K], vg[K], vx[K], vh[K], vn[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = row * a.d + (lane + tpr * k) * VEC;
      vy[k] = typename X::V{};
      vg[k] = vx[k] = vh[k] = vn[k] = vy[k];
      if (live && ok[k]) {
        vy[k] = X::load(a.y, i);
        vh[k] = X::load(g.dh, i);
        if (a.g) vg[k] = X::load(a.g, i);
        if (a.w2) {
          if (a.x) vx[k] = X::load(a.x, i);
          vn[k] = X::load(g.dn, i);
        }
      }
    }
    float r1 = 1.f;
    if (a.w) {
      float ss[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] += X::get(vy[k], e) * X::get(vy[k], e);
      row_sum<1, NT>(ss, tpr, red, half);
      // with eps = 0 a thread without a row would add inf * 0 to its sums over rows
      r1 = live ? 1.f / sqrtf(ss[0] * inv_d + a.eps) : 0.f;
    }
    float D[EPL], act[EPL], dact[EPL];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        D[j] = X::get(vh[k], e);
        act[j] = 1.f;
        dact[j] = 0.f;
        if (a.g) {
          const float gg = X::get(vg[k], e);
          float p, q;
          sigmoid_and_slope<IO>(gg, p, q);
          act[j] = a.act == kActSilu ? (p == 0.f ? 0.f : gg * p) : p;
          dact[j] = a.act == kActSilu ? (p == 0.f ? 0.f : p + gg * q) : q;
        }
      }
    if (a.w2) {
      float ss[2] = {0.f, 0.f};
      float h[EPL];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = k * VEC + e;
          const float v = X::get(vy[k], e) * r1 * w[j] * act[j] * s[j];
          h[j] = a.x ? X::get(vx[k], e) + v : v;
          if (!ok[k]) h[j] = 0.f;
          ss[0] += h[j] * h[j];
          ss[1] += X::get(vn[k], e) * w2[j] * h[j];
        }
      row_sum<2, NT>(ss, tpr, red, half);
      const float r2 = live ? 1.f / sqrtf(ss[0] * inv_d + a.eps) : 0.f, m = ss[1] * r2 * inv_d;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = k * VEC + e;
          const float hn = h[j] * r2, dn = X::get(vn[k], e);
          dw2[j] += dn * hn;
          D[j] += r2 * (dn * w2[j] - hn * m);
        }
    }
    if (g.dx && live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(g.dx, row * a.d + (lane + tpr * k) * VEC, D + k * VEC);
    }
    float ss[1] = {0.f};
    float dg[EPL];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = k * VEC + e;
        const float yn = X::get(vy[k], e) * r1, u = yn * w[j];
        ds[j] += D[j] * u * act[j];
        const float dv = D[j] * s[j];
        dg[j] = dv * u * dact[j];
        const float du = dv * act[j];
        dw[j] += du * yn;
        D[j] = du * w[j];
        ss[0] += D[j] * yn;
      }
    if (a.g && live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(g.dg, row * a.d + (lane + tpr * k) * VEC, dg + k * VEC);
    }
    if (a.w) {
      row_sum<1, NT>(ss, tpr, red, half);
      const float m = ss[0] * inv_d;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = k * VEC + e;
          D[j] = r1 * (D[j] - X::get(vy[k], e) * r1 * m);
        }
    }
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k]) X::store(g.dy, row * a.d + (lane + tpr * k) * VEC, D + k * VEC);
    }
  }
  // sums over the rows of this workgroup, row groups in order
  float* out = g.part + static_cast<int64_t>(blockIdx.x) * 3 * a.d;
  float* const sums[3] = {dw, ds, dw2};
  const bool want[3] = {a.w != nullptr, a.s != nullptr, a.w2 != nullptr};
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (!want[q]) continue;
    if (rpb == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k])
#pragma unroll
          for (int e = 0; e < VEC; ++e) out[q * a.d + (lane + tpr * k) * VEC + e] = sums[q][k * VEC + e];
    } else {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (ok[k])
#pragma unroll
          for (int e = 0; e < VEC; ++e) cols[(t / tpr) * a.d + (lane + tpr * k) * VEC + e] = sums[q][k * VEC + e];
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
__global__ __launch_bounds__(1024) void norm_cols_kernel(const float* part, int parts, int d, float* dw,
                                                        float* ds, float* dw2) {
  __shared__ float red[32][33];
  const int q = blockIdx.y, l = threadIdx.x & 31, c = blockIdx.x * 32 + l, grp = threadIdx.x >> 5;
  float* out = q == 0 ? dw : (q == 1 ? ds : dw2);
  if (!out) return;
  float v = 0.f;
  if (c < d)
    for (int p = grp; p < parts; p += 32) v += part[(static_cast<int64_t>(p) * 3 + q) * d + c];
  red[grp][l] = v;
  __syncthreads();
  if (grp == 0 && c < d) {
    for (int i = 1; i < 32; ++i) v += red[i][l];
    out[c] = v;
  }
}

// How rows of d elements are held: EPL elements a thread, TPR threads.
struct Shape {
  int vec, epl, tpr, nt;
};
Shape shape_of(int d, int es) {
  Shape s;
  s.vec = 16 / es;
  while (d % s.vec != 0) s.vec /= 2;
  // past 8192 the gradients' registers spill a little at 16 elements a thread,
  // and by kilobytes at 32 in 512 threads
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

// Workgroups: as many as the 256 CUs hold at once by their registers, each
// walking over rows.  A second round of a few costs as much as a full one
// (gradients of 32768 rows of 2048 in bf16, where three fit a CU: 213 us with
// 768 workgroups, 27% more with 512, 35% more with 1024; forward of 524288 rows of 128:
// 71 us with 1024, 82 with 2048).
constexpr int64_t kFwdGroups = 1024;
int64_t bwd_groups(const Shape& s) { return s.nt == 1024 ? 256 : (s.epl == 8 ? 768 : 512); }

template <class IO, int VEC, int EPL, int NT>
launch_result launch_one(const NormArgs& a, const NormGrads* g, const Shape& s, hipStream_t st) {
  if (!g) {
    hipLaunchKernelGGL((norm_fwd_kernel<IO, VEC, EPL, NT>),
                       dim3(static_cast<unsigned>(grid_of(a.rows, s, kFwdGroups))), dim3(NT), 0, st, a, s.tpr);
    return hipGetLastError();
  }
  const int64_t grid = grid_of(a.rows, s, bwd_groups(s));
  const int rpb = NT / s.tpr;
  const size_t lds = rpb > 1 ? static_cast<size_t>(rpb) * a.d * 4 : 0;
  hipLaunchKernelGGL((norm_bwd_kernel<IO, VEC, EPL, NT>), dim3(static_cast<unsigned>(grid)), dim3(NT), lds, st,
                     a, *g, s.tpr);
  const launch_result e = hipGetLastError();
  if (e != hipSuccess || (!g->dw && !g->ds && !g->dw2)) return e;
  hipLaunchKernelGGL(norm_cols_kernel, dim3((a.d + 31) / 32, 3), dim3(1024), 0, st, g->part,
                     static_cast<int>(grid), a.d, g->dw, g->ds, g->dw2);
  return hipGetLastError();
}

template <class IO, int VEC>
launch_result launch_vec(const NormArgs& a, const NormGrads* g, const Shape& s, hipStream_t st) {
  if (s.nt == 1024) return launch_one<IO, VEC, 16, 1024>(a, g, s, st);
  if (s.epl == 8) return launch_one<IO, VEC, 8, 256>(a, g, s, st);
  if (s.epl == 16) return launch_one<IO, VEC, 16, 256>(a, g, s, st);
  return launch_one<IO, VEC, 32, 256>(a, g, s, st);
}

launch_result launch(const NormArgs& a, const NormGrads* g, int32_t io_dtype, hipStream_t st) {
  const Shape s = shape_of(a.d, io_dtype == CKDA_DTYPE_BF16 ? 2 : 4);
  if (io_dtype == CKDA_DTYPE_BF16) {
    if (s.vec == 8) return launch_vec<io_bf16, 8>(a, g, s, st);
    if (s.vec == 4) return launch_vec<io_bf16, 4>(a, g, s, st);
    if (s.vec == 2) return launch_vec<io_bf16, 2>(a, g, s, st);
    return launch_vec<io_bf16, 1>(a, g, s, st);
  }
  if (s.vec == 4) return launch_vec<io_f32, 4>(a, g, s, st);
  if (s.vec == 2) return launch_vec<io_f32, 2>(a, g, s, st);
  return launch_vec<io_f32, 1>(a, g, s, st);
}

}  // namespace

size_t norm_bwd_workspace(int64_t rows, int32_t d, int32_t io_dtype) {
  const Shape s = shape_of(d, io_dtype == CKDA_DTYPE_BF16 ? 2 : 4);
  return static_cast<size_t>(grid_of(rows, s, bwd_groups(s))) * 3 * d * 4;
}

launch_result launch_norm_fwd(const NormArgs& a, int32_t io_dtype, hipStream_t s) {
  return launch(a, nullptr, io_dtype, s);
}

launch_result launch_norm_bwd(const NormArgs& a, NormGrads g, int32_t io_dtype, void* ws, hipStream_t s) {
  g.part = static_cast<float*>(ws);
  return launch(a, &g, io_dtype, s);
}

}  // namespace ckda
