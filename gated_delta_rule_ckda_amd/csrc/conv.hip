// Short causal convolution, a channel and K taps (2 to 4):
//
//   e_t = b + sum_j w_j x_{t-K+1+j},   y_t = act(e_t)        act: none or silu
//
// the inputs before a sequence's first token coming from its cache h0 (the last
// K-1 inputs of what went before; zeros without).  Backwards, g_t = dy_t act'(e_t):
//
//   dx_s = sum_j w_j g_{s+K-1-j},  dw_j = sum_t g_t x_{t-K+1+j},  db = sum_t g_t
//
// with dht (what the cache left behind is worth) added to the inputs it holds.
// Bound by HBM: x is read and y written once.  A thread walks over a tile of
// tokens for a vector of channels with the last K-1 rows in registers, so a row
// is read again only at tile edges, and consecutive threads take consecutive
// channels, so a wave reads whole lines.  Four channels a thread: with two
// and with eight the forward took 56 and 60 us instead of 55, the gradients 133 and
// 105 instead of 98.  8 x 4096 tokens of 2048 channels, 4 taps: bf16 54 us (5.0
// TB/s), gradients 96 (4.2); float32 109 (4.9), gradients 159 (5.1).
#include "row_ops.h"
#include "spans.h"

namespace ckda {
namespace {

template <int VEC, int K>
struct Taps {
  float w[VEC][K], b[VEC];
  __device__ __forceinline__ Taps(const ConvArgs& a, int c) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int64_t at = c + e < a.D ? c + e : 0;
#pragma unroll
      for (int j = 0; j < K; ++j) w[e][j] = a.w[at * K + j];
      b[e] = a.bias ? a.bias[at] : 0.f;
    }
  }
};

// The K-1 inputs before token t0 of sequence n, whose tokens begin at `begin`.
template <class X, int VEC, int K>
__device__ __forceinline__ void window(const ConvArgs& a, int n, int64_t begin, int t0, int c, float (&x)[K - 1][VEC]) {
#pragma unroll
  for (int r = 0; r < K - 1; ++r) {
    const int t = t0 - (K - 1) + r;
    if (t >= 0) {
      X::row(a.x, (begin + t) * a.sx + c, a.D - c, x[r]);
    } else if (a.h0) {
      X::row(a.h0, (static_cast<int64_t>(n) * (K - 1) + (K - 1 + t)) * a.D + c, a.D - c, x[r]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[r][e] = 0.f;
    }
  }
}

template <class IO, int VEC, bool ALIGNED, int K>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int cx, int ny) {
  using X = Chans<IO, VEC, ALIGNED>;
  constexpr int U = 4;
  const int chunk = blockIdx.x % ny, py = 256 / cx;
  const int slot = (blockIdx.x / ny) * py + threadIdx.x / cx;
  const int c = (chunk * cx + (threadIdx.x & (cx - 1))) * VEC;
  if (c >= a.D || slot >= a.slots) return;
  const Piece p = piece_of_thread(a, slot, a.tile);
  if (p.n < 0) return;
  const Taps<VEC, K> w(a, c);
  const Seq q = sequence(a, p.n);
  float x[K - 1 + U][VEC];
  {
    float first[K - 1][VEC];
    window<X, VEC, K>(a, p.n, q.begin, p.s * a.tile, c, first);
#pragma unroll
    for (int r = 0; r < K - 1; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[r][e] = first[r][e];
  }
  typename X::V next[U];
  const auto load = [&](int t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      next[u] = typename X::V{};
      if (t + u < p.len) next[u] = X::load(a.x, (p.begin + t + u) * a.sx + c, a.D - c);
    }
  };
  load(0);
  for (int t = 0; t < p.len; t += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[K - 1 + u][e] = X::get(next[u], e);
    load(t + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u >= p.len) break;
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float s = w.b[e];
#pragma unroll
        for (int j = 0; j < K; ++j) s += w.w[e][j] * x[u + j][e];
        y[e] = a.act ? silu_of<IO>(s) : s;
      }
      X::store(a.y, (p.begin + t + u) * a.D + c, a.D - c, y);
    }
#pragma unroll
    for (int r = 0; r < K - 1; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[r][e] = x[U + r][e];
  }
  if (a.ht && p.s == 0) {
    // by the thread that read the cache, since ht may be h0's buffer
    const int64_t at = static_cast<int64_t>(p.n) * (K - 1) * a.D + c;
#pragma unroll
    for (int r = 0; r < K - 1; ++r) {
      const int t = q.len - (K - 1) + r;
      float v[VEC];
      if (t >= 0) {
        X::row(a.x, (q.begin + t) * a.sx + c, a.D - c, v);
      } else if (a.h0) {
        X::row(a.h0, at + static_cast<int64_t>(K - 1 + t) * a.D, a.D - c, v);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = 0.f;
      }
      X::store(a.ht, at + static_cast<int64_t>(r) * a.D, a.D - c, v);
    }
  }
}

// Gradients.  At step t a thread forms g_t from the window of inputs, then the
// gradient of the input K-1 tokens back, whose last tap g_t was; it walks K-1
// tokens past its tile for the inputs at the tile's end.  Each workgroup leaves
// its tiles' sums for dw and db in part[workgroup][K + 1][D].
template <class IO, int VEC, bool ALIGNED, int K>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, ConvGrads gr, int cx, int ny) {
  using X = Chans<IO, VEC, ALIGNED>;
  __shared__ float red[256 * VEC];
  const int chunk = blockIdx.x % ny, py = 256 / cx, grp = blockIdx.x / ny;
  const int slot = grp * py + threadIdx.x / cx;
  const int c = (chunk * cx + (threadIdx.x & (cx - 1))) * VEC;
  float dw[K][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = 0.f;
  }
  Piece p;
  p.n = -1;
  if (c < a.D && slot < a.slots) p = piece_of_thread(a, slot, a.tile);
  if (p.n >= 0) {
    const Taps<VEC, K> w(a, c);
    const Seq q = sequence(a, p.n);
    const int t0 = p.s * a.tile;
    float x[K][VEC], g[K][VEC];  // inputs t-K+1..t, gradients g_{t-K+1}..g_t
    {
      float first[K - 1][VEC];
      window<X, VEC, K>(a, p.n, q.begin, t0, c, first);
#pragma unroll
      for (int r = 0; r < K; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[r][e] = r > 0 ? first[r - 1][e] : 0.f;
          g[r][e] = 0.f;
        }
    }
    typename X::V nx = typename X::V{}, ng = nx;
    const auto load = [&](int t) {
      if (t < q.len) {
        nx = X::load(a.x, (q.begin + t) * a.sx + c, a.D - c);
        ng = X::load(gr.dy, (q.begin + t) * a.D + c, a.D - c);
      }
    };
    const int end = t0 + p.len + K - 1;
    load(t0);
    for (int t = t0; t < end; ++t) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
          x[r][e] = x[r + 1][e];
          g[r][e] = g[r + 1][e];
        }
        x[K - 1][e] = X::get(nx, e);
        g[K - 1][e] = t < q.len ? X::get(ng, e) : 0.f;
      }
      load(t + 1 < end ? t + 1 : q.len);
      if (a.act && t < q.len) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float s = w.b[e];
#pragma unroll
          for (int j = 0; j < K; ++j) s += w.w[e][j] * x[j][e];
          float y, slope;
          silu_and_slope<IO>(s, y, slope);
          g[K - 1][e] *= slope;
        }
      }
      if (t < t0 + p.len) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          db[e] += g[K - 1][e];
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][e] += g[K - 1][e] * x[j][e];
        }
      }
      // the input before the window's second: token t-K+1, or the cache's row t
      const int s = t - (K - 1);
      if (s < t0 && !(s < 0 && gr.dh0)) continue;
      float dx[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        dx[e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dx[e] += w.w[e][j] * g[K - 1 - j][e];
      }
      if (gr.dht && t >= q.len) {
        float more[VEC];
        X::row(gr.dht, (static_cast<int64_t>(p.n) * (K - 1) + (t - q.len)) * a.D + c, a.D - c, more);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dx[e] += more[e];
      }
      if (s >= 0)
        X::store(gr.dx, (q.begin + s) * a.D + c, a.D - c, dx);
      else if (t0 == 0)
        X::store(gr.dh0, (static_cast<int64_t>(p.n) * (K - 1) + t) * a.D + c, a.D - c, dx);
    }
  }
  // sums over the workgroup's tiles, in order
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    if (py > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) red[threadIdx.x * VEC + e] = j < K ? dw[j < K ? j : 0][e] : db[e];
      __syncthreads();
    }
    if (threadIdx.x < cx && c < a.D) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float v = j < K ? dw[j < K ? j : 0][e] : db[e];
        for (int r = 1; r < py; ++r) v += red[(threadIdx.x + r * cx) * VEC + e];
        if (c + e < a.D) gr.part[(static_cast<int64_t>(grp) * (K + 1) + j) * a.D + c + e] = v;
      }
    }
  }
}

// dw[c][j] and db[c]: 32 columns of part a workgroup, its 32 groups of lanes
// taking every 32nd row; their sums are added in order.
__global__ __launch_bounds__(1024) void conv_cols_kernel(const float* part, int parts, int D, int K, float* dw,
                                                         float* db) {
  __shared__ float red[32][33];
  const int l = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t cols = static_cast<int64_t>(K + 1) * D, i = static_cast<int64_t>(blockIdx.x) * 32 + l;
  float v = 0.f;
  if (i < cols) {
#pragma unroll 8
    for (int p = grp; p < parts; p += 32) v += part[p * cols + i];
  }
  red[grp][l] = v;
  __syncthreads();
  if (grp == 0 && i < cols) {
    for (int r = 1; r < 32; ++r) v += red[r][l];
    const int64_t j = i / D, c = i - j * D;
    if (j < K)
      dw[c * K + j] = v;
    else if (db)
      db[c] = v;
  }
}

// One token a sequence: the cache moves up a row in place.
template <class IO, int VEC, bool ALIGNED, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, int nv) {
  using X = Chans<IO, VEC, ALIGNED>;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = i / nv;
  const int c = static_cast<int>(i - n * nv) * VEC;
  if (n >= a.N) return;
  const int64_t at = n * (K - 1) * a.D + c;
  float x[K][VEC], y[VEC];
#pragma unroll
  for (int r = 0; r < K - 1; ++r) X::row(a.h0, at + static_cast<int64_t>(r) * a.D, a.D - c, x[r]);
  X::row(a.x, n * a.sx + c, a.D - c, x[K - 1]);
  const Taps<VEC, K> w(a, c);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float s = w.b[e];
#pragma unroll
    for (int j = 0; j < K; ++j) s += w.w[e][j] * x[j][e];
    y[e] = a.act ? silu_of<IO>(s) : s;
  }
  X::store(a.y, n * a.D + c, a.D - c, y);
#pragma unroll
  for (int r = 0; r < K - 1; ++r) X::store(a.ht, at + static_cast<int64_t>(r) * a.D, a.D - c, x[r + 1]);
}

// Whether every vector of VEC channels lies at a multiple of its size.
bool aligned(const ConvArgs& a, int vec, int es) {
  return a.D % vec == 0 && a.sx % vec == 0 && reinterpret_cast<uintptr_t>(a.x) % (vec * es) == 0;
}

struct Grid {
  int cx, ny;         // lanes over channels, workgroups over channels
  int64_t groups;     // workgroups over slots
};
Grid grid_of(const ConvArgs& a, int vec) {
  const int nv = (a.D + vec - 1) / vec;
  Grid g{1, 0, 0};
  while (g.cx < 64 && g.cx < nv) g.cx *= 2;
  g.ny = (nv + g.cx - 1) / g.cx;
  const int py = 256 / g.cx;
  g.groups = (static_cast<int64_t>(a.slots) + py - 1) / py;
  return g;
}

constexpr int kVec = 4;  // channels a thread

int32_t slots_of(const ConvArgs& a, int tile) {
  if (a.N == 0) return 0;  // a packed batch of no sequences
  if (a.cu) return a.T / tile + a.N;
  return a.N * (a.T > 0 ? (a.T + tile - 1) / tile : 1);
}
// Tokens of a tile: long ones read fewer rows twice and leave fewer partial sums,
// but there have to be waves enough to hide the loads.  Measured: gradients of
// 2 x 4096 tokens of 2001 channels (1000 waves with tiles of 64) 82 us with 64,
// 54 with 32; of 8 x 4096 of 2048 in bf16 (4096 waves) 96 with 64, 106 with 32;
// forward of the latter 53 with 32 and with 64, 55 with 16.
void set_tile(ConvArgs& a, bool grads) {
  const int64_t nv = (a.D + kVec - 1) / kVec;
  a.tile = grads ? 64 : 32;
  while (a.tile > 8 && slots_of(a, a.tile) * nv < 2048 * 64) a.tile /= 2;
  a.slots = slots_of(a, a.tile);
}

enum Pass { kFwd, kBwd, kStep };

template <class IO, int VEC, bool ALIGNED, int K>
launch_result launch_one(const ConvArgs& a, const ConvGrads* g, Pass pass, hipStream_t s) {
  if (pass == kStep) {
    const int nv = (a.D + VEC - 1) / VEC;
    const int64_t grid = (static_cast<int64_t>(a.N) * nv + 255) / 256;
    hipLaunchKernelGGL((conv_step_kernel<IO, VEC, ALIGNED, K>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a,
                       nv);
    return hipGetLastError();
  }
  const Grid r = grid_of(a, VEC);
  const dim3 grid(static_cast<unsigned>(r.groups * r.ny));
  if (pass == kFwd) {
    hipLaunchKernelGGL((conv_fwd_kernel<IO, VEC, ALIGNED, K>), grid, dim3(256), 0, s, a, r.cx, r.ny);
    return hipGetLastError();
  }
  if (r.groups > 0) {
    hipLaunchKernelGGL((conv_bwd_kernel<IO, VEC, ALIGNED, K>), grid, dim3(256), 0, s, a, *g, r.cx, r.ny);
    const launch_result e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t cols = static_cast<int64_t>(K + 1) * a.D;
  hipLaunchKernelGGL(conv_cols_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(1024), 0, s, g->part,
                     static_cast<int>(r.groups), a.D, K, g->dw, g->dbias);
  return hipGetLastError();
}

template <class IO, int VEC, bool ALIGNED>
launch_result launch_taps(const ConvArgs& a, const ConvGrads* g, Pass pass, hipStream_t s) {
  if (a.K == 2) return launch_one<IO, VEC, ALIGNED, 2>(a, g, pass, s);
  if (a.K == 3) return launch_one<IO, VEC, ALIGNED, 3>(a, g, pass, s);
  return launch_one<IO, VEC, ALIGNED, 4>(a, g, pass, s);
}

template <class IO>
launch_result launch_io(const ConvArgs& a, const ConvGrads* g, Pass pass, hipStream_t s) {
  if (aligned(a, kVec, sizeof(typename IO::storage))) return launch_taps<IO, kVec, true>(a, g, pass, s);
  return launch_taps<IO, kVec, false>(a, g, pass, s);
}
launch_result launch(const ConvArgs& a, const ConvGrads* g, int32_t io_dtype, Pass pass, hipStream_t s) {
  return io_dtype == CKDA_DTYPE_BF16 ? launch_io<io_bf16>(a, g, pass, s) : launch_io<io_f32>(a, g, pass, s);
}

}  // namespace

int64_t conv_threads(const ConvArgs& a0, bool grads) {
  ConvArgs a = a0;
  const int64_t most = a.cu ? a.T / 8 + static_cast<int64_t>(a.N) : static_cast<int64_t>(a.N) * (a.T / 8 + 1);
  if (most >= (int64_t(1) << 31)) return int64_t(1) << 62;
  set_tile(a, grads);
  const Grid g = grid_of(a, kVec);
  return g.groups * g.ny * 256;
}

// A column sum a workgroup.
size_t conv_bwd_workspace(const ConvArgs& a0) {
  ConvArgs a = a0;
  set_tile(a, true);
  return static_cast<size_t>(grid_of(a, kVec).groups) * (a.K + 1) * a.D * 4;
}

launch_result launch_conv_fwd(ConvArgs a, int32_t io_dtype, hipStream_t s) {
  set_tile(a, false);
  return launch(a, nullptr, io_dtype, kFwd, s);
}

launch_result launch_conv_bwd(ConvArgs a, ConvGrads g, int32_t io_dtype, void* ws, hipStream_t s) {
  set_tile(a, true);
  g.part = static_cast<float*>(ws);
  return launch(a, &g, io_dtype, kBwd, s);
}

launch_result launch_conv_step(const ConvArgs& a, int32_t io_dtype, hipStream_t s) {
  return launch(a, nullptr, io_dtype, kStep, s);
}

}  // namespace ckda
