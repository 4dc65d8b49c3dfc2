// Gradients of the selective scan.  With g_t = dy_t silu(z_t) and the adjoint
// c_t that later tokens hand back (c_T from dht),
//
//   G_t = c_t + g_t C_t,   w_t = exp(d_t A) G_t h_{t-1},   c_{t-1} = exp(d_t A) G_t
//   dx_t = d_t (G_t . B_t) + D g_t        dd_t = x_t (G_t . B_t) + w_t . A
//   ddt_t = dd_t sigmoid(dt_t + bias)     dz_t = dy_t silu'(z_t) (C_t . h_t + D x_t)
//   dA = sum_t w_t d_t,  dD = sum_t g_t x_t,  dbias = sum_t ddt_t
//   dB_t = sum_ch G_t d_t x_t,  dC_t = sum_ch g_t h_t       over the channels of a group
//
// The states are formed again: a first walk leaves the one entering every kMark
// tokens, and the walk backwards takes kMark tokens at a time, forwards into
// registers and then back.  In a cut sequence the pieces' first walks start from
// zero, and what enters a piece is added to its marks, decayed over the steps
// since, as they are read: so the states are walked once.  Bound by vector
// instructions, 22 a token, channel and state here, 4 of them for the sums over
// channels.  8 x 4096 tokens of 2048 channels and 16 states: bf16 1293 us, of which
// this kernel 858, the walks of states and adjoints 211 and 155, dB and dC 37;
// float32 1512, where the 16-state kernel keeps 44 bytes a lane in scratch.
#include "scan_ops.h"

namespace ckda {
namespace {

template <class IO, class C>
__global__ __launch_bounds__(64 * C::W, 2) void scan_grads_kernel(ScanArgs a) {
  constexpr int CH = C::CH, NR = C::NR, NL = C::NL, SP = C::SP, NSL = C::NSL;
  constexpr int TT = kMark, NT = 64 * C::W, EP = TT * CH / NT, EB = (TT * SP + NT - 1) / NT;
  constexpr int GV = 16 / NL, TG = GV / (2 * NR);  // values summed over channels at a time, their tokens
  constexpr int ES = sizeof(typename IO::storage);
  constexpr float kLn2 = 0.6931471805599453f;
  using Row = RowBits<IO, EP>;
  __shared__ __align__(16) float sd[TT][CH], su[TT][CH], sg[TT][CH], sB[TT][SP], sC[TT][SP];
  __shared__ __align__(16) float sP[3][NSL][TT][CH];  // a slice's G . B, w . A2 and C . h
  __shared__ __align__(16) float sbc[TT][2][SP];      // sums over the block's channels for dB and dC
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const ScanBlock<C> b(a);
  const int blocks = scan_blocks(a.D, a.G, CH);
  const Piece p = piece_of(a, b.slot, a.seg, lane);
  const int ch = lane % CH, sl = wave * NL + lane / CH;
  const int64_t own = static_cast<int64_t>(b.slot) * blocks + b.blk;
  const bool mine = ch < b.cols;
  const int64_t chan = b.chan + ch;
  float A2[NR], c[NR], dA[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int n = sl * NR + i;
    const bool ok = mine && n < a.S;
    A2[i] = ok ? log2_rate(a.A[chan * a.S + n]) : 0.f;
    dA[i] = c[i] = 0.f;
    if (p.n >= 0) {
      if (a.cut)
        c[i] = a.leave[(own * SP + n) * CH + ch];
      else if (a.dht && ok)
        c[i] = a.dht[(static_cast<int64_t>(p.n) * a.D + chan) * a.S + n];
    }
  }
  const int row = tid / (CH / EP), col = tid % (CH / EP) * EP, left = b.cols - col;
  float bias[EP], Dv[EP], dD[EP], db[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) {
    bias[e] = a.bias && e < left ? a.bias[b.chan + col + e] : 0.f;
    Dv[e] = a.Dv && e < left ? a.Dv[b.chan + col + e] : 0.f;
    dD[e] = db[e] = 0.f;
  }
  const int64_t mark0 = p.n >= 0 ? first_slot(a, p.n, kMark) + static_cast<int64_t>(p.s) * a.seg / kMark : 0;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T;

  // where this lane's sum over channels goes: (token, dB or dC, state) of sbc
  const int vi = sum_index<NL>(lane);
  const int sum_at = (vi / (2 * NR) * 2 + vi / NR % 2) * SP + sl * NR + vi % NR;

  Row nx, ndt, ndy, nz;
  uint32_t rB[EB], rC[EB];
  float nh[NR], ne[NR], ns = 0.f;  // a tile's first state: the piece's part, what entered, the steps since
  const auto load = [&](int t0) {
    const bool some = t0 >= 0;
    const int rows = !some ? 0 : (p.len - t0 < TT ? p.len - t0 : TT);
    const int64_t at = p.begin + (some ? t0 : 0);
    const bool ok = row < rows && left > 0;
    nx.load(rows_rsrc<IO>(a.x, at, a.sx, b.chan, rows, b.cols), ok ? static_cast<int>(row * a.sx + col) * ES : kOut, left, a.vec);
    ndt.load(rows_rsrc<IO>(a.dt, at, a.sdt, b.chan, rows, b.cols), ok ? static_cast<int>(row * a.sdt + col) * ES : kOut, left, a.vec);
    ndy.load(rows_rsrc<IO>(a.dy, at, a.D, b.chan, rows, b.cols), ok ? static_cast<int>(static_cast<int64_t>(row) * a.D + col) * ES : kOut, left, a.vec);
    if (a.z)
      nz.load(rows_rsrc<IO>(a.z, at, a.sz, b.chan, rows, b.cols), ok ? static_cast<int>(row * a.sz + col) * ES : kOut, left, a.vec);
    const rsrc_t rb = rows_rsrc<IO>(a.Bm, at, a.sb, static_cast<int64_t>(b.g) * a.S, rows, a.S);
    const rsrc_t rc = rows_rsrc<IO>(a.Cm, at, a.sc, static_cast<int64_t>(b.g) * a.S, rows, a.S);
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int t = (tid + NT * i) / SP, n = (tid + NT * i) % SP;
      const bool in = t < rows && n < a.S;
      ldraw<ES>(rb, in ? static_cast<int>(t * a.sb + n) * ES : kOut, rB + i);
      ldraw<ES>(rc, in ? static_cast<int>(t * a.sc + n) * ES : kOut, rC + i);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      nh[i] = some ? a.marks[(((mark0 + t0 / kMark) * blocks + b.blk) * SP + sl * NR + i) * CH + ch] : 0.f;
      if (a.cut) ne[i] = a.entry[(own * SP + sl * NR + i) * CH + ch];
    }
    if (a.cut && some) ns = a.mspan[((mark0 + t0 / kMark) * blocks + b.blk) * CH + ch];
  };

  const int last = p.n >= 0 && p.len > 0 ? (p.len - 1) / TT * TT : -1;
  if (last >= 0) load(last);
  for (int t0 = last; t0 >= 0; t0 -= TT) {
    const int rows = p.len - t0 < TT ? p.len - t0 : TT;
    // kept for the outputs; d and g are read back from this thread's places in LDS
    const Row rx = nx;
    float slope[EP], dz[EP];
    {
      float u[EP], d[EP], g[EP];
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        d[e] = ndt.get(e) + bias[e];
        slope[e] = 1.f;
        g[e] = ndy.get(e);
        dz[e] = 0.f;
      }
      if (a.softplus)
#pragma unroll
        for (int e = 0; e < EP; ++e) softplus_and_slope(d[e], d[e], slope[e]);
      if (a.z)
#pragma unroll
        for (int e = 0; e < EP; ++e) {
          float act, s;
          silu_and_slope<IO>(nz.get(e), act, s);
          dz[e] = g[e] * s;
          g[e] *= act;
        }
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        d[e] = row < rows ? d[e] : 0.f;
        u[e] = d[e] * rx.get(e);
      }
      lds_put<EP>(&sd[row][col], d);
      lds_put<EP>(&su[row][col], u);
      lds_put<EP>(&sg[row][col], g);
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const int k = tid + NT * i;
        if (k < TT * SP) {
          sB[k / SP][k % SP] = dec<IO>(rB + i, 0);
          sC[k / SP][k % SP] = dec<IO>(rC + i, 0);
        }
      }
    }
    float h[TT + 1][NR], ex[TT][NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) h[0][i] = nh[i];
    if (a.cut) enter(ns, A2, ne, nh, h[0]);
    __syncthreads();
    load(t0 - TT);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float dd = sd[t][ch], uu = su[t][ch];
      float B[NR], Cv[NR], y = 0.f;
      lds_run<NR>(&sB[t][sl * NR], B);
      lds_run<NR>(&sC[t][sl * NR], Cv);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        ex[t][i] = decay_by(dd, A2[i]);
        h[t + 1][i] = __builtin_fmaf(ex[t][i], h[t][i], uu * B[i]);
        y = __builtin_fmaf(Cv[i], h[t + 1][i], y);
      }
      sP[2][sl][t][ch] = y;
    }
#pragma unroll
    for (int tg = TT / TG - 1; tg >= 0; --tg) {
      float v[GV];
#pragma unroll
      for (int j = TG - 1; j >= 0; --j) {
        const int t = tg * TG + j;
        const float dd = sd[t][ch], uu = su[t][ch], gg = sg[t][ch];
        float B[NR], Cv[NR], gb = 0.f, wa = 0.f;
        lds_run<NR>(&sB[t][sl * NR], B);
        lds_run<NR>(&sC[t][sl * NR], Cv);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float G = __builtin_fmaf(gg, Cv[i], c[i]);
          gb = __builtin_fmaf(G, B[i], gb);
          c[i] = ex[t][i] * G;
          const float w = c[i] * h[t][i];
          wa = __builtin_fmaf(w, A2[i], wa);
          dA[i] = __builtin_fmaf(w, dd, dA[i]);
          v[(j * 2) * NR + i] = G * uu;
          v[(j * 2 + 1) * NR + i] = gg * h[t + 1][i];
        }
        sP[0][sl][t][ch] = gb;
        sP[1][sl][t][ch] = wa;
      }
      const float sum = sum_channels<NL>(v);
      if ((lane & 3) == 0) (&sbc[0][0][0])[tg * TG * 2 * SP + sum_at] = sum;
    }
    __syncthreads();
    for (int k = tid; k < rows * 2 * SP; k += NT)
      a.partbc[(static_cast<int64_t>(b.blk) * tokens + p.begin + t0) * 2 * SP + k] = (&sbc[0][0][0])[k];
    if (row < rows && left > 0) {
      float gb[EP], wa[EP], y[EP], dx[EP], dt[EP], x[EP], d[EP], g[EP];
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        gb[e] = wa[e] = d[e] = g[e] = 0.f;
        x[e] = rx.get(e);
        y[e] = Dv[e] * x[e];
      }
      lds_add<EP>(&sd[row][col], d);
      lds_add<EP>(&sg[row][col], g);
#pragma unroll
      for (int s = 0; s < NSL; ++s) {
        lds_add<EP>(&sP[0][s][row][col], gb);
        lds_add<EP>(&sP[1][s][row][col], wa);
        lds_add<EP>(&sP[2][s][row][col], y);
      }
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        dx[e] = __builtin_fmaf(d[e], gb[e], Dv[e] * g[e]);
        // a slope of 0 is a masked token's, whose w . A may have left float32
        dt[e] = slope[e] == 0.f ? 0.f : __builtin_fmaf(x[e], gb[e], wa[e] * kLn2) * slope[e];
        dz[e] *= y[e];
        dD[e] = __builtin_fmaf(g[e], x[e], dD[e]);
        db[e] += dt[e];
      }
      const int off = static_cast<int>(static_cast<int64_t>(row) * a.D + col) * ES;
      const int64_t at = p.begin + t0;
      Row::store(rows_rsrc<IO>(a.dx, at, a.D, b.chan, rows, b.cols), off, left, a.vec, dx);
      Row::store(rows_rsrc<IO>(a.ddt, at, a.D, b.chan, rows, b.cols), off, left, a.vec, dt);
      if (a.z) Row::store(rows_rsrc<IO>(a.dz, at, a.D, b.chan, rows, b.cols), off, left, a.vec, dz);
    }
  }
  if (a.dh0 && p.n >= 0 && p.s == 0 && mine) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (sl * NR + i < a.S) a.dh0[(static_cast<int64_t>(p.n) * a.D + chan) * a.S + sl * NR + i] = c[i];
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) a.partA[(own * SP + sl * NR + i) * CH + ch] = dA[i];
  // the rows' sums for dD and dbias, in order
  __syncthreads();
  float* red = &sP[0][0][0][0];
#pragma unroll
  for (int e = 0; e < EP; ++e) {
    red[row * CH + col + e] = dD[e];
    red[(TT + row) * CH + col + e] = db[e];
  }
  __syncthreads();
  for (int k = tid; k < 2 * CH; k += NT) {
    float v = 0.f;
    for (int r = 0; r < TT; ++r) v += red[((k / CH) * TT + r) * CH + k % CH];
    a.partD[own * 2 * CH + k] = v;
  }
}

// dB and dC: the blocks' sums of a group, in order.
template <class IO, class C>
__global__ __launch_bounds__(256) void scan_bc_kernel(ScanArgs a) {
  constexpr int SP = C::SP;
  using T = typename IO::storage;
  const int nb = (a.D / a.G + C::CH - 1) / C::CH;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T, row = 2 * SP;
  const int64_t first = a.cu ? cu_at(a, 0) : 0, end = a.cu ? cu_at(a, a.N) : tokens;
  const int64_t total = tokens * a.G * row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t tg = i / row, t = tg / a.G;
    const int k = static_cast<int>(i - tg * row), g = static_cast<int>(tg - t * a.G), n = k % SP;
    if (n >= a.S || t < first || t >= end) continue;
    float v = 0.f;
    for (int j = 0; j < nb; ++j) v += a.partbc[(static_cast<int64_t>(g * nb + j) * tokens + t) * row + k];
    IO::store(static_cast<T*>(k < SP ? a.dB : a.dC), tg * a.S + n, v);
  }
}

// dA (what = 0) and dD, dbias (what = 1): the pieces' sums, 32 columns a
// workgroup at a time, its 32 groups of lanes taking every 32nd piece's; their sums
// are added in order.
template <class C>
__global__ __launch_bounds__(1024) void scan_cols_kernel(ScanArgs a, int what) {
  constexpr int CH = C::CH, SP = C::SP;
  __shared__ float red[32][33];
  const int per = a.D / a.G, nb = (per + CH - 1) / CH, blocks = a.G * nb;
  const int l = threadIdx.x & 31, grp = threadIdx.x >> 5, rows = what ? 2 : SP;
  const int64_t cols = static_cast<int64_t>(blocks) * rows * CH;
  const float* part = what ? a.partD : a.partA;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * 32; first < cols; first += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t i = first + l;
    float v = 0.f;
    if (i < cols)
      for (int s = grp; s < a.slots; s += 32) v += part[s * cols + i];
    red[grp][l] = v;
    __syncthreads();
    if (grp == 0 && i < cols) {
      for (int r = 1; r < 32; ++r) v += red[r][l];
      const int blk = static_cast<int>(i / (rows * CH)), k = static_cast<int>(i - static_cast<int64_t>(blk) * rows * CH);
      const int n = k / CH, g = blk / nb, c = (blk - g * nb) * CH + k % CH;
      const int64_t chan = static_cast<int64_t>(g) * per + c;
      if (c < per) {
        if (what == 0) {
          if (n < a.S) a.dA[chan * a.S + n] = v;
        } else {
          float* out = n == 0 ? a.dD : a.dbias;
          if (out) out[chan] = v;
        }
      }
    }
    __syncthreads();
  }
}

// Workgroups for the sums of `rows` values a channel: a launch counts its threads in 32
// bits, which groups of a channel each, at 64 columns a group, would pass.
dim3 cols_grid(int64_t cols, int rows) {
  const int64_t n = (cols * rows + 31) / 32;
  return dim3(static_cast<unsigned>(n < (1 << 20) ? n : 1 << 20));
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// The workspace at ws: pieces, marks, and the partial sums.
size_t layout(ScanArgs& a, const ScanPlan& p, unsigned char* ws) {
  a.seg = p.seg;
  a.slots = p.slots;
  a.cut = p.cut;
  const size_t lanes = static_cast<size_t>(p.blocks) * p.CH * 4, at = lanes * p.SP;
  size_t n = 0;
  const auto take = [&](size_t bytes) {
    float* r = reinterpret_cast<float*>(ws + n);
    n += up256(bytes);
    return r;
  };
  a.entry = take(p.cut ? at * p.slots : 0);
  a.leave = take(p.cut ? at * p.slots : 0);
  a.mspan = take(p.cut ? lanes * p.mslots : 0);
  a.span = take(p.cut ? lanes * p.slots : 0);
  a.marks = take(at * p.mslots);
  a.partbc = take(static_cast<size_t>(p.blocks) * a.B * a.T * 2 * p.SP * 4);
  a.partA = take(at * p.slots);
  a.partD = take(2 * lanes * p.slots);
  return n;
}

template <class IO>
launch_result launch_io(const ScanArgs& a, const ScanPlan& p, hipStream_t s) {
  return scan_config(p.which, [&](auto cfg) -> launch_result {
    using C = decltype(cfg);
    if (p.slots > 0) {
      hipLaunchKernelGGL((scan_grads_kernel<IO, C>), dim3(static_cast<unsigned>(static_cast<int64_t>(p.slots) * p.blocks)),
                         dim3(64 * C::W), 0, s, a);
      const launch_result e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const int64_t total = (static_cast<int64_t>(a.B) * a.T * a.G * 2 * C::SP + 255) / 256;
    if (total > 0) {
      hipLaunchKernelGGL((scan_bc_kernel<IO, C>), dim3(static_cast<unsigned>(total < 16384 ? total : 16384)), dim3(256), 0, s, a);
      const launch_result e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const int64_t cols = static_cast<int64_t>(p.blocks) * C::CH;
    hipLaunchKernelGGL((scan_cols_kernel<C>), cols_grid(cols, C::SP), dim3(1024), 0, s, a, 0);
    const launch_result e = hipGetLastError();
    if (e != hipSuccess || (!a.dD && !a.dbias)) return e;
    hipLaunchKernelGGL((scan_cols_kernel<C>), cols_grid(cols, 2), dim3(1024), 0, s, a, 1);
    return hipGetLastError();
  });
}

}  // namespace

size_t scan_bwd_workspace(const ScanArgs& a0) {
  ScanArgs a = a0;
  return layout(a, scan_plan(a, true), nullptr);
}

launch_result launch_scan_bwd(ScanArgs a, int32_t io_dtype, void* ws, hipStream_t s) {
  const ScanPlan p = scan_plan(a, true);
  layout(a, p, static_cast<unsigned char*>(ws));
  if (p.slots > 0) {
    const launch_result e = launch_scan_marks(a, p, io_dtype, s);
    if (e != hipSuccess) return e;
  }
  return io_dtype == CKDA_DTYPE_BF16 ? launch_io<io_bf16>(a, p, s) : launch_io<io_f32>(a, p, s);
}

}  // namespace ckda
