// Selective scan: whole prompts, and one token a sequence (see scan_ops.h for the
// formulas and how a workgroup holds channels and states).
//
// Bound by the vector instructions and the LDS beside each other.  A token, channel
// and state takes a power and four multiplications or additions; on a SIMD a power
// costs 8.4 cycles a wave, the others 2.5 to 2.9 where two waves or more take turns
// and about 4 where powers come between them, which is why they run in groups.  B
// and C, the same for all channels, reach the lanes as broadcast reads, so a lane
// holds several states.  8 x 4096 tokens of 2048 channels and 16 states: bf16 364 us
// (1.5 TB/s), float32 394 (2.7).  The bytes alone would take 106 (212) us, the
// states' instructions 131, with the input waves' (38% of all) about 200.
#include "scan_ops.h"

namespace ckda {
namespace {

// What a walk over a piece leaves behind.
enum Walk {
  kOutputs,   // y, and ht after a sequence's last piece
  kSums,      // the state it would end in from zero, and the sum of its steps
  kMarks,     // the states entering every kMark tokens; in a piece of a cut sequence
              // from zero, with the sums of steps up to them, and what kSums leaves
  kBack,      // kSums for the adjoint, against the tokens:
              //   c_{t-1} = exp(d_t A) (c_t + g_t C_t),  g_t = dy_t silu(z_t)
};

// The operands of four tokens on their way from LDS to the states.
template <int NR, bool Y>
struct Four {
  float d[4], u[4], B[4][NR], C[4][NR];
  __device__ __forceinline__ void load(const float* sd, const float* su, const float* sB, const float* sC, int CH, int SP) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = sd[j * CH];
      u[j] = su[j * CH];
      lds_run<NR>(sB + j * SP, B[j]);
      if (Y) lds_run<NR>(sC + j * SP, C[j]);
    }
  }
};

// W waves walk the states over a tile of TT tokens; four more, spread over the same
// SIMDs, form the steps and writes of tiles to come in LDS and finish the outputs
// of the one before.  Tiles are laid down two
// ahead, so that the states' operands are asked for four tokens ahead across
// tiles.
template <class IO, class C, int WALK>
__global__ __launch_bounds__(64 * (C::W + 4), 4) void scan_walk_kernel(ScanArgs a) {
  constexpr int CH = C::CH, NR = C::NR, NL = C::NL, SP = C::SP, NSL = C::NSL;
  constexpr int TT = 16, EP = TT * CH / 256, EB = (TT * SP + 255) / 256;
  constexpr int ES = sizeof(typename IO::storage);
  constexpr bool kY = WALK == kOutputs, kRev = WALK == kBack, kSum = WALK == kSums || kRev;
  using Row = RowBits<IO, EP>;
  __shared__ __align__(16) float sd[3][TT][CH], su[3][TT][CH], sB[3][TT][SP], sC[kY ? 3 : 1][kY ? TT : 1][SP];
  __shared__ __align__(16) float sY[2][kY ? NSL : 1][TT][CH];
  const int lane = threadIdx.x & 63, wave = uniform32(threadIdx.x >> 6);
  const ScanBlock<C> b(a);
  const Piece p = piece_of(a, b.slot, a.seg, lane);
  if (p.n < 0) return;
  // nothing enters a piece after a sequence's last one, or from before its first
  if (WALK == kSums && p.s == p.count - 1) return;
  if (kRev && p.s == 0) return;
  const int tiles = (p.len + TT - 1) / TT;
  const int64_t blocks = scan_blocks(a.D, a.G, CH);

  if (wave < C::W) {
    // The outputs' walk takes longer than the other waves' part of a tile, and waits
    // less with priority (packed prompts: 404 us against 442).  In the shorter walks
    // the others' loads come late, so they go first (sums of states: 340 us with
    // priority here, 255 without any, gradients of a layer 1297 against 1335).
    if (kY) __builtin_amdgcn_s_setprio(2);
    // ---- states
    const int ch = lane % CH, sl = wave * NL + lane / CH;
    const bool mine = ch < b.cols;
    const int64_t chan = b.chan + ch;
    const int64_t own = (b.slot * blocks + b.blk) * SP + sl * NR;
    float A2[NR], h[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int n = sl * NR + i;
      const bool ok = mine && n < a.S;
      A2[i] = ok ? log2_rate(a.A[chan * a.S + n]) : 0.f;
      h[i] = 0.f;
      if (!kSum && !(WALK == kMarks && a.cut)) {
        if (a.cut)
          h[i] = a.entry[(own + i) * CH + ch];
        else if (a.h0 && ok)
          h[i] = a.h0[(static_cast<int64_t>(p.n) * a.D + chan) * a.S + n];
      }
    }
    const int64_t mark0 = WALK == kMarks ? first_slot(a, p.n, kMark) + static_cast<int64_t>(p.s) * a.seg / kMark : 0;
    float span = 0.f;
    Four<NR, kY> ops[2];
    const auto fetch = [&](Four<NR, kY>& o, int q, int t) {
      o.load(&sd[q][t][ch], &su[q][t][ch], &sB[q][t][sl * NR], kY ? &sC[kY ? q : 0][kY ? t : 0][sl * NR] : nullptr, CH, SP);
    };
    __syncthreads();
    int q = 0, half = 0;
    if (tiles > 0) fetch(ops[0], 0, kRev ? TT - 4 : 0);
    for (int k = 0; k < tiles; ++k) {
      if (WALK == kMarks) {
        static_assert(TT == kMark, "a state a tile");
#pragma unroll
        for (int i = 0; i < NR; ++i)
          a.marks[(((mark0 + k) * blocks + b.blk) * SP + sl * NR + i) * CH + ch] = h[i];
        if (a.cut && sl == 0) a.mspan[((mark0 + k) * blocks + b.blk) * CH + ch] = span;
      }
      const int next = q == 2 ? 0 : q + 1;
#pragma unroll
      for (int g = 0; g < TT / 4; ++g) {
        Four<NR, kY>& o = ops[g & 1];
        float e[4][NR];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < NR; ++i) e[j][i] = decay_arg(o.d[j], A2[i]);
        // past the last tile this reads what an earlier one left
        const int to = (g + 1) % (TT / 4) * 4;
        fetch(ops[(g + 1) & 1], g + 1 < TT / 4 ? q : next, kRev ? TT - 4 - to : to);
        __builtin_amdgcn_sched_barrier(0);
        // powers run together: a switch between them and other operations costs both
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < NR; ++i) e[j][i] = __builtin_amdgcn_exp2f(e[j][i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int j = kRev ? 3 - jj : jj;
          float y = 0.f;
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            if (kRev)
              h[i] = e[j][i] * __builtin_fmaf(o.u[j], o.B[j][i], h[i]);
            else
              h[i] = __builtin_fmaf(e[j][i], h[i], o.u[j] * o.B[j][i]);
            if (kY) y = __builtin_fmaf(o.C[j][i], h[i], y);
          }
          if (kY) sY[half][sl][4 * g + j][ch] = y;
          if (kSum || WALK == kMarks) span += o.d[j];
        }
      }
      q = next;
      half ^= 1;
      __syncthreads();
    }
    if (kSum || (WALK == kMarks && a.cut)) {
      float* to = kRev ? a.leave : a.entry;
#pragma unroll
      for (int i = 0; i < NR; ++i) to[(own + i) * CH + ch] = h[i];
      if (sl == 0) a.span[(b.slot * blocks + b.blk) * CH + ch] = span;
    }
    if (WALK == kOutputs && a.ht && p.s == p.count - 1 && mine) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (sl * NR + i < a.S) a.ht[(static_cast<int64_t>(p.n) * a.D + chan) * a.S + sl * NR + i] = h[i];
    }
    return;
  }

  // ---- inputs and outputs: this thread's part of a tile is EP channels of one row
  if (!kY) __builtin_amdgcn_s_setprio(2);
  const int tid = threadIdx.x - 64 * C::W;
  const int row = tid / (CH / EP), col = tid % (CH / EP) * EP, left = b.cols - col;
  float bias[EP], Dv[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) {
    bias[e] = a.bias && e < left ? a.bias[b.chan + col + e] : 0.f;
    Dv[e] = kY && a.Dv && e < left ? a.Dv[b.chan + col + e] : 0.f;
  }
  Row nx, ndt, nz;
  Row x0, x1, x2, z0, z1, z2;  // of the tiles whose outputs are to come
  uint32_t rB[EB], rC[EB];
  // against the tokens the writes are dy's gated and B's place is C's
  const void* px = kRev ? a.dy : a.x;
  const int64_t sx = kRev ? a.D : a.sx, sb = kRev ? a.sc : a.sb;
  // tile k in the order of the walk
  const auto first = [&](int k) { return (kRev ? tiles - 1 - k : k) * TT; };
  const auto load = [&](int k) {
    const int t0 = k < tiles ? first(k) : p.len;
    const int rows = p.len - t0 < TT ? p.len - t0 : TT;
    const int64_t at = p.begin + (rows > 0 ? t0 : 0);
    const bool ok = row < rows && left > 0;
    nx.load(rows_rsrc<IO>(px, at, sx, b.chan, rows, b.cols), ok ? static_cast<int>(row * sx + col) * ES : kOut, left, a.vec);
    ndt.load(rows_rsrc<IO>(a.dt, at, a.sdt, b.chan, rows, b.cols), ok ? static_cast<int>(row * a.sdt + col) * ES : kOut, left, a.vec);
    if ((kY || kRev) && a.z)
      nz.load(rows_rsrc<IO>(a.z, at, a.sz, b.chan, rows, b.cols), ok ? static_cast<int>(row * a.sz + col) * ES : kOut, left, a.vec);
    const rsrc_t rb = rows_rsrc<IO>(kRev ? a.Cm : a.Bm, at, sb, static_cast<int64_t>(b.g) * a.S, rows, a.S);
    const rsrc_t rc = rows_rsrc<IO>(kY ? a.Cm : a.Bm, at, kY ? a.sc : a.sb, static_cast<int64_t>(b.g) * a.S, rows, a.S);
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int t = (tid + 256 * i) / SP, n = (tid + 256 * i) % SP;
      const bool in = t < rows && n < a.S;
      ldraw<ES>(rb, in ? static_cast<int>(t * sb + n) * ES : kOut, rB + i);
      if (kY) ldraw<ES>(rc, in ? static_cast<int>(t * a.sc + n) * ES : kOut, rC + i);
    }
  };
  const auto stage = [&](int k, int q) {
    const int rows = k < tiles ? p.len - first(k) : 0;
    float d[EP], u[EP];
#pragma unroll
    for (int e = 0; e < EP; ++e) d[e] = ndt.get(e) + bias[e];
    if (a.softplus)
#pragma unroll
      for (int e = 0; e < EP; ++e) d[e] = softplus_of(d[e]);
#pragma unroll
    for (int e = 0; e < EP; ++e) {
      d[e] = row < rows ? d[e] : 0.f;
      u[e] = kRev ? nx.get(e) : d[e] * nx.get(e);
    }
    if (kRev && a.z)
#pragma unroll
      for (int e = 0; e < EP; ++e) u[e] *= silu_of<IO>(nz.get(e));
    lds_put<EP>(&sd[q][row][col], d);
    lds_put<EP>(&su[q][row][col], u);
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int j = tid + 256 * i;
      if (TT * SP % 256 == 0 || j < TT * SP) {
        sB[q][j / SP][j % SP] = dec<IO>(rB + i, 0);
        if (kY) sC[q][j / SP][j % SP] = dec<IO>(rC + i, 0);
      }
    }
  };
  const auto outputs = [&](int k, const Row& rx, const Row& rz) {
    const int rows = p.len - k * TT < TT ? p.len - k * TT : TT;
    if (row >= rows || left <= 0) return;
    float y[EP];
#pragma unroll
    for (int e = 0; e < EP; ++e) y[e] = Dv[e] * rx.get(e);
#pragma unroll
    for (int s = 0; s < NSL; ++s) lds_add<EP>(&sY[k & 1][s][row][col], y);
    if (a.z)
#pragma unroll
      for (int e = 0; e < EP; ++e) y[e] *= silu_of<IO>(rz.get(e));
    Row::store(rows_rsrc<IO>(a.y, p.begin + k * TT, a.D, b.chan, rows, b.cols),
               static_cast<int>(static_cast<int64_t>(row) * a.D + col) * ES, left, a.vec, y);
  };
  // before tile k: tiles k and k+1 lie in LDS, k+2 is on its way
  load(0);
  stage(0, 0);
  x1 = nx;
  z1 = nz;
  load(1);
  stage(1, 1);
  x2 = nx;
  z2 = nz;
  load(2);
  __syncthreads();
  int q = 2;
  for (int k = 0; k < tiles; ++k) {
    if (k + 2 < tiles) stage(k + 2, q);
    q = q == 2 ? 0 : q + 1;
    if (kY && k > 0) outputs(k - 1, x0, z0);
    x0 = x1;
    z0 = z1;
    x1 = x2;
    z1 = z2;
    x2 = nx;
    z2 = nz;
    if (k + 2 < tiles) load(k + 3);
    __syncthreads();
  }
  if (kY && tiles > 0) outputs(tiles - 1, x0, z0);
}

// entry[s], the pieces' own sums, become what enters them: R <- exp(A span_s) R + sum_s
// along a sequence's pieces (backwards: against them), from h0 (dht).  A thread takes
// N states of one channel, whose loads share the wait, and asks for the next piece's
// before it stores this one's.
template <class C, bool REV>
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs a) {
  constexpr int CH = C::CH, SP = C::SP, N = SP * CH / 256;
  static_assert(256 % CH == 0 && SP * CH % 256 == 0, "a thread's states are of one channel");
  const int blocks = scan_blocks(a.D, a.G, CH), per = a.D / a.G, nb = (per + CH - 1) / CH;
  const int n = blockIdx.x / blocks, blk = blockIdx.x - n * blocks, g = blk / nb, c0 = (blk - g * nb) * CH;
  const Seq q = sequence(a, n);
  const int first = first_slot(a, n, a.seg), count = q.len > 0 ? (q.len + a.seg - 1) / a.seg : 1;
  const float* from = REV ? a.dht : a.h0;
  float* const to = REV ? a.leave : a.entry;
  const int ch = threadIdx.x % CH;
  const int64_t chan = static_cast<int64_t>(g) * per + c0 + ch;
  float A2[N], R[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int st = (threadIdx.x + 256 * i) / CH;
    const bool ok = c0 + ch < per && st < a.S;
    A2[i] = ok ? log2_rate(a.A[chan * a.S + st]) : 0.f;
    R[i] = ok && from ? from[(static_cast<int64_t>(n) * a.D + chan) * a.S + st] : 0.f;
  }
  // the last one's own sum enters no piece and was not formed
  const auto slot = [&](int j) { return static_cast<int64_t>(first + (REV ? count - 1 - j : j)) * blocks + blk; };
  float sum[N], span = 0.f;
  const auto load = [&](int j) {
    const bool some = j < count - 1;
    const int64_t own = slot(some ? j : 0);
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = some ? to[own * SP * CH + threadIdx.x + 256 * i] : 0.f;
    span = some ? a.span[own * CH + ch] : 0.f;
  };
  load(0);
  for (int j = 0; j < count; ++j) {
    float own[N], h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) own[i] = sum[i];
    const float d = span;
    load(j + 1);
#pragma unroll
    for (int i = 0; i < N; ++i) to[slot(j) * SP * CH + threadIdx.x + 256 * i] = R[i];
    enter(d, A2, R, own, h);
#pragma unroll
    for (int i = 0; i < N; ++i) R[i] = h[i];
  }
}

// One token a sequence.  LPC lanes hold the S states of a channel, VEC each; a
// workgroup takes 256 / LPC channels of one sequence at a time.  Bound by HBM: the
// states are read and written once, in 16-byte accesses where S is a multiple of 4.
template <class IO, int VEC, bool STREAM>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a, int lpc, int groups) {
  using State = Chans<io_f32, VEC, STREAM>;
  using Token = Chans<IO, VEC, false>;
  using T = typename IO::storage;
  const int n = blockIdx.x / groups;
  const int c = ((blockIdx.x - n * groups) * 256 + threadIdx.x) / lpc;
  const int s = (threadIdx.x & (lpc - 1)) * VEC;
  if (c >= a.D) return;  // whole channels leave
  float y = 0.f, x = 0.f;
  const bool some = s < a.S;
  if (some) {
    const int64_t at = (static_cast<int64_t>(n) * a.D + c) * a.S + s;
    const int64_t group = static_cast<int64_t>(c / (a.D / a.G)) * a.S + s;
    float h[VEC], B[VEC], Cv[VEC], A2[VEC];
    State::row(a.h0, at, VEC, h);
    x = IO::load(static_cast<const T*>(a.x), n * a.sx + c);
    float d = IO::load(static_cast<const T*>(a.dt), n * a.sdt + c) + (a.bias ? a.bias[c] : 0.f);
    Token::row(a.Bm, n * a.sb + group, VEC, B);
    Token::row(a.Cm, n * a.sc + group, VEC, Cv);
#pragma unroll
    for (int i = 0; i < VEC; ++i) A2[i] = log2_rate(a.A[static_cast<int64_t>(c) * a.S + s + i]);
    if (a.softplus) d = softplus_of(d);
    const float u = d * x;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      h[i] = __builtin_fmaf(decay_by(d, A2[i]), h[i], u * B[i]);
      y = __builtin_fmaf(Cv[i], h[i], y);
    }
    State::store(a.ht, at, VEC, h);
  }
  for (int m = lpc >> 1; m >= 1; m >>= 1) y += __shfl_xor(y, m, 64);
  if (s != 0) return;
  y += (a.Dv ? a.Dv[c] : 0.f) * x;
  if (a.z) y *= silu_of<IO>(IO::load(static_cast<const T*>(a.z), n * a.sz + c));
  const __bf16 b = static_cast<__bf16>(y);
  if constexpr (sizeof(T) == 2)
    static_cast<T*>(a.y)[static_cast<int64_t>(n) * a.D + c] = __builtin_bit_cast(uint16_t, b);
  else
    static_cast<T*>(a.y)[static_cast<int64_t>(n) * a.D + c] = y;
}

struct StepShape {
  int vec, lpc, groups;  // states and lanes of a channel, workgroups of a sequence
};
StepShape step_shape(const ScanArgs& a) {
  StepShape r;
  r.vec = a.S % 4 == 0 ? 4 : 1;
  r.lpc = 1;
  while (r.lpc * r.vec < a.S) r.lpc *= 2;
  r.groups = (a.D * r.lpc + 255) / 256;
  return r;
}

template <class IO>
launch_result launch_walk(const ScanArgs& a, const ScanPlan& p, Walk walk, hipStream_t s) {
  return scan_config(p.which, [&](auto cfg) -> launch_result {
    using C = decltype(cfg);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.slots) * p.blocks));
    if (walk == kOutputs)
      hipLaunchKernelGGL((scan_walk_kernel<IO, C, kOutputs>), grid, dim3(64 * (C::W + 4)), 0, s, a);
    else if (walk == kSums)
      hipLaunchKernelGGL((scan_walk_kernel<IO, C, kSums>), grid, dim3(64 * (C::W + 4)), 0, s, a);
    else if (walk == kBack)
      hipLaunchKernelGGL((scan_walk_kernel<IO, C, kBack>), grid, dim3(64 * (C::W + 4)), 0, s, a);
    else
      hipLaunchKernelGGL((scan_walk_kernel<IO, C, kMarks>), grid, dim3(64 * (C::W + 4)), 0, s, a);
    return hipGetLastError();
  });
}
launch_result launch_walk_io(const ScanArgs& a, const ScanPlan& p, Walk walk, int32_t io_dtype, hipStream_t s) {
  return io_dtype == CKDA_DTYPE_BF16 ? launch_walk<io_bf16>(a, p, walk, s) : launch_walk<io_f32>(a, p, walk, s);
}

}  // namespace

bool scan_supported(int32_t S) { return S >= 1 && S <= 64; }

ScanPlan scan_plan(const ScanArgs& a, bool grads) {
  ScanPlan p;
  const int per = a.D / a.G;
  // Workgroups for whole sequences, of 64 channels or, past 16 states, of 32; a GPU
  // holds two a CU (of 32 channels and 16 states three), 512 at a time.
  const int wide = a.S <= 16 ? 64 : 32;
  const int64_t whole = static_cast<int64_t>(a.N) * a.G * ((per + wide - 1) / wide);
  const int64_t want = a.cu || grads ? 1024 : 512;
  // Sequences are cut where whole ones leave CUs idle, and in packed batches, whose
  // lengths are not known here.  Measured in us on sequences of 2048 tokens of 2048 channels
  // in bf16, by workgroups of whole sequences, cut and whole:
  //   forward     up to 128                            160 and more
  //    8 states   128: 106, 169                        160: 139, 169   192: 194, 170
  //   16          128: 133, 149                        160: 175, 182   192: 248, 184
  //   32           64: 70, 192     128: 122, 198       192: 225, 199
  //   64           64: 137, 284    128: 249, 287       192: 386, 289
  //   gradients   up to 341                            352 and more
  //    8 states   256: 494, 674    320: 648, 803       384: 759, 806
  //   16          256: 662, 753    320: 883, 1158      384: 1103, 1116  480: 1280, 1127
  //   32          256: 652, 841    320: 874, 1085      384: 1047, 1095  512: 1232, 1114
  //   64          192: 1088, 1125  320: 1758, 2199     384: 1921, 2206
  // One rule for all of them: it gives up a fifth at 160 workgroups and 8 states, and
  // an eighth at 384 and 64 with gradients, which cuts would have gained.
  const bool few = a.T > 256 && (a.cu || whole <= (grads ? 341 : 128));
  // 8 to 16 states of whole sequences: 32 channels a workgroup use more CUs (forward
  // of 256 workgroups of 64: 186 us, 203 with 64; of 384 245 and 276), up to where
  // they no longer fit in one round (of 416 368 and 276; gradients of 256 745 and
  // 869, of 384 1160 and 1119).
  if (a.S <= 8)
    p.which = 0;
  else if (a.S <= 16)
    p.which = !few && whole <= (grads ? 341 : 384) ? 2 : 1;
  else
    p.which = a.S <= 32 ? 3 : 4;
  p.CH = p.which <= 1 ? 64 : 32;
  p.SP = p.which == 0 ? 8 : (p.which <= 2 ? 16 : (p.which == 3 ? 32 : 64));
  p.blocks = scan_blocks(a.D, a.G, p.CH);
  p.seg = scan_whole(a.T);
  p.cut = 0;
  if (a.N > 0 && few) {
    // no more than `want` workgroups, in pieces of one length: a last round of a
    // few, or a short last piece, would leave the rest waiting (forward of 96
    // workgroups whole: 112 us in 5 pieces, 136 in 6; gradients of 160: 487 and 506)
    const int64_t own = static_cast<int64_t>(a.N) * p.blocks, pieces = want > own ? want / own : 1;
    int64_t L = a.cu ? static_cast<int64_t>(a.T) * p.blocks / want : (a.T + pieces - 1) / pieces;
    L = L < 128 ? 128 : (L + 31) / 32 * 32;
    if (L < a.T) {
      p.seg = static_cast<int>(L);
      p.cut = 1;
    }
  }
  // none in a packed batch of no sequences
  p.slots = a.N == 0 ? 0 : (a.cu ? a.T / p.seg + a.N : a.N * (a.T > 0 ? (a.T + p.seg - 1) / p.seg : 1));
  p.mslots = grads && a.N > 0 ? (a.cu ? a.T / kMark + a.N : a.N * (a.T > 0 ? (a.T + kMark - 1) / kMark : 1)) : 0;
  return p;
}

int64_t scan_step_threads(const ScanArgs& a) {
  return static_cast<int64_t>(a.N) * step_shape(a).groups * 256;
}
int64_t scan_threads(const ScanArgs& a) {
  // slots and threads in 64 bits, for narrow blocks and pieces of 128 tokens
  const int64_t blocks = static_cast<int64_t>(a.G) * ((a.D / a.G + 31) / 32);
  const int64_t slots = a.cu ? a.T / 128 + static_cast<int64_t>(a.N) : static_cast<int64_t>(a.N) * (a.T / 128 + 1);
  return slots * blocks * 768;
}

namespace {
// entry and span of the pieces, at ws; returns the bytes taken
size_t layout_pieces(ScanArgs& a, const ScanPlan& p, unsigned char* ws) {
  a.seg = p.seg;
  a.slots = p.slots;
  a.cut = p.cut;
  if (!p.cut) return 0;
  const size_t n = static_cast<size_t>(p.slots) * p.blocks * p.CH * 4;
  const size_t entry = (n * p.SP + 255) & ~size_t(255), span = (n + 255) & ~size_t(255);
  a.entry = reinterpret_cast<float*>(ws);
  a.span = reinterpret_cast<float*>(ws + entry);
  return entry + span;
}
}  // namespace

size_t scan_fwd_workspace(const ScanArgs& a0) {
  ScanArgs a = a0;
  return layout_pieces(a, scan_plan(a, false), nullptr);
}

launch_result launch_scan_join(const ScanArgs& a, const ScanPlan& p, bool rev, hipStream_t s) {
  return scan_config(p.which, [&](auto cfg) -> launch_result {
    using C = decltype(cfg);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.N) * p.blocks));
    if (rev)
      hipLaunchKernelGGL((scan_join_kernel<C, true>), grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((scan_join_kernel<C, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

launch_result launch_scan_marks(const ScanArgs& a, const ScanPlan& p, int32_t io_dtype, hipStream_t s) {
  launch_result e = launch_walk_io(a, p, kMarks, io_dtype, s);
  if (e != hipSuccess || !p.cut) return e;
  e = launch_scan_join(a, p, false, s);
  if (e == hipSuccess) e = launch_walk_io(a, p, kBack, io_dtype, s);
  return e == hipSuccess ? launch_scan_join(a, p, true, s) : e;
}

launch_result launch_scan_fwd(ScanArgs a, int32_t io_dtype, void* ws, hipStream_t s) {
  const ScanPlan p = scan_plan(a, false);
  layout_pieces(a, p, static_cast<unsigned char*>(ws));
  if (p.cut) {
    launch_result e = launch_walk_io(a, p, kSums, io_dtype, s);
    if (e == hipSuccess) e = launch_scan_join(a, p, false, s);
    if (e != hipSuccess) return e;
  }
  return launch_walk_io(a, p, kOutputs, io_dtype, s);
}

namespace {
template <class IO>
void launch_step(const ScanArgs& a, const StepShape& r, dim3 grid, hipStream_t s) {
  // States that the 256 MiB last-level cache keeps from one token to the next stay
  // cached, others are streamed: 256 sequences of 4096 channels (67 MB) 26.5 us
  // cached, 29.9 streamed; 1024 sequences (268 MB) 132 cached, 115 streamed.
  const bool stream = static_cast<int64_t>(a.N) * a.D * a.S > (int64_t(1) << 25);
  if (r.vec != 4)
    hipLaunchKernelGGL((scan_step_kernel<IO, 1, false>), grid, dim3(256), 0, s, a, r.lpc, r.groups);
  else if (stream)
    hipLaunchKernelGGL((scan_step_kernel<IO, 4, true>), grid, dim3(256), 0, s, a, r.lpc, r.groups);
  else
    hipLaunchKernelGGL((scan_step_kernel<IO, 4, false>), grid, dim3(256), 0, s, a, r.lpc, r.groups);
}
}  // namespace

launch_result launch_scan_step(const ScanArgs& a, int32_t io_dtype, hipStream_t s) {
  const StepShape r = step_shape(a);
  const dim3 grid(static_cast<unsigned>(a.N * r.groups));
  if (io_dtype == CKDA_DTYPE_BF16)
    launch_step<io_bf16>(a, r, grid, s);
  else
    launch_step<io_f32>(a, r, grid, s);
  return hipGetLastError();
}

}  // namespace ckda
