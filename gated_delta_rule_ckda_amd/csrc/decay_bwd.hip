// Gradients of the decay linear attention.  With the state S0 entering a chunk
// and the adjoint A of the state leaving it (both kept by the state passes of
// decay.hip), D_ij, E_i, W_j as in decay_ops.h, P_ij = q_i . k_j and
// N_ij = scale dout_i . v_j,
//
//   dq_i = scale E_i S0 dout_i + sum_{j <= i} D_ij N_ij k_j
//   dk_j = W_j A v_j           + sum_{i >= j} D_ij N_ij q_i
//   dv_j = W_j A^T k_j         + scale sum_{i >= j} D_ij P_ij dout_i
//
// and for the gates: a_t appears in every pair of a write before it and a read
// at or after it.  With M_ij = P_ij N_ij, z_i = scale q_i . S0 dout_i,
// y_j = k_j . A v_j and x = <A, S0>,
//
//   a_t da_t = sum_{i >= t} (E_i z_i + sum_{j < t} D_ij M_ij) + sum_{j < t} W_j y_j + g x:
//
// sums of terms that all hold the factor a_t, with nothing subtracted, so that
// dividing by it costs no accuracy.  In a chunk with gates of zero or under
// 2^-30, or products beyond 2^+-60, the factor is left out instead,
//
//   R_1(i) = z_i,  R_{t+1}(i) = a_t R_t(i) + M_it     (writes before t, read i)
//   da_t = sum_{i >= t} D_it R_t(i) + W_t X_t,   X_1 = x,  X_{t+1} = a_t X_t + y_t.
//
// A workgroup takes (chunk, query/key head) items in turn and runs over the
// value heads that share the head, summing their dq and dk in registers; a
// wave owns DP / 8 columns of dq, dk and dv for all tokens.  One workgroup
// fills a CU's LDS, so the next head's or item's rows are on their way into
// registers while one is computed.
//
// P and N rounded to the io type once each, as the states are: half a step of
// each gradient.  Measured at 8 x 4096 tokens, 16 heads of 128, bf16: 424 us
// (1.47 GB, 3.5 TB/s).  Without the loads 373 us were left of 540, without the
// products 422: LDS (half of its cycles busy, nearly half of those with bank
// conflicts: 5.4e7 of 1.1e8) and the loads share the time.
// Four waves took 900 us, loads all at once 528, stores straight from the
// accumulators 466.
#include "decay_ops.h"

namespace ckda {
namespace {

constexpr int kNT = 512;  // 8 waves
constexpr int kWaves = kNT / 64;

template <class Op, int DP, int C>
struct GradCfg {
  using T = typename Op::T;
  static constexpr int ES = sizeof(T);
  static constexpr int LD = frag_stride(DP, ES), LDC = frag_stride(C, ES), LDM = C + 1;
  static constexpr int ROWS = C * LD * ES;
  static constexpr int O_Q = 0, O_K = ROWS, O_V = 2 * ROWS, O_O = 3 * ROWS, O_A = 4 * ROWS,
                       O_P = O_A + DP * LD * ES, O_N = O_P + C * LDC * ES,
                       O_M = O_N + C * LDC * ES, O_Z = O_M + C * LDM * 4, O_Y = O_Z + kWaves * C * 4,
                       O_X = O_Y + kWaves * C * 4, O_G = align16(O_X + 2 * (C + 4) * 4),
                       BYTES = O_G + 2 * static_cast<int>(sizeof(Gates<C>));
};

template <class Op, int DP, int C>
__global__ __launch_bounds__(kNT, 2) void decay_grad_kernel(DecayArgs a, DecayGrads gr) {
  using Cfg = GradCfg<Op, DP, C>;
  using X = Fr<Op>;
  using T = typename Op::T;
  using F = typename X::F;
  constexpr int LD = Cfg::LD, LDC = Cfg::LDC, LDM = Cfg::LDM, KS = X::KS, EPP = 16 / sizeof(T);
  // tiles of 16 columns: DP / 16 of them over 8 waves (with 4, half of the waves take none)
  constexpr int RT = C / 16, ND = DP / KS, NC = C / KS, CW = DP / 16;
  static_assert(CW == 4 || CW == 8, "column tiles");
  extern __shared__ __align__(16) unsigned char smem[];
  T* sQ = reinterpret_cast<T*>(smem + Cfg::O_Q);
  T* sK = reinterpret_cast<T*>(smem + Cfg::O_K);
  T* sV = reinterpret_cast<T*>(smem + Cfg::O_V);
  T* sO = reinterpret_cast<T*>(smem + Cfg::O_O);
  T* sA = reinterpret_cast<T*>(smem + Cfg::O_A);  // adjoint state [dk][dv]
  T* sP = reinterpret_cast<T*>(smem + Cfg::O_P);  // scale D P  [i][j]
  T* sN = reinterpret_cast<T*>(smem + Cfg::O_N);  // D N        [i][j]
  float* sM = reinterpret_cast<float*>(smem + Cfg::O_M);   // D M with fast gates, else M
  float* sZ = reinterpret_cast<float*>(smem + Cfg::O_Z);   // waves' parts of z, then of da
  float* sY = reinterpret_cast<float*>(smem + Cfg::O_Y);
  float* sX = reinterpret_cast<float*>(smem + Cfg::O_X);  // gates, then x; two of them
  Gates<C>* sG = reinterpret_cast<Gates<C>*>(smem + Cfg::O_G);

  const int t = threadIdx.x, lane = t & 63, w = uniform32(t >> 6), l16 = lane & 15, lq = lane >> 4;
  const int group = a.H / a.Hk;
  const int ldq = a.Hk * a.dk, ldv = a.H * a.dv;
  const bool ckda = a.gate_range == CKDA_GATE_CKDA;
  const int nslab = (a.dv + decay_slab(a.dv) - 1) / decay_slab(a.dv);
  // with 4 column tiles, waves 4..7 take the upper half of the tokens
  const int col0 = 16 * (w % CW), n0 = CW == 8 ? 0 : (w / 4) * (RT / 2);
  constexpr int NT = CW == 8 ? RT : RT / 2;  // token tiles a wave
  const unsigned items = static_cast<unsigned>(a.cslots) * a.Hk;  // below 2^31

  // one (item, value head): where its rows are
  struct Work {
    unsigned item;
    int slot, hk, hv;
    Piece pc;
  };
  auto seek = [&](Work& k) {  // the first item at or after k.item that has tokens
    for (; k.item < items; k.item += gridDim.x) {
      k.slot = k.item / static_cast<unsigned>(a.Hk);
      k.hk = k.item - k.slot * a.Hk;
      k.pc = piece_of(a, k.slot, C, lane);
      if (k.pc.n >= 0 && k.pc.len > 0) return;
    }
  };
  auto advance = [&](Work& k) {
    if (++k.hv < group) return;
    k.hv = 0;
    k.item += gridDim.x;
    seek(k);
  };
  using R = RowTile<T, C, DP, kNT>;
  using RA = RowTile<T, DP, DP, kNT>;
  R tq, tv;
  RA ta;
  tq.init(ldq, a.dk, t);
  tv.init(ldv, a.dv, t);
  ta.init(a.dv, a.dv, t);
  int offs[ND];  // this wave's rows of the state, as operands
#pragma unroll
  for (int s = 0; s < ND; ++s) {
    const int r = col0 + l16, c = KS * s + EPP * lq;
    offs[s] = r < a.dk && c < a.dv ? (r * a.dv + c) * Cfg::ES : kNoOffset;
  }
  typename R::Regs rq, rk, rv, ro;
  typename RA::Regs ra;
  uint4 rs[ND];
  GateBits bits;
  uint32_t rx[2];  // slabs' parts of x (dv <= 128: two at most)
  // A CU takes in some 16 bytes a clock, and a load that finds its queue full
  // holds its wave: the next rows are asked for in parts, between the products.
  auto chain_of = [&](const Work& k) { return (k.item < items ? k.slot : 0) * static_cast<int64_t>(a.H) + k.hk * group + k.hv; };
  auto load_qk = [&](const Work& k) {  // nothing past the last item, in all three
    const bool in = k.item < items;
    const int rows = in ? k.pc.len : 0;
    const int64_t tok = in ? k.pc.begin : 0;
    bits = load_gate_bits(a, tok, rows, in ? k.hk * group + k.hv : 0, lane);
    const rsrc_t rd = make_rsrc(reinterpret_cast<const void*>(uniform64(reinterpret_cast<int64_t>(a.dots + (in ? chain_of(k) : 0) * nslab))),
                                uniform32(in ? 4 * nslab : 0));
    ldraw<4>(rd, 0, &rx[0]);
    ldraw<4>(rd, 4, &rx[1]);
    if (k.hv == 0) {
      const int64_t oq = tok * ldq + static_cast<int64_t>(in ? k.hk : 0) * a.dk;
      tq.load(rq, static_cast<const T*>(a.q) + oq, ldq, rows, a.dk);
      tq.load(rk, static_cast<const T*>(a.k) + oq, ldq, rows, a.dk);
    }
  };
  auto load_vo = [&](const Work& k) {
    const bool in = k.item < items;
    const int64_t ov = in ? k.pc.begin * ldv + static_cast<int64_t>(k.hk * group + k.hv) * a.dv : 0;
    tv.load(rv, static_cast<const T*>(a.v) + ov, ldv, in ? k.pc.len : 0, a.dv);
    tv.load(ro, static_cast<const T*>(gr.dout) + ov, ldv, in ? k.pc.len : 0, a.dv);
  };
  auto load_states = [&](const Work& k) {
    const bool in = k.item < items;
    const int64_t rec = (in ? chain_of(k) : 0) * a.dk * a.dv;
    ta.load(ra, static_cast<const T*>(a.adjoints) + rec, a.dv, in ? a.dk : 0, a.dv);
    const rsrc_t r = rows_rsrc(static_cast<const T*>(a.states) + rec, a.dv, in ? a.dk : 0, a.dv, DP);
#pragma unroll
    for (int s = 0; s < ND; ++s) rs[s] = load_piece(r, offs[s]);
  };

  Work cur{blockIdx.x, 0, 0, 0, {}};
  seek(cur);
  if (cur.item >= items) return;
  load_qk(cur);
  load_vo(cur);
  load_states(cur);
  // the gates of what `load` fetched last, into place b, by one wave
  auto fill = [&](const Work& k, int b) {
    const bool ok = k.item < items && lane < C && lane < k.pc.len;
    const float x = gate_of_bits(bits, a.gate_input);
    gates_fill<C>(sG[b], x, ok, a.gate_input, ckda, lane);
    if (lane < C) sX[b * (C + 4) + lane] = ok ? gate_value(x, a.gate_input, ckda) : 1.f;
    if (lane == 0) sX[b * (C + 4) + C] = __uint_as_float(rx[0]) + __uint_as_float(rx[1]);
  };
  if (w == 1) fill(cur, 0);
  f32x4 dq[NT], dk[NT];
  for (int turn = 0; cur.item < items; turn ^= 1) {
    const Gates<C>& G = sG[turn];
    const float* sAl = sX + turn * (C + 4);
    const Piece pc = cur.pc;
    const int hk = cur.hk, h = hk * group + cur.hv;
    const bool first = cur.hv == 0, last = cur.hv == group - 1;
    const bool tok = lane < C && lane < pc.len;
    const float xg = gate_of_bits(bits, a.gate_input);
    if (first) {
#pragma unroll
      for (int n = 0; n < NT; ++n) dq[n] = dk[n] = f32x4{0.f, 0.f, 0.f, 0.f};
      tq.store(rq, sQ, LD, t);
      tq.store(rk, sK, LD, t);
    }
    tv.store(rv, sV, LD, t);
    tv.store(ro, sO, LD, t);
    ta.store(ra, sA, LD, t);
    F fs[ND];
#pragma unroll
    for (int s = 0; s < ND; ++s) fs[s] = *reinterpret_cast<const F*>(&rs[s]);
    __syncthreads();
    Work next = cur;
    advance(next);
    const bool fast = G.fast != 0;

    // P^T and N^T tiles: column i = 16 ti + l16, rows j = 16 tj + 4 lq + r
    for (int tile = w; tile < RT * RT; tile += kWaves) {
      const int ti = RT - 1 - tile / RT, tj = tile % RT, i = 16 * ti + l16, j0 = 16 * tj + 4 * lq;
      f32x4 p = {0.f, 0.f, 0.f, 0.f}, n = p;
      if (tj <= ti) {
#pragma unroll
        for (int s = 0; s < ND; ++s) {
          Op::mma(p, X::row(sK + (16 * tj + l16) * LD, s, lq), X::row(sQ + i * LD, s, lq));
          Op::mma(n, X::row(sV + (16 * tj + l16) * LD, s, lq), X::row(sO + i * LD, s, lq));
        }
        const f32x4 d = decay_of(G, i, j0, fast);
        n *= a.scale;
#pragma unroll
        for (int r = 0; r < 4; ++r) sM[i * LDM + j0 + r] = fast ? (d[r] != 0.f ? p[r] * d[r] * n[r] : 0.f) : p[r] * n[r];
        p = decayed(p, d) * a.scale;
        n = decayed(n, d);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) sM[i * LDM + j0 + r] = 0.f;
      }
      Op::store4(sP + i * LDC + j0, p);
      Op::store4(sN + i * LDC + j0, n);
    }
    __syncthreads();

    load_qk(next);
    __builtin_amdgcn_sched_barrier(0);
    // dq: columns dk = col0 + 4 lq + r, token 16 n + l16
    {
      F fk[NC];
#pragma unroll
      for (int ks = 0; ks < NC; ++ks) fk[ks] = X::across(sK, LD, KS * ks, col0, lane);
#pragma unroll
      for (int nn = 0; nn < NT; ++nn) {
        const int i = 16 * (n0 + nn) + l16;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < ND; ++s) Op::mma(acc, fs[s], X::row(sO + i * LD, s, lq));
        const T* qr = sQ + i * LD + col0 + 4 * lq;
        float z = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) z += acc[r] * static_cast<float>(qr[r]);
        dq[nn] += acc * (G.E[i] * a.scale);
#pragma unroll
        for (int ks = 0; ks < NC; ++ks) Op::mma(dq[nn], fk[ks], X::rowp(sN + i * LDC, ks, lq));
        z += __shfl_xor(z, 16, 64);
        z += __shfl_xor(z, 32, 64);
        if (lq == 0) sZ[(w % CW) * C + i] = z * a.scale;
      }
    }
    load_vo(next);
    __builtin_amdgcn_sched_barrier(0);  // hoisted across, the operands spill
    // dk, token 16 n + l16
    {
      F fa[ND], fq[NC];
#pragma unroll
      for (int s = 0; s < ND; ++s) fa[s] = X::row(sA + (col0 + l16) * LD, s, lq);
#pragma unroll
      for (int ks = 0; ks < NC; ++ks) fq[ks] = X::across(sQ, LD, KS * ks, col0, lane);
#pragma unroll
      for (int nn = 0; nn < NT; ++nn) {
        const int j = 16 * (n0 + nn) + l16;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < ND; ++s) Op::mma(acc, fa[s], X::row(sV + j * LD, s, lq));
        const T* kr = sK + j * LD + col0 + 4 * lq;
        float y = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) y += acc[r] * static_cast<float>(kr[r]);
        dk[nn] += acc * G.W[j];
#pragma unroll
        for (int ks = 0; ks < NC; ++ks) Op::mma(dk[nn], fq[ks], X::across(sN, LDC, KS * ks, 16 * (n0 + nn), lane));
        y += __shfl_xor(y, 16, 64);
        y += __shfl_xor(y, 32, 64);
        if (lq == 0) sY[(w % CW) * C + j] = y;
      }
    }
    load_states(next);
    __builtin_amdgcn_sched_barrier(0);
    // dv: columns dv = col0 + 4 lq + r
    f32x4 dv[NT];
    {
      F fa[ND], fo[NC];
#pragma unroll
      for (int s = 0; s < ND; ++s) fa[s] = X::across(sA, LD, KS * s, col0, lane);
#pragma unroll
      for (int ks = 0; ks < NC; ++ks) fo[ks] = X::across(sO, LD, KS * ks, col0, lane);
#pragma unroll
      for (int nn = 0; nn < NT; ++nn) {
        const int j = 16 * (n0 + nn) + l16;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < ND; ++s) Op::mma(acc, fa[s], X::rowp(sK + j * LD, s, lq));
        acc *= G.W[j];
#pragma unroll
        for (int ks = 0; ks < NC; ++ks) Op::mma(acc, fo[ks], X::across(sP, LDC, KS * ks, 16 * (n0 + nn), lane));
        dv[nn] = acc;
      }
    }
    __syncthreads();  // z, y and M are in LDS; the rows there are done with

    // the gradients leave through LDS as whole rows
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
      const int at = (16 * (n0 + nn) + l16) * LD + col0 + 4 * lq;
      Op::store4(sV + at, dv[nn]);
      if (last) {
        Op::store4(sQ + at, dq[nn]);
        Op::store4(sK + at, dk[nn]);
      }
    }
    const int i = lane < C ? lane : C - 1;  // this lane's token, for the gates
    float da = 0.f;
    if (gr.dalpha) {
      float z = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < CW; ++k) {
        z += sZ[k * C + i];
        y += sY[k * C + i];
      }
      if (fast) {
        // wave w: reads w, w + 8, ... (lane t: the writes before t)
        const float ez = G.E[i] * z;
#pragma unroll
        for (int u = 0; u < C / kWaves; ++u) {
          const int r = w + kWaves * u;
          const float before = wave_scan(lane > 0 && lane <= C ? sM[r * LDM + lane - 1] : 0.f);
          const float e = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ez), r));
          da += lane <= r ? before + e : 0.f;
        }
        if (w == 0) {
          const float wy = __shfl_up(lane < C ? G.W[i] * y : 0.f, 1, 64);
          da += wave_scan(lane > 0 ? wy : 0.f) + G.g * sAl[C];
        }
      } else if (w == 0) {  // one gate after the other
        float Rr = z, Xr = sAl[C];
        for (int s0 = 0; s0 < C; s0 += 4) {
          const f32x4 d = decay_of(G, i, s0, false);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int s = s0 + e;
            const float al = sAl[s], ys = __shfl(y, s, 64), m = sM[i * LDM + s];
            sM[i * LDM + s] = d[e] != 0.f ? d[e] * Rr : 0.f;  // past the diagonal: 0
            Rr = al * Rr + m;
            da = s == i ? G.W[s] * Xr : da;
            Xr = al * Xr + ys;
          }
        }
        wave_lds_sync();
        for (int r = i; r < C; ++r) da += sM[r * LDM + i];
      }
    }
    __syncthreads();  // the gradients are in LDS; z is read: its place takes the waves' parts of da
    auto flush = [&](const T* from, const R& tile, void* to, int64_t at, int ld, int cols) {
      const rsrc_t r = rows_rsrc(static_cast<const T*>(to) + at, ld, pc.len, cols, C);
#pragma unroll
      for (int u = 0; u < R::NP; ++u) {
        const int p = t + kNT * u;
        store_piece(r, tile.off[u], *reinterpret_cast<const uint4*>(from + (p / R::PPR) * LD + (p % R::PPR) * R::EPP));
      }
    };
    flush(sV, tv, gr.dv, pc.begin * ldv + static_cast<int64_t>(h) * a.dv, ldv, a.dv);
    if (last) {
      const int64_t oq = pc.begin * ldq + static_cast<int64_t>(hk) * a.dk;
      flush(sQ, tq, gr.dq, oq, ldq, a.dk);
      flush(sK, tq, gr.dk, oq, ldq, a.dk);
    }
    if (gr.dalpha) {
      if (fast && lane < C) sZ[w * C + lane] = da;
      __syncthreads();
      if (w == 0) {
        if (fast) {
          da = 0.f;
#pragma unroll
          for (int k = 0; k < kWaves; ++k) da += sZ[k * C + i];
          da *= 1.f / sAl[i];
        }
        if (tok) {
          if (a.gate_input != CKDA_GATES_F32) {
            const float e = expf(-fabsf(xg));
            da *= (ckda ? 2.f : 1.f) * e / ((1.f + e) * (1.f + e));
          }
          const int64_t at = (pc.begin + lane) * a.H + h;
          if (a.per_head)
            gr.per_token[at] = da;
          else
            static_cast<T*>(gr.dalpha)[at] = static_cast<T>(da);
        }
      }
    }
    if (w == 1) fill(next, turn ^ 1);
    __syncthreads();  // LDS is free; the next gates are there
    cur = next;
  }
}

// dalpha [H] from the tokens' gradients, in a fixed order: thread t of a
// head's workgroup takes tokens t, t + 1024, ..., then a tree over threads.
// Without sequences there is nothing to read: zeros.
template <class IO>
__global__ __launch_bounds__(1024) void decay_gate_sum_kernel(DecayArgs a, const float* per_token,
                                                             void* dalpha) {
  __shared__ float part[16];
  const int h = blockIdx.x, t = threadIdx.x;
  const int64_t n = a.N == 0 ? 0 : a.cu ? cu_at(a, a.N) : static_cast<int64_t>(a.B) * a.T;
  float s = 0.f;
  for (int64_t i = t; i < n; i += 1024) s += per_token[i * a.H + h];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
  if ((t & 63) == 0) part[t >> 6] = s;
  __syncthreads();
  if (t == 0) {
    for (int i = 1; i < 16; ++i) s += part[i];
    using T = typename IO::storage;
    IO::store(static_cast<T*>(dalpha), h, s);
  }
}

template <class Op, int DP, int C>
launch_result launch_grad_t(const DecayArgs& a, const DecayGrads& g, hipStream_t s) {
  constexpr int lds = GradCfg<Op, DP, C>::BYTES;
  static_assert(lds <= 160 * 1024, "LDS of a CU");
  const launch_result e = allow_lds<decay_grad_kernel<Op, DP, C>>(lds);
  if (e != hipSuccess) return e;
  // as many workgroups as are resident on 256 CUs, each taking items in turn
  const int64_t items = static_cast<int64_t>(a.cslots) * a.Hk, most = 256 * (160 * 1024 / lds < 2 ? 1 : 2);
  const int64_t grid = items < most ? items : most;
  hipLaunchKernelGGL((decay_grad_kernel<Op, DP, C>), dim3(static_cast<unsigned>(grid)), dim3(kNT), lds, s,
                     a, g);
  return hipGetLastError();
}

launch_result launch_gate_sum(const DecayArgs& a, const DecayGrads& g, int32_t io_dtype, hipStream_t s) {
  if (io_dtype == CKDA_DTYPE_BF16)
    hipLaunchKernelGGL(decay_gate_sum_kernel<io_bf16>, dim3(a.H), dim3(1024), 0, s, a, g.per_token, g.dalpha);
  else
    hipLaunchKernelGGL(decay_gate_sum_kernel<io_f32>, dim3(a.H), dim3(1024), 0, s, a, g.per_token, g.dalpha);
  return hipGetLastError();
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: segments' records (used forwards, then again backwards), then
// the chunks' states, adjoints and partial dots, then the tokens' gate
// gradients of a head's one gate.
size_t lay_out(DecayArgs& a, DecayGrads& g, int32_t io_dtype, unsigned char* ws) {
  size_t off = up256(decay_layout_segments(a, ws));
  const int C = decay_bwd_chunk(io_dtype);
  const size_t es = io_dtype == CKDA_DTYPE_BF16 ? 2 : 4;
  a.cslots = static_cast<int32_t>(decay_slots(a, C));
  const size_t chains = static_cast<size_t>(a.cslots) * a.H;
  a.states = ws + off;
  off += up256(chains * a.dk * a.dv * es);
  a.adjoints = ws + off;
  off += up256(chains * a.dk * a.dv * es);
  a.dots = reinterpret_cast<float*>(ws + off);
  off += up256(chains * decay_dots_per_chunk(a.dv) * 4);
  g.per_token = reinterpret_cast<float*>(ws + off);
  if (a.per_head) off += up256(static_cast<size_t>(a.B) * a.T * a.H * 4);
  return off;
}

}  // namespace

size_t decay_bwd_workspace(const DecayArgs& a, int32_t io_dtype) {
  DecayArgs b = a;
  DecayGrads g{};
  return lay_out(b, g, io_dtype, nullptr);
}

launch_result launch_decay_bwd(const DecayArgs& a, DecayGrads g, int32_t io_dtype, void* ws,
                               hipStream_t s) {
  if (a.N == 0)  // one gate a head still has its gradient, a sum over no tokens
    return g.dalpha && a.per_head ? launch_gate_sum(a, g, io_dtype, s) : hipSuccess;
  DecayArgs f = a;
  lay_out(f, g, io_dtype, static_cast<unsigned char*>(ws));
  f.ht = nullptr;
  launch_result e = launch_decay_segments(f, io_dtype, false, s);
  if (e != hipSuccess) return e;
  if ((e = launch_decay_chunks(f, io_dtype, false, s)) != hipSuccess) return e;
  DecayArgs r = f;
  r.h0 = g.dht;
  r.ht = g.dh0;
  r.o = const_cast<void*>(g.dout);
  if ((e = launch_decay_segments(r, io_dtype, true, s)) != hipSuccess) return e;
  if ((e = launch_decay_chunks(r, io_dtype, true, s)) != hipSuccess) return e;
  constexpr int CB = decay_bwd_chunk(CKDA_DTYPE_BF16), CF = decay_bwd_chunk(CKDA_DTYPE_F32);
  const bool wide = a.dk > 64 || a.dv > 64;
  if (io_dtype == CKDA_DTYPE_BF16)
    e = wide ? launch_grad_t<OpBF16, 128, CB>(f, g, s) : launch_grad_t<OpBF16, 64, CB>(f, g, s);
  else
    e = wide ? launch_grad_t<OpF32, 128, CF>(f, g, s) : launch_grad_t<OpF32, 64, CF>(f, g, s);
  if (e != hipSuccess || !g.dalpha || !a.per_head) return e;
  return launch_gate_sum(f, g, io_dtype, s);
}

}  // namespace ckda
