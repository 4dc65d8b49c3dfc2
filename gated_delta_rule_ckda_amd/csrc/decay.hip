// Decay linear attention: the chunked forward, the state passes that the
// backward and long prompts run, and the single-token step.
//
//     S_t = a_t S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t
#include <type_traits>

#include "decay_ops.h"

namespace ckda {
namespace {

constexpr int kNT = 256;  // of the join

// ---- forward -------------------------------------------------------------------
// One workgroup walks one (segment, head) over its chunks for DVS columns of
// the state; per chunk
//
//   P^T = K Q^T
//   O^T = E S^T Q^T + V^T (D P)^T
//   S   = g S + K^T (W V)
//
// Four waves read out (wave w: the 16 tokens 16w.. of Q, all DVS columns); four
// for every 32 columns keep the state (DKP/4 rows each, in the matrix
// accumulators, in float32) and bring K and V in.  The two kinds run side by
// side on one chunk, since the read-out takes the state from before it, and
// everything they hand on in LDS (K, V, W V, a copy of S in the io type) is
// held twice, so that a chunk's step has one barrier: with one copy the
// hand-over itself, between two barriers, took as long as the products.  P^T
// leaves the accumulators as the next product's operand (each term rounded
// once to the io type, as the copy of S is: half a step of o each).
//
// Measured at 8 x 4096 tokens, 16 heads of 128, bf16: 150 us, 3.6 TB/s of the
// bytes it cannot do without, each read from HBM once (411 MB fetched of 402).
// Without the loads it takes 119 us, without the products 131: LDS (58% of its
// cycles busy) bounds the one, what a CU takes in (16 to 22 bytes a clock, q and
// k once a slab) the other, and the two overlap in part.  Nearly half of the LDS
// cycles are bank conflicts (2.6e7 of 5.4e7): by a model of 64 banks those of
// the reads across rows of W V (2 ways) and, columns 16 apart, of V (4 ways),
// whose rows lie 16 bytes past a multiple of 128; K, Q and P have none.  Half
// as many state waves with twice the rows each read W V less but take as long
// (152 us).
// Earlier forms: one role and two barriers 246 us, two roles 207, rows loaded
// two chunks ahead 187, slabs of 64 columns 155.
template <class Op, int DKP, int DVS>
struct FwdCfg {
  using T = typename Op::T;
  static constexpr int C = kDecayChunk, ES = sizeof(T), NU = DVS / 8, NT = 64 * (4 + NU);
  static constexpr int LDK = frag_stride(DKP, ES), LDV = cross_stride(DVS, ES), LDS = DKP + 16 / ES;
  static constexpr int NV = 1 + Fr<Op>::kTerms;  // V, then the terms of W V
  static constexpr int KB = C * LDK * ES, VB = NV * C * LDV * ES, SB = DVS * LDS * ES;
  static constexpr int O_K = 0, O_V = O_K + 2 * KB, O_S = O_V + 2 * VB, O_G = align16(O_S + 2 * SB),
                       BYTES = O_G + 8 * static_cast<int>(sizeof(Gates<C>));
  static_assert(BYTES <= 160 * 1024, "LDS of a CU");
};

template <class Op, int DKP, int DVS>
__global__ __launch_bounds__((FwdCfg<Op, DKP, DVS>::NT)) void decay_fwd_kernel(DecayArgs a) {
  using Cfg = FwdCfg<Op, DKP, DVS>;
  using X = Fr<Op>;
  using T = typename Op::T;
  using F = typename X::F;
  constexpr int C = Cfg::C, LDK = Cfg::LDK, LDV = Cfg::LDV, KS = X::KS, NW = 64 * Cfg::NU;
  constexpr int NQ = DKP / KS, MT = DKP / 64, NTO = DVS / 16, NTS = 2, EPP = 16 / sizeof(T);
  extern __shared__ __align__(16) unsigned char smem[];
  // by the chunk's parity
  auto sK = [&](int c) { return reinterpret_cast<T*>(smem + Cfg::O_K + (c & 1) * Cfg::KB); };
  auto sV = [&](int c) { return reinterpret_cast<T*>(smem + Cfg::O_V + (c & 1) * Cfg::VB); };
  auto sS = [&](int c) { return reinterpret_cast<T*>(smem + Cfg::O_S + (c & 1) * Cfg::SB); };
  Gates<C>* sG = reinterpret_cast<Gates<C>*>(smem + Cfg::O_G);

  const int lane = threadIdx.x & 63, l16 = lane & 15, lq = lane >> 4;
  const int wave = uniform32(threadIdx.x >> 6);
  const int nslab = (a.dv + DVS - 1) / DVS;
  int64_t chain;
  int slab;
  item_of(blockIdx.x, gridDim.x, nslab, chain, slab);
  const int slot = static_cast<int>(chain / a.H), h = static_cast<int>(chain % a.H);
  Piece pc;
  if (a.seg > 0) {
    pc = piece_of(a, slot, a.seg, lane);
    if (pc.n < 0) return;
  } else {
    const Seq s = sequence(a, slot);
    pc = Piece{slot, 0, 1, s.begin, s.len};
  }
  const int hk = h / (a.H / a.Hk), c0 = slab * DVS;
  const int vcols = a.dv - c0 < DVS ? a.dv - c0 : DVS;
  const int ldq = a.Hk * a.dk, ldv = a.H * a.dv;
  const int64_t oq = pc.begin * ldq + static_cast<int64_t>(hk) * a.dk;
  const int64_t ov = pc.begin * ldv + static_cast<int64_t>(h) * a.dv + c0;
  const int nch = (pc.len + C - 1) / C;
  auto first_token = [&](int c) { return static_cast<int64_t>(c) * C; };  // past the end: nothing is read there

  if (wave < 4) {  // ---- read-out
    const int w = wave, r = 16 * w + l16;  // this lane's token
    T* go = static_cast<T*>(a.o) + ov;
    // tile n of the output holds, in lane (l16, lq), columns RUN lq + 4 n + i of
    // token l16: RUN columns in a row
    constexpr int RUN = 4 * NTO;
    int offo[RUN / EPP];
#pragma unroll
    for (int u = 0; u < RUN / EPP; ++u) {
      const int col = RUN * lq + EPP * u;
      offo[u] = col < vcols ? (r * ldv + col) * Cfg::ES : kNoOffset;
    }
    const T* gq = static_cast<const T*>(a.q) + oq;
    uint4 rq[NQ];
    int offq[NQ];
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      const int col = KS * s + EPP * lq;
      offq[s] = col < a.dk ? (r * ldq + col) * Cfg::ES : kNoOffset;
    }
    auto load = [&](int c) {
      const rsrc_t rs = rows_rsrc(gq + first_token(c) * ldq, ldq, pc.len - c * C, a.dk, C);
#pragma unroll
      for (int s = 0; s < NQ; ++s) rq[s] = load_piece(rs, offq[s]);
    };
    if (nch > 0) {
      load(0);
      __syncthreads();
    }
    for (int c = 0; c < nch; ++c) {
      __syncthreads();  // rows, state copy and gates of chunk c are in LDS
      const Gates<C>& G = sG[c & 7];
      const bool fast = G.fast != 0;
      const T *tK = sK(c), *tV = sV(c), *tS = sS(c);
      F fq[NQ];
#pragma unroll
      for (int s = 0; s < NQ; ++s) fq[s] = *reinterpret_cast<const F*>(&rq[s]);
      f32x4 p[C / 16];
#pragma unroll
      for (int j = 0; j < C / 16; ++j) p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto tile_pair = [&](auto J) {
        constexpr int j0 = decltype(J)::value;
#pragma unroll
        for (int j = j0; j < j0 + 2; ++j) {
          const T* rowk = tK + (16 * j + l16) * LDK;
#pragma unroll
          for (int s = 0; s < NQ; ++s) Op::mma(p[j], X::row(rowk, s, lq), fq[s]);
        }
      };
      tile_pair(std::integral_constant<int, 0>{});
      if (w >= 2) tile_pair(std::integral_constant<int, 2>{});
      f32x4 o[NTO], x[NTO];
#pragma unroll
      for (int n = 0; n < NTO; ++n) {
        o[n] = x[n] = f32x4{0.f, 0.f, 0.f, 0.f};
        const T* rows = tS + (RUN * (l16 >> 2) + 4 * n + (l16 & 3)) * Cfg::LDS;
#pragma unroll
        for (int s = 0; s < NQ; ++s) Op::mma(x[n], X::row(rows, s, lq), fq[s]);
      }
      load(c + 1);
      // where D factors, its row part multiplies the sum instead of each term
      float row = 1.f;
      if (fast) {
        row = G.u[r];
#pragma unroll
        for (int j = 0; j < C / 16; ++j) {
          p[j] *= *reinterpret_cast<const f32x4*>(&G.v[16 * j + 4 * lq]);
          if (j >= w) {  // this wave's diagonal tile, or past it
#pragma unroll
            for (int i = 0; i < 4; ++i) p[j][i] = 16 * j + 4 * lq + i <= r ? p[j][i] : 0.f;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < C / 16; ++j) p[j] = decayed(p[j], decay_of(G, r, 16 * j + 4 * lq, false));
      }
      F pf[C / KS];
      Op::template frags<C>(pf, p);
#pragma unroll
      for (int ks = 0; ks < C / KS; ++ks)
        if (2 * ks < C / KS || w >= 2) {
#pragma unroll
          for (int n = 0; n < NTO; ++n) Op::mma(o[n], X::across(tV, LDV, KS * ks, 4 * n, lane, RUN), pf[ks]);
        }
      const float e = G.E[r] * a.scale;
      row *= a.scale;
      const rsrc_t ro = rows_rsrc(go + first_token(c) * ldv, ldv, pc.len - c * C, vcols, C);
      alignas(16) T y[RUN];
#pragma unroll
      for (int n = 0; n < NTO; ++n) Op::store4(y + 4 * n, x[n] * e + o[n] * row);
#pragma unroll
      for (int u = 0; u < RUN / EPP; ++u) store_piece(ro, offo[u], *reinterpret_cast<const uint4*>(y + EPP * u));
    }
    return;
  }

  // ---- state tile (m, n): rows dk = row0 + 16 m + 4 lq + i, column c0 + colw + 16 n + l16
  const int w = (wave - 4) & 3, t = threadIdx.x - 256;
  const int row0 = w * (DKP / 4), colw = 32 * ((wave - 4) >> 2);
  const int64_t sbase = (static_cast<int64_t>(pc.n) * a.H + h) * a.dk * a.dv;
  f32x4 S[MT][NTS];
  auto each = [&](auto f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NTS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = row0 + 16 * m + 4 * lq + i, c = colw + 16 * n + l16;
          f(S[m][n], i, r < a.dk && c < vcols, static_cast<int64_t>(r) * a.dv + c0 + c);
        }
  };
  const float* src = a.seg > 0 ? a.entry + (static_cast<int64_t>(slot) * a.H + h) * a.dk * a.dv
                               : (a.h0 ? a.h0 + sbase : nullptr);
  each([&](f32x4& x, int i, bool in, int64_t at) { x[i] = src && in ? src[at] : 0.f; });
  auto stage_state = [&](int c) {  // as chunk c meets it
    T* dst = sS(c) + (colw + l16) * Cfg::LDS + row0 + 4 * lq;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NTS; ++n) Op::store4(dst + 16 * n * Cfg::LDS + 16 * m, S[m][n]);
  };
  const bool ckda = a.gate_range == CKDA_GATE_CKDA;
  const T* gk = static_cast<const T*>(a.k) + oq;
  const T* gv = static_cast<const T*>(a.v) + ov;
  using RK = RowTile<T, C, DKP, NW>;
  using RV = RowTile<T, C, DVS, NW>;
  RK tk;
  RV tv;
  tk.init(ldq, a.dk, t);
  tv.init(ldv, vcols, t);
  // Rows wait in registers for two chunks; the loop takes two a turn, so that
  // the registers are fixed.
  typename RK::Regs rk[2];
  typename RV::Regs rv[2];
  auto load = [&](auto P, int c) {
    constexpr int b = decltype(P)::value;
    const int rows = pc.len - c * C;
    tv.load(rv[b], gv + first_token(c) * ldv, ldv, rows, vcols);
    tk.load(rk[b], gk + first_token(c) * ldq, ldq, rows, a.dk);
  };
  // Gates four chunks at a time, one a wave: formed one after the other they
  // were the longest part of a chunk's step.
  GateBits bits;
  auto load_gates = [&](int c) {
    const int cw = c + w;
    bits = load_gate_bits(a, pc.begin + first_token(cw), pc.len - cw * C, h, lane);
  };
  auto fill_gates = [&](int c) {
    const int cw = c + w;
    if (colw == 0)
      gates_fill<C>(sG[cw & 7], gate_of_bits(bits, a.gate_input), cw * C + lane < pc.len, a.gate_input, ckda, lane);
  };
  auto stage_rows = [&](auto P, int c) {
    constexpr int b = decltype(P)::value;
    T* dst = sV(c);
    const Gates<C>& G = sG[c & 7];
    tv.store(rv[b], dst, LDV, t);
#pragma unroll
    for (int u = 0; u < RV::NP; ++u) {
      const int p = t + NW * u, row = p / RV::PPR, col = (p % RV::PPR) * RV::EPP;
      store_scaled<T>(rv[b].r[u], G.W[row], dst + C * LDV + row * LDV + col, C * LDV);
    }
    tk.store(rk[b], sK(c), LDK, t);
  };
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;
  // chunk c, whose rows were in registers P and are in LDS now
  auto step = [&](auto P, auto Q, int c) {
    __syncthreads();  // rows, state copy and gates of chunk c are in LDS
    const float g = sG[c & 7].g;
    const T *tK = sK(c), *tH = sV(c) + C * LDV;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NTS; ++n) S[m][n] *= g;
#pragma unroll
    for (int ks = 0; ks < C / KS; ++ks) {
      F ka[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) ka[m] = X::across(tK, LDK, KS * ks, row0 + 16 * m, lane);
#pragma unroll
      for (int p = 0; p < X::kTerms; ++p)
#pragma unroll
        for (int n = 0; n < NTS; ++n) {
          const F vb = X::across(tH + p * C * LDV, LDV, KS * ks, colw + 16 * n, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m) Op::mma(S[m][n], ka[m], vb);
        }
    }
    load(P, c + 2);
    stage_state(c + 1);
    stage_rows(Q, c + 1);
    if ((c & 3) == 0) load_gates(c + 4);
    if ((c & 3) == 2) fill_gates(c + 2);  // ready when chunk c + 2 is staged, a barrier on
  };
  if (nch > 0) {
    load_gates(0);
    load(P0{}, 0);
    load(P1{}, 1);
    fill_gates(0);
    stage_state(0);
    __syncthreads();
    stage_rows(P0{}, 0);
  }
  int c = 0;
  for (; c + 1 < nch; c += 2) {
    step(P0{}, P1{}, c);
    step(P1{}, P0{}, c + 1);
  }
  if (c < nch) step(P0{}, P1{}, c);
  if (a.ht && pc.s == pc.count - 1) {
    float* dst = a.ht + sbase;
    each([&](const f32x4& x, int i, bool in, int64_t at) {
      if (in) dst[at] = x[i];
    });
  }
}

// ---- state passes ---------------------------------------------------------------
// The same walk without the read-out, in either direction:
//   forward    S <- g S + sum_j k_j (W_j v_j)^T,              x = k, y = v
//   backwards  S <- g S + sum_i q_i (scale E_i dout_i)^T,     x = q, y = dout,
// over the chunks from the last to the first.  kSegment starts from zero and
// leaves a segment's own sum and gate product (joined by decay_join_kernel);
// kChunks starts from the segment's entry and keeps the state met at every
// chunk in the io type (backwards with its product with the forward's one),
// and the state at the end of the walk in float32.
//
// Measured at 8 x 4096 tokens, 16 heads of 128, bf16: kChunks 135 us forward
// (4.0 TB/s of k, v and the states) and 198 backwards (4.1 TB/s of q, dout, the
// adjoints and the forward's states).  kSegment over 15/16 of 65536 tokens, 16
// heads: 168 us with all 128 columns and 64 x 32 a wave, 197 with 32 x 32, 207
// in slabs of 64 columns; with one of the three terms of W V a third less, so
// the reads of those terms from LDS bound it, bank conflicts among them (in
// kChunks 1.3e7 of 2.7e7 LDS cycles; the 128 columns of kSegment conflict more).
enum { kSegment = 0, kChunks = 1 };

template <class Op, int DKP, int DVS, int C>
struct StateCfg {
  using T = typename Op::T;
  // WK waves for every 32 columns, each with DKP / WK rows: fewer where all
  // columns are here, since each reads its columns' terms of the whole chunk
  static constexpr int ES = sizeof(T), WK = DVS == 128 ? 2 : 4, NT = 64 * WK * (DVS / 32);
  static constexpr int LDK = frag_stride(DKP, ES), LDV = cross_stride(DVS, ES);
  static constexpr int KB = C * LDK * ES, VB = Fr<Op>::kTerms * C * LDV * ES;
  static constexpr int O_K = 0, O_H = O_K + 2 * KB, O_G = align16(O_H + 2 * VB),
                       O_R = O_G + 8 * static_cast<int>(sizeof(Gates<C>)), BYTES = O_R + 2 * 16 * 4;
};

template <class Op, int DKP, int DVS, int C, bool REV, int MODE>
__global__ __launch_bounds__((StateCfg<Op, DKP, DVS, C>::NT)) void decay_state_kernel(DecayArgs a) {
  using Cfg = StateCfg<Op, DKP, DVS, C>;
  using X = Fr<Op>;
  using T = typename Op::T;
  using F = typename X::F;
  constexpr int LDK = Cfg::LDK, LDV = Cfg::LDV, KS = X::KS, MT = DKP / 16 / Cfg::WK, NTL = 2, NT = Cfg::NT;
  extern __shared__ __align__(16) unsigned char smem[];
  auto sK = [&](int i) { return reinterpret_cast<T*>(smem + Cfg::O_K + (i & 1) * Cfg::KB); };
  auto sH = [&](int i) { return reinterpret_cast<T*>(smem + Cfg::O_H + (i & 1) * Cfg::VB); };
  Gates<C>* sG = reinterpret_cast<Gates<C>*>(smem + Cfg::O_G);
  float* sR = reinterpret_cast<float*>(smem + Cfg::O_R);

  const int t = threadIdx.x, lane = t & 63, wave = uniform32(t >> 6), w = wave & 3, l16 = lane & 15, lq = lane >> 4;
  const int nslab = (a.dv + DVS - 1) / DVS;
  int64_t chain;
  int slab;
  item_of(blockIdx.x, gridDim.x, nslab, chain, slab);
  const int slot = static_cast<int>(chain / a.H), h = static_cast<int>(chain % a.H);
  Piece pc;
  if (a.seg > 0) {
    pc = piece_of(a, slot, a.seg, lane);
    if (pc.n < 0) return;
  } else {
    const Seq s = sequence(a, slot);
    pc = Piece{slot, 0, 1, s.begin, s.len};
  }
  // nobody enters a state after the walk's last segment
  if (MODE == kSegment && pc.s == (REV ? 0 : pc.count - 1)) return;
  const int hk = h / (a.H / a.Hk), c0 = slab * DVS;
  const int vcols = a.dv - c0 < DVS ? a.dv - c0 : DVS;
  const int ldx = a.Hk * a.dk, ldy = a.H * a.dv;
  const T* gx = static_cast<const T*>(REV ? a.q : a.k) + pc.begin * ldx + static_cast<int64_t>(hk) * a.dk;
  const T* gy = static_cast<const T*>(REV ? a.o : a.v) + pc.begin * ldy + static_cast<int64_t>(h) * a.dv + c0;
  const bool ckda = a.gate_range == CKDA_GATE_CKDA;
  const int nch = (pc.len + C - 1) / C;

  // tile (m, n) of S^T: column dk = row0 + 16 m + l16, rows dv = c0 + colw +
  // RUN lq + 4 n + i: a lane holds RUN columns of the state in a row
  constexpr int RUN = 4 * NTL;
  const int row0 = (wave % Cfg::WK) * (DKP / Cfg::WK), colw = 32 * (wave / Cfg::WK);
  const int64_t seq_state = (static_cast<int64_t>(pc.n) * a.H + h) * a.dk * a.dv;
  const int64_t seg_state = (static_cast<int64_t>(slot) * a.H + h) * a.dk * a.dv;
  f32x4 S[MT][NTL];
  // place of S[m][n] in a state, -1 outside it
  auto place = [&](int m, int n) {
    const int r = row0 + 16 * m + l16, c = colw + RUN * lq + 4 * n;
    return r < a.dk && c < vcols ? r * a.dv + c0 + c : -1;
  };
  const float* src = MODE == kSegment ? nullptr
                     : (a.seg > 0 ? a.entry + seg_state : (a.h0 ? a.h0 + seq_state : nullptr));
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NTL; ++n) {
      const int at = place(m, n);
      S[m][n] = src && at >= 0 ? *reinterpret_cast<const f32x4*>(src + at) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  auto save = [&](float* dst) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NTL; ++n) {
        const int at = place(m, n);
        if (at >= 0) *reinterpret_cast<f32x4*>(dst + at) = S[m][n];
      }
  };

  using RX = RowTile<T, C, DKP, NT>;
  using RY = RowTile<T, C, DVS, NT>;
  RX tx;
  RY ty;
  tx.init(ldx, a.dk, t);
  ty.init(ldy, vcols, t);
  // rows wait in registers two chunks ahead; the loop takes two chunks a turn
  typename RX::Regs rx[2];
  typename RY::Regs ry[2];
  uint4 rf[2][MT][RUN * sizeof(T) / 16];  // backwards: the forward's state at the chunk
  int64_t cslot = 0;
  if (MODE == kChunks) cslot = first_slot(a, pc.n, C) + (a.seg > 0 ? pc.s * (a.seg / C) : 0);
  auto chunk_at = [&](int i) { return REV ? nch - 1 - i : i; };
  auto rows_at = [&](int i) {  // none past the last
    const int left = REV ? min(pc.len - (nch - 1 - i) * C, C) : pc.len - i * C;
    return i < nch ? left : 0;
  };
  auto record = [&](int i) { return ((cslot + chunk_at(i)) * a.H + h) * a.dk * a.dv; };
  auto load_chunk = [&](auto P, int i) {  // zeros past the last
    constexpr int b = decltype(P)::value;
    const int rows = rows_at(i);
    const int64_t o = static_cast<int64_t>(chunk_at(i)) * C;
    tx.load(rx[b], gx + o * ldx, ldx, rows, a.dk);
    ty.load(ry[b], gy + o * ldy, ldy, rows, vcols);
    if constexpr (REV && MODE == kChunks) {
      const T* fwd = static_cast<const T*>(a.states) + record(i);
      const rsrc_t r = rows_rsrc(fwd, a.dv, i < nch ? a.dk : 0, a.dv, DKP);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int u = 0; u < RUN * static_cast<int>(sizeof(T)) / 16; ++u) {
          const int at = place(m, u * (4 / static_cast<int>(sizeof(T))));
          rf[b][m][u] = load_piece(r, at >= 0 ? at * static_cast<int>(sizeof(T)) : kNoOffset);
        }
    }
  };
  GateBits bits;  // gates four chunks at a time, one a wave
  auto load_gates = [&](int i) {
    const int iw = i + w;
    bits = load_gate_bits(a, pc.begin + static_cast<int64_t>(chunk_at(iw)) * C, min(rows_at(iw), C), h, lane);
  };
  auto fill_gates = [&](int i) {
    const int iw = i + w;
    const bool ok = iw < nch && lane < C && chunk_at(iw) * C + lane < pc.len;
    if (wave < 4) gates_fill<C>(sG[iw & 7], gate_of_bits(bits, a.gate_input), ok, a.gate_input, ckda, lane);
  };
  auto stage_rows = [&](auto P, int i) {
    constexpr int b = decltype(P)::value;
    const Gates<C>& G = sG[i & 7];
#pragma unroll
    for (int u = 0; u < RY::NP; ++u) {
      const int p = t + NT * u, row = p / RY::PPR, c = (p % RY::PPR) * RY::EPP;
      store_scaled<T>(ry[b].r[u], REV ? G.E[row] * a.scale : G.W[row], sH(i) + row * LDV + c, C * LDV);
    }
    tx.store(rx[b], sK(i), LDK, t);
  };
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;

  float gain = 1.f;
  auto step = [&](auto P, auto Q, int i) {
    if (MODE == kChunks) {  // the state met at this chunk
      const rsrc_t dst = rows_rsrc(static_cast<const T*>(REV ? a.adjoints : a.states) + record(i), a.dv, a.dk, a.dv, DKP);
      float dot = 0.f;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        alignas(16) T y[RUN];
#pragma unroll
        for (int n = 0; n < NTL; ++n) Op::store4(y + 4 * n, S[m][n]);
#pragma unroll
        for (int u = 0; u < RUN * static_cast<int>(sizeof(T)) / 16; ++u) {
          const int at = place(m, u * (4 / static_cast<int>(sizeof(T))));
          store_piece(dst, at >= 0 ? at * static_cast<int>(sizeof(T)) : kNoOffset, reinterpret_cast<const uint4*>(y)[u]);
          if (REV) {
            constexpr int E = 16 / sizeof(T);
#pragma unroll
            for (int e = 0; e < E; ++e)
              dot += S[m][(u * E + e) / 4][(u * E + e) % 4] * piece_elem<T>(rf[decltype(P)::value][m][u], e);
          }
        }
      }
      if (REV) {
#pragma unroll
        for (int mm = 32; mm >= 1; mm >>= 1) dot += __shfl_xor(dot, mm, 64);
        if (lane == 0) sR[16 * (i & 1) + wave] = dot;
      }
    }
    __syncthreads();  // rows and gates of chunk i are in LDS
    if (MODE == kChunks && REV && t == 0) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < NT / 64; ++k) x += sR[16 * (i & 1) + k];
      a.dots[((cslot + chunk_at(i)) * a.H + h) * nslab + slab] = x;
    }
    const float g = sG[i & 7].g;
    gain *= g;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NTL; ++n) S[m][n] *= g;
#pragma unroll
    for (int ks = 0; ks < C / KS; ++ks) {
      F ka[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) ka[m] = X::across(sK(i), LDK, KS * ks, row0 + 16 * m, lane);
#pragma unroll
      for (int p = 0; p < X::kTerms; ++p)
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          const F vb = X::across(sH(i) + p * C * LDV, LDV, KS * ks, colw + 4 * n, lane, RUN);
#pragma unroll
          for (int m = 0; m < MT; ++m) Op::mma(S[m][n], vb, ka[m]);
        }
    }
    load_chunk(P, i + 2);
    stage_rows(Q, i + 1);
    if ((i & 3) == 0) load_gates(i + 4);
    if ((i & 3) == 2) fill_gates(i + 2);
  };
  if (nch > 0) {
    load_gates(0);
    load_chunk(P0{}, 0);
    load_chunk(P1{}, 1);
    fill_gates(0);
    __syncthreads();
    stage_rows(P0{}, 0);
  }
  int i = 0;
  for (; i + 1 < nch; i += 2) {
    step(P0{}, P1{}, i);
    step(P1{}, P0{}, i + 1);
  }
  if (i < nch) step(P0{}, P1{}, i);
  if (MODE == kSegment) {
    save(a.entry + seg_state);
    if (slab == 0 && t == 0) a.gain[static_cast<int64_t>(slot) * a.H + h] = gain;
  } else if (a.ht && pc.s == (REV ? 0 : pc.count - 1)) {
    save(a.ht + seq_state);
  }
}

// entry[s], the sums of the segments alone, become the states entering them:
// R <- gain_s R + sum_s along each sequence's segments, elements side by side.
template <bool REV>
__global__ __launch_bounds__(kNT) void decay_join_kernel(DecayArgs a) {
  const int64_t per = static_cast<int64_t>(a.dk) * a.dv / 4;
  const int parts = static_cast<int>((per + kNT - 1) / kNT);
  const int64_t nh = blockIdx.x / parts, e = (blockIdx.x % parts) * static_cast<int64_t>(kNT) + threadIdx.x;
  if (e >= per) return;
  const int n = static_cast<int>(nh / a.H), h = static_cast<int>(nh % a.H);
  const Seq q = sequence(a, n);
  const int first = first_slot(a, n, a.seg), count = q.len > 0 ? (q.len + a.seg - 1) / a.seg : 1;
  f32x4 R = a.h0 ? reinterpret_cast<const f32x4*>(a.h0)[(static_cast<int64_t>(n) * a.H + h) * per + e]
                 : f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4* base = reinterpret_cast<f32x4*>(a.entry);
  for (int i = 0; i < count; ++i) {
    const int64_t s = static_cast<int64_t>(first + (REV ? count - 1 - i : i)) * a.H + h;
    f32x4 u = {0.f, 0.f, 0.f, 0.f};
    float g = 0.f;
    if (i + 1 < count) {
      u = base[s * per + e];
      g = a.gain[s];
    }
    base[s * per + e] = R;
    R = R * g + u;
  }
}

// ---- single-token step -----------------------------------------------------------
//   S <- a S + k v^T,  o = scale S^T q
// HBM-bound: the state is read once and written once.  One workgroup owns 32
// columns of one (sequence, head) state; each thread holds one float4 of two
// rows between the read and the write (8 rows a wave, so 1 to 8 waves by dk).
// The column sums of o run over the rows a wave holds, then over the waves in
// LDS.  256 sequences, 32 heads of 128: 179 us, 6.0 TB/s.
struct DecayStepArgs {
  int32_t N, H, Hk, dk, dv, gate_range, gate_input, per_head;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const void* alpha;
  const float* h0;
  float* ht;
  void* o;
};

template <class IO, int NW>
__global__ __launch_bounds__(64 * NW) void decay_step_kernel(DecayStepArgs a) {
  using T = typename IO::storage;
  __shared__ f32x4 part[NW][8];
  const int nslab = (a.dv + 31) / 32;
  int64_t nh;
  int slab;
  item_of(blockIdx.x, gridDim.x, nslab, nh, slab);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int n = static_cast<int>(nh / a.H), h = static_cast<int>(nh % a.H);
  const int c = slab * 32 + 4 * (lane & 7), r0 = wave * 8 + lane / 8;  // rows r0 + 8 NW i
  const bool col = c < a.dv;
  const int64_t sb = nh * a.dk * a.dv + c;
  f32x4 s[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * NW * i;
    s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (col && r < a.dk)
      s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.h0 + sb + static_cast<int64_t>(r) * a.dv));
  }
  const bool ckda = a.gate_range == CKDA_GATE_CKDA;
  const float g = load_alpha_rt(a.alpha, a.per_head ? h : nh, a.gate_input, ckda);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (col) {
    const T* p = static_cast<const T*>(a.v) + nh * a.dv + c;
    v = f32x4{IO::load(p, 0), IO::load(p, 1), IO::load(p, 2), IO::load(p, 3)};
  }
  const int64_t kb = (static_cast<int64_t>(n) * a.Hk + h / (a.H / a.Hk)) * a.dk;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * NW * i;
    if (r < a.dk) {
      const float k = IO::load(static_cast<const T*>(a.k), kb + r);
      const float q = IO::load(static_cast<const T*>(a.q), kb + r);
      s[i] = s[i] * g + k * v;
      y += s[i] * q;
      if (col)
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(a.ht + sb + static_cast<int64_t>(r) * a.dv));
    }
  }
#pragma unroll
  for (int m = 8; m < 64; m <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], m, 64);
  if (NW > 1) {
    if (lane < 8) part[wave][lane] = y;
    __syncthreads();
    if (t < 8) {
      y = part[0][t];
#pragma unroll
      for (int i = 1; i < NW; ++i) y += part[i][t];
    }
  }
  if (t < 8 && col) IO::store4(static_cast<T*>(a.o) + nh * a.dv + c, y * a.scale);
}

constexpr int step_waves(int dk) { return dk <= 16 ? 1 : (dk <= 32 ? 2 : (dk <= 64 ? 4 : 8)); }
template <class IO>
launch_result launch_step_io(const DecayStepArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.N) * a.H * ((a.dv + 31) / 32));
  const int waves = step_waves(a.dk);
  if (waves == 1)
    hipLaunchKernelGGL((decay_step_kernel<IO, 1>), dim3(grid), dim3(64), 0, s, a);
  else if (waves == 2)
    hipLaunchKernelGGL((decay_step_kernel<IO, 2>), dim3(grid), dim3(128), 0, s, a);
  else if (waves == 4)
    hipLaunchKernelGGL((decay_step_kernel<IO, 4>), dim3(grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((decay_step_kernel<IO, 8>), dim3(grid), dim3(512), 0, s, a);
  return hipGetLastError();
}

// ---- launches ----------------------------------------------------------------------

template <class Op, int DKP, int DVS>
launch_result launch_fwd_t(const DecayArgs& a, hipStream_t s) {
  using Cfg = FwdCfg<Op, DKP, DVS>;
  const launch_result e = allow_lds<decay_fwd_kernel<Op, DKP, DVS>>(Cfg::BYTES);
  if (e != hipSuccess) return e;
  const int64_t grid = static_cast<int64_t>(a.seg > 0 ? a.slots : a.N) * a.H * ((a.dv + DVS - 1) / DVS);
  hipLaunchKernelGGL((decay_fwd_kernel<Op, DKP, DVS>), dim3(static_cast<unsigned>(grid)), dim3(Cfg::NT),
                     Cfg::BYTES, s, a);
  return hipGetLastError();
}
// Columns of the state a workgroup of the forward takes.  Slabs of 64 read q and
// k and form Q K^T half as often as slabs of 32 (8 x 4096 tokens, 16 heads of
// 128: 155 us against 187); in float32 with rows of 128 only 32 fit the LDS.
// With up to 128 walks half the columns each still find CUs of their own and
// shorten a chunk's step: 2 x 100 tokens, 4 heads of 64, 11 us against 14 in
// float32 and 7.3 against 8.1 in bf16; 128 walks of 512 tokens 32 against 42
// (float32, heads of 64) and 19 against 23 (bf16, heads of 128).  From 256 walks
// on it is the other way round: 61 against 46, 35 against 25.
int fwd_slab(const DecayArgs& a, bool bf16) {
  const int64_t walks = static_cast<int64_t>(a.seg > 0 ? a.slots : a.N) * a.H * ((a.dv + 63) / 64);
  return a.dv <= 32 || walks <= 128 || (a.dk > 64 && !bf16) ? 32 : 64;
}
template <class Op>
launch_result launch_fwd_op(const DecayArgs& a, hipStream_t s) {
  constexpr bool bf16 = sizeof(typename Op::T) == 2;
  const bool narrow = fwd_slab(a, bf16) == 32;
  if (a.dk <= 64) return narrow ? launch_fwd_t<Op, 64, 32>(a, s) : launch_fwd_t<Op, 64, 64>(a, s);
  return narrow ? launch_fwd_t<Op, 128, 32>(a, s) : launch_fwd_t<Op, 128, (bf16 ? 64 : 32)>(a, s);
}

template <class Op, int DKP, int DVS, int C, bool REV, int MODE>
launch_result launch_state_t(const DecayArgs& a, hipStream_t s) {
  using Cfg = StateCfg<Op, DKP, DVS, C>;
  constexpr int lds = Cfg::BYTES;
  const int64_t grid = static_cast<int64_t>(a.seg > 0 ? a.slots : a.N) * a.H * ((a.dv + DVS - 1) / DVS);
  const launch_result e = allow_lds<decay_state_kernel<Op, DKP, DVS, C, REV, MODE>>(lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decay_state_kernel<Op, DKP, DVS, C, REV, MODE>), dim3(static_cast<unsigned>(grid)),
                     dim3(Cfg::NT), lds, s, a);
  return hipGetLastError();
}

template <bool REV>
launch_result launch_join(const DecayArgs& a, hipStream_t s) {
  const int64_t per = static_cast<int64_t>(a.dk) * a.dv / 4;
  const int64_t grid = static_cast<int64_t>(a.N) * a.H * ((per + kNT - 1) / kNT);
  hipLaunchKernelGGL(decay_join_kernel<REV>, dim3(static_cast<unsigned>(grid)), dim3(kNT), 0, s, a);
  return hipGetLastError();
}

template <class Op, bool REV, int MODE>
launch_result launch_state_op(const DecayArgs& a, hipStream_t s) {
  constexpr int C = decay_bwd_chunk(sizeof(typename Op::T) == 2 ? CKDA_DTYPE_BF16 : CKDA_DTYPE_F32);
  // a segment's own sum: all columns in one workgroup, which reads k once
  if constexpr (MODE == kSegment)
    if (a.dk > 64 && a.dv > 64) return launch_state_t<Op, 128, 128, C, REV, MODE>(a, s);
  if (decay_slab(a.dv) == 32)
    return a.dk <= 64 ? launch_state_t<Op, 64, 32, C, REV, MODE>(a, s) : launch_state_t<Op, 128, 32, C, REV, MODE>(a, s);
  return a.dk <= 64 ? launch_state_t<Op, 64, 64, C, REV, MODE>(a, s) : launch_state_t<Op, 128, 64, C, REV, MODE>(a, s);
}
template <bool REV, int MODE>
launch_result launch_state(const DecayArgs& a, int32_t io_dtype, hipStream_t s) {
  return io_dtype == CKDA_DTYPE_BF16 ? launch_state_op<OpBF16, REV, MODE>(a, s)
                                     : launch_state_op<OpF32, REV, MODE>(a, s);
}

}  // namespace

bool decay_supported(int32_t dk, int32_t dv) {
  return dk >= 8 && dk <= 128 && dk % 8 == 0 && dv >= 8 && dv <= 128 && dv % 8 == 0;
}

// Tokens of a segment for these sizes (0: sequences are not cut).  Sequences
// are cut where there are fewer (sequence, head, slab) walks than CUs, into
// pieces that give each CU one segment of one head: a cut costs another read
// of k and v.  One prompt of 65536 tokens, 16 heads of 128: 441 us so, 482 with
// half as many segments, 469 with twice as many, 505 with three quarters (256
// CUs do not divide into them).  A packed batch is always cut, since its
// longest sequence would walk alone (40000 tokens, the longest 8191: 298 us).
// Batches of little more than 256 walks pay for a second round of CUs: 8, 9, 12
// and 16 sequences of 4096 tokens, 16 heads of 128, take 160, 258, 265, 308 us,
// gradients 677, 946, 1118, 1337.
int32_t decay_segment(const DecayArgs& a) {
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T;
  if (!a.cu && static_cast<int64_t>(a.N) * a.H * ((a.dv + 63) / 64) >= 256) return 0;
  int64_t seg = (tokens * a.H / 256 + 63) / 64 * 64;
  if (seg < 512) seg = 512;
  return seg < a.T ? static_cast<int32_t>(seg) : 0;
}

// Lays the segments' records out in `ws`; returns the bytes taken.
size_t decay_layout_segments(DecayArgs& a, unsigned char* ws) {
  a.seg = decay_segment(a);
  a.slots = 0;
  if (a.seg == 0) return 0;
  a.slots = static_cast<int32_t>(decay_slots(a, a.seg));
  const size_t st = static_cast<size_t>(a.slots) * a.H * a.dk * a.dv * 4;
  a.entry = reinterpret_cast<float*>(ws);
  a.gain = reinterpret_cast<float*>(ws + st);
  return st + ((static_cast<size_t>(a.slots) * a.H * 4 + 255) & ~size_t(255));
}

size_t decay_segment_bytes(const DecayArgs& a) {
  DecayArgs b = a;
  return decay_layout_segments(b, nullptr);
}

launch_result launch_decay_segments(const DecayArgs& a, int32_t io_dtype, bool rev, hipStream_t s) {
  if (a.seg == 0) return hipSuccess;
  launch_result e = rev ? launch_state<true, kSegment>(a, io_dtype, s)
                        : launch_state<false, kSegment>(a, io_dtype, s);
  if (e != hipSuccess) return e;
  return rev ? launch_join<true>(a, s) : launch_join<false>(a, s);
}

launch_result launch_decay_chunks(const DecayArgs& a, int32_t io_dtype, bool rev, hipStream_t s) {
  return rev ? launch_state<true, kChunks>(a, io_dtype, s) : launch_state<false, kChunks>(a, io_dtype, s);
}

int64_t decay_grid(const DecayArgs& a, int32_t io_dtype) {
  const int64_t parts = static_cast<int64_t>(a.H) * ((a.dv + 31) / 32);
  const int64_t walks = (a.cu || a.T > 0 ? decay_slots(a, 512) : a.N) * parts;
  const int64_t chunks = decay_slots(a, decay_bwd_chunk(io_dtype)) * a.H;
  const int64_t joins = static_cast<int64_t>(a.N) * a.H * ((static_cast<int64_t>(a.dk) * a.dv / 4 + kNT - 1) / kNT);
  const int64_t m = walks > chunks ? walks : chunks;
  return m > joins ? m : joins;
}

int64_t decay_threads(const DecayArgs& given, int32_t io_dtype, DecayCall call) {
  DecayArgs a = given;
  const int64_t heads = static_cast<int64_t>(a.N) * a.H;
  if (call == kDecayStep) return heads * ((a.dv + 31) / 32) * 64 * step_waves(a.dk);
  decay_layout_segments(a, nullptr);
  const int64_t walks = a.seg > 0 ? decay_slots(a, a.seg) * a.H : heads;
  const int slab = call == kDecayFwd ? fwd_slab(a, io_dtype == CKDA_DTYPE_BF16) : decay_slab(a.dv);
  // the forward's walk has four waves more than a state walk's four for every 32 columns
  const int64_t walk = walks * ((a.dv + slab - 1) / slab) * (8 * slab + (call == kDecayFwd ? 256 : 0));
  const int64_t sums = a.seg > 0 ? walks * ((a.dv + 63) / 64) * 512 : 0;
  const int64_t join = a.seg > 0 ? heads * ((static_cast<int64_t>(a.dk) * a.dv / 4 + kNT - 1) / kNT) * kNT : 0;
  const int64_t m = walk > sums ? walk : sums;
  return m > join ? m : join;
}

int decay_dots_per_chunk(int32_t dv) { return (dv + decay_slab(dv) - 1) / decay_slab(dv); }

launch_result launch_decay_fwd(DecayArgs a, int32_t io_dtype, void* ws, hipStream_t s) {
  decay_layout_segments(a, static_cast<unsigned char*>(ws));
  launch_result e = launch_decay_segments(a, io_dtype, false, s);
  if (e != hipSuccess) return e;
  return io_dtype == CKDA_DTYPE_BF16 ? launch_fwd_op<OpBF16>(a, s) : launch_fwd_op<OpF32>(a, s);
}

launch_result launch_decay_step(const DecayArgs& a, int32_t io_dtype, hipStream_t s) {
  const DecayStepArgs p{a.N, a.H, a.Hk, a.dk, a.dv, a.gate_range, a.gate_input, a.per_head, a.scale,
                        a.q, a.k, a.v, a.alpha, a.h0, a.ht, a.o};
  return io_dtype == CKDA_DTYPE_BF16 ? launch_step_io<io_bf16>(p, s) : launch_step_io<io_f32>(p, s);
}

}  // namespace ckda
