// Device building blocks of the decay linear attention
//
//     S_t = a_t S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t
//
// (one gate a head and token, or one a head): the products of gates inside a
// chunk, the spans of tokens a workgroup works on, tiles of rows on their way
// from memory to LDS, and operand fragments read across the rows of LDS.
//
// A chunk of C tokens entered with the state S0 is, with D_ij = a_{j+1}..a_i
// for j <= i (0 otherwise), E_i = a_1..a_i, W_j = a_{j+1}..a_C and g = E_C,
//
//     o_i = scale (E_i S0^T q_i + sum_{j <= i} D_ij (q_i . k_j) v_j)
//     S_C = g S0 + sum_j W_j k_j v_j^T
//
// exactly the recurrence for any gates, zeros and negative ones included.
#pragma once

#include <atomic>

#include "mfma_ops.h"

namespace ckda {


// ---- spans -------------------------------------------------------------------
// Sequence n owns the tokens [begin, begin + len).  cu_seqlens is clamped to
// [0, T], so a malformed one cannot lead outside the tensors.
struct Seq {
  int64_t begin;
  int32_t len;
};
__device__ __forceinline__ int32_t cu_at(const DecayArgs& a, int i) {
  const int32_t c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? a.T : c);
}
__device__ __forceinline__ Seq sequence(const DecayArgs& a, int n) {
  if (!a.cu) return Seq{static_cast<int64_t>(n) * a.T, a.T};
  const int32_t b = cu_at(a, n), e = cu_at(a, n + 1);
  return Seq{b, e > b ? e - b : 0};
}

// Sequences are cut into pieces of L tokens (at least one a sequence), and
// piece s of sequence n has slot first_slot(n, L) + s.  A packed sequence
// starting at token b takes slots from floor(b / L) + n on: those ranges never
// meet and need no sum over the lengths before.
__device__ __forceinline__ int32_t first_slot(const DecayArgs& a, int n, int L) {
  if (!a.cu) return n * (a.T > 0 ? (a.T + L - 1) / L : 1);
  return cu_at(a, n) / L + n;
}
struct Piece {
  int32_t n;       // sequence, -1 for an unused slot
  int32_t s, count;  // piece s of `count` of the sequence
  int64_t begin;   // first token
  int32_t len;
};
// The piece of a slot, the same in all lanes of a wave: dense by division,
// packed by a search that tests 64 sequences at a time.
__device__ __forceinline__ Piece piece_of(const DecayArgs& a, int slot, int L, int lane) {
  Piece p;
  if (!a.cu) {
    const int per = a.T > 0 ? (a.T + L - 1) / L : 1;
    p.n = slot / per;
  } else {
    int lo = 0, cnt = a.N;
    while (cnt > 1) {
      const int step = (cnt + 63) / 64;
      const int off = lane * step;
      const bool below = off < cnt && first_slot(a, lo + off, L) <= slot;
      int m = __popcll(__ballot(below));
      m = m > 0 ? m - 1 : 0;
      const int left = cnt - m * step;
      lo += m * step;
      cnt = left < step ? left : step;
    }
    p.n = uniform32(lo);
  }
  const Seq q = sequence(a, p.n);
  p.s = slot - first_slot(a, p.n, L);
  p.count = q.len > 0 ? (q.len + L - 1) / L : 1;
  if (p.s < 0 || p.s >= p.count) {
    p.n = -1;
    p.len = 0;
    return p;
  }
  p.begin = q.begin + static_cast<int64_t>(p.s) * L;
  const int rest = q.len - p.s * L;
  p.len = rest < L ? rest : L;
  return p;
}

// ---- gates -------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;

// log2|a| of a gate, whether it is negative, and whether it is zero (then the
// logarithm is 0 and the zero is tracked apart).  The logarithm comes from the
// logit itself where there is one: forming the gate first would lose the
// distance of a gate from 1, which a memory of thousands of tokens multiplies.
// A gate under the least float32, 2^-149, is a zero: the single-token step has
// it so, and a running sum with a logit of -1e9 in it, or of the type's lowest
// value, would lose the gates behind it.  So no logarithm here is under -150,
// and a chunk's sum stays within 2^14.
struct GateLog {
  float l2;
  bool neg, zero;
};
// v_log_f32 is within 1.2e-7 of the value over all normal floats, also next to
// 1 (measured); smaller ones are scaled up first.
__device__ __forceinline__ float log2_of(float a) {  // a > 0
  const bool tiny = a < 0x1p-100f;
  return __builtin_amdgcn_logf(tiny ? a * 0x1p64f : a) - (tiny ? 64.f : 0.f);
}
// log2(1 + y), -1 < y <= 1: the rounding of 1 + y is undone by the factor
__device__ __forceinline__ float log2_1p(float y) {
  const float u = 1.f + y, r = u - 1.f;
  return r == 0.f ? y * kLog2e : __builtin_amdgcn_logf(u) * (y * __builtin_amdgcn_rcpf(r));
}
__device__ __forceinline__ GateLog gate_log(float x, int gate_input, bool ckda) {
  GateLog r;
  if (gate_input == CKDA_GATES_F32) {
    r.neg = x < 0.f;
    r.l2 = log2_of(fabsf(x));
  } else if (!ckda) {  // sigmoid
    r.neg = false;
    r.l2 = (x < 0.f ? x * kLog2e : 0.f) - log2_1p(exp_neg(fabsf(x)));
  } else {  // 2 sigmoid - 1 = tanh(x / 2)
    const float m = fabsf(x), e = exp_neg(m);
    r.neg = x < 0.f;
    r.l2 = m < 0.5f ? log2_of(alpha_from_logit(m, true)) : log2_1p(-e) - log2_1p(e);
  }
  r.zero = r.l2 < -149.5f;  // -inf of a gate of 0 too
  if (r.zero) r.l2 = 0.f;
  return r;
}
// the gate itself (for the recurrences that multiply by it)
__device__ __forceinline__ float gate_value(float x, int gate_input, bool ckda) {
  return gate_input == CKDA_GATES_F32 ? x : alpha_from_logit(x, ckda);
}
// Inclusive sum over the lanes of a wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_moved(double x) {  // 0 where no lane moves in
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_moved<0x111, 0xf>(x);  // within rows of 16 lanes: from 1, 2, 4, 8 below
  x += dpp_moved<0x112, 0xf>(x);
  x += dpp_moved<0x114, 0xf>(x);
  x += dpp_moved<0x118, 0xf>(x);
  x += dpp_moved<0x142, 0xa>(x);  // row 0's last lane into row 1, 2's into 3
  x += dpp_moved<0x143, 0xc>(x);  // lane 31 into rows 2 and 3
  return x;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_moved(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_scan(float x) {
  x += dpp_moved<0x111, 0xf>(x);
  x += dpp_moved<0x112, 0xf>(x);
  x += dpp_moved<0x114, 0xf>(x);
  x += dpp_moved<0x118, 0xf>(x);
  x += dpp_moved<0x142, 0xa>(x);
  x += dpp_moved<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ double lane_value(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), l);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// 2^x of a double whose integer part may leave float's exponent range
__device__ __forceinline__ float exp2_wide(double x) {
  const double n = rint(x);
  return ldexpf(__builtin_amdgcn_exp2f(static_cast<float>(x - n)), static_cast<int>(n));
}

// A chunk's gates in LDS.  L is the running sum of log2|a| (kept in double:
// with gates near 0.1 a float sum of 64 of them is off by 1e-5), split into an
// integer and a fraction so that differences of two are exact to float.
// `fast`: no gate under 2^-30 (zeros among them) and all running products
// within 2^+-60 of the middle one, so D_ij = er_i ej_j, signs included, and a
// sum of terms that hold a gate may be divided by it.
template <int C>
struct alignas(16) Gates {
  float E[C], W[C];  // products from the chunk's start, to its end
  float u[C], v[C];  // er, ej; without `fast` the integer and fraction of L
  int sz[C];         // without `fast`: 2 z + (1 where the running sign is negative),
                     // z the last zero gate at or before i (-1: none)
  float g;           // product of all
  int fast;
};

// One wave fills G from its lanes' gates (lane i: token i; tokens past the
// chunk's length count as gates of 1).
template <int C>
__device__ __forceinline__ void gates_fill(Gates<C>& G, float x, bool valid, int gate_input,
                                           bool ckda, int lane) {
  const GateLog gl = gate_log(x, gate_input, ckda);
  const uint64_t zm = __ballot(valid && gl.zero), nm = __ballot(valid && gl.neg);
  const double L = wave_scan(valid ? static_cast<double>(gl.l2) : 0.0);
  const double end = lane_value(L, 63), mid = lane_value(L, C / 2 - 1);
  const uint64_t upto = ~0ull >> (63 - lane);
  const uint64_t zz = zm & upto;
  const int z = zz ? 63 - __clzll(zz) : -1;
  const int zend = zm ? 63 - __clzll(zm) : -1;
  const float sg = (__popcll(nm & upto) & 1) ? -1.f : 1.f;
  const float sgend = (__popcll(nm) & 1) ? -1.f : 1.f;
  const bool far = !(fabs(L - mid) <= 60.0) || (valid && !(fabsf(gl.l2) <= 30.f));
  const bool fast = zm == 0 && __ballot(far) == 0;
  if (fast) {  // powers of differences up to 60, the others from them
    const float er = sg * __builtin_amdgcn_exp2f(static_cast<float>(L - mid));
    const float ej = __builtin_amdgcn_rcpf(er);
    const float g = sgend * exp2_wide(end), em = exp2_wide(mid), ee = sgend * exp2_wide(end - mid);
    if (lane < C) {
      G.E[lane] = er * em;
      G.W[lane] = ej * ee;
      G.u[lane] = er;
      G.v[lane] = ej;
    }
    if (lane == 0) {
      G.g = g;
      G.fast = 1;
    }
  } else {
    const double n = rint(L);
    if (lane < C) {
      G.E[lane] = z < 0 ? sg * exp2_wide(L) : 0.f;
      G.W[lane] = zend <= lane ? sg * sgend * exp2_wide(end - L) : 0.f;
      G.u[lane] = static_cast<float>(n);
      G.v[lane] = static_cast<float>(L - n);
      G.sz[lane] = 2 * z + (sg < 0.f ? 1 : 0);
    }
    if (lane == 0) {
      G.g = zend < 0 ? sgend * exp2_wide(end) : 0.f;
      G.fast = 0;
    }
  }
}

// D_ij for one i and j = j0 .. j0 + 3 (j0 a multiple of 4), 0 for j > i
template <int C>
__device__ __forceinline__ f32x4 decay_of(const Gates<C>& G, int i, int j0, bool fast) {
  f32x4 d;
  if (fast) {
    d = *reinterpret_cast<const f32x4*>(&G.v[j0]) * G.u[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = j0 + e <= i ? d[e] : 0.f;
  } else {
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&G.u[j0]);
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&G.v[j0]);
    const int4 sz = *reinterpret_cast<const int4*>(&G.sz[j0]);
    const int szj[4] = {sz.x, sz.y, sz.z, sz.w};
    const float h = G.u[i], l = G.v[i];
    const int si = G.sz[i], z = si >> 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __builtin_amdgcn_exp2f((h - hi[e]) + (l - lo[e]));
      d[e] = (j0 + e <= i && z <= j0 + e) ? (((si ^ szj[e]) & 1) ? -x : x) : 0.f;
    }
  }
  return d;
}
// x D, nothing passing a D of exactly 0 (a zero gate, j > i)
__device__ __forceinline__ f32x4 decayed(f32x4 x, f32x4 d) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = d[e] != 0.f ? x[e] * d[e] : 0.f;
  return x;
}

// ---- tiles of rows, memory -> registers -> LDS ------------------------------
// ROWS x COLS elements of T in 16-byte pieces by NT threads, read through a
// buffer resource that ends with the last valid row's last column: rows past
// it read as zeros without a branch, and pieces past the first `cols` columns
// (a multiple of a piece) carry an offset past any resource.  A thread's
// offsets are formed once; ld in elements, ROWS * ld * sizeof(T) < 2^31.
constexpr int kNoOffset = 0x7ffffff0;
template <class T>
__device__ __forceinline__ rsrc_t rows_rsrc(const T* base, int ld, int rows, int cols, int most) {
  // no branch (a wait after one would count the path with fewer loads)
  const int r = min(rows, most), bytes = ((r - 1) * ld + cols) * static_cast<int>(sizeof(T));
  const T* b = reinterpret_cast<const T*>(uniform64(reinterpret_cast<int64_t>(base)));
  return make_rsrc(b, uniform32(bytes & ~((r - 1) >> 31)));
}
__device__ __forceinline__ uint4 load_piece(rsrc_t r, int off) {
  uint4 x;
  ldraw<16>(r, off, reinterpret_cast<uint32_t*>(&x));
  return x;
}
// Stores through such a resource drop what lies past it.
__device__ __forceinline__ void store_piece(rsrc_t r, int off, const uint4& x) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(u32x4{x.x, x.y, x.z, x.w}, r, off, 0, 0);
}
template <class T, int ROWS, int COLS, int NT>
struct RowTile {
  static constexpr int EPP = 16 / sizeof(T), PPR = COLS / EPP, NP = ROWS * PPR / NT;
  static_assert(ROWS * PPR % NT == 0, "whole pieces a thread");
  struct Regs {
    uint4 r[NP];
  };
  int off[NP];
  __device__ __forceinline__ void init(int ld, int cols, int t) {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = t + NT * u, row = p / PPR, c = (p % PPR) * EPP;
      off[u] = c < cols ? (row * ld + c) * static_cast<int>(sizeof(T)) : kNoOffset;
    }
  }
  __device__ __forceinline__ void load(Regs& d, const T* base, int ld, int rows, int cols) const {
    const rsrc_t rs = rows_rsrc(base, ld, rows, cols, ROWS);
#pragma unroll
    for (int u = 0; u < NP; ++u) d.r[u] = load_piece(rs, off[u]);
  }
  static __device__ __forceinline__ void store(const Regs& d, T* lds, int ldl, int t) {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = t + NT * u, row = p / PPR, c = (p % PPR) * EPP;
      *reinterpret_cast<uint4*>(lds + row * ldl + c) = d.r[u];
    }
  }
};

// LDS row stride for tiles that are read across their rows (four rows of 16
// columns a lane group and read): 16 bytes past the row.
constexpr int cross_stride(int n, int es) { return n + 16 / es; }

// The stored gate of token `lane` of `rows` tokens from `token` on, as raw
// bits (0 past them): issued with a chunk's rows and decoded after them.
struct GateBits {
  uint32_t lo, hi;
};
__device__ __forceinline__ GateBits load_gate_bits(const DecayArgs& a, int64_t token, int rows, int h,
                                                   int lane) {
  // two loads of two bytes each, at any type, in the place of a branch on it
  const int gs = a.gate_input == CKDA_GATES_LOGITS_BF16 ? 2 : 4;
  const int64_t at = (a.per_head ? 0 : token * a.H) + h;
  const unsigned char* b = static_cast<const unsigned char*>(a.alpha) + at * gs;
  const int ld = a.per_head ? 0 : a.H, n = min(rows, 64), bytes = ((n - 1) * ld + 1) * gs;
  const rsrc_t r = make_rsrc(reinterpret_cast<const void*>(uniform64(reinterpret_cast<int64_t>(b))),
                             uniform32(bytes & ~((n - 1) >> 31)));
  GateBits x;
  ldraw<2>(r, lane * ld * gs, &x.lo);
  ldraw<2>(r, lane * ld * gs + (gs - 2), &x.hi);  // of a bf16 gate, its bits again
  return x;
}
__device__ __forceinline__ float gate_of_bits(const GateBits& x, int gate_input) {
  return __uint_as_float((x.hi << 16) | (gate_input == CKDA_GATES_LOGITS_BF16 ? 0 : x.lo));
}

// ---- operand fragments --------------------------------------------------------
// Beside the row fragments of mfma_ops.h, fragments read ACROSS rows: from
// X[k][n] in LDS, lane (l16, lq) takes column n0 + l16 and the K-values of the
// accumulators' order (16-row tile, lq, i), so products of accumulators with
// them need no pass through LDS.  `row`: natural K order; `rowp`: a row in
// the accumulators' K order.
template <class Op>
struct Fr;

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <>
struct Fr<OpBF16> {
  using Op = OpBF16;
  using T = __bf16;
  using F = bf16x8;
  static constexpr int KS = 32;
  static constexpr int kTerms = 3;  // of a weighted operand
  using IO = io_bf16;
  static __device__ __forceinline__ s16x4 tr4(const T* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(const_cast<T*>(p)));
  }
  // the 16 columns in groups of 4, `apart` columns apart: lane l16 takes column
  // n0 + apart (l16 / 4) + l16 % 4
  static __device__ __forceinline__ F across(const T* x, int ld, int k0, int n0, int lane, int apart = 4) {
    const int l16 = lane & 15, lq = lane >> 4;
    const T* p = x + (k0 + 4 * lq + (l16 >> 2)) * ld + n0 + apart * (l16 & 3);
    union {
      s16x4 s[2];
      F f;
    } u;
    u.s[0] = tr4(p);
    u.s[1] = tr4(p + 16 * ld);
    return u.f;
  }
  static __device__ __forceinline__ F row(const T* r, int s, int lq) {
    return *reinterpret_cast<const F*>(r + 32 * s + 8 * lq);
  }
  static __device__ __forceinline__ F rowp(const T* r, int s, int lq) {
    union {
      bf16x4 h[2];
      F f;
    } u;
    u.h[0] = *reinterpret_cast<const bf16x4*>(r + 32 * s + 4 * lq);
    u.h[1] = *reinterpret_cast<const bf16x4*>(r + 32 * s + 16 + 4 * lq);
    return u.f;
  }
};

template <>
struct Fr<OpF32> {
  using Op = OpF32;
  using T = float;
  using F = f32x4;
  static constexpr int KS = 16;
  static constexpr int kTerms = 1;
  using IO = io_f32;
  static __device__ __forceinline__ F across(const T* x, int ld, int k0, int n0, int lane, int apart = 4) {
    const T* p = x + (k0 + 4 * (lane >> 4)) * ld + n0 + apart * ((lane & 15) >> 2) + (lane & 3);
    return F{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  static __device__ __forceinline__ F row(const T* r, int s, int lq) {
    return *reinterpret_cast<const F*>(r + 16 * s + 4 * lq);
  }
  static __device__ __forceinline__ F rowp(const T* r, int s, int lq) { return row(r, s, lq); }
};

// element e of a 16-byte piece, widened
template <class T>
__device__ __forceinline__ float piece_elem(const uint4& u, int e) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 2)
    return __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
  else
    return __uint_as_float(w[e]);
}

// A piece times w, stored for the state update.  bf16: as three terms, each
// the nearest bf16 of what the ones before leave (2^-24 of it is lost: as
// float32), because the state is kept, and handed out, in float32; k and v
// themselves are exact.  Two terms would leave 2e-6 of the state.
template <class T>
__device__ __forceinline__ void store_scaled(const uint4& u, float w, T* dst, int plane) {
  constexpr int E = 16 / sizeof(T), NP = sizeof(T) == 2 ? 3 : 1;
  alignas(16) T h[NP][E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float x = piece_elem<T>(u, e) * w;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      h[p][e] = static_cast<T>(x);
      if constexpr (NP > 1) x -= static_cast<float>(h[p][e]);
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p)
    *reinterpret_cast<uint4*>(dst + p * plane) = *reinterpret_cast<const uint4*>(h[p]);
}

// Work items of a grid: `outer` items of `inner` parts.  Workgroups go to the
// 8 XCDs in turn, so the parts of one item are placed 8 workgroups apart: they
// share what they read through one L2.
__device__ __forceinline__ void item_of(int64_t block, int64_t grid, int inner, int64_t& outer,
                                        int& part) {
  if (inner > 1 && grid % (8 * static_cast<int64_t>(inner)) == 0) {
    const int64_t r = block / 8;
    part = static_cast<int>(r % inner);
    outer = (r / inner) * 8 + block % 8;
  } else {
    part = static_cast<int>(block % inner);
    outer = block / inner;
  }
}

// ---- host side ----------------------------------------------------------------
// Lets `Kernel` take more than 64 KB of LDS, once for each device.
template <auto Kernel>
launch_result allow_lds(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return hipSuccess;
  const hipError_t r = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (r == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return r;
}
constexpr int kDecayChunk = 64;
// state columns a workgroup of the state walks takes
__host__ __device__ constexpr int decay_slab(int dv) { return dv <= 32 ? 32 : 64; }
// chunk of the backward's records and gradients
constexpr int decay_bwd_chunk(int32_t io_dtype) { return io_dtype == CKDA_DTYPE_BF16 ? 64 : 32; }
// slots of pieces of L tokens
inline int64_t decay_slots(const DecayArgs& a, int L) {
  if (a.cu) return a.T / L + static_cast<int64_t>(a.N);
  return static_cast<int64_t>(a.N) * (a.T > 0 ? (a.T + L - 1) / L : 1);
}

size_t decay_layout_segments(DecayArgs& a, unsigned char* ws);
int decay_dots_per_chunk(int32_t dv);
// Segment entries (nothing where sequences are not cut), then the walks that
// keep the state met at every chunk.  Backwards, a.o holds dout, a.h0 the
// adjoint of the final states and a.ht receives that of the initial ones.
launch_result launch_decay_segments(const DecayArgs& a, int32_t io_dtype, bool rev, hipStream_t s);
launch_result launch_decay_chunks(const DecayArgs& a, int32_t io_dtype, bool rev, hipStream_t s);

}  // namespace ckda
