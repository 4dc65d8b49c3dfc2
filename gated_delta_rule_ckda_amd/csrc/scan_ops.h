// Device building blocks of the selective scan: for every channel with S states,
//
//   d_t = softplus(dt_t + bias)   (or dt_t + bias itself)
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,     y_t = C_t . h_t + D x_t
//
// and, with a gate, y_t silu(z_t).  B and C are shared by the channels of a group.
//
// W waves of a workgroup walk over the tokens of one piece of a sequence for CH
// channels.  Lanes hold channels, and the states of a channel are dealt out to W NL
// slices (NL slices a wave, side by side in its lanes), NR a lane, so that a
// lane's sums over states are its own and only W NL partial sums a token and
// channel meet in LDS.
#pragma once

#include "decay_ops.h"
#include "row_ops.h"

namespace ckda {

template <int W_, int NL_, int NR_>
struct ScanCfg {
  static constexpr int W = W_, NL = NL_, NR = NR_;
  static constexpr int CH = 64 / NL;     // channels of a workgroup
  static constexpr int NSL = W * NL;     // slices of the states
  static constexpr int SP = NSL * NR;    // states, the last ones possibly padding
};

// A / ln 2, kept finite for the largest A (past 2.358e38 rates count as that one): an
// infinite one would make no number of a step of 0, of the rows that fill a tile's
// end, and of its product with a decay of 0.
__device__ __forceinline__ float log2_rate(float A) {
  const float r = A * kLog2e, most = 3.4028234663852886e38f;
  return r < -most ? -most : (r > most ? most : r);
}

// The decay of a step d by A = A2 ln 2.  v_exp_f32 is low by 6.8e-9 of the value on
// average for arguments next to 0, 3.5e-9 at -0.01 and 2e-9 to 4e-9 from there on
// (measured over 2^20 arguments each; its rounding is 1.8e-8): nothing in one step,
// but a product over a memory of a thousand tokens keeps every step's.  The sum
// with kLift, in the product's own rounding, takes most of it back; an argument of
// 0 still gives 1.
constexpr float kLift = 8e-9f;
__device__ __forceinline__ float decay_arg(float d, float A2) { return __builtin_fmaf(d, A2, kLift); }
__device__ __forceinline__ float decay_by(float d, float A2) { return __builtin_amdgcn_exp2f(decay_arg(d, A2)); }

// h = own + R exp(span A): the states R that enter a part of a sequence added to the
// part's own, whose steps sum to `span`.  For rates that grow the power may leave
// float32 where its product with R does not: past 2^126 the exponent's whole part
// goes to the product instead, and an R of 0 stays 0.  Decays take the one power: a
// wave branches where any of its lanes grows that far (both ways in every lane:
// gradients of a layer 1326 us against 1297).  Steps of the largest finite size may
// sum to infinity, of which a rate of 0 would make no number.
template <int N>
__device__ __forceinline__ void enter(float span, const float (&A2)[N], const float (&R)[N], const float (&own)[N],
                                      float (&h)[N]) {
  constexpr float kMost = 3.4028234663852886e38f;
  span = __builtin_amdgcn_fmed3f(span, -kMost, kMost);
  float x[N], top = -kMost;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = decay_arg(span, A2[i]);
    top = fmaxf(top, x[i]);
  }
  if (__any(top > 126.f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // more than 2^277 takes the least float32 past the largest
      const float y = __builtin_amdgcn_fmed3f(x[i], -300.f, 300.f), k = rintf(y);
      h[i] = own[i] + __builtin_amdgcn_ldexpf(R[i] * __builtin_amdgcn_exp2f(y - k), static_cast<int>(k));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(x[i]), R[i], own[i]);
  }
}

// exp(-m) for m >= 0, the rounding of m log2(e) undone (it would cost m / 2 half
// steps of the value); zeros from about 87 on.
__device__ __forceinline__ float exp_minus(float m) {
  m = fminf(m, 200.f);
  const float t = m * -kLog2e, e = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(m, -kLog2e, -t);  // what t lost
  return __builtin_fmaf(e * 0.6931471805599453f, r, e);
}
// softplus: max(v, 0) + log(1 + e), e = exp(-|v|).  u = 1 + e is off by c, which
// the last step puts back, so a small e keeps its digits (c counts 1 / u times;
// leaving that out costs less than half a step).  -inf gives 0, NaN stays.
__device__ __forceinline__ float softplus_of(float v) {
  const float e = exp_minus(fabsf(v)), u = 1.f + e, c = e - (u - 1.f);
  return (v < 0.f ? 0.f : v) + __builtin_fmaf(__builtin_amdgcn_logf(u), 0.6931471805599453f, c);
}
// with its derivative, the sigmoid
__device__ __forceinline__ void softplus_and_slope(float v, float& d, float& slope) {
  const float e = exp_minus(fabsf(v)), u = 1.f + e, c = e - (u - 1.f), r = __builtin_amdgcn_rcpf(u);
  d = (v < 0.f ? 0.f : v) + __builtin_fmaf(__builtin_amdgcn_logf(u), 0.6931471805599453f, c);
  slope = v < 0.f ? e * r : r;
}

// ---- rows in memory --------------------------------------------------------
// EP consecutive channels of a row as they lie in memory.  Offsets that are out
// of the resource's range load zeros and store nothing; kOut is one.
constexpr int kOut = 0x7ffffff0;

template <class IO, int EP>
struct RowBits {
  static constexpr int ES = sizeof(typename IO::storage), BYTES = EP * ES, W = BYTES >= 4 ? BYTES / 4 : 1;
  uint32_t w[W];
  // off: bytes to the first channel (kOut: none); cols: channels left in the row
  __device__ __forceinline__ void load(rsrc_t r, int off, int cols, bool vec) {
    static_assert(EP == 1 || EP == 2 || EP == 4, "channels a thread");
    if (vec) {
      ldraw<BYTES, kStream>(r, off, w);
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int e = 0; e < EP; ++e) ldraw<4>(r, e < cols && off != kOut ? off + 4 * e : kOut, w + e);
    } else {
      uint32_t x[EP];
#pragma unroll
      for (int e = 0; e < EP; ++e) ldraw<2>(r, e < cols && off != kOut ? off + 2 * e : kOut, x + e);
#pragma unroll
      for (int e = 0; e < EP; e += 2) w[e / 2] = (x[e] & 0xffffu) | (e + 1 < EP ? x[e + 1 < EP ? e + 1 : e] << 16 : 0);
    }
  }
  __device__ __forceinline__ float get(int e) const { return dec<IO>(w, e); }
  static __device__ __forceinline__ void store(rsrc_t r, int off, int cols, bool vec, const float* x) {
    if constexpr (ES == 4) {
      if (vec) {
        if constexpr (EP == 4) {
          typedef uint32_t u4 __attribute__((ext_vector_type(4)));
          const u4 v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
          __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, kStream);
          return;
        }
      }
#pragma unroll
      for (int e = 0; e < EP; ++e)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[e]), r, e < cols && off != kOut ? off + 4 * e : kOut, 0, 0);
    } else {
      uint32_t u[W];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        bf16x2 b;
        b[0] = static_cast<__bf16>(x[2 * k]);
        b[1] = static_cast<__bf16>(x[2 * k + 1 < EP ? 2 * k + 1 : 2 * k]);
        u[k] = __builtin_bit_cast(uint32_t, b);
      }
      if (vec) {
        if constexpr (EP == 4) {
          typedef uint32_t u2 __attribute__((ext_vector_type(2)));
          __builtin_amdgcn_raw_buffer_store_b64(u2{u[0], u[1]}, r, off, 0, kStream);
          return;
        } else if constexpr (EP == 2) {
          __builtin_amdgcn_raw_buffer_store_b32(u[0], r, off, 0, kStream);
          return;
        }
      }
#pragma unroll
      for (int e = 0; e < EP; ++e)
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1))), r,
                                              e < cols && off != kOut ? off + 2 * e : kOut, 0, 0);
    }
  }
};

// The resource of `rows` rows of `cols` channels from channel c of token t on.
template <class IO>
__device__ __forceinline__ rsrc_t rows_rsrc(const void* p, int64_t t, int64_t stride, int64_t c, int rows, int cols) {
  constexpr int ES = sizeof(typename IO::storage);
  const int64_t at = uniform64((t * stride + c) * ES);
  const int bytes = rows > 0 ? static_cast<int>((rows - 1) * stride + cols) * ES : 0;
  return make_rsrc(static_cast<const char*>(p) + at, uniform32(bytes));
}

// ---- workgroups ------------------------------------------------------------
// Blocks of channels: CH of one group each.
__host__ __device__ __forceinline__ int scan_blocks(int D, int G, int CH) { return G * ((D / G + CH - 1) / CH); }

// Workgroups whose channels share 128-byte lines are put on one XCD (workgroups
// go to the 8 XCDs in turn): NL neighbours 8 apart.
template <int NL>
__device__ __forceinline__ int scan_order(int id, int total) {
  const int span = 8 * NL, base = id / span * span;
  if (NL == 1 || base + span > total) return id;
  const int r = id - base;
  return base + (r & 7) * NL + (r >> 3);
}

template <class C>
struct ScanBlock {
  int slot, blk;   // piece slot, block of channels
  int g, chan, cols;  // group, first channel, channels of the block
  __device__ __forceinline__ ScanBlock(const ScanArgs& a) {
    const int per = a.D / a.G, nb = (per + C::CH - 1) / C::CH, blocks = a.G * nb;
    const int id = scan_order<C::NL>(blockIdx.x, gridDim.x);
    slot = id / blocks;
    blk = id - slot * blocks;
    g = blk / nb;
    const int c0 = (blk - g * nb) * C::CH;
    chan = g * per + c0;
    cols = per - c0 < C::CH ? per - c0 : C::CH;
  }
};

// NR consecutive floats in LDS (16-byte aligned rows), the same for all lanes of a slice
template <int NR>
__device__ __forceinline__ void lds_run(const float* p, float* v) {
  if constexpr (NR % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NR; i += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + i);
      v[i] = x[0]; v[i + 1] = x[1]; v[i + 2] = x[2]; v[i + 3] = x[3];
    }
  } else {
    static_assert(NR == 2, "states a lane");
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x;
    v[1] = x.y;
  }
}
template <int EP>
__device__ __forceinline__ void lds_put(float* p, const float* v) {
  if constexpr (EP % 4 == 0) {
#pragma unroll
    for (int e = 0; e < EP; e += 4) *reinterpret_cast<f32x4*>(p + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
  } else if constexpr (EP == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
    p[0] = v[0];
  }
}
template <int EP>
__device__ __forceinline__ void lds_add(const float* p, float* v) {
  if constexpr (EP % 4 == 0) {
#pragma unroll
    for (int e = 0; e < EP; e += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[e + i] += x[i];
    }
  } else {
#pragma unroll
    for (int e = 0; e < EP; ++e) v[e] += p[e];
  }
}

// ---- sums over a wave's channels ---------------------------------------------
// 16 / NL values a lane, to be summed over the lanes of each slice: halves of the
// wave and neighbouring rows of 16 lanes are added while pairs of values become one
// register, then the lanes of a row, four registers becoming one.  Lane l, for l a
// multiple of 4, ends with the sum of value sum_index(l) of slice l / (64 / NL).
template <int NL>
__device__ __forceinline__ float sum_channels(const float (&v)[16 / NL]) {
  const auto swap = [](float x, float y, auto f) {
    const auto r = f(__float_as_uint(x), __float_as_uint(y));
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const auto halves = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane32_swap(x, y, false, false); };
  const auto rows = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane16_swap(x, y, false, false); };
  float s[8], q[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = NL == 1 ? swap(v[2 * k], v[NL == 1 ? 2 * k + 1 : 0], halves) : v[NL == 1 ? 0 : k];
#pragma unroll
  for (int k = 0; k < 4; ++k) q[k] = swap(s[2 * k], s[2 * k + 1], rows);
  // banks of 4 lanes: 0 and 1 from q0 (q2), 2 and 3 from q1 (q3); then bank 1 from
  // q0, 3 from q1, 0 from q2, 2 from q3; then all four lanes of a bank.  A lane's
  // register is read by its neighbours two wait states after it is written.
  float t0, t1, r;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %0, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %2, %0, %0 row_ror:4 row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %1, %1 row_ror:12 row_mask:0xf bank_mask:0x5\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %2, %2, %2 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %2, %2, %2 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf"
      : "=&v"(t0), "=&v"(t1), "=&v"(r)
      : "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]));
  return r;
}
template <int NL>
__device__ __forceinline__ int sum_index(int lane) {
  const int row = lane >> 4, bank = (lane >> 2) & 3, q = (0x1302 >> (4 * bank)) & 3;  // 2, 0, 3, 1
  if (NL == 1) return 4 * q + ((row & 1) << 1 | row >> 1);
  return 2 * q + (row & 1);
}

constexpr int kMark = 16;  // tokens between the states kept for the gradients

// Tokens of a piece where sequences are not cut: past every sequence's end.
__host__ __device__ __forceinline__ int scan_whole(int T) { return T + 1; }

// What the kernels of one call share out: which lanes hold which states.
template <class F>
launch_result scan_config(int which, F f) {
  switch (which) {
    case 0: return f(ScanCfg<4, 1, 2>{});
    case 1: return f(ScanCfg<4, 1, 4>{});
    case 2: return f(ScanCfg<4, 2, 2>{});
    case 3: return f(ScanCfg<4, 2, 4>{});
    default: return f(ScanCfg<8, 2, 4>{});
  }
}
struct ScanPlan {
  int which, CH, SP;
  int blocks, slots, seg, cut, mslots;
};
ScanPlan scan_plan(const ScanArgs& a, bool grads);

// What the gradients need of the states: the marks and, where sequences are cut,
// the state and the adjoint entering every piece.
launch_result launch_scan_marks(const ScanArgs& a, const ScanPlan& p, int32_t io_dtype, hipStream_t s);

}  // namespace ckda
