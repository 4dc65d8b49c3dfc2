// The tokens of a batch's sequences, and the pieces that sequences are cut into.
// An argument struct that uses these has T (tokens of a sequence, or of a whole
// packed batch), N (sequences) and cu (their offsets, null for a dense batch).
#pragma once

#include "mfma_ops.h"

namespace ckda {

// Sequence n owns the tokens [begin, begin + len).  cu_seqlens is clamped to
// [0, T], so a malformed one cannot lead outside the tensors.
struct Seq {
  int64_t begin;
  int32_t len;
};
template <class Args>
__device__ __forceinline__ int32_t cu_at(const Args& a, int i) {
  const int32_t c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? a.T : c);
}
template <class Args>
__device__ __forceinline__ Seq sequence(const Args& a, int n) {
  if (!a.cu) return Seq{static_cast<int64_t>(n) * a.T, a.T};
  const int32_t b = cu_at(a, n), e = cu_at(a, n + 1);
  return Seq{b, e > b ? e - b : 0};
}

// Sequences are cut into pieces of L tokens (at least one a sequence), and
// piece s of sequence n has slot first_slot(n, L) + s.  A packed sequence
// starting at token b takes slots from floor(b / L) + n on: those ranges never
// meet and need no sum over the lengths before.
template <class Args>
__device__ __forceinline__ int32_t first_slot(const Args& a, int n, int L) {
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
template <class Args>
__device__ __forceinline__ Piece piece_of(const Args& a, int slot, int L, int lane) {
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

// The same for a slot of this thread's own: packed by halving.
template <class Args>
__device__ __forceinline__ Piece piece_of_thread(const Args& a, int slot, int L) {
  Piece p;
  if (!a.cu) {
    const int per = a.T > 0 ? (a.T + L - 1) / L : 1;
    p.n = slot / per;
  } else {
    int lo = 0, hi = a.N;  // the last sequence whose slots start at or before this one
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (first_slot(a, m, L) <= slot)
        lo = m;
      else
        hi = m;
    }
    p.n = lo;
  }
  const Seq q = sequence(a, p.n);
  p.s = slot - first_slot(a, p.n, L);
  p.count = q.len > 0 ? (q.len + L - 1) / L : 1;
  p.begin = q.begin;
  p.len = 0;
  if (p.s < 0 || p.s >= p.count) {
    p.n = -1;
    return p;
  }
  p.begin += static_cast<int64_t>(p.s) * L;
  const int rest = q.len - p.s * L;
  p.len = rest < L ? rest : L;
  return p;
}

}  // namespace ckda
