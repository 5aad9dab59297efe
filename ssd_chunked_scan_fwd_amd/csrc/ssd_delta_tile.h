// ssd_delta_tile.h -- what the delta rule's kernels share: fp32 values as sums
// of bf16 terms, operands of v_mfma_f32_16x16x32_bf16 made of them, rows of a
// chunk as operands.
//
// The rule feeds what it computes back into itself (the state, and the inverse
// of I + A), its states and gate gradients are fp32 results, and o may be small
// beside the terms that it is summed of (a query that is almost orthogonal to what
// the state holds), far below where 16 bits of them end. So every
// computed operand enters its products as the sum of three bf16 terms, which
// hold all 24 bits of an fp32 value; bf16 inputs are exact with one, fp32 inputs
// take three. Of a product of terms i and j those with i + j < 3 are formed: what
// is left out is below 2^-24 of the product.
#pragma once

#include <type_traits>

#include "ssd_delta.h"
#include "ssd_device.h"
#include "ssd_lin_chunk.h"

namespace ssd {

constexpr int kTerms = 3;

// Eight (four) floats as the sum of N terms each.
template <int N>
__device__ __forceinline__ void split8(const float* x, u32x4* out) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float lo = x[2 * c], hi = x[2 * c + 1];
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const uint32_t w = pack_bf16x2(lo, hi);
      out[t][c] = w;
      lo -= bf16_lo(w);
      hi -= bf16_hi(w);
    }
  }
}
template <int N>
__device__ __forceinline__ void split4(f32x4 x, u32x2* out) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float lo = x[2 * c], hi = x[2 * c + 1];
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const uint32_t w = pack_bf16x2(lo, hi);
      out[t][c] = w;
      lo -= bf16_lo(w);
      hi -= bf16_hi(w);
    }
  }
}

// acc += a b, of terms i and j with i + j < ORD; the small ones first.
template <int NA, int NB, int ORD>
__device__ __forceinline__ f32x4 mma(const u32x4* a, const u32x4* b, f32x4 acc) {
#pragma unroll
  for (int s = ORD - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) acc = mfma16x16x32(a[i], b[s - i], acc);
  return acc;
}

// acc += a b of one term of a, the i-th.
template <int NA, int NB, int ORD>
__device__ __forceinline__ f32x4 mma(const u32x4* a, const u32x4* b, int i, f32x4 acc) {
#pragma unroll
  for (int j = NB - 1; j >= 0; --j)
    if (i + j < ORD) acc = mfma16x16x32(a[0], b[j], acc);
  return acc;
}

// Eight values of a row as they come from memory, and as terms. NX: terms of an
// input, 1 for bf16 and 3 for fp32.
template <int NX>
struct Raw8 {
  u32x4 w[NX == 1 ? 1 : 2];
};
// Columns col .. col + 7 at byte offset `off` (kOffNone: zeros).
template <int NX>
__device__ __forceinline__ Raw8<NX> load8(rsrc_t r, uint32_t off) {
  Raw8<NX> x;
  x.w[0] = buf_load16(r, off);
  if constexpr (NX > 1) x.w[1] = buf_load16(r, off + 16);
  return x;
}
// Columns col .. col + 3 and col + 16 .. col + 19, the order of an accumulator pair.
template <int NX>
__device__ __forceinline__ Raw8<NX> load_pair(rsrc_t r, uint32_t lo, uint32_t hi) {
  Raw8<NX> x;
  if constexpr (NX == 1) {
    const u32x2 a = buf_load8(r, lo), b = buf_load8(r, hi);
    x.w[0] = u32x4{a.x, a.y, b.x, b.y};
  } else {
    x.w[0] = buf_load16(r, lo);
    x.w[1] = buf_load16(r, hi);
  }
  return x;
}
__device__ __forceinline__ void floats8(const Raw8<1>& x, float* f) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f[2 * c] = bf16_lo(x.w[0][c]);
    f[2 * c + 1] = bf16_hi(x.w[0][c]);
  }
}
__device__ __forceinline__ void floats8(const Raw8<3>& x, float* f) {
#pragma unroll
  for (int c = 0; c < 8; ++c) f[c] = __uint_as_float(x.w[c >> 2][c & 3]);
}
template <int NX>
__device__ __forceinline__ void terms8(const Raw8<NX>& x, u32x4* out) {
  if constexpr (NX == 1) {
    out[0] = x.w[0];
  } else {
    float f[8];
    floats8(x, f);
    split8<NX>(f, out);
  }
}

// Four values of a row.
template <int NX>
struct Raw4 {
  uint32_t w[NX == 1 ? 2 : 4];
};
template <int NX>
__device__ __forceinline__ Raw4<NX> load4(rsrc_t r, uint32_t off) {
  Raw4<NX> x;
  if constexpr (NX == 1) {
    const u32x2 a = buf_load8(r, off);
    x.w[0] = a.x;
    x.w[1] = a.y;
  } else {
    const u32x4 a = buf_load16(r, off);
#pragma unroll
    for (int c = 0; c < 4; ++c) x.w[c] = a[c];
  }
  return x;
}
template <int NX>
__device__ __forceinline__ f32x4 floats4(const Raw4<NX>& x) {
  if constexpr (NX == 1) return f32x4{bf16_lo(x.w[0]), bf16_hi(x.w[0]), bf16_lo(x.w[1]), bf16_hi(x.w[1])};
  else return f32x4{__uint_as_float(x.w[0]), __uint_as_float(x.w[1]), __uint_as_float(x.w[2]), __uint_as_float(x.w[3])};
}
template <int NX>
__device__ __forceinline__ void store4(f32x4 x, rsrc_t r, uint32_t off) {
  if constexpr (NX == 1) buf_store8(u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, r, off);
  else buf_store16(__builtin_bit_cast(u32x4, x), r, off);
}

// C x C matrices in the workspace as operands of 16 rows and 32 columns, columns in the order of an accumulator
// pair, in fp32: 64 lanes of the columns 4 g .., then 64 of the columns 16 + 4 g .., split into terms where they are
// used. What a CU has on its way from memory bounds the walks of few heads: with three terms in memory, half as much
// again, they took 9 to 13 % longer. A triangle's zero operands are not loaded.
constexpr int kOperand = 512;   // elements
__host__ __device__ constexpr long operands(int C) { return (long)(C / 16) * (C / 32) * kOperand; }
__device__ __forceinline__ int operand_at(int C, int rb, int kp) { return (rb * (C / 32) + kp) * kOperand; }
struct RawOperand {
  u32x4 w[2];
};
// P of fp32 inputs is there as its three terms, each 64 lanes of 16 bytes, one behind the other: the waves that take it
// have all other operands to split, and 8192 tokens, 32 heads on 16 of 128 x 128, took 833 us with it in fp32 for 794. With
// bf16 inputs it is the memory that counts, as above: 16384 tokens 579 us in fp32, 604 in terms (with two value blocks a
// workgroup the other way round: 2 x 4096 tokens 244 and 239).
template <int NX>
using ScoresIn = std::conditional_t<NX == 1, float, uint16_t>;
template <int C>
__device__ __forceinline__ long scores_at(const float*, long sh) { return sh * operands(C); }
template <int C>
__device__ __forceinline__ long scores_at(const uint16_t*, long sh) { return sh * kTerms * operands(C); }
struct TermOperand {
  u32x4 w[kTerms];
};
template <int NX>
using Scores = std::conditional_t<NX == 1, RawOperand, TermOperand>;
template <int N>
__device__ __forceinline__ void terms8(const RawOperand& x, u32x4* out) {
  float f[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) f[c] = __uint_as_float(x.w[c >> 2][c & 3]);
  split8<N>(f, out);
}
template <int N>
__device__ __forceinline__ void terms8(const TermOperand& x, u32x4* out) {
#pragma unroll
  for (int t = 0; t < N; ++t) out[t] = x.w[t];
}
// Row block rb of matrix sh; the operands from `least` to `most`, zeros in the place of the others.
template <int C>
__device__ __forceinline__ void load_operands(const float* from, long sh, int rb, int least, int most, int lane, RawOperand* to) {
  const rsrc_t r = make_rsrc(from + sh * operands(C), (uint32_t)(operands(C) * 4));
#pragma unroll
  for (int kp = 0; kp < C / 32; ++kp) {
    const uint32_t off = kp >= least && kp <= most ? (uint32_t)(operand_at(C, rb, kp) * 4 + lane * 16) : kOffNone;
    to[kp].w[0] = buf_load16(r, off);
    to[kp].w[1] = buf_load16(r, off + 1024);
  }
}
template <int C>
__device__ __forceinline__ void load_operands(const uint16_t* from, long sh, int rb, int least, int most, int lane, TermOperand* to) {
  const rsrc_t r = make_rsrc(from + scores_at<C>(from, sh), (uint32_t)(kTerms * operands(C) * 2));
#pragma unroll
  for (int kp = 0; kp < C / 32; ++kp) {
    const uint32_t off = kp >= least && kp <= most ? (uint32_t)(kTerms * operand_at(C, rb, kp) * 2 + lane * 16) : kOffNone;
#pragma unroll
    for (int t = 0; t < kTerms; ++t) to[kp].w[t] = buf_load16(r, off + t * kOperand * 2);
  }
}

// Element (16 rb + row, col) of such a matrix.
template <int C>
__device__ __forceinline__ float operand_value(const float* m, int rb, int row, int col) {
  return m[operand_at(C, rb, col / 32) + 256 * (col / 16 & 1) + (row + 16 * (col / 4 & 3)) * 4 + (col & 3)];
}
template <int C>
__device__ __forceinline__ float operand_value(const uint16_t* m, int rb, int row, int col) {
  const uint16_t* at = m + kTerms * operand_at(C, rb, col / 32) + (row + 16 * (col / 4 & 3)) * 8 + 4 * (col / 16 & 1) + (col & 3);
  float x = 0.f;
#pragma unroll
  for (int t = kTerms - 1; t >= 0; --t) x += bf16_to_f32(at[t * kOperand]);
  return x;
}

__device__ __forceinline__ bool not_finite(f32x4 x) {
  const float y = fmaf(x[0], 0.f, fmaf(x[1], 0.f, fmaf(x[2], 0.f, x[3] * 0.f)));
  return y != y;
}

// Everything loaded so far is there. Before a loop that loads ahead: the compiler's waits inside it are for the order
// of its own loads then, not for that of the loads before it.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// LDS rows of 16 nv values of a token, written 8 bytes a lane (16 rows) and read transposed (8 rows a half wave). One
// block of 16: rows of 32 bytes, one behind the other, the two halves of every second 8 rows exchanged; both accesses
// then cover the 64 banks once. (Padded rows of 48 bytes cost a walk 760 of its 1710 LDS cycles a chunk in conflicts;
// a third of them are left, and neither their number nor other pitches of the keys' rows show in its time.)
// More blocks: an odd multiple of 32 bytes.
__host__ __device__ constexpr int value_pitch(int nv) { return nv == 1 ? 16 : lds_pitch(16 * nv); }
template <int PITCH>
__device__ __forceinline__ int value_at(int row, int col) {
  return row * PITCH + (PITCH == 16 ? col ^ (row & 8) : col);
}

// e^x to an ulp or two, with the hardware's 2^y: what rounds off y = x log2(e) is put back to first order, and so is
// what log2(e) itself has below 24 bits, 1.3e-8 of it, which would be 9 ulp at x = -80. (With the library's exponential
// the matrices of 16384 tokens, 32 heads, took 119 us for 108.)
constexpr float kLog2eLow = 1.925963033e-8f;
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * kLog2e, rest = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -y));
  const float p = fast_exp2(y);
  return fmaf(p, rest * 0.69314718f, p);
}

// The chunk of a workgroup.
struct DeltaChunk {
  LinPiece p;    // p.blk < 0: none
  long row0;     // first token, flattened
  int n;         // tokens
};
template <int C>
__device__ __forceinline__ DeltaChunk delta_slot(const DeltaArgs& a, long slot) {
  DeltaChunk c;
  c.p = lin_piece(a.cu, a.S, a.T, C, a.slots_per_row, slot);
  c.row0 = c.p.start + (long)max(c.p.blk, 0) * C;
  c.n = min(C, c.p.len - max(c.p.blk, 0) * C);
  return c;
}
// Rows of a chunk of one head: row 0 at the buffer's start.
__device__ __forceinline__ rsrc_t chunk_rows(const void* base, long row0, long row, long col, int n, int esz) {
  return make_rsrc(static_cast<const char*>(base) + (row0 * row + col) * esz, (uint32_t)(n * row * esz));
}

}  // namespace ssd
