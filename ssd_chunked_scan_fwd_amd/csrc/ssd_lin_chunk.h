// ssd_lin_chunk.h -- what the linear-attention kernels on matrix instructions
// share: chunks of 64 tokens, powers of the decay in LDS, rows staged by
// 16-byte pieces, LDS operands in the order of an accumulator pair.
#pragma once

#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

constexpr int kC = 64;                       // tokens a chunk
constexpr int kPitchP = lds_pitch(kC);       // LDS row of 64 scores

// Powers of the decay, pw[kPowZero + e] = lam^e for e = 0 .. 64 and 0 for e = -64
// .. -1, spw scale times them, pw[kPowHi] and the next lam as a sum of two floats:
// the weight of every pair and token of a chunk is one LDS read (an exponential
// costs a wave as long as sixteen multiplies, and a chunk has some forty weights a
// lane). They are rounded once, from 64 bits: lam^64 carries the state from chunk
// to chunk, and an error in it compounds.
constexpr int kPowZero = 64, kPowHi = 130, kPowSize = 132;
__device__ __forceinline__ void fill_powers(float* pw, float* spw, float log_decay, float scale) {
  for (int i = threadIdx.x; i < kPowHi; i += blockDim.x) {
    const double x = i < kPowZero ? 0.0 : lin_power(log_decay, i - kPowZero);
    pw[i] = (float)x;
    if (spw) spw[i] = (float)(x * (double)scale);
    if (i == kPowZero + 1) {
      const LinDecay lam = lin_split(x);
      pw[kPowHi] = lam.hi;
      pw[kPowHi + 1] = lam.lo;
    }
  }
}

// Weights of the tokens 32 kp + 16 (s / 4) + 4 g + s % 4, s = 0 .. 7, of a chunk
// of n: lam^(n - 1 - token), 0 behind the chunk. pw is 16-byte aligned.
__device__ __forceinline__ void token_weights(const float* pw, int n, int kp, int g, float* w) {
  if (n == kC) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(pw + kPowZero + 60 - 32 * kp - 16 * t - 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) w[4 * t + r] = x[3 - r];
    }
  } else {
    const float* at = pw + kPowZero + n - 1 - 32 * kp - 4 * g;
#pragma unroll
    for (int s = 0; s < 8; ++s) w[s] = at[-16 * (s >> 2) - (s & 3)];
  }
}

// v w, element by element, as the sum of TERMS bf16 values, each rounded to
// nearest: two leave 2^-16 of it, three 2^-24.
template <int TERMS>
__device__ __forceinline__ void split_weighted(u32x4 v, const float* w, u32x4* part) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x = bf16_lo(v[c]) * w[2 * c], y = bf16_hi(v[c]) * w[2 * c + 1];
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      part[t][c] = pack_bf16x2(x, y);
      x -= bf16_lo(part[t][c]);
      y -= bf16_hi(part[t][c]);
    }
  }
}

// A load of rows that no later launch reads again: it leaves the caches to
// those that are. With it the forward pass of 16384 tokens takes 200 us instead
// of 208. Calls whose rows are all in the caches already, as back to back on the
// same tensors, take longer: backwards, 8192 tokens, 256 us instead of 243, the
// ragged batch of 5087 tokens 37 instead of 34.
__device__ __forceinline__ u32x4 buf_load16_once(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2));
}

// Byte offset, from a chunk's lowest row in memory, of a piece at row r and
// column col: fixed for whole chunks (`full`); a short reversed chunk starts
// nearer. Rows behind the chunk and columns behind `end` give kOffNone.
struct Piece {
  uint32_t full;
  int row;   // chunk row, or kC where the columns end before
};
__device__ __forceinline__ Piece make_piece(int r, int col, int end, int row_bytes, int esz, int rev) {
  return Piece{(uint32_t)((rev ? kC - 1 - r : r) * row_bytes + col * esz), col < end ? r : kC};
}
__device__ __forceinline__ uint32_t piece_offset(const Piece& p, int n, int row_bytes, int rev) {
  return p.row < n ? p.full - (rev ? (uint32_t)((kC - n) * row_bytes) : 0u) : kOffNone;
}

// A 16-byte piece c8 (of four) of 32 columns, stored in the order of an
// accumulator pair: column 16 t + 4 g + k at 8 g + 4 t + k.
__device__ __forceinline__ void store_paired(uint16_t* row, int j, int c8, u32x4 v) {
  uint16_t* at = row + 32 * j + 16 * (c8 & 1) + 4 * (c8 >> 1);
  *reinterpret_cast<u32x2*>(at) = u32x2{v.x, v.y};
  *reinterpret_cast<u32x2*>(at + 8) = u32x2{v.z, v.w};
}
// Tiles in the columns' own order that are read in that one: rows 8..15 of every
// 16 lie 8 elements further on (inside the padding), so that the 8-byte accesses
// of half a wave, two of each of 16 rows, cover the 64 banks once where rows r
// and r + 8 would share them (dK and dV of 8192 tokens: 6.7 instead of 12.5
// million cycles of conflicts, 122 instead of 126 us).
__device__ __forceinline__ int row_shift(int r) { return r & 8; }
// Rows row0 + c16, k in the order of an accumulator pair.
__device__ __forceinline__ u32x4 frag_k_cols_pairs(const uint16_t* W, int pitch, int row0, int col0, int lane) {
  const int r = lane & 15;
  const uint16_t* at = W + (row0 + r) * pitch + row_shift(r) + col0 + 4 * (lane >> 4);
  const u32x2 lo = *reinterpret_cast<const u32x2*>(at), hi = *reinterpret_cast<const u32x2*>(at + 16);
  return u32x4{lo.x, lo.y, hi.x, hi.y};
}
// frag_k_rows_accpair of such a tile.
__device__ __forceinline__ u32x4 frag_k_rows_shifted(const uint16_t* W, int pitch, int row0, int col0, int lane) {
  return frag_k_rows_accpair(W + row_shift(4 * (lane >> 4)), pitch, row0, col0, lane);
}

// Two blocks of 16 weighted scores as bf16 operand (slots of an accumulator pair)
// at `at`. The first 32 tokens of a sequence have few scores, whose roundings do
// not average out: what rounding leaves of those goes 32 columns on, a place that
// their rows do not use (its keys are later), for a product of its own.
__device__ __forceinline__ void store_scores(uint16_t* at, f32x4 s0, f32x4 s1, bool rest) {
  const u32x4 hi = {pack_bf16x2(s0[0], s0[1]), pack_bf16x2(s0[2], s0[3]), pack_bf16x2(s1[0], s1[1]), pack_bf16x2(s1[2], s1[3])};
  *reinterpret_cast<u32x4*>(at) = hi;
  if (!rest) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    s0[r] -= r & 1 ? bf16_hi(hi[r >> 1]) : bf16_lo(hi[r >> 1]);
    s1[r] -= r & 1 ? bf16_hi(hi[2 + (r >> 1)]) : bf16_lo(hi[2 + (r >> 1)]);
  }
  *reinterpret_cast<u32x4*>(at + 32) =
      u32x4{pack_bf16x2(s0[0], s0[1]), pack_bf16x2(s0[2], s0[3]), pack_bf16x2(s1[0], s1[1]), pack_bf16x2(s1[2], s1[3])};
}

// A pointer that all lanes hold, in scalar registers.
template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t at = (uint64_t)p;
  return (const T*)((uint64_t)(uint32_t)uniform((int)at) | (uint64_t)(uint32_t)uniform((int)(at >> 32)) << 32);
}
__device__ __forceinline__ f32x4 four(u32x2 w) { return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)}; }

}  // namespace ssd
