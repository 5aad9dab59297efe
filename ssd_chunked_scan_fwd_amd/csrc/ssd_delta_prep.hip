// ssd_delta_prep.hip -- the delta rule's matrices of every chunk: the gates'
// powers, P = scale D o Q K^T and the inverse T = (I + A)^-1 (ssd_delta.h).
//
// One workgroup takes a chunk of one query and key head and, one after the
// other, the value heads that share it: K K^T and Q K^T are formed once, on
// matrix instructions, and stay in registers.
// The inverse is taken by blocks, in fp32 throughout (matrix instructions on
// fp32): diagonal blocks of 16 by substitution, a lane a column, and twice
// T21 = -T22 A21 T11. That is substitution in another order, whose error is that
// of 32-bit sums for any A; sums of powers of A, which would need no
// substitution, cancel to nothing when keys repeat (A^32 of 64 equal keys
// reaches 10^17).
// T (with beta of its columns folded in) and P are stored as the operands that
// the walk over the chunks loads, and for the gradients their transposes.
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;

template <int C>
constexpr int kPitch = C + 4;   // floats; rows of 16-byte pieces

// Inclusive sum over the lanes 0..l, in 64 bits.
__device__ __forceinline__ double lanes_up(double x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ f32x4 mfma_f32(f32x4 a, f32x4 b, f32x4 c) {
  // Four steps of k = 4 each; step r takes k = 4 g + r, so that an accumulator is an operand as it stands.
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}
template <int C>
__device__ __forceinline__ f32x4 block_rows(const float* M, int rb, int cb, int c16, int g) {   // [c16][4 g + r]
  return *reinterpret_cast<const f32x4*>(M + (16 * rb + c16) * kPitch<C> + 16 * cb + 4 * g);
}
template <int C>
__device__ __forceinline__ f32x4 block_cols(const float* M, int rb, int cb, int c16, int g) {   // [4 g + r][c16]
  f32x4 x;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = M[(16 * rb + 4 * g + r) * kPitch<C> + 16 * cb + c16];
  return x;
}
template <int C>
__device__ __forceinline__ void put_cols(float* M, int rb, int cb, int c16, int g, f32x4 x) {
#pragma unroll
  for (int r = 0; r < 4; ++r) M[(16 * rb + 4 * g + r) * kPitch<C> + 16 * cb + c16] = -x[r];
}

// Tm := (I + Am)^-1, lower triangles. Tm's blocks above the diagonal are zero.
template <int C>
__device__ __forceinline__ void invert(const float* Am, float* Tm, int wave, int lane) {
  const int c16 = lane & 15, g = lane >> 4;
  if (wave == 0 && lane < C) {
    float t[16];
    const float* A = Am + 16 * g * kPitch<C> + 16 * g;
    float* out = Tm + 16 * g * kPitch<C> + 16 * g + c16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f32x4 row[4];
#pragma unroll
      for (int j = 0; 4 * j < i; ++j) row[j] = *reinterpret_cast<const f32x4*>(A + i * kPitch<C> + 4 * j);
      float x = c16 == i ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) x = fmaf(-row[j >> 2][j & 3], t[j], x);
      t[i] = x;
      out[i * kPitch<C>] = x;
    }
  }
  __syncthreads();
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if (wave < C / 32) {
    const int lo = 2 * wave, hi = lo + 1;
    const f32x4 R = mfma_f32(block_rows<C>(Am, hi, lo, c16, g), block_cols<C>(Tm, lo, lo, c16, g), zero);
    put_cols<C>(Tm, hi, lo, c16, g, mfma_f32(block_rows<C>(Tm, hi, hi, c16, g), R, zero));
  }
  if constexpr (C == 64) {
    __syncthreads();
    const int ir = wave >> 1, jc = wave & 1;
    f32x4 x = zero;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      f32x4 R = zero;
#pragma unroll
      for (int n = 0; n < 2; ++n) R = mfma_f32(block_rows<C>(Am, 2 + m, n, c16, g), block_cols<C>(Tm, n, jc, c16, g), R);
      x = mfma_f32(block_rows<C>(Tm, 2 + ir, 2 + m, c16, g), R, x);
    }
    put_cols<C>(Tm, 2 + ir, jc, c16, g, x);
  }
}

// Operand (rb, kp) of a matrix, or of its transpose, its columns times w.
template <int C, bool TR>
__device__ __forceinline__ void put_operand(const float* M, float* to, int rb, int kp, const float* w, int lane) {
  const int c16 = lane & 15, g = lane >> 4, row = 16 * rb + c16;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int col = 32 * kp + 16 * t + 4 * g;
    f32x4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = TR ? M[(col + r) * kPitch<C> + row] : M[row * kPitch<C> + col + r];
      if (w) x[r] *= w[col + r];
    }
    *reinterpret_cast<f32x4*>(to + operand_at(C, rb, kp) + 256 * t + lane * 4) = x;
  }
}

// The pairs of 16 rows and 16 columns on or below the diagonal that wave w takes: (row, column), -1: none.
template <int C>
__device__ __forceinline__ void tile_of(int wave, int e, int& ib, int& jb) {
  constexpr int kOf64[4][3] = {{12, 13, 0}, {14, 15, 4}, {8, 9, -1}, {10, 5, -1}};
  constexpr int kOf32[4] = {0, 4, 5, -1};
  int t = -1;
  if constexpr (C == 64) {
#pragma unroll
    for (int w = 0; w < 4; ++w) t = wave == w ? kOf64[w][e] : t;
  } else {
#pragma unroll
    for (int w = 0; w < 4; ++w) t = wave == w ? kOf32[w] : t;
  }
  ib = t < 0 ? -1 : t >> 2;
  jb = t & 3;
}

template <int C, int KB, int NX, bool BWD>
__global__ __launch_bounds__(kThreads, 2) void delta_prep_kernel(DeltaArgs a) {
  constexpr int kTiles = C == 64 ? 3 : 1;   // a wave
  constexpr int kEsz = NX == 1 ? 2 : 4;
  __shared__ __align__(16) float Am[C * kPitch<C>], Tm[C * kPitch<C>], Pm[C * kPitch<C>];
  __shared__ __align__(16) float Gh[C], Gl[C], Be[C];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const long unit = xcd_unit(blockIdx.x, gridDim.x);
  const int hk = (int)(unit % a.Hk);
  const long slot = unit / a.Hk;
  const DeltaChunk ch = delta_slot<C>(a, slot);
  if (ch.p.blk < 0 || ch.n <= 0) return;
  const int n = ch.n, rep = a.H / a.Hk;
  const rsrc_t rk = chunk_rows(a.k, ch.row0, a.k_row, (long)hk * a.dk, n, kEsz);
  const rsrc_t rq = chunk_rows(a.q, ch.row0, a.q_row, (long)hk * a.dk, n, kEsz);
  const int krow = (int)a.k_row * kEsz, qrow = (int)a.q_row * kEsz;
  for (int i = threadIdx.x; i < C * kPitch<C>; i += kThreads) Tm[i] = Pm[i] = 0.f;

  f32x4 kk[kTiles], qk[kTiles];   // of queries and keys i (columns c16) and keys j (rows 4 g + r)
#pragma unroll
  for (int e = 0; e < kTiles; ++e) {
    kk[e] = qk[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    int ib, jb;
    tile_of<C>(wave, e, ib, jb);
    if (ib < 0) continue;
    const int i = 16 * ib + c16, j = 16 * jb + c16;
    Raw8<NX> xi[KB], xj[KB], xq[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int col = 32 * b + 8 * g;
      const bool in = col < a.dk;
      xi[b] = load8<NX>(rk, in && i < n ? (uint32_t)(i * krow + col * kEsz) : kOffNone);
      xj[b] = load8<NX>(rk, in && j < n ? (uint32_t)(j * krow + col * kEsz) : kOffNone);
      xq[b] = load8<NX>(rq, in && i < n ? (uint32_t)(i * qrow + col * kEsz) : kOffNone);
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      u32x4 ti[NX], tj[NX], tq[NX];
      terms8<NX>(xi[b], ti);
      terms8<NX>(xj[b], tj);
      terms8<NX>(xq[b], tq);
      kk[e] = mma<NX, NX, NX>(tj, ti, kk[e]);
      qk[e] = mma<NX, NX, NX>(tj, tq, qk[e]);
    }
  }

  for (int m = 0; m < rep; ++m) {
    const int h = hk * rep + m;
    const long sh = slot * a.H + h;
    float* gates = a.gates + sh * kGateRows * C;
    if (m > 0) __syncthreads();   // the last head's operands are out
    if (wave == 0) {
      const bool in = lane < n;
      const long at = (ch.row0 + min(lane, n - 1)) * a.H + h;
      // Below -200 a decay is 0 in fp32, as e^-200 is, and its sums stay finite.
      float x = in && a.g ? a.g[at] : 0.f;
      x = x < -200.f ? -200.f : x;
      const float be = in ? a.beta[at] : 0.f;
      const double G = lanes_up((double)x, lane), end = __shfl(G, C - 1);
      if (lane < C) {
        const float hi = (float)G, lo = (float)(G - (double)hi);
        Gh[lane] = hi;
        Gl[lane] = lo;
        Be[lane] = be;
        gates[lane] = (float)exp(G);
        gates[C + lane] = in ? (float)exp(end - G) : 0.f;
        gates[2 * C + lane] = be;
        gates[3 * C + lane] = hi;
        gates[4 * C + lane] = lo;
        if (lane == 0) gates[5 * C] = (float)exp(end);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kTiles; ++e) {
      int ib, jb;
      tile_of<C>(wave, e, ib, jb);
      if (ib < 0) continue;
      const int i = 16 * ib + c16, j = 16 * jb + 4 * g;
      const float hi = Gh[i], lo = Gl[i], be = Be[i];
      f32x4 A, P;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float d = j + r <= i ? expf((hi - Gh[j + r]) + (lo - Gl[j + r])) : 0.f;
        A[r] = j + r < i ? be * d * kk[e][r] : 0.f;
        P[r] = j + r <= i ? a.scale * d * qk[e][r] : 0.f;
      }
      *reinterpret_cast<f32x4*>(Am + i * kPitch<C> + j) = A;
      *reinterpret_cast<f32x4*>(Pm + i * kPitch<C> + j) = P;
    }
    __syncthreads();
    invert<C>(Am, Tm, wave, lane);
    __syncthreads();
    // Operands on or below the diagonal, of the transposes on or above it.
    const long at = sh * operands(C);
    for (int t = wave; t < (C / 16) * (C / 32); t += 4) {
      const int rb = t / (C / 32), kp = t % (C / 32);
      if (kp <= rb / 2) {
        put_operand<C, false>(Tm, a.tf + at, rb, kp, Be, lane);
        if (!BWD) put_operand<C, false>(Pm, a.pf + at, rb, kp, nullptr, lane);
      }
      if (BWD && kp >= rb / 2) {
        put_operand<C, true>(Tm, a.tt + at, rb, kp, nullptr, lane);
        put_operand<C, true>(Pm, a.pt + at, rb, kp, nullptr, lane);
      }
    }
  }
}

template <int C, int NX, bool BWD>
void prep(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.slots * a.Hk));
  if (a.dk <= 32) hipLaunchKernelGGL((delta_prep_kernel<C, 1, NX, BWD>), grid, dim3(kThreads), 0, stream, a);
  else if (a.dk <= 64) hipLaunchKernelGGL((delta_prep_kernel<C, 2, NX, BWD>), grid, dim3(kThreads), 0, stream, a);
  else if (a.dk <= 128) hipLaunchKernelGGL((delta_prep_kernel<C, 4, NX, BWD>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((delta_prep_kernel<C, 8, NX, BWD>), grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

size_t delta_gates_bytes(bool bf16) { return (size_t)kGateRows * delta_chunk(bf16) * 4; }
size_t delta_matrix_bytes(bool bf16) { return (size_t)operands(delta_chunk(bf16)) * 4; }
int delta_prep_threads() { return kThreads; }

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream) {
  if (a.bf16) backward ? prep<64, 1, true>(a, stream) : prep<64, 1, false>(a, stream);
  else backward ? prep<32, 3, true>(a, stream) : prep<32, 3, false>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
