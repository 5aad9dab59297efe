// ssd_delta_prep.hip -- the delta rule's matrices of every chunk: the gates'
// powers, P = scale D o Q K^T and the inverse T = (I + A)^-1 (ssd_delta.h).
//
// One workgroup takes a chunk of one query and key head and, one after the
// other, the value heads that share it: K K^T and Q K^T are formed once, on
// matrix instructions, and stay in registers.
// The inverse is taken by blocks, in place in LDS, in fp32 throughout (matrix
// instructions on fp32): diagonal blocks of 16 by substitution, a lane a column, and
// twice T21 = -T22 A21 T11. That is substitution in another order, whose error is
// that of 32-bit sums for any A; sums of powers of A, which would need no
// substitution, cancel to nothing when keys repeat (A^32 of 64 equal keys
// reaches 10^17).
// T (with beta of its columns folded in) and P are stored as the operands that
// the walk over the chunks loads, and for the gradients their transposes. A tile of
// P is such an operand as its accumulators hold it.
// 16384 tokens, 32 heads on 16 of 128 x 128: 100 us, 143 MB read and 237 MB written (3.8 TB/s), the vector units
// busy 33 % of the time, matrix units 17 %, LDS 28 %: the inverse's dependent steps bound it, four workgroups a CU.
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;

template <int C>
constexpr int kPitch = C + 4;   // floats; rows of 16-byte pieces

// Inclusive sum over the lanes 0..l, in 64 bits: wave_incl_scan on both halves of a double.
template <int CTRL, int ROWS>
__device__ __forceinline__ double pick64(double x) {
  const long v = __builtin_bit_cast(long, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v & 0xffffffffL), CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lanes_up(double x) {
  x += pick64<0x111, 0xF>(x);
  x += pick64<0x112, 0xF>(x);
  x += pick64<0x114, 0xF>(x);
  x += pick64<0x118, 0xF>(x);
  x += pick64<0x142, 0xA>(x);
  x += pick64<0x143, 0xC>(x);
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

// M := (I + M)^-1, lower triangles; M's blocks above the diagonal are zero.
template <int C>
__device__ __forceinline__ void invert(float* M, int wave, int lane) {
  const int c16 = lane & 15, g = lane >> 4;
  if (wave == 0 && lane < C) {
    float t[16];
    float* A = M + 16 * g * kPitch<C> + 16 * g;
    f32x4 row[3][4];   // two rows ahead
    auto load = [&](int i) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * j < i && i < 16) row[i % 3][j] = *reinterpret_cast<const f32x4*>(A + i * kPitch<C> + 4 * j);
    };
    load(1);
    load(2);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = c16 == i ? 1.f : 0.f, y = 0.f;   // two chains
#pragma unroll
      for (int j = 0; j < i; ++j) {
        float& to = j & 1 ? y : x;
        to = fmaf(-row[i % 3][j >> 2][j & 3], t[j], to);
      }
      t[i] = x + y;
      load(i + 3);
      A[i * kPitch<C> + c16] = t[i];
    }
  }
  __syncthreads();
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if (wave < C / 32) {
    const int lo = 2 * wave, hi = lo + 1;
    const f32x4 R = mfma_f32(block_rows<C>(M, hi, lo, c16, g), block_cols<C>(M, lo, lo, c16, g), zero);
    put_cols<C>(M, hi, lo, c16, g, mfma_f32(block_rows<C>(M, hi, hi, c16, g), R, zero));
  }
  if constexpr (C == 64) {
    __syncthreads();
    const int ir = wave >> 1, jc = wave & 1;
    f32x4 x = zero;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      f32x4 R = zero;
#pragma unroll
      for (int n = 0; n < 2; ++n) R = mfma_f32(block_rows<C>(M, 2 + m, n, c16, g), block_cols<C>(M, n, jc, c16, g), R);
      x = mfma_f32(block_rows<C>(M, 2 + ir, 2 + m, c16, g), R, x);
    }
    __syncthreads();   // all have read what is replaced
    put_cols<C>(M, 2 + ir, jc, c16, g, x);
  }
}

// Operand (rb, kp) of a matrix, or of its transpose, its columns times w, in fp32.
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
// Half of an operand, the columns 16 cb ..: a tile as its accumulators hold it (rows c16, columns 4 g + r).
template <int C>
__device__ __forceinline__ void put_tile(f32x4 x, float* to, int rb, int cb, int lane) {
  *reinterpret_cast<f32x4*>(to + operand_at(C, rb, cb / 2) + 256 * (cb & 1) + lane * 4) = x;
}
template <int C>
__device__ __forceinline__ void put_tile(f32x4 x, uint16_t* to, int rb, int cb, int lane) {
  u32x2 part[kTerms];
  split4<kTerms>(x, part);
  uint16_t* at = to + kTerms * operand_at(C, rb, cb / 2) + lane * 8 + 4 * (cb & 1);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) *reinterpret_cast<u32x2*>(at + t * kOperand) = part[t];
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
__global__ __launch_bounds__(kThreads, BWD ? 3 : 4) void delta_prep_kernel(DeltaArgs a, int heads) {
  constexpr int kTiles = C == 64 ? 3 : 1;   // a wave
  constexpr int kEsz = NX == 1 ? 2 : 4;
  // Rows of K and Q, kSlab pieces of 32 columns at a time, and in their place the matrix.
  constexpr int kSlab = NX == 1 ? (KB < 4 ? KB : 4) : (KB < 2 ? KB : 2), kPitchK = lds_pitch(32 * kSlab);
  constexpr int kRows = NX * C * kPitchK, kBytes = 4 * kRows > 4 * C * kPitch<C> ? 4 * kRows : 4 * C * kPitch<C>;
  __shared__ __align__(16) char shared[kBytes];
  uint16_t* const Kl = reinterpret_cast<uint16_t*>(shared);
  uint16_t* const Ql = Kl + kRows;
  float* const Am = reinterpret_cast<float*>(shared);
  __shared__ __align__(16) float Gh[4][C], Gl[4][C], Be[4][C];   // of four heads at a time
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const long unit = xcd_unit(blockIdx.x, gridDim.x);
  const int rep = a.H / a.Hk, parts = (rep + heads - 1) / heads;   // `heads` value heads a workgroup
  const int part = (int)(unit % parts), hk = (int)((unit / parts) % a.Hk), first = part * heads, end = min(first + heads, rep);
  const long slot = unit / ((long)parts * a.Hk);
  const DeltaChunk ch = delta_slot<C>(a, slot);
  if (ch.p.blk < 0 || ch.n <= 0) return;
  const int n = ch.n;
  const rsrc_t rk = chunk_rows(a.k, ch.row0, a.k_row, (long)hk * a.dk, n, kEsz);
  const rsrc_t rq = chunk_rows(a.q, ch.row0, a.q_row, (long)hk * a.dk, n, kEsz);
  const int krow = (int)a.k_row * kEsz, qrow = (int)a.q_row * kEsz;
  float gx = 0.f, bx = 0.f;   // the gates of this lane's token, of head m0 + wave
  auto load_gates = [&](int m0) {
    const long at = (ch.row0 + min(lane, n - 1)) * a.H + hk * rep + min(m0 + wave, end - 1);
    if (a.g) gx = a.g[at];
    bx = a.beta[at];
  };
  load_gates(first);
  // Of keys j (rows 4 g + r) and queries or keys i (columns c16); BWD: Q K^T the other way round, as its transpose is stored.
  f32x4 kk[kTiles], qk[kTiles];
#pragma unroll
  for (int e = 0; e < kTiles; ++e) kk[e] = qk[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s0 = 0; s0 < KB; s0 += kSlab) {
    if (s0 > 0) __syncthreads();
    // A wave's 16 rows of K and of Q; with 32 tokens of one of the two. Rows behind the chunk lie behind the buffers' ends.
    Raw8<NX> xk[kSlab], xq[kSlab];
    const int rb = wave % (C / 16), row = 16 * rb + c16;
    const bool of_k = C == 64 || wave < 2, of_q = C == 64 || wave >= 2;
#pragma unroll
    for (int b = 0; b < kSlab; ++b) {
      const int col = 32 * (s0 + b) + 8 * g;
      xk[b] = load8<NX>(rk, of_k && col < a.dk ? (uint32_t)(row * krow + col * kEsz) : kOffNone);
      xq[b] = load8<NX>(rq, of_q && col < a.dk ? (uint32_t)(row * qrow + col * kEsz) : kOffNone);
    }
#pragma unroll
    for (int b = 0; b < kSlab; ++b) {
      u32x4 tk[NX], tq[NX];
      terms8<NX>(xk[b], tk);
      terms8<NX>(xq[b], tq);
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        if (of_k) *reinterpret_cast<u32x4*>(Kl + (t * C + row) * kPitchK + 32 * b + 8 * g) = tk[t];
        if (of_q) *reinterpret_cast<u32x4*>(Ql + (t * C + row) * kPitchK + 32 * b + 8 * g) = tq[t];
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kTiles; ++e) {
      int ib, jb;
      tile_of<C>(wave, e, ib, jb);
      if (ib < 0) continue;
#pragma unroll
      for (int b = 0; b < kSlab; ++b) {
        u32x4 ti[NX], tj[NX], tq[NX];
#pragma unroll
        for (int t = 0; t < NX; ++t) {
          ti[t] = frag_k_cols(Kl + t * C * kPitchK, kPitchK, 16 * ib, 32 * b, lane);
          tj[t] = frag_k_cols(Kl + t * C * kPitchK, kPitchK, 16 * jb, 32 * b, lane);
          tq[t] = frag_k_cols(Ql + t * C * kPitchK, kPitchK, 16 * ib, 32 * b, lane);
        }
        kk[e] = mma<NX, NX, NX>(tj, ti, kk[e]);
        qk[e] = BWD ? mma<NX, NX, NX>(tq, tj, qk[e]) : mma<NX, NX, NX>(tj, tq, qk[e]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < C * kPitch<C>; i += kThreads) Am[i] = 0.f;

  for (int m = first; m < end; ++m) {
    const int h = hk * rep + m, mw = (m - first) & 3;
    const long sh = slot * a.H + h;
    if (m > first) __syncthreads();   // the last head's operands are out
    if (mw == 0) {
      if (m + wave < end) {
        float* gates = a.gates + (sh + wave) * kGateRows * C;
        const bool in = lane < n;
        // Below -200 a decay is 0 in fp32, as e^-200 is, and its sums stay finite.
        const float x = !in ? 0.f : gx < -200.f ? -200.f : gx, be = in ? bx : 0.f;
        const double G = lanes_up((double)x), end = __shfl(G, C - 1);
        if (lane < C) {
          const float hi = (float)G, lo = (float)(G - (double)hi);
          Gh[wave][lane] = hi;
          Gl[wave][lane] = lo;
          Be[wave][lane] = be;
          const double left = end - G;
          const float lh = (float)left, ll = (float)(left - (double)lh);
          gates[lane] = exp_of(hi) * (1.f + lo);
          gates[C + lane] = in ? exp_of(lh) * (1.f + ll) : 0.f;
          gates[2 * C + lane] = be;
          gates[3 * C + lane] = hi;
          gates[4 * C + lane] = lo;
          if (lane == C - 1) gates[5 * C] = exp_of(hi) * (1.f + lo);
        }
      }
      if (m + 4 < end) load_gates(m + 4);
      __syncthreads();
    }
    const float *gh = Gh[mw], *gl = Gl[mw], *bt = Be[mw];
#pragma unroll
    for (int e = 0; e < kTiles; ++e) {
      int ib, jb;
      tile_of<C>(wave, e, ib, jb);
      if (ib < 0) continue;
      const int i = 16 * ib + c16, j = 16 * jb + 4 * g;
      const f32x4 hj = *reinterpret_cast<const f32x4*>(gh + j), lj = *reinterpret_cast<const f32x4*>(gl + j);
      const float hi = gh[i], lo = gl[i], be = bt[i];
      f32x4 d, A, P;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        d[r] = j + r <= i ? exp_of((hi - hj[r]) + (lo - lj[r])) : 0.f;
        A[r] = j + r < i ? be * d[r] * kk[e][r] : 0.f;
      }
      *reinterpret_cast<f32x4*>(Am + i * kPitch<C> + j) = A;
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      if (BWD) {
        const int i4 = 16 * ib + 4 * g, j1 = 16 * jb + c16;
        const f32x4 hr = *reinterpret_cast<const f32x4*>(gh + i4), lr = *reinterpret_cast<const f32x4*>(gl + i4);
        const float h1 = gh[j1], l1 = gl[j1];
#pragma unroll
        for (int r = 0; r < 4; ++r) P[r] = j1 <= i4 + r ? a.scale * exp_of((hr[r] - h1) + (lr[r] - l1)) * qk[e][r] : 0.f;
        float* to = a.pt + sh * operands(C);
        put_tile<C>(P, to, jb, ib, lane);
        if (ib == jb && (ib & 1)) put_tile<C>(zero, to, jb, ib - 1, lane);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) P[r] = j + r <= i ? a.scale * d[r] * qk[e][r] : 0.f;
        ScoresIn<NX>* to = static_cast<ScoresIn<NX>*>(a.pf);
        to += scores_at<C>(to, sh);
        put_tile<C>(P, to, ib, jb, lane);
        if (ib == jb && !(ib & 1)) put_tile<C>(zero, to, ib, jb + 1, lane);
      }
    }
    __syncthreads();
    invert<C>(Am, wave, lane);
    __syncthreads();
    // Operands on or below the diagonal, of the transpose on or above it.
    for (int t = wave; t < (C / 16) * (C / 32); t += 4) {
      const int rb = t / (C / 32), kp = t % (C / 32);
      if (kp <= rb / 2) put_operand<C, false>(Am, a.tf + sh * operands(C), rb, kp, bt, lane);
      if (BWD && kp >= rb / 2) put_operand<C, true>(Am, a.tt + sh * operands(C), rb, kp, nullptr, lane);
    }
  }
}

// Value heads a workgroup: all that share its keys, whose products it makes once, or so few that the launch has
// four workgroups for every CU. A workgroup's time is mostly waits: 5087 tokens of 16 heads on 4, 348 workgroups of four
// heads took 25.4 us, 1392 of one 22.5; 8192 of 4 on 2, 256 of two 15.7 and 512 of one 14.3. From 1024 on the products count
// (calls, us): 4096 tokens of 32 on 16, 128 x 128, 1024 of two 140, 2048 of one 146; 4 x 2048 of 32 on 8, 64 x 64, 1024 of
// four 105, 4096 of one 128; 16384 of 32 on 16, 4096 of two 581, 8192 of one 605.
int heads_a_workgroup(const DeltaArgs& a) {
  const int rep = a.H / a.Hk;
  int heads = rep;
  while (heads > 1 && a.slots * a.Hk * ((rep + heads - 1) / heads) < 1024) heads = (heads + 1) / 2;
  return heads;
}

template <int C, int NX, bool BWD>
void prep(const DeltaArgs& a, hipStream_t stream) {
  const int heads = heads_a_workgroup(a), rep = a.H / a.Hk;
  const dim3 grid((unsigned)(a.slots * a.Hk * ((rep + heads - 1) / heads)));
  if (a.dk <= 32) hipLaunchKernelGGL((delta_prep_kernel<C, 1, NX, BWD>), grid, dim3(kThreads), 0, stream, a, heads);
  else if (a.dk <= 64) hipLaunchKernelGGL((delta_prep_kernel<C, 2, NX, BWD>), grid, dim3(kThreads), 0, stream, a, heads);
  else if (a.dk <= 128) hipLaunchKernelGGL((delta_prep_kernel<C, 4, NX, BWD>), grid, dim3(kThreads), 0, stream, a, heads);
  else hipLaunchKernelGGL((delta_prep_kernel<C, 8, NX, BWD>), grid, dim3(kThreads), 0, stream, a, heads);
}

}  // namespace

size_t delta_gates_bytes(bool bf16) { return (size_t)kGateRows * delta_chunk(bf16) * 4; }
size_t delta_tf_bytes(bool bf16) { return (size_t)operands(delta_chunk(bf16)) * 4; }
size_t delta_pf_bytes(bool bf16) { return (size_t)operands(delta_chunk(bf16)) * (bf16 ? 4 : 2 * kTerms); }
int delta_prep_threads() { return kThreads; }

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream) {
  if (a.bf16) backward ? prep<64, 1, true>(a, stream) : prep<64, 1, false>(a, stream);
  else backward ? prep<32, 3, true>(a, stream) : prep<32, 3, false>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
