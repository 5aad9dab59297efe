// ssd_delta_bwd.hip -- the delta rule's gradients of q, k, beta and the log
// decays, for all chunks at once, from what the walks left of each: the state S0
// before it, the gradient dS1 of the state behind it, U and U' (ssd_delta.h).
// With Z1_ij = dO_i . U_j and Z2_ij = U'_i . U_j:
//     r_i  = -(e^G_i (U' S0)_i + sum_{j < i} D_ij Z2_ij k_j)        reads of k
//     w_j  = e^(G_C - G_j) (U dS1)_j + scale sum_{i >= j} D_ij Z1_ij q_i
//            - sum_{i > j} beta_i D_ij Z2_ij k_i                    writes of k
//     dq_i = scale (e^G_i (dO S0)_i + sum_{j <= i} D_ij Z1_ij k_j)
//     dk   = beta r + w,   dbeta_i = U'_i . v_i + k_i . r_i.
// e^G_i stands before q_i and the reads of k_i, e^-G_j before its writes, so with
// E_i = q_i . dq_i + beta_i k_i . r_i - k_i . w_i
//     dg_t = <dS1, S1> + sum_{i >= t} E_i   (tokens of the chunk),
//     <dS1, S1> = e^(G_C) <dS1, S0> + sum_j e^(G_C - G_j) k_j . (U dS1)_j.
//
// A workgroup takes one chunk of one head, two waves 16 tokens, each half of the key
// columns. First, over the value columns 32 at a time, the products with the states
// (contraction over the columns, the states' terms in LDS) and, one of the two waves
// each, Z1 and Z2 of the tokens, both as rows and as columns; then the products of
// the masked Z, which go round through LDS, with Q and K, whose rows take the
// states' place there.
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int threads_of(int C) { return 8 * C; }   // two waves for 16 tokens
constexpr int kPitchT = lds_pitch(32);   // rows of 32 value columns, in the order of an accumulator pair

template <int C, int KB, int NX>
__global__ __launch_bounds__(threads_of(C), C == 64 ? 2 : 1) void delta_grads_kernel(DeltaArgs a) {
  constexpr int kEsz = NX == 1 ? 2 : 4, kTb = C / 16, kKp = C / 32, kHalves = 2, kB = KB, kThreads = threads_of(C);
  constexpr int kPitchK = lds_pitch(32 * KB);
  // [S0, dS1][term][32 value columns] and U, U', dO [term][C]; then K, Q [term][C] and, of every wave, three operands.
  constexpr int kStates = 2 * kTerms * 32 * kPitchK, kTokens = (2 * kTerms + NX) * C * kPitchT;
  constexpr int kRows = 2 * NX * C * kPitchK, kWave = 3 * kTerms * kOperand, kMasked = kThreads / 64 * kWave;
  constexpr int kSize = kStates + kTokens > kRows + kMasked ? kStates + kTokens : kRows + kMasked;
  __shared__ __align__(16) uint16_t Sl[kSize];
  __shared__ __align__(16) float Gh[C], Gl[C], Be[C], Ev[C], Sw[C], Kr[C], dots[kThreads / 64];
  uint16_t* const Tl = Sl + kStates;
  uint16_t* const Ut = Tl;
  uint16_t* const Vt = Tl + kTerms * C * kPitchT;       // U'
  uint16_t* const Ot = Tl + 2 * kTerms * C * kPitchT;   // dO
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int tb = wave % kTb, half = wave / kTb, tok = 16 * tb + c16;
  const long unit = xcd_unit(blockIdx.x, gridDim.x);
  const int h = (int)(unit % a.H);
  const long slot = unit / a.H;
  const DeltaChunk ch = delta_slot<C>(a, slot);
  if (ch.p.blk < 0 || ch.n <= 0) return;
  const int n = ch.n, hk = h / (a.H / a.Hk);
  const long sh = slot * a.H + h, mat = (long)a.dk * a.dv;
  const float* gates = a.gates + sh * kGateRows * C;
  if (threadIdx.x < C) {
    Gh[threadIdx.x] = gates[3 * C + threadIdx.x];
    Gl[threadIdx.x] = gates[4 * C + threadIdx.x];
    Be[threadIdx.x] = gates[2 * C + threadIdx.x];
    Ev[threadIdx.x] = Sw[threadIdx.x] = Kr[threadIdx.x] = 0.f;
  }
  const float eg = gates[tok], wt = gates[C + tok], keep = gates[5 * C];
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  const float* S0 = a.states + sh * mat;
  const float* S1 = a.dstates + sh * mat;
  const rsrc_t ru = make_rsrc(a.u + sh * C * a.dv, (uint32_t)(C * a.dv * 4));
  const rsrc_t rb = make_rsrc(a.ub + sh * C * a.dv, (uint32_t)(C * a.dv * 4));
  const rsrc_t ro = chunk_rows(a.d_o, ch.row0, (long)a.H * a.dv, (long)h * a.dv, n, kEsz);
  const rsrc_t rv = chunk_rows(a.v, ch.row0, a.v_row, (long)h * a.dv, n, kEsz);
  constexpr int kPieces = (256 * KB + kThreads - 1) / kThreads;
  f32x4 s0[kPieces], s1[kPieces];   // this thread's pieces of four of the states' rows
  Raw8<3> xu, xb;
  Raw8<NX> xo, xv;
  auto load = [&](int kv) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = threadIdx.x + kThreads * i, dv = 32 * kv + at / (8 * KB), dk = 4 * (at % (8 * KB));
      const bool in = at < 256 * KB && dv < a.dv && dk < a.dk;
      s0[i] = in ? *reinterpret_cast<const f32x4*>(S0 + (long)dv * a.dk + dk) : zero;
      s1[i] = in ? *reinterpret_cast<const f32x4*>(S1 + (long)dv * a.dk + dk) : zero;
    }
    const int lo = 32 * kv + 4 * g, hi = lo + 16;
    auto pair = [&](bool row, int pitch, int esz, uint32_t& x, uint32_t& y) {
      x = row && lo < a.dv ? (uint32_t)(tok * pitch + lo * esz) : kOffNone;
      y = row && hi < a.dv ? (uint32_t)(tok * pitch + hi * esz) : kOffNone;
    };
    uint32_t x, y;
    pair(true, a.dv * 4, 4, x, y);
    xu = load_pair<3>(ru, x, y);
    xb = load_pair<3>(rb, x, y);
    pair(tok < n, a.H * a.dv * kEsz, kEsz, x, y);
    xo = load_pair<NX>(ro, x, y);
    pair(tok < n, (int)a.v_row * kEsz, kEsz, x, y);
    xv = load_pair<NX>(rv, x, y);
  };

  // Lane: token tok, key columns 16 (half kB + b) + 4 g + r.
  f32x4 dQ[kB], R[kB], W[kB];
#pragma unroll
  for (int b = 0; b < kB; ++b) dQ[b] = R[b] = W[b] = zero;
  // Products with the tokens 16 blk + 4 g + r: entry e <= tb has blk = e and tok as the row (i), the others
  // blk = e - 1 and tok as the column (j).
  // The first of the tokens' two waves makes Z1, the second Z2.
  f32x4 Z[kTb + 1];
#pragma unroll
  for (int e = 0; e <= kTb; ++e) Z[e] = zero;
  float uv = 0.f, dot = 0.f;

  const int steps = (a.dv + 31) / 32;
  load(0);
  for (int kv = 0; kv < steps; ++kv) {
    u32x4 ut[kTerms], vt[kTerms], ot[NX];
    {
      float x[8], y[8];
      floats8(xu, x);
      split8<kTerms>(x, ut);
      floats8(xb, x);
      split8<kTerms>(x, vt);
      floats8(xv, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) uv = fmaf(x[i], y[i], uv);
      terms8<NX>(xo, ot);
    }
    {
      const int at = tok * kPitchT + 8 * g;
#pragma unroll
      for (int t = 0; t < kTerms; ++t) *reinterpret_cast<u32x4*>((half ? Vt : Ut) + t * C * kPitchT + at) = half ? vt[t] : ut[t];
#pragma unroll
      for (int t = 0; t < NX; ++t)
        if (half == 0) *reinterpret_cast<u32x4*>(Ot + t * C * kPitchT + at) = ot[t];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = threadIdx.x + kThreads * i, row = at / (8 * KB), col = 4 * (at % (8 * KB));
      if (256 * KB % kThreads && at >= 256 * KB) continue;
      u32x2 p0[kTerms], p1[kTerms];
      split4<kTerms>(s0[i], p0);
      split4<kTerms>(s1[i], p1);
#pragma unroll
      for (int r = 0; r < 4; ++r) dot = fmaf(s0[i][r], s1[i][r], dot);
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        *reinterpret_cast<u32x2*>(Sl + (t * 32 + row) * kPitchK + col) = p0[t];
        *reinterpret_cast<u32x2*>(Sl + ((kTerms + t) * 32 + row) * kPitchK + col) = p1[t];
      }
    }
    if (kv + 1 < steps) load(kv + 1);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int col = 16 * (half * kB + b);
      u32x4 st[kTerms], dt[kTerms];
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        st[t] = frag_k_rows_accpair(Sl + t * 32 * kPitchK, kPitchK, 0, col, lane);
        dt[t] = frag_k_rows_accpair(Sl + (kTerms + t) * 32 * kPitchK, kPitchK, 0, col, lane);
      }
      dQ[b] = mma<kTerms, NX, kTerms>(st, ot, dQ[b]);
      R[b] = mma<kTerms, kTerms, kTerms>(st, vt, R[b]);
      W[b] = mma<kTerms, kTerms, kTerms>(dt, ut, W[b]);
    }
#pragma unroll
    for (int e = 0; e <= kTb; ++e) {
      const bool row = e <= tb;
      const int at = 16 * (row ? e : e - 1);
      u32x4 x[kTerms];
      if (half == 0) {
        if (row) {
#pragma unroll
          for (int t = 0; t < kTerms; ++t) x[t] = frag_k_cols(Ut + t * C * kPitchT, kPitchT, at, 0, lane);
          Z[e] = mma<kTerms, NX, kTerms>(x, ot, Z[e]);
        } else {
#pragma unroll
          for (int t = 0; t < NX; ++t) x[t] = frag_k_cols(Ot + t * C * kPitchT, kPitchT, at, 0, lane);
          Z[e] = mma<NX, kTerms, kTerms>(x, ut, Z[e]);
        }
      } else {
        const uint16_t* from = row ? Ut : Vt;
#pragma unroll
        for (int t = 0; t < kTerms; ++t) x[t] = frag_k_cols(from + t * C * kPitchT, kPitchT, at, 0, lane);
        if (row) Z[e] = mma<kTerms, kTerms, kTerms>(x, vt, Z[e]);
        else Z[e] = mma<kTerms, kTerms, kTerms>(x, ut, Z[e]);
      }
    }
    __syncthreads();
  }

  // Rows of K and Q where the states were.
  uint16_t* const Kl = Sl;
  uint16_t* const Ql = Sl + NX * C * kPitchK;
  {
    // The tokens' first wave stages K, the second Q.
    const int xrow = (int)(half ? a.q_row : a.k_row) * kEsz;
    const rsrc_t rx = chunk_rows(half ? a.q : a.k, ch.row0, half ? a.q_row : a.k_row, (long)hk * a.dk, n, kEsz);
    uint16_t* const to = half ? Ql : Kl;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int col = 32 * b + 8 * g;
      u32x4 x[NX];
      terms8<NX>(load8<NX>(rx, col < a.dk ? (uint32_t)(tok * xrow + col * kEsz) : kOffNone), x);
#pragma unroll
      for (int t = 0; t < NX; ++t) *reinterpret_cast<u32x4*>(to + (t * C + tok) * kPitchK + col) = x[t];
    }
  }
  // Weights of the pairs; masked ones are 0 whatever their product was. As operands, of every wave: row blocks kp up
  // to tb / 2 at kp, columns from tb / 2 on at kp + 1.
  uint16_t* const Ml = Sl + kRows;
  {
    const float hi = Gh[tok], lo = Gl[tok];
#pragma unroll
    for (int e = 0; e <= kTb; ++e) {
      const bool row = e <= tb;
      const int o = 16 * (row ? e : e - 1) + 4 * g;
      const f32x4 ho = *reinterpret_cast<const f32x4*>(Gh + o), lo4 = *reinterpret_cast<const f32x4*>(Gl + o);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = row ? tok : o + r, j = row ? o + r : tok;
        const float dh = hi - ho[r], dl = lo - lo4[r];
        const float d = i >= j ? exp_of(row ? dh + dl : -dh - dl) : 0.f;
        const float w = half ? -d * (row ? 1.f : Be[o + r]) : d * (row ? 1.f : a.scale);
        Z[e][r] = i > j || (i == j && half == 0) ? Z[e][r] * w : 0.f;
      }
    }
    uint16_t* const to = Ml + wave * kWave + lane * 8;
#pragma unroll
    for (int m = 0; m < kKp; ++m) {
      float x[8], y[8];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int b = 2 * m + t;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[4 * t + r] = b <= tb ? Z[b][r] : 0.f;
          y[4 * t + r] = b >= tb ? Z[b + 1][r] : 0.f;
        }
      }
      u32x4 part[kTerms];
      if (m <= tb / 2) {
        split8<kTerms>(x, part);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) *reinterpret_cast<u32x4*>(to + (m * kTerms + t) * kOperand) = part[t];
      }
      if (m >= tb / 2) {
        split8<kTerms>(y, part);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) *reinterpret_cast<u32x4*>(to + ((m + 1) * kTerms + t) * kOperand) = part[t];
      }
    }
  }
  __syncthreads();
  const uint16_t *const z1 = Ml + tb * kWave + lane * 8, *const z2 = Ml + (tb + kTb) * kWave + lane * 8;
  const float be = Be[tok];
  const bool shared = a.part_q != nullptr;
  const long heads = shared ? a.H : a.Hk, hout = shared ? h : hk;
  const rsrc_t wq = chunk_rows(shared ? (void*)a.part_q : a.dq, ch.row0, heads * a.dk, hout * a.dk, n, shared ? 4 : kEsz);
  const rsrc_t wk = chunk_rows(shared ? (void*)a.part_k : a.dk_out, ch.row0, heads * a.dk, hout * a.dk, n, shared ? 4 : kEsz);
  float e_q = 0.f, e_r = 0.f, e_w = 0.f, e_s = 0.f;
  auto row_of = [&](const uint16_t* L, int b) {   // this lane's four of the token's row
    f32x4 x = zero;
#pragma unroll
    for (int t = NX - 1; t >= 0; --t) x += four(*reinterpret_cast<const u32x2*>(L + (t * C + tok) * kPitchK + 16 * (half * kB + b) + 4 * g));
    return x;
  };
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const f32x4 kv = row_of(Kl, b);
    dQ[b] *= eg;
    R[b] *= -eg;
    W[b] *= wt;
#pragma unroll
    for (int r = 0; r < 4; ++r) e_s = fmaf(kv[r], W[b][r], e_s);
  }
  auto masked = [&](const uint16_t* z, int at, u32x4* out) {
#pragma unroll
    for (int t = 0; t < kTerms; ++t) out[t] = *reinterpret_cast<const u32x4*>(z + (at * kTerms + t) * kOperand);
  };
#pragma unroll
  for (int m = 0; m < kKp; ++m) {
    u32x4 x[kTerms], y[kTerms];
    if (m <= tb / 2) {
      masked(z1, m, x);
      masked(z2, m, y);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        u32x4 kt[NX];
#pragma unroll
        for (int t = 0; t < NX; ++t) kt[t] = frag_k_rows_accpair(Kl + t * C * kPitchK, kPitchK, 32 * m, 16 * (half * kB + b), lane);
        dQ[b] = mma<NX, kTerms, kTerms>(kt, x, dQ[b]);
        R[b] = mma<NX, kTerms, kTerms>(kt, y, R[b]);
      }
    }
    if (m >= tb / 2) {
      masked(z1, m + 1, x);
      masked(z2, m + 1, y);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        u32x4 kt[NX], qt[NX];
#pragma unroll
        for (int t = 0; t < NX; ++t) {
          kt[t] = frag_k_rows_accpair(Kl + t * C * kPitchK, kPitchK, 32 * m, 16 * (half * kB + b), lane);
          qt[t] = frag_k_rows_accpair(Ql + t * C * kPitchK, kPitchK, 32 * m, 16 * (half * kB + b), lane);
        }
        W[b] = mma<NX, kTerms, kTerms>(qt, x, W[b]);
        W[b] = mma<NX, kTerms, kTerms>(kt, y, W[b]);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const int dk = 16 * (half * kB + b) + 4 * g;
    const f32x4 kv = row_of(Kl, b), qv = row_of(Ql, b);
    dQ[b] *= a.scale;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      e_q = fmaf(qv[r], dQ[b][r], e_q);
      e_r = fmaf(kv[r], R[b][r], e_r);
      e_w = fmaf(kv[r], W[b][r], e_w);
    }
    const f32x4 dk4 = R[b] * be + W[b];
    const bool in = tok < n && dk < a.dk;
    if (shared) {
      const uint32_t off = in ? (uint32_t)((tok * (int)heads * a.dk + dk) * 4) : kOffNone;
      store4<3>(dQ[b], wq, off);
      store4<3>(dk4, wk, off);
    } else {
      const uint32_t off = in ? (uint32_t)((tok * (int)heads * a.dk + dk) * kEsz) : kOffNone;
      store4<NX>(dQ[b], wq, off);
      store4<NX>(dk4, wk, off);
    }
  }
  auto over_g = [](float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
  };
  e_q = over_g(e_q);
  e_r = over_g(e_r);
  e_w = over_g(e_w);
  e_s = over_g(e_s);
  uv = over_g(uv);
  dot = lanes_sum<64>(dot, 64);
  if (lane == 0) dots[wave] = dot;
#pragma unroll
  for (int s = 0; s < kHalves; ++s) {   // one half of the key columns after the other
    if (half == s && g == 0) {
      Ev[tok] += e_q + be * e_r - e_w;
      Sw[tok] += e_s;
      Kr[tok] += e_r;
    }
    __syncthreads();
  }
  if (half == 0 && g == 0 && tok < n) a.dbeta[(ch.row0 + tok) * a.H + h] = uv + Kr[tok];
  if (wave == 0 && a.dg) {
    const double ev = lane < C ? (double)Ev[lane] : 0.0;
    double up = ev, all = ev, sw = lane < C ? (double)Sw[lane] : 0.0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double y = __shfl_up(up, d);
      if (lane >= d) up += y;
      all += __shfl_xor(all, d);
      sw += __shfl_xor(sw, d);
    }
    double cross = 0.0;
    for (int i = 0; i < kThreads / 64; ++i) cross += (double)dots[i];
    cross = (double)keep * cross + sw;
    if (lane < n) a.dg[(ch.row0 + lane) * a.H + h] = (float)(cross + (all - up + ev));
  }
}

template <int C, int NX>
void grads(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)delta_bwd_blocks(a));
  if (a.dk <= 32) hipLaunchKernelGGL((delta_grads_kernel<C, 1, NX>), grid, dim3(threads_of(C)), 0, stream, a);
  else if (a.dk <= 64) hipLaunchKernelGGL((delta_grads_kernel<C, 2, NX>), grid, dim3(threads_of(C)), 0, stream, a);
  else if (a.dk <= 128) hipLaunchKernelGGL((delta_grads_kernel<C, 4, NX>), grid, dim3(threads_of(C)), 0, stream, a);
  else hipLaunchKernelGGL((delta_grads_kernel<C, 8, NX>), grid, dim3(threads_of(C)), 0, stream, a);
}

}  // namespace

long delta_bwd_blocks(const DeltaArgs& a) { return a.slots * a.H; }
int delta_bwd_threads() { return threads_of(64); }

hipError_t launch_delta_grads(const DeltaArgs& a, hipStream_t stream) {
  if (a.bf16) grads<64, 1>(a, stream);
  else grads<32, 3>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
