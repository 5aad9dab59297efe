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
// A workgroup takes one chunk of one head. First, over the value columns 32 at a
// time, the products with the states (contraction over the columns, the states'
// terms in LDS) and Z1, Z2 of the wave's own tokens, both as rows and as columns;
// then the products of the masked Z with Q and K, whose rows take the states'
// place in LDS.
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kPitchT = lds_pitch(32);   // rows of 32 value columns, in the order of an accumulator pair

template <int C, int KB, int NX>
__global__ __launch_bounds__(kThreads, 1) void delta_grads_kernel(DeltaArgs a) {
  constexpr int kEsz = NX == 1 ? 2 : 4, kTb = C / 16, kKp = C / 32, kHalves = 4 / kTb, kB = 2 * KB / kHalves;
  constexpr int kPitchK = lds_pitch(32 * KB);
  constexpr int kStateRows = 2 * kTerms * 32;
  static_assert(kStateRows >= 2 * NX * C, "Q and K take the states' place");
  __shared__ __align__(16) uint16_t Sl[kStateRows * kPitchK];   // [S0, dS1][term][32 value columns]; K, Q [term][C]
  __shared__ __align__(16) uint16_t Tl[(2 * kTerms + NX) * C * kPitchT];   // U, U', dO [term][C]
  __shared__ float Gh[C], Gl[C], Be[C], Ev[C], Sw[C], Kr[C], dots[4];
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
  f32x4 s0[KB], s1[KB];   // this thread's pieces of four of the states' rows
  Raw8<3> xu, xb;
  Raw8<NX> xo, xv;
  auto load = [&](int kv) {
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int at = threadIdx.x + kThreads * i, dv = 32 * kv + at / (8 * KB), dk = 4 * (at % (8 * KB));
      const bool in = dv < a.dv && dk < a.dk;
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
  f32x4 Z1[kTb + 1], Z2[kTb + 1];
#pragma unroll
  for (int e = 0; e <= kTb; ++e) Z1[e] = Z2[e] = zero;
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
    if (half == 0) {
      const int at = tok * kPitchT + 8 * g;
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        *reinterpret_cast<u32x4*>(Ut + t * C * kPitchT + at) = ut[t];
        *reinterpret_cast<u32x4*>(Vt + t * C * kPitchT + at) = vt[t];
      }
#pragma unroll
      for (int t = 0; t < NX; ++t) *reinterpret_cast<u32x4*>(Ot + t * C * kPitchT + at) = ot[t];
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int at = threadIdx.x + kThreads * i, row = at / (8 * KB), col = 4 * (at % (8 * KB));
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
      u32x4 x[kTerms], y[kTerms];
      if (e <= tb) {
#pragma unroll
        for (int t = 0; t < kTerms; ++t) x[t] = frag_k_cols(Ut + t * C * kPitchT, kPitchT, 16 * e, 0, lane);
        Z1[e] = mma<kTerms, NX, kTerms>(x, ot, Z1[e]);
        Z2[e] = mma<kTerms, kTerms, kTerms>(x, vt, Z2[e]);
      } else {
#pragma unroll
        for (int t = 0; t < NX; ++t) x[t] = frag_k_cols(Ot + t * C * kPitchT, kPitchT, 16 * (e - 1), 0, lane);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) y[t] = frag_k_cols(Vt + t * C * kPitchT, kPitchT, 16 * (e - 1), 0, lane);
        Z1[e] = mma<NX, kTerms, kTerms>(x, ut, Z1[e]);
        Z2[e] = mma<kTerms, kTerms, kTerms>(y, ut, Z2[e]);
      }
    }
    __syncthreads();
  }

  // Rows of K and Q where the states were.
  uint16_t* const Kl = Sl;
  uint16_t* const Ql = Sl + NX * C * kPitchK;
  {
    const rsrc_t rk = chunk_rows(a.k, ch.row0, a.k_row, (long)hk * a.dk, n, kEsz);
    const rsrc_t rq = chunk_rows(a.q, ch.row0, a.q_row, (long)hk * a.dk, n, kEsz);
    const int krow = (int)a.k_row * kEsz, qrow = (int)a.q_row * kEsz;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if (kHalves > 1 && KB > 1 && b % kHalves != half) continue;
      const int col = 32 * b + 8 * g;
      const bool in = tok < n && col < a.dk;
      u32x4 kt[NX], qt[NX];
      terms8<NX>(load8<NX>(rk, in ? (uint32_t)(tok * krow + col * kEsz) : kOffNone), kt);
      terms8<NX>(load8<NX>(rq, in ? (uint32_t)(tok * qrow + col * kEsz) : kOffNone), qt);
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        *reinterpret_cast<u32x4*>(Kl + (t * C + tok) * kPitchK + col) = kt[t];
        *reinterpret_cast<u32x4*>(Ql + (t * C + tok) * kPitchK + col) = qt[t];
      }
    }
  }
  // Weights of the pairs; masked ones are 0 whatever their product was.
  {
    const float hi = Gh[tok], lo = Gl[tok];
#pragma unroll
    for (int e = 0; e <= kTb; ++e) {
      const bool row = e <= tb;
      const int o = 16 * (row ? e : e - 1) + 4 * g;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = row ? tok : o + r, j = row ? o + r : tok;
        const float dh = hi - Gh[o + r], dl = lo - Gl[o + r];
        const float d = i >= j ? expf(row ? dh + dl : -dh - dl) : 0.f;
        Z1[e][r] = i >= j ? Z1[e][r] * d * (row ? 1.f : a.scale) : 0.f;
        Z2[e][r] = i > j ? -Z2[e][r] * d * (row ? 1.f : Be[o + r]) : 0.f;
      }
    }
  }
  __syncthreads();
  u32x4 r1[kKp][kTerms], r2[kKp][kTerms], c1[kKp][kTerms], c2[kKp][kTerms];
#pragma unroll
  for (int m = 0; m < kKp; ++m) {
    float x1[8], x2[8], y1[8], y2[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int b = 2 * m + t;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x1[4 * t + r] = b <= tb ? Z1[b][r] : 0.f;
        x2[4 * t + r] = b <= tb ? Z2[b][r] : 0.f;
        y1[4 * t + r] = b >= tb ? Z1[b + 1][r] : 0.f;
        y2[4 * t + r] = b >= tb ? Z2[b + 1][r] : 0.f;
      }
    }
    split8<kTerms>(x1, r1[m]);
    split8<kTerms>(x2, r2[m]);
    split8<kTerms>(y1, c1[m]);
    split8<kTerms>(y2, c2[m]);
  }
  const float be = Be[tok];
  const bool shared = a.part_q != nullptr;
  const long heads = shared ? a.H : a.Hk, hout = shared ? h : hk;
  const rsrc_t wq = chunk_rows(shared ? (void*)a.part_q : a.dq, ch.row0, heads * a.dk, hout * a.dk, n, shared ? 4 : kEsz);
  const rsrc_t wk = chunk_rows(shared ? (void*)a.part_k : a.dk_out, ch.row0, heads * a.dk, hout * a.dk, n, shared ? 4 : kEsz);
  float e_q = 0.f, e_r = 0.f, e_w = 0.f, e_s = 0.f;
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const int col = 16 * (half * kB + b), dk = col + 4 * g;
    f32x4 kv = zero, qv = zero;
#pragma unroll
    for (int t = NX - 1; t >= 0; --t) {
      kv += four(*reinterpret_cast<const u32x2*>(Kl + (t * C + tok) * kPitchK + dk));
      qv += four(*reinterpret_cast<const u32x2*>(Ql + (t * C + tok) * kPitchK + dk));
    }
    dQ[b] *= eg;
    R[b] *= -eg;
    W[b] *= wt;
#pragma unroll
    for (int r = 0; r < 4; ++r) e_s = fmaf(kv[r], W[b][r], e_s);
#pragma unroll
    for (int m = 0; m < kKp; ++m) {
      u32x4 kt[NX], qt[NX];
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        kt[t] = frag_k_rows_accpair(Kl + t * C * kPitchK, kPitchK, 32 * m, col, lane);
        qt[t] = frag_k_rows_accpair(Ql + t * C * kPitchK, kPitchK, 32 * m, col, lane);
      }
      dQ[b] = mma<NX, kTerms, kTerms>(kt, r1[m], dQ[b]);
      R[b] = mma<NX, kTerms, kTerms>(kt, r2[m], R[b]);
      W[b] = mma<NX, kTerms, kTerms>(qt, c1[m], W[b]);
      W[b] = mma<NX, kTerms, kTerms>(kt, c2[m], W[b]);
    }
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
    const double cross = (double)keep * ((double)dots[0] + (double)dots[1] + (double)dots[2] + (double)dots[3]) + sw;
    if (lane < n) a.dg[(ch.row0 + lane) * a.H + h] = (float)(cross + (all - up + ev));
  }
}

template <int C, int NX>
void grads(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)delta_bwd_blocks(a));
  if (a.dk <= 32) hipLaunchKernelGGL((delta_grads_kernel<C, 1, NX>), grid, dim3(kThreads), 0, stream, a);
  else if (a.dk <= 64) hipLaunchKernelGGL((delta_grads_kernel<C, 2, NX>), grid, dim3(kThreads), 0, stream, a);
  else if (a.dk <= 128) hipLaunchKernelGGL((delta_grads_kernel<C, 4, NX>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((delta_grads_kernel<C, 8, NX>), grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

long delta_bwd_blocks(const DeltaArgs& a) { return a.slots * a.H; }
int delta_bwd_threads() { return kThreads; }

hipError_t launch_delta_grads(const DeltaArgs& a, hipStream_t stream) {
  if (a.bf16) grads<64, 1>(a, stream);
  else grads<32, 3>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
