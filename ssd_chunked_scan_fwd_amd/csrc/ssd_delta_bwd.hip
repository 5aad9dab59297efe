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
// A workgroup takes one chunk of one head, two waves 16 tokens: one makes what belongs to their reads (dq and r, from
// S0, U', dO and the Z of the tokens as rows i), the other what belongs to their writes (w, from dS1, U and the Z of
// the tokens as columns j). First, over the value columns 32 at a time, the products with the states (contraction over
// the columns, the states' terms in LDS) and the Z; then the products of the masked Z, which stay in registers, with Q
// and K, whose rows take the states' place in LDS.
// 8192 tokens, 32 heads on 16 of 128 x 128: 430 to 450 us. 1.2 GB are read, the states of all chunks and U twice half
// of it, and 0.2 GB written: 3.2 TB/s, with one workgroup a CU, whose waves keep 256 registers: a step of 32 columns
// takes 4 us, of which 1 is a wait for memory, the vector units are busy 37 % of the time, matrix units 21 %. (Rows of
// Q and K loaded with the first columns: no faster, fp32 412 -> 447 us. With both kinds of waves for half of the key
// columns each, U and U' split twice: 30 us more.)
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int threads_of(int C) { return 8 * C; }   // two waves for 16 tokens
constexpr int kPitchT = lds_pitch(32);   // rows of 32 value columns, in the order of an accumulator pair

// ALL: all value heads that share their keys, one after the other; else one.
template <int C, int KB, int NX, bool ALL>
__global__ __launch_bounds__(threads_of(C), C == 64 ? 2 : 1) void delta_grads_kernel(DeltaArgs a) {
  constexpr int kEsz = NX == 1 ? 2 : 4, kTb = C / 16, kKp = C / 32, kB = 2 * KB, kThreads = threads_of(C);
  constexpr int kPitchK = lds_pitch(32 * KB);
  // [S0, dS1][term][32 value columns] and U, U', dO [term][C]; then K, Q [term][C] and beta r in fp32.
  constexpr int kStates = 2 * kTerms * 32 * kPitchK, kTokens = (2 * kTerms + NX) * C * kPitchT;
  constexpr int kRows = 2 * NX * C * kPitchK, kReads = kTb * kB * 64 * 8;
  constexpr int kSize = kStates + kTokens > kRows + kReads ? kStates + kTokens : kRows + kReads;
  __shared__ __align__(16) uint16_t Sl[kSize];
  __shared__ __align__(16) float Gh[C], Gl[C], Be[C], Ev[C], Sw[C], dots[kThreads / 64];
  uint16_t* const Ut = Sl + kStates;
  uint16_t* const Vt = Ut + kTerms * C * kPitchT;       // U'
  uint16_t* const Ot = Ut + 2 * kTerms * C * kPitchT;   // dO
  const int wave = uniform(threadIdx.x >> 6), tb = wave % kTb;
  const bool reads = wave < kTb;   // else the writes
  const long unit = xcd_unit(blockIdx.x, gridDim.x);
  const int rep = a.H / a.Hk, here = ALL ? rep : 1, units = a.H / here;
  const long slot = unit / units;
  const DeltaChunk ch = delta_slot<C>(a, slot);
  if (ch.p.blk < 0 || ch.n <= 0) return;
  const int n = ch.n, h0 = (int)(unit % units) * here;
  for (int h = h0; h < h0 + here; ++h) {
    // A thread's number that the compiler does not know from one head to the next: the places that follow from it are
    // made anew, not kept in registers.
    int tid = threadIdx.x;
    if (ALL) asm volatile("" : "+v"(tid));
    const int lane = tid & 63, c16 = lane & 15, g = lane >> 4, tok = 16 * tb + c16, hk = h / rep;
    const long sh = slot * a.H + h, mat = (long)a.dk * a.dv;
    const float* gates = a.gates + sh * kGateRows * C;
    if (tid < C) {
      Gh[tid] = gates[3 * C + tid];
      Gl[tid] = gates[4 * C + tid];
      Be[tid] = gates[2 * C + tid];
    }
    const float eg = gates[tok], wt = gates[C + tok], keep = gates[5 * C];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    const rsrc_t rs0 = make_rsrc(a.states + sh * mat, (uint32_t)(mat * 4)), rs1 = make_rsrc(a.dstates + sh * mat, (uint32_t)(mat * 4));
    const rsrc_t ru = make_rsrc((reads ? a.ub : a.u) + sh * C * a.dv, (uint32_t)(C * a.dv * 4));
    const rsrc_t ro = chunk_rows(a.d_o, ch.row0, (long)a.H * a.dv, (long)h * a.dv, n, kEsz);
    const rsrc_t rv = chunk_rows(a.v, ch.row0, a.v_row, (long)h * a.dv, n, kEsz);
    constexpr int kPieces = (256 * KB + kThreads - 1) / kThreads;
    f32x4 s0[kPieces], s1[kPieces];   // this thread's pieces of four of the states' rows
    Raw8<3> xu;                       // of U' or U
    Raw8<NX> xo, xv;
    auto load = [&](int kv) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = tid + kThreads * i, dv = 32 * kv + at / (8 * KB), dk = 4 * (at % (8 * KB));
        const uint32_t off = at < 256 * KB && dv < a.dv && dk < a.dk ? (uint32_t)((dv * a.dk + dk) * 4) : kOffNone;
        s0[i] = __builtin_bit_cast(f32x4, buf_load16(rs0, off));
        s1[i] = __builtin_bit_cast(f32x4, buf_load16(rs1, off));
      }
      const int lo = 32 * kv + 4 * g, hi = lo + 16;
      auto pair = [&](bool row, int pitch, int esz, uint32_t& x, uint32_t& y) {
        x = row && lo < a.dv ? (uint32_t)(tok * pitch + lo * esz) : kOffNone;
        y = row && hi < a.dv ? (uint32_t)(tok * pitch + hi * esz) : kOffNone;
      };
      uint32_t x, y;
      pair(true, a.dv * 4, 4, x, y);
      xu = load_pair<3>(ru, x, y);
      pair(reads && tok < n, a.H * a.dv * kEsz, kEsz, x, y);
      xo = load_pair<NX>(ro, x, y);
      pair(reads && tok < n, (int)a.v_row * kEsz, kEsz, x, y);
      xv = load_pair<NX>(rv, x, y);
    };

    // Lane: token tok, key columns 16 b + 4 g + r. P: r or w. Z of the tokens 16 blk + 4 g + r, before tok and in its
    // block (reads) or behind it and in its block (writes); zeros of the other blocks.
    f32x4 dQ[kB], P[kB], Z1[kTb], Z2[kTb];
#pragma unroll
    for (int b = 0; b < kB; ++b) dQ[b] = P[b] = zero;
#pragma unroll
    for (int e = 0; e < kTb; ++e) Z1[e] = Z2[e] = zero;
    float uv = 0.f, dot = 0.f;

    // Gradients of shared rows: fp32, of every head (added up by another launch), or of the heads so far, the last
    // head's sum as the result.
    const bool each = here < rep, part = each || h + 1 < h0 + here;
    const long heads = each ? a.H : a.Hk, hout = each ? h : hk;
    auto out = [&](float* sums, void* whole) {
      return chunk_rows(part ? (void*)sums : whole, ch.row0, heads * a.dk, hout * a.dk, n, part ? 4 : kEsz);
    };
    const rsrc_t wx = out(reads ? a.part_q : a.part_k, reads ? a.dq : a.dk_out);
    const rsrc_t rsums = chunk_rows(reads ? a.part_q : a.part_k, ch.row0, heads * a.dk, hout * a.dk, n, 4);
    auto place = [&](int b) { return tok < n && 16 * b + 4 * g < a.dk ? (uint32_t)(tok * (int)heads * a.dk + 16 * b + 4 * g) : kOffNone; };
    auto store = [&](f32x4 x, int b) {
      const uint32_t at = place(b);
      if (part) store4<3>(x, wx, at == kOffNone ? at : at * 4);
      else store4<NX>(x, wx, at == kOffNone ? at : at * kEsz);
    };

    const int steps = (a.dv + 31) / 32;
    load(0);
    loads_done();
    for (int kv = 0; kv < steps; ++kv) {
      u32x4 own[kTerms], ot[NX];
      {
        float x[8], y[8];
        floats8(xu, x);
        split8<kTerms>(x, own);
        floats8(xv, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) uv = fmaf(x[i], y[i], uv);
        terms8<NX>(xo, ot);
      }
      {
        const int at = tok * kPitchT + 8 * g;
#pragma unroll
        for (int t = 0; t < kTerms; ++t) *reinterpret_cast<u32x4*>((reads ? Vt : Ut) + t * C * kPitchT + at) = own[t];
#pragma unroll
        for (int t = 0; t < NX; ++t)
          if (reads) *reinterpret_cast<u32x4*>(Ot + t * C * kPitchT + at) = ot[t];
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = tid + kThreads * i, row = at / (8 * KB), col = 4 * (at % (8 * KB));
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
      load(min(kv + 1, steps - 1));
      __syncthreads();
      const uint16_t* const states = Sl + (reads ? 0 : kTerms * 32 * kPitchK);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        u32x4 st[kTerms];
#pragma unroll
        for (int t = 0; t < kTerms; ++t) st[t] = frag_k_rows_accpair(states + t * 32 * kPitchK, kPitchK, 0, 16 * b, lane);
        P[b] = mma<kTerms, kTerms, kTerms>(st, own, P[b]);
        if (reads) dQ[b] = mma<kTerms, NX, kTerms>(st, ot, dQ[b]);
      }
#pragma unroll
      for (int e = 0; e < kTb; ++e) {
        if (reads ? e > tb : e < tb) continue;
        u32x4 x[kTerms], y[NX];
#pragma unroll
        for (int t = 0; t < kTerms; ++t) x[t] = frag_k_cols((reads ? Ut : Vt) + t * C * kPitchT, kPitchT, 16 * e, 0, lane);
        Z2[e] = mma<kTerms, kTerms, kTerms>(x, own, Z2[e]);
        if (reads) {
          Z1[e] = mma<kTerms, NX, kTerms>(x, ot, Z1[e]);
        } else {
#pragma unroll
          for (int t = 0; t < NX; ++t) y[t] = frag_k_cols(Ot + t * C * kPitchT, kPitchT, 16 * e, 0, lane);
          Z1[e] = mma<NX, kTerms, kTerms>(y, own, Z1[e]);
        }
      }
      __syncthreads();
    }

    // Rows of K and Q where the states were: the reads' waves stage K, the others Q.
    uint16_t* const Kl = Sl;
    uint16_t* const Ql = Sl + NX * C * kPitchK;
    f32x4* const Rl = reinterpret_cast<f32x4*>(Sl + kRows) + tb * kB * 64 + lane;   // beta r, as the lanes hold it
    {
      const int xrow = (int)(reads ? a.k_row : a.q_row) * kEsz;
      const rsrc_t rx = chunk_rows(reads ? a.k : a.q, ch.row0, reads ? a.k_row : a.q_row, (long)hk * a.dk, n, kEsz);
      uint16_t* const to = reads ? Kl : Ql;
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const int col = 32 * b + 8 * g;
        u32x4 x[NX];
        terms8<NX>(load8<NX>(rx, col < a.dk ? (uint32_t)(tok * xrow + col * kEsz) : kOffNone), x);
#pragma unroll
        for (int t = 0; t < NX; ++t) *reinterpret_cast<u32x4*>(to + (t * C + tok) * kPitchK + col) = x[t];
      }
    }
    // Weights of the pairs; masked ones are 0 whatever their product was.
    u32x4 z1[kKp][kTerms], z2[kKp][kTerms];
    {
      const float hi = Gh[tok], lo = Gl[tok];
#pragma unroll
      for (int e = 0; e < kTb; ++e) {
        const int o = 16 * e + 4 * g;
        const f32x4 ho = *reinterpret_cast<const f32x4*>(Gh + o), lo4 = *reinterpret_cast<const f32x4*>(Gl + o),
                    beo = *reinterpret_cast<const f32x4*>(Be + o);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = reads ? tok : o + r, j = reads ? o + r : tok;
          const float dh = hi - ho[r], dl = lo - lo4[r];
          const float d = exp_of(reads ? dh + dl : -dh - dl);
          Z1[e][r] = i >= j ? Z1[e][r] * (d * (reads ? 1.f : a.scale)) : 0.f;
          Z2[e][r] = i > j ? Z2[e][r] * (d * (reads ? -1.f : -beo[r])) : 0.f;
        }
      }
#pragma unroll
      for (int m = 0; m < kKp; ++m) {
        float x[8], y[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          x[t] = Z1[2 * m + t / 4][t % 4];
          y[t] = Z2[2 * m + t / 4][t % 4];
        }
        split8<kTerms>(x, z1[m]);
        split8<kTerms>(y, z2[m]);
      }
    }
    __syncthreads();
    f32x4 sum[kB];   // of the heads so far, this thread's own stores
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const uint32_t at = ALL && h > h0 ? place(b) : kOffNone;
      sum[b] = ALL ? __builtin_bit_cast(f32x4, buf_load16(rsums, at == kOffNone ? at : at * 4)) : zero;
    }
    const float be = Be[tok];
    auto row_of = [&](const uint16_t* L, int b) {   // this lane's four of the token's row
      f32x4 x = zero;
#pragma unroll
      for (int t = NX - 1; t >= 0; --t) x += four(*reinterpret_cast<const u32x2*>(L + (t * C + tok) * kPitchK + 16 * b + 4 * g));
      return x;
    };
    auto operand = [&](const uint16_t* L, int m, int b, u32x4* x) {
#pragma unroll
      for (int t = 0; t < NX; ++t) x[t] = frag_k_rows_accpair(L + t * C * kPitchK, kPitchK, 32 * m, 16 * b, lane);
    };
    auto over_g = [](float x) {
      x += __shfl_xor(x, 16);
      return x + __shfl_xor(x, 32);
    };
    float e_r = 0.f;
    if (reads) {
      float e_q = 0.f;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        dQ[b] *= eg;
        P[b] *= -eg;
#pragma unroll
        for (int m = 0; m < kKp; ++m) {
          if (m > tb / 2) continue;
          u32x4 kt[NX];
          operand(Kl, m, b, kt);
          dQ[b] = mma<NX, kTerms, kTerms>(kt, z1[m], dQ[b]);
          P[b] = mma<NX, kTerms, kTerms>(kt, z2[m], P[b]);
        }
        dQ[b] *= a.scale;
        const f32x4 kv = row_of(Kl, b), qv = row_of(Ql, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e_q = fmaf(qv[r], dQ[b][r], e_q);
          e_r = fmaf(kv[r], P[b][r], e_r);
        }
        Rl[b * 64] = P[b] * be;
        store(sum[b] + dQ[b], b);
      }
      e_r = over_g(e_r);
      e_q = over_g(e_q);
      if (g == 0) Ev[tok] = e_q + be * e_r;
      uv = over_g(uv);
      if (g == 0 && tok < n) a.dbeta[(ch.row0 + tok) * a.H + h] = uv + e_r;
    } else {
      float e_s = 0.f;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        P[b] *= wt;
        const f32x4 kv = row_of(Kl, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) e_s = fmaf(kv[r], P[b][r], e_s);
#pragma unroll
        for (int m = 0; m < kKp; ++m) {
          if (m < tb / 2) continue;
          u32x4 kt[NX], qt[NX];
          operand(Kl, m, b, kt);
          operand(Ql, m, b, qt);
          P[b] = mma<NX, kTerms, kTerms>(qt, z1[m], P[b]);
          P[b] = mma<NX, kTerms, kTerms>(kt, z2[m], P[b]);
        }
      }
      e_s = over_g(e_s);
      if (g == 0) Sw[tok] = e_s;
    }
    dot = lanes_sum<64>(dot, 64);
    if (lane == 0) dots[wave] = dot;
    __syncthreads();
    if (!reads) {
      float e_w = 0.f;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const f32x4 kv = row_of(Kl, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) e_w = fmaf(kv[r], P[b][r], e_w);
        store(sum[b] + (Rl[b * 64] + P[b]), b);
      }
      e_w = over_g(e_w);
      if (g == 0) Ev[tok] -= e_w;
    }
    __syncthreads();
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
    __syncthreads();
  }
}

template <int C, int KB, int NX>
void grads(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)delta_bwd_blocks(a)), block(threads_of(C));
  if constexpr (KB <= 4) {
    if (a.grad_heads > 1) {
      hipLaunchKernelGGL((delta_grads_kernel<C, KB, NX, true>), grid, block, 0, stream, a);
      return;
    }
  }
  hipLaunchKernelGGL((delta_grads_kernel<C, KB, NX, false>), grid, block, 0, stream, a);
}
template <int C, int NX>
void grads(const DeltaArgs& a, hipStream_t stream) {
  if (a.dk <= 32) grads<C, 1, NX>(a, stream);
  else if (a.dk <= 64) grads<C, 2, NX>(a, stream);
  else if (a.dk <= 128) grads<C, 4, NX>(a, stream);
  else grads<C, 8, NX>(a, stream);
}

}  // namespace

// Value heads a workgroup, one after the other: all that share their keys, where that leaves a workgroup for every CU, in
// fp32 two (no partial sums of every head to write and to add up then); else one, and so with keys of 256, which leave no registers for
// the sums. With the walks, us with one and with all, heads of 128 x 128 two on a key (the workgroups of all): 8192 tokens of
// 32 (2048) 1114 and 1069, 4096 of 24 (768) 472 and 452, 1024 of 32 (256) 148 and 141, 768 of 32 (192) 122 and 118, 512 of
// 32 (128) 86 and 101; four on a key, 64 x 64: 2 x 2048 of 16 (256) 175 and 169, half of them (128) 130 and 142. fp32, 64 x
// 64: 2048 of 32 (1024) 249 and 238, 128 x 64 2048 of 16 (512) 275 and 272; 64 x 64, four on a key, 1024 of 32 (256) 145
// and 151, half of them (128) 96 and 116.
int delta_grad_heads(long slots, int H, int Hk, int dk, bool bf16) { return slots * Hk >= (bf16 ? 256 : 512) && dk <= 128 ? H / Hk : 1; }
long delta_bwd_blocks(const DeltaArgs& a) { return a.slots * (a.H / a.grad_heads); }
int delta_bwd_threads() { return threads_of(64); }

hipError_t launch_delta_grads(const DeltaArgs& a, hipStream_t stream) {
  if (a.bf16) grads<64, 1>(a, stream);
  else grads<32, 3>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
