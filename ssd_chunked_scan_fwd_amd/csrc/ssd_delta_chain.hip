// ssd_delta_chain.hip -- the walk of the delta rule over the chunks of each
// sequence, forwards and, for the gradients, backwards (formulas: ssd_delta.h).
//
// Columns of V, rows of the state, do not mix: a workgroup of four waves takes
// NV blocks of 16 of them of one head and carries their state [16 NV][dk] in the
// accumulators of its own products. What a chunk waits for is a chain of three
// phases, each ending in a barrier:
//     state times keys (a wave 16 tokens: X, or Y)  ->  times T  ->  state update
//     (a wave a quarter of dk).
// The longest chain of a call is its longest sequence's chunks times these three;
// so the phases are cut over the waves of a workgroup and kept short, O is made
// beside them, and the next chunk's rows and operands are loaded into the registers
// of this one's as soon as these have been used.
#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;

// What a wave takes of 16 NV value columns and C tokens: in the products over
// tokens block tb of 16 tokens and value blocks vb(0 .. kV - 1); of the state,
// blocks of 16 key columns kb(0 .. kB - 1) and value blocks sb(0 .. kS - 1).
template <int C, int KB, int NV>
struct Share {
  static constexpr int kTb = C / 16, kGroups = 4 / kTb, kV = (NV + kGroups - 1) / kGroups;
  static constexpr int kBlocks = 2 * KB, kB = kBlocks >= 4 ? kBlocks / 4 : 1;
  static constexpr int kS = kBlocks >= 4 ? NV : (NV + 1) / 2;
  int wave, tb, group;
  __device__ __forceinline__ explicit Share(int w) : wave(w), tb(w % kTb), group(kGroups > 1 ? w / kTb : 0) {}
  __device__ __forceinline__ int vb(int i) const { return group + kGroups * i; }
  __device__ __forceinline__ int kb(int i) const { return kBlocks >= 4 ? wave * kB + i : wave & 1; }
  __device__ __forceinline__ int sb(int i) const { return kBlocks >= 4 ? i : (wave >> 1) + 2 * i; }
};

struct Unit {
  int dv0, h, seq, len, chunks;
  long start, slot0;
};
template <int C, int NV>
__device__ __forceinline__ Unit delta_unit(const DeltaArgs& a) {
  Unit u;
  const int tiles = (a.dv + 16 * NV - 1) / (16 * NV);
  const long id = xcd_unit(blockIdx.x, gridDim.x);
  u.dv0 = (int)(id % tiles) * 16 * NV;
  u.h = (int)((id / tiles) % a.H);
  u.seq = (int)(id / ((long)tiles * a.H));
  if (a.cu) {
    const int c0 = min(max(a.cu[u.seq], 0), a.T), c1 = min(max(a.cu[u.seq + 1], c0), a.T);
    u.start = c0;
    u.len = c1 - c0;
    u.slot0 = (long)c0 / C + u.seq;
  } else {
    u.start = (long)u.seq * a.T;
    u.len = a.T;
    u.slot0 = (long)u.seq * a.slots_per_row;
  }
  u.chunks = (u.len + C - 1) / C;
  return u;
}

template <int C, int KB, int NV>
using State = f32x4[Share<C, KB, NV>::kB][Share<C, KB, NV>::kS];   // lane: value column c16, key columns 4 g + r

template <int C, int KB, int NV>
__device__ __forceinline__ void read_state(const DeltaArgs& a, const float* from, int dv0, const Share<C, KB, NV>& w, int c16, int g,
                                           State<C, KB, NV>& S) {
#pragma unroll
  for (int i = 0; i < w.kB; ++i)
#pragma unroll
    for (int j = 0; j < w.kS; ++j) {
      const int dk = 16 * w.kb(i) + 4 * g, dv = dv0 + 16 * w.sb(j) + c16;
      const bool in = from && w.sb(j) < NV && dk < a.dk && dv < a.dv;
      S[i][j] = in ? *reinterpret_cast<const f32x4*>(from + (long)dv * a.dk + dk) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
}
// Bytes of this lane's pieces of a state from its start, kOffNone where they lie outside.
template <int C, int KB, int NV>
struct StatePieces {
  uint32_t at[Share<C, KB, NV>::kB][Share<C, KB, NV>::kS];
  __device__ __forceinline__ StatePieces(const DeltaArgs& a, int dv0, const Share<C, KB, NV>& w, int c16, int g) {
#pragma unroll
    for (int i = 0; i < w.kB; ++i)
#pragma unroll
      for (int j = 0; j < w.kS; ++j) {
        const int dk = 16 * w.kb(i) + 4 * g, dv = dv0 + 16 * w.sb(j) + c16;
        at[i][j] = w.sb(j) < NV && dk < a.dk && dv < a.dv ? (uint32_t)((dv * a.dk + dk) * 4) : kOffNone;
      }
  }
  __device__ __forceinline__ void store(const DeltaArgs& a, float* to, const State<C, KB, NV>& S) const {
    const rsrc_t r = make_rsrc(to, (uint32_t)(a.dk * a.dv * 4));
#pragma unroll
    for (int i = 0; i < Share<C, KB, NV>::kB; ++i)
#pragma unroll
      for (int j = 0; j < Share<C, KB, NV>::kS; ++j) buf_store16(__builtin_bit_cast(u32x4, S[i][j]), r, at[i][j]);
  }
};
// The state's terms in LDS, [term][16 NV][kPitchK].
template <int C, int KB, int NV>
__device__ __forceinline__ void stage_state(uint16_t* Sl, const Share<C, KB, NV>& w, int c16, int g, const State<C, KB, NV>& S) {
  constexpr int kPitchK = lds_pitch(32 * KB);
#pragma unroll
  for (int i = 0; i < w.kB; ++i)
#pragma unroll
    for (int j = 0; j < w.kS; ++j) {
      if (w.sb(j) >= NV) continue;
      u32x2 part[kTerms];
      split4<kTerms>(S[i][j], part);
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        *reinterpret_cast<u32x2*>(Sl + (t * 16 * NV + 16 * w.sb(j) + c16) * kPitchK + 16 * w.kb(i) + 4 * g) = part[t];
    }
}
// Four values of token row in LDS, [term][C][pitch], at column col.
template <int C, int N, int PITCH>
__device__ __forceinline__ void stage4(uint16_t* L, int row, int col, f32x4 x) {
  u32x2 part[N];
  split4<N>(x, part);
#pragma unroll
  for (int t = 0; t < N; ++t) *reinterpret_cast<u32x2*>(L + (t * C + row) * PITCH + col) = part[t];
}
// Rows of the wave's tokens, 32 columns a piece, in LDS [term][C][kPitchK]. Waves that hold the same rows share the pieces out.
template <int C, int KB, int NV, int NX>
__device__ __forceinline__ void stage_rows(uint16_t* L, const Share<C, KB, NV>& w, int c16, int g, int b, const u32x4* part) {
  constexpr int kPitchK = lds_pitch(32 * KB);
  if (w.kGroups > 1 && b % w.kGroups != w.group && KB > 1) return;
#pragma unroll
  for (int t = 0; t < NX; ++t)
    *reinterpret_cast<u32x4*>(L + (t * C + 16 * w.tb + c16) * kPitchK + 32 * b + 8 * g) = part[t];
}
// Operands with k along the tokens 32 kp .. (order of an accumulator pair), N terms.
template <int C, int N, int PITCH>
__device__ __forceinline__ void tokens_operand(const uint16_t* L, int kp, int col, int lane, u32x4* out) {
#pragma unroll
  for (int t = 0; t < N; ++t) out[t] = frag_k_rows_accpair(L + t * C * PITCH, PITCH, 32 * kp, col, lane);
}
template <int N>
__device__ __forceinline__ void load_operand(const uint16_t* from, int lane, u32x4* out) {
#pragma unroll
  for (int t = 0; t < N; ++t) out[t] = *reinterpret_cast<const u32x4*>(from + t * kOperand + lane * 8);
}

// NX: terms of an input. KEEP: for the gradients; the states before the chunks and U are written, not O.
template <int C, int KB, int NV, int NX, bool KEEP>
__global__ __launch_bounds__(kThreads, KB <= 4 ? 2 : 1) void delta_fwd_kernel(DeltaArgs a) {
  using Sh = Share<C, KB, NV>;
  constexpr int kEsz = NX == 1 ? 2 : 4, kOut = out_terms(NX), kKp = C / 32;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = value_pitch(NV);
  __shared__ __align__(16) uint16_t Sl[kTerms * 16 * NV * kPitchK];
  __shared__ __align__(16) uint16_t Kl[NX * C * kPitchK];
  __shared__ __align__(16) uint16_t Xl[kTerms * C * kPitchV], Wl[kTerms * C * kPitchV];
  __shared__ __align__(16) uint16_t Ul[KEEP ? 8 : kOut * C * kPitchV];
  const Sh w(uniform(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const Unit u = delta_unit<C, NV>(a);
  const int hk = u.h / (a.H / a.Hk), tok = 16 * w.tb + c16;
  const long mat = (long)a.dk * a.dv;
  State<C, KB, NV> S;
  read_state<C, KB, NV>(a, a.init ? a.init + ((long)u.seq * a.H + u.h) * mat : nullptr, u.dv0, w, c16, g, S);
  stage_state<C, KB, NV>(Sl, w, c16, g, S);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  Raw8<NX> kr[KB], qr[KEEP ? 1 : KB];
  Raw4<NX> vr[Sh::kV];
  u32x4 tf[kKp][kTerms], pf[KEEP ? 1 : kKp][kOut];
  float eg = 0.f, wt = 0.f, keep = 0.f;
  // Byte offsets of this lane's pieces from a chunk's first row; rows behind the chunk lie behind its buffer's end.
  const int krow = (int)a.k_row * kEsz, qrow = (int)a.q_row * kEsz, vrow = (int)a.v_row * kEsz, orow = a.H * a.dv * kEsz;
  uint32_t kat[KB], qat[KB], vat[Sh::kV], oat[Sh::kV], uat[Sh::kV];
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    const int col = 32 * b + 8 * g;
    kat[b] = col < a.dk ? (uint32_t)(tok * krow + col * kEsz) : kOffNone;
    qat[b] = col < a.dk ? (uint32_t)(tok * qrow + col * kEsz) : kOffNone;
  }
#pragma unroll
  for (int i = 0; i < Sh::kV; ++i) {
    const int col = u.dv0 + 16 * w.vb(i) + 4 * g;
    const bool in = w.vb(i) < NV && col < a.dv;
    vat[i] = in ? (uint32_t)(tok * vrow + col * kEsz) : kOffNone;
    oat[i] = in ? (uint32_t)(tok * orow + col * kEsz) : kOffNone;
    uat[i] = in ? (uint32_t)((tok * a.dv + col) * 4) : kOffNone;
  }
  const StatePieces<C, KB, NV> pieces(a, u.dv0, w, c16, g);
  auto rows_of = [&](int c) { return min(C, u.len - c * C); };
  auto load_rows = [&](int c) {
    const int n = rows_of(c);
    const long row0 = u.start + (long)c * C;
    const rsrc_t rk = chunk_rows(a.k, row0, a.k_row, (long)hk * a.dk, n, kEsz);
    const rsrc_t rq = chunk_rows(a.q, row0, a.q_row, (long)hk * a.dk, n, kEsz);
    const rsrc_t rv = chunk_rows(a.v, row0, a.v_row, (long)u.h * a.dv, n, kEsz);
#pragma unroll
    for (int b = 0; b < KB; ++b) kr[b] = load8<NX>(rk, kat[b]);
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) vr[i] = load4<NX>(rv, vat[i]);
    const float* gates = a.gates + ((u.slot0 + c) * a.H + u.h) * kGateRows * C;
    eg = gates[tok];
    wt = gates[C + tok];
    keep = gates[5 * C];
#pragma unroll
    for (int b = 0; b < (KEEP ? 0 : KB); ++b) qr[b] = load8<NX>(rq, qat[b]);
  };
  // Operands above the diagonal are not used: the wave's last one again.
  auto load_t = [&](int c) {
    const uint16_t* at = a.tf + ((u.slot0 + c) * a.H + u.h) * operands(C, kTerms);
#pragma unroll
    for (int kp = 0; kp < kKp; ++kp) load_operand<kTerms>(at + operand_at(C, kTerms, w.tb, min(kp, w.tb / 2)), lane, tf[kp]);
  };
  auto load_p = [&](int c) {
    const uint16_t* at = a.pf + ((u.slot0 + c) * a.H + u.h) * operands(C, kOut);
#pragma unroll
    for (int kp = 0; kp < (KEEP ? 0 : kKp); ++kp)
      load_operand<kOut>(at + operand_at(C, kOut, w.tb, min(kp, w.tb / 2)), lane, pf[kp]);
  };
  if (u.chunks > 0) {
    load_rows(0);
    load_t(0);
    if (!KEEP) load_p(0);
  }
  loads_done();
  __syncthreads();

  for (int c = 0; c < u.chunks; ++c) {
    const int n = rows_of(c);
    const long row0 = u.start + (long)c * C, sh = (u.slot0 + c) * a.H + u.h;
    const int ahead = min(c + 1, u.chunks - 1);   // loaded without a branch, which would wait for the loads in flight
    if (KEEP) pieces.store(a, a.states + sh * mat, S);
    // X = V - e^G (K S^T), and Q S^T: lane token c16, value columns 4 g + r.
    f32x4 X[Sh::kV], O[Sh::kV];
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) X[i] = O[i] = zero;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      u32x4 kt[NX], qt[NX];
      terms8<NX>(kr[b], kt);
      stage_rows<C, KB, NV, NX>(Kl, w, c16, g, b, kt);
      if (!KEEP) terms8<NX>(qr[b], qt);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
        u32x4 st[kTerms];
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          st[t] = frag_k_cols(Sl + t * 16 * NV * kPitchK, kPitchK, 16 * w.vb(i), 32 * b, lane);
        X[i] = mma<kTerms, NX, kTerms>(st, kt, X[i]);
        if (!KEEP) O[i] = mma<kOut, NX, kOut>(st, qt, O[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) {
      if (w.vb(i) >= NV) continue;
      const f32x4 v = floats4<NX>(vr[i]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        X[i][r] = fmaf(-eg, X[i][r], v[r]);
        O[i][r] *= eg * a.scale;
      }
      stage4<C, kTerms, kPitchV>(Xl, tok, 16 * w.vb(i) + 4 * g, X[i]);
    }
    const float wt_now = wt, keep_now = keep;
    load_rows(ahead);
    __syncthreads();

    // U = T diag(beta) X.
    f32x4 U[Sh::kV];
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) {
      if (w.vb(i) >= NV) continue;
      U[i] = zero;
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) {
        if (kp > w.tb / 2) continue;
        u32x4 xt[kTerms];
        tokens_operand<C, kTerms, kPitchV>(Xl, kp, 16 * w.vb(i), lane, xt);
        U[i] = mma<kTerms, kTerms, kTerms>(xt, tf[kp], U[i]);
      }
      if (!KEEP) stage4<C, kOut, kPitchV>(Ul, tok, 16 * w.vb(i) + 4 * g, U[i]);
      stage4<C, kTerms, kPitchV>(Wl, tok, 16 * w.vb(i) + 4 * g, U[i] * wt_now);
      if (KEEP) buf_store16(__builtin_bit_cast(u32x4, U[i]), make_rsrc(a.u + sh * C * a.dv, (uint32_t)(C * a.dv * 4)), uat[i]);
    }
    load_t(ahead);
    __syncthreads();

    // S = e^(G_C) S + (e^(G_C - G) U)^T K.
#pragma unroll
    for (int i = 0; i < Sh::kB; ++i)
#pragma unroll
      for (int j = 0; j < Sh::kS; ++j) S[i][j] *= keep_now;
#pragma unroll
    for (int kp = 0; kp < kKp; ++kp) {
      u32x4 ut[Sh::kS][kTerms];
#pragma unroll
      for (int j = 0; j < Sh::kS; ++j)
        if (w.sb(j) < NV) tokens_operand<C, kTerms, kPitchV>(Wl, kp, 16 * w.sb(j), lane, ut[j]);
#pragma unroll
      for (int i = 0; i < Sh::kB; ++i) {
        u32x4 kt[NX];
        tokens_operand<C, NX, kPitchK>(Kl, kp, 16 * w.kb(i), lane, kt);
#pragma unroll
        for (int j = 0; j < Sh::kS; ++j)
          if (w.sb(j) < NV) S[i][j] = mma<NX, kTerms, kTerms>(kt, ut[j], S[i][j]);
      }
    }
    stage_state<C, KB, NV>(Sl, w, c16, g, S);
    if (!KEEP) {
      const rsrc_t ro = chunk_rows(a.o, row0, (long)a.H * a.dv, (long)u.h * a.dv, n, kEsz);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
#pragma unroll
        for (int kp = 0; kp < kKp; ++kp) {
          if (kp > w.tb / 2) continue;
          u32x4 ut[kOut];
          tokens_operand<C, kOut, kPitchV>(Ul, kp, 16 * w.vb(i), lane, ut);
          O[i] = mma<kOut, kOut, kOut>(ut, pf[kp], O[i]);
        }
        store4<NX>(O[i], ro, oat[i]);
      }
      load_p(ahead);
    }
    __syncthreads();
  }
  if (a.fin) pieces.store(a, a.fin + ((long)u.seq * a.H + u.h) * mat, S);
}

// The adjoint, from the last chunk to the first: U', dV, the gradients of the states before the chunks.
template <int C, int KB, int NV, int NX>
__global__ __launch_bounds__(kThreads, KB <= 4 && NX == 1 ? 2 : 1) void delta_rev_kernel(DeltaArgs a) {
  using Sh = Share<C, KB, NV>;
  constexpr int kEsz = NX == 1 ? 2 : 4, kKp = C / 32;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = value_pitch(NV);
  __shared__ __align__(16) uint16_t Ll[kTerms * 16 * NV * kPitchK];
  __shared__ __align__(16) uint16_t Kl[NX * C * kPitchK], Ql[NX * C * kPitchK];
  __shared__ __align__(16) uint16_t Ol[NX * C * kPitchV];                                  // dO
  __shared__ __align__(16) uint16_t Gl[kTerms * C * kPitchV], Yl[kTerms * C * kPitchV];    // scale e^G dO; Y
  __shared__ __align__(16) uint16_t Xl[kTerms * C * kPitchV];                              // -e^G beta U'
  const Sh w(uniform(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const Unit u = delta_unit<C, NV>(a);
  const int hk = u.h / (a.H / a.Hk), tok = 16 * w.tb + c16;
  const long mat = (long)a.dk * a.dv;
  State<C, KB, NV> L;
  read_state<C, KB, NV>(a, a.dfin ? a.dfin + ((long)u.seq * a.H + u.h) * mat : nullptr, u.dv0, w, c16, g, L);
  stage_state<C, KB, NV>(Ll, w, c16, g, L);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  Raw8<NX> kr[KB], qr[KB];
  Raw4<NX> dor[Sh::kV];
  u32x4 tt[kKp][kTerms], pt[kKp][kTerms];
  float eg = 0.f, wt = 0.f, be = 0.f, keep = 0.f;
  // Byte offsets of this lane's pieces from a chunk's first row; rows behind the chunk lie behind its buffer's end.
  const int krow = (int)a.k_row * kEsz, qrow = (int)a.q_row * kEsz, orow = a.H * a.dv * kEsz;
  uint32_t kat[KB], qat[KB], oat[Sh::kV], uat[Sh::kV];
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    const int col = 32 * b + 8 * g;
    kat[b] = col < a.dk ? (uint32_t)(tok * krow + col * kEsz) : kOffNone;
    qat[b] = col < a.dk ? (uint32_t)(tok * qrow + col * kEsz) : kOffNone;
  }
#pragma unroll
  for (int i = 0; i < Sh::kV; ++i) {
    const int col = u.dv0 + 16 * w.vb(i) + 4 * g;
    const bool in = w.vb(i) < NV && col < a.dv;
    oat[i] = in ? (uint32_t)(tok * orow + col * kEsz) : kOffNone;
    uat[i] = in ? (uint32_t)((tok * a.dv + col) * 4) : kOffNone;
  }
  const StatePieces<C, KB, NV> pieces(a, u.dv0, w, c16, g);
  auto rows_of = [&](int c) { return min(C, u.len - c * C); };
  auto load_rows = [&](int c) {
    const int n = rows_of(c);
    const long row0 = u.start + (long)c * C;
    const rsrc_t rk = chunk_rows(a.k, row0, a.k_row, (long)hk * a.dk, n, kEsz);
    const rsrc_t rq = chunk_rows(a.q, row0, a.q_row, (long)hk * a.dk, n, kEsz);
    const rsrc_t ro = chunk_rows(a.d_o, row0, (long)a.H * a.dv, (long)u.h * a.dv, n, kEsz);
#pragma unroll
    for (int b = 0; b < KB; ++b) kr[b] = load8<NX>(rk, kat[b]);
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) dor[i] = load4<NX>(ro, oat[i]);
    const float* gates = a.gates + ((u.slot0 + c) * a.H + u.h) * kGateRows * C;
    eg = gates[tok];
    wt = gates[C + tok];
    be = gates[2 * C + tok];
    keep = gates[5 * C];
#pragma unroll
    for (int b = 0; b < KB; ++b) qr[b] = load8<NX>(rq, qat[b]);
  };
  // Operands below the diagonal are not used: the wave's first one again.
  auto load_operands = [&](const uint16_t* from, int c, u32x4 (*to)[kTerms]) {
    const uint16_t* at = from + ((u.slot0 + c) * a.H + u.h) * operands(C, kTerms);
#pragma unroll
    for (int kp = 0; kp < kKp; ++kp) load_operand<kTerms>(at + operand_at(C, kTerms, w.tb, max(kp, w.tb / 2)), lane, to[kp]);
  };
  auto stage_do = [&]() {
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i)
      if (w.vb(i) < NV) stage4<C, NX, kPitchV>(Ol, tok, 16 * w.vb(i) + 4 * g, floats4<NX>(dor[i]));
  };
  if (u.chunks > 0) {
    load_rows(u.chunks - 1);
    load_operands(a.tt, u.chunks - 1, tt);
    load_operands(a.pt, u.chunks - 1, pt);
    stage_do();
  }
  loads_done();
  __syncthreads();

  for (int c = u.chunks - 1; c >= 0; --c) {
    const int n = rows_of(c);
    const long row0 = u.start + (long)c * C, sh = (u.slot0 + c) * a.H + u.h;
    const int ahead = max(c - 1, 0);   // loaded without a branch, which would wait for the loads in flight
    pieces.store(a, a.dstates + sh * mat, L);
    // Y = e^(G_C - G) (K L^T) + P^T dO.
    f32x4 Y[Sh::kV];
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) Y[i] = zero;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      u32x4 kt[NX], qt[NX];
      terms8<NX>(kr[b], kt);
      terms8<NX>(qr[b], qt);
      stage_rows<C, KB, NV, NX>(Kl, w, c16, g, b, kt);
      stage_rows<C, KB, NV, NX>(Ql, w, c16, g, b, qt);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
        u32x4 st[kTerms];
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          st[t] = frag_k_cols(Ll + t * 16 * NV * kPitchK, kPitchK, 16 * w.vb(i), 32 * b, lane);
        Y[i] = mma<kTerms, NX, kTerms>(st, kt, Y[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) {
      if (w.vb(i) >= NV) continue;
      Y[i] *= wt;
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) {
        if (kp < w.tb / 2) continue;
        u32x4 ot[NX];
        tokens_operand<C, NX, kPitchV>(Ol, kp, 16 * w.vb(i), lane, ot);
        Y[i] = mma<NX, kTerms, kTerms>(ot, pt[kp], Y[i]);
      }
      const int col = 16 * w.vb(i) + 4 * g;
      stage4<C, kTerms, kPitchV>(Gl, tok, col, floats4<NX>(dor[i]) * (eg * a.scale));
      stage4<C, kTerms, kPitchV>(Yl, tok, col, Y[i]);
    }
    const float eg_now = eg, be_now = be, keep_now = keep;
    load_rows(ahead);
    load_operands(a.pt, ahead, pt);
    __syncthreads();

    // U' = T^T Y, dV = beta U'.
    f32x4 U[Sh::kV];
    const rsrc_t rv = chunk_rows(a.dv_out, row0, (long)a.H * a.dv, (long)u.h * a.dv, n, kEsz);
#pragma unroll
    for (int i = 0; i < Sh::kV; ++i) {
      if (w.vb(i) >= NV) continue;
      U[i] = zero;
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) {
        if (kp < w.tb / 2) continue;
        u32x4 yt[kTerms];
        tokens_operand<C, kTerms, kPitchV>(Yl, kp, 16 * w.vb(i), lane, yt);
        U[i] = mma<kTerms, kTerms, kTerms>(yt, tt[kp], U[i]);
      }
      buf_store16(__builtin_bit_cast(u32x4, U[i]), make_rsrc(a.ub + sh * C * a.dv, (uint32_t)(C * a.dv * 4)), uat[i]);
      store4<NX>(U[i] * be_now, rv, oat[i]);
      stage4<C, kTerms, kPitchV>(Xl, tok, 16 * w.vb(i) + 4 * g, U[i] * (-eg_now * be_now));
    }
    load_operands(a.tt, ahead, tt);
    __syncthreads();

    // L = e^(G_C) L + scale (e^G dO)^T Q - (e^G beta U')^T K.
#pragma unroll
    for (int i = 0; i < Sh::kB; ++i)
#pragma unroll
      for (int j = 0; j < Sh::kS; ++j) L[i][j] *= keep_now;
#pragma unroll
    for (int kp = 0; kp < kKp; ++kp) {
      u32x4 gt[Sh::kS][kTerms], xt[Sh::kS][kTerms];
#pragma unroll
      for (int j = 0; j < Sh::kS; ++j) {
        if (w.sb(j) >= NV) continue;
        tokens_operand<C, kTerms, kPitchV>(Gl, kp, 16 * w.sb(j), lane, gt[j]);
        tokens_operand<C, kTerms, kPitchV>(Xl, kp, 16 * w.sb(j), lane, xt[j]);
      }
#pragma unroll
      for (int i = 0; i < Sh::kB; ++i) {
        u32x4 kt[NX], qt[NX];
        tokens_operand<C, NX, kPitchK>(Kl, kp, 16 * w.kb(i), lane, kt);
        tokens_operand<C, NX, kPitchK>(Ql, kp, 16 * w.kb(i), lane, qt);
#pragma unroll
        for (int j = 0; j < Sh::kS; ++j) {
          if (w.sb(j) >= NV) continue;
          L[i][j] = mma<NX, kTerms, kTerms>(qt, gt[j], L[i][j]);
          L[i][j] = mma<NX, kTerms, kTerms>(kt, xt[j], L[i][j]);
        }
      }
    }
    stage_state<C, KB, NV>(Ll, w, c16, g, L);
    stage_do();
    __syncthreads();
  }
  if (a.dinit) pieces.store(a, a.dinit + ((long)u.seq * a.H + u.h) * mat, L);
}

// Value blocks a workgroup: with keys of 256, fp32 rows leave LDS for one.
constexpr int kNv64 = 1;
constexpr int nv32(int kb) { return kb > 4 ? 1 : 2; }

template <int KB>
void fwd(const DeltaArgs& a, bool keep, hipStream_t stream) {
  const dim3 grid((unsigned)delta_chain_blocks(a, false));
  if (a.bf16) {
    if (keep) hipLaunchKernelGGL((delta_fwd_kernel<64, KB, kNv64, 1, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((delta_fwd_kernel<64, KB, kNv64, 1, false>), grid, dim3(kThreads), 0, stream, a);
  } else {
    if (keep) hipLaunchKernelGGL((delta_fwd_kernel<32, KB, nv32(KB), 3, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((delta_fwd_kernel<32, KB, nv32(KB), 3, false>), grid, dim3(kThreads), 0, stream, a);
  }
}
template <int KB>
void rev(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)delta_chain_blocks(a, true));
  if (a.bf16) hipLaunchKernelGGL((delta_rev_kernel<64, KB, kNv64, 1>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((delta_rev_kernel<32, KB, nv32(KB), 3>), grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

long delta_chain_blocks(const DeltaArgs& a, bool) {
  const int cols = 16 * (a.bf16 ? kNv64 : nv32((a.dk + 31) / 32));
  return (long)(a.S > 0 ? a.S : a.batch) * a.H * ((a.dv + cols - 1) / cols);
}
int delta_chain_threads() { return kThreads; }

hipError_t launch_delta_fwd(const DeltaArgs& a, bool keep, hipStream_t stream) {
  if (a.dk <= 32) fwd<1>(a, keep, stream);
  else if (a.dk <= 64) fwd<2>(a, keep, stream);
  else if (a.dk <= 128) fwd<4>(a, keep, stream);
  else fwd<8>(a, keep, stream);
  return hipGetLastError();
}

hipError_t launch_delta_rev(const DeltaArgs& a, hipStream_t stream) {
  if (a.dk <= 32) rev<1>(a, stream);
  else if (a.dk <= 64) rev<2>(a, stream);
  else if (a.dk <= 128) rev<4>(a, stream);
  else rev<8>(a, stream);
  return hipGetLastError();
}

}  // namespace ssd
