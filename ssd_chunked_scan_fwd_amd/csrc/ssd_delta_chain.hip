// ssd_delta_chain.hip -- the walk of the delta rule over the chunks of each
// sequence, forwards and, for the gradients, backwards (formulas: ssd_delta.h).
//
// Columns of V, rows of the state, do not mix: a workgroup takes NV blocks of 16
// of them of one head. What a chunk waits for is a chain of three phases, each
// ending in a barrier: state times keys (X, or Y)  ->  times T (U, or U')  ->  state
// update. The longest chain of a call is its longest sequence's chunks times these
// three, and few heads leave a SIMD one wave of it. So the phases are kept short:
// four waves, the token waves, take the first two, 16 tokens each, and do nothing
// else; four others, the state waves, hold the state in the accumulators of its
// update, a quarter of dk each, and make what nothing waits for (O; backwards the
// terms of dO) while the token waves work. The next chunk's rows and operands are
// loaded into the registers of this one's as soon as these have been used.
// 16384 tokens, 32 heads on 16 of 128 x 128: 506 us for 256 chunks, 2.0 a chunk, at the least in a trace, which slows
// calls (back to back matrices and walk take 580, of which the matrices 100); 475 MB read, 136 MB written: 1.2 TB/s. Its
// products, 28 million operations a chunk and head in their terms, would take 213 us at the rate of a large product.
// Backwards 8192 tokens 321 us. LDS is busy 38 % of the time, the vector units 35 %, the matrix units 20 %, hardly at the
// same time: the phases' dependent reads, products and splits into terms bound it. With the loads of every chunk from the
// first's rows, out of the caches, the walk of 8192 tokens took 30 us less of 234; two workgroups on a CU together gained
// a tenth on one after the other (both with two terms in o's products). Where the workgroups of ragged sequences fall,
// long ones side by side on a CU or not, moves a call by up to 20 us of 100 with anything that shifts their start.
#include <algorithm>

#include "ssd_delta_tile.h"

namespace ssd {

namespace {

constexpr int kThreads = 512;   // four token waves, four state waves

// What wave w of four takes of 16 NV value columns and C tokens: in the products
// over tokens block tb of 16 tokens and value blocks vb(0 .. kV - 1); of the state,
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

// What a workgroup walks: columns dv0 .. of one head over a sequence, or over one of its segments. Of a segment's own
// states, after those of its value columns, the rows of its map: V = 0, and the rows of the unit matrix as the state
// before it.
struct Unit {
  int dv0, h, len, chunks, rows;   // rows of the state
  long start, slot0;
  bool map, none;
  const float* from;               // the state before, null: zero
  float* to;                       // the state behind, null: not wanted
};
// REV: backwards, `first` and `last` the gradients of the last and of the first state.
template <int C, int NV, bool OWN, bool REV>
__device__ __forceinline__ Unit delta_unit(const DeltaArgs& a, int block, const float* first, float* last) {
  Unit u;
  const int values = (a.dv + 16 * NV - 1) / (16 * NV), tiles = values + (OWN && !REV ? (a.dk + 16 * NV - 1) / (16 * NV) : 0);
  const long id = xcd_unit(block, gridDim.x), mat = (long)a.dk * a.dv, map = (long)a.dk * a.dk;
  const int tile = (int)(id % tiles);
  // Sequence or segment before head: an XCD takes a contiguous range of units, and all sequences, long and short, of
  // its heads. (Heads first, an XCD had one of eight ragged sequences: 102 us for what then took 70.)
  const long all = a.seg ? a.segs : (long)(a.S > 0 ? a.S : a.batch), n = (id / tiles) % all;
  u.h = (int)(id / (tiles * all));
  u.map = OWN && !REV && tile >= values;
  u.dv0 = (u.map ? tile - values : tile) * 16 * NV;
  u.rows = u.map ? a.dk : a.dv;
  u.none = false;
  LinPiece q;
  if (a.seg) {
    q = lin_piece(a.cu, a.S, a.T, a.seg * C, a.segs_per_row, n);
  } else {
    const int c0 = a.cu ? min(max(a.cu[n], 0), a.T) : 0;
    q.seq = (int)n;
    q.blk = 0;
    q.start = a.cu ? c0 : n * a.T;
    q.len = a.cu ? min(max(a.cu[n + 1], c0), a.T) - c0 : a.T;
  }
  const int blk = q.blk;
  if (blk < 0) {
    u.none = true;
    return u;
  }
  const long begin = (long)blk * a.seg * C;
  u.len = a.seg ? (int)min((long)q.len - begin, (long)a.seg * C) : q.len;
  u.chunks = (u.len + C - 1) / C;
  u.start = q.start + begin;
  u.slot0 = (a.cu ? q.start / C + q.seq : (long)q.seq * a.slots_per_row) + begin / C;
  const bool at_end = begin + u.len >= q.len, entry = REV ? at_end : blk == 0, exit = REV ? blk == 0 : at_end;
  const long sh = (long)q.seq * a.H + u.h;
  float* const states = REV ? a.seg_adj : a.seg_states;
  if (OWN) {
    u.none = exit || (u.map && entry);   // nothing comes behind it; the state before it is known
    u.from = entry && first && !u.map ? first + sh * mat : nullptr;
    u.to = u.map ? a.seg_maps + (n * a.H + u.h) * map : states + (n * a.H + u.h) * mat;
  } else {
    u.from = !entry ? states + ((REV ? n + 1 : n - 1) * a.H + u.h) * mat : first ? first + sh * mat : nullptr;
    u.to = exit && last ? last + sh * mat : nullptr;
  }
  return u;
}

template <int C, int KB, int NV>
using State = f32x4[Share<C, KB, NV>::kB][Share<C, KB, NV>::kS];   // lane: value column c16, key columns 4 g + r

template <int C, int KB, int NV>
__device__ __forceinline__ void read_state(const DeltaArgs& a, const Unit& u, const Share<C, KB, NV>& w, int c16, int g,
                                           State<C, KB, NV>& S) {
#pragma unroll
  for (int i = 0; i < w.kB; ++i)
#pragma unroll
    for (int j = 0; j < w.kS; ++j) {
      const int dk = 16 * w.kb(i) + 4 * g, dv = u.dv0 + 16 * w.sb(j) + c16;
      const bool in = u.from && w.sb(j) < NV && dk < a.dk && dv < u.rows;
      S[i][j] = in ? *reinterpret_cast<const f32x4*>(u.from + (long)dv * a.dk + dk) : f32x4{0.f, 0.f, 0.f, 0.f};
      if (u.map) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][j][r] = dk + r == dv ? 1.f : 0.f;
      }
    }
}
// Bytes of this lane's pieces of a state from its start, kOffNone where they lie outside.
template <int C, int KB, int NV>
struct StatePieces {
  uint32_t at[Share<C, KB, NV>::kB][Share<C, KB, NV>::kS];
  uint32_t bytes;
  __device__ __forceinline__ StatePieces(const DeltaArgs& a, const Unit& u, const Share<C, KB, NV>& w, int c16, int g)
      : bytes((uint32_t)(a.dk * u.rows * 4)) {
#pragma unroll
    for (int i = 0; i < w.kB; ++i)
#pragma unroll
      for (int j = 0; j < w.kS; ++j) {
        const int dk = 16 * w.kb(i) + 4 * g, dv = u.dv0 + 16 * w.sb(j) + c16;
        at[i][j] = w.sb(j) < NV && dk < a.dk && dv < u.rows ? (uint32_t)((dv * a.dk + dk) * 4) : kOffNone;
      }
  }
  __device__ __forceinline__ void store(float* to, const State<C, KB, NV>& S) const {
    const rsrc_t r = make_rsrc(to, bytes);
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
  for (int t = 0; t < N; ++t) *reinterpret_cast<u32x2*>(L + t * C * PITCH + value_at<PITCH>(row, col)) = part[t];
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
// Operands with k along the tokens 32 kp .. (order of an accumulator pair), N terms, of rows of values
template <int C, int N, int PITCH>
__device__ __forceinline__ void values_operand(const uint16_t* L, int kp, int col, int lane, u32x4* out) {
  const int i = lane & 15, g = lane >> 4;
  const uint16_t* p0 = L + value_at<PITCH>(32 * kp + 4 * g + (i >> 2), col + 4 * (i & 3));
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const u32x2 lo = lds_read_tr16(p0 + t * C * PITCH), hi = lds_read_tr16(p0 + (t * C + 16) * PITCH);
    out[t] = u32x4{lo.x, lo.y, hi.x, hi.y};
  }
}
// and of rows of keys, [term][C][PITCH].
template <int C, int N, int PITCH>
__device__ __forceinline__ void tokens_operand(const uint16_t* L, int kp, int col, int lane, u32x4* out) {
#pragma unroll
  for (int t = 0; t < N; ++t) out[t] = frag_k_rows_accpair(L + t * C * PITCH, PITCH, 32 * kp, col, lane);
}
// The lane's pieces of a chunk, byte offsets from its first row: of rows of keys (row elements apart), 32 columns
// a piece, and of rows of values, 16 columns a piece; kOffNone behind the columns. Rows behind the chunk lie behind
// its buffer's end.
template <int KB>
struct KeyPieces {
  uint32_t at[KB];
  __device__ __forceinline__ KeyPieces(int tok, int g, long row, int end, int esz) {
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int col = 32 * b + 8 * g;
      at[b] = col < end ? (uint32_t)((tok * (int)row + col) * esz) : kOffNone;
    }
  }
};
template <int C, int KB, int NV>
struct ValuePieces {
  uint32_t at[Share<C, KB, NV>::kV];
  __device__ __forceinline__ ValuePieces(const Share<C, KB, NV>& w, int tok, int g, int dv0, long row, int end, int esz) {
#pragma unroll
    for (int i = 0; i < Share<C, KB, NV>::kV; ++i) {
      const int col = dv0 + 16 * w.vb(i) + 4 * g;
      at[i] = w.vb(i) < NV && col < end ? (uint32_t)((tok * (int)row + col) * esz) : kOffNone;
    }
  }
};
// The state (N of its terms, value block vb) times rows of keys: lane token c16, value columns 4 g + r. The operands
// of four pieces are on their way at once, and the terms' products are chains of their own.
template <int KB, int NV, int NX, int N>
__device__ __forceinline__ f32x4 state_times(const uint16_t* Sl, int vb, const u32x4 (*kt)[NX], int lane) {
  constexpr int kPitchK = lds_pitch(32 * KB), kAtOnce = KB < 4 ? KB : 4;
  f32x4 sum[N];
#pragma unroll
  for (int t = 0; t < N; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b0 = 0; b0 < KB; b0 += kAtOnce) {
    u32x4 st[kAtOnce][N];
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b)
#pragma unroll
      for (int t = 0; t < N; ++t) st[b][t] = frag_k_cols(Sl + t * 16 * NV * kPitchK, kPitchK, 16 * vb, 32 * (b0 + b), lane);
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b)
#pragma unroll
      for (int t = 0; t < N; ++t) sum[t] = mma<1, NX, N>(&st[b][t], kt[b0 + b], t, sum[t]);
  }
  f32x4 x = sum[N - 1];
#pragma unroll
  for (int t = N - 2; t >= 0; --t) x += sum[t];
  return x;
}
// S += M^T Y over the tokens 32 kp .., M rows of keys and Y of values in LDS.
template <int C, int KB, int NV, int NX>
__device__ __forceinline__ void state_update(const uint16_t* M, const uint16_t* Y, const Share<C, KB, NV>& w, int kp, int lane,
                                             State<C, KB, NV>& S) {
  using Sh = Share<C, KB, NV>;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = value_pitch(NV);
  u32x4 yt[Sh::kS][kTerms];
#pragma unroll
  for (int j = 0; j < Sh::kS; ++j)
    if (w.sb(j) < NV) values_operand<C, kTerms, kPitchV>(Y, kp, 16 * w.sb(j), lane, yt[j]);
#pragma unroll
  for (int i = 0; i < Sh::kB; ++i) {
    u32x4 mt[NX];
    tokens_operand<C, NX, kPitchK>(M, kp, 16 * w.kb(i), lane, mt);
#pragma unroll
    for (int j = 0; j < Sh::kS; ++j)
      if (w.sb(j) < NV) S[i][j] = mma<NX, kTerms, kTerms>(mt, yt[j], S[i][j]);
  }
}
template <int C, int KB, int NV>
__device__ __forceinline__ void scale_state(State<C, KB, NV>& S, float by) {
#pragma unroll
  for (int i = 0; i < Share<C, KB, NV>::kB; ++i)
#pragma unroll
    for (int j = 0; j < Share<C, KB, NV>::kS; ++j) S[i][j] *= by;
}

// x, of token tok and four value columns, is not finite: where its own share is, the sum over the tokens up to tok alone,
// which those behind it do not reach. (Matrix instructions take all tokens, the later ones times zero: what is not
// finite in one of them would run against time.) w: a row of weights of the tokens, L: [term][C][PITCH] of their values.
template <int C, int PITCH, typename Matrix>
__device__ __forceinline__ f32x4 sum_so_far(f32x4 x, f32x4 own, const Matrix* w, const uint16_t* L, int tok, int col) {
  f32x4 sum = own;
#pragma unroll 1
  for (int k = 0; k <= tok; ++k) {
    const float weight = operand_value<C>(w, tok / 16, tok & 15, k);
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = kTerms - 1; t >= 0; --t) y += four(*reinterpret_cast<const u32x2*>(L + t * C * PITCH + value_at<PITCH>(k, col)));
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] = fmaf(weight, y[r], sum[r]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (x[r] * 0.f != 0.f && own[r] * 0.f == 0.f) x[r] = sum[r];
  return x;
}
// U of a chunk's n tokens one after the other, U_i = beta_i (X_i - sum_{j < i} D_ij k_i.k_j U_j), a lane a value column: as
// the inverse, made by blocks, holds zeros times what is not finite in rows that this does not reach. One wave.
template <int C, int KB, int NV, int NX, int PITCH>
__device__ __forceinline__ void updates_by_token(const float* gates, const uint16_t* Kl, const uint16_t* Xl, float* Uf, int n, int lane) {
  constexpr int kPitchK = lds_pitch(32 * KB), kWide = 16 * NV;
  const int col = min(lane, kWide - 1);
  auto key = [&](int row) {   // this lane's four of it
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (4 * lane < 32 * KB) {
#pragma unroll
      for (int t = NX - 1; t >= 0; --t) x += four(*reinterpret_cast<const u32x2*>(Kl + (t * C + row) * kPitchK + 4 * lane));
    }
    return x;
  };
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const f32x4 ki = key(i);
    float x = 0.f;
#pragma unroll
    for (int t = kTerms - 1; t >= 0; --t) x += bf16_to_f32(Xl[t * C * PITCH + value_at<PITCH>(i, col)]);
#pragma unroll 1
    for (int j = 0; j < i; ++j) {
      const f32x4 kj = key(j);
      const float kk = lanes_sum<64>(fmaf(ki[0], kj[0], fmaf(ki[1], kj[1], fmaf(ki[2], kj[2], ki[3] * kj[3]))), 64);
      const float d = exp_of((gates[3 * C + i] - gates[3 * C + j]) + (gates[4 * C + i] - gates[4 * C + j]));
      x = fmaf(-d * kk, Uf[j * kWide + col], x);
    }
    if (lane < kWide) Uf[i * kWide + col] = gates[2 * C + i] * x;
    __builtin_amdgcn_wave_barrier();
  }
}

// What a forward walk writes: O; for the gradients, the states before the chunks and U; of a segment, its own last
// state or map.
enum { kOutputs, kKeep, kOwn };

// NX: terms of an input.
template <int C, int KB, int NV, int NX, int WHAT>
__global__ __launch_bounds__(kThreads, KB <= 4 && NX == 1 && NV == 1 ? 4 : 2) void delta_fwd_kernel(DeltaArgs args) {
  using Sh = Share<C, KB, NV>;
  constexpr bool KEEP = WHAT != kOutputs;
  constexpr int kEsz = NX == 1 ? 2 : 4, kKp = C / 32;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = value_pitch(NV);
  __shared__ __align__(16) uint16_t Sl[kTerms * 16 * NV * kPitchK];
  __shared__ __align__(16) uint16_t Kl[NX * C * kPitchK];
  __shared__ __align__(16) uint16_t Xl[kTerms * C * kPitchV], Wl[kTerms * C * kPitchV];   // X; e^(G_C - G) U
  constexpr int kU = kTerms * C * kPitchV;
  __shared__ __align__(16) uint16_t Ul[KEEP ? 8 : 2 * kU];   // U of this chunk and of the one before
  __shared__ int lost, again;   // the last state is not finite; updates of a chunk are to be made again
  // CAREFUL: with what is not finite kept to where the rule brings it. A walk of outputs that ends in a state that is not
  // finite (once it is not, no later one is) is walked once more so, in code of its own, which leaves the other's time as
  // it is (16384 tokens 579 us for 580; a check of every chunk's O in one walk for both took 617, 8192 tokens of fp32 901 for
  // 795). The walks that keep or make states alone need none of it: U that is not finite makes its state so.
  auto walk = [&](auto careful, const DeltaArgs& a) {
    constexpr bool CAREFUL = decltype(careful)::value;
    int tid = threadIdx.x, block = blockIdx.x;
    if (CAREFUL) asm volatile("" : "+v"(tid), "+s"(block));   // what follows from them is made anew, not kept over the walk
    const int wave = uniform(tid >> 6);
    const Sh w(wave & 3);
    const int lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const Unit u = delta_unit<C, NV, WHAT == kOwn, false>(a, block, a.init, a.fin);
    if (u.none) return false;
    const int hk = u.h / (a.H / a.Hk), tok = 16 * w.tb + c16, last = u.chunks - 1;
    const long mat = (long)a.dk * a.dv, sh0 = u.slot0 * a.H + u.h;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    auto rows = [&](const void* x, int c, long row, long col) {
      return chunk_rows(x, u.start + (long)c * C, row, col, min(C, u.len - c * C), kEsz);
    };

    if (wave < 4) {
      const KeyPieces<KB> kat(tok, g, a.k_row, a.dk, kEsz);
      const ValuePieces<C, KB, NV> vat(w, tok, g, u.dv0, a.v_row, u.map ? 0 : a.dv, kEsz), uat(w, tok, g, u.dv0, a.dv, a.dv, 4);
      Raw8<NX> kr[KB];
      Raw4<NX> vr[Sh::kV];
      u32x4 tf[kKp][kTerms];
      RawOperand tn[kKp];   // of the next chunk
      float eg, wt, eg_next, wt_next;
      auto load_rows = [&](int c) {
        const rsrc_t rk = rows(a.k, c, a.k_row, (long)hk * a.dk), rv = rows(a.v, c, a.v_row, (long)u.h * a.dv);
#pragma unroll
        for (int b = 0; b < KB; ++b) kr[b] = load8<NX>(rk, kat.at[b]);
#pragma unroll
        for (int i = 0; i < Sh::kV; ++i) vr[i] = load4<NX>(rv, vat.at[i]);
      };
      auto load_gates = [&](int c) {
        const float* gates = a.gates + (sh0 + (long)c * a.H) * kGateRows * C;
        eg_next = gates[tok];
        wt_next = gates[C + tok];
      };
      auto next = [&]() {
        eg = eg_next;
        wt = wt_next;
#pragma unroll
        for (int kp = 0; kp < kKp; ++kp) terms8<kTerms>(tn[kp], tf[kp]);
      };
      auto load_t = [&](int c) { load_operands<C>(a.tf, sh0 + (long)c * a.H, w.tb, 0, w.tb / 2, lane, tn); };
      if (last >= 0) {
        load_rows(0);
        load_gates(0);
        load_t(0);
        next();
        load_t(min(1, last));
        load_gates(min(1, last));
      }
      loads_done();
      __syncthreads();
      for (int c = 0; c <= last; ++c) {
        const long sh = sh0 + (long)c * a.H;
        // X = V - e^G (K S^T): lane token c16, value columns 4 g + r.
        f32x4 X[Sh::kV];
        u32x4 kt[KB][NX];
#pragma unroll
        for (int b = 0; b < KB; ++b) terms8<NX>(kr[b], kt[b]);
#pragma unroll
        for (int i = 0; i < Sh::kV; ++i) {
          if (w.vb(i) >= NV) continue;
          const f32x4 v = floats4<NX>(vr[i]);
          X[i] = state_times<KB, NV, NX, kTerms>(Sl, w.vb(i), kt, lane);
#pragma unroll
          for (int r = 0; r < 4; ++r) X[i][r] = fmaf(-eg, X[i][r], v[r]);
          stage4<C, kTerms, kPitchV>(Xl, tok, 16 * w.vb(i) + 4 * g, X[i]);
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) stage_rows<C, KB, NV, NX>(Kl, w, c16, g, b, kt[b]);
        load_rows(min(c + 1, last));
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
            values_operand<C, kTerms, kPitchV>(Xl, kp, 16 * w.vb(i), lane, xt);
            U[i] = mma<kTerms, kTerms, kTerms>(xt, tf[kp], U[i]);
          }
          if (CAREFUL) continue;
          stage4<C, kTerms, kPitchV>(Wl, tok, 16 * w.vb(i) + 4 * g, U[i] * wt);
          if (WHAT == kKeep) buf_store16(__builtin_bit_cast(u32x4, U[i]), make_rsrc(a.u + sh * C * a.dv, (uint32_t)(C * a.dv * 4)), uat.at[i]);
          if (WHAT == kOutputs) stage4<C, kTerms, kPitchV>(Ul + (c & 1) * kU, tok, 16 * w.vb(i) + 4 * g, U[i]);
        }
        if constexpr (CAREFUL) {
          float* const Uf = reinterpret_cast<float*>(Wl);   // [C][16 NV], until W is staged
          const float* gates = a.gates + sh * kGateRows * C;
#pragma unroll
          for (int i = 0; i < Sh::kV; ++i) {
            if (w.vb(i) >= NV) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (U[i][r] * 0.f != 0.f && X[i][r] * 0.f == 0.f) again = 1;
          }
          __syncthreads();
          if (uniform(again) && wave == 0) updates_by_token<C, KB, NV, NX, kPitchV>(gates, Kl, Xl, Uf, min(C, u.len - c * C), lane);
          __syncthreads();
#pragma unroll
          for (int i = 0; i < Sh::kV; ++i) {
            if (w.vb(i) >= NV) continue;
            const f32x4 by_token = *reinterpret_cast<const f32x4*>(Uf + tok * 16 * NV + 16 * w.vb(i) + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (uniform(again) && tok < u.len - c * C && U[i][r] * 0.f != 0.f && X[i][r] * 0.f == 0.f) U[i][r] = by_token[r];
          }
          __syncthreads();
          if (tid == 0) again = 0;
#pragma unroll
          for (int i = 0; i < Sh::kV; ++i) {
            if (w.vb(i) >= NV) continue;
            stage4<C, kTerms, kPitchV>(Wl, tok, 16 * w.vb(i) + 4 * g, U[i] * wt);
            stage4<C, kTerms, kPitchV>(Ul + (c & 1) * kU, tok, 16 * w.vb(i) + 4 * g, U[i]);
          }
        }
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);   // while the state is updated, and not before the barrier
        next();
        load_t(min(c + 2, last));
        load_gates(min(c + 2, last));
        __syncthreads();
      }
    } else {
      const KeyPieces<KB> qat(tok, g, a.q_row, a.dk, kEsz);
      const ValuePieces<C, KB, NV> oat(w, tok, g, u.dv0, (long)a.H * a.dv, a.dv, kEsz);
      const StatePieces<C, KB, NV> pieces(a, u, w, c16, g);
      State<C, KB, NV> S;
      read_state<C, KB, NV>(a, u, w, c16, g, S);
      stage_state<C, KB, NV>(Sl, w, c16, g, S);
      Raw8<NX> qr[KEEP ? 1 : KB];
      Scores<NX> pr[KEEP ? 1 : kKp];
      f32x4 O[Sh::kV];
      float eg = 0.f, keep = 0.f;
      auto load_q = [&](int c) {
        const float* gates = a.gates + (sh0 + (long)c * a.H) * kGateRows * C;
        eg = gates[tok];
        const rsrc_t rq = rows(a.q, c, a.q_row, (long)hk * a.dk);
#pragma unroll
        for (int b = 0; b < (KEEP ? 0 : KB); ++b) qr[b] = load8<NX>(rq, qat.at[b]);
      };
      auto load_keep = [&](int c) { keep = a.gates[((sh0 + (long)c * a.H) * kGateRows + 5) * C]; };
      // O += P U of a chunk: while the token waves make U of the next.
      auto finish = [&](int c) {
        const rsrc_t ro = rows(a.o, c, (long)a.H * a.dv, (long)u.h * a.dv);
#pragma unroll
        for (int i = 0; i < Sh::kV; ++i) {
          if (w.vb(i) >= NV) continue;
          const f32x4 own = O[i];
#pragma unroll
          for (int kp = 0; kp < kKp; ++kp) {
            if (kp > w.tb / 2) continue;
            u32x4 ut[kTerms], pt[kTerms];
            values_operand<C, kTerms, kPitchV>(Ul + (c & 1) * kU, kp, 16 * w.vb(i), lane, ut);
            terms8<kTerms>(pr[kp], pt);
            O[i] = mma<kTerms, kTerms, kTerms>(ut, pt, O[i]);
          }
          if (CAREFUL && __any(not_finite(O[i]))) {
            const ScoresIn<NX>* p = static_cast<const ScoresIn<NX>*>(a.pf);
            p += scores_at<C>(p, sh0 + (long)c * a.H);
            O[i] = sum_so_far<C, kPitchV>(O[i], own, p, Ul + (c & 1) * kU, tok, 16 * w.vb(i) + 4 * g);
          }
          store4<NX>(O[i], ro, oat.at[i]);
        }
      };
      if (last >= 0) {
        load_keep(0);
        if (!KEEP) load_q(0);
      }
      if (!KEEP && !CAREFUL && tid == kThreads / 2) lost = again = 0;
      loads_done();
      __syncthreads();
      for (int c = 0; c <= last; ++c) {
        const int ahead = min(c + 1, last);
        f32x4 Q[Sh::kV];
        if (WHAT == kKeep) pieces.store(a.states + (sh0 + (long)c * a.H) * mat, S);
        if constexpr (!KEEP) {   // scale e^G (Q S^T)
          u32x4 qt[KB][NX];
#pragma unroll
          for (int b = 0; b < KB; ++b) terms8<NX>(qr[b], qt[b]);
#pragma unroll
          for (int i = 0; i < Sh::kV; ++i)
            if (w.vb(i) < NV) Q[i] = state_times<KB, NV, NX, kTerms>(Sl, w.vb(i), qt, lane) * (eg * a.scale);
          load_q(ahead);
        }
        __syncthreads();
        if constexpr (!KEEP) {
          if (c > 0) finish(c - 1);
          load_operands<C>(static_cast<const ScoresIn<NX>*>(a.pf), sh0 + (long)c * a.H, w.tb, 0, w.tb / 2, lane, pr);
#pragma unroll
          for (int i = 0; i < Sh::kV; ++i) O[i] = Q[i];
        }
        scale_state<C, KB, NV>(S, keep);
        load_keep(ahead);
        if constexpr (CAREFUL) {   // the token waves' three
          __syncthreads();
          __syncthreads();
          __syncthreads();
        }
        __syncthreads();
        // S = e^(G_C) S + (e^(G_C - G) U)^T K.
#pragma unroll
        for (int kp = 0; kp < kKp; ++kp) state_update<C, KB, NV, NX>(Kl, Wl, w, kp, lane, S);
        stage_state<C, KB, NV>(Sl, w, c16, g, S);
        __syncthreads();
      }
      if (!KEEP && last >= 0) finish(last);
      if (u.to) pieces.store(u.to, S);
      if (!KEEP && !CAREFUL) {
#pragma unroll
        for (int i = 0; i < w.kB; ++i)
#pragma unroll
          for (int j = 0; j < w.kS; ++j)
            if (not_finite(S[i][j])) lost = 1;
      }
    }
    return true;
  };
  const bool walked = walk(std::false_type{}, args);
  if constexpr (!KEEP) {
    if (!walked) return;
    __syncthreads();
    if (uniform(lost)) {
      auto anew = __builtin_amdgcn_kernarg_segment_ptr();   // the arguments too
      asm volatile("" : "+s"(anew));
      walk(std::true_type{}, *(const DeltaArgs*)anew);
    }
  }
}

// The adjoint, from the last chunk to the first: U', dV, the gradients of the states before the chunks. What the
// state waves make ahead of the token waves: dO's terms of the state, (e^G dO)^T Q, while these make Y, and P^T dO
// of the next chunk while they make U'.
// OWN: of a segment, its own gradient of the state before it alone.
template <int C, int KB, int NV, int NX, bool OWN>
__global__ __launch_bounds__(kThreads, 2) void delta_rev_kernel(DeltaArgs a) {
  using Sh = Share<C, KB, NV>;
  constexpr int kEsz = NX == 1 ? 2 : 4, kKp = C / 32;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = value_pitch(NV), kPitchD = 16 * NV + 4;
  __shared__ __align__(16) uint16_t Ll[kTerms * 16 * NV * kPitchK];
  __shared__ __align__(16) uint16_t Kl[NX * C * kPitchK], Ql[NX * C * kPitchK];
  __shared__ __align__(16) uint16_t Ol[NX * C * kPitchV];                                  // dO of the next chunk
  __shared__ __align__(16) uint16_t Gl[kTerms * C * kPitchV], Yl[kTerms * C * kPitchV];    // scale e^G dO; Y
  __shared__ __align__(16) uint16_t Xl[kTerms * C * kPitchV];                              // -e^G beta U'
  __shared__ __align__(16) float Dl[C * kPitchD];                                          // P^T dO
  const int wave = uniform(threadIdx.x >> 6);
  const Sh w(wave & 3);
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const Unit u = delta_unit<C, NV, OWN, true>(a, blockIdx.x, a.dfin, a.dinit);
  if (u.none) return;
  const int hk = u.h / (a.H / a.Hk), tok = 16 * w.tb + c16, last = u.chunks - 1;
  const long mat = (long)a.dk * a.dv, sh0 = u.slot0 * a.H + u.h;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto rows = [&](const void* x, int c, long row, long col) {
    return chunk_rows(x, u.start + (long)c * C, row, col, min(C, u.len - c * C), kEsz);
  };

  if (wave < 4) {
    const KeyPieces<KB> kat(tok, g, a.k_row, a.dk, kEsz);
    const ValuePieces<C, KB, NV> vat(w, tok, g, u.dv0, (long)a.H * a.dv, a.dv, kEsz), uat(w, tok, g, u.dv0, a.dv, a.dv, 4);
    Raw8<NX> kr[KB];
    u32x4 tt[kKp][kTerms];
    RawOperand tn[kKp];   // of the next chunk
    float eg, wt, be, eg_next, wt_next, be_next;
    auto load_rows = [&](int c) {
      const rsrc_t rk = rows(a.k, c, a.k_row, (long)hk * a.dk);
#pragma unroll
      for (int b = 0; b < KB; ++b) kr[b] = load8<NX>(rk, kat.at[b]);
    };
    auto load_gates = [&](int c) {
      const float* gates = a.gates + (sh0 + (long)c * a.H) * kGateRows * C;
      eg_next = gates[tok];
      wt_next = gates[C + tok];
      be_next = gates[2 * C + tok];
    };
    auto next = [&]() {
      eg = eg_next;
      wt = wt_next;
      be = be_next;
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) terms8<kTerms>(tn[kp], tt[kp]);
    };
    auto load_t = [&](int c) { load_operands<C>(a.tt, sh0 + (long)c * a.H, w.tb, w.tb / 2, kKp - 1, lane, tn); };
    if (last >= 0) {
      load_rows(last);
      load_gates(last);
      load_t(last);
      next();
      load_t(max(last - 1, 0));
      load_gates(max(last - 1, 0));
    }
    loads_done();
    __syncthreads();
    __syncthreads();
    for (int c = last; c >= 0; --c) {
      const long sh = sh0 + (long)c * a.H;
      // Y = e^(G_C - G) (K L^T) + P^T dO.
      f32x4 Y[Sh::kV];
      u32x4 kt[KB][NX];
#pragma unroll
      for (int b = 0; b < KB; ++b) terms8<NX>(kr[b], kt[b]);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
        const int col = 16 * w.vb(i) + 4 * g;
        const f32x4 d = *reinterpret_cast<const f32x4*>(Dl + tok * kPitchD + col);
        Y[i] = state_times<KB, NV, NX, kTerms>(Ll, w.vb(i), kt, lane);
#pragma unroll
        for (int r = 0; r < 4; ++r) Y[i][r] = fmaf(wt, Y[i][r], d[r]);
        stage4<C, kTerms, kPitchV>(Yl, tok, col, Y[i]);
      }
#pragma unroll
      for (int b = 0; b < KB; ++b) stage_rows<C, KB, NV, NX>(Kl, w, c16, g, b, kt[b]);
      load_rows(max(c - 1, 0));
      __syncthreads();

      // U' = T^T Y, dV = beta U'.
      f32x4 U[Sh::kV];
      const rsrc_t rv = rows(a.dv_out, c, (long)a.H * a.dv, (long)u.h * a.dv);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
        U[i] = zero;
#pragma unroll
        for (int kp = 0; kp < kKp; ++kp) {
          if (kp < w.tb / 2) continue;
          u32x4 yt[kTerms];
          values_operand<C, kTerms, kPitchV>(Yl, kp, 16 * w.vb(i), lane, yt);
          U[i] = mma<kTerms, kTerms, kTerms>(yt, tt[kp], U[i]);
        }
        stage4<C, kTerms, kPitchV>(Xl, tok, 16 * w.vb(i) + 4 * g, U[i] * (-eg * be));
        if (OWN) continue;
        buf_store16(__builtin_bit_cast(u32x4, U[i]), make_rsrc(a.ub + sh * C * a.dv, (uint32_t)(C * a.dv * 4)), uat.at[i]);
        store4<NX>(U[i] * be, rv, vat.at[i]);
      }
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);   // while the state is updated, and not before the barrier
      next();
      load_t(max(c - 2, 0));
      load_gates(max(c - 2, 0));
      __syncthreads();
    }
  } else {
    const KeyPieces<KB> qat(tok, g, a.q_row, a.dk, kEsz);
    const ValuePieces<C, KB, NV> oat(w, tok, g, u.dv0, (long)a.H * a.dv, a.dv, kEsz);
    const StatePieces<C, KB, NV> pieces(a, u, w, c16, g);
    State<C, KB, NV> L;
    read_state<C, KB, NV>(a, u, w, c16, g, L);
    stage_state<C, KB, NV>(Ll, w, c16, g, L);
    Raw8<NX> qr[KB];
    Raw4<NX> d1[Sh::kV], d2[Sh::kV];   // dO of the chunk before the present one, and of the one before that
    RawOperand pr[kKp];
    float eg1 = 0.f, eg2 = 0.f, keep = 0.f;
    auto load_do = [&](int c, Raw4<NX>* to, float& eg) {
      const rsrc_t ro = rows(a.d_o, c, (long)a.H * a.dv, (long)u.h * a.dv);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) to[i] = load4<NX>(ro, oat.at[i]);
      eg = a.gates[(sh0 + (long)c * a.H) * kGateRows * C + tok];
    };
    auto load_q = [&](int c) {
      const rsrc_t rq = rows(a.q, c, a.q_row, (long)hk * a.dk);
#pragma unroll
      for (int b = 0; b < KB; ++b) qr[b] = load8<NX>(rq, qat.at[b]);
    };
    auto load_p = [&](int c) { load_operands<C>(a.pt, sh0 + (long)c * a.H, w.tb, w.tb / 2, kKp - 1, lane, pr); };
    auto load_keep = [&](int c) { keep = a.gates[((sh0 + (long)c * a.H) * kGateRows + 5) * C]; };
    auto stage_q = [&]() {
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        u32x4 qt[NX];
        terms8<NX>(qr[b], qt);
        stage_rows<C, KB, NV, NX>(Ql, w, c16, g, b, qt);
      }
    };
    auto stage_g = [&](const Raw4<NX>* x, float eg) {
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i)
        if (w.vb(i) < NV) stage4<C, kTerms, kPitchV>(Gl, tok, 16 * w.vb(i) + 4 * g, floats4<NX>(x[i]) * (eg * a.scale));
    };
    auto stage_o = [&](const Raw4<NX>* x) {
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i)
        if (w.vb(i) < NV) stage4<C, NX, kPitchV>(Ol, tok, 16 * w.vb(i) + 4 * g, floats4<NX>(x[i]));
    };
    auto scores = [&]() {   // P^T dO of the chunk whose dO is staged
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) {
        if (w.vb(i) >= NV) continue;
        f32x4 D = zero;
#pragma unroll
        for (int kp = 0; kp < kKp; ++kp) {
          if (kp < w.tb / 2) continue;
          u32x4 ot[NX], pt[kTerms];
          values_operand<C, NX, kPitchV>(Ol, kp, 16 * w.vb(i), lane, ot);
          terms8<kTerms>(pr[kp], pt);
          D = mma<NX, kTerms, kTerms>(ot, pt, D);
        }
        *reinterpret_cast<f32x4*>(Dl + tok * kPitchD + 16 * w.vb(i) + 4 * g) = D;
      }
    };
    if (last >= 0) {
      load_do(last, d1, eg1);
      load_q(last);
      load_p(last);
      load_keep(last);
      stage_q();
      stage_g(d1, eg1);
      stage_o(d1);
    }
    __syncthreads();
    if (last >= 0) {
      scores();
      load_do(max(last - 1, 0), d1, eg1);
      load_do(max(last - 2, 0), d2, eg2);
      load_q(max(last - 1, 0));
      load_p(max(last - 1, 0));
    }
    loads_done();
    __syncthreads();
    if (last >= 0) stage_o(d1);
    for (int c = last; c >= 0; --c) {
      if (!OWN) pieces.store(a.dstates + (sh0 + (long)c * a.H) * mat, L);
      // L = e^(G_C) L + scale (e^G dO)^T Q - (e^G beta U')^T K, the last term when U' is there.
      scale_state<C, KB, NV>(L, keep);
      load_keep(max(c - 1, 0));
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) state_update<C, KB, NV, NX>(Ql, Gl, w, kp, lane, L);
      __syncthreads();
      scores();
      load_p(max(c - 2, 0));
      __syncthreads();
#pragma unroll
      for (int kp = 0; kp < kKp; ++kp) state_update<C, KB, NV, NX>(Kl, Xl, w, kp, lane, L);
      stage_state<C, KB, NV>(Ll, w, c16, g, L);
      stage_q();
      load_q(max(c - 2, 0));
      stage_g(d1, eg1);
      stage_o(d2);
#pragma unroll
      for (int i = 0; i < Sh::kV; ++i) d1[i] = d2[i];
      eg1 = eg2;
      load_do(max(c - 3, 0), d2, eg2);
      __syncthreads();
    }
    if (u.to) pieces.store(u.to, L);
  }
}

// The states behind the segments of a sequence, one after the other: R := R M + own (REV: the gradients of the states
// before them, from the last to the first, R := R M^T + own), of 16 rows of one head, in fp32
// (matrix instructions on fp32). A wave makes 16 of the key columns; R goes round through LDS, and the next segment's
// map is on its way while this one's is taken.
template <int KB, bool REV>
__global__ __launch_bounds__(128 * KB) void delta_join_kernel(DeltaArgs a, int C) {
  constexpr int kBlocks = 2 * KB;   // waves
  __shared__ __align__(16) f32x4 Rl[kBlocks * 64];   // blocks of 16 key columns as accumulators hold them
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int tiles = (a.dv + 15) / 16, tile = (int)(blockIdx.x % tiles), h = (int)((blockIdx.x / tiles) % a.H);
  const long seq = blockIdx.x / ((long)tiles * a.H), mat = (long)a.dk * a.dv, map = (long)a.dk * a.dk;
  const int L = a.seg * C;
  long n0, len;
  if (a.cu) {
    const int c0 = min(max(a.cu[seq], 0), a.T);
    len = min(max(a.cu[seq + 1], c0), a.T) - c0;
    n0 = (long)c0 / L + seq;
  } else {
    len = a.T;
    n0 = seq * a.segs_per_row;
  }
  const int segs = (int)((len + L - 1) / L), dv = 16 * tile + c16;
  if (segs < 3) return;   // the state behind the first segment is its own
  f32x4 R, own, M[kBlocks];   // M: rows 16 k + 4 g + t of the map, column c16 of this wave's block; REV: of its transpose
  const int dk = 16 * wave + 4 * g, col = 16 * wave + c16;
  const uint32_t at = dv < a.dv && dk < a.dk ? (uint32_t)((dv * a.dk + dk) * 4) : kOffNone;
  const uint32_t mat0 = col >= a.dk ? kOffNone : REV ? (uint32_t)(col * a.dk * 4) : (uint32_t)((4 * g * a.dk + col) * 4);
  float* const states = REV ? a.seg_adj : a.seg_states;
  auto state = [&](int s) { return make_rsrc(states + ((n0 + s) * a.H + h) * mat, (uint32_t)(mat * 4)); };
  auto load = [&](int s) {
    const rsrc_t rm = make_rsrc(a.seg_maps + ((n0 + s) * a.H + h) * map, (uint32_t)(map * 4));
    own = __builtin_bit_cast(f32x4, buf_load16(state(s), at));
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      if constexpr (REV) {
        M[k] = __builtin_bit_cast(f32x4, buf_load16(rm, 16 * k + 4 * g < a.dk ? mat0 + (uint32_t)((16 * k + 4 * g) * 4) : kOffNone));
      } else {   // rows behind the map lie behind its end
#pragma unroll
        for (int t = 0; t < 4; ++t) M[k][t] = buf_load_f32(rm, mat0 + (uint32_t)((16 * k + t) * a.dk * 4));
      }
    }
  };
  const int first = REV ? segs - 1 : 0, step = REV ? -1 : 1, middle = segs - 2;   // segments between the first and the last
  R = __builtin_bit_cast(f32x4, buf_load16(state(first), at));
  load(first + step);
  loads_done();
  for (int i = 1; i <= middle; ++i) {
    const int s = first + step * i;
    Rl[wave * 64 + lane] = R;
    __syncthreads();
    f32x4 x[2] = {own, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      const f32x4 r = Rl[k * 64 + lane];
#pragma unroll
      for (int t = 0; t < 4; ++t) x[k & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(M[k][t], r[t], x[k & 1], 0, 0, 0);
    }
    R = x[0] + x[1];
    buf_store16(__builtin_bit_cast(u32x4, R), state(s), at);
    load(first + step * min(i + 1, middle));
    __syncthreads();
  }
}

// Value blocks a workgroup. Two, which read a chunk's rows and operands once, where workgroups of one would be more
// than the CUs; else one. Prompts, us with one and with two (the workgroups of one): heads of 128 x 128, 2 x 4096 tokens of
// 32 (512) 269 and 243, 4096 of 40 (320) 227 and 205, 2 x 2048 of 17 (272) 128 and 119, 4096 of 32 (256) 141 and 208; heads
// of 64 x 64 gain nothing (8 x 1024 of 16 (512) 66 and 67, with gradients 254 and 241). Packed sequences take one: what
// counts there is the longest, which two make longer: 8 of 5117 tokens, 16 heads of 64 x 96 (768) 110 and 123, 32 heads
// (1536) 125 and 144, 8 of 7996, 16 of 128 x 128 (1024) 187 and 241, 64 of 7652, 8 heads (4096) 119 and 127 (sequences that are
// equally long, which the host cannot know, would gain: 8 of 1024, 16 heads of 128 x 128, 161 and 150). fp32: two; with
// keys of 256, whose rows leave LDS for one, one. Walks that are cut fill the card as they are: one (bf16).
constexpr int nv32(int kb) { return kb > 4 ? 1 : 2; }
int value_blocks(const DeltaArgs& a) {
  if (!a.bf16) return nv32((a.dk + 31) / 32);
  if (a.seg || a.S > 0) return 1;
  return (long)a.batch * a.H * ((a.dv + 15) / 16) > 256 && a.dk <= 128 ? 2 : 1;
}

template <int KB, int WHAT>
void walk(const DeltaArgs& a, long blocks, hipStream_t stream) {
  const dim3 grid((unsigned)blocks);
  if constexpr (KB <= 4 && WHAT != kOwn) {
    if (a.bf16 && value_blocks(a) == 2) {
      hipLaunchKernelGGL((delta_fwd_kernel<64, KB, 2, 1, WHAT>), grid, dim3(kThreads), 0, stream, a);
      return;
    }
  }
  if (a.bf16) hipLaunchKernelGGL((delta_fwd_kernel<64, KB, 1, 1, WHAT>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((delta_fwd_kernel<32, KB, nv32(KB), 3, WHAT>), grid, dim3(kThreads), 0, stream, a);
}
template <int KB, bool REV>
void join(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((long)(a.S > 0 ? a.S : a.batch) * a.H * ((a.dv + 15) / 16)));
  hipLaunchKernelGGL((delta_join_kernel<KB, REV>), grid, dim3(128 * KB), 0, stream, a, delta_chunk(a.bf16));
}
template <int KB>
void fwd(const DeltaArgs& a, bool keep, hipStream_t stream) {
  if (a.seg) {
    walk<KB, kOwn>(a, delta_segment_blocks(a), stream);
    join<KB, false>(a, stream);
  }
  if (keep) walk<KB, kKeep>(a, delta_chain_blocks(a), stream);
  else walk<KB, kOutputs>(a, delta_chain_blocks(a), stream);
}
template <int KB, bool OWN>
void walk_back(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)delta_chain_blocks(a));
  if constexpr (KB <= 4 && !OWN) {
    if (a.bf16 && value_blocks(a) == 2) {
      hipLaunchKernelGGL((delta_rev_kernel<64, KB, 2, 1, OWN>), grid, dim3(kThreads), 0, stream, a);
      return;
    }
  }
  if (a.bf16) hipLaunchKernelGGL((delta_rev_kernel<64, KB, 1, 1, OWN>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((delta_rev_kernel<32, KB, nv32(KB), 3, OWN>), grid, dim3(kThreads), 0, stream, a);
}
template <int KB>
void rev(const DeltaArgs& a, hipStream_t stream) {   // the maps are those of the forward walk
  if (a.seg) {
    walk_back<KB, true>(a, stream);
    join<KB, true>(a, stream);
  }
  walk_back<KB, false>(a, stream);
}

}  // namespace

static int tiles_of(int d, int blocks) { return (d + 16 * blocks - 1) / (16 * blocks); }
long delta_chain_blocks(const DeltaArgs& a) {
  return (a.seg ? a.segs : (long)(a.S > 0 ? a.S : a.batch)) * a.H * tiles_of(a.dv, value_blocks(a));
}
long delta_segment_blocks(const DeltaArgs& a) {
  return a.segs * a.H * (tiles_of(a.dv, value_blocks(a)) + tiles_of(a.dk, value_blocks(a)));
}

// A walk of few heads leaves most of the card idle for as long as its longest sequence is. Cut into segments, every
// segment's own last state (from a state of zero) and its map of a state are made at once, the states behind the
// segments follow from these one after the other, and all segments are walked at once: twice to three times the
// work, in chains of a segment's length (8192 tokens, 4 heads of 128 x 128: 220 us whole, 93 in eight segments). The
// backward walk is cut alike, its maps the forward's transposed (both with the gradients 462 us whole, 240 cut; 8 heads
// of 4096 tokens 272 and 218; fp32, 2048 tokens of 4 heads of 64 x 128, 249 and 114). The
// number of segments is the one of least cost, counted in steps of a chunk: a walk takes as long as its longest chain,
// or as its steps shared out over 256 CUs, one at a time (workgroups on one CU do not overlap by more than a tenth);
// a step without O 0.8 of one with it; a segment's join about one step, the two launches five. The host does not
// know the lengths of packed sequences: the longest is taken to be three times the mean. (Eight ragged sequences of
// 5087 tokens, 16 heads of 64 x 96: 99 us whole, 110 in segments of nine chunks.)
int delta_segment(int batch, int T, int S, int H, int dk, int dv, bool bf16) {
  const int C = delta_chunk(bf16);
  const long seqs = S > 0 ? S : batch, tokens = (long)batch * T;
  const long longest = S > 0 ? std::min((long)T, 3 * ((tokens + S - 1) / S)) : T;
  const long chunks = (longest + C - 1) / C, all = (tokens + C - 1) / C;
  const int blocks = bf16 ? 1 : nv32((dk + 31) / 32), values = tiles_of(dv, blocks), rows = values + tiles_of(dk, blocks);
  auto steps = [](double chain, double work) { return std::max(chain, work / 256); };
  const double outputs = (double)all * H * values;
  double least = 0.9 * steps((double)chunks, outputs);
  int best = 0;
  for (long n = 2; n <= 64 && n <= chunks; ++n) {
    const long c = (chunks + n - 1) / n;
    const double own = std::max((double)all - (double)seqs * c, 0.0) * H * rows;   // not of the last segments
    const double cost = 0.8 * steps((double)c, own) + (double)n + 5.0 + steps((double)c, outputs);
    if (cost < least) {
      least = cost;
      best = (int)c;
    }
  }
  return best;
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
