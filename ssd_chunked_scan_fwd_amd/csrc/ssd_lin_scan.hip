// ssd_lin_scan.hip -- linear attention with one decay a head over prompts, on
// bf16 matrix instructions (v_mfma_f32_16x16x32_bf16).
//
// Chunks of C = 64 tokens of one (block, head). With D the state [dv][dk]
// before the chunk and i, j its tokens (lam^(i-j) masked to i >= j):
//     O  = (lam^(i-j) o Q K^T) V + lam^(i+1) Q D^T
//     D' = lam^C D + (lam^(C-1-j) V)^T K.
// Wave w owns 16 value columns of D, in the fp32 accumulators of its own
// products, over the whole chunk loop:
//   scores  S^T = K Q^T, 16 queries by 32 keys a task, weighted and left in LDS as bf16;
//   inter   O^T = D Q^T: the accumulators of two blocks of dk, rounded to bf16,
//           are the operand as they stand (their k order is that of an
//           accumulator pair; Q's columns lie in LDS in that order);
//   intra   O^T += V^T P^T;
//   state   D^T += K^T (lam^(C-1-j) V), the weighted V as the sum of two bf16
//           values: the state is carried on, and one bf16 rounding of each term
//           would weigh as much as that of the state itself as an operand. Of
//           three where the last state is asked for, an fp32 result: its error
//           is then that of 32-bit sums.
// Roundings to bf16: the weighted scores (of a sequence's first 32 tokens as the
// sum of two, store_scores) and the state as operands, and O.
//
// A chunk moves C (2 dk + 2 dv) 2 bytes, reads of k and v by the blocks' own sums
// apart, and makes 2 C (C + 3 dk) dv multiplies (the doubled state product
// included). The next chunk's rows are in flight in registers while this one is
// computed. T = 16384, 32 heads of 128 x 128, 16 blocks a head: 200 - 213 us a call.
// Under the trace, which lengthens them, means of 19 and the least: own sums 70 us
// and 58 for 283 MB (4.1 and 4.9 TB/s; a copy reaches 4.9), entering states 13.5,
// this scan 149 and 125 for 571 MB (3.8 and 4.6 TB/s). Memory bounds the sums, and
// with the chain scores - barrier - outputs - state of each chunk (four waves a
// SIMD, all that registers allow) the scan: without its loads it took 106 us, with
// matrix pipes busy a third of the time and LDS 40 %. Heads of 256 x 256 (T 4096, 16
// heads) leave one workgroup a CU: 104 - 114 us for 138 MB.
#include <type_traits>

#include "ssd_lin_chunk.h"

namespace ssd {

namespace {

// What a workgroup takes: 128 or 64 value columns (DV) of one head's block.
struct LinUnit {
  int dv0, h, pos0, total;   // first column, head, the block's first token and tokens in the sequence
  long slot;
  bool last;                 // of the sequence
  LinPiece p;                // p.blk < 0: nothing
};
template <int DV>
__device__ __forceinline__ LinUnit lin_unit(const LinScan& a, long bid, long blocks) {
  LinUnit w;
  const int tiles = (a.dv + DV - 1) / DV;
  const long u = xcd_unit(bid, blocks);
  w.dv0 = (int)(u % tiles) * DV;
  w.h = (int)((u / tiles) % a.H);
  w.slot = u / ((long)tiles * a.H);
  w.p = lin_piece(a, w.slot);
  w.pos0 = w.p.blk * a.L;
  w.total = min(w.p.len - w.pos0, a.L);
  w.last = w.pos0 + w.total >= w.p.len;
  return w;
}

// The state that enters the block: S[b] holds D[dvc][dk] at dk = 16 b + 4 g + r.
template <int KB, bool STATE_ONLY>
__device__ __forceinline__ void enter_state(const LinScan& a, const LinUnit& w, int dvc, int g, f32x4 (&S)[2 * KB]) {
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b) S[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (STATE_ONLY) return;
  const long mat = (long)a.dv * a.dk;
  const float* src = w.p.blk > 0 ? a.states + (w.slot * a.H + w.h) * mat : a.init;
  if (w.p.blk == 0 && src) src += ((long)w.p.seq * a.H + w.h) * mat;
  const bool tr = w.p.blk == 0 && a.init_tr;
  const float sc = w.p.blk == 0 ? a.init_scale : 1.f;
  if (!src || dvc >= a.dv) return;
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b) {
    const int dk = 16 * b + 4 * g;
    if (dk >= a.dk) continue;
    if (tr) {
#pragma unroll
      for (int r = 0; r < 4; ++r) S[b][r] = sc * src[(long)(dk + r) * a.dv + dvc];
    } else {
      S[b] = *reinterpret_cast<const f32x4*>(src + (long)dvc * a.dk + dk) * sc;
    }
  }
}

// The state that leaves it, where it is wanted: the block's own sum or the last state.
template <int KB, bool STATE_ONLY>
__device__ __forceinline__ void leave_state(const LinScan& a, const LinUnit& w, int dvc, int g, const f32x4 (&S)[2 * KB],
                                            const float* pw) {
  const long mat = (long)a.dv * a.dk;
  float* dst = nullptr;
  float sc = 1.f;
  if (STATE_ONLY) {
    dst = a.states + (w.slot * a.H + w.h) * mat;
  } else if (w.last && a.fin) {
    dst = a.fin + ((long)w.p.seq * a.H + w.h) * mat;
    sc = a.fin_scale * (a.rev && w.p.len > 0 ? pw[kPowZero + 1] : 1.f);
  }
  if (!dst || dvc >= a.dv) return;
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b) {
    const int dk = 16 * b + 4 * g;
    if (dk < a.dk) *reinterpret_cast<f32x4*>(dst + (long)dvc * a.dk + dk) = S[b] * sc;
  }
}

// What a wave needs to find its block again. It lies in LDS, and the arguments
// are read from where the launch put them: kept at hand through the loop of the
// matrix form they take scalar registers that cost it up to 6 % (heads of 256).
struct LinAgain {
  const LinScan* args;
  int bid, blocks;
};
__device__ __forceinline__ void remember(LinAgain* to, int which, long bid, long blocks) {
  static_assert(sizeof(LinScan) % 8 == 0, "scans lie one behind the other from the first argument on");
  if (threadIdx.x == 0) *to = LinAgain{(const LinScan*)__builtin_amdgcn_kernarg_segment_ptr() + which, (int)bid, (int)blocks};
}

// A wave's columns of a block by the recurrence itself, token by token in fp32.
// In a matrix product a masked score (0) times an infinity or NaN of v is a NaN in
// the output of an earlier token, and the bf16 terms of an infinity are that
// infinity and a NaN; here a value meets only what it belongs to. Some 1.1 us a
// token, the way from one state to the next with the next rows in flight: a NaN in
// 16384 tokens of 32 heads of 128 x 128, 16 blocks a head, makes 0.2 ms 2.3.
template <int KB, int W, bool STATE_ONLY>
__device__ __forceinline__ void lin_by_token(const LinAgain* again, const float* pw) {
  int tid = threadIdx.x;
  asm volatile("s_waitcnt vmcnt(0)" : "+v"(tid) : : "memory");   // the outputs of the first time are written
  const LinScan& a = *uniform(again->args);
  const int bid = uniform(again->bid), blocks = uniform(again->blocks);
  const LinUnit u = lin_unit<16 * W>(a, bid, blocks);
  const int g = (tid & 63) >> 4, dvc = u.dv0 + 16 * (tid >> 6) + (tid & 15);
  f32x4 S[2 * KB];
  enter_state<KB, STATE_ONLY>(a, u, dvc, g, S);
  const float lam_hi = pw[kPowHi], lam_lo = pw[kPowHi + 1];
  const int end = a.dk - 4 * g, dv = a.dv, rev = a.rev, o_f32 = a.o_f32;
  const bool in = dvc < dv;
  const long krow = a.k.row, qrow = a.q.row, vrow = a.v.row, orow = (long)a.H * dv;
  const uint16_t* k0 = static_cast<const uint16_t*>(a.k.base) + (long)(u.h / a.k.div) * a.dk + 4 * g;
  const uint16_t* q0 = static_cast<const uint16_t*>(a.q.base) + (long)(u.h / a.q.div) * a.dk + 4 * g;
  const uint16_t* v0 = static_cast<const uint16_t*>(a.v.base) + (long)(u.h / a.v.div) * dv + (in ? dvc : 0);
  const long o0 = (long)u.h * dv + dvc;
  void* const out = a.o;
  const float scale = a.scale;
  u32x2 k[2 * KB], q[2 * KB];   // the next token's rows
  uint16_t v = 0;
  auto token = [&](int j) { return u.p.start + (rev ? u.p.len - 1 - (u.pos0 + j) : u.pos0 + j); };
  auto load = [&](int j) {
    const long tok = token(min(j, u.total - 1));
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      const int col = 16 * b < end ? 16 * b : -4 * g;   // behind the end: the head's first (with dk = 8 all that g >= 2 has)
      k[b] = *reinterpret_cast<const u32x2*>(k0 + tok * krow + col);
      if (!STATE_ONLY) q[b] = *reinterpret_cast<const u32x2*>(q0 + tok * qrow + col);
    }
    v = v0[tok * vrow];
  };
  load(0);
#pragma unroll 1
  for (int j = 0; j < u.total; ++j) {
    const bool keep = rev && u.pos0 + j == 0;   // the state handed to a reversed scan is not decayed first
    const float hi = keep ? kOneHi : lam_hi, lo = keep ? kOneLo : lam_lo, x = bf16_to_f32(v);
    float part = 0.f;
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      const f32x4 kb = four(k[b]), qb = four(STATE_ONLY ? k[b] : q[b]);
      if (16 * b >= end) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        S[b][r] = fmaf(S[b][r], hi, fmaf(S[b][r], lo, x * kb[r]));
        if (!STATE_ONLY) part = fmaf(S[b][r], qb[r], part);
      }
    }
    load(j + 1);
    if (STATE_ONLY) continue;
    part += __shfl_xor(part, 16);
    part = (part + __shfl_xor(part, 32)) * scale;
    const long at = token(j) * orow + o0;
    if (g == 0 && in) {
      if (o_f32) static_cast<float*>(out)[at] = part;
      else static_cast<uint16_t*>(out)[at] = f32_to_bf16(part);
    }
  }
  leave_state<KB, STATE_ONLY>(a, u, dvc, g, S, pw);
}

// KB: dk in units of 32. W waves of 16 value columns. TERMS: bf16 terms of the
// weighted V in the state product. `which` of the launch's scans is a.
template <int KB, int W, int TERMS, bool STATE_ONLY>
__device__ __forceinline__ void lin_mfma(const LinScan& a, int which, long bid, long blocks) {
  constexpr int kDk = 32 * KB, kDv = 16 * W, kThreads = 64 * W;
  constexpr int kPitchK = lds_pitch(kDk), kPitchV = lds_pitch(kDv);
  __shared__ __align__(16) uint16_t Ks[kC * kPitchK];
  __shared__ __align__(16) uint16_t Vs[kC * kPitchV];
  __shared__ __align__(16) uint16_t Qs[STATE_ONLY ? 8 : kC * kPitchK];
  __shared__ __align__(16) uint16_t Ps[STATE_ONLY ? 8 : kC * kPitchP];
  __shared__ __align__(16) float pw[kPowSize], spw[STATE_ONLY ? 4 : kPowSize];   // powers of lam, and scale times them
  constexpr int kQK = (256 * KB + kThreads - 1) / kThreads;   // 16-byte pieces a thread stages of q and of k,
  constexpr int kV = 2;                                       // and of v

  __shared__ LinAgain again;
  remember(&again, which, bid, blocks);
  const LinUnit u = lin_unit<kDv>(a, bid, blocks);
  if (u.p.blk < 0) return;
  if (STATE_ONLY && u.last) return;  // the scan carries the last block's state itself
  const LinPiece& p = u.p;
  const int dv0 = u.dv0, h = u.h, pos0 = u.pos0, total = u.total;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;

  const int dvc = dv0 + 16 * wave + c16;
  f32x4 S[2 * KB];
  enter_state<KB, STATE_ONLY>(a, u, dvc, g, S);

  constexpr int kTasks = 8 / W;   // score tasks (16 queries by 32 keys) a wave

  fill_powers(pw, STATE_ONLY ? nullptr : spw, a.ld[h], a.scale);

  const int qrow = (int)a.q.row * 2, krow = (int)a.k.row * 2, vrow = (int)a.v.row * 2;  // 64 rows are fewer than 2^31 bytes
  Piece qp[STATE_ONLY ? 1 : kQK], kp_[kQK], vp[kV];
#pragma unroll
  for (int j = 0; j < kQK; ++j) {
    const int i = threadIdx.x + kThreads * j;
    const int r = i / (4 * KB), col = 8 * (i % (4 * KB));
    kp_[j] = make_piece(r, col, a.dk, krow, 2, a.rev);
    if (!STATE_ONLY) qp[j] = make_piece(r, col, a.dk, qrow, 2, a.rev);
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + kThreads * j;
    vp[j] = make_piece(i / (kDv / 8), 8 * (i % (kDv / 8)), a.dv - dv0, vrow, 2, a.rev);
  }
  u32x4 qn[kQK], kn[kQK], vn[kV];
  auto load = [&](int t0) {  // rows of the chunk that starts t0 tokens into the block
    const int n = min(kC, total - t0);
    const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
    auto rows = [&](const LinOperand& x, int d, int col0) {
      const uint16_t* base = static_cast<const uint16_t*>(x.base) + low * x.row + (long)(h / x.div) * d + col0;
      return make_rsrc(base, (uint32_t)(n * x.row * 2));
    };
    const rsrc_t rk = rows(a.k, a.dk, 0), rv = rows(a.v, a.dv, dv0);
#pragma unroll
    for (int j = 0; j < kQK; ++j) kn[j] = buf_load16(rk, piece_offset(kp_[j], n, krow, a.rev));
    if (!STATE_ONLY) {
      const rsrc_t rq = rows(a.q, a.dk, 0);
#pragma unroll
      for (int j = 0; j < kQK; ++j) {
        const uint32_t off = piece_offset(qp[j], n, qrow, a.rev);
        qn[j] = a.q_once ? buf_load16_once(rq, off) : buf_load16(rq, off);
      }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) vn[j] = buf_load16(rv, piece_offset(vp[j], n, vrow, a.rev));
  };

  // This lane's piece of O at token c16; those of the other token blocks lie 16 rows on.
  const Piece o0 = make_piece(c16, dv0 + 16 * wave + 4 * g, a.dv, a.H * a.dv * (a.o_f32 ? 4 : 2), a.o_f32 ? 4 : 2, a.rev);

  // The blocks' own sums walk their chunks backwards, weighting each V by its whole
  // distance to the block's end: the scan, which walks forwards and comes next,
  // finds the rows that were read last in the memory-side cache.
  const int chunks = (total + kC - 1) / kC;
  if (chunks > 0) load(STATE_ONLY ? (chunks - 1) * kC : 0);
  float behind = 1.f;   // STATE_ONLY: lam to the tokens of the block behind the chunk
  for (int ci = 0; ci < chunks; ++ci) {
    const int t0 = (STATE_ONLY ? chunks - 1 - ci : ci) * kC;
    const int n = min(kC, total - t0);
    const bool first = pos0 + t0 == 0;
    const int lead = a.rev && first ? 0 : 1;   // the state handed to a reversed scan is not decayed first
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQK; ++j) {
      const int i = threadIdx.x + kThreads * j;
      const int row = i / (4 * KB), col = i % (4 * KB);
      if (kThreads <= 256 * KB || i < 256 * KB) {
        *reinterpret_cast<u32x4*>(Ks + row * kPitchK + row_shift(row) + 8 * col) = kn[j];
        if (!STATE_ONLY) store_paired(Qs + row * kPitchK, col >> 2, col & 3, qn[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + kThreads * j;
      *reinterpret_cast<u32x4*>(Vs + i / (kDv / 8) * kPitchV + 8 * (i % (kDv / 8))) = vn[j];
    }
    if (ci + 1 < chunks) load(STATE_ONLY ? t0 - kC : t0 + kC);
    __syncthreads();

    if (!STATE_ONLY) {
#pragma unroll
      for (int k = 0; k < kTasks; ++k) {
        const int qb = wave & 3, kp = W == 8 ? wave >> 2 : k;
        if (kp > qb / 2) continue;   // all keys are later; never read
        f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const u32x4 q = frag_k_cols(Qs, kPitchK, 16 * qb, 32 * j, lane);
          s0 = mfma16x16x32(frag_k_cols_pairs(Ks, kPitchK, 32 * kp, 32 * j, lane), q, s0);
          s1 = mfma16x16x32(frag_k_cols_pairs(Ks, kPitchK, 32 * kp + 16, 32 * j, lane), q, s1);
        }
        // Query minus key, of the first key (r = 0); weighted, or 0 (selected: a later key may hold anything).
        const int diff = 16 * qb - 32 * kp + c16 - 4 * g;
        const float* w = spw + kPowZero + diff;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s0[r] = diff >= r ? s0[r] * w[-r] : 0.f;
          s1[r] = diff - 16 >= r ? s1[r] * w[-16 - r] : 0.f;
        }
        store_scores(Ps + (16 * qb + c16) * kPitchP + 32 * kp + 8 * g, s0, s1, first && qb < 2);
      }
    }

    u32x4 vf[2];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) vf[kp] = frag_k_rows_accpair(Vs, kPitchV, 32 * kp, 16 * wave, lane);

    if (!STATE_ONLY) {
      f32x4 O[4];
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) O[qb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const f32x4 x = S[2 * j], y = S[2 * j + 1];
        const u32x4 sf = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
#pragma unroll
        for (int qb = 0; qb < 4; ++qb) O[qb] = mfma16x16x32(sf, frag_k_cols(Qs, kPitchK, 16 * qb, 32 * j, lane), O[qb]);
      }
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) O[qb] *= spw[kPowZero + 16 * qb + c16 + lead];
      __syncthreads();
#pragma unroll
      for (int qb = 0; qb < 4; ++qb)
#pragma unroll
        for (int kp = 0; kp <= qb / 2; ++kp)
          O[qb] = mfma16x16x32(vf[kp], frag_k_cols(Ps, kPitchP, 16 * qb, 32 * kp, lane), O[qb]);
      if (first) {
#pragma unroll
        for (int qb = 0; qb < 2; ++qb) O[qb] = mfma16x16x32(vf[0], frag_k_cols(Ps, kPitchP, 16 * qb, 32, lane), O[qb]);
      }
      // O^T: column c16 is the query, rows 4 g + r the value columns.
      const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
      const int esz = a.o_f32 ? 4 : 2, orow = a.H * a.dv * esz;
      const rsrc_t ro = make_rsrc(static_cast<char*>(a.o) + low * orow + (long)h * a.dv * esz, (uint32_t)(n * orow));
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) {
        const Piece at = {o0.full + (uint32_t)((a.rev ? -16 : 16) * qb * orow), o0.row + 16 * qb};
        const uint32_t off = piece_offset(at, n, orow, a.rev);
        const f32x4 o = O[qb];
        if (a.o_f32) buf_store16(__builtin_bit_cast(u32x4, o), ro, off);
        else buf_store8(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, ro, off);
      }
    }

    // State: decay by the chunk, add K^T (weighted V). Token of slot s of pair kp: 32 kp + 16 (s / 4) + 4 g + s % 4.
    u32x4 part[2][TERMS];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      float w[8];
      token_weights(pw, n, kp, g, w);
      if (STATE_ONLY) {
#pragma unroll
        for (int s = 0; s < 8; ++s) w[s] *= behind;
      }
      split_weighted<TERMS>(vf[kp], w, part[kp]);
    }
    behind *= pw[kPowZero + n];
    const float keep = pw[kPowZero + n - 1 + lead];
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      if (!STATE_ONLY) S[b] *= keep;
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const u32x4 kf = frag_k_rows_shifted(Ks, kPitchK, 32 * kp, 16 * b, lane);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) S[b] = mfma16x16x32(kf, part[kp][t], S[b]);
      }
    }
  }

  // A value of v or k that is not finite is left in its columns of the state, whatever comes behind it:
  // a wave that finds one there takes them again. (A sequence without tokens has none to take.)
  float none = 0.f;
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) none = fmaf(S[b][r], 0.f, none);
  if (__builtin_expect(__ballot(none != 0.f) != 0 && u.p.len > 0, 0)) return lin_by_token<KB, W, STATE_ONLY>(&again, pw);
  leave_state<KB, STATE_ONLY>(a, u, dvc, g, S, pw);
}

template <int KB, int W, int TERMS>
__global__ __launch_bounds__(64 * W, KB <= 4 ? W / 2 : W / 4) void lin_mfma_kernel(LinScan a) {
  lin_mfma<KB, W, TERMS, false>(a, 0, blockIdx.x, gridDim.x);
}

// The blocks' own sums of one scan, or of two: the first `na` workgroups are a's.
// Five waves a SIMD up to dk = 64, as the matrix form takes: without the bound
// lin_by_token's registers left four.
template <int KB, int W, int TERMS>
__global__ __launch_bounds__(64 * W, KB <= 2 ? 5 : KB <= 4 ? 4 : W / 4) void lin_mfma_states_kernel(LinScan a, LinScan b, long na) {
  if ((long)blockIdx.x < na) lin_mfma<KB, W, TERMS, true>(a, 0, blockIdx.x, na);
  else lin_mfma<KB, W, TERMS, true>(b, 1, blockIdx.x - na, gridDim.x - na);
}

long mfma_blocks(const LinScan& a) {
  const long slots = a.S > 0 ? a.slots_per_row : a.slots_per_row * a.batch;
  const int tile = lin_mfma_tile(a.dv);
  return slots * a.H * ((a.dv + tile - 1) / tile);
}

// The instance for sizes dk and dv and a state that is an fp32 result or not:
// f(KB, W, TERMS) as integral constants.
template <typename F>
void mfma_instance(int dk, int dv, bool fine, F f) {
  using std::integral_constant;
  auto wide = [&](auto kb) {
    auto terms = [&](auto w) {
      if (fine) f(kb, w, integral_constant<int, 3>{});
      else f(kb, w, integral_constant<int, 2>{});
    };
    if (lin_mfma_tile(dv) == 128) terms(integral_constant<int, 8>{});
    else terms(integral_constant<int, 4>{});
  };
  if (dk <= 32) wide(integral_constant<int, 1>{});
  else if (dk <= 64) wide(integral_constant<int, 2>{});
  else if (dk <= 128) wide(integral_constant<int, 4>{});
  else wide(integral_constant<int, 8>{});
}

int k_class(int dk) { return dk <= 32 ? 1 : dk <= 64 ? 2 : dk <= 128 ? 4 : 8; }

}  // namespace

// Value columns of one workgroup: 64 up to dv = 64, else 128. Sums and scan with
// 64 and with 128, in us: heads of 128 x 128, T = 16384: 66 + 162 and 57 + 125 (q
// and k are read once, not twice); heads of 64 x 64, 5087 ragged tokens: 12 + 16
// and 15 + 29 (half of the columns would be empty).
int lin_mfma_tile(int dv) { return dv <= 64 ? 64 : 128; }

// Four waves a SIMD with dk up to 64, and with eight-wave workgroups up to 128
// (launch bounds, and LDS of two of them a CU); one workgroup a CU above.
int lin_mfma_target(int dk, int dv) {
  const int cus = 256;
  if (dk > 128) return cus;
  return lin_mfma_tile(dv) == 128 ? 2 * cus : dk <= 64 ? 4 * cus : 2 * cus;
}

hipError_t launch_lin_mfma(const LinScan& a, hipStream_t stream) {
  mfma_instance(a.dk, a.dv, a.fine(), [&](auto kb, auto w, auto terms) {
    constexpr int KB = decltype(kb)::value, W = decltype(w)::value, TERMS = decltype(terms)::value;
    hipLaunchKernelGGL((lin_mfma_kernel<KB, W, TERMS>), dim3((unsigned)mfma_blocks(a)), dim3(64 * W), 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_lin_mfma_states(const LinScan& a, const LinScan* b, hipStream_t stream) {
  if (b && (k_class(a.dk) != k_class(b->dk) || lin_mfma_tile(a.dv) != lin_mfma_tile(b->dv))) {
    const hipError_t e = launch_lin_mfma_states(a, nullptr, stream);
    return e == hipSuccess ? launch_lin_mfma_states(*b, nullptr, stream) : e;
  }
  mfma_instance(a.dk, a.dv, a.fine() || (b && b->fine()), [&](auto kb, auto w, auto terms) {
    constexpr int KB = decltype(kb)::value, W = decltype(w)::value, TERMS = decltype(terms)::value;
    const long na = mfma_blocks(a), all = na + (b ? mfma_blocks(*b) : 0);
    hipLaunchKernelGGL((lin_mfma_states_kernel<KB, W, TERMS>), dim3((unsigned)all), dim3(64 * W), 0, stream, a, b ? *b : a, na);
  });
  return hipGetLastError();
}

}  // namespace ssd
