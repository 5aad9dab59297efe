// ssd_lin_bwd.hip -- linear attention with one decay a head: the gradients of
// keys and values in one reversed scan, on bf16 matrix instructions.
//
// With R the adjoint state [dv][dk] that enters a chunk from behind, and i, j
// its tokens, i not before j (lam^(i-j) masked to that):
//     dV = (lam^(i-j) o K Q^T) dO + lam^(.) K R^T
//     dK = (lam^(i-j) o V dO^T) Q + lam^(.) V R
//     R' = lam^C R + (lam^(.) dO)^T Q.
// Both need the rows of q, k, v and dO and the same R, so one scan reads
// 2 dk + 2 dv and writes dk + dv values a token, where two scans would read
// 4 dk + 4 dv (2 reads of q, dO for the state each) and carry R twice. Chunk
// order, products, layouts and roundings are those of ssd_lin_scan.hip with
// q := K, k := Q, v := dO for dV; dK contracts over R's other index, for which
// R is laid down in LDS once a chunk as the bf16 operand it is rounded to
// anyway. 4 VB waves, four a SIMD: value block w % 2 VB of R and dV a wave, of R
// one half of the key columns and of dV one half of the chunk's tokens; dK's
// blocks of 16 key columns by 16 tokens are dealt over the waves.
//
// T = 8192, 32 heads of 128 x 128: mean 127 us, least 111, for 417 MB (3.3 and 3.8
// TB/s), 254 - 258 us a backward call (own sums of both scans 73, entering states
// 18, dQ 73); the
// one scan in place of two took such a call from 347 to 295 us. Heads of more
// than 128 take two scans: R and its bf16 copy would not fit. It is bound by its
// phases between barriers in the one workgroup that a CU holds (matrix pipes 20 %
// busy, LDS half the time); leaving out any one product gains 8 to 14 us.
#include "ssd_lin_chunk.h"

namespace ssd {

namespace {

struct KvArgs {
  LinScan a;        // the scan for dv
  LinOperand v;
  void* dk_out;
};

// What a workgroup takes: one head's block.
struct KvUnit {
  int h, pos0, total;   // head, the block's first token and tokens in the sequence
  long slot;
  bool last;            // of the sequence
  LinPiece p;           // p.blk < 0: nothing
};
__device__ __forceinline__ KvUnit kv_unit(const LinScan& a) {
  KvUnit w;
  const long u = xcd_unit(blockIdx.x, gridDim.x);
  w.h = (int)(u % a.H);
  w.slot = u / a.H;
  w.p = lin_piece(a, w.slot);
  w.pos0 = w.p.blk * a.L;
  w.total = min(w.p.len - w.pos0, a.L);
  w.last = w.pos0 + w.total >= w.p.len;
  return w;
}

// A wave's part of R, dv = dvc and dk = dk0 + 16 b + r: as it enters the block,
template <int KB>
__device__ __forceinline__ void enter_state(const LinScan& a, const KvUnit& w, int dvc, int dk0, f32x4 (&R)[KB]) {
  const long mat = (long)a.dv * a.dk;
#pragma unroll
  for (int b = 0; b < KB; ++b) R[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* src = w.p.blk > 0 ? a.states + (w.slot * a.H + w.h) * mat : a.init;
  if (w.p.blk == 0 && src) src += ((long)w.p.seq * a.H + w.h) * mat;
  const float sc = w.p.blk == 0 ? a.init_scale : 1.f;
  if (!src || dvc >= a.dv) return;
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    const int dk = dk0 + 16 * b;
    if (dk < a.dk) R[b] = *reinterpret_cast<const f32x4*>(src + (long)dvc * a.dk + dk) * sc;
  }
}
// and as it leaves the sequence.
template <int KB>
__device__ __forceinline__ void leave_state(const LinScan& a, const KvUnit& w, int dvc, int dk0, const f32x4 (&R)[KB],
                                            const float* pw) {
  if (!w.last || !a.fin || dvc >= a.dv) return;
  const float sc = a.fin_scale * (w.p.len > 0 ? pw[kPowZero + 1] : 1.f);
  float* dst = a.fin + ((long)w.p.seq * a.H + w.h) * a.dv * a.dk;
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    const int dk = dk0 + 16 * b;
    if (dk < a.dk) *reinterpret_cast<f32x4*>(dst + (long)dvc * a.dk + dk) = R[b] * sc;
  }
}

// The block by the recurrence itself, token by token in fp32, where a value of q
// or dO is not finite (see lin_by_token). R lies over the waves as in the matrix
// form. Of every token each wave leaves its sums over its part of R in `part`, of
// even tokens in one half and of odd ones in the other, and behind a barrier they
// are joined in order. `again`, in LDS: where the launch put the arguments.
template <int KB, int VB>
__device__ __forceinline__ void kv_by_token(const KvArgs* const* again, float* part, const float* pw) {
  constexpr int kThreads = 256 * VB, kHalf = 2 * 32 * VB + 2 * VB * 32 * KB;
  static_assert(2 * kHalf * 4 <= 2 * kC * kPitchP * 2, "lies in the scores' place");
  int tid = threadIdx.x;
  asm volatile("s_waitcnt vmcnt(0)" : "+v"(tid) : : "memory");   // the outputs of the first time are written
  const KvArgs* args = uniform(*again);
  const LinScan& a = args->a;
  const KvUnit u = kv_unit(a);
  const int wave = uniform(tid >> 6), c16 = tid & 15, g = (tid & 63) >> 4;
  const int vb = wave % (2 * VB), half = wave / (2 * VB);
  const int dvc = 16 * vb + c16, dk0 = 16 * KB * half + 4 * g;
  const int dk = a.dk, dv = a.dv, H = a.H, o_f32 = a.o_f32;
  const bool in = dvc < dv;
  const long krow = a.q.row, qrow = a.k.row, grow = a.v.row, vrow = args->v.row;
  auto base = [&](const LinOperand& x, int d) { return static_cast<const uint16_t*>(x.base) + (long)(u.h / x.div) * d; };
  const uint16_t *k0 = base(a.q, dk), *q0 = base(a.k, dk), *g0 = base(a.v, dv) + (in ? dvc : 0),
                 *v0 = base(args->v, dv) + (in ? dvc : 0);
  void *const out_v = a.o, *const out_k = args->dk_out;
  const float scale = a.scale, lam_hi = pw[kPowHi], lam_lo = pw[kPowHi + 1];
  f32x4 R[KB];
  enter_state<KB>(a, u, dvc, dk0, R);
  u32x2 k[KB], q[KB];   // the next token's rows
  uint16_t dO = 0, v = 0;
  auto token = [&](int j) { return u.p.start + (u.p.len - 1 - (u.pos0 + j)); };
  auto load = [&](int j) {
    const long tok = token(min(j, u.total - 1));
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int col = dk0 + 16 * b < dk ? dk0 + 16 * b : 0;
      k[b] = *reinterpret_cast<const u32x2*>(k0 + tok * krow + col);
      q[b] = *reinterpret_cast<const u32x2*>(q0 + tok * qrow + col);
    }
    dO = g0[tok * grow];
    v = v0[tok * vrow];
  };
  auto put = [&](void* out, int d, int j, int i, float o) {
    const long at = (token(j) * H + u.h) * d + i;
    if (o_f32) static_cast<float*>(out)[at] = o * scale;
    else static_cast<uint16_t*>(out)[at] = f32_to_bf16(o * scale);
  };
  load(0);
#pragma unroll 1
  for (int j = 0; j < u.total; ++j) {
    const bool keep = u.pos0 + j == 0;   // the state handed in is not decayed before the last token
    const float hi = keep ? kOneHi : lam_hi, lo = keep ? kOneLo : lam_lo;
    const float x = bf16_to_f32(dO), y = bf16_to_f32(v);
    float *sum_v = part + (j & 1) * kHalf, *sum_k = sum_v + 2 * 32 * VB, to_v = 0.f;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const f32x4 kb = four(k[b]), qb = four(q[b]);
      f32x4 to_k = {0.f, 0.f, 0.f, 0.f};
      if (in && dk0 + 16 * b < dk) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          R[b][r] = fmaf(R[b][r], hi, fmaf(R[b][r], lo, x * qb[r]));
          to_v = fmaf(R[b][r], kb[r], to_v);
          to_k[r] = R[b][r] * y;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) to_k[r] = lanes_sum(to_k[r], 16);
      if (c16 == 0) *reinterpret_cast<f32x4*>(sum_k + vb * 32 * KB + dk0 + 16 * b) = to_k;
    }
    load(j + 1);
    to_v += __shfl_xor(to_v, 16);
    to_v += __shfl_xor(to_v, 32);
    if (g == 0) sum_v[half * 32 * VB + dvc] = to_v;
    __syncthreads();
    if (tid < dk) {
      float o = 0.f;
      for (int i = 0; i < 2 * VB; ++i) o += sum_k[i * 32 * KB + tid];
      put(out_k, dk, j, tid, o);
    }
    const int i = kThreads - 1 - tid;
    if (i < dv) put(out_v, dv, j, i, sum_v[i] + sum_v[32 * VB + i]);
  }
  leave_state<KB>(a, u, dvc, dk0, R, pw);
}

// KB, VB: dk and dv in units of 32 (2 or 4). TERMS: as in ssd_lin_scan.hip.
template <int KB, int VB, int TERMS>
__global__ __launch_bounds__(256 * VB, 4) void lin_kv_kernel(KvArgs args) {
  const LinScan& a = args.a;
  const LinOperand& vop = args.v;
  void* const dk_out = args.dk_out;
  constexpr int kWaves = 4 * VB, kThreads = 64 * kWaves;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = lds_pitch(32 * VB);
  __shared__ __align__(16) uint16_t Qs[kC * kPitchK], Gs[kC * kPitchV];   // q and dO, rows by row_shift
  __shared__ __align__(16) uint16_t Ks[kC * kPitchK], Vs[kC * kPitchV];   // k and v, columns in pair order
  __shared__ __align__(16) uint16_t Ps[2][kC * kPitchP];            // weighted K Q^T and V dO^T
  __shared__ __align__(16) uint16_t Rs[32 * VB * kPitchK];          // R, rounded, rows by row_shift
  __shared__ __align__(16) float pw[kPowSize], spw[kPowSize];       // powers of lam, and scale times them
  // 16-byte pieces: with sixteen waves half of the threads stage q and k, the others dO and v.
  constexpr bool kHalves = VB == 4;
  constexpr int kStage = kHalves ? kThreads / 2 : kThreads;
  constexpr int kK = 256 * KB / kStage, kV = 256 * VB / kStage;
  constexpr int kMost = kK > kV ? kK : kV;
  // Score tasks (16 tokens j by 32 tokens i): 6 of K Q^T and 6 of V dO^T that are not all masked.
  constexpr int kTasks = 16 / kWaves;
  // dK: blocks of 16 key columns by 16 tokens a wave.
  constexpr int kDkTok = 2 * KB / VB;

  __shared__ const KvArgs* again;
  if (threadIdx.x == 0) again = (const KvArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const KvUnit u = kv_unit(a);
  if (u.p.blk < 0) return;
  const LinPiece& p = u.p;
  const int h = u.h, pos0 = u.pos0, total = u.total;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int vb = wave % (2 * VB), half = wave / (2 * VB);     // value block; half of dk (R) and of the tokens (dV)
  const int kb0 = wave % (2 * KB), tb0 = wave / (2 * KB) * kDkTok;   // dK: key block, first token block
  fill_powers(pw, spw, a.ld[h], a.scale);

  const int dvc = 16 * vb + c16, dk0 = 16 * KB * half + 4 * g;
  f32x4 R[KB];   // dv = dvc, dk = dk0 + 16 b + r
  enter_state<KB>(a, u, dvc, dk0, R);

  const int qrow = (int)a.k.row * 2, krow = (int)a.q.row * 2, grow = (int)a.v.row * 2, vrow = (int)vop.row * 2;
  const int tid = kHalves ? threadIdx.x % kStage : threadIdx.x;
  const bool stage_k = !kHalves || threadIdx.x < kStage, stage_v = !kHalves || threadIdx.x >= kStage;
  // This thread's pieces: of q and k, and of dO and v (one of the two in halves).
  u32x4 x0[kHalves ? kMost : kK], x1[kHalves ? kMost : kK], y0[kHalves ? 1 : kV], y1[kHalves ? 1 : kV];
  auto load = [&](int t0) {
    const int n = min(kC, total - t0);
    const long low = p.start + (long)p.len - (pos0 + t0) - n;
    auto rows = [&](const LinOperand& x, int d) {
      return make_rsrc(static_cast<const uint16_t*>(x.base) + low * x.row + (long)(h / x.div) * d, (uint32_t)(n * x.row * 2));
    };
    if (stage_k) {
      const rsrc_t rq = rows(a.k, a.dk), rk = rows(a.q, a.dk);
#pragma unroll
      for (int j = 0; j < kK; ++j) {
        const int i = tid + kStage * j, r = i / (4 * KB), col = 8 * (i % (4 * KB));
        x0[j] = buf_load16_once(rq, piece_offset(make_piece(r, col, a.dk, qrow, 2, 1), n, qrow, 1));
        x1[j] = buf_load16_once(rk, piece_offset(make_piece(r, col, a.dk, krow, 2, 1), n, krow, 1));
      }
    }
    if (stage_v) {
      u32x4 *to0 = kHalves ? x0 : y0, *to1 = kHalves ? x1 : y1;
      const rsrc_t rg = rows(a.v, a.dv), rv = rows(vop, a.dv);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int i = tid + kStage * j, r = i / (4 * VB), col = 8 * (i % (4 * VB));
        to0[j] = buf_load16_once(rg, piece_offset(make_piece(r, col, a.dv, grow, 2, 1), n, grow, 1));
        to1[j] = buf_load16_once(rv, piece_offset(make_piece(r, col, a.dv, vrow, 2, 1), n, vrow, 1));
      }
    }
  };

  if (total > 0) load(0);
  for (int t0 = 0; t0 < total; t0 += kC) {
    const int n = min(kC, total - t0);
    const bool first = pos0 + t0 == 0;
    const int lead = first ? 0 : 1;  // the state handed in is not decayed before the last token
    __syncthreads();
    if (stage_k) {
#pragma unroll
      for (int j = 0; j < kK; ++j) {
        const int i = tid + kStage * j, r = i / (4 * KB), col = i % (4 * KB);
        *reinterpret_cast<u32x4*>(Qs + r * kPitchK + row_shift(r) + 8 * col) = x0[j];
        store_paired(Ks + r * kPitchK, col >> 2, col & 3, x1[j]);
      }
    }
    if (stage_v) {
      const u32x4 *from0 = kHalves ? x0 : y0, *from1 = kHalves ? x1 : y1;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int i = tid + kStage * j, r = i / (4 * VB), col = i % (4 * VB);
        *reinterpret_cast<u32x4*>(Gs + r * kPitchV + row_shift(r) + 8 * col) = from0[j];
        store_paired(Vs + r * kPitchV, col >> 2, col & 3, from1[j]);
      }
    }
#pragma unroll
    for (int b = 0; b < KB; ++b)
      *reinterpret_cast<u32x2*>(Rs + dvc * kPitchK + row_shift(dvc) + 16 * (KB * half + b) + 4 * g) =
          u32x2{pack_bf16x2(R[b][0], R[b][1]), pack_bf16x2(R[b][2], R[b][3])};
    if (t0 + kC < total) load(t0 + kC);
    __syncthreads();

    // Scores: token j = 16 qb + c16 (columns) with tokens i = 32 kp + 16 t + 4 g + r (rows).
#pragma unroll
    for (int k = 0; k < kTasks; ++k) {
      const int task = wave + kWaves * k, qb = task & 3, kp = (task >> 2) & 1, of_v = task >> 3;
      if (kp > qb / 2) continue;   // all masked; never read
      f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
      if (of_v) {
#pragma unroll
        for (int j = 0; j < VB; ++j) {
          const u32x4 x = frag_k_cols(Vs, kPitchV, 16 * qb, 32 * j, lane);
          s0 = mfma16x16x32(frag_k_cols_pairs(Gs, kPitchV, 32 * kp, 32 * j, lane), x, s0);
          s1 = mfma16x16x32(frag_k_cols_pairs(Gs, kPitchV, 32 * kp + 16, 32 * j, lane), x, s1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const u32x4 x = frag_k_cols(Ks, kPitchK, 16 * qb, 32 * j, lane);
          s0 = mfma16x16x32(frag_k_cols_pairs(Qs, kPitchK, 32 * kp, 32 * j, lane), x, s0);
          s1 = mfma16x16x32(frag_k_cols_pairs(Qs, kPitchK, 32 * kp + 16, 32 * j, lane), x, s1);
        }
      }
      const int diff = 16 * qb - 32 * kp + c16 - 4 * g;
      const float* w = spw + kPowZero + diff;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s0[r] = diff >= r ? s0[r] * w[-r] : 0.f;
        s1[r] = diff - 16 >= r ? s1[r] * w[-16 - r] : 0.f;
      }
      store_scores(Ps[of_v] + (16 * qb + c16) * kPitchP + 32 * kp + 8 * g, s0, s1, first && qb < 2);
    }

    // Terms of R: dV^T (rows: the wave's value block; two token blocks) and dK^T (rows: its key block).
    f32x4 OV[2], OK[kDkTok];
#pragma unroll
    for (int t = 0; t < 2; ++t) OV[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < kDkTok; ++t) OK[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // The wave's own half of R is at hand as the operand; the other half is its partner's.
#pragma unroll
    for (int own = 1; own >= 0; --own)
#pragma unroll
      for (int j = 0; j < KB / 2; ++j) {
        const int col = 16 * KB * (own ? half : 1 - half) + 32 * j;
        u32x4 rf;
        if (own) {
          rf = u32x4{pack_bf16x2(R[2 * j][0], R[2 * j][1]), pack_bf16x2(R[2 * j][2], R[2 * j][3]),
                     pack_bf16x2(R[2 * j + 1][0], R[2 * j + 1][1]), pack_bf16x2(R[2 * j + 1][2], R[2 * j + 1][3])};
        } else {
          rf = frag_k_cols_pairs(Rs, kPitchK, 16 * vb, col, lane);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) OV[t] = mfma16x16x32(rf, frag_k_cols(Ks, kPitchK, 32 * half + 16 * t, col, lane), OV[t]);
      }
#pragma unroll
    for (int j = 0; j < VB; ++j) {
      const u32x4 rt = frag_k_rows_shifted(Rs, kPitchK, 32 * j, 16 * kb0, lane);
#pragma unroll
      for (int t = 0; t < kDkTok; ++t)
        OK[t] = mfma16x16x32(rt, frag_k_cols(Vs, kPitchV, 16 * (tb0 + t), 32 * j, lane), OK[t]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) OV[t] *= spw[kPowZero + 32 * half + 16 * t + c16 + lead];
#pragma unroll
    for (int t = 0; t < kDkTok; ++t) OK[t] *= spw[kPowZero + 16 * (tb0 + t) + c16 + lead];
    u32x4 gf[2];   // dO^T of this wave's value block
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) gf[kp] = frag_k_rows_shifted(Gs, kPitchV, 32 * kp, 16 * vb, lane);
    __syncthreads();

    // Terms of the chunk's own tokens.
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      if (kp <= half) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          OV[t] = mfma16x16x32(gf[kp], frag_k_cols(Ps[0], kPitchP, 32 * half + 16 * t, 32 * kp, lane), OV[t]);
      }
      const u32x4 qf = frag_k_rows_shifted(Qs, kPitchK, 32 * kp, 16 * kb0, lane);
#pragma unroll
      for (int t = 0; t < kDkTok; ++t)
        if (kp <= (tb0 + t) / 2) OK[t] = mfma16x16x32(qf, frag_k_cols(Ps[1], kPitchP, 16 * (tb0 + t), 32 * kp, lane), OK[t]);
      if (first && kp == 0) {   // what rounding left of the first 32 tokens' scores
        if (half == 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t) OV[t] = mfma16x16x32(gf[0], frag_k_cols(Ps[0], kPitchP, 16 * t, 32, lane), OV[t]);
        }
#pragma unroll
        for (int t = 0; t < kDkTok; ++t)
          if (tb0 + t < 2) OK[t] = mfma16x16x32(qf, frag_k_cols(Ps[1], kPitchP, 16 * (tb0 + t), 32, lane), OK[t]);
      }
    }

    const long low = p.start + (long)p.len - (pos0 + t0) - n;
    const int esz = a.o_f32 ? 4 : 2;
    auto put = [&](void* out, int d, int tok, int col, f32x4 o) {
      const int row = a.H * d * esz;
      const rsrc_t ro = make_rsrc(static_cast<char*>(out) + low * row + (long)h * d * esz, (uint32_t)(n * row));
      const uint32_t off = piece_offset(make_piece(tok, col, d, row, esz, 1), n, row, 1);
      if (a.o_f32) buf_store16(__builtin_bit_cast(u32x4, o), ro, off);
      else buf_store8(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, ro, off);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) put(a.o, a.dv, 32 * half + 16 * t + c16, 16 * vb + 4 * g, OV[t]);
#pragma unroll
    for (int t = 0; t < kDkTok; ++t) put(dk_out, a.dk, 16 * (tb0 + t) + c16, 16 * kb0 + 4 * g, OK[t]);

    // R: decay by the chunk, add Q^T (weighted dO).
    u32x4 part[2][TERMS];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      float w[8];
      token_weights(pw, n, kp, g, w);
      split_weighted<TERMS>(gf[kp], w, part[kp]);
    }
    const float keep = pw[kPowZero + n - 1 + lead];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      R[b] *= keep;
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const u32x4 qf = frag_k_rows_shifted(Qs, kPitchK, 32 * kp, 16 * (KB * half + b), lane);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) R[b] = mfma16x16x32(qf, part[kp][t], R[b]);
      }
    }
  }

  // A value of q or dO that is not finite is left in R, whatever comes behind it. (A sequence without
  // tokens has none, and none to read: it may start at the tensors' end.)
  float none = 0.f;
#pragma unroll
  for (int b = 0; b < KB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) none = fmaf(R[b][r], 0.f, none);
  if (__builtin_expect(__syncthreads_or(none != 0.f && u.p.len > 0), 0))
    return kv_by_token<KB, VB>(&again, reinterpret_cast<float*>(&Ps[0][0]), pw);
  leave_state<KB>(a, u, dvc, dk0, R, pw);
}

}  // namespace

bool lin_kv_supported(int dk, int dv, int bf16) { return bf16 && dk <= 128 && dv <= 128; }

// Workgroups that run at once: one of sixteen waves a CU, or two of eight where LDS holds them.
int lin_kv_target(int dk, int dv) { return dv <= 64 && dk <= 64 ? 512 : 256; }
int lin_kv_threads(int dv) { return dv <= 64 ? 512 : 1024; }

namespace {
template <int KB, int VB>
void kv_launch(const LinScan& a, const LinOperand& v, void* dk_out, hipStream_t stream) {
  const long slots = a.S > 0 ? a.slots_per_row : a.slots_per_row * a.batch;
  const dim3 grid((unsigned)(slots * a.H)), block(256 * VB);
  const KvArgs args = {a, v, dk_out};
  if (a.fine()) hipLaunchKernelGGL((lin_kv_kernel<KB, VB, 3>), grid, block, 0, stream, args);
  else hipLaunchKernelGGL((lin_kv_kernel<KB, VB, 2>), grid, block, 0, stream, args);
}
}  // namespace

hipError_t launch_lin_kv(const LinScan& a, const LinOperand& v, void* dk_out, hipStream_t stream) {
  if (a.dv <= 64) a.dk <= 64 ? kv_launch<2, 2>(a, v, dk_out, stream) : kv_launch<4, 2>(a, v, dk_out, stream);
  else a.dk <= 64 ? kv_launch<2, 4>(a, v, dk_out, stream) : kv_launch<4, 4>(a, v, dk_out, stream);
  return hipGetLastError();
}

}  // namespace ssd
