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
//           values (2^-16 of it is dropped): the state is an fp32 result that
//           is carried on, and one bf16 rounding of each term would show in it.
// Roundings to bf16: the weighted scores and the state as operands, and O.
//
// A chunk moves C (2 dk + 2 dv) 2 bytes and makes 2 C (C + 3 dk) dv multiplies
// (the doubled state product included), so at dk = dv = 128 the memory's rate
// bounds it once the matrix pipes are a third busy. The next chunk's rows are in flight
// in registers while this one is computed.
#include <type_traits>

#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

namespace {

constexpr int kC = 64;
constexpr int kPitchP = lds_pitch(kC);

// Keeps what is computed from v where it is: the weights are powers with
// exponents known before the loop, but held over it they would cost registers
// that the fourth wave of a SIMD needs, and computing them is cheap.
__device__ __forceinline__ void here(int& v) { asm volatile("" : "+v"(v)); }

// A 16-byte piece c8 (of four) of 32 columns, stored in the order of an
// accumulator pair: column 16 t + 4 g + k at 8 g + 4 t + k.
__device__ __forceinline__ void store_paired(uint16_t* row, int j, int c8, u32x4 v) {
  uint16_t* at = row + 32 * j + 16 * (c8 & 1) + 4 * (c8 >> 1);
  *reinterpret_cast<u32x2*>(at) = u32x2{v.x, v.y};
  *reinterpret_cast<u32x2*>(at + 8) = u32x2{v.z, v.w};
}
// The operand of rows row0 + c16 in that order, from columns stored as they are.
__device__ __forceinline__ u32x4 frag_k_cols_paired(const uint16_t* W, int pitch, int row0, int col0, int lane) {
  const uint16_t* at = W + (row0 + (lane & 15)) * pitch + col0 + 4 * (lane >> 4);
  const u32x2 lo = *reinterpret_cast<const u32x2*>(at), hi = *reinterpret_cast<const u32x2*>(at + 16);
  return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// KB: dk in units of 32. NB: 64 NB value columns a workgroup of 4 NB waves.
template <int KB, int NB, bool STATE_ONLY>
__device__ __forceinline__ void lin_mfma(const LinScan& a, long bid, long blocks) {
  constexpr int kDk = 32 * KB, kDv = 64 * NB, kThreads = 256 * NB;
  constexpr int kPitchK = lds_pitch(kDk), kPitchV = lds_pitch(kDv);
  __shared__ __align__(16) uint16_t Ks[kC * kPitchK];
  __shared__ __align__(16) uint16_t Vs[kC * kPitchV];
  __shared__ __align__(16) uint16_t Qs[STATE_ONLY ? 8 : kC * kPitchK];
  __shared__ __align__(16) uint16_t Ps[STATE_ONLY ? 8 : kC * kPitchP];
  constexpr int kQK = (256 * KB + kThreads - 1) / kThreads;   // 16-byte pieces a thread stages of q and of k

  const int tiles = (a.dv + kDv - 1) / kDv;
  const long u = xcd_unit(bid, blocks);
  const int dv0 = (int)(u % tiles) * kDv;
  const int h = (int)((u / tiles) % a.H);
  const long slot = u / ((long)tiles * a.H);
  const LinPiece p = lin_piece(a, slot);
  if (p.blk < 0) return;
  const int pos0 = p.blk * a.L;
  const int total = min(p.len - pos0, a.L);
  const bool last = pos0 + total >= p.len;
  if (STATE_ONLY && last) return;  // the scan carries the last block's state itself
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const float g2 = lin_log2_decay(a.ld, h);
  const long mat = (long)a.dv * a.dk;
  const int dvc = dv0 + 16 * wave + c16;

  // The state: block b holds D[dvc][dk] at dk = 16 b + 4 g + r.
  f32x4 S[2 * KB];
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b) S[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!STATE_ONLY) {
    const float* src = p.blk > 0 ? a.states + (slot * a.H + h) * mat : a.init;
    if (p.blk == 0 && src) src += ((long)p.seq * a.H + h) * mat;
    const bool tr = p.blk == 0 && a.init_tr;
    const float sc = p.blk == 0 ? a.init_scale : 1.f;
    if (src && dvc < a.dv) {
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
  }

  constexpr int kTasks = 2 / NB;   // score tasks (16 queries by 32 keys) a wave

  u32x4 qn[kQK], kn[kQK], vn[2];
  auto load = [&](int t0) {  // rows of the chunk that starts t0 tokens into the block
    const int n = min(kC, total - t0);
    const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
    auto rows = [&](const LinOperand& x, int d, int col0) {
      const uint16_t* base = static_cast<const uint16_t*>(x.base) + low * x.row + (long)(h / x.div) * d + col0;
      return make_rsrc(base, (uint32_t)(n * x.row * 2));
    };
    auto offset = [&](const LinOperand& x, int r, int col, int end) {  // 64 rows are fewer than 2^31 bytes
      const int row = (int)x.row * 2;
      return r < n && col < end ? (uint32_t)((a.rev ? n - 1 - r : r) * row + col * 2) : kOffNone;
    };
    const rsrc_t rk = rows(a.k, a.dk, 0), rv = rows(a.v, a.dv, dv0);
#pragma unroll
    for (int j = 0; j < kQK; ++j) {
      const int i = threadIdx.x + kThreads * j;
      kn[j] = buf_load16(rk, offset(a.k, i / (4 * KB), 8 * (i % (4 * KB)), a.dk));
    }
    if (!STATE_ONLY) {
      const rsrc_t rq = rows(a.q, a.dk, 0);
#pragma unroll
      for (int j = 0; j < kQK; ++j) {
        const int i = threadIdx.x + kThreads * j;
        qn[j] = buf_load16(rq, offset(a.q, i / (4 * KB), 8 * (i % (4 * KB)), a.dk));
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = threadIdx.x + kThreads * j;
      vn[j] = buf_load16(rv, offset(a.v, i / (8 * NB), 8 * (i % (8 * NB)), a.dv - dv0));
    }
  };

  // The blocks' own sums walk their chunks backwards, weighting each V by its whole
  // distance to the block's end: the scan, which walks forwards and comes next,
  // finds the rows that were read last in the memory-side cache.
  const int chunks = (total + kC - 1) / kC;
  if (chunks > 0) load(STATE_ONLY ? (chunks - 1) * kC : 0);
  for (int ci = 0; ci < chunks; ++ci) {
    const int t0 = (STATE_ONLY ? chunks - 1 - ci : ci) * kC;
    const int n = min(kC, total - t0);
    const int after = STATE_ONLY ? total - t0 - n : 0;  // tokens of the block behind this chunk
    const int lead = a.rev && pos0 + t0 == 0 ? 0 : 1;   // the state handed to a reversed scan is not decayed first
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQK; ++j) {
      const int i = threadIdx.x + kThreads * j;
      const int row = i / (4 * KB), col = i % (4 * KB);
      if (kThreads <= 256 * KB || i < 256 * KB) {
        *reinterpret_cast<u32x4*>(Ks + row * kPitchK + 8 * col) = kn[j];
        if (!STATE_ONLY) store_paired(Qs + row * kPitchK, col >> 2, col & 3, qn[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = threadIdx.x + kThreads * j;
      *reinterpret_cast<u32x4*>(Vs + i / (8 * NB) * kPitchV + 8 * (i % (8 * NB))) = vn[j];
    }
    __syncthreads();

    if (!STATE_ONLY) {
#pragma unroll
      for (int k = 0; k < kTasks; ++k) {
        const int qb = wave & 3, kp = NB == 2 ? wave >> 2 : k;
        if (kp > qb / 2) continue;   // all keys are later; never read
        f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const u32x4 q = frag_k_cols(Qs, kPitchK, 16 * qb, 32 * j, lane);
          s0 = mfma16x16x32(frag_k_cols_paired(Ks, kPitchK, 32 * kp, 32 * j, lane), q, s0);
          s1 = mfma16x16x32(frag_k_cols_paired(Ks, kPitchK, 32 * kp + 16, 32 * j, lane), q, s1);
        }
        // Query minus key, of the first key (r = 0); weighted, or 0 (selected: a later key may hold anything).
        int diff = 16 * qb - 32 * kp + c16 - 4 * g;
        here(diff);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s0[r] = diff >= r ? s0[r] * fast_exp2(g2 * (float)(diff - r)) : 0.f;
          s1[r] = diff - 16 >= r ? s1[r] * fast_exp2(g2 * (float)(diff - 16 - r)) : 0.f;
        }
        *reinterpret_cast<u32x4*>(Ps + (16 * qb + c16) * kPitchP + 32 * kp + 8 * g) =
            u32x4{pack_bf16x2(s0[0], s0[1]), pack_bf16x2(s0[2], s0[3]), pack_bf16x2(s1[0], s1[1]), pack_bf16x2(s1[2], s1[3])};
      }
    }
    if (ci + 1 < chunks) load(STATE_ONLY ? t0 - kC : t0 + kC);

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
      for (int qb = 0; qb < 4; ++qb) O[qb] *= fast_exp2(g2 * (float)(16 * qb)) * fast_exp2(g2 * (float)(c16 + lead));
      __syncthreads();
#pragma unroll
      for (int qb = 0; qb < 4; ++qb)
#pragma unroll
        for (int kp = 0; kp <= qb / 2; ++kp)
          O[qb] = mfma16x16x32(vf[kp], frag_k_cols(Ps, kPitchP, 16 * qb, 32 * kp, lane), O[qb]);
      // O^T: column c16 is the query, rows 4 g + r the value columns.
      const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
      const int esz = a.o_f32 ? 4 : 2, orow = a.H * a.dv;
      const rsrc_t ro = make_rsrc(static_cast<char*>(a.o) + (low * orow + (long)h * a.dv) * esz, (uint32_t)(n * orow * esz));
      const int dv = dv0 + 16 * wave + 4 * g;
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) {
        const int r = 16 * qb + c16;
        const uint32_t off = r < n && dv < a.dv ? (uint32_t)(((a.rev ? n - 1 - r : r) * orow + dv) * esz) : kOffNone;
        const f32x4 o = O[qb] * a.scale;
        if (a.o_f32) buf_store16(__builtin_bit_cast(u32x4, o), ro, off);
        else buf_store8(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, ro, off);
      }
    }

    // State: decay by the chunk, add K^T (weighted V). Token of slot s of pair kp: 32 kp + 16 (s / 4) + 4 g + s % 4.
    u32x4 hi[2], lo[2];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      float w[8];
      int first = 32 * kp + 4 * g;
      here(first);
#pragma unroll
      for (int s = 0; s < 8; ++s) w[s] = fast_exp2(g2 * (float)(after + max(n - 1 - (first + 16 * (s >> 2) + (s & 3)), 0)));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = bf16_lo(vf[kp][c]) * w[2 * c], y = bf16_hi(vf[kp][c]) * w[2 * c + 1];
        hi[kp][c] = pack_bf16x2(x, y);
        lo[kp][c] = pack_bf16x2(x - bf16_lo(hi[kp][c]), y - bf16_hi(hi[kp][c]));
      }
    }
    const float keep = fast_exp2(g2 * (float)(n - 1 + lead));
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      if (!STATE_ONLY) S[b] *= keep;
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const u32x4 kf = frag_k_rows_accpair(Ks, kPitchK, 32 * kp, 16 * b, lane);
        S[b] = mfma16x16x32(kf, hi[kp], S[b]);
        S[b] = mfma16x16x32(kf, lo[kp], S[b]);
      }
    }
  }

  float* dst = nullptr;
  float sc = 1.f;
  if (STATE_ONLY) {
    dst = a.states + (slot * a.H + h) * mat;
  } else if (last && a.fin) {
    dst = a.fin + ((long)p.seq * a.H + h) * mat;
    sc = a.fin_scale * (a.rev && p.len > 0 ? fast_exp2(g2) : 1.f);
  }
  if (dst && dvc < a.dv) {
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      const int dk = 16 * b + 4 * g;
      if (dk < a.dk) *reinterpret_cast<f32x4*>(dst + (long)dvc * a.dk + dk) = S[b] * sc;
    }
  }
}

// Four waves a SIMD (two workgroups of eight waves a CU) hide the barriers'
// and LDS reads' waits; dk above 128 leaves registers and LDS for half of that.
template <int KB, int NB>
__global__ __launch_bounds__(256 * NB, KB <= 4 ? 4 : 2) void lin_mfma_kernel(LinScan a) {
  lin_mfma<KB, NB, false>(a, blockIdx.x, gridDim.x);
}

// The blocks' own sums of one scan, or of two: the first `na` workgroups are a's.
template <int KB, int NB>
__global__ __launch_bounds__(256 * NB, KB <= 4 ? 4 : 2) void lin_mfma_states_kernel(LinScan a, LinScan b, long na) {
  if ((long)blockIdx.x < na) lin_mfma<KB, NB, true>(a, blockIdx.x, na);
  else lin_mfma<KB, NB, true>(b, blockIdx.x - na, gridDim.x - na);
}

template <int KB, int NB>
long mfma_blocks(const LinScan& a) {
  const long slots = a.S > 0 ? a.slots_per_row : a.slots_per_row * a.batch;
  return slots * a.H * ((a.dv + 64 * NB - 1) / (64 * NB));
}

// The instance for sizes dk and dv: f(KB, NB) as integral constants.
template <typename F>
void mfma_instance(int dk, int dv, F f) {
  using std::integral_constant;
  auto wide = [&](auto kb) {
    if (lin_mfma_tile(dv) == 128) f(kb, integral_constant<int, 2>{});
    else f(kb, integral_constant<int, 1>{});
  };
  if (dk <= 32) wide(integral_constant<int, 1>{});
  else if (dk <= 64) wide(integral_constant<int, 2>{});
  else if (dk <= 128) wide(integral_constant<int, 4>{});
  else wide(integral_constant<int, 8>{});
}

int k_class(int dk) { return dk <= 32 ? 1 : dk <= 64 ? 2 : dk <= 128 ? 4 : 8; }

}  // namespace

// Value columns of one workgroup: 64 up to dv = 64, else 128.
int lin_mfma_tile(int dv) { return dv <= 64 ? 64 : 128; }

hipError_t launch_lin_mfma(const LinScan& a, hipStream_t stream) {
  mfma_instance(a.dk, a.dv, [&](auto kb, auto nb) {
    constexpr int KB = decltype(kb)::value, NB = decltype(nb)::value;
    hipLaunchKernelGGL((lin_mfma_kernel<KB, NB>), dim3((unsigned)mfma_blocks<KB, NB>(a)), dim3(256 * NB), 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_lin_mfma_states(const LinScan& a, const LinScan* b, hipStream_t stream) {
  if (b && (k_class(a.dk) != k_class(b->dk) || lin_mfma_tile(a.dv) != lin_mfma_tile(b->dv))) {
    const hipError_t e = launch_lin_mfma_states(a, nullptr, stream);
    return e == hipSuccess ? launch_lin_mfma_states(*b, nullptr, stream) : e;
  }
  mfma_instance(a.dk, a.dv, [&](auto kb, auto nb) {
    constexpr int KB = decltype(kb)::value, NB = decltype(nb)::value;
    const long na = mfma_blocks<KB, NB>(a), all = na + (b ? mfma_blocks<KB, NB>(*b) : 0);
    hipLaunchKernelGGL((lin_mfma_states_kernel<KB, NB>), dim3((unsigned)all), dim3(256 * NB), 0, stream, a, b ? *b : a, na);
  });
  return hipGetLastError();
}

}  // namespace ssd
