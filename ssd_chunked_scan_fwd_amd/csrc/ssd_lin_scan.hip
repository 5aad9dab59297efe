// ssd_lin_scan.hip -- linear attention with one decay a head over prompts, on
// bf16 matrix instructions (v_mfma_f32_16x16x32_bf16).
//
// Chunks of C = 64 tokens of one (block, head). With D the state [dv][dk]
// before the chunk and i, j its tokens (lam^(i-j) masked to i >= j):
//     O  = (lam^(i-j) o Q K^T) V + lam^(i+1) Q D^T
//     D' = lam^C D + (lam^(C-1-j) V)^T K.
// Four waves; wave w owns NB blocks of 16 value columns of D, in the fp32
// accumulators of its own products, over the whole chunk loop:
//   scores  wave w forms S^T = K Q^T for queries 16 w .. 16 w + 15 and the keys up
//           to them, weights them, and leaves them in LDS as bf16;
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
// in registers while this one is computed. Q's loads have the layout of the
// score product's operand, which so needs no LDS read for it.
#include <type_traits>

#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

namespace {

constexpr int kC = 64;
constexpr int kPitchP = lds_pitch(kC);

template <int KB, int NB, bool STATE_ONLY>
__device__ __forceinline__ void lin_mfma(const LinScan& a, long bid, long blocks) {
  constexpr int kDk = 32 * KB, kDv = 64 * NB;
  constexpr int kPitchK = lds_pitch(kDk), kPitchV = lds_pitch(kDv);
  __shared__ __align__(16) uint16_t Ks[kC * kPitchK];
  __shared__ __align__(16) uint16_t Vs[kC * kPitchV];
  __shared__ __align__(16) uint16_t Qs[STATE_ONLY ? 8 : kC * kPitchK];
  __shared__ __align__(16) uint16_t Ps[STATE_ONLY ? 8 : kC * kPitchP];

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

  // The state: block b of wave column block nb holds D[dv][dk] at
  // dv = dv0 + 16 (NB wave + nb) + c16, dk = 16 b + 4 g + r.
  f32x4 S[NB][2 * KB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) S[nb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (!STATE_ONLY) {
    const float* src = p.blk > 0 ? a.states + (slot * a.H + h) * mat : a.init;
    if (p.blk == 0 && src) src += ((long)p.seq * a.H + h) * mat;
    const bool tr = p.blk == 0 && a.init_tr;
    const float sc = p.blk == 0 ? a.init_scale : 1.f;
    if (src) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int dv = dv0 + 16 * (NB * wave + nb) + c16;
#pragma unroll
        for (int b = 0; b < 2 * KB; ++b) {
          const int dk = 16 * b + 4 * g;
          if (dv < a.dv && dk < a.dk) {
            if (tr) {
#pragma unroll
              for (int r = 0; r < 4; ++r) S[nb][b][r] = sc * src[(long)(dk + r) * a.dv + dv];
            } else {
              S[nb][b] = *reinterpret_cast<const f32x4*>(src + (long)dv * a.dk + dk) * sc;
            }
          }
        }
      }
    }
  }

  u32x4 qn[KB], kn[KB], vn[2 * NB];
  auto load = [&](int t0) {  // rows of the chunk that starts t0 tokens into the block
    const int n = min(kC, total - t0);
    const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
    auto rows = [&](const LinOperand& x, int d, int col0) {
      const uint16_t* base = static_cast<const uint16_t*>(x.base) + low * x.row + (long)(h / x.div) * d + col0;
      return make_rsrc(base, (uint32_t)(n * x.row * 2));
    };
    auto offset = [&](const LinOperand& x, int r, int col, int end) {
      return r < n && col < end ? (uint32_t)(((a.rev ? n - 1 - r : r) * x.row + col) * 2) : kOffNone;
    };
    const rsrc_t rk = rows(a.k, a.dk, 0), rv = rows(a.v, a.dv, dv0);
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const int i = threadIdx.x + 256 * j;
      kn[j] = buf_load16(rk, offset(a.k, i / (4 * KB), 8 * (i % (4 * KB)), a.dk));
    }
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {
      const int i = threadIdx.x + 256 * j;
      vn[j] = buf_load16(rv, offset(a.v, i / (8 * NB), 8 * (i % (8 * NB)), a.dv - dv0));
    }
    if (!STATE_ONLY) {
      const rsrc_t rq = rows(a.q, a.dk, 0);
#pragma unroll
      for (int j = 0; j < KB; ++j) qn[j] = buf_load16(rq, offset(a.q, 16 * wave + c16, 32 * j + 8 * g, a.dk));
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
    const int lead = a.rev && pos0 + t0 == 0 ? 0 : 1;  // the state handed to a reversed scan is not decayed first
    __syncthreads();
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const int i = threadIdx.x + 256 * j;
      *reinterpret_cast<u32x4*>(Ks + i / (4 * KB) * kPitchK + 8 * (i % (4 * KB))) = kn[j];
    }
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {
      const int i = threadIdx.x + 256 * j;
      *reinterpret_cast<u32x4*>(Vs + i / (8 * NB) * kPitchV + 8 * (i % (8 * NB))) = vn[j];
    }
    if (!STATE_ONLY) {
      // Q's columns in the order of an accumulator pair: column 16 t + 4 g' + k at 8 g' + 4 t + k of each 32.
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        uint16_t* at = Qs + (16 * wave + c16) * kPitchK + 32 * j + 16 * (g & 1) + 4 * (g >> 1);
        *reinterpret_cast<u32x2*>(at) = u32x2{qn[j].x, qn[j].y};
        *reinterpret_cast<u32x2*>(at + 8) = u32x2{qn[j].z, qn[j].w};
      }
    }
    __syncthreads();

    if (!STATE_ONLY) {
      // Scores of queries 16 wave + c16 (columns) with keys 16 kb + 4 g + r (rows).
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb <= wave) {
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < KB; ++j) s = mfma16x16x32(frag_k_cols(Ks, kPitchK, 16 * kb, 32 * j, lane), qn[j], s);
          const int diff = 16 * (wave - kb) + c16 - 4 * g;
#pragma unroll
          for (int r = 0; r < 4; ++r) s[r] = diff >= r ? s[r] * fast_exp2(g2 * (float)(diff - r)) : 0.f;
          uint16_t* at = Ps + (16 * wave + c16) * kPitchP + 32 * (kb >> 1) + 8 * g + 4 * (kb & 1);
          *reinterpret_cast<u32x2*>(at) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        } else if (kb == wave + 1 && (kb & 1)) {  // the pair's other half, read with it
          *reinterpret_cast<u32x2*>(Ps + (16 * wave + c16) * kPitchP + 32 * (kb >> 1) + 8 * g + 4) = u32x2{0u, 0u};
        }
      }
    }
    if (ci + 1 < chunks) load(STATE_ONLY ? t0 - kC : t0 + kC);

    u32x4 vf[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int kp = 0; kp < 2; ++kp)
        vf[nb][kp] = frag_k_rows_accpair(Vs, kPitchV, 32 * kp, 16 * (NB * wave + nb), lane);

    if (!STATE_ONLY) {
      f32x4 O[4][NB];
#pragma unroll
      for (int qb = 0; qb < 4; ++qb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) O[qb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        u32x4 sf[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const f32x4 x = S[nb][2 * j], y = S[nb][2 * j + 1];
          sf[nb] = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        }
#pragma unroll
        for (int qb = 0; qb < 4; ++qb) {
          const u32x4 qf = frag_k_cols(Qs, kPitchK, 16 * qb, 32 * j, lane);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) O[qb][nb] = mfma16x16x32(sf[nb], qf, O[qb][nb]);
        }
      }
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) {
        const float w = fast_exp2(g2 * (float)(16 * qb + c16 + lead));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) O[qb][nb] *= w;
      }
      __syncthreads();
#pragma unroll
      for (int qb = 0; qb < 4; ++qb)
#pragma unroll
        for (int kp = 0; kp <= qb / 2; ++kp) {
          const u32x4 pf = frag_k_cols(Ps, kPitchP, 16 * qb, 32 * kp, lane);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) O[qb][nb] = mfma16x16x32(vf[nb][kp], pf, O[qb][nb]);
        }
      // O^T: column c16 is the query, rows 4 g + r the value columns.
      const long low = p.start + (a.rev ? (long)p.len - (pos0 + t0) - n : (long)pos0 + t0);
      const int esz = a.o_f32 ? 4 : 2, orow = a.H * a.dv;
      const rsrc_t ro = make_rsrc(static_cast<char*>(a.o) + (low * orow + (long)h * a.dv) * esz, (uint32_t)(n * orow * esz));
#pragma unroll
      for (int qb = 0; qb < 4; ++qb) {
        const int r = 16 * qb + c16;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int dv = dv0 + 16 * (NB * wave + nb) + 4 * g;
          const uint32_t off = r < n && dv < a.dv ? (uint32_t)(((a.rev ? n - 1 - r : r) * orow + dv) * esz) : kOffNone;
          const f32x4 o = O[qb][nb] * a.scale;
          if (a.o_f32) buf_store16(__builtin_bit_cast(u32x4, o), ro, off);
          else buf_store8(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, ro, off);
        }
      }
    }

    // State: decay by the chunk, add K^T (weighted V). Token of slot s of pair kp: 32 kp + 16 (s / 4) + 4 g + s % 4.
    u32x4 hi[NB][2], lo[NB][2];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      float w[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) w[s] = fast_exp2(g2 * (float)(after + max(n - 1 - (32 * kp + 16 * (s >> 2) + 4 * g + (s & 3)), 0)));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float x = bf16_lo(vf[nb][kp][c]) * w[2 * c], y = bf16_hi(vf[nb][kp][c]) * w[2 * c + 1];
          const uint32_t top = pack_bf16x2(x, y);
          hi[nb][kp][c] = top;
          lo[nb][kp][c] = pack_bf16x2(x - bf16_lo(top), y - bf16_hi(top));
        }
    }
    const float keep = fast_exp2(g2 * (float)(n - 1 + lead));
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (!STATE_ONLY) S[nb][b] *= keep;
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const u32x4 kf = frag_k_rows_accpair(Ks, kPitchK, 32 * kp, 16 * b, lane);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          S[nb][b] = mfma16x16x32(kf, hi[nb][kp], S[nb][b]);
          S[nb][b] = mfma16x16x32(kf, lo[nb][kp], S[nb][b]);
        }
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
  if (dst) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int dv = dv0 + 16 * (NB * wave + nb) + c16;
#pragma unroll
      for (int b = 0; b < 2 * KB; ++b) {
        const int dk = 16 * b + 4 * g;
        if (dv < a.dv && dk < a.dk) *reinterpret_cast<f32x4*>(dst + (long)dv * a.dk + dk) = S[nb][b] * sc;
      }
    }
  }
}

template <int KB, int NB>
__global__ __launch_bounds__(256, KB <= 4 ? 2 : 1) void lin_mfma_kernel(LinScan a) {
  lin_mfma<KB, NB, false>(a, blockIdx.x, gridDim.x);
}

// The blocks' own sums of one scan, or of two: the first `na` workgroups are a's.
template <int KB, int NB>
__global__ __launch_bounds__(256, KB <= 4 ? 2 : 1) void lin_mfma_states_kernel(LinScan a, LinScan b, long na) {
  const bool first = (long)blockIdx.x < na;
  const LinScan& s = first ? a : b;
  lin_mfma<KB, NB, true>(s, first ? blockIdx.x : blockIdx.x - na, first ? na : gridDim.x - na);
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
    hipLaunchKernelGGL((lin_mfma_kernel<KB, NB>), dim3((unsigned)mfma_blocks<KB, NB>(a)), dim3(256), 0, stream, a);
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
    hipLaunchKernelGGL((lin_mfma_states_kernel<KB, NB>), dim3((unsigned)all), dim3(256), 0, stream, a, b ? *b : a, na);
  });
  return hipGetLastError();
}

}  // namespace ssd
