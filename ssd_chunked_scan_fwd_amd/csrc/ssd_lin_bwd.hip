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
// anyway. Two VB waves; wave w owns value block w of R and dV, and dK's blocks of
// key columns (and, where there are fewer blocks than waves, of tokens) are
// dealt over the waves.
#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

namespace {

constexpr int kC = 64;
constexpr int kPitchP = lds_pitch(kC);

// Row order of an accumulator pair in each 32 columns: columns 8 g + 4 e + 0..3
// of a 16-byte piece g go to 16 (g & 1) + 8 e + 4 (g >> 1).
__device__ __forceinline__ void store_paired(uint16_t* row, int j, int g, u32x4 v) {
  uint16_t* at = row + 32 * j + 16 * (g & 1) + 4 * (g >> 1);
  *reinterpret_cast<u32x2*>(at) = u32x2{v.x, v.y};
  *reinterpret_cast<u32x2*>(at + 8) = u32x2{v.z, v.w};
}

// KB, VB: dk and dv in units of 32 (2 or 4).
template <int KB, int VB>
__global__ __launch_bounds__(128 * VB, 2) void lin_kv_kernel(LinScan a, LinOperand vop, void* dk_out) {
  constexpr int kWaves = 2 * VB, kThreads = 64 * kWaves;
  constexpr int kPitchK = lds_pitch(32 * KB), kPitchV = lds_pitch(32 * VB);
  __shared__ __align__(16) uint16_t Qs[kC * kPitchK], Gs[kC * kPitchV];   // q and dO
  __shared__ __align__(16) uint16_t Ks[kC * kPitchK], Vs[kC * kPitchV];   // k and v, columns in pair order
  __shared__ __align__(16) uint16_t Ps[2][kC * kPitchP];                  // weighted K Q^T and V dO^T
  __shared__ __align__(16) uint16_t Rs[32 * VB * kPitchK];                // R, rounded
  // Pieces of 16 bytes a thread stages of q and of dO.
  constexpr int kQ = kC * 4 * KB / kThreads, kG = kC * 4 * VB / kThreads;
  // Score blocks: with eight waves the first four take K Q^T and the others V dO^T,
  // with four each wave takes both.
  constexpr bool kSplit = kWaves == 8;
  // dK: blocks of 16 key columns a wave, and blocks of 16 tokens.
  constexpr int kDkBlocks = 2 * KB >= kWaves ? 2 * KB / kWaves : 1;
  constexpr int kDkTok = 2 * KB >= kWaves ? 4 : 4 * 2 * KB / kWaves;

  const long u = xcd_unit(blockIdx.x, gridDim.x);
  const int h = (int)(u % a.H);
  const long slot = u / a.H;
  const LinPiece p = lin_piece(a, slot);
  if (p.blk < 0) return;
  const int pos0 = p.blk * a.L;
  const int total = min(p.len - pos0, a.L);
  const bool last = pos0 + total >= p.len;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int qb0 = wave & 3;                       // token block whose scores this wave forms
  const bool do_k = !kSplit || wave < 4, do_v = !kSplit || wave >= 4;
  const int kb0 = 2 * KB >= kWaves ? wave * kDkBlocks : wave % (2 * KB);
  const int tb0 = 2 * KB >= kWaves ? 0 : wave / (2 * KB) * kDkTok;
  const float g2 = lin_log2_decay(a.ld, h);
  const long mat = (long)a.dv * a.dk;

  f32x4 R[2 * KB];   // dv = 16 wave + c16, dk = 16 b + 4 g + r
#pragma unroll
  for (int b = 0; b < 2 * KB; ++b) R[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int dvc = 16 * wave + c16;
  {
    const float* src = p.blk > 0 ? a.states + (slot * a.H + h) * mat : a.init;
    if (p.blk == 0 && src) src += ((long)p.seq * a.H + h) * mat;
    const float sc = p.blk == 0 ? a.init_scale : 1.f;
    if (src && dvc < a.dv) {
#pragma unroll
      for (int b = 0; b < 2 * KB; ++b)
        if (16 * b + 4 * g < a.dk) R[b] = *reinterpret_cast<const f32x4*>(src + (long)dvc * a.dk + 16 * b + 4 * g) * sc;
    }
  }

  u32x4 qn[kQ], gn[kG], kn[KB], vn[VB];
  auto load = [&](int t0) {
    const int n = min(kC, total - t0);
    const long low = p.start + (long)p.len - (pos0 + t0) - n;
    auto rows = [&](const LinOperand& x, int d) {
      return make_rsrc(static_cast<const uint16_t*>(x.base) + low * x.row + (long)(h / x.div) * d, (uint32_t)(n * x.row * 2));
    };
    auto offset = [&](const LinOperand& x, int r, int col, int d) {
      return r < n && col < d ? (uint32_t)(((n - 1 - r) * x.row + col) * 2) : kOffNone;
    };
    const rsrc_t rq = rows(a.k, a.dk), rg = rows(a.v, a.dv), rk = rows(a.q, a.dk), rv = rows(vop, a.dv);
#pragma unroll
    for (int j = 0; j < kQ; ++j) {
      const int i = threadIdx.x + kThreads * j;
      qn[j] = buf_load16(rq, offset(a.k, i / (4 * KB), 8 * (i % (4 * KB)), a.dk));
    }
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int i = threadIdx.x + kThreads * j;
      gn[j] = buf_load16(rg, offset(a.v, i / (4 * VB), 8 * (i % (4 * VB)), a.dv));
    }
    if (do_k) {
#pragma unroll
      for (int j = 0; j < KB; ++j) kn[j] = buf_load16(rk, offset(a.q, 16 * qb0 + c16, 32 * j + 8 * g, a.dk));
    }
    if (do_v) {
#pragma unroll
      for (int j = 0; j < VB; ++j) vn[j] = buf_load16(rv, offset(vop, 16 * qb0 + c16, 32 * j + 8 * g, a.dv));
    }
  };

  if (total > 0) load(0);
  for (int t0 = 0; t0 < total; t0 += kC) {
    const int n = min(kC, total - t0);
    const int lead = pos0 + t0 == 0 ? 0 : 1;  // the state handed in is not decayed before the last token
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQ; ++j) {
      const int i = threadIdx.x + kThreads * j;
      *reinterpret_cast<u32x4*>(Qs + i / (4 * KB) * kPitchK + 8 * (i % (4 * KB))) = qn[j];
    }
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      const int i = threadIdx.x + kThreads * j;
      *reinterpret_cast<u32x4*>(Gs + i / (4 * VB) * kPitchV + 8 * (i % (4 * VB))) = gn[j];
    }
    if (do_k) {
#pragma unroll
      for (int j = 0; j < KB; ++j) store_paired(Ks + (16 * qb0 + c16) * kPitchK, j, g, kn[j]);
    }
    if (do_v) {
#pragma unroll
      for (int j = 0; j < VB; ++j) store_paired(Vs + (16 * qb0 + c16) * kPitchV, j, g, vn[j]);
    }
    // R as an operand: in registers by pairs of blocks, and in LDS for the other contraction.
    u32x4 rf[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const f32x4 x = R[2 * j], y = R[2 * j + 1];
      rf[j] = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
      uint16_t* at = Rs + dvc * kPitchK + 32 * j + 4 * g;
      *reinterpret_cast<u32x2*>(at) = u32x2{rf[j].x, rf[j].y};
      *reinterpret_cast<u32x2*>(at + 16) = u32x2{rf[j].z, rf[j].w};
    }
    __syncthreads();

    // Scores: token j = 16 qb0 + c16 (columns) with tokens i = 16 kb + 4 g + r (rows).
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (kb <= qb0) {
        const int diff = 16 * (qb0 - kb) + c16 - 4 * g;
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = fast_exp2(g2 * (float)max(diff - r, 0));
        const int at = (16 * qb0 + c16) * kPitchP + 32 * (kb >> 1) + 8 * g + 4 * (kb & 1);
        auto put = [&](uint16_t* P, f32x4 s) {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[r] = diff >= r ? s[r] * w[r] : 0.f;
          *reinterpret_cast<u32x2*>(P + at) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        };
        if (do_k) {
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < KB; ++j) s = mfma16x16x32(frag_k_cols(Qs, kPitchK, 16 * kb, 32 * j, lane), kn[j], s);
          put(Ps[0], s);
        }
        if (do_v) {
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < VB; ++j) s = mfma16x16x32(frag_k_cols(Gs, kPitchV, 16 * kb, 32 * j, lane), vn[j], s);
          put(Ps[1], s);
        }
      } else if (kb == qb0 + 1 && (kb & 1)) {  // the pair's other half, read with it
        const int at = (16 * qb0 + c16) * kPitchP + 32 * (kb >> 1) + 8 * g + 4;
        if (do_k) *reinterpret_cast<u32x2*>(Ps[0] + at) = u32x2{0u, 0u};
        if (do_v) *reinterpret_cast<u32x2*>(Ps[1] + at) = u32x2{0u, 0u};
      }
    }
    if (t0 + kC < total) load(t0 + kC);

    // Terms of R: dV^T (rows: value block of this wave) and dK^T (rows: its key blocks).
    f32x4 OV[4], OK[kDkBlocks][kDkTok];
#pragma unroll
    for (int qb = 0; qb < 4; ++qb) {
      OV[qb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KB; ++j) OV[qb] = mfma16x16x32(rf[j], frag_k_cols(Ks, kPitchK, 16 * qb, 32 * j, lane), OV[qb]);
    }
#pragma unroll
    for (int b = 0; b < kDkBlocks; ++b)
#pragma unroll
      for (int t = 0; t < kDkTok; ++t) OK[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VB; ++j) {
      u32x4 rt[kDkBlocks];
#pragma unroll
      for (int b = 0; b < kDkBlocks; ++b) rt[b] = frag_k_rows_accpair(Rs, kPitchK, 32 * j, 16 * (kb0 + b), lane);
#pragma unroll
      for (int t = 0; t < kDkTok; ++t) {
        const u32x4 vf = frag_k_cols(Vs, kPitchV, 16 * (tb0 + t), 32 * j, lane);
#pragma unroll
        for (int b = 0; b < kDkBlocks; ++b) OK[b][t] = mfma16x16x32(rt[b], vf, OK[b][t]);
      }
    }
#pragma unroll
    for (int qb = 0; qb < 4; ++qb) OV[qb] *= fast_exp2(g2 * (float)(16 * qb + c16 + lead));
#pragma unroll
    for (int t = 0; t < kDkTok; ++t) {
      const float w = fast_exp2(g2 * (float)(16 * (tb0 + t) + c16 + lead));
#pragma unroll
      for (int b = 0; b < kDkBlocks; ++b) OK[b][t] *= w;
    }
    u32x4 gf[2];   // dO^T of this wave's value block
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) gf[kp] = frag_k_rows_accpair(Gs, kPitchV, 32 * kp, 16 * wave, lane);
    __syncthreads();

    // Terms of the chunk's own tokens.
#pragma unroll
    for (int qb = 0; qb < 4; ++qb)
#pragma unroll
      for (int kp = 0; kp <= qb / 2; ++kp)
        OV[qb] = mfma16x16x32(gf[kp], frag_k_cols(Ps[0], kPitchP, 16 * qb, 32 * kp, lane), OV[qb]);
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      u32x4 qf[kDkBlocks];
#pragma unroll
      for (int b = 0; b < kDkBlocks; ++b) qf[b] = frag_k_rows_accpair(Qs, kPitchK, 32 * kp, 16 * (kb0 + b), lane);
#pragma unroll
      for (int t = 0; t < kDkTok; ++t) {
        if (kp > (tb0 + t) / 2) continue;
        const u32x4 pf = frag_k_cols(Ps[1], kPitchP, 16 * (tb0 + t), 32 * kp, lane);
#pragma unroll
        for (int b = 0; b < kDkBlocks; ++b) OK[b][t] = mfma16x16x32(qf[b], pf, OK[b][t]);
      }
    }

    const long low = p.start + (long)p.len - (pos0 + t0) - n;
    const int esz = a.o_f32 ? 4 : 2;
    auto put = [&](void* out, int d, int tok, int col, f32x4 v) {
      const int row = a.H * d;
      const rsrc_t ro = make_rsrc(static_cast<char*>(out) + (low * row + (long)h * d) * esz, (uint32_t)(n * row * esz));
      const uint32_t off = tok < n && col < d ? (uint32_t)(((n - 1 - tok) * row + col) * esz) : kOffNone;
      const f32x4 o = v * a.scale;
      if (a.o_f32) buf_store16(__builtin_bit_cast(u32x4, o), ro, off);
      else buf_store8(u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])}, ro, off);
    };
#pragma unroll
    for (int qb = 0; qb < 4; ++qb) put(a.o, a.dv, 16 * qb + c16, 16 * wave + 4 * g, OV[qb]);
#pragma unroll
    for (int t = 0; t < kDkTok; ++t)
#pragma unroll
      for (int b = 0; b < kDkBlocks; ++b) put(dk_out, a.dk, 16 * (tb0 + t) + c16, 16 * (kb0 + b) + 4 * g, OK[b][t]);

    // R: decay by the chunk, add Q^T (weighted dO), dO's weighted values as two bf16 values each.
    u32x4 hi[2], lo[2];
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      float w[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) w[s] = fast_exp2(g2 * (float)max(n - 1 - (32 * kp + 16 * (s >> 2) + 4 * g + (s & 3)), 0));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = bf16_lo(gf[kp][c]) * w[2 * c], y = bf16_hi(gf[kp][c]) * w[2 * c + 1];
        hi[kp][c] = pack_bf16x2(x, y);
        lo[kp][c] = pack_bf16x2(x - bf16_lo(hi[kp][c]), y - bf16_hi(hi[kp][c]));
      }
    }
    const float keep = fast_exp2(g2 * (float)(n - 1 + lead));
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      R[b] *= keep;
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const u32x4 qf = frag_k_rows_accpair(Qs, kPitchK, 32 * kp, 16 * b, lane);
        R[b] = mfma16x16x32(qf, hi[kp], R[b]);
        R[b] = mfma16x16x32(qf, lo[kp], R[b]);
      }
    }
  }

  if (last && a.fin && dvc < a.dv) {
    const float sc = a.fin_scale * (p.len > 0 ? fast_exp2(g2) : 1.f);
    float* dst = a.fin + ((long)p.seq * a.H + h) * mat;
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b)
      if (16 * b + 4 * g < a.dk) *reinterpret_cast<f32x4*>(dst + (long)dvc * a.dk + 16 * b + 4 * g) = R[b] * sc;
  }
}

}  // namespace

bool lin_kv_supported(int dk, int dv, int bf16) { return bf16 && dk <= 128 && dv <= 128; }

// Workgroups that fill the chip: two of four waves a CU, or one of eight.
int lin_kv_target(int dv) { return dv <= 64 ? 512 : 256; }

hipError_t launch_lin_kv(const LinScan& a, const LinOperand& v, void* dk_out, hipStream_t stream) {
  const long slots = a.S > 0 ? a.slots_per_row : a.slots_per_row * a.batch;
  const dim3 grid((unsigned)(slots * a.H));
  if (a.dv <= 64) {
    if (a.dk <= 64) hipLaunchKernelGGL((lin_kv_kernel<2, 2>), grid, dim3(256), 0, stream, a, v, dk_out);
    else hipLaunchKernelGGL((lin_kv_kernel<4, 2>), grid, dim3(256), 0, stream, a, v, dk_out);
  } else {
    if (a.dk <= 64) hipLaunchKernelGGL((lin_kv_kernel<2, 4>), grid, dim3(512), 0, stream, a, v, dk_out);
    else hipLaunchKernelGGL((lin_kv_kernel<4, 4>), grid, dim3(512), 0, stream, a, v, dk_out);
  }
  return hipGetLastError();
}

}  // namespace ssd
