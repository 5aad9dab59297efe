// ssd_lin_attn.hip -- linear attention with one fixed decay a head: the scan
// token by token (fp32 operands), the states passed between blocks of tokens,
// the sums over shared heads, and the one-token step on a pool of states.
#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

namespace {

template <bool BF16>
__device__ __forceinline__ float load_el(const void* p, long i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// ----------------------------------------------------------------------------
// The recurrence itself, token by token, for fp32 operands. A workgroup takes
// 16 rows of the state of one (block, head): 16 lanes a row, 4 NQ columns a lane,
// all in registers; the next 16 tokens are in flight while 16 are taken from LDS.
// Bound by its own arithmetic: 2 multiply-adds a state element for the decay
// (LinDecay), one for the product and one for the output.
// STATE_ONLY leaves each block's own sum (from a zero state) in a.states;
// the other form starts from the block's entering state and writes o. 256 tokens
// of 2 heads of 16 x 16: 8 + 3 + 16 us of three launches, 26 us a call (442 in
// plain operations). 16384 tokens of 32 heads of 128 x 128: 2300 us, the chain of
// 4096 tokens a block; backwards, 8192 tokens, three such scans, 3300.
// ----------------------------------------------------------------------------
constexpr int kRecRows = 16, kRecTok = 16, kC64 = 64;

template <int NQ, bool STATE_ONLY>
__global__ __launch_bounds__(256) void lin_rec_kernel(LinScan a) {
  constexpr int kCols = 64 * NQ, kPiecesT = kRecTok * kCols / 4 / 256;   // 16-byte pieces a thread stages
  __shared__ __align__(16) float ks[kRecTok][kCols], qs[STATE_ONLY ? 1 : kRecTok][STATE_ONLY ? 4 : kCols];
  __shared__ float vs[kRecTok][kRecRows];
  const int tiles = (a.dv + kRecRows - 1) / kRecRows;
  const long u = blockIdx.x;
  const int row0 = (int)(u % tiles) * kRecRows;
  const int h = (int)((u / tiles) % a.H);
  const long slot = u / ((long)tiles * a.H);
  const LinPiece p = lin_piece(a, slot);
  if (p.blk < 0) return;
  const int pos0 = p.blk * a.L;
  const int n = min(p.len - pos0, a.L);
  const bool last = pos0 + n >= p.len;
  if (STATE_ONLY && last) return;  // the scan carries the last block's state itself
  const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int row = row0 + r;
  const LinDecay lam = lin_decay(a.ld[h]);

  f32x4 s[NQ];  // columns 64 m + 4 c + 0..3
#pragma unroll
  for (int m = 0; m < NQ; ++m) s[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const long mat = (long)a.dv * a.dk;
  if (!STATE_ONLY) {
    const float* src = p.blk > 0 ? a.states + (slot * a.H + h) * mat : a.init;
    if (p.blk == 0 && src) src += ((long)p.seq * a.H + h) * mat;
    const bool tr = p.blk == 0 && a.init_tr;
    const float sc = p.blk == 0 ? a.init_scale : 1.f;
    if (src && row < a.dv) {
#pragma unroll
      for (int m = 0; m < NQ; ++m) {
        const int col = 64 * m + 4 * c;
        if (col >= a.dk) continue;
        if (tr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][i] = sc * src[(long)(col + i) * a.dv + row];
        } else {
          s[m] = *reinterpret_cast<const f32x4*>(src + (long)row * a.dk + col) * sc;
        }
      }
    }
  }

  f32x4 kn[kPiecesT], qn[kPiecesT];
  float vn;
  auto token = [&](int pos) { return p.start + (a.rev ? p.len - 1 - pos : pos); };
  auto load = [&](int t0) {
#pragma unroll
    for (int j = 0; j < kPiecesT; ++j) {
      const int i = threadIdx.x + 256 * j, t = i / (kCols / 4), col = 4 * (i % (kCols / 4));
      kn[j] = qn[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (t0 + t < n && col < a.dk) {
        const long tok = token(pos0 + t0 + t);
        kn[j] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.k.base) + tok * a.k.row + (long)(h / a.k.div) * a.dk + col);
        if (!STATE_ONLY)
          qn[j] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q.base) + tok * a.q.row + (long)(h / a.q.div) * a.dk + col);
      }
    }
    vn = 0.f;
    if (t0 + r < n && row0 + c < a.dv)
      vn = static_cast<const float*>(a.v.base)[token(pos0 + t0 + r) * a.v.row + (long)(h / a.v.div) * a.dv + row0 + c];
  };

  if (n > 0) load(0);
  for (int t0 = 0; t0 < n; t0 += kRecTok) {
    const int nt = min(kRecTok, n - t0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPiecesT; ++j) {
      const int i = threadIdx.x + 256 * j;
      *reinterpret_cast<f32x4*>(&ks[0][0] + 4 * i) = kn[j];
      if (!STATE_ONLY) *reinterpret_cast<f32x4*>(&qs[0][0] + 4 * i) = qn[j];
    }
    vs[r][c] = vn;
    __syncthreads();
    if (t0 + kRecTok < n) load(t0 + kRecTok);
    auto step = [&](int t) {
      const bool keep = a.rev && pos0 + t0 + t == 0;  // the state handed to a reversed scan is not decayed first
      const float hi = keep ? kOneHi : lam.hi, lo = keep ? kOneLo : lam.lo;
      const float v = vs[t][r];
      float part = 0.f;
#pragma unroll
      for (int m = 0; m < NQ; ++m) {
        const f32x4 k = *reinterpret_cast<const f32x4*>(&ks[t][64 * m + 4 * c]);
        f32x4 q = {0.f, 0.f, 0.f, 0.f};
        if (!STATE_ONLY) q = *reinterpret_cast<const f32x4*>(&qs[t][64 * m + 4 * c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[m][i] = fmaf(s[m][i], hi, fmaf(s[m][i], lo, v * k[i]));
          part = fmaf(s[m][i], q[i], part);
        }
      }
      if (!STATE_ONLY) {
        part = lanes_sum(part, 16) * a.scale;
        if (c == 0 && row < a.dv) static_cast<float*>(a.o)[(token(pos0 + t0 + t) * a.H + h) * a.dv + row] = part;
      }
    };
    if (nt == kRecTok) {
#pragma unroll 4
      for (int t = 0; t < kRecTok; ++t) step(t);
    } else {
      for (int t = 0; t < nt; ++t) step(t);
    }
  }

  float* dst = nullptr;
  float sc = 1.f;
  if (STATE_ONLY) {
    dst = a.states + (slot * a.H + h) * mat;
  } else if (last && a.fin) {
    dst = a.fin + ((long)p.seq * a.H + h) * mat;
    sc = a.fin_scale * (a.rev && p.len > 0 ? lam.hi + lam.lo : 1.f);
  }
  if (dst && row < a.dv) {
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
      const int col = 64 * m + 4 * c;
      if (col < a.dk) *reinterpret_cast<f32x4*>(dst + (long)row * a.dk + col) = s[m] * sc;
    }
  }
}

// ----------------------------------------------------------------------------
// Entering states: for blocks b = 0, 1, ... of a sequence, with own sums s_b,
// D = initial state; states[b] = D (b >= 1); D = lam^n_b D + s_b. Four
// elements a thread; kAhead blocks' sums are in flight at a time. Bound by the
// states' way through memory, read and written once: 32 heads of 128 x 128 in 16
// blocks, 63 MB, 13 us (4.9 TB/s). Folding it into the scan's start, each block
// summing those before it, took longer.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void lin_pass(const LinScan& a, int s) {
  const int h = blockIdx.y;
  const int mat = a.dv * a.dk;
  const int e = 4 * (int)(blockIdx.x * 256 + threadIdx.x);
  long slot0;
  int len;
  if (a.cu) {
    const int c0 = min(max(a.cu[s], 0), a.T), c1 = min(max(a.cu[s + 1], c0), a.T);
    slot0 = (long)c0 / a.L + s;
    len = c1 - c0;
  } else {
    slot0 = s * a.slots_per_row;
    len = a.T;
  }
  const int nb = (len + a.L - 1) / a.L;
  if (nb < 2 || e >= mat) return;
  f32x4 D = {0.f, 0.f, 0.f, 0.f};
  if (a.init) {
    const float* src = a.init + ((long)s * a.H + h) * mat;
    if (a.init_tr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) D[i] = src[(long)((e + i) % a.dk) * a.dv + (e + i) / a.dk] * a.init_scale;
    } else {
      D = *reinterpret_cast<const f32x4*>(src + e) * a.init_scale;
    }
  }
  // A block's decay is at least the smallest normal number, unless the head remembers nothing: an infinity
  // times a power that fp32 rounds to 0 would be a NaN.
  const float ld = a.ld[h], least = ld == -INFINITY ? 0.f : 0x1p-126f;
  auto decay = [&](int tokens) {
    const float w = (float)lin_power(ld, tokens);
    return w < least ? least : w;
  };
  const float w0 = decay(a.L - (a.rev ? 1 : 0)), w = decay(a.L);
  const long step = (long)a.H * mat;
  float* at = a.states + (slot0 * a.H + h) * mat + e;
  constexpr int kAhead = 8;
  f32x4 own = *reinterpret_cast<const f32x4*>(at);   // of block b0, before its place is taken by D
  for (int b0 = 0; b0 + 1 < nb; b0 += kAhead) {
    f32x4 next[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) next[k] = *reinterpret_cast<const f32x4*>(at + min(b0 + k + 1, nb - 1) * step);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int b = b0 + k + 1;
      D = D * (b == 1 ? w0 : w) + own;
      if (b < nb) *reinterpret_cast<f32x4*>(at + b * step) = D;
      own = next[k];
    }
  }
}

// One scan's states, or two scans' (of equal dv * dk) in the halves of grid.z.
__global__ __launch_bounds__(256) void lin_passing_kernel(LinScan a) { lin_pass(a, blockIdx.z); }
__global__ __launch_bounds__(256) void lin_passing2_kernel(LinScan a, LinScan b) {
  const int half = gridDim.z / 2;
  if ((int)blockIdx.z < half) lin_pass(a, blockIdx.z);
  else lin_pass(b, blockIdx.z - half);
}

// Sum over the heads that share a key head, eight values a thread, in head
// order: the gradients of keys (blockIdx.y = 0) and of values. Packed batches:
// tokens before the first and behind the last sequence are left as they were.
template <bool BF16>
__global__ __launch_bounds__(256) void lin_share_sum_kernel(LinShareSum a) {
  const int d = blockIdx.y ? a.dv : a.dk;
  const float* __restrict__ in = blockIdx.y ? a.in_v : a.in_k;
  void* __restrict__ out = blockIdx.y ? a.out_v : a.out_k;
  const int pieces = d >> 3;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * a.Hk * pieces) return;
  const int c = (int)(i % pieces);
  const long th = i / pieces;
  const long tok = th / a.Hk;
  const int hk = (int)(th % a.Hk), rep = a.H / a.Hk;
  if (a.cu && (tok < max(a.cu[0], 0) || tok >= min(a.cu[a.S], a.T))) return;
  const float* src = in + (tok * a.H + (long)hk * rep) * d + 8 * c;
  f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
  for (int j = 1; j < rep; ++j) {
    lo += *reinterpret_cast<const f32x4*>(src + (long)j * d);
    hi += *reinterpret_cast<const f32x4*>(src + (long)j * d + 4);
  }
  const long at = (tok * a.Hk + hk) * d + 8 * c;
  if constexpr (BF16) {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) =
        u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = lo;
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at + 4) = hi;
  }
}

// ----------------------------------------------------------------------------
// The one-token step: D = lam D + v k^T, o = scale D q, for the state of each
// entry's slot. The state's read and write bound it (2 dv dk 4 bytes a head): 64
// streams of 32 heads of 128 x 128, 271 MB, take 48.5 us (5.6 TB/s; a copy of
// that size reaches 5.45), non-temporal, as the states of a model's layers do not
// stay in the caches between two steps.
// A state row takes `tpr` lanes of four columns each (a power of two; lanes
// past dk / 4 idle), a thread ROWS rows; a workgroup one (entry, head, row
// range). Entries whose slot is outside the pool are padding: o = 0 and no
// state is touched. Entries that name the same slot are taken in the order of
// the batch: the first one's workgroup runs them all, so a stream may bring
// several tokens in one call and nothing is raced.
// ----------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* p, long i) {
  if constexpr (BF16) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
  } else {
    return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  }
}

template <bool BF16, int ROWS>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStep a, int tpr, int parts) {
  const int h = (int)(blockIdx.x / parts), part = (int)(blockIdx.x % parts);
  int e = blockIdx.y;
  const int hk = h / (a.H / a.Hk);
  const int c4 = threadIdx.x & (tpr - 1), rpp = 256 / tpr, lane = threadIdx.x & 63;
  const int r0 = part * ROWS * rpp + (int)threadIdx.x / tpr;
  const bool col_in = 4 * c4 < a.dk;
  const int slot = a.slots ? a.slots[e] : e;
  if (slot < 0 || slot >= a.num_slots) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = r0 + j * rpp;
      if (c4 == 0 && r < a.dv) {
        const long at = ((long)e * a.H + h) * a.dv + r;
        if (BF16) static_cast<uint16_t*>(a.o)[at] = 0;
        else static_cast<float*>(a.o)[at] = 0.f;
      }
    }
    return;
  }
  // Rows and columns past the ends read their nearest neighbour inside, and are not written.
  float* st = a.state + ((long)slot * a.H + h) * a.dv * a.dk + (col_in ? 4 * c4 : 0);
  f32x4 s[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    s[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(st + (long)min(r0 + j * rpp, a.dv - 1) * a.dk));
  const LinDecay lam = lin_decay(a.ld[h]);
  int next = a.batch;
  if (a.slots && step_peers(a.slots, a.batch, e, slot, lane, next)) return;  // an earlier entry's workgroup runs this one
  for (;;) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const long ek = (long)e * a.Hk + hk, eh = (long)e * a.H + h;
    f32x4 k = load4<BF16>(a.k, ek * a.dk + (col_in ? 4 * c4 : 0));
    f32x4 q = load4<BF16>(a.q, eh * a.dk + (col_in ? 4 * c4 : 0));
    float v[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) v[j] = load_el<BF16>(a.v, ek * a.dv + min(r0 + j * rpp, a.dv - 1));
    if (!col_in) k = q = zero;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = r0 + j * rpp;
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] = fmaf(s[j][i], lam.hi, fmaf(s[j][i], lam.lo, v[j] * k[i]));
        acc = fmaf(s[j][i], q[i], acc);
      }
      if (next == a.batch && col_in && r < a.dv)
        __builtin_nontemporal_store(s[j], reinterpret_cast<f32x4*>(st + (long)r * a.dk));
      acc = lanes_sum(col_in ? acc : 0.f, tpr) * a.scale;
      if (c4 == 0 && r < a.dv) {
        if (BF16) static_cast<uint16_t*>(a.o)[eh * a.dv + r] = f32_to_bf16(acc);
        else static_cast<float*>(a.o)[eh * a.dv + r] = acc;
      }
    }
    if (next == a.batch) break;
    e = next;
    step_peers(a.slots, a.batch, e, slot, lane, next);
  }
}

}  // namespace

// Sequences are cut so that the chip is filled, but every cut costs its state's
// way through memory, and the products k v^T a second time; and workgroups that
// do not fit at once cost a whole further round. So the number of blocks a
// sequence (of mean length, where packed) is the one of least cost, counted in
// chunks of 64 tokens: rounds of (chunks + start-up) each, times 1.45 for the
// blocks' own sums, plus the passing launch and the states' bytes. The times of a
// chunk were measured for heads of 128 x 128 and of 64 x 64. The host does not know
// the lengths of packed sequences: one long sequence among many short ones, whose
// mean needs no cut, is one block (16384 tokens and 15 single ones, 32 heads of 128
// x 128: 1060 us, the long one alone 210).
int lin_block_tokens(int batch, int T, int S, int H, int dk, int dv, int bf16, bool kv) {
  const long seqs = S > 0 ? S : batch;
  const int tile = kv ? dv : bf16 ? lin_mfma_tile(dv) : kRecRows;
  const long units = (long)H * ((dv + tile - 1) / tile) * seqs;
  const long fit = kv ? lin_kv_target(dk, dv) : bf16 ? lin_mfma_target(dk, dv) : 1024;   // workgroups that run at once
  const double start = bf16 ? 2.0 : 0.5, pass = bf16 ? 2.5 : 0.7;
  const double chunk_us = bf16 ? (dk > 64 && dv > 64 ? 7.0 : 2.5) : 6.4;
  const long len = ((long)T * batch + seqs - 1) / seqs, chunks = (len + kC64 - 1) / kC64;
  const double state = (double)seqs * H * dk * dv * 4 * 4 / 5e6 / chunk_us;   // four passes over a block's states, at 5 TB/s
  long best = chunks;
  double least = 0.0;
  for (long nb = 1; nb <= chunks && nb <= 512; ++nb) {
    const long c = (chunks + nb - 1) / nb, blocks = (chunks + c - 1) / c;
    const long rounds = (units * blocks + fit - 1) / fit;
    const double cost = (double)rounds * (double)(c + start) * (blocks > 1 ? 1.45 : 1.0) +
                        (blocks > 1 ? pass + (double)(blocks - 1) * state : 0.0);
    if (nb == 1 || cost < least) {
      least = cost;
      best = c;
    }
  }
  // One block a sequence: as long as the longest can be.
  if (best == chunks) return (int)(((long)T + kC64 - 1) / kC64 * kC64);
  return (int)(best * kC64);
}

int lin_slot_threads(int dv, int bf16, bool kv) {
  if (kv) return lin_kv_threads(dv);
  const int tile = bf16 ? lin_mfma_tile(dv) : kRecRows;
  return (bf16 ? 4 * tile : 256) * ((dv + tile - 1) / tile);
}

namespace {
template <bool STATE_ONLY>
void launch_rec(const LinScan& a, hipStream_t stream) {
  const long slots = a.S > 0 ? a.slots_per_row : a.slots_per_row * a.batch;
  const dim3 grid((unsigned)(slots * a.H * ((a.dv + kRecRows - 1) / kRecRows)));
  if (a.dk <= 64) hipLaunchKernelGGL((lin_rec_kernel<1, STATE_ONLY>), grid, dim3(256), 0, stream, a);
  else if (a.dk <= 128) hipLaunchKernelGGL((lin_rec_kernel<2, STATE_ONLY>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((lin_rec_kernel<4, STATE_ONLY>), grid, dim3(256), 0, stream, a);
}
}  // namespace

hipError_t launch_lin_states(const LinScan& a, const LinScan* b, hipStream_t stream) {
  if (b && !b->states) b = nullptr;
  if (!a.states) return b ? launch_lin_states(*b, nullptr, stream) : hipSuccess;
  if (a.bf16) {
    // The scan with the longer blocks first, so that the shorter ones fill the last round.
    const hipError_t e = b && b->L > a.L ? launch_lin_mfma_states(*b, &a, stream) : launch_lin_mfma_states(a, b, stream);
    if (e != hipSuccess) return e;
  } else {
    launch_rec<true>(a, stream);
    if (b) launch_rec<true>(*b, stream);
  }
  const unsigned seqs = (unsigned)(a.S > 0 ? a.S : a.batch);
  dim3 grid((unsigned)((a.dv * a.dk / 4 + 255) / 256), (unsigned)a.H, b ? 2 * seqs : seqs);
  if (b) hipLaunchKernelGGL(lin_passing2_kernel, grid, dim3(256), 0, stream, a, *b);
  else hipLaunchKernelGGL(lin_passing_kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_lin_outputs(const LinScan& a, hipStream_t stream) {
  if (a.bf16) return launch_lin_mfma(a, stream);
  launch_rec<false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_lin_scan(const LinScan& a, hipStream_t stream) {
  const hipError_t e = launch_lin_states(a, nullptr, stream);
  return e == hipSuccess ? launch_lin_outputs(a, stream) : e;
}

hipError_t launch_lin_share_sum(const LinShareSum& a, hipStream_t stream) {
  const long n = a.tokens * a.Hk * ((a.dk > a.dv ? a.dk : a.dv) / 8);
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (a.bf16) hipLaunchKernelGGL(lin_share_sum_kernel<true>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(lin_share_sum_kernel<false>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

namespace {
template <bool BF16>
void step_launch(const LinStep& a, int rows, int tpr, int parts, hipStream_t stream) {
  const dim3 grid((unsigned)(a.H * parts), (unsigned)a.batch);
  if (rows == 8) hipLaunchKernelGGL((lin_step_kernel<BF16, 8>), grid, dim3(256), 0, stream, a, tpr, parts);
  else if (rows == 4) hipLaunchKernelGGL((lin_step_kernel<BF16, 4>), grid, dim3(256), 0, stream, a, tpr, parts);
  else if (rows == 2) hipLaunchKernelGGL((lin_step_kernel<BF16, 2>), grid, dim3(256), 0, stream, a, tpr, parts);
  else hipLaunchKernelGGL((lin_step_kernel<BF16, 1>), grid, dim3(256), 0, stream, a, tpr, parts);
}
}  // namespace

hipError_t launch_lin_step(const LinStep& a, hipStream_t stream) {
  int tpr = 2;
  while (tpr * 4 < a.dk) tpr *= 2;
  const int rpp = 256 / tpr;
  // Rows a thread: as many (up to 8, the loads each thread keeps in flight) as
  // still leave two workgroups for every CU and as fewer would not cover dv with
  // less to spare. us with 8, 4, 2 and 1 rows a thread, heads of 128 x 128: 64 MB
  // of states 12.3, 13.0, 14.6, 19.4; 256 MB 48.7, 49.0, 46-49, 68; 1 GB 192, 189,
  // 207, 345; 144 MB in heads of 96 x 96, of which 8 cover 128 rows: 34.7, 29.7, 34.8, 54.
  auto parts_of = [&](int r) { return (a.dv + r * rpp - 1) / (r * rpp); };
  int rows = 8;
  while (rows > 1 && (parts_of(rows) * 2 > parts_of(rows / 2) || (long)a.batch * a.H * parts_of(rows) < 512)) rows /= 2;
  const int parts = parts_of(rows);
  if (a.bf16) step_launch<true>(a, rows, tpr, parts, stream);
  else step_launch<false>(a, rows, tpr, parts, stream);
  return hipGetLastError();
}

}  // namespace ssd
