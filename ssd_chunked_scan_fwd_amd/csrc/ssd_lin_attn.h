// ssd_lin_attn.h -- internal interface of the linear-attention kernels
// (one fixed decay a head): the scan over prompts and the one-token step.
//
// A scan computes, for every head of every sequence,
//     D_t = lam D_{t-1} + v_t k_t^T,   o_t = scale D_t q_t,   D [dv][dk],
// over the tokens in order or, reversed, from each sequence's last token to
// its first. The backward pass is three scans with the roles exchanged:
//     dq: forwards, q := do, k := v, v := k, from the transposed initial state;
//     dv: reversed, q := k, k := q, v := do, from dfinal;
//     dk: reversed, q := v, k := do, v := q, from the transposed dfinal.
// In a reversed scan the state handed in is added where the last token's own
// product is (L_T = scale do_T q_T^T + dfinal), so it is not decayed before
// that token; `lead` below is 0 there and 1 in a forward scan.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// One operand: element (token, head, i) at base + token * row + (head / div) * d + i.
struct LinOperand {
  const void* base = nullptr;
  long row = 0;
  int div = 1;
};

struct LinScan {
  LinOperand q, k, v;
  void* o = nullptr;           // [tokens][H][dv], bf16 or fp32
  int o_f32 = 0;               // bf16 operands only: write o in fp32 (partials summed over shared heads)
  const float* ld = nullptr;   // [H] natural log decay
  float scale = 1.f;
  const float* init = nullptr; // [nseq][H] matrices, or null for zero
  float init_scale = 1.f;
  int init_tr = 0;             // the matrices are [dk][dv] instead of [dv][dk]
  float* fin = nullptr;        // [nseq][H][dv][dk] or null: the state after the last token,
  float fin_scale = 1.f;       //   times this,
  int rev = 0;                 //   and in a reversed scan of at least one token times lam
  const int32_t* cu = nullptr; // packed sequence starts, or null
  int S = 0;                   // packed sequences
  int batch = 1, T = 0, H = 0; // rows, tokens a row, heads
  int dk = 0, dv = 0;          // this scan's contraction and value sizes
  int bf16 = 0;
  int q_once = 0;              // no later launch of the call reads q's rows
  bool fine() const { return fin != nullptr; }   // the state is an fp32 result: carry it in full
  // Sequences are cut into blocks of L tokens (from the end in a reversed
  // scan); block b of packed sequence s has slot floor(cu[s] / L) + s + b, of
  // row r slot r * slots_per_row + b. A sequence without tokens has one block.
  int L = 0;
  long slots_per_row = 0;
  float* states = nullptr;     // [slots][H][dv][dk]: each block's own sum, then its entering state
};

// Tokens a block for a scan of these sizes (kv: the scan of launch_lin_kv); a
// value >= T means that no sequence is cut and no block states are needed.
int lin_block_tokens(int batch, int T, int S, int H, int dk, int dv, int bf16, bool kv = false);
// Threads of a launch for one block of one head.
int lin_slot_threads(int dv, int bf16, bool kv);
inline long lin_slots_per_row(int T, int S, int L) { return S > 0 ? (long)(T / L) + S : (T + (long)L - 1) / L; }

hipError_t launch_lin_scan(const LinScan& a, hipStream_t stream);
// The two parts of it: the states that enter the blocks (nothing without
// a.states), for one scan or for two at once, and the outputs.
hipError_t launch_lin_states(const LinScan& a, const LinScan* b, hipStream_t stream);
hipError_t launch_lin_outputs(const LinScan& a, hipStream_t stream);

// bf16 operands: the scan on matrix instructions (ssd_lin_scan.hip), either the
// blocks' own sums or, from the entering states, the outputs.
int lin_mfma_tile(int dv);
int lin_mfma_target(int dk, int dv);   // workgroups that run at once
hipError_t launch_lin_mfma(const LinScan& a, hipStream_t stream);
hipError_t launch_lin_mfma_states(const LinScan& a, const LinScan* b, hipStream_t stream);

// dk and dv of the backward pass in one reversed scan, bf16, dk and dv up to
// 128 (ssd_lin_bwd.hip): `a` is the scan for dv; `v` and `dk_out` are what dk
// takes besides.
bool lin_kv_supported(int dk, int dv, int bf16);
int lin_kv_target(int dk, int dv);
int lin_kv_threads(int dv);   // of a workgroup
hipError_t launch_lin_kv(const LinScan& a, const LinOperand& v, void* dk_out, hipStream_t stream);

// out[token][key head][i] = sum of in over the query heads that share it, in
// head order, for keys (size dk) and values (dv).
struct LinShareSum {
  const float *in_k = nullptr, *in_v = nullptr;
  void *out_k = nullptr, *out_v = nullptr;
  const int32_t* cu = nullptr;
  long tokens = 0;
  int S = 0, T = 0, H = 0, Hk = 0, dk = 0, dv = 0, bf16 = 0;
};
hipError_t launch_lin_share_sum(const LinShareSum& a, hipStream_t stream);

struct LinStep {
  float* state = nullptr;      // [num_slots][H][dv][dk]
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  const float* ld = nullptr;
  const int32_t* slots = nullptr;
  void* o = nullptr;
  float scale = 1.f;
  int batch = 0, H = 0, Hk = 0, dk = 0, dv = 0, num_slots = 0, bf16 = 0;
};
hipError_t launch_lin_step(const LinStep& a, hipStream_t stream);

#ifdef __HIPCC__

// ---- device side ----------------------------------------------------------

struct LinPiece {
  int seq;     // sequence
  int blk;     // block in the sequence, -1: the slot holds no block
  int len;     // tokens of the sequence
  long start;  // its first token, flattened over rows
};

// The sequence and block of a slot: rows or packed sequences (cu, S of them) of T
// tokens in all, cut into blocks of L. cu's entries are brought into [0, T] and
// into order, so that no content of cu leads outside the tensors. Every lane of
// the calling wave must be active; all receive the same answer.
__device__ __forceinline__ LinPiece lin_piece(const int32_t* cu, int S, int T, int L, long slots_per_row, long slot) {
  LinPiece p;
  if (!cu) {
    p.seq = (int)(slot / slots_per_row);
    p.blk = (int)(slot % slots_per_row);
    p.len = T;
    p.start = (long)p.seq * T;
    return p;
  }
  // Slots of sequence s begin at floor(cu[s] / L) + s, which grows with s: count those at or before `slot`,
  // halving the range down to a wave's width, the rest with one load a lane.
  const int lane = (int)threadIdx.x & 63;
  auto begins = [&](int i) { return (long)min(max(cu[i], 0), T) / L + i; };
  int lo = 0, hi = S;
  while (hi - lo > 64) {
    const int mid = __builtin_amdgcn_readfirstlane((lo + hi) / 2);
    if (begins(mid) <= slot) lo = mid;
    else hi = mid;
  }
  const bool in = lo + lane < hi && begins(lo + lane) <= slot;
  const int n = lo + __popcll(__ballot(in));
  p.seq = __builtin_amdgcn_readfirstlane(n - 1);
  if (p.seq < 0) {
    p.seq = 0;
    p.blk = -1;
    p.len = 0;
    p.start = 0;
    return p;
  }
  const int c0 = min(max(cu[p.seq], 0), T);
  const int c1 = min(max(cu[p.seq + 1], c0), T);
  p.start = c0;
  p.len = c1 - c0;
  const long b = slot - ((long)c0 / L + p.seq);
  p.blk = b >= 0 && (b == 0 || b * L < p.len) ? (int)b : -1;
  return p;
}
__device__ __forceinline__ LinPiece lin_piece(const LinScan& a, long slot) {
  return lin_piece(a.cu, a.S, a.T, a.L, a.slots_per_row, slot);
}

// lam^e in 64 bits (a log decay of -inf: 0 for e > 0, 1 for e = 0).
__device__ __forceinline__ double lin_power(float log_decay, int e) {
  return exp((double)(log_decay < -11356.f ? -11356.f : log_decay) * (double)e);
}

// lam as a sum of two floats: rounded to one, the same error would enter with
// every token and compound. Both are above 0 (unless lam is 0): an infinity in
// a state times a low part of 0 or below would be, or end in, a NaN.
struct LinDecay {
  float hi, lo;
};
constexpr float kOneHi = 1.f - 0x1p-24f, kOneLo = 0x1p-24f;   // 1, for a token that is not decayed
__device__ __forceinline__ LinDecay lin_split(double lam) {
  float hi = (float)lam;
  if ((double)hi >= lam && hi > 0.f) hi = __uint_as_float(__float_as_uint(hi) - 1);   // the nearest float below
  return LinDecay{hi, (float)(lam - (double)hi)};
}
__device__ __forceinline__ LinDecay lin_decay(float log_decay) { return lin_split(lin_power(log_decay, 1)); }

// The one-token steps. Whether an earlier entry names entry e's slot, and the next
// entry that does (batch if none). Each wave looks for itself: no barrier stands
// between the state's loads and their use.
__device__ __forceinline__ bool step_peers(const int32_t* slots, int batch, int e, int slot, int lane, int& next) {
  next = batch;
  bool before = false;
  for (int i0 = 0; i0 < batch; i0 += 64) {
    const int i = i0 + lane;
    const bool same = i < batch && i != e && slots[i] == slot;
    before |= __ballot(same && i < e) != 0;
    const unsigned long long later = __ballot(same && i > e);
    if (later && next == batch) next = i0 + __builtin_ctzll(later);
  }
  return before;
}

#endif

}  // namespace ssd
