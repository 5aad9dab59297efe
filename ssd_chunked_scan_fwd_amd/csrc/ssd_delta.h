// ssd_delta.h -- internal interface of the gated delta rule's kernels.
//
// Per value head, with a = exp(log_decay) and S the state [dv][dk]:
//     u_t = beta_t (v_t - a_t S_{t-1} k_t),  S_t = a_t S_{t-1} + u_t k_t^T,  o_t = scale S_t q_t.
// Chunks of C tokens of one sequence, S0 the state before the chunk, G the log
// decays summed within it, D_ij = e^(G_i - G_j) for j <= i:
//     A_ij = beta_i D_ij k_i.k_j (j < i),  T = (I + A)^-1,  P = scale D o Q K^T
//     X = V - e^G (K S0^T),  U = T diag(beta) X
//     O = scale e^G (Q S0^T) + P U
//     S1 = e^(G_C) S0 + (e^(G_C - G) U)^T K.
// The adjoint, dS1 the gradient of S1 and U' that of U with all it leads to:
//     Y = P^T dO + e^(G_C - G) (K dS1^T),  U' = T^T Y,  dV = beta U'
//     dS0 = e^(G_C) dS1 + scale (e^G dO)^T Q - (e^G beta U')^T K.
// A first kernel makes T and P of every chunk (ssd_delta_prep.hip), a second
// walks the chunks of each sequence (ssd_delta_chain.hip), forwards or, for the
// gradients, forwards and then backwards; what the gradients take besides is made
// for all chunks at once (ssd_delta_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

struct DeltaArgs {
  const void *q = nullptr, *k = nullptr, *v = nullptr;   // element (token, head, i) at token * row + head * d + i
  long q_row = 0, k_row = 0, v_row = 0;
  const float *g = nullptr, *beta = nullptr;             // [tokens][H]; g null: no decay
  const int32_t* cu = nullptr;                           // packed sequence starts, or null
  int S = 0;                                             // packed sequences
  int batch = 1, T = 0, H = 0, Hk = 0, dk = 0, dv = 0;
  int bf16 = 0;
  float scale = 1.f;
  const float* init = nullptr;   // [nseq][H][dv][dk] or null for zero
  float* fin = nullptr;          // the state after the last token, or null
  void* o = nullptr;             // [tokens][H][dv]
  // Workspace. A sequence's chunks have consecutive slots, chunk c of packed
  // sequence s slot floor(cu[s] / C) + s + c, of row r slot r * slots_per_row + c.
  long slots_per_row = 0, slots = 0;
  float* gates = nullptr;        // [slots][H][kGateRows][C]
  float* tf = nullptr;           // T diag(beta) and
  void* pf = nullptr;            // P, operands (ssd_delta_tile.h)
  // Sequences cut into segments of `seg` chunks (0: not cut), numbered as chunks are, by which one long sequence
  // of few heads fills the card (ssd_delta_chain.hip).
  int seg = 0;
  long segs_per_row = 0, segs = 0;
  float* seg_states = nullptr;   // [segs][H][dv][dk]: a segment's own last state, then the state behind it
  float* seg_maps = nullptr;     // [segs][H][dk][dk]: what the segment makes of a state's row
  float* seg_adj = nullptr;      // [segs][H][dv][dk]: the gradient of the state before a segment, its own, then all of it
  // Gradients.
  float *tt = nullptr, *pt = nullptr;            // T^T and P^T, operands
  const void* d_o = nullptr;     // [tokens][H][dv]
  const float* dfin = nullptr;   // gradient of the last state, or null
  float* dinit = nullptr;        // of the first, or null
  void *dq = nullptr, *dk_out = nullptr, *dv_out = nullptr;   // contiguous
  float *dg = nullptr, *dbeta = nullptr;                      // [tokens][H]; dg may be null
  float *states = nullptr, *dstates = nullptr;   // [slots][H][dv][dk]: S0 and dS1 of every chunk
  float *u = nullptr, *ub = nullptr;             // [slots][H][C][dv]: U and U'
  int grad_heads = 1;            // value heads that a workgroup of the gradients takes
  float *part_q = nullptr, *part_k = nullptr;   // where heads share q and k: [tokens][H][dk], or with all of them in a
                                                // workgroup [tokens][Hk][dk]
};

// Tokens a chunk.
constexpr int delta_chunk(bool bf16) { return bf16 ? 64 : 32; }
// Bytes of a chunk's workspace arrays, of one head.
constexpr int kGateRows = 6;     // e^G, e^(G_C - G), beta, G as the sum of two floats, e^(G_C) (its first element)
size_t delta_gates_bytes(bool bf16);
size_t delta_tf_bytes(bool bf16);   // of T and the transposes, each
size_t delta_pf_bytes(bool bf16);

// Chunks a segment of a walk over these sizes, 0: no sequence is cut.
int delta_segment(int batch, int T, int S, int H, int dk, int dv, bool bf16);

int delta_prep_threads();
long delta_chain_blocks(const DeltaArgs& a);
long delta_segment_blocks(const DeltaArgs& a);   // of the segments' own states and maps
int delta_chain_threads();
int delta_grad_heads(long slots, int H, int Hk, int dk, bool bf16);
long delta_bwd_blocks(const DeltaArgs& a);
int delta_bwd_threads();

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t stream);
hipError_t launch_delta_fwd(const DeltaArgs& a, bool keep, hipStream_t stream);   // keep: states and u instead of o
hipError_t launch_delta_rev(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_grads(const DeltaArgs& a, hipStream_t stream);

struct DeltaStep {
  float* state = nullptr;        // [num_slots][H][dv][dk]
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  const float *g = nullptr, *beta = nullptr;
  const int32_t* slots = nullptr;
  void* o = nullptr;
  float scale = 1.f;
  int batch = 0, H = 0, Hk = 0, dk = 0, dv = 0, num_slots = 0, bf16 = 0;
};
hipError_t launch_delta_step(const DeltaStep& a, hipStream_t stream);

}  // namespace ssd
