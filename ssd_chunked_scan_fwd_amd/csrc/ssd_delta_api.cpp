// ssd_delta_api.cpp -- the C ABI (include/ssd.h) of the gated delta rule and of
// rotary positions. As in ssd_api.cpp, every argument is checked on the host
// before any HIP call; nothing is allocated, synchronised or thrown.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "ssd.h"
#include "ssd_api_check.h"
#include "ssd_delta.h"
#include "ssd_layer.h"
#include "ssd_lin_attn.h"

namespace {

// ---------------------------------------------------------------- gated delta rule

struct DeltaDims {
  int64_t q_row, k_row, v_row, tokens, nseq, spr, slots, segs_per_row, segs;
  int grad_heads;
  int esz, seg;
};

ssd_status check_delta_heads(const ssd_delta_shape* s) {
  if (!s) return SSD_ERR_INVALID_ARGUMENT;
  if (s->nheads < 1 || s->nqk_heads < 1 || s->dk < 1 || s->dv < 1 || s->batch < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->nheads % s->nqk_heads) return SSD_ERR_INVALID_ARGUMENT;
  if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->dk % 8 || s->dv % 8 || s->dk > 256 || s->dv > 256) return SSD_ERR_UNSUPPORTED;
  if (s->nheads > 65535 || s->batch > 65535) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd::DeltaArgs delta_args(const ssd_delta_shape* s, const DeltaDims& d) {
  ssd::DeltaArgs a;
  a.q_row = (long)d.q_row;
  a.k_row = (long)d.k_row;
  a.v_row = (long)d.v_row;
  a.S = s->num_seqs;
  a.batch = s->batch;
  a.T = s->seqlen;
  a.H = s->nheads;
  a.Hk = s->nqk_heads;
  a.dk = s->dk;
  a.dv = s->dv;
  a.bf16 = s->dtype == SSD_DTYPE_BF16;
  a.slots_per_row = (long)d.spr;
  a.slots = (long)d.slots;
  a.seg = d.seg;
  a.grad_heads = d.grad_heads;
  a.segs_per_row = (long)d.segs_per_row;
  a.segs = (long)d.segs;
  return a;
}

ssd_status check_delta(const ssd_delta_shape* s, DeltaDims* d, bool backward) {
  ssd_status st = check_delta_heads(s);
  if (st != SSD_OK) return st;
  if (s->seqlen < 1 || s->num_seqs < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > 0 && s->batch != 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > 65535) return SSD_ERR_UNSUPPORTED;
  d->esz = s->dtype == SSD_DTYPE_BF16 ? 2 : 4;
  const int64_t qk = (int64_t)s->nqk_heads * s->dk, vs = (int64_t)s->nheads * s->dv;
  d->q_row = s->q_row ? s->q_row : qk;
  d->k_row = s->k_row ? s->k_row : qk;
  d->v_row = s->v_row ? s->v_row : vs;
  if (d->q_row < qk || d->k_row < qk || d->v_row < vs) return SSD_ERR_INVALID_ARGUMENT;
  // rows start on 16-byte boundaries
  if ((d->q_row | d->k_row | d->v_row) * d->esz % 16) return SSD_ERR_UNSUPPORTED;
  // 64 rows are addressed as one buffer range of fewer than 2^31 bytes
  const int64_t most = INT32_MAX / 64 / 4;
  if (d->q_row > most || d->k_row > most || d->v_row > most || vs > most || (int64_t)s->nheads * s->dk > most)
    return SSD_ERR_UNSUPPORTED;
  d->tokens = (int64_t)s->batch * s->seqlen;
  if (d->tokens > INT32_MAX / 2) return SSD_ERR_UNSUPPORTED;
  d->nseq = s->num_seqs > 0 ? s->num_seqs : s->batch;
  const int C = ssd::delta_chunk(s->dtype == SSD_DTYPE_BF16);
  d->spr = ssd::lin_slots_per_row(s->seqlen, s->num_seqs, C);
  d->slots = s->num_seqs > 0 ? d->spr : d->spr * s->batch;
  d->grad_heads = ssd::delta_grad_heads(d->slots, s->nheads, s->nqk_heads, s->dk, s->dtype == SSD_DTYPE_BF16);
  d->seg = ssd::delta_segment(s->batch, s->seqlen, s->num_seqs, s->nheads, s->dk, s->dv, s->dtype == SSD_DTYPE_BF16);
  d->segs_per_row = d->seg ? ssd::lin_slots_per_row(s->seqlen, s->num_seqs, d->seg * C) : 0;
  d->segs = s->num_seqs > 0 ? d->segs_per_row : d->segs_per_row * s->batch;
  const ssd::DeltaArgs a = delta_args(s, *d);
  if (!ssd::launchable(a.slots * a.Hk, ssd::delta_prep_threads()) ||
      !ssd::launchable(ssd::delta_chain_blocks(a), ssd::delta_chain_threads()) ||
      !ssd::launchable(ssd::delta_segment_blocks(a), ssd::delta_chain_threads()))
    return SSD_ERR_UNSUPPORTED;
  if (backward && (!ssd::launchable(ssd::delta_bwd_blocks(a), ssd::delta_bwd_threads()) ||
                   !ssd::launchable(d->tokens * s->nqk_heads * (s->dk / 8) / 256 + 1, 256)))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

struct DeltaLayout {
  size_t gates, tf, pf, seg_states, seg_maps, seg_adj, tt, pt, states, dstates, u, ub, part_q, part_k, total;
};
DeltaLayout delta_layout(const ssd_delta_shape* s, const DeltaDims& d, bool backward) {
  DeltaLayout L{};
  const bool bf16 = s->dtype == SSD_DTYPE_BF16, shared = s->nheads != s->nqk_heads;
  const size_t units = (size_t)d.slots * s->nheads, mat = (size_t)s->dk * s->dv * 4;
  const size_t rows = (size_t)ssd::delta_chunk(bf16) * s->dv * 4, part = (size_t)d.tokens * (d.grad_heads > 1 ? s->nqk_heads : s->nheads) * s->dk * 4;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off = align256(off + b);
    return o;
  };
  L.gates = take(units * ssd::delta_gates_bytes(bf16));
  L.tf = take(units * ssd::delta_tf_bytes(bf16));
  L.seg_states = take((size_t)d.segs * s->nheads * mat);
  L.seg_maps = take((size_t)d.segs * s->nheads * s->dk * s->dk * 4);
  if (!backward) {
    L.pf = take(units * ssd::delta_pf_bytes(bf16));
  } else {
    L.seg_adj = take((size_t)d.segs * s->nheads * mat);
    L.tt = take(units * ssd::delta_tf_bytes(bf16));
    L.pt = take(units * ssd::delta_tf_bytes(bf16));
    L.states = take(units * mat);
    L.dstates = take(units * mat);
    L.u = take(units * rows);
    L.ub = take(units * rows);
    L.part_q = take(shared ? part : 0);
    L.part_k = take(shared ? part : 0);
  }
  L.total = off;
  return L;
}

// The memory of a call's tensors.
struct DeltaSpans {
  const ssd_delta_shape* s;
  DeltaDims d;
  DeltaSpans(const ssd_delta_shape* shape, const DeltaDims& dims) : s(shape), d(dims) {}
  Span rows(const void* p, int64_t row, int64_t heads, int64_t size) const {
    return Span{p, d.tokens, row * d.esz, heads * size * d.esz};
  }
  Span q(const void* p) const { return rows(p, d.q_row, s->nqk_heads, s->dk); }
  Span k(const void* p) const { return rows(p, d.k_row, s->nqk_heads, s->dk); }
  Span v(const void* p) const { return rows(p, d.v_row, s->nheads, s->dv); }
  Span keys(const void* p) const { return whole(p, d.tokens * s->nqk_heads * s->dk * d.esz); }
  Span values(const void* p) const { return whole(p, d.tokens * s->nheads * s->dv * d.esz); }
  Span gates(const void* p) const { return whole(p, d.tokens * s->nheads * 4); }
  Span starts(const void* p) const { return whole(p, s->num_seqs > 0 ? (d.nseq + 1) * 4 : 0); }
  Span state(const void* p) const { return whole(p, d.nseq * s->nheads * s->dk * s->dv * 4); }
};

bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

// ---------------------------------------------------------------- rotary positions

// Whether two sets of rows share a byte; sets of different pitch count as sharing where their ranges do.
bool rows_meet(const Span& a, const Span& b) {
  if (!a.base || !b.base) return false;
  const uintptr_t a0 = (uintptr_t)a.base, b0 = (uintptr_t)b.base;
  const uintptr_t a1 = a0 + (uintptr_t)((a.rows - 1) * a.pitch + a.width), b1 = b0 + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t p = a.pitch, shift = (((int64_t)(b0 - a0)) % p + p) % p;
  return shift < a.width || p - shift < b.width;
}

}  // namespace

extern "C" {

ssd_status ssd_gated_delta_workspace_bytes(const ssd_delta_shape* shape, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  DeltaDims d;
  const ssd_status st = check_delta(shape, &d, false);
  if (st == SSD_OK) *bytes = delta_layout(shape, d, false).total;
  return st;
}

ssd_status ssd_gated_delta_bwd_workspace_bytes(const ssd_delta_shape* shape, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  DeltaDims d;
  const ssd_status st = check_delta(shape, &d, true);
  if (st == SSD_OK) *bytes = delta_layout(shape, d, true).total;
  return st;
}

ssd_status ssd_gated_delta_fwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const int32_t* cu_seqlens, float scale, const float* initial_state, void* o,
                               float* final_state, const ssd_delta_shape* shape, void* workspace, size_t workspace_bytes,
                               void* stream) {
  DeltaDims d;
  ssd_status st = check_delta(shape, &d, false);
  if (st != SSD_OK) return st;
  if (!q || !k || !v || !beta || !o || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if ((cu_seqlens != nullptr) != (shape->num_seqs > 0)) return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned4(log_decay) || !aligned4(beta) || !aligned4(cu_seqlens)) return SSD_ERR_INVALID_ARGUMENT;
  const DeltaLayout L = delta_layout(shape, d, false);
  if ((st = check_ws(workspace, workspace_bytes, L.total)) != SSD_OK) return st;
  const DeltaSpans t(shape, d);
  if (overlap({t.values(o), t.state(final_state), whole(workspace, (int64_t)L.total)},
              {t.q(q), t.k(k), t.v(v), t.gates(log_decay), t.gates(beta), t.state(initial_state), t.starts(cu_seqlens)}))
    return SSD_ERR_INVALID_ARGUMENT;
  char* ws = static_cast<char*>(workspace);
  ssd::DeltaArgs a = delta_args(shape, d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = log_decay;
  a.beta = beta;
  a.cu = cu_seqlens;
  a.scale = scale;
  a.init = initial_state;
  a.fin = final_state;
  a.o = o;
  a.gates = reinterpret_cast<float*>(ws + L.gates);
  a.tf = reinterpret_cast<float*>(ws + L.tf);
  a.pf = ws + L.pf;
  a.seg_states = reinterpret_cast<float*>(ws + L.seg_states);
  a.seg_maps = reinterpret_cast<float*>(ws + L.seg_maps);
  const hipError_t e = ssd::launch_delta_prep(a, false, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(ssd::launch_delta_fwd(a, false, (hipStream_t)stream));
}

ssd_status ssd_gated_delta_bwd(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                               const int32_t* cu_seqlens, float scale, const float* initial_state, const void* d_o,
                               const float* dfinal_state, void* dq, void* dk, void* dv, float* dlog_decay, float* dbeta,
                               float* dinitial_state, const ssd_delta_shape* shape, void* workspace,
                               size_t workspace_bytes, void* stream) {
  DeltaDims d;
  ssd_status st = check_delta(shape, &d, true);
  if (st != SSD_OK) return st;
  if (!q || !k || !v || !beta || !d_o || !dq || !dk || !dv || !dbeta || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if ((cu_seqlens != nullptr) != (shape->num_seqs > 0)) return SSD_ERR_INVALID_ARGUMENT;
  for (const void* t : {q, k, v, d_o, (const void*)initial_state, (const void*)dfinal_state, (const void*)dq, (const void*)dk,
                        (const void*)dv, (const void*)dinitial_state})
    if (!aligned16(t)) return SSD_ERR_INVALID_ARGUMENT;
  for (const void* t : {(const void*)log_decay, (const void*)beta, (const void*)dlog_decay, (const void*)dbeta, (const void*)cu_seqlens})
    if (!aligned4(t)) return SSD_ERR_INVALID_ARGUMENT;
  const DeltaLayout L = delta_layout(shape, d, true);
  if ((st = check_ws(workspace, workspace_bytes, L.total)) != SSD_OK) return st;
  const DeltaSpans t(shape, d);
  if (overlap({t.keys(dq), t.keys(dk), t.values(dv), t.gates(dlog_decay), t.gates(dbeta), t.state(dinitial_state),
               whole(workspace, (int64_t)L.total)},
              {t.q(q), t.k(k), t.v(v), t.values(d_o), t.gates(log_decay), t.gates(beta), t.state(initial_state),
               t.state(dfinal_state), t.starts(cu_seqlens)}))
    return SSD_ERR_INVALID_ARGUMENT;
  char* ws = static_cast<char*>(workspace);
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  ssd::DeltaArgs a = delta_args(shape, d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = log_decay;
  a.beta = beta;
  a.cu = cu_seqlens;
  a.scale = scale;
  a.init = initial_state;
  a.gates = floats(L.gates);
  a.tf = reinterpret_cast<float*>(ws + L.tf);
  a.seg_states = floats(L.seg_states);
  a.seg_maps = floats(L.seg_maps);
  a.seg_adj = floats(L.seg_adj);
  a.tt = floats(L.tt);
  a.pt = floats(L.pt);
  a.d_o = d_o;
  a.dfin = dfinal_state;
  a.dinit = dinitial_state;
  a.dq = dq;
  a.dk_out = dk;
  a.dv_out = dv;
  a.dg = dlog_decay;
  a.dbeta = dbeta;
  a.states = floats(L.states);
  a.dstates = floats(L.dstates);
  a.u = floats(L.u);
  a.ub = floats(L.ub);
  const bool shared = shape->nheads != shape->nqk_heads;
  if (shared) {
    a.part_q = floats(L.part_q);
    a.part_k = floats(L.part_k);
  }
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = ssd::launch_delta_prep(a, true, s);
  if (e == hipSuccess) e = ssd::launch_delta_fwd(a, true, s);
  if (e == hipSuccess) e = ssd::launch_delta_rev(a, s);
  if (e == hipSuccess) e = ssd::launch_delta_grads(a, s);
  if (e == hipSuccess && shared && d.grad_heads == 1) {
    ssd::LinShareSum p;
    p.in_k = a.part_q;
    p.in_v = a.part_k;
    p.out_k = dq;
    p.out_v = dk;
    p.cu = cu_seqlens;
    p.tokens = (long)d.tokens;
    p.S = shape->num_seqs;
    p.T = shape->seqlen;
    p.H = shape->nheads;
    p.Hk = shape->nqk_heads;
    p.dk = p.dv = shape->dk;
    p.bf16 = a.bf16;
    e = ssd::launch_lin_share_sum(p, s);
  }
  return hip_status(e);
}

ssd_status ssd_gated_delta_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                                const float* beta, const int32_t* slots, int32_t num_slots, float scale, void* o,
                                const ssd_delta_shape* shape, void* stream) {
  const ssd_status st = check_delta_heads(shape);
  if (st != SSD_OK) return st;
  if (!state || !q || !k || !v || !beta || !o || !scale_ok(scale) || num_slots < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (!slots && num_slots < shape->batch) return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned16(state) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned4(log_decay) || !aligned4(beta) || !aligned4(slots)) return SSD_ERR_INVALID_ARGUMENT;
  // A workgroup of 256 threads for every head and up to 64 row ranges of it (4 rows each at least): below 2^31 threads.
  const int64_t b = shape->batch, H = shape->nheads, Hk = shape->nqk_heads, esz = shape->dtype == SSD_DTYPE_BF16 ? 2 : 4;
  const int64_t slot = H * shape->dk * shape->dv * 4;
  const Span states = whole(state, std::min<int64_t>(num_slots, INT64_MAX / 8 / slot) * slot), out = whole(o, b * H * shape->dv * esz);
  if (overlap({out, states}, {whole(q, b * Hk * shape->dk * esz), whole(k, b * Hk * shape->dk * esz),
                              whole(v, b * H * shape->dv * esz), whole(log_decay, b * H * 4), whole(beta, b * H * 4),
                              whole(slots, b * 4)}))
    return SSD_ERR_INVALID_ARGUMENT;
  ssd::DeltaStep a;
  a.state = state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = log_decay;
  a.beta = beta;
  a.slots = slots;
  a.o = o;
  a.scale = scale;
  a.batch = shape->batch;
  a.H = shape->nheads;
  a.Hk = shape->nqk_heads;
  a.dk = shape->dk;
  a.dv = shape->dv;
  a.num_slots = num_slots;
  a.bf16 = shape->dtype == SSD_DTYPE_BF16;
  return hip_status(ssd::launch_delta_step(a, (hipStream_t)stream));
}

ssd_status ssd_rotary(const void* q, const void* k, const float* freq, const int32_t* positions,
                      const int32_t* cu_seqlens, const int32_t* offsets, float scale, void* q_out, void* k_out,
                      const ssd_rotary_shape* shape, void* stream) {
  const ssd_rotary_shape* s = shape;
  if (!s) return SSD_ERR_INVALID_ARGUMENT;
  if (s->batch < 1 || s->seqlen < 1 || s->q_heads < 1 || s->k_heads < 0 || s->dim < 1 || s->num_seqs < 0)
    return SSD_ERR_INVALID_ARGUMENT;
  if (s->rot < 2 || s->rot > s->dim || s->rot % 2) return SSD_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > 0 && s->batch != 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->inverse != 0 && s->inverse != 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->layout != SSD_ROTARY_HALF && s->layout != SSD_ROTARY_INTERLEAVED) return SSD_ERR_UNSUPPORTED;
  if (s->dim > 1024 || s->q_heads > 65535 || s->k_heads > 65535 || s->batch > 65535 || s->num_seqs > 65535) return SSD_ERR_UNSUPPORTED;
  if (!q || !q_out || !freq || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if ((k != nullptr) != (s->k_heads > 0) || (k_out != nullptr) != (s->k_heads > 0)) return SSD_ERR_INVALID_ARGUMENT;
  if ((cu_seqlens != nullptr) != (s->num_seqs > 0) || (positions && offsets)) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t esz = s->dtype == SSD_DTYPE_BF16 ? 2 : 4, tokens = (int64_t)s->batch * s->seqlen;
  if (tokens > INT32_MAX / 2) return SSD_ERR_UNSUPPORTED;
  const int64_t wide[2] = {(int64_t)s->q_heads * s->dim, (int64_t)s->k_heads * s->dim};
  const int64_t in[2] = {s->q_row ? s->q_row : wide[0], s->k_row ? s->k_row : wide[1]};
  const int64_t out[2] = {s->q_out_row ? s->q_out_row : wide[0], s->k_out_row ? s->k_out_row : wide[1]};
  const void* from[2] = {q, k};
  void* to[2] = {q_out, k_out};
  Span x[2], y[2];
  for (int w = 0; w < 2; ++w) {
    if (in[w] < wide[w] || out[w] < wide[w]) return SSD_ERR_INVALID_ARGUMENT;
    if (in[w] > INT32_MAX || out[w] > INT32_MAX) return SSD_ERR_UNSUPPORTED;
    if (((uintptr_t)from[w] | (uintptr_t)to[w]) % (uintptr_t)esz) return SSD_ERR_INVALID_ARGUMENT;
    x[w] = Span{from[w], tokens, in[w] * esz, wide[w] * esz};
    y[w] = Span{to[w], tokens, out[w] * esz, wide[w] * esz};
  }
  for (const void* t : {(const void*)freq, (const void*)positions, (const void*)cu_seqlens, (const void*)offsets})
    if (!aligned4(t)) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t seqs = s->num_seqs > 0 ? s->num_seqs : s->batch;
  const Span plain[4] = {whole(freq, s->rot / 2 * 4), whole(positions, tokens * 4),
                         whole(cu_seqlens, s->num_seqs > 0 ? (seqs + 1) * 4 : 0), whole(offsets, seqs * 4)};
  for (int w = 0; w < 2; ++w) {
    for (int i = 0; i < 2; ++i) {
      const bool same = w == i && y[w].base == x[i].base && y[w].pitch == x[i].pitch;   // in place
      if (!same && rows_meet(y[w], x[i])) return SSD_ERR_INVALID_ARGUMENT;
    }
    for (const Span& p : plain)
      if (meet(p, y[w])) return SSD_ERR_INVALID_ARGUMENT;
  }
  if (rows_meet(y[0], y[1])) return SSD_ERR_INVALID_ARGUMENT;
  ssd::RotaryArgs a;
  for (int w = 0; w < 2; ++w) {
    a.x[w] = from[w];
    a.y[w] = to[w];
    a.x_row[w] = (long)in[w];
    a.y_row[w] = (long)out[w];
  }
  a.heads[0] = s->q_heads;
  a.heads[1] = s->k_heads;
  a.freq = freq;
  a.positions = positions;
  a.cu = cu_seqlens;
  a.offsets = offsets;
  a.scale = scale;
  a.batch = s->batch;
  a.T = s->seqlen;
  a.S = s->num_seqs;
  a.d = s->dim;
  a.rot = s->rot;
  a.interleaved = s->layout == SSD_ROTARY_INTERLEAVED;
  a.inverse = s->inverse;
  a.bf16 = s->dtype == SSD_DTYPE_BF16;
  if (!ssd::rotary_launchable(a)) return SSD_ERR_UNSUPPORTED;
  return hip_status(ssd::launch_rotary(a, (hipStream_t)stream));
}

}  // extern "C"
