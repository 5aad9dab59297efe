// ssd_layer_api.cpp -- the C ABI (include/ssd.h) of the layer operators around
// the scan: linear attention with one decay a head, the group norm with its
// gate, and the pages of a state pool. As in ssd_api.cpp, every argument is
// checked on the host before any HIP call; nothing is allocated, synchronised
// or thrown.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ssd.h"
#include "ssd_layer.h"
#include "ssd_lin_attn.h"

namespace {

ssd_status hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool scale_ok(float s) { return std::isnormal(s); }  // its reciprocal is taken

// Rows of `width` bytes, `pitch` bytes apart; a null base has none.
struct Span {
  const void* base;
  int64_t rows, pitch, width;
};
Span whole(const void* p, int64_t bytes) { return Span{p, 1, bytes, bytes}; }
// Whether a, one row, and b share a byte.
bool meet(const Span& a, const Span& b) {
  if (!a.base || !b.base || a.width < 1 || b.width < 1 || b.rows < 1) return false;
  const intptr_t at = (intptr_t)a.base - (intptr_t)b.base, end = at + a.width;   // a, from b's first row on
  if (end <= 0) return false;
  // the first of b's rows that ends behind a's start
  const int64_t first = at < b.width ? 0 : (at - b.width) / b.pitch + 1;
  return first < b.rows && first * b.pitch < end;
}
// Whether one of the outputs shares memory with an input or another output: kernels
// read the one while others write the other.
bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (const Span* p = outs.begin(); p != o; ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}

// ---------------------------------------------------------------- linear attention

struct LinDims {
  int64_t q_row, k_row, v_row, tokens, nseq;
  int esz;
};

ssd_status check_heads(const ssd_lin_shape* s) {
  if (s->nheads < 1 || s->nkv_heads < 1 || s->dk < 1 || s->dv < 1 || s->batch < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->nheads % s->nkv_heads) return SSD_ERR_INVALID_ARGUMENT;
  if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->dk % 8 || s->dv % 8 || s->dk > 256 || s->dv > 256) return SSD_ERR_UNSUPPORTED;
  if (s->nheads > 65535 || s->batch > 65535) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status check_lin(const ssd_lin_shape* s, LinDims* d) {
  if (!s) return SSD_ERR_INVALID_ARGUMENT;
  ssd_status st = check_heads(s);
  if (st != SSD_OK) return st;
  if (s->seqlen < 1 || s->num_seqs < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > 0 && s->batch != 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > 65535) return SSD_ERR_UNSUPPORTED;
  d->esz = s->dtype == SSD_DTYPE_BF16 ? 2 : 4;
  d->q_row = s->q_row ? s->q_row : (int64_t)s->nheads * s->dk;
  d->k_row = s->k_row ? s->k_row : (int64_t)s->nkv_heads * s->dk;
  d->v_row = s->v_row ? s->v_row : (int64_t)s->nkv_heads * s->dv;
  if (d->q_row < (int64_t)s->nheads * s->dk || d->k_row < (int64_t)s->nkv_heads * s->dk ||
      d->v_row < (int64_t)s->nkv_heads * s->dv)
    return SSD_ERR_INVALID_ARGUMENT;
  // rows start on 16-byte boundaries
  if ((d->q_row | d->k_row | d->v_row) * d->esz % 16) return SSD_ERR_UNSUPPORTED;
  // 64 rows are addressed as one buffer range of fewer than 2^31 bytes
  const int64_t most = INT32_MAX / 64 / 4;
  if (d->q_row > most || d->k_row > most || d->v_row > most || (int64_t)s->nheads * (s->dk > s->dv ? s->dk : s->dv) > most)
    return SSD_ERR_UNSUPPORTED;
  d->tokens = (int64_t)s->batch * s->seqlen;
  if (d->tokens > INT32_MAX / 2) return SSD_ERR_UNSUPPORTED;
  d->nseq = s->num_seqs > 0 ? s->num_seqs : s->batch;
  return SSD_OK;
}

// The memory of a call's tensors.
struct LinSpans {
  const ssd_lin_shape* s;
  LinDims d;
  LinSpans(const ssd_lin_shape* shape, const LinDims& dims) : s(shape), d(dims) {}
  Span rows(const void* p, int64_t row, int64_t heads, int64_t size) const {
    return Span{p, d.tokens, row * d.esz, heads * size * d.esz};
  }
  Span q(const void* p) const { return rows(p, d.q_row, s->nheads, s->dk); }
  Span k(const void* p) const { return rows(p, d.k_row, s->nkv_heads, s->dk); }
  Span v(const void* p) const { return rows(p, d.v_row, s->nkv_heads, s->dv); }
  Span queries(const void* p) const { return whole(p, d.tokens * s->nheads * s->dk * d.esz); }
  Span values(const void* p) const { return whole(p, d.tokens * s->nheads * s->dv * d.esz); }
  Span keys(const void* p, int64_t size) const { return whole(p, d.tokens * s->nkv_heads * size * d.esz); }
  Span decays(const void* p) const { return whole(p, s->nheads * 4); }
  Span starts(const void* p) const { return whole(p, (d.nseq + 1) * 4); }
  Span state(const void* p) const { return whole(p, d.nseq * s->nheads * s->dk * s->dv * 4); }
};

// The blocks of one scan with contraction size dk and value size dv.
struct LinPlan {
  int L;
  int64_t spr, slots;
  size_t state_bytes;  // 0: no sequence is cut
};
// `scans` of them may share a launch.
ssd_status lin_plan(const ssd_lin_shape* s, int dk, int dv, LinPlan* p, int scans = 1, bool kv = false) {
  p->L = ssd::lin_block_tokens(s->batch, s->seqlen, s->num_seqs, s->nheads, dk, dv, s->dtype == SSD_DTYPE_BF16, kv);
  p->spr = ssd::lin_slots_per_row(s->seqlen, s->num_seqs, p->L);
  p->slots = s->num_seqs > 0 ? p->spr : p->spr * s->batch;
  if (!ssd::launchable(p->slots * s->nheads * scans, ssd::lin_slot_threads(dv, s->dtype == SSD_DTYPE_BF16, kv)))
    return SSD_ERR_UNSUPPORTED;
  p->state_bytes = p->L >= s->seqlen ? 0 : (size_t)p->slots * s->nheads * dk * dv * 4;
  return SSD_OK;
}

struct LinBwdLayout {
  LinPlan dq, dv, dk;
  bool kv;  // dk and dv come from one scan
  size_t st_dq, st_dv, st_dk, part_k, part_v, total;
};
ssd_status lin_bwd_layout(const ssd_lin_shape* s, LinBwdLayout* L) {
  LinDims d;
  ssd_status st = check_lin(s, &d);
  if (st != SSD_OK) return st;
  if ((st = lin_plan(s, s->dv, s->dk, &L->dq, 2)) != SSD_OK) return st;
  L->kv = ssd::lin_kv_supported(s->dk, s->dv, s->dtype == SSD_DTYPE_BF16);
  if ((st = lin_plan(s, s->dk, s->dv, &L->dv, 2, L->kv)) != SSD_OK) return st;
  L->dk = LinPlan{};
  if (!L->kv && (st = lin_plan(s, s->dv, s->dk, &L->dk)) != SSD_OK) return st;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off = align256(off + b);
    return o;
  };
  L->st_dq = take(L->dq.state_bytes);
  L->st_dv = take(L->dv.state_bytes);
  L->st_dk = take(L->dk.state_bytes);
  const bool shared = s->nheads != s->nkv_heads;
  const int64_t pieces = (s->dk > s->dv ? s->dk : s->dv) / 8;   // a thread's share of the sums over shared heads
  if (shared && !ssd::launchable(d.tokens * s->nkv_heads * pieces / 256 + 1, 256)) return SSD_ERR_UNSUPPORTED;
  L->part_k = take(shared ? (size_t)d.tokens * s->nheads * s->dk * 4 : 0);
  L->part_v = take(shared ? (size_t)d.tokens * s->nheads * s->dv * 4 : 0);
  L->total = off;
  return SSD_OK;
}

ssd::LinScan base_scan(const ssd_lin_shape* s, const float* ld, const int32_t* cu, float scale) {
  ssd::LinScan a;
  a.ld = ld;
  a.scale = scale;
  a.cu = cu;
  a.S = s->num_seqs;
  a.batch = s->batch;
  a.T = s->seqlen;
  a.H = s->nheads;
  a.bf16 = s->dtype == SSD_DTYPE_BF16;
  return a;
}

void set_plan(ssd::LinScan* a, const LinPlan& p, char* states) {
  a->L = p.L;
  a->slots_per_row = (long)p.spr;
  a->states = p.state_bytes ? reinterpret_cast<float*>(states) : nullptr;
}

ssd_status check_ws(const void* workspace, size_t have, size_t need) {
  if (need == 0) return SSD_OK;
  if (!workspace || ((uintptr_t)workspace & 255)) return SSD_ERR_INVALID_ARGUMENT;
  return have < need ? SSD_ERR_WORKSPACE_TOO_SMALL : SSD_OK;
}

// ---------------------------------------------------------------- group norm

ssd_status check_norm(const ssd_norm_shape* s) {
  if (!s) return SSD_ERR_INVALID_ARGUMENT;
  if (s->samples < 1 || s->positions < 1 || s->channels < 1 || s->groups < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->channels % s->groups) return SSD_ERR_INVALID_ARGUMENT;
  if (s->x_row != 0 && s->x_row < s->channels) return SSD_ERR_INVALID_ARGUMENT;
  if (s->z_row != 0 && s->z_row < s->channels) return SSD_ERR_INVALID_ARGUMENT;
  if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->act != SSD_ACT_NONE && s->act != SSD_ACT_SILU) return SSD_ERR_UNSUPPORTED;
  if (s->gate != SSD_GATE_NONE && s->gate != SSD_GATE_AFTER && s->gate != SSD_GATE_BEFORE) return SSD_ERR_UNSUPPORTED;
  if (s->center != 0 && s->center != 1) return SSD_ERR_INVALID_ARGUMENT;
  // rows, and what of a launch is counted in 32 bits by the kernels (its threads: norm_launchable)
  const int64_t rows = (int64_t)s->samples * s->positions;
  if (rows > INT32_MAX / 4 || rows * s->groups > INT32_MAX / 4) return SSD_ERR_UNSUPPORTED;
  if (rows * ((s->channels + 63) / 64) > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd::NormArgs norm_args(const ssd_norm_shape* s) {
  ssd::NormArgs a;
  a.n = s->samples;
  a.s = s->positions;
  a.C = s->channels;
  a.G = s->groups;
  a.x_row = s->x_row ? s->x_row : s->channels;
  a.z_row = s->z_row ? s->z_row : s->channels;
  a.bf16 = s->dtype == SSD_DTYPE_BF16;
  a.silu = s->act == SSD_ACT_SILU;
  a.gate = s->gate;
  a.center = s->center;
  return a;
}

// Elements start on their own size; 8-channel pieces need 16-byte rows throughout.
ssd_status norm_align(ssd::NormArgs* a) {
  const int esz = a->bf16 ? 2 : 4;
  const uintptr_t all = (uintptr_t)a->x | (uintptr_t)a->z | (uintptr_t)a->dy | (uintptr_t)a->y | (uintptr_t)a->dx |
                        (uintptr_t)a->dz;
  if (all % esz) return SSD_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)a->w | (uintptr_t)a->bias | (uintptr_t)a->stats | (uintptr_t)a->dw | (uintptr_t)a->db) & 3)
    return SSD_ERR_INVALID_ARGUMENT;
  a->vec = all % 16 == 0 && a->C % 8 == 0 && a->x_row % 8 == 0 && a->z_row % 8 == 0;
  return SSD_OK;
}

// An output of contiguous rows over an input: they may be the same rows, which a
// thread reads before it writes them, or lie apart.
bool norm_apart(const ssd::NormArgs& a, const void* out, const void* in, long in_row) {
  const int64_t esz = a.bf16 ? 2 : 4, rows = a.n * a.s;
  if (out == in && in_row == a.C) return true;
  return !meet(whole(out, rows * a.C * esz), Span{in, rows, std::min<int64_t>(in_row, INT64_MAX / 32) * esz, a.C * esz});
}

ssd_status check_pages(const ssd_pages_shape* s) {
  if (!s) return SSD_ERR_INVALID_ARGUMENT;
  if (s->layers < 1 || s->slots < 1 || s->page_bytes < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (s->layers > 65535 || s->slots > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  if (s->page_bytes > ((int64_t)1 << 40)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}
ssd::PagesArgs pages_args(void* pool, const ssd_pages_shape* s) {
  ssd::PagesArgs a;
  a.pool = static_cast<char*>(pool);
  a.layers = s->layers;
  a.slots = s->slots;
  a.page = (long)s->page_bytes;
  return a;
}

}  // namespace

extern "C" {

ssd_status ssd_lin_attn_workspace_bytes(const ssd_lin_shape* shape, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  LinDims d;
  LinPlan p;
  ssd_status st = check_lin(shape, &d);
  if (st == SSD_OK) st = lin_plan(shape, shape->dk, shape->dv, &p);
  if (st == SSD_OK) *bytes = p.state_bytes;
  return st;
}

ssd_status ssd_lin_attn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                            const int32_t* cu_seqlens, float scale, const float* initial_state, void* o,
                            float* final_state, const ssd_lin_shape* shape, void* workspace, size_t workspace_bytes,
                            void* stream) {
  LinDims d;
  LinPlan p;
  ssd_status st = check_lin(shape, &d);
  if (st != SSD_OK) return st;
  if (!q || !k || !v || !log_decay || !o || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if ((cu_seqlens != nullptr) != (shape->num_seqs > 0)) return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state))
    return SSD_ERR_INVALID_ARGUMENT;
  if ((st = lin_plan(shape, shape->dk, shape->dv, &p)) != SSD_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, p.state_bytes)) != SSD_OK) return st;
  const LinSpans t(shape, d);
  if (overlap({t.values(o), t.state(final_state), whole(workspace, p.state_bytes)},
              {t.q(q), t.k(k), t.v(v), t.state(initial_state), t.decays(log_decay), t.starts(cu_seqlens)}))
    return SSD_ERR_INVALID_ARGUMENT;
  const int rep = shape->nheads / shape->nkv_heads;
  ssd::LinScan a = base_scan(shape, log_decay, cu_seqlens, scale);
  a.q = {q, (long)d.q_row, 1};
  a.k = {k, (long)d.k_row, rep};
  a.v = {v, (long)d.v_row, rep};
  a.o = o;
  a.dk = shape->dk;
  a.dv = shape->dv;
  a.init = initial_state;
  a.fin = final_state;
  a.q_once = 1;
  set_plan(&a, p, static_cast<char*>(workspace));
  return hip_status(ssd::launch_lin_scan(a, (hipStream_t)stream));
}

ssd_status ssd_lin_attn_bwd_workspace_bytes(const ssd_lin_shape* shape, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  LinBwdLayout L;
  ssd_status st = lin_bwd_layout(shape, &L);
  if (st == SSD_OK) *bytes = L.total;
  return st;
}

ssd_status ssd_lin_attn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                            const int32_t* cu_seqlens, float scale, const float* initial_state, const void* d_o,
                            const float* dfinal_state, void* dq, void* dk, void* dv, float* dinitial_state,
                            const ssd_lin_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
  LinDims d;
  LinBwdLayout L;
  ssd_status st = check_lin(shape, &d);
  if (st != SSD_OK) return st;
  if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if ((cu_seqlens != nullptr) != (shape->num_seqs > 0)) return SSD_ERR_INVALID_ARGUMENT;
  for (const void* t : {q, k, v, d_o, (const void*)initial_state, (const void*)dfinal_state, (const void*)dq, (const void*)dk,
                        (const void*)dv, (const void*)dinitial_state})
    if (!aligned16(t)) return SSD_ERR_INVALID_ARGUMENT;
  if ((st = lin_bwd_layout(shape, &L)) != SSD_OK) return st;
  if ((st = check_ws(workspace, workspace_bytes, L.total)) != SSD_OK) return st;
  const LinSpans t(shape, d);
  if (overlap({t.queries(dq), t.keys(dk, shape->dk), t.keys(dv, shape->dv), t.state(dinitial_state), whole(workspace, L.total)},
              {t.q(q), t.k(k), t.v(v), t.values(d_o), t.state(initial_state), t.state(dfinal_state), t.decays(log_decay),
               t.starts(cu_seqlens)}))
    return SSD_ERR_INVALID_ARGUMENT;
  char* ws = static_cast<char*>(workspace);
  hipStream_t hs = (hipStream_t)stream;
  const int H = shape->nheads, Hk = shape->nkv_heads, rep = H / Hk;
  const ssd::LinOperand oq{q, (long)d.q_row, 1}, ok{k, (long)d.k_row, rep}, ov{v, (long)d.v_row, rep},
      og{d_o, (long)H * shape->dv, 1};
  ssd::LinScan sq = base_scan(shape, log_decay, cu_seqlens, scale);
  sq.q = og;
  sq.k = ov;
  sq.v = ok;
  sq.o = dq;
  sq.dk = shape->dv;
  sq.dv = shape->dk;
  sq.init = initial_state;
  sq.init_tr = 1;
  set_plan(&sq, L.dq, ws + L.st_dq);
  // The reversed scans carry the adjoint divided by `scale`, which multiplies their outputs.
  void* const dv_out = rep > 1 ? static_cast<void*>(ws + L.part_v) : dv;
  void* const dk_out = rep > 1 ? static_cast<void*>(ws + L.part_k) : dk;
  ssd::LinScan sv = base_scan(shape, log_decay, cu_seqlens, scale);
  sv.q = ok;
  sv.k = oq;
  sv.v = og;
  sv.o = dv_out;
  sv.o_f32 = rep > 1;
  sv.dk = shape->dk;
  sv.dv = shape->dv;
  sv.init = dfinal_state;
  sv.init_scale = 1.f / scale;
  sv.fin = dinitial_state;
  sv.fin_scale = scale;
  sv.rev = 1;
  set_plan(&sv, L.dv, ws + L.st_dv);
  hipError_t e = ssd::launch_lin_states(sq, &sv, hs);
  if (e == hipSuccess) e = ssd::launch_lin_outputs(sq, hs);
  if (e == hipSuccess) e = L.kv ? ssd::launch_lin_kv(sv, ov, dk_out, hs) : ssd::launch_lin_outputs(sv, hs);
  if (e == hipSuccess && !L.kv) {
    ssd::LinScan sk = base_scan(shape, log_decay, cu_seqlens, scale);
    sk.q = ov;
    sk.k = og;
    sk.v = oq;
    sk.o = dk_out;
    sk.o_f32 = rep > 1;
    sk.dk = shape->dv;
    sk.dv = shape->dk;
    sk.init = dfinal_state;
    sk.init_scale = 1.f / scale;
    sk.init_tr = 1;
    sk.rev = 1;
    set_plan(&sk, L.dk, ws + L.st_dk);
    e = ssd::launch_lin_scan(sk, hs);
  }
  if (e != hipSuccess) return SSD_ERR_HIP;
  if (rep > 1) {
    ssd::LinShareSum sum;
    sum.in_k = static_cast<const float*>(dk_out);
    sum.in_v = static_cast<const float*>(dv_out);
    sum.out_k = dk;
    sum.out_v = dv;
    sum.cu = cu_seqlens;
    sum.tokens = (long)d.tokens;
    sum.S = shape->num_seqs;
    sum.T = shape->seqlen;
    sum.H = H;
    sum.Hk = Hk;
    sum.dk = shape->dk;
    sum.dv = shape->dv;
    sum.bf16 = shape->dtype == SSD_DTYPE_BF16;
    e = ssd::launch_lin_share_sum(sum, hs);
  }
  return hip_status(e);
}

ssd_status ssd_lin_attn_step(float* state, const void* q, const void* k, const void* v, const float* log_decay,
                             const int32_t* slots, int32_t num_slots, float scale, void* o, const ssd_lin_shape* shape,
                             void* stream) {
  if (!shape) return SSD_ERR_INVALID_ARGUMENT;
  ssd_status st = check_heads(shape);
  if (st != SSD_OK) return st;
  if (!state || !q || !k || !v || !log_decay || !o || !scale_ok(scale)) return SSD_ERR_INVALID_ARGUMENT;
  if (num_slots < 1 || (!slots && num_slots < shape->batch)) return SSD_ERR_INVALID_ARGUMENT;
  if (!aligned16(state) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t esz = shape->dtype == SSD_DTYPE_BF16 ? 2 : 4, heads = shape->nheads, keys = shape->nkv_heads;
  const auto entries = [&](const void* p, int64_t values) { return whole(p, shape->batch * values * esz); };
  const int64_t slot = heads * shape->dk * shape->dv * 4;
  if (overlap({entries(o, heads * shape->dv), whole(state, std::min<int64_t>(num_slots, INT64_MAX / 8 / slot) * slot)},
              {entries(q, heads * shape->dk), entries(k, keys * shape->dk), entries(v, keys * shape->dv),
               whole(log_decay, heads * 4), whole(slots, shape->batch * 4)}))
    return SSD_ERR_INVALID_ARGUMENT;
  ssd::LinStep a;
  a.state = state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld = log_decay;
  a.slots = slots;
  a.o = o;
  a.scale = scale;
  a.batch = shape->batch;
  a.H = shape->nheads;
  a.Hk = shape->nkv_heads;
  a.dk = shape->dk;
  a.dv = shape->dv;
  a.num_slots = num_slots;
  a.bf16 = shape->dtype == SSD_DTYPE_BF16;
  return hip_status(ssd::launch_lin_step(a, (hipStream_t)stream));
}

ssd_status ssd_group_norm_workspace_bytes(const ssd_norm_shape* shape, int32_t backward, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  ssd_status st = check_norm(shape);
  if (st != SSD_OK) return st;
  *bytes = 4 * ssd::norm_ws_floats(shape->samples, shape->positions, shape->channels, shape->groups, backward != 0);
  return SSD_OK;
}

ssd_status ssd_group_norm(const void* x, const void* z, const float* weight, const float* bias, float eps, void* y,
                          float* stats, const ssd_norm_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
  ssd_status st = check_norm(shape);
  if (st != SSD_OK) return st;
  if (!x || !y || (z != nullptr) != (shape->gate != SSD_GATE_NONE)) return SSD_ERR_INVALID_ARGUMENT;
  if (!(eps > 0.f) || !std::isfinite(eps)) return SSD_ERR_INVALID_ARGUMENT;
  ssd::NormArgs a = norm_args(shape);
  a.x = x;
  a.z = z;
  a.w = weight;
  a.bias = bias;
  a.eps = eps;
  a.y = y;
  a.stats = stats;
  if ((st = norm_align(&a)) != SSD_OK) return st;
  if (!ssd::norm_launchable(a)) return SSD_ERR_UNSUPPORTED;
  size_t need = 0;
  ssd_group_norm_workspace_bytes(shape, 0, &need);
  if ((st = check_ws(workspace, workspace_bytes, need)) != SSD_OK) return st;
  if (!norm_apart(a, y, x, a.x_row) || !norm_apart(a, y, z, a.z_row)) return SSD_ERR_INVALID_ARGUMENT;
  a.ws = static_cast<float*>(workspace);
  return hip_status(ssd::launch_group_norm(a, (hipStream_t)stream));
}

ssd_status ssd_group_norm_bwd(const void* x, const void* z, const float* weight, const float* bias, const float* stats,
                              const void* dy, void* dx, void* dz, float* dweight, float* dbias, const ssd_norm_shape* shape,
                              void* workspace, size_t workspace_bytes, void* stream) {
  ssd_status st = check_norm(shape);
  if (st != SSD_OK) return st;
  if (!x || !stats || !dy || !dx) return SSD_ERR_INVALID_ARGUMENT;
  if ((z != nullptr) != (shape->gate != SSD_GATE_NONE) || (dz != nullptr) != (z != nullptr)) return SSD_ERR_INVALID_ARGUMENT;
  ssd::NormArgs a = norm_args(shape);
  a.x = x;
  a.z = z;
  a.w = weight;
  a.bias = bias;
  a.stats = const_cast<float*>(stats);  // read only here
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.dw = dweight;
  a.db = dbias;
  if ((st = norm_align(&a)) != SSD_OK) return st;
  if (!ssd::norm_launchable(a)) return SSD_ERR_UNSUPPORTED;
  size_t need = 0;
  ssd_group_norm_workspace_bytes(shape, 1, &need);
  if ((st = check_ws(workspace, workspace_bytes, need)) != SSD_OK) return st;
  for (const void* out : {(const void*)dx, (const void*)dz})
    if (!norm_apart(a, out, x, a.x_row) || !norm_apart(a, out, z, a.z_row) || !norm_apart(a, out, dy, a.C))
      return SSD_ERR_INVALID_ARGUMENT;
  if (overlap({whole(dx, a.n * a.s * a.C * (a.bf16 ? 2 : 4))}, {whole(dz, a.n * a.s * a.C * (a.bf16 ? 2 : 4))}))
    return SSD_ERR_INVALID_ARGUMENT;
  a.ws = static_cast<float*>(workspace);
  return hip_status(ssd::launch_group_norm_bwd(a, (hipStream_t)stream));
}

ssd_status ssd_pages_copy(void* pool, const int32_t* src, const int32_t* dst, int32_t pairs, const ssd_pages_shape* shape,
                          void* stream) {
  ssd_status st = check_pages(shape);
  if (st != SSD_OK) return st;
  if (!pool || !src || !dst || pairs < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (pairs > ssd::kMaxPagePairs) return SSD_ERR_UNSUPPORTED;
  return hip_status(ssd::launch_pages_copy(pages_args(pool, shape), src, dst, pairs, (hipStream_t)stream));
}

ssd_status ssd_pages_clear(void* pool, const int32_t* slots, int32_t count, const ssd_pages_shape* shape, void* stream) {
  ssd_status st = check_pages(shape);
  if (st != SSD_OK) return st;
  if (!pool || !slots || count < 1) return SSD_ERR_INVALID_ARGUMENT;
  if (count > 65535) return SSD_ERR_UNSUPPORTED;
  return hip_status(ssd::launch_pages_clear(pages_args(pool, shape), slots, count, (hipStream_t)stream));
}

ssd_status ssd_pages_compact_workspace_bytes(const ssd_pages_shape* shape, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  ssd_status st = check_pages(shape);
  if (st == SSD_OK) *bytes = ssd::pages_compact_ws_bytes(shape->slots);
  return st;
}

ssd_status ssd_pages_compact(void* pool, const uint8_t* live, int32_t* where, int32_t* count, const ssd_pages_shape* shape,
                             void* workspace, size_t workspace_bytes, void* stream) {
  ssd_status st = check_pages(shape);
  if (st != SSD_OK) return st;
  if (!pool || !live || !where || !count) return SSD_ERR_INVALID_ARGUMENT;
  if ((st = check_ws(workspace, workspace_bytes, ssd::pages_compact_ws_bytes(shape->slots))) != SSD_OK) return st;
  return hip_status(ssd::launch_pages_compact(pages_args(pool, shape), live, where, count, workspace, (hipStream_t)stream));
}

}  // extern "C"
