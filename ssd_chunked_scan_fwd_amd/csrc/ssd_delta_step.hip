// ssd_delta_step.hip -- the delta rule's one-token step against a pool of states:
//     u = beta (v - a S k),  S = a S + u k^T,  o = scale S q,  a = exp(log_decay).
// The state's read and write bound it (2 dv dk 4 bytes a head). A row of the state
// is read once: S k and S q of the state as it came are summed together, and
// o = scale (a (S q) + u (k . q)).
// The layout is that of the step of linear attention: a row takes `tpr` lanes of
// four columns each (a power of two; lanes past dk / 4 idle), a thread ROWS rows, a
// workgroup one (entry, head, row range); states move non-temporally, as those of
// a model's layers do not stay in the caches between two steps. Entries whose slot
// is outside the pool are padding: o = 0 and no state is touched. Entries that name
// the same slot are taken in the order of the batch by the first one's workgroup.
// 64 of 80 states, 32 heads of 128 x 128: 50 us, 5.4 TB/s, the rate of a copy.
#include "ssd_delta.h"
#include "ssd_device.h"
#include "ssd_lin_attn.h"

namespace ssd {

namespace {

template <bool BF16>
__device__ __forceinline__ float one(const void* p, long i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ f32x4 four_of(const void* p, long i) {
  if constexpr (BF16) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
  } else {
    return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  }
}
template <bool BF16>
__device__ __forceinline__ void put(void* p, long i, float x) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
  else static_cast<float*>(p)[i] = x;
}

template <bool BF16, int ROWS>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStep a, int tpr, int parts) {
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
      if (c4 == 0 && r < a.dv) put<BF16>(a.o, ((long)e * a.H + h) * a.dv + r, 0.f);
    }
    return;
  }
  // Rows and columns past the ends read their nearest neighbour inside, and are not written.
  float* st = a.state + ((long)slot * a.H + h) * a.dv * a.dk + (col_in ? 4 * c4 : 0);
  f32x4 s[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    s[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(st + (long)min(r0 + j * rpp, a.dv - 1) * a.dk));
  int next = a.batch;
  if (a.slots && step_peers(a.slots, a.batch, e, slot, lane, next)) return;  // an earlier entry's workgroup runs this one
  for (;;) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const long ek = (long)e * a.Hk + hk, eh = (long)e * a.H + h;
    f32x4 k = four_of<BF16>(a.k, ek * a.dk + (col_in ? 4 * c4 : 0));
    f32x4 q = four_of<BF16>(a.q, ek * a.dk + (col_in ? 4 * c4 : 0));
    const float decay = a.g ? expf(a.g[eh]) : 1.f, beta = a.beta[eh];
    float v[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) v[j] = one<BF16>(a.v, eh * a.dv + min(r0 + j * rpp, a.dv - 1));
    if (!col_in) k = q = zero;
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) kq = fmaf(k[i], q[i], kq);
    kq = lanes_sum(kq, tpr);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = r0 + j * rpp;
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] *= decay;
        sk = fmaf(s[j][i], k[i], sk);
        sq = fmaf(s[j][i], q[i], sq);
      }
      sk = lanes_sum(col_in ? sk : 0.f, tpr);
      sq = lanes_sum(col_in ? sq : 0.f, tpr);
      const float u = beta * (v[j] - sk);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = fmaf(u, k[i], s[j][i]);
      if (next == a.batch && col_in && r < a.dv)
        __builtin_nontemporal_store(s[j], reinterpret_cast<f32x4*>(st + (long)r * a.dk));
      if (c4 == 0 && r < a.dv) put<BF16>(a.o, eh * a.dv + r, a.scale * fmaf(u, kq, sq));
    }
    if (next == a.batch) break;
    e = next;
    step_peers(a.slots, a.batch, e, slot, lane, next);
  }
}

template <bool BF16>
void step_launch(const DeltaStep& a, int rows, int tpr, int parts, hipStream_t stream) {
  const dim3 grid((unsigned)(a.H * parts), (unsigned)a.batch);
  if (rows == 8) hipLaunchKernelGGL((delta_step_kernel<BF16, 8>), grid, dim3(256), 0, stream, a, tpr, parts);
  else if (rows == 4) hipLaunchKernelGGL((delta_step_kernel<BF16, 4>), grid, dim3(256), 0, stream, a, tpr, parts);
  else if (rows == 2) hipLaunchKernelGGL((delta_step_kernel<BF16, 2>), grid, dim3(256), 0, stream, a, tpr, parts);
  else hipLaunchKernelGGL((delta_step_kernel<BF16, 1>), grid, dim3(256), 0, stream, a, tpr, parts);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStep& a, hipStream_t stream) {
  int tpr = 2;
  while (tpr * 4 < a.dk) tpr *= 2;
  const int rpp = 256 / tpr;
  // Rows a thread: as many (up to 8, the loads each thread keeps in flight) as still leave two workgroups for
  // every CU and as fewer would not cover dv with less to spare.
  auto parts_of = [&](int r) { return (a.dv + r * rpp - 1) / (r * rpp); };
  int rows = 8;
  while (rows > 1 && (parts_of(rows) * 2 > parts_of(rows / 2) || (long)a.batch * a.H * parts_of(rows) < 512)) rows /= 2;
  const int parts = parts_of(rows);
  if (a.bf16) step_launch<true>(a, rows, tpr, parts, stream);
  else step_launch<false>(a, rows, tpr, parts, stream);
  return hipGetLastError();
}

}  // namespace ssd
