// ssd_rotary.hip -- rotary positions: pairs (x, y) of a head's first `rot`
// elements turned by the angle position * freq_i,
//     (x cos - y sin, y cos + x sin) * scale,
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) interleaved; the rest of the head is
// copied. The gradient of a turned pair is turned back (the same with -sin).
//
// Memory bounds it: every element is read once and written once (16384 tokens of 32 and 8 heads of 128: 67 us, 5.0 TB/s,
// the rate of a copy). The angles are
// those of a token, whatever the head: a workgroup takes a few tokens, makes their
// sines and cosines once, in LDS, and turns all heads of queries and keys with
// them. An angle is a product of 64 bits, brought into half a turn before it is
// rounded: a position of 10^6 times a frequency of 1 leaves 32 bits some 0.03 of a
// radian.
#include "ssd_device.h"
#include "ssd_layer.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 16;      // a workgroup
constexpr int kTable = 2048;         // angles a workgroup

struct RotaryPlan {
  int tokens;              // a workgroup
  int turned, units;       // of a head: units of a turn, and with those that are copied
  int du, dh, dt;          // kThreads units on: unit, head, token
};

// The position of a token; false where it belongs to no sequence.
__device__ __forceinline__ bool position_of(const RotaryArgs& a, long tok, double& pos) {
  int s = (int)(tok / a.T);
  long first = (long)s * a.T;
  if (a.cu) {
    // The last sequence that begins at or before tok (empty ones begin where the next one does).
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= tok) lo = mid;
      else hi = mid;
    }
    s = lo;
    first = min(max(a.cu[s], 0), a.T);
    if (tok < first || tok >= a.cu[a.S]) return false;
  }
  if (a.positions) pos = (double)a.positions[tok];
  else pos = (double)(tok - first) + (a.offsets ? (double)a.offsets[s] : 0.0);
  return true;
}

template <bool BF16>
__device__ __forceinline__ void load_piece(const void* p, long i, float* x) {   // 8 elements
  if constexpr (BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[2 * c] = bf16_lo(w[c]);
      x[2 * c + 1] = bf16_hi(w[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + 4 * c);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * c + r] = w[r];
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store_piece(void* p, long i, const float* x) {
  if constexpr (BF16) {
    u32x4 w;
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i + 4 * c) = f32x4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
  }
}
template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, long i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, long i, float x) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(x);
  else static_cast<float*>(p)[i] = x;
}

// VEC: units of 16-byte pieces, of a turn two pieces of 8 (a half apart) or one (4 pairs side by side); else
// units of one pair and one element.
template <bool BF16, bool VEC, bool INTER>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, RotaryPlan p) {
  __shared__ float cs[kTable], sn[kTable];
  __shared__ double pos[kMostTokens];
  __shared__ int in[kMostTokens];
  const int half = a.rot / 2, H = a.heads[0] + a.heads[1];
  const long all = (long)a.batch * a.T, tok0 = (long)blockIdx.x * p.tokens;
  const int tokens = (int)min((long)p.tokens, all - tok0);
  if ((int)threadIdx.x < tokens) {
    double x = 0.0;
    in[threadIdx.x] = position_of(a, tok0 + threadIdx.x, x);
    pos[threadIdx.x] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const double turns = pos[i / half] * (double)a.freq[i % half] * 0.15915494309189533577;   // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = c * a.scale;
    sn[i] = a.inverse ? -s * a.scale : s * a.scale;
  }
  __syncthreads();
  int u = threadIdx.x % p.units, h = threadIdx.x / p.units % H, t = threadIdx.x / p.units / H;
  for (; t < tokens; u += p.du, h += p.dh, t += p.dt) {
    if (u >= p.units) {
      u -= p.units;
      ++h;
    }
    if (h >= H) {
      h -= H;
      ++t;
    }
    if (t >= tokens) break;
    if (!in[t]) continue;
    const int w = h >= a.heads[0];
    const int hd = w ? h - a.heads[0] : h;
    const void* x = a.x[w];
    void* y = a.y[w];
    const long xi = (tok0 + t) * a.x_row[w] + (long)hd * a.d, yi = (tok0 + t) * a.y_row[w] + (long)hd * a.d;
    const float *c = cs + t * half, *s = sn + t * half;
    if constexpr (VEC) {
      if (u >= p.turned) {
        const int at = a.rot + 8 * (u - p.turned);
        float v[8];
        load_piece<BF16>(x, xi + at, v);
        store_piece<BF16>(y, yi + at, v);
      } else if constexpr (INTER) {
        float v[8], r[8];
        load_piece<BF16>(x, xi + 8 * u, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ci = c[4 * u + i], si = s[4 * u + i];
          r[2 * i] = fmaf(v[2 * i], ci, -v[2 * i + 1] * si);
          r[2 * i + 1] = fmaf(v[2 * i + 1], ci, v[2 * i] * si);
        }
        store_piece<BF16>(y, yi + 8 * u, r);
      } else {
        float v[8], z[8], r[8], q[8];
        load_piece<BF16>(x, xi + 8 * u, v);
        load_piece<BF16>(x, xi + half + 8 * u, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float ci = c[8 * u + i], si = s[8 * u + i];
          r[i] = fmaf(v[i], ci, -z[i] * si);
          q[i] = fmaf(z[i], ci, v[i] * si);
        }
        store_piece<BF16>(y, yi + 8 * u, r);
        store_piece<BF16>(y, yi + half + 8 * u, q);
      }
    } else {
      if (u >= p.turned) {
        const int at = a.rot + u - p.turned;
        store_one<BF16>(y, yi + at, load_one<BF16>(x, xi + at));
      } else {
        const int ia = INTER ? 2 * u : u, ib = INTER ? 2 * u + 1 : u + half;
        const float v = load_one<BF16>(x, xi + ia), z = load_one<BF16>(x, xi + ib);
        store_one<BF16>(y, yi + ia, fmaf(v, c[u], -z * s[u]));
        store_one<BF16>(y, yi + ib, fmaf(z, c[u], v * s[u]));
      }
    }
  }
}

bool vectors(const RotaryArgs& a) {
  const int esz = a.bf16 ? 2 : 4;
  uintptr_t all = 0;
  for (int w = 0; w < 2; ++w)
    if (a.heads[w])
      all |= (uintptr_t)a.x[w] | (uintptr_t)a.y[w] | (uintptr_t)(a.x_row[w] * esz) | (uintptr_t)(a.y_row[w] * esz);
  return all % 16 == 0 && a.d % 8 == 0 && a.rot % (a.interleaved ? 8 : 16) == 0;
}

RotaryPlan plan_of(const RotaryArgs& a, bool vec) {
  RotaryPlan p;
  const int H = a.heads[0] + a.heads[1];
  p.turned = vec ? a.rot / (a.interleaved ? 8 : 16) : a.rot / 2;
  p.units = p.turned + (vec ? (a.d - a.rot) / 8 : a.d - a.rot);
  // Tokens a workgroup: so many that a thread has some eight units, which hides the table's making, while the
  // launch still has four workgroups for every CU.
  const long all = (long)a.batch * a.T;
  p.tokens = 1;
  while (p.tokens < kMostTokens && (p.tokens * 2) * (a.rot / 2) <= kTable && (long)p.tokens * H * p.units < 8 * kThreads &&
         all / (p.tokens * 2) >= 1024)
    p.tokens *= 2;
  p.du = kThreads % p.units;
  p.dh = kThreads / p.units % H;
  p.dt = kThreads / p.units / H;
  return p;
}

template <bool BF16, bool VEC>
void launch(const RotaryArgs& a, const RotaryPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)(((long)a.batch * a.T + p.tokens - 1) / p.tokens));
  if (a.interleaved) hipLaunchKernelGGL((rotary_kernel<BF16, VEC, true>), grid, dim3(kThreads), 0, stream, a, p);
  else hipLaunchKernelGGL((rotary_kernel<BF16, VEC, false>), grid, dim3(kThreads), 0, stream, a, p);
}

}  // namespace

bool rotary_launchable(const RotaryArgs& a) {
  const RotaryPlan p = plan_of(a, vectors(a));
  return launchable(((long)a.batch * a.T + p.tokens - 1) / p.tokens, kThreads);
}

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream) {
  const bool vec = vectors(a);
  const RotaryPlan p = plan_of(a, vec);
  if (a.bf16) vec ? launch<true, true>(a, p, stream) : launch<true, false>(a, p, stream);
  else vec ? launch<false, true>(a, p, stream) : launch<false, false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace ssd
