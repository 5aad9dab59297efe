// ssd_group_norm.hip -- group norm over channels-last rows with an activation
// or a gate, forwards and backwards. All of it is bound by the bytes of x, z,
// y and their gradients.
//
// Over the channels of a group and the s positions of a sample:
//     u = x or x silu(z),  xh = (u - mean) rstd,  t = xh w + bias,
//     y = a or a silu(z),  a = t or silu(t).
// With g = dL/dt and M values a group:
//     du = rstd (g w - mean(g w) - xh mean(g w xh)),  dw = sum g xh,  dbias = sum g.
//
// Two forms. One position a sample (s = 1: the norm of a token): a group is
// one run of channels, held in registers by the lanes that share it, so that
// x is read once. More positions: the rows are cut into slabs; a first launch
// leaves each slab's mean and squared deviations per channel, a second joins
// them per group, a third applies them (reading x twice, but with every slab at
// work at once). Means and deviations are joined about their own means, in 32
// bits; nothing subtracts two large sums.
//
// 16384 tokens of 32 gated groups of 128: 85 us for 403 MB, 4.7 TB/s; backwards,
// 8192 tokens of 5120 gated channels: 82 us for 420 MB, 5.1 TB/s. 8 samples of
// 2256 positions, 320 channels, 23 MB (in cache): 7 + 4 + 10 us of three launches,
// 21 a call, 35 backwards; the 376 workgroups of 256 threads of the first and the
// third hide little of each other's waits. Groups that are no whole pieces of
// eight channels are read channel by channel: 16384 tokens of 32 groups of 10, 21
// MB, 47 us, of 70, 147 MB, 404 us. Groups beyond the registers take the slabs with
// one row each: 4096 tokens of 10240 channels, 168 MB, 652 us.
#include <type_traits>

#include "ssd_device.h"
#include "ssd_layer.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kCus = 256, kMaxParts = 1024;
constexpr int kMaxWaves = 16;   // of a workgroup that shares one group

// Sums over the `lanes` threads that share a group: a power of two up to 64, or
// the whole workgroup, then through LDS (`red`, a slot of two floats a wave;
// calls in turn use the two halves of it, so that one barrier a call is enough).
__device__ __forceinline__ void group_totals(float& v0, float& v1, int lanes, float* red, int half) {
  const int n = lanes < 64 ? lanes : 64;
  v0 = lanes_sum(v0, n);
  v1 = lanes_sum(v1, n);
  if (lanes <= 64) return;
  float* at = red + 2 * kMaxWaves * half;
  if ((threadIdx.x & 63) == 0) {
    at[2 * (threadIdx.x >> 6)] = v0;
    at[2 * (threadIdx.x >> 6) + 1] = v1;
  }
  __syncthreads();
  v0 = v1 = 0.f;
  for (int w = 0; w < (int)blockDim.x >> 6; ++w) {
    v0 += at[2 * w];
    v1 += at[2 * w + 1];
  }
}

__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + fast_exp2(-v * kLog2e)); }
// silu'(v) = s (1 + v (1 - s))
__device__ __forceinline__ float silu_slope(float v, float s) { return s * (1.f + v * (1.f - s)); }

// VEC consecutive elements (8: sixteen-byte pieces; 1: any alignment).
template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void* p, long i, float* v) {
  if constexpr (VEC == 8) {
    if constexpr (BF16) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(w[j]);
        v[2 * j + 1] = bf16_hi(w[j]);
      }
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
      const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
      }
    }
  } else {
    v[0] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  }
}
template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(void* p, long i, const float* v) {
  if constexpr (VEC == 8) {
    if constexpr (BF16) {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) =
          u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
    if (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v[0]);
    else static_cast<float*>(p)[i] = v[0];
  }
}
// Parameters of VEC channels, `other` where the pointer is null.
template <int VEC>
__device__ __forceinline__ void load_par(const float* p, int c, float other, float* v) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = p ? p[c + j] : other;
}

// A form of the norm fixed at compile time (GATE and SILU), or read from the
// arguments (GATE < 0).
template <int GATE, bool SILU>
struct Form {
  static __device__ __forceinline__ int gate(const NormArgs& a) { return GATE < 0 ? a.gate : GATE; }
  static __device__ __forceinline__ bool silu(const NormArgs& a) { return GATE < 0 ? a.silu != 0 : SILU; }
};

// t -> y for one element; sz = silu(z) where the gate comes after.
template <class F>
__device__ __forceinline__ float finish(const NormArgs& a, float t, float sz) {
  const float v = F::silu(a) ? t * sigmoid(t) : t;
  return F::gate(a) == kGateAfter ? v * sz : v;
}
// dL/dt from dL/dy, and the gate's own gradient where it comes after.
template <class F>
__device__ __forceinline__ float unfinish(const NormArgs& a, float t, float z, float dy, float& dz) {
  float slope = 1.f, v = t;
  if (F::silu(a)) {
    const float s = sigmoid(t);
    v = t * s;
    slope = silu_slope(t, s);
  }
  if (F::gate(a) == kGateAfter) {
    const float s = sigmoid(z);
    dz = dy * v * silu_slope(z, s);
    dy *= z * s;
  }
  return dy * slope;
}
typedef Form<-1, false> AnyForm;

// ---------------------------------------------------------------- one position a sample

// VEC elements as they lie in memory, so that the next row's loads wait in few registers.
template <bool BF16, int VEC>
struct Raw {
  u32x4 w[VEC == 8 ? (BF16 ? 1 : 2) : 1];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (auto& x : w) x = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void load(const void* p, long i) {
    if constexpr (VEC == 8) {
      const u32x4* at = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
      for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = at[k];
    } else {
      w[0].x = BF16 ? (uint32_t)static_cast<const uint16_t*>(p)[i] << 16 : static_cast<const uint32_t*>(p)[i];
    }
  }
  // The same, for rows that no launch of the call reads again: marked so, they do
  // not push other lines out of the caches. 16384 tokens of 4096 gated channels:
  // 92 -> 88 us back to back, 114 -> 95 after 1 GB of writes; backwards, 8192 x
  // 5120: 78 -> 72 and 118 -> 86. (Results so marked gained back to back and lost
  // 4 to 13 % after the writes, so they are stored as usual.)
  __device__ __forceinline__ void load_once(const void* p, long i) {
    if constexpr (VEC == 8) {
      const u32x4* at = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
      for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = __builtin_nontemporal_load(at + k);
    } else {
      load(p, i);
    }
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (VEC == 8 && BF16) return j & 1 ? bf16_hi(w[0][j >> 1]) : bf16_lo(w[0][j >> 1]);
    else return __uint_as_float(w[VEC == 8 ? j >> 2 : 0][j & 3]);
  }
};

// `lanes` threads share one (row, group), NV pieces of VEC channels each; WHOLE:
// all threads of the workgroup do.
template <bool BF16, int VEC, int NV, int GATE, bool SILU, bool WHOLE>
__global__ __launch_bounds__(WHOLE ? 1024 : kThreads) void norm_row_kernel(NormArgs a, int lanes) {
  using F = Form<GATE, SILU>;
  __shared__ float red[4 * kMaxWaves];
  const int Cg = a.C / a.G;
  const int l = WHOLE ? (int)threadIdx.x : (int)threadIdx.x & (lanes - 1);
  const long item = WHOLE ? (long)blockIdx.x : (long)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  const bool on = item < a.n * a.G;
  const long row = on ? item / a.G : 0;
  const int g = on ? (int)(item % a.G) : 0;
  Raw<BF16, VEC> rx[NV], rz[NV];
  float u[NV][VEC], z[NV][VEC];
  float sum = 0.f, none = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (l + i * lanes) * VEC;
    rx[i].zero();
    rz[i].zero();
    if (on && c < Cg) {
      rx[i].load_once(a.x, row * a.x_row + g * Cg + c);
      if (F::gate(a)) rz[i].load_once(a.z, row * a.z_row + g * Cg + c);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      u[i][j] = rx[i][j];
      z[i][j] = 0.f;
      if (F::gate(a)) z[i][j] = rz[i][j] * sigmoid(rz[i][j]);
      if (F::gate(a) == kGateBefore) u[i][j] *= z[i][j];
      sum += u[i][j];
    }
  const float inv = 1.f / (float)Cg;
  float mean = 0.f;
  if (a.center) {
    group_totals(sum, none, lanes, red, 0);
    mean = sum * inv;
  }
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (l + i * lanes) * VEC < Cg;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      u[i][j] = in ? u[i][j] - mean : 0.f;
      sq += u[i][j] * u[i][j];
    }
  }
  group_totals(sq, none, lanes, red, 1);
  const float rstd = 1.f / sqrtf(sq * inv + a.eps);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (l + i * lanes) * VEC;
    if (c >= Cg) break;
    float w[VEC], b[VEC];
    load_par<VEC>(a.w, g * Cg + c, 1.f, w);
    load_par<VEC>(a.bias, g * Cg + c, 0.f, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) u[i][j] = finish<F>(a, u[i][j] * rstd * w[j] + b[j], z[i][j]);
    store_vec<BF16, VEC>(a.y, row * a.C + g * Cg + c, u[i]);
  }
  if (a.stats && l == 0) {
    a.stats[2 * (row * a.G + g)] = mean;
    a.stats[2 * (row * a.G + g) + 1] = rstd;
  }
}

// Backwards: `lanes` threads keep one group and walk rows, so that dw and
// dbias of their channels stay in registers; each leaves one row of partial
// sums in ws ([part][2][C]). The next row's loads are issued before this row's
// sums are taken.
template <bool BF16, int VEC, int NV, int GATE, bool SILU, bool WHOLE>
__global__ __launch_bounds__(WHOLE ? 1024 : kThreads) void norm_row_bwd_kernel(NormArgs a, int lanes, int groups, int rows, int row_blocks) {
  using F = Form<GATE, SILU>;
  __shared__ float red[4 * kMaxWaves];
  const int Cg = a.C / a.G;
  const int l = WHOLE ? (int)threadIdx.x : (int)threadIdx.x & (lanes - 1), worker = WHOLE ? 0 : (int)threadIdx.x / lanes;
  const int tiles = (a.G + groups - 1) / groups;
  const int g = (int)(blockIdx.x % tiles) * groups + worker % groups;
  const int part = (int)(blockIdx.x / tiles) * rows + worker / groups;
  const int parts = row_blocks * rows;
  const bool on = worker < groups * rows && g < a.G;
  const int c0 = (on ? g : 0) * Cg;
  const float inv = 1.f / (float)Cg;
  float dw[NV][VEC], db[NV][VEC], w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (l + i * lanes) * VEC;
    load_par<VEC>(a.w, c0 + (c < Cg ? c : 0), 1.f, w[i]);
    load_par<VEC>(a.bias, c0 + (c < Cg ? c : 0), 0.f, b[i]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  Raw<BF16, VEC> nx[NV], nz[NV], ng[NV];
  float nmean = 0.f, nrstd = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    nx[i].zero();
    nz[i].zero();
    ng[i].zero();
  }
  auto fetch = [&](long row) {
    if (!on || row >= a.n) return;
    nmean = a.stats[2 * (row * a.G + g)];
    nrstd = a.stats[2 * (row * a.G + g) + 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (l + i * lanes) * VEC;
      if (c >= Cg) break;
      nx[i].load_once(a.x, row * a.x_row + c0 + c);
      if (F::gate(a)) nz[i].load_once(a.z, row * a.z_row + c0 + c);
      ng[i].load_once(a.dy, row * a.C + c0 + c);
    }
  };
  fetch(part);
  int half = 0;
  // Every thread of the workgroup makes the same number of rounds (the sums meet at a barrier).
  for (long r0 = 0; r0 < a.n; r0 += parts, half ^= 1) {
    const long row = r0 + part;
    const bool live = on && row < a.n;
    Raw<BF16, VEC> x[NV], z[NV], dy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = nx[i];
      z[i] = nz[i];
      dy[i] = ng[i];
    }
    const float mean = nmean, rstd = nrstd;
    fetch(row + parts);
    // g w and xh; with the gate before also silu(z) and x silu'(z). dz of a gate after is final here.
    float xh[NV][VEC], gw[NV][VEC], p[NV][VEC], q[NV][VEC];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (l + i * lanes) * VEC;
      const bool in = live && c < Cg;
      float dzv[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float u = x[i][j], dz = 0.f;
        if (F::gate(a) == kGateBefore) {
          const float s = sigmoid(z[i][j]);
          p[i][j] = z[i][j] * s;
          q[i][j] = u * (s + p[i][j] * (1.f - s));
          u *= p[i][j];
        }
        xh[i][j] = (u - mean) * rstd;
        float gt = unfinish<F>(a, xh[i][j] * w[i][j] + b[i][j], z[i][j], dy[i][j], dz);
        dzv[j] = dz;
        if (!in) xh[i][j] = gt = 0.f;
        dw[i][j] += gt * xh[i][j];
        db[i][j] += gt;
        gw[i][j] = gt * w[i][j];
        s0 += gw[i][j];
        s1 += gw[i][j] * xh[i][j];
      }
      if (F::gate(a) == kGateAfter && in) store_vec<BF16, VEC>(a.dz, row * a.C + c0 + c, dzv);
    }
    group_totals(s0, s1, lanes, red, half);
    if (!live) continue;
    const float m0 = a.center ? s0 * inv : 0.f, m1 = s1 * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (l + i * lanes) * VEC;
      if (c >= Cg) break;
      float dx[VEC], dz[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dx[j] = rstd * (gw[i][j] - m0 - xh[i][j] * m1);
        if (F::gate(a) == kGateBefore) {
          dz[j] = dx[j] * q[i][j];
          dx[j] *= p[i][j];
        }
      }
      store_vec<BF16, VEC>(a.dx, row * a.C + c0 + c, dx);
      if (F::gate(a) == kGateBefore) store_vec<BF16, VEC>(a.dz, row * a.C + c0 + c, dz);
    }
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (l + i * lanes) * VEC;
    if (c >= Cg) break;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (a.dw) a.ws[((long)part * 2) * a.C + c0 + c + j] = dw[i][j];
      if (a.db) a.ws[((long)part * 2 + 1) * a.C + c0 + c + j] = db[i][j];
    }
  }
}

// out[c] = sum over parts of ws[part][which][c] (which = blockIdx.y: dw or
// dbias): 16 channels by 16 lanes of parts a workgroup, joined in a fixed order.
__global__ __launch_bounds__(kThreads) void norm_sum_parts_kernel(const float* __restrict__ ws, int parts, int C,
                                                                  float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float acc[16][17];
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int cl = threadIdx.x & 15, pl = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cl;
  const float* src = ws + (long)blockIdx.y * C + (c < C ? c : 0);
  constexpr int kAhead = 8;
  float s[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) s[k] = 0.f;
  int p = pl;
  for (; p + 16 * (kAhead - 1) < parts; p += 16 * kAhead)
#pragma unroll
    for (int k = 0; k < kAhead; ++k) s[k] += src[(long)(p + 16 * k) * 2 * C];
  for (; p < parts; p += 16) s[0] += src[(long)p * 2 * C];
#pragma unroll
  for (int k = 1; k < kAhead; ++k) s[0] += s[k];
  acc[pl][cl] = s[0];
  __syncthreads();
  if (pl == 0 && c < C) {
    float t = 0.f;
    for (int k = 0; k < 16; ++k) t += acc[k][cl];
    out[c] = t;
  }
}

// ---------------------------------------------------------------- several positions a sample

// A workgroup takes `cols` columns of VEC channels by kThreads / cols rows at a
// time, kSlabRounds rounds: one slab.
constexpr int kSlabRounds = 8;

struct Slabs {
  int cols, rows, tiles;   // thread columns, rows a round, column tiles
  long count;              // slabs a sample
};
inline Slabs slabs_of(long s, int C, int vec) {
  Slabs b;
  const int pieces = (C + vec - 1) / vec;
  b.tiles = (pieces + 63) / 64;
  b.cols = (pieces + b.tiles - 1) / b.tiles;
  b.rows = kThreads / b.cols;
  b.count = (s + (long)b.rows * kSlabRounds - 1) / ((long)b.rows * kSlabRounds);
  return b;
}

// Sum of v[VEC] over the workgroup's thread rows, in row order; every thread receives its column's.
template <int VEC>
__device__ __forceinline__ void rows_total(float* v, int cols, int rows, float* lds) {
  const int tx = threadIdx.x % cols, ty = threadIdx.x / cols;
  __syncthreads();
  if (ty < rows) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) lds[(ty * VEC + j) * cols + tx] = v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = 0.f;
#pragma unroll 2
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] += lds[(r * VEC + j) * cols + tx];
}

// The rows of one thread's column in a slab, all in flight at once: rows past
// the sample's end read its last row, columns past C the first column; neither counts.
template <bool BF16, int VEC>
struct SlabRows {
  Raw<BF16, VEC> v[kSlabRounds];
  __device__ __forceinline__ void load(const void* p, long row0, long pitch, int rows, int ty, long have, int c) {
#pragma unroll
    for (int k = 0; k < kSlabRounds; ++k) v[k].load(p, (row0 + min(ty + (long)k * rows, have - 1)) * pitch + c);
  }
};

// A thread's place in the slab form.
struct SlabAt {
  int tx, ty, c;       // thread column and row, first channel
  long slab, n;        // slab and sample
  long row0, have;     // first row of the slab, its rows
};
template <int VEC>
__device__ __forceinline__ SlabAt slab_at(const NormArgs& a, const Slabs& b) {
  SlabAt s;
  const int tile = (int)(blockIdx.x % b.tiles);
  s.slab = blockIdx.x / b.tiles % b.count;
  s.n = blockIdx.x / b.tiles / b.count;
  s.tx = threadIdx.x % b.cols;
  s.ty = threadIdx.x / b.cols;
  s.c = s.ty < b.rows ? (tile * b.cols + s.tx) * VEC : a.C;   // threads beyond the last row stand outside
  const long r0 = s.slab * b.rows * kSlabRounds;
  s.row0 = s.n * a.s + r0;
  s.have = min((long)b.rows * kSlabRounds, a.s - r0);
  return s;
}

// The groups of VEC channels from c on.
template <int VEC>
__device__ __forceinline__ void groups_of(int c, int Cg, int* g) {
  int at = c / Cg, left = Cg - c % Cg;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    g[j] = at;
    if (--left == 0) {
      ++at;
      left = Cg;
    }
  }
}

// First launch: ws [n][slab][2][C]: each slab's mean and squared deviations from it, per channel.
template <bool BF16, int VEC>
__global__ __launch_bounds__(kThreads) void norm_slab_kernel(NormArgs a, Slabs b) {
  __shared__ float lds[kThreads * VEC];
  const SlabAt at = slab_at<VEC>(a, b);
  const bool in = at.c < a.C;
  const int c = in ? at.c : 0;
  SlabRows<BF16, VEC> x, z;
  x.load(a.x, at.row0, a.x_row, b.rows, at.ty, at.have, c);
  if (a.gate == kGateBefore) z.load(a.z, at.row0, a.z_row, b.rows, at.ty, at.have, c);
  float u[kSlabRounds][VEC], sum[VEC], dev[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[j] = dev[j] = 0.f;
#pragma unroll
  for (int k = 0; k < kSlabRounds; ++k) {
    const bool row = at.ty + (long)k * b.rows < at.have;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      u[k][j] = x.v[k][j];
      if (a.gate == kGateBefore) u[k][j] *= z.v[k][j] * sigmoid(z.v[k][j]);
      sum[j] += row ? u[k][j] : 0.f;
    }
  }
  rows_total<VEC>(sum, b.cols, b.rows, lds);
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[j] /= (float)at.have;   // divided, so that equal values have exactly their mean
#pragma unroll
  for (int k = 0; k < kSlabRounds; ++k) {
    const bool row = at.ty + (long)k * b.rows < at.have;
#pragma unroll
    for (int j = 0; j < VEC; ++j) dev[j] += row ? (u[k][j] - sum[j]) * (u[k][j] - sum[j]) : 0.f;
  }
  rows_total<VEC>(dev, b.cols, b.rows, lds);
  if (at.ty == 0 && in) {
    float* out = a.ws + (at.n * b.count + at.slab) * 2 * a.C + c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      out[j] = sum[j];
      out[a.C + j] = dev[j];
    }
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = lanes_sum(v, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < kThreads / 64; ++w) t += red[w];
  return t;
}

// One group of one sample: joins its slabs and channels about their common
// mean. Threads take a channel's slabs one after the other, several at a time
// where a group has few channels; two in flight (1 x 1024 positions of 512
// channels in 8 groups: a call of 18.5 us without, 16.0 with two, 15 with four,
// which cost 64 x 256 positions of 512 in 32 groups 1 us of 22).
__global__ __launch_bounds__(kThreads) void norm_join_kernel(NormArgs a, int slabs, int slab_rows, float* stats) {
  __shared__ float red[kThreads / 64];
  const int Cg = a.C / a.G;
  const long n = blockIdx.x / a.G;
  const int g = (int)(blockIdx.x % a.G);
  const float* ws = a.ws + n * slabs * 2 * a.C + (long)g * Cg;
  const int per = Cg < kThreads ? Cg : kThreads, lanes = kThreads / per;   // threads across a slab's channels; slabs at a time
  const int l = threadIdx.x % per, s0 = threadIdx.x / per;
  const int last = (int)(a.s - (long)(slabs - 1) * slab_rows);             // rows of the last slab
  float sum = 0.f;
  if (s0 < lanes)
    for (int c = l; c < Cg; c += per)
#pragma unroll 2
      for (int i = s0; i < slabs; i += lanes) sum += ws[(long)i * 2 * a.C + c] * (float)(i + 1 < slabs ? slab_rows : last);
  const float mean = block_sum(sum, red) / ((float)a.s * (float)Cg);
  float d = 0.f;
  if (s0 < lanes)
    for (int c = l; c < Cg; c += per)
#pragma unroll 2
      for (int i = s0; i < slabs; i += lanes) {
        const float off = ws[(long)i * 2 * a.C + c] - mean;
        d += ws[((long)i * 2 + 1) * a.C + c] + (float)(i + 1 < slabs ? slab_rows : last) * off * off;
      }
  float var = block_sum(d, red) / ((float)a.s * (float)Cg);
  if (!a.center) var += mean * mean;
  if (threadIdx.x == 0) {
    stats[2 * blockIdx.x] = a.center ? mean : 0.f;
    stats[2 * blockIdx.x + 1] = 1.f / sqrtf(var + a.eps);
  }
}

template <bool BF16, int VEC>
__global__ __launch_bounds__(kThreads) void norm_apply_kernel(NormArgs a, Slabs b, const float* __restrict__ stats) {
  const SlabAt at = slab_at<VEC>(a, b);
  if (at.c >= a.C) return;
  const int c = at.c;
  SlabRows<BF16, VEC> x, z;
  x.load(a.x, at.row0, a.x_row, b.rows, at.ty, at.have, c);
  if (a.gate) z.load(a.z, at.row0, a.z_row, b.rows, at.ty, at.have, c);
  float mean[VEC], rstd[VEC], w[VEC], bias[VEC];
  load_par<VEC>(a.w, c, 1.f, w);
  load_par<VEC>(a.bias, c, 0.f, bias);
  int g[VEC];
  groups_of<VEC>(c, a.C / a.G, g);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    mean[j] = stats[2 * (at.n * a.G + g[j])];
    rstd[j] = stats[2 * (at.n * a.G + g[j]) + 1];
  }
#pragma unroll
  for (int k = 0; k < kSlabRounds; ++k) {
    const long r = at.ty + (long)k * b.rows;
    if (r >= at.have) break;
    float u[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float sz = a.gate ? z.v[k][j] * sigmoid(z.v[k][j]) : 0.f;
      const float v = a.gate == kGateBefore ? x.v[k][j] * sz : x.v[k][j];
      u[j] = finish<AnyForm>(a, (v - mean[j]) * rstd[j] * w[j] + bias[j], sz);
    }
    store_vec<BF16, VEC>(a.y, (at.row0 + r) * a.C + c, u);
  }
}

// Backwards, first launch: ws [n][slab][2][C]: each slab's sums of g xh and g per channel.
template <bool BF16, int VEC>
__global__ __launch_bounds__(kThreads) void norm_slab_bwd_kernel(NormArgs a, Slabs b) {
  __shared__ float lds[kThreads * VEC];
  const SlabAt at = slab_at<VEC>(a, b);
  const bool in = at.c < a.C;
  const int c = in ? at.c : 0;
  SlabRows<BF16, VEC> x, z, dy;
  x.load(a.x, at.row0, a.x_row, b.rows, at.ty, at.have, c);
  if (a.gate) z.load(a.z, at.row0, a.z_row, b.rows, at.ty, at.have, c);
  dy.load(a.dy, at.row0, a.C, b.rows, at.ty, at.have, c);
  float mean[VEC], rstd[VEC], w[VEC], bias[VEC], s0[VEC], s1[VEC];
  int g[VEC];
  groups_of<VEC>(c, a.C / a.G, g);
  load_par<VEC>(a.w, c, 1.f, w);
  load_par<VEC>(a.bias, c, 0.f, bias);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    mean[j] = a.stats[2 * (at.n * a.G + g[j])];
    rstd[j] = a.stats[2 * (at.n * a.G + g[j]) + 1];
    s0[j] = s1[j] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < kSlabRounds; ++k) {
    if (at.ty + (long)k * b.rows >= at.have) break;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float zj = a.gate ? z.v[k][j] : 0.f;
      const float v = a.gate == kGateBefore ? x.v[k][j] * zj * sigmoid(zj) : x.v[k][j];
      const float xh = (v - mean[j]) * rstd[j];
      float dz;
      const float gt = unfinish<AnyForm>(a, xh * w[j] + bias[j], zj, dy.v[k][j], dz);
      s0[j] += gt * xh;
      s1[j] += gt;
    }
  }
  rows_total<VEC>(s0, b.cols, b.rows, lds);
  rows_total<VEC>(s1, b.cols, b.rows, lds);
  if (at.ty == 0 && in) {
    float* out = a.ws + (at.n * b.count + at.slab) * 2 * a.C + c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      out[j] = s0[j];
      out[a.C + j] = s1[j];
    }
  }
}

// means[n][G][2]: a group's means of g w xh and of g w.
__global__ __launch_bounds__(kThreads) void norm_join_bwd_kernel(NormArgs a, int slabs, float* means) {
  __shared__ float red[kThreads / 64];
  const int Cg = a.C / a.G;
  const long n = blockIdx.x / a.G;
  const int g = (int)(blockIdx.x % a.G);
  const float* ws = a.ws + n * slabs * 2 * a.C + (long)g * Cg;
  const int per = Cg < kThreads ? Cg : kThreads, lanes = kThreads / per;
  const int l = threadIdx.x % per, i0 = threadIdx.x / per;
  float s0 = 0.f, s1 = 0.f;
  if (i0 < lanes)
    for (int c = l; c < Cg; c += per) {
      const float w = a.w ? a.w[g * Cg + c] : 1.f;
#pragma unroll 2
      for (int i = i0; i < slabs; i += lanes) {
        s0 += w * ws[(long)i * 2 * a.C + c];
        s1 += w * ws[((long)i * 2 + 1) * a.C + c];
      }
    }
  const float inv = 1.f / ((float)a.s * (float)Cg);
  const float t0 = block_sum(s0, red) * inv, t1 = block_sum(s1, red) * inv;
  if (threadIdx.x == 0) {
    means[2 * blockIdx.x] = t0;
    means[2 * blockIdx.x + 1] = a.center ? t1 : 0.f;
  }
}

template <bool BF16, int VEC>
__global__ __launch_bounds__(kThreads) void norm_apply_bwd_kernel(NormArgs a, Slabs b, const float* __restrict__ means) {
  const SlabAt at = slab_at<VEC>(a, b);
  if (at.c >= a.C) return;
  const int c = at.c;
  SlabRows<BF16, VEC> x, z, dy;
  x.load(a.x, at.row0, a.x_row, b.rows, at.ty, at.have, c);
  if (a.gate) z.load(a.z, at.row0, a.z_row, b.rows, at.ty, at.have, c);
  dy.load(a.dy, at.row0, a.C, b.rows, at.ty, at.have, c);
  float mean[VEC], rstd[VEC], w[VEC], bias[VEC], m0[VEC], m1[VEC];
  int g[VEC];
  groups_of<VEC>(c, a.C / a.G, g);
  load_par<VEC>(a.w, c, 1.f, w);
  load_par<VEC>(a.bias, c, 0.f, bias);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const long q = 2 * (at.n * a.G + g[j]);
    mean[j] = a.stats[q];
    rstd[j] = a.stats[q + 1];
    m1[j] = means[q];
    m0[j] = means[q + 1];
  }
#pragma unroll
  for (int k = 0; k < kSlabRounds; ++k) {
    const long r = at.ty + (long)k * b.rows;
    if (r >= at.have) break;
    float dx[VEC], dzv[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float zj = a.gate ? z.v[k][j] : 0.f;
      const float sg = a.gate == kGateBefore ? sigmoid(zj) : 0.f;
      const float u = a.gate == kGateBefore ? x.v[k][j] * zj * sg : x.v[k][j];
      const float xh = (u - mean[j]) * rstd[j];
      dzv[j] = 0.f;
      const float gt = unfinish<AnyForm>(a, xh * w[j] + bias[j], zj, dy.v[k][j], dzv[j]);
      dx[j] = rstd[j] * (gt * w[j] - m0[j] - xh * m1[j]);
      if (a.gate == kGateBefore) {
        dzv[j] = dx[j] * x.v[k][j] * silu_slope(zj, sg);
        dx[j] *= zj * sg;
      }
    }
    store_vec<BF16, VEC>(a.dx, (at.row0 + r) * a.C + c, dx);
    if (a.gate) store_vec<BF16, VEC>(a.dz, (at.row0 + r) * a.C + c, dzv);
  }
}

// Whether (and how) a group fits the registers of the threads that share it:
// up to 64 pieces a power of two of lanes, one piece each; above that the
// workgroup, in as many whole waves as the pieces fill (up to 16), so that no
// lane idles for a power of two. Beyond that (8192 channels in pieces of 8,
// 2048 in single ones, two a lane) the slab form takes over.
struct RowPlan {
  int vec, nv, lanes, threads;
};
bool row_plan(const NormArgs& a, RowPlan* p) {
  if (a.s != 1) return false;
  const int Cg = a.C / a.G;
  p->vec = a.vec && Cg % 8 == 0 ? 8 : 1;
  const int pieces = Cg / p->vec;
  p->threads = kThreads;
  p->nv = 1;
  if (pieces <= 64) {
    p->lanes = 1;
    while (p->lanes < pieces) p->lanes *= 2;
    return true;
  }
  p->nv = (pieces + 1023) / 1024;
  if (p->nv > (p->vec == 8 ? 1 : 2)) return false;
  p->lanes = ((pieces + p->nv - 1) / p->nv + 63) / 64 * 64;
  p->threads = p->lanes;
  return true;
}

// Rows of partial sums of the one-position backward pass: workgroups of eight
// waves for every CU, which with the next row's loads in flight keep the
// memory busy, and no more rows than there are.
struct RowParts {
  int groups, rows, tiles, blocks;
};
RowParts row_parts(const NormArgs& a, const RowPlan& p) {
  RowParts r;
  const int workers = p.lanes > 64 ? 1 : kThreads / p.lanes;
  r.groups = a.G < workers ? a.G : workers;
  r.rows = workers / r.groups;
  r.tiles = (a.G + r.groups - 1) / r.groups;
  const int want = kCus * (p.threads > 512 ? 1 : 512 / p.threads);
  long blocks = (want + r.tiles - 1) / r.tiles;
  const long most = (a.n + r.rows - 1) / r.rows;
  if (blocks > most) blocks = most;
  if (blocks * r.rows > kMaxParts) blocks = kMaxParts / r.rows;
  r.blocks = blocks < 1 ? 1 : (int)blocks;
  return r;
}

}  // namespace

size_t norm_ws_floats(long n, long s, int C, int G, bool backward) {
  // The slab form with the narrowest pieces has the most slabs; the
  // one-position backward pass leaves at most 1024 rows of partial sums.
  size_t most = 0;
  for (int vec : {1, 8}) {
    const Slabs b = slabs_of(s, C, vec);
    const size_t f = (size_t)n * b.count * 2 * C + (size_t)n * G * 2;
    if (f > most) most = f;
  }
  if (s == 1) {
    const size_t rows = (n < kMaxParts ? (size_t)n : kMaxParts) + kThreads;
    const size_t parts = backward ? 2 * rows * C : 0;
    if (C / G <= 2048) return parts;  // fits registers with any alignment
    if (parts > most) most = parts;
  }
  return most;
}

namespace {

template <bool BF16, int VEC, int NV, int GATE, bool SILU, bool WHOLE>
void row_form(const NormArgs& a, const RowPlan& p, bool backward, hipStream_t stream) {
  const dim3 block((unsigned)p.threads);
  if (!backward) {
    const long workers = p.lanes > 64 ? 1 : kThreads / p.lanes;
    const dim3 grid((unsigned)((a.n * a.G + workers - 1) / workers));
    hipLaunchKernelGGL((norm_row_kernel<BF16, VEC, NV, GATE, SILU, WHOLE>), grid, block, 0, stream, a, p.lanes);
    return;
  }
  const RowParts r = row_parts(a, p);
  hipLaunchKernelGGL((norm_row_bwd_kernel<BF16, VEC, NV, GATE, SILU, WHOLE>), dim3((unsigned)(r.tiles * r.blocks)), block, 0,
                     stream, a, p.lanes, r.groups, r.rows, r.blocks);
  if (a.dw || a.db)
    hipLaunchKernelGGL(norm_sum_parts_kernel, dim3((unsigned)((a.C + 15) / 16), 2), dim3(kThreads), 0, stream, a.ws,
                       r.rows * r.blocks, a.C, a.dw, a.db);
}

// Pieces of eight: the form is fixed at compile time, as the arithmetic of the
// gate is a good part of the time; single channels read it from the arguments.
template <bool BF16, int VEC, bool WHOLE>
void row_launch(const NormArgs& a, const RowPlan& p, bool backward, hipStream_t stream) {
  if constexpr (VEC == 8) {
    switch (2 * a.gate + (a.silu ? 1 : 0)) {
      case 0: return row_form<BF16, 8, 1, 0, false, WHOLE>(a, p, backward, stream);
      case 1: return row_form<BF16, 8, 1, 0, true, WHOLE>(a, p, backward, stream);
      case 2: return row_form<BF16, 8, 1, 1, false, WHOLE>(a, p, backward, stream);
      case 3: return row_form<BF16, 8, 1, 1, true, WHOLE>(a, p, backward, stream);
      case 4: return row_form<BF16, 8, 1, 2, false, WHOLE>(a, p, backward, stream);
      default: return row_form<BF16, 8, 1, 2, true, WHOLE>(a, p, backward, stream);
    }
  } else if (p.nv == 1) {
    row_form<BF16, 1, 1, -1, false, WHOLE>(a, p, backward, stream);
  } else {
    row_form<BF16, 1, 2, -1, false, true>(a, p, backward, stream);
  }
}

template <bool BF16, int VEC>
void slab_launch(const NormArgs& a, hipStream_t stream) {
  const Slabs b = slabs_of(a.s, a.C, VEC);
  const dim3 grid((unsigned)(a.n * b.count * b.tiles)), groups((unsigned)(a.n * a.G)), block(kThreads);
  float* stats = a.stats ? a.stats : a.ws + a.n * b.count * 2 * a.C;
  hipLaunchKernelGGL((norm_slab_kernel<BF16, VEC>), grid, block, 0, stream, a, b);
  hipLaunchKernelGGL(norm_join_kernel, groups, block, 0, stream, a, (int)b.count, b.rows * kSlabRounds, stats);
  hipLaunchKernelGGL((norm_apply_kernel<BF16, VEC>), grid, block, 0, stream, a, b, (const float*)stats);
}

template <bool BF16, int VEC>
void slab_bwd_launch(const NormArgs& a, hipStream_t stream) {
  const Slabs b = slabs_of(a.s, a.C, VEC);
  const dim3 grid((unsigned)(a.n * b.count * b.tiles)), groups((unsigned)(a.n * a.G)), block(kThreads);
  float* means = a.ws + a.n * b.count * 2 * a.C;
  hipLaunchKernelGGL((norm_slab_bwd_kernel<BF16, VEC>), grid, block, 0, stream, a, b);
  hipLaunchKernelGGL(norm_join_bwd_kernel, groups, block, 0, stream, a, (int)b.count, means);
  hipLaunchKernelGGL((norm_apply_bwd_kernel<BF16, VEC>), grid, block, 0, stream, a, b, (const float*)means);
  if (a.dw || a.db)
    hipLaunchKernelGGL(norm_sum_parts_kernel, dim3((unsigned)((a.C + 15) / 16), 2), block, 0, stream, a.ws,
                       (int)(a.n * b.count), a.C, a.dw, a.db);
}

template <typename F>
void by_type(bool bf16, bool vec, F f) {
  using T = std::true_type;
  using N = std::false_type;
  if (bf16) {
    if (vec) f(T{}, std::integral_constant<int, 8>{});
    else f(T{}, std::integral_constant<int, 1>{});
  } else {
    if (vec) f(N{}, std::integral_constant<int, 8>{});
    else f(N{}, std::integral_constant<int, 1>{});
  }
}

}  // namespace

bool norm_launchable(const NormArgs& a) {
  RowPlan p;
  if (row_plan(a, &p)) {
    const long workers = p.lanes > 64 ? 1 : kThreads / p.lanes;
    return launchable((a.n * a.G + workers - 1) / workers, p.threads);
  }
  const Slabs b = slabs_of(a.s, a.C, a.vec ? 8 : 1);
  return launchable(a.n * b.count * b.tiles, kThreads) && launchable(a.n * a.G, kThreads);
}

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream) {
  RowPlan p;
  const bool row = row_plan(a, &p);
  by_type(a.bf16, row ? p.vec == 8 : a.vec, [&](auto bf, auto vec) {
    if (row && p.lanes > 64) row_launch<decltype(bf)::value, decltype(vec)::value, true>(a, p, false, stream);
    else if (row) row_launch<decltype(bf)::value, decltype(vec)::value, false>(a, p, false, stream);
    else slab_launch<decltype(bf)::value, decltype(vec)::value>(a, stream);
  });
  return hipGetLastError();
}

hipError_t launch_group_norm_bwd(const NormArgs& a, hipStream_t stream) {
  RowPlan p;
  const bool row = row_plan(a, &p);
  by_type(a.bf16, row ? p.vec == 8 : a.vec, [&](auto bf, auto vec) {
    if (row && p.lanes > 64) row_launch<decltype(bf)::value, decltype(vec)::value, true>(a, p, true, stream);
    else if (row) row_launch<decltype(bf)::value, decltype(vec)::value, false>(a, p, true, stream);
    else slab_bwd_launch<decltype(bf)::value, decltype(vec)::value>(a, stream);
  });
  return hipGetLastError();
}

}  // namespace ssd
