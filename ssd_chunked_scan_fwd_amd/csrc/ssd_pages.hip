// ssd_pages.hip -- pages of a pool of states, [layers][slots][page]: copied
// (forked, permuted), compacted, cleared. All are bound by the bytes they
// read and write: 4 sequences' pages forked to 28, 2 layers of 1 MB a page, 67 MB
// with each source read once: 16 us (4.2 TB/s). Lists of disjoint pairs, 2 layers
// of 1 MB a page: 64 pairs 42 us (6.4 TB/s), 256 238 (4.5), 1024 1520 (2.8), as longer
// lists leave shorter runs. 60 live pages of 96 of 393 KB made dense, 18 MB: 3 + 6
// us of two launches, 15 us a call. 28 pages cleared, 59 MB: 10 us (6.0 TB/s).
#include "ssd_device.h"
#include "ssd_layer.h"

namespace ssd {

namespace {

constexpr int kPageThreads = 256;
constexpr int kCopyHeld = 16;   // pieces a thread holds between the reads and the writes

// ----------------------------------------------------------------------------
// pool[dst[i]] = pool[src[i]] for all pairs at once: every source is read
// before any destination is written, whatever the lists share. Pages are only
// ever exchanged at equal offsets, so a workgroup that owns a range of offsets
// (`lanes` consecutive pieces) of one layer reads that range of every source
// into registers, waits, and writes it; nothing crosses workgroups. Of several
// pairs with one destination the last is kept; a pair with an index outside the
// pool is left out. A workgroup walks several ranges, so the pairs are checked
// once.
// ----------------------------------------------------------------------------
template <typename W>
__global__ __launch_bounds__(kPageThreads) void pages_copy_kernel(PagesArgs a, const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst, int n, int lanes,
                                                                  long ranges) {
  __shared__ int from[kMaxPagePairs], to[kMaxPagePairs];
  for (int i = threadIdx.x; i < n; i += kPageThreads) {
    const int f = src[i], t = dst[i];
    const bool in = f >= 0 && f < a.slots && t >= 0 && t < a.slots;
    from[i] = f;
    to[i] = in ? t : -1;
  }
  __syncthreads();
  bool lost[kMaxPagePairs / kPageThreads];
#pragma unroll
  for (int m = 0; m < kMaxPagePairs / kPageThreads; ++m) {
    const int i = threadIdx.x + m * kPageThreads;
    lost[m] = false;
    if (i < n)
      for (int j = i + 1; j < n; ++j) lost[m] |= to[j] == to[i];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kMaxPagePairs / kPageThreads; ++m) {
    const int i = threadIdx.x + m * kPageThreads;
    if (i < n && (lost[m] || from[i] == to[i])) to[i] = -1;
  }
  __syncthreads();

  const int c = threadIdx.x % lanes, p0 = threadIdx.x / lanes, per = kPageThreads / lanes;
  const long pieces = a.page / (long)sizeof(W);
  const long across = (pieces + lanes - 1) / lanes;
  for (long r = blockIdx.x; r < ranges; r += gridDim.x) {
    const long layer = r / across, col = (r % across) * lanes + c;
    W* base = reinterpret_cast<W*>(a.pool) + layer * a.slots * pieces + col;
    W v[kCopyHeld];
    const bool in = col < pieces;
#pragma unroll
    for (int k = 0; k < kCopyHeld; ++k) {
      const int i = p0 + k * per;
      if (in && i < n && to[i] >= 0) v[k] = base[(long)from[i] * pieces];
    }
    // The reads have returned in every wave before the first write is issued.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCopyHeld; ++k) {
      const int i = p0 + k * per;
      if (in && i < n && to[i] >= 0) base[(long)to[i] * pieces] = v[k];
    }
  }
}

template <typename W>
__global__ __launch_bounds__(kPageThreads) void pages_clear_kernel(PagesArgs a, const int32_t* __restrict__ slots) {
  const int s = slots[blockIdx.y];
  if (s < 0 || s >= a.slots) return;
  const long pieces = a.page / (long)sizeof(W);
  W* base = reinterpret_cast<W*>(a.pool) + ((long)blockIdx.z * a.slots + s) * pieces;
  for (long i = (long)blockIdx.x * kPageThreads + threadIdx.x; i < pieces; i += (long)gridDim.x * kPageThreads) base[i] = W{};
}

// ----------------------------------------------------------------------------
// Compaction. With `count` live pages, the k-th live page at or above `count`
// moves into the k-th hole below it; live pages below stay. No page is both
// read and written, so the moves need no order. One workgroup draws up the list
// (ws: the number of moves, then sources, then destinations), then a second
// launch moves the pages.
// ----------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// Exclusive prefix of two 0/1 flags over the workgroup's threads, and their totals.
__device__ __forceinline__ void block_ranks(bool f0, bool f1, int* part, int& r0, int& r1, int& n0, int& n1) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned long long b0 = __ballot(f0), b1 = __ballot(f1), below = (1ull << lane) - 1;
  if (lane == 0) {
    part[2 * wave] = __popcll(b0);
    part[2 * wave + 1] = __popcll(b1);
  }
  __syncthreads();
  r0 = __popcll(b0 & below);
  r1 = __popcll(b1 & below);
  n0 = n1 = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) {
      r0 += part[2 * w];
      r1 += part[2 * w + 1];
    }
    n0 += part[2 * w];
    n1 += part[2 * w + 1];
  }
  __syncthreads();
}

__global__ __launch_bounds__(kPlanThreads) void pages_plan_kernel(const uint8_t* __restrict__ live, int slots,
                                                                  int32_t* __restrict__ where, int32_t* __restrict__ count,
                                                                  int32_t* __restrict__ ws) {
  __shared__ int part[2 * kPlanThreads / 64];
  const int half = slots / 2 + 1;
  int32_t *from = ws + 64, *to = from + half;
  int total = 0, r0, r1, n0, n1;
  for (int i0 = 0; i0 < slots; i0 += kPlanThreads) {
    const int i = i0 + (int)threadIdx.x;
    block_ranks(i < slots && live[i] != 0, false, part, r0, r1, n0, n1);
    total += n0;
  }
  int holes = 0, highs = 0;
  for (int i0 = 0; i0 < slots; i0 += kPlanThreads) {
    const int i = i0 + (int)threadIdx.x;
    const bool in = i < slots, on = in && live[i] != 0;
    const bool hole = in && !on && i < total, high = on && i >= total;
    block_ranks(hole, high, part, r0, r1, n0, n1);
    if (hole) to[holes + r0] = i;
    if (high) from[highs + r1] = i;
    if (in && !high) where[i] = on ? i : -1;
    holes += n0;
    highs += n1;
  }
  __threadfence_block();
  __syncthreads();
  for (int k = threadIdx.x; k < highs; k += kPlanThreads) where[from[k]] = to[k];
  if (threadIdx.x == 0) {
    ws[0] = highs;
    *count = total;
  }
}

template <typename W>
__global__ __launch_bounds__(kPageThreads) void pages_move_kernel(PagesArgs a, const int32_t* __restrict__ ws) {
  const int half = a.slots / 2 + 1;
  const int32_t *from = ws + 64, *to = from + half;
  const long pieces = a.page / (long)sizeof(W);
  constexpr int kHeld = 4;
  const long across = (pieces + kHeld * kPageThreads - 1) / (kHeld * kPageThreads);
  const long total = (long)ws[0] * a.layers * across;
  for (long u = blockIdx.x; u < total; u += gridDim.x) {
    const long pair = u / (a.layers * across), layer = u / across % a.layers;
    const long c0 = (u % across) * kHeld * kPageThreads + threadIdx.x;
    W* base = reinterpret_cast<W*>(a.pool) + layer * a.slots * pieces;
    const W* f = base + (long)from[pair] * pieces;
    W* t = base + (long)to[pair] * pieces;
    W v[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (c0 + k * kPageThreads < pieces) v[k] = f[c0 + k * kPageThreads];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (c0 + k * kPageThreads < pieces) t[c0 + k * kPageThreads] = v[k];
  }
}

// The widest piece (16, 4 or 1 bytes) that pages and pool are whole numbers of.
int piece_bytes(const PagesArgs& a) {
  const uintptr_t m = (uintptr_t)a.pool | (uintptr_t)a.page;
  return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : 1;
}

template <typename F>
void with_piece(const PagesArgs& a, F f) {
  switch (piece_bytes(a)) {
    case 16: f(u32x4{}); break;
    case 4: f(uint32_t{}); break;
    default: f(uint8_t{}); break;
  }
}

}  // namespace

hipError_t launch_pages_copy(const PagesArgs& a, const int32_t* src, const int32_t* dst, int n, hipStream_t stream) {
  // As many consecutive pieces of a page as let a workgroup hold all n pairs:
  // 64 (1 KiB of a page) up to 64 pairs, 4 (64 bytes) at 1024. 28 pairs with 64,
  // 16 and 4: 16, 19 and 45 us.
  int lanes = 64;
  while (lanes > 4 && n > kCopyHeld * (kPageThreads / lanes)) lanes /= 2;
  with_piece(a, [&](auto w) {
    using W = decltype(w);
    const long pieces = a.page / (long)sizeof(W);
    const long ranges = a.layers * ((pieces + lanes - 1) / lanes);
    // Two ranges or more a workgroup, so that its list is checked less often (28
    // pages of 2 MiB forked from 4: 17 us with 1024 workgroups, 19 with 2048, 18.5 with 512).
    const unsigned blocks = (unsigned)(ranges < 1024 ? ranges : 1024);
    hipLaunchKernelGGL(pages_copy_kernel<W>, dim3(blocks), dim3(kPageThreads), 0, stream, a, src, dst, n, lanes, ranges);
  });
  return hipGetLastError();
}

hipError_t launch_pages_clear(const PagesArgs& a, const int32_t* slots, int n, hipStream_t stream) {
  with_piece(a, [&](auto w) {
    using W = decltype(w);
    const long pieces = a.page / (long)sizeof(W);
    const long want = (pieces + 4 * kPageThreads - 1) / (4 * kPageThreads);
    const dim3 grid((unsigned)(want < 256 ? want : 256), (unsigned)n, (unsigned)a.layers);
    hipLaunchKernelGGL(pages_clear_kernel<W>, grid, dim3(kPageThreads), 0, stream, a, slots);
  });
  return hipGetLastError();
}

size_t pages_compact_ws_bytes(int slots) { return 256 + 2 * ((size_t)slots / 2 + 1) * 4; }

hipError_t launch_pages_compact(const PagesArgs& a, const uint8_t* live, int32_t* where, int32_t* count, void* ws,
                                hipStream_t stream) {
  int32_t* list = static_cast<int32_t*>(ws);
  hipLaunchKernelGGL(pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, live, a.slots, where, count, list);
  with_piece(a, [&](auto w) {
    using W = decltype(w);
    const long across = (a.page / (long)sizeof(W) + 4 * kPageThreads - 1) / (4 * kPageThreads);
    const long most = (long)(a.slots / 2) * a.layers * across;  // no more than half of the pages move
    const unsigned blocks = (unsigned)(most < 1 ? 1 : most < 2048 ? most : 2048);
    hipLaunchKernelGGL(pages_move_kernel<W>, dim3(blocks), dim3(kPageThreads), 0, stream, a, list);
  });
  return hipGetLastError();
}

}  // namespace ssd
