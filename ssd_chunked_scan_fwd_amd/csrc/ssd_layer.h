// ssd_layer.h -- internal launchers of the group norm, of the pages of a state
// pool and of rotary positions. Arguments have been validated by the C-ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

enum { kGateNone = 0, kGateAfter = 1, kGateBefore = 2 };

struct NormArgs {
  const void *x = nullptr, *z = nullptr, *dy = nullptr;  // rows of `C` channels; x and z may have a row pitch
  const float *w = nullptr, *bias = nullptr;             // [C] or null (1 and 0)
  void *y = nullptr, *dx = nullptr, *dz = nullptr;       // contiguous rows
  float *stats = nullptr;                                // [n][G][2]: mean (0 when not centred), 1 / deviation
  float *dw = nullptr, *db = nullptr;                    // [C], each may be null
  float* ws = nullptr;
  long n = 0, s = 0;                                     // samples, positions a sample
  int C = 0, G = 0;
  long x_row = 0, z_row = 0;
  float eps = 0.f;
  int bf16 = 0, silu = 0, gate = 0, center = 1;
  bool vec = false;                                      // every row of 8-channel pieces is 16-byte aligned
};

// Floats of workspace of a forward and of a backward call (an upper bound over
// alignments).
size_t norm_ws_floats(long n, long s, int C, int G, bool backward);
bool norm_launchable(const NormArgs& a);
hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_group_norm_bwd(const NormArgs& a, hipStream_t stream);

struct PagesArgs {
  char* pool = nullptr;     // [layers][slots][page] bytes
  int layers = 0, slots = 0;
  long page = 0;
};
// Whether the runtime, which counts the threads of a grid's dimension in 32
// bits, takes that many workgroups.
inline bool launchable(long workgroups, int threads) { return workgroups <= (long)(UINT32_MAX / (unsigned)threads); }

constexpr int kMaxPagePairs = 1024;
hipError_t launch_pages_copy(const PagesArgs& a, const int32_t* src, const int32_t* dst, int n, hipStream_t stream);
hipError_t launch_pages_clear(const PagesArgs& a, const int32_t* slots, int n, hipStream_t stream);
size_t pages_compact_ws_bytes(int slots);
hipError_t launch_pages_compact(const PagesArgs& a, const uint8_t* live, int32_t* where, int32_t* count, void* ws,
                                hipStream_t stream);

struct RotaryArgs {
  const void* x[2] = {nullptr, nullptr};   // queries and keys, rows x_row apart
  void* y[2] = {nullptr, nullptr};
  long x_row[2] = {0, 0}, y_row[2] = {0, 0};
  int heads[2] = {0, 0};
  const float* freq = nullptr;             // [rot / 2]
  const int32_t* positions = nullptr;      // [tokens] or null: the token's place in its sequence
  const int32_t* cu = nullptr;
  const int32_t* offsets = nullptr;        // [sequences] added to those places, or null
  float scale = 1.f;
  int batch = 1, T = 0, S = 0, d = 0, rot = 0, interleaved = 0, inverse = 0, bf16 = 0;
};
bool rotary_launchable(const RotaryArgs& a);
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);

}  // namespace ssd
