// fl_serving.h -- what the serving operators' translation units share: argument
// checks, the tensor maps of strided caches, and the prefix attention's launch
// (also made by a context's decode step).
#pragma once
#include <cstdio>
#include <string>

#include "flashloop.h"
#include "fl_internal.h"

namespace fl {

inline int ceil_div_i(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }
inline size_t align256_sz(size_t v) { return (v + 255) & ~size_t(255); }
inline bool is_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Failures leave their reason where flashloop_last_cuda_error(NULL) reports it.
// (Keeping the reason may need memory: without any, the status alone is left, and no exception crosses a C entry.)
inline fl_status refuse(fl_status st, const char* why) {
  try {
    set_last_error(why);
  } catch (...) {
  }
  return st;
}
inline fl_status refuse_scratch(size_t need) {
  char why[96];
  std::snprintf(why, sizeof why, "scratch must be 256-byte aligned and hold %zu bytes", need);
  return refuse(FL_ERR_WORKSPACE, why);
}
inline fl_status cuda_status(cudaError_t e) {
  return e == cudaSuccess ? FL_OK : refuse(FL_ERR_CUDA, cudaGetErrorString(e));
}

// A ring of `slots` barriers, load n on slot n % slots in its phase n / slots: wait(slot, parity) for each of the
// `issued` loads that may still be under way, the oldest first (those before them had to arrive for their slots).
template <class N, class Wait>
__host__ __device__ inline void each_in_flight(N issued, int slots, Wait wait) {
  for (N n = issued > slots ? issued - slots : 0; n < issued; ++n)
    wait(static_cast<int>(n % slots), static_cast<int>(n / slots) & 1);
}

// A stride is usable when its dimension has one element or it is a positive multiple of `unit`.
inline bool stride_ok(int64_t stride, int64_t dim, int64_t unit) {
  return dim <= 1 || (stride > 0 && stride % unit == 0 && stride < (int64_t(1) << 38));
}

// Tensor map over bf16 rows [n2][n1][rows][hd] with element strides, as [n2][n1][hd / 64][rows][64]: one copy brings
// box_rows rows of all dims, the halves of a 128-dim row one behind the other, 128-byte swizzle.
bool encode_tmap_rows(CUtensorMap* map, const void* base, int hd, int64_t rows, int64_t n1, int64_t n2,
                      int64_t s_row, int64_t s1, int64_t s2, uint32_t box_rows);

// Tensor map over bf16 queries [B][Tq][H][hd] with element strides, 128-byte
// swizzle, box 64 dims x box_heads heads x box_queries queries.
bool encode_tmap_queries(CUtensorMap* map, const void* base, int hd, int H, int Tq, int B, int64_t s_h, int64_t s_t,
                         int64_t s_b, uint32_t box_heads, uint32_t box_queries);

// The prefix attention as launched: the C arguments, or a context's decode step
// (fp32 queries, an fp32 copy of the output, lengths offset by lens_add).
struct PrefixLaunch {
  flashloop_prefix_args a;
  const float* q32;     // fp32 queries [B][Tq][H][hd] by q_stride (a.q unused), or nullptr
  float* out32;         // fp32 copy of the output rows [B*Tq*H][hd], or nullptr
  int lens_add;         // added to lens[b] before it is clamped
  bool pdl;             // the first launch may overlap its predecessor
  int* status;          // fp32 queries: error bits of waits that ran out, or nullptr
};
size_t prefix_scratch_bytes(int B, int Tq, int H, int Hkv, int hd, int P, int S, bool fp32_queries);
cudaError_t launch_prefix(const PrefixLaunch& L, void* scratch, cudaStream_t s);
cudaError_t serving_init_attrs();   // opt the kernels in to their shared memory (per device)

}  // namespace fl
