// fl_evict.cu -- eviction from a cache by accumulated attention weight.
//
// Two launches.  The selection finds, per (sequence, KV head), the keep-th key in
// the order (protected, weight bits descending, slot ascending) by a radix select
// and writes the source slot of every destination slot; the move copies rows.  A kept row
// below the budget stays where it is and the freed slots take the kept rows from
// beyond it, so in place the sources (slots >= keep) and the destinations (slots
// < keep) never meet and no order of the copies matters.
#include <algorithm>
#include <climits>
#include <cooperative_groups.h>

#include "fl_device.cuh"
#include "fl_serving.h"

namespace cg = cooperative_groups;

namespace fl {
namespace {

constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;
constexpr int kEvDigit = 11, kEvBins = 1 << kEvDigit;   // bits of a digit (the last has 10): four bins a thread
constexpr int kEvHeld = 16;               // slots a thread holds the positions of
constexpr int kEvCluster = 16;            // CTAs of one (sequence, KV head) at most (over 8: non-portable)
constexpr int kEvKeys = 32 * kEvThreads;  // keys one CTA holds in shared memory (64 KB), a word of 32 slots per thread
constexpr int kEvSlots = kEvCluster * kEvKeys;

struct EvictArgs {
  flashloop_evict_args c;
  int cap;              // min(keep, S): slots of a segment's map
  int chunk;            // slots per CTA of the selection
  int32_t* src;         // [B * Hkv][cap] source slot of each destination slot
  int32_t* n_kept;      // [B * Hkv]
};

// Exclusive prefix sums of the warps' counts, in place, and their total (one warp; kEvWarps of them).
__device__ __forceinline__ void scan_warps(int* v, int* total) {
  const int lane = threadIdx.x & 31, x = lane < kEvWarps ? v[lane] : 0;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane < kEvWarps) v[lane] = incl - x;
  if (lane == 31) *total = incl;
}

// ============================================================================
// Selection: a cluster of 1-16 CTAs per (sequence, KV head), each with a contiguous
// chunk of slots, its keys in shared memory.  Key: 0xFFFFFFFF when protected, else the
// weight's bits (at most 0xFFFFFFFE).  Three digits of 11, 11 and 10 bits, largest first
// (weights share their leading bits, so wide digits part more of them): every
// CTA histograms the keys that match the digits found so far, and after a
// cluster barrier sums all CTAs' histograms over distributed shared memory and
// finds the next digit by itself.  The freed slots' list stays in shared memory, where
// the CTAs look up where their kept slots go.  Latency-bound (a round trip to memory, then
// about ten barriers): 10 us at 32 segments of 4160 slots, 20 us at 32 of 65536 (8 bytes a slot
// would take 3 us).  Digits of 8 bits with 8 copies of the counters took 12 and 27 us; reading every
// bin of the other CTAs instead of sums of 64 first, 33 us at 65536.
// ============================================================================
__global__ void __launch_bounds__(kEvThreads, 2) k_evict_select(const EvictArgs a) {
  pdl_trigger();   // the move is launched, and waits for the result, while this runs
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ uint32_t keys[];        // [chunk]; in the end the freed and the moving slots' lists
  __shared__ __align__(16) int hist[2][kEvBins];   // this CTA's, one per digit parity: a cluster barrier per digit suffices
  __shared__ int group[2][32];              // its sums of 64 bins
  __shared__ int newest_sm, sel_digit, sel_before, sel_count, move_base;
  __shared__ int warp_a[kEvWarps];
  __shared__ int cta_eq, cta_both;
  __shared__ uint32_t kept_w[kEvThreads];   // kept slots, a bit each: word t is thread t's
  __shared__ int list_at[kEvThreads];       // before a word: freed slots (low half) and moving ones of this CTA
  __shared__ int hole_base[kEvCluster + 1]; // freed slots before each CTA's, and all of them
  const flashloop_evict_args& c = a.c;
  const int nc = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y, b = blockIdx.z;
  const long long seg = static_cast<long long>(b) * c.Hkv + g;
  const int len = c.lens[b];
  // ---- weights and positions (requested before the length is known: the slots are there, used or not)
  const int lo = min(c.S, rank * a.chunk), cap = min(c.S, lo + a.chunk) - lo;
  const float* acc = c.acc + b * c.acc_stride[0] + g * c.acc_stride[1] + lo;
  const int32_t* pos = c.pos + b * c.pos_stride[0] + g * c.pos_stride[1] + lo;
  int held[kEvHeld];
  {
    float w[kEvHeld];
#pragma unroll
    for (int j = 0; j < kEvHeld; ++j) {
      const int i = tid + j * kEvThreads;
      if (i < cap) {
        w[j] = acc[i];
        held[j] = pos[i];
      }
    }
#pragma unroll
    for (int j = 0; j < kEvHeld; ++j) {
      const int i = tid + j * kEvThreads;
      if (i < cap) keys[i] = min(__float_as_uint(w[j]), 0xFFFFFFFEu);
    }
  }
  const int n = min(max(len, 0), c.S), m = max(0, min(n - lo, cap));
  int32_t* src = a.src + seg * a.cap;
  if (rank == 0 && tid == 0) a.n_kept[seg] = min(n, c.keep);
  if (n <= c.keep) {   // the whole cluster alike
    for (int i = rank * kEvThreads + tid; i < n; i += nc * kEvThreads) src[i] = i;
    return;
  }
  // ---- the newest token
  int newest = INT_MIN;
#pragma unroll
  for (int j = 0; j < kEvHeld; ++j)
    if (tid + j * kEvThreads < m) newest = max(newest, held[j]);
  for (int i = tid + kEvHeld * kEvThreads; i < m; i += kEvThreads) {
    keys[i] = min(__float_as_uint(acc[i]), 0xFFFFFFFEu);
    newest = max(newest, pos[i]);
  }
  if (tid == 0) newest_sm = INT_MIN;
  *reinterpret_cast<int4*>(&hist[0][4 * tid]) = make_int4(0, 0, 0, 0);
  *reinterpret_cast<int4*>(&hist[1][4 * tid]) = make_int4(0, 0, 0, 0);
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) atomicMax(&newest_sm, newest);
  auto sync_all = [&]() {   // the cluster, or its one CTA
    if (nc > 1) cl.sync();
    else __syncthreads();
  };
  sync_all();
  newest = __reduce_max_sync(0xffffffffu, lane < nc ? *cl.map_shared_rank(&newest_sm, lane) : INT_MIN);
  const long long oldest_safe = static_cast<long long>(newest) - c.recent;   // protected above it
  auto scan_warp = [&](int v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  auto scan_block = [&](int v, int* total) {   // exclusive prefix sum over the threads (two barriers)
    const int incl = scan_warp(v);
    if (lane == 31) warp_a[warp] = incl;
    __syncthreads();
    if (warp == 0) scan_warps(warp_a, total);
    __syncthreads();
    return warp_a[warp] + incl - v;
  };
  // ---- the digits of the keep-th key
  uint32_t prefix = 0, mask = 0;
  int k_rem = c.keep;      // keys still to keep among those that match the digits so far
  bool ties = true;        // more keys than that match
#pragma unroll 1
  for (int d = 0; d < 3 && ties; ++d) {
    const int shift = d == 2 ? 0 : 32 - kEvDigit * (d + 1);
    const uint32_t digit = d == 2 ? (1u << (32 - 2 * kEvDigit)) - 1u : kEvBins - 1u;
    int* h = hist[d & 1];
    if (d == 0) {   // every key: the protected ones are found, and odd lanes count apart
      int* const hl = hist[lane & 1];
      auto count = [&](int i, int p) {
        uint32_t u = 0xFFFFFFFFu;
        if (p < c.sinks || p > oldest_safe) keys[i] = u;
        else u = keys[i];
        atomicAdd(&hl[u >> (32 - kEvDigit)], 1);
      };
#pragma unroll
      for (int j = 0; j < kEvHeld; ++j)
        if (tid + j * kEvThreads < m) count(tid + j * kEvThreads, held[j]);
      for (int i = tid + kEvHeld * kEvThreads; i < m; i += kEvThreads) count(i, pos[i]);
    } else {
#pragma unroll 8
      for (int i = tid; i < m; i += kEvThreads) {
        const uint32_t u = keys[i];
        if ((u & mask) == prefix) atomicAdd(&h[u >> shift & digit], 1);
      }
    }
    __syncthreads();
    // sums of 64 bins first: the crossing one's bins are all that is read of the others' histograms
    int4 x = *reinterpret_cast<int4*>(&h[4 * tid]);
    if (d == 0) {
      const int4 y = *reinterpret_cast<int4*>(&hist[1][4 * tid]);
      x = make_int4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      *reinterpret_cast<int4*>(&h[4 * tid]) = x;
    }
    int sum = x.x + x.y + x.z + x.w;
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((lane & 15) == 0) group[d & 1][tid >> 4] = sum;
    sync_all();
    // the next digit's counters: no other CTA reads them any more (it passed this digit's barrier)
    *reinterpret_cast<int4*>(&hist[(d & 1) ^ 1][4 * tid]) = make_int4(0, 0, 0, 0);
    if (warp == 0) {
      int cnt = 0;   // of a lane's group, the largest digits first
#pragma unroll 8
      for (int r = 0; r < nc; ++r) cnt += cl.map_shared_rank(group[d & 1], r)[31 - lane];
      int at = __ffs(__ballot_sync(0xffffffffu, scan_warp(cnt) >= k_rem)) - 1;
      const int above = __shfl_sync(0xffffffffu, scan_warp(cnt) - cnt, at);
      const int top = 64 * (31 - at) + 62 - 2 * lane;   // a lane's two bins are top and top + 1
      int2 two = make_int2(0, 0);
#pragma unroll 8
      for (int r = 0; r < nc; ++r) {
        const int2 y = *reinterpret_cast<const int2*>(cl.map_shared_rank(h, r) + top);
        two = make_int2(two.x + y.x, two.y + y.y);
      }
      const int incl = above + scan_warp(two.x + two.y), mid = incl - two.x, low = mid - two.y;
      if (low < k_rem && incl >= k_rem) {
        const bool upper = mid >= k_rem;
        sel_digit = top + upper;
        sel_before = upper ? low : mid;
        sel_count = upper ? two.y : two.x;
      }
    }
    __syncthreads();
    k_rem -= sel_before;
    prefix |= static_cast<uint32_t>(sel_digit) << shift;
    mask |= digit << shift;
    ties = sel_count > k_rem;   // else every key with these digits is kept: the threshold is found
  }
  // ---- kept: every key from the threshold on or, when keys equal to it are left out, those above it
  // and the k_rem lowest slots equal to it.  32 slots to a word, a word to a thread.
  const unsigned below = (1u << lane) - 1u;
  const int words = (m + 31) / 32;
#pragma unroll 4
  for (int w = warp; w < words; w += kEvWarps) {
    const int i = w * 32 + lane;
    const uint32_t u = i < m ? keys[i] : 0u;
    const unsigned k = __ballot_sync(0xffffffffu, i < m && (ties ? u > prefix : u >= prefix));
    const unsigned e = ties ? __ballot_sync(0xffffffffu, i < m && u == prefix) : 0u;
    if (lane == 0) {
      kept_w[w] = k;
      list_at[w] = static_cast<int>(e);
    }
  }
  __syncthreads();
  if (ties) {   // (the cluster alike)
    uint32_t e = tid < words ? static_cast<uint32_t>(list_at[tid]) : 0u;
    int seen = scan_block(__popc(e), &cta_eq);
    sync_all();
    seen += __reduce_add_sync(0xffffffffu, lane < rank ? *cl.map_shared_rank(&cta_eq, lane) : 0);
    for (; e && seen < k_rem; e &= e - 1, ++seen) kept_w[tid] |= e & (0u - e);
    __syncthreads();
  }
  const uint32_t kw = tid < words ? kept_w[tid] : 0u;
  const int s0 = tid * 32, n_low = min(32, max(0, c.keep - lo - s0));   // the word's slots below the budget
  const uint32_t low = n_low >= 32 ? 0xFFFFFFFFu : (1u << n_low) - 1u;
  const uint32_t there = m - s0 >= 32 ? 0xFFFFFFFFu : (m - s0 > 0 ? (1u << (m - s0)) - 1u : 0u);
  // holes in the low half, moves in the high one: at most kEvKeys = 2^14 of each in a CTA
  const int both = scan_block(__popc(~kw & low & there) | __popc(kw & ~low) << 16, &cta_both);
  list_at[tid] = both;
  __syncthreads();
  uint16_t* holes = reinterpret_cast<uint16_t*>(keys);   // [chunk] each, of this CTA's slots; the keys are done with
  uint16_t* moves = holes + a.chunk;
#pragma unroll 4
  for (int w = warp; w < words; w += kEvWarps) {
    const int i = w * 32 + lane, slot = lo + i, at = list_at[w];
    const uint32_t k = kept_w[w];
    const bool kept = k >> lane & 1u, is_low = slot < c.keep;
    const unsigned lowb = __ballot_sync(0xffffffffu, is_low), hb = __ballot_sync(0xffffffffu, i < m && is_low && !kept);
    if (hb >> lane & 1u) holes[(at & 0xFFFF) + __popc(hb & below)] = static_cast<uint16_t>(i);
    if (kept && !is_low) moves[(at >> 16) + __popc(k & ~lowb & below)] = static_cast<uint16_t>(i);
  }
  sync_all();   // every CTA's lists and counts are written (and nothing else yet: a barrier waits for its CTA's stores)
  for (int w = warp; w < words; w += kEvWarps) {
    const int slot = lo + w * 32 + lane;
    if ((kept_w[w] >> lane & 1u) && slot < c.keep) src[slot] = slot;
  }
  if (warp == 0) {
    const int x = lane < nc ? *cl.map_shared_rank(&cta_both, lane) : 0;
    const int ih = scan_warp(x & 0xFFFF), im = scan_warp(x >> 16);
    if (lane < nc) hole_base[lane + 1] = ih;
    if (lane == 0) hole_base[0] = 0;
    if (lane == rank) move_base = im - (x >> 16);
  }
  __syncthreads();
  // ---- the i-th moving slot takes the i-th freed one (as many of the ones as of the others)
  const int n_moves = cta_both >> 16;
  int r = 0;
#pragma unroll 2
  for (int i = tid; i < n_moves; i += kEvThreads) {
    const int x = move_base + i;
    while (r + 1 < nc && x >= hole_base[r + 1]) ++r;
    src[r * a.chunk + cl.map_shared_rank(holes, r)[x - hole_base[r]]] = lo + moves[i];
  }
  if (nc > 1)   // nobody reads another's shared memory any more
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// ============================================================================
// Move: a row's K and V as 16-byte vectors, kEvVecs of them per thread in flight
// at once; in place only rows whose source is another slot.  HBM-bound: 8 hd
// bytes per copied row.  W: vectors of a K or V row as a constant (head_dim 64, 128; 0: any).
//   Four vectors and five CTAs per SM: 1 GB out of place (32 x 8 heads, 4160 slots to 4096, hd 128,
// with the selection) in 181 us, 90 % of the measured copy bandwidth; 8 vectors and 3 or 4 CTAs
// 190-193, 4 and 6 or 8 190-231 (registers spill), 2 and 8 193.
// ============================================================================
constexpr int kEvVecs = 4;
template <int W>
__global__ void __launch_bounds__(256, 5) k_evict_move(const EvictArgs a, int vec_any, int rows_cta) {
  pdl_wait();
  const flashloop_evict_args& c = a.c;
  const int vec = W ? W : vec_any;
  const int g = blockIdx.y, b = blockIdx.z;
  const long long seg = static_cast<long long>(b) * c.Hkv + g;
  const int n = a.n_kept[seg];
  const bool in_place = c.k_out == c.k;
  if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0) c.lens_out[b] = n;
  const int32_t* src = a.src + seg * a.cap;
  const int row0 = blockIdx.x * rows_cta, row1 = min(n, row0 + rows_cta);
  if (row0 >= row1) return;
  const uint16_t* k = c.k + b * c.k_stride[0] + g * c.k_stride[1];
  const uint16_t* v = c.v + b * c.v_stride[0] + g * c.v_stride[1];
  uint16_t* ko = c.k_out + b * c.k_out_stride[0] + g * c.k_out_stride[1];
  uint16_t* vo = c.v_out + b * c.v_out_stride[0] + g * c.v_out_stride[1];
  const int total = (row1 - row0) * 2 * vec;   // vectors of this CTA's rows: K then V of each row
  for (int e0 = threadIdx.x; e0 < total; e0 += 256 * kEvVecs) {
    uint4 x[kEvVecs];
    int from[kEvVecs];
#pragma unroll
    for (int u = 0; u < kEvVecs; ++u) {
      const int e = e0 + u * 256;
      from[u] = e < total ? src[row0 + e / (2 * vec)] : -1;
      if (in_place && from[u] == row0 + e / (2 * vec)) from[u] = -1;   // it stays where it is
    }
#pragma unroll
    for (int u = 0; u < kEvVecs; ++u) {
      const int w = (e0 + u * 256) % (2 * vec);
      if (from[u] >= 0)
        x[u] = __ldcs(reinterpret_cast<const uint4*>(w < vec ? k + from[u] * c.k_stride[2] + w * 8
                                                             : v + from[u] * c.v_stride[2] + (w - vec) * 8));
    }
#pragma unroll
    for (int u = 0; u < kEvVecs; ++u) {
      const int e = e0 + u * 256, w = e % (2 * vec);
      const long long row = row0 + e / (2 * vec);
      if (from[u] >= 0)
        __stcs(reinterpret_cast<uint4*>(w < vec ? ko + row * c.k_out_stride[2] + w * 8
                                                : vo + row * c.v_out_stride[2] + (w - vec) * 8), x[u]);
    }
  }
  for (int r = row0 + threadIdx.x; r < row1; r += 256) {
    const int f = src[r];
    if (in_place && f == r) continue;
    c.acc_out[b * c.acc_out_stride[0] + g * c.acc_out_stride[1] + r] = c.acc[b * c.acc_stride[0] + g * c.acc_stride[1] + f];
    c.pos_out[b * c.pos_out_stride[0] + g * c.pos_out_stride[1] + r] = c.pos[b * c.pos_stride[0] + g * c.pos_stride[1] + f];
  }
}

bool evict_shape_ok(int B, int Hkv, int S, int keep) {
  return B >= 1 && Hkv >= 1 && S >= 0 && keep >= 1 && S <= kEvSlots && B <= 65535 && Hkv <= 65535;
}
size_t evict_bytes(int B, int Hkv, int S, int keep) {
  const size_t seg = static_cast<size_t>(B) * Hkv, cap = std::min(keep, S);
  return align256_sz(seg * cap * 4) + align256_sz(seg * 4) + 256;
}

}  // namespace
}  // namespace fl

using namespace fl;

extern "C" {

size_t flashloop_evict_scratch_bytes(int B, int Hkv, int S, int keep) {
  return evict_shape_ok(B, Hkv, S, keep) ? evict_bytes(B, Hkv, S, keep) : 0;
}

fl_status flashloop_evict(const flashloop_evict_args* c, void* scratch, size_t scratch_bytes, fl_stream_t stream) {
  if (!c) return refuse(FL_ERR_INVALID_ARG, "NULL arguments");
  if (!evict_shape_ok(c->B, c->Hkv, c->S, c->keep) || c->hd < 8 || c->hd % 8 || c->hd > 1024)
    return refuse(FL_ERR_INVALID_ARG, "B, Hkv, S (<= 262144), keep (>= 1) or hd (a multiple of 8, <= 1024) out of range");
  if (c->recent < 0 || c->sinks < 0 || static_cast<long long>(c->recent) + c->sinks > c->keep)
    return refuse(FL_ERR_INVALID_ARG, "recent and sinks must not be negative, nor more than keep together");
  if (c->S == 0) return refuse(FL_ERR_INVALID_ARG, "S must be at least 1");
  const void* p16[4] = {c->k, c->v, c->k_out, c->v_out};
  for (const void* p : p16)
    if (!p || !is_aligned(p, 16)) return refuse(FL_ERR_INVALID_ARG, "k, v, k_out and v_out must be non-NULL and 16-byte aligned");
  const void* p4[6] = {c->acc, c->pos, c->lens, c->acc_out, c->pos_out, c->lens_out};
  for (const void* p : p4)
    if (!p || !is_aligned(p, 4)) return refuse(FL_ERR_INVALID_ARG, "acc, pos, lens and their outputs must be non-NULL and 4-byte aligned");
  const int same = (c->k_out == c->k) + (c->v_out == c->v) + (c->acc_out == c->acc) + (c->pos_out == c->pos) +
                   (c->lens_out == c->lens);
  if (same != 0 && same != 5) return refuse(FL_ERR_INVALID_ARG, "either every output is its input (in place) or none is");
  const int64_t in[3] = {c->B, c->Hkv, c->S}, out[3] = {c->B, c->Hkv, c->keep};
  for (int i = 0; i < 3; ++i) {
    if (!stride_ok(c->k_stride[i], in[i], 8) || !stride_ok(c->v_stride[i], in[i], 8) ||
        !stride_ok(c->k_out_stride[i], out[i], 8) || !stride_ok(c->v_out_stride[i], out[i], 8))
      return refuse(FL_ERR_INVALID_ARG, "k, v, k_out and v_out strides must be positive multiples of 8");
    if (same == 5 && in[i] > 1 &&
        (c->k_stride[i] != c->k_out_stride[i] || c->v_stride[i] != c->v_out_stride[i] ||
         (i < 2 && (c->acc_stride[i] != c->acc_out_stride[i] || c->pos_stride[i] != c->pos_out_stride[i]))))
      return refuse(FL_ERR_INVALID_ARG, "in place, the outputs' strides must be the inputs'");
    if (i < 2 && (!stride_ok(c->acc_stride[i], in[i], 1) || !stride_ok(c->pos_stride[i], in[i], 1) ||
                  !stride_ok(c->acc_out_stride[i], in[i], 1) || !stride_ok(c->pos_out_stride[i], in[i], 1)))
      return refuse(FL_ERR_INVALID_ARG, "acc, pos and their outputs' strides must be positive");
  }
  const size_t need = evict_bytes(c->B, c->Hkv, c->S, c->keep);
  if (!scratch || scratch_bytes < need || !is_aligned(scratch, 256))
    return refuse_scratch(need);
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvKeys * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_status(e);
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  EvictArgs a{};
  a.c = *c;
  a.cap = std::min(c->keep, c->S);
  const size_t seg = static_cast<size_t>(c->B) * c->Hkv, list = align256_sz(seg * a.cap * 4);
  uint8_t* ws = static_cast<uint8_t*>(scratch);
  a.src = reinterpret_cast<int32_t*>(ws);
  a.n_kept = reinterpret_cast<int32_t*>(ws + list);
  // CTAs per segment: chunks of at most 8192 slots (8 per thread and pass) while the cluster allows
  int nc = 1;
  while ((nc < 8 && c->S > nc * 8192) || c->S > nc * kEvKeys) nc *= 2;
  a.chunk = ceil_div_i(c->S, nc);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, c->Hkv, c->B);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.chunk) * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nc;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_evict_select, a);
  if (e != cudaSuccess) return cuda_status(e);
  const int vec = c->hd / 8;
  const int rows_cta = std::max(1, 256 * kEvVecs / (2 * vec));   // one round of every thread's vectors
  const dim3 grid(ceil_div_i(a.cap, rows_cta), c->Hkv, c->B);
  if (vec == 16) return cuda_status(launch_k(true, k_evict_move<16>, grid, dim3(256), 0, s, a, vec, rows_cta));
  if (vec == 8) return cuda_status(launch_k(true, k_evict_move<8>, grid, dim3(256), 0, s, a, vec, rows_cta));
  return cuda_status(launch_k(true, k_evict_move<0>, grid, dim3(256), 0, s, a, vec, rows_cta));
}

}  // extern "C"
