// fl_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Two launches.  The first reads every row of logits once and leaves, per
// chunk, the maximum, where it is, and the sum of exponentials relative to it.  The second
// decides the accepted drafts, forms again, in 64 bits, the sums of the one row that
// decides the last token, and finds the token.  64 bits because a token
// is the index where a running sum crosses u times its total: with V tokens between 0 and
// 1 that index is only well defined when the sum is known far better than 1 / V.
#include <algorithm>
#include <climits>
#include <cmath>

#include "fl_device.cuh"
#include "fl_serving.h"

namespace fl {
namespace {

constexpr int kVfThreads = 256;
constexpr int kVfChunk = 32 * kVfThreads - 4;   // logits per CTA of the first launch: 32 per thread, 4 spare for alignment
constexpr int kMaxDraft = 64;

struct alignas(16) RowPart {   // one chunk of one row
  float m, s;      // maximum, sum of 2^((x - m) c)
  int at, pad;     // lowest index of the maximum
};
struct VerifyArgs {
  flashloop_verify_args c;
  int n_chunks;
  double scale2;   // log2(e) / temperature
  double reach;    // logits further than this below the maximum, 2^-1000 of it, count as nothing
  RowPart* part;   // [B][2D + 1][n_chunks]: target rows, then draft rows
  unsigned* done;              // [B] finished CTAs of the second launch
  struct Sums* sums;           // [B][n_sub] of the deciding row's token ranges
  int n_sub, sub_len;
  unsigned* tickets;           // [B][D] finished chunks of a draft's rows, minus one (EARLY)
  unsigned* dead;              // [B] the first position known to be rejected
};
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kSumMaxCtas = kSumThreads / kSumWarps;   // CTAs of one sequence: n_sub <= kSumThreads

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int b) {
  return a.c.n_draft ? min(max(a.c.n_draft[b], 0), a.c.D) : a.c.D;
}
__device__ __forceinline__ const float* row_of(const VerifyArgs& a, int b, int r) {
  const flashloop_verify_args& c = a.c;
  return r <= c.D ? c.logits + b * c.logits_stride[0] + r * c.logits_stride[1]
                  : c.draft_logits + b * c.draft_logits_stride[0] + (r - c.D - 1) * c.draft_logits_stride[1];
}

// exp((x - m) / temperature) in 64 bits, to 4e-14: with z = 64 log2(e) (x - m) / temperature = k + r, k = rint(z),
// it is 2^(k / 64) e^(r ln 2 / 64); table[i] = 2^(i / 64), and the second factor's series to
// its fourth power, |r ln 2 / 64| <= 0.0055 (the next term is below 4e-14).  z = scale64 (x - m), x and m 32-bit
// values, z in [-65000, 0].  The difference comes first: as scale64 x + (-scale64 m), one operation less, z would be off by
// the rounding of scale64 m, which is beyond any exponent at low temperatures or with large logits.
constexpr int kExpTable = 64;
__device__ __forceinline__ double exp64(float x, double scale64, double m, const double* table) {
  const double z = (static_cast<double>(x) - m) * scale64;
  const double t = z + 6755399441055744.0;                  // + 1.5 * 2^52: k in the low word
  const int k = __double2loint(t);
  const double r = z - (t - 6755399441055744.0);
  constexpr double h = 0.693147180559945309417 / kExpTable;
  constexpr double c1 = h, c2 = h * h / 2, c3 = c2 * h / 3, c4 = c3 * h / 4;
  const double p = fma(fma(fma(fma(c4, r, c3), r, c2), r, c1), r, 1.0);
  const double f = table[k & (kExpTable - 1)];
  return p * __hiloint2double(__double2hiint(f) + ((k >> 6) << 20), __double2loint(f));
}

// The same, 0 for x below lo.
__device__ __forceinline__ double exp64_from(float x, float lo, double scale64, double m, const double* table) {
  const double e = exp64(fmaxf(x, lo), scale64, m, table);
  return x >= lo ? e : 0.0;
}

// The deciding row of a sequence, from 32-bit sums: target row `row`, draft row
// `row` when with_draft, their maxima, ratio = the draft's total over the target's.
struct Deciding {
  int row;          // drafts accepted in front of it
  int near;         // whether draft `row` is rejected is too near to say from 32-bit sums
  int with_draft;   // the weights are max(p - q, 0)
  int x_out;        // a token left out (the rejected one of a draft without probabilities), or -1
  int fine;         // both rows have finite, positive totals
  // Logits below these (2^-1000 of the maximum, -inf among them) count as nothing.  Rounded up, so that no logit counts
  // whose exponent would not fit, and finite however far they reach.
  float lo_p, lo_q;
  double mp, mq;    // the rows' maxima
  double ratio;
};

// Sum and maximum of a row from the first launch (one warp).
__device__ __forceinline__ void row_norm(const VerifyArgs& a, int b, int r, float& m, double& z) {
  const int lane = threadIdx.x & 31;
  const RowPart* part = a.part + (static_cast<size_t>(b) * (2 * a.c.D + 1) + r) * a.n_chunks;
  m = -INFINITY;
  z = 0.0;
  for (int k0 = 0; k0 < a.n_chunks; k0 += 32) {
    RowPart p{-INFINITY, 0.f, 0, 0};
    if (k0 + lane < a.n_chunks) {   // (through L2: another SM may have written it in this launch)
      const float4 f = __ldcg(reinterpret_cast<const float4*>(&part[k0 + lane]));
      p.m = f.x;
      p.s = f.y;
    }
    const float mn = fmaxf(m, warp_max(p.m));
    if (mn > m) z *= static_cast<double>(exp2f(static_cast<float>((static_cast<double>(m) - mn) * a.scale2)));
    z += p.m == -INFINITY ? p.s : p.s * exp2f(static_cast<float>((static_cast<double>(p.m) - mn) * a.scale2));   // (no finite logit: 0, or NaN)
    m = mn;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}

// Sums and maxima of the rows looked at, from the first launch: target rows and draft rows.
struct Norms {
  float mp[kMaxDraft + 1], mq[kMaxDraft + 1];
  double zp[kMaxDraft + 1], zq[kMaxDraft + 1];
};

// Verdict on a draft from the 32-bit sums: 0 rejected, 1 accepted, 2 too near to say (closer than 1e-4 of p;
// the sums and exponentials are good to about 1e-6).  u q < p without the divisions: u e_q Z_p < e_p Z_q.
__device__ __forceinline__ int verdict_on(const VerifyArgs& a, int x, double u, float xp, float mp, double zp, float xq, float mq,
                                          double zq) {
  if (x < 0 || x >= a.c.V) return 0;
  const double ep = exp2((static_cast<double>(xp) - mp) * a.scale2);
  const double eq = a.c.draft_logits ? exp2((static_cast<double>(xq) - mq) * a.scale2) : 1.0;
  const double l = u * eq * zp, r = ep * zq;
  return isfinite(r) && fabs(l - r) <= 1e-4 * r ? 2 : (l < r ? 1 : 0);
}
// ... on draft i (one warp)
__device__ __forceinline__ int judge_one(const VerifyArgs& a, int b, int i) {
  const flashloop_verify_args& c = a.c;
  const int x = c.draft[static_cast<size_t>(b) * c.D + i];
  const bool in = x >= 0 && x < c.V;
  const float xp = in ? row_of(a, b, i)[x] : 0.f, xq = in && c.draft_logits ? row_of(a, b, c.D + 1 + i)[x] : 0.f;
  const float u = c.u[static_cast<size_t>(b) * (c.D + 1) + i];
  float mp, mq = 0.f;
  double zp, zq = 1.0;
  row_norm(a, b, i, mp, zp);
  if (c.draft_logits) row_norm(a, b, c.D + 1 + i, mq, zq);
  return verdict_on(a, x, u, xp, mp, zp, xq, mq, zq);
}

// ============================================================================
// One chunk of one row: 32 logits per thread in registers (16-byte loads where the
// row's alignment allows, whatever V is), then maximum and sum.  HBM-bound, by CTAs that come
// and go (five of 32 KB per SM): 32 x 11 rows of 32000 logits in 7.3 us.
// Rows go position by position, each position's rows of all sequences together.
//   EARLY: rows behind a rejected draft decide nothing; a CTA takes its chunk of a position's
// target row and then of its draft row, the one that finishes a draft (a ticket) judges it, and
// later positions that have not started by then are not read.  For large calls: the
// tickets need a memset in front.  64 sequences, 8 drafts, 131071 logits with the samples' usual
// rejections: 54 us, the whole call 93; a CTA per row 60 (skipped CTAs cost 1 us of their place each,
// and a row as many tickets), persistent CTAs fed from a ring of bulk copies 67.
// ============================================================================
template <bool EARLY>
__global__ void __launch_bounds__(kVfThreads, 5) k_verify_rows(const VerifyArgs a) {
  __shared__ float red[kVfThreads / 32];
  __shared__ int red_i[kVfThreads / 32];
  __shared__ int last;
  pdl_trigger();
  const flashloop_verify_args& c = a.c;
  const bool pairs = c.draft_logits != nullptr;
  // position i; EARLY: its target row and then its draft row, else one of the two
  const int chunk = blockIdx.x, b = blockIdx.y, i = !EARLY && pairs ? blockIdx.z >> 1 : blockIdx.z;
  int r = !EARLY && pairs && (blockIdx.z & 1) ? c.D + 1 + i : i;
  const int n = drafts_of(a, b);
  if (r == 0 && chunk == 0 && threadIdx.x == 0) a.done[b] = 0;   // (row 0 is always read)
  if (r <= c.D ? r > n : i >= n) return;   // rows of drafts that were not made
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (EARLY) {
    if (tid == 0) last = static_cast<unsigned>(i) > __ldcg(&a.dead[b]);
    __syncthreads();
    if (last) return;
  }
  const int lo = chunk * kVfChunk, hi = min(c.V, lo + kVfChunk);
#pragma unroll 1
  for (;;) {   // (EARLY: the target row, then the draft row)
    const float* x = row_of(a, b, r) + lo;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);   // floats past a 16-byte boundary
    const int len = hi - lo;
    float v[8][4];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = (u * kVfThreads + tid) * 4 - off;   // index of the vector's first logit
      if (j >= 0 && j + 4 <= len) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(x + j));
        v[u][0] = f.x; v[u][1] = f.y; v[u][2] = f.z; v[u][3] = f.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = j + e >= 0 && j + e < len ? x[j + e] : -INFINITY;
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = fmaxf(m, v[u][e]);
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kVfThreads / 32; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    RowPart* out = a.part + (static_cast<size_t>(b) * (2 * c.D + 1) + r) * a.n_chunks + chunk;
    if (c.temperature == 0.f) {
      int at = INT_MAX;
#pragma unroll
      for (int u = 7; u >= 0; --u)
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const int j = (u * kVfThreads + tid) * 4 - off + e;
          if (v[u][e] == m && j >= 0 && j < len) at = lo + j;
        }
      at = __reduce_min_sync(0xffffffffu, at);
      if (lane == 0) red_i[warp] = at;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kVfThreads / 32; ++w) at = min(at, red_i[w]);
        *out = RowPart{m, 0.f, at, 0};
      }
      return;
    }
    // (halves, exact but for denormals: the difference of two logits may be beyond fp32)
    const float c2 = static_cast<float>(2.0 * a.scale2), ms = m == -INFINITY ? 0.f : 0.5f * m;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += exp2f(fmaf(v[u][e], 0.5f, -ms) * c2);
    s = warp_sum(s);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (tid == 0) {
      float t = 0.f;
      for (int w = 0; w < kVfThreads / 32; ++w) t += red[w];
      *out = RowPart{m, t, 0, 0};
    }
    if (!EARLY || !pairs || r > c.D || i >= n) break;
    r = c.D + 1 + i;
    __syncthreads();   // red
  }
  if (EARLY) {
    if (tid == 0) {
      __threadfence();
      last = i < n && atomicAdd(&a.tickets[static_cast<size_t>(b) * c.D + i], 1u) + 2u == a.n_chunks;
    }
    __syncthreads();
    if (!last || warp != 0) return;
    __threadfence();
    if (judge_one(a, b, i) == 0 && lane == 0) atomicMin(&a.dead[b], static_cast<unsigned>(i));
  }
}

// What the verdicts need of the inputs, read while the first launch still runs.
struct Ahead {
  int x[kMaxDraft];
  float xp[kMaxDraft], xq[kMaxDraft], u[kMaxDraft + 1];
};
__device__ __forceinline__ void look_ahead(const VerifyArgs& a, int b, int n, Ahead* h) {
  const flashloop_verify_args& c = a.c;
  const int i = threadIdx.x;
  if (i <= c.D) h->u[i] = c.u[static_cast<size_t>(b) * (c.D + 1) + i];
  if (i >= n) return;
  const int x = c.draft[static_cast<size_t>(b) * c.D + i];
  const bool in = x >= 0 && x < c.V;
  h->x[i] = x;
  h->xp[i] = in ? row_of(a, b, i)[x] : 0.f;
  h->xq[i] = in && c.draft_logits ? row_of(a, b, c.D + 1 + i)[x] : 0.f;
}

// Norms of target rows [first, n] and draft rows [first, n), a warp each, then the drafts' verdicts, a thread
// each.  Whole block.  (Rows behind a sure rejection may not have been summed: what is made of them is not looked at.)
__device__ void judge(const VerifyArgs& a, int b, int first, int n, const Ahead& h, int* verdict, Norms* norms) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const bool pairs = a.c.draft_logits != nullptr;
  const int targets = n - first + 1;
  for (int k = warp; k < targets + (pairs ? targets - 1 : 0); k += nw) {
    float m;
    double z;
    const int i = first + (k < targets ? k : k - targets);
    row_norm(a, b, k < targets ? i : a.c.D + 1 + i, m, z);
    if (lane == 0) {
      (k < targets ? norms->mp : norms->mq)[i] = m;
      (k < targets ? norms->zp : norms->zq)[i] = z;
    }
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i >= first && i < n)
    verdict[i] = verdict_on(a, h.x[i], h.u[i], h.xp[i], norms->mp[i], norms->zp[i], h.xq[i], pairs ? norms->mq[i] : 0.f,
                            pairs ? norms->zq[i] : 1.0);
  __syncthreads();
}

// The deciding row when drafts [0, row) are accepted (thread 0 fills *d; then a block barrier).
__device__ void describe(const VerifyArgs& a, int row, int n, const Ahead& h, const Norms& norms, const int* verdict, Deciding* d) {
  if (threadIdx.x == 0) {
    const bool residual = row < n, with_draft = residual && a.c.draft_logits;
    const float mp = norms.mp[row], mq = with_draft ? norms.mq[row] : 0.f;
    const double zp = norms.zp[row], zq = with_draft ? norms.zq[row] : 1.0;
    const bool fine = isfinite(zp) && zp > 0.0 && (!with_draft || (isfinite(zq) && zq > 0.0));
    *d = Deciding{row, residual && verdict[row] == 2, with_draft,
                  residual && !with_draft ? h.x[row] : -1, fine, __double2float_ru(mp - a.reach), __double2float_ru(mq - a.reach),
                  mp, mq, zq / zp};
  }
  __syncthreads();
}

// 64-bit sums over tokens [j0, j1) of the deciding row (one warp; every lane returns them): p and q,
// all exponentials; ap and aq, those of tokens whose weight is positive.  The weight of token j is
//   max(e_p / Z_p - e_q / Z_q, 0) = max(ratio e_p - e_q, 0) / Z_q,  ratio = Z_q / Z_p,
// so a range's weight is ratio * ap - aq, and the exact ratio need not be known
// before the pass: which tokens are positive is decided with the 32-bit one (good to 4e-6, by its sums' roundings), and
// a token it gets wrong weighs less than the ratios' difference times its e_q.  `near` is the e_q of all tokens that it
// could get wrong, those whose two terms are within kNearWords of each other in the high words (kNearReach of either at
// the least): that difference times `near` is what the pick allows for.
struct Sums {
  double p, q, ap, aq, near, pad;
};
constexpr int kNearWords = 22;
constexpr double kNearReach = 1e-5;
template <bool DRAFT>
__device__ Sums range_sums_of(const VerifyArgs& a, int b, const Deciding& d, int j0, int j1, const double* table) {
  constexpr int U = DRAFT ? 4 : 8;   // tokens of a lane in flight
  const int lane = threadIdx.x & 31;
  const float* xp = row_of(a, b, d.row);
  const float* xq = DRAFT ? row_of(a, b, a.c.D + 1 + d.row) : nullptr;
  const double s64 = 64.0 * a.scale2, mp = d.mp, mq = d.mq, ratio = d.ratio;
  const float lo_p = d.lo_p, lo_q = d.lo_q;
  const int x_out = d.x_out;
  double ap = 0.0, aq = 0.0, np = 0.0, nq = 0.0, near = 0.0;   // tokens of positive weight, the others, those near 0
  auto add = [&](float fp, float fq, int j) {
    const double ep = exp64_from(fp, lo_p, s64, mp, table);
    if (DRAFT) {
      const double eq = exp64_from(fq, lo_q, s64, mq, table);
      const double rp = ratio * ep;
      if (abs(__double2hiint(rp) - __double2hiint(eq)) <= kNearWords) near += eq;
      if (rp > eq) {
        ap += ep;
        aq += eq;
      } else {
        np += ep;
        nq += eq;
      }
    } else if (j != x_out) {
      ap += ep;
    } else {
      np += ep;
    }
  };
  // full rounds of U tokens a lane, the next round's loads under this one's arithmetic
  const int rounds = j1 > j0 ? (j1 - j0) / (32 * U) : 0;
  float fp[U], fq[U];
  auto load = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + (r * U + u) * 32 + lane;
      fp[u] = xp[j];
      fq[u] = DRAFT ? xq[j] : 0.f;
    }
  };
  if (rounds) load(0);
  for (int r = 0; r < rounds; ++r) {
    float gp[U], gq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      gp[u] = fp[u];
      gq[u] = fq[u];
    }
    if (r + 1 < rounds) load(r + 1);
#pragma unroll
    for (int u = 0; u < U; ++u) add(gp[u], gq[u], j0 + (r * U + u) * 32 + lane);
  }
  int j = j0 + rounds * 32 * U + lane;
  for (; j < j1; j += 32) add(xp[j], DRAFT ? xq[j] : 0.f, j);
  Sums s{ap + np, aq + nq, ap, aq, near, 0.0};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.p += __shfl_xor_sync(0xffffffffu, s.p, o);
    s.q += __shfl_xor_sync(0xffffffffu, s.q, o);
    s.ap += __shfl_xor_sync(0xffffffffu, s.ap, o);
    s.aq += __shfl_xor_sync(0xffffffffu, s.aq, o);
  }
  if (DRAFT && __any_sync(0xffffffffu, near > 0.0)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s.near += __shfl_xor_sync(0xffffffffu, s.near, o);
  }
  return s;
}
__device__ __forceinline__ Sums range_sums(const VerifyArgs& a, int b, const Deciding& d, int j0, int j1, const double* table) {
  if (!d.fine) return Sums{};   // (the token will be -1)
  return d.with_draft ? range_sums_of<true>(a, b, d, j0, j1, table) : range_sums_of<false>(a, b, d, j0, j1, table);
}

// the sums of x, y and z over the block
struct Three {
  double x, y, z;
};
__device__ Three block_sums_f64(Three v, Three* buf /*[kSumWarps]*/) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  Three t{0.0, 0.0, 0.0};
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) t = Three{t.x + buf[w].x, t.y + buf[w].y, t.z + buf[w].z};
  return t;
}
// exclusive prefix sum over the block's threads, in thread order, and the sum of all
__device__ double block_scan_f64(double v, Three* buf, double& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp].x = incl;
  __syncthreads();
  double base = 0.0;
  total = 0.0;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) {
    if (w == warp) base = total;
    total += buf[w].x;
  }
  const double excl = __shfl_up_sync(0xffffffffu, incl, 1);
  return base + (lane ? excl : 0.0);
}

// ============================================================================
// Second launch: every CTA finds its sequence's deciding row from the first
// launch's sums, then each of its warps forms the 64-bit sums of a contiguous
// range of that row's tokens, two exponentials a token, once.  Bound by the 64-bit pipe
// (about 12 operations per exponential) and its conversions for many sequences, by a chain of round
// trips for few: 64 rows of 131071 tokens about 37 us (18 of them the sums), one sequence of
// 32000 8 us.  Four CTAs per SM leave 64 registers a thread, of which 160 bytes spill.
//   The CTA that finishes a sequence's last ranges picks its token: totals of the
// ranges' sums, the range that holds the crossing, and the crossing token in it.  A near
// decision is settled by the 64-bit totals of its row; when it turns out accepted, this CTA
// goes on to the next rows by itself (about one call in ten thousand per draft).
// ============================================================================
__global__ void __launch_bounds__(kSumThreads, 4) k_verify_sums(const VerifyArgs a) {
  __shared__ double table[kExpTable], start_of[kSumThreads];
  __shared__ Three buf[kSumWarps];
  __shared__ Ahead ahead;
  __shared__ int verdict[kMaxDraft];
  __shared__ Norms norms;
  __shared__ Deciding d;
  __shared__ int last, cross[2], top[2];
  __shared__ bool sure;
  const flashloop_verify_args& c = a.c;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kExpTable) table[tid] = exp2(tid * (1.0 / kExpTable));
  const int n = drafts_of(a, b), D = c.D;
  int32_t* tokens = c.tokens + static_cast<size_t>(b) * (D + 1);
  look_ahead(a, b, n, &ahead);
  if (tid < 2) cross[tid] = INT_MAX, top[tid] = -1;
  Sums* sums = a.sums + static_cast<size_t>(b) * a.n_sub;
  pdl_wait();
  judge(a, b, 0, n, ahead, verdict, &norms);
  {
    int row = 0;
    while (row < n && verdict[row] == 1) ++row;
    describe(a, row, n, ahead, norms, verdict, &d);
    const int sub = blockIdx.x * kSumWarps + warp;
    const int j0 = min(c.V, sub * a.sub_len), j1 = min(c.V, j0 + a.sub_len);
    const Sums s = range_sums(a, b, d, j0, j1, table);
    if (lane == 0) sums[sub] = s;
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(&a.done[b], 1u) + 1u == gridDim.x;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  const double s64 = 64.0 * a.scale2;
  auto prob = [&](float x, float lo, double m) { return exp64_from(x, lo, s64, m, table); };
  Sums s{};                     // n_sub <= threads: one range each
  double zp, zq, unsure;
  auto totals = [&]() {
    if (tid < a.n_sub) {   // (from L2: other CTAs wrote most of them)
      const double2* from = reinterpret_cast<const double2*>(&sums[tid]);
      const double2 x = __ldcg(from), y = __ldcg(from + 1), z = __ldcg(from + 2);
      s = Sums{x.x, x.y, y.x, y.y, z.x, 0.0};
    }
    const Three t = block_sums_f64(Three{s.p, s.q, s.near}, buf);
    zp = t.x;
    zq = t.y;
    // The ranges' weights may be off, together, by what the 32-bit ratio got wrong; so may the target.  (1e-13: this
    // one's own roundings; a 32-bit ratio beyond its bound: nothing is sure.)
    const double off = fabs(zq / zp / d.ratio - 1.0) + 1e-13;
    unsure = !d.with_draft || !d.fine ? 0.0 : off <= kNearReach ? 2.0 * off * t.z : INFINITY;
  };
  totals();
  while (d.near && d.fine) {
    const double p = prob(ahead.xp[d.row], d.lo_p, d.mp) / zp;   // (a token outside the vocabulary is never near)
    const double q = c.draft_logits ? prob(ahead.xq[d.row], d.lo_q, d.mq) / zq : 1.0;
    if (!(static_cast<double>(ahead.u[d.row]) * q < p)) break;   // rejected after all
    int row = d.row + 1;
    judge(a, b, row, n, ahead, verdict, &norms);
    while (row < n && verdict[row] == 1) ++row;
    describe(a, row, n, ahead, norms, verdict, &d);
    for (int sub = warp; sub < a.n_sub; sub += kSumWarps) {
      const int j0 = min(c.V, sub * a.sub_len), j1 = min(c.V, j0 + a.sub_len);
      const Sums t = range_sums(a, b, d, j0, j1, table);
      if (lane == 0) sums[sub] = t;
    }
    __syncthreads();
    totals();
  }
  const int acc = d.row;
  const bool with_draft = d.with_draft;
  const double ratio = with_draft ? zq / zp : 1.0;
  const float* xp = row_of(a, b, acc);
  const float* xq = with_draft ? row_of(a, b, D + 1 + acc) : nullptr;
  auto weight = [&](int j) {
    const double ep = prob(xp[j], d.lo_p, d.mp);
    if (with_draft) return fmax(ratio * ep - prob(xq[j], d.lo_q, d.mq), 0.0);
    return j == d.x_out ? 0.0 : ep;
  };
  for (int i = tid; i <= D; i += kSumThreads)
    if (i != acc) tokens[i] = i < acc ? ahead.x[i] : -1;
  if (tid == 0) c.n_accepted[b] = acc;
  double mine = fmax(ratio * s.ap - s.aq, 0.0);   // (0 for NaN)
  for (;;) {
    double total;
    const double before = block_scan_f64(mine, buf, total);
    const bool fine = d.fine && isfinite(total) && total > 0.0;
    if (fine) {
      const double target = static_cast<double>(ahead.u[D]) * total;
      // the first range whose end is past the target (the last with any weight, should rounding leave none)
      start_of[tid] = before;
      if (mine > 0.0) {
        atomicMax(&top[0], tid);
        if (target < before + mine) atomicMin(&cross[0], tid);
      }
      __syncthreads();
      const int sub = cross[0] != INT_MAX ? cross[0] : top[0];
      const double start = start_of[sub];
      const int j0 = min(c.V, sub * a.sub_len), j1 = min(c.V, j0 + a.sub_len);
      const int per = (j1 - j0 + kSumThreads - 1) / kSumThreads;
      const int t0 = min(j1, j0 + tid * per), t1 = min(j1, t0 + per);
      double mass = 0.0;
      for (int j = t0; j < t1; ++j) mass += weight(j);
      double all;
      const double at = start + block_scan_f64(mass, buf, all);
      if (mass > 0.0) {
        atomicMax(&top[1], tid);
        if (target < at + mass) atomicMin(&cross[1], tid);
      }
      __syncthreads();
      if (tid == (cross[1] != INT_MAX ? cross[1] : max(top[1], 0))) {
        double run = at, x = 0.0;
        int y = -1;   // (no weight at all where p and q differ by roundings alone: empty)
        for (int j = t0; j < t1; ++j) {
          x = weight(j);
          run += x;
          if (x > 0.0) {
            y = j;
            if (run > target) break;
          }
        }
        sure = run - target > unsure && target - (run - x) >= unsure;
        if (unsure == 0.0 || sure) tokens[acc] = y;
      }
      if (unsure == 0.0) return;
      __syncthreads();
      if (sure) return;
    } else if (unsure == 0.0) {
      if (tid == 0) tokens[acc] = -1;
      return;
    }
    // Too near to say: the ranges' weights again, token by token from the exact ratio (where target and draft
    // nearly agree: a call on 64 equal rows of 131071 tokens, the slowest, takes 275 us, on unlike ones 50).
    unsure = 0.0;
    for (int r = warp; r < a.n_sub; r += kSumWarps) {
      const int j0 = min(c.V, r * a.sub_len), j1 = min(c.V, j0 + a.sub_len);
      double x = 0.0;
      for (int j = j0 + lane; j < j1; j += 32) x += weight(j);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) start_of[r] = x;
    }
    if (tid < 2) cross[tid] = INT_MAX, top[tid] = -1;
    __syncthreads();
    mine = tid < a.n_sub ? start_of[tid] : 0.0;
  }
}

// ============================================================================
// Greedy: one CTA per sequence; the first launch left every chunk's maximum.  Latency-bound (16 sequences of up to
// 5 rows x 50001 tokens: 5.6 us with the first launch).
// ============================================================================
__global__ void __launch_bounds__(256) k_verify_greedy(const VerifyArgs a) {
  __shared__ int best[kMaxDraft + 1];
  const flashloop_verify_args& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const int n = drafts_of(a, b), D = c.D;
  const int32_t* draft = c.draft + static_cast<size_t>(b) * D;
  int32_t* tokens = c.tokens + static_cast<size_t>(b) * (D + 1);
  const RowPart* part = a.part + static_cast<size_t>(b) * (2 * D + 1) * a.n_chunks;
  pdl_wait();
  for (int i = warp; i <= n; i += 8) {
    float m = -INFINITY;
    int at = INT_MAX;
    for (int k = lane; k < a.n_chunks; k += 32) {
      const RowPart p = part[static_cast<size_t>(i) * a.n_chunks + k];
      if (p.m > m || at == INT_MAX) {
        m = p.m;
        at = p.at;
      }
    }
    const float mm = warp_max(m);
    at = __reduce_min_sync(0xffffffffu, m == mm ? at : INT_MAX);
    if (lane == 0) best[i] = mm > -INFINITY ? at : -1;   // (only NaN, or nothing above -inf: no candidate)
  }
  __syncthreads();
  int acc = 0;
  while (acc < n && best[acc] >= 0 && draft[acc] == best[acc]) ++acc;
  for (int i = tid; i <= D; i += 256) tokens[i] = i < acc ? draft[i] : i == acc ? best[acc] : -1;
  if (tid == 0) c.n_accepted[b] = acc;
}

bool verify_shape_ok(int B, int D, int V) {
  return B >= 1 && B <= 65535 && D >= 0 && D <= kMaxDraft && V >= 1 && V <= (1 << 30);
}
// Ranges of the deciding row: the CTAs of the whole batch resident at once (four per SM), none with
// fewer than 1024 tokens (4 a thread), at most one range per thread of the CTA that picks the token.
void plan_sums(int B, int V, int& ctas, int& sub_len) {
  ctas = std::min(std::min(kSumMaxCtas, std::max(1, 4 * kNumSM / B)), std::max(1, V / 1024));
  sub_len = (ceil_div_i(V, ctas * kSumWarps) + 31) & ~31;
}
int verify_chunks(int V) { return ceil_div_i(V, kVfChunk); }

}  // namespace
}  // namespace fl

using namespace fl;

extern "C" {

size_t flashloop_verify_draft_scratch_bytes(int B, int D, int V) {
  if (!verify_shape_ok(B, D, V)) return 0;
  return align256_sz(static_cast<size_t>(B) * (2 * D + 1) * verify_chunks(V) * sizeof(RowPart)) +
         align256_sz(static_cast<size_t>(B) * kSumThreads * sizeof(Sums)) +
         align256_sz(static_cast<size_t>(B) * (D + 2) * 4) + 256;
}

fl_status flashloop_verify_draft(const flashloop_verify_args* c, void* scratch, size_t scratch_bytes,
                                 fl_stream_t stream) {
  if (!c) return refuse(FL_ERR_INVALID_ARG, "NULL arguments");
  if (!verify_shape_ok(c->B, c->D, c->V)) return refuse(FL_ERR_INVALID_ARG, "B, D (0 to 64) or V out of range");
  if (!(c->temperature == 0.f || c->temperature >= 1e-20f) || !std::isfinite(c->temperature))
    return refuse(FL_ERR_INVALID_ARG, "temperature must be 0, or finite and at least 1e-20");
  if (!c->logits || !c->tokens || !c->n_accepted || (c->D > 0 && !c->draft) || (c->temperature > 0.f && !c->u))
    return refuse(FL_ERR_INVALID_ARG, "logits, draft, u, tokens and n_accepted must be non-NULL");
  const void* p4[7] = {c->logits, c->draft_logits, c->draft, c->u, c->n_draft, c->tokens, c->n_accepted};
  for (const void* p : p4)
    if (!is_aligned(p, 4)) return refuse(FL_ERR_INVALID_ARG, "every pointer must be 4-byte aligned");
  if (!stride_ok(c->logits_stride[0], c->B, 1) || !stride_ok(c->logits_stride[1], c->D + 1, 1) ||
      (c->draft_logits && (!stride_ok(c->draft_logits_stride[0], c->B, 1) || !stride_ok(c->draft_logits_stride[1], c->D, 1))))
    return refuse(FL_ERR_INVALID_ARG, "strides must be positive");
  const size_t need = flashloop_verify_draft_scratch_bytes(c->B, c->D, c->V);
  if (!scratch || scratch_bytes < need || !is_aligned(scratch, 256))
    return refuse_scratch(need);
  VerifyArgs a{};
  a.c = *c;
  if (c->temperature == 0.f) a.c.draft_logits = nullptr;   // greedy: the target's rows alone
  a.n_chunks = verify_chunks(c->V);
  a.scale2 = c->temperature > 0.f ? 1.4426950408889634 / static_cast<double>(c->temperature) : 0.0;
  a.reach = c->temperature > 0.f ? 1000.0 / a.scale2 : 0.0;
  a.part = static_cast<RowPart*>(scratch);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = c->D + 1 + (a.c.draft_logits ? c->D : 0);
  int ctas;
  plan_sums(c->B, c->V, ctas, a.sub_len);
  a.n_sub = ctas * kSumWarps;
  uint8_t* ws = static_cast<uint8_t*>(scratch) +
                align256_sz(static_cast<size_t>(c->B) * (2 * c->D + 1) * a.n_chunks * sizeof(RowPart));
  a.sums = reinterpret_cast<Sums*>(ws);
  ws += align256_sz(static_cast<size_t>(c->B) * kSumThreads * sizeof(Sums));
  a.tickets = reinterpret_cast<unsigned*>(ws);
  a.dead = a.tickets + static_cast<size_t>(c->B) * c->D;
  a.done = a.dead + c->B;
  // Skipping rows behind a rejection costs a memset in front, a ticket per chunk and the place of each skipped CTA, and pays
  // when most rows have not started by the first verdicts.  With against without it, us, where 1 to 2 drafts are accepted,
  // and where nearly all are: 45 MB of logits 29 / 22 and 29 / 22, 141 MB 47 / 42 and 50 / 41, 218 MB 53 / 53 and 61 / 54,
  // 359 MB 68 / 80 and 85 / 78, 570 MB 92 / 119 and 124 / 117.  The host cannot know which it will be: from 350 MB on,
  // where the first case wins about twice what the second loses.
  const bool early = c->temperature > 0.f && c->D >= 2 && static_cast<double>(c->B) * rows * c->V * 4.0 > 350e6;
  cudaError_t e;
  const dim3 grid(a.n_chunks, c->B, rows);
  if (early) {
    e = cudaMemsetAsync(a.tickets, 0xFF, static_cast<size_t>(c->B) * (c->D + 1) * 4, s);
    if (e == cudaSuccess) e = launch_k(false, k_verify_rows<true>, dim3(a.n_chunks, c->B, c->D + 1), dim3(kVfThreads), 0, s, a);
  } else {
    e = launch_k(false, k_verify_rows<false>, grid, dim3(kVfThreads), 0, s, a);
  }
  if (e != cudaSuccess) return cuda_status(e);
  if (c->temperature == 0.f)
    return cuda_status(launch_k(true, k_verify_greedy, dim3(c->B), dim3(256), 0, s, a));
  return cuda_status(launch_k(true, k_verify_sums, dim3(ctas, c->B), dim3(kSumThreads), 0, s, a));
}

}  // extern "C"
