// fl_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Two launches.  The first reads every row of logits once and leaves, per chunk, the
// maximum, where it is, and the sum of exponentials relative to it.  The second
// (a cluster per sequence) decides the accepted drafts and samples the last
// token from the one row that decides it, whose sums it forms again in 64 bits:
// a token is the index where a running sum crosses u times its total, and with
// V tokens between 0 and 1 that index is only well defined when the sum is
// known far better than 1 / V.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cooperative_groups.h>

#include "fl_device.cuh"
#include "fl_serving.h"

namespace cg = cooperative_groups;

namespace fl {
namespace {

constexpr int kVfThreads = 256;
constexpr int kVfChunk = 32 * kVfThreads - 4;   // logits per CTA of the first launch: 32 per thread, 4 spare for alignment
constexpr int kVfCluster = 8;
constexpr int kMaxDraft = 64;

struct RowPart {   // one chunk of one row
  float m, s;      // maximum, sum of 2^((x - m) c)
  int at, pad;     // lowest index of the maximum
};
struct VerifyArgs {
  flashloop_verify_args c;
  int n_chunks;
  double scale2;   // log2(e) / temperature
  RowPart* part;   // [B][2D + 1][n_chunks]: target rows, then draft rows
};

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int b) {
  return a.c.n_draft ? min(max(a.c.n_draft[b], 0), a.c.D) : a.c.D;
}
__device__ __forceinline__ const float* row_of(const VerifyArgs& a, int b, int r) {
  const flashloop_verify_args& c = a.c;
  return r <= c.D ? c.logits + b * c.logits_stride[0] + r * c.logits_stride[1]
                  : c.draft_logits + b * c.draft_logits_stride[0] + (r - c.D - 1) * c.draft_logits_stride[1];
}

// ============================================================================
// One chunk of one row: 32 logits per thread in registers (16-byte loads where the
// row's alignment allows, whatever V is), then maximum and sum.  HBM-bound.
// ============================================================================
__global__ void __launch_bounds__(kVfThreads) k_verify_rows(const VerifyArgs a) {
  __shared__ float red[kVfThreads / 32];
  __shared__ int red_i[kVfThreads / 32];
  pdl_trigger();
  const flashloop_verify_args& c = a.c;
  const int chunk = blockIdx.x, r = blockIdx.y, b = blockIdx.z;
  const int n = drafts_of(a, b);
  if (r <= c.D ? r > n : r - c.D - 1 >= n) return;   // rows of drafts that were not made
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = chunk * kVfChunk, hi = min(c.V, lo + kVfChunk);
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
  const float c2 = static_cast<float>(a.scale2), ms = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) s += exp2f((v[u][e] - ms) * c2);
  s = warp_sum(s);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
    for (int w = 0; w < kVfThreads / 32; ++w) t += red[w];
    *out = RowPart{m, t, 0, 0};
  }
}

// ============================================================================
// One cluster per sequence.  Every CTA decides the accepted drafts from the
// first launch's sums (32-bit, good to about 1e-6); a decision closer to its
// border than 1e-4 is taken again from 64-bit sums of that row.  Then each CTA
// has a contiguous range of the deciding row's tokens, each warp a contiguous
// part of it: their sums, scanned over warps and CTAs, give the warp that holds
// the crossing, which walks its part once more.
// ============================================================================
struct Near {
  int at;    // first draft not surely accepted (n: all are)
  int sure;  // it is surely rejected
};

__global__ void __launch_bounds__(kVfThreads) k_verify_pick(const VerifyArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  constexpr int NW = kVfThreads / 32;
  __shared__ int verdict[kMaxDraft];      // 0 rejected, 1 accepted, 2 too near to say
  __shared__ double wsum[2][NW];
  __shared__ double cta_sum[2][2];        // [buffer][row kind]
  __shared__ float row_max[2];
  const flashloop_verify_args& c = a.c;
  const int nc = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y;
  pdl_wait();
  const int n = drafts_of(a, b), V = c.V, D = c.D;
  const int32_t* draft = c.draft + static_cast<size_t>(b) * D;
  int32_t* tokens = c.tokens + static_cast<size_t>(b) * (D + 1);
  const RowPart* part = a.part + static_cast<size_t>(b) * (2 * D + 1) * a.n_chunks;
  auto best_of = [&](int r, float& m, int& at) {   // (one warp)
    m = -INFINITY;
    at = INT_MAX;
    for (int k = lane; k < a.n_chunks; k += 32) {
      const RowPart p = part[static_cast<size_t>(r) * a.n_chunks + k];
      if (p.m > m || at == INT_MAX) {
        m = p.m;
        at = p.at;
      }
    }
    const float mm = warp_max(m);
    at = __reduce_min_sync(0xffffffffu, m == mm ? at : INT_MAX);
    m = mm;
  };
  if (c.temperature == 0.f) {
    if (rank != 0) return;
    for (int i = warp; i <= n; i += NW) {
      float m;
      int at;
      best_of(i, m, at);
      if (lane == 0 && i < n) verdict[i] = draft[i] == at ? 1 : 0;
    }
    __syncthreads();
    int acc = 0;
    while (acc < n && verdict[acc] == 1) ++acc;
    if (warp == 0) {
      float m;
      int at;
      best_of(acc, m, at);
      for (int i = lane; i <= D; i += 32) tokens[i] = i < acc ? draft[i] : i == acc ? at : -1;
      if (lane == 0) c.n_accepted[b] = acc;
    }
    return;
  }
  // sum and maximum of a row from the first launch (one warp)
  auto norm_of = [&](int r, float& m, double& z) {
    m = -INFINITY;
    for (int k = lane; k < a.n_chunks; k += 32) m = fmaxf(m, part[static_cast<size_t>(r) * a.n_chunks + k].m);
    m = warp_max(m);
    z = 0.0;
    for (int k = lane; k < a.n_chunks; k += 32) {
      const RowPart p = part[static_cast<size_t>(r) * a.n_chunks + k];
      if (p.m == -INFINITY)
        z += p.s;   // 0, or NaN
      else
        z += p.s * exp2(static_cast<double>(p.m - m) * a.scale2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  };
  for (int i = warp; i < n; i += NW) {
    const int x = draft[i];
    float m;
    double z;
    norm_of(i, m, z);
    double p = 0.0, q = 1.0;
    const bool in = x >= 0 && x < V;
    if (in) p = exp2(static_cast<double>(row_of(a, b, i)[x] - m) * a.scale2) / z;
    if (c.draft_logits && in) {
      norm_of(D + 1 + i, m, z);
      q = exp2(static_cast<double>(row_of(a, b, D + 1 + i)[x] - m) * a.scale2) / z;
    }
    const double uq = static_cast<double>(c.u[static_cast<size_t>(b) * (D + 1) + i]) * q;
    if (lane == 0) verdict[i] = in && fabs(uq - p) <= 1e-4 * p ? 2 : (in && uq < p ? 1 : 0);
  }
  __syncthreads();
  // this CTA's tokens, and this warp's
  const int per = ((V + nc - 1) / nc + 31) & ~31;
  const int c0 = min(V, rank * per), c1 = min(V, c0 + per);
  const int pw = ((c1 - c0 + NW - 1) / NW + 31) & ~31;
  const int w0 = min(c1, c0 + warp * pw), w1 = min(c1, w0 + pw);
  int buf = 0;
  // 64-bit sums of 2^((x - m) scale2) of target row i and draft row i over the cluster
  auto exact_sums = [&](int i, bool with_draft, float& mp, float& mq, double& zp, double& zq) {
    if (warp < 2) {
      float m = 0.f;
      double z;
      if (warp == 0 || with_draft) norm_of(warp == 0 ? i : D + 1 + i, m, z);
      if (lane == 0) row_max[warp] = m;
    }
    __syncthreads();
    mp = row_max[0];
    mq = row_max[1];
    const float* xp = row_of(a, b, i);
    double sp = 0.0, sq = 0.0;
    for (int j = w0 + lane; j < w1; j += 32) sp += exp2(static_cast<double>(xp[j] - mp) * a.scale2);
    if (with_draft) {
      const float* xq = row_of(a, b, D + 1 + i);
      for (int j = w0 + lane; j < w1; j += 32) sq += exp2(static_cast<double>(xq[j] - mq) * a.scale2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sp += __shfl_xor_sync(0xffffffffu, sp, o);
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
    }
    if (lane == 0) {
      wsum[0][warp] = sp;
      wsum[1][warp] = sq;
    }
    __syncthreads();
    if (tid < 2) {
      double t = 0.0;
      for (int w = 0; w < NW; ++w) t += wsum[tid][w];
      cta_sum[buf][tid] = t;
    }
    cl.sync();
    zp = zq = 0.0;
    for (int r = 0; r < nc; ++r) {
      const double* s = cl.map_shared_rank(&cta_sum[buf][0], r);
      zp += s[0];
      zq += s[1];
    }
    buf ^= 1;
  };
  int acc = 0;
  float mp = 0.f, mq = 0.f;
  double zp = 0.0, zq = 0.0;
  bool have = false;   // the exact sums of row acc are at hand
  while (acc < n && verdict[acc] != 0) {   // (the same in every CTA of the cluster)
    if (verdict[acc] == 2) {
      exact_sums(acc, c.draft_logits != nullptr, mp, mq, zp, zq);
      const int x = draft[acc];
      const double p = exp2(static_cast<double>(row_of(a, b, acc)[x] - mp) * a.scale2) / zp;
      const double q = c.draft_logits ? exp2(static_cast<double>(row_of(a, b, D + 1 + acc)[x] - mq) * a.scale2) / zq : 1.0;
      if (!(static_cast<double>(c.u[static_cast<size_t>(b) * (D + 1) + acc]) * q < p)) {
        have = true;
        break;
      }
    }
    ++acc;
  }
  const bool residual = acc < n;
  const bool with_draft = residual && c.draft_logits != nullptr;
  if (!have) exact_sums(acc, with_draft, mp, mq, zp, zq);
  const float* xp = row_of(a, b, acc);
  const float* xq = with_draft ? row_of(a, b, D + 1 + acc) : nullptr;
  const int x_out = residual && !with_draft ? draft[acc] : -1;   // a draft without probabilities: its own token is out
  const double ip = 1.0 / zp, iq = with_draft ? 1.0 / zq : 0.0;
  auto weight = [&](int j) {
    double w = exp2(static_cast<double>(xp[j] - mp) * a.scale2) * ip;
    if (with_draft) w = fmax(w - exp2(static_cast<double>(xq[j] - mq) * a.scale2) * iq, 0.0);
    return j == x_out ? 0.0 : w;
  };
  double s = 0.0;
  for (int j = w0 + lane; j < w1; j += 32) s += weight(j);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) wsum[0][warp] = s;
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < NW; ++w) t += wsum[0][w];
    cta_sum[buf][0] = t;
  }
  cl.sync();
  double total = 0.0, before = 0.0;
  int last_cta = -1;   // the last CTA with any weight
  for (int r = 0; r < nc; ++r) {
    const double t = *cl.map_shared_rank(&cta_sum[buf][0], r);
    if (r < rank) before += t;
    total += t;
    if (t > 0.0) last_cta = r;
  }
  cl.sync();   // nobody's shared memory is read from here on
  const bool fine = isfinite(total) && total > 0.0 && isfinite(zp) && (!with_draft || (isfinite(zq) && zq > 0.0));
  if (rank == 0) {
    for (int i = tid; i <= D; i += kVfThreads)
      if (i != acc || !fine) tokens[i] = i < acc ? draft[i] : -1;
    if (tid == 0) c.n_accepted[b] = acc;
  }
  if (!fine) return;
  const double target = static_cast<double>(c.u[static_cast<size_t>(b) * (D + 1) + D]) * total;
  const double mine = cta_sum[buf][0];
  // the CTA whose range holds the crossing (the last with any weight, should rounding leave none)
  if (!(before <= target && (target < before + mine || rank == last_cta)) || mine <= 0.0) return;
  int last_warp = -1, w_at = -1;
  double run = before, start = before;
  for (int w = 0; w < NW; ++w) {
    if (wsum[0][w] > 0.0) last_warp = w;
    if (w_at < 0 && target < run + wsum[0][w]) {
      w_at = w;
      start = run;
    }
    run += wsum[0][w];
  }
  if (w_at < 0) {
    w_at = last_warp;
    start = before;
    for (int w = 0; w < w_at; ++w) start += wsum[0][w];
  }
  if (warp != w_at) return;
  int found = INT_MAX, last_pos = -1;
  for (int j0 = w0; j0 < w1 && found == INT_MAX; j0 += 32) {
    const double w = j0 + lane < w1 ? weight(j0 + lane) : 0.0;
    double incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && start + incl > target);
    const unsigned any = __ballot_sync(0xffffffffu, w > 0.0);
    if (any) last_pos = j0 + 31 - __clz(any);
    if (over) found = j0 + __ffs(over) - 1;
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) tokens[acc] = found != INT_MAX ? found : last_pos;
}

bool verify_shape_ok(int B, int D, int V) {
  return B >= 1 && B <= 65535 && D >= 0 && D <= kMaxDraft && V >= 1 && V <= (1 << 30);
}
int verify_chunks(int V) { return ceil_div_i(V, kVfChunk); }

}  // namespace
}  // namespace fl

using namespace fl;

extern "C" {

size_t flashloop_verify_draft_scratch_bytes(int B, int D, int V) {
  if (!verify_shape_ok(B, D, V)) return 0;
  return align256_sz(static_cast<size_t>(B) * (2 * D + 1) * verify_chunks(V) * sizeof(RowPart)) + 256;
}

fl_status flashloop_verify_draft(const flashloop_verify_args* c, void* scratch, size_t scratch_bytes,
                                 fl_stream_t stream) {
  if (!c) return refuse(FL_ERR_INVALID_ARG, "NULL arguments");
  if (!verify_shape_ok(c->B, c->D, c->V)) return refuse(FL_ERR_INVALID_ARG, "B, D (0 to 64) or V out of range");
  if (!(c->temperature >= 0.f) || !std::isfinite(c->temperature))
    return refuse(FL_ERR_INVALID_ARG, "temperature must be finite and not negative");
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
    return refuse(FL_ERR_WORKSPACE, "scratch must be 256-byte aligned and hold " + std::to_string(need) + " bytes");
  VerifyArgs a{};
  a.c = *c;
  if (c->temperature == 0.f) a.c.draft_logits = nullptr;   // greedy: the target's rows alone
  a.n_chunks = verify_chunks(c->V);
  a.scale2 = c->temperature > 0.f ? 1.4426950408889634 / static_cast<double>(c->temperature) : 0.0;
  a.part = static_cast<RowPart*>(scratch);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = c->D + 1 + (a.c.draft_logits ? c->D : 0);
  cudaError_t e = launch_k(false, k_verify_rows, dim3(a.n_chunks, rows, c->B), dim3(kVfThreads), 0, s, a);
  if (e != cudaSuccess) return cuda_status(e);
  int nc = 1;   // a CTA per 4096 tokens of a row, at most 8
  while (nc < kVfCluster && c->V > nc * 4096) nc *= 2;
  if (c->temperature == 0.f) nc = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, c->B);
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nc;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, k_verify_pick, a));
}

}  // extern "C"
