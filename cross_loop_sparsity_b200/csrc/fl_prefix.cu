// fl_prefix.cu -- attention of a batch that shares a prefix, and the attention
// weight of key columns.
//
// Shared prefix: the batch's queries of one KV head form one matrix, so a tile
// of the prefix is read once for all of them instead of once per sequence.  The
// columns -- the prefix, and each sequence's own rows -- are split over CTAs;
// every split leaves (max, sum, unnormalised output) per row in fp32, and one
// merge forms the softmax over all of them:
//   M = max_i m_i,  L = sum_i e^(m_i - M) l_i,  out = sum_i e^(m_i - M) o_i / L.
#include <algorithm>
#include <cmath>

#include "fl_mma.cuh"
#include "fl_serving.h"

namespace fl {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPxTile = 32;                       // keys of one warp's tile
constexpr int kPxWarps = 4;
constexpr int kPxRing = kPxWarps * 24 * 1024;     // bytes of the four warps' tile rings (two CTAs per SM)
constexpr int kMaxGroup = 64;                     // query heads per KV head
constexpr int kMaxTq = 64;

struct PrefixArgs {
  const uint16_t* q;      // bf16 queries, or
  const float* q32;       // fp32 queries (hi + lo products)
  long long q_sb, q_st, q_sh;
  uint16_t* out;
  long long o_sb, o_st, o_sh;
  float* out32;
  float* lse;
  const uint16_t *k, *v;  // each sequence's own rows (the merge reads the causal tail itself)
  long long k_sb, k_sg, k_sr, v_sb, v_sg, v_sr;
  const int32_t* lens;
  const int32_t* q_lens;
  int lens_add;
  int B, Tq, H, Hkv, G, P, S;
  float scale2;           // scale * log2(e): the softmax runs in powers of two
  int rb_p, n_p;          // prefix: row blocks per KV head, column splits
  int rb_s, n_s;          // own rows: row blocks per (sequence, KV head), column splits
  int items_p;            // row blocks x splits of the prefix part (CTAs, or warps of k_prefix_rows)
  long long rows;         // B * Tq * H
  float* part_o;          // [n_p + n_s][rows][hd]
  float2* part_ml;        // [n_p + n_s][rows]: max (log2 domain), sum
  int tc_ctas;            // > 0: the prefix part runs on k_prefix_tc with at most this many CTAs (n_p = items_p = 0)
  float* tc_o;            // [tc_ctas + Hkv * row blocks][kTcRows][hd]
  float2* tc_ml;          // [tc_ctas + Hkv * row blocks][kTcRows]
  int* status;            // where a context's step records a wait that ran out, or nullptr (its result is NaN either way)
};

// a / b for a, b >= 0: most quotients here fit the 32-bit divider, several times faster than the 64-bit one
__device__ __forceinline__ long long quick_div(long long a, long long b) {
  return (static_cast<unsigned long long>(a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                                                         : a / b;
}

// How k_prefix_tc divides the prefix: row blocks of kTcRows packed query rows, 128-key tiles; the
// (row block, KV head, tile) units in this order, evenly over the CTAs by cost, so a CTA's
// range covers few (row block, head) pairs.  CTA c's part of pair p is partial c + p.  A unit of a
// block with more than 128 rows is two products of 128 rows; one of a shorter block is one,
// at 0.7 of the cost (it reads the same keys and values).
constexpr int kTcRows = 256, kTcTile = 128, kTcMinTiles = 2;
struct TcPlan {
  int nblk, ntiles, ctas;
  long long units, full;     // all units; those of blocks with more than 128 rows, which come first
  __device__ TcPlan(const PrefixArgs& a, int queries) {
    const int rows = queries * a.G;
    nblk = (rows + kTcRows - 1) / kTcRows;
    ntiles = (a.P + kTcTile - 1) / kTcTile;
    const long long per_block = static_cast<long long>(a.Hkv) * ntiles;
    units = nblk * per_block;
    full = rows - (nblk - 1) * kTcRows > 128 ? units : units - per_block;
    ctas = static_cast<int>(min(static_cast<long long>(a.tc_ctas), max(1LL, quick_div(units, kTcMinTiles))));
  }
  __device__ long long cost(long long u) const { return u <= full ? 10 * u : 10 * full + 7 * (u - full); }
  __device__ long long begin(int c) const {   // first unit of CTA c: at least two units' cost apart
    const long long x = quick_div(c * cost(units), ctas);
    return x <= 10 * full ? quick_div(x + 9, 10) : full + quick_div(x - 10 * full + 6, 7);
  }
  __device__ int cta_of(long long u) const {
    int c = min(ctas - 1, static_cast<int>(quick_div(cost(u) * ctas, cost(units))));
    while (c > 0 && begin(c) > u) --c;
    while (c + 1 < ctas && begin(c + 1) <= u) ++c;
    return c;
  }
};

__device__ __forceinline__ int q_len_of(const PrefixArgs& a, int b) {
  return a.q_lens ? min(max(a.q_lens[b], 0), a.Tq) : a.Tq;
}
__device__ __forceinline__ int len_of(const PrefixArgs& a, int b) {
  return a.S ? min(max(a.lens[b] + a.lens_add, 0), a.S) : 0;
}

// The valid queries of the batch, packed: query number i of all sequences'
// first q_lens[b] ones, i in [first, first + count), as slots b * Tq + t (-1 past
// the last).  Called by one warp with the lanes' q_len_of sequences 0..31 (0 past the last); returns how
// many queries there are in all.
__device__ int pack_queries(const PrefixArgs& a, int first, int count, int n, int* slot) {
  const int lane = threadIdx.x & 31;
  if (!a.q_lens) {
    const int total = a.B * a.Tq;
    for (int i = lane; i < count; i += 32) slot[i] = first + i < total ? first + i : -1;
    return total;
  }
  for (int i = lane; i < count; i += 32) slot[i] = -1;
  __syncwarp();
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (b0) n = b0 + lane < a.B ? q_len_of(a, b0 + lane) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int start = base + incl - n - first;
    for (int t = max(0, -start); t < n && start + t < count; ++t) slot[start + t] = (b0 + lane) * a.Tq + t;
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  return base;
}

// byte offset of 16-byte chunk c (8 dims) of row r in a tile of 128-byte swizzled boxes of `rows` rows
__device__ __forceinline__ uint32_t sw_off(int rows, int r, int c) {
  return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// two fp32 to packed bf16 (low half: the first), one conversion
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One warp's tiles: scores, running softmax and products for its 16 NM query rows (bf16 in shared memory at qs,
// HILO: their low parts QBYTES behind).  tile(n): where load n lies (K even, V odd); columns(i): those of tile i that
// are in range; arrived(n), refill(): wait for a load, give its slot to the next.  Returns the tiles
// done, fewer than `mine` when a load never arrived.
template <int HD, int NM, bool HILO, class Tile, class Columns, class Arrived, class Refill>
__device__ __forceinline__ int warp_tiles(int mine, uint32_t qs, float scale2, Tile tile, Columns columns, Arrived arrived,
                                          Refill refill, float (&m_run)[NM][2], float (&l_run)[NM][2],
                                          float (&acc)[NM][HD / 8][4]) {
  constexpr int RB = 16 * NM, QBYTES = RB * HD * 2, NT = HD / 8;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    m_run[i][0] = m_run[i][1] = -INFINITY;
    l_run[i][0] = l_run[i][1] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
  }
  int done = 0;
  for (; done < mine; ++done) {
    if (!arrived(2 * done)) break;
    const uint32_t Kt = smem_u32(tile(2 * done));
    const int nc = min(kPxTile, columns(done));   // columns of this tile in range
    // ---- scores of the tile's 32 keys
    float s[NM][4][4] = {};
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
      uint32_t kf[2][4];
#pragma unroll
      for (int n2 = 0; n2 < 2; ++n2)
        ldsm_x4(Kt + sw_off(kPxTile, n2 * 16 + (lane & 7) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1)), kf[n2]);
#pragma unroll
      for (int i = 0; i < NM; ++i) {
#pragma unroll
        for (int part = 0; part < (HILO ? 2 : 1); ++part) {
          uint32_t qf[4];
          ldsm_x4(qs + part * QBYTES + sw_off(RB, i * 16 + (lane & 15), k * 2 + (lane >> 4)), qf);
#pragma unroll
          for (int n2 = 0; n2 < 2; ++n2) {
            mma_bf16_16816(s[i][n2 * 2], qf, kf[n2][0], kf[n2][1]);
            mma_bf16_16816(s[i][n2 * 2 + 1], qf, kf[n2][2], kf[n2][3]);
          }
        }
      }
    }
    refill();
    // ---- running softmax: thread holds rows lane/4 (+8), columns 8n + 2(lane%4) + {0, 1}
    uint32_t pf[NM][2][4], pl[HILO ? NM : 1][2][4];
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[i][n][e] * scale2;
          if (nc < kPxTile && n * 8 + 2 * (lane & 3) + (e & 1) >= nc) x = -INFINITY;
          s[i][n][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      float al[2], ms[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        const float mn = fmaxf(m_run[i][e], mx[e]);
        ms[e] = mn == -INFINITY ? 0.f : mn;   // nothing finite yet: weights of 0, not NaN
        al[e] = exp2f(m_run[i][e] - ms[e]);
        m_run[i][e] = mn;
        l_run[i][e] *= al[e];
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2f(s[i][n][e] - ms[e >> 1]);
          s[i][n][e] = p;
          l_run[i][e >> 1] += p;
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[i][n][0] *= al[0];
        acc[i][n][1] *= al[0];
        acc[i][n][2] *= al[1];
        acc[i][n][3] *= al[1];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = s[i][2 * k + (j >> 1)][(j & 1) * 2], x1 = s[i][2 * k + (j >> 1)][(j & 1) * 2 + 1];
          pf[i][k][j] = pack_bf16x2(x0, x1);
          if (HILO)
            pl[HILO ? i : 0][k][j] = pack_bf16x2(x0 - bf16_to_f(pf[i][k][j] & 0xFFFF), x1 - bf16_to_f(pf[i][k][j] >> 16));
        }
    }
    // ---- output += P V
    if (!arrived(2 * done + 1)) break;
    uint8_t* vt = tile(2 * done + 1);
    const uint32_t Vt = smem_u32(vt);
    if (nc < kPxTile) {
      // rows past the range (another query's tokens, or never written): their
      // probabilities are 0, and 0 times what they hold must stay 0
      for (int e = lane; e < (kPxTile - nc) * (HD / 8); e += 32)
        *reinterpret_cast<uint4*>(vt + sw_off(kPxTile, nc + e / (HD / 8), e % (HD / 8))) = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int n2 = 0; n2 < NT / 2; ++n2) {
        uint32_t vf[4];
        ldsm_x4_t(Vt + sw_off(kPxTile, k * 16 + (lane & 15), n2 * 2 + (lane >> 4)), vf);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          mma_bf16_16816(acc[i][n2 * 2], pf[i][k], vf[0], vf[1]);
          mma_bf16_16816(acc[i][n2 * 2 + 1], pf[i][k], vf[2], vf[3]);
          if (HILO) {
            mma_bf16_16816(acc[i][n2 * 2], pl[HILO ? i : 0][k], vf[0], vf[1]);
            mma_bf16_16816(acc[i][n2 * 2 + 1], pl[HILO ? i : 0][k], vf[2], vf[3]);
          }
        }
      }
    }
    refill();
  }
  // the sums of a row, over its four lanes
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l_run[i][e] += __shfl_xor_sync(0xffffffffu, l_run[i][e], 1);
      l_run[i][e] += __shfl_xor_sync(0xffffffffu, l_run[i][e], 2);
    }
  return done;
}

// ============================================================================
// One split: up to 16 NM query rows of one KV head over a range of columns of
// the prefix (rows of every sequence, packed) or of one sequence's own rows.
// Four warps take alternate 32-key tiles, each from a TMA ring of its own, with
// its own running (max, sum, output): no barrier between warps until the end.
// HBM-bound: a tile's 16 KB feed 16 NM rows.  mma.sync, because a query row block of a decode
// step has 1 to 32 rows: a 128-row tcgen05 tile would be mostly padding (k_prefix_tc takes over from 33 rows).
// Two CTAs per SM, 24 KB of ring per warp, reused by halves (K, then V): with 64 samples' own 500 to 1000
// columns of 8 heads x 128 behind an 8192-column prefix the whole call took 68 us then, 74 with one
// CTA per SM and twice the ring (70 now, with the merge's later form).  A row sees every column of
// the range -- a sequence's columns stop at the last one all its queries see;
// the few that only later queries see are added by the merge -- so what a masked
// row of V holds never meets a product.  HILO: fp32 queries and probabilities as
// bf16 hi + lo pairs (about 16 significant bits); otherwise P enters the
// product with V rounded to bf16, as one product of the tensor cores takes it: a weight is off by at most 2^-8 of
// itself, and the outputs' error against 64 bits goes from 0.0017 (their own rounding to bf16) to 0.0018 relative.
// ============================================================================
template <int HD, int NM, bool HILO>
__global__ void __launch_bounds__(128, 2)
    k_prefix_split(const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp,
                   const __grid_constant__ CUtensorMap ks, const __grid_constant__ CUtensorMap vs, const PrefixArgs a) {
  constexpr int RB = 16 * NM;                       // query rows
  constexpr int TILE_BYTES = kPxTile * HD * 2;      // K or V of one tile
  constexpr int SLOTS = kPxRing / kPxWarps / TILE_BYTES;   // a warp's ring: K_0 V_0 K_1 V_1 .., a slot each
  constexpr int QBYTES = RB * HD * 2;
  constexpr int NT = HD / 8;                        // 8-dim output tiles
  constexpr int OLD = HD + 8;                       // padded row of the merge buffer
  extern __shared__ uint8_t sm_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qsm = ring + kPxRing;
  __shared__ __align__(8) uint64_t full[kPxWarps][12];
  __shared__ int slot_sm[RB + 1];
  __shared__ long long row_id[RB], q_at[RB];   // of a row: its number in the call (-1: none), its place in q
  __shared__ float sm_w[RB][kPxWarps];
  __shared__ float sm_m[kPxWarps][RB], sm_l[kPxWarps][RB];
  __shared__ int n_valid_sm, bad_sm;
  static_assert(SLOTS <= 12, "barriers");

  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (lane == 0) {   // a warp's barriers are its own
    for (int i = 0; i < SLOTS; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    fence_mbar_init();
    if (warp == 0) bad_sm = 0;
  }
  __syncwarp();
  // Behind k_prefix_tc (which started after everything this call reads was
  // written, and shares nothing with this kernel) the wait moves to the end: the
  // two overlap, and the merge, which waits for this kernel, finds both complete.
  if (!a.tc_ctas) pdl_wait();
  // ---- which rows, which columns
  const bool pre = static_cast<int>(blockIdx.x) < a.items_p;
  int it = pre ? blockIdx.x : blockIdx.x - a.items_p;
  const int rbs = pre ? a.rb_p : a.rb_s, nsp = pre ? a.n_p : a.n_s;
  const int rb = it % rbs;
  it /= rbs;
  const int sp = it % nsp;
  it /= nsp;
  const int g = it % a.Hkv, b = it / a.Hkv;
  const int r0 = rb * RB;
  int ncols = a.P, nrows;
  int ql = 0;   // (pre: of the lane's sequence, for pack_queries)
  if (!pre) {
    const int len = len_of(a, b);
    ql = q_len_of(a, b);
    nrows = ql * a.G;
    ncols = min(max(len - ql + 1, 0), len);
  } else if (warp == 0 && lane < a.B) {
    ql = q_len_of(a, lane);
  }
  // ---- this warp's tiles, the first of them requested while the rows are still being looked up
  const int ntiles = (ncols + kPxTile - 1) / kPxTile;
  const int tb = static_cast<int>(quick_div(static_cast<long long>(sp) * ntiles, nsp));
  const int te = static_cast<int>(quick_div(static_cast<long long>(sp + 1) * ntiles, nsp));
  const int mine = te - tb > warp ? (te - tb - warp + kPxWarps - 1) / kPxWarps : 0;
  const CUtensorMap* km = pre ? &kp : &ks;
  const CUtensorMap* vm = pre ? &vp : &vs;
  uint8_t* wring = ring + warp * (kPxRing / kPxWarps);
  auto issue = [&](int n) {   // load n: K (even) or V (odd) of this warp's tile n / 2
    const int y = (tb + warp + (n >> 1) * kPxWarps) * kPxTile;
    const uint32_t st = smem_u32(wring + (n % SLOTS) * TILE_BYTES), fb = smem_u32(&full[warp][n % SLOTS]);
    const CUtensorMap* map = (n & 1) ? vm : km;
    mbar_arrive_expect_tx(fb, TILE_BYTES);
    tma_load_5d(st, map, fb, 0, y, 0, g, pre ? 0 : b);
  };
  int issued = 0;             // (lane 0)
  if (lane == 0 && (pre || r0 < nrows))
    for (; issued < SLOTS && issued < 2 * mine; ++issued) issue(issued);
  // whole warp: load n has arrived, or (false) its wait ran out
  auto arrived = [&](int n) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[warp][n % SLOTS]), (n / SLOTS) & 1, a.status)) != 0;
  };
  // whole warp: a slot has been read; the next load takes it
  auto refill = [&]() {
    __syncwarp();
    if (lane == 0 && issued < 2 * mine) issue(issued++);
  };
  // lane 0: the copies in flight land (bounded) before the block can end
  auto land = [&]() {
    each_in_flight(issued, SLOTS, [&](int slot, int parity) { mbar_wait(smem_u32(&full[warp][slot]), parity, a.status); });
  };
  auto place = [&](int slot, int in_group) {   // (thread tid's row)
    const int h = g * a.G + in_group, sb = slot / a.Tq;
    row_id[tid] = slot < 0 ? -1 : static_cast<long long>(slot) * a.H + h;
    q_at[tid] = sb * a.q_sb + (slot - sb * a.Tq) * a.q_st + h * a.q_sh;
  };
  if (pre) {
    const int first = r0 / a.G, count = (r0 + RB - 1) / a.G - first + 1;
    if (warp == 0) {
      const int total = pack_queries(a, first, count, ql, slot_sm);
      if (lane == 0) n_valid_sm = total;
    }
    __syncthreads();
    nrows = n_valid_sm * a.G;
    if (tid < RB) {
      const int q = (r0 + tid) / a.G;
      place(r0 + tid < nrows ? slot_sm[q - first] : -1, r0 + tid - q * a.G);
    }
  } else if (tid < RB) {
    const int q = (r0 + tid) / a.G;
    place(r0 + tid < nrows ? b * a.Tq + q : -1, r0 + tid - q * a.G);
  }
  __syncthreads();   // row_id
  if (r0 >= nrows) {
    if (lane == 0) land();   // (no rows after all)
    if (a.tc_ctas) pdl_wait();
    return;
  }

  // ---- queries to shared memory (rows past the last: zero)
#pragma unroll
  for (int e = tid; e < RB * (HD / 8); e += 128) {
    const int r = e / (HD / 8), c = e % (HD / 8);
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (row_id[r] >= 0) {
      const long long off = q_at[r] + c * 8;
      if (!HILO) {
        hi = *reinterpret_cast<const uint4*>(a.q + off);
      } else {
        const float4 x0 = *reinterpret_cast<const float4*>(a.q32 + off);
        const float4 x1 = *reinterpret_cast<const float4*>(a.q32 + off + 4);
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        float h8[8], l8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split_bf16(x[i], h8[i], l8[i]);
        hi = make_uint4(pack_bf16x2(h8[0], h8[1]), pack_bf16x2(h8[2], h8[3]), pack_bf16x2(h8[4], h8[5]),
                        pack_bf16x2(h8[6], h8[7]));
        lo = make_uint4(pack_bf16x2(l8[0], l8[1]), pack_bf16x2(l8[2], l8[3]), pack_bf16x2(l8[4], l8[5]),
                        pack_bf16x2(l8[6], l8[7]));
      }
    }
    *reinterpret_cast<uint4*>(qsm + sw_off(RB, r, c)) = hi;
    if (HILO) *reinterpret_cast<uint4*>(qsm + QBYTES + sw_off(RB, r, c)) = lo;
  }
  __syncthreads();

  float m_run[NM][2], l_run[NM][2], acc[NM][NT][4];
  const int done = warp_tiles<HD, NM, HILO>(
      mine, smem_u32(qsm), a.scale2, [&](int n) { return wring + n % SLOTS * TILE_BYTES; },
      [&](int i) { return ncols - (tb + warp + i * kPxWarps) * kPxTile; }, arrived, refill, m_run, l_run, acc);
  if (done < mine && lane == 0) {
    // a tile never arrived; the result becomes NaN
    bad_sm = 1;
    land();
  }
  // ---- the four warps' parts become one
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if ((lane & 3) == 0) {
        sm_m[warp][i * 16 + e * 8 + (lane >> 2)] = m_run[i][e];
        sm_l[warp][i * 16 + e * 8 + (lane >> 2)] = l_run[i][e];
      }
    }
  __syncthreads();   // every warp is done with its ring
  float* om = reinterpret_cast<float*>(ring);   // [warps][RB][OLD]
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* d0 = om + (warp * RB + i * 16 + (lane >> 2)) * OLD + n * 8 + 2 * (lane & 3);
      *reinterpret_cast<float2*>(d0) = make_float2(acc[i][n][0], acc[i][n][1]);
      *reinterpret_cast<float2*>(d0 + 8 * OLD) = make_float2(acc[i][n][2], acc[i][n][3]);
    }
  const long long split = pre ? sp : a.n_p + sp;
  if (tid < RB) {
    const long long id = row_id[tid];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kPxWarps; ++w) M = fmaxf(M, sm_m[w][tid]);
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kPxWarps; ++w) {
      const float wt = exp2f(sm_m[w][tid] - ms);
      sm_w[tid][w] = wt;
      L += wt * sm_l[w][tid];
    }
    if (id >= 0) a.part_ml[split * a.rows + id] = bad_sm ? make_float2(0.f, NAN) : make_float2(M, L);
  }
  __syncthreads();
  // (a row with nothing finite too: the merge does not look at what stands behind a maximum of -inf)
#pragma unroll 4
  for (int e = tid; e < RB * (HD / 4); e += 128) {
    const int r = e / (HD / 4), d = (e % (HD / 4)) * 4;
    const long long id = row_id[r];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPxWarps; ++w) {
      const float wt = sm_w[r][w];
      const float4 x = *reinterpret_cast<const float4*>(om + (w * RB + r) * OLD + d);
      o.x += wt * x.x;
      o.y += wt * x.y;
      o.z += wt * x.z;
      o.w += wt * x.w;
    }
    if (id >= 0) *reinterpret_cast<float4*>(a.part_o + (split * a.rows + id) * HD + d) = o;
  }
  if (a.tc_ctas) pdl_wait();
}

// ============================================================================
// The same for many rows and few columns: a row block per warp over all tiles of its
// split, with rows, queries and results of its own and no step that the CTA takes together.  The
// queries take the first slot of the warp's ring.  Bound by each warp's chain of latencies (lengths,
// rows, queries, tile, products), which four row blocks per CTA share instead of one.
// ============================================================================
template <int HD, int NM>
__global__ void __launch_bounds__(128, 2)
    k_prefix_rows(const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp,
                  const __grid_constant__ CUtensorMap ks, const __grid_constant__ CUtensorMap vs, const PrefixArgs a, int items) {
  constexpr int RB = 16 * NM, TILE_BYTES = kPxTile * HD * 2, NT = HD / 8;
  constexpr int SLOTS = kPxRing / kPxWarps / TILE_BYTES - 1;   // of tiles, behind the queries
  static_assert(RB * HD * 2 <= TILE_BYTES && SLOTS >= 2 && SLOTS <= 12, "the warp's ring");
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[kPxWarps][12];
  __shared__ int slot_sm[kPxWarps][RB + 1];
  __shared__ long long row_id[kPxWarps][RB], q_at[kPxWarps][RB];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* wring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023)) +
                   warp * (kPxRing / kPxWarps);
  if (!a.tc_ctas) pdl_wait();   // (else at the end, as in k_prefix_split)
  int it = blockIdx.x * kPxWarps + warp;
  if (it >= items) {
    if (a.tc_ctas) pdl_wait();
    return;
  }
  if (lane == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    fence_mbar_init();
  }
  __syncwarp();
  const bool pre = it < a.items_p;
  if (!pre) it -= a.items_p;
  const int rbs = pre ? a.rb_p : a.rb_s, nsp = pre ? a.n_p : a.n_s;
  const int rb = it % rbs;
  it /= rbs;
  const int sp = it % nsp;
  it /= nsp;
  const int g = it % a.Hkv, b = it / a.Hkv, r0 = rb * RB;
  int ncols = a.P, nrows = 0, ql = 0;
  if (!pre) {
    const int len = len_of(a, b);
    ql = q_len_of(a, b);
    nrows = ql * a.G;
    ncols = min(max(len - ql + 1, 0), len);
  } else if (lane < a.B) {
    ql = q_len_of(a, lane);
  }
  const int ntiles = (ncols + kPxTile - 1) / kPxTile;
  const int tb = static_cast<int>(quick_div(static_cast<long long>(sp) * ntiles, nsp));
  const int mine = static_cast<int>(quick_div(static_cast<long long>(sp + 1) * ntiles, nsp)) - tb;
  auto slot_at = [&](int n) { return wring + (1 + n % SLOTS) * TILE_BYTES; };
  auto issue = [&](int n) {   // load n: K (even) or V (odd) of tile n / 2
    const uint32_t fb = smem_u32(&full[warp][n % SLOTS]);
    mbar_arrive_expect_tx(fb, TILE_BYTES);
    tma_load_5d(smem_u32(slot_at(n)), pre ? ((n & 1) ? &vp : &kp) : ((n & 1) ? &vs : &ks), fb, 0, (tb + (n >> 1)) * kPxTile, 0, g,
                pre ? 0 : b);
  };
  int issued = 0;             // (lane 0)
  if (lane == 0 && (pre || r0 < nrows))
    for (; issued < SLOTS && issued < 2 * mine; ++issued) issue(issued);
  auto arrived = [&](int n) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[warp][n % SLOTS]), (n / SLOTS) & 1, nullptr)) != 0;
  };
  auto refill = [&]() {
    __syncwarp();
    if (lane == 0 && issued < 2 * mine) issue(issued++);
  };
  // lane 0: the copies in flight land (bounded) before the block can end
  auto land = [&]() {
    each_in_flight(issued, SLOTS, [&](int slot, int parity) { mbar_wait(smem_u32(&full[warp][slot]), parity, nullptr); });
  };
  const int first = r0 / a.G;
  if (pre) {
    nrows = pack_queries(a, first, (r0 + RB - 1) / a.G - first + 1, ql, slot_sm[warp]) * a.G;
    __syncwarp();
  }
  if (r0 >= nrows) {
    if (lane == 0) land();    // (no rows after all)
    if (a.tc_ctas) pdl_wait();
    return;
  }
  if (lane < RB) {
    const int q = (r0 + lane) / a.G, h = g * a.G + r0 + lane - q * a.G;
    const int slot = r0 + lane >= nrows ? -1 : pre ? slot_sm[warp][q - first] : b * a.Tq + q, sb = slot / a.Tq;
    row_id[warp][lane] = slot < 0 ? -1 : static_cast<long long>(slot) * a.H + h;
    q_at[warp][lane] = sb * a.q_sb + (slot - sb * a.Tq) * a.q_st + h * a.q_sh;
  }
  __syncwarp();
#pragma unroll 8
  for (int e = lane; e < RB * (HD / 8); e += 32) {   // (rows past the last: zero)
    const int r = e / (HD / 8), c = e % (HD / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row_id[warp][r] >= 0) x = *reinterpret_cast<const uint4*>(a.q + q_at[warp][r] + c * 8);
    *reinterpret_cast<uint4*>(wring + sw_off(RB, r, c)) = x;
  }
  __syncwarp();
  float m_run[NM][2], l_run[NM][2], acc[NM][NT][4];
  const int done = warp_tiles<HD, NM, false>(
      mine, smem_u32(wring), a.scale2, slot_at, [&](int i) { return ncols - (tb + i) * kPxTile; }, arrived, refill, m_run, l_run,
      acc);
  if (done < mine && lane == 0) land();   // a tile never arrived; the rows become NaN
  const long long split = pre ? sp : a.n_p + sp;
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long id = row_id[warp][i * 16 + e * 8 + (lane >> 2)];
      if (id < 0) continue;
      const long long at = split * a.rows + id;
      if ((lane & 3) == 0) a.part_ml[at] = done < mine ? make_float2(0.f, NAN) : make_float2(m_run[i][e], l_run[i][e]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(a.part_o + at * HD + n * 8 + 2 * (lane & 3)) =
            make_float2(acc[i][n][2 * e], acc[i][n][2 * e + 1]);
    }
  if (a.tc_ctas) pdl_wait();
}

// ============================================================================
// The prefix on the 5th-generation tensor cores, when the batch has more query
// rows per KV head than two warp tiles: 256 rows share every K and V tile, so
// the kernel is bound by the tensor pipe (4 * 256 FLOP per byte) for full row
// blocks and by HBM for a few.  Four softmax warpgroups, one MMA warp, one TMA
// thread.  A job is one 128-row x 128-key product: S = Q K^T into the job's half
// of TMEM, softmax on S by its two warpgroups (a thread owns 64 columns of a
// row; the two halves of a row exchange their maxima), P as bf16 over S, O += P V with P
// read from TMEM.  Jobs alternate between the two halves, so one half's
// products run under the other's softmax.  With more than 128 rows the halves
// are two row tiles of the same keys; with fewer they are the same rows over
// alternate key tiles, joined at the end.
//   Running maximum: O is rescaled only when a row's maximum has grown by more
// than 8 (log2 domain) -- until then the old one stays, the probabilities are at
// most 2^8, and bf16's relative precision is the same there.
//   P enters the second product rounded to bf16 (as in the prefill attention), by at most 2^-8 of a weight, so that it takes
// one product instead of two; the sums use the fp32 values.  Outputs are then 0.0022 from 64 bits, relative, 0.0017
// of it their own rounding to bf16.
//   Measured: 256 rows x 65536 columns x 8 heads, hd 128, 69 GFLOP: 75 us (42 at the measured GEMM rate; about 20
// of the 75 are start and end: queries in, TMEM, pipeline fill, partial results out).  Two softmax
// warpgroups instead of four took 84.  In the steady state Q K^T, with both operands in
// shared memory, is what the rest waits for (128 x 128 x 128 in about 890 clocks, 512 ideal), so
// exponentials on the FMA pipe gained nothing here.
// ============================================================================
template <int HD>
struct TcSmem {
  static constexpr int kBox = 128 * 128;                 // 128 rows of 64 dims
  static constexpr int kTileBytes = (HD / 64) * kBox;    // 128 rows
  static constexpr int kKSlots = HD == 128 ? 3 : 6, kVSlots = HD == 128 ? 2 : 4;
  static constexpr int kTiles = (2 + kKSlots + kVSlots) * kTileBytes;
  static constexpr int kBytes = kTiles + 2048 + 256;     // then the maxima (or row places), barriers and flags
};
constexpr int kTcThreads = 576;   // 16 softmax warps, the MMA warp, the TMA warp

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_prefix_tc(const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp, const PrefixArgs a) {
  using C = TcSmem<HD>;
  constexpr int KS = C::kKSlots, VS = C::kVSlots;
  constexpr int OLD = HD + 4;                            // padded row of the join buffer
  // no static shared memory: the tiles start at the (1024-byte aligned) start of the block's, which they nearly fill
  extern __shared__ __align__(1024) uint8_t tc_sm[];
  uint8_t* qsm = tc_sm;
  uint8_t* ksm = qsm + 2 * C::kTileBytes;
  uint8_t* vsm = ksm + KS * C::kTileBytes;
  float* max_sm = reinterpret_cast<float*>(tc_sm + C::kTiles);          // [half][column half][row]; then the sums
  uint32_t* row_off = reinterpret_cast<uint32_t*>(max_sm);               // while no maxima are there: a query row's
                                                                         // place in q, in 16-byte units (~0: no row)
  uint64_t* bars = reinterpret_cast<uint64_t*>(tc_sm + C::kTiles + 2048);
  uint64_t *k_full = bars, *k_empty = k_full + KS, *v_full = k_empty + KS, *v_empty = v_full + VS, *s_full = v_empty + VS,
           *p_ready = s_full + 2, *p_first = p_ready + 2, *o_done = p_first + 2;
  static_assert((2 * KS + 2 * VS + 8) * 8 + 16 <= 256, "barriers");
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(tc_sm + C::kTiles + 2048 + 240);
  int& total_sm = *reinterpret_cast<int*>(tc_sm + C::kTiles + 2048 + 244);
  volatile int& bad = *reinterpret_cast<volatile int*>(tc_sm + C::kTiles + 2048 + 248);
  int* slot_sm = reinterpret_cast<int*>(qsm);            // while the query tiles are not there yet
  float2* join_ml = reinterpret_cast<float2*>(ksm + 128 * OLD * 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 17 * 32) {
    tma_prefetch_desc(&kp);
    tma_prefetch_desc(&vp);
  }
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(smem_u32(&v_full[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 256);
      mbar_init(smem_u32(&p_first[i]), 256);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    fence_mbar_init();
    bad = 0;
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();   // (the next launch may run beside this one; see its wait)
  if (warp == 0) {
    const int total = pack_queries(a, 0, 0, lane < a.B ? q_len_of(a, lane) : 0, slot_sm);
    if (lane == 0) total_sm = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int queries = total_sm, nrows = queries * a.G;
  // a negative scale: negated queries and its magnitude, so that the largest score is the largest product
  const float scale2 = fabsf(a.scale2);
  const uint32_t flip = a.scale2 < 0.f ? 0x80008000u : 0u;
  // counts of the barriers' phases, running over the CTA's segments
  int nk = 0, nv = 0;            // tiles loaded (TMA thread) or consumed (MMA thread)
  int ns[2] = {0, 0};            // jobs per half (MMA thread), or [0]: this warpgroup's jobs
  const TcPlan plan(a, queries);
  long long u = 0, u_end = 0;
  if (queries > 0 && static_cast<int>(blockIdx.x) < plan.ctas) {
    u = plan.begin(blockIdx.x);
    u_end = plan.begin(blockIdx.x + 1);
  }
  while (u < u_end && !bad) {
    const int pair = static_cast<int>(quick_div(u, plan.ntiles)), t0 = static_cast<int>(u - static_cast<long long>(pair) * plan.ntiles);
    const int nt = static_cast<int>(min(static_cast<long long>(plan.ntiles - t0), u_end - u));
    const int g = pair % a.Hkv, r0 = pair / a.Hkv * kTcRows;
    const int rows = min(kTcRows, nrows - r0);
    const bool two = rows > 128;               // the halves are two row tiles
    const int jobs = two ? 2 * nt : nt;        // job n: half n & 1, tile t0 + (two ? n / 2 : n)
    auto load_k = [&](int i) {                 // (TMA thread)
      const uint32_t bar = smem_u32(&k_full[nk % KS]), dst = smem_u32(ksm + (nk % KS) * C::kTileBytes);
      mbar_arrive_expect_tx(bar, C::kTileBytes);
      tma_load_5d(dst, &kp, bar, 0, (t0 + i) * kTcTile, 0, g, 0);
      ++nk;
    };
    auto load_v = [&](int i) {
      const uint32_t bar = smem_u32(&v_full[nv % VS]), dst = smem_u32(vsm + (nv % VS) * C::kTileBytes);
      mbar_arrive_expect_tx(bar, C::kTileBytes);
      tma_load_5d(dst, &vp, bar, 0, (t0 + i) * kTcTile, 0, g, 0);
      ++nv;
    };
    // ---- the segment's queries (every thread); the K and V rings fill meanwhile
    int k_at = 0, v_at = 0;                    // next tile to load (TMA thread): K_0 K_1 V_0 K_2 V_1 ...
    bool stop = false;
    if (tid == 17 * 32) {
      // the first tiles of a segment: their slots' last readers finished with the previous segment
      while (k_at < nt && k_at < KS) {
        stop = nk >= KS && !mbar_wait(smem_u32(&k_empty[nk % KS]), ((nk / KS) - 1) & 1, nullptr);
        if (stop) break;
        load_k(k_at++);
      }
      while (!stop && v_at < nt && v_at < VS) {
        stop = nv >= VS && !mbar_wait(smem_u32(&v_empty[nv % VS]), ((nv / VS) - 1) & 1, nullptr);
        if (stop) break;
        load_v(v_at++);
      }
    }
    // (warps 0-16: the TMA warp is not waited for, nor does it read the queries)
    if (warp == 0) {
      const int first = r0 / a.G, count = (r0 + rows - 1) / a.G - first + 1;
      pack_queries(a, first, count, lane < a.B ? q_len_of(a, lane) : 0, slot_sm);
    }
    if (warp < 16) {
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (tid < kTcRows) {
        const int r = r0 + tid, sl = tid < rows ? slot_sm[r / a.G - r0 / a.G] : 0;
        const long long off = (sl / a.Tq) * a.q_sb + (sl % a.Tq) * a.q_st + (g * a.G + r % a.G) * a.q_sh;
        row_off[tid] = tid < rows ? static_cast<uint32_t>(off >> 3) : ~0u;
      }
      asm volatile("bar.sync 1, 512;" ::: "memory");
      constexpr int CH = HD / 8, RP = 512 / CH;    // chunks of a row: thread t copies chunk t % CH of every RP-th row
      const int c = tid % CH;
#pragma unroll
      for (int i = 0; i < 256 / RP; ++i) {
        const int qr = tid / CH + i * RP;
        if (qr < 128 || two) {
          const uint32_t off16 = row_off[qr];
          cp_async_16(smem_u32(qsm + (qr >> 7) * C::kTileBytes + sw_off(128, qr & 127, c)),
                      a.q + (off16 == ~0u ? 0 : static_cast<long long>(off16) * 8 + c * 8), off16 == ~0u ? 0u : 16u);
        }
      }
      cp_async_wait_all();
      if (flip)
        for (int i = 0; i < 256 / RP; ++i) {       // the chunks this thread copied
          const int qr = tid / CH + i * RP;
          uint4* x = reinterpret_cast<uint4*>(qsm + (qr >> 7) * C::kTileBytes + sw_off(128, qr & 127, c));
          if (qr < 128 || two) *x = make_uint4(x->x ^ flip, x->y ^ flip, x->z ^ flip, x->w ^ flip);
        }
      fence_proxy_async();
    }
    if (warp < 17) asm volatile("bar.sync 2, 544;" ::: "memory");   // the MMA warp too

    if (warp < 16) {
      // ================= two softmax warpgroups of one half =================
      const int q = warp >> 3, sub = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + q * 128, to = tmem + lanes + 256 + q * HD + sub * (HD / 2);
      float* my_max = max_sm + (q * 2 + sub) * 128 + row;
      const float* other_max = max_sm + (q * 2 + (sub ^ 1)) * 128 + row;
      auto half_sync = [&]() {                 // the half's 256 threads
        if (q == 0) asm volatile("bar.sync 3, 256;" ::: "memory");
        else asm volatile("bar.sync 4, 256;" ::: "memory");
      };
      const int mine = (jobs + 1 - q) / 2;     // this half's jobs
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {   // the warp's threads agree: what follows is warp-wide
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase & 1, nullptr)) != 0;
      };
      for (int j = 0; j < mine; ++j, ++ns[0]) {
        // (after a wait that ran out the loop goes on without waiting, so that the barriers still meet)
        ok = ok && wait(&s_full[q], ns[0]);
        tc_fence_after();
        const uint32_t tj = ts + sub * 64;               // these 64 columns of S; P goes over their first 32
        const int ncol = a.P - (t0 + (two ? j : 2 * j + q)) * kTcTile - sub * 64;   // valid ones of them
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        uint32_t r[32];
        auto load = [&](int c) {
          tmem_ld32(tj + c * 32, r);
          tc_wait_ld();
          if (ncol < 64) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= ncol) r[e] = 0xFF800000u;   // -inf
          }
        };
#pragma unroll
        for (int c = 0; c < 2; ++c) {                    // (columns 32-63 stay in registers)
          load(c);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
        }
        *my_max = fmax3(fmax3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        half_sync();
        const float mrow = fmax3(*my_max, *other_max, *other_max);
        const float mn = mrow == -INFINITY ? -INFINITY : mrow * scale2;
        const bool grow = mn > m + 8.f || (m == -INFINITY && mn > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? mn : m;
          if (j > 0) {
            // this warpgroup's half of the row's output so far
            const float al = m == m_new ? 1.f : ex2_approx(m - m_new);
            ok = ok && wait(&o_done[q], ns[0] - 1);
            tc_fence_after();
            l *= al;
            if (ok) {
#pragma unroll 1
              for (int c = 0; c < HD / 2; c += 16) {
                float o[16];
                tmem_ld16(to + c, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= al;
                tmem_st16(to + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          m = m_new;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        const uint64_t sc2 = f2_pack(scale2, scale2), ms2 = f2_pack(-ms, -ms);
        uint64_t sum2[2] = {0, 0};
        auto probs = [&](uint32_t* pk) {   // (a column out of range: score -inf, probability 0)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc2, ms2);
            float p0, p1;
            f2_unpack(y2, p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum2[(e >> 1) & 1] = f2_add(sum2[(e >> 1) & 1], f2_pack(p0, p1));
            pk[e >> 1] = pack2(p0, p1);
          }
        };
        uint32_t pk[16];
        probs(pk);
        load(0);                               // before P of columns 32-63 goes over its second half
        tmem_st16(tj + 16, pk);
        tc_wait_st();
        tc_fence_before();
        if (ok) mbar_arrive(smem_u32(&p_first[q]));      // half of P: its products can start
        probs(pk);
        tmem_st16(tj, pk);
        {
          float x, y;
          f2_unpack(f2_add(sum2[0], sum2[1]), x, y);
          l += x + y;
        }
        tc_wait_st();
        tc_fence_before();
        if (ok) mbar_arrive(smem_u32(&p_ready[q]));
      }
      if (mine > 0) ok = ok && wait(&o_done[q], ns[0] - 1);
      if (!ok) bad = 1;
      tc_fence_after();
      // ---- this segment's part of the rows: (max, sum) and the unnormalised output, half a row at a
      // time by bulk copies from shared memory (the rings are idle: every product is done)
      const int at_row = (two ? q * 128 : 0) + row;
      const bool have = at_row < rows;
      const long long at = (blockIdx.x + pair) * static_cast<long long>(kTcRows) + at_row;
      float* so = reinterpret_cast<float*>(ksm) + at_row * OLD + sub * (HD / 2);
      *my_max = l;                                     // (every maximum has been read)
      asm volatile("bar.sync 1, 512;" ::: "memory");   // every softmax warp
      l += *other_max;                                 // the whole row's sum
      float w0 = 1.f, w1 = 0.f, M = m, L = l;
      if (!two) {
        // the halves are the same rows over alternate tiles: the second leaves its sums and output, the first joins
        if (q == 1) {
          if (sub == 0) join_ml[row] = make_float2(mine > 0 ? m : -INFINITY, l);
          if (mine > 0 && ok) {
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 16) {
              float o[16];
              tmem_ld16(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(so + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (q == 0) {
          const float2 x = join_ml[row];
          M = fmaxf(m, x.x);
          const float ms = M == -INFINITY ? 0.f : M;
          w0 = ex2_approx(m - ms);
          w1 = ex2_approx(x.x - ms);
          L = l * w0 + x.y * w1;
        }
      }
      if (two || q == 0) {
#pragma unroll 1
        for (int c = 0; c < HD / 2; c += 32) {
          uint32_t o[32];
          tmem_ld32(to + c, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 x = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                   __uint_as_float(o[e + 3]));
            if (!two && jobs > 1) {
              const float4 y = *reinterpret_cast<const float4*>(so + c + e);
              x = make_float4(x.x * w0 + y.x * w1, x.y * w0 + y.y * w1, x.z * w0 + y.z * w1, x.w * w0 + y.w * w1);
            }
            *reinterpret_cast<float4*>(so + c + e) = x;
          }
        }
        if (have) {
          if (sub == 0) a.tc_ml[at] = bad ? make_float2(0.f, NAN) : make_float2(M, L);
          fence_proxy_async();
          bulk_store(a.tc_o + at * HD + sub * (HD / 2), smem_u32(so), HD * 2);
          bulk_commit();
          bulk_wait_read();
        }
        __syncwarp();
      }
      fence_proxy_async();   // the join buffer becomes a ring again
      tc_fence_before();
    } else if (warp == 16) {
      // ================= MMA warp =================
      // The whole warp runs the loop and one elected lane issues: the operands are
      // then warp-uniform, as the instruction wants them.
      constexpr uint32_t id_s = umma_idesc_bf16(128, 128), id_o = umma_idesc_bf16(128, HD) | kIdescBMn;
      const int k0 = nk, v0 = nv, s0 = ns[0], s1 = ns[1];   // counts at the segment's start
      auto tile_of = [&](int n) { return two ? n >> 1 : n; };
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase & 1, nullptr)) != 0;
      };
      const uint64_t q_desc = umma_desc_sw128(smem_u32(qsm)), k_desc = umma_desc_sw128(smem_u32(ksm));
      const uint64_t v_desc = umma_desc_sw128_mn(smem_u32(vsm), C::kBox);
      auto do_qk = [&](int n) -> bool {
        const int q = n & 1, i = tile_of(n), kt = k0 + i, st = kt % KS;
        if (!wait(&k_full[st], kt / KS)) return false;
        tc_fence_after();
        const uint64_t da = q_desc + (two ? q : 0) * (C::kTileBytes >> 4), db = k_desc + st * (C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            tc_mma_bf16(tmem + q * 128, da + (k >> 2) * (C::kBox >> 4) + (k & 3) * 2,
                        db + (k >> 2) * (C::kBox >> 4) + (k & 3) * 2, id_s, k > 0);
          tc_commit(smem_u32(&s_full[q]));
          if (!two || q == 1) tc_commit(smem_u32(&k_empty[st]));
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      for (int n = 0; n < 2 && n < jobs; ++n) ok = ok && do_qk(n);
      for (int n = 0; ok && n < jobs; ++n) {
        const int q = n & 1, i = tile_of(n), vt = v0 + i, st = vt % VS, j = n >> 1;
        const uint64_t db = v_desc + st * (C::kTileBytes >> 4);
        // O += P V for the keys of one half of P: columns 32-63 (first) or 0-31 of each 64
        auto half_pv = [&](bool first) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = (k >> 1) * 4 + (first ? 2 : 0) + (k & 1);   // 16 keys
              tc_mma_bf16_ts(tmem + 256 + q * HD, tmem + q * 128 + (kk >> 2) * 64 + (kk & 3) * 8, db + kk * (2048 >> 4), id_o,
                             j > 0 || !first || k > 0);
            }
          }
          __syncwarp();
        };
        if (!wait(&p_first[q], (q ? s1 : s0) + j) || !wait(&v_full[st], vt / VS)) {
          ok = false;
          break;
        }
        half_pv(true);
        if (!wait(&p_ready[q], (q ? s1 : s0) + j)) {
          ok = false;
          break;
        }
        half_pv(false);
        if (elect_one()) {
          tc_commit(smem_u32(&o_done[q]));
          if (!two || q == 1) tc_commit(smem_u32(&v_empty[st]));
        }
        __syncwarp();
        if (n + 2 < jobs) ok = do_qk(n + 2);
      }
      nk += nt;
      nv += nt;
      ns[0] += (jobs + 1) / 2;
      ns[1] += jobs / 2;
      if (!ok) bad = 1;
    } else if (tid == 17 * 32) {
      // ================= TMA thread =================
      if (stop) bad = 1;
      while ((k_at < nt || v_at < nt) && !bad) {
        // V_i in front of K_{i+2}, as the products need them
        const bool vk = v_at < nt && (k_at >= nt || v_at <= k_at - 2);
        if (vk) {
          if (nv >= VS && !mbar_wait(smem_u32(&v_empty[nv % VS]), ((nv / VS) - 1) & 1, nullptr)) {
            bad = 1;
            break;
          }
          load_v(v_at++);
        } else {
          if (nk >= KS && !mbar_wait(smem_u32(&k_empty[nk % KS]), ((nk / KS) - 1) & 1, nullptr)) {
            bad = 1;
            break;
          }
          load_k(k_at++);
        }
      }
      if (bad) {   // let every copy in flight land (bounded) before the block can end
        each_in_flight(nk, KS, [&](int slot, int parity) { mbar_wait(smem_u32(&k_full[slot]), parity, nullptr); });
        each_in_flight(nv, VS, [&](int slot, int parity) { mbar_wait(smem_u32(&v_full[slot]), parity, nullptr); });
      }
    }
    __syncthreads();
    tc_fence_after();
    u += nt;
  }
  if (bad)   // a wait ran out: every part of this CTA becomes NaN, never a silently wrong sum
    for (long long w = plan.begin(blockIdx.x); w < u_end; w += plan.ntiles - w % plan.ntiles)
      if (tid < kTcRows) a.tc_ml[(blockIdx.x + w / plan.ntiles) * kTcRows + tid] = make_float2(0.f, NAN);
  bulk_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================
// Merge.  A group is HD/4 lanes, 4 dims each.  ALL: the CTA's groups share one
// output row -- each takes every n-th split (a few loads in flight) and every
// n-th column of the causal tail, and their (max, sum, output) meet in shared
// memory; for few rows, where latency counts.  Otherwise a row per group.  The
// causal tail: columns this query sees and an earlier one of its sequence does
// not, at most Tq - 1, as fp32 dot products, while the launch in front still runs.
//   A row per group: eight CTAs per SM and four splits requested together (117 x 6 queries of 64 heads, two splits:
// the whole call 70 us; five CTAs and eight splits 83, six and eight 81, eight and six 73; 160 queries
// over a long prefix 130 us against 132, 64 with 18 parts a row 70 against 69).
// ============================================================================
template <int HD, bool Q32, bool ALL>
__global__ void __launch_bounds__(128, ALL ? 4 : 8) k_prefix_merge(const PrefixArgs a) {
  constexpr int LPG = HD / 4;          // lanes of a group, 4 dims each
  constexpr int NG = 128 / LPG;        // groups
  constexpr int MB = ALL ? 8 : 4;      // splits requested together
  __shared__ float gm[NG], gl[NG];
  __shared__ float4 go[NG][LPG];
  __shared__ int cnt[2][4];
  pdl_trigger();
  const int grp = ALL ? threadIdx.x / LPG : 0, gl_lane = threadIdx.x % LPG;
  constexpr int GS = ALL ? NG : 1;     // groups that share a row
  const int row = ALL ? blockIdx.x : min(static_cast<int>(a.rows) - 1, static_cast<int>(blockIdx.x * NG + threadIdx.x / LPG));
  const bool last = ALL || static_cast<int>(blockIdx.x * NG + threadIdx.x / LPG) < a.rows;   // (a group past the end repeats the last row)
  const int slot = row / a.H, h = row - slot * a.H, b = slot / a.Tq, t = slot - b * a.Tq;
  // (a decode step's fp32 queries and lengths come from kernels the wait covers; a caller's were there before the first launch)
  if (Q32) pdl_wait();
  const int ql = q_len_of(a, b), len = len_of(a, b);
  const bool valid = last && t < ql;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float ms, float ls, const float4& x) {   // a part with maximum ms, sum ls, output x
    if (ms == -INFINITY) {   // nothing there: its output was never written
      l += ls;               // 0, or NaN
      return;
    }
    const float mn = fmaxf(m, ms);
    const float w0 = exp2f(m - mn), w1 = exp2f(ms - mn);
    l = l * w0 + ls * w1;
    o.x = o.x * w0 + x.x * w1;
    o.y = o.y * w0 + x.y * w1;
    o.z = o.z * w0 + x.z * w1;
    o.w = o.w * w0 + x.w * w1;
    m = mn;
  };
  // n partials of this row, `step` rows apart from row `at`
  auto add_parts = [&](const float* po, const float2* pml, long long at, long long step, int n) {
    for (int i0 = grp; i0 < n; i0 += GS * MB) {
      float2 ml[MB];
      float4 x[MB];
#pragma unroll
      for (int u = 0; u < MB; ++u) {
        const int i = i0 + u * GS;
        ml[u] = i < n ? __ldcg(&pml[at + i * step]) : make_float2(-INFINITY, 0.f);
        x[u] = i < n ? __ldcg(reinterpret_cast<const float4*>(&po[(at + i * step) * HD + gl_lane * 4]))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < MB; ++u)
        if (i0 + u * GS < n) add(ml[u].x, ml[u].y, x[u]);
    }
  };
  // the causal tail (a caller's inputs: before the wait, four columns' loads together)
  const int base = min(max(len - ql + 1, 0), len), lim = min(max(len - ql + t + 1, 0), len);
  if (valid && lim > base) {
    const int g = h / a.G;
    float4 q4;
    const long long qo = b * a.q_sb + t * a.q_st + h * a.q_sh + gl_lane * 4;
    if (Q32) {
      q4 = *reinterpret_cast<const float4*>(a.q32 + qo);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(a.q + qo);
      q4 = make_float4(bf16_to_f(u.x & 0xFFFF), bf16_to_f(u.x >> 16), bf16_to_f(u.y & 0xFFFF), bf16_to_f(u.y >> 16));
    }
    const unsigned mask = LPG == 32 ? 0xffffffffu : (0xffffu << (threadIdx.x & 16));
    constexpr int TB = Q32 ? 1 : 4;   // (a decode step's tail is empty: one query)
    for (int j0 = base + grp; j0 < lim; j0 += GS * TB) {
      uint2 ku[TB], vu[TB];
      float sc[TB];
#pragma unroll
      for (int u = 0; u < TB; ++u) {
        const int j = min(j0 + u * GS, lim - 1);
        ku[u] = *reinterpret_cast<const uint2*>(a.k + b * a.k_sb + g * a.k_sg + j * a.k_sr + gl_lane * 4);
        vu[u] = *reinterpret_cast<const uint2*>(a.v + b * a.v_sb + g * a.v_sg + j * a.v_sr + gl_lane * 4);
      }
#pragma unroll
      for (int u = 0; u < TB; ++u)
        sc[u] = q4.x * bf16_to_f(ku[u].x & 0xFFFF) + q4.y * bf16_to_f(ku[u].x >> 16) + q4.z * bf16_to_f(ku[u].y & 0xFFFF) +
                q4.w * bf16_to_f(ku[u].y >> 16);
#pragma unroll
      for (int d = LPG / 2; d > 0; d >>= 1)
#pragma unroll
        for (int u = 0; u < TB; ++u) sc[u] += __shfl_xor_sync(mask, sc[u], d);
#pragma unroll
      for (int u = 0; u < TB; ++u)
        if (j0 + u * GS < lim)
          add(sc[u] * a.scale2, 1.f, make_float4(bf16_to_f(vu[u].x & 0xFFFF), bf16_to_f(vu[u].x >> 16),
                                                 bf16_to_f(vu[u].y & 0xFFFF), bf16_to_f(vu[u].y >> 16)));
    }
  }
  if (!Q32) pdl_wait();
  if (ALL && t >= ql) return;
  add_parts(a.part_o, a.part_ml, row, a.rows, valid ? a.n_p + a.n_s : 0);
  if (a.tc_ctas > 0) {
    // this query's number among the valid ones, and all of them
    int before = b * a.Tq, all = a.B * a.Tq;
    if (a.q_lens) {
      before = all = 0;
      if (ALL) {
        for (int i = threadIdx.x; i < a.B; i += 128) {
          const int x = q_len_of(a, i);
          all += x;
          if (i < b) before += x;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        all = __reduce_add_sync(0xffffffffu, all);
        if ((threadIdx.x & 31) == 0) {
          cnt[0][threadIdx.x >> 5] = before;
          cnt[1][threadIdx.x >> 5] = all;
        }
        __syncthreads();
        before = cnt[0][0] + cnt[0][1] + cnt[0][2] + cnt[0][3];
        all = cnt[1][0] + cnt[1][1] + cnt[1][2] + cnt[1][3];
      } else {
        for (int i = gl_lane; i < a.B; i += LPG) {
          const int x = q_len_of(a, i);
          all += x;
          if (i < b) before += x;
        }
#pragma unroll
        for (int d = LPG / 2; d > 0; d >>= 1) {
          before += __shfl_xor_sync(0xffffffffu, before, d);
          all += __shfl_xor_sync(0xffffffffu, all, d);
        }
      }
    }
    const TcPlan plan(a, max(all, 1));
    const int r = (valid ? before + t : 0) * a.G + h % a.G;
    const int pair = r / kTcRows * a.Hkv + h / a.G;
    const int c0 = plan.cta_of(static_cast<long long>(pair) * plan.ntiles);
    const int c1 = plan.cta_of(static_cast<long long>(pair + 1) * plan.ntiles - 1);
    add_parts(a.tc_o, a.tc_ml, static_cast<long long>(c0 + pair) * kTcRows + r % kTcRows, kTcRows, valid ? c1 - c0 + 1 : 0);
  }
  float M = m, L = l;
  float4 r = o;
  if (ALL) {
    if (gl_lane == 0) {
      gm[grp] = m;
      gl[grp] = l;
    }
    go[grp][gl_lane] = o;
    __syncthreads();
    if (threadIdx.x >= LPG) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < NG; ++i) M = fmaxf(M, gm[i]);
    const float ms = M == -INFINITY ? 0.f : M;
    L = 0.f;
    r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const float w = exp2f(gm[i] - ms);
      const float4 x = go[i][gl_lane];
      L += w * gl[i] + (gm[i] == -INFINITY ? gl[i] : 0.f);
      r.x += w * x.x;
      r.y += w * x.y;
      r.z += w * x.z;
      r.w += w * x.w;
    }
  }
  if (!valid) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;   // nothing visible: 0 and -inf
  r.x *= inv;
  r.y *= inv;
  r.z *= inv;
  r.w *= inv;
  *reinterpret_cast<uint2*>(a.out + b * a.o_sb + t * a.o_st + h * a.o_sh + gl_lane * 4) =
      make_uint2(pack_bf16x2(r.x, r.y), pack_bf16x2(r.z, r.w));
  if (a.out32) *reinterpret_cast<float4*>(a.out32 + static_cast<long long>(row) * HD + gl_lane * 4) = r;
  if (a.lse && gl_lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// ============================================================================
// Attention weight of key columns: out = acc + sum over rows of
// 2^(scale2 q.k - lse2).  Every sum stays in one thread over all rows of a part, and
// parts meet in a fixed order: no atomics.
// ============================================================================
struct WeightsArgs {
  const uint16_t* q;
  long long q_sb, q_st, q_sh;
  const float* lse;
  const float* acc;
  float* out;
  const int32_t* lens;
  const int32_t* q_lens;
  int B, Tq, H, Hkv, G, S;
  float scale2;
  int nt;             // k_weights_tc: queries (of G rows) per row block
  int ctas;           // k_weights_tc: CTAs at most
  float* part;        // k_weights_tc: [ctas + key tiles][kWtCols]
};
// What the queries of sequence b see: query t columns j < min(j0 + t + 1, len) (every column when not causal).
struct Seen {
  int ql, len, j0;
  bool causal;
  __device__ Seen(const WeightsArgs& a, int b) {
    causal = a.lens != nullptr;
    ql = a.q_lens ? min(max(a.q_lens[b], 0), a.Tq) : a.Tq;
    len = causal ? min(max(a.lens[b], 0), a.S) : a.S;
    j0 = causal ? len - ql : len;
  }
  __device__ int limit(int t) const { return causal ? min(j0 + t + 1, len) : len; }
};

// ---- few rows (decode): 32-key tiles streamed by each warp from a TMA ring of its own, the
// rows' fragments in registers.  HBM-bound: the keys are read once and nothing else is large (8 sequences x 4097
// columns x 4 heads x 128, 34 MB: 10.5 us, launch included; tiles shared by the whole CTA took 13.7).
// Warps take contiguous runs of the tiles of all (sequence, KV head) pairs.
constexpr int kWsWarps = 8, kWsStages = 3;
template <int HD, int NM>
__global__ void __launch_bounds__(32 * kWsWarps) k_weights_stream(const __grid_constant__ CUtensorMap km, const WeightsArgs a) {
  constexpr int STAGE = kPxTile * HD * 2;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kWsWarps][kWsStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kWsWarps * kWsStages; ++i) mbar_init(smem_u32(&full[0][0] + i), 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int tiles = (a.S + kPxTile - 1) / kPxTile;
  const long long units = static_cast<long long>(a.B) * a.Hkv * tiles;
  const long long w = static_cast<long long>(blockIdx.x) * kWsWarps + warp, nw = static_cast<long long>(gridDim.x) * kWsWarps;
  const long long u0 = w * units / nw, u1 = (w + 1) * units / nw;
  uint8_t* wring = ring + warp * kWsStages * STAGE;
  auto issue = [&](long long u) {
    const int st = static_cast<int>((u - u0) % kWsStages), pair = static_cast<int>(u / tiles);
    const uint32_t dst = smem_u32(wring + st * STAGE), bar = smem_u32(&full[warp][st]);
    mbar_arrive_expect_tx(bar, STAGE);
    tma_load_5d(dst, &km, bar, 0, static_cast<int>(u % tiles) * kPxTile, 0, pair % a.Hkv, pair / a.Hkv);
  };
  long long last = u0 - 1;   // the last tile requested (lane 0)
  if (lane == 0)
    for (; last + 1 < u1 && last + 1 < u0 + kWsStages; ++last) issue(last + 1);
  int pair_at = -1;
  uint32_t qf[NM][HD / 16][4];
  float lse2[NM][2];
  int lim[NM][2], lim_max = 0;
  bool ok = true;
  for (long long u = u0; u < u1; ++u) {
    const int pair = static_cast<int>(u / tiles), b = pair / a.Hkv, g = pair % a.Hkv;
    const int col0 = static_cast<int>(u % tiles) * kPxTile;
    const long long at = static_cast<long long>(pair) * a.S + col0 + (lane >> 3) * 8 + 2 * (lane & 3) + ((lane >> 2) & 1);
    const bool inside = at < static_cast<long long>(pair + 1) * a.S;
    const float old = inside ? a.acc[at] : 0.f;
    if (pair != pair_at) {
      // the rows of this (sequence, KV head): row r is query r / G, head g G + r % G
      pair_at = pair;
      const Seen see(a, b);
      lim_max = 0;
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = i * 16 + e * 8 + (lane >> 2), t = r / a.G, h = g * a.G + r % a.G;
          const bool valid = t < see.ql;
          const float l = valid ? a.lse[(static_cast<long long>(b) * a.Tq + t) * a.H + h] : -INFINITY;
          lse2[i][e] = l * kLog2e;
          lim[i][e] = l == -INFINITY ? 0 : see.limit(t);
          lim_max = max(lim_max, lim[i][e]);
          const uint16_t* q = a.q + b * a.q_sb + t * a.q_st + h * a.q_sh + 2 * (lane & 3);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            qf[i][k][e] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
            qf[i][k][2 + e] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
          }
        }
      lim_max = __reduce_max_sync(0xffffffffu, lim_max);
    }
    const int st = static_cast<int>((u - u0) % kWsStages);
    ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[warp][st]), static_cast<int>((u - u0) / kWsStages) & 1,
                                                 nullptr));
    float sum[4][2] = {};   // columns 8n + 2(lane%4) + {0, 1}
    if (col0 < lim_max) {
      const uint32_t Kt = smem_u32(wring + st * STAGE);
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        float s[4][4] = {};
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          uint32_t kf[4];
#pragma unroll
          for (int n2 = 0; n2 < 2; ++n2) {
            ldsm_x4(Kt + sw_off(kPxTile, n2 * 16 + (lane & 7) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1)), kf);
            mma_bf16_16816(s[n2 * 2], qf[i][k], kf[0], kf[1]);
            mma_bf16_16816(s[n2 * 2 + 1], qf[i][k], kf[2], kf[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int left = lim[i][e >> 1] - (col0 + 2 * (lane & 3) + (e & 1));
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float p = exp2f(fmaf(s[n][e], a.scale2, -lse2[i][e >> 1]));
            sum[n][e & 1] += n * 8 < left ? p : 0.f;
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0 && ok && u + kWsStages < u1) {
      issue(u + kWsStages);
      last = u + kWsStages;
    }
    // over the 8 row groups; then lane l writes column (l >> 3) * 8 + 2 (l & 3) + ((l >> 2) & 1)
    float mine = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = sum[n][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if ((lane >> 2) == n * 2 + e) mine = v;
      }
    if (inside) a.out[at] = old + (ok ? mine : NAN);
    __syncwarp();
  }
  if (!ok && lane == 0)   // a tile never arrived: let the copies in flight land (bounded) before the warp ends
    each_in_flight(last + 1 - u0, kWsStages,
                   [&](int slot, int parity) { mbar_wait(smem_u32(&full[warp][slot]), parity, nullptr); });
}

// ---- many rows: S^T = K Q^T on tcgen05, blocks of 256 keys (two products of 128) x 128 rows, so that a
// thread owns a key and its sum needs no exchange.  Persistent: the (sequence, KV head, 256 keys,
// row block) units, in this order, are divided evenly over the CTAs; a CTA's part of a
// tile's sums is partial (CTA + tile).  One TMA thread, one MMA warp, four warpgroups (all 256 keys x
// a quarter of a block's rows each; two TMEM buffers, so that the next block's products run under
// this one's exponentials).  Bound by the exponentials, 16 a clock and SM, with shared memory
// (the products' operands) close behind.  512 queries of 16 heads x 16384 columns of 4 KV heads x 128, causal: 52 us,
// of which the exponentials alone would take 30 and the products 21; warpgroups that take alternate
// blocks 54, or half the rows of a key 57, mma.sync warp tiles 206.  18 warps leave 96 registers a thread, beside
// two score tiles of 32: 116 bytes are spilled (264 read back).
// Of 8 pairs of exponentials, those formed on the FMA pipe: 0 / 1 / 2 / 3 of them take, us, there 54 / 51 / 50 / 52, with heads of
// 64 53 / 50 / 50 / 52, 4 x 128 queries of 32/8 heads x 8192 columns 74 / 71 / 71 / 72 (64: 71 / 69 / 70 / 70), 8 x 40
// queries x 30000 columns 87 / 86 / 86 / 85.
constexpr int kWtPoly = 1;
constexpr int kWtCols = 256, kWtRows = 128, kWtThreads = 576;
constexpr int kWtStaged = 24;   // row blocks whose lse are in shared memory at once
template <int HD>
struct WtSmem {
  static constexpr int kBox = 128 * 128, kTile = (HD / 64) * kBox;   // 128 rows
  static constexpr int kQSlots = HD == 128 ? 2 : 4;      // and two slots of 256 keys
  static constexpr int kBytes = 1024 + (4 + kQSlots) * kTile;
};
struct WtPlan {
  int tiles_s, nb, ctas;   // key tiles per (sequence, KV head), row blocks of nt queries, CTAs
  long long units;
  __host__ __device__ WtPlan(int B, int Hkv, int S, int Tq, int nt, int max_ctas) {
    tiles_s = (S + kWtCols - 1) / kWtCols;
    nb = (Tq + nt - 1) / nt;
    units = static_cast<long long>(B) * Hkv * tiles_s * nb;
    ctas = static_cast<int>(units < max_ctas ? units : max_ctas);
  }
  __host__ __device__ long long begin(int c) const { return c * units / ctas; }
  __host__ __device__ int cta_of(long long u) const { return static_cast<int>(((u + 1) * ctas - 1) / units); }
};

template <int HD>
__global__ void __launch_bounds__(kWtThreads, 1)
    k_weights_tc(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap qm, const WeightsArgs a) {
  using C = WtSmem<HD>;
  constexpr int NB = HD / 64, QS = C::kQSlots;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* ksm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qsm = ksm + 4 * C::kTile;
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], q_full[QS], q_empty[QS], d_full[2], d_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float lse_s[kWtStaged][kWtRows];   // of the segment's next blocks: -lse log2(e), or -inf
  __shared__ uint8_t none_s[kWtStaged][4];                    // some row of the block's quarter adds nothing
  __shared__ float join[4][kWtCols];
  __shared__ volatile int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < QS; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), 1);
      mbar_init(smem_u32(&d_full[i]), 1);
      mbar_init(smem_u32(&d_empty[i]), 512);
    }
    fence_mbar_init();
    bad = 0;
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = tmem_slot;
  const WtPlan plan(a.B, a.Hkv, a.S, a.Tq, a.nt, a.ctas);
  const long long u0 = plan.begin(blockIdx.x), u1 = plan.begin(blockIdx.x + 1);
  // a segment: one key tile of the CTA's range, and the row blocks [first, first + count) of it that see any of its columns
  struct Segment {
    int b, g, col0, first, count;
    long long tile;
  };
  auto segment = [&](long long u) {
    Segment x;
    x.tile = u / plan.nb;
    const int pair = static_cast<int>(x.tile / plan.tiles_s);
    x.b = pair / a.Hkv;
    x.g = pair % a.Hkv;
    x.col0 = static_cast<int>(x.tile % plan.tiles_s) * kWtCols;
    const Seen see(a, x.b);
    int lo = static_cast<int>(u % plan.nb), hi = static_cast<int>(min(static_cast<long long>(plan.nb), lo + (u1 - u)));
    hi = x.col0 < see.len ? min(hi, (see.ql + a.nt - 1) / a.nt) : 0;   // queries there are
    if (see.causal) lo = max(lo, max(0, x.col0 - see.j0) / a.nt);      // queries that see column col0
    x.first = lo;
    x.count = max(0, hi - lo);
    return x;
  };
  if (warp < 16) {
    // ================= a warpgroup: a quarter of the rows of every block, keys `key` and 128 + key a thread ====
    // (two keys a thread: a row's lse is then read from shared memory, whose bandwidth the products'
    // operands need too, once for both)
    const int wg = warp >> 2, key = (warp & 3) * 32 + lane;
    const uint32_t td = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 32;
    const uint64_t sc2 = f2_pack(a.scale2, a.scale2);
    int seen = 0;             // blocks of the CTA so far
    bool ok = true;
    for (long long u = u0; u < u1; u += plan.nb - u % plan.nb) {
      const Segment sg = segment(u);
      const Seen see(a, sg.b);
      float sum[2] = {0.f, 0.f};
      uint64_t sum2[2][2] = {{0, 0}, {0, 0}};
      for (int n = 0; n < sg.count; ++n) {
        const int tb = (sg.first + n) * a.nt, blk = seen + n;    // the block's first query; its number in the CTA
        if (n % kWtStaged == 0) {
          // the next blocks' lse: a warp's 32 consecutive rows at a time
          asm volatile("bar.sync 5, 512;" ::: "memory");         // (the last ones have been read)
          const int todo = min(kWtStaged, sg.count - n) * 4;
          for (int x0 = warp; x0 < todo; x0 += 64) {
            float l[4];                                          // four in flight
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int x = x0 + v * 16, row = (x & 3) * 32 + lane, row_t = row / a.G, t = tb + (x >> 2) * a.nt + row_t;
              l[v] = x < todo && row_t < a.nt && t < see.ql
                         ? a.lse[(static_cast<long long>(sg.b) * a.Tq + t) * a.H + sg.g * a.G + row - row_t * a.G]
                         : -INFINITY;
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int x = x0 + v * 16;
              if (x >= todo) break;
              lse_s[x >> 2][(x & 3) * 32 + lane] = l[v] == -INFINITY ? -INFINITY : -l[v] * kLog2e;
              const bool none = __any_sync(0xffffffffu, l[v] == -INFINITY);
              if (lane == 0) none_s[x >> 2][x & 3] = none;
            }
          }
          asm volatile("bar.sync 5, 512;" ::: "memory");
        }
        const float* lse_b = &lse_s[n % kWtStaged][wg * 32];
        // rows that add nothing, or columns that the block's first queries do not see: each weight is looked at
        const bool edge = none_s[n % kWtStaged][wg] || (see.causal && see.limit(tb) < min(sg.col0 + kWtCols, see.len));
        // (after a wait that ran out the loop goes on without waiting, so that the barriers above still meet)
        const int par = blk & 1;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&d_full[par]), (blk >> 1) & 1, nullptr));
        if (!ok) continue;
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(td + par * 256, r[0]);
        tmem_ld32(td + par * 256 + 128, r[1]);
        tc_wait_ld();
        tc_fence_before();
        mbar_arrive(smem_u32(&d_empty[par]));       // in registers: the buffer is free
        if (!edge) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(&lse_b[e]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t l2 = h ? f2_pack(l4.z, l4.w) : f2_pack(l4.x, l4.y);
#pragma unroll
              for (int kt = 0; kt < 2; ++kt) {
                const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(r[kt][e + 2 * h]), __uint_as_float(r[kt][e + 2 * h + 1])), sc2, l2);
                if ((e / 2 + h) % 8 < kWtPoly) {   // part of the exponentials on the FMA pipe
                  sum2[kt][h] = f2_add(sum2[kt][h], exp2_poly2(y2));
                } else {
                  float p0, p1;
                  f2_unpack(y2, p0, p1);
                  sum2[kt][h] = f2_add(sum2[kt][h], f2_pack(ex2_approx(p0), ex2_approx(p1)));
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            // the first of these rows (query) that sees this key
            const int r_min = (see.causal ? max(0, sg.col0 + kt * 128 + key - see.j0 - tb) * a.G : 0) - wg * 32;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float l2 = lse_b[e];
              const float p = ex2_approx(fmaf(__uint_as_float(r[kt][e]), a.scale2, l2));
              sum[kt] += e >= r_min && l2 != -INFINITY ? p : 0.f;
            }
          }
        }
      }
      seen += sg.count;
      if (!ok) bad = 1;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        float total, odd;
        f2_unpack(f2_add(sum2[kt][0], sum2[kt][1]), total, odd);
        total = (total + odd) + sum[kt];
        join[wg][kt * 128 + key] = sg.col0 + kt * 128 + key < see.len ? total : 0.f;   // (past the sequence: nobody sees it)
      }
      asm volatile("bar.sync 5, 512;" ::: "memory");
      if (tid < kWtCols)
        a.part[(blockIdx.x + sg.tile) * kWtCols + tid] = bad ? NAN : (join[0][tid] + join[1][tid]) + (join[2][tid] + join[3][tid]);
      asm volatile("bar.sync 5, 512;" ::: "memory");   // join read
    }
  } else if (warp == 16) {
    // ================= MMA warp (one elected lane issues) =================
    constexpr uint32_t idesc = umma_idesc_bf16(128, 128);
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase & 1, nullptr)) != 0;
    };
    const uint64_t k_desc = umma_desc_sw128(smem_u32(ksm)), q_desc = umma_desc_sw128(smem_u32(qsm));
    int blocks = 0, segs = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1; u += plan.nb - u % plan.nb) {
      const Segment sg = segment(u);
      if (sg.count == 0) continue;
      const int ks = segs & 1;
      ok = wait(&k_full[ks], segs++ >> 1);
      for (int n = 0; ok && n < sg.count; ++n, ++blocks) {
        const int st = blocks % QS, par = blocks & 1, use = blocks >> 1;
        ok = wait(&q_full[st], blocks / QS) && (use == 0 || wait(&d_empty[par], use - 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              tc_mma_bf16(tmem + par * 256 + kt * 128, k_desc + (ks * 2 + kt) * (C::kTile >> 4) + (k >> 2) * (C::kBox >> 4) + (k & 3) * 2,
                          q_desc + st * (C::kTile >> 4) + (k >> 2) * (C::kBox >> 4) + (k & 3) * 2, idesc, k > 0);
          tc_commit(smem_u32(&d_full[par]));
          tc_commit(smem_u32(&q_empty[st]));
          if (n + 1 == sg.count) tc_commit(smem_u32(&k_empty[ks]));
        }
        __syncwarp();
      }
    }
    if (!ok) bad = 1;
  } else if (tid == 17 * 32) {
    // ================= TMA thread =================
    int blocks = 0, segs = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1; u += plan.nb - u % plan.nb) {
      const Segment sg = segment(u);
      if (sg.count == 0) continue;
      const int ks = segs & 1;
      ok = segs < 2 || mbar_wait(smem_u32(&k_empty[ks]), ((segs >> 1) - 1) & 1, nullptr);
      if (!ok) break;
      ++segs;
      mbar_arrive_expect_tx(smem_u32(&k_full[ks]), 2 * C::kTile);
      for (int i = 0; i < 2; ++i)   // (keys past the tensor's last read as zero)
        tma_load_5d(smem_u32(ksm) + (ks * 2 + i) * C::kTile, &km, smem_u32(&k_full[ks]), 0, sg.col0 + i * 128, 0, sg.g, sg.b);
      for (int n = 0; n < sg.count; ++n) {
        const int st = blocks % QS;
        ok = blocks < QS || mbar_wait(smem_u32(&q_empty[st]), (blocks / QS - 1) & 1, nullptr);
        if (!ok) break;
        ++blocks;
        mbar_arrive_expect_tx(smem_u32(&q_full[st]), a.nt * a.G * HD * 2);
        // rows in the order (query, head of the group); queries past the tensor's last read as zero
        for (int bx = 0; bx < NB; ++bx)
          tma_load_4d(smem_u32(qsm) + st * C::kTile + bx * C::kBox, &qm, smem_u32(&q_full[st]), bx * 64, sg.g * a.G,
                      (sg.first + n) * a.nt, sg.b);
      }
    }
    if (!ok) {   // the products stopped: let the copies in flight land (bounded) before the block can end
      bad = 1;
      each_in_flight(segs, 2, [&](int slot, int parity) { mbar_wait(smem_u32(&k_full[slot]), parity, nullptr); });
      each_in_flight(blocks, QS, [&](int slot, int parity) { mbar_wait(smem_u32(&q_full[slot]), parity, nullptr); });
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// the parts of each key tile, in order, added to acc
__global__ void __launch_bounds__(256) k_weights_add(const WeightsArgs a) {
  const WtPlan plan(a.B, a.Hkv, a.S, a.Tq, a.nt, a.ctas);
  const long long tile = blockIdx.x;
  const int pair = static_cast<int>(tile / plan.tiles_s), j = static_cast<int>(tile % plan.tiles_s) * kWtCols + threadIdx.x;
  const int c0 = plan.cta_of(tile * plan.nb), c1 = plan.cta_of((tile + 1) * plan.nb - 1);
  if (j >= a.S) return;
  const long long at = static_cast<long long>(pair) * a.S + j;
  const float acc = a.acc[at];
  pdl_wait();
  float s = 0.f;
  for (int c = c0; c <= c1; ++c) s += __ldcg(&a.part[(c + tile) * kWtCols + threadIdx.x]);
  a.out[at] = acc + s;
}

// ---------------------------------------------------------------- host side
// A CTA per row up to four rows per SM (latency: the splits are spread over the CTA), else a row per group: with 4096 +
// 257 columns, a CTA per row against a row per group, whole calls in us: 128 rows 12.4 / 13.8, 512 17.3 / 17.8,
// 768 22.7 / 20.5, 2048 45.0 / 40.2.
template <int HD>
cudaError_t run_merge(bool q32, const PrefixArgs& a, bool pdl, cudaStream_t s) {
  constexpr int NG = 128 / (HD / 4);
  const unsigned rows = static_cast<unsigned>(a.rows);
  if (a.rows <= 4 * kNumSM)
    return q32 ? launch_k(pdl, k_prefix_merge<HD, true, true>, dim3(rows), dim3(128), 0, s, a)
               : launch_k(pdl, k_prefix_merge<HD, false, true>, dim3(rows), dim3(128), 0, s, a);
  return q32 ? launch_k(pdl, k_prefix_merge<HD, true, false>, dim3((rows + NG - 1) / NG), dim3(128), 0, s, a)
             : launch_k(pdl, k_prefix_merge<HD, false, false>, dim3((rows + NG - 1) / NG), dim3(128), 0, s, a);
}

// Rows per CTA and column splits of both parts.  About two CTAs per SM in all,
// none shorter than 256 columns: a shorter split costs more in partial results
// (hd + 2 floats per row) than its keys and values cost to read.
struct PrefixPlan {
  int nm;
  int rb_p, n_p, rb_s, n_s;
  int tc_ctas;         // > 0: the prefix on the 5th-generation tensor cores
  size_t rows, tc_parts;
  size_t off_ml, off_tc_o, off_tc_ml, bytes;
};
// The prefix goes to the 5th-generation tensor cores when its rows take two blocks of warp tiles (which then read
// every column twice) and there is enough of it for their 16 us of start and end: blocks x columns x KV heads x
// head_dim.  Whole calls with 8 heads x 128, tensor cores against warp tiles, us: 36 rows x 1024 columns 16.3 / 12.3,
// x 4096 19.5 / 15.3, x 32768 38.8 / 42.6; 64 rows x 512 16.5 / 12.8, x 4096 20.3 / 19.3, x 32768
// 40.0 / 46.7; 128 rows x 4096 22.4 / 25.8; and of one block, 32 rows x 4096 19.3 / 13.4, x 32768 38.7 / 37.8.
constexpr int kTcMinRows = 33;
constexpr double kTcMinWork = 1.2e7;
PrefixPlan plan_prefix(int B, int Tq, int H, int Hkv, int hd, int P, int S, bool warp_tiles) {
  PrefixPlan p{};
  const int G = H / Hkv;
  const long long rows_p = static_cast<long long>(B) * Tq * G, rows_s = static_cast<long long>(Tq) * G;
  if (!warp_tiles && P >= kTcTile && rows_p >= kTcMinRows &&
      static_cast<double>(ceil_div_i(rows_p, 32)) * P * Hkv * hd >= kTcMinWork) {
    const long long pairs = static_cast<long long>(Hkv) * ceil_div_i(rows_p, kTcRows);
    p.tc_ctas = static_cast<int>(std::min<long long>(kNumSM, std::max(1LL, pairs * ceil_div_i(P, kTcTile) / kTcMinTiles)));
    p.tc_parts = static_cast<size_t>(p.tc_ctas + pairs);
    P = 0;   // nothing of it is left for the warp tiles
  }
  p.nm = (P > 0 && rows_p > 16) || rows_s > 16 ? 2 : 1;
  const int RB = 16 * p.nm;
  p.rb_p = ceil_div_i(rows_p, RB);
  p.rb_s = ceil_div_i(rows_s, RB);
  const double cols = static_cast<double>(p.rb_p) * Hkv * P + static_cast<double>(p.rb_s) * Hkv * B * S;
  const double per = std::max(256.0, cols / (2.0 * kNumSM));
  auto splits = [&](int n) { return n ? std::min(64, std::max(1, static_cast<int>(n / per + 0.5))) : 0; };
  p.n_p = splits(P);
  p.n_s = splits(S);
  p.rows = static_cast<size_t>(B) * Tq * H;
  const size_t n = p.n_p + p.n_s;
  p.off_ml = align256_sz(n * p.rows * hd * 4);
  p.off_tc_o = p.off_ml + align256_sz(n * p.rows * 8);
  p.off_tc_ml = p.off_tc_o + align256_sz(p.tc_parts * kTcRows * hd * 4);
  p.bytes = p.off_tc_ml + align256_sz(p.tc_parts * kTcRows * 8) + 256;
  return p;
}

size_t split_smem(int hd, int nm, bool hilo) { return 1024 + kPxRing + static_cast<size_t>(16 * nm) * hd * 2 * (hilo ? 2 : 1); }

template <int HD, int NM, bool HILO>
cudaError_t run_split(const CUtensorMap* m, const PrefixArgs& a, int grid, bool pdl, cudaStream_t s) {
  return launch_k(pdl, k_prefix_split<HD, NM, HILO>, dim3(grid), dim3(128), split_smem(HD, NM, HILO), s, m[0], m[1],
                  m[2], m[3], a);
}
template <int HD>
cudaError_t run_split_hd(int nm, bool hilo, const CUtensorMap* m, const PrefixArgs& a, int grid, bool pdl,
                         cudaStream_t s) {
  if (nm == 1)
    return hilo ? run_split<HD, 1, true>(m, a, grid, pdl, s) : run_split<HD, 1, false>(m, a, grid, pdl, s);
  return hilo ? run_split<HD, 2, true>(m, a, grid, pdl, s) : run_split<HD, 2, false>(m, a, grid, pdl, s);
}

// A row block per warp when the CTAs of a block each would take more than one wave and no split is long (a chain of up
// to eight tiles per warp, half of that for half the blocks).  Whole calls, a block per warp against one per
// CTA, us: 117 x 6 queries of 64/8 heads x 128, 2 + 8 columns 70 / 114; 128 x 1, 32/8 heads, 100 + 200 columns 28 / 41; 49 x 7,
// 64/8 heads x 64, 103 + 20 columns 22 / 35; but 64 x 1, 32/8 heads, 8192 + 250 columns 47 / 45, and 32 x 3, 320 + 43 25 / 16.
constexpr int kRowsMaxCols = 256;
template <int HD>
cudaError_t run_rows(int nm, const CUtensorMap* m, const PrefixArgs& a, int items, bool pdl, cudaStream_t s) {
  const dim3 grid((items + kPxWarps - 1) / kPxWarps);
  return nm == 1 ? launch_k(pdl, k_prefix_rows<HD, 1>, grid, dim3(128), 1024 + kPxRing, s, m[0], m[1], m[2], m[3], a, items)
                 : launch_k(pdl, k_prefix_rows<HD, 2>, grid, dim3(128), 1024 + kPxRing, s, m[0], m[1], m[2], m[3], a, items);
}

size_t stream_smem(int hd) { return 1024 + static_cast<size_t>(kWsWarps) * kWsStages * kPxTile * hd * 2; }

// Column weights on tcgen05 when a (sequence, KV head) has more rows than two warp tiles hold (tensor cores
// against warp tiles: 32 rows, 8 x 4096 columns x 4 heads 23.4 / 15.7 us, 65536 columns 37.8 / 22.9).
constexpr int kStreamRows = 32;
struct WeightsPlan {
  bool tc;
  int nt;
  long long tiles;
  size_t bytes;
};
WeightsPlan plan_weights(int B, int Tq, int H, int Hkv, int S) {
  WeightsPlan p{};
  const int G = H / Hkv;
  p.tc = static_cast<long long>(Tq) * G > kStreamRows;
  p.bytes = 256;
  if (!p.tc) return p;
  p.nt = std::min(kWtRows / G, 256);
  p.tiles = static_cast<long long>(B) * Hkv * ceil_div_i(S, kWtCols);
  p.bytes += static_cast<size_t>(p.tiles + kNumSM) * kWtCols * 4;
  return p;
}

}  // namespace

cudaError_t serving_init_attrs() {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  auto set = [&](auto* kern, size_t bytes) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) e = r;
  };
  set(k_prefix_split<64, 1, false>, split_smem(64, 1, false));
  set(k_prefix_split<64, 1, true>, split_smem(64, 1, true));
  set(k_prefix_split<64, 2, false>, split_smem(64, 2, false));
  set(k_prefix_split<64, 2, true>, split_smem(64, 2, true));
  set(k_prefix_split<128, 1, false>, split_smem(128, 1, false));
  set(k_prefix_split<128, 1, true>, split_smem(128, 1, true));
  set(k_prefix_split<128, 2, false>, split_smem(128, 2, false));
  set(k_prefix_split<128, 2, true>, split_smem(128, 2, true));
  set(k_prefix_rows<64, 1>, 1024 + kPxRing);
  set(k_prefix_rows<64, 2>, 1024 + kPxRing);
  set(k_prefix_rows<128, 1>, 1024 + kPxRing);
  set(k_prefix_rows<128, 2>, 1024 + kPxRing);
  set(k_prefix_tc<64>, TcSmem<64>::kBytes);
  set(k_prefix_tc<128>, TcSmem<128>::kBytes);
  set(k_weights_stream<64, 1>, stream_smem(64));
  set(k_weights_stream<64, 2>, stream_smem(64));
  set(k_weights_stream<128, 1>, stream_smem(128));
  set(k_weights_stream<128, 2>, stream_smem(128));
  set(k_weights_tc<64>, WtSmem<64>::kBytes);
  set(k_weights_tc<128>, WtSmem<128>::kBytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

size_t prefix_scratch_bytes(int B, int Tq, int H, int Hkv, int hd, int P, int S, bool fp32_queries) {
  // either of the prefix's kernels (the scale, known at the call, has a say)
  const size_t warp = plan_prefix(B, Tq, H, Hkv, hd, P, S, true).bytes;
  return fp32_queries ? warp : std::max(warp, plan_prefix(B, Tq, H, Hkv, hd, P, S, false).bytes);
}

cudaError_t launch_prefix(const PrefixLaunch& L, void* scratch, cudaStream_t s) {
  const flashloop_prefix_args& c = L.a;
  cudaError_t e = serving_init_attrs();
  if (e != cudaSuccess) return e;
  PrefixArgs a{};
  a.scale2 = c.scale * kLog2e;   // 0: k_prefix_tc masks by scores of -inf, which 0 would turn to NaN
  const PrefixPlan p = plan_prefix(c.B, c.Tq, c.H, c.Hkv, c.hd, c.P, c.S, L.q32 != nullptr || a.scale2 == 0.f);
  a.q = c.q; a.q32 = L.q32; a.q_sb = c.q_stride[0]; a.q_st = c.q_stride[1]; a.q_sh = c.q_stride[2];
  a.out = c.out; a.o_sb = c.out_stride[0]; a.o_st = c.out_stride[1]; a.o_sh = c.out_stride[2];
  a.out32 = L.out32; a.lse = c.lse; a.k = c.k; a.v = c.v;
  a.k_sb = c.k_stride[0]; a.k_sg = c.k_stride[1]; a.k_sr = c.k_stride[2];
  a.v_sb = c.v_stride[0]; a.v_sg = c.v_stride[1]; a.v_sr = c.v_stride[2];
  a.lens = c.lens; a.q_lens = c.q_lens; a.lens_add = L.lens_add; a.status = L.status;
  a.B = c.B; a.Tq = c.Tq; a.H = c.H; a.Hkv = c.Hkv; a.G = c.H / c.Hkv; a.P = c.P; a.S = c.S;
  a.rb_p = p.rb_p; a.n_p = p.n_p; a.rb_s = p.rb_s; a.n_s = p.n_s;
  a.items_p = p.rb_p * p.n_p * c.Hkv;
  a.rows = static_cast<long long>(p.rows);
  uint8_t* ws = static_cast<uint8_t*>(scratch);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
  a.tc_ctas = p.tc_ctas;
  a.tc_o = reinterpret_cast<float*>(ws + p.off_tc_o);
  a.tc_ml = reinterpret_cast<float2*>(ws + p.off_tc_ml);
  CUtensorMap m[4] = {};
  const uint32_t box = p.tc_ctas ? kTcTile : kPxTile;
  if (c.P > 0) {
    if (!encode_tmap_rows(&m[0], c.k_prefix, c.hd, c.P, c.Hkv, 1, c.kp_stride[1], c.kp_stride[0], 0, box) ||
        !encode_tmap_rows(&m[1], c.v_prefix, c.hd, c.P, c.Hkv, 1, c.vp_stride[1], c.vp_stride[0], 0, box))
      return cudaErrorInvalidValue;
  }
  if (c.S > 0) {
    if (!encode_tmap_rows(&m[2], c.k, c.hd, c.S, c.Hkv, c.B, c.k_stride[2], c.k_stride[1], c.k_stride[0], kPxTile) ||
        !encode_tmap_rows(&m[3], c.v, c.hd, c.S, c.Hkv, c.B, c.v_stride[2], c.v_stride[1], c.v_stride[0], kPxTile))
      return cudaErrorInvalidValue;
  }
  if (c.P == 0) m[0] = m[2], m[1] = m[3];
  if (c.S == 0) m[2] = m[0], m[3] = m[1];
  const long long grid = a.items_p + static_cast<long long>(p.rb_s) * p.n_s * c.Hkv * c.B;
  bool pdl = L.pdl;
  if (p.tc_ctas) {
    const int smem = c.hd == 128 ? TcSmem<128>::kBytes : TcSmem<64>::kBytes;
    e = c.hd == 128 ? launch_k(pdl, k_prefix_tc<128>, dim3(p.tc_ctas), dim3(kTcThreads), smem, s, m[0], m[1], a)
                    : launch_k(pdl, k_prefix_tc<64>, dim3(p.tc_ctas), dim3(kTcThreads), smem, s, m[0], m[1], a);
    if (e != cudaSuccess) return e;
    pdl = true;
  }
  if (grid > 0) {
    const int cols = std::max(p.n_p ? ceil_div_i(c.P, p.n_p) : 0, p.n_s ? ceil_div_i(c.S, p.n_s) : 0);   // of a split
    if (!L.q32 && grid > 2 * kNumSM && cols <= std::min<long long>(kRowsMaxCols, grid / 4))
      e = c.hd == 128 ? run_rows<128>(p.nm, m, a, static_cast<int>(grid), pdl, s)
                      : run_rows<64>(p.nm, m, a, static_cast<int>(grid), pdl, s);
    else
      e = c.hd == 128 ? run_split_hd<128>(p.nm, L.q32 != nullptr, m, a, static_cast<int>(grid), pdl, s)
                      : run_split_hd<64>(p.nm, L.q32 != nullptr, m, a, static_cast<int>(grid), pdl, s);
    if (e != cudaSuccess) return e;
    pdl = true;
  }
  return c.hd == 128 ? run_merge<128>(L.q32 != nullptr, a, pdl, s) : run_merge<64>(L.q32 != nullptr, a, pdl, s);
}

}  // namespace fl

using namespace fl;

namespace {
// Head shapes that the attention operators take.
constexpr int kMaxCols = 1 << 30;   // columns of a prefix or a sequence (tile ends are held in 32 bits)
bool heads_ok(int B, int Tq, int H, int Hkv, int hd) {
  return B >= 1 && Tq >= 1 && H >= 1 && Hkv >= 1 && H % Hkv == 0 && H / Hkv <= kMaxGroup && (hd == 64 || hd == 128) &&
         Hkv <= 65535 && B <= 65535 && static_cast<long long>(B) * Tq * H <= (1LL << 30);
}
}  // namespace

extern "C" {

size_t flashloop_prefix_attention_scratch_bytes(int B, int Tq, int H, int Hkv, int hd, int P, int S) {
  if (!heads_ok(B, Tq, H, Hkv, hd) || Tq > kMaxTq || P < 0 || S < 0 || P > kMaxCols || S > kMaxCols) return 0;
  return prefix_scratch_bytes(B, Tq, H, Hkv, hd, P, S, false);
}

fl_status flashloop_prefix_attention(const flashloop_prefix_args* a, void* scratch, size_t scratch_bytes,
                                     fl_stream_t stream) {
  if (!a) return refuse(FL_ERR_INVALID_ARG, "NULL arguments");
  if (!heads_ok(a->B, a->Tq, a->H, a->Hkv, a->hd) || a->Tq > kMaxTq || a->P < 0 || a->S < 0 || a->P > kMaxCols || a->S > kMaxCols)
    return refuse(FL_ERR_INVALID_ARG, "B, Tq (<= 64), H, Hkv (H % Hkv == 0, H / Hkv <= 64), hd (64 or 128), P or S out of range");
  if (!std::isfinite(a->scale)) return refuse(FL_ERR_INVALID_ARG, "scale must be finite");
  if (!a->q || !a->out || !is_aligned(a->q, 16) || !is_aligned(a->out, 16) || !is_aligned(a->lse, 4) ||
      !is_aligned(a->q_lens, 4))
    return refuse(FL_ERR_INVALID_ARG, "q and out must be non-NULL and 16-byte aligned, lse and q_lens 4-byte aligned");
  if (a->P > 0 && (!a->k_prefix || !a->v_prefix || !is_aligned(a->k_prefix, 16) || !is_aligned(a->v_prefix, 16)))
    return refuse(FL_ERR_INVALID_ARG, "k_prefix and v_prefix must be non-NULL and 16-byte aligned when P > 0");
  if (a->S > 0 && (!a->k || !a->v || !a->lens || !is_aligned(a->k, 16) || !is_aligned(a->v, 16) || !is_aligned(a->lens, 4)))
    return refuse(FL_ERR_INVALID_ARG, "k, v (16-byte aligned) and lens must be non-NULL when S > 0");
  const int64_t qd[3] = {a->B, a->Tq, a->H}, kd[3] = {a->B, a->Hkv, a->S}, pd[2] = {a->Hkv, a->P};
  for (int i = 0; i < 3; ++i) {
    if (!stride_ok(a->q_stride[i], qd[i], 8) || !stride_ok(a->out_stride[i], qd[i], 8))
      return refuse(FL_ERR_INVALID_ARG, "q and out strides must be positive multiples of 8");
    if (a->S > 0 && (!stride_ok(a->k_stride[i], kd[i], 8) || !stride_ok(a->v_stride[i], kd[i], 8)))
      return refuse(FL_ERR_INVALID_ARG, "k and v strides must be positive multiples of 8");
    if (i < 2 && a->P > 0 && (!stride_ok(a->kp_stride[i], pd[i], 8) || !stride_ok(a->vp_stride[i], pd[i], 8)))
      return refuse(FL_ERR_INVALID_ARG, "k_prefix and v_prefix strides must be positive multiples of 8");
  }
  int64_t span = 0;   // the tensor-core kernel holds a query row's place in 32 bits of 16-byte units
  for (int i = 0; i < 3; ++i) span += qd[i] > 1 ? (qd[i] - 1) * a->q_stride[i] : 0;
  if (span >= (int64_t(1) << 34)) return refuse(FL_ERR_INVALID_ARG, "q must span less than 2^34 elements");
  const size_t need = prefix_scratch_bytes(a->B, a->Tq, a->H, a->Hkv, a->hd, a->P, a->S, false);
  if (!scratch || scratch_bytes < need || !is_aligned(scratch, 256))
    return refuse_scratch(need);
  PrefixLaunch L{};
  L.a = *a;
  return cuda_status(launch_prefix(L, scratch, reinterpret_cast<cudaStream_t>(stream)));
}

size_t flashloop_column_weights_scratch_bytes(int B, int Tq, int H, int Hkv, int hd, int S) {
  if (!heads_ok(B, Tq, H, Hkv, hd) || S < 0 || S > kMaxCols) return 0;
  return plan_weights(B, Tq, H, Hkv, S).bytes;
}

fl_status flashloop_column_weights(const flashloop_weights_args* a, void* scratch, size_t scratch_bytes,
                                   fl_stream_t stream) {
  if (!a) return refuse(FL_ERR_INVALID_ARG, "NULL arguments");
  if (!heads_ok(a->B, a->Tq, a->H, a->Hkv, a->hd) || a->S < 0 || a->S > kMaxCols)
    return refuse(FL_ERR_INVALID_ARG, "B, Tq, H, Hkv (H % Hkv == 0, H / Hkv <= 64), hd (64 or 128) or S out of range");
  if (!std::isfinite(a->scale)) return refuse(FL_ERR_INVALID_ARG, "scale must be finite");
  if (a->S == 0) return FL_OK;
  if (!a->q || !a->k || !a->lse || !a->acc || !a->out || !is_aligned(a->q, 16) || !is_aligned(a->k, 16) ||
      !is_aligned(a->lse, 4) || !is_aligned(a->acc, 4) || !is_aligned(a->out, 4) || !is_aligned(a->lens, 4) ||
      !is_aligned(a->q_lens, 4))
    return refuse(FL_ERR_INVALID_ARG, "q and k must be 16-byte aligned, lse, acc, out, lens and q_lens 4-byte aligned");
  const int64_t qd[3] = {a->B, a->Tq, a->H}, kd[3] = {a->B, a->Hkv, a->S};
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(a->q_stride[i], qd[i], 8) || !stride_ok(a->k_stride[i], kd[i], 8))
      return refuse(FL_ERR_INVALID_ARG, "q and k strides must be positive multiples of 8");
  const size_t need = flashloop_column_weights_scratch_bytes(a->B, a->Tq, a->H, a->Hkv, a->hd, a->S);
  if (!scratch || scratch_bytes < need || !is_aligned(scratch, 256))
    return refuse_scratch(need);
  cudaError_t e = serving_init_attrs();
  if (e != cudaSuccess) return cuda_status(e);
  WeightsArgs w{};
  w.q = a->q; w.q_sb = a->q_stride[0]; w.q_st = a->q_stride[1]; w.q_sh = a->q_stride[2];
  w.lse = a->lse; w.acc = a->acc; w.out = a->out; w.lens = a->lens; w.q_lens = a->lens ? a->q_lens : nullptr;
  w.B = a->B; w.Tq = a->Tq; w.H = a->H; w.Hkv = a->Hkv; w.G = a->H / a->Hkv; w.S = a->S;
  w.scale2 = a->scale * kLog2e;
  const WeightsPlan p = plan_weights(a->B, a->Tq, a->H, a->Hkv, a->S);
  CUtensorMap km, qm;
  if (!encode_tmap_rows(&km, a->k, a->hd, a->S, a->Hkv, a->B, a->k_stride[2], a->k_stride[1], a->k_stride[0],
                        p.tc ? 128 : kPxTile))
    return refuse(FL_ERR_INVALID_ARG, "tensor map encoding failed");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!p.tc) {
    const long long units = static_cast<long long>(a->B) * a->Hkv * ceil_div_i(a->S, kPxTile);
    const dim3 grid(static_cast<unsigned>(std::min<long long>(kNumSM, (units + kWsWarps - 1) / kWsWarps)));
    const int block = 32 * kWsWarps;
    const size_t sm = stream_smem(a->hd);
    if (a->Tq * w.G > 16)
      return cuda_status(a->hd == 128 ? launch_k(false, k_weights_stream<128, 2>, grid, dim3(block), sm, s, km, w)
                                      : launch_k(false, k_weights_stream<64, 2>, grid, dim3(block), sm, s, km, w));
    return cuda_status(a->hd == 128 ? launch_k(false, k_weights_stream<128, 1>, grid, dim3(block), sm, s, km, w)
                                    : launch_k(false, k_weights_stream<64, 1>, grid, dim3(block), sm, s, km, w));
  }
  // the queries as [B][Tq][H][hd] with boxes of nt queries x the group's heads
  if (!encode_tmap_queries(&qm, a->q, a->hd, a->H, a->Tq, a->B, a->q_stride[2], a->q_stride[1], a->q_stride[0], w.G, p.nt))
    return refuse(FL_ERR_INVALID_ARG, "tensor map encoding failed");
  w.nt = p.nt;
  w.ctas = kNumSM;
  w.part = static_cast<float*>(scratch);
  const dim3 grid(WtPlan(a->B, a->Hkv, a->S, a->Tq, p.nt, kNumSM).ctas);
  e = a->hd == 128 ? launch_k(false, k_weights_tc<128>, grid, dim3(kWtThreads), WtSmem<128>::kBytes, s, km, qm, w)
                   : launch_k(false, k_weights_tc<64>, grid, dim3(kWtThreads), WtSmem<64>::kBytes, s, km, qm, w);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_k(true, k_weights_add, dim3(static_cast<unsigned>(p.tiles)), dim3(256), 0, s, w));
}

}  // extern "C"
