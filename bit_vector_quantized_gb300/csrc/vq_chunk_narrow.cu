// vq_chunk_narrow.cu -- chunk attention for few query rows per (sequence, KV head) (sm_103a),
// and the merge of the chunk kernels' partials.
//
// What is computed, per query row (VecInfer, section 方法细节 "注意力机制中的向量量化KV缓存", for
// several new tokens at once):
//   q~ = q diag(lambda) H_D,  s_p = q~ . VQ^-1(K~_p) * scale over the visible p,
//   o = softmax(s) VQ^-1(V).
//
// Each warp takes every n-th 16-token block of a tile's keys and keeps its own
// online softmax (running maximum, sum and 128-wide output); the warps join at
// the end of the piece.  Both products are m16n8k16 warp mma, with centroids
// gathered from the replicated, bank-conflict-free table straight into one
// operand.  Two kernels:
//
//   * 8 rows and fewer (single decode tokens, a few drafted ones): tokens as
//     rows, scores^T [16 tok x 8] = K~ q~^T and o^T [128 x 8] += V^T p^T, the
//     form with the fewest products (16 or 24 per block) and registers (32 of
//     output), so 16 warps share an SM and hide the latency of the codes.
//     With 4 rows and fewer, columns 2h and 2h + 1 hold the high and low fp16
//     parts of q~ and of p, and both products keep about fp32 accuracy.
//   * up to 16 rows: the query rows as rows, the centroids as columns; a
//     gather of a V centroid serves four output blocks.
//
// q~ is split into high and low fp16 parts everywhere (scores keep about fp32
// accuracy); p is rounded to fp16 once where it is not split (p <= 2^8,
// relative 2^-11): a choice, which leaves the outputs off by 2.6e-4 to 2.8e-4
// against 64 bits where their own rounding is 2.1e-4.  Splitting it for 5 to 8
// rows too left 2.1e-4 and took 105 us instead of 97 in the case below.  Sums
// and maxima are fp32.
//
// What bounds them: latency at 16 warps per SM (the table takes the shared
// memory that more would need).  Nothing is full: the few-row kernel issues in
// 54 % of the cycles, the shared-memory pipe is 65 % busy, DRAM 29 %; a warp
// waits between two instructions first for the one before (1.9 cycles), then
// for a gather (1.0), for its turn (0.9), for the tensor pipe (0.7) and for the
// codes (0.5).
// Measured for one token of each of 64 sequences with a window of 4096 and 4
// sinks: 97 us for 40 heads of 8 KV heads and 100 B of codes per token (211 MB,
// 2.2 TB/s, floor 31 us), 72 us for 32 heads and 64 B.  The 16-row kernel, 3
// new tokens of each of 8 sequences of 4000 to 8000 tokens, 32 heads of 8 KV
// heads and 64 B: 42 us and a merge of 8 (25 MB, floor 3.7 us).  It has 8 warps
// and 216 registers a thread, so it is further from filling anything: issue
// 30 %, shared memory 28 %, tensor pipe 22 %, DRAM 8 %.  Groups of four warps
// with pieces of their own came together with the end of the spilled registers:
// 146 to 104 us; which of the two did how much was not taken apart.

#include "vq_chunk_common.cuh"
#include "vq_gather.cuh"

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kSlack = 8.f;    // the running maximum may lag by this much (log2 units): p <= 2^8
constexpr int kNarrowWarps = 8;  // of the 16-row kernel
constexpr int kFewWarps = 16;    // of the kernel for 8 rows and fewer
constexpr int kGroupWarps = kFewWarps / kFewGroups, kGroupThreads = kGroupWarps * 32;
constexpr int kBlock = 16;       // tokens per block
constexpr int kQStride = 132;    // halves between q~ rows in shared memory

template <int DK, int BK, int DV, int BV>
struct NarrowTable {
  static constexpr bool kWide = DK == 8;
  static constexpr int kRows = 1 << (BK > BV ? BK : BV);
  static constexpr int kBytes = kWide ? 131072 : kRows * kTabRow;
};

// Codebooks into the gather table: 256-byte rows, K centroid j 16 (or 32)
// times in bytes 0..127 and V centroid j in bytes 128..255; the 1.5-bit format
// as two plain 64 KB tables.
template <int DK, int BK, int DV, int BV>
__device__ __forceinline__ void fill_table(const ChunkParams& p) {
  using T = NarrowTable<DK, BK, DV, BV>;
  uint4* tab = reinterpret_cast<uint4*>(g_smem);
  const int tid = threadIdx.x, n = blockDim.x;
  if constexpr (T::kWide) {
    for (int i = tid; i < 4096; i += n) {
      tab[i] = __ldg(static_cast<const uint4*>(p.cb_k) + i);
      tab[4096 + i] = __ldg(static_cast<const uint4*>(p.cb_v) + i);
    }
  } else {
    for (int i = tid; i < T::kRows * 16; i += n) {
      const int row = i >> 4;
      const bool v = (i & 8) != 0;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < (v ? 1 << BV : 1 << BK)) {
        if ((v ? DV : DK) == 4) {
          const uint2 c = __ldg(static_cast<const uint2*>(v ? p.cb_v : p.cb_k) + row);
          x = make_uint4(c.x, c.y, c.x, c.y);
        } else {
          const uint32_t c = __ldg(static_cast<const uint32_t*>(v ? p.cb_v : p.cb_k) + row);
          x = make_uint4(c, c, c, c);
        }
      }
      tab[i] = x;
    }
  }
}

// Shared memory of both kernels before q~ and the join buffers.
struct NarrowWorker {
  ChunkWalk<kBlock> walk;  // its first thread's
  ChunkPiece piece[2];     // the piece under way and the next one
  int more[2];
  // piece k, into its buffer
  __device__ __forceinline__ void plan(const ChunkParams& p, int k) { more[k & 1] = walk.next(p, piece[k & 1]); }
};
struct NarrowHead {
  long long pre[kChunkMaxBatch + 1];
  long long scratch[33];
  NarrowWorker worker[kFewGroups];
};
constexpr size_t kHeadBytes = (sizeof(NarrowHead) + 15) / 16 * 16;

// Elements e of two fp16 pairs as one operand register: (a.e, b.e).
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// Row r of a tile's q~ (one warp) as high and low fp16 parts: rows r and kRows + r of qs; 0 where there is none.
template <int kRows>
__device__ __forceinline__ void query_row(const ChunkParams& p, const ChunkPiece& u, int r, bool live, __half* qs, int lane) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const int G = p.group;
    const long long row = static_cast<long long>(u.s.row0 + u.tile * p.tile_tok + r / G) * p.hq + u.kvh * G + r % G;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __half*>(p.q) + row * kHeadDim) + lane);
    const float4 lam = __ldg(reinterpret_cast<const float4*>(p.lambda + u.kvh * kHeadDim) + lane);
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    x[0] = lo.x * lam.x;
    x[1] = lo.y * lam.y;
    x[2] = hi.x * lam.z;
    x[3] = hi.y * lam.w;
    fwht128_warp(x, lane);
  }
  uint2 vh, vl;
  split_pair(x[0] * p.qscale, x[1] * p.qscale, vh.x, vl.x);
  split_pair(x[2] * p.qscale, x[3] * p.qscale, vh.y, vl.y);
  *reinterpret_cast<uint2*>(qs + r * kQStride + 4 * lane) = vh;
  *reinterpret_cast<uint2*>(qs + (kRows + r) * kQStride + 4 * lane) = vl;
}

// Row r of a piece from its warps' partials (one warp; mo [warps][rows][128], ml [warps][rows]): to
// `out`, or as one partial to the workspace.
template <int kWarps, int kRows>
__device__ __forceinline__ void join_row(const ChunkParams& p, const ChunkPiece& u, const float* mo, const float2* ml, int r,
                                         bool live, int slot_rows, int lane) {
  if (!live) return;
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + r].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float Mu = M == -INFINITY ? 0.f : M;  // a row that sees nothing: sums of 0 (or of its NaN)
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 v = ml[w * kRows + r];
    const float f = fast_exp2(v.x - Mu);
    L = fmaf(f, v.y, L);
    const float4 x = *reinterpret_cast<const float4*>(mo + (w * kRows + r) * kHeadDim + 4 * lane);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  if (u.slot >= 0) {
    const long long at = static_cast<long long>(u.slot) * slot_rows + r;
    reinterpret_cast<float4*>(p.ws_o + at * kHeadDim)[lane] = acc;
    if (lane == 0) p.ws_ml[at] = make_float2(M, L);
  } else {
    const float f = L == 0.f ? 0.f : 1.f / L;
    const long long row = static_cast<long long>(u.s.row0 + u.tile * p.tile_tok + r / p.group) * p.hq + u.kvh * p.group + r % p.group;
    const __half2 h0 = __floats2half2_rn(acc.x * f, acc.y * f), h1 = __floats2half2_rn(acc.z * f, acc.w * f);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&h0);
    w.y = *reinterpret_cast<const uint32_t*>(&h1);
    reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + row * kHeadDim)[lane] = w;
  }
}

// ---- up to 16 rows: the query rows as the rows of the products --------------------------------
template <int DK, int BK, int DV, int BV>
__global__ void __launch_bounds__(kNarrowWarps * 32, 1) vq_chunk_narrow_kernel(const ChunkParams p) {
  using T = NarrowTable<DK, BK, DV, BV>;
  constexpr int kRows = 16;
  constexpr bool kWide = T::kWide;
  constexpr int KROW = ((kHeadDim / DK) * BK + 31) / 32 * 4, VROW = ((kHeadDim / DV) * BV + 31) / 32 * 4;
  uint8_t* const sm = g_smem + T::kBytes;
  NarrowHead* const head = reinterpret_cast<NarrowHead*>(sm);
  __half* const qs = reinterpret_cast<__half*>(sm + kHeadBytes);           // [2][kRows][kQStride] high, low
  float* const mo = reinterpret_cast<float*>(qs + 2 * kRows * kQStride);   // [warps][kRows][128]
  float2* const ml = reinterpret_cast<float2*>(mo + kNarrowWarps * kRows * kHeadDim);  // [warps][kRows]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_trigger();
  fill_table<DK, BK, DV, BV>(p);
  chunk_plan(p, head->pre, head->scratch);
  NarrowWorker* const me = head->worker;
  if (tid == 0) {
    me->walk.start(p, head->pre, blockIdx.x, gridDim.x);
    me->plan(p, 0);
  }
  __syncthreads();
  const uint32_t lwk = kWide ? 0u : DK == 4 ? (lane & 15) * 8 : lane * 4;
  const uint32_t lwv = kWide ? 65536u : 128u + (DV == 4 ? (lane & 15) * 8 : lane * 4);
  const int G = p.group;
  bool recorded = false;

  for (int k = 0; me->more[k & 1]; ++k) {
    const ChunkPiece& u = me->piece[k & 1];
    const ChunkKeys keys = u.k;
    const int blk1 = u.blk1, limit = u.s.limit;
    const int i0 = u.tile * p.tile_tok;
    const int rows = min(p.tile_tok, u.s.n - i0) * G;
    // ---- q~ of the tile's rows, as high and low fp16 parts ------------------------
    for (int r = warp; r < kRows; r += kNarrowWarps) query_row<kRows>(p, u, r, r < rows, qs, lane);
    __syncthreads();
    if (tid == 0) me->plan(p, k + 1);
    uint32_t qa[8][4], ql[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 32 * c + 4 * j;
      const uint2 h0 = *reinterpret_cast<const uint2*>(qs + g * kQStride + e);
      const uint2 h1 = *reinterpret_cast<const uint2*>(qs + (g + 8) * kQStride + e);
      qa[j][0] = h0.x;
      qa[j][1] = h1.x;
      qa[j][2] = h0.y;
      qa[j][3] = h1.y;
      const uint2 l0 = *reinterpret_cast<const uint2*>(qs + (kRows + g) * kQStride + e);
      const uint2 l1 = *reinterpret_cast<const uint2*>(qs + (kRows + g + 8) * kQStride + e);
      ql[j][0] = l0.x;
      ql[j][1] = l1.x;
      ql[j][2] = l0.y;
      ql[j][3] = l1.y;
    }
    // positions of the lane's rows g and g + 8 (rows past the tile see nothing)
    constexpr int NR = 2;
    int pos[NR];
    float m[NR], l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = g + 8 * i;
      pos[i] = r < rows ? u.s.base + i0 + r / G : -1;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    const int first_pos = u.s.base + i0, last_pos = u.s.base + min(i0 + p.tile_tok, u.s.n) - 1;
    float o[16][4];
#pragma unroll
    for (int nb = 0; nb < 16; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nb][e] = 0.f;

    KCodes<DK> kc[2];
    VCodes<DV, BV> vc[4];
    auto load = [&](int i, KCodes<DK>(&kx)[2], VCodes<DV, BV>(&vx)[4]) {  // false: no such page
      const int t0 = keys.block(i) * kBlock;
      const int lp = t0 / p.page_size;
      const int pg = __ldg(p.page_table + static_cast<long long>(u.b) * p.max_pages + lp);
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) report(p.status, kDevBadPage);
        return false;
      }
      const long long row = (static_cast<long long>(pg) * p.hkv + u.kvh) * p.page_size + (t0 - lp * p.page_size);
      const uint8_t* kr = p.k_pool + row * KROW;
      const uint8_t* vr = p.v_pool + row * VROW;
      kx[0].load(kr + g * KROW, c);
      kx[1].load(kr + (g + 8) * KROW, c);
      vx[0].load(vr + (2 * c) * VROW, g);
      vx[1].load(vr + (2 * c + 1) * VROW, g);
      vx[2].load(vr + (2 * c + 8) * VROW, g);
      vx[3].load(vr + (2 * c + 9) * VROW, g);
      return true;
    };
    bool have = false;
    if (u.blk0 + warp < blk1) have = load(u.blk0 + warp, kc, vc);
    for (int i = u.blk0 + warp; i < blk1; i += kNarrowWarps) {
      KCodes<DK> kn[2];
      VCodes<DV, BV> vn[4];
      bool have_n = false;
      if (i + kNarrowWarps < blk1) have_n = load(i + kNarrowWarps, kn, vn);
      const int t0 = keys.block(i) * kBlock;
      if (have) {
        // ---- scores: s[nb][..]: row g (and g + 8), tokens 8 nb + 2c, 2c + 1 ----------
        float s[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            uint32_t b[4];  // two k-steps
            if constexpr (kWide) {
              const uint4 w = tab128(kc[nb].off16(j >> 1, lwk));
              b[0] = w.x, b[1] = w.y, b[2] = w.z, b[3] = w.w;
            } else if constexpr (DK == 4) {
              const uint2 w0 = tab64(kc[nb].off(j, lwk)), w1 = tab64(kc[nb].off(j + 1, lwk));
              b[0] = w0.x, b[1] = w0.y, b[2] = w1.x, b[3] = w1.y;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] = tab32(kc[nb].off(2 * j + e, lwk));
            }
            mma16816(s[nb], qa[j][0], qa[j][1], qa[j][2], qa[j][3], b[0], b[1]);
            mma16816(s[nb], qa[j + 1][0], qa[j + 1][1], qa[j + 1][2], qa[j + 1][3], b[2], b[3]);
            mma16816(s[nb], ql[j][0], ql[j][1], ql[j][2], ql[j][3], b[0], b[1]);
            mma16816(s[nb], ql[j + 1][0], ql[j + 1][1], ql[j + 1][2], ql[j + 1][3], b[2], b[3]);
          }
        }
        // ---- masks --------------------------------------------------------------------
        const bool whole = t0 + kBlock - 1 <= first_pos && t0 + kBlock <= limit &&
                           (p.window == 0 || t0 > last_pos - p.window || t0 + kBlock <= p.sinks);
        if (!whole) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = t0 + 8 * nb + 2 * c + e;
                const bool see = t <= pos[r] && t < limit &&
                                 (p.window == 0 || t > pos[r] - p.window || t < p.sinks);
                if (!see) s[nb][2 * r + e] = -INFINITY;
              }
        }
        // ---- online softmax ------------------------------------------------------------
        float pr[NR][4];  // the row's tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
          const bool raise = mx > m[r] + kSlack || (m[r] == -INFINITY && mx > -INFINITY);
          if (__any_sync(kAll, raise)) {
            const float mn = raise ? mx : m[r];
            const float a = raise ? fast_exp2(m[r] - mn) : 1.f;  // 0 while nothing is accumulated
            m[r] = mn;
            l[r] *= a;
#pragma unroll
            for (int nb = 0; nb < 16; ++nb) {
              o[nb][2 * r] *= a;
              o[nb][2 * r + 1] *= a;
            }
          }
          const float mu = m[r] == -INFINITY ? 0.f : m[r];
          pr[r][0] = fast_exp2(s[0][2 * r] - mu);
          pr[r][1] = fast_exp2(s[0][2 * r + 1] - mu);
          pr[r][2] = fast_exp2(s[1][2 * r] - mu);
          pr[r][3] = fast_exp2(s[1][2 * r + 1] - mu);
          l[r] += (pr[r][0] + pr[r][1]) + (pr[r][2] + pr[r][3]);
        }
        auto pack = [](float a, float b) {
          const __half2 h = __floats2half2_rn(a, b);
          return *reinterpret_cast<const uint32_t*>(&h);
        };
        const uint32_t a0 = pack(pr[0][0], pr[0][1]), a1 = pack(pr[1][0], pr[1][1]);
        const uint32_t a2 = pack(pr[0][2], pr[0][3]), a3 = pack(pr[1][2], pr[1][3]);
        // ---- o += p V -------------------------------------------------------------------
        auto pv = [&](int nb, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
          mma16816(o[nb], a0, a1, a2, a3, pair_lo(w0, w1), pair_lo(w2, w3));
          mma16816(o[nb + 1], a0, a1, a2, a3, pair_hi(w0, w1), pair_hi(w2, w3));
        };
        if constexpr (kWide) {
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            uint4 w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab128(vc[t].off16(i2, lwv));
            pv(8 * i2, w[0].x, w[1].x, w[2].x, w[3].x);
            pv(8 * i2 + 2, w[0].y, w[1].y, w[2].y, w[3].y);
            pv(8 * i2 + 4, w[0].z, w[1].z, w[2].z, w[3].z);
            pv(8 * i2 + 6, w[0].w, w[1].w, w[2].w, w[3].w);
          }
        } else if constexpr (DV == 4) {
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) {
            uint2 w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab64(vc[t].off(i2, lwv));
            pv(4 * i2, w[0].x, w[1].x, w[2].x, w[3].x);
            pv(4 * i2 + 2, w[0].y, w[1].y, w[2].y, w[3].y);
          }
        } else {
#pragma unroll
          for (int i2 = 0; i2 < 8; ++i2) {
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab32(vc[t].off(i2, lwv));
            pv(2 * i2, w[0], w[1], w[2], w[3]);
          }
        }
      }
      kc[0] = kn[0], kc[1] = kn[1];
#pragma unroll
      for (int t = 0; t < 4; ++t) vc[t] = vn[t];
      have = have_n;
    }
    // ---- the warps' partials join ------------------------------------------------------
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor_sync(kAll, l[r], 1);
      l[r] += __shfl_xor_sync(kAll, l[r], 2);
      if (c == 0) ml[warp * kRows + g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
      for (int nb = 0; nb < 16; ++nb) {
        float* dst = mo + (warp * kRows + g + 8 * r) * kHeadDim;
        dst[32 * c + nb] = o[nb][2 * r];
        dst[32 * c + 16 + nb] = o[nb][2 * r + 1];
      }
    }
    __syncthreads();
    for (int r = warp; r < kRows; r += kNarrowWarps)
      join_row<kNarrowWarps, kRows>(p, u, mo, ml, r, r < rows, kRows, lane);
    if (u.slot >= 0 && (u.slot & 1) && tid == 0) {
      write_record(p, blockIdx.x, &u);
      recorded = true;
    }
    __syncthreads();  // q~ and the join buffers are free again; the next piece is known
  }
  if (tid == 0 && !recorded) write_record(p, blockIdx.x, nullptr);
}

// A lane's code words as they lie in the pools, loaded ahead of their use: the loads are volatile, so
// that they stay where they are issued, and nothing is computed from the words until get().
__device__ __forceinline__ uint32_t ld_words1(const uint8_t* at) {
  uint32_t x;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(x) : "l"(at));
  return x;
}
template <int DK>
struct KWords;
template <>
struct KWords<4> {
  KCodes<4> k;
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(k.w.x), "=r"(k.w.y) : "l"(row + 8 * c));
  }
  __device__ __forceinline__ KCodes<4> get(int) const { return k; }
};
template <>
struct KWords<2> {
  KCodes<2> k;
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(k.w.x), "=r"(k.w.y), "=r"(k.w.z), "=r"(k.w.w)
                 : "l"(row + 16 * c));
  }
  __device__ __forceinline__ KCodes<2> get(int) const { return k; }
};
template <>
struct KWords<8> {  // 48 bits from bit 48 c
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    const uint8_t* at = row + (48 * c) / 32 * 4;
    lo = ld_words1(at);
    hi = ld_words1(at + 4);
  }
  __device__ __forceinline__ KCodes<8> get(int c) const {
    KCodes<8> k;
    k.a = __funnelshift_r(lo, hi, (48 * c) & 31);
    k.b = hi >> ((48 * c) & 31);
    return k;
  }
};
template <int DV, int BV>
struct VWords;
template <>
struct VWords<4, 8> {
  VCodes<4, 8> v;
  __device__ __forceinline__ void load(const uint8_t* row, int r) { v.w = ld_words1(row + 4 * r); }
  __device__ __forceinline__ VCodes<4, 8> get(int) const { return v; }
};
template <>
struct VWords<2, 8> {
  VCodes<2, 8> v;
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.w.x), "=r"(v.w.y) : "l"(row + 8 * r));
  }
  __device__ __forceinline__ VCodes<2, 8> get(int) const { return v; }
};
template <>
struct VWords<4, 9> {  // 36 bits from bit 36 r
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    lo = ld_words1(row + 4 * r);
    hi = ld_words1(row + 4 * r + 4);
  }
  __device__ __forceinline__ VCodes<4, 9> get(int r) const {
    VCodes<4, 9> v;
    v.a = __funnelshift_r(lo, hi, 4 * r);
    v.b = hi >> (4 * r);
    return v;
  }
};
template <>
struct VWords<8, 12> {  // 24 bits from bit 24 r; the last lane's lie in its first word
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    const uint8_t* at = row + (24 * r) / 32 * 4;
    lo = ld_words1(at);
    hi = ld_words1(r < 7 ? at + 4 : at);
  }
  __device__ __forceinline__ VCodes<8, 12> get(int r) const {
    VCodes<8, 12> v;
    v.x = __funnelshift_r(lo, hi, (24 * r) & 31);
    return v;
  }
};

// ---- 8 rows or fewer per (sequence, KV head): tokens as the rows of the products ---------------
// kPair: up to 4 query rows, columns 2h and 2h + 1 of the 8-wide operand being the high and low
// fp16 parts of row h; else up to 8 rows, a column each, and two mma per step for q~.
template <int DK, int BK, int DV, int BV, bool kPair>
__global__ void __launch_bounds__(kFewWarps * 32, 1) vq_chunk_few_kernel(const ChunkParams p) {
  using T = NarrowTable<DK, BK, DV, BV>;
  constexpr bool kWide = T::kWide;
  constexpr int kRows = 8;                 // rows of a tile's slots in the workspace
  constexpr int NR = kPair ? 1 : 2;        // rows of one lane
  constexpr int kTileRows = kPair ? 4 : 8;
  constexpr int KROW = ((kHeadDim / DK) * BK + 31) / 32 * 4, VROW = ((kHeadDim / DV) * BV + 31) / 32 * 4;
  uint8_t* const sm = g_smem + T::kBytes;
  NarrowHead* const head = reinterpret_cast<NarrowHead*>(sm);
  // The CTA's warps work in groups, each with pieces of its own, so that one group's waits (page, codes,
  // join) pass under the others' products.
  const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads;
  const int worker = group * gridDim.x + blockIdx.x;  // (few pieces go to different SMs)
  __half* const qs = reinterpret_cast<__half*>(sm + kHeadBytes) + group * 2 * kRows * kQStride;  // [2][kRows][kQStride] high, low
  float* const mo = reinterpret_cast<float*>(sm + kHeadBytes + kFewGroups * 2 * kRows * kQStride * sizeof(__half)) +
                    group * kGroupWarps * kTileRows * (kHeadDim + 2);                     // [warps][kTileRows][128]
  float2* const ml = reinterpret_cast<float2*>(mo + kGroupWarps * kTileRows * kHeadDim);  // [warps][kTileRows]
  auto group_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory"); };

  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_trigger();
  fill_table<DK, BK, DV, BV>(p);
  chunk_plan(p, head->pre, head->scratch);
  NarrowWorker* const me = head->worker + group;
  if (tid == 0) {
    me->walk.start(p, head->pre, worker, kFewGroups * gridDim.x);
    me->plan(p, 0);
  }
  __syncthreads();
  const uint32_t lwk = kWide ? 0u : DK == 4 ? (lane & 15) * 8 : lane * 4;
  const uint32_t lwv = kWide ? 65536u : 128u + (DV == 4 ? (lane & 15) * 8 : lane * 4);
  const int G = p.group;
  bool recorded = false;

  for (int k = 0; me->more[k & 1]; ++k) {
    const ChunkPiece& u = me->piece[k & 1];
    const ChunkKeys keys = u.k;
    const int blk1 = u.blk1, limit = u.s.limit, kvh = u.kvh;
    const int i0 = u.tile * p.tile_tok;
    const int rows = min(p.tile_tok, u.s.n - i0) * G;
    const int32_t* const pages = p.page_table + static_cast<long long>(u.b) * p.max_pages;
    // The pipeline of a warp's blocks (every kGroupWarps-th): codes in registers one block ahead, the page
    // looked up two ahead.  A block's page and offset follow from the block before, by 64 tokens, where
    // blocks adjoin; rows are counted by 16.
    const int per_page = p.page_size / kBlock, step_page = kGroupWarps / per_page, step_off = kGroupWarps - step_page * per_page;
    int at = u.blk0 + warp, lp = 0, off = 0;  // the iterator's block, its page and its offset in blocks
    bool fresh = true;
    struct Where {
      int page, off;  // page -1: no block, or none that can be read
    };
    auto advance = [&]() {
      Where x = {-1, 0};
      if (at >= blk1) return x;
      if (fresh) {
        const int b = keys.block(at);
        lp = p.page_shift >= 0 ? b >> (p.page_shift - 4) : b / per_page;
        off = b - lp * per_page;
      }
      // (volatile: the load is to be issued here, ahead of its use)
      asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x.page) : "l"(pages + lp));
      x.off = off;
      fresh = at < keys.sink && at + kGroupWarps >= keys.sink;  // on from the sinks to the window
      at += kGroupWarps;
      lp += step_page;
      off += step_off;
      if (off >= per_page) {
        off -= per_page;
        ++lp;
      }
      return x;
    };
    auto row_of = [&](const Where& x, bool there) {  // the block's rows in the pools, in blocks of 16, or -1
      if (static_cast<unsigned long long>(x.page) < static_cast<unsigned long long>(p.num_pages)) return (x.page * p.hkv + kvh) * per_page + x.off;
      if (there && lane == 0) report(p.status, kDevBadPage);
      return -1;
    };
    KWords<DK> kw[2];
    VWords<DV, BV> vw[4];
    auto load = [&](int row, KWords<DK>(&kx)[2], VWords<DV, BV>(&vx)[4]) {
      if (row < 0) return;
      const uint8_t* kr = p.k_pool + static_cast<long long>(row) * (kBlock * KROW);
      const uint8_t* vr = p.v_pool + static_cast<long long>(row) * (kBlock * VROW);
      kx[0].load(kr + g * KROW, c);
      kx[1].load(kr + (g + 8) * KROW, c);
      vx[0].load(vr + (2 * c) * VROW, g);
      vx[1].load(vr + (2 * c + 1) * VROW, g);
      vx[2].load(vr + (2 * c + 8) * VROW, g);
      vx[3].load(vr + (2 * c + 9) * VROW, g);
    };
    const int first = u.blk0 + warp;
    const Where w0 = advance();
    Where ahead = advance();
    int row0 = row_of(w0, first < blk1);
    load(row0, kw, vw);
    // ---- q~ of the tile's rows, as high and low fp16 parts ------------------------
    for (int r = warp; r < kTileRows; r += kGroupWarps) query_row<kRows>(p, u, r, r < rows, qs, lane);
    group_sync();
    if (tid == 0) me->plan(p, k + 1);
    uint32_t qb[8][2];  // (the low parts of more than 4 rows are read again for every block: registers are short)
    const uint32_t ql_at = smem_addr(qs + (kRows + g) * kQStride + 32 * c);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = (kPair ? (g & 1) * kRows + (g >> 1) : g) * kQStride + 32 * c + 4 * j;
      const uint2 h = *reinterpret_cast<const uint2*>(qs + at);
      qb[j][0] = h.x;
      qb[j][1] = h.y;
    }
    int pos[NR];  // positions of the lane's rows (rows past the tile see nothing)
    float m[NR], l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = kPair ? c : 2 * c + i;
      pos[i] = r < rows ? u.s.base + i0 + r / G : -1;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    const int first_pos = u.s.base + i0, last_pos = u.s.base + min(i0 + p.tile_tok, u.s.n) - 1;
    float o[8][4];  // dims 16 g + 2 mb and + 1, columns 2c and 2c + 1
#pragma unroll
    for (int mb = 0; mb < 8; ++mb)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mb][e] = 0.f;

    for (int i = first; i < blk1; i += kGroupWarps) {
      const KCodes<DK> kc[2] = {kw[0].get(c), kw[1].get(c)};
      const VCodes<DV, BV> vc[4] = {vw[0].get(g), vw[1].get(g), vw[2].get(g), vw[3].get(g)};
      const int row1 = row_of(ahead, i + kGroupWarps < blk1);
      load(row1, kw, vw);
      ahead = advance();
      if (row0 >= 0) {
        const int t0 = keys.block(i) * kBlock;
        // ---- scores: tokens g and g + 8 ------------------------------------------------
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint32_t a[2][4];  // two k-steps
          if constexpr (kWide) {
            const uint4 w0 = tab128(kc[0].off16(j >> 1, lwk)), w1 = tab128(kc[1].off16(j >> 1, lwk));
            a[0][0] = w0.x, a[0][1] = w1.x, a[0][2] = w0.y, a[0][3] = w1.y;
            a[1][0] = w0.z, a[1][1] = w1.z, a[1][2] = w0.w, a[1][3] = w1.w;
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (DK == 4) {
                const uint2 w0 = tab64(kc[0].off(j + e, lwk)), w1 = tab64(kc[1].off(j + e, lwk));
                a[e][0] = w0.x, a[e][1] = w1.x, a[e][2] = w0.y, a[e][3] = w1.y;
              } else {
                a[e][0] = tab32(kc[0].off(2 * (j + e), lwk));
                a[e][1] = tab32(kc[1].off(2 * (j + e), lwk));
                a[e][2] = tab32(kc[0].off(2 * (j + e) + 1, lwk));
                a[e][3] = tab32(kc[1].off(2 * (j + e) + 1, lwk));
              }
            }
          }
          mma16816(s, a[0][0], a[0][1], a[0][2], a[0][3], qb[j][0], qb[j][1]);
          mma16816(s2, a[1][0], a[1][1], a[1][2], a[1][3], qb[j + 1][0], qb[j + 1][1]);
          if constexpr (!kPair) {
            uint32_t w[4];
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(ql_at + 8 * j));
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[2]), "=r"(w[3]) : "r"(ql_at + 8 * j + 8));
            mma16816(s, a[0][0], a[0][1], a[0][2], a[0][3], w[0], w[1]);
            mma16816(s2, a[1][0], a[1][1], a[1][2], a[1][3], w[2], w[3]);
          }
        }
        float x[NR][2];  // the lane's rows, tokens g and g + 8
        if constexpr (kPair) {
          x[0][0] = (s[0] + s2[0]) + (s[1] + s2[1]);
          x[0][1] = (s[2] + s2[2]) + (s[3] + s2[3]);
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[r][0] = s[r] + s2[r];
            x[r][1] = s[2 + r] + s2[2 + r];
          }
        }
        const bool whole = t0 + kBlock - 1 <= first_pos && t0 + kBlock <= limit &&
                           (p.window == 0 || t0 > last_pos - p.window || t0 + kBlock <= p.sinks);
        if (!whole) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = t0 + g + 8 * e;
              const bool see = t <= pos[r] && t < limit && (p.window == 0 || t > pos[r] - p.window || t < p.sinks);
              if (!see) x[r][e] = -INFINITY;
            }
        }
        // ---- online softmax: the maxima move only when a score passes them by kSlack ----------
        bool over = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float mx = fmaxf(x[r][0], x[r][1]);
          over |= mx > m[r] + kSlack || (m[r] == -INFINITY && mx > -INFINITY);
        }
        if (__any_sync(kAll, over)) {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float mx = fmaxf(fmaxf(x[r][0], x[r][1]), m[r]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
            const float a = mx == m[r] ? 1.f : fast_exp2(m[r] - mx);  // 0 while nothing is accumulated
            m[r] = mx;
            l[r] *= a;
#pragma unroll
            for (int mb = 0; mb < 8; ++mb) {
              o[mb][r] *= a;
              o[mb][2 + r] *= a;
              if constexpr (kPair) {
                o[mb][1] *= a;
                o[mb][3] *= a;
              }
            }
          }
        }
        uint32_t b[2];  // tokens 0..7 and 8..15
        float pr[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float mu = m[r] == -INFINITY ? 0.f : m[r];
          pr[r][0] = fast_exp2(x[r][0] - mu);
          pr[r][1] = fast_exp2(x[r][1] - mu);
          l[r] += pr[r][0] + pr[r][1];
        }
        if constexpr (kPair) {
          uint32_t hi, lo;
          split_pair(pr[0][0], pr[0][1], hi, lo);
          b[0] = movmatrix_trans(pair_lo(hi, lo));
          b[1] = movmatrix_trans(pair_hi(hi, lo));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const __half2 h = __floats2half2_rn(pr[0][e], pr[NR - 1][e]);
            b[e] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h));
          }
        }
        // ---- o^T += V^T p ------------------------------------------------------------------
        auto pv = [&](int mb, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
          mma16816(o[mb], pair_lo(w0, w1), pair_hi(w0, w1), pair_lo(w2, w3), pair_hi(w2, w3), b[0], b[1]);
        };
        if constexpr (kWide) {
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            uint4 w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab128(vc[t].off16(i2, lwv));
            pv(4 * i2, w[0].x, w[1].x, w[2].x, w[3].x);
            pv(4 * i2 + 1, w[0].y, w[1].y, w[2].y, w[3].y);
            pv(4 * i2 + 2, w[0].z, w[1].z, w[2].z, w[3].z);
            pv(4 * i2 + 3, w[0].w, w[1].w, w[2].w, w[3].w);
          }
        } else if constexpr (DV == 4) {
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) {
            uint2 w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab64(vc[t].off(i2, lwv));
            pv(2 * i2, w[0].x, w[1].x, w[2].x, w[3].x);
            pv(2 * i2 + 1, w[0].y, w[1].y, w[2].y, w[3].y);
          }
        } else {
#pragma unroll
          for (int i2 = 0; i2 < 8; ++i2) {
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = tab32(vc[t].off(i2, lwv));
            pv(i2, w[0], w[1], w[2], w[3]);
          }
        }
      }
      row0 = row1;
    }
    // ---- the warps' partials join ------------------------------------------------------
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(kAll, l[r], d);
      const int row = kPair ? c : 2 * c + r;
      if (g == 0) ml[warp * kTileRows + row] = make_float2(m[r], l[r]);
      float* dst = mo + (warp * kTileRows + row) * kHeadDim + 16 * g;
#pragma unroll
      for (int mb = 0; mb < 8; ++mb) {
        float2 v;
        v.x = kPair ? o[mb][0] + o[mb][1] : o[mb][r];
        v.y = kPair ? o[mb][2] + o[mb][3] : o[mb][2 + r];
        *reinterpret_cast<float2*>(dst + 2 * mb) = v;
      }
    }
    group_sync();
    for (int r = warp; r < kTileRows; r += kGroupWarps)
      join_row<kGroupWarps, kTileRows>(p, u, mo, ml, r, r < rows, kRows, lane);
    if (u.slot >= 0 && (u.slot & 1) && tid == 0) {
      write_record(p, worker, &u);
      recorded = true;
    }
    group_sync();  // q~ and the join buffers are free again; the next piece is known
  }
  if (tid == 0 && !recorded) write_record(p, worker, nullptr);
}

template <int DK, int BK, int DV, int BV, bool kPair>
cudaError_t launch_few(const ChunkParams& p, int grid, cudaStream_t stream) {
  static SmemOptIn opt;
  constexpr size_t smem = NarrowTable<DK, BK, DV, BV>::kBytes + kHeadBytes +
                          kFewGroups * 2 * 8 * kQStride * sizeof(__half) + kFewWarps * (kPair ? 4 : 8) * (kHeadDim + 2) * sizeof(float);
  cudaError_t e = ensure_smem(vq_chunk_few_kernel<DK, BK, DV, BV, kPair>, smem, opt);
  if (e != cudaSuccess) return e;
  return launch_pdl(vq_chunk_few_kernel<DK, BK, DV, BV, kPair>, dim3(grid), dim3(kFewWarps * 32), smem, stream, p, false);
}

template <int DK, int BK, int DV, int BV>
cudaError_t launch_narrow(const ChunkParams& p, int grid, cudaStream_t stream) {
  if (p.tile_rows == 8)
    return p.tile_tok * p.group <= 4 ? launch_few<DK, BK, DV, BV, true>(p, grid, stream)
                                     : launch_few<DK, BK, DV, BV, false>(p, grid, stream);
  static SmemOptIn opt;
  constexpr size_t smem = NarrowTable<DK, BK, DV, BV>::kBytes + kHeadBytes +
                          2 * 16 * kQStride * sizeof(__half) + kNarrowWarps * 16 * (kHeadDim + 2) * sizeof(float);
  cudaError_t e = ensure_smem(vq_chunk_narrow_kernel<DK, BK, DV, BV>, smem, opt);
  if (e != cudaSuccess) return e;
  return launch_pdl(vq_chunk_narrow_kernel<DK, BK, DV, BV>, dim3(grid), dim3(kNarrowWarps * 32), smem, stream, p, false);
}

// ---- merge of the pieces of tiles that several CTAs took -----------------------------
// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the tile's pieces, in the workers' order.
// blockIdx.x: the worker that began the tile; one warp per row, four elements per lane.
__global__ void __launch_bounds__(256) vq_chunk_merge_kernel(const ChunkParams p) {
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.records + c0));
  const int half = p.tile_rows == 256 ? 128 : p.tile_rows, half_tok = p.tile_tok * half / p.tile_rows;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < p.tile_rows; r += gridDim.y * 8) {
    // row r: of 256 rows, each 128 hold half of the tile's tokens
    const int in_half = r % half, token = r / half * half_tok + in_half / p.group;
    if (in_half >= half_tok * p.group || token >= rec.x) continue;
    auto at = [&](int w) {
      return static_cast<long long>(w == c0 ? 2 * c0 + 1 : 2 * w) * p.tile_rows + r;
    };
    float M = -INFINITY;
    for (int i = c0 + lane; i <= rec.w; i += 32) M = fmaxf(M, __ldcg(p.ws_ml + at(i)).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    const float Mu = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int i = c0; i <= rec.w; ++i) {
      const float2 v = __ldcg(p.ws_ml + at(i));
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p.ws_o + at(i) * kHeadDim) + lane);
      const float f = fast_exp2(v.x - Mu);
      L = fmaf(f, v.y, L);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
    const float f = L == 0.f ? 0.f : 1.f / L;
    const __half2 h0 = __floats2half2_rn(acc.x * f, acc.y * f), h1 = __floats2half2_rn(acc.z * f, acc.w * f);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&h0);
    w.y = *reinterpret_cast<const uint32_t*>(&h1);
    const long long row = static_cast<long long>(rec.y + token) * p.hq + rec.z * p.group + in_half % p.group;
    reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + row * kHeadDim)[lane] = w;
  }
}

}  // namespace

cudaError_t launch_chunk_narrow(const ChunkParams& p, int k_sub, int k_bits, int v_sub, int v_bits, int grid,
                                cudaStream_t stream) {
  if (k_sub == 8 && k_bits == 12 && v_sub == 8 && v_bits == 12) return launch_narrow<8, 12, 8, 12>(p, grid, stream);
  if (k_bits == 8 && (k_sub == 2 || k_sub == 4)) {
    const bool k4 = k_sub == 4;
    if (v_sub == 4 && v_bits == 8) return k4 ? launch_narrow<4, 8, 4, 8>(p, grid, stream) : launch_narrow<2, 8, 4, 8>(p, grid, stream);
    if (v_sub == 4 && v_bits == 9) return k4 ? launch_narrow<4, 8, 4, 9>(p, grid, stream) : launch_narrow<2, 8, 4, 9>(p, grid, stream);
    if (v_sub == 2 && v_bits == 8) return k4 ? launch_narrow<4, 8, 2, 8>(p, grid, stream) : launch_narrow<2, 8, 2, 8>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_chunk_merge(const ChunkParams& p, int workers, cudaStream_t stream) {
  return launch_pdl(vq_chunk_merge_kernel, dim3(workers, (p.tile_rows + 7) / 8), dim3(256), 0, stream, p, true);
}

}  // namespace vqk
