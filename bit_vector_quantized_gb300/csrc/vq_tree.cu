// vq_tree.cu -- attention of drafted trees for few query rows per (sequence, KV head) (sm_103a).
//
// The mathematics of vq_chunk_narrow.cu, with a tree's masks: a row sees the context, and of the drafted tokens
// those that its bits name.  Tens of rows, and every code of the context to expand for them: what costs is not the
// products but the way of the centroids through shared memory.  So the products stand the other way round than in
// vq_chunk_wide.cu, the tokens as rows of the scores and the dims as rows of the output, N query rows as columns:
//   S^T [128 tokens x N] = K~ Q~^T,  P^T = 2^(S^T - m),  O^T [128 dims x N] += V^T P^T  (N = 16 or 32).
//
//   * K~ goes from the gathers straight into tensor memory (a thread's token is a lane), V as 16-byte pieces into
//     swizzled shared memory (rows of dims, the token as k), so of a block of 128 tokens 96 KB are gathered and stored
//     and 32 KB read by the tensor core, where tiles of query rows take 128 KB and 96 KB.
//   * Q~ stays in shared memory, high and low fp16 parts, for the tile (scores keep about fp32 accuracy), and so does P of a
//     block (vq_chunk_wide.cuh has why).  High and low parts are columns of one product of 2 N, in either product.
//   * Four or eight warps do the softmax: a thread has one token and 16 rows.  The rows' maxima are in shared memory and
//     may lag by 2^8, so the usual block needs no maximum over the tokens, only a vote whether one moved.
//   * Eight warps expand K, eight V, four of them every other block, a thread a whole token; one thread issues, one warp
//     plans, as in vq_chunk_wide.cu, whose rings, barriers and bounded waits these are.  (All of them at every block, a
//     thread half a token: 249 us instead of 190 for 16 tiles of 16 rows over 32K tokens, by instructions.)
//   * The planning warp plans while the others fill the table, and one warp sends the codes to L2 ahead of the others.
//
// What bounds it.  No pipe is full by counters (16 rows of each of 8 sequences of 4000 to 8000, (4,8)): shared memory 29 %,
// issue 27 %, tensor 7 %; the warps wait for codes and, around the blocks, for one another (a piece's q~, first
// maxima, sums and output cost about 5 us, the start 6).  A block of 128 tokens takes 1110 wavefronts of shared memory there,
// 1940 at 1.5 bit, where half of them are the plain tables' bank conflicts (pipe 60 % busy).  Measured, merge included, 8 KV
// heads: 16 rows of each of those 8 sequences 42 us, 32 rows 49 (tiles of 128 rows 55 and 56); of each of
// 16 sequences of 32K 202 and 275 at (4,8), 226 and 305 at (2,8), (4,9), 296 for 16 rows at 1.5 bit; 32 rows over one
// sequence of 32K 39.  A variant for 64 rows did not beat tiles of 128: its softmax threads, 32 rows each, spilled.
#include <type_traits>

#include "vq_chunk_wide.cuh"

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kSlack = 8.f;        // the running maximum may lag by this much (log2 units): p <= 2^(8 + kLift)
constexpr float kUnset = 1e30f;      // in place of kLift minus the maximum, of a row that has seen nothing
constexpr int kBlockTok = 128;       // tokens of a block
constexpr int kCodeWarps = 16;
constexpr uint32_t kKStages = 4;
constexpr int kCodeSets = 2;         // the code warps of a side take every other block
constexpr uint32_t kPieces = kTreePieces;
constexpr int kBarriers = 20 + 2 * kTreePieces;  // (one to spare: what follows is 16-byte aligned)
static_assert(kTreeAhead == 2 * kCodeSets, "a code warp arrives for a block once it has looked two of its own further");

// A softmax thread takes one token and 16 rows.
constexpr int kColumns = 16;
template <int N>
struct TreeShape {
  static constexpr int kSoftWarps = 4 * (N / kColumns), kThreads = (kSoftWarps + kCodeWarps + 4) * 32;
  // Registers per thread: 80 at the launch of 768 threads, 72 of 896, then their shares
  static constexpr int kLaunch = N == 16 ? 80 : 72, kSoft = N == 16 ? 128 : 80, kCode = 72, kIssue = N == 16 ? 56 : 40;
  static_assert(kSoftWarps * kSoft + kCodeWarps * kCode + 4 * kIssue <= (kThreads / 32) * kLaunch, "the block's registers at the launch");
  // Tensor memory: S of high and low parts, twice; O; K~ of blocks under way.
  static constexpr uint32_t kColS = 0, kColO = 4 * N, kCols = 512, kColK = kCols - 64 * kKStages;
  static_assert(kColO + 2 * N <= kColK, "columns");
};
constexpr int kMasks = 4;            // token masks in flight (vq_chunk_wide.cu has why four are enough)

template <int DK, int BK, int DV, int BV, int N>
struct TreeSmem {
  using Table = WideTable<DK, BV>;
  static constexpr int kVTile = kBlockTok * kHeadDim * 2, kVStages = 2;
  // P of two blocks: rows of tokens of 128 bytes, the rows' high parts and then their low ones; N = 16: two blocks' in a row.
  static constexpr uint32_t kPNext = N == 16 ? 64 : kBlockTok * 128;  // from an even block's to an odd one's
  static constexpr int kPTile = (N == 16 ? 1 : 2) * kBlockTok * 128;
  static constexpr int kQTile = 2 * N * kHeadDim * 2;  // rows of high parts, then of low parts
  static constexpr int kV = Table::kBytes;
  static constexpr int kP = kV + kVStages * kVTile;
  static constexpr int kQ = kP + kPTile;
  static constexpr int kMisc = kQ + kQTile;
  static constexpr int kBars = kBarriers * 8 + kTreePieces * 64 + kMasks * 16 + 16;
  static constexpr int kTops = kMisc + kBars;  // [N] minus the maxima, [N] scales, [4][N] maxima or sums of the warps
  static constexpr int kTotal = kTops + 6 * N * 4;
  static_assert(kTotal <= 232448, "shared memory of one CTA");
  static_assert((kChunkMaxBatch + 1) * 8 <= kVTile, "the plan shares a tile");
};

__device__ __forceinline__ float warp_max(float x) {  // (numbers before NaN)
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <int DK, int BK, int DV, int BV, int N>
__global__ void __launch_bounds__(TreeShape<N>::kThreads, 1) vq_tree_kernel(const ChunkParams p) {
  using W = TreeSmem<DK, BK, DV, BV, N>;
  using Shape = TreeShape<N>;
  constexpr int NV = W::kVStages, NC = kColumns, kSoftWarps = Shape::kSoftWarps;
  constexpr uint32_t kColS = Shape::kColS, kColO = Shape::kColO, kColK = Shape::kColK, kCols = Shape::kCols;
  constexpr int KROW = ((kHeadDim / DK) * BK + 31) / 32 * 4, VROW = ((kHeadDim / DV) * BV + 31) / 32 * 4;
  constexpr bool kWideCodes = W::Table::kWideCodes, kSplitTable = W::Table::kSplitTable;
  uint8_t* const tiles = g_smem + W::kV;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(g_smem + W::kMisc);
  uint64_t* const ready = bars;            // [4] by block b: P of b, the V tile of b, the K tile of b + 2
  uint64_t* const start = ready + 4;       // K tiles of blocks 0 and 1
  uint64_t* const k_empty = start + 1;     // [kKStages] scores done, the tile is free
  uint64_t* const v_empty = k_empty + 4;   // [2]
  uint64_t* const s_full = v_empty + 2;    // [4] by block: the scores are done, the tokens' masks are there
  uint64_t* const o_full = s_full + 4;     // [2] values of a piece's last block but one, and of its last
  uint64_t* const q_full = o_full + 2;     // Q~ stored, O read
  uint64_t* const drain = q_full + 1;
  uint64_t* const piece_full = drain + 1;              // [kPieces] planning warp -> everybody
  uint64_t* const piece_empty = piece_full + kPieces;  // [kPieces]
  WidePiece* const pieces = reinterpret_cast<WidePiece*>(bars + kBarriers);           // [kPieces]
  uint32_t* const masks = reinterpret_cast<uint32_t*>(pieces + kPieces);              // [kMasks][4] tokens that have a page
  uint32_t* const tmem_at = masks + kMasks * 4;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
  volatile uint32_t* const done = tmem_at + 2;  // blocks whose values are under way
  float* const neg_max = reinterpret_cast<float*>(g_smem + W::kTops);  // [N] kLift minus the maxima
  float* const scales = neg_max + N;                                   // [N]
  float* const tops = scales + N;                                      // [4][N]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, worker = blockIdx.x;
  pdl_trigger();
  if (smem_addr(tiles) & 1023u) {  // the swizzled tiles need it (and dynamic shared memory alone gives it)
    if (tid == 0) report(p.status, kDevBadConfig);
    if (tid == 0) write_record(p, worker, nullptr);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(ready + i, kSoftWarps + 4 + 4);
      mbar_init(s_full + i, 1 + 4);
    }
    mbar_init(start, 8);
    for (uint32_t i = 0; i < kKStages; ++i) mbar_init(k_empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(v_empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(o_full + i, 1);
    mbar_init(q_full, kSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < static_cast<int>(kPieces); ++i) {
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, kSoftWarps + kCodeWarps + 2);
    }
    mbar_init_fence();
    *abort_flag = 0;
    *done = 0;
  }
  if (warp == kSoftWarps + kCodeWarps) tmem_alloc<false>(tmem_at, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All 512 columns are this CTA's, so they start at column 0; the constant keeps the products' operands uniform.
  constexpr uint32_t tmem = 0;
  if (*tmem_at != tmem) {
    if (tid == 0) report(p.status, kDevBadConfig);
    if (tid == 0) write_record(p, worker, nullptr);
    __syncthreads();
    if (warp == kSoftWarps + kCodeWarps) tmem_free<false>(*tmem_at, kCols);
    return;
  }

  // The planning warp plans while the others fill the table.
  if (warp != kSoftWarps + kCodeWarps + 1) {
    fill_wide_table<DK, BK, DV, BV>(p, warp > kSoftWarps + kCodeWarps + 1 ? tid - 32 : tid, Shape::kThreads - 32);
    asm volatile("bar.sync 6, %0;" ::"n"(Shape::kThreads - 32) : "memory");
  }

  // Bounded wait, uniform over the warp; on a timeout the CTA is given up.
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    bool ok = mbar_wait_bounded(bar, phase, abort_flag, p.timeout_ns);
    if (!ok && !*abort_flag) {
      *abort_flag = 1;
      report(p.status, kDevTimeout);
    }
    return __all_sync(kAll, ok) != 0;
  };
  // The next piece (whole warps); false when there is none or the CTA was given up.
  Ring rp;
  auto next_piece = [&](WidePiece& u) {
    if (!wait(piece_full + rp.slot, rp.phase)) return false;
    u = pieces[rp.slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty + rp.slot);
    rp.next(kPieces);
    return u.more != 0;
  };
  WidePiece u = {};

  if (warp < kSoftWarps) {
    // ====== a thread per token, and all rows or half of them: columns NC g .. NC g + NC - 1 ==============
    reg_inc<Shape::kSoft>();
    const int quarter = warp & 3, g = warp >> 2, G = p.group, tok = 32 * quarter + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t inv_g = 65536u / G + 1u;  // r / G = r * inv_g >> 16 for r < 128
    uint8_t* const qs = g_smem + W::kQ;
    uint8_t* const ps = g_smem + W::kP;
    // Barriers have no limit, so a warp that gave up goes on to meet the others at all of them, without the work
    // between, and they leave together: whether there is another piece, and whether a half's maxima moved, is voted on.
    auto half_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); };
    auto vote = [](int bar, int threads, bool x, bool all) {
      uint32_t r;
      if (all)
        asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbar.red.and.pred b, %2, %3, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                     : "=r"(r) : "r"(static_cast<uint32_t>(x)), "r"(bar), "r"(threads) : "memory");
      else
        asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbar.red.or.pred b, %2, %3, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                     : "=r"(r) : "r"(static_cast<uint32_t>(x)), "r"(bar), "r"(threads) : "memory");
      return r != 0;
    };
    uint32_t blocks = 0, ends0 = 0, ends1 = 0;  // blocks so far, phases of o_full so far
    bool ok = true;
    for (;;) {
      ok = ok && next_piece(u);
      if (!vote(5, kSoftWarps * 32, ok, true)) break;  // (the last piece's Q~, maxima and sums are free)
      // ---- q~ = q diag(lambda) H of rows warp, warp + 8, .., 0 where there is none ----------------------
      const float4 lam = __ldg(reinterpret_cast<const float4*>(p.lambda + u.kvh * kHeadDim) + lane);
#pragma unroll 2
      for (int r = warp; r < N; r += kSoftWarps) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < u.rows) {
          const int token = static_cast<int>(r * inv_g >> 16);
          const long long row = static_cast<long long>(u.row0 + token) * p.hq + u.kvh * G + (r - token * G);
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __half*>(p.q) + row * kHeadDim) + lane);
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
        uint8_t* const at = qs + (lane >> 4) * (2 * N * 128) + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8;
        *reinterpret_cast<uint2*>(at) = vh;
        *reinterpret_cast<uint2*>(at + N * 128) = vl;  // (N is a multiple of eight)
      }
      if (tid < N) neg_max[tid] = kUnset;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();  // (O's reads of the last piece)
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      vote(5, kSoftWarps * 32, true, true);  // the maxima are there
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;

      const int nblk = u.blk1 - u.blk0, ctx = u.first_pos + 1;
      for (int j = 0; j < nblk; ++j) {
        ok = ok && wait(s_full + (blocks & 3u), (blocks >> 2) & 1u);
        const uint32_t col_s = tmem + lanes + kColS + 2 * N * (blocks & 1u) + NC * g;
        uint32_t s[NC];
        // a token's scores, minus infinity where a row does not see it
        auto scores = [&]() {
          uint32_t low[NC];
          tmem_ld16(col_s, s);
          tmem_ld16(col_s + N, low);
          const int t0 = u.block(u.blk0 + j) * kBlockTok, t = t0 + tok;
          const uint4 seen = *reinterpret_cast<const uint4*>(masks + (blocks % kMasks) * 4);
          const bool whole = t0 + kBlockTok <= ctx && (p.window == 0 || t0 > u.last_pos - p.window || t0 + kBlockTok <= p.sinks) &&
                             (seen.x & seen.y & seen.z & seen.w) == kAll;
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            float x0 = __uint_as_float(s[c]), x1 = __uint_as_float(s[c + 1]);
            add2(x0, x1, __uint_as_float(low[c]), __uint_as_float(low[c + 1]));
            s[c] = __float_as_uint(x0), s[c + 1] = __float_as_uint(x1);
          }
          if (whole) return;
          const uint32_t here = quarter == 0 ? seen.x : quarter == 1 ? seen.y : quarter == 2 ? seen.z : seen.w;
          const bool there = here >> lane & 1u;
          const int at = t - ctx;  // among the drafted tokens
          const bool drafted = at >= 0;
          const int its = drafted && there && p.window > 0 ? max(__ldg(p.positions + u.seq_row + at), ctx) : t;
          const unsigned long long* const bits = p.masks + static_cast<long long>(u.row0) * p.mask_words + (drafted && there ? at >> 6 : 0);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int r = NC * g + c, token = static_cast<int>(r * inv_g >> 16);
            bool see = there && r < u.rows;
            if (see && drafted) see = __ldg(bits + static_cast<long long>(token) * p.mask_words) >> (at & 63) & 1ULL;
            if (see && p.window > 0) see = its > max(__ldg(p.positions + u.row0 + token), ctx) - p.window || its < p.sinks;
            if (!see) s[c] = __float_as_uint(-INFINITY);
          }
        };
        // minus the maxima so far, plus kLift; whether one is passed
        auto shift = [&]() {
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 m = *reinterpret_cast<const float4*>(neg_max + NC * g + c);
            float x0 = __uint_as_float(s[c]), x1 = __uint_as_float(s[c + 1]), x2 = __uint_as_float(s[c + 2]), x3 = __uint_as_float(s[c + 3]);
            add2(x0, x1, m.x, m.y);
            add2(x2, x3, m.z, m.w);
            s[c] = __float_as_uint(x0), s[c + 1] = __float_as_uint(x1), s[c + 2] = __float_as_uint(x2), s[c + 3] = __float_as_uint(x3);
          }
          float top = max3(s[0], s[1], s[2]);
#pragma unroll
          for (int c = 3; c + 1 < NC; c += 2) top = max3(__float_as_uint(top), s[c], s[c + 1]);
          return fmaxf(top, __uint_as_float(s[NC - 1])) > kSlack + kLift;
        };
        bool passed = false;
        if (ok) {
          tc_fence_after();
          scores();
          passed = shift();
        }
        if (vote(1 + g, 128, passed, false)) {  // ---- the maxima move, and O and the sums with them
          const int col = NC * g + (lane & (NC - 1));
          const float old = -neg_max[col];
          if (ok) {
            scores();
            float mine = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float m = warp_max(__uint_as_float(s[c]));
              if ((lane & (NC - 1)) == c) mine = m;
            }
            if (lane < NC) tops[quarter * N + col] = mine;
          }
          half_sync();
          if (quarter == 0 && lane < NC) {
            const float top = fmaxf(fmaxf(tops[col], tops[N + col]), fmaxf(tops[2 * N + col], tops[3 * N + col]));
            const bool unset = old == -kUnset;
            const bool moves = top > -INFINITY && (unset || top > old + (kSlack + kLift));
            const float next = kLift - top;
            scales[col] = moves && !unset ? fast_exp2(old + next) : 1.f;  // (unset: nothing is accumulated)
            if (moves) neg_max[col] = next;
          }
          half_sync();
          if (ok) {
            shift();
#pragma unroll
            for (int c = 0; c < NC; ++c) l[c] *= scales[NC * g + c];
            if (j > 0) {  // O follows, once the values of block - 1 are in (the next scores come after them)
              ok = j + 1 < nblk ? wait(s_full + ((blocks + 1) & 3u), ((blocks + 1) >> 2) & 1u) : wait(o_full, ends0 & 1u);
              if (ok) {
                tc_fence_after();
                uint32_t o[NC];
                tmem_ld16(tmem + lanes + kColO + NC * g, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * scales[NC * g + c]);
                tmem_st16(tmem + lanes + kColO + NC * g, o);
                tmem_ld16(tmem + lanes + kColO + N + NC * g, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * scales[NC * g + c]);
                tmem_st16(tmem + lanes + kColO + N + NC * g, o);
                tmem_wait_st();
              }
            }
          }
        }
        if (ok) {
          // p and its sums; P^T as rows of tokens.  (The scores of this block came after the values of the one before
          // the last, so its place in shared memory is free.)
          const uint32_t row = smem_addr(ps) + tok * 128;
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x0 = fast_exp2(__uint_as_float(s[c0 + 2 * i])), x1 = fast_exp2(__uint_as_float(s[c0 + 2 * i + 1]));
              add2(l[c0 + 2 * i], l[c0 + 2 * i + 1], x0, x1);
              cut_pair(x0, x1, hi[i], lo[i]);
            }
            const uint32_t piece = (NC * g + c0) / 8 + (N == 16 ? 4 * (blocks & 1u) : 0u);
            const uint32_t tile = row + (N == 16 ? 0u : (blocks & 1u) * W::kPNext);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile + ((piece ^ (tok & 7)) << 4)), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile + (((piece + N / 8) ^ (tok & 7)) << 4)), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
                         "r"(lo[3])
                         : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + (blocks & 3u));
        }
        ++blocks;
      }
      // ---- the rows' sums over the tokens: over a warp, then the four warps of a half --------------------
      ok = ok && (nblk < 2 || wait(o_full, ends0 & 1u)) && wait(o_full + 1, ends1 & 1u);
      if (nblk >= 2) ++ends0;
      ++ends1;
#pragma unroll
      for (int m = NC / 2; m > 0; m >>= 1)  // lane keeps columns whose bit m is its own
#pragma unroll
        for (int c = 0; c < m; ++c) {
          const float mine = lane & m ? l[c + m] : l[c], other = lane & m ? l[c] : l[c + m];
          l[c] = mine + __shfl_xor_sync(kAll, other, m);
        }
#pragma unroll
      for (int m = NC; m < 32; m <<= 1) l[0] += __shfl_xor_sync(kAll, l[0], m);
      if (lane < NC) tops[quarter * N + NC * g + lane] = l[0];
      half_sync();
      if (quarter == 0 && lane < NC) {
        const int r = NC * g + lane;
        const float sum = (tops[r] + tops[N + r]) + (tops[2 * N + r] + tops[3 * N + r]);
        scales[r] = sum == 0.f ? 0.f : 1.f / sum;
        if (u.slot >= 0 && r < u.rows)
          p.ws_ml[static_cast<long long>(u.slot) * N + r] = make_float2(neg_max[r] == kUnset ? -INFINITY : -neg_max[r], sum);
      }
      half_sync();
      if (ok) {
        tc_fence_after();
        const int dim = tok;  // lanes are dims now
        uint32_t o[NC];
        tmem_ld16(tmem + lanes + kColO + NC * g, o);
        tmem_wait_ld();
        {  // of the low parts
          uint32_t low[NC];
          tmem_ld16(tmem + lanes + kColO + N + NC * g, low);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(low[c]));
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int r = NC * g + c;
          if (r >= u.rows) continue;
          if (u.slot >= 0) {
            p.ws_o[(static_cast<long long>(u.slot) * N + r) * kHeadDim + dim] = __uint_as_float(o[c]);
          } else {
            const int token = static_cast<int>(r * inv_g >> 16);
            const long long row = static_cast<long long>(u.row0 + token) * p.hq + u.kvh * G + (r - token * G);
            static_cast<__half*>(p.out)[row * kHeadDim + dim] = __float2half_rn(__uint_as_float(o[c]) * scales[r]);
          }
        }
      }
    }
  } else if (warp < kSoftWarps + kCodeWarps) {
    // ================================= code warps ======================================
    reg_dec<Shape::kCode>();
    // Eight expand K, eight V, four of them every other block; a thread takes one token's 128 dims.  K: a warp's tokens
    // are the lanes of tensor memory that it may write.  (A token that cannot be read gets what stands in the
    // registers for codes: some centroid of K, whose score is masked, and zeros of V: p is 0, but a centroid that no code
    // names may be no number.)
    const int set = (warp >> 2) & 1, tok = 32 * (warp & 3) + lane;
    auto expand = [&](auto codes, auto row_bytes, const uint8_t* pool, uint32_t table, auto is_k) {
      using Codes = decltype(codes);
      constexpr int kRow = decltype(row_bytes)::value;
      constexpr bool kIsK = decltype(is_k)::value;
      constexpr int kShift = kWideCodes ? 4 : kSplitTable ? 7 : 8;
      constexpr uint32_t kStages = kIsK ? kKStages : NV;
      uint64_t* const empty = kIsK ? k_empty : v_empty;
      // The set's blocks: a block's page is looked up two ahead of it, its codes are asked for one ahead.
      pool += (tok % 16) * kRow;
      const int per_page = p.page_size / 16;
      bool more = true;
      int i = set;
      const int32_t* pages = nullptr;
      u.blk1 = 0;
      struct Where {
        int page, off, kvh;
        bool in, any;  // the token exists; the block exists
      };
      auto advance = [&]() {
        Where x = {0, 0, 0, false, false};
        while (more && i >= u.blk1) {
          const int over = i - u.blk1;
          more = next_piece(u);
          i = more ? u.blk0 + over : 0;
          pages = p.page_table + static_cast<long long>(u.b) * p.max_pages;
        }
        if (!more) return x;
        const int t = u.block(i) * kBlockTok + tok, lp = p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
        i += kCodeSets;
        x.any = true;
        x.in = t < u.limit;
        x.kvh = u.kvh;
        x.off = (t - lp * p.page_size) / 16;
        // (volatile like the codes' loads: it is to be under way before its use)
        if (x.in) asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x.page) : "l"(pages + lp));
        return x;
      };
      Codes now;
      auto fetch = [&](const Where& x) {  // whether the token can be read
        const bool good = x.in && static_cast<unsigned long long>(x.page) < static_cast<unsigned long long>(p.num_pages);
        if (good) {
          const uint32_t row16 = static_cast<uint32_t>(x.page * p.hkv + x.kvh) * per_page + x.off;
          now.load(pool + static_cast<unsigned long long>(row16) * (16 * kRow));
        } else if (x.in) {
          report(p.status, kDevBadPage);
        }
        return good;
      };
      const uint32_t v_at = smem_addr(tiles) + tok * 128 + ((tok & 7) << 4);
      const uint32_t k_at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kColK;
      const Where first = advance();
      Where ahead = advance();
      bool any = first.any, has = any && fetch(first);
      uint32_t blk = set, stage = set, phase = 1;
      auto next_stage = [&]() {
        blk += kCodeSets;
        stage += kCodeSets;
        if (stage >= kStages) {
          stage -= kStages;
          phase ^= 1u;
        }
      };
      auto arrive = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(!kIsK ? ready + (blk & 3u) : blk < 2 ? start : ready + ((blk - 2) & 3u));
      };
      while (any) {
        if constexpr (!kIsK) {  // the tokens of the block that can be read
          const uint32_t seen = __ballot_sync(kAll, has);
          if (lane == 0) {
            masks[(blk % kMasks) * 4 + (warp & 3)] = seen;
            mbar_arrive(s_full + (blk & 3u));
          }
        }
        if (!wait(empty + stage, phase)) break;
        now.align(0);
        if constexpr (kIsK) {
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < 16; c0 += 4) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 v = gather_piece<Codes, kShift>(now, c0 + c, table);
              w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
            }
            tmem_st16(k_at + 64 * stage + 4 * c0, w);
          }
        } else {
          const uint32_t at = v_at + stage * W::kVTile;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 v = has ? gather_piece<Codes, kShift>(now, c, table) : make_uint4(0, 0, 0, 0);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"((at ^ ((c & 7) << 4)) + (c >> 3) * (kBlockTok * 128)), "r"(v.x), "r"(v.y), "r"(v.z),
                         "r"(v.w)
                         : "memory");
          }
        }
        const Where then = ahead;
        any = then.any;
        has = any && fetch(then);
        ahead = advance();  // (may wait for pieces up to kTreeAhead blocks on, before this block's arrival: the ring holds them)
        if constexpr (kIsK) {
          tmem_wait_st();
          tc_fence_before();
        } else {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        arrive();
        next_stage();
      }
      // The last two blocks have no K tile to wait for; its arrivals come in their turn all the same, one of either set
      // (unless the CTA was given up).
      if (kIsK && !any && wait(empty + stage, phase)) arrive();
    };
    const uint32_t rep_k = DK == 4 ? (lane & 15) * 8 : lane * 4, rep_v = DV == 4 ? (lane & 15) * 8 : lane * 4;
    if (warp < kSoftWarps + kCodeWarps / 2)
      expand(PartCodes<DK, BK, kHeadDim>{}, std::integral_constant<int, KROW>{}, p.k_pool, kWideCodes ? 0u : rep_k, std::true_type{});
    else
      expand(PartCodes<DV, BV, kHeadDim>{}, std::integral_constant<int, VROW>{}, p.v_pool,
             kWideCodes ? 65536u : (kSplitTable ? 32768u : 128u) + rep_v, std::false_type{});
  } else {
    // ================================= the products ====================================
    reg_dec<Shape::kIssue>();
    if (warp == kSoftWarps + kCodeWarps) {
      constexpr uint32_t kScores = tc_idesc(kBlockTok, 2 * N, false), kValues = tc_idesc_rows_k(kHeadDim, 2 * N);
      const uint32_t v0 = smem_addr(tiles), q0 = smem_addr(g_smem + W::kQ), p0 = smem_addr(g_smem + W::kP);
      Ring rk, rv;
      uint32_t blocks = 0, tiles_done = 0;
      bool ok = true;
      while (ok && next_piece(u)) {
        const int nblk = u.blk1 - u.blk0;
        ok = wait(q_full, tiles_done++ & 1u);
        auto scores = [&](uint32_t blk) {  // of block blk, whose K tile is there
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // columns: the rows' high parts, then their low parts
              tc_mma_ts<false>(tmem + kColS + 2 * N * (blk & 1u), tmem + kColK + 64 * rk.slot + 8 * ks,
                               tc_desc(q0 + (ks >> 2) * (2 * N * 128) + (ks & 3) * 32, 16), kScores, ks > 0);
            tc_commit<false>(s_full + (blk & 3u));
            tc_commit<false>(k_empty + rk.slot);
          }
          __syncwarp();
          rk.next(kKStages);
        };
        // scores of blocks 0 and 1 (their K tiles were there with the blocks before), then values of block j and scores
        // of block j + 2 (into j's columns)
        if (ok && blocks == 0) ok = wait(start, 0);
        tc_fence_after();
        for (int j = 0; ok && j < min(nblk, 2); ++j) scores(blocks + j);
        for (int j = 0; ok && j < nblk; ++j) {
          const uint32_t blk = blocks + j;
          ok = wait(ready + (blk & 3u), (blk >> 2) & 1u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vt = v0 + rv.slot * W::kVTile, pt = p0 + (blk & 1u) * W::kPNext;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_ss(tmem + kColO, tc_desc(vt + ks * 2048, kBlockTok * 128), tc_desc(pt + ks * 2048, kBlockTok * 128), kValues,
                        j > 0 || ks > 0);
            tc_commit<false>(v_empty + rv.slot);
            if (j + 2 >= nblk) tc_commit<false>(o_full + (j + 1 == nblk));
          }
          __syncwarp();
          rv.next(NV);
          if (lane == 0) *done = blk;
          if (j + 2 < nblk) scores(blk + 2);
        }
        blocks += nblk;
      }
      // (given up or not) the products in flight end before the tensor memory goes back
      if (elect_one()) tc_commit<false>(drain);
      __syncwarp();
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < p.timeout_ns) {
      }
    } else if (warp == kSoftWarps + kCodeWarps + 1) {
      // ================================== planning =======================================
      long long* const pre = reinterpret_cast<long long*>(tiles);  // the plan: the tiles over it wait for the first piece
      tree_plan(p, pre);
      ChunkWalk<kBlockTok, true> walk;
      walk.start(p, pre, worker, gridDim.x);
      ChunkPiece q;
      Ring ro;
      bool recorded = false;
      for (bool more = true; more;) {
        more = walk.next(p, q);
        const int i0 = q.tile * p.tile_tok, n = more ? min(p.tile_tok, q.s.n - i0) : 0;
        if (more && q.slot >= 0 && (q.slot & 1)) {
          if (lane == 0) write_record(p, worker, &q);
          recorded = true;
        }
        if (more && q.blk0 >= q.blk1) {  // rows that see nothing here: zero, or an empty partial
          for (int r = 0; r < n * p.group; ++r) {
            if (q.slot >= 0) {
              const long long at = static_cast<long long>(q.slot) * N + r;
              reinterpret_cast<float4*>(p.ws_o + at * kHeadDim)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (lane == 0) p.ws_ml[at] = make_float2(-INFINITY, 0.f);
            } else {
              const long long row = static_cast<long long>(q.s.row0 + i0 + r / p.group) * p.hq + q.kvh * p.group + r % p.group;
              reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + row * kHeadDim)[lane] = make_uint2(0, 0);
            }
          }
          continue;
        }
        if (more) {  // the query rows, for the softmax warps a piece later
          const char* rows = reinterpret_cast<const char*>(static_cast<const __half*>(p.q) +
                                                           (static_cast<long long>(q.s.row0 + i0) * p.hq + q.kvh * p.group) * kHeadDim);
          const int lines = 2 * p.group;  // a token's rows, 128 bytes each line
          for (int i = lane; i < n * lines; i += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + static_cast<long long>(i / lines) * p.hq * (kHeadDim * 2) + (i % lines) * 128));
        }
        int last = 0;  // of the rows, the furthest position
        if (more && p.window > 0) {
          for (int i = lane; i < n; i += 32) last = max(last, __ldg(p.positions + q.s.row0 + i0 + i));
          last = max(__reduce_max_sync(kAll, last), q.s.base);
        }
        if (!wait(piece_empty + ro.slot, ro.phase ^ 1u)) break;
        if (lane == 0) {
          WidePiece w = {};
          w.more = more;
          if (more) {
            w.b = q.b;
            w.kvh = q.kvh;
            w.row0 = q.s.row0 + i0;
            w.rows = n * p.group;
            w.first_pos = q.s.base - 1;
            w.last_pos = last;
            w.limit = q.s.limit;
            w.sink = q.k.sink;
            w.lo = q.k.lo;
            w.blk0 = q.blk0;
            w.blk1 = q.blk1;
            w.slot = q.slot;
            w.seq_row = q.s.row0;
          }
          pieces[ro.slot] = w;
          mbar_arrive(piece_full + ro.slot);
        }
        __syncwarp();
        ro.next(kPieces);
      }
      if (!recorded && lane == 0) write_record(p, worker, nullptr);
    } else if (warp == kSoftWarps + kCodeWarps + 2) {
      CodePrefetch prefetch;
      while (next_piece(u)) prefetch.piece(p, u, KROW, VROW, 0, 16, done, abort_flag);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kCodeWarps) {
    __syncwarp();
    tc_fence_after();
    tmem_free<false>(tmem, kCols);
  }
}

template <int DK, int BK, int DV, int BV, int N>
cudaError_t launch_rows(const ChunkParams& p, int grid, cudaStream_t stream) {
  static SmemOptIn opt;
  auto kern = vq_tree_kernel<DK, BK, DV, BV, N>;
  constexpr size_t smem = TreeSmem<DK, BK, DV, BV, N>::kTotal;
  cudaError_t e = ensure_smem(kern, smem, opt);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(TreeShape<N>::kThreads), smem, stream, p, false);
}

template <int DK, int BK, int DV, int BV>
cudaError_t launch_format(const ChunkParams& p, int grid, cudaStream_t stream) {
  if (p.tile_rows == 16) return launch_rows<DK, BK, DV, BV, 16>(p, grid, stream);
  // (32 rows not beside the 1.5-bit format's tables, which leave no room for P's second tile)
  if constexpr (BK != 12) return launch_rows<DK, BK, DV, BV, 32>(p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree(const ChunkParams& p, int k_sub, int k_bits, int v_sub, int v_bits, int grid, cudaStream_t stream) {
  if (k_sub == 8 && k_bits == 12 && v_sub == 8 && v_bits == 12) return launch_format<8, 12, 8, 12>(p, grid, stream);
  if (k_bits == 8 && (k_sub == 2 || k_sub == 4)) {
    const bool k4 = k_sub == 4;
    if (v_sub == 4 && v_bits == 8) return k4 ? launch_format<4, 8, 4, 8>(p, grid, stream) : launch_format<2, 8, 4, 8>(p, grid, stream);
    if (v_sub == 4 && v_bits == 9) return k4 ? launch_format<4, 8, 4, 9>(p, grid, stream) : launch_format<2, 8, 4, 9>(p, grid, stream);
    if (v_sub == 2 && v_bits == 8) return k4 ? launch_format<4, 8, 2, 8>(p, grid, stream) : launch_format<2, 8, 2, 8>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace vqk
