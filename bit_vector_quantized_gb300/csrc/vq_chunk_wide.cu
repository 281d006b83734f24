// vq_chunk_wide.cu -- chunk attention for many query rows per (sequence, KV head) (sm_103a).
//
// The mathematics of vq_chunk_narrow.cu for tiles of 128 query rows per CTA, on
// the fifth-generation tensor cores: per block of 128 tokens
//   S [128 x 128] = Q~ K~^T,  P = 2^(S - m),  O [128 x 128] += P V.
//
// Two shapes.  Alone, a CTA expands a block's codes for its 128 rows.  With
// more than 128 rows two CTAs form a pair (cta_group::2): one product of 256
// rows, each CTA holding half of the expanded tile (K of 64 of the block's
// tokens, 64 dims of V), so each expands, stores and reads half as much.
//
//   * Sixteen warps expand codes, eight K and eight V: a thread takes one
//     token's codes of 64 dims (32 in a pair; loaded a block ahead, their page
//     two ahead), gathers their centroids from the replicated,
//     bank-conflict-free table and stores 16-byte pieces into the swizzled
//     tiles that the tensor core reads (K rows of dims, V rows of dims with
//     the token as k: one layout for both).
//   * One thread issues the products, values of block j and then scores of
//     block j + 2 into the same columns; the tensor pipe works on one block
//     while the softmax works on the next.  Operands are uniform (an elected
//     lane of a converged warp): from a divergent branch an issue took 190
//     cycles in a loop of products alone, 68 from uniform operands.
//   * Eight warps hold half a query row per thread: the Walsh-Hadamard transform
//     of their q row in registers, the online softmax (maximum and sum in
//     fp32; the maximum may lag by 2^8, so O is seldom rescaled), P rounded
//     to fp16 once (p <= 2^8, relative 2^-11).  That rounding is a choice: the
//     outputs are off by 2.3e-4 to 2.9e-4 (relative, against 64 bits), their own
//     rounding to fp16 being 2.1e-4 of it.  With P's low part as a second operand
//     (tensor memory has its columns) 2.1e-4 is all that is left, but a block has
//     32 products instead of 24: a chunk of 2048 in 32K took 1215 us instead of
//     943, chunks of 1000 with a window of 1024 161 instead of 132, 5 drafted
//     tokens 203 instead of 158.  (Trees of drafted tokens have P's low part: 66 us instead of 60 for a
//     tree of 64 in 32K, 270 instead of 225 for trees of 26, batch 16 at (2,8), (4,9).)
//   * One warp walks the CTA's pieces and hands them to the others, so that
//     none of them carries the walk in registers.
//   * Tensor memory, all 512 columns: S twice (P overwrites its S, so the
//     values read it from there), O, and Q~ high and low.
//   * Every wait on an mbarrier is bounded: on a timeout the CTA raises an abort
//     flag, everybody leaves, the products in flight are drained and
//     VQ_DEV_TIMEOUT is reported.  The softmax warps also meet at barriers
//     without a limit; vq_chunk_soft.cuh has the order in which none of them
//     leaves another there.
//
// What bounds it.  A block costs 24 products of 64 cycles (16 for the scores,
// q~ in high and low fp16 parts so that they keep about fp32 accuracy, and 8
// for the values): 1536 cycles, against which the floor of 4 D operations per
// (row, token) is 1024.  Measured (2048 new tokens in 32K, 32 heads of 8 KV
// heads, 64 B of codes per token): this kernel alone 946 us, 1.13 PFLOP/s of
// the floor's operations (0.60 of the measured 1.889), tensor pipe 72 % busy;
// the call on one input again and again 941 to 990 with the clock, on
// changing inputs 1022 (1.04 PFLOP/s).  What is
// missing is the way from scores to P and back (two blocks of scores are all
// that tensor memory holds).  The same with one CTA per tile, in an earlier
// state: 1056 us; there a block's gathers, stores and
// product reads are about 1800 cycles of shared memory, by count (5 drafted
// tokens, batch 16: its pipe is 55 % busy, the tensor pipe 43 %).  A tile's
// start and end (q~, first scores, output)
// take 12 000 to 15 000 cycles by clock reads in an earlier state of the
// kernel, which short contexts feel: 128 us, with the merge 132, for chunks
// of 1000 with a window of 1024 (floor 34).  The 1.5-bit format's plain table,
// whose gathers meet in the same banks, costs little beside that: prompts of
// 512 to 8192 tokens take 3 to 12 % longer than at 8 bits.
#include <type_traits>

#include "vq_chunk_soft.cuh"
#include "vq_chunk_wide.cuh"

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kSlack = 8.f;        // the running maximum may lag by this much (log2 units): p <= 2^8 (a tree's 2^15)
constexpr int kTile = 128;           // query rows of a CTA's tile, and tokens of a block
constexpr int kSoftWarps = 8, kCodeWarps = 16;
constexpr int kWideThreads = (kSoftWarps + kCodeWarps + 4) * 32;  // the issuer's warpgroup has two busy warps
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kCols = 512;
constexpr uint32_t kPieces = kWidePieces;

// One CTA alone, or the two CTAs of a pair that share a block's tiles.
template <bool kPair>
struct WideShape {
  // Registers per thread: 72 at the launch (896 threads), then 256 soft + 512 code + 128 issue = 896 x 72
  // (112, 56, 56 or 104, 64, 40).  Alone, a code thread's 64 dims need the 64: with 56 it spills, and
  // spilled registers go to L2 beside this much shared memory (5 drafted tokens, batch 16: 174 -> 158 us).
  // In a pair its 32 dims do not, and the others use theirs (chunks of 1000, window 1024: 131 against 142 us).
  static constexpr int kSoftRegs = kPair ? 112 : 104, kCodeRegs = kPair ? 56 : 64, kIssueRegs = kPair ? 56 : 40;
  static_assert(8 * kSoftRegs + 16 * kCodeRegs + 4 * kIssueRegs <= 28 * 72, "the block's registers at the launch");
  static constexpr int kTileBytes = kTile * kHeadDim * 2 / (kPair ? 2 : 1);  // of K or V, this CTA's part
  static constexpr int kKStages = kPair ? 3 : 2;
  // Token masks in flight: block b's is written when the V tile of block b - 1 has been, so the values of
  // block b - 1 - (V stages) are done, and the softmax of that block.
  static constexpr int kMasks = 4;
};

template <int DK, int BK, int DV, int BV, bool kPair>
struct WideSmem {
  using Shape = WideShape<kPair>;
  static constexpr bool kWideCodes = DK == 8;      // 1.5-bit format: plain 64 KB tables
  static constexpr bool kSplitTable = BV == 9;     // 128-byte rows, K then V; else 256-byte rows (K, V)
  static constexpr int kTable = WideTable<DK, BV>::kBytes;
  static constexpr int kVStages = kPair ? 3 : kWideCodes ? 1 : 2;
  static constexpr int kTiles = kTable;                             // K stages, then V stages
  static constexpr int kMisc = kTiles + (Shape::kKStages + kVStages) * Shape::kTileBytes;
  static constexpr int kEnd = kMisc + 704 + 2 * 2 * kTile * 4;
  // 4 KB per softmax warp, where they fit (all but the 1.5-bit format, and the split table alone): its 32
  // rows' half of q and of the output pass through, so that global accesses are whole 128-byte lines.
  static constexpr bool kStaged = kEnd + 128 + kSoftWarps * 4096 <= 232448;
  static constexpr int kStage = (kEnd + 127) / 128 * 128;
  static constexpr int kTotal = kStaged ? kStage + kSoftWarps * 4096 : kEnd;
  static_assert(Shape::kMasks >= kVStages + 1, "a mask's slot comes round after its reader");
  static_assert(kTotal <= 232448, "shared memory of one CTA");
  static_assert((kChunkMaxBatch + 1 + 32) * 8 <= Shape::kTileBytes, "the plan shares a tile");
};

// Unnormalised Walsh-Hadamard transform of 64 registers.
__device__ __forceinline__ void fwht64(float (&x)[64]) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if (!(i & s)) {
        const float a = x[i], b = x[i + s];
        x[i] = a + b;
        x[i + s] = a - b;
      }
}

// Which of tokens t .. t + 31 a row of a tree sees among the drafted ones, which begin at token `ctx` (its
// bits, and with a window their positions against its own, pos).
__device__ __forceinline__ uint32_t tree_bits(const ChunkParams& p, int row, int seq_row, int ctx, int t, int pos) {
  const unsigned long long* const m = p.masks + static_cast<long long>(row) * p.mask_words;
  const int at = t - ctx, w = at >> 6, s = at & 63;  // (at > -32; w -1 where the context's tokens come first)
  unsigned long long x = w >= 0 && w < p.mask_words ? __ldg(m + w) >> s : 0ULL;
  if (s > 32 && w + 1 < p.mask_words) x |= __ldg(m + w + 1) << (64 - s);
  uint32_t see = static_cast<uint32_t>(x);
  if (p.window > 0) {
    uint32_t todo = see;
    while (todo) {
      const int i = __ffs(todo) - 1;
      todo &= todo - 1u;
      if (at + i < p.max_new_len && seq_row + at + i < p.num_tokens) {  // (a bit past the sequence names nothing: `seen` clears it)
        const int its = max(__ldg(p.positions + seq_row + at + i), ctx);
        if (its <= pos - p.window && its >= p.sinks) see &= ~(1u << i);
      }
    }
  }
  return see;
}

template <int DK, int BK, int DV, int BV, bool kPair, bool kTree>
__global__ void __launch_bounds__(kWideThreads, 1) vq_chunk_wide_kernel(const ChunkParams p) {
  using W = WideSmem<DK, BK, DV, BV, kPair>;
  using Shape = WideShape<kPair>;
  constexpr int NV = W::kVStages, kKStages = Shape::kKStages, kMasks = Shape::kMasks, kTileBytes = Shape::kTileBytes;
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int KROW = ((kHeadDim / DK) * BK + 31) / 32 * 4, VROW = ((kHeadDim / DV) * BV + 31) / 32 * 4;
  uint8_t* const tiles = g_smem + W::kTiles;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(g_smem + W::kMisc);
  // A wait costs 100 to 300 cycles here, ready or not (mbarrier operations queue behind the code warps'
  // shared-memory accesses), so what is needed together is collected on one barrier.
  // In a pair the first CTA's thread issues for both.  The second CTA's Q~ and P are arrived on there directly.
  // Its tiles are arrived on at home, and a warp passes each phase on as one arrival that releases them to the
  // cluster: the release takes 500 to 800 cycles, which tiles, ready blocks ahead, have and P has not (chunk of
  // 2048 in 32K, one input: 961 us; with Q~ and P passed on as well 1117).
  uint64_t* const ready = bars;            // [4] by block b: P of b, the V tile of b, the K tile of b + 2
  uint64_t* const start = ready + 4;       // K tiles of blocks 0 and 1
  uint64_t* const k_empty = start + 1;     // [kKStages] scores done, the tile is free
  uint64_t* const v_empty = k_empty + 3;   // [NV]
  uint64_t* const s_full = v_empty + 3;    // [4] by block: the scores are done, the tokens' masks are there
  uint64_t* const o_full = s_full + 4;     // [2] values of a piece's last block but one, and of its last
  uint64_t* const q_full = o_full + 2;     // Q~ stored, O read
  uint64_t* const drain = q_full + 1;
  uint64_t* const piece_full = drain + 1;              // [kPieces] planning warp -> everybody
  uint64_t* const piece_empty = piece_full + kPieces;  // [kPieces]
  WidePiece* const pieces = reinterpret_cast<WidePiece*>(bars + 48);  // [kPieces]
  uint32_t* const masks = reinterpret_cast<uint32_t*>(bars + 28);  // [kMasks][4] tokens that have a page
  uint32_t* const tmem_at = masks + kMasks * 4;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
  volatile uint32_t* const done = tmem_at + 2;  // (a tree:) blocks whose values are under way
  float* const tops = reinterpret_cast<float*>(g_smem + W::kMisc + 704);  // [2][2][128] maxima of a row's two halves

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  const uint32_t rank = kPair ? cluster_rank() : 0u;
  const int worker = static_cast<int>(blockIdx.x) / kCtas;
  const bool lead = rank == 0;
  const uint32_t passed = kPair && lead ? 1u : 0u;       // the arrival that stands for the second CTA's tiles
  const uint32_t soft = lead ? kCtas * kSoftWarps : 0u;  // softmax warps that arrive here
  if (smem_addr(tiles) & 1023u) {  // the swizzled tiles need it (and dynamic shared memory alone gives it)
    if (tid == 0) report(p.status, kDevBadConfig);
    if (tid == 0 && rank == 0) write_record(p, worker, nullptr);
    return;
  }
  if constexpr (!kTree) fill_wide_table<DK, BK, DV, BV>(p);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(ready + i, soft + kCodeWarps + passed);
      mbar_init(s_full + i, 1 + 4);
    }
    mbar_init(start, kCodeWarps + passed);  // (the K warps, for two blocks each)
    for (int i = 0; i < kKStages; ++i) mbar_init(k_empty + i, 1);
    for (int i = 0; i < NV; ++i) mbar_init(v_empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(o_full + i, 1);
    mbar_init(q_full, kCtas * kSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < static_cast<int>(kPieces); ++i) {
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, kSoftWarps + kCodeWarps + 1 + (kTree ? 1 : 0));
    }
    mbar_init_fence();
    *abort_flag = 0;
    if constexpr (kTree) *done = 0;
  }
  if (warp == kSoftWarps + kCodeWarps) tmem_alloc<kPair>(tmem_at, kCols);
  long long* const pre = reinterpret_cast<long long*>(tiles);  // the plan, before the first tile is written
  tc_fence_before();
  if constexpr (kTree) __syncthreads();
  else chunk_plan(p, pre, pre + kChunkMaxBatch + 1);
  tc_fence_after();
  // All 512 columns are this CTA's, so they start at column 0; the constant keeps the
  // products' operands in uniform registers.
  constexpr uint32_t tmem = 0;
  if (*tmem_at != tmem) {  // (in both CTAs of a pair, which allocate together)
    if (tid == 0) report(p.status, kDevBadConfig);
    if (tid == 0 && rank == 0) write_record(p, worker, nullptr);
    __syncthreads();
    if (warp == kSoftWarps + kCodeWarps) tmem_free<kPair>(*tmem_at, kCols);
    return;
  }
  if constexpr (kPair) cluster_sync();  // the barriers of both are there before either arrives on the other's

  if constexpr (kTree) {  // the planning warp plans while the others fill the table
    if (warp != kSoftWarps + kCodeWarps + 1) {
      fill_wide_table<DK, BK, DV, BV>(p, warp > kSoftWarps + kCodeWarps + 1 ? tid - 32 : tid, kWideThreads - 32);
      asm volatile("bar.sync 6, %0;" ::"n"(kWideThreads - 32) : "memory");
    }
  }

  // Bounded wait; on a timeout the CTA is given up.  The warps' form is uniform over the warp.
  auto wait_one = [&](uint64_t* bar, uint32_t phase, auto cluster) {
    if (mbar_wait_bounded<decltype(cluster)::value>(bar, phase, abort_flag, p.timeout_ns)) return true;
    if (!*abort_flag) {
      *abort_flag = 1;
      report(p.status, kDevTimeout);
    }
    return false;
  };
  auto wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(kAll, wait_one(bar, phase, std::false_type{})) != 0; };
  // (the issuer's, for what both CTAs of a pair have ready)
  auto wait_both = [&](uint64_t* bar, uint32_t phase) {
    return __all_sync(kAll, wait_one(bar, phase, std::integral_constant<bool, kPair>{})) != 0;
  };
  // An arrival for what a softmax warp did in tensor memory, which the issuing thread waits for.
  auto arrive_issuer = [&](uint64_t* bar) {
    if (kPair && !lead) mbar_arrive_at_tmem(bar, 0);
    else mbar_arrive(bar);
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
    // ====== two threads per query row: columns (and dims) 0 .. 63 and 64 .. 127 of a block ======
    reg_inc<Shape::kSoftRegs>();
    const int r = tid & (kTile - 1), g = tid >> 7, G = p.group;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // the two warps of a row meet here
    auto row_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory"); };
    uint32_t blocks = 0;  // blocks so far, over all pieces
    uint32_t ends0 = 0, ends1 = 0;  // phases of o_full so far
    // Staging: 128 bytes of each of the warp's rows, 16-byte piece c of row i at piece c ^ (i & 7).  A warp
    // moves pieces (row 4 k + lane / 8, piece lane % 8) between it and global memory, k = 0 .. 7.
    uint8_t* const stage = g_smem + W::kStage + warp * 4096;
    const int row_k = lane >> 3, piece = lane & 7;
    auto staged = [&](int i, int c) { return reinterpret_cast<uint4*>(stage + i * 128 + ((c ^ (i & 7)) << 4)); };
    const uint32_t inv_g = 65536u / G + 1u;  // r / G = r * inv_g >> 16 for r < 128
    auto row_of = [&](int i) {  // row of q and out of tile row i
      const int token = static_cast<int>(i * inv_g >> 16);
      return static_cast<long long>(u.row0 + token) * p.hq + u.kvh * G + (i - token * G);
    };
    // What a warp does between its waits and barriers, whose order (and the way out when a wait gave up)
    // is soft_warp's.
    bool live = false;  // the thread has a row of the tile
    long long row = 0;
    int pos = -1;
    float m = -INFINITY, l = 0.f;
    uint4 raw[8];             // the thread's half of its q row
    float x[64];              // and of its q~
    uint32_t s0[32], s1[32];  // its half of a row of scores
    float mx = 0.f, sum[4];
    bool again = false;
    float* const lam = tops;  // lambda by way of shared memory (the maxima's place), 64 elements in one round trip
    auto take = [&]() { return next_piece(u); };
    auto load_query = [&]() {  // (without a piece: no row's, or once more the last piece's)
      live = r < u.rows;
      row = row_of(live ? r : 0);
      m = -INFINITY;
      l = 0.f;
      if (tid < kHeadDim && u.more) lam[tid] = __ldg(p.lambda + u.kvh * kHeadDim + tid) * p.qscale;
      const __half* const q = static_cast<const __half*>(p.q) + 64 * g;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = W::kStaged ? (warp & 3) * 32 + 4 * i + row_k : r;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (at < u.rows) raw[i] = __ldg(reinterpret_cast<const uint4*>(q + (W::kStaged ? row_of(at) : row) * kHeadDim) + (W::kStaged ? piece : i));
      }
      if constexpr (W::kStaged) {
#pragma unroll
        for (int i = 0; i < 8; ++i) *staged(4 * i + row_k, piece) = raw[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = *staged(lane, i);
      }
    };
    auto all_took = [&](bool took) {  // the eight warps meet: lambda is there, and all have the piece
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbar.red.and.pred b, 5, %2, a;\n\t"
          "selp.u32 %0, 1, 0, b;\n\t}"
          : "=r"(all)
          : "r"(static_cast<uint32_t>(took)), "n"(kSoftWarps * 32)
          : "memory");
      return all != 0;
    };
    // ---- q~ = q diag(lambda) H: 64 elements here, then the butterfly of the two halves ----------
    auto turn_half = [&]() {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
          const float2 v = *reinterpret_cast<const float2*>(lam + 64 * g + 8 * i + 2 * e);
          x[8 * i + 2 * e] = f.x * v.x;
          x[8 * i + 2 * e + 1] = f.y * v.y;
        }
      }
      fwht64(x);
      __syncwarp();
      // the last butterfly joins the row's two threads, by way of the scores' columns (free by now)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(x[32 * c + i]);
        tmem_st32(tmem + lanes + kColS + 64 * g + 32 * c, y);
      }
      tmem_wait_st();
      tc_fence_before();
    };
    auto turn = [&]() {
      tc_fence_after();
      const float sg = g ? -1.f : 1.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t y[32];
        tmem_ld32(tmem + lanes + kColS + 64 * (g ^ 1) + 32 * c, y);
        tmem_wait_ld();
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          split_pair(fmaf(x[32 * c + 2 * i], sg, __uint_as_float(y[2 * i])),
                     fmaf(x[32 * c + 2 * i + 1], sg, __uint_as_float(y[2 * i + 1])), hi[i], lo[i]);
        tmem_st16(tmem + lanes + kColQ + 32 * g + 16 * c, hi);
        tmem_st16(tmem + lanes + kColQ + 64 + 32 * g + 16 * c, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_issuer(q_full);
      const int token = static_cast<int>(r * inv_g >> 16);
      if constexpr (kTree) pos = live && p.window > 0 ? max(__ldg(p.positions + u.row0 + token), u.first_pos + 1) : 0;
      else pos = live ? u.first_pos + token : -1;
      return u.blk1 - u.blk0;
    };
    // ---- a block: its scores, their masks and maximum, P with the maximum so far -----------------
    constexpr float kLead = kTree ? kLift : 0.f;  // (m: the maximum so far less this)
    auto passes = [&](float v) { return v > m + (kSlack + kLead) || (m == -INFINITY && v > -INFINITY); };
    auto col_s = [&]() { return tmem + lanes + kColS + 128 * (blocks & 1u) + 64 * g; };
    auto meet = [&]() { return tops + (blocks & 1u) * 2 * kTile; };
    // p, its sum, and P in fp16 over its own scores (of a tree two parts, the low one 16 columns behind the high one)
    auto store_p = [&](const uint32_t(&s)[32], uint32_t at, float mu) {
      if constexpr (kTree) {
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = c + j;
            float x0 = __uint_as_float(s[2 * i]), x1 = __uint_as_float(s[2 * i + 1]);
            add2(x0, x1, mu, mu);
            x0 = fast_exp2(x0);
            x1 = fast_exp2(x1);
            add2(sum[2 * (i & 1)], sum[2 * (i & 1) + 1], x0, x1);
            cut_pair(x0, x1, hi[j], lo[j]);
          }
          tmem_st4(at + c, hi);
          tmem_st4(at + 16 + c, lo);
        }
      } else {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x0 = __uint_as_float(s[2 * i]), x1 = __uint_as_float(s[2 * i + 1]);
          add2(x0, x1, mu, mu);
          x0 = fast_exp2(x0);
          x1 = fast_exp2(x1);
          add2(sum[2 * (i & 1)], sum[2 * (i & 1) + 1], x0, x1);
          const __half2 h = __floats2half2_rn(x0, x1);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st16(at, w);
      }
    };
    auto scores_wait = [&]() { return wait(s_full + (blocks & 3u), (blocks >> 2) & 1u); };
    auto block_half = [&](int j) {
      tc_fence_after();
      tmem_ld32(col_s(), s0);
      tmem_ld32(col_s() + 32, s1);
      const int t0 = u.block(u.blk0 + j) * kTile;
      const uint4 seen = *reinterpret_cast<const uint4*>(masks + (blocks % kMasks) * 4);
      const bool whole = t0 + kTile - 1 <= u.first_pos && (p.window == 0 || t0 > u.last_pos - p.window || t0 + kTile <= p.sinks) &&
                         (seen.x & seen.y & seen.z & seen.w) == kAll;
      tmem_wait_ld();
      if (!whole) {
        // the row sees tokens up to pos, from `from` on, and the sinks: as bits of a half's two words
        const int from = p.window > 0 ? (kTree ? max(pos - p.window + 1, 0) : pos - p.window + 1) : 0;
        auto bits = [](int lo, int hi) {  // bits lo .. hi - 1 of 32, whatever the two are
          const uint32_t up = hi >= 32 ? kAll : hi <= 0 ? 0u : (1u << hi) - 1u;
          const uint32_t down = lo >= 32 ? kAll : lo <= 0 ? 0u : (1u << lo) - 1u;
          return up & ~down;
        };
        auto mask = [&](uint32_t(&s)[32], int t, uint32_t here) {
          // (tokens past the sequence's end are not in `seen`)
          uint32_t see;
          if constexpr (kTree) {
            const int ctx = u.first_pos + 1;  // the context's end
            see = here & bits(0, ctx - t);
            if (p.window > 0) see &= bits(from - t, 32) | bits(0, p.sinks - t);
            if (live && t + 32 > ctx) see |= here & tree_bits(p, u.row0 + static_cast<int>(r * inv_g >> 16), u.seq_row, ctx, t, pos);
          } else {
            see = here & bits(0, pos + 1 - t) & (bits(from - t, 32) | bits(0, p.sinks - t));
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = see >> i & 1u ? s[i] : __float_as_uint(-INFINITY);
        };
        mask(s0, t0 + 64 * g, g ? seen.z : seen.x);
        mask(s1, t0 + 64 * g + 32, g ? seen.w : seen.y);
      }
      float a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t* v = k < 2 ? s0 + 16 * k : s1 + 16 * (k - 2);
        a[k] = max3(v[0], v[1], v[2]);
#pragma unroll
        for (int i = 3; i < 15; i += 2) a[k] = max3(__float_as_uint(a[k]), v[i], v[i + 1]);
        a[k] = fmaxf(a[k], __uint_as_float(v[15]));
      }
      mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
      meet()[g * kTile + r] = mx;
      // The maximum so far nearly always stays; whether the other half of the row passes it is seen on the way.
      again = __any_sync(kAll, passes(mx));
      sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
      if (!again) store_p(s0, col_s(), m == -INFINITY ? 0.f : -m);
    };
    // (false: the wait for O's values gave up)
    auto block = [&](int j, int nblk) {
      const float other = meet()[(g ^ 1) * kTile + r];
      if (!again) store_p(s1, col_s() + 32, m == -INFINITY ? 0.f : -m);
      again = again || __any_sync(kAll, passes(other));
      if (again) {  // (both warps of the rows come here)
        mx = fmaxf(mx, other);
        const float m_new = passes(mx) ? mx - kLead : m;
        const float scale = m_new == m ? 1.f : fast_exp2(m - m_new);  // 0 while nothing is accumulated
        m = m_new;
        l *= scale;
        sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
        const float mu = m == -INFINITY ? 0.f : -m;
        store_p(s0, col_s(), mu);
        store_p(s1, col_s() + 32, mu);
        if (j > 0) {  // O follows the maximum, once the values of block - 1 are in (the next scores come after them)
          if (!(j + 1 < nblk ? wait(s_full + ((blocks + 1) & 3u), ((blocks + 1) >> 2) & 1u) : wait(o_full, ends0 & 1u))) return false;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld32(tmem + lanes + kColO + 64 * g + 32 * c, s0);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) s0[i] = __float_as_uint(__uint_as_float(s0[i]) * scale);
            tmem_st32(tmem + lanes + kColO + 64 * g + 32 * c, s0);
          }
        }
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_issuer(ready + (blocks & 3u));
      ++blocks;
      return true;
    };
    auto output_wait = [&](int nblk) { return (nblk < 2 || wait(o_full, ends0++ & 1u)) && wait(o_full + 1, ends1++ & 1u); };
    auto put_sum = [&]() {
      tc_fence_after();
      meet()[g * kTile + r] = l;  // (not the last block's maxima)
    };
    // ---- the piece's rows: to `out`, or as a partial to the workspace ----------------------------
    auto store = [&]() {
      l = meet()[r] + meet()[kTile + r];  // (the same order in both threads)
      const float f = u.slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const long long at = static_cast<long long>(u.slot) * (kCtas * kTile) + rank * kTile + r;
      __half* const out = static_cast<__half*>(p.out);
      if (u.slot >= 0) {
        float* const ws = p.ws_o + (at - r) * kHeadDim + 64 * g;  // of the tile's row 0
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t s[32];
          tmem_ld32(tmem + lanes + kColO + 64 * g + 32 * c, s);
          tmem_wait_ld();
          if constexpr (W::kStaged) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) *staged(lane, i) = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 4 * i + row_k;
              reinterpret_cast<uint4*>(ws + ((warp & 3) * 32 + k) * kHeadDim + 32 * c)[piece] = *staged(k, piece);
            }
          } else if (live) {
            uint4* dst = reinterpret_cast<uint4*>(ws + r * kHeadDim + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
          }
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t s[32];
          tmem_ld32(tmem + lanes + kColO + 64 * g + 32 * c, s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 h = __floats2half2_rn(__uint_as_float(s[8 * i + 2 * e]) * f, __uint_as_float(s[8 * i + 2 * e + 1]) * f);
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (W::kStaged) *staged(lane, 4 * c + i) = v;
            else if (live) reinterpret_cast<uint4*>(out + row * kHeadDim + 64 * g)[4 * c + i] = v;
          }
          __syncwarp();
        }
        if constexpr (W::kStaged) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 4 * i + row_k, tile_row = (warp & 3) * 32 + k;
            if (tile_row < u.rows) reinterpret_cast<uint4*>(out + row_of(tile_row) * kHeadDim + 64 * g)[piece] = *staged(k, piece);
          }
          __syncwarp();
        }
      }
      if (u.slot >= 0 && live && g == 0) p.ws_ml[at] = make_float2(m, l);
      tc_fence_before();  // (O's reads, before the next piece's arrival on q_full)
    };
    soft_warp(take, load_query, all_took, turn_half, row_sync, turn, scores_wait, block_half, block, output_wait, put_sum, store);
  } else if (warp < kSoftWarps + kCodeWarps) {
    // ================================= code warps ======================================
    reg_dec<Shape::kCodeRegs>();
    // The first half of the warps expand K, the others V, each at its own pace.  Alone, a thread takes 64
    // dims of a token; in a pair 32, and the CTA has the K of half the block's tokens (columns of B) and
    // half the dims of V (columns of B again).
    constexpr int kDims = kPair ? 32 : 64;
    const int w = (warp - kSoftWarps) % (kCodeWarps / 2);
    auto expand = [&](auto codes, auto row_bytes, const uint8_t* pool, int tok, int part, uint32_t dst, uint32_t table,
                      uint32_t stages, uint64_t* empty, bool is_k, bool masking) {
      using Codes = decltype(codes);
      constexpr int kRow = decltype(row_bytes)::value;
      constexpr int kShift = W::kWideCodes ? 4 : W::kSplitTable ? 7 : 8;
      // Block iterator, two blocks ahead of the tiles: the token's page; then its codes one ahead.  The
      // page and the offset in it follow from the block before, by 128 tokens, where blocks adjoin; rows are
      // counted by 16 (a token's place among 16 is its own).
      pool += (tok % 16) * kRow + Codes::first_byte(part);
      const int per_page = p.page_size / 16, step_page = kTile / p.page_size, step_off = kTile / 16 - step_page * per_page;
      bool more = true;
      int i = 0, t = 0, lp = 0, off = 0;
      const int32_t* pages = nullptr;
      u.blk1 = 0;
      u.sink = -1;
      struct Where {
        int page, off, kvh;
        bool in, any;  // the token exists; the block exists
      };
      auto advance = [&]() {
        Where x = {0, 0, 0, false, false};
        bool jump = i == u.sink;
        while (more && i >= u.blk1) {
          more = next_piece(u);
          i = more ? u.blk0 : 0;
          jump = true;
          pages = p.page_table + static_cast<long long>(u.b) * p.max_pages;
        }
        if (!more) return x;
        if (jump) {
          t = u.block(i) * kTile + tok;
          lp = t / p.page_size;
          off = (t - lp * p.page_size) / 16;
        } else {
          t += kTile;
          lp += step_page;
          off += step_off;
          if (off >= per_page) {
            off -= per_page;
            ++lp;
          }
        }
        ++i;
        x.any = true;
        x.in = t < u.limit;
        x.kvh = u.kvh;
        x.off = off;
        // (volatile like the codes' loads: it is to be under way an iteration before its use)
        if (x.in) asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(x.page) : "l"(pages + lp));
        return x;
      };
      bool has = false, has_next = false;  // the token can be read
      Codes now, next;
      auto fetch = [&](const Where& x, Codes& y) {
        const bool good = x.in && static_cast<unsigned long long>(x.page) < static_cast<unsigned long long>(p.num_pages);
        if (good) {
          const uint32_t row16 = static_cast<uint32_t>(x.page * p.hkv + x.kvh) * per_page + x.off;
          y.load(pool + static_cast<unsigned long long>(row16) * (16 * kRow));
        } else if (x.in) {
          report(p.status, kDevBadPage);
        }
        return good;
      };
      const Where first = advance();
      Where ahead = advance();
      bool any = first.any;
      if (any) has = fetch(first, now);
      Ring ring;
      uint32_t blocks = 0;
      while (any) {
        const Where then = ahead;
        ahead = advance();
        has_next = then.any && fetch(then, next);
        if (masking) {  // the tokens of the block that can be read
          const uint32_t seen = __ballot_sync(kAll, has);
          if (lane == 0) {
            masks[(blocks % kMasks) * 4 + tok / 32] = seen;
            mbar_arrive(s_full + (blocks & 3u));
          }
        }
        if (!wait(empty + ring.slot, ring.phase ^ 1u)) break;
        const uint32_t at = dst + ring.slot * kTileBytes;
        now.align(part);
#pragma unroll
        for (int c = 0; c < Codes::kPieces; ++c) {
          // (a tree's token that cannot be read: some centroid of K, whose score is masked, but zeros of V: p is 0, and a
          // centroid that no code names may be no number)
          const uint4 v = (kTree && is_k) || has ? gather_piece<Codes, kShift>(now, c, table) : make_uint4(0, 0, 0, 0);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (c << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(!is_k ? ready + (blocks & 3u) : blocks < 2 ? start : ready + ((blocks - 2) & 3u));
        ring.next(stages);
        ++blocks;
        now = next;
        has = has_next;
        any = then.any;
      }
      // The last two blocks have no K tile to wait for; its arrivals come in their turn all the same (unless
      // the CTA was given up).
      if (is_k && !any) {
        for (uint32_t end = blocks + 2; blocks < end; ++blocks) {
          if (!wait(empty + ring.slot, ring.phase ^ 1u)) break;
          if (lane == 0) mbar_arrive(blocks < 2 ? start : ready + ((blocks - 2) & 3u));
          ring.next(stages);
        }
      }
    };
    // The first 16-byte piece of the thread's part, swizzled (its others: this address ^ (c << 4)).
    auto place = [&](int row, int rows, int part) {
      const int first = part * (kDims / 8);
      return smem_addr(tiles) + first / 8 * (rows * 128) + row * 128 + (((row & 7) ^ (first & 7)) << 4);
    };
    const uint32_t rep_k = DK == 4 ? (lane & 15) * 8 : lane * 4, rep_v = DV == 4 ? (lane & 15) * 8 : lane * 4;
    if (warp < kSoftWarps + kCodeWarps / 2) {
      const int row = kPair ? 32 * (w & 1) + lane : 32 * (w >> 1) + lane, part = kPair ? w >> 1 : w & 1;
      expand(PartCodes<DK, BK, kDims>{}, std::integral_constant<int, KROW>{}, p.k_pool,
             static_cast<int>(64 * rank) + row, part, place(row, kPair ? 64 : kTile, part), W::kWideCodes ? 0u : rep_k, kKStages,
             k_empty, true, false);
    } else {
      const int row = kPair ? 32 * (w & 3) + lane : 32 * (w >> 1) + lane, part = kPair ? w >> 2 : w & 1;
      expand(PartCodes<DV, BV, kDims>{}, std::integral_constant<int, VROW>{}, p.v_pool, row,
             (kPair ? static_cast<int>(2 * rank) : 0) + part, place(row, kTile, part) + kKStages * kTileBytes,
             W::kWideCodes ? 65536u : (W::kSplitTable ? 32768u : 128u) + rep_v, NV, v_empty, false, part == 0);
    }
  } else {
    // ================================= the products ====================================
    reg_dec<Shape::kIssueRegs>();
    if (warp == kSoftWarps + kCodeWarps && rank != 0) {
      // The first CTA issues; this one's tiles are passed on.
      uint32_t blocks = 0;
      auto pass = [&](uint64_t* bar, uint32_t phase) {
        if (!wait(bar, phase)) return false;
        if (lane == 0) mbar_arrive_at(bar, 0);
        return true;
      };
      bool ok = true;
      while (ok && next_piece(u)) {
        if (blocks == 0) ok = pass(start, 0);
        for (int j = u.blk0; ok && j < u.blk1; ++j, ++blocks) {
          ok = pass(ready + (blocks & 3u), (blocks >> 2) & 1u);
          if constexpr (kTree)
            if (lane == 0) *done = blocks;
        }
      }
    } else if (warp == kSoftWarps + kCodeWarps) {
      constexpr uint32_t kScores = tc_idesc(kCtas * kTile, kTile, false), kValues = tc_idesc(kCtas * kTile, kHeadDim, true);
      constexpr uint32_t kHalfBytes = kPair ? 64 * 128 : kTile * 128;  // K: 64 dims of this CTA's tokens
      const uint32_t tile0 = smem_addr(tiles);
      Ring rk, rv;
      uint32_t blocks = 0, tiles_done = 0;
      bool ok = true;
      while (ok && next_piece(u)) {
        const int nblk = u.blk1 - u.blk0;
        ok = wait_both(q_full, tiles_done++ & 1u);
        auto scores = [&](uint32_t blk) {  // of block blk, whose K tile is there
          if (elect_one()) {
            const uint32_t kt = tile0 + rk.slot * kTileBytes;
#pragma unroll
            for (int part = 0; part < 2; ++part)  // high and low part of q~
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc_mma_ts<kPair>(tmem + kColS + 128 * (blk & 1u), tmem + kColQ + 64 * part + 8 * ks,
                                 tc_desc(kt + (ks >> 2) * kHalfBytes + (ks & 3) * 32, 16), kScores, part > 0 || ks > 0);
            tc_commit<kPair>(s_full + (blk & 3u));
            tc_commit<kPair>(k_empty + rk.slot);
          }
          __syncwarp();
          rk.next(kKStages);
        };
        // scores of blocks 0 and 1 (their K tiles were there with the blocks before), then values of block j
        // and scores of block j + 2 (into j's columns)
        if (ok && blocks == 0) ok = wait_both(start, 0);
        tc_fence_after();
        for (int j = 0; ok && j < min(nblk, 2); ++j) scores(blocks + j);
        for (int j = 0; ok && j < nblk; ++j) {
          const uint32_t blk = blocks + j, sb = blk & 1u;
          ok = wait_both(ready + (blk & 3u), (blk >> 2) & 1u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vt = tile0 + (kKStages * kTileBytes) + rv.slot * kTileBytes;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // P of tokens 32 c .. 32 c + 31 sits at column 32 c
              tc_mma_ts<kPair>(tmem + kColO, tmem + kColS + 128 * sb + 32 * (ks >> 1) + 8 * (ks & 1),
                               tc_desc(vt + ks * 2048, kTile * 128), kValues, j > 0 || ks > 0);
            if constexpr (kTree) {  // P's low parts
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc_mma_ts<kPair>(tmem + kColO, tmem + kColS + 128 * sb + 16 + 32 * (ks >> 1) + 8 * (ks & 1),
                                 tc_desc(vt + ks * 2048, kTile * 128), kValues, true);
            }
            tc_commit<kPair>(v_empty + rv.slot);
            if (j + 2 >= nblk) tc_commit<kPair>(o_full + (j + 1 == nblk));
          }
          __syncwarp();
          rv.next(NV);
          if constexpr (kTree)
            if (lane == 0) *done = blk;
          if (j + 2 < nblk) scores(blk + 2);
        }
        blocks += nblk;
      }
      // (given up or not) the products in flight end before the tensor memory goes back
      if (elect_one()) tc_commit<kPair>(drain);
      __syncwarp();
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < p.timeout_ns) {
      }
    } else if (warp == kSoftWarps + kCodeWarps + 1) {
      // ================================== planning =======================================
      ChunkWalk<kTile, kTree> walk;
      if constexpr (kTree) tree_plan(p, pre);
      walk.start(p, pre, worker, static_cast<int>(gridDim.x) / kCtas);  // (the tiles over the plan wait for the first piece)
      ChunkPiece q;
      Ring ro;
      bool recorded = false;
      for (bool more = true; more;) {
        more = walk.next(p, q);
        // this CTA's tokens of the tile (a pair's second CTA may have none)
        const int tokens = p.tile_tok / kCtas, i0 = q.tile * p.tile_tok + static_cast<int>(rank) * tokens;
        const int n = more ? max(min(tokens, q.s.n - i0), 0) : 0;
        if (more && q.slot >= 0 && (q.slot & 1)) {
          if (lane == 0 && rank == 0) write_record(p, worker, &q);
          recorded = true;
        }
        if (more && q.blk0 >= q.blk1) {  // rows that see nothing here: zero, or an empty partial
          for (int r = 0; r < n * p.group; ++r) {
            if (q.slot >= 0) {
              const long long at = static_cast<long long>(q.slot) * (kCtas * kTile) + rank * kTile + r;
              reinterpret_cast<float4*>(p.ws_o + at * kHeadDim)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (lane == 0) p.ws_ml[at] = make_float2(-INFINITY, 0.f);
            } else {
              const long long row = static_cast<long long>(q.s.row0 + i0 + r / p.group) * p.hq + q.kvh * p.group + r % p.group;
              reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + row * kHeadDim)[lane] = make_uint2(0, 0);
            }
          }
          continue;
        }
        if (more) {  // the tile's query rows, for the softmax warps a piece later
          const char* rows = reinterpret_cast<const char*>(static_cast<const __half*>(p.q) +
                                                           (static_cast<long long>(q.s.row0 + i0) * p.hq + q.kvh * p.group) * kHeadDim);
          const int lines = 2 * p.group;  // a token's rows, 128 bytes each line
          for (int i = lane; i < n * lines; i += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + static_cast<long long>(i / lines) * p.hq * (kHeadDim * 2) + (i % lines) * 128));
        }
        int last = 0;  // of a tree's rows, the furthest position
        if (kTree && more && p.window > 0) {
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
            w.first_pos = kTree ? q.s.base - 1 : q.s.base + i0;
            w.last_pos = kTree ? last : q.s.base + i0 + n - 1;
            w.seq_row = q.s.row0;
            w.limit = q.s.limit;
            w.sink = q.k.sink;
            w.lo = q.k.lo;
            w.blk0 = q.blk0;
            w.blk1 = q.blk1;
            w.slot = q.slot;
          }
          pieces[ro.slot] = w;
          mbar_arrive(piece_full + ro.slot);
        }
        __syncwarp();
        ro.next(kPieces);
      }
      if (!recorded && lane == 0 && rank == 0) write_record(p, worker, nullptr);
    } else if (kTree && warp == kSoftWarps + kCodeWarps + 2) {
      CodePrefetch prefetch;  // (of a pair one CTA K, one V)
      while (next_piece(u)) prefetch.piece(p, u, KROW, VROW, rank ? 8 : 0, kPair && !rank ? 8 : 16, done, abort_flag);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // neither leaves while the other's barriers or products need it
  if (warp == kSoftWarps + kCodeWarps) {
    __syncwarp();
    tc_fence_after();
    tmem_free<kPair>(tmem, kCols);
  }
}

template <int DK, int BK, int DV, int BV, bool kPair, bool kTree>
cudaError_t launch_wide(const ChunkParams& p, int grid, cudaStream_t stream) {
  static SmemOptIn opt;
  auto kern = vq_chunk_wide_kernel<DK, BK, DV, BV, kPair, kTree>;
  constexpr size_t smem = WideSmem<DK, BK, DV, BV, kPair>::kTotal;
  cudaError_t e = ensure_smem(kern, smem, opt);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DK, int BK, int DV, int BV, bool kTree>
cudaError_t launch_wide(const ChunkParams& p, int grid, cudaStream_t stream) {
  return p.tile_rows == 2 * kTile ? launch_wide<DK, BK, DV, BV, true, kTree>(p, grid, stream)
                                  : launch_wide<DK, BK, DV, BV, false, kTree>(p, grid, stream);
}

template <bool kTree>
cudaError_t launch_format(const ChunkParams& p, int k_sub, int k_bits, int v_sub, int v_bits, int grid, cudaStream_t stream) {
  if (k_sub == 8 && k_bits == 12 && v_sub == 8 && v_bits == 12) return launch_wide<8, 12, 8, 12, kTree>(p, grid, stream);
  if (k_bits == 8 && (k_sub == 2 || k_sub == 4)) {
    const bool k4 = k_sub == 4;
    if (v_sub == 4 && v_bits == 8) return k4 ? launch_wide<4, 8, 4, 8, kTree>(p, grid, stream) : launch_wide<2, 8, 4, 8, kTree>(p, grid, stream);
    if (v_sub == 4 && v_bits == 9) return k4 ? launch_wide<4, 8, 4, 9, kTree>(p, grid, stream) : launch_wide<2, 8, 4, 9, kTree>(p, grid, stream);
    if (v_sub == 2 && v_bits == 8) return k4 ? launch_wide<4, 8, 2, 8, kTree>(p, grid, stream) : launch_wide<2, 8, 2, 8, kTree>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_chunk_wide(const ChunkParams& p, int k_sub, int k_bits, int v_sub, int v_bits, int grid,
                              cudaStream_t stream) {
  return launch_format<false>(p, k_sub, k_bits, v_sub, v_bits, grid, stream);
}

cudaError_t launch_tree_wide(const ChunkParams& p, int k_sub, int k_bits, int v_sub, int v_bits, int grid,
                             cudaStream_t stream) {
  return launch_format<true>(p, k_sub, k_bits, v_sub, v_bits, grid, stream);
}

}  // namespace vqk
