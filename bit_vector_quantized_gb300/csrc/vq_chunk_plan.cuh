// vq_chunk_plan.cuh -- the plan of the chunk-attention kernels: which tokens a tile of query rows sees, and
// how the tiles are divided over the grid.  Compiles for the host too.
//
// Sequence b brings n new tokens; the last of them stands at position
// len - 1, so token i stands at t = len - n + i and sees p <= t, with a window
// only p > t - window or p < sinks.  A tile is TT consecutive new tokens and
// the G query heads of one KV head (row r: token r / G, head r % G); its
// keys are the blocks of CW tokens that any of its rows sees: the sinks'
// blocks, then the window's.
//
// Work division.  The tiles are laid end to end, each as long as an estimate
// of its keys plus a fixed cost, and worker c (a CTA, or a group of its warps)
// takes [c W, (c + 1) W), whatever the mix of lengths, so that the last
// worker ends with the others.  The
// estimate is min(len - n + (t + 1) TT, cap) for tile t, whose sums have a
// closed form: a worker finds its first tile by two binary searches, without a
// list of tiles.  A cut inside a tile falls on a block; the tile's pieces
// leave unnormalised partials in the workspace: a worker has at most one tile
// that began before it (slot 2c) and one that it begins but does not end
// (slot 2c + 1), so 2 slots per worker are enough for any batch.  The worker
// that begins such a tile writes its record, and the merge kernel joins the
// pieces, in order.
//
// W is total / workers, but at least 512 tokens and the root of 32 times the
// mean length of a (sequence, KV head).  A smaller W shortens the scan and
// lengthens the merge, which walks a tile's length / W pieces, so the best W
// grows as the root of that length.  Device time of one new token of one
// sequence (32 heads of 8 KV heads; one graph replayed, so the codes were in
// L2), W at least 512 | 768 | 1024 | 2048:
// 4K tokens 18.5 | 19.3 | 21.4 | 28.9 us, 16K 27.0 | 24.6 | 25.6 | 30.7, 32K
// 38.8 | 33.6 | 31.7 | 33.5; no constant is best at all three.  The root as
// built: 18.8, 25.9, 32.0.  The root of the
// total work instead (2 sqrt(total)) took four sequences of 32K from 40.6 to
// 44.1.  (total / (hkv batch) is taken over idle sequences too: they lower W,
// towards 512.)
//
// kTree: the new tokens are a tree of drafted ones.  Every one of them sees the context
// (tokens p < len - n, with a window those near its own position, which is len - n at
// least), and of the new ones those that its bits name, so all tiles of a
// sequence have the same keys.
#pragma once

#include "vq_kernels.h"

namespace vqk {
namespace {

// Slots of the ring by which a planning warp hands pieces to a CTA's other warps (vq_chunk_wide.cu, vq_tree.cu; a piece
// has a block at least).  A slot is used again once every warp has taken its piece, and the warps that expand codes take
// pieces ahead of the blocks that they store, so with too few slots the warps wait in a circle.  The products of block b
// need the K tile of block b + 2, and the warps that store that one have looked kAhead blocks further: where every
// piece is one block, at piece b + 2 + kAhead, whose slot must be that of a piece which the issuing warp has taken, b at the
// latest.  (Fewer blocks than that at the end or the start wait for fewer pieces.)  A slot less is too few.
constexpr int kWideAhead = 2, kWidePieces = 2 + kWideAhead;  // every block, and its page two ahead
constexpr int kTreeAhead = 4, kTreePieces = 2 + kTreeAhead;  // every other block, and its page two of its own ahead

struct ChunkSeq {
  int row0;   // first row (new token) in q and out
  int n;      // new tokens (0: nothing to do)
  int base;   // position of the first new token: len - n (may be negative)
  int limit;  // keys end here: len
};

__host__ __device__ __forceinline__ int plan_load(const int32_t* at) {
#ifdef __CUDA_ARCH__
  return __ldg(at);
#else
  return *at;
#endif
}

// (bad: set where the sequence is outside its bounds and left out)
template <bool kTree = false>
__host__ __device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b, bool& bad) {
  ChunkSeq s;
  const int len = plan_load(p.seq_lens + b);
  int c0 = b, c1 = b + 1;  // one token per sequence
  if (p.cu != nullptr) {
    c0 = plan_load(p.cu + b);
    c1 = plan_load(p.cu + b + 1);
  }
  s.row0 = c0;
  s.n = 0;
  s.limit = 0;
  if (c1 != c0) {
    if (len < 0 || len > p.max_seq_len || c0 < 0 || c1 < c0 || c1 > p.num_tokens || c1 - c0 > p.max_new_len ||
        (kTree && c1 - c0 > len)) {
      bad = true;
    } else {
      s.n = c1 - c0;
      s.limit = len;
    }
  }
  s.base = s.limit - s.n;
  return s;
}
template <bool kTree = false>
__host__ __device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b) {
  bool bad = false;
  return chunk_seq<kTree>(p, b, bad);
}

// The keys of tile t in blocks of CW tokens: `sink` blocks from token 0, then
// `count - sink` blocks from block `lo`.
struct ChunkKeys {
  int sink, lo, count;
  __host__ __device__ __forceinline__ int block(int i) const { return i < sink ? i : lo + (i - sink); }
};

template <int CW, bool kTree = false>
__host__ __device__ __forceinline__ ChunkKeys chunk_keys(const ChunkParams& p, const ChunkSeq& s, int t) {
  ChunkKeys k;
  const int i0 = kTree ? 0 : t * p.tile_tok, i1 = kTree ? s.n : min(i0 + p.tile_tok, s.n);
  const int hi = max(min(s.base + i1, s.limit), 0);
  int lo = 0;
  k.sink = 0;
  if (p.window > 0) {
    lo = min(max(s.base + i0 - p.window + 1, 0), hi);
    k.sink = (min(p.sinks, lo) + CW - 1) / CW;
  }
  k.lo = max(lo / CW, k.sink);
  k.count = hi > 0 ? k.sink + max((hi + CW - 1) / CW - k.lo, 0) : 0;
  return k;
}

// Estimated length of tiles 0 .. j-1 of one (sequence, KV head): each
// kGap + clamp(base + (t + 1) TT, 0, cap).
template <bool kTree = false>
__host__ __device__ __forceinline__ long long chunk_sum(const ChunkParams& p, const ChunkSeq& s, int j) {
  if constexpr (kTree) {
    const int keys = p.window > 0 ? static_cast<int>(min(static_cast<long long>(s.limit), static_cast<long long>(p.window) + p.sinks + s.n)) : s.limit;
    return static_cast<long long>(j) * (p.gap + keys);
  }
  const int TT = p.tile_tok, base = max(s.base, 0);
  const int cap = p.window > 0 ? static_cast<int>(min(static_cast<long long>(s.limit), static_cast<long long>(p.window) + p.sinks + TT)) : s.limit;
  const long long rise = min(cap > base ? static_cast<int>(static_cast<unsigned>(cap - base) / static_cast<unsigned>(TT)) : 0, j);  // tiles below the cap
  return static_cast<long long>(j) * p.gap + rise * base + TT * (rise * (rise + 1) / 2) + (j - rise) * cap;
}

struct ChunkPiece {
  int b, kvh, tile;
  ChunkSeq s;
  ChunkKeys k;
  int blk0, blk1;  // blocks [blk0, blk1) of the tile's keys
  int slot;        // partial slot, or -1: the piece is the whole tile
  int last;        // the worker that ends the tile (slot 2c + 1 only)
};

// Walks the pieces of worker `me` of `workers` (one thread does, for all of it).
template <int CW, bool kTree = false>
struct ChunkWalk {
  long long x, x1, W;    // position, end of the range, range per CTA
  long long tile_x;      // where the current tile begins
  int me;
  int b, kvh, tile, tiles;
  ChunkSeq s;

  // pre: [B + 1] estimated length of the sequences before b, all KV heads
  __host__ __device__ __forceinline__ void start(const ChunkParams& p, const long long* pre, int me_, int workers) {
    me = me_;
    const long long total = pre[p.batch];
    W = max((total + workers - 1) / static_cast<long long>(workers), static_cast<long long>(p.min_range));
    W = max(W, static_cast<long long>(sqrtf(32.0f * static_cast<float>(total / (static_cast<long long>(p.hkv) * p.batch)))));
    x = min(W * me, total);
    x1 = min(x + W, total);
    if (x >= x1) return;
    int lo = 0, hi = p.batch;  // the last b with pre[b] <= x; its own length is not 0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid;
      else hi = mid;
    }
    b = lo;
    s = chunk_seq<kTree>(p, b);
    tiles = (s.n + p.tile_tok - 1) / p.tile_tok;
    const long long per_head = chunk_sum<kTree>(p, s, tiles);
    kvh = static_cast<int>((x - pre[b]) / per_head);
    const long long off = x - pre[b] - kvh * per_head;
    lo = 0;
    hi = tiles;  // the last tile with chunk_sum(tile) <= off
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (chunk_sum<kTree>(p, s, mid) <= off) lo = mid;
      else hi = mid;
    }
    tile = lo;
    tile_x = pre[b] + kvh * per_head + chunk_sum<kTree>(p, s, tile);
  }

  // The next piece; false when the range is done.
  __host__ __device__ __forceinline__ bool next(const ChunkParams& p, ChunkPiece& q) {
    if (x >= x1) return false;
    const long long w = chunk_sum<kTree>(p, s, tile + 1) - chunk_sum<kTree>(p, s, tile);
    const long long o0 = x - tile_x, o1 = min(w, o0 + (x1 - x));
    q.b = b;
    q.kvh = kvh;
    q.tile = tile;
    q.s = s;
    q.k = chunk_keys<CW, kTree>(p, s, tile);
    q.blk0 = o0 == 0 ? 0 : static_cast<int>(o0 * q.k.count / w);
    q.blk1 = o1 == w ? q.k.count : static_cast<int>(o1 * q.k.count / w);
    q.slot = o0 > 0 ? 2 * me : o1 < w ? 2 * me + 1 : -1;
    q.last = static_cast<int>((tile_x + w - 1) / W);
    x += o1 - o0;
    if (o1 == w) {  // on to the next tile
      tile_x += w;
      if (++tile == tiles) {
        tile = 0;
        if (++kvh == p.hkv) {
          kvh = 0;
          if (x < x1) {
            do s = chunk_seq<kTree>(p, ++b);
            while (s.n == 0);
            tiles = (s.n + p.tile_tok - 1) / p.tile_tok;
          }
        }
      }
    }
    return true;
  }
};

}  // namespace
}  // namespace vqk
