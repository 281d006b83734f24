// vq_chunk_wide.cuh -- what the tcgen05 attention kernels share: codes of a token's part, gathers from the centroid
// table, register splits and packed arithmetic.
#pragma once

#include "vq_chunk_common.cuh"
#include "vq_gather.cuh"
#include "vq_tcgen05.cuh"

namespace vqk {
namespace {

// Codes of kDims dims of a token (32 or 64; part 0 .. 128 / kDims - 1), loaded ahead of their use: the
// loads are volatile, so that they stay where they are issued, and nothing is computed from the words
// before align().
template <int D, int B, int kDims>
struct PartCodes {
  static constexpr int kBits = B, kSub = D, kPieces = kDims / 8;  // 16-byte pieces of centroids
  static constexpr int kCodes = kDims / D;
  static constexpr int kWords = (kCodes * B + 31) / 32;  // (9- and 12-bit codes may start inside their first word)
  uint32_t w[kWords];
  static __device__ __forceinline__ int first_byte(int part) { return part * kCodes * B / 32 * 4; }
  __device__ __forceinline__ void load(const uint8_t* at) {
    if constexpr (B == 8 && kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                     : "l"(at + 4 * i));
    } else if constexpr (B == 8) {
      asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(at));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[i]) : "l"(at + 4 * i));
    }
  }
  // Code 0 to bit 0.
  __device__ __forceinline__ void align(int part) {
    if constexpr (kCodes * B % 32) {
      const int s = part * kCodes * B & 31;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = i + 1 < kWords ? __funnelshift_r(w[i], w[i + 1], s) : w[i] >> s;
    }
  }
  __device__ __forceinline__ uint32_t code(int i) const {
    if constexpr (B == 8) {
      return __byte_perm(w[i >> 2], 0u, 0x4440 | (i & 3));
    } else {
      const int bit = i * B, k = bit >> 5, s = bit & 31;
      const uint32_t x = s + B > 32 ? __funnelshift_r(w[k], w[k + 1 < kWords ? k + 1 : k], s) : w[k] >> s;
      return x & ((1u << B) - 1u);
    }
  }
};
static_assert(PartCodes<4, 9, 32>::kWords == 3 && PartCodes<4, 9, 64>::kWords == 5 && PartCodes<8, 12, 32>::kWords == 2 &&
                  PartCodes<8, 12, 64>::kWords == 3,
              "72 + 24, 144 + 16, 48 + 16 and 96 bits");

// 16-byte piece c (dims 8c .. 8c + 7) of the part: its centroids.
// kRowShift: log2 of the table's row bytes; lane: the lane's byte in a row.
template <typename Codes, int kRowShift>
__device__ __forceinline__ uint4 gather_piece(const Codes& x, int c, uint32_t lane) {
  constexpr int D = Codes::kSub;
  auto off = [&](int i) {
    if constexpr (Codes::kBits == 8 && kRowShift == 8) return row_addr(x.w[i >> 2], lane, i & 3);
    else return (x.code(i) << kRowShift) + lane;
  };
  if constexpr (D == 8) {
    return tab128(off(c));
  } else if constexpr (D == 4) {
    const uint2 a = tab64(off(2 * c)), b = tab64(off(2 * c + 1));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    return make_uint4(tab32(off(4 * c)), tab32(off(4 * c + 1)), tab32(off(4 * c + 2)), tab32(off(4 * c + 3)));
  }
}

// The gather table: replicated centroids, K and V side by side in 256-byte rows, or (9-bit codes) in 128-byte rows
// one after the other; the 1.5-bit format's are plain tables of 64 KB.
template <int DK, int BV>
struct WideTable {
  static constexpr bool kWideCodes = DK == 8, kSplitTable = BV == 9;
  static constexpr int kBytes = kWideCodes ? 131072 : kSplitTable ? (256 + 512) * 128 : 65536;
};

// (By thread `thread` of `threads`, or, with 0, by all of the CTA's.  Those step by the built-in variables themselves: with the
// kernel's own copies of them 5 drafted tokens, batch 16, take 158.4 us instead of 156.5.)
template <int DK, int BK, int DV, int BV>
__device__ __forceinline__ void fill_wide_table(const ChunkParams& p, int thread = 0, int threads = 0) {
  using W = WideTable<DK, BV>;
  uint4* tab = reinterpret_cast<uint4*>(g_smem);
  auto replicas = [](const void* cb, int row, bool four) {
    if (four) {
      const uint2 c = __ldg(static_cast<const uint2*>(cb) + row);
      return make_uint4(c.x, c.y, c.x, c.y);
    }
    const uint32_t c = __ldg(static_cast<const uint32_t*>(cb) + row);
    return make_uint4(c, c, c, c);
  };
  auto put = [&](int i) {
    if constexpr (W::kWideCodes) {
      tab[i] = i < 4096 ? __ldg(static_cast<const uint4*>(p.cb_k) + i) : __ldg(static_cast<const uint4*>(p.cb_v) + i - 4096);
    } else if constexpr (W::kSplitTable) {
      tab[i] = i < 2048 ? replicas(p.cb_k, i >> 3, DK == 4) : replicas(p.cb_v, (i - 2048) >> 3, DV == 4);
    } else {
      tab[i] = i & 8 ? replicas(p.cb_v, i >> 4, DV == 4) : replicas(p.cb_k, i >> 4, DK == 4);
    }
  };
  if (threads) {
    for (int i = thread; i < W::kBytes / 16; i += threads) put(i);
  } else {
    for (int i = threadIdx.x; i < W::kBytes / 16; i += blockDim.x) put(i);
  }
}

// The warpgroup's registers per thread from here on (all four warps call it).
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Maximum of three (fp32 bits), and a packed pair of fp32 additions.
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}

// A tree's weights p = 2^(s - m) are products' operands as two fp16 parts, 22 bits: with the first alone outputs were off by
// 2.0e-4 to 2.8e-4 (relative, against 64 bits), of which their own rounding is 1.9e-4 to 2.1e-4, and that is all that is left.
// m is the maximum less kLift.  The maximum may lag by 2^8, so p stays under 2^15, and fp16, which ends at 2^16 above and is
// subnormal under 2^-14, has all bits down to 2^-21 of the largest weight; below it p is off by up to 2^-31 of that.  (The
// tensor core's fp32 sums drop what is under 2^-24 of what they hold already.)
constexpr float kLift = 7.f;

// p0 and p1 (not negative) -> fp16 pairs of their first 11 bits and of the next 11.
__device__ __forceinline__ void cut_pair(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1), "f"(p0));
  add2(p0, p1, __uint_as_float((__float_as_uint(p0) & 0xffffe000u) | 0x80000000u), __uint_as_float((__float_as_uint(p1) & 0xffffe000u) | 0x80000000u));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(p1), "f"(p0));
}

// A ring slot's position: phase flips each time the ring wraps.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// One piece of a tile as the planning warp hands it to the others.
struct __align__(16) WidePiece {
  int b, kvh;
  int row0, rows;            // the tile's first row in q and out, and its rows (tokens x G)
  int first_pos, last_pos;   // positions of its first and last token
  int limit;                 // keys end here
  int sink, lo, blk0, blk1;  // blocks [blk0, blk1) of its keys (ChunkKeys)
  int slot;                  // partial slot or -1
  int more;                  // 0: there is no piece, the range is done
  int seq_row;               // (a tree:) row of the sequence's first drafted token; first_pos is the context's last token
  int pad[2];
  __device__ __forceinline__ int block(int i) const { return i < sink ? i : lo + (i - sink); }
};
static_assert(sizeof(WidePiece) == 64, "the pieces' place in shared memory");
// pre[b]: the estimated length of the sequences before b, all KV heads (one warp).
__device__ __forceinline__ void tree_plan(const ChunkParams& p, long long* pre) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    long long w = 0;
    if (b < p.batch) {
      bool bad = false;
      const ChunkSeq s = chunk_seq<true>(p, b, bad);
      if (bad && blockIdx.x == 0) report(p.status, kDevBadLength);
      w = p.hkv * chunk_sum<true>(p, s, (s.n + p.tile_tok - 1) / p.tile_tok);
    }
    long long in = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    if (b < p.batch) pre[b] = before + in - w;
    before += __shfl_sync(0xffffffffu, in, 31);
  }
  if (lane == 0) pre[p.batch] = before;
  __syncwarp();
}

// Codes on their way to L2 ahead of the warps that expand them (one warp, a piece at a time).  Those ask for a block's
// codes one block ahead, which covers L2's latency and not the memory's; where few tiles share a sequence nearly
// every code comes from there.  A lane takes 16 tokens of K or V; at most kAhead blocks ahead of `done`, which the
// issuing warp moves on.  (26 drafted tokens of each of 16 sequences of 8000 to 16 000: 230 -> 225 us; 12 tokens with
// tiles of 16 rows 610 -> 526; nothing where the codes were in L2 already.)  Granules of a block: 0 .. 7 K, 8 .. 15 V,
// taken from `from` to `to` - 1.
constexpr int kAhead = 16;
struct CodePrefetch {
  uint32_t blocks = 0;  // over all pieces
  __device__ __forceinline__ void piece(const ChunkParams& p, const WidePiece& u, int k_row, int v_row, int from, int to, volatile uint32_t* done,
                                        volatile int* abort) {
    const int lane = threadIdx.x & 31, per = to - from, at_once = 32 / per;
    const int32_t* const pages = p.page_table + static_cast<long long>(u.b) * p.max_pages;
    const int granule = from + lane % per;
    for (int i0 = u.blk0; i0 < u.blk1; i0 += at_once) {
      // (only a pace: whoever does not move for long is not waited for)
      for (int spin = 0; spin < 200 && static_cast<int>(blocks + (i0 - u.blk0) - *done) > kAhead && !*abort; ++spin) __nanosleep(100);
      const int i = i0 + lane / per, t = i < u.blk1 ? u.block(i) * 128 + (granule & 7) * 16 : u.limit;
      if (t < u.limit) {
        const int page = __ldg(pages + t / p.page_size);
        if (page >= 0 && page < p.num_pages) {
          const int row = granule < 8 ? k_row : v_row;
          const long long at = (static_cast<long long>(page) * p.hkv + u.kvh) * p.page_size + t % p.page_size;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((granule < 8 ? p.k_pool : p.v_pool) + at * row), "r"(16 * row) : "memory");
        }
      }
      __syncwarp();
    }
    blocks += u.blk1 - u.blk0;
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

}  // namespace
}  // namespace vqk
