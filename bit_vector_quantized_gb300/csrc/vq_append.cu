// vq_append.cu -- keys and values from a projection's rows to codes in the paged pools, keys turned by their
// positions on the way, queries turned beside them (sm_103a).
//
// For token t and KV head h (VecInfer, section 方法细节 "异常值抑制的向量量化"; the rotation as in vq_rotary.cu):
//   k' = R(position) k,  k~ = k' diag(lambda)^-1 H_D,  code i = argmin_j ||k~_i - C_k[j]||^2,
//   v's code i = argmin_j ||v_i - C_v[j]||^2,  the lowest j where several are equal.
//
// The search is a product: ||c||^2 - 2 x . c orders centroids as the distance does, so sub-vectors against centroids
// are a matrix product with a very short k, in tf32: -2 c is fp16 and exact in it, x goes in as high and low part side
// by side in k, ||c||^2 in three parts against ones (or as the sums' start).  Of a group of centroids a lane keeps the
// smallest score only, with the smallest and second smallest so far and which group the smallest was.
//
// Codes are exact.  In steps, each for the sub-vectors that the one before cannot tell:
//   1. the group with the smallest score, if no other comes within the products' error and, for keys, that of x itself;
//   2. its centroids by fp32 distances ||x - c||^2 (their error is relative to the distance, not to x):
//      the nearest, if no other comes within the error of these and, for keys, of x itself (turn_key counts it);
//   3. the group's centroids (all, where step 1 could not tell) by fp32 distances once more (one warp): those as near as that,
//      equal ones counting as one;
//   4. these in 64 bits, for keys from the rows on (one warp).
// The errors are bounds, not deviations: what fp32 tells is so for every key.  They leave one to three of 10 000
// sub-vectors of drawn keys to steps 3 and 4, where the errors themselves are some fifteen times smaller.  Those
// wait for the end of a CTA's vectors, when its warps share them (at once they held up their teams: 202 us instead of 195 for 4099
// bf16 tokens at (2,8) and (4,9), 244 instead of 234 for 8192 at (4,8), 149 instead of 135 for 333 at 1.5 bit).
//
// Two kernels.  8- and 9-bit codes: tcgen05, 128 sub-vectors by 128 centroids a product; tensor memory gives the
// minima of 16 columns as it is read (tcgen05.ld.red).  12-bit codes, whose 4096 centroids do not fit shared memory as
// operands of 128 bytes: m16n8k8 warp mma, groups of 32 of which a lane holds 8 scores.  Warp mma for the others
// too took 209 us where tcgen05 took 177 (4099 bf16 tokens of 8 KV heads at (2,8) and (4,9)), 271 and 215 (8192
// tokens at (4,8)), 16 and 15.5 (64 tokens), all with narrower bounds on a key's error than now.
//
// What bounds them.  tcgen05: instructions and latency at 16 warps an SM (128 registers; with 80 for 24 warps they
// spill: 265 us), issuing in 55 % of the cycles, about 1100 warp instructions for a vector of 32 sub-vectors: a quarter the
// scores and their minima, a quarter step 2, rotation, transform and bound of a key 330, its queries 120.  The queries' CTAs
// come last and take 20 to 27 us of 229, steps 3 and 4 about 8.  The floor is 25 us, the bytes of 8192 tokens.  In an earlier
// state (215 us) two chunks of 64 centroids under way instead of one of 128 took 280 us, minima of 8 columns instead of 16
// nothing for it and 199 us instead of 183 at (2,8), (4,9).  Warp mma: the
// tensor pipe is 49 % busy with products of k = 8 (333 tokens of 8 KV heads: 135 us, floor 3).
#include "vq_rotary.cuh"
#include "vq_tcgen05.cuh"
#include "vq_turn.cuh"

#include <algorithm>

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kAppThreads = 512;  // of the warp-mma kernel, whose codebook leaves room for one CTA an SM

__device__ __forceinline__ double row_value(const AppendParams& p, const uint16_t* row, int e) {
  const uint16_t x = __ldg(row + e);
  return p.bf16 ? to_float<true>(x) : to_float<false>(x);
}

// Elements 4 lane .. 4 lane + 3 of a vector as they are coded, in 64 bits (one warp).  64-bit instructions issue at a
// fifteenth of the 32-bit ones' rate, so an angle's sine and cosine are formed once and by turn_sincos.
__device__ __forceinline__ void exact_vector(const AppendParams& p, int which, long long t, int h, int lane, double (&x)[4]) {
  const uint16_t* const row = static_cast<const uint16_t*>(p.src[which]) + t * p.stride[which] + h * kHeadDim;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = row_value(p, row, 4 * lane + i);
  if (which != 0) return;
  const int r = p.rotary_dim, half = r / 2;
  const unsigned long long pos = static_cast<unsigned long long>(__ldg(p.positions + t));
  auto first = [&](int e) { return p.interleaved ? !(e & 1) : e < half; };
  auto pair = [&](int e) { return p.interleaved ? e >> 1 : e < half ? e : e - half; };
  double si[4], co[4];
  const bool shared = p.interleaved || (half & 3) == 0;  // two of the lane's elements have one angle, or two lanes have the same four
  const int step = p.interleaved ? 2 : 1, count = shared ? 2 : 4, from = shared && !p.interleaved && 4 * lane >= half ? 2 : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    si[i] = 0.0;
    co[i] = 1.0;
    if (i < count && 4 * lane + from + step * i < r) turn_sincos(p.freq[pair(4 * lane + from + step * i)] * pos, si[i], co[i]);
  }
  if (p.interleaved) {
    si[2] = si[3] = si[1], co[2] = co[3] = co[1];
    si[1] = si[0], co[1] = co[0];
  } else if (shared) {
    const int other = 4 * lane >= r ? lane : 4 * lane < half ? lane + half / 4 : lane - half / 4;
    const double s0 = __shfl_sync(kAll, si[0], other), s1 = __shfl_sync(kAll, si[1], other);
    const double c0 = __shfl_sync(kAll, co[0], other), c1 = __shfl_sync(kAll, co[1], other);
    const bool low = from == 0;
    si[2] = low ? s0 : si[0], si[3] = low ? s1 : si[1], co[2] = low ? c0 : co[0], co[3] = low ? c1 : co[1];
    si[0] = low ? si[0] : s0, si[1] = low ? si[1] : s1, co[0] = low ? co[0] : c0, co[1] = low ? co[1] : c1;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    if (e < r) {
      const double y = row_value(p, row, p.interleaved ? e ^ 1 : e < half ? e + half : e - half);
      x[i] = p.factor * (first(e) ? x[i] * co[i] - y * si[i] : x[i] * co[i] + y * si[i]);
    }
    x[i] /= __ldg(p.lambda + h * kHeadDim + e);
  }
  // Walsh-Hadamard: strides 1 and 2 in registers, 4 .. 64 across lanes
  const double a0 = x[0] + x[1], a1 = x[0] - x[1], a2 = x[2] + x[3], a3 = x[2] - x[3];
  x[0] = a0 + a2;
  x[1] = a1 + a3;
  x[2] = a0 - a2;
  x[3] = a1 - a3;
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double y = __shfl_xor_sync(kAll, x[i], m);
      x[i] = lane & m ? y - x[i] : x[i] + y;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= 0.08838834764831845;  // 1 / sqrt(128)
}

// Sub-vector s of such a vector, in all lanes.
template <int D>
__device__ __forceinline__ void exact_part(int s, const double (&x)[4], double (&y)[D]) {
#pragma unroll
  for (int i = 0; i < D; ++i) {
    const int e = s * D + i;
    const double v0 = __shfl_sync(kAll, x[0], e >> 2), v1 = __shfl_sync(kAll, x[1], e >> 2);
    const double v2 = __shfl_sync(kAll, x[2], e >> 2), v3 = __shfl_sync(kAll, x[3], e >> 2);
    y[i] = (e & 3) == 0 ? v0 : (e & 3) == 1 ? v1 : (e & 3) == 2 ? v2 : v3;
  }
}

__device__ __forceinline__ uint32_t* code_row(const AppendParams& p, int which, long long slot, int h) {
  const unsigned P = p.page_size;
  const long long page = slot >> 32 ? slot / P : static_cast<unsigned>(slot) / P, off = slot - page * P;
  return reinterpret_cast<uint32_t*>(p.pool[which] + ((page * p.hkv + h) * P + off) * p.row_bytes[which]);
}

// Codes first .. first + count - 1 of a vector into its row of the pool (one warp), a word a lane; the words that they
// fill are theirs alone.
__device__ __forceinline__ void store_codes(const AppendParams& p, int which, const uint16_t* codes, int first, int count, long long slot, int h,
                                            int lane) {
  const int bits = p.bits[which], words = count * bits / 32;  // (whole words in every format)
  uint32_t* const row = code_row(p, which, slot, h) + first * bits / 32;
  for (int w = lane; w < words; w += 32) {
    uint32_t x = 0;
    if (bits == 8) {  // four codes a word
      const uint2 c = *reinterpret_cast<const uint2*>(codes + 4 * w);
      x = __byte_perm(c.x, c.y, 0x6420);
    } else {
      for (int i = 32 * w / bits; i < count && i * bits < 32 * w + 32; ++i) {
        const int at = i * bits - 32 * w;
        x |= at >= 0 ? static_cast<uint32_t>(codes[i]) << at : static_cast<uint32_t>(codes[i]) >> -at;
      }
    }
    row[w] = x;
  }
}

// The slot that token t is stored in, or -1.
__device__ __forceinline__ long long append_slot(const AppendParams& p, long long t, bool tell) {
  if (__ldg(p.positions + t) < 0) return -1;
  const long long slot = __ldg(p.slots + t);
  if (slot >= p.num_slots && tell) report(p.status, kDevBadSlot);
  return slot >= 0 && slot < p.num_slots ? slot : -1;
}

// ---- the codebook in shared memory: -2 c, 8 centroids a block, and ||c||^2 -------------------------------------
// Word of element e of centroid j: j d + e, but for d = 8 the lower and the upper halves of a block's 8 centroids
// one after the other, so that warp mma's operands are one word a lane without bank conflicts.
template <int D>
__device__ __forceinline__ int centroid_word(int j, int e) {
  return D == 8 ? (j >> 3) * 64 + (e >> 2) * 32 + (j & 7) * 4 + (e & 3) : j * D + e;
}

template <int D>
__device__ __forceinline__ void fill_codebook(const __half* cb, int n, float* tab, float2* norm, int* top) {
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    float c[D], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D; ++e) {
      c[e] = __half2float(__ldg(cb + j * D + e));
      sum = fmaf(c[e], c[e], sum);
    }
#pragma unroll
    for (int e = 0; e < D; ++e) tab[centroid_word<D>(j, e)] = -2.f * c[e];
    float* const at = reinterpret_cast<float*>(norm + (j & ~1)) + (j & 1);  // a pair of norms twice, as a product's start
    at[0] = at[2] = sum;
    const int high = __reduce_max_sync(kAll, __float_as_int(sum));  // (not negative: ordered like their bits; n is a multiple of the threads)
    if ((threadIdx.x & 31) == 0) atomicMax(top, high);
  }
}

// Centroid j times -2.
template <int D>
__device__ __forceinline__ void load_centroid(const float* tab, int j, float (&c)[D]) {
#pragma unroll
  for (int e = 0; e < D; e += D < 4 ? 2 : 4) {
    const float* at = tab + centroid_word<D>(j, e);
    if constexpr (D == 2) {
      const float2 v = *reinterpret_cast<const float2*>(at);
      c[0] = v.x, c[1] = v.y;
    } else {
      const float4 v = *reinterpret_cast<const float4*>(at);
      c[e] = v.x, c[e + 1] = v.y, c[e + 2] = v.z, c[e + 3] = v.w;
    }
  }
}

template <int D>
__device__ __forceinline__ float distance(const float (&x)[D], const float (&c)[D]) {  // c: times -2
  float d = 0.f;
#pragma unroll
  for (int e = 0; e < D; ++e) {
    const float y = fmaf(0.5f, c[e], x[e]);
    d = fmaf(y, y, d);
  }
  return d;
}

// ---- products -----------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                       float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (fp32's own square root takes as long as a centroid's distance, and what it is for here has room)
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether a centroid at fp32 distance d is farther off than one at `best` in truth too: the two distances are off by 2^-19 of
// the farther together, and by what the vector's own error makes of them (of_x).
__device__ __forceinline__ bool apart(float d, float best, float of_x) { return d > best + d * 1.9073486e-6f + of_x * root(d); }

// Smallest and second smallest of two such pairs, with what the smallest is (the lower of equals).
__device__ __forceinline__ void join_best(float& best, float& second, int& at, int lanes) {
  const float ob = __shfl_xor_sync(kAll, best, lanes), os = __shfl_xor_sync(kAll, second, lanes);
  const int oa = __shfl_xor_sync(kAll, at, lanes);
  second = min3(second, os, fmaxf(best, ob));
  at = ob < best || (ob == best && oa < at) ? oa : at;
  best = fminf(best, ob);
}

// Elements 4 lane .. 4 lane + 3 of a vector as they are coded (one warp).  Of keys the angles' sines and cosines
// stay with the lane while the token stays the same.
struct Angles {
  long long t = -1;
  float co[4], si[4];
};
__device__ __forceinline__ void raw_values(const AppendParams& p, uint2 w, float (&x)[4]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t v = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
    x[i] = p.bf16 ? to_float<true>(v) : to_float<false>(v);
  }
}

__device__ __forceinline__ void load_raw(const AppendParams& p, const uint16_t* row, int e, float (&x)[4]) {
  raw_values(p, __ldg(reinterpret_cast<const uint2*>(row + e)), x);
}

// The other members of the lane's pairs, where they are one aligned piece of the row (else found by turn_key).
__device__ __forceinline__ bool pair_piece(const AppendParams& p, int lane, int& e) {
  const int half = p.rotary_dim / 2;
  e = 4 * lane < half ? 4 * lane + half : 4 * lane - half;
  return !p.interleaved && (half & 3) == 0 && 4 * lane < p.rotary_dim;
}

// Squared norm of a rotated pair (x, y) under one of its channels' factor / lambda.
__device__ __forceinline__ float smoothed_pair(float x, float y, float inv) {
  const float a = x * inv, b = y * inv;
  return fmaf(a, a, b * b);
}

// Turns, smooths and transforms a key's elements 4 lane .. 4 lane + 3.  Returns four times the most that the key as it is
// here can be off by in a sub-vector, which is what apart() wants: a difference of two distances moves by 2 error . (c - c'),
// and |c - c'| is up to twice the root of the farther one.  With u = 2^-24 (half a step of 1, relative), the pairs' norms w
// (unturned, times the factor, by a channel's own lambda, so that a strong channel counts beside a partner of small lambda), |k~|:
//   * rotation, of a pair's norm: the angle's rounding pi / 4 u, sine and cosine an ulp each (1.42 u), the two products
//     and their sum 2 u, together under 4.3 u; the factor's own rounding and the products with it, where it is not 1, 2 u;
//   * of |k~|: the division u, seven butterflies 7 u, the last product and its constant 1.3 u: under 9.4 u.
// The transform keeps norms, so that is the most in all of the key, and also the most that one sub-vector can get of it: it does
// where the key follows a row of the transform and its elements round alike.  (a |w| + b |k~|)^2 <= (1 + t) a^2 |w|^2 +
// (1 + 1 / t) b^2 |k~|^2 for any t; t = 1.04 gives at most 13.2 u root(|k~|^2 + 0.22 |w|^2), 0.47 with a factor.
__device__ __forceinline__ float turn_key(const AppendParams& p, const uint16_t* row, uint2 pair, long long t, int h, int lane, Angles& a, float (&x)[4]) {
  const int r = p.rotary_dim, half = r / 2;
  const float4 lam = __ldg(reinterpret_cast<const float4*>(p.lambda + h * kHeadDim) + lane);
  const float factor = static_cast<float>(p.factor), inv[4] = {__fdividef(factor, lam.x), __fdividef(factor, lam.y), __fdividef(factor, lam.z),
                                                               __fdividef(factor, lam.w)};
  float pairs = 0.f;
  if (a.t != t) {
    a.t = t;
    const unsigned long long pos = static_cast<unsigned long long>(__ldg(p.positions + t));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (p.interleaved && (i & 1)) {
        a.co[i] = a.co[i - 1];
        a.si[i] = a.si[i - 1];
      } else if (e < r) {
        const unsigned long long turn = p.freq[p.interleaved ? e >> 1 : e < half ? e : e - half] * pos;
        // (folded to half a turn around none, where its rounding to fp32 is half as far off)
        const uint32_t at = static_cast<uint32_t>(turn >> 32);
        const bool fold = (at + 0x40000000u) >> 31;
        sincospif(static_cast<float>(static_cast<int>(fold ? 0x80000000u - at : at)) * 4.656612873077393e-10f, a.si + i, a.co + i);  // 2^-31
        if (fold) a.co[i] = -a.co[i];
        a.co[i] *= static_cast<float>(p.factor);
        a.si[i] *= static_cast<float>(p.factor);
      }
    }
  }
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      if (4 * lane + i < r) {
        pairs += smoothed_pair(x[i], x[i + 1], inv[i]) + smoothed_pair(x[i], x[i + 1], inv[i + 1]);
        const float y = x[i] * a.co[i] - x[i + 1] * a.si[i];
        x[i + 1] = x[i + 1] * a.co[i] + x[i] * a.si[i];
        x[i] = y;
      }
  } else if (4 * lane < r) {
    float y[4];
    if ((half & 3) == 0) {
      raw_values(p, pair, y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i;
        const uint16_t v = __ldg(row + (e < half ? e + half : e < r ? e - half : e));
        y[i] = p.bf16 ? to_float<true>(v) : to_float<false>(v);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < r) {
        pairs += smoothed_pair(x[i], y[i], inv[i]);
        x[i] = e < half ? x[i] * a.co[i] - y[i] * a.si[i] : x[i] * a.co[i] + y[i] * a.si[i];
      }
    }
  }
  x[0] /= lam.x;
  x[1] /= lam.y;
  x[2] /= lam.z;
  x[3] /= lam.w;
  fwht128_warp(x, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
  float sum = fmaf(__double_as_longlong(p.factor) == 0x3ff0000000000000LL ? 0.22f : 0.47f, pairs, fmaf(x[0], x[0], fmaf(x[1], x[1], fmaf(x[2], x[2], x[3] * x[3]))));
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(kAll, sum, m);
  return 53.f * 5.9604645e-8f * root(sum);
}

// Steps 3 and 4 of sub-vector s, of which the steps before found `code` (not told apart from others): among its group's
// centroids, or with `all` all of them (one warp; rare, so not inlined).
template <int D>
__device__ __noinline__ int settle(const AppendParams& p, int which, long long t, int h, int s, const float* xs, const float* tab, float of_x, int code,
                                   bool all) {
  constexpr int kGroup = D == 8 ? 32 : 16;  // of step 1
  const int lane = threadIdx.x & 31, j0 = all ? 0 : code & -kGroup, end = all ? 1 << p.bits[which] : j0 + kGroup;
  float x[D], c[D], near[D];
#pragma unroll
  for (int e = 0; e < D; ++e) x[e] = xs[s * D + e];
  load_centroid<D>(tab, code, near);
  const float best = distance<D>(x, near);
  // Whatever is past this is apart() from `best`: its root is past root(best) + of_x.
  const float limit = (best + of_x * fmaf(2.f, root(best), of_x)) * 1.0000038f;  // 1 + 2^-18
  int open[2] = {}, count = 0;  // of this lane
  bool other = false;           // one that is not `code`'s centroid by another index
  for (int j = j0 + lane; j < end; j += 32) {
    load_centroid<D>(tab, j, c);
    if (distance<D>(x, c) > limit) continue;  // (all are open where fp32 tells nothing: too far off, or not a number)
    if (count < 2) open[count] = j;
    ++count;
#pragma unroll
    for (int e = 0; e < D; ++e) other |= !(c[e] == near[e]);
  }
  const bool few = __all_sync(kAll, count <= 2);
  if (!__any_sync(kAll, other)) return __reduce_min_sync(kAll, count ? open[0] : code);
  // ---- in 64 bits ----------------------------------------------------------------------------------------------
  double full[4], y[D], nearest = INFINITY;
  exact_vector(p, which, t, h, lane, full);
  exact_part<D>(s, full, y);
  int at = code;
  auto look = [&](int j) {
    load_centroid<D>(tab, j, c);
    double score = 0.0;
#pragma unroll
    for (int e = 0; e < D; ++e) score += 0.25 * c[e] * (c[e] + 4.0 * y[e]);  // (c: times -2)
    if (score < nearest) {
      nearest = score;
      at = j;
    }
  };
  if (few) {
    if (count > 0) look(open[0]);
    if (count > 1) look(open[1]);
  } else {
    for (int j = j0 + lane; j < end; j += 32) look(j);
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const double its = __shfl_xor_sync(kAll, nearest, m);
    const int j = __shfl_xor_sync(kAll, at, m);
    if (its < nearest || (its == nearest && j < at)) {
      nearest = its;
      at = j;
    }
  }
  return at;
}

// What steps 1 and 2 leave open waits for the end of the CTA's vectors: its warps share it then, where each would hold up its
// team at once.  (A team of the tcgen05 kernel that has one tile settles them at once, which is less work: 64 tokens 20 us
// on the device instead of 22.  With 12 bits, where a look at all centroids takes long, at once took 158 us instead of 135.)
struct OpenCode {
  int t, h, s, code;  // s: the sub-vector, and kAllGroups where step 1 told none
};
constexpr int kOpenCodes = 64, kAllGroups = 0x10000;
struct OpenList {
  int count;  // (may pass kOpenCodes: those were settled at once)
  OpenCode at[kOpenCodes];
};

// Puts the lanes' open codes (`todo`: one bit a lane) on the list; returns those that found no place.
__device__ __forceinline__ uint32_t put_open(OpenList& list, uint32_t todo, int t, int h, int s, int code, bool all) {
  const int lane = threadIdx.x & 31;
  int at = 0;
  if (lane == 0) at = atomicAdd(&list.count, __popc(todo));
  at = __shfl_sync(kAll, at, 0) + __popc(todo & ((1u << lane) - 1u));
  const bool mine = todo >> lane & 1u, room = at < kOpenCodes;
  if (mine && room) list.at[at] = {t, h, all ? s | kAllGroups : s, code};
  return __ballot_sync(kAll, mine && !room);
}

// One of them (one warp; xs: 128 floats of the warp's): the vector once more, steps 3 and 4, the code in its row put right.
template <int D>
__device__ __noinline__ void settle_open(const AppendParams& p, int which, const OpenCode& open, const float* tab, float* xs) {
  const int lane = threadIdx.x & 31, t = open.t, h = open.h, s = open.s & (kAllGroups - 1);
  const uint16_t* const src = static_cast<const uint16_t*>(p.src[which]) + t * p.stride[which] + h * kHeadDim;
  float raw[4], of_x = 0.f;
  load_raw(p, src, 4 * lane, raw);
  if (which == 0) {
    uint2 pair = make_uint2(0u, 0u);
    int e;
    if (pair_piece(p, lane, e)) pair = __ldg(reinterpret_cast<const uint2*>(src + e));
    Angles angles;
    of_x = turn_key(p, src, pair, t, h, lane, angles, raw);
  }
  __syncwarp();
  *reinterpret_cast<float4*>(xs + 4 * lane) = make_float4(raw[0], raw[1], raw[2], raw[3]);
  __syncwarp();
  const int code = settle<D>(p, which, t, h, s, xs, tab, of_x, open.code, open.s & kAllGroups);
  if (code == open.code || lane != 0) return;
  // Bits of the row's words; another warp may be at others of them.
  const int bit = s * p.bits[which];
  const unsigned long long change = static_cast<unsigned long long>(code ^ open.code) << (bit & 31);
  uint32_t* const word = code_row(p, which, append_slot(p, t, false), h) + (bit >> 5);
  atomicXor(word, static_cast<uint32_t>(change));
  if (change >> 32) atomicXor(word + 1, static_cast<uint32_t>(change >> 32));
}

template <int D>
constexpr float kBand = D == 8 ? 7.6293945e-6f : 3.8146973e-6f;  // 2^-17, 2^-18: two scores' errors

// Step 1: whether the second best group of a sub-vector may hold the nearest centroid, from the two groups' scores and |x|^2.
// The products' error: at most 2^-18 (sub-vectors of 8; of fewer 2^-19) of ||c||^2 + 2 |x| |c| each: products of 11 bits by
// 11 are exact, each of up to 19 sums is off by 2^-23 of it at most, x without its high and low parts by 2^-22, of centroids
// that are as near as the nearest, so with |c| up to |x| + distance (and no longer than the longest).
// And the vector's own: apart() holds for what is farther than root(nearest) + of_x.
template <int D>
__device__ __forceinline__ bool groups_near(float best, float second, float x2, float cmax2, float of_x) {
  const float x1 = root(x2), nearest = fmaxf(best + x2, 0.f), reach = fmaf(1.01f, x1, root(nearest));
  const float c2 = fminf(reach * reach, cmax2), band = kBand<D> * fmaf(2.f * x1, root(c2), c2);
  return !(second > best + band + of_x * fmaf(2.f, root(nearest + band), of_x));
}

// Rows, codebook and scratch of the CTA.  Shared memory: the table, the norms, then for each warp its vectors in fp32
// and their codes.
template <int D, int R>
struct AppendShape {
  static constexpr int kVectors = R * 16 * D / kHeadDim;  // of a warp's pass: R tiles of 16 sub-vectors
  static_assert(kVectors >= 1 && kVectors * kHeadDim == R * 16 * D, "whole vectors");
  static constexpr int kWarpBytes = kVectors * kHeadDim * 4 + R * 16 * 2;
};

// One tensor's vectors by warp mma: R tiles of 16 sub-vectors a pass and warp.
template <int D, int R>
__device__ __forceinline__ void append_tensor(const AppendParams& p, int which, int cta, int ctas, uint8_t* smem, int* top, OpenList& list) {
  using Shape = AppendShape<D, R>;
  constexpr int NV = Shape::kVectors, kSubs = kHeadDim / D;  // sub-vectors of a vector
  const int n = 1 << p.bits[which];
  float* const tab = reinterpret_cast<float*>(smem);
  float2* const norm = reinterpret_cast<float2*>(tab + n * D);  // (|c_j|^2, |c_j+1|^2) of the pair, for either of it
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* const mine = smem + n * (D + 2) * 4 + warp * Shape::kWarpBytes;
  float* const xs = reinterpret_cast<float*>(mine);
  uint16_t* const codes = reinterpret_cast<uint16_t*>(xs + NV * kHeadDim);
  fill_codebook<D>(static_cast<const __half*>(p.cb[which]), n, tab, norm, top);
  __syncthreads();
  const float cmax2 = __int_as_float(*top);
  // A warp's passes are next to each other, so that a token's angles serve its heads.
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv, passes = (vectors + NV - 1) / NV;
  const long long per = (passes + static_cast<long long>(ctas) * warps - 1) / (static_cast<long long>(ctas) * warps);
  long long v0 = (static_cast<long long>(cta) * warps + warp) * per * NV;
  const long long v1 = min(v0 + per * NV, vectors);
  int t0 = static_cast<int>(v0 / p.hkv), h0 = static_cast<int>(v0 - static_cast<long long>(t0) * p.hkv);
  Angles angles;

  for (; v0 < v1; v0 += NV) {
    int tok[NV], head[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      tok[v] = t0;
      head[v] = h0;
      if (++h0 == p.hkv) h0 = 0, ++t0;
    }
    // ---- the vectors as they are coded ---------------------------------------------------------------------
    long long slot[NV];
    uint2 pair[NV];
    float raw[NV][4], of_x[NV];  // of_x: turn_key's, of values (which are exact) 0
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      slot[v] = v0 + v < v1 ? append_slot(p, tok[v], lane == 0) : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[v][i] = 0.f;
      pair[v] = make_uint2(0u, 0u);
      if (slot[v] >= 0) {
        const uint16_t* const src = static_cast<const uint16_t*>(p.src[which]) + tok[v] * p.stride[which] + head[v] * kHeadDim;
        load_raw(p, src, 4 * lane, raw[v]);
        int e;
        if (which == 0 && pair_piece(p, lane, e)) pair[v] = __ldg(reinterpret_cast<const uint2*>(src + e));
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      of_x[v] = 0.f;
      if (which == 0 && slot[v] >= 0)
        of_x[v] = turn_key(p, static_cast<const uint16_t*>(p.src[0]) + tok[v] * p.stride[0] + head[v] * kHeadDim, pair[v], tok[v], head[v], lane, angles,
                           raw[v]);
      *reinterpret_cast<float4*>(xs + v * kHeadDim + 4 * lane) = make_float4(raw[v][0], raw[v][1], raw[v][2], raw[v][3]);
    }
    __syncwarp();
    // ---- operands: lane (g, c) has rows g and g + 8 of each tile -----------------------------------------------
    uint32_t a[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int half = 0; half < 2; ++half)  // row g + 8 half
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // high parts of the eight elements, then a product of the low parts
          const float y = xs[r * 16 * D + (g + 8 * half) * D + 4 * e + c];
          const uint32_t hi = to_tf32(y);
          a[r][2 * e + half] = hi;
          a[r][4 + 2 * e + half] = to_tf32(y - __uint_as_float(hi));
        }
    // ---- groups of 32 centroids, 8 of a row's scores a lane --------------------------------------------------
    float best[R][2], second[R][2];
    int at[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        best[r][half] = second[r][half] = INFINITY;
        at[r][half] = 0;
      }
    for (int group = 0; group < n / 32; ++group) {
      float low[R][2];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int nb = 4 * group + b;
        const float4 start = *reinterpret_cast<const float4*>(norm + 8 * nb + 2 * c);
        const uint32_t b0 = __float_as_uint(tab[64 * nb + lane]), b1 = __float_as_uint(tab[64 * nb + 32 + lane]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float s[4];
          mma_k8(s, a[r][0], a[r][1], a[r][2], a[r][3], b0, b1, start.x, start.y, start.z, start.w);
          mma_k8(s, a[r][4], a[r][5], a[r][6], a[r][7], b0, b1, s[0], s[1], s[2], s[3]);
          low[r][0] = b == 0 ? fminf(s[0], s[1]) : min3(low[r][0], s[0], s[1]);
          low[r][1] = b == 0 ? fminf(s[2], s[3]) : min3(low[r][1], s[2], s[3]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          second[r][half] = fminf(second[r][half], fmaxf(best[r][half], low[r][half]));
          at[r][half] = low[r][half] < best[r][half] ? group : at[r][half];
          best[r][half] = fminf(best[r][half], low[r][half]);
        }
    }
    // ---- steps 1 and 2: a quad has two rows; lanes c < 2 go on with row g, the others with row g + 8 ------------
    uint32_t open[R];  // of lanes 4 g + 2 i: row g + 8 i is not told yet, and found no place on the list
    int found[R];      // (of the lane's row, and kAllGroups)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int half = c >> 1, row = 16 * r + g + 8 * half;
      float b = half ? best[r][1] : best[r][0], sec = half ? second[r][1] : second[r][0];
      int id = 4 * (half ? at[r][1] : at[r][0]) + c;
      {  // the other pair's share of this row, for this pair's share of its row
        const float ob = __shfl_xor_sync(kAll, half ? best[r][0] : best[r][1], 2), os = __shfl_xor_sync(kAll, half ? second[r][0] : second[r][1], 2);
        const int oi = __shfl_xor_sync(kAll, 4 * (half ? at[r][0] : at[r][1]) + c, 2);
        sec = min3(sec, os, fmaxf(b, ob));
        id = ob < b ? oi : id;
        b = fminf(b, ob);
      }
      join_best(b, sec, id, 1);
      float x[D], y[D], x2 = 0.f;
#pragma unroll
      for (int e = 0; e < D; ++e) {
        x[e] = xs[row * D + e];
        x2 = fmaf(x[e], x[e], x2);
      }
      const bool near = groups_near<D>(b, sec, x2, cmax2, of_x[16 * r / kSubs]);
      // of the group's four blocks this lane's two, two centroids each
      const int j = 32 * (id >> 2) + 16 * (c & 1) + 2 * (id & 3);
      float d0 = INFINITY, far = INFINITY;
      int code = j;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = j + 8 * (i >> 1) + (i & 1);
        load_centroid<D>(tab, k, y);
        const float d = distance<D>(x, y);
        far = fminf(far, fmaxf(d0, d));
        code = d < d0 ? k : code;
        d0 = fminf(d0, d);
      }
      join_best(d0, far, code, 1);
      // (not a number or too far off for fp32: not told)
      const bool unsure = near || !apart(far, d0, of_x[16 * r / kSubs]);
      if (!(c & 1)) codes[row] = static_cast<uint16_t>(code);
      found[r] = near ? code | kAllGroups : code;
      open[r] = __ballot_sync(kAll, unsure && !(c & 1) && slot[16 * r / kSubs] >= 0);
      if (open[r]) open[r] = put_open(list, open[r], tok[16 * r / kSubs], head[16 * r / kSubs], row % kSubs, code, near);
    }
    __syncwarp();
    // ---- steps 3 and 4 ------------------------------------------------------------------------------------------
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t todo = open[r];
      while (todo) {
        constexpr int kTiles = kSubs / 16;  // of a vector
        const int v = r / kTiles, bit = __ffs(todo) - 1, row = 16 * r + (bit >> 2) + 4 * (bit & 2), was = __shfl_sync(kAll, found[r], bit);
        todo &= todo - 1u;
        const int code = settle<D>(p, which, tok[v], head[v], row % kSubs, xs + v * kHeadDim, tab, of_x[v], was & (kAllGroups - 1), was & kAllGroups);
        if (lane == 0) codes[row] = static_cast<uint16_t>(code);
      }
    }
    __syncwarp();
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (slot[v] >= 0) store_codes(p, which, codes + v * kSubs, 0, kSubs, slot[v], head[v], lane);
    __syncwarp();
  }
  __syncthreads();
  for (int i = warp; i < min(list.count, kOpenCodes); i += warps) settle_open<D>(p, which, list.at[i], tab, xs);
}

// The CTAs from `first` on turn queries.
__device__ __forceinline__ void append_queries(const AppendParams& p, int first) {
  const long long b = static_cast<long long>(blockIdx.x) - first, shares = (p.q.heads[0] + p.q.heads_per_y - 1) / p.q.heads_per_y;
  if (threadIdx.x >= kRotThreads) return;
  const bool whole = p.interleaved || p.rotary_dim % 16 == 0;
  const int y = static_cast<int>(b % shares);
  if (p.bf16) whole ? rotary_share<true, true>(p.q, b / shares, y) : rotary_share<true, false>(p.q, b / shares, y);
  else whole ? rotary_share<false, true>(p.q, b / shares, y) : rotary_share<false, false>(p.q, b / shares, y);
}

__global__ void __launch_bounds__(kAppThreads, 1) vq_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) uint8_t app_smem[];
  __shared__ int top;  // the largest ||c||^2
  __shared__ OpenList list;
  const int ctas0 = p.kv_ctas[0], ctas = ctas0 + p.kv_ctas[1];
  if (static_cast<int>(blockIdx.x) >= ctas) {  // queries
    append_queries(p, ctas);
    return;
  }
  const int which = static_cast<int>(blockIdx.x) >= ctas0, cta = static_cast<int>(blockIdx.x) - which * ctas0;
  if (threadIdx.x == 0) top = list.count = 0;
  __syncthreads();
  if (p.few) append_tensor<8, 1>(p, which, cta, p.kv_ctas[which], app_smem, &top, list);
  else append_tensor<8, 2>(p, which, cta, p.kv_ctas[which], app_smem, &top, list);
}

// ---- 8- and 9-bit codes: the products on the tensor cores ----------------------------------------------------------
// A team of four warps takes 128 sub-vectors at a time, a lane one of them (sub-vectors of 2: a vector is two warps',
// who both prepare it); two teams a CTA, two CTAs an SM, 128 columns of tensor memory a team.  Operands are rows of
// 128 bytes, of which a product's k takes 32: (x high, x low | 1, 1, 1, 0 ..) against (-2 c, -2 c | ||c||^2 in three
// parts), for sub-vectors of 2 all in one.
constexpr int kTcThreads = 256, kTcChunk = 128, kTcGroup = 16;

template <int D>
__device__ __forceinline__ void fill_products(const __half* cb, int n, uint8_t* rows, float* tab, int* top) {
  for (int j = threadIdx.x; j < n; j += kTcThreads) {
    float c[D], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D; ++e) {
      c[e] = __half2float(__ldg(cb + j * D + e));
      sum = fmaf(c[e], c[e], sum);
      c[e] *= -2.f;
    }
#pragma unroll
    for (int e = 0; e < D; ++e) tab[j * D + e] = c[e];
    const uint32_t n1 = to_tf32(sum), n2 = to_tf32(sum - __uint_as_float(n1));
    const uint32_t n3 = to_tf32(sum - __uint_as_float(n1) - __uint_as_float(n2));
    auto piece = [&](int i) { return reinterpret_cast<uint4*>(rows + j * 128 + ((i ^ (j & 7)) << 4)); };
    if constexpr (D == 2) {
      const uint32_t c0 = __float_as_uint(c[0]), c1 = __float_as_uint(c[1]);
      *piece(0) = make_uint4(c0, c1, c0, c1);
      *piece(1) = make_uint4(n1, n2, n3, 0u);
    } else {
      const uint4 v = make_uint4(__float_as_uint(c[0]), __float_as_uint(c[1]), __float_as_uint(c[2]), __float_as_uint(c[3]));
      *piece(0) = v;
      *piece(1) = v;
      *piece(2) = make_uint4(n1, n2, n3, 0u);
      *piece(3) = make_uint4(0u, 0u, 0u, 0u);
    }
    const int high = __reduce_max_sync(kAll, __float_as_int(sum));  // (not negative: ordered like their bits; n is a multiple of the threads)
    if ((threadIdx.x & 31) == 0) atomicMax(top, high);
  }
}

struct TcSmem {  // offsets from the 1024-aligned start
  int rows[2], cb, tab, xs, codes, total;
};
__host__ __device__ inline TcSmem tc_smem(int d, int n) {
  TcSmem s;
  s.rows[0] = 0;
  s.rows[1] = 128 * 128;
  s.cb = 2 * 128 * 128;
  s.tab = s.cb + n * 128;
  s.xs = s.tab + n * d * 4;
  s.codes = s.xs + (kTcThreads / 32) * kHeadDim * 4;
  s.total = s.codes + (kTcThreads / 32) * 32 * 2;
  return s;
}

template <int D>
__device__ __forceinline__ void append_products(const AppendParams& p, int which, int cta, int ctas, uint8_t* smem, int* top, uint32_t tmem,
                                                uint64_t* bars, volatile int* abort_flag, OpenList& list) {
  constexpr int kVectors = 128 * D / kHeadDim;  // of a team's tile
  const int n = 1 << p.bits[which];
  const TcSmem at = tc_smem(D, n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp >> 2, w = warp & 3;
  uint8_t* const rows = smem + at.rows[team];
  float* const tab = reinterpret_cast<float*>(smem + at.tab);
  float* const xs = reinterpret_cast<float*>(smem + at.xs) + warp * kHeadDim;
  uint16_t* const codes = reinterpret_cast<uint16_t*>(smem + at.codes) + warp * 32;
  uint64_t* const bar = bars + team;
  const uint32_t cols = tmem + kTcChunk * team, mine = cols + (static_cast<uint32_t>(32 * w) << 16);
  auto row_piece = [&](int row, int i) { return reinterpret_cast<uint4*>(rows + row * 128 + ((i ^ (row & 7)) << 4)); };
  auto team_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory"); };
  fill_products<D>(static_cast<const __half*>(p.cb[which]), n, smem + at.cb, tab, top);
  {  // the ones that take the norms
    const int row = 32 * w + lane;
    const uint32_t one = __float_as_uint(1.f);
    *row_piece(row, D == 2 ? 1 : 2) = make_uint4(one, one, one, 0u);
    if constexpr (D == 4) *row_piece(row, 3) = make_uint4(0u, 0u, 0u, 0u);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  const float cmax2 = __int_as_float(*top);
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv, tiles = (vectors + kVectors - 1) / kVectors;
  const long long per = (tiles + 2LL * ctas - 1) / (2LL * ctas);
  const long long tile0 = (2LL * cta + team) * per, tile1 = min(tile0 + per, tiles);
  // This warp's vector of a tile, and which half of its sub-vectors.  One tile's are as far apart as there are tiles, so that
  // a warp's follow each other and a token's angles serve its heads.
  const int vec = D == 4 ? w : w >> 1, half = D == 4 ? 0 : w & 1;
  const long long v0 = tile0 * kVectors, v1 = min(tile1 * kVectors, vectors), run = tile1 - tile0;
  long long v = v0 + vec * run;
  const long long v_end = min(v + run, v1);
  int tok = static_cast<int>(v / p.hkv), head = static_cast<int>(v - static_cast<long long>(tok) * p.hkv);
  uint32_t phase = 0;
  Angles angles;
  // A tile's rows are asked for one tile ahead.
  struct Ahead {
    long long slot;
    uint2 raw, pair;
  } next;
  auto ask = [&](long long at, int t, int h) {
    Ahead a = {-1, make_uint2(0u, 0u), make_uint2(0u, 0u)};
    if (at >= v_end) return a;
    a.slot = append_slot(p, t, lane == 0);
    const uint16_t* const src = static_cast<const uint16_t*>(p.src[which]) + t * p.stride[which] + h * kHeadDim;
    a.raw = __ldg(reinterpret_cast<const uint2*>(src + 4 * lane));
    int e;
    if (which == 0 && pair_piece(p, lane, e)) a.pair = __ldg(reinterpret_cast<const uint2*>(src + e));
    return a;
  };
  next = ask(v, tok, head);

  for (long long tile = tile0; tile < tile1; ++tile) {
    // ---- the vector as it is coded; its rows of the operand --------------------------------------------------------
    const long long slot = next.slot;
    float raw[4] = {0.f, 0.f, 0.f, 0.f}, of_x = 0.f;
    if (slot >= 0) {
      raw_values(p, next.raw, raw);
      if (which == 0)
        of_x = turn_key(p, static_cast<const uint16_t*>(p.src[0]) + tok * p.stride[0] + head * kHeadDim, next.pair, tok, head, lane, angles, raw);
    }
    *reinterpret_cast<float4*>(xs + 4 * lane) = make_float4(raw[0], raw[1], raw[2], raw[3]);
    __syncwarp();
    float x[D], x2 = 0.f;
    uint32_t hi[D], lo[D];
#pragma unroll
    for (int e = 0; e < D; ++e) {
      x[e] = D == 4 ? raw[e & 3] : xs[(32 * half + lane) * D + e];
      x2 = fmaf(x[e], x[e], x2);
      hi[e] = to_tf32(x[e]);
      lo[e] = to_tf32(x[e] - __uint_as_float(hi[e]));
    }
    if constexpr (D == 2) {
      *row_piece(32 * w + lane, 0) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
    } else {
      *row_piece(32 * w + lane, 0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *row_piece(32 * w + lane, 1) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    ++v;
    const int tok1 = head + 1 == p.hkv ? tok + 1 : tok, head1 = head + 1 == p.hkv ? 0 : head + 1;
    next = ask(v, tok1, head1);
    // ---- scores of 128 centroids at a time; of 16 their minimum ------------------------------------------------------
    float best = INFINITY, second = INFINITY;
    int id = 0;
    bool ok = true;
    for (int c0 = 0; c0 < n; c0 += kTcChunk) {
      tc_fence_before();
      team_sync();  // the operand is there, the columns are read
      tc_fence_after();
      if (w == 0) {
        if (lane == 0) {
          const uint32_t a = smem_addr(rows), b = smem_addr(smem + at.cb) + c0 * 128;
          tc_mma_tf32(cols, tc_desc(a, 16), tc_desc(b, 16), tc_idesc_tf32(128, kTcChunk), false);
          if constexpr (D == 4) tc_mma_tf32(cols, tc_desc(a + 32, 16), tc_desc(b + 32, 16), tc_idesc_tf32(128, kTcChunk), true);
          tc_commit<false>(bar);
        }
        __syncwarp();
      }
      ok = __all_sync(kAll, mbar_wait_bounded(bar, phase, abort_flag, p.timeout_ns)) && ok;
      phase ^= 1u;
      tc_fence_after();
#pragma unroll 1
      for (int g0 = 0; g0 < kTcChunk / kTcGroup; g0 += 2) {
        const float m0 = tmem_min16(mine + kTcGroup * g0), m1 = tmem_min16(mine + kTcGroup * (g0 + 1));
        tmem_wait_ld();
        const float low[2] = {m0, m1};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          second = fminf(second, fmaxf(best, low[i]));
          id = low[i] < best ? c0 + kTcGroup * (g0 + i) : id;
          best = fminf(best, low[i]);
        }
      }
    }
    // ---- steps 1 and 2: a lane's group, each lane beginning elsewhere in it (banks) ----------------------------------
    const bool near = groups_near<D>(best, second, x2, cmax2, of_x);
    float d0 = INFINITY, far = INFINITY;
    int code = id;
#pragma unroll
    for (int i = 0; i < kTcGroup; ++i) {
      const int j = id + ((i + lane) & (kTcGroup - 1));
      float y[D];
      load_centroid<D>(tab, j, y);
      const float d = distance<D>(x, y);
      far = fminf(far, fmaxf(d0, d));
      code = d < d0 ? j : code;
      d0 = fminf(d0, d);
    }
    const bool unsure = near || !apart(far, d0, of_x);
    // ---- steps 3 and 4 ------------------------------------------------------------------------------------------------
    uint32_t todo = slot >= 0 ? __ballot_sync(kAll, unsure) : 0u;
    if (todo && run > 1) todo = put_open(list, todo, tok, head, 32 * half + lane, code, near);
    while (todo) {
      const int i = __ffs(todo) - 1, was = __shfl_sync(kAll, near ? code | kAllGroups : code, i);
      todo &= todo - 1u;
      const int told = settle<D>(p, which, tok, head, 32 * half + i, xs, tab, of_x, was & (kAllGroups - 1), was & kAllGroups);
      if (lane == i) code = told;
    }
    codes[lane] = static_cast<uint16_t>(code);
    __syncwarp();
    if (slot >= 0) store_codes(p, which, codes, 32 * half, 32, slot, head, lane);
    __syncwarp();
    tok = tok1;
    head = head1;
    // (a wait that gave up: the team leaves together, here)
    uint32_t all;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbar.red.and.pred b, %2, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(all) : "r"(static_cast<uint32_t>(ok)), "r"(1 + team) : "memory");
    if (!all) {
      if (w == 0 && lane == 0) report(p.status, kDevTimeout);
      break;
    }
  }
  __syncthreads();
  for (int i = warp; i < min(list.count, kOpenCodes); i += kTcThreads / 32) settle_open<D>(p, which, list.at[i], tab, xs);
}

__global__ void __launch_bounds__(kTcThreads, 2) vq_append_tc_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) uint8_t app_smem[];
  __shared__ int top, abort_flag;  // the largest ||c||^2
  __shared__ OpenList list;
  __shared__ uint32_t tmem_at;
  __shared__ uint64_t bars[2];
  const int ctas0 = p.kv_ctas[0], ctas = ctas0 + p.kv_ctas[1];
  if (static_cast<int>(blockIdx.x) >= ctas) {  // queries
    append_queries(p, ctas);
    return;
  }
  const int which = static_cast<int>(blockIdx.x) >= ctas0, cta = static_cast<int>(blockIdx.x) - which * ctas0;
  uint8_t* const smem = app_smem + (-smem_addr(app_smem) & 1023u);
  if (threadIdx.x == 0) {
    top = abort_flag = list.count = 0;
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    mbar_init_fence();
  }
  if (threadIdx.x < 32) tmem_alloc<false>(&tmem_at, 2 * kTcChunk);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  if (p.sub[which] == 2) append_products<2>(p, which, cta, p.kv_ctas[which], smem, &top, tmem, bars, &abort_flag, list);
  else append_products<4>(p, which, cta, p.kv_ctas[which], smem, &top, tmem, bars, &abort_flag, list);
  tc_fence_before();
  __syncthreads();  // (a product that a team gave up on has had the wait's limit to end)
  tc_fence_after();
  if (threadIdx.x < 32) tmem_free<false>(tmem, 2 * kTcChunk);
}

}  // namespace

namespace {

// CTAs of the two tensors: `most` of each where they fit the GPU at once, else shared by what they cost.
void share_ctas(AppendParams& p, const long long (&most)[2], const double (&cost)[2], int slots) {
  for (int i = 0; i < 2; ++i) {
    const long long share = static_cast<long long>(slots * cost[i] / (cost[0] + cost[1]));
    p.kv_ctas[i] = static_cast<int>(most[0] + most[1] <= slots || most[i] < share ? most[i] : share < 1 ? 1 : share);
  }
}

cudaError_t launch_products(AppendParams p, int sms, long long queries, cudaStream_t stream) {
  static SmemOptIn opt;
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv;
  size_t smem = 80 * 1024;  // (no third CTA on an SM: it would wait for tensor memory)
  long long most[2];
  double cost[2];
  for (int i = 0; i < 2; ++i) {
    const int d = p.sub[i], n = 1 << p.bits[i], per_cta = 2 * 128 * d / kHeadDim;
    smem = std::max(smem, static_cast<size_t>(tc_smem(d, n).total + 1024));
    most[i] = (vectors + per_cta - 1) / per_cta;
    // scores and what else the sub-vectors take, a key's rotation and open codes (240: 8192 tokens at (4,8) 228 us, without 233;
    // as part of the sub-vectors' it would be twice as much at (2,8): 4099 tokens 201 us instead of 195)
    cost[i] = (4.0 / d) * (n + (i == 0 ? 380 : 250)) + (i == 0 ? 240 : 0);
  }
  cudaError_t e = ensure_smem(vq_append_tc_kernel, smem, opt);
  if (e != cudaSuccess) return e;
  share_ctas(p, most, cost, 2 * sms);
  p.timeout_ns = 2000000000ULL;
  vq_append_tc_kernel<<<static_cast<unsigned>(p.kv_ctas[0] + p.kv_ctas[1] + queries), kTcThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(AppendParams p, int sms, cudaStream_t stream) {
  static SmemOptIn opt;
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv;
  long long queries = 0;  // CTAs
  if (p.q.heads[0] > 0) {
    const dim3 g = rotary_grid(p.q, sms);
    queries = static_cast<long long>(g.x) * g.y;
  }
  if (p.bits[0] < 10 && p.bits[1] < 10) return launch_products(p, sms, queries, stream);
  // one vector per warp and pass while that leaves no warp without work
  const int warps = kAppThreads / 32;
  p.few = vectors <= static_cast<long long>(sms) * warps / 2;
  size_t smem = 0;
  long long most[2];
  double cost[2];
  for (int i = 0; i < 2; ++i) {
    const int d = p.sub[i], n = 1 << p.bits[i], per_pass = p.few ? 1 : 2;
    if (d != 8) return cudaErrorInvalidValue;
    smem = std::max(smem, static_cast<size_t>(n) * (d + 2) * 4 + warps * per_pass * (kHeadDim * 4 + kHeadDim / d * 2));
    most[i] = (vectors + warps * per_pass - 1) / (warps * per_pass);
    cost[i] = 2.0 * (kHeadDim / d) * n + (i == 0 ? 3000 : 1000);  // scores, and what comes before them
  }
  cudaError_t e = ensure_smem(vq_append_kernel, smem, opt);
  if (e != cudaSuccess) return e;
  share_ctas(p, most, cost, sms);
  vq_append_kernel<<<static_cast<unsigned>(p.kv_ctas[0] + p.kv_ctas[1] + queries), kAppThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vqk
