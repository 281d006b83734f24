// vq_rotary.cuh -- one CTA's share of turning rows by their positions (vq_rotary.cu has the mathematics and
// the figures), for the rotary kernel and for the queries of the append kernel.
#pragma once

#include <cuda_bf16.h>

#include "vq_device.cuh"
#include "vq_kernels.h"

namespace vqk {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotLanes = 8;    // threads per token
constexpr int kRotUnroll = 4;   // heads in flight

template <bool kBf16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if constexpr (kBf16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  else return __half2float(__ushort_as_half(x));
}

// kWhole: the thread's 16 elements are two aligned 16-byte pieces (every
// format but split halves with rotary_dim not a multiple of 16).
template <bool kBf16, bool kWhole>
__device__ __forceinline__ void rotary_share(const RotaryParams& p, long long block_x, int block_y) {
  const int j = threadIdx.x & (kRotLanes - 1);
  const long long t = block_x * (kRotThreads / kRotLanes) + threadIdx.x / kRotLanes;
  if (t >= p.num_tokens) return;
  const int pos = __ldg(p.positions + t);
  if (pos < 0) return;  // a padding token: its rows are left as they were
  const int heads = p.heads[0] + p.heads[1] + p.heads[2];
  const int h0 = block_y * p.heads_per_y, h1 = min(h0 + p.heads_per_y, heads);

  // The thread's pairs P = 8j .. 8j + 7 of the head's 64.  Pair P < r / 2
  // turns; split halves put it at elements (P, P + r / 2), and every other
  // pair (all of them when interleaved) is elements (2P, 2P + 1).
  const int half = p.rotary_dim / 2;
  float co[8], si[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pair = 8 * j + e;
    co[e] = 1.f;
    si[e] = 0.f;
    if (pair < half) {
      const unsigned long long turn = p.freq[pair] * static_cast<unsigned long long>(pos);
      const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, si + e, co + e);
      co[e] *= p.factor;
      si[e] *= p.factor;
    }
  }
  const bool split = !p.interleaved && 8 * j < half;
  const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + half : 16 * j + 8;  // the two pieces (kWhole)

  auto tensor = [&](int h, int& hh) {
    hh = h < p.heads[0] ? h : h < p.heads[0] + p.heads[1] ? h - p.heads[0] : h - p.heads[0] - p.heads[1];
    return h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
  };
  auto element = [&](int e, int which) {  // element of pair 8j + e (which: 0 first, 1 second)
    const int pair = 8 * j + e;
    return !p.interleaved && pair < half ? pair + which * half : 2 * pair + which;
  };
  for (int hb = h0; hb < h1; hb += kRotUnroll) {
    union Piece {
      uint4 v[2];
      uint16_t s[16];
    } x[kRotUnroll];
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      if (hb + u >= h1) break;
      int hh;
      const int w = tensor(hb + u, hh);
      const uint16_t* src = static_cast<const uint16_t*>(p.src[w]) + t * p.stride[w] + hh * kHeadDim;
      if constexpr (kWhole) {
        x[u].v[0] = *reinterpret_cast<const uint4*>(src + e0);
        x[u].v[1] = *reinterpret_cast<const uint4*>(src + e1);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[u].s[e] = src[element(e, 0)];
          x[u].s[8 + e] = src[element(e, 1)];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      if (hb + u >= h1) break;
      int hh;
      const int w = tensor(hb + u, hh);
      __half* dst = static_cast<__half*>(p.dst[w]) + (t * p.heads[w] + hh) * kHeadDim;
      Piece y;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // pieces of split halves hold the pair's members apart, others side by side
        const bool apart = kWhole ? split : true;
        const float a = to_float<kBf16>(apart ? x[u].s[e] : x[u].s[2 * e]);
        const float b = to_float<kBf16>(apart ? x[u].s[8 + e] : x[u].s[2 * e + 1]);
        const bool turns = w != 2 && 8 * j + e < half;
        const uint16_t ya = __half_as_ushort(__float2half_rn(turns ? a * co[e] - b * si[e] : a));
        const uint16_t yb = __half_as_ushort(__float2half_rn(turns ? b * co[e] + a * si[e] : b));
        if constexpr (kWhole) {
          if (split) {
            y.s[e] = ya;
            y.s[8 + e] = yb;
          } else {
            y.s[2 * e] = ya;
            y.s[2 * e + 1] = yb;
          }
        } else {
          dst[element(e, 0)] = __ushort_as_half(ya);
          dst[element(e, 1)] = __ushort_as_half(yb);
        }
      }
      if constexpr (kWhole) {
        *reinterpret_cast<uint4*>(dst + e0) = y.v[0];
        *reinterpret_cast<uint4*>(dst + e1) = y.v[1];
      }
    }
  }
}

// Head shares (p.heads_per_y) and the grid: enough CTAs for four per SM, no share below the unroll.
inline dim3 rotary_grid(RotaryParams& p, int sms) {
  const int heads = p.heads[0] + p.heads[1] + p.heads[2];
  const int per_cta = kRotThreads / kRotLanes;
  const unsigned grid_x = static_cast<unsigned>((p.num_tokens + per_cta - 1) / per_cta);
  const long long want = (4LL * sms + grid_x - 1) / grid_x;
  const int most = (heads + kRotUnroll - 1) / kRotUnroll;
  const int shares = static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  p.heads_per_y = (heads + shares - 1) / shares;
  return dim3(grid_x, (heads + p.heads_per_y - 1) / p.heads_per_y);
}

}  // namespace
}  // namespace vqk
