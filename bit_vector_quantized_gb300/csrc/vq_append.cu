// vq_append.cu -- keys and values from a projection's rows to codes in the paged pools, keys turned by their
// positions on the way, queries turned beside them (sm_103a).
//
// For token t and KV head h (VecInfer, section 方法细节 "异常值抑制的向量量化"; the rotation as in vq_rotary.cu):
//   k' = R(position) k,  k~ = k' diag(lambda)^-1 H_D,  code i = argmin_j ||k~_i - C_k[j]||^2,
//   v's code i = argmin_j ||v_i - C_v[j]||^2,  the lowest j where several are equal.
//
// One warp per vector, everything in 64 bits.
#include "vq_rotary.cuh"

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kAppThreads = kRotThreads, kAppWarps = kAppThreads / 32;

__device__ __forceinline__ double row_value(const AppendParams& p, const uint16_t* row, int e) {
  const uint16_t x = __ldg(row + e);
  return p.bf16 ? to_float<true>(x) : to_float<false>(x);
}

// Elements 4 lane .. 4 lane + 3 of a vector as they are coded, in 64 bits (one warp).
__device__ __forceinline__ void exact_vector(const AppendParams& p, int which, long long t, int h, int lane, double (&x)[4]) {
  const uint16_t* const row = static_cast<const uint16_t*>(p.src[which]) + t * p.stride[which] + h * kHeadDim;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = row_value(p, row, 4 * lane + i);
  if (which != 0) return;
  const int half = p.rotary_dim / 2;
  const unsigned long long pos = static_cast<unsigned long long>(__ldg(p.positions + t));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    if (e < p.rotary_dim) {
      const bool first = p.interleaved ? !(e & 1) : e < half;
      const int pair = p.interleaved ? e >> 1 : first ? e : e - half;
      const int other = p.interleaved ? e ^ 1 : first ? e + half : e - half;
      double si, co;  // (the fraction of a turn, in half turns)
      sincospi(static_cast<double>(static_cast<long long>(p.freq[pair] * pos)) * 1.0842021724855044e-19, &si, &co);
      const double y = row_value(p, row, other);
      x[i] = p.factor * (first ? x[i] * co - y * si : x[i] * co + y * si);
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

// Nearest centroid of sub-vector s in 64 bits (one warp; the same in all lanes).
__device__ __forceinline__ int exact_code(const AppendParams& p, int which, int s, const double (&x)[4], int lane) {
  const int d = p.sub[which], n = 1 << p.bits[which];
  double y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = (s * d + i) % kHeadDim;  // (past the sub-vector: not used)
    const double v0 = __shfl_sync(kAll, x[0], e >> 2), v1 = __shfl_sync(kAll, x[1], e >> 2);
    const double v2 = __shfl_sync(kAll, x[2], e >> 2), v3 = __shfl_sync(kAll, x[3], e >> 2);
    y[i] = (e & 3) == 0 ? v0 : (e & 3) == 1 ? v1 : (e & 3) == 2 ? v2 : v3;
  }
  const __half* const cb = static_cast<const __half*>(p.cb[which]);
  double best = INFINITY;
  int at = 0;
  for (int j = lane; j < n; j += 32) {
    double score = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < d) {
        const double c = __half2float(__ldg(cb + j * d + i));
        score += c * (c - 2.0 * y[i]);
      }
    if (score < best) {
      best = score;
      at = j;
    }
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const double other = __shfl_xor_sync(kAll, best, m);
    const int its = __shfl_xor_sync(kAll, at, m);
    if (other < best || (other == best && its < at)) {
      best = other;
      at = its;
    }
  }
  return at;
}

// A vector's codes into its row of the pool (one warp): lane w makes words w, w + 32, .. of the row.
__device__ __forceinline__ void store_codes(const AppendParams& p, int which, const uint16_t* codes, long long slot, int h, int lane) {
  const int bits = p.bits[which], count = kHeadDim / p.sub[which], words = p.row_bytes[which] / 4;
  const long long page = slot / p.page_size, off = slot % p.page_size;
  uint32_t* const row = reinterpret_cast<uint32_t*>(p.pool[which] + ((page * p.hkv + h) * p.page_size + off) * p.row_bytes[which]);
  for (int w = lane; w < words; w += 32) {
    uint32_t x = 0;
    for (int i = 32 * w / bits; i < count && i * bits < 32 * w + 32; ++i) {
      const int at = i * bits - 32 * w;
      x |= at >= 0 ? static_cast<uint32_t>(codes[i]) << at : static_cast<uint32_t>(codes[i]) >> -at;
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

template <bool kBf16, bool kWhole>
__global__ void __launch_bounds__(kAppThreads) vq_append_kernel(const __grid_constant__ AppendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= 2 * p.kv_ctas) {  // queries
    const long long b = static_cast<long long>(blockIdx.x) - 2 * p.kv_ctas, shares = (p.q.heads[0] + p.q.heads_per_y - 1) / p.q.heads_per_y;
    rotary_share<kBf16, kWhole>(p.q, b / shares, static_cast<int>(b % shares));
    return;
  }
  const int which = blockIdx.x & 1;
  __shared__ uint16_t codes[kAppWarps][kHeadDim];
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv;
  for (long long v = static_cast<long long>(blockIdx.x >> 1) * kAppWarps + warp; v < vectors; v += static_cast<long long>(p.kv_ctas) * kAppWarps) {
    const long long t = v / p.hkv;
    const int h = static_cast<int>(v % p.hkv);
    const long long slot = append_slot(p, t, lane == 0);
    if (slot < 0) continue;
    double x[4];
    exact_vector(p, which, t, h, lane, x);
    for (int s = 0; s < kHeadDim / p.sub[which]; ++s) {
      const int code = exact_code(p, which, s, x, lane);
      if (lane == 0) codes[warp][s] = static_cast<uint16_t>(code);
    }
    __syncwarp();
    store_codes(p, which, codes[warp], slot, h, lane);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_append(AppendParams p, int sms, cudaStream_t stream) {
  const long long vectors = static_cast<long long>(p.num_tokens) * p.hkv;
  const long long most = (vectors + kAppWarps - 1) / kAppWarps;
  p.kv_ctas = static_cast<int>(most < 4LL * sms ? most : 4LL * sms);
  long long grid = 2LL * p.kv_ctas;
  if (p.q.heads[0] > 0) {
    const dim3 g = rotary_grid(p.q, sms);
    grid += static_cast<long long>(g.x) * g.y;
  }
  const bool whole = p.interleaved || p.rotary_dim % 16 == 0;
  auto kern = p.bf16 ? (whole ? vq_append_kernel<true, true> : vq_append_kernel<true, false>)
                     : (whole ? vq_append_kernel<false, true> : vq_append_kernel<false, false>);
  kern<<<static_cast<unsigned>(grid), kAppThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vqk
